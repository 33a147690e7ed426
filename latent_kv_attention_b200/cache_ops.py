"""Operators around the attention calls: rotary positions and the cache append, attention over a shared prefix,
the attention weight each cached key received, and the eviction of keys by it.

Same contract as the attention functions of the package: the functions check tensors, allocate outputs and pass
pointers to the library on the current stream of the tensors' device; there is no fallback.  q, k, v and the rotary
operands may be strided views whose last dimension is contiguous (a projection's [B, s, h, d] seen as [B, h, s, d]);
caches, pools and everything else is contiguous.

Calls captured into a CUDA graph get scratch of their own from the graph's memory, so graphs that hold the same call
can replay at the same time; their flags go to one header per device that device_status reads too.
"""
from __future__ import annotations

import ctypes
import math
import threading

import torch

from . import _DT, _check, library, workspaces

_E4M3 = torch.float8_e4m3fn
_Tensor = torch.Tensor
_CACHE_DT = {torch.bfloat16: 0, torch.float32: 1, _E4M3: 2}
_HEADER = 256  # bytes of a workspace that hold the status word
_TOO_SMALL = 3  # LKA_ERR_WORKSPACE

_captured = {}
_captured_lock = threading.Lock()


def captured_status(device, create=False):
    """The address of the status header that captured calls on `device` raise their flags in (None before the first one):
    one per device, of the library's, because a graph keeps the address and no graph may own or clear the header."""
    index = device.index if device.index is not None else torch.cuda.current_device()
    with _captured_lock:
        address = _captured.get(index)
        if address is None and create:
            with torch.cuda.device(index):
                address = library().lka_captured_header()
            if not address:
                raise RuntimeError(f"no status header on cuda:{index}")
            _captured[index] = address
        return address


# The checks below run on every call, a decode step's included: they compare first and word the message only when
# something is wrong.
def _require(cond, msg):
    if not cond:
        raise ValueError(msg)


def _code(t, name):
    """(device, dtype code) of the tensor that sets both for a call."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _DT.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype} (bf16 or fp32)")
    return t.device, code


def _dense(t, name, dtype, device, shape=None):
    """The address of a contiguous tensor of this type, device and shape."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous() and
            (shape is None or t.shape == shape)):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {device}" +
                         (f" of shape {list(shape)}" if shape is not None else ""))
    return t.data_ptr()


def _strided(t, name, dtype, device):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.dim() == 4):
        raise ValueError(f"{name} must be a 4-D {dtype} tensor on {device}")
    st = t.stride()
    if st[3] != 1 and t.shape[3] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return st


def _distinct(shape, strides):
    """Every element lies at an address of its own (each stride reaches past all that the smaller ones span)."""
    span = 1
    for st, n in sorted((st, n) for st, n in zip(strides, shape) if n > 1):
        if st < span:
            return False
        span += (n - 1) * st
    return True


def _separate(out, os, x, xs, name, itself=False):
    """out (strides os) shares no memory with x (strides xs), or, if `itself`, is x."""
    a, b, e = out.data_ptr(), x.data_ptr(), x.element_size()
    if itself and a == b and all(n == 1 or i == j for n, i, j in zip(x.shape, os, xs)):
        _require(_distinct(x.shape, xs), f"in place needs {name} without repeated or overlapping rows")
        return
    if out.numel() and x.numel():
        end_a, end_b = (at + e * (1 + sum((n - 1) * st for n, st in zip(t.shape, sts)))
                        for t, at, sts in ((out, a, os), (x, b, xs)))
        _require(a >= end_b or b >= end_a,
                 f"the output must be {name} itself or share no memory with it" if itself else
                 f"the output must share no memory with {name}")


def _lens(cache_lens, B, device):
    return _dense(cache_lens, "cache_lens", torch.int32, device, (B,))


def _positions(positions, B, s, device):
    return None if positions is None else _dense(positions, "positions", torch.int32, device, (B, s))


def _table(block_table, B, device):
    p = _dense(block_table, "block_table", torch.int32, device)
    _require(block_table.dim() == 2 and block_table.shape[0] == B and block_table.shape[1] >= 1,
             "block_table must be int32 [B, max_pages]")
    return p, block_table.shape[1]


_I3, _I9 = ctypes.c_int64 * 3, ctypes.c_int64 * 9
_functions = {}
_device_now, _stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing


def _function(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(library(), name)
    return f


def _call(name, device, args, sizes=None):
    """Calls the library on the device's current stream, with a workspace after `args`: the stream's own, of the status
    header alone or, with `sizes` (the arguments of the matching *_workspace_size), of what the call needs.  A captured
    call gets its scratch from the graph's memory."""
    index = device.index
    if _device_now() != index:
        with torch.cuda.device(device):
            return _call(name, device, args, sizes)
    f, stream = _function(name), _stream_now(index)
    if not _capturing():
        ws = workspaces._ws.get((index, stream))
        if ws is None:
            ws = workspaces.get(_HEADER, device)
        rc = f(*args, ws.data_ptr(), ws.numel(), stream)
        if rc == _TOO_SMALL and sizes is not None:  # nothing was enqueued
            ws = workspaces.get(_function(name + "_workspace_size")(*sizes), device)
            rc = f(*args, ws.data_ptr(), ws.numel(), stream)
    elif sizes is None:
        rc = f(*args, captured_status(device, create=True), _HEADER, stream)
    else:
        ws = torch.empty(max(_function(name + "_workspace_size")(*sizes), _HEADER), dtype=torch.uint8, device=device)
        ws[:_HEADER].zero_()
        rc = f(*args, ws.data_ptr(), ws.numel(), stream)
        # the captured call's flags outlive its scratch
        rc = rc or _function("lka_add_status")(captured_status(device, create=True), ws.data_ptr(), stream)
    if rc:
        _check(name, rc)


def rope_inv_freq(d_rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                  original_length: int = 8192, low: float = 1.0, high: float | None = None, device="cuda"):
    """(inv_freq, amplitude) for the rotary operators: fp64 [d_rot / 2] radians per token on `device`, and the factor
    on cos and sin.  theta_i = base^(-2i / d_rot), scaled for contexts `factor` times the trained length by

      None      nothing
      "linear"  theta / factor (positions interpolated)
      "ntk"     base times factor^(d_rot / (d_rot - 2)): the slowest pair is interpolated, the fastest kept
      "bands"   by the turns r = original_length * theta / 2 pi a pair makes over the trained length: r < low is
                interpolated, r > high kept, linear in r between (default high 4: Llama-3.1)
      "yarn"    the same with high 32, and amplitude 0.1 ln(factor) + 1 (Peng et al. 2023, whose ramp is linear in the
                turns; code that ramps over the pair index between the two borders gives the pairs there other
                frequencies: take the one a checkpoint was trained with)
    """
    _require(d_rot >= 2 and d_rot % 2 == 0, "d_rot must be even")
    _require(base > 0 and factor > 0, "base and factor must be positive")
    i = torch.arange(0, d_rot, 2, dtype=torch.float64)
    if scaling == "ntk":
        _require(d_rot > 2, "ntk scaling needs more than one pair")
        base = base * factor ** (d_rot / (d_rot - 2))
    theta = float(base) ** (-i / d_rot)
    amplitude = 1.0
    if scaling == "linear":
        theta = theta / factor
    elif scaling in ("bands", "yarn"):
        high = (4.0 if scaling == "bands" else 32.0) if high is None else high
        _require(high > low, "high must be greater than low")
        keep = ((original_length * theta / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        theta = theta * (keep + (1.0 - keep) / factor)
        amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    else:
        _require(scaling in (None, "ntk"), f"unknown scaling {scaling!r}")
    return theta.to(device), amplitude


def rope(x, positions, inv_freq, interleaved: bool = False, amplitude: float = 1.0, backward: bool = False, out=None):
    """Rotary positions on the first 2 * len(inv_freq) values of x's last dimension: x [B,h,s,d] bf16 or fp32 (strided
    views allowed), positions int32 [B,s], inv_freq fp64 radians per token.  Pairs (i, i + n), or (2i, 2i + 1) if
    interleaved.  backward=True applies the transpose: the gradient of x from the gradient of the result.
    out: a contiguous tensor of x's shape, or x itself (in place)."""
    dev, code = _code(x, "x")
    xs = _strided(x, "x", x.dtype, dev)
    shape = B, h, s, d = x.shape
    freq = _dense(inv_freq, "inv_freq", torch.float64, dev)
    pos = _dense(positions, "positions", torch.int32, dev, (B, s))
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        same = out is x or out.data_ptr() == x.data_ptr()
        _strided(out, "out", x.dtype, dev) if same else _dense(out, "out", x.dtype, dev, shape)
        _require(out.shape == shape, "out must have x's shape")
        _separate(out, out.stride(), x, xs, "x", itself=True)
    os = out.stride()
    args = (x.data_ptr(), _I3(xs[0], xs[1], xs[2]), pos, freq, out.data_ptr(), _I3(os[0], os[1], os[2]), B, h, s, d,
            2 * inv_freq.numel(), bool(interleaved), bool(backward), amplitude, code)
    if _device_now() == dev.index:
        rc = _function("rope_apply")(*args, _stream_now(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = _function("rope_apply")(*args, _stream_now(dev.index))
    if rc:
        _check("rope_apply", rc)
    return out


def _append_out(q_out, dt, dev, q, qs, k, ks, v, vs):
    _dense(q_out, "q_out", dt, dev, q.shape)
    os = q_out.stride()
    _separate(q_out, os, q, qs, "the queries", itself=True)
    _separate(q_out, os, k, ks, "the new keys")
    _separate(q_out, os, v, vs, "the new values")


def _append_operands(q, k, v, cache_lens, inv_freq, positions, q_out):
    """The checked operands of an append: sizes, and the arguments up to q_out."""
    dev, code = _code(q, "q")
    dt = q.dtype
    qs = _strided(q, "q", dt, dev)
    shape = B, h_q, s, d = q.shape
    ks, vs = _strided(k, "k", dt, dev), _strided(v, "v", dt, dev)
    h_kv = k.shape[1]
    if k.shape != (B, h_kv, s, d) or v.shape != k.shape:
        raise ValueError("q [B,h_q,s,d], k and v [B,h_kv,s,d]")
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _append_out(q_out, dt, dev, q, qs, k, ks, v, vs)
    freq = _dense(inv_freq, "inv_freq", torch.float64, dev)
    return (dev, code, B, h_q, h_kv, s, d, q_out, _lens(cache_lens, B, dev), _positions(positions, B, s, dev), freq,
            2 * inv_freq.numel(), (q.data_ptr(), k.data_ptr(), v.data_ptr(), _I9(*qs[:3], *ks[:3], *vs[:3])))


def _cache_shape(cache, B, h_kv, d):
    if not isinstance(cache, torch.Tensor) or cache.dim() != 4:
        raise ValueError("caches must be [B,h_kv,Lmax,d]")
    return (B, h_kv, cache.shape[2], d)


def _pages_shape(pages, h_kv, d, name="k_pages/v_pages"):
    if not isinstance(pages, torch.Tensor) or pages.dim() != 4:
        raise ValueError(f"{name} must be [num_pages,h_kv,page_size,d]")
    return (pages.shape[0], h_kv, pages.shape[2], d)


def gqa_rope_append(q, k, v, k_cache, v_cache, cache_lens, inv_freq, positions=None, interleaved: bool = False,
                    amplitude: float = 1.0, q_out=None):
    """Rotary positions on a step's queries and keys, and its keys and values into the cache: q [B,h_q,s,d], k, v
    [B,h_kv,s,d] (strided views allowed); token t is written at row cache_lens[b] - s + t of k_cache, v_cache
    [B,h_kv,Lmax,d], and stands at that position unless positions int32 [B,s] says otherwise.  Tokens before row 0
    are padding (not written, their query 0).  Returns the rotated queries [B,h_q,s,d] for gqa_attn (q_out, contiguous,
    where given: q itself, or memory of its own)."""
    dev, code, B, h_q, h_kv, s, d, q_out, lens, pos, freq, d_rot, qkv = _append_operands(
        q, k, v, cache_lens, inv_freq, positions, q_out)
    shape = _cache_shape(k_cache, B, h_kv, d)
    kc, vc = _dense(k_cache, "k_cache", q.dtype, dev, shape), _dense(v_cache, "v_cache", q.dtype, dev, shape)
    _call("gqa_rope_append", dev, (*qkv, lens, pos, freq, q_out.data_ptr(), kc, vc, B, h_q, h_kv, s, d, d_rot, shape[2],
                                   bool(interleaved), amplitude, code))
    return q_out


def gqa_rope_append_paged(q, k, v, k_pages, v_pages, block_table, cache_lens, inv_freq, positions=None,
                          interleaved: bool = False, amplitude: float = 1.0, q_out=None):
    """gqa_rope_append into paged caches: k_pages, v_pages [num_pages,h_kv,page_size,d], block_table int32
    [B,max_pages].  A token whose page is outside the pool is not written (reported in device_status)."""
    dev, code, B, h_q, h_kv, s, d, q_out, lens, pos, freq, d_rot, qkv = _append_operands(
        q, k, v, cache_lens, inv_freq, positions, q_out)
    shape = _pages_shape(k_pages, h_kv, d)
    kc, vc = _dense(k_pages, "k_pages", q.dtype, dev, shape), _dense(v_pages, "v_pages", q.dtype, dev, shape)
    table, max_pages = _table(block_table, B, dev)
    _call("gqa_rope_append_paged", dev, (*qkv, table, lens, pos, freq, q_out.data_ptr(), kc, vc, B, h_q, h_kv, s, d,
                                         d_rot, shape[2], max_pages, shape[0], bool(interleaved), amplitude, code))
    return q_out


def gqa_rope_append_fp8kv(q, k, v, k_cache, v_cache, k_scale, v_scale, cache_lens, inv_freq, positions=None,
                          interleaved: bool = False, amplitude: float = 1.0, q_out=None):
    """gqa_rope_append into e4m3 caches (torch.float8_e4m3fn) with fp32 scales [h_kv]: the caches hold key / k_scale
    and value / v_scale, rounded to nearest even and saturated.  q, k, v bf16."""
    _require(isinstance(q, torch.Tensor) and q.dtype == torch.bfloat16, "q must be torch.bfloat16")
    dev, _, B, h_q, h_kv, s, d, q_out, lens, pos, freq, d_rot, qkv = _append_operands(
        q, k, v, cache_lens, inv_freq, positions, q_out)
    shape = _cache_shape(k_cache, B, h_kv, d)
    kc, vc = _dense(k_cache, "k_cache", _E4M3, dev, shape), _dense(v_cache, "v_cache", _E4M3, dev, shape)
    ks = _dense(k_scale, "k_scale", torch.float32, dev, (h_kv,))
    vs = _dense(v_scale, "v_scale", torch.float32, dev, (h_kv,))
    _call("gqa_rope_append_fp8kv", dev, (*qkv, ks, vs, lens, pos, freq, q_out.data_ptr(), kc, vc, B, h_q, h_kv, s, d,
                                         d_rot, shape[2], bool(interleaved), amplitude))
    return q_out


def _latent_operands(q_r, c_kv, k_r, cache_lens, inv_freq, positions, q_out):
    dev, code = _code(q_r, "q_r")
    dt = q_r.dtype
    qs = _strided(q_r, "q_r", dt, dev)
    shape = B, h_q, s, d_r = q_r.shape
    cs, ks = _strided(c_kv, "c_kv", dt, dev), _strided(k_r, "k_r", dt, dev)
    _require(c_kv.shape[:3] == (B, 1, s) and k_r.shape == (B, 1, s, d_r),
             "q_r [B,h_q,s,d_r], c_kv [B,1,s,r_kv], k_r [B,1,s,d_r]")
    freq = _dense(inv_freq, "inv_freq", torch.float64, dev)
    _require(2 * inv_freq.numel() == d_r, "inv_freq must hold d_r / 2 values")
    if q_out is None:
        q_out = torch.empty_like(q_r, memory_format=torch.contiguous_format)
    else:
        _append_out(q_out, dt, dev, q_r, qs, c_kv, cs, k_r, ks)
    return (dev, code, B, h_q, s, c_kv.shape[3], d_r, q_out, _lens(cache_lens, B, dev),
            _positions(positions, B, s, dev), freq,
            (q_r.data_ptr(), c_kv.data_ptr(), k_r.data_ptr(), _I9(*qs[:3], *ks[:3], *cs[:3])))


def _latent_rows(t, name, n0, width):
    _require(isinstance(t, torch.Tensor) and t.dim() == 3, f"{name} must be 3-D")
    return (t.shape[0] if n0 is None else n0, t.shape[1], width)


def latent_rope_append(q_r, c_kv, k_r, latent, cache_lens, inv_freq, positions=None, interleaved: bool = False,
                       amplitude: float = 1.0, q_out=None):
    """The latent cache's append: q_r [B,h_q,s,d_r] and k_r [B,1,s,d_r] are rotated, and [c_kv ; k_r] (c_kv
    [B,1,s,r_kv]) is written to rows cache_lens[b] - s + t of latent [B,Lmax,r_kv+d_r].  Returns the rotated q_r."""
    dev, code, B, h_q, s, r_kv, d_r, q_out, lens, pos, freq, qck = _latent_operands(
        q_r, c_kv, k_r, cache_lens, inv_freq, positions, q_out)
    shape = _latent_rows(latent, "latent", B, r_kv + d_r)
    cache = _dense(latent, "latent", q_r.dtype, dev, shape)
    _call("latent_rope_append", dev, (*qck, lens, pos, freq, q_out.data_ptr(), cache, B, h_q, s, r_kv, d_r, shape[1],
                                      bool(interleaved), amplitude, code))
    return q_out


def latent_rope_append_paged(q_r, c_kv, k_r, latent_pages, block_table, cache_lens, inv_freq, positions=None,
                             interleaved: bool = False, amplitude: float = 1.0, q_out=None):
    """latent_rope_append into a paged latent cache [num_pages,page_size,r_kv+d_r] through block_table."""
    dev, code, B, h_q, s, r_kv, d_r, q_out, lens, pos, freq, qck = _latent_operands(
        q_r, c_kv, k_r, cache_lens, inv_freq, positions, q_out)
    shape = _latent_rows(latent_pages, "latent_pages", None, r_kv + d_r)
    cache = _dense(latent_pages, "latent_pages", q_r.dtype, dev, shape)
    table, max_pages = _table(block_table, B, dev)
    _call("latent_rope_append_paged", dev, (*qck, table, lens, pos, freq, q_out.data_ptr(), cache, B, h_q, s, r_kv, d_r,
                                            shape[1], max_pages, shape[0], bool(interleaved), amplitude, code))
    return q_out


def latent_rope_append_fp8kv(q_r, c_kv, k_r, latent, kv_scale, cache_lens, inv_freq, positions=None,
                             interleaved: bool = False, amplitude: float = 1.0, q_out=None):
    """latent_rope_append into an e4m3 latent cache with kv_scale fp32 [2]: c_kv / kv_scale[0], k_r / kv_scale[1]."""
    _require(isinstance(q_r, torch.Tensor) and q_r.dtype == torch.bfloat16, "q_r must be torch.bfloat16")
    dev, _, B, h_q, s, r_kv, d_r, q_out, lens, pos, freq, qck = _latent_operands(
        q_r, c_kv, k_r, cache_lens, inv_freq, positions, q_out)
    shape = _latent_rows(latent, "latent", B, r_kv + d_r)
    cache = _dense(latent, "latent", _E4M3, dev, shape)
    sc = _dense(kv_scale, "kv_scale", torch.float32, dev, (2,))
    _call("latent_rope_append_fp8kv", dev, (*qck, sc, lens, pos, freq, q_out.data_ptr(), cache, B, h_q, s, r_kv, d_r,
                                            shape[1], bool(interleaved), amplitude))
    return q_out


def _attn_outputs(q, out, return_lse):
    B, h_q, s, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    else:
        _dense(out, "out", q.dtype, q.device, q.shape)
    lse = torch.empty((B, h_q, s), dtype=torch.float32, device=q.device) if return_lse else None
    return out, lse, lse.data_ptr() if return_lse else None


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _prefix_len(prefix_len, device):
    return None if prefix_len is None else _dense(prefix_len, "prefix_len", torch.int32, device, (1,))


def gqa_attn_shared_prefix(q, k_prefix, v_prefix, k, v, cache_lens, prefix_len=None, causal: bool = True,
                           scale: float | None = None, out=None, return_lse: bool = False):
    """GQA attention of a batch whose sequences share one prefix: q [B,h_q,s_q,d]; k_prefix, v_prefix [h_kv,Lp,d]
    (prefix_len int32 [1] on the device, or all Lp); k, v [B,h_kv,Lmax,d] with cache_lens int32 [B] the suffix
    lengths including the s_q new tokens.  Every query sees the whole prefix, then its suffix as in gqa_attn.
    Returns out [B,h_q,s_q,d] (and lse [B,h_q,s_q] fp32 over all keys if return_lse)."""
    dev, code = _code(q, "q")
    dt = q.dtype
    qp = _dense(q, "q", dt, dev)
    if q.dim() != 4 or k.dim() != 4 or k_prefix.dim() != 3:
        raise ValueError("q [B,h_q,s_q,d], k/v [B,h_kv,Lmax,d], prefix [h_kv,Lp,d]")
    B, h_q, s, d = q.shape
    h_kv, Lmax, Lp = k.shape[1], k.shape[2], k_prefix.shape[1]
    own, shared = (B, h_kv, Lmax, d), (h_kv, Lp, d)
    kp, vp = _dense(k_prefix, "k_prefix", dt, dev, shared), _dense(v_prefix, "v_prefix", dt, dev, shared)
    ko, vo = _dense(k, "k", dt, dev, own), _dense(v, "v", dt, dev, own)
    lens, plen = _lens(cache_lens, B, dev), _prefix_len(prefix_len, dev)
    out, lse, lp = _attn_outputs(q, out, return_lse)
    _call("gqa_attn_shared_prefix", dev, (qp, kp, vp, plen, ko, vo, lens, out.data_ptr(), lp, B, h_q, h_kv, s, d, Lp,
                                          Lmax, bool(causal), _scale(scale, d), code),
          (B, h_q, h_kv, s, d, Lp, Lmax, code))
    return (out, lse) if return_lse else out


def gqa_attn_shared_prefix_paged(q, k_pages, v_pages, prefix_table, prefix_len, block_table, cache_lens,
                                 causal: bool = True, scale: float | None = None, out=None, return_lse: bool = False):
    """gqa_attn_shared_prefix over one paged pool [num_pages,h_kv,page_size,d]: the prefix's pages are prefix_table
    int32 [max_prefix_pages] (prefix_len int32 [1] on the device, or None for all their rows), a sequence's suffix
    starts at row 0 of block_table[b, 0]."""
    dev, code = _code(q, "q")
    dt = q.dtype
    qp = _dense(q, "q", dt, dev)
    _require(q.dim() == 4, "q [B,h_q,s_q,d]")
    B, h_q, s, d = q.shape
    _require(isinstance(k_pages, torch.Tensor) and k_pages.dim() == 4, "k_pages/v_pages [num_pages,h_kv,page_size,d]")
    num_pages, h_kv, page_size, _ = shape = _pages_shape(k_pages, k_pages.shape[1], d)
    kp, vp = _dense(k_pages, "k_pages", dt, dev, shape), _dense(v_pages, "v_pages", dt, dev, shape)
    ptab = _dense(prefix_table, "prefix_table", torch.int32, dev)
    _require(prefix_table.dim() == 1, "prefix_table must be int32 [max_prefix_pages]")
    mp, (table, max_pages) = prefix_table.shape[0], _table(block_table, B, dev)
    lens, plen = _lens(cache_lens, B, dev), _prefix_len(prefix_len, dev)
    out, lse, lp = _attn_outputs(q, out, return_lse)
    _call("gqa_attn_shared_prefix_paged", dev, (qp, kp, vp, ptab, plen, table, lens, out.data_ptr(), lp, B, h_q, h_kv,
                                                s, d, page_size, mp, max_pages, num_pages, bool(causal),
                                                _scale(scale, d), code),
          (B, h_q, h_kv, s, d, page_size, mp, max_pages, code))
    return (out, lse) if return_lse else out


def _weights_out(weights, shape, dev):
    if weights is None:
        return torch.empty(shape, dtype=torch.float32, device=dev), 0
    _dense(weights, "weights", torch.float32, dev, shape)
    return weights, 1


def gqa_key_weights(q, k, lse, cache_lens, weights=None, causal: bool = True, scale: float | None = None):
    """The attention weight each cached key received from these queries, summed over the queries and the heads of its
    group: q, k, cache_lens, causal and scale as given to gqa_attn and lse [B,h_q,s_q] as it returned it.  Returns
    weights fp32 [B,h_kv,Lmax] (0 from cache_lens on), or adds to the given `weights` and returns them."""
    dev, code = _code(q, "q")
    qp = _dense(q, "q", q.dtype, dev)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q [B,h_q,s_q,d], k [B,h_kv,Lmax,d]")
    B, h_q, s, d = q.shape
    shape = _cache_shape(k, B, k.shape[1], d)
    kp, lp = _dense(k, "k", q.dtype, dev, shape), _dense(lse, "lse", torch.float32, dev, (B, h_q, s))
    lens = _lens(cache_lens, B, dev)
    weights, add = _weights_out(weights, shape[:3], dev)
    _call("gqa_key_weights", dev, (qp, kp, lp, lens, weights.data_ptr(), B, h_q, shape[1], s, d, shape[2], bool(causal),
                                   add, _scale(scale, d), code))
    return weights


def gqa_key_weights_paged(q, k_pages, lse, block_table, cache_lens, weights=None, causal: bool = True,
                          scale: float | None = None):
    """gqa_key_weights over a paged key cache [num_pages,h_kv,page_size,d]; weights fp32 [B,h_kv,max_pages*page_size]
    in token order."""
    dev, code = _code(q, "q")
    qp = _dense(q, "q", q.dtype, dev)
    _require(q.dim() == 4 and isinstance(k_pages, torch.Tensor) and k_pages.dim() == 4,
             "q [B,h_q,s_q,d], k_pages [num_pages,h_kv,page_size,d]")
    B, h_q, s, d = q.shape
    num_pages, h_kv, page_size, _ = shape = _pages_shape(k_pages, k_pages.shape[1], d, "k_pages")
    kp, lp = _dense(k_pages, "k_pages", q.dtype, dev, shape), _dense(lse, "lse", torch.float32, dev, (B, h_q, s))
    table, max_pages = _table(block_table, B, dev)
    lens = _lens(cache_lens, B, dev)
    weights, add = _weights_out(weights, (B, h_kv, max_pages * page_size), dev)
    _call("gqa_key_weights_paged", dev, (qp, kp, lp, table, lens, weights.data_ptr(), B, h_q, h_kv, s, d, page_size,
                                         max_pages, num_pages, bool(causal), add, _scale(scale, d), code))
    return weights


def _evict_counts(budget, sinks, recent):
    """The three as the library takes them: no more sinks or recent keys than the budget (larger numbers mean the same,
    and might not fit its integers)."""
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    return budget, min(sinks, max(budget, 0)), min(recent, max(budget, 0))


def _evict_outputs(cache_lens, h_kv, budget):
    return torch.empty_like(cache_lens), cache_lens.new_empty((cache_lens.shape[0], h_kv, budget))


def gqa_evict(k, v, weights, cache_lens, budget: int, sinks: int = 0, recent: int = 0, k_out=None, v_out=None,
              weights_out=None):
    """Cuts k, v [B,h_kv,Lmax,d] (bf16, fp32 or e4m3) to at most `budget` keys per KV head: the first `sinks`, the
    last `recent`, and of the rest those with the largest weights (fp32 [B,h_kv,Lmax]; ties to the lowest position),
    in the order of their positions.  Outputs go to k_out, v_out [B,h_kv,Lout,d] and weights_out [B,h_kv,Lout]
    (allocated with Lout = budget, zero, where not given); k_out=k, v_out=v, weights_out=weights works in place.
    Returns (k_out, v_out, weights_out, new_lens int32 [B], kept int32 [B,h_kv,budget], -1 behind the kept)."""
    _require(isinstance(k, torch.Tensor) and k.dtype in _CACHE_DT and k.dim() == 4,
             "k must be bf16, fp32 or e4m3 [B,h_kv,Lmax,d]")
    dev, dt = k.device, k.dtype
    _require(k.is_cuda, "k must be a CUDA tensor")
    B, h_kv, Lmax, d = shape = k.shape
    budget, sinks, recent = _evict_counts(budget, sinks, recent)
    if budget < 1 or sinks < 0 or recent < 0:
        raise ValueError("budget must be at least 1, sinks and recent at least 0")
    kp, vp = _dense(k, "k", dt, dev, shape), _dense(v, "v", dt, dev, shape)
    wp, lens = _dense(weights, "weights", torch.float32, dev, (B, h_kv, Lmax)), _lens(cache_lens, B, dev)
    _require((k_out is None) == (v_out is None), "k_out and v_out come together")
    if k_out is None:
        k_out, v_out = (torch.zeros((B, h_kv, budget, d), dtype=torch.uint8 if dt == _E4M3 else dt, device=dev).view(dt)
                        for _ in range(2))
    to = _cache_shape(k_out, B, h_kv, d)
    ko, vo = _dense(k_out, "k_out", dt, dev, to), _dense(v_out, "v_out", dt, dev, to)
    _require(to[2] >= budget, "k_out holds fewer rows than the budget")
    if weights_out is None:
        _require(ko != kp or k.numel() == 0, "in place needs weights_out=weights")
        weights_out = weights.new_empty(to[:3])
    wo = _dense(weights_out, "weights_out", torch.float32, dev, to[:3])
    new_lens, kept = _evict_outputs(cache_lens, h_kv, budget)
    _call("gqa_evict", dev, (kp, vp, wp, lens, ko, vo, wo, new_lens.data_ptr(), kept.data_ptr(), B, h_kv, d, Lmax, to[2],
                             budget, sinks, recent, _CACHE_DT[dt]))
    return k_out, v_out, weights_out, new_lens, kept


def gqa_evict_paged(k_pages, v_pages, weights, block_table, cache_lens, budget: int, sinks: int = 0, recent: int = 0):
    """gqa_evict in place over paged caches [num_pages,h_kv,page_size,d] and weights fp32 [B,h_kv,max_pages*page_size]
    in token order.  A sequence's pages must be its own; those its new length no longer reaches are free afterwards.
    Returns (new_lens int32 [B], kept int32 [B,h_kv,budget])."""
    _require(isinstance(k_pages, torch.Tensor) and k_pages.dtype in _CACHE_DT and k_pages.dim() == 4,
             "k_pages must be bf16, fp32 or e4m3 [num_pages,h_kv,page_size,d]")
    dev, dt = k_pages.device, k_pages.dtype
    _require(k_pages.is_cuda, "k_pages must be a CUDA tensor")
    num_pages, h_kv, page_size, d = shape = k_pages.shape
    kp, vp = _dense(k_pages, "k_pages", dt, dev, shape), _dense(v_pages, "v_pages", dt, dev, shape)
    _require(isinstance(block_table, torch.Tensor) and block_table.dim() == 2, "block_table must be int32 [B, max_pages]")
    B = block_table.shape[0]
    table, max_pages = _table(block_table, B, dev)
    wp = _dense(weights, "weights", torch.float32, dev, (B, h_kv, max_pages * page_size))
    lens = _lens(cache_lens, B, dev)
    budget, sinks, recent = _evict_counts(budget, sinks, recent)
    _require(1 <= budget <= max_pages * page_size and sinks >= 0 and recent >= 0,
             "budget must be between 1 and the table's capacity, sinks and recent at least 0")
    new_lens, kept = _evict_outputs(cache_lens, h_kv, budget)
    _call("gqa_evict_paged", dev, (kp, vp, wp, table, lens, new_lens.data_ptr(), kept.data_ptr(), B, h_kv, d, page_size,
                                   max_pages, num_pages, budget, sinks, recent, _CACHE_DT[dt]))
    return new_lens, kept
