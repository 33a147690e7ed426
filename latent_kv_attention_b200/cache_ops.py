"""Operators around the attention calls: rotary positions and the cache append, attention over a shared prefix,
the attention weight each cached key received, and the eviction of keys by it.

Same contract as the attention functions of the package: the functions check tensors, allocate outputs and pass
pointers to the library on the current stream of the tensors' device; there is no fallback.  q, k, v and the rotary
operands may be strided views whose last dimension is contiguous (a projection's [B, s, h, d] seen as [B, h, s, d]);
caches, pools and everything else is contiguous.

Calls captured into a CUDA graph get scratch of their own from the graph's memory, so graphs that hold the same call
can replay at the same time.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import threading

import torch

from . import (_check, _device_tensor, _dtype_code, _lens_tensor, _ptr, _require, library, workspaces)

_E4M3 = torch.float8_e4m3fn
_CACHE_DT = {torch.bfloat16: 0, torch.float32: 1, _E4M3: 2}
_HEADER = 256  # bytes of a workspace that hold the status word

_captured = {}
_captured_lock = threading.Lock()


def captured_status(device, create=False):
    """The status header that captured calls on `device` raise their flags in (None before the first one): one per
    device, never replaced, because a graph keeps its address."""
    index = device.index if device.index is not None else torch.cuda.current_device()
    with _captured_lock:
        t = _captured.get(index)
        if t is None and create:
            t = _captured[index] = torch.zeros(_HEADER, dtype=torch.uint8, device=device)
        return t


@contextlib.contextmanager
def _on(device):
    """The device's current stream (as a pointer) and whether it is being captured, with the device made current."""
    if device.index == torch.cuda.current_device():
        s = torch.cuda.current_stream()
        yield ctypes.c_void_p(s.cuda_stream), torch.cuda.is_current_stream_capturing()
    else:
        with torch.cuda.device(device):
            s = torch.cuda.current_stream()
            yield ctypes.c_void_p(s.cuda_stream), torch.cuda.is_current_stream_capturing()


def _header(device, capturing):
    return captured_status(device, create=True) if capturing else workspaces.get(_HEADER, device)


def _strided(t, name, dtype, device=None):
    _require(isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 4, f"{name} must be a 4-D CUDA tensor")
    _require(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
    _require(t.stride(3) == 1 or t.shape[3] == 1, f"the last dimension of {name} must be contiguous")
    _require(device is None or t.device == device, f"{name} must be on {device}")


def _dense(t, name, dtype, device, shape=None):
    _device_tensor(t, name, dtype)
    _require(t.device == device, f"{name} must be on {device}")
    _require(shape is None or tuple(t.shape) == tuple(shape), f"{name} must have shape {list(shape or ())}")


def _strides(*ts):
    return (ctypes.c_int64 * (3 * len(ts)))(*[s for t in ts for s in t.stride()[:3]])


def _frequencies(inv_freq, device):
    _dense(inv_freq, "inv_freq", torch.float64, device)
    return 2 * inv_freq.numel()


def _positions(positions, B, s, device):
    if positions is not None:
        _dense(positions, "positions", torch.int32, device, (B, s))
    return positions


def _table(block_table, B, device):
    _dense(block_table, "block_table", torch.int32, device)
    _require(block_table.dim() == 2 and block_table.shape[0] == B and block_table.shape[1] >= 1,
             "block_table must be int32 [B, max_pages]")
    return block_table.shape[1]


def rope_inv_freq(d_rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                  original_length: int = 8192, low: float = 1.0, high: float | None = None, device="cuda"):
    """(inv_freq, amplitude) for the rotary operators: fp64 [d_rot / 2] radians per token on `device`, and the factor
    on cos and sin.  theta_i = base^(-2i / d_rot), scaled for contexts `factor` times the trained length by

      None      nothing
      "linear"  theta / factor (positions interpolated)
      "ntk"     base times factor^(d_rot / (d_rot - 2)): the slowest pair is interpolated, the fastest kept
      "bands"   by the turns r = original_length * theta / 2 pi a pair makes over the trained length: r < low is
                interpolated, r > high kept, linear in r between (default high 4: Llama-3.1)
      "yarn"    the same with high 32, and amplitude 0.1 ln(factor) + 1 (Peng et al. 2023)
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
    code = _dtype_code(x)
    _strided(x, "x", x.dtype)
    B, h, s, d = x.shape
    dev = x.device
    d_rot = _frequencies(inv_freq, dev)
    _dense(positions, "positions", torch.int32, dev, (B, s))
    if out is None:
        out = torch.empty((B, h, s, d), dtype=x.dtype, device=dev)
    elif out.data_ptr() != x.data_ptr() or out.stride() != x.stride():
        _dense(out, "out", x.dtype, dev, x.shape)
        span = 1 + sum((n - 1) * abs(st) for n, st in zip(x.shape, x.stride())) if x.numel() else 0
        e = x.element_size()
        _require(out.data_ptr() >= x.data_ptr() + span * e or x.data_ptr() >= out.data_ptr() + out.numel() * e,
                 "out must be x itself or share no memory with it")
    else:
        _strided(out, "out", x.dtype, dev)
        _require(out.shape == x.shape, "out must have x's shape")
        _require(all(st != 0 or n == 1 for n, st in zip(x.shape, x.stride())), "in place needs x without repeated rows")
    with _on(dev) as (stream, _):
        rc = library().rope_apply(_ptr(x), _strides(x), _ptr(positions), _ptr(inv_freq), _ptr(out), _strides(out), B,
                                  h, s, d, d_rot, int(bool(interleaved)), int(bool(backward)), float(amplitude), code,
                                  stream)
    _check("rope_apply", rc)
    return out


def _append_operands(q, k, v, cache_lens, inv_freq, positions, q_out):
    _strided(q, "q", q.dtype)
    dev = q.device
    B, h_q, s, d = q.shape
    _strided(k, "k", q.dtype, dev)
    _strided(v, "v", q.dtype, dev)
    _require(k.shape[0] == B and k.shape[2:] == (s, d) and v.shape == k.shape, "q [B,h_q,s,d], k and v [B,h_kv,s,d]")
    _lens_tensor(cache_lens, B, dev)
    _positions(positions, B, s, dev)
    if q_out is None:
        q_out = torch.empty((B, h_q, s, d), dtype=q.dtype, device=dev)
    else:
        _dense(q_out, "q_out", q.dtype, dev, q.shape)
    return dev, B, h_q, k.shape[1], s, d, _frequencies(inv_freq, dev), q_out


def gqa_rope_append(q, k, v, k_cache, v_cache, cache_lens, inv_freq, positions=None, interleaved: bool = False,
                    amplitude: float = 1.0, q_out=None):
    """Rotary positions on a step's queries and keys, and its keys and values into the cache: q [B,h_q,s,d], k, v
    [B,h_kv,s,d] (strided views allowed); token t is written at row cache_lens[b] - s + t of k_cache, v_cache
    [B,h_kv,Lmax,d], and stands at that position unless positions int32 [B,s] says otherwise.  Tokens before row 0
    are padding (not written, their query 0).  Returns the rotated queries [B,h_q,s,d] for gqa_attn."""
    code = _dtype_code(q)
    dev, B, h_q, h_kv, s, d, d_rot, q_out = _append_operands(q, k, v, cache_lens, inv_freq, positions, q_out)
    _dense(k_cache, "k_cache", q.dtype, dev)
    _require(k_cache.dim() == 4 and k_cache.shape[:2] == (B, h_kv) and k_cache.shape[3] == d, "caches [B,h_kv,Lmax,d]")
    _dense(v_cache, "v_cache", q.dtype, dev, k_cache.shape)
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().gqa_rope_append(_ptr(q), _ptr(k), _ptr(v), _strides(q, k, v), _ptr(cache_lens), _ptr(positions),
                                       _ptr(inv_freq), _ptr(q_out), _ptr(k_cache), _ptr(v_cache), B, h_q, h_kv, s, d,
                                       d_rot, k_cache.shape[2], int(bool(interleaved)), float(amplitude), code,
                                       _ptr(ws), ws.numel(), stream)
    _check("gqa_rope_append", rc)
    return q_out


def gqa_rope_append_paged(q, k, v, k_pages, v_pages, block_table, cache_lens, inv_freq, positions=None,
                          interleaved: bool = False, amplitude: float = 1.0, q_out=None):
    """gqa_rope_append into paged caches: k_pages, v_pages [num_pages,h_kv,page_size,d], block_table int32
    [B,max_pages].  A token whose page is outside the pool is not written (reported in device_status)."""
    code = _dtype_code(q)
    dev, B, h_q, h_kv, s, d, d_rot, q_out = _append_operands(q, k, v, cache_lens, inv_freq, positions, q_out)
    _dense(k_pages, "k_pages", q.dtype, dev)
    _require(k_pages.dim() == 4 and k_pages.shape[1] == h_kv and k_pages.shape[3] == d,
             "k_pages/v_pages [num_pages,h_kv,page_size,d]")
    _dense(v_pages, "v_pages", q.dtype, dev, k_pages.shape)
    max_pages = _table(block_table, B, dev)
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().gqa_rope_append_paged(_ptr(q), _ptr(k), _ptr(v), _strides(q, k, v), _ptr(block_table),
                                             _ptr(cache_lens), _ptr(positions), _ptr(inv_freq), _ptr(q_out),
                                             _ptr(k_pages), _ptr(v_pages), B, h_q, h_kv, s, d, d_rot, k_pages.shape[2],
                                             max_pages, k_pages.shape[0], int(bool(interleaved)), float(amplitude),
                                             code, _ptr(ws), ws.numel(), stream)
    _check("gqa_rope_append_paged", rc)
    return q_out


def gqa_rope_append_fp8kv(q, k, v, k_cache, v_cache, k_scale, v_scale, cache_lens, inv_freq, positions=None,
                          interleaved: bool = False, amplitude: float = 1.0, q_out=None):
    """gqa_rope_append into e4m3 caches (torch.float8_e4m3fn) with fp32 scales [h_kv]: the caches hold key / k_scale
    and value / v_scale, rounded to nearest even and saturated.  q, k, v bf16."""
    _require(isinstance(q, torch.Tensor) and q.dtype == torch.bfloat16, "q must be torch.bfloat16")
    dev, B, h_q, h_kv, s, d, d_rot, q_out = _append_operands(q, k, v, cache_lens, inv_freq, positions, q_out)
    _dense(k_cache, "k_cache", _E4M3, dev)
    _require(k_cache.dim() == 4 and k_cache.shape[:2] == (B, h_kv) and k_cache.shape[3] == d, "caches [B,h_kv,Lmax,d]")
    _dense(v_cache, "v_cache", _E4M3, dev, k_cache.shape)
    _dense(k_scale, "k_scale", torch.float32, dev, (h_kv,))
    _dense(v_scale, "v_scale", torch.float32, dev, (h_kv,))
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().gqa_rope_append_fp8kv(_ptr(q), _ptr(k), _ptr(v), _strides(q, k, v), _ptr(k_scale),
                                             _ptr(v_scale), _ptr(cache_lens), _ptr(positions), _ptr(inv_freq),
                                             _ptr(q_out), _ptr(k_cache), _ptr(v_cache), B, h_q, h_kv, s, d, d_rot,
                                             k_cache.shape[2], int(bool(interleaved)), float(amplitude), _ptr(ws),
                                             ws.numel(), stream)
    _check("gqa_rope_append_fp8kv", rc)
    return q_out


def _latent_operands(q_r, c_kv, k_r, cache_lens, inv_freq, positions, q_out):
    _strided(q_r, "q_r", q_r.dtype)
    dev = q_r.device
    B, h_q, s, d_r = q_r.shape
    _strided(c_kv, "c_kv", q_r.dtype, dev)
    _strided(k_r, "k_r", q_r.dtype, dev)
    _require(c_kv.shape[:3] == (B, 1, s) and k_r.shape == (B, 1, s, d_r), "q_r [B,h_q,s,d_r], c_kv [B,1,s,r_kv], k_r [B,1,s,d_r]")
    _lens_tensor(cache_lens, B, dev)
    _positions(positions, B, s, dev)
    _require(_frequencies(inv_freq, dev) == d_r, "inv_freq must hold d_r / 2 values")
    if q_out is None:
        q_out = torch.empty((B, h_q, s, d_r), dtype=q_r.dtype, device=dev)
    else:
        _dense(q_out, "q_out", q_r.dtype, dev, q_r.shape)
    return dev, B, h_q, s, c_kv.shape[3], d_r, q_out


def latent_rope_append(q_r, c_kv, k_r, latent, cache_lens, inv_freq, positions=None, interleaved: bool = False,
                       amplitude: float = 1.0, q_out=None):
    """The latent cache's append: q_r [B,h_q,s,d_r] and k_r [B,1,s,d_r] are rotated, and [c_kv ; k_r] (c_kv
    [B,1,s,r_kv]) is written to rows cache_lens[b] - s + t of latent [B,Lmax,r_kv+d_r].  Returns the rotated q_r."""
    code = _dtype_code(q_r)
    dev, B, h_q, s, r_kv, d_r, q_out = _latent_operands(q_r, c_kv, k_r, cache_lens, inv_freq, positions, q_out)
    _dense(latent, "latent", q_r.dtype, dev)
    _require(latent.dim() == 3 and latent.shape[0] == B and latent.shape[2] == r_kv + d_r, "latent [B,Lmax,r_kv+d_r]")
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().latent_rope_append(_ptr(q_r), _ptr(c_kv), _ptr(k_r), _strides(q_r, k_r, c_kv), _ptr(cache_lens),
                                          _ptr(positions), _ptr(inv_freq), _ptr(q_out), _ptr(latent), B, h_q, s, r_kv,
                                          d_r, latent.shape[1], int(bool(interleaved)), float(amplitude), code,
                                          _ptr(ws), ws.numel(), stream)
    _check("latent_rope_append", rc)
    return q_out


def latent_rope_append_paged(q_r, c_kv, k_r, latent_pages, block_table, cache_lens, inv_freq, positions=None,
                             interleaved: bool = False, amplitude: float = 1.0, q_out=None):
    """latent_rope_append into a paged latent cache [num_pages,page_size,r_kv+d_r] through block_table."""
    code = _dtype_code(q_r)
    dev, B, h_q, s, r_kv, d_r, q_out = _latent_operands(q_r, c_kv, k_r, cache_lens, inv_freq, positions, q_out)
    _dense(latent_pages, "latent_pages", q_r.dtype, dev)
    _require(latent_pages.dim() == 3 and latent_pages.shape[2] == r_kv + d_r, "latent_pages [num_pages,page_size,r_kv+d_r]")
    max_pages = _table(block_table, B, dev)
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().latent_rope_append_paged(_ptr(q_r), _ptr(c_kv), _ptr(k_r), _strides(q_r, k_r, c_kv),
                                                _ptr(block_table), _ptr(cache_lens), _ptr(positions), _ptr(inv_freq),
                                                _ptr(q_out), _ptr(latent_pages), B, h_q, s, r_kv, d_r,
                                                latent_pages.shape[1], max_pages, latent_pages.shape[0],
                                                int(bool(interleaved)), float(amplitude), code, _ptr(ws), ws.numel(),
                                                stream)
    _check("latent_rope_append_paged", rc)
    return q_out


def latent_rope_append_fp8kv(q_r, c_kv, k_r, latent, kv_scale, cache_lens, inv_freq, positions=None,
                             interleaved: bool = False, amplitude: float = 1.0, q_out=None):
    """latent_rope_append into an e4m3 latent cache with kv_scale fp32 [2]: c_kv / kv_scale[0], k_r / kv_scale[1]."""
    _require(isinstance(q_r, torch.Tensor) and q_r.dtype == torch.bfloat16, "q_r must be torch.bfloat16")
    dev, B, h_q, s, r_kv, d_r, q_out = _latent_operands(q_r, c_kv, k_r, cache_lens, inv_freq, positions, q_out)
    _dense(latent, "latent", _E4M3, dev)
    _require(latent.dim() == 3 and latent.shape[0] == B and latent.shape[2] == r_kv + d_r, "latent [B,Lmax,r_kv+d_r]")
    _dense(kv_scale, "kv_scale", torch.float32, dev, (2,))
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().latent_rope_append_fp8kv(_ptr(q_r), _ptr(c_kv), _ptr(k_r), _strides(q_r, k_r, c_kv),
                                                _ptr(kv_scale), _ptr(cache_lens), _ptr(positions), _ptr(inv_freq),
                                                _ptr(q_out), _ptr(latent), B, h_q, s, r_kv, d_r, latent.shape[1],
                                                int(bool(interleaved)), float(amplitude), _ptr(ws), ws.numel(), stream)
    _check("latent_rope_append_fp8kv", rc)
    return q_out


def _attn_outputs(q, scale, out, return_lse):
    B, h_q, s, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    else:
        _dense(out, "out", q.dtype, q.device, q.shape)
    lse = torch.empty((B, h_q, s), dtype=torch.float32, device=q.device) if return_lse else None
    return scale, out, lse


def _prefix_scratch(nbytes, dev, capturing):
    if not capturing:
        return workspaces.get(nbytes, dev)
    ws = torch.empty(max(nbytes, _HEADER), dtype=torch.uint8, device=dev)
    ws[:_HEADER].zero_()
    return ws


def _prefix_done(ws, dev, capturing):
    if capturing:  # the captured call's flags outlive its scratch
        captured_status(dev, create=True)[:4].view(torch.int32).bitwise_or_(ws[:4].view(torch.int32))


def _prefix_len(prefix_len, device):
    if prefix_len is not None:
        _dense(prefix_len, "prefix_len", torch.int32, device)
        _require(prefix_len.numel() == 1, "prefix_len must be int32 [1] on the device")


def gqa_attn_shared_prefix(q, k_prefix, v_prefix, k, v, cache_lens, prefix_len=None, causal: bool = True,
                           scale: float | None = None, out=None, return_lse: bool = False):
    """GQA attention of a batch whose sequences share one prefix: q [B,h_q,s_q,d]; k_prefix, v_prefix [h_kv,Lp,d]
    (prefix_len int32 [1] on the device, or all Lp); k, v [B,h_kv,Lmax,d] with cache_lens int32 [B] the suffix
    lengths including the s_q new tokens.  Every query sees the whole prefix, then its suffix as in gqa_attn.
    Returns out [B,h_q,s_q,d] (and lse [B,h_q,s_q] fp32 over all keys if return_lse)."""
    code = _dtype_code(q)
    _device_tensor(q, "q", q.dtype)
    dev = q.device
    _require(q.dim() == 4 and k.dim() == 4 and k_prefix.dim() == 3, "q [B,h_q,s_q,d], k/v [B,h_kv,Lmax,d], prefix [h_kv,Lp,d]")
    B, h_q, s, d = q.shape
    h_kv, Lmax, Lp = k.shape[1], k.shape[2], k_prefix.shape[1]
    _dense(k, "k", q.dtype, dev, (B, h_kv, Lmax, d))
    _dense(v, "v", q.dtype, dev, k.shape)
    _dense(k_prefix, "k_prefix", q.dtype, dev, (h_kv, Lp, d))
    _dense(v_prefix, "v_prefix", q.dtype, dev, k_prefix.shape)
    _lens_tensor(cache_lens, B, dev)
    _prefix_len(prefix_len, dev)
    scale, out, lse = _attn_outputs(q, scale, out, return_lse)
    lib = library()
    with _on(dev) as (stream, capturing):
        ws = _prefix_scratch(lib.gqa_attn_shared_prefix_workspace_size(B, h_q, h_kv, s, d, Lp, Lmax, code), dev, capturing)
        rc = lib.gqa_attn_shared_prefix(_ptr(q), _ptr(k_prefix), _ptr(v_prefix), _ptr(prefix_len), _ptr(k), _ptr(v),
                                        _ptr(cache_lens), _ptr(out), _ptr(lse), B, h_q, h_kv, s, d, Lp, Lmax,
                                        int(bool(causal)), scale, code, _ptr(ws), ws.numel(), stream)
        _check("gqa_attn_shared_prefix", rc)
        _prefix_done(ws, dev, capturing)
    return (out, lse) if return_lse else out


def gqa_attn_shared_prefix_paged(q, k_pages, v_pages, prefix_table, prefix_len, block_table, cache_lens,
                                 causal: bool = True, scale: float | None = None, out=None, return_lse: bool = False):
    """gqa_attn_shared_prefix over one paged pool [num_pages,h_kv,page_size,d]: the prefix's pages are prefix_table
    int32 [max_prefix_pages] (prefix_len int32 [1] on the device, or None for all their rows), a sequence's suffix
    starts at row 0 of block_table[b, 0]."""
    code = _dtype_code(q)
    _device_tensor(q, "q", q.dtype)
    dev = q.device
    _require(q.dim() == 4 and k_pages.dim() == 4, "q [B,h_q,s_q,d], k_pages/v_pages [num_pages,h_kv,page_size,d]")
    B, h_q, s, d = q.shape
    num_pages, h_kv, page_size, dk = k_pages.shape
    _require(dk == d, "q and the pages disagree on d")
    _dense(k_pages, "k_pages", q.dtype, dev)
    _dense(v_pages, "v_pages", q.dtype, dev, k_pages.shape)
    _dense(prefix_table, "prefix_table", torch.int32, dev)
    _require(prefix_table.dim() == 1, "prefix_table must be int32 [max_prefix_pages]")
    mp, max_pages = prefix_table.shape[0], _table(block_table, B, dev)
    _lens_tensor(cache_lens, B, dev)
    _prefix_len(prefix_len, dev)
    scale, out, lse = _attn_outputs(q, scale, out, return_lse)
    lib = library()
    with _on(dev) as (stream, capturing):
        nbytes = lib.gqa_attn_shared_prefix_paged_workspace_size(B, h_q, h_kv, s, d, page_size, mp, max_pages, code)
        ws = _prefix_scratch(nbytes, dev, capturing)
        rc = lib.gqa_attn_shared_prefix_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(prefix_table),
                                              _ptr(prefix_len), _ptr(block_table), _ptr(cache_lens), _ptr(out),
                                              _ptr(lse), B, h_q, h_kv, s, d, page_size, mp, max_pages, num_pages,
                                              int(bool(causal)), scale, code, _ptr(ws), ws.numel(), stream)
        _check("gqa_attn_shared_prefix_paged", rc)
        _prefix_done(ws, dev, capturing)
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
    code = _dtype_code(q)
    for n, t in (("q", q), ("k", k)):
        _device_tensor(t, n, q.dtype)
    dev = q.device
    _require(q.dim() == 4 and k.dim() == 4 and k.device == dev, "q [B,h_q,s_q,d], k [B,h_kv,Lmax,d]")
    B, h_q, s, d = q.shape
    _, h_kv, Lmax, dk = k.shape
    _require(dk == d and k.shape[0] == B, "q and k disagree on B or d")
    _dense(lse, "lse", torch.float32, dev, (B, h_q, s))
    _lens_tensor(cache_lens, B, dev)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    weights, add = _weights_out(weights, (B, h_kv, Lmax), dev)
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().gqa_key_weights(_ptr(q), _ptr(k), _ptr(lse), _ptr(cache_lens), _ptr(weights), B, h_q, h_kv, s,
                                       d, Lmax, int(bool(causal)), add, scale, code, _ptr(ws), ws.numel(), stream)
    _check("gqa_key_weights", rc)
    return weights


def gqa_key_weights_paged(q, k_pages, lse, block_table, cache_lens, weights=None, causal: bool = True,
                          scale: float | None = None):
    """gqa_key_weights over a paged key cache [num_pages,h_kv,page_size,d]; weights fp32 [B,h_kv,max_pages*page_size]
    in token order."""
    code = _dtype_code(q)
    for n, t in (("q", q), ("k_pages", k_pages)):
        _device_tensor(t, n, q.dtype)
    dev = q.device
    _require(q.dim() == 4 and k_pages.dim() == 4 and k_pages.device == dev,
             "q [B,h_q,s_q,d], k_pages [num_pages,h_kv,page_size,d]")
    B, h_q, s, d = q.shape
    num_pages, h_kv, page_size, dk = k_pages.shape
    _require(dk == d, "q and the pages disagree on d")
    max_pages = _table(block_table, B, dev)
    _dense(lse, "lse", torch.float32, dev, (B, h_q, s))
    _lens_tensor(cache_lens, B, dev)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    weights, add = _weights_out(weights, (B, h_kv, max_pages * page_size), dev)
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().gqa_key_weights_paged(_ptr(q), _ptr(k_pages), _ptr(lse), _ptr(block_table), _ptr(cache_lens),
                                             _ptr(weights), B, h_q, h_kv, s, d, page_size, max_pages, num_pages,
                                             int(bool(causal)), add, scale, code, _ptr(ws), ws.numel(), stream)
    _check("gqa_key_weights_paged", rc)
    return weights


def _evict_outputs(B, h_kv, budget, dev):
    return (torch.empty((B,), dtype=torch.int32, device=dev),
            torch.empty((B, h_kv, budget), dtype=torch.int32, device=dev))


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
    B, h_kv, Lmax, d = k.shape
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    _require(budget >= 1 and sinks >= 0 and recent >= 0, "budget must be at least 1, sinks and recent at least 0")
    _dense(k, "k", dt, dev)
    _dense(v, "v", dt, dev, k.shape)
    _dense(weights, "weights", torch.float32, dev, (B, h_kv, Lmax))
    _lens_tensor(cache_lens, B, dev)
    _require((k_out is None) == (v_out is None), "k_out and v_out come together")
    if k_out is None:
        k_out, v_out = (torch.zeros((B, h_kv, budget, d), dtype=torch.uint8 if dt == _E4M3 else dt, device=dev).view(dt)
                        for _ in range(2))
    _dense(k_out, "k_out", dt, dev)
    _require(k_out.dim() == 4 and k_out.shape[:2] == (B, h_kv) and k_out.shape[3] == d, "k_out [B,h_kv,Lout,d]")
    Lout = k_out.shape[2]
    _require(Lout >= budget, "k_out holds fewer rows than the budget")
    _dense(v_out, "v_out", dt, dev, k_out.shape)
    if weights_out is None:
        _require(k_out.data_ptr() != k.data_ptr() or k.numel() == 0, "in place needs weights_out=weights")
        weights_out = torch.empty((B, h_kv, Lout), dtype=torch.float32, device=dev)
    _dense(weights_out, "weights_out", torch.float32, dev, (B, h_kv, Lout))
    new_lens, kept = _evict_outputs(B, h_kv, budget, dev)
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().gqa_evict(_ptr(k), _ptr(v), _ptr(weights), _ptr(cache_lens), _ptr(k_out), _ptr(v_out),
                                 _ptr(weights_out), _ptr(new_lens), _ptr(kept), B, h_kv, d, Lmax, Lout, budget, sinks,
                                 recent, _CACHE_DT[dt], _ptr(ws), ws.numel(), stream)
    _check("gqa_evict", rc)
    return k_out, v_out, weights_out, new_lens, kept


def gqa_evict_paged(k_pages, v_pages, weights, block_table, cache_lens, budget: int, sinks: int = 0, recent: int = 0):
    """gqa_evict in place over paged caches [num_pages,h_kv,page_size,d] and weights fp32 [B,h_kv,max_pages*page_size]
    in token order.  A sequence's pages must be its own; those its new length no longer reaches are free afterwards.
    Returns (new_lens int32 [B], kept int32 [B,h_kv,budget])."""
    _require(isinstance(k_pages, torch.Tensor) and k_pages.dtype in _CACHE_DT and k_pages.dim() == 4,
             "k_pages must be bf16, fp32 or e4m3 [num_pages,h_kv,page_size,d]")
    dev, dt = k_pages.device, k_pages.dtype
    num_pages, h_kv, page_size, d = k_pages.shape
    _dense(k_pages, "k_pages", dt, dev)
    _dense(v_pages, "v_pages", dt, dev, k_pages.shape)
    _require(isinstance(block_table, torch.Tensor) and block_table.dim() == 2, "block_table must be int32 [B, max_pages]")
    B = block_table.shape[0]
    max_pages = _table(block_table, B, dev)
    _dense(weights, "weights", torch.float32, dev, (B, h_kv, max_pages * page_size))
    _lens_tensor(cache_lens, B, dev)
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    _require(1 <= budget <= max_pages * page_size and sinks >= 0 and recent >= 0,
             "budget must be between 1 and the table's capacity, sinks and recent at least 0")
    new_lens, kept = _evict_outputs(B, h_kv, budget, dev)
    with _on(dev) as (stream, capturing):
        ws = _header(dev, capturing)
        rc = library().gqa_evict_paged(_ptr(k_pages), _ptr(v_pages), _ptr(weights), _ptr(block_table),
                                       _ptr(cache_lens), _ptr(new_lens), _ptr(kept), B, h_kv, d, page_size, max_pages,
                                       num_pages, budget, sinks, recent, _CACHE_DT[dt], _ptr(ws), ws.numel(), stream)
    _check("gqa_evict_paged", rc)
    return new_lens, kept
