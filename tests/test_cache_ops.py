"""Host side of the cache operators (CPU only): frequencies, refusals of the C ABI before anything is enqueued, and of
the binding before the library is called."""
import ctypes
import math

import pytest
import torch

import latent_kv_attention_b200 as lka
from latent_kv_attention_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lka.library()


P = ctypes.c_void_p
A = P(1 << 20)  # an aligned address that is never read: these calls are refused on the host
A2 = P(1 << 21)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


# ------------------------------------------------------------------ frequencies
def test_plain_frequencies():
    f, a = lka.rope_inv_freq(8, base=100.0, device="cpu")
    assert f.dtype == torch.float64 and a == 1.0
    assert f.tolist() == pytest.approx([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], rel=1e-14)


def test_linear_and_ntk_scaling():
    f, _ = lka.rope_inv_freq(64, device="cpu")
    lin, a = lka.rope_inv_freq(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-14) and a == 1.0
    ntk, _ = lka.rope_inv_freq(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == f[0] and ntk[-1].item() == pytest.approx(f[-1].item() / 4, rel=1e-12)


@pytest.mark.parametrize("scaling,low,high", [("bands", 1.0, 4.0), ("yarn", 1.0, 32.0)])
def test_scaling_by_turns(scaling, low, high):
    f, _ = lka.rope_inv_freq(128, base=500000.0, device="cpu")
    g, a = lka.rope_inv_freq(128, base=500000.0, scaling=scaling, factor=8.0, original_length=8192, device="cpu")
    assert a == pytest.approx(0.1 * math.log(8.0) + 1 if scaling == "yarn" else 1.0)
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(g[turns > high], f[turns > high])
    assert torch.allclose(g[turns < low], f[turns < low] / 8, rtol=1e-14)
    mid = (turns >= low) & (turns <= high)
    keep = (turns[mid] - low) / (high - low)
    assert mid.any() and torch.allclose(g[mid], f[mid] * keep + f[mid] / 8 * (1 - keep), rtol=1e-12)


@pytest.mark.parametrize("kw", [dict(d_rot=7), dict(d_rot=0), dict(d_rot=8, scaling="other"),
                                dict(d_rot=8, scaling="bands", low=4.0, high=4.0), dict(d_rot=2, scaling="ntk"),
                                dict(d_rot=8, factor=0.0)])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        lka.rope_inv_freq(device="cpu", **kw)


# ------------------------------------------------------------------ the C ABI
def rope_apply(lib, B=1, h=2, s=3, d=64, d_rot=64, dtype=0, x=A, out=A, pos=A, freq=A, amp=1.0, st=True):
    xs = strides(h * s * d, s * d, d) if st else None
    return lib.rope_apply(x, xs, pos, freq, out, xs, B, h, s, d, d_rot, 0, 0, amp, dtype, None)


def test_rope_apply_refusals(lib):
    assert rope_apply(lib, B=0, x=None) == OK
    assert rope_apply(lib, d_rot=63) == INVALID
    assert rope_apply(lib, d_rot=66) == INVALID
    assert rope_apply(lib, h=0) == INVALID
    assert rope_apply(lib, s=0) == INVALID
    assert rope_apply(lib, B=-1) == INVALID
    assert rope_apply(lib, amp=float("nan")) == INVALID
    assert rope_apply(lib, amp=float("inf")) == INVALID
    assert rope_apply(lib, dtype=2) == UNSUPPORTED
    assert rope_apply(lib, d=1024, d_rot=1024) == UNSUPPORTED
    assert rope_apply(lib, x=None) == INVALID
    assert rope_apply(lib, x=P((1 << 20) + 1)) == INVALID  # half an element
    assert rope_apply(lib, pos=None) == INVALID
    assert rope_apply(lib, freq=P((1 << 20) + 4)) == INVALID
    assert rope_apply(lib, st=False) == INVALID


def append(lib, B=1, h_q=8, h_kv=2, s=1, d=64, d_rot=64, Lmax=32, dtype=0, q=A, kc=A, ws=A, ws_bytes=256, lens=A):
    st = strides(*([s * d] * 9))
    return lib.gqa_rope_append(q, A, A, st, lens, None, A, A, kc, A2, B, h_q, h_kv, s, d, d_rot, Lmax, 0, 1.0, dtype, ws,
                               ws_bytes, None)


def test_append_refusals(lib):
    assert append(lib, B=0, q=None, ws=None) == OK
    assert append(lib, d_rot=0) == INVALID
    assert append(lib, Lmax=0) == INVALID
    assert append(lib, dtype=2) == UNSUPPORTED
    assert append(lib, kc=None) == INVALID
    assert append(lib, kc=A2) == INVALID  # one cache for keys and values
    assert append(lib, lens=None) == INVALID
    assert append(lib, ws=None) == WORKSPACE
    assert append(lib, ws_bytes=255) == WORKSPACE
    assert append(lib, ws=P((1 << 20) + 8)) == INVALID
    st = strides(*([64] * 9))

    def paged(page_size=16, max_pages=2, num_pages=4, table=A):
        return lib.gqa_rope_append_paged(A, A, A, st, table, A, None, A, A, A, A2, 1, 8, 2, 1, 64, 64, page_size,
                                         max_pages, num_pages, 0, 1.0, 0, None, 0, None)
    assert paged() == WORKSPACE  # everything else is in order
    assert paged(page_size=12) == INVALID
    assert paged(page_size=4) == INVALID
    assert paged(max_pages=0) == INVALID
    assert paged(num_pages=0) == INVALID
    assert paged(table=None) == INVALID
    assert paged(page_size=1 << 20, max_pages=1 << 12) == INVALID

    def fp8(scale=A):
        return lib.gqa_rope_append_fp8kv(A, A, A, st, scale, A, A, None, A, A, A, A2, 1, 8, 2, 1, 64, 64, 32, 0, 1.0,
                                         None, 0, None)
    assert fp8() == WORKSPACE
    assert fp8(scale=None) == INVALID
    assert lib.latent_rope_append(A, A, A, st, A, None, A, A, None, 1, 8, 1, 512, 64, 32, 0, 1.0, 0, A, 256, None) == INVALID
    assert lib.latent_rope_append(A, A, A, st, A, None, A, A, A, 1, 8, 1, 0, 64, 32, 0, 1.0, 0, A, 256, None) == INVALID


def prefix(lib, B=1, h_q=8, h_kv=2, s=1, d=64, Lp=100, Lmax=32, dtype=0, q=A, kp=A, plen=None, ws=None, ws_bytes=0,
           scale=1.0):
    return lib.gqa_attn_shared_prefix(q, kp, A, plen, A, A, A, A, None, B, h_q, h_kv, s, d, Lp, Lmax, 1, scale, dtype,
                                      ws, ws_bytes, None)


def test_prefix_refusals(lib):
    assert prefix(lib) == WORKSPACE
    assert prefix(lib, B=0, q=None) == OK
    assert prefix(lib, h_q=6, h_kv=4) == INVALID
    assert prefix(lib, d=96) == UNSUPPORTED
    assert prefix(lib, d=256, dtype=1) == UNSUPPORTED
    assert prefix(lib, dtype=2) == UNSUPPORTED
    assert prefix(lib, Lp=-1) == INVALID
    assert prefix(lib, Lmax=0) == INVALID
    assert prefix(lib, q=P((1 << 20) + 8)) == INVALID
    assert prefix(lib, kp=None) == INVALID
    assert prefix(lib, Lp=0, kp=None) == WORKSPACE  # no prefix, no pointer needed
    assert prefix(lib, plen=P((1 << 20) + 2)) == INVALID
    assert prefix(lib, scale=float("nan")) == INVALID
    need = lib.gqa_attn_shared_prefix_workspace_size(1, 8, 2, 1, 64, 100, 32, 0)
    assert need > 256 and prefix(lib, ws=A, ws_bytes=need - 1) == WORKSPACE
    assert lib.gqa_attn_shared_prefix_workspace_size(1, 6, 4, 1, 64, 100, 32, 0) == 0
    assert lib.gqa_attn_shared_prefix_paged_workspace_size(1, 8, 2, 1, 64, 12, 4, 4, 0) == 0
    assert lib.gqa_attn_shared_prefix_paged(A, A, A, None, None, A, A, A, None, 1, 8, 2, 1, 64, 16, 4, 4, 8, 1, 1.0, 0,
                                            A, 1 << 20, None) == INVALID  # no prefix table


def weights(lib, B=1, h_q=8, h_kv=2, s=1, d=64, Lmax=32, dtype=0, lse=A, ws=None, ws_bytes=0):
    return lib.gqa_key_weights(A, A, lse, A, A, B, h_q, h_kv, s, d, Lmax, 1, 0, 1.0, dtype, ws, ws_bytes, None)


def test_key_weight_refusals(lib):
    assert weights(lib) == WORKSPACE
    assert weights(lib, B=0) == OK
    assert weights(lib, h_q=6, h_kv=4) == INVALID
    assert weights(lib, d=80) == UNSUPPORTED
    assert weights(lib, d=256, dtype=1) == UNSUPPORTED
    assert weights(lib, dtype=2) == UNSUPPORTED
    assert weights(lib, lse=None) == INVALID
    assert lib.gqa_key_weights_paged(A, A, A, A, A, A, 1, 8, 2, 1, 64, 24, 2, 4, 1, 0, 1.0, 0, A, 256, None) == INVALID


def evict(lib, B=1, h_kv=2, d=64, Lmax=32, Lout=16, budget=16, sinks=0, recent=0, dtype=0, base=1 << 24, ws=None,
          same_lens=False, ko=None, vo=None, wo=None):
    k, v, w = base, base + (1 << 20), base + (2 << 20)
    ko = base + (3 << 20) if ko is None else ko
    vo = base + (4 << 20) if vo is None else vo
    wo = base + (5 << 20) if wo is None else wo
    lens, new, kept = base + (6 << 20), base + (7 << 20), base + (8 << 20)
    return lib.gqa_evict(P(k), P(v), P(w), P(lens), P(ko), P(vo), P(wo), P(lens if same_lens else new), P(kept), B,
                         h_kv, d, Lmax, Lout, budget, sinks, recent, dtype, ws, 256 if ws else 0, None)


def test_evict_refusals(lib):
    base = 1 << 24
    assert evict(lib) == WORKSPACE
    assert evict(lib, B=0) == OK
    assert evict(lib, budget=0) == INVALID
    assert evict(lib, budget=17) == INVALID                 # more than Lout
    assert evict(lib, sinks=-1) == INVALID
    assert evict(lib, recent=-1) == INVALID
    assert evict(lib, dtype=3) == UNSUPPORTED
    assert evict(lib, d=12) == UNSUPPORTED                  # rows of 24 bytes
    assert evict(lib, d=24, dtype=2) == UNSUPPORTED         # e4m3 rows of 24 bytes
    assert evict(lib, d=32, dtype=2) == WORKSPACE
    assert evict(lib, same_lens=True) == INVALID
    assert evict(lib, ko=base) == INVALID                   # k in place, v not
    assert evict(lib, ko=base, vo=base + (1 << 20), wo=base + (2 << 20)) == INVALID            # in place, Lout != Lmax
    assert evict(lib, ko=base, vo=base + (1 << 20), wo=base + (2 << 20), Lout=32) == WORKSPACE  # in place
    assert evict(lib, ko=base + 128) == INVALID             # overlaps k
    assert evict(lib, ko=base + (4 << 20)) == INVALID       # k_out is v_out
    assert evict(lib, ko=base + (4 << 20) - 128) == INVALID  # and a part of it
    assert lib.gqa_evict_paged(A, A, A2, A, A, P(3 << 20), A, 1, 2, 64, 16, 2, 4, 8, 0, 0, 0, A, 256, None) == INVALID
    assert evict(lib, ko=base + (1 << 20) + 128) == INVALID  # overlaps v
    assert evict(lib, wo=base + (2 << 20) + 16) == INVALID  # overlaps the weights
    assert lib.gqa_evict_paged(A, A, A, A, A, P(1 << 21), A, 1, 2, 64, 16, 2, 4, 33, 0, 0, 0, A, 256, None) == INVALID


# ------------------------------------------------------------------ the binding
def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    lens = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        lka.rope(x, torch.zeros(1, 3, dtype=torch.int32), f)
    with pytest.raises(ValueError):
        lka.gqa_rope_append(x, x, x, x, x, lens, f)
    with pytest.raises(ValueError):
        lka.gqa_attn_shared_prefix(x, x[0], x[0], x, x, lens)
    with pytest.raises(ValueError):
        lka.gqa_key_weights(x, x, torch.zeros(1, 2, 3), lens)
    with pytest.raises(ValueError):
        lka.gqa_evict(x, x, torch.zeros(1, 2, 3), lens, 2)
    with pytest.raises(ValueError):
        lka.gqa_evict(x, x, torch.zeros(1, 2, 3), lens, 0)
    with pytest.raises(ValueError):
        lka.rope(x.half(), torch.zeros(1, 3, dtype=torch.int32), f)


# ------------------------------------------------------------------ byte and FLOP counts
def test_costs_against_counting():
    from latent_kv_attention_b200 import costs

    assert costs.rope_append_bytes(3, 8, 2, 64) == 3 * 64 * 2 * (8 + 8 + 2 + 2 + 2 + 2)
    assert costs.rope_append_bytes(1, 8, 2, 64, 2, 1) == 64 * (8 * 4 + 2 * 6)
    # 2 sequences of suffix 3 and 5 over a prefix of 10, two causal queries each: 10 + 2 and 10 + 3, 10 + 4 and 10 + 5 keys
    assert costs.shared_prefix_flops(10, [3, 5], 4, 64, 2, True) == (12 + 13 + 14 + 15) * 4 * 4 * 64
    assert costs.shared_prefix_bytes(10, [3, 5], 4, 2, 64, 2) == 18 * 2 * 2 * 64 * 2 + 2 * 4 * 2 * 64 * 2 * 2
    assert costs.key_weights_flops([3, 5], 4, 64, 2, True) == (2 + 3 + 4 + 5) * 4 * 2 * 64
    assert costs.key_weights_bytes([3, 5], 4, 2, 64, 2, 8) == 8 * 2 * 64 * 2 + 2 * 4 * 2 * (128 + 4) + 2 * 2 * 8 * 4
    assert costs.evict_bytes([3, 9], 2, 64, 4) == 2 * (12 + 3 * 516 + 16) + 2 * (36 + 4 * 516 + 16)
