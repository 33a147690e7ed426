"""The timing hook on the cache operators (marked gpu): every call is one timed launch, of its main kernels."""
import pytest
import torch

import latent_kv_attention_b200 as lka
from test_gpu_cache_ops import DEV, E4M3, _clean_status, gen, ints, prefix_case, randn, to_pool  # noqa: F401

pytestmark = pytest.mark.gpu


def calls():
    g = gen(1)
    f, _ = lka.rope_inv_freq(64)
    B, h_q, h_kv, s, d, cap = 3, 8, 2, 2, 64, 64
    q, k = randn(g, B, h_q, s, d), randn(g, B, h_kv, s, d)
    kc, vc = randn(g, B, h_kv, cap, d), randn(g, B, h_kv, cap, d)
    lens = ints(64, 5, 30)
    (kp, table), (vp, _) = to_pool(kc, 16, gen(2)), to_pool(vc, 16, gen(2))
    k8, v8 = kc.to(E4M3), vc.to(E4M3)
    scale = torch.full((h_kv,), 0.1, device=DEV)
    qr, ckv, kr = randn(g, B, h_q, s, d), randn(g, B, 1, s, 128), randn(g, B, 1, s, d)
    lat = randn(g, B, cap, 192)
    _, lse = lka.gqa_attn(q, kc, vc, lens, return_lse=True)
    w = torch.rand(B, h_kv, cap, generator=g, device=DEV)
    long_q, long_lens = randn(g, B, h_q, 64, d), ints(64, 64, 64)
    _, long_lse = lka.gqa_attn(long_q, kc, vc, long_lens, return_lse=True)
    pre = {n: prefix_case(c, 1)[:6] for n, c in {
        "few": (2, 4, 2, 1, 64, 64, 30, True, "bf16", 0), "many": (64, 4, 2, 1, 64, 64, 30, True, "bf16", 0),
        "none": (64, 4, 2, 1, 64, 0, 30, True, "bf16", 0), "d256": (64, 4, 2, 1, 256, 64, 30, True, "bf16", 0),
        "fp32": (5, 4, 2, 1, 64, 64, 30, True, "fp32", 0), "fp32 twice": (40, 32, 2, 1, 128, 9000, 70, True, "fp32", 0)}.items()}
    yield "rope", lambda: lka.rope(q, torch.zeros((B, s), dtype=torch.int32, device=DEV), f)
    yield "append", lambda: lka.gqa_rope_append(q, k, k, kc, vc, lens, f)
    yield "append paged", lambda: lka.gqa_rope_append_paged(q, k, k, kp, vp, table, lens, f)
    yield "append e4m3", lambda: lka.gqa_rope_append_fp8kv(q, k, k, k8, v8, scale, scale, lens, f)
    yield "latent", lambda: lka.latent_rope_append(qr, ckv, kr, lat, lens, f)
    yield "latent paged", lambda: lka.latent_rope_append_paged(qr, ckv, kr, lat.view(B * 4, 16, 192), table, lens, f)
    yield "latent e4m3", lambda: lka.latent_rope_append_fp8kv(qr, ckv, kr, lat.to(E4M3), scale, lens, f)
    for n, c in pre.items():
        yield "prefix " + n, lambda c=c: lka.gqa_attn_shared_prefix(*c)
    yield "prefix paged", lambda: lka.gqa_attn_shared_prefix_paged(q, kp, vp, table[0].contiguous(), ints(50), table, lens)
    yield "weights", lambda: lka.gqa_key_weights(q, kc, lse, lens)
    yield "weights paged", lambda: lka.gqa_key_weights_paged(q, kp, lse, table, lens)
    yield "weights of a prompt", lambda: lka.gqa_key_weights(long_q, kc, long_lse, long_lens)
    yield "weights fp32", lambda: lka.gqa_key_weights(q.float(), kc.float(), lse, lens)
    yield "evict", lambda: lka.gqa_evict(kc, vc, w, lens, 10)
    yield "evict in place", lambda: lka.gqa_evict(kc, vc, w, lens, 60, k_out=kc, v_out=vc, weights_out=w)
    yield "evict paged", lambda: lka.gqa_evict_paged(kp, vp, w, table, lens, 10)


def test_every_call_is_one_timed_launch():
    seen = {}
    for name, call in calls():
        lka.kernel_timing(True)
        try:
            call()
            seen[name] = lka.kernel_timing_read()
        finally:
            lka.kernel_timing(False)
    assert {n: c for n, (c, _) in seen.items()} == dict.fromkeys(seen, 1)
    assert all(0 < ms < 50 for _, ms in seen.values()), seen
