"""Shared-prefix attention and key weights at every number of tiles around their rings (marked gpu): the copies, the
products and the releases of a ring's stages have to match from one tile to several turns of it, in whole and in
started tiles, with one row tile and with two.  Against the definitions in fp64; tolerances as in
test_gpu_cache_ops.py."""
import pytest
import torch

import latent_kv_attention_b200 as lka
from test_gpu_cache_ops import DEV, _clean_status, check_prefix, gen, ints, randn, want_weights  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [20, 40])  # 80 rows: one tile; 160: two
def test_prefixes_around_the_ring(d, B):
    h_q, h_kv, L = 8, 2, 3
    g = gen(d + B)
    q, k, v = randn(g, B, h_q, 1, d), randn(g, B, h_kv, L, d), randn(g, B, h_kv, L, d)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    prev = lka.set_split_tokens(1 << 20)  # one split: one block walks all tiles
    try:
        for tiles in range(1, 14):
            for n in (128 * tiles - 127, 128 * tiles - 64, 128 * tiles - 63, 128 * tiles):
                kp, vp = randn(g, h_kv, n, d), randn(g, h_kv, n, d)
                out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens, return_lse=True)
                check_prefix(out, lse, q, kp, vp, k, v, lens, n, True, q.dtype)
                assert lka.device_status() == 0, n
    finally:
        lka.set_split_tokens(prev)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q", [1, 3])
def test_key_weights_around_the_ring(d, h_q):
    """1 to 3 x 9 query tiles of one key head, dealt to the blocks of clusters of one to eight."""
    g = gen(3 * d + h_q)
    for s in [64, 128] + [128 * t + 1 for t in range(1, 9)]:
        for causal in (True, False):
            n = s + 37
            q, k, v = randn(g, 1, h_q, s, d), randn(g, 1, 1, n, d), randn(g, 1, 1, n, d)
            lens = ints(n)
            _, lse = lka.gqa_attn(q, k, v, lens, causal=causal, return_lse=True)
            w = lka.gqa_key_weights(q, k, lse, lens, causal=causal)
            ref = want_weights(q, k, lse, lens, causal, d ** -0.5)
            assert ((w - ref).abs() <= 1e-5 * ref + 1e-30).all(), s
            assert lka.device_status() == 0, s
