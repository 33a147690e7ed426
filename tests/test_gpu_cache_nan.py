"""NaN and infinities in the operands of the cache operators (marked gpu): what a NaN score reaches is what it reaches in
gqa_attn, and rows that are marked as empty give nothing, whatever they hold."""
import math

import pytest
import torch

import latent_kv_attention_b200 as lka
from test_gpu_cache_ops import _clean_status, gen, ints, prefix_case, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,d,dtype", [(3, 128, "bf16"), (1, 64, "bf16"), (40, 64, "bf16"), (40, 128, "bf16"), (12, 256, "bf16"),
                                       (3, 64, "fp32"), (40, 128, "fp32")])
@pytest.mark.parametrize("where", ["query", "prefix", "suffix", "whole prefix"])
def test_nan_reaches_the_rows_it_reaches_in_gqa_attn(B, d, dtype, where):
    """A NaN in a query, a prefix key or a suffix key makes NaN of the outputs and the normalisers of the rows that score
    it, and of no other."""
    case = (B, 8, 2, 1, d, 900, 100, True, dtype, 0)
    q, kp, vp, k, v, lens, n, dt = prefix_case(case, 90 + B)
    k, v = torch.nan_to_num(k, 0.0, 0.0, 0.0), torch.nan_to_num(v, 0.0, 0.0, 0.0)
    if where == "query":
        q[-1, 2, 0, 3] = math.nan
    elif where == "prefix":
        kp[0, 700, 5] = math.nan
    elif where == "whole prefix":
        kp[1] = math.nan
    else:
        k[-1, 1, 0, 5] = math.nan
    out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens, return_lse=True)
    kk, vv = (torch.cat((a[None].expand(B, -1, -1, -1), b), 2).contiguous() for a, b in ((kp, k), (vp, v)))
    ref, ref_lse = lka.gqa_attn(q, kk, vv, lens + 900, return_lse=True)
    assert ref_lse.isnan().any()
    assert torch.equal(lse.isnan(), ref_lse.isnan()) and torch.equal(out.isnan(), ref.isnan())
    assert not lse.isinf().any()


@pytest.mark.parametrize("s,dtype,d,causal", [(1, "bf16", 128, True), (3, "bf16", 256, True), (40, "bf16", 64, False),
                                              (130, "bf16", 64, True), (300, "bf16", 128, False), (70, "bf16", 256, True),
                                              (3, "fp32", 64, True), (40, "fp32", 128, False)])
def test_weights_of_empty_rows_that_hold_nan(s, dtype, d, causal):
    """Rows whose lse is -inf add nothing to any key, even where their queries are NaN or infinite."""
    g = gen(4)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v = (randn(g, 2, h, n, d, dtype=dt) for h, n in ((8, s), (2, 350), (2, 350)))
    lens = ints(350, 310)
    _, lse = lka.gqa_attn(q, k, v, lens, causal=causal, return_lse=True)
    for row in ((0, 1, 0), (1, 7, s - 1), (1, 2, s // 2)):
        lse[row] = -math.inf
    want = lka.gqa_key_weights(q, k, lse, lens, causal=causal)
    assert not want.isnan().any()
    for bad in (math.nan, math.inf, -math.inf):
        for row in ((0, 1, 0), (1, 7, s - 1), (1, 2, s // 2)):
            q[row] = bad
        assert torch.equal(lka.gqa_key_weights(q, k, lse, lens, causal=causal), want)
