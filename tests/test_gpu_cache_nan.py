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
