"""The split knob at its ends (host logic, CPU only): plans round it up to whole tiles, and hold one split at least."""
import pytest

import latent_kv_attention_b200 as lka
from latent_kv_attention_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lka.library()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B", [2, 40])
def test_the_largest_split_is_one_split(lib, B, dtype):
    def sizes():
        return (lib.gqa_attn_shared_prefix_workspace_size(B, 8, 2, 1, 128, 5000, 300, dtype),
                lib.gqa_attn_shared_prefix_paged_workspace_size(B, 8, 2, 1, 64, 16, 100, 20, dtype),
                lka.gqa_split_count(B, 8, 2, 1, 128, 5000), lka.gqa_split_count(B, 8, 2, 100, 128, 5000))
    prev = lka.set_split_tokens(1 << 20)
    try:
        want = sizes()
        rows = B * 8
        # two partial results a row, one of the prefix and one of the suffix: outputs and normalisers
        assert want[0] >= rows * 2 * (128 + 1) * 4 and want[2:] == (1, 1)
        for knob in ((1 << 31) - 1, 1 << 30, (1 << 31) - 127):
            lka.set_split_tokens(knob)
            assert sizes() == want
        assert lka.set_split_tokens(-5) == 1 << 30 and lka.set_split_tokens(0) == 0
    finally:
        lka.set_split_tokens(prev)
