"""The binding's workspaces (host logic, on CPU tensors)."""
from types import SimpleNamespace

import torch

import latent_kv_attention_b200 as lka

CPU = torch.device("cpu", 0)


def test_a_larger_workspace_takes_over_the_status():
    w, stream = lka._Workspaces(), SimpleNamespace(cuda_stream=7)
    small = w.get(100, CPU, stream)
    assert small.numel() >= 256 and not small.any()
    small[0] = 2    # a raised flag
    small[64] = 9   # and scratch of a call
    assert w.get(200, CPU, stream) is small
    large = w.get(small.numel() + 1, CPU, stream)
    assert large is not small and large[0] == 2 and not large[4:].any()
    assert w.get(256, CPU, stream) is large
    other = w.get(256, CPU, SimpleNamespace(cuda_stream=8))
    assert not other.any()
