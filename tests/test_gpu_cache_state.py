"""Status words, workspaces and captured graphs of the cache operators (marked gpu): what one call raises or leaves
behind, no other call loses, clears or takes for its own."""
import os
import subprocess
import sys

import pytest
import torch

import latent_kv_attention_b200 as lka
from test_gpu_cache_ops import DEV, gen, prefix_case, randn

pytestmark = pytest.mark.gpu
BAD_LENGTH = 6
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _clear_status():
    lka.clear_status()
    yield
    lka.clear_status()


def append_args(length, B=2):
    """Operands of a gqa_rope_append of one token per sequence into caches of 16 rows."""
    g = gen(1)
    f, _ = lka.rope_inv_freq(64)
    q, k = randn(g, B, 4, 1, 64), randn(g, B, 2, 1, 64)
    kc, vc = randn(g, B, 2, 16, 64), randn(g, B, 2, 16, 64)
    return q, k, k, kc, vc, torch.full((B,), length, dtype=torch.int32, device=DEV), f


def captured(call):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_graphs_that_replay_together_lose_no_flag():
    """One graph raises a flag in the shared header while another adds the (empty) flags of its calls to it."""
    q, kp, vp, k, v, lens, _, _ = prefix_case((2, 4, 2, 1, 64, 64, 30, True, "bf16", 0), 1)
    a = append_args(17)
    lka.gqa_rope_append(*a)
    lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens)
    raises = captured(lambda: lka.gqa_rope_append(*a))
    adds = captured(lambda: [lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens) for _ in range(30)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(500):
        lka.clear_status()
        torch.cuda.synchronize()
        for s, g in zip(streams, (adds, raises)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert lka.device_status() == BAD_LENGTH


CAPTURE_FIRST = """
import sys
sys.path[:0] = ["tests", "."]
import torch
import latent_kv_attention_b200 as lka
from test_gpu_cache_ops import gen, ints, randn
g = gen(1)
sets = []
f = torch.ones(32, dtype=torch.float64, device="cuda")
for i in range(2):
    q, k = randn(g, 1, 4, 1, 64), randn(g, 1, 2, 1, 64)
    sets.append((q, k, k.clone(), randn(g, 1, 2, 16, 64), randn(g, 1, 2, 16, 64), ints(3), f))
p = randn(g, 2, 100, 64)
junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
del junk
torch.cuda.synchronize()
torch.cuda.empty_cache()  # what the graphs allocate may hold anything
graphs = []
for s in sets:
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        q = lka.gqa_rope_append(*s)
        lka.gqa_attn_shared_prefix(q, p, p, s[3], s[4], s[5])
    graphs.append(gr)
seen = [lka.device_status()]
for gr in graphs:
    gr.replay()
seen.append(lka.device_status())
sets[1][5].fill_(99)
graphs[1].replay()
graphs[0].replay()
seen.append(lka.device_status())
lka.clear_status()
graphs[0].replay()
seen.append(lka.device_status())
print(*seen)
"""


def test_first_calls_of_a_process_in_captures():
    """Graphs captured before any eager call: no status before the first replay, and a replay of one clears no flag of
    another's."""
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    assert r.stdout.split() == ["0", "0", str(BAD_LENGTH), "0"]


@pytest.mark.parametrize("later", ["prefix", "gqa_attn"])
def test_status_outlives_the_growth_of_a_workspace(later):
    """The flags of a call on a small workspace are still there when a later call on the stream needs a larger one."""
    with torch.cuda.stream(torch.cuda.Stream()):
        lka.gqa_rope_append(*append_args(17))
        q, kp, vp, k, v, lens, _, _ = prefix_case((64, 32, 8, 1, 128, 4000, 30, True, "bf16", 0), 1)
        before = lka.workspaces.get(256, q.device)
        if later == "prefix":
            lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens)
        else:
            kk = torch.randn(2, 8, 60000, 128, device=DEV).to(q.dtype)
            lka.gqa_attn(q[:2].contiguous(), kk, kk, torch.full((2,), 60000, dtype=torch.int32, device=DEV))
        assert lka.workspaces.get(256, q.device) is not before
        assert lka.device_status() == BAD_LENGTH
        lka.clear_status()
        assert lka.device_status() == 0


def gqa_args(n, g):
    """A gqa_attn call over n keys whose splits need a workspace of about 10 n bytes."""
    q, k = randn(g, 2, 32, 1, 128), randn(g, 2, 8, n, 128)
    return q, k, k, torch.full((2,), n, dtype=torch.int32, device=DEV)


def test_a_workspace_of_a_capture_is_no_eager_call_s():
    """A capture that needs a larger workspace than its stream has takes one of its graph's memory, whose zeros come with
    the replay: an eager call on the stream must not find it."""
    g = gen(5)
    args = gqa_args(60000, g)
    case = prefix_case((80, 8, 8, 1, 64, 300, 300, True, "bf16", 0), 2)[:6]
    want, want_lse = (x.clone() for x in lka.gqa_attn_shared_prefix(*case, return_lse=True))
    junk = torch.full((64 << 20,), 17, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    del junk
    torch.cuda.empty_cache()  # what the graph allocates may hold anything
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = lka.gqa_attn(*args)
    assert (args[0].device.index, s.cuda_stream) not in lka.workspaces._ws
    with torch.cuda.stream(s):
        got, lse = lka.gqa_attn_shared_prefix(*case, return_lse=True)
        assert lka.device_status() == 0
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, lka.gqa_attn(*args))


def test_a_captured_workspace_outlives_a_larger_one():
    """A graph keeps the address of the workspace that its stream had: it stays the graph's when a later eager call on
    the stream gets a larger one, and a replay writes to nothing else."""
    g = gen(6)
    s = torch.cuda.Stream()
    args, larger = gqa_args(60000, g), gqa_args(240000, g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        want = lka.gqa_attn(*args).clone()
        size = lka.workspaces.get(256, args[0].device).numel()
    with torch.cuda.graph(graph, stream=s):
        out = lka.gqa_attn(*args)
    with torch.cuda.stream(s):
        lka.gqa_attn(*larger)
        assert lka.workspaces.get(256, args[0].device).numel() > size
        others = [torch.full((size,), 5, dtype=torch.uint8, device=DEV) for _ in range(8)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all((t == 5).all() for t in others)


def refused(n, call):
    """The call fails at the n-th of its launches behind the first kernel, on the host."""
    assert lka.library().lka_selftest_refuse_launch(n) == 0
    with pytest.raises(lka.LkaError):
        call()
    assert lka.library().lka_selftest_refuse_launch(0) == 0


@pytest.mark.parametrize("what", ["evict", "fp32 prefix"])
def test_a_call_after_a_failed_one(what):
    """A call that failed leaves no error behind for the next."""
    g = gen(7)
    if what == "evict":
        k, w = randn(g, 2, 3, 400, 64), torch.rand(2, 3, 400, generator=g, device=DEV)
        lens = torch.full((2,), 400, dtype=torch.int32, device=DEV)
        call = lambda: lka.gqa_evict(k, k, w, lens, 50)  # noqa: E731
    else:
        case = prefix_case((5, 4, 2, 1, 64, 300, 30, True, "fp32", 0), 3)[:6]
        call = lambda: lka.gqa_attn_shared_prefix(*case, return_lse=True)  # noqa: E731
    want = [x.clone() for x in call()]
    refused(1, call)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))


@pytest.mark.parametrize("B,n", [(80, 1), (80, 2), (1, 1)])
def test_a_shared_prefix_after_a_failed_one(B, n):
    """A call whose merge (or suffix kernel) was refused leaves the counter of its work items as the next call expects it.
    80 x 8 suffix items are more than the blocks that take them; one sequence of 8 x 2 heads takes its prefix in items."""
    shape = (B, 16 if B == 1 else 8, 8, 1, 64, 4000 if B == 1 else 300, 300, True, "bf16", 0)
    calls = [lambda case=prefix_case(shape, seed)[:6]: lka.gqa_attn_shared_prefix(*case, return_lse=True) for seed in (2, 3)]
    prev = lka.set_split_tokens(64 if B == 1 else 0)
    try:
        want = [x.clone() for x in calls[1]()]
        calls[0]()  # other partial results in the workspace
        refused(n, calls[0])
        assert all(torch.equal(a, b) for a, b in zip(calls[1](), want))
    finally:
        lka.set_split_tokens(prev)
    assert lka.device_status() == 0
