"""Cache operators called together (marked gpu): from threads and streams at once, over outputs in their own operands, and
a captured loop replayed as a server does."""
import threading

import pytest
import torch

import latent_kv_attention_b200 as lka
from test_gpu_cache_ops import DEV, _clean_status, check_prefix, gen, ints, prefix_case, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [(3, 8, 2, 1, 128, 500, 30, True, "bf16", 0), (40, 8, 2, 1, 128, 500, 30, True, "bf16", 0),
                                  (40, 8, 2, 1, 256, 500, 30, True, "bf16", 0), (40, 8, 2, 1, 64, 500, 30, True, "fp32", 0)])
def test_shared_prefix_into_its_queries(case):
    """The output may be the queries: the merge, which alone writes it, is the last kernel of the call."""
    q, kp, vp, k, v, lens, n, dt = prefix_case(case, 4)
    want, want_lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens, return_lse=True)
    x = q.clone()
    out, lse = lka.gqa_attn_shared_prefix(x, kp, vp, k, v, lens, out=x, return_lse=True)
    assert out is x and torch.equal(x, want) and torch.equal(lse, want_lse)


def step(st, f, kp, vp):
    q = lka.gqa_rope_append(st["q"], st["k"], st["v"], st["kc"], st["vc"], st["lens"], f)
    out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, st["kc"], st["vc"], st["lens"], return_lse=True)
    w = lka.gqa_key_weights(q, st["kc"], lse, st["lens"])
    return (q, out, lse, w) + lka.gqa_evict(st["kc"], st["vc"], w, st["lens"], 40, sinks=2, recent=9)


def states(n, B=24):
    g = gen(31)
    f, _ = lka.rope_inv_freq(128)
    kp, vp = randn(g, 8, 2000, 128), randn(g, 8, 2000, 128)
    sets = [dict(q=randn(g, B, 32, 1, 128), k=randn(g, B, 8, 1, 128), v=randn(g, B, 8, 1, 128), kc=randn(g, B, 8, 150, 128),
                 vc=randn(g, B, 8, 150, 128), lens=torch.randint(1, 151, (B,), generator=g, device=DEV).to(torch.int32))
            for _ in range(n)]
    return sets, f, kp, vp


def test_threads_on_their_own_streams():
    sets, f, kp, vp = states(4)
    want = [[x.clone() for x in step(s, f, kp, vp)] for s in sets]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = step(sets[i], f, kp, vp)
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    failed.append(f"thread {i}: other results")
        except Exception as e:  # noqa: BLE001 -- a thread's exception would be lost
            failed.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_a_captured_step_follows_its_operands():
    """A captured decode step, replayed as the lengths and the tokens in its buffers change, between eager calls on the
    same stream."""
    (st,), f, kp, vp = states(1)
    st["lens"].clamp_(max=100)
    eager = {n: x.clone() for n, x in st.items()}
    step(st, f, kp, vp)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = step(st, f, kp, vp)
    for n, x in eager.items():
        st[n].copy_(x)
    g = gen(8)
    with torch.cuda.stream(stream):
        stream.wait_stream(torch.cuda.default_stream())
        for i in range(30):
            for n in ("q", "k", "v"):
                new = randn(g, *st[n].shape)
                st[n].copy_(new)
                eager[n].copy_(new)
            st["lens"] += 1
            eager["lens"] += 1
            graph.replay()
            want = step(eager, f, kp, vp)
            assert all(torch.equal(a, b) for a, b in zip(out, want)), i
            assert torch.equal(st["kc"], eager["kc"]) and torch.equal(st["vc"], eager["vc"])
    torch.cuda.synchronize()
    assert lka.device_status() == 0
