"""The cache operators at the sizes from which their kernels loop (marked gpu): several tokens per block of the rotation,
several key tiles per block of the key weights, more work items than blocks of the shared prefix, rows of weights that are
read again or shared by two blocks, offsets past 2^31 elements.  Against the definitions in fp64; tolerances as in
test_gpu_cache_ops.py."""
import math

import pytest
import torch

import latent_kv_attention_b200 as lka
from parity import assert_close, assert_lse_close
from test_gpu_cache_ops import (DEV, E4M3, _clean_status, assert_rotated, attend, check_prefix, e4m3_near, from_pool,  # noqa: F401
                                gen, ints, prefix_case, randn, spin, to_pool, want_weights)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rotation: 2 to 16 tokens per block
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,h,s,d,d_rot,inter", [(1, 2, 3001, 64, 64, False), (3, 1, 1001, 72, 48, True), (7, 1, 431, 21, 10, False),
                                                 (5, 1, 9001, 64, 32, True), (1, 1, 21312, 32, 32, False), (2, 3, 1500, 512, 512, False)])
def test_rope_of_many_tokens(B, h, s, d, d_rot, inter, dtype):
    g = gen(s)
    x = randn(g, B, s, h, d, dtype=dtype).transpose(1, 2)
    pos = torch.randint(0, 500_000, (B, s), generator=g, device=DEV, dtype=torch.int32)
    f, _ = lka.rope_inv_freq(d_rot)
    y = lka.rope(x, pos, f, interleaved=inter)
    assert_rotated(y, x, spin(x, pos, f, inter), dtype)
    back = lka.rope(x, pos, f, interleaved=inter, backward=True)
    assert_rotated(back, x, spin(x, pos, f, inter, sign=-1.0), dtype)
    assert lka.rope(x, pos, f, interleaved=inter, out=x) is x and torch.equal(x, y)


@pytest.mark.parametrize("kind,page,d,d_rot", [("bf16", 0, 64, 64), ("bf16", 16, 64, 32), ("bf16", 0, 18, 6), ("fp32", 64, 64, 64),
                                               ("e4m3", 0, 64, 64), ("e4m3", 0, 22, 22)])
@pytest.mark.parametrize("B,s", [(7, 431), (23, 1000)])
def test_append_of_many_tokens(B, s, kind, page, d, d_rot):
    h_q, h_kv, cap, inter = 2, 1, 1024, d_rot < d
    g = gen(s + d)
    wide = torch.float32 if kind == "fp32" else torch.bfloat16
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": E4M3}[kind]
    q, k, v = (randn(g, B, s, h, d, dtype=wide).transpose(1, 2) for h in (h_q, h_kv, h_kv))
    lens = torch.randint(s, cap + 1, (B,), generator=g, device=DEV).to(torch.int32)
    lens[0], lens[1], lens[2], lens[3] = cap, 0, s - 77, s  # a full cache, no tokens, padding in front
    row = lens[:, None].long() - s + torch.arange(s, device=DEV)
    f, _ = lka.rope_inv_freq(d_rot)
    caches = [randn(g, B, h_kv, cap, d, dtype=torch.float32).to(dt) for _ in range(2)]
    before = [c.clone() for c in caches]
    sc = torch.full((h_kv,), 0.01, device=DEV)
    if kind == "e4m3":
        out = lka.gqa_rope_append_fp8kv(q, k, v, *caches, sc, sc, lens, f, interleaved=inter)
    elif page:
        (kp, table), (vp, _) = to_pool(caches[0], page, gen(5)), to_pool(caches[1], page, gen(5))
        out = lka.gqa_rope_append_paged(q, k, v, kp, vp, table, lens, f, interleaved=inter)
        caches = [from_pool(p, table) for p in (kp, vp)]
    else:
        out = lka.gqa_rope_append(q, k, v, *caches, lens, f, interleaved=inter)
    live = (row >= 0)[:, None, :, None]
    assert_rotated(out, q, spin(q, row, f, inter) * live, wide)
    for i, (x, new) in enumerate(((k, spin(k, row, f, inter)), (v, v.double()))):
        want = before[i].double()
        at = torch.zeros((B, cap), dtype=torch.bool, device=DEV)
        for b in range(B):
            r = row[b][row[b] >= 0]
            at[b, r] = True
            want[b, :, r] = new[b][:, row[b] >= 0] / (0.01 if kind == "e4m3" else 1.0)
        got, touched = caches[i].double(), at[:, None, :, None].expand(want.shape)
        assert torch.equal(got[~touched], before[i].double()[~touched])
        if kind == "e4m3":
            assert e4m3_near(got[touched], want[touched], 600.0)
        elif i:
            assert torch.equal(got, want)
        else:
            tol = torch.finfo(dt).eps / 2 * want.abs() + 2.0 ** -21 * 2 * x.double().abs().max()
            assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_latent_append_of_many_tokens(kind):
    B, h_q, s, cap, r_kv, d_r = 5, 2, 700, 800, 96, 64
    g = gen(3)
    q_r, joint = randn(g, B, h_q, s, d_r), randn(g, B, s, r_kv + d_r)
    c_kv, k_r = joint[:, None, :, :r_kv], joint[:, None, :, r_kv:]
    lens = ints(800, 700, 699, 0, 750)
    row = lens[:, None].long() - s + torch.arange(s, device=DEV)
    f, _ = lka.rope_inv_freq(d_r)
    cache = randn(g, B, cap, r_kv + d_r, dtype=torch.float32).to(torch.bfloat16 if kind == "bf16" else E4M3)
    before = cache.clone()
    if kind == "bf16":
        out = lka.latent_rope_append(q_r, c_kv, k_r, cache, lens, f)
    else:
        out = lka.latent_rope_append_fp8kv(q_r, c_kv, k_r, cache, torch.tensor([0.01, 0.02], device=DEV), lens, f)
    assert_rotated(out, q_r, spin(q_r, row, f, False) * (row >= 0)[:, None, :, None], torch.bfloat16)
    k_new = spin(k_r, row, f, False)[:, 0]
    got = cache.float()
    for b in range(B):
        ok = row[b] >= 0
        r = row[b][ok]
        if kind == "bf16":
            assert torch.equal(got[b, r, :r_kv], c_kv[b, 0][ok].float())
            assert_rotated(got[b, r, r_kv:], k_r[b, 0][ok], k_new[b][ok], torch.bfloat16) if len(r) else None
        else:
            assert torch.equal(got[b, r, :r_kv], (c_kv[b, 0][ok].float() / 0.01).clamp(-448, 448).to(E4M3).float())
            assert e4m3_near(got[b, r, r_kv:], k_new[b][ok] / 0.02, 500.0)
        rest = torch.ones(cap, dtype=torch.bool, device=DEV)
        rest[r] = False
        assert torch.equal(got[b, rest], before[b].float()[rest])


# ------------------------------------------------------------------ key weights: 2 to 8 key tiles per block
@pytest.mark.parametrize("B,h_kv,ratio,s,d,cap,page", [(64, 8, 1, 1, 64, 600, 0), (64, 8, 4, 1, 128, 608, 16), (40, 8, 2, 3, 128, 1300, 0),
                                                       (80, 8, 1, 2, 256, 320, 64), (256, 1, 4, 1, 64, 5 * 128, 128)])
def test_key_weights_of_many_sequences(B, h_kv, ratio, s, d, cap, page):
    g = gen(cap + d)
    q, k = randn(g, B, ratio * h_kv, s, d), randn(g, B, h_kv, cap, d)
    lens = torch.randint(s, cap + 1, (B,), generator=g, device=DEV).to(torch.int32)
    border = torch.tensor([s, 63, 64, 65, 128, 129, 256, 257, 512, 513, cap - 1, cap], device=DEV, dtype=torch.int32)
    lens[:border.numel()] = border.clamp(s, cap)
    _, lse = lka.gqa_attn(q, k, k, lens, return_lse=True)
    for b, L in enumerate(lens.tolist()):
        k[b, :, L:] = math.nan
    ref = want_weights(q, k, lse, lens, True, d ** -0.5)
    w = lka.gqa_key_weights(q, k, lse, lens)
    assert ((w - ref).abs() <= 1e-5 * ref + 1e-30).all()
    old = torch.rand(w.shape, generator=g, device=DEV)
    assert torch.equal(lka.gqa_key_weights(q, k, lse, lens, weights=old.clone()), old + w)
    if page:
        pool, table = to_pool(torch.nan_to_num(k, 0.0), page, g)
        table = torch.where(torch.arange(table.shape[1], device=DEV) * page < lens[:, None], table, torch.full_like(table, -3))
        assert torch.equal(w, lka.gqa_key_weights_paged(q, pool, lse, table, lens))


# ------------------------------------------------------------------ shared prefix: more items than blocks
@pytest.mark.parametrize("split", [0, 64])
@pytest.mark.parametrize("case", [
    (100, 8, 8, 1, 128, 300, 200, True, "bf16", 0), (90, 16, 8, 2, 64, 129, 150, True, "bf16", 16),
    (50, 16, 4, 2, 256, 100, 140, True, "bf16", 0), (2, 32, 8, 1, 64, 8000, 700, True, "bf16", 0),
    (1, 16, 8, 3, 128, 8000, 70, True, "bf16", 64), (3, 8, 8, 1, 256, 5000, 300, False, "bf16", 0),
    (60, 32, 8, 1, 64, 700, 90, True, "fp32", 0)], ids=lambda c: f"{c[8]}B{c[0]}d{c[4]}P{c[5]}p{c[9]}")
def test_shared_prefix_of_many_items(case, split):
    B, h_q, h_kv, s, d, Lp, Lmax, causal, _, page = case
    q, kp, vp, k, v, lens, n, dt = prefix_case(case, Lp + B)
    prev = lka.set_split_tokens(split)
    try:
        for _ in range(3):  # the counter of the items goes back to 0 every time
            out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens, causal=causal, return_lse=True)
        if page:
            up = lambda x: torch.nn.functional.pad(x, (0, 0, 0, -x.shape[-2] % page))  # noqa: E731
            mp, sp, g = -(-Lp // page), -(-Lmax // page), gen(7)
            perm = torch.randperm(mp + B * sp, generator=g, device=DEV).to(torch.int32)
            ptab, tab = perm[:mp].contiguous(), perm[mp:].view(B, sp).contiguous()
            pools = []
            for x, y in ((kp, k), (vp, v)):
                pool = torch.full((mp + B * sp, h_kv, page, d), math.nan, dtype=dt, device=DEV)
                pool[ptab.long()] = up(x).view(h_kv, mp, page, d).transpose(0, 1)
                pool[tab.flatten().long()] = up(y).view(B, h_kv, sp, page, d).transpose(1, 2).reshape(-1, h_kv, page, d)
                pools.append(pool)
            o2, l2 = lka.gqa_attn_shared_prefix_paged(q, *pools, ptab, ints(Lp), tab, lens, causal=causal, return_lse=True)
            check_prefix(o2, l2, q, kp, vp, k, v, lens, n, causal, dt)
    finally:
        lka.set_split_tokens(prev)
    check_prefix(out, lse, q, kp, vp, k, v, lens, n, causal, dt)


# ------------------------------------------------------------------ eviction: long rows, by many heads
def sorted_kept(w, lens, budget, sinks, recent):
    """Positions kept per (sequence, head), ascending, -1 behind them: a stable sort by weight."""
    at, L = torch.arange(w.shape[2], device=DEV), lens[:, None, None].long()
    w = torch.where(((at < sinks) | (at >= L - recent)) & (at < L), math.inf, w.double()).masked_fill(at >= L, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.where(torch.arange(budget, device=DEV) < L, order, w.shape[2])
    kept = torch.sort(order, dim=-1).values
    return torch.where(kept < w.shape[2], kept, -1)


@pytest.mark.parametrize("B,h,cap,budget", [(20, 2, 33000, 1500), (5, 8, 9000, 4000), (20, 4, 40000, 300), (37, 1, 33000, 12000),
                                            (3, 3, 8193, 8000)])
@pytest.mark.parametrize("place", ["new", "same", "pages"])
def test_evict_long_rows_of_many_heads(B, h, cap, budget, place):
    """Rows past 8192 weights that a block reads again for every digit, and pairs and fours of blocks per row."""
    d, sinks, recent, page = 16, 5, 100, 16
    cap += -cap % page if place == "pages" else 0
    g = gen(cap + h)
    k, v = randn(g, B, h, cap, d), randn(g, B, h, cap, d)
    w = torch.rand((B, h, cap), generator=g, device=DEV)
    w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.3, (w * 64).round() / 64, w)
    lens = torch.randint(cap // 3, cap + 1, (B,), generator=g, device=DEV).to(torch.int32)
    lens[0], lens[1], lens[2] = cap, budget + 1, budget - 1
    want = sorted_kept(w, lens, budget, sinks, recent)
    if place == "pages":
        (kp, table), (vp, _) = to_pool(k, page, gen(1)), to_pool(v, page, gen(1))
        wo = w.clone()
        new, kept = lka.gqa_evict_paged(kp, vp, wo, table, lens, budget, sinks=sinks, recent=recent)
        ko, vo = from_pool(kp, table), from_pool(vp, table)
    elif place == "same":
        ko, vo, wo = k.clone(), v.clone(), w.clone()
        new, kept = lka.gqa_evict(ko, vo, wo, lens, budget, sinks=sinks, recent=recent, k_out=ko, v_out=vo, weights_out=wo)[3:]
    else:
        ko, vo, wo, new, kept = lka.gqa_evict(k, v, w, lens, budget, sinks=sinks, recent=recent)
    assert torch.equal(kept.long(), want) and torch.equal(new, lens.clamp(max=budget))
    live, at = want >= 0, want.clamp_min(0)
    for got, x in ((ko, k), (vo, v)):
        moved = torch.gather(x, 2, at[..., None].expand(-1, -1, -1, d))
        assert torch.equal(got[:, :, :budget][live], moved[live])
        if place != "new":
            keep = torch.arange(cap, device=DEV) >= new[:, None]
            assert torch.equal(got.transpose(1, 2)[keep], x.transpose(1, 2)[keep])
    assert torch.equal(wo[:, :, :budget], torch.gather(w, 2, at) * live) and not wo[:, :, budget:].any()


# ------------------------------------------------------------------ offsets past 2^31 elements
def test_caches_past_two_to_the_31_elements():
    """One loop over caches of 2.25e9 elements: append, attend over a short prefix, weigh, cut; the last sequence is long,
    the others hold one token."""
    B, h, cap, d = 8, 2, 1_100_000, 128
    assert B * h * cap * d > 2 ** 31
    g = gen(1)
    kc, vc = (torch.zeros((B, h, cap, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kc[-1].normal_(generator=g)
    vc[-1].normal_(generator=g)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    lens[-1] = cap
    q, k, v = (randn(g, B, h, 1, d) for _ in range(3))
    q = q * 3
    f, _ = lka.rope_inv_freq(d)
    qr = lka.gqa_rope_append(q, k, v, kc, vc, lens, f)
    row = lens[:, None].long() - 1
    assert_rotated(qr, q, spin(q, row, f, False), torch.bfloat16)
    assert_rotated(kc[-1, :, -1:][None], k[-1:], spin(k[-1:], row[-1:], f, False), torch.bfloat16)
    assert torch.equal(vc[-1, :, -1], v[-1, :, 0]) and torch.equal(vc[:-1, :, 0], v[:-1, :, 0])
    assert not vc[:-1, :, 1:].any()
    kp, vp = randn(g, h, 100, d), randn(g, h, 100, d)
    out, lse = lka.gqa_attn_shared_prefix(qr, kp, vp, kc, vc, lens, return_lse=True)
    ref, ref_lse = attend(qr[-1], torch.cat((kp, kc[-1]), 1), torch.cat((vp, vc[-1]), 1), 100, True)
    assert_close(out[-1], ref, torch.bfloat16, "last sequence")
    assert_lse_close(lse[-1], ref_lse, torch.bfloat16, "last lse")
    ref, ref_lse = attend(qr[0], torch.cat((kp, kc[0, :, :1]), 1), torch.cat((vp, vc[0, :, :1]), 1), 100, True)
    assert_close(out[0], ref, torch.bfloat16, "first sequence")
    del ref
    w = lka.gqa_key_weights(qr, kc, lse, lens)
    for b, L in ((0, 1), (B - 1, cap)):
        want = want_weights(qr[b:b + 1], kc[b:b + 1, :, :L], lse[b:b + 1], lens[b:b + 1], True, d ** -0.5)
        assert ((w[b:b + 1, :, :L] - want).abs() <= 1e-5 * want + 1e-30).all()
        assert not w[b, :, L:].any()
    kept_want = sorted_kept(w[-1:], lens[-1:], 1000, 1, 50)
    ko, vo, wo, new, kept = lka.gqa_evict(kc, vc, w, lens, 1000, sinks=1, recent=50)
    assert torch.equal(kept[-1:].long(), kept_want) and new.tolist() == [1] * (B - 1) + [1000]
    for got, x in ((ko, kc), (vo, vc)):
        assert torch.equal(got[-1], torch.gather(x[-1], 1, kept_want[0][..., None].expand(-1, -1, d)))
        assert torch.equal(got[:-1, :, 0], x[:-1, :, 0])


def test_pools_past_two_to_the_31_elements():
    """The same over paged pools of 2.2e9 elements, whose last pages hold the tokens."""
    B, h, page, d, pages, mp = 3, 8, 128, 128, 17_000, 20
    assert pages * h * page * d > 2 ** 31
    g = gen(2)
    kp, vp = (torch.zeros((pages, h, page, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kp[-100:].normal_(generator=g)
    vp[-100:].normal_(generator=g)
    table = (pages - 1 - torch.randperm(100, generator=g, device=DEV)[:B * mp]).to(torch.int32).view(B, mp)
    ptab = (pages - 1 - torch.randperm(100, generator=g, device=DEV)[:7]).to(torch.int32)
    lens = ints(mp * page, 1, 1000)
    q, k, v = randn(g, B, 32, 1, d), randn(g, B, h, 1, d), randn(g, B, h, 1, d)
    f, _ = lka.rope_inv_freq(d)
    qr = lka.gqa_rope_append_paged(q, k, v, kp, vp, table, lens, f)
    kc, vc = from_pool(kp, table), from_pool(vp, table)
    for b, L in enumerate(lens.tolist()):
        assert torch.equal(vc[b, :, L - 1], v[b, :, 0])
    shared = [from_pool(x, ptab[None])[0, :, :800] for x in (kp, vp)]
    out, lse = lka.gqa_attn_shared_prefix_paged(qr, kp, vp, ptab, ints(800), table, lens, return_lse=True)
    check_prefix(out, lse, qr, *shared, kc, vc, lens, 800, True, torch.bfloat16)
    w = lka.gqa_key_weights_paged(qr, kp, lse, table, lens)
    want = want_weights(qr, kc, lse, lens, True, d ** -0.5)
    assert ((w - want).abs() <= 1e-5 * want + 1e-30).all()
    rest = kp[:-100].any() | vp[:-100].any()
    want = sorted_kept(w, lens, 700, 3, 60)
    new, kept = lka.gqa_evict_paged(kp, vp, w, table, lens, 700, sinks=3, recent=60)
    assert torch.equal(kept.long(), want) and new.tolist() == [700, 1, 700] and not rest
    live, at = want >= 0, want.clamp_min(0)
    for pool, x in ((kp, kc), (vp, vc)):
        moved = torch.gather(x, 2, at[..., None].expand(-1, -1, -1, d))
        assert torch.equal(from_pool(pool, table)[:, :, :700][live], moved[live])
        assert not pool[:-100].any()


# ------------------------------------------------------------------ many query rows per head
@pytest.mark.parametrize("split", [0, 128])
@pytest.mark.parametrize("case", [
    (2, 8, 2, 70, 128, 700, 90, True, "bf16", 0), (3, 4, 4, 200, 64, 333, 260, True, "bf16", 16), (1, 8, 1, 40, 256, 200, 64, True, "bf16", 0),
    (2, 40, 2, 7, 128, 300, 50, False, "bf16", 64), (1, 4, 4, 129, 64, 1000, 129, True, "bf16", 0), (5, 64, 1, 2, 128, 450, 70, True, "bf16", 0),
    (2, 4, 2, 50, 64, 300, 70, True, "fp32", 0), (1, 8, 2, 130, 128, 150, 140, True, "fp32", 8)],
    ids=lambda c: f"{c[8]}B{c[0]}h{c[1]}kv{c[2]}s{c[3]}d{c[4]}p{c[9]}")
def test_prompts_after_a_shared_prefix(case, split):
    """More than 128 rows per sequence and KV head: row tiles of one sequence's, the last one started."""
    test_shared_prefix_of_many_items(case, split)


@pytest.mark.parametrize("B,h_q,h_kv,s,d,cap,causal,dtype", [(2, 64, 2, 30, 128, 300, True, "bf16"), (3, 32, 1, 63, 64, 130, False, "bf16"),
                                                             (1, 16, 2, 33, 256, 200, True, "bf16"), (2, 64, 1, 63, 64, 100, True, "fp32"),
                                                             (1, 24, 2, 150, 128, 190, True, "fp32"), (1, 128, 1, 64, 128, 500, True, "bf16")])
def test_key_weights_of_many_rows(B, h_q, h_kv, s, d, cap, causal, dtype):
    """Groups of more rows than are staged at a time, and heads that end inside a stage."""
    g = gen(h_q + s)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k = randn(g, B, h_q, s, d, dtype=dt), randn(g, B, h_kv, cap, d, dtype=dt)
    lens = torch.randint(s, cap + 1, (B,), generator=g, device=DEV).to(torch.int32)
    lens[0] = cap
    _, lse = lka.gqa_attn(q, k, k, lens, causal=causal, return_lse=True)
    ref = want_weights(q, k, lse, lens, causal, d ** -0.5)
    w = lka.gqa_key_weights(q, k, lse, lens, causal=causal)
    assert ((w - ref).abs() <= 1e-5 * ref + 1e-30).all()


@pytest.mark.parametrize("many", [50, 10 ** 6, 2 ** 31, 2 ** 32, 2 ** 32 + 3])
def test_evict_counts_past_the_budget(many):
    """More sinks or recent keys than the budget are the budget's worth of them, however many."""
    g = gen(12)
    k, w, lens = randn(g, 1, 2, 300, 16), torch.rand(1, 2, 300, generator=g, device=DEV), ints(300)
    for kw in (dict(sinks=many), dict(recent=many), dict(sinks=20, recent=many)):
        like = {n: min(x, 50) for n, x in kw.items()}
        want, got = lka.gqa_evict(k, k, w, lens, 50, **like), lka.gqa_evict(k, k, w, lens, 50, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    pool, table = to_pool(k[:, :, :288].contiguous(), 16, g)
    got = lka.gqa_evict_paged(pool, pool.clone(), w[:, :, :288].contiguous(), table, ints(288), 50, recent=many)[1]
    assert (got == torch.arange(238, 288, device=DEV)).all()
