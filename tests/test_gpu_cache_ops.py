"""GPU parity of the cache operators against their definitions in fp64 (marked gpu).

Tolerances: a result held in type t is off by at most half a step of it, eps(t) / 2 relative, plus the fp32 arithmetic
before.  Rotation: three fp32 roundings and the table's (cos, sin within 2^-22 of amplitude) on |x0| + |x1|: 2^-21 of it.
Attention: the library's parity tolerances.  Key weights: each term's exponent is off by at most 2^-18 (a 256-term fp32
sum of products of a few units, log2 normaliser below 32), so a sum is by 2^-18 relative, and 4e-6 < 1e-5 is asked.
Eviction copies: equality."""
import math

import pytest
import torch

import latent_kv_attention_b200 as lka
from parity import assert_close, assert_lse_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _clean_status():
    lka.clear_status()
    yield
    assert lka.device_status() == 0, lka.status_string(lka.device_status())


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def spin(x, pos, f, interleaved, amplitude=1.0, sign=1.0):
    """The rotation's definition, in fp64: x [B,h,s,d], pos [B,s]."""
    n = f.numel()
    x = x.double()
    ang = (pos.double()[..., None] * f)[:, None]
    c, s = amplitude * torch.cos(ang), sign * amplitude * torch.sin(ang)
    y = x.clone()
    i0, i1 = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def assert_rotated(got, x, ref, dtype, amplitude=1.0):
    size = amplitude * 2 * x.double().abs().amax(-1, keepdim=True)
    tol = torch.finfo(dtype).eps / 2 * ref.abs() + 2.0 ** -21 * size
    assert ((got.double() - ref).abs() <= tol).all(), (got.double() - ref).abs().max().item()


# ------------------------------------------------------------------ rope
ROPE = [  # B, h, s, d, d_rot, interleaved, strided
    (1, 1, 1, 64, 64, False, False), (2, 3, 5, 128, 128, True, True), (3, 2, 7, 128, 64, False, True),
    (2, 5, 3, 256, 64, True, False), (1, 4, 9, 20, 6, False, False), (2, 2, 3, 21, 10, True, True),
    (1, 2, 300, 24, 24, False, False), (2, 1, 2, 40, 16, False, False), (1, 3, 2, 512, 512, True, False),
    (700, 2, 1, 72, 40, False, True), (1, 2, 2, 3, 2, True, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", ROPE, ids=[f"h{c[1]}d{c[3]}r{c[4]}{'i' if c[5] else 'h'}{'s' if c[6] else ''}" for c in ROPE])
def test_rope(case, dtype):
    B, h, s, d, d_rot, inter, strided = case
    g = gen(d + s)
    x = randn(g, B, s, h, d, dtype=dtype).transpose(1, 2) if strided else randn(g, B, h, s, d, dtype=dtype)
    pos = torch.randint(-5, 2_000_000, (B, s), generator=g, device=DEV, dtype=torch.int32)
    f, amp = lka.rope_inv_freq(d_rot, base=10000.0, scaling="yarn" if d_rot > 2 else None, factor=4.0)
    y = lka.rope(x, pos, f, interleaved=inter, amplitude=amp)
    assert_rotated(y, x, spin(x, pos, f, inter, amp), dtype, amp)
    back = lka.rope(x, pos, f, interleaved=inter, amplitude=amp, backward=True)
    assert_rotated(back, x, spin(x, pos, f, inter, amp, -1.0), dtype, amp)
    # in place, through the same strides
    z = x.clone(memory_format=torch.preserve_format)
    assert lka.rope(z, pos, f, interleaved=inter, amplitude=amp, out=z) is z
    assert torch.equal(z, y)


def test_rope_backward_is_the_gradient():
    """<grad, rope(x)> as a function of x has the gradient rope(grad, backward=True): by differences (the function is
    linear, so a difference of step 1 is exact up to fp32 rounding) and as the adjoint."""
    g = gen(1)
    x, w = randn(g, 2, 3, 4, 16, dtype=torch.float32), randn(g, 2, 3, 4, 16, dtype=torch.float32)
    pos = torch.randint(0, 5000, (2, 4), generator=g, device=DEV, dtype=torch.int32)
    f, _ = lka.rope_inv_freq(12)
    grad = lka.rope(w, pos, f, amplitude=1.25, backward=True)
    base = (lka.rope(x, pos, f, amplitude=1.25).double() * w).sum()
    for at in [(0, 0, 0, 0), (1, 2, 3, 5), (0, 1, 2, 11), (1, 0, 3, 15), (0, 2, 1, 6)]:
        x1 = x.clone()
        x1[at] += 1.0
        diff = (lka.rope(x1, pos, f, amplitude=1.25).double() * w).sum() - base
        # 384 terms of at most about 10, each rounded to 2^-24 twice
        assert abs(diff.item() - grad[at].item()) <= 384 * 10 * 2.0 ** -23
    assert ((w.double() * lka.rope(x, pos, f, amplitude=1.25)).sum() - (x.double() * grad).sum()).abs() <= 384 * 10 * 2.0 ** -22


def test_rope_refusals():
    g = gen(2)
    x = randn(g, 2, 3, 4, 64)
    pos = torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    f, _ = lka.rope_inv_freq(64)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:1]), dict(inv_freq=f.float()), dict(inv_freq=f.cpu()),
                dict(x=x.transpose(2, 3)), dict(x=x[..., ::2]), dict(x=x.half()), dict(out=x[:, :, :, :32]),
                dict(out=x.flatten()[64:].new_empty(0)), dict(x=x[:, :1].expand(2, 3, 4, 64), out=x[:, :1].expand(2, 3, 4, 64))):
        kw = dict(x=x, positions=pos, inv_freq=f) | bad
        with pytest.raises(ValueError):
            lka.rope(**kw)
    with pytest.raises(lka.LkaError):
        lka.rope(x[..., :32], pos, f)  # more rotated values than the head has
    buf = randn(g, 2 * 3 * 4 * 64 + 64)
    with pytest.raises(ValueError):  # shifted by a row
        lka.rope(buf[:-64].view(2, 3, 4, 64), pos, f, out=buf[64:].view(2, 3, 4, 64))


def test_outputs_in_place_and_overlapping():
    """out and q_out may be the rotated tensor itself, through any view of the same rows, and nothing else of it."""
    g = gen(9)
    B, h, s, d = 1, 4, 3, 64
    f, _ = lka.rope_inv_freq(d)
    pos = torch.arange(s, dtype=torch.int32, device=DEV).view(1, s)
    buf = randn(g, (2 * h + 2) * s * d).bfloat16()
    q, k, v = (buf[n * s * d:].as_strided((B, n2, s, d), (99 * 64, s * d, d, 1)) for n, n2 in ((0, h), (h, 2), (h + 2, 2)))
    want = lka.rope(q, pos, f)
    copy = buf.clone()
    view = copy[:h * s * d].view(B, h, s, d)  # the same memory, another stride of the dimension of one
    assert lka.rope(copy[:h * s * d].as_strided(q.shape, q.stride()), pos, f, out=view) is view
    assert torch.equal(view, want)
    assert torch.equal(copy[h * s * d:], buf[h * s * d:])
    kc, vc = (torch.zeros((B, 2, 8, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lens = torch.full((B,), s, dtype=torch.int32, device=DEV)
    for q_out in (k.as_strided(q.shape, (h * s * d, s * d, d, 1)), v.as_strided(q.shape, (h * s * d, s * d, d, 1)),
                  buf[d:].as_strided(q.shape, (h * s * d, s * d, d, 1))):
        with pytest.raises(ValueError):
            lka.gqa_rope_append(q, k, v, kc, vc, lens, f, q_out=q_out)
    assert not kc.any() and torch.equal(want, lka.rope(q, pos, f))
    want_k = lka.rope(k, pos, f)
    q_out = buf[:h * s * d].view(B, h, s, d)
    assert lka.gqa_rope_append(q, k, v, kc, vc, lens, f, q_out=q_out) is q_out
    assert torch.equal(q_out, want) and torch.equal(kc[:, :, :s], want_k) and torch.equal(vc[:, :, :s], v)


# ------------------------------------------------------------------ append
def to_pool(x, page, g):
    """Cache [B,h,cap,d] -> pool with shuffled pages and its table."""
    B, h, cap, d = x.shape
    n = B * (cap // page)
    table = torch.randperm(n, generator=g, device=DEV).to(torch.int32).view(B, -1)
    raw = x.view(torch.uint8) if x.dtype == E4M3 else x
    pool = torch.empty((n, h, page, raw.shape[3]), dtype=raw.dtype, device=DEV)
    pool[table.flatten().long()] = raw.view(B, h, cap // page, page, -1).transpose(1, 2).reshape(n, h, page, -1)
    return pool.view(x.dtype), table


def from_pool(pool, table):
    raw = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
    x = raw[table.long()].transpose(1, 2)
    return x.reshape(table.shape[0], pool.shape[1], -1, raw.shape[3]).view(pool.dtype)


def e4m3_near(got, want, x_max):
    """e4m3 values within half a step of the fp64 quotient (2^-4 relative, subnormal step 2^-9 / 2), plus fp32's error."""
    tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 + 2.0 ** -20 * x_max
    return ((got.double() - want.clamp(-448, 448)).abs() <= tol).all()


APPEND = [  # B, h_q, h_kv, s, d, d_rot, interleaved, kind, page
    (3, 8, 2, 1, 128, 128, False, "bf16", 0), (2, 4, 4, 5, 64, 32, True, "bf16", 16), (2, 32, 8, 130, 128, 128, False, "bf16", 64),
    (2, 6, 2, 3, 64, 64, True, "fp32", 0), (1, 4, 1, 9, 64, 16, False, "fp32", 8), (3, 8, 2, 4, 128, 64, True, "e4m3", 0),
    (2, 16, 1, 1, 256, 256, False, "e4m3", 0), (2, 2, 2, 7, 20, 12, False, "bf16", 0), (2, 2, 1, 3, 18, 6, True, "e4m3", 0),
    (2, 3, 3, 2, 15, 10, False, "fp32", 8)]


@pytest.mark.parametrize("case", APPEND, ids=[f"{c[7]}s{c[3]}d{c[4]}r{c[5]}p{c[8]}" for c in APPEND])
@pytest.mark.parametrize("with_positions", [False, True])
def test_gqa_append(case, with_positions):
    B, h_q, h_kv, s, d, d_rot, inter, kind, page = case
    g = gen(10 * d + s)
    cap = 256 if page else 250
    wide = torch.float32 if kind == "fp32" else torch.bfloat16
    q, k, v = (randn(g, B, s, h, d, dtype=wide).transpose(1, 2) for h in (h_q, h_kv, h_kv))
    lens = torch.randint(s, 250, (B,), generator=g, device=DEV).to(torch.int32)
    lens[0] = 250
    if B > 1:
        lens[1] = s - 1 if s > 1 else 0  # the first token is padding (or the sequence has none)
    if B > 2:
        lens[2] = s
    row = lens[:, None].long() - s + torch.arange(s, device=DEV)
    pos = torch.randint(0, 100000, (B, s), generator=g, device=DEV, dtype=torch.int32) if with_positions else None
    at = pos if with_positions else row
    f, amp = lka.rope_inv_freq(d_rot, base=500000.0, scaling="yarn", factor=2.0)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": E4M3}[kind]
    caches = [randn(g, B, h_kv, cap, d, dtype=torch.float32).to(dt) for _ in range(2)]
    before = [c.clone() for c in caches]
    sc = [torch.rand(h_kv, generator=g, device=DEV) * 0.02 + 0.004 for _ in range(2)]
    kw = dict(positions=pos, interleaved=inter, amplitude=amp)
    if kind == "e4m3":
        out = lka.gqa_rope_append_fp8kv(q, k, v, *caches, *sc, lens, f, **kw)
    elif page:
        pools = []
        for c in caches:
            pool, table = to_pool(c, page, gen(5))
            pools.append(pool)
        out = lka.gqa_rope_append_paged(q, k, v, *pools, table, lens, f, **kw)
        caches = [from_pool(p, table) for p in pools]
    else:
        out = lka.gqa_rope_append(q, k, v, *caches, lens, f, **kw)
    live = row >= 0
    want_q = spin(q, at, f, inter, amp) * live[:, None, :, None]
    assert_rotated(out, q, want_q, wide, amp)
    new = [spin(k, at, f, inter, amp), v.double()]
    for i in range(2):
        got, old = caches[i].float(), before[i].float()
        touched = torch.zeros((B, cap), dtype=torch.bool, device=DEV)
        for b in range(B):
            r = row[b][live[b]]
            touched[b, r] = True
            w, x = new[i][b][:, live[b]], (k, v)[i][b][:, live[b]]
            if kind == "e4m3":
                quotient = w / sc[i].double()[:, None, None]
                assert e4m3_near(got[b][:, r], quotient, (x.double().abs().max() / sc[i].min() if x.numel() else 0.0))
                if i == 1:  # values are not rotated: the very bits
                    exact = (x.float() / sc[1][:, None, None]).clamp(-448, 448).to(E4M3).float()
                    assert torch.equal(got[b][:, r], exact)
            elif i == 1:
                assert torch.equal(got[b][:, r], x.float())
            elif x.numel():
                assert_rotated(got[b][:, r], x, w, dt, amp)
        keep = ~touched[:, None, :, None].expand_as(got)
        assert torch.equal(got[keep], old[keep])


@pytest.mark.parametrize("kind,page,r_kv,d_r", [("bf16", 0, 512, 64), ("bf16", 16, 512, 64), ("fp32", 0, 48, 16),
                                                ("e4m3", 0, 512, 64), ("fp32", 8, 13, 6), ("bf16", 8, 512, 62)])
def test_latent_append(kind, page, r_kv, d_r):
    B, h_q, s, cap = 3, 5, 4, 64
    g = gen(r_kv + d_r + page)
    wide = torch.float32 if kind == "fp32" else torch.bfloat16
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": E4M3}[kind]
    q_r = randn(g, B, s, h_q, d_r, dtype=wide).transpose(1, 2)
    joint = randn(g, B, s, r_kv + d_r, dtype=wide)  # one projection, split into its two parts
    c_kv, k_r = joint[:, None, :, :r_kv], joint[:, None, :, r_kv:]
    lens = ints(64, 2, 31)
    row = lens[:, None].long() - s + torch.arange(s, device=DEV)
    f, _ = lka.rope_inv_freq(d_r)
    cache = randn(g, B, cap, r_kv + d_r, dtype=torch.float32).to(dt)
    before = cache.clone()
    sc = torch.tensor([0.01, 0.02], device=DEV)
    if kind == "e4m3":
        out = lka.latent_rope_append_fp8kv(q_r, c_kv, k_r, cache, sc, lens, f)
    elif page:
        pool, table = to_pool(cache[:, None], page, g)
        flat = pool[:, 0].contiguous()
        out = lka.latent_rope_append_paged(q_r, c_kv, k_r, flat, table, lens, f)
        cache = from_pool(flat[:, None], table)[:, 0]
    else:
        out = lka.latent_rope_append(q_r, c_kv, k_r, cache, lens, f)
    live = row >= 0
    assert_rotated(out, q_r, spin(q_r, row, f, False) * live[:, None, :, None], wide)
    k_new = spin(k_r, row, f, False)[:, 0]
    got, old = cache.float(), before.float()
    for b in range(B):
        r = row[b][live[b]]
        if kind == "e4m3":
            assert torch.equal(got[b, r, :r_kv], (c_kv[b, 0][live[b]].float() / sc[0]).clamp(-448, 448).to(E4M3).float())
            assert e4m3_near(got[b, r, r_kv:], k_new[b][live[b]] / 0.02, 500.0)
        else:
            assert torch.equal(got[b, r, :r_kv], c_kv[b, 0][live[b]].float())
            assert_rotated(got[b, r, r_kv:], k_r[b, 0][live[b]], k_new[b][live[b]], dt)
        rest = torch.ones(cap, dtype=torch.bool, device=DEV)
        rest[r] = False
        assert torch.equal(got[b, rest], old[b, rest])


def test_e4m3_append_of_extreme_values_and_scales():
    """Values and scales of every size divide as the fp32 division does: infinities and overflows saturate to 448, NaN
    stays NaN, a zero scale gives what division by zero gives."""
    x = torch.tensor([0.0, -0.0, 1.0, -1.0, 3e38, -3e38, math.inf, -math.inf, math.nan, 1e-38, 7.5, 0.013, 448.0, 464.0, 1e30, -2e-3],
                     device=DEV).to(torch.bfloat16)
    v = x.view(1, 1, 1, 16).expand(1, 6, 1, 16).contiguous()
    scale = torch.tensor([1.0, 1e-38, 3e38, 0.0, 0.0123, 1e25], device=DEV)
    f, _ = lka.rope_inv_freq(2)
    caches = [torch.zeros(1, 6, 8, 16, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    lka.gqa_rope_append_fp8kv(v, v, v, *caches, scale, scale, ints(1), f)
    want = (v.float() / scale[None, :, None, None])[0, :, 0]
    got = caches[1][0, :, 0].float()
    want8 = want.clamp(-448, 448).to(E4M3).float()
    assert torch.equal(got.isnan(), want8.isnan()) and torch.equal(got.nan_to_num(1.0), want8.nan_to_num(1.0))


def test_append_reports_bad_lengths_and_pages():
    g = gen(3)
    q, k = randn(g, 3, 4, 2, 64), randn(g, 3, 2, 2, 64)
    f, _ = lka.rope_inv_freq(64)
    cache = [randn(g, 3, 2, 32, 64) for _ in range(2)]
    old = [c.clone() for c in cache]
    out = lka.gqa_rope_append(q, k, k, *cache, ints(33, -1, 32), f)
    assert lka.device_status() == 6  # LKA_ERR_BAD_LENGTH
    lka.clear_status()
    for c, o in zip(cache, old):  # neither sequence is written, the third is
        assert torch.equal(c[:2], o[:2]) and not torch.equal(c[2, :, 30:], o[2, :, 30:]) and torch.equal(c[2, :, :30], o[2, :, :30])
    assert (out[:2] == 0).all() and (out[2] != 0).any()
    pools = [randn(g, 6, 2, 16, 64) for _ in range(2)]
    old = [p.clone() for p in pools]
    table = ints(0, 6, 1, -1, 2, 3).view(3, 2)
    lka.gqa_rope_append_paged(q, k, k, *pools, table, ints(17, 18, 32), f)
    assert lka.device_status() == 7  # LKA_ERR_BAD_PAGE
    lka.clear_status()
    for p, o in zip(pools, old):
        changed = (p != o).flatten(1).any(1)
        assert changed.tolist() == [True, False, False, True, False, False]  # row 15 of page 0; rows 14, 15 of page 3


# ------------------------------------------------------------------ shared prefix
def attend(q, k, v, n_shared, causal):
    """fp64 attention of one sequence: q [h_q,s,d], k, v [h_kv,n,d]; the first n_shared keys are seen by every query."""
    h_q, s, d = q.shape
    r = h_q // k.shape[0]
    k, v = k.double().repeat_interleave(r, 0), v.double().repeat_interleave(r, 0)
    x = q.double() @ k.transpose(1, 2) / math.sqrt(d)
    if causal:
        n = k.shape[1]
        last = n - s + torch.arange(s, device=DEV)
        x = x.masked_fill(torch.arange(n, device=DEV) > last[:, None], -math.inf)
    return torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)


PREFIX = [  # B, h_q, h_kv, s, d, Lp, Lmax, causal, dtype, page
    (1, 8, 2, 1, 64, 1, 1, True, "bf16", 0), (3, 8, 2, 1, 128, 333, 40, True, "bf16", 0),
    (5, 32, 8, 2, 128, 1000, 90, True, "bf16", 16), (4, 4, 4, 3, 64, 257, 65, True, "bf16", 64),
    (3, 16, 1, 1, 256, 190, 70, True, "bf16", 0), (40, 8, 2, 1, 256, 130, 20, True, "bf16", 8),
    (37, 8, 2, 1, 128, 700, 33, True, "bf16", 0), (70, 4, 2, 2, 64, 500, 129, False, "bf16", 0),
    (2, 8, 2, 5, 128, 64, 5, True, "bf16", 128), (33, 12, 4, 3, 128, 1500, 17, True, "bf16", 0),
    (2, 40, 2, 3, 128, 300, 50, True, "bf16", 0), (130, 8, 1, 1, 128, 2100, 9, False, "bf16", 16),
    (3, 8, 2, 1, 64, 200, 30, True, "fp32", 0), (2, 6, 3, 4, 128, 77, 20, True, "fp32", 8),
    (9, 4, 1, 2, 64, 130, 40, False, "fp32", 16), (1, 4, 1, 1, 128, 500, 60, True, "fp32", 0),
    (40, 32, 8, 1, 128, 1300, 70, True, "fp32", 16), (3, 20, 2, 5, 64, 200, 90, True, "fp32", 0),
    (2, 24, 2, 3, 128, 300, 100, False, "fp32", 8), (40, 16, 1, 2, 64, 5000, 33, True, "fp32", 0),
    (3, 12, 1, 1, 64, 700, 200, True, "fp32", 0)]


def prefix_case(case, seed, plen=None):
    B, h_q, h_kv, s, d, Lp, Lmax, causal, dtype, page = case
    g = gen(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = randn(g, B, h_q, s, d, dtype=dt)
    kp, vp = randn(g, h_kv, Lp, d, dtype=dt), randn(g, h_kv, Lp, d, dtype=dt)
    k, v = randn(g, B, h_kv, Lmax, d, dtype=dt), randn(g, B, h_kv, Lmax, d, dtype=dt)
    lens = torch.randint(min(s, Lmax), Lmax + 1, (B,), generator=g, device=DEV).to(torch.int32)
    lens[0], lens[-1] = Lmax, min(s, Lmax)
    n = Lp if plen is None else plen
    # what lies behind a length may be anything
    kp[:, n:], vp[:, n:] = math.nan, math.inf
    for b, L in enumerate(lens.tolist()):
        k[b, :, L:], v[b, :, L:] = math.nan, -math.inf
    return q, kp, vp, k, v, lens, n, dt


def check_prefix(out, lse, q, kp, vp, k, v, lens, n, causal, dt):
    for b, L in enumerate(lens.tolist()):
        ref, ref_lse = attend(q[b], torch.cat((kp[:, :n], k[b, :, :L]), 1), torch.cat((vp[:, :n], v[b, :, :L]), 1), n, causal)
        assert_close(out[b], ref, dt, f"sequence {b}")
        assert_lse_close(lse[b], ref_lse, dt, f"lse {b}")


@pytest.mark.parametrize("split", [0, 64, 192])
@pytest.mark.parametrize("case", PREFIX, ids=[f"{c[8]}B{c[0]}h{c[1]}kv{c[2]}s{c[3]}d{c[4]}P{c[5]}p{c[9]}" for c in PREFIX])
def test_shared_prefix(case, split):
    B, h_q, h_kv, s, d, Lp, Lmax, causal, _, page = case
    q, kp, vp, k, v, lens, n, dt = prefix_case(case, Lp + B)
    prev = lka.set_split_tokens(split)
    try:
        out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens, causal=causal, return_lse=True)
        if page:
            up = lambda x: torch.nn.functional.pad(x.float(), (0, 0, 0, -x.shape[-2] % page)).to(dt)  # noqa: E731
            mp, sp = -(-Lp // page), -(-Lmax // page)
            pools, g = [], gen(7)
            perm = torch.randperm(mp + B * sp + 3, generator=g, device=DEV).to(torch.int32)
            ptab, tab = perm[:mp].contiguous(), perm[mp:mp + B * sp].view(B, sp).contiguous()
            for x, y in ((kp, k), (vp, v)):
                pool = torch.full((mp + B * sp + 3, h_kv, page, d), math.nan, dtype=dt, device=DEV)
                pool[ptab.long()] = up(x).view(h_kv, mp, page, d).transpose(0, 1)
                pool[tab.flatten().long()] = up(y).view(B, h_kv, sp, page, d).transpose(1, 2).reshape(-1, h_kv, page, d)
                pools.append(pool)
            used = torch.arange(sp, device=DEV) * page < lens[:, None]
            tab = torch.where(used, tab, torch.full_like(tab, -7))  # entries behind the length may hold anything
            o2, l2 = lka.gqa_attn_shared_prefix_paged(q, *pools, ptab, ints(Lp), tab, lens, causal=causal, return_lse=True)
            check_prefix(o2, l2, q, kp, vp, k, v, lens, n, causal, dt)
    finally:
        lka.set_split_tokens(prev)
    check_prefix(out, lse, q, kp, vp, k, v, lens, n, causal, dt)


@pytest.mark.parametrize("dtype,B", [("bf16", 3), ("bf16", 64), ("fp32", 3)])
@pytest.mark.parametrize("plen", [0, 1, 63, 64, 65, 400])
def test_prefix_length_on_the_device(dtype, B, plen):
    case = (B, 8, 2, 1, 128, 400, 30, True, dtype, 0)
    q, kp, vp, k, v, lens, n, dt = prefix_case(case, 50 + plen, plen)
    out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens, prefix_len=ints(plen), return_lse=True)
    check_prefix(out, lse, q, kp, vp, k, v, lens, n, True, dt)
    if plen == 0:
        none = kp[:, :0].contiguous()
        o2, l2 = lka.gqa_attn_shared_prefix(q, none, none, k, v, lens, return_lse=True)
        check_prefix(o2, l2, q, kp, vp, k, v, lens, 0, True, dt)


def test_prefix_equals_gqa_attn_over_the_joined_cache():
    """Peaked scores (queries times 8) in one part or the other, against gqa_attn on the concatenated cache."""
    g = gen(9)
    B, h_q, h_kv, d, P, L = 20, 16, 4, 128, 900, 100
    q = randn(g, B, h_q, 1, d) * 8
    kp, vp = randn(g, h_kv, P, d), randn(g, h_kv, P, d)
    k, v = randn(g, B, h_kv, L, d), randn(g, B, h_kv, L, d)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens, return_lse=True)
    kk, vv = (torch.cat((a[None].expand(B, -1, -1, -1), b), 2).contiguous() for a, b in ((kp, k), (vp, v)))
    ref, ref_lse = lka.gqa_attn(q, kk, vv, lens + P, return_lse=True)
    assert_close(out, ref.float(), torch.bfloat16, "joined")
    assert_lse_close(lse, ref_lse, torch.bfloat16, "joined lse")


@pytest.mark.parametrize("scale", [-0.09, 0.0, 0.5])
@pytest.mark.parametrize("B,d,dtype", [(3, 128, "bf16"), (40, 64, "bf16"), (40, 128, "bf16"), (12, 256, "bf16"), (3, 64, "fp32")])
def test_prefix_scales_and_growing_scores(B, d, dtype, scale):
    """Scores that grow along the keys move the reference maximum again and again; negative and zero scales turn and
    flatten them."""
    case = (B, 8, 2, 1, d, 900, 100, True, dtype, 0)
    q, kp, vp, k, v, lens, n, dt = prefix_case(case, 90 + B)
    if scale > 0:  # up to about e^30 from the first key to the last
        kp *= torch.linspace(0.2, 4.0 / d ** 0.5 * 4, 900, device=DEV).view(1, -1, 1).to(dt)
    out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, lens, scale=scale, return_lse=True)
    fix = scale * math.sqrt(d)  # attend() divides by sqrt(d)
    for b, L in enumerate(lens.tolist()):
        ref, ref_lse = attend(q[b].double() * fix, torch.cat((kp, k[b, :, :L]), 1), torch.cat((vp, v[b, :, :L]), 1), n, True)
        assert_close(out[b], ref, dt, f"sequence {b}")
        assert_lse_close(lse[b], ref_lse, dt, f"lse {b}")


def test_prefix_reports_bad_lengths_and_pages():
    case = (4, 8, 2, 1, 128, 100, 30, True, "bf16", 0)
    q, kp, vp, k, v, lens, n, dt = prefix_case(case, 60)
    kp, vp, k, v = (torch.nan_to_num(x, 0.0, 0.0, 0.0) for x in (kp, vp, k, v))
    for bad_len, bad_prefix in ((ints(31, 30, 30, 30), None), (ints(0, 30, 30, 30), None), (lens, ints(101)), (lens, ints(-1))):
        out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, k, v, bad_len, prefix_len=bad_prefix, return_lse=True)
        assert lka.device_status() == 6  # LKA_ERR_BAD_LENGTH
        lka.clear_status()
        n = 100 if bad_prefix is None else int(bad_prefix.clamp(0, 100))
        check_prefix(out, lse, q, kp, vp, k, v, bad_len.clamp(1, 30), n, True, dt)
    pool = randn(gen(61), 8, 2, 16, 128)
    lka.gqa_attn_shared_prefix_paged(q, pool, pool, ints(0, 9), ints(20), ints(1, 2, 3, 4).view(4, 1), ints(9, 9, 9, 9))
    assert lka.device_status() == 7  # LKA_ERR_BAD_PAGE
    lka.clear_status()


# ------------------------------------------------------------------ key weights
def want_weights(q, k, lse, lens, causal, scale):
    B, h_q, s, d = q.shape
    h_kv, cap = k.shape[1], k.shape[2]
    w = torch.zeros((B, h_kv, cap), dtype=torch.float64, device=DEV)
    for b, L in enumerate(lens.tolist()):
        x = (q[b].double().view(h_kv, -1, s, d) @ k[b, :, None, :L].double().transpose(2, 3)) * scale
        if causal:
            last = L - s + torch.arange(s, device=DEV)
            x = x.masked_fill(torch.arange(L, device=DEV) > last[:, None], -math.inf)
        e = torch.exp(x - lse[b].double().view(h_kv, -1, s, 1))
        w[b, :, :L] = torch.where(torch.isinf(lse[b]).view(h_kv, -1, s, 1), 0.0, e).sum((1, 2))
    return w


WEIGHTS = [  # B, h_q, h_kv, s, d, Lmax, causal, dtype, page
    (3, 8, 2, 1, 128, 200, True, "bf16", 0), (2, 32, 8, 2, 128, 130, True, "bf16", 0), (2, 4, 4, 5, 64, 96, True, "bf16", 16),
    (2, 16, 1, 1, 256, 100, True, "bf16", 0), (1, 8, 2, 70, 128, 128, True, "bf16", 64), (2, 4, 2, 200, 64, 333, True, "bf16", 0),
    (1, 2, 1, 131, 256, 192, True, "bf16", 8), (2, 4, 1, 100, 128, 90, False, "bf16", 0), (1, 8, 8, 1, 64, 1, True, "bf16", 0),
    (2, 40, 2, 3, 128, 65, True, "bf16", 0), (1, 4, 2, 300, 128, 300, True, "bf16", 0), (1, 8, 2, 257, 128, 520, True, "bf16", 0),
    (1, 4, 4, 190, 64, 512, True, "bf16", 128),
    (3, 8, 2, 1, 64, 70, True, "fp32", 0), (2, 6, 3, 4, 128, 64, True, "fp32", 8), (1, 4, 2, 90, 64, 100, True, "fp32", 0)]


@pytest.mark.parametrize("case", WEIGHTS, ids=[f"{c[7]}B{c[0]}h{c[1]}kv{c[2]}s{c[3]}d{c[4]}L{c[5]}p{c[8]}" for c in WEIGHTS])
def test_key_weights(case):
    B, h_q, h_kv, s, d, Lmax, causal, dtype, page = case
    g = gen(s + Lmax)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v = randn(g, B, h_q, s, d, dtype=dt), randn(g, B, h_kv, Lmax, d, dtype=dt), randn(g, B, h_kv, Lmax, d, dtype=dt)
    lens = torch.randint(min(s, Lmax), Lmax + 1, (B,), generator=g, device=DEV).to(torch.int32)
    lens[0] = Lmax
    _, lse = lka.gqa_attn(q, k, v, lens, causal=causal, return_lse=True)
    lse[0, 0, 0] = -math.inf  # a row that saw nothing
    for b, L in enumerate(lens.tolist()):
        k[b, :, L:] = math.nan
    ref = want_weights(q, k, lse, lens, causal, d ** -0.5)
    w = lka.gqa_key_weights(q, k, lse, lens, causal=causal)
    assert ((w - ref).abs() <= 1e-5 * ref + 1e-30).all(), ((w - ref).abs() / (ref + 1e-30)).max().item()
    assert torch.equal(w, lka.gqa_key_weights(q, k, lse, lens, causal=causal))  # the same bits
    acc = torch.rand((B, h_kv, Lmax), generator=g, device=DEV)
    old = acc.clone()
    assert lka.gqa_key_weights(q, k, lse, lens, weights=acc, causal=causal) is acc
    assert torch.equal(acc, old + w)  # one fp32 addition; nothing from the length on
    if page:
        k0 = torch.nan_to_num(k, 0.0)
        pool, table = to_pool(k0, page, g)
        used = torch.arange(table.shape[1], device=DEV) * page < lens[:, None]
        table = torch.where(used, table, torch.full_like(table, -3))
        assert torch.equal(w, lka.gqa_key_weights_paged(q, pool, lse, table, lens, causal=causal))


def test_weights_of_a_causal_prompt_sum_to_its_rows():
    """Every query row's probabilities sum to 1, so a KV head's weights sum to its group's rows."""
    g = gen(11)
    q, k, v = randn(g, 1, 8, 600, 128), randn(g, 1, 2, 600, 128), randn(g, 1, 2, 600, 128)
    lens = ints(600)
    _, lse = lka.gqa_attn(q, k, v, lens, return_lse=True)
    w = lka.gqa_key_weights(q, k, lse, lens)
    # 2400 rows; lse from bf16-probability sums is fp32-accurate: relative 1e-5 as above
    assert torch.allclose(w.double().sum(-1), torch.full((1, 2), 2400.0, dtype=torch.float64, device=DEV), rtol=1e-5)


@pytest.mark.parametrize("s,dtype", [(1, "bf16"), (130, "bf16"), (3, "fp32")])
@pytest.mark.parametrize("scale", [-0.07, 0.0])
def test_weights_of_other_scales(s, dtype, scale):
    g = gen(13)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v = (randn(g, 2, h, n, 64, dtype=dt) for h, n in ((8, s), (2, 200), (2, 200)))
    lens = ints(200, 150)
    _, lse = lka.gqa_attn(q, k, v, lens, scale=scale, return_lse=True)
    ref = want_weights(q, k, lse, lens, True, scale)
    w = lka.gqa_key_weights(q, k, lse, lens, scale=scale)
    assert ((w - ref).abs() <= 1e-5 * ref).all()


def test_weights_report_bad_lengths_and_pages():
    g = gen(12)
    q, k, lse = randn(g, 2, 4, 1, 64), randn(g, 2, 2, 32, 64), torch.zeros(2, 4, 1, device=DEV)
    lka.gqa_key_weights(q, k, lse, ints(33, 4))
    assert lka.device_status() == 6
    lka.clear_status()
    lka.gqa_key_weights_paged(q, randn(g, 3, 2, 16, 64), lse, ints(0, 3, 1, -1).view(2, 2), ints(32, 16))
    assert lka.device_status() == 7
    lka.clear_status()


# ------------------------------------------------------------------ eviction
def want_kept(w, L, budget, sinks, recent):
    """Positions of one head: a stable sort by weight (NaN least), sinks first where the budget is small."""
    if L <= budget:
        return list(range(L))
    sinks = min(sinks, budget)
    recent = min(recent, budget - sinks)
    w = w[:L].tolist()
    mid = sorted(range(sinks, L - recent), key=lambda i: (1, 0.0, i) if math.isnan(w[i]) else (0, -w[i], i))
    mid = mid[:budget - sinks - recent]
    return list(range(sinks)) + sorted(mid) + list(range(L - recent, L))


EVICT = [  # B, h_kv, d, Lmax, budget, sinks, recent, dtype
    (2, 2, 128, 300, 64, 4, 16, "bf16"), (3, 1, 64, 1000, 999, 0, 0, "bf16"), (1, 4, 256, 2100, 500, 7, 100, "fp32"),
    (2, 2, 128, 5000, 1, 0, 0, "bf16"), (2, 3, 128, 257, 100, 60, 90, "e4m3"), (1, 2, 16, 3000, 2048, 2048, 0, "e4m3"),
    (2, 1, 64, 40, 64, 4, 4, "bf16"), (1, 8, 128, 9000, 1500, 4, 700, "bf16"), (1, 1, 40, 70000, 3000, 1, 1, "bf16"),
    (2, 2, 128, 600, 200, 0, 200, "fp32")]


def evict_case(case, seed):
    B, h, d, Lmax, budget, sinks, recent, dtype = case
    g = gen(seed)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": E4M3}[dtype]
    k, v = (randn(g, B, h, Lmax, d, dtype=torch.float32).to(dt) for _ in range(2))
    w = torch.rand((B, h, Lmax), generator=g, device=DEV)
    w = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.3, (w * 4).round() / 4, w)  # many ties
    w[:, :, 1::97] = -0.0
    w[:, :, 5::89] = -1.5
    lens = torch.randint(1, Lmax + 1, (B,), generator=g, device=DEV).to(torch.int32)
    lens[0] = Lmax
    return g, k, v, w, lens


def check_evict(k, v, w, lens, ko, vo, wo, new, kept, budget, sinks, recent, rest):
    f = lambda x: x.float()  # noqa: E731
    for b, L in enumerate(lens.tolist()):
        n = min(L, budget)
        assert new[b].item() == n
        for h in range(k.shape[1]):
            idx = want_kept(w[b, h], L, budget, sinks, recent)
            assert kept[b, h].tolist() == idx + [-1] * (budget - n)
            at = torch.tensor(idx, device=DEV, dtype=torch.long)
            assert torch.equal(f(ko[b, h, :n]), f(k[b, h])[at]) and torch.equal(f(vo[b, h, :n]), f(v[b, h])[at])
            assert torch.equal(wo[b, h, :n].nan_to_num(7.0), w[b, h][at].nan_to_num(7.0)) and (wo[b, h, n:] == 0).all()
            assert torch.equal(f(ko[b, h, n:]), f(rest[0][b, h, n:])) and torch.equal(f(vo[b, h, n:]), f(rest[1][b, h, n:]))


@pytest.mark.parametrize("case", EVICT, ids=[f"{c[7]}h{c[1]}d{c[2]}L{c[3]}n{c[4]}" for c in EVICT])
def test_evict(case):
    B, h, d, Lmax, budget, sinks, recent, dtype = case
    g, k, v, w, lens = evict_case(case, Lmax)
    # new buffers, with rows to spare whose contents stay
    Lout = budget + 5
    rest = [randn(g, B, h, Lout, d, dtype=torch.float32).to(k.dtype) for _ in range(2)]
    ko, vo = rest[0].clone(), rest[1].clone()
    out = lka.gqa_evict(k, v, w, lens, budget, sinks=sinks, recent=recent, k_out=ko, v_out=vo)
    assert out[0] is ko and out[1] is vo
    check_evict(k, v, w, lens, *out, budget, sinks, recent, rest)
    # allocated by the call
    out = lka.gqa_evict(k, v, w, lens, budget, sinks=sinks, recent=recent)
    check_evict(k, v, w, lens, *out, budget, sinks, recent, [torch.zeros(B, h, budget, d, device=DEV)] * 2)
    if budget <= Lmax:  # in place
        k1, v1, w1 = k.clone(), v.clone(), w.clone()
        out = lka.gqa_evict(k1, v1, w1, lens, budget, sinks=sinks, recent=recent, k_out=k1, v_out=v1, weights_out=w1)
        check_evict(k, v, w, lens, *out, budget, sinks, recent, (k1, v1))
        for b, L in enumerate(lens.tolist()):  # rows behind the kept ones keep their contents
            n = min(L, budget)
            assert torch.equal(k1[b, :, n:].float(), k[b, :, n:].float()) and torch.equal(v1[b, :, n:].float(), v[b, :, n:].float())


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("e4m3", 64), ("fp32", 8)])
def test_evict_paged(dtype, page):
    B, h, d, cap, budget, sinks, recent = 2, 3, 64, 1024, 200, 3, 50
    g, k, v, w, lens = evict_case((B, h, d, cap, budget, sinks, recent, dtype), page)
    lens[1] = 700
    (kp, table), (vp, _) = to_pool(k, page, gen(1)), to_pool(v, page, gen(1))
    w1 = w.clone()
    new, kept = lka.gqa_evict_paged(kp, vp, w1, table, lens, budget, sinks=sinks, recent=recent)
    k1, v1 = from_pool(kp, table), from_pool(vp, table)
    check_evict(k, v, w, lens, k1, v1, w1, new, kept, budget, sinks, recent, (k, v))


def test_evict_nan_infinite_and_equal_weights():
    w = torch.tensor([[[math.nan, 1.0, math.inf, -math.inf, 1.0, 0.0, -0.0, 1.0, math.nan, 2.0]]], device=DEV)
    k = torch.arange(10, device=DEV, dtype=torch.float32).view(1, 1, 10, 1).expand(1, 1, 10, 4).contiguous()
    for budget, want in ((1, [2]), (2, [2, 9]), (3, [1, 2, 9]), (4, [1, 2, 4, 9]), (5, [1, 2, 4, 7, 9]), (6, [1, 2, 4, 5, 7, 9]),
                         (7, [1, 2, 4, 5, 6, 7, 9]), (8, [1, 2, 3, 4, 5, 6, 7, 9]), (9, [0, 1, 2, 3, 4, 5, 6, 7, 9])):
        ko, _, _, new, kept = lka.gqa_evict(k, k, w, ints(10), budget)
        assert kept[0, 0].tolist() == want and new.item() == budget and ko[0, 0, :, 0].tolist() == want
    same = torch.ones_like(w)
    assert lka.gqa_evict(k, k, same, ints(10), 4, sinks=1, recent=1)[4][0, 0].tolist() == [0, 1, 2, 9]


@pytest.mark.parametrize("L", [300, 20000, 70000])
@pytest.mark.parametrize("kind", ["binades", "digits", "last"])
def test_evict_thresholds_between_digits(L, kind):
    """Weights that agree in their leading bits, cut at the border of a group of equal ones and one key beside it."""
    i = torch.arange(L, device=DEV)
    bits = {"binades": lambda: (120 + i % 8) << 23, "digits": lambda: (0x3f800000 + (i % 16 << 10)),
            "last": lambda: 0x3f800000 + i * 7 % 5}[kind]().to(torch.int32)
    w = bits.view(torch.float32).view(1, 1, L).contiguous()
    k = torch.zeros((1, 1, L, 16), dtype=torch.bfloat16, device=DEV)
    order = torch.argsort(w[0, 0], descending=True, stable=True)
    group = int((w == w.max()).sum())
    for budget in (1, group - 1, group, group + 1, 3 * group, 3 * group + 1, L - 1):
        kept = lka.gqa_evict(k, k, w, ints(L), budget)[4]
        assert torch.equal(kept[0, 0].long(), order[:budget].sort().values), budget


def test_evict_empty_and_bad_lengths():
    g, k, v, w, _ = evict_case((3, 2, 64, 50, 20, 1, 1, "bf16"), 4)
    ko, vo, wo, new, kept = lka.gqa_evict(k, v, w, ints(0, 1, 50), 20)
    assert new.tolist() == [0, 1, 20] and (kept[0] == -1).all() and (wo[0] == 0).all() and (ko[0] == 0).all()
    new = lka.gqa_evict(k, v, w, ints(51, -2, 50), 20)[3]
    assert lka.device_status() == 6 and new.tolist() == [20, 0, 20]
    lka.clear_status()
    kp = randn(g, 4, 2, 16, 64)
    old = kp.clone()
    lka.gqa_evict_paged(kp, kp.clone(), torch.rand(1, 2, 48, device=DEV), ints(0, 9, 2).view(1, 3), ints(48), 30, recent=14)
    assert lka.device_status() == 7  # the destination rows 16 .. 29 lie in a page outside the pool: not written
    assert torch.equal(kp[1], old[1]) and torch.equal(kp[2:], old[2:])
    lka.clear_status()


# ------------------------------------------------------------------ together, streams, graphs
def test_generation_with_a_budget():
    """A decode loop as a server runs it: append, attend, add up the weights, cut the cache when it is full, go on with
    the true positions; against the same loop in fp64 on the kept tokens."""
    g = gen(20)
    B, h_q, h_kv, d, cap, budget, sinks, recent = 2, 8, 2, 64, 48, 32, 2, 8
    f, _ = lka.rope_inv_freq(d, base=500000.0, scaling="bands", factor=8.0)
    kc, vc = torch.zeros(B, h_kv, cap, d, device=DEV), torch.zeros(B, h_kv, cap, d, device=DEV)
    weights = torch.zeros(B, h_kv, cap, device=DEV)
    lens, seen = ints(0, 0), 0
    hist = [[([], [], []) for _ in range(h_kv)] for _ in range(B)]  # keys, values, weights kept so far, fp64
    cuts = 0
    for step in range(40):
        s = 20 if step == 0 else 1
        q, k, v = (randn(g, B, s, h, d, dtype=torch.float32).transpose(1, 2) for h in (h_q, h_kv, h_kv))
        pos = (seen + torch.arange(s, device=DEV, dtype=torch.int32)).expand(B, s).contiguous()
        seen += s
        lens = lens + s
        qr = lka.gqa_rope_append(q, k, v, kc, vc, lens, f, positions=pos)
        out, lse = lka.gqa_attn(qr, kc, vc, lens, return_lse=True)
        lka.gqa_key_weights(qr, kc, lse, lens, weights=weights)
        q64, k64 = spin(q, pos, f, False), spin(k, pos, f, False)
        for b in range(B):
            for h in range(h_kv):
                K, V, W = hist[b][h]
                for t in range(s):
                    K.append(k64[b, h, t])
                    V.append(v[b, h, t].double())
                    W.append(0.0)
                r = h_q // h_kv
                ref, _ = attend(q64[b, h * r:(h + 1) * r], torch.stack(K)[None], torch.stack(V)[None], 0, True)
                assert (out[b, h * r:(h + 1) * r] - ref).abs().max() <= 1e-5
                x = q64[b, h * r:(h + 1) * r] @ torch.stack(K).T / math.sqrt(d)
                n = len(K)
                x = x.masked_fill(torch.arange(n, device=DEV) > (n - s + torch.arange(s, device=DEV))[:, None], -math.inf)
                add = torch.softmax(x, -1).sum((0, 1)).tolist()
                for j in range(n):
                    W[j] += add[j]
        if int(lens[0]) == cap:
            cuts += 1
            got_w = weights.clone()
            _, _, _, lens, kept = lka.gqa_evict(kc, vc, weights, lens, budget, sinks=sinks, recent=recent, k_out=kc, v_out=vc,
                                                weights_out=weights)
            for b in range(B):
                for h in range(h_kv):
                    K, V, W = hist[b][h]
                    assert (got_w[b, h] - torch.tensor(W, device=DEV)).abs().max() <= 1e-4
                    idx = kept[b, h].tolist()
                    hist[b][h] = tuple([X[i] for i in idx] for X in (K, V, W))
    assert cuts >= 1


def test_prefix_after_append_with_graphs_on_two_streams():
    """Two captured graphs of append + shared-prefix attention replay at the same time on two streams, and give what
    the eager calls give; flags raised inside a graph reach device_status."""
    f, _ = lka.rope_inv_freq(128)
    g = gen(21)
    kp, vp = randn(g, 8, 3000, 128), randn(g, 8, 3000, 128)
    sets = []
    for i in range(2):
        st = dict(q=randn(g, 24, 32, 1, 128), k=randn(g, 24, 8, 1, 128), v=randn(g, 24, 8, 1, 128),
                  kc=randn(g, 24, 8, 200, 128), vc=randn(g, 24, 8, 200, 128),
                  lens=torch.randint(1, 201, (24,), generator=g, device=DEV).to(torch.int32))
        sets.append(st)

    def call(st):
        q = lka.gqa_rope_append(st["q"], st["k"], st["v"], st["kc"], st["vc"], st["lens"], f)
        out, lse = lka.gqa_attn_shared_prefix(q, kp, vp, st["kc"], st["vc"], st["lens"], return_lse=True)
        w = lka.gqa_key_weights(q, st["kc"], lse, st["lens"])
        return (out, lse, w) + lka.gqa_evict(st["kc"], st["vc"], w, st["lens"], 50, recent=5)
    want = [[x.clone() for x in call(st)] for st in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for st in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call(st))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x, y in zip(o, w):
            assert torch.equal(x, y)
    sets[1]["lens"][3] = 999
    graphs[1].replay()
    assert lka.device_status() == 6
    lka.clear_status()


def test_calls_on_another_stream_do_not_share_scratch():
    case = (64, 16, 4, 1, 128, 1500, 60, True, "bf16", 0)
    sets = [prefix_case(case, 70 + i) for i in range(2)]
    want = [lka.gqa_attn_shared_prefix(*s[:6]).clone() for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        outs = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                outs.append(lka.gqa_attn_shared_prefix(*s[:6]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_empty_batch():
    f, _ = lka.rope_inv_freq(64)
    z = torch.empty(0, 4, 1, 64, dtype=torch.bfloat16, device=DEV)
    c = torch.empty(0, 2, 16, 64, dtype=torch.bfloat16, device=DEV)
    n = torch.empty(0, dtype=torch.int32, device=DEV)
    assert lka.rope(z, torch.empty(0, 1, dtype=torch.int32, device=DEV), f).shape == z.shape
    assert lka.gqa_rope_append(z, z[:, :2], z[:, :2], c, c, n, f).shape == z.shape
    p = torch.zeros(2, 5, 64, dtype=torch.bfloat16, device=DEV)
    assert lka.gqa_attn_shared_prefix(z, p, p, c, c, n).shape == z.shape
    assert lka.gqa_key_weights(z, c, torch.empty(0, 4, 1, device=DEV), n).shape == (0, 2, 16)
    assert lka.gqa_evict(c, c, torch.empty(0, 2, 16, device=DEV), n, 4)[0].shape == (0, 2, 4, 64)
