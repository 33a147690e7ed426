"""The cache operators around the attention calls, as a serving or training program calls them, with plain forms.

Four operators of the life of a grouped KV cache, on cases over the range each is used in:

  append   gqa_rope_append(_paged / _fp8kv): rotary positions on the new queries and keys, new rows into the cache;
           rope: the rotation of one tensor, here as the backward pass of a training step
  prefix   gqa_attn_shared_prefix(_paged): attention of a batch whose sequences share one cached prefix
  weights  gqa_key_weights(_paged): the attention weight every cached key received, summed per KV head
  evict    gqa_evict: the cache cut to a budget of keys, by that weight

`own` selects the library's calls; otherwise run() computes the definitions with elementary torch operations in fp32
(angles in fp64).  exact() computes the same in fp64.
"""
from __future__ import annotations

import math

import torch

own = False
DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    """The shapes are this repository's Llama-3.1-8B layer (32 / 8 heads of 128) unless a comment says otherwise."""
    layer = dict(h_q=32, h_kv=8, d=128)
    return [
        # one decode step of 64 sequences: 64 new tokens, where launch and latency are all there is
        dict(name="append_step_b64", op="append", B=64, s=1, lo=1024, hi=8192, cap=8192, page=0, cache="bf16",
             d_rot=128, interleaved=False, **layer),
        # two prompts of 4096 tokens into a paged cache: the largest append
        dict(name="append_prompt_paged", op="append", B=2, s=4096, lo=4096, hi=4096, cap=4096, page=64, cache="bf16",
             d_rot=128, interleaved=False, **layer),
        # a ragged chunk of odd size into an e4m3 cache, half of each head rotated, interleaved pairs
        dict(name="append_chunk_fp8", op="append", B=8, s=509, lo=600, hi=4000, cap=4096, page=0, cache="e4m3",
             d_rot=64, interleaved=True, **layer),
        # the gradient of a training step's queries, a strided view of the projection's [B, s, h, d]
        dict(name="rope_backward", op="rope", B=4, h=32, s=2048, d=128, d_rot=128, interleaved=False, dtype="bf16",
             strided=True),
        # four users of one system prompt: few rows, bound by reading the prefix once
        dict(name="prefix_b4", op="prefix", B=4, s=1, Lp=2000, lo=1, hi=128, cap=128, page=0, dtype="bf16", **layer),
        # 64 users of a long shared document
        dict(name="prefix_b64", op="prefix", B=64, s=1, Lp=8192, lo=1, hi=512, cap=512, page=0, dtype="bf16", **layer),
        # 256 samples of one long prompt, two-token steps, paged cache: bound by the tensor cores
        dict(name="prefix_b256_paged", op="prefix", B=256, s=2, Lp=16384, lo=2, hi=1024, cap=1024, page=64,
             dtype="bf16", **layer),
        # the glossary example's heads (8 / 2 of 64) in fp32, odd lengths
        dict(name="prefix_fp32", op="prefix", B=7, s=3, Lp=1001, lo=3, hi=77, cap=80, page=0, dtype="fp32", h_q=8,
             h_kv=2, d=64),
        # the decode layer's step: 64 sequences, one query each, ragged lengths
        dict(name="weights_step_b64", op="weights", B=64, s=1, lo=1024, hi=8192, cap=8192, page=0, dtype="bf16",
             **layer),
        # after a causal prompt of 4096 tokens: every query against every key
        dict(name="weights_prompt", op="weights", B=1, s=4096, lo=4096, hi=4096, cap=4096, page=0, dtype="bf16",
             **layer),
        # 16 prompts cut to a quarter and less
        dict(name="evict_b16", op="evict", B=16, lo=4096, hi=8192, cap=8192, budget=1024, sinks=4, recent=256,
             cache="bf16", h_kv=8, d=128),
        # one long sequence in an e4m3 cache: few rows to choose for, many keys to choose from
        dict(name="evict_long_fp8", op="evict", B=1, lo=65536, hi=65536, cap=65536, budget=4096, sinks=16, recent=512,
             cache="e4m3", h_kv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: batch, lengths, heads, head dim, pages and types over the ranges the listed cases stand for."""
    op = rng.choice(["append", "append", "rope", "prefix", "prefix", "weights", "weights", "evict"])
    ratio, h_kv, d = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    page = rng.choice([0, 0, 16, 64, 128])
    if op in ("append", "rope"):
        cache = rng.choice(["bf16", "bf16", "fp32", "e4m3"] if op == "append" else ["bf16", "fp32"])
        h_kv = min(h_kv, 32 // ratio)
        tokens = _log_int(rng, 1, 8192 * 256 // (d * (4 if cache == "fp32" else 2)))
        B = min(tokens, _log_int(rng, 1, 128))
        s, d_rot = max(1, tokens // B), rng.choice([d, d, d // 2, d // 4])
        if op == "rope":
            return dict(op=op, B=B, h=ratio * h_kv, s=s, d=d, d_rot=d_rot, interleaved=rng.random() < 0.5, dtype=cache,
                        strided=rng.random() < 0.5)
        hi = s + rng.randrange(0, 2048)
        return dict(op=op, B=B, h_q=ratio * h_kv, h_kv=h_kv, d=d, s=s, lo=s, hi=hi, cap=-(-hi // 128) * 128,
                    page=0 if cache == "e4m3" else page, cache=cache, d_rot=d_rot, interleaved=rng.random() < 0.5)
    if op == "prefix":
        dtype = "bf16" if rng.random() < 0.8 or d == 256 else "fp32"
        B, s = _log_int(rng, 1, 256 if dtype == "bf16" else 16), rng.choice([1, 1, 2, 4])
        Lp = _log_int(rng, 64, 16384 if dtype == "bf16" else 2048)
        heads = max(1, min(h_kv, 8192 // (B * s * ratio)))
        Lp = min(Lp, max(64, 2 ** 33 // (B * s * ratio * heads * d)))
        hi = s + rng.randrange(0, 768)
        return dict(op=op, B=B, s=s, Lp=Lp, lo=s, hi=hi, cap=-(-hi // 128) * 128, page=page, dtype=dtype,
                    h_q=ratio * heads, h_kv=heads, d=d)
    if op == "weights":
        if rng.random() < 0.3:  # after a prompt or a chunk of one
            s, h_kv, ratio = _log_int(rng, 8, 4096), min(h_kv, 4), min(ratio, 4)
            hi, B = min(6000, s + rng.randrange(0, 1024)), 1
        else:
            s, hi, B = rng.choice([1, 1, 2, 4]), _log_int(rng, 64, 8192), _log_int(rng, 1, 64)
        dtype = "bf16" if rng.random() < 0.8 or d == 256 or s > 64 else "fp32"
        B = max(1, min(B, 2 ** 30 // (hi * h_kv * d * (2 if dtype == "bf16" else 4))))
        return dict(op=op, B=B, s=s, lo=max(s, hi // 4), hi=hi, cap=-(-hi // 128) * 128, page=page, dtype=dtype,
                    h_q=ratio * h_kv, h_kv=h_kv, d=d)
    hi, cache = _log_int(rng, 512, 65536), rng.choice(["bf16", "fp32", "e4m3"])
    B = max(1, min(16, 131072 // hi))
    most = 2 ** 27 // (B * h_kv * d * {"bf16": 2, "fp32": 4, "e4m3": 1}[cache])
    budget = _log_int(rng, 64, max(64, min(hi // 2, most)))
    return dict(op=op, B=B, lo=max(1, hi // 2), hi=hi, cap=hi + rng.randrange(0, 64), budget=budget,
                sinks=rng.randrange(0, 17), recent=rng.randrange(0, budget // 2), cache=cache, h_kv=h_kv, d=d)


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rand(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _frequencies(d_rot):
    """Radians per token of every pair: base 500000, as the layer's positions are."""
    i = torch.arange(0, d_rot, 2, dtype=torch.float64, device=DEV)
    return torch.pow(torch.tensor(500000.0, dtype=torch.float64, device=DEV), -i / d_rot)


def _page_table(g, B, pages):
    return torch.randperm(B * pages, generator=g, device=DEV).to(torch.int32).view(B, pages)


def _pool(x, table, page):
    """The pages [num_pages, h, page, d] that hold the cache x [B, h, cap, d] as the table says."""
    B, h, cap, d = x.shape
    pool = torch.empty((table.numel(), h, page, d), dtype=x.dtype, device=DEV)
    pool[table.flatten().long()] = x.view(B, h, cap // page, page, d).transpose(1, 2).reshape(-1, h, page, d)
    return pool


def _lens(g, c):
    return torch.randint(c["lo"], c["hi"] + 1, (c["B"],), generator=g, device=DEV).to(torch.int32)


def prepare(case, seed):
    g, c, st = _gen(seed), case, dict(case=case)
    if c["op"] == "rope":
        dt = _TYPES[c["dtype"]]
        x = _rand(g, c["B"], c["s"], c["h"], c["d"], dtype=dt) if c["strided"] else _rand(g, c["B"], c["h"], c["s"], c["d"], dtype=dt)
        st["grad"] = x.transpose(1, 2) if c["strided"] else x
        first = torch.randint(0, 100000, (c["B"], 1), generator=g, device=DEV)
        st["positions"] = (first + torch.arange(c["s"], device=DEV)).to(torch.int32).contiguous()
        st["inv_freq"] = _frequencies(c["d_rot"])
        return st
    lens = st["lens"] = _lens(g, c)
    B, h_kv, d, cap = c["B"], c["h_kv"], c["d"], c["cap"]
    if c["op"] == "evict":
        dt = _TYPES[c["cache"]]
        for n in ("k", "v"):
            st[n] = _rand(g, B, h_kv, cap, d).mul_(4.0 if c["cache"] == "e4m3" else 1.0).to(dt)
            st[n + "_out"] = torch.zeros((B, h_kv, c["budget"], d), device=DEV).to(dt)
        # what keys receive: heavy-tailed, and whole groups of keys with exactly equal weights
        w = torch.exp(2.0 * _rand(g, B, h_kv, cap)) * 1e-3
        st["weights"] = torch.where(_rand(g, B, h_kv, cap) > 1.0, torch.full_like(w, 1e-3), w)
        st["weights"] *= torch.arange(cap, device=DEV) < lens[:, None, None]
        return st
    if c["op"] == "append":
        wide = torch.float32 if c["cache"] == "fp32" else torch.bfloat16
        # the projections' outputs, [B, s, h, d] seen as [B, h, s, d]
        st["q"] = _rand(g, B, c["s"], c["h_q"], d, dtype=wide).transpose(1, 2)
        st["k"] = _rand(g, B, c["s"], h_kv, d, dtype=wide).transpose(1, 2)
        st["v"] = _rand(g, B, c["s"], h_kv, d, dtype=wide).transpose(1, 2)
        st["inv_freq"] = _frequencies(c["d_rot"])
        st["scale"] = (torch.rand((2, h_kv), generator=g, device=DEV) * 0.02 + 0.01)
        dt = _TYPES[c["cache"]]
        for n in ("k_cache", "v_cache"):
            shape = (B * (cap // c["page"]), h_kv, c["page"], d) if c["page"] else (B, h_kv, cap, d)
            st[n] = torch.zeros(shape, device=DEV, dtype=torch.uint8 if c["cache"] == "e4m3" else dt)
            st[n] = st[n].view(dt) if c["cache"] == "e4m3" else st[n]
        if c["page"]:
            st["table"] = _page_table(g, B, cap // c["page"])
        return st
    dt = _TYPES[c["dtype"]]
    st["q"] = _rand(g, B, c["h_q"], c["s"], d, dtype=dt)
    k = _rand(g, B, h_kv, cap, d, dtype=dt)
    if c["op"] == "weights":
        # the normalisers that the attention call over the same queries and keys returned
        s = _scores(st["q"], k, lens)
        st["lse"] = torch.logsumexp(s, -1).view(B, c["h_q"], c["s"]).contiguous()
        del s
        if c["page"]:
            st["table"] = _page_table(g, B, cap // c["page"])
            k = _pool(k, st["table"], c["page"])
        st["k"] = k
        return st
    v = _rand(g, B, h_kv, cap, d, dtype=dt)
    if not c["page"]:
        st["k"], st["v"] = k, v
        st["k_prefix"] = _rand(g, h_kv, c["Lp"], d, dtype=dt)
        st["v_prefix"] = _rand(g, h_kv, c["Lp"], d, dtype=dt)
        return st
    own_pages, shared = B * (cap // c["page"]), -(-c["Lp"] // c["page"])
    perm = torch.randperm(own_pages + shared, generator=g, device=DEV).to(torch.int32)
    st["table"], st["prefix_table"] = perm[:own_pages].view(B, -1).contiguous(), perm[own_pages:].contiguous()
    st["prefix_len"] = torch.tensor([c["Lp"]], dtype=torch.int32, device=DEV)
    for n, x in (("k", k), ("v", v)):
        pool = _rand(g, own_pages + shared, h_kv, c["page"], d, dtype=dt)
        pool[st["table"].flatten().long()] = x.view(B, h_kv, -1, c["page"], d).transpose(1, 2).reshape(-1, h_kv, c["page"], d)
        st[n] = pool
    return st


# ---------------------------------------------------------------------------------------------------- plain forms
def _from_pages(pool, table):
    """Pages [n, h, page, d] and a table [B, m] -> [B, h, m * page, d]."""
    x = pool[table.long().clamp_min(0)]
    return x.transpose(1, 2).reshape(table.shape[0], pool.shape[1], -1, pool.shape[3])


def _scores(q, k, lens):
    """Scaled, causally masked scores [B, h_kv, ratio * s, cap] in fp32 (query t sees keys 0 .. len - s + t)."""
    B, h_q, s, d = q.shape
    h_kv, cap = k.shape[1], k.shape[2]
    x = torch.matmul(q.float().view(B, h_kv, -1, d) / math.sqrt(d), k.float().transpose(2, 3))
    last = lens[:, None].long() - s + torch.arange(s, device=q.device)
    seen = torch.arange(cap, device=q.device) <= last[..., None]
    return x.masked_fill(~seen.repeat(1, h_q // h_kv, 1)[:, None], -math.inf)


def _rotate(x, positions, inv_freq, interleaved, backward=False):
    """x [B, h, s, d] with its first 2 * len(inv_freq) values rotated by position * frequency, in fp32."""
    n = inv_freq.numel()
    angle = (positions.double()[..., None] * inv_freq)[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float() * (-1.0 if backward else 1.0)
    x = x.float()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1 if interleaved else -2).flatten(-2)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _to_cache(x, dtype, scale=None):
    return (x / scale[None, :, None, None]).clamp(-448.0, 448.0).to(dtype) if scale is not None else x.to(dtype)


def _plain_append(st):
    c, lens = st["case"], st["lens"].long()
    B, s, page = c["B"], c["s"], c["page"]
    pos = lens[:, None] - s + torch.arange(s, device=lens.device)
    q = _rotate(st["q"], pos, st["inv_freq"], c["interleaved"]).to(st["q"].dtype)
    k = _rotate(st["k"], pos, st["inv_freq"], c["interleaved"])
    ks, vs = (st["scale"][0], st["scale"][1]) if c["cache"] == "e4m3" else (None, None)
    k, v = _to_cache(k, st["k_cache"].dtype, ks), _to_cache(st["v"].float(), st["v_cache"].dtype, vs)
    if page:
        at, row = torch.gather(st["table"].long(), 1, pos // page), pos % page
    else:
        at, row = torch.arange(B, device=lens.device)[:, None].expand(B, s), pos
    raw = (lambda x: x.view(torch.uint8)) if c["cache"] == "e4m3" else (lambda x: x)
    raw(st["k_cache"])[at, :, row] = raw(k).transpose(1, 2)
    raw(st["v_cache"])[at, :, row] = raw(v).transpose(1, 2)
    return [q, st["k_cache"], st["v_cache"]]


def _plain_prefix(st):
    c, q = st["case"], st["q"]
    B, h_q, s, d = q.shape
    h_kv = c["h_kv"]
    if c["page"]:
        kp, vp = (_from_pages(st[n], st["prefix_table"][None])[0, :, :c["Lp"]] for n in ("k", "v"))
        k, v = _from_pages(st["k"], st["table"]), _from_pages(st["v"], st["table"])
    else:
        kp, vp, k, v = st["k_prefix"], st["v_prefix"], st["k"], st["v"]
    rows = q.float().view(B, h_kv, -1, d) / math.sqrt(d)
    shared = torch.matmul(rows.transpose(0, 1).reshape(h_kv, -1, d), kp.float().transpose(1, 2))
    single = _scores(q, k, st["lens"])
    m = torch.maximum(shared.amax(-1).view(h_kv, B, -1).transpose(0, 1), single.amax(-1))
    shared = torch.exp(shared - m.transpose(0, 1).reshape(h_kv, -1, 1))
    single = torch.exp(single - m[..., None])
    total = shared.sum(-1).view(h_kv, B, -1).transpose(0, 1) + single.sum(-1)
    out = torch.matmul(shared, vp.float()).view(h_kv, B, -1, d).transpose(0, 1) + torch.matmul(single, v.float())
    lse = (m + torch.log(total)).reshape(B, h_q, s)
    return [(out / total[..., None]).reshape(B, h_q, s, d).to(q.dtype), lse]


def _plain_weights(st):
    c = st["case"]
    k = _from_pages(st["k"], st["table"]) if c["page"] else st["k"]
    s = _scores(st["q"], k, st["lens"])
    return torch.exp(s - st["lse"].view(c["B"], c["h_kv"], -1, 1)).sum(2)


def _plain_evict(st):
    c, lens = st["case"], st["lens"].long()
    budget, cap = c["budget"], c["cap"]
    at = torch.arange(cap, device=lens.device)
    L = lens[:, None, None]
    kept = (at < c["sinks"]) | (at >= L - c["recent"])
    w = torch.where(kept & (at < L), math.inf, st["weights"]).masked_fill(at >= L, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    n = torch.clamp(L, max=budget)
    order = torch.where(torch.arange(budget, device=lens.device) < n, order, cap)
    keep = torch.sort(order, dim=-1).values
    live, idx = keep < cap, keep.clamp_max(cap - 1)
    out = []
    wide = idx[..., None].expand(-1, -1, -1, c["d"])
    raw = (lambda x: x.view(torch.uint8)) if c["cache"] == "e4m3" else (lambda x: x)
    for n_ in ("k", "v"):
        new = torch.gather(raw(st[n_]), 2, wide)
        raw(st[n_ + "_out"]).copy_(torch.where(live[..., None], new, raw(st[n_ + "_out"])))
        out.append(st[n_ + "_out"])
    weights = torch.gather(st["weights"], 2, idx) * live
    return out + [weights, n[:, 0, 0].to(torch.int32), torch.where(live, keep, -1).to(torch.int32)]


# ---------------------------------------------------------------------------------------------------- the calls
def _call(st):
    import latent_kv_attention_b200 as lka

    c = st["case"]
    if c["op"] == "rope":
        return lka.rope(st["grad"], st["positions"], st["inv_freq"], interleaved=c["interleaved"], backward=True)
    if c["op"] == "append":
        if c["cache"] == "e4m3":
            q = lka.gqa_rope_append_fp8kv(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["scale"][0],
                                          st["scale"][1], st["lens"], st["inv_freq"], interleaved=c["interleaved"])
        elif c["page"]:
            q = lka.gqa_rope_append_paged(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"],
                                          st["lens"], st["inv_freq"], interleaved=c["interleaved"])
        else:
            q = lka.gqa_rope_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["lens"],
                                    st["inv_freq"], interleaved=c["interleaved"])
        return [q, st["k_cache"], st["v_cache"]]
    if c["op"] == "prefix":
        if c["page"]:
            return list(lka.gqa_attn_shared_prefix_paged(st["q"], st["k"], st["v"], st["prefix_table"],
                                                         st["prefix_len"], st["table"], st["lens"], return_lse=True))
        return list(lka.gqa_attn_shared_prefix(st["q"], st["k_prefix"], st["v_prefix"], st["k"], st["v"], st["lens"],
                                               return_lse=True))
    if c["op"] == "weights":
        if c["page"]:
            return lka.gqa_key_weights_paged(st["q"], st["k"], st["lse"], st["table"], st["lens"])
        return lka.gqa_key_weights(st["q"], st["k"], st["lse"], st["lens"])
    return list(lka.gqa_evict(st["k"], st["v"], st["weights"], st["lens"], c["budget"], sinks=c["sinks"],
                              recent=c["recent"], k_out=st["k_out"], v_out=st["v_out"]))


def run(state):
    if own:
        return _call(state)
    c = state["case"]
    if c["op"] == "rope":
        x = state["grad"]
        return _rotate(x, state["positions"], state["inv_freq"], c["interleaved"], backward=True).to(x.dtype)
    return {"append": _plain_append, "prefix": _plain_prefix, "weights": _plain_weights, "evict": _plain_evict}[c["op"]](state)


# ---------------------------------------------------------------------------------------------------- the work
def work(case):
    """Bytes read and written once and the floating operations of one pass (lengths at the mean of their range)."""
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["h"] * c["s"]
        return {"bytes": 2 * n * c["d"] * (2 if c["dtype"] == "bf16" else 4) + 4 * c["B"] * c["s"], "flops": 3 * n * c["d_rot"]}
    B, d, L = c["B"], c["d"], (c["lo"] + c["hi"]) / 2
    if c["op"] == "append":
        e_in, e_out = (4 if c["cache"] == "fp32" else 2), {"bf16": 2, "fp32": 4, "e4m3": 1}[c["cache"]]
        n = B * c["s"] * d
        b = n * (2 * c["h_q"] * e_in + 2 * c["h_kv"] * (e_in + e_out))
        return {"bytes": b + 4 * B, "flops": 3 * B * c["s"] * (c["h_q"] + c["h_kv"]) * c["d_rot"]}
    if c["op"] == "evict":
        e = {"bf16": 2, "fp32": 4, "e4m3": 1}[c["cache"]]
        keep = min(L, c["budget"])
        return {"bytes": int(B * c["h_kv"] * (4 * L + keep * (4 * d * e + 4) + 4 * c["budget"])), "flops": int(B * c["h_kv"] * L)}
    e = 2 if c["dtype"] == "bf16" else 4
    rows = B * c["h_q"] * c["s"]
    seen = L - (c["s"] - 1) / 2
    if c["op"] == "weights":
        return {"bytes": int(B * L * c["h_kv"] * d * e + rows * (d * e + 4) + 4 * B * c["h_kv"] * c["cap"]), "flops": int(rows * seen * 2 * d)}
    kv = 2 * c["h_kv"] * d * e
    return {"bytes": int((B * L + c["Lp"]) * kv + rows * (2 * d * e + 4)), "flops": int(rows * (seen + c["Lp"]) * 4 * d)}


# ---------------------------------------------------------------------------------------------------- fp64
def _spin(x, positions, inv_freq, interleaved, sign=1.0):
    """The rotation as a product of complex numbers."""
    n = inv_freq.numel()
    x = x.double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), sign * positions.double()[:, None, :, None] * inv_freq)
    pair = x[..., :2 * n].unflatten(-1, (n, 2)) if interleaved else x[..., :2 * n].unflatten(-1, (2, n)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    y = y if interleaved else y.transpose(-1, -2)
    return torch.cat((y.flatten(-2), x[..., 2 * n:]), -1)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "evict":
        return None
    if c["op"] == "rope":
        return _spin(st["grad"], st["positions"], st["inv_freq"], c["interleaved"], -1.0)
    lens = st["lens"].tolist()
    B, s = c["B"], c["s"]
    if c["op"] == "append":
        pos = torch.stack([torch.arange(L - s, L, device=DEV) for L in lens])
        q, k, v = (f(st[n]) for n, f in (("q", lambda x: _spin(x, pos, st["inv_freq"], c["interleaved"])),
                                         ("k", lambda x: _spin(x, pos, st["inv_freq"], c["interleaved"])),
                                         ("v", lambda x: x.double())))
        if c["cache"] == "e4m3":
            k, v = (torch.clamp(x / st["scale"][i].double()[:, None, None], -448.0, 448.0) for i, x in enumerate((k, v)))
        caches = [torch.zeros(st[n].shape, dtype=torch.float64, device=DEV) for n in ("k_cache", "v_cache")]
        for b in range(B):
            for cache, x in zip(caches, (k, v)):
                if c["page"]:
                    pages = st["table"][b].long()[pos[b] // c["page"]]
                    cache[pages, :, pos[b] % c["page"]] = x[b].transpose(0, 1)
                else:
                    cache[b, :, lens[b] - s:lens[b]] = x[b]
        return [q] + caches
    ratio, d, q = c["h_q"] // c["h_kv"], c["d"], st["q"].double()
    step = torch.arange(s, device=DEV)

    def one(pool, table, n):
        return pool[table.long()].transpose(0, 1).flatten(1, 2)[:, :n].double()

    outs = []
    for b, L in enumerate(lens):
        k = one(st["k"], st["table"][b], L) if c["page"] else st["k"][b, :, :L].double()
        hidden = torch.arange(L, device=DEV) > (L - s + step)[:, None]
        x = torch.einsum("hrsd,hld->hrsl", q[b].unflatten(0, (c["h_kv"], ratio)), k) * d ** -0.5
        x = x.masked_fill(hidden, -math.inf)
        if c["op"] == "weights":
            lse = st["lse"][b].double().unflatten(0, (c["h_kv"], ratio))
            w = torch.zeros((c["h_kv"], c["cap"]), dtype=torch.float64, device=DEV)
            w[:, :L] = torch.exp(x - lse[..., None]).sum((1, 2))
            outs.append(w)
            continue
        v = one(st["v"], st["table"][b], L) if c["page"] else st["v"][b, :, :L].double()
        if c["page"] and b == 0:
            kp, vp = one(st["k"], st["prefix_table"], c["Lp"]), one(st["v"], st["prefix_table"], c["Lp"])
        elif b == 0:
            kp, vp = st["k_prefix"].double(), st["v_prefix"].double()
        y = torch.einsum("hrsd,hld->hrsl", q[b].unflatten(0, (c["h_kv"], ratio)), kp) * d ** -0.5
        x = torch.cat((y, x), -1)
        p = torch.softmax(x, -1)
        o = torch.einsum("hrsl,hld->hrsd", p, torch.cat((vp, v), 1))
        outs.append((o.flatten(0, 1), torch.logsumexp(x, -1).flatten(0, 1)))
    if c["op"] == "weights":
        return torch.stack(outs)
    return [torch.stack([o for o, _ in outs]), torch.stack([x for _, x in outs])]
