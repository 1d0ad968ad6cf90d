"""Measured cases of what stands around the exact-attention and incremental layers: the norms of
queries and keys with the position rotation, forward and backward, and attention over the paged
8-bit cache for requests that share a prefix (its plan and the attention).

Between a projection and a layer, ``qk_norm_rope`` normalises every head's queries and keys (root
mean square with weights, or to unit length as the incremental layer wants them) and rotates
them by their tokens' positions; ``qk_norm_rope_bwd`` is its gradient.  ``kv8_shared_plan`` finds, once a
step, the pages that the requests of a group have in common, and ``kv8_attn_shared`` attends to
these once for all of the group and to the rest of each request alone: ``kv8_attn``'s result.

``own`` selects the library's calls; otherwise every operator runs in its plain form:
elementary torch operations in 32 bits (angles in 64).  ``exact`` restates the definitions in 64 bits.

A case is a dict of plain values.  Lengths are drawn from the case itself (``mix`` seeds them),
contents from the seed that ``prepare`` gets.
"""
from __future__ import annotations

import math
import random

import torch

own = False

CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 64 requests with contexts of up to a million tokens: latency
        dict(name="norm decode 64", op="norm", T=64, seqs=64, pos_max=1048576, Hq=32, Hk=8, D=128, norm="rms",
             rot=128, pairs="half", dtype="bf16", mix=1),
        # four prompts of the prefill length, grouped heads
        dict(name="norm prefill 4 x 4096", op="norm", T=16384, seqs=4, pos_max=4096, Hq=32, Hk=8, D=128,
             norm="rms", rot=128, pairs="half", dtype="bf16", mix=2),
        # unit queries and keys of an incremental layer, the long prefill
        dict(name="norm delta 65536", op="norm", T=65536, seqs=1, pos_max=0, Hq=32, Hk=32, D=128, norm="l2",
             rot=0, pairs="half", dtype="bf16", mix=3),
        # a small packed training batch in fp32: narrow heads, half of them rotated, adjacent pairs
        dict(name="grad ragged f32 d64", op="grad", T=777, seqs=9, pos_max=70000, Hq=6, Hk=2, D=64, norm="rms",
             rot=32, pairs="adjacent", dtype="f32", mix=4),
        # the training step of an exact layer, four sequences of the prefill length
        dict(name="grad 4 x 4096", op="grad", T=16384, seqs=4, pos_max=4096, Hq=32, Hk=8, D=128, norm="rms",
             rot=128, pairs="half", dtype="bf16", mix=5),
        # the training step of an incremental layer with 16 heads
        dict(name="grad delta 16384", op="grad", T=16384, seqs=4, pos_max=0, Hq=16, Hk=16, D=128, norm="l2",
             rot=0, pairs="half", dtype="bf16", mix=6),
        # a busy server: eight system prompts, 256 requests
        dict(name="plan 256 in 8", op="plan", S=256, groups=8, prefix=8192, own_min=1, own_max=4096, q="one",
             q_max=1, page=64, mix=7),
        # one very long common document, small pages: the tables are the work
        dict(name="plan 1000 on 64k", op="plan", S=1000, groups=1, prefix=65536, own_min=1, own_max=2000,
             q="one", q_max=1, page=16, mix=8),
        # a few requests on a short system prompt: latency
        dict(name="shared decode 8 on 2k", op="shared", S=8, groups=1, prefix=2048, own_min=10, own_max=400,
             q="one", q_max=1, Hq=32, Hkv=8, D=128, page=64, dtype="bf16", kv="e4m3", mix=9),
        # a busy server: 256 requests, four documents of up to 32 k tokens
        dict(name="shared decode 256 on 4 x 32k", op="shared", S=256, groups=4, prefix=32768, own_min=20,
             own_max=2000, q="one", q_max=1, Hq=32, Hkv=4, D=128, page=64, dtype="bf16", kv="int8", mix=10),
        # drafted tokens in fp32, narrow heads, three heads to a cached head, pages gone, requests that idle
        dict(name="shared draft f32 d64", op="shared", S=21, groups=3, prefix=3000, own_min=5, own_max=300,
             q="ragged", q_max=5, Hq=6, Hkv=2, D=64, page=16, dtype="f32", kv="e4m3", gone=0.03, mix=11),
        # two dozen questions of up to 200 tokens about one document
        dict(name="shared questions 24 on 20k", op="shared", S=24, groups=1, prefix=20000, own_min=200,
             own_max=500, q="ragged", q_max=200, Hq=32, Hkv=8, D=128, page=32, dtype="bf16", kv="e4m3", mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "grad", "plan", "shared", "shared", "shared"])
    mix = rng.randrange(1 << 30)
    if op in ("norm", "grad"):
        D = rng.choice([64, 128, 128])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hk * rng.choice([1, 1, 2, 4, 7])
        T = _log(rng, 1, min(65536, (1 << 28) // ((Hq + Hk) * D)))
        norm = rng.choice(["rms", "rms", "l2", "none"])
        rot = 0 if norm == "l2" else rng.choice([D, D, D // 2])
        return dict(op=op, T=T, seqs=rng.randint(1, min(T, 32)), pos_max=_log(rng, 100, 1048576), Hq=Hq, Hk=Hk,
                    D=D, norm=norm, rot=rot, pairs=rng.choice(["half", "adjacent"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), mix=mix)
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        S = _log(rng, 4, 1500)
        return dict(op=op, S=S, groups=rng.randint(1, max(1, S // 4)), prefix=_log(rng, 16 * page, 65536),
                    own_min=rng.choice([1, 1, 40]), own_max=_log(rng, 50, 8192),
                    q=rng.choice(["one", "ragged"]), q_max=rng.randint(1, 30), page=page, mix=mix)
    Hkv, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128])
    dtype, kv = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["e4m3", "int8"])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8])
    mode = rng.choice(["decode", "decode", "draft", "questions"])
    if mode == "decode":
        S, q, q_max, own_max = _log(rng, 2, 256), "one", 1, _log(rng, 10, 4096)
    elif mode == "draft":
        S, q, q_max, own_max = _log(rng, 2, 64), rng.choice(["all", "ragged"]), rng.randint(2, 8), _log(rng, 20, 4096)
    else:
        S, q, q_max = _log(rng, 2, 24), rng.choice(["all", "ragged"]), _log(rng, 9, 300)
        own_max = q_max + _log(rng, 1, 1000)
    prefix = _log(rng, 100, 32768)
    if dtype == "f32":              # the accuracy path: moderate sizes
        q_max, prefix = min(q_max, 64), min(prefix, 8192)
    while S * Hq * q_max * (prefix + own_max) > 2_000_000_000 or S * Hkv * D * own_max > 400_000_000:
        S, prefix, own_max = max(2, S // 2), max(100, prefix // 2), max(q_max, own_max // 2)
    return dict(op=op, S=S, groups=rng.randint(1, max(1, S // 3)), prefix=prefix, own_min=q_max,
                own_max=max(q_max, own_max), q=q, q_max=q_max, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype,
                kv=kv, gone=rng.choice([0.0, 0.0, 0.02]), mix=mix)


# ------------------------------------------------------------------ lengths of a case
def _ceil(a, b):
    return -(-a // b)


def _runs(c):
    """(first position, tokens) of every packed sequence of a norm case."""
    rng = random.Random(c["mix"])
    n = c["seqs"]
    cuts = sorted(rng.sample(range(1, c["T"]), n - 1)) if n > 1 else []
    size = [b - a for a, b in zip([0] + cuts, cuts + [c["T"]])]
    return [(rng.randint(0, max(0, c["pos_max"] - m)), m) for m in size]


def _batch(c):
    """Lengths of a shared case: (prefix tokens, requests) of every group, then own tokens (the new
    ones among them) and new tokens of every request.  Every fifth group has one request or no prefix."""
    rng = random.Random(c["mix"])
    S, n = c["S"], c["groups"]
    cuts = sorted(rng.sample(range(1, S), n - 1)) if n > 1 else []
    size = [b - a for a, b in zip([0] + cuts, cuts + [S])]
    groups = []
    for i, m in enumerate(size):
        p = c["prefix"] if n == 1 else rng.randint(c["prefix"] // 2, c["prefix"])
        groups.append((0 if i % 5 == 4 else max(1, p // c["page"]) * c["page"], m))
    if c["q"] == "ragged":
        q = [rng.randint(1, c["q_max"]) if rng.random() > 0.08 else 0 for _ in range(S)]
        q = q if any(q) else [1] + q[1:]
    else:
        q = [c["q_max"] if c["q"] == "all" else 1] * S
    mine = [max(k, rng.randint(c["own_min"], max(c["own_min"], c["own_max"]))) for k in q]
    return groups, mine, q


def _elem(c):
    return 2 if c["dtype"] == "bf16" else 4


def work(case):
    c = case
    if c["op"] in ("norm", "grad"):
        n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
        small = (4 * c["T"] + 4 * c["rot"] if c["rot"] else 0) + (8 * c["D"] if c["norm"] == "rms" else 0)
        if c["op"] == "norm":
            return {"bytes": 2 * n * _elem(c) + small, "flops": 7 * n}
        return {"bytes": 3 * n * _elem(c) + small + (8 * c["D"] if c["norm"] == "rms" else 0), "flops": 14 * n}
    groups, mine, q = _batch(c)
    at, tokens, pages, entries, pairs = 0, 0, 0, 0, 0
    for p, m in groups:
        rows = [i for i in range(at, at + m) if q[i]]
        at += m
        tokens += (p if rows else 0) + sum(mine[i] for i in rows)
        pages += (p // c["page"] if rows else 0) + sum(_ceil(mine[i], c["page"]) for i in rows)
        if len(rows) > 1:
            entries += len(rows) * (p // c["page"] * 3 // 4 + 1)     # the least, see prepare
        pairs += sum(q[i] * p + q[i] * (mine[i] - q[i]) + q[i] * (q[i] + 1) // 2 for i in rows)
    if c["op"] == "plan":
        return {"bytes": 4 * entries + 12 * c["S"] + 8 * len(groups), "flops": 0}
    e, rows = _elem(c), sum(q) * c["Hq"]
    by = tokens * c["Hkv"] * c["D"] * 2 + pages * (4 + 8 * c["Hkv"]) + rows * (2 * c["D"] * e + 4)
    return {"bytes": by, "flops": 4 * pairs * c["Hq"] * c["D"]}


# ------------------------------------------------------------------ inputs
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + k) % (1 << 62))
    return g


def _randn(shape, seed, k):
    return torch.randn(shape, generator=_gen(seed, k), device="cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _activations(T, heads, D, seed, k):
    """A projection's output: channels and tokens of uneven size."""
    x = _randn((T, heads, D), seed, k)
    x *= torch.exp(0.5 * _randn((1, heads, D), seed, k + 1))
    return x.mul_(torch.exp(0.4 * _randn((T, 1, 1), seed, k + 2)))


def _cache(pages, c, seed, k):
    """Codes and scales as earlier appends left them: the scale a power of two that holds the page."""
    H, P, D, kv = c["Hkv"], c["page"], c["D"], c["kv"]
    x = _randn((pages, H, P, D), seed, k)
    x *= torch.exp(0.5 * _randn((1, H, 1, D), seed, k + 1))
    s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / QMAX[kv])).clamp(-40, 40))
    x = (x / s[:, :, None, None]).clamp(-QMAX[kv], QMAX[kv])
    return (x.to(CODE[kv]) if kv == "e4m3" else torch.round(x).to(torch.int8)), s


def prepare(case, seed):
    c = case
    if c["op"] in ("norm", "grad"):
        T, Hq, Hk, D, dt = c["T"], c["Hq"], c["Hk"], c["D"], DTYPE[c["dtype"]]
        # queries, keys and values side by side, as one product writes them
        q, k, _ = _activations(T, Hq + 2 * Hk, D, seed, 1).to(dt).split([Hq, Hk, Hk], 1)
        s = dict(c=c, q=q, k=k, wq=None, wk=None, pos=None, freq=None, eps=1e-6)
        if c["norm"] == "rms":
            s["wq"], s["wk"] = (1 + 0.2 * _randn((D,), seed, i) for i in (5, 6))
        if c["rot"]:
            s["pos"] = _i32([p + i for p, n in _runs(c) for i in range(n)])
            i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
            s["freq"] = 10000.0 ** (-2 * i / c["rot"])
        if c["op"] == "grad":
            s["gq"], s["gk"] = (_randn((T, h, D), seed, i).to(dt) for h, i in ((Hq, 7), (Hk, 8)))
        return s
    groups, mine, q = _batch(c)
    P, S = c["page"], c["S"]
    first = [p for p, m in groups for _ in range(m)]
    kv = [a + b for a, b in zip(first, mine)]
    # a group's rows begin with the same pages; every page is somewhere else in a shuffled pool
    pool = sum(p // P for p, _ in groups) + sum(_ceil(m, P) for m in mine) + 5
    order = torch.randperm(pool, generator=_gen(seed, 1), device="cuda").to(torch.int32)
    W = max(_ceil(k, P) for k in kv)
    start, at = [], 0
    for p, m in groups:
        start += [at] * m
        at += p // P
    behind = torch.cumsum(_i32([_ceil(m, P) for m in mine]), 0) - _i32([_ceil(m, P) for m in mine]) + at
    col = torch.arange(W, device="cuda")
    f, start = _i32(first)[:, None] // P, _i32(start)[:, None]
    place = torch.where(col < f, start + col, behind[:, None] + col - f).clamp(max=pool - 1)
    table = torch.where(col < _i32([_ceil(k, P) for k in kv])[:, None], order[place.long()], _i32([-1]))
    if c["op"] == "plan":           # in every group one request's prompt leaves the others' in the last quarter
        rng = random.Random(seed)
        at = 0
        for p, m in groups:
            n = p // P
            if m > 1 and n:
                j = rng.randint(n * 3 // 4, n - 1)
                table[at + rng.randrange(m), j:n] = torch.randint(0, pool, (n - j,), generator=_gen(seed, 8),
                                                                  device="cuda", dtype=torch.int32)
            at += m
    if c.get("gone"):               # pages the server dropped, for all that had them
        drop = torch.rand(pool, generator=_gen(seed, 2), device="cuda") < c["gone"]
        table = torch.where((table >= 0) & drop[table.clamp(min=0).long()], _i32([-1]), table)
    ends = [0]
    for _, m in groups:
        ends.append(ends[-1] + m)
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    s = dict(c=c, table=table.contiguous(), kv_len=_i32(kv), cu=None if c["q"] == "one" else _i32(cu),
             group=_i32(ends), S=S, max_q=max(q), max_group_q=max(cu[b] - cu[a] for a, b in zip(ends, ends[1:])))
    if c["op"] == "plan":
        return s
    got = _plain_plan(s)
    s["shared"], s["lead"] = got["shared"], got["lead"]
    s["kc"], s["ks"] = _cache(pool, c, seed, 3)
    s["vc"], s["vs"] = _cache(pool, c, seed, 5)
    s["q"] = _randn((sum(q), c["Hq"], c["D"]), seed, 7).to(DTYPE[c["dtype"]])
    s["scale"] = 1.0 / math.sqrt(c["D"])
    # what a server has on its host anyway; the plain form slices by it
    s["ends"], s["cu_host"], s["lens"] = ends, cu, kv
    s["first"] = got["shared"].tolist()
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    op = c["op"]
    if own:
        import gated_delta_rule_gdr_gb300 as gdr
        if op in ("norm", "grad"):
            how = dict(norm=c["norm"], q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"], positions=s["pos"],
                       freq=s["freq"], pairs=c["pairs"])
            if op == "norm":
                q, k = gdr.qk_norm_rope(s["q"], s["k"], **how)
                return dict(q=q, k=k)
            dq, dk, dwq, dwk = gdr.qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], **how)
            return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
        if op == "plan":
            shared, lead = gdr.kv8_shared_plan(s["table"], s["kv_len"], s["group"], c["page"], cu_q=s["cu"])
            return dict(shared=shared, lead=lead)
        out, lse = gdr.kv8_attn_shared(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["kv_len"],
                                       s["scale"], s["group"], s["shared"], s["lead"], cu_q=s["cu"],
                                       max_q=s["max_q"], max_group_q=s["max_group_q"], want_lse=True)
        return dict(out=out, lse=lse)
    if op == "norm":
        return dict(q=_plain_norm(s, s["q"], s["wq"]), k=_plain_norm(s, s["k"], s["wk"]))
    if op == "grad":
        dq, dwq = _plain_grad(s, s["q"], s["wq"], s["gq"])
        dk, dwk = _plain_grad(s, s["k"], s["wk"], s["gk"])
        return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    return _plain_plan(s) if op == "plan" else _plain_attn(s)


def _turn(s):
    """cos and sin of every token's angles, [T, 1, rot / 2]."""
    a = s["pos"].double()[:, None] * s["freq"]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, s, back):
    rot = s["c"]["rot"]
    if not rot:
        return x
    cos, sin = _turn(s)
    sin = -sin if back else sin
    y = x.clone()
    if s["c"]["pairs"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _inverse_norm(s, x):
    kind, D = s["c"]["norm"], s["c"]["D"]
    if kind == "none":
        return None
    return torch.rsqrt((x * x).sum(-1, keepdim=True) / (D if kind == "rms" else 1) + s["eps"])


def _plain_norm(s, x, w):
    y = x.float()
    r = _inverse_norm(s, y)
    y = y if r is None else y * r
    y = y if w is None else y * w
    return _rotate(y, s, False).to(x.dtype)


def _plain_grad(s, x, w, g):
    f, g = x.float(), _rotate(g.float(), s, True)
    r = _inverse_norm(s, f)
    if r is None:
        return g.to(x.dtype), None
    dw = None if w is None else (g * f * r).sum((0, 1))
    g = g if w is None else g * w
    n = s["c"]["D"] if s["c"]["norm"] == "rms" else 1
    return (r * g - f * (r * r * r * (g * f).sum(-1, keepdim=True) / n)).to(x.dtype), dw


def _plain_plan(s):
    """shared [S]: tokens of the pages that a request's group has in common; lead [groups]: a request to
    read them from (-1: none).  Only requests with queries count, two at least, and all of their
    queries see the pages."""
    table, kv, P = s["table"], s["kv_len"].long(), s["c"]["page"]
    S, W = table.shape
    dev, ends = table.device, s["group"].long()
    n = torch.ones_like(kv) if s["cu"] is None else (s["cu"][1:] - s["cu"][:-1]).long()
    r, groups = torch.arange(S, device=dev), ends.numel() - 1
    g = torch.searchsorted(ends[1:].contiguous(), r, right=True)
    live = n > 0
    count = torch.zeros(groups, dtype=torch.long, device=dev).index_add_(0, g, live.long())
    lead = torch.full((groups,), S, dtype=torch.long, device=dev)
    lead = lead.scatter_reduce_(0, g, torch.where(live, r, S), "amin")
    limit = ((kv - n + 1).clamp(min=0) // P).clamp(max=W)
    col = torch.arange(W, device=dev)
    same = (table == table[lead[g].clamp(max=S - 1)]) & (col < limit[:, None])
    pages = torch.where(same, W, col).amin(1)
    most = torch.full((groups,), W, dtype=torch.long, device=dev)
    most = most.scatter_reduce_(0, g, torch.where(live, pages, W), "amin")
    most = torch.where(count > 1, most, 0)
    return dict(shared=torch.where(live, most[g] * P, 0).to(torch.int32),
                lead=torch.where(most > 0, lead, -1).to(torch.int32))


def _read(s, name, pages):
    """Codes times scales of some pages in 32 bits, [H, tokens, D]; and which tokens are there."""
    cache, scale = s[name + "c"], s[name + "s"]
    there = (pages >= 0) & (pages < cache.shape[0])
    at = torch.where(there, pages, 0).long()
    x = cache.view(torch.uint8)[at].view(cache.dtype).float() * scale[at][..., None, None]
    return x.movedim(-3, 0).flatten(-3, -2), there.repeat_interleave(cache.shape[2], -1)


def _plain_attn(s):
    """The pages in common once for a group, the rest request by request (padded to the longest)."""
    c, table, cu, ends, kv, first = s["c"], s["table"], s["cu_host"], s["ends"], s["lens"], s["first"]
    P, D, H, G = c["page"], c["D"], c["Hkv"], c["Hq"] // c["Hkv"]
    S, dev, T = c["S"], table.device, s["q"].shape[0]
    x = s["q"].float().view(T, H, G, D).permute(1, 0, 2, 3) * s["scale"]             # [H, T, G, D]
    top = torch.full((H, T, G, 1), -math.inf, device=dev)
    tot = torch.zeros((H, T, G, 1), device=dev)
    acc = torch.zeros((H, T, G, D), device=dev)

    def join(rows, m, t, o):
        """A part's maximum, sum and products into those of some queries."""
        new = torch.maximum(top[:, rows], m)
        ref = torch.where(new == -math.inf, 0.0, new)
        a, b = torch.exp(top[:, rows] - ref), torch.exp(m - ref)
        tot[:, rows] = tot[:, rows] * a + t * b
        acc[:, rows] = acc[:, rows] * a + o * b
        top[:, rows] = new

    for a, b in zip(ends, ends[1:]):
        live = [i for i in range(a, b) if cu[i + 1] > cu[i]]
        p = first[live[0]] if live else 0
        if p == 0:
            continue
        rows = slice(cu[a], cu[b])
        row = table[live[0], :p // P]
        k, there = _read(s, "k", row)
        v, _ = _read(s, "v", row)
        z = torch.matmul(x[:, rows].flatten(1, 2), k.transpose(1, 2)).masked_fill_(~there, -math.inf)
        m = z.amax(-1, keepdim=True)
        z.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
        shape = (H, cu[b] - cu[a], G, -1)
        join(rows, m.view(shape), z.sum(-1, keepdim=True).view(shape), torch.matmul(z, v).view(shape))
    # the rest: [S, H, max_q * G, longest]
    M = s["max_q"]
    skip, n = s["shared"].long(), _i32(cu[1:]) - _i32(cu[:-1])
    W = max(_ceil(k - f, P) for k, f in zip(kv, first))
    col = skip[:, None] // P + torch.arange(W, device=dev)
    pages = torch.where(col < table.shape[1], table.gather(1, col.clamp(max=table.shape[1] - 1)), -1)
    at = (_i32(cu[:-1])[:, None] + torch.arange(M, device=dev)).clamp(max=max(T - 1, 0)).long()
    rest = x[:, at].movedim(1, 0).flatten(2, 3)
    k, there = _read(s, "k", pages)
    v, _ = _read(s, "v", pages)
    k, v = k.movedim(1, 0), v.movedim(1, 0)
    z = torch.matmul(rest, k.transpose(2, 3)).view(S, H, M, G, -1)
    j = skip[:, None] + torch.arange(z.shape[-1], device=dev)
    i = torch.arange(M, device=dev)
    see = (j[:, None] < (s["kv_len"] - n + 1)[:, None, None] + i[:, None]) & (j < s["kv_len"][:, None])[:, None]
    z.masked_fill_(~(see & there[:, None])[:, None, :, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    z.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    t = z.sum(-1, keepdim=True)
    o = torch.matmul(z.flatten(2, 3), v).view(S, H, M, G, D)
    r = torch.repeat_interleave(torch.arange(S, device=dev), n, output_size=T)
    k = torch.arange(T, device=dev) - _i32(cu)[r]
    join(slice(0, T), *(y[r, :, k].movedim(0, 1) for y in (m, t, o)))
    out = torch.where(tot > 0, acc / tot, 0.0).permute(1, 0, 2, 3).reshape(T, H * G, D)
    lse = (torch.log(tot) + top).permute(1, 0, 2, 3).reshape(T, H * G)
    return dict(out=out.to(s["q"].dtype), lse=lse)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "plan":
        return None                  # whole numbers only
    if c["op"] in ("norm", "grad"):
        T, D, rot = c["T"], c["D"], c["rot"]
        got = {}
        for name, x, w, g in (("q", s["q"], s["wq"], s.get("gq")), ("k", s["k"], s["wk"], s.get("gk"))):
            x = x.double()
            if rot:                  # a token's rotation as complex factors of its pairs
                z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                s["pos"].double()[:, None] * s["freq"])[:, None]

            def turn(y, by):
                if not rot:
                    return y
                y = y.clone()
                if c["pairs"] == "half":
                    v = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * by
                    y[..., :rot // 2], y[..., rot // 2:rot] = v.real, v.imag
                else:
                    v = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2)) * by
                    y[..., :rot] = torch.view_as_real(v).flatten(-2)
                return y

            if c["norm"] == "none":
                size = torch.ones((T, 1, 1), dtype=torch.float64, device="cuda")
            else:
                size = torch.sqrt(x.square().sum(-1, keepdim=True) / (D if c["norm"] == "rms" else 1) + s["eps"])
            unit = x / size
            weight = torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()
            if c["op"] == "norm":
                got[name] = turn(unit * weight, z if rot else None)
                continue
            g = turn(g.double(), z.conj() if rot else None)
            got["dw" + name] = None if w is None else (g * unit).sum((0, 1))
            g = g * weight
            if c["norm"] != "none":
                along = (g * unit).sum(-1, keepdim=True) / (D if c["norm"] == "rms" else 1)
                g = (g - unit * along) / size
            got["d" + name] = g
        return got if c["op"] == "norm" else {k: got[k] for k in ("dq", "dk", "dwq", "dwk")}
    # attention of every request over all that it has, by its own row of the table
    cu, kv = s["cu_host"], s["lens"]
    H, G, P, N = c["Hkv"], c["Hq"] // c["Hkv"], c["page"], s["kc"].shape[0]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for r in range(c["S"]):
        n, a, b = kv[r], cu[r], cu[r + 1]
        if a == b or n == 0:
            continue
        row = s["table"][r, :_ceil(n, P)].long()
        ok = ((row >= 0) & (row < N)).repeat_interleave(P)[:n]
        row = row.clamp(min=0)
        last = n - (b - a) + torch.arange(b - a, device="cuda")
        sees = ((torch.arange(n, device="cuda") <= last[:, None]) & ok)[:, None]
        for h in range(H):
            k, v = ((x[row, h].double() if x.dtype is torch.int8 else x[:, h].contiguous().view(torch.uint8)[row]
                     .view(x.dtype).double()) * y[row, h].double()[:, None, None]
                    for x, y in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            x = s["q"][a:b, h * G:(h + 1) * G].double().reshape(-1, c["D"])
            z = (x @ k.reshape(-1, c["D"])[:n].T).view(b - a, G, n) * s["scale"]
            z = torch.where(sees, z, torch.full((), -math.inf, dtype=z.dtype, device="cuda"))
            e = torch.logsumexp(z, -1)
            w = torch.exp(z - torch.where(e > -math.inf, e, 0.0)[..., None])
            out[a:b, h * G:(h + 1) * G] = (w.view(-1, n) @ v.reshape(-1, c["D"])[:n]).view(b - a, G, -1)
            lse[a:b, h * G:(h + 1) * G] = e
    return dict(out=out, lse=lse)
