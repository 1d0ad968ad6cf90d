"""Attention of requests that share a prefix (gdr_kv8_shared_plan, gdr_kv8_attn_shared) against the
fp64 oracle of the attention over each request's whole row, and against gdr_kv8_attn.

Tolerances are those of gdr_kv8_attn, whose operands and sums both passes have: bf16 3e-3 in relative L2
(the output's one rounding, uniform in half a step of 2^-8, is 2^-8 / sqrt(3) = 2.26e-3, and weights of
11 bits 2^-11), fp32 1e-5; joining two fp32 sums adds 2^-23.  The plan gives whole numbers: equal."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
import oracle
from oracle import kv8 as O

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TOL = {BF16: 3e-3, F32: 1e-5}
LSE_TOL = 1e-5
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    with gdr.option(shared_least=1):        # both passes, however little there is to share
        yield
    torch.cuda.synchronize()
    assert gdr.last_device_error() == 0


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def plan_oracle(table, kv, n, group, page):
    """shared, lead from the definition, request by request."""
    S, W = table.shape
    shared, lead = [0] * S, []
    for a, b in zip(group, group[1:]):
        live = [s for s in range(a, b) if n[s] > 0]
        most = 0
        if len(live) > 1:
            most = min(max(0, min(kv[s], W * page) - n[s] + 1) // page for s in live)
            for c in range(most):
                if len({int(table[s, c]) for s in live}) > 1:
                    most = c
                    break
        for s in live:
            shared[s] = most * page
        lead.append(live[0] if most else -1)
    return shared, lead


def case(groups, Hq, Hkv, D, page, dtype, kv, seed=0, gone=0.0, q_scale=1.0, spare=2):
    """groups: a list of (prefix pages, [(own tokens, queries), ...]); a request's queries are its last."""
    g = torch.Generator().manual_seed(seed)
    lens, qs, ends, rows = [], [], [0], []
    at = 0
    for pre, reqs in groups:
        common, at = list(range(at, at + pre)), at + pre
        for mine, n in reqs:
            k = -(-mine // page)
            rows.append(common + list(range(at, at + k)))
            at += k
            lens.append(pre * page + mine)
            qs.append(n)
        ends.append(len(lens))
    N, W = at + 3, max(max(map(len, rows)), 1) + spare
    order = torch.randperm(N, generator=g)
    drop = torch.rand(N, generator=g) < gone
    table = torch.full((len(lens), W), -1, dtype=torch.int32)
    for s, r in enumerate(rows):
        for c, p in enumerate(r):
            table[s, c] = N + 5 if drop[p] else int(order[p])

    def cache():
        if kv == "int8":
            c = torch.randint(-127, 128, (N, Hkv, page, D), generator=g, dtype=torch.int8)
        else:
            c = (torch.randn((N, Hkv, page, D), generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        return c, torch.exp2(torch.randint(-8, -4, (N, Hkv), generator=g).float())

    (kc, ks), (vc, vs) = cache(), cache()
    # what no request has: NaN codes (int8: the largest)
    live = torch.zeros((N, page), dtype=torch.bool)
    for s, n in enumerate(lens):
        for i in range(-(-n // page)):
            if table[s, i] < N:
                live[int(table[s, i]), :min(page, n - i * page)] = True
    for c in (kc, vc):
        c.view(torch.uint8).permute(0, 2, 1, 3)[~live] = 0x7f
    q = (torch.randn((sum(qs), Hq, D), generator=g) * q_scale).to(dtype)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=lens, qs=qs, ends=ends, kv=kv,
                cu=[sum(qs[:i]) for i in range(len(qs) + 1)], scale=1 / math.sqrt(D), page=page)


def on_gpu(x):
    return dict(q=x["q"].cuda(), cache=[x[k].cuda() for k in ("kc", "vc", "ks", "vs")], table=x["table"].cuda(),
                kv_len=i32(x["lens"]), cu=i32(x["cu"]), group=i32(x["ends"]))


def attend(x, d=None, plan=None, **kw):
    d = d or on_gpu(x)
    packed = kw.pop("packed", False)
    one = all(n == 1 for n in x["qs"]) and not packed
    cu = None if one else d["cu"]
    shared, lead = plan or gdr.kv8_shared_plan(d["table"], d["kv_len"], d["group"], x["page"], cu_q=cu)
    sizes = dict(max_q=max(x["qs"]),
                 max_group_q=max(x["cu"][b] - x["cu"][a] for a, b in zip(x["ends"], x["ends"][1:])), want_lse=True)
    return gdr.kv8_attn_shared(d["q"], *d["cache"], d["table"], d["kv_len"], x["scale"], d["group"], shared, lead, cu_q=cu,
                               **{**sizes, **kw})


def check(x, got=None):
    out, lse = attend(x) if got is None else got
    ro, rl = O.attention(x["q"].double().numpy(), x["kc"].view(torch.uint8).numpy(), x["vc"].view(torch.uint8).numpy(),
                         x["ks"].double().numpy(), x["vs"].double().numpy(), x["table"].numpy(), x["lens"], x["cu"],
                         x["scale"], x["kv"])
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(out).all()
    empty = rl == -math.inf
    assert np.array_equal(lse == -math.inf, empty) and (out[empty] == 0).all()
    if (~empty).any():
        assert np.abs(lse - rl)[~empty].max() <= LSE_TOL * max(1.0, np.abs(rl[~empty]).max())
    for a, b in zip(x["cu"], x["cu"][1:]):              # every request for itself
        if b > a and not empty[a:b].all():
            assert oracle.rel_l2(out[a:b], ro[a:b]) <= TOL[x["q"].dtype], (a, oracle.rel_l2(out[a:b], ro[a:b]))


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("seed", range(12))
def test_plan(seed):
    rng = np.random.default_rng(seed)
    S, page = int(rng.integers(1, 70)), int(rng.choice([16, 32, 64, 128]))
    W = int(rng.integers(1, 5000 if seed % 3 == 0 else 60))
    table = rng.integers(0, 1000, (1, W)).repeat(S, 0).astype(np.int32)
    for s in range(S):                      # rows leave the common one somewhere, or not; gone pages are equal too
        c = int(rng.integers(0, 2 * W))
        if c < W and rng.random() < 0.7:
            table[s, c] = -1 if rng.random() < 0.2 else 2000 + s
    table[:, :1] = -1 if seed % 4 == 1 else 7
    kv = rng.integers(0, W * page + 40, S)
    kv[rng.random(S) < 0.5] = W * page
    n = np.where(rng.random(S) < 0.2, 0, rng.integers(1, 6, S)) if seed % 2 else np.ones(S, np.int64)
    cuts = np.sort(rng.integers(0, S + 1, int(rng.integers(0, 6))))
    group = [int(c) for c in cuts] if seed % 5 == 4 and len(cuts) > 1 else [0, *map(int, cuts), S]
    want = plan_oracle(table, kv, n, group, page)
    cu = None if (n == 1).all() and seed % 2 == 0 else i32(np.concatenate([[0], np.cumsum(n)]))
    shared, lead = gdr.kv8_shared_plan(i32(table), i32(kv), i32(group), page, cu_q=cu)
    assert shared.tolist() == want[0] and lead.tolist() == want[1]


def test_plan_of_many():
    """The most requests there may be, in one group; and each in a group of its own."""
    S, W = 8192, 40
    table = torch.arange(W, dtype=torch.int32).repeat(S, 1)
    table[5000, 33] = -3
    kv = torch.full((S,), W * 16, dtype=torch.int32)
    shared, lead = gdr.kv8_shared_plan(table.cuda(), kv.cuda(), i32([0, S]), 16)
    assert (shared == 33 * 16).all() and lead.tolist() == [0]
    shared, lead = gdr.kv8_shared_plan(table.cuda(), kv.cuda(), torch.arange(S + 1, dtype=torch.int32).cuda(), 16)
    assert (shared == 0).all() and (lead == -1).all()


# ------------------------------------------------------------------ attention
CASES = [
    # groups, Hq, Hkv, D, page
    ([(4, [(1, 1), (1, 1)])], 2, 2, 64, 16),                                       # nothing of their own but the token
    ([(9, [(5, 1), (30, 1), (17, 1)])], 8, 2, 128, 16),                            # split kernel twice
    ([(40, [(3, 1)] * 20), (7, [(100, 1)] * 3), (3, [(9, 1)]), (0, [(40, 1), (50, 1)])], 16, 2, 128, 32),
    ([(3, [(300, 1)] * 70)], 16, 4, 128, 64),                                      # 280 rows: pairs of tiles, divided
    ([(20, [(10, 1)] * 40)], 6, 2, 64, 16),                                        # 120 rows: one tile
    ([(25, [(4, 1)] * 9), (12, [(7, 1)] * 9)], 10, 2, 128, 128),                   # 45 rows: two copies
    ([(8, [(2, 1)] * 6)], 8, 2, 64, 64),                                           # 24 rows: four copies
    ([(30, [(8, 5), (20, 2), (6, 0), (9, 5)]), (5, [(40, 3), (12, 12)])], 8, 2, 128, 16),
    ([(6, [(60, 40), (200, 33), (50, 50)])], 4, 4, 64, 32),
    ([(10, [(300, 200), (180, 150), (90, 1)]), (2, [(130, 129), (140, 140)])], 8, 2, 128, 64),
    ([(70, [(1, 1), (40, 17), (33, 33), (900, 2)])], 5, 1, 128, 16),
    ([(1, [(16, 1)] * 2)], 64, 1, 128, 16),
    ([(75, [(3, 1)] * 33)], 28, 4, 64, 16),                                        # 231 rows of many parts
    ([(19, [(1, 1)] * 37), (4, [(3, 1)] * 2)], 21, 3, 128, 64),                    # 259
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_whole(dtype, kv, i):
    check(case(*CASES[i], dtype, kv, seed=i))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gone", [0.3, 1.0])
def test_pages_gone(dtype, gone):
    check(case([(30, [(8, 2), (20, 1), (6, 3)]), (9, [(5, 1)] * 30)], 8, 2, 128, 16, dtype, "e4m3", seed=3, gone=gone))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("own", [1, 90])
@pytest.mark.parametrize("up", [True, False])
def test_scores_far_apart(dtype, own, up):
    """The common pages' scores far above or below a request's own: one part weighs next to nothing."""
    x = case([(12, [(own, 1), (own, 1), (own + 60, 1)] * 8)], 8, 2, 64, 16, dtype, "int8", seed=5)
    first = x["table"][0, :12].long()
    x["ks"][first] *= 16.0 if up else 1 / 64
    if not up:
        others = torch.ones(len(x["ks"]), dtype=torch.bool)
        others[first] = False
        x["ks"][others] *= 16.0
    check(x)


def test_one_request_and_no_prefix():
    """Groups of one, idle requests, requests outside every group: as gdr_kv8_attn."""
    x = case([(5, [(30, 2)]), (0, [(9, 1)] * 4), (3, [(8, 0), (9, 0), (4, 1)])], 8, 2, 128, 16, BF16, "e4m3", seed=9)
    check(x)
    x["ends"] = [1, 3, 3]
    check(x)


@pytest.mark.parametrize("max_q,max_group_q", [(1, 1), (1, 1000), (300, 2), (0, 0)])
def test_bounds_that_are_off(max_q, max_group_q):
    x = case([(20, [(10, 3), (50, 7), (9, 9)]), (6, [(7, 1)] * 3)], 8, 2, 128, 16, BF16, "e4m3", seed=11)
    check(x, attend(x, max_q=max_q, max_group_q=max_group_q))


def test_plans_that_are_off():
    """Entries outside their ranges read nothing outside the tensors; other groups are as they were."""
    x = case([(20, [(10, 1)] * 5), (6, [(7, 1)] * 3)], 8, 2, 128, 16, BF16, "e4m3", seed=12)
    d = on_gpu(x)
    want, _ = attend(x, d)
    shared, lead = gdr.kv8_shared_plan(d["table"], d["kv_len"], d["group"], 16)
    for bad_lead, bad_shared in ((-9, 320), (8, 2 ** 31 - 1), (2 ** 31 - 1, -7), (0, -1), (0, 2 ** 31 - 1), (-2 ** 31, 5)):
        s, l = shared.clone(), lead.clone()
        l[0] = bad_lead
        s[:5] = bad_shared
        out, _ = attend(x, d, plan=(s, l))
        assert torch.equal(out[5:], want[5:])


def test_strides_streams_graphs_and_rows_behind():
    x = case([(20, [(10, 3), (50, 2), (9, 4)] * 3), (6, [(7, 1)] * 3)], 8, 2, 128, 16, BF16, "int8", seed=13)
    d = on_gpu(x)
    want = attend(x, d)
    check(x, want)
    T = d["q"].shape[0]
    wide = torch.randn((T + 5, 12, 128), device="cuda").bfloat16()
    wide[:T, :8] = d["q"]
    wide[T:] = math.nan
    e = dict(d, q=wide[:, :8])
    out = torch.full((T + 5, 8, 128), 7.0, device="cuda", dtype=BF16)
    ws = torch.empty(gdr.kv8_attn_shared_workspace_size(12, 4, 2, 27, T + 5, 8, 2, 128), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    got, lse = attend(x, e, out=out, workspace=ws)
    assert torch.equal(got[:T], want[0]) and torch.equal(lse[:T], want[1]) and (got[T:] == 7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = attend(x, d)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attend(x, e, workspace=ws)
        again = attend(x, e, workspace=ws)              # the second follows on the first's workspace
    for _ in range(3):
        ws.fill_(255)
        got[0].zero_(), again[0].zero_()
        graph.replay()
        assert torch.equal(got[0][:T], want[0]) and torch.equal(again[0][:T], want[0])


def test_many_times_as_kv8_attn():
    """A batch as a server has it, against gdr_kv8_attn on the same rows, one bf16 step apart at most."""
    x = case([(60, [(20, 1)] * 50), (33, [(100, 1)] * 30)], 32, 4, 128, 64, BF16, "e4m3", seed=14)
    d = on_gpu(x)
    a, la = attend(x, d)
    b, lb = gdr.kv8_attn(d["q"], *d["cache"], d["table"], d["kv_len"], x["scale"], want_lse=True)
    # each is within half a step of the exact value and 2^-10 of the row's largest weight's share
    assert oracle.rel_l2(a.cpu(), b.cpu()) <= 2 * TOL[BF16]
    assert (la - lb).abs().max() <= 2 * LSE_TOL * max(1.0, float(lb.abs().max()))


@pytest.mark.parametrize("qs,rows", [(1, 2), (2, 3), (3, 30), (30, 30)])
def test_waits_give_up(qs, rows):
    x = case([(20, [(qs + 5, qs)] * rows)], 8, 2, 128, 16, BF16, "e4m3", seed=15)
    d = on_gpu(x)
    plan = gdr.kv8_shared_plan(d["table"], d["kv_len"], d["group"], 16, cu_q=d["cu"])
    torch.cuda.synchronize()
    with gdr.option(wait_limit_ns=0):
        attend(x, d, plan=plan, packed=True)
        assert gdr.last_device_error() == 5
    check(x, attend(x, d, plan=plan, packed=True))
    assert gdr.last_device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_chosen_by_sizes(dtype):
    """By the cost model, and with a bound between two groups' prefixes: in one pass, in two, mixed."""
    for groups in ([(4, [(9, 1)] * 5)], [(400, [(20, 1)] * 30), (2, [(7, 1)] * 4)],
                   [(90, [(9, 2), (40, 3)]), (20, [(9, 1)] * 6)]):
        x = case(groups, 16, 2, 128, 16, dtype, "e4m3", seed=16)
        for least in (0, 500, 2 ** 31 - 1):
            with gdr.option(shared_least=least):
                check(x)


def test_option():
    for bad in (-1, 2 ** 31):
        with pytest.raises(gdr.GdrError):
            gdr.set_option("shared_least", bad)
    with gdr.option(shared_least=77):
        assert gdr.get_option("shared_least") == 77


def test_another_device(monkeypatch):
    """Tensors that are not on the current device are refused (the current one is made out to be another)."""
    x = case([(2, [(9, 1)] * 3)], 2, 2, 64, 16, BF16, "int8")
    d = on_gpu(x)
    plan = gdr.kv8_shared_plan(d["table"], d["kv_len"], d["group"], 16)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        gdr.kv8_shared_plan(d["table"], d["kv_len"], d["group"], 16)
    with pytest.raises(ValueError, match="current device"):
        attend(x, d, plan=plan)


@pytest.mark.parametrize("size", [2, 3, 1024])
def test_the_most_requests(size):
    """8192 requests in groups of two, of three (some left over, outside every group) and of 1024."""
    S, page, D, Hkv, Hq = 8192, 16, 64, 1, 2
    groups = S // size
    g = torch.Generator().manual_seed(size)
    N = 3 * groups + S
    order = torch.randperm(N, generator=g).to(torch.int32)
    r = torch.arange(S)
    table = torch.stack([order[(r // size).clamp(max=groups - 1) * 3 + c] for c in range(3)]
                        + [order[3 * groups + r]], 1)
    kv = torch.randint(3 * page + 1, 4 * page + 1, (S,), generator=g, dtype=torch.int32)
    cache = [torch.randint(-127, 128, (N, Hkv, page, D), generator=g, dtype=torch.int8).cuda() for _ in range(2)]
    scale = [torch.exp2(torch.randint(-8, -4, (N, Hkv), generator=g).float()).cuda() for _ in range(2)]
    q = torch.randn((S, Hq, D), generator=g).bfloat16().cuda()
    group = torch.arange(groups + 1, dtype=torch.int32).cuda() * size
    shared, lead = gdr.kv8_shared_plan(table.cuda(), kv.cuda(), group, page)
    inside = groups * size
    assert (shared[:inside] == 48).all() and (shared[inside:] == 0).all()
    assert torch.equal(lead.cpu(), torch.arange(groups, dtype=torch.int32) * size)
    a, la = gdr.kv8_attn_shared(q, *cache, *scale, table.cuda(), kv.cuda(), 0.125, group, shared, lead, max_group_q=size,
                                want_lse=True)
    b, lb = gdr.kv8_attn(q, *cache, *scale, table.cuda(), kv.cuda(), 0.125, want_lse=True)
    assert oracle.rel_l2(a.cpu(), b.cpu()) <= 2 * TOL[BF16]
    assert (la - lb).abs().max() <= 2 * LSE_TOL * max(1.0, float(lb.abs().max()))
