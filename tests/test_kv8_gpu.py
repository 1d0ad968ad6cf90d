"""The paged 8-bit cache on the GPU (gdr_page_plan, gdr_kv8_append, gdr_kv8_attn, through the
C ABI) against the fp64 / integer oracle on the same seeded inputs.

Plan and append give whole numbers, codes and power-of-two scales: they are equal to the
oracle's.  Attention: a bf16 output is rounded once (an error uniform in half a unit of the
last of 8 bits: at most 2^-7 / sqrt(12) = 2.26e-3 in relative L2) and its weights to 11 bits
(at most 2^-11 = 4.9e-4): 3e-3 is asked.  fp32 runs on 22-bit operands: 1e-5, the library's
fp32 tolerance, on outputs and lse."""
from __future__ import annotations

import math
import random

import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
import oracle
from oracle import kv8 as O

pytestmark = pytest.mark.gpu
TOL = {torch.bfloat16: 3e-3, torch.float32: 1e-5}
LSE_TOL = 1e-5
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    yield
    assert gdr.last_device_error() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def codes_np(t):
    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------ plan
def plan_case(S, W, page, seed, q_max, free, finished=0.1, extra=9, max_tokens=None, kv_max=None):
    r = random.Random(seed)
    kv = [r.randint(0, kv_max or W * page) for _ in range(S)]
    q = [-1 if r.random() < finished else r.randint(0, q_max) for _ in range(S)]
    used = sum(-(-k // page) for k in kv)
    N = used + free
    perm = list(range(N))
    r.shuffle(perm)
    table = np.full((S, W), -7)
    it = iter(perm)
    for s, k in enumerate(kv):
        for i in range(-(-k // page)):
            table[s, i] = next(it)
    head = r.randrange(N)
    ring = np.full(N, -3)
    for i, p in enumerate(it):
        ring[(head + i) % N] = p
    T = sum(n for n in q if n > 0) + extra if max_tokens is None else max_tokens
    return kv, q, table, ring, [head, free], T


@pytest.mark.parametrize("S,W,page,q_max,free,kw", [
    (1, 4, 16, 1, 3, {}), (1, 64, 16, 700, 60, dict(finished=0.0, kv_max=100)),
    (7, 40, 32, 90, 40, {}), (300, 24, 64, 1, 200, {}), (257, 33, 16, 64, 300, dict(kv_max=300)),
    (1500, 20, 128, 40, 900, {}), (4097, 4, 16, 3, 2000, {}), (40, 30, 16, 50, 25, {}),
    (64, 16, 16, 60, 1000, {}),                                    # some outgrow their table
    (30, 64, 16, 100, 500, dict(max_tokens=700)), (5, 8, 16, 9, 9, dict(finished=1.0)),
    (8192, 2, 16, 1, 100, {}), (3, 5, 16, 4, 0, dict(kv_max=40, extra=0)),
])
def test_plan_equals_oracle(S, W, page, q_max, free, kw):
    if free == 0:
        free = 1
    kv, q, table, ring, state, T = plan_case(S, W, page, S + W, q_max, free, **kw)
    t, r = i32(table), i32(ring)
    for _ in range(2):              # a plan repeats: outputs depend on the inputs alone
        got = gdr.page_plan(i32(kv), i32(q), t, r, i32(state), page, T)
        want = O.plan(kv, q, table, ring, state, page, T)
        for g, w, name in zip((*got, t, r), want, ("kv", "cu", "slots", "pos", "granted", "state", "table", "ring")):
            assert np.array_equal(g.cpu().numpy(), np.asarray(w)), name


def test_plan_no_requests():
    kv, cu, slots, pos, ok, st = gdr.page_plan(i32([]), i32([]), torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                                               i32([0, 1, 2]), i32([1, 2]), 16, 5)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 5 and st.tolist() == [1, 2]


# ------------------------------------------------------------------ append
def random_cache(N, H, P, D, kv, g, spread=0.0):
    """Codes of any value but NaN, power-of-two scales."""
    c = torch.randint(0, 256, (N, H, P, D), dtype=torch.uint8, generator=g)
    if kv == "e4m3":
        c[(c & 0x7f) == 0x7f] = 0x30
    else:
        c[c == 0x80] = 0x81
    s = torch.exp2(torch.randint(-3, 3, (N, H), generator=g).float() + spread * torch.randn((N, H), generator=g).round())
    return c, s


def check_append(k, v, slots, kc, vc, ks, vs, page, kv):
    want = []
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        cn, sn = c.numpy().copy(), s.numpy().astype(np.float64).copy()
        O.append(x.double().cpu().numpy(), slots, cn, sn, page, kv)
        want.append((cn, sn))
    dev = [t.view(CODE[kv]).cuda() for t in (kc, vc)] + [ks.cuda(), vs.cuda()]
    gdr.kv8_append(k, v, i32(slots), *dev)
    for c, s, (cn, sn) in ((dev[0], dev[2], want[0]), (dev[1], dev[3], want[1])):
        assert np.array_equal(s.cpu().numpy().astype(np.float64), sn)
        got = codes_np(c)
        same = got == cn
        if kv == "e4m3":            # -0 and 0 are one value
            same |= ((got | cn) & 0x7f) == 0
        assert same.all()


def runs(lens, page, N, seed, drop=False):
    """Slots of requests that append lens tokens each, at random places of their first page."""
    r = random.Random(seed)
    pages = list(range(N))
    r.shuffle(pages)
    it, slots = iter(pages), []
    for n in lens:
        off = r.choice([0, r.randrange(page)])
        p = None
        for i in range(n):
            if p is None or (off + i) % page == 0:
                p = next(it)
            slots.append(p * page + (off + i) % page)
        if drop and n:
            slots += [-1, N * page + 3]
    return slots


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("H,D,page,lens", [
    (1, 64, 16, [1]), (3, 128, 16, [1, 0, 17, 40, 1, 1, 5]), (8, 128, 64, [1] * 70),
    (2, 64, 128, [300, 2, 129, 1, 128]), (5, 64, 32, [33] * 9), (1, 128, 128, [1000]),
    (4, 128, 32, [2, 3, 4, 5, 6, 7, 8, 9, 10, 31, 32, 33]),
])
def test_append_equals_oracle(dtype, kv, H, D, page, lens):
    g = torch.Generator().manual_seed(sum(lens) + H)
    N = sum(-(-n // page) + 1 for n in lens) + 3
    slots = runs(lens, page, N, H + D, drop=True)
    T = len(slots)
    x = [(torch.randn((T, H, D), generator=g) * torch.exp2(3 * torch.randn((T, H, 1), generator=g))).to(dtype).cuda()
         for _ in range(2)]
    (kc, ks), (vc, vs) = random_cache(N, H, page, D, kv, g), random_cache(N, H, page, D, kv, g)
    check_append(*x, slots, kc, vc, ks, vs, page, kv)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
def test_append_special_values_and_strides(kv):
    g = torch.Generator().manual_seed(3)
    H, D, page, N, T = 2, 64, 16, 6, 30
    # keys and values as slices of one projection: token stride (2 H + 2 H) D
    qkv = torch.randn((T, 4 * H, D), generator=g)
    qkv[3, 2, 5], qkv[4, 3, 6], qkv[5, 4, 7] = math.nan, math.inf, -math.inf
    qkv[7] = 0.0
    qkv[9, :, :3] = 1e-30
    qkv[20] = 3e38
    qkv[21:] = 0.0
    qkv = qkv.to(BF16).cuda()
    k, v = qkv[:, 2:4], qkv[:, 4:6]
    assert not k.is_contiguous()
    slots = list(range(5, 16)) + list(range(32, 48)) + [64, 65, 66]
    (kc, ks), (vc, vs) = random_cache(N, H, page, D, kv, g), random_cache(N, H, page, D, kv, g)
    check_append(k, v, slots, kc, vc, ks, vs, page, kv)
    # all rows zero, a page whose only values are NaN, a page that holds zeros grows
    z = torch.zeros((2, H, D), device="cuda", dtype=BF16)
    check_append(z, z, [0, 17], kc, vc, ks, vs, page, kv)
    check_append(z * math.nan, z + 1, [16, 17], kc, vc, ks, vs, page, kv)
    check_append(z + 1e-3, z + 7, [3, 4], kc * 0, vc * 0, ks * 0 + 2.0 ** -40, vs * 0 + 2.0 ** -40, page, kv)


def test_append_nothing():
    kc = torch.zeros((2, 1, 16, 64), dtype=torch.int8, device="cuda")
    s = torch.ones((2, 1), device="cuda")
    e = torch.empty((0, 1, 64), device="cuda")
    gdr.kv8_append(e, e, i32([]), kc, kc.clone(), s, s.clone())
    gdr.kv8_append(torch.ones((2, 1, 64), device="cuda"), torch.ones((2, 1, 64), device="cuda"), i32([-1, 32]),
                   kc, kc.clone(), s, s.clone())
    assert not kc.any() and (s == 1).all()


# ------------------------------------------------------------------ attention
def attn_case(lens, qs, Hq, Hkv, D, page, dtype, kv, seed=0, gone=0.0, spread=0.0, q_scale=1.0, slack=3):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    N, W = sum(need) + 4, max(max(need), 1) + slack
    perm = torch.randperm(N, generator=g).tolist()
    table = torch.full((len(lens), W), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    if gone:
        table[torch.rand(table.shape, generator=g) < gone] = N + 5
    (kc, ks), (vc, vs) = random_cache(N, Hkv, page, D, kv, g), random_cache(N, Hkv, page, D, kv, g, spread)
    ks = ks / (16 if kv == "int8" else 64)
    q = (torch.randn((sum(qs), Hq, D), generator=g) * q_scale).to(dtype)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=lens,
                cu=[sum(qs[:i]) for i in range(len(qs) + 1)], kv=kv, scale=1 / math.sqrt(D))


def poison(x):
    """NaN codes (int8: the largest) wherever a page holds no token of its request, and in
    pages that no request has."""
    kc, vc = x["kc"].clone(), x["vc"].clone()
    N, _, P, _ = kc.shape
    live = torch.zeros((N, P), dtype=torch.bool)
    for s, n in enumerate(x["lens"]):
        for i in range(-(-n // P)):
            p = int(x["table"][s, i])
            if 0 <= p < N:
                live[p, :max(0, min(P, n - i * P))] = True
    for c in (kc, vc):
        c.permute(0, 2, 1, 3)[~live] = 0x7f
    return dict(x, kc=kc, vc=vc)


def attend(x, want_lse=True, **kw):
    n = [b - a for a, b in zip(x["cu"], x["cu"][1:])]
    one = all(v == 1 for v in n)
    return gdr.kv8_attn(x["q"].cuda(), x["kc"].view(CODE[x["kv"]]).cuda(), x["vc"].view(CODE[x["kv"]]).cuda(),
                        x["ks"].cuda(), x["vs"].cuda(), x["table"].cuda(), i32(x["lens"]), x["scale"],
                        cu_q=None if one and "cu_q" not in kw else i32(x["cu"]), max_q=max(n + [1]),
                        want_lse=want_lse)


def want(x):
    return O.attention(x["q"].double().numpy(), x["kc"].numpy(), x["vc"].numpy(), x["ks"].double().numpy(),
                       x["vs"].double().numpy(), x["table"].numpy(), x["lens"], x["cu"], x["scale"], x["kv"])


def check(x, got=None):
    out, lse = attend(x) if got is None else got
    ro, rl = want(x)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(out).all()
    empty = rl == -math.inf
    assert np.array_equal(lse == -math.inf, empty) and (out[empty] == 0).all()
    if (~empty).any():
        assert np.abs(lse - rl)[~empty].max() <= LSE_TOL * max(1.0, np.abs(rl[~empty]).max())
    assert oracle.rel_l2(out, ro) <= TOL[x["q"].dtype], oracle.rel_l2(out, ro)
    for a, b in zip(x["cu"], x["cu"][1:]):              # every request for itself
        if b > a and not empty[a:b].all():
            assert oracle.rel_l2(out[a:b], ro[a:b]) <= TOL[x["q"].dtype]


DECODE = [
    ([1], 1, 1, 64, 16), ([17], 8, 8, 128, 16), ([1000], 32, 8, 128, 16), ([1, 0, 33, 2, 64], 12, 4, 64, 32),
    ([300, 299, 1, 128, 129, 0, 4096], 16, 2, 128, 64), ([513] * 9, 7, 1, 128, 128), ([777, 3], 48, 3, 64, 16),
    ([5000], 16, 1, 128, 128), ([64] * 70, 4, 2, 64, 64), ([2500, 40], 40, 2, 128, 32), ([700, 90], 64, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", DECODE)
def test_one_token(dtype, kv, lens, Hq, Hkv, D, page):
    check(poison(attn_case(lens, [1] * len(lens), Hq, Hkv, D, page, dtype, kv, seed=len(lens))))


MANY = [
    ([5], [5], 2, 2, 64, 16), ([40], [2], 8, 1, 128, 16), ([300, 17, 200], [5, 5, 5], 16, 2, 128, 32),
    ([130], [130], 4, 4, 64, 64), ([257, 31, 0, 90], [257, 31, 4, 0], 6, 2, 128, 16),
    ([700, 3, 900], [100, 7, 1], 8, 2, 128, 64), ([2000], [33], 32, 8, 128, 128), ([520, 520], [260, 520], 5, 1, 64, 16),
    ([1, 2, 3], [9, 2, 30], 3, 1, 64, 32), ([385], [129], 10, 2, 128, 128), ([1200], [65], 4, 4, 128, 64),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,qs,Hq,Hkv,D,page", MANY)
def test_several_tokens(dtype, kv, lens, qs, Hq, Hkv, D, page):
    check(poison(attn_case(lens, qs, Hq, Hkv, D, page, dtype, kv, seed=sum(qs))))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("qs", [[1, 1, 1], [3, 1, 2], [70, 150, 1]])
def test_pages_gone(dtype, qs):
    x = attn_case([600, 150, 80], qs, 8, 2, 128, 16, dtype, "e4m3", seed=5, gone=0.3)
    x["table"][2] = -1                       # a request whose pages are all gone
    check(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("qs", [[1, 1], [4, 3], [20, 9], [31, 5], [140, 80]])
@pytest.mark.parametrize("lens,page,every", [([900, 640], 16, 8), ([900, 640], 16, 1), ([1100, 129], 64, 1), ([128, 257], 32, 2)])
def test_growing_scores(dtype, qs, lens, page, every):
    """Key scales that grow along the cache: the running maximum moves inside and between
    tiles, to the last one of a request."""
    x = attn_case(lens, qs, 8, 2, 128, page, dtype, "int8", seed=6)
    for s in range(2):
        for i, p in enumerate(x["table"][s].tolist()):
            if p >= 0:
                x["ks"][p] = 2.0 ** (min(i // every, 18) / (2 if every == 1 else 1) - 9)
    check(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("qs", [[1, 1], [4, 3], [140, 80]])
def test_value_scales_far_apart(dtype, qs):
    """Value scales 2^-12 .. 2^12 apart, and scales that are no powers of two."""
    x = attn_case([700, 333], qs, 8, 2, 128, 32, dtype, "e4m3", seed=7, spread=4.0)
    check(x)
    x["vs"] = x["vs"] * 1.37
    x["ks"] = x["ks"] * 0.81
    check(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("q_scale", [1e-20, 30.0])
@pytest.mark.parametrize("qs", [[1, 1], [60, 80]])
def test_query_magnitudes(dtype, q_scale, qs):
    check(attn_case([400, 333], qs, 4, 2, 64, 32, dtype, "int8", seed=8, q_scale=q_scale))


@pytest.mark.parametrize("qs", [[1, 1], [1, 70]])
def test_zero_and_nonfinite_queries(qs):
    x = attn_case([400, 333], qs, 4, 2, 128, 32, BF16, "int8", seed=9)
    x["q"][0] = 0
    check(x)
    a, la = attend(x)
    x["q"][-1, 1] = math.nan
    b, lb = attend(x)
    assert b[-1, 1].isnan().all()            # that row alone
    keep = torch.ones(a.shape[:2], dtype=torch.bool)
    keep[-1, 1] = False
    assert torch.equal(a[keep], b[keep]) and torch.equal(la[keep], lb[keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("qs", [[1, 1, 1], [150, 7, 260]])
def test_strided_queries_streams_and_repeats(dtype, qs):
    x = attn_case([1500, 20, 300], qs, 8, 2, 128, 64, dtype, "e4m3", seed=10)
    a, la = attend(x)
    check(x, (a, la))
    wide = torch.zeros((sum(qs), 12, 128), dtype=dtype, device="cuda")
    wide[:, 2:10] = x["q"].cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = [x["kc"].view(CODE["e4m3"]).cuda(), x["vc"].view(CODE["e4m3"]).cuda(), x["ks"].cuda(), x["vs"].cuda(),
            x["table"].cuda(), i32(x["lens"])]
    need = gdr.kv8_attn_workspace_size(3, max(qs), sum(qs), 8, 2, 128, dtype)
    ws = torch.full((max(need, 16),), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            b, lb = gdr.kv8_attn(wide[:, 2:10], *args, x["scale"], cu_q=i32(x["cu"]), max_q=max(qs), want_lse=True,
                                 workspace=ws)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_rows_outside_requests_are_left_alone():
    for qs in ([1, 1], [40, 90]):
        x = attn_case([200, 300], qs, 4, 2, 64, 16, BF16, "int8", seed=11)
        q = torch.cat([x["q"], torch.full((5, 4, 64), math.nan, dtype=BF16)]).cuda()
        out = torch.full_like(q, 7.0)
        gdr.kv8_attn(q, x["kc"].view(torch.int8).cuda(), x["vc"].view(torch.int8).cuda(), x["ks"].cuda(),
                     x["vs"].cuda(), x["table"].cuda(), i32(x["lens"]), x["scale"], cu_q=i32(x["cu"]),
                     max_q=max(qs), out=out)
        n = sum(qs)
        assert (out[n:] == 7).all()
        assert oracle.rel_l2(out[:n], want(x)[0]) <= TOL[BF16]


def test_max_q_does_not_change_the_result():
    x = attn_case([300, 200, 90], [2, 1, 2], 8, 2, 128, 16, BF16, "e4m3", seed=12)
    ro = want(x)[0]
    for max_q in (2, 3, 200):
        out = gdr.kv8_attn(x["q"].cuda(), x["kc"].view(CODE["e4m3"]).cuda(), x["vc"].view(CODE["e4m3"]).cuda(),
                           x["ks"].cuda(), x["vs"].cuda(), x["table"].cuda(), i32(x["lens"]), x["scale"],
                           cu_q=i32(x["cu"]), max_q=max_q)
        assert oracle.rel_l2(out, ro) <= TOL[BF16]


def test_length_beyond_the_table_is_clamped():
    x = attn_case([64], [1], 2, 1, 64, 16, BF16, "int8", seed=13, slack=0)
    a, _ = attend(x)
    b, _ = attend(dict(x, lens=[70]))
    assert torch.equal(a, b)
    c, _ = attend(dict(x, lens=[-5]))
    assert (c == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[17], [700, 33, 0, 1290], [150000, 33]])
@pytest.mark.parametrize("rows", [8, 16, 24, 96, 320])
def test_injected_timeout_is_reported_and_recovers(dtype, lens, rows):
    """Every kernel of the attention with waits that give up at once (no fault, no hang): the
    error word says so, and the next call gives the results of the one before.  A wait that
    finds its data there is no timeout (short work, or fp32 whose products take longer than its
    loads): then the call's results stand."""
    x = attn_case(lens, [rows // 8] * len(lens), 16, 2, 128, 16, dtype, "e4m3", seed=rows)
    args = [x["q"].cuda(), x["kc"].view(CODE["e4m3"]).cuda(), x["vc"].view(CODE["e4m3"]).cuda(), x["ks"].cuda(),
            x["vs"].cuda(), x["table"].cuda(), i32(lens), x["scale"]]
    kw = dict(cu_q=i32(x["cu"]), max_q=rows // 8, want_lse=True)
    before = gdr.kv8_attn(*args, **kw)
    other = torch.ones(1 << 28, dtype=torch.uint8, device="cuda")    # nothing of the cache is in the L2
    assert gdr.last_device_error() == 0
    with gdr.option(wait_limit_ns=0):
        got = gdr.kv8_attn(*args, **kw)
        error = gdr.last_device_error()
    assert error == 5 or (error == 0 and (dtype == F32 or max(lens) < 2000))     # GDR_ERR_TIMEOUT
    assert gdr.last_device_error() == 0 and other[-1] == 1
    if error == 0:
        assert all(torch.equal(u, v) for u, v in zip(got, before))
    for u, v in zip(gdr.kv8_attn(*args, **kw), before):
        assert torch.equal(u, v)


@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,qs,Hq,Hkv,D,page", [
    ([33, 64, 500, 1], [3, 2, 4, 1], 16, 2, 128, 16),       # 8 to 32 rows: warps with whole, part and no rows
    ([1025, 31, 700], [9, 7, 8], 6, 2, 64, 32),             # 21 to 27 rows, tokens split by 3
    ([90, 3000], [17, 1], 4, 4, 128, 64),                   # one query head a cached head
    ([2000, 0, 64], [1, 1, 1], 64, 2, 64, 128),             # 32 rows of single tokens
])
def test_seventeen_to_thirty_two_rows(kv, lens, qs, Hq, Hkv, D, page):
    check(attn_case(lens, qs, Hq, Hkv, D, page, BF16, kv, seed=7 + D))
    check(attn_case(lens, qs, Hq, Hkv, D, page, BF16, kv, seed=8 + D, gone=0.3))


@pytest.mark.parametrize("S,q,kv_max", [(700, 1, 300), (700, 2, 200), (1100, 5, 150), (530, 20, 140)])
def test_many_requests(S, q, kv_max):
    """More requests than a CTA has threads, of no to a few units each, some without queries:
    the places that the CTAs find for themselves, and items that end where a CTA's share does."""
    r = random.Random(S + q)
    lens = [r.choice([0, 1, r.randint(0, kv_max), kv_max]) for _ in range(S)]
    qs = [1] * S if q == 1 else [r.choice([0, 1, q, q]) for _ in range(S)]
    qs[5] = q
    check(attn_case(lens, qs, 8, 1, 64, 16, BF16, "int8", seed=S))


@pytest.mark.slow
def test_offsets_past_32_bits():
    """A cache of over 2^32 bytes of keys: the request's pages lie at its end."""
    N, H, P, D = 270000, 2, 64, 128
    g = torch.Generator().manual_seed(14)
    small, ss = random_cache(40, H, P, D, "int8", g)
    kc = torch.zeros((N, H, P, D), dtype=torch.int8, device="cuda")
    vc = torch.zeros_like(kc)
    ks = torch.ones((N, H), device="cuda")
    vs = torch.ones((N, H), device="cuda")
    kc[-40:], vc[-40:] = small.view(torch.int8).cuda(), small.flip(0).contiguous().view(torch.int8).cuda()
    ks[-40:], vs[-40:] = ss.cuda() / 16, ss.flip(0).cuda()
    local = torch.randperm(40, generator=g).to(torch.int32)[None]
    for qs in ([1], [70]):
        q = torch.randn((qs[0], 8, D), generator=g).to(BF16)
        out = gdr.kv8_attn(q.cuda(), kc, vc, ks, vs, (local + N - 40).cuda(), i32([40 * P - 9]), 0.09,
                           cu_q=i32([0, qs[0]]), max_q=qs[0])
        ro, _ = O.attention(q.double().numpy(), small.numpy(), small.flip(0).numpy(), ss.double().numpy() / 16,
                            ss.flip(0).double().numpy(), local.numpy(), [40 * P - 9], [0, qs[0]], 0.09, "int8")
        assert oracle.rel_l2(out, ro) <= TOL[BF16]
    # and an append there
    x = torch.randn((3, H, D), generator=g).cuda()
    gdr.kv8_append(x, x, i32([(N - 1) * P + 7, (N - 1) * P + 8, (N - 1) * P + 9]), kc, vc, ks, vs)
    err = (kc[-1, :, 7:10].float() * ks[-1][:, None, None] - x.transpose(0, 1)).abs().amax()
    assert err <= 0.5 * float(ks[-1].max())


# ------------------------------------------------------------------ the three together
@pytest.mark.parametrize("kv,dtype", [("e4m3", BF16), ("int8", F32)])
def test_a_serving_loop(kv, dtype):
    """Prompts, chunks and single tokens through plan, append and attention; the cache the
    oracle keeps by itself from the same activations gives the same attention."""
    r = random.Random(1)
    S, W, P, H, G, D, N = 5, 12, 16, 2, 3, 64, 40
    g = torch.Generator().manual_seed(15)
    table = torch.full((S, W), -1, dtype=torch.int32, device="cuda")
    ring, state = i32(r.sample(range(N), N)), i32([11, N])
    kv_len = i32([0] * S)
    caches = [torch.zeros((N, H, P, D), dtype=CODE[kv], device="cuda") for _ in range(2)]
    scales = [torch.ones((N, H), device="cuda") for _ in range(2)]
    mine = [np.zeros((N, H, P, D), np.uint8) for _ in range(2)], [np.ones((N, H)) for _ in range(2)]
    for step in range(6):
        q_len = [33, 1, 0, 20, 7] if step == 0 else [1, 17, 40, -1, 1] if step == 2 else \
            [1, 1, 1, 5 * (step > 2), 3]
        T = sum(n for n in q_len if n > 0) + 2
        kv_len, cu, slots, pos, ok, state = gdr.page_plan(kv_len, i32(q_len), table, ring, state, P, T)
        assert ok.all()
        q = torch.randn((T, H * G, D), generator=g).to(dtype)
        x = [torch.randn((T, H, D), generator=g).to(dtype) for _ in range(2)]
        gdr.kv8_append(x[0].cuda(), x[1].cuda(), slots, *caches, *scales)
        out, lse = gdr.kv8_attn(q.cuda(), *caches, *scales, table, kv_len, 0.125, cu_q=cu,
                                max_q=max(q_len), want_lse=True)
        for i in range(2):
            O.append(x[i].double().numpy(), slots.tolist(), mine[0][i], mine[1][i], P, kv)
        n = int(cu[-1])
        ro, rl = O.attention(q.double().numpy(), *mine[0], *mine[1], table.cpu().numpy(), kv_len.tolist(),
                             cu.tolist(), 0.125, kv)
        assert oracle.rel_l2(out[:n], ro[:n]) <= TOL[dtype]
        assert np.abs(lse[:n].double().cpu().numpy() - rl[:n]).max() <= LSE_TOL * 10
