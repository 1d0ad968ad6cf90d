"""Norms of queries and keys with the rotation, forward and backward, against the definitions in 64
bits (numpy) and, for the gradients, against differences of the 64-bit forward.

Tolerances (u = 2^-24, an fp32 rounding).  A sum over a head is a chain of 16 additions and a tree of
at most 5: 21 u of the sum of magnitudes.  Forward: the factor r takes half of that and 3 u of its own
(4 with the hardware's root), the products 2 u, the rotation 3 u and the sine and cosine 2^-23 (fp32,
the angle's 2^-25 included) or 2^-20 (bf16): 19 u + 2^-23 below 2^-19 and 19 u + 2^-20 below 2^-18 of the
row's largest weighted value times sqrt(2) (a pair's length), and one rounding of the result: 2^-24 or 2^-8
of it.  Backward: g as above; the row's sum <w g, x> 21 u and g's own error, r^3 another 3 (10.5 + 3) u, 6
products: 75 u + 2^-20 below 2^-17 of r max |w g| + max |x| r^3 max |w g| sum |x| / N.  Weights'
gradients: a term's error is 19 u + 2^-20 below 2^-18 of max |g| |x r|; a thread adds at most T H / 1000
terms (the tensors here have 240 warps or more), then 5 lanes' steps, 8 warps, at most 76 CTAs' sums in a
thread and 64 of those: 128 + T H / 1000 additions, u of the sum of magnitudes each."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    yield
    torch.cuda.synchronize()
    assert gdr.last_device_error() == 0


def angles(pos, freq):
    """cos, sin [T, 1, rot / 2] of pos * freq; the product's whole turns come off exactly enough: 2^31
    positions times a 53-bit frequency is off by 2^-22 radians at most, so long doubles are used."""
    a = pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)
    return np.cos(a).astype(np.float64)[:, None], np.sin(a).astype(np.float64)[:, None]


def turn(x, cs, pairs, rot, back=False):
    if not rot:
        return x
    c, s = cs
    s = -s if back else s
    y = x.copy()
    ia, ib = (slice(0, rot // 2), slice(rot // 2, rot)) if pairs == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def factor(x, norm, eps):
    if norm == "none":
        return np.ones(x.shape[:-1] + (1,))
    n = x.shape[-1] if norm == "rms" else 1
    return 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)


def forward(x, w, norm, eps, cs, pairs, rot):
    return turn(x * factor(x, norm, eps) * w, cs, pairs, rot)


def backward(x, w, g, norm, eps, cs, pairs, rot):
    """dx, dw, and bounds of the magnitudes that dx and dw are sums of."""
    r = factor(x, norm, eps)
    g0 = g
    g = turn(g, cs, pairs, rot, back=True)
    dw = (g * x * r).sum((0, 1))
    g = g * w
    big = np.abs(g).max(-1, keepdims=True) * r
    size = (np.abs(g0).max(-1, keepdims=True) * math.sqrt(2) * np.abs(x) * r).sum((0, 1))
    if norm == "none":
        return g, dw, big, size
    n = x.shape[-1] if norm == "rms" else 1
    dot = (g * x).sum(-1, keepdims=True) / n
    big = big + (np.abs(x).max(-1, keepdims=True) * r ** 3 * np.abs(g).max(-1, keepdims=True)
                 * np.abs(x).sum(-1, keepdims=True) / n)
    return r * g - x * r ** 3 * dot, dw, big, size


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, Hq, Hk, D, dtype, seed=0, packed=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hq + 2 * Hk + 1, D), generator=g) * torch.exp(torch.randn((T, 1, 1), generator=g))
    x = x.to(DT[dtype]).cuda()
    q, k = x[:, 1:1 + Hq], x[:, 1 + Hq:1 + Hq + Hk]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    gq, gk = (torch.randn((T, h, D), generator=g).to(DT[dtype]).cuda() for h in (Hq, Hk))
    return q, k, wq, wk, gq, gk


def freq_of(rot, theta=10000.0):
    return (theta ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)).cuda() if rot else None


def near(got, want, size, dtype, bits):
    """|got - want| within one rounding of the value and 2^-bits of `size`."""
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    off = np.abs(f64(got) - want) - (np.abs(want) * step + size * 2.0 ** -bits + 1e-38)
    assert off.max(initial=-1) <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))


CASES = [
    # T, Hq, Hk, D, rot, pairs, norm, dtype, weights
    (1, 1, 1, 128, 128, "half", "rms", "bf16", True),
    (1, 32, 8, 128, 128, "half", "rms", "bf16", True),
    (5, 7, 3, 128, 64, "half", "rms", "bf16", True),
    (33, 6, 2, 64, 32, "adjacent", "rms", "f32", True),
    (200, 3, 1, 64, 64, "adjacent", "none", "bf16", False),
    (77, 4, 4, 32, 32, "half", "l2", "f32", False),
    (130, 5, 2, 16, 16, "half", "rms", "bf16", True),
    (130, 5, 2, 16, 16, "adjacent", "rms", "f32", False),
    (19, 2, 1, 512, 64, "half", "rms", "bf16", True),
    (19, 2, 1, 512, 512, "adjacent", "rms", "f32", True),
    (41, 9, 5, 256, 240, "half", "none", "f32", True),
    (3000, 16, 16, 128, 0, "half", "l2", "bf16", False),
    (2000, 33, 1, 128, 128, "half", "rms", "bf16", True),
    (2000, 1, 33, 128, 112, "adjacent", "rms", "f32", True),
    (9000, 8, 2, 64, 64, "half", "rms", "bf16", False),
    (3001, 1, 2, 128, 128, "half", "rms", "bf16", True),         # rows of several tokens in a warp's pass
    (777, 3, 5, 32, 32, "adjacent", "rms", "f32", True),
    (1500, 7, 1, 16, 16, "half", "l2", "bf16", False),
    (400, 3, 3, 256, 128, "half", "rms", "f32", True),
]


def prepare(T, Hq, Hk, D, rot, pairs, norm, dtype, weights, seed=0):
    q, k, wq, wk, gq, gk = make(T, Hq, Hk, D, dtype, seed)
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(seed + 1), dtype=torch.int32).cuda()
    how = dict(norm=norm, eps=1e-6, pairs=pairs, positions=pos if rot else None, freq=freq_of(rot))
    if weights:
        how.update(q_weight=wq, k_weight=wk)
    cs = angles(pos.cpu().numpy(), f64(how["freq"])) if rot else None
    return q, k, gq, gk, how, cs


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward(case):
    T, Hq, Hk, D, rot, pairs, norm, dtype, weights = case
    q, k, _, _, how, cs = prepare(*case)
    got = gdr.qk_norm_rope(q, k, **how)
    for x, w, y in ((q, how.get("q_weight"), got[0]), (k, how.get("k_weight"), got[1])):
        w = np.ones(D) if w is None else f64(w)
        want = forward(f64(x), w, norm, 1e-6, cs, pairs, rot)
        near(y, want, np.abs(want).max(-1, keepdims=True) * math.sqrt(2), dtype, 18 if dtype == "bf16" else 19)
        assert y.is_contiguous() and y.dtype is x.dtype


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_backward(case):
    T, Hq, Hk, D, rot, pairs, norm, dtype, weights = case
    q, k, gq, gk, how, cs = prepare(*case)
    dq, dk, dwq, dwk = gdr.qk_norm_rope_bwd(q, k, gq, gk, **how)
    for x, g, w, dx, dw, H in ((q, gq, how.get("q_weight"), dq, dwq, Hq), (k, gk, how.get("k_weight"), dk, dwk, Hk)):
        want, wdw, big, size = backward(f64(x), np.ones(D) if w is None else f64(w), f64(g), norm, 1e-6, cs, pairs, rot)
        near(dx, want, big * math.sqrt(2), dtype, 17)
        if w is None:
            assert dw is None
        else:
            assert (np.abs(f64(dw) - wdw) <= ((T * H / 1000 + 128) * 2.0 ** -24 + 2.0 ** -18) * size).all()


def test_gradient_is_that_of_differences():
    """The formula that the gradients are tested against, against central differences of the forward."""
    rng = np.random.default_rng(3)
    for norm in ("rms", "l2", "none"):
        for pairs in ("half", "adjacent"):
            x, w, g = rng.standard_normal((2, 2, 16)), rng.standard_normal(16), rng.standard_normal((2, 2, 16))
            cs = angles(np.array([3, 70000]), 100.0 ** -np.linspace(0, 1, 8))
            loss = lambda x, w: (forward(x, w, norm, 1e-3, cs, pairs, 16) * g).sum()  # noqa: E731
            dx, dw, _, _ = backward(x, w, g, norm, 1e-3, cs, pairs, 16)
            for _ in range(5):
                ex, ew, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-5
                diff = (loss(x + h * ex, w + h * ew) - loss(x - h * ex, w - h * ew)) / (2 * h)
                assert abs(diff - (dx * ex).sum() - (dw * ew).sum()) <= 1e-7 * max(1.0, abs(diff))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_positions(dtype):
    """The last position there is, with frequencies from a radian down."""
    T, D = 64, 128
    q, _, _, _, _, _ = make(T, 2, 1, D, dtype)
    pos = torch.tensor([2 ** 31 - 1 - i for i in range(T)], dtype=torch.int32).cuda()
    freq = freq_of(D, 1e6)
    y, none = gdr.qk_norm_rope(q, norm="none", positions=pos, freq=freq)
    assert none is None
    cs = angles(pos.cpu().numpy(), f64(freq))
    want = turn(f64(q), cs, "half", D)
    near(y, want, np.abs(f64(q)).max(-1, keepdims=True) * math.sqrt(2), dtype, 18 if dtype == "bf16" else 19)


@pytest.mark.parametrize("rot", [0, 64])
def test_rows_that_are_no_tokens(rot):
    q, k, wq, wk, gq, gk = make(50, 4, 2, 128, "bf16")
    pos = torch.arange(50, dtype=torch.int32).cuda()
    gone = torch.arange(50).cuda() % 7 == 3
    pos[gone] = -1
    q2, k2 = q.clone(), k.clone()
    q2[gone] = math.nan
    how = dict(q_weight=wq, k_weight=wk, positions=pos, freq=freq_of(rot))
    qo, ko = torch.full_like(q2, 7.0), torch.full_like(k2, 7.0)
    gdr.qk_norm_rope(q2, k2, q_out=qo, k_out=ko, **how)
    assert (qo[gone] == 7).all() and (ko[gone] == 7).all()
    a, b = gdr.qk_norm_rope(q, k, **how)
    assert torch.equal(qo[~gone], a[~gone]) and torch.equal(ko[~gone], b[~gone])
    dq, dk, dwq, dwk = gdr.qk_norm_rope_bwd(q2, k2, gq, gk, **how)
    assert (dq[gone] == 0).all() and (dk[gone] == 0).all()
    keep = dict(how, positions=pos[~gone].contiguous())
    eq, ek, ewq, ewk = gdr.qk_norm_rope_bwd(q[~gone].contiguous(), k[~gone].contiguous(), gq[~gone].contiguous(),
                                            gk[~gone].contiguous(), **keep)
    assert torch.equal(dq[~gone], eq) and torch.equal(dk[~gone], ek)
    assert torch.allclose(dwq, ewq, rtol=1e-5, atol=1e-4) and torch.allclose(dwk, ewk, rtol=1e-5, atol=1e-4)


def test_in_place_and_strides():
    """Slices of one projection turned where they are; other columns stay; gradients onto the given ones."""
    T, Hq, Hk, D = 300, 6, 2, 64
    x = torch.randn((T, Hq + 2 * Hk, D), device="cuda").bfloat16()
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), freq_of(64)
    want = gdr.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hk], positions=pos, freq=freq)
    y = x.clone()
    gdr.qk_norm_rope(y[:, :Hq], y[:, Hq:Hq + Hk], positions=pos, freq=freq, q_out=y[:, :Hq], k_out=y[:, Hq:Hq + Hk])
    assert torch.equal(y[:, :Hq], want[0]) and torch.equal(y[:, Hq:Hq + Hk], want[1])
    assert torch.equal(y[:, Hq + Hk:], x[:, Hq + Hk:])
    gq, gk = torch.randn_like(x[:, :Hq]), torch.randn_like(x[:, :Hk])
    want = gdr.qk_norm_rope_bwd(x[:, :Hq], x[:, Hq:Hq + Hk], gq, gk, positions=pos, freq=freq)
    z = torch.cat([gq, gk], 1)
    gdr.qk_norm_rope_bwd(x[:, :Hq], x[:, Hq:Hq + Hk], z[:, :Hq], z[:, Hq:], positions=pos, freq=freq, d_q=z[:, :Hq],
                         d_k=z[:, Hq:])
    assert torch.equal(z[:, :Hq], want[0]) and torch.equal(z[:, Hq:], want[1])


def test_values_that_are_not_finite_stay_in_their_row():
    """An infinity among the values that are not turned reaches no other value without a norm, and no
    other row with one; rows of zeros give zeros, and gradients as the formula has them."""
    q, _, _, _, gq, _ = make(9, 3, 1, 64, "f32")
    q = q.contiguous()
    pos, freq = torch.arange(9, dtype=torch.int32).cuda(), freq_of(32)
    ref, _ = gdr.qk_norm_rope(q, norm="none", positions=pos, freq=freq)
    q[4, 1, 40] = math.inf
    y, _ = gdr.qk_norm_rope(q, norm="none", positions=pos, freq=freq)
    assert y[4, 1, 40] == math.inf
    y[4, 1, 40] = ref[4, 1, 40]
    assert torch.equal(y, ref)
    ref, _ = gdr.qk_norm_rope(q, positions=pos, freq=freq)
    q[4, 1] = 0
    y, _ = gdr.qk_norm_rope(q, positions=pos, freq=freq)
    assert (y[4, 1] == 0).all()
    keep = torch.ones((9, 3), dtype=torch.bool, device="cuda")
    keep[4, 1] = False
    assert torch.equal(y[keep], ref[keep])
    dq, _, _, _ = gdr.qk_norm_rope_bwd(q, None, gq, None, positions=pos, freq=freq)
    want = turn(f64(gq), angles(np.arange(9), f64(freq)), "half", 32, back=True)[4, 1] * 1e3
    assert np.abs(f64(dq[4, 1]) - want).max() <= 2.0 ** -19 * np.abs(want).max() * math.sqrt(2)


def test_no_tokens_and_no_heads():
    w = torch.ones(64, device="cuda")
    x = torch.zeros((0, 4, 64), device="cuda")
    q, k = gdr.qk_norm_rope(x, x[:, :2], q_weight=w)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    dq, dk, dwq, dwk = gdr.qk_norm_rope_bwd(x, x[:, :2], x, x[:, :2], q_weight=w, k_weight=w)
    assert (dwq == 0).all() and (dwk == 0).all() and dq.shape == (0, 4, 64)
    x = torch.ones((5, 0, 64), device="cuda")
    y = torch.ones((5, 3, 64), device="cuda")
    q, k = gdr.qk_norm_rope(x, y, norm="l2", eps=0.0)
    assert q.shape == (5, 0, 64) and torch.allclose(k, torch.full_like(k, 0.125))
    _, dk, dwq, dwk = gdr.qk_norm_rope_bwd(x, y, x, y, q_weight=w, k_weight=w)
    assert (dwq == 0).all() and torch.isfinite(dwk).all()


def test_repeats_streams_and_graphs():
    """The same bits every time, on another stream, and replayed; two captures share a workspace in turn."""
    q, k, wq, wk, gq, gk = make(700, 8, 2, 128, "bf16")
    pos = torch.arange(700, dtype=torch.int32).cuda()
    how = dict(q_weight=wq, k_weight=wk, positions=pos, freq=freq_of(128))
    ws = torch.empty(gdr.qk_norm_rope_bwd_workspace_size(128), dtype=torch.uint8, device="cuda")
    want = [*gdr.qk_norm_rope(q, k, **how), *gdr.qk_norm_rope_bwd(q, k, gq, gk, workspace=ws, **how)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [*gdr.qk_norm_rope(q, k, **how), *gdr.qk_norm_rope_bwd(q, k, gq, gk, workspace=ws, **how)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [*gdr.qk_norm_rope(q, k, **how), *gdr.qk_norm_rope_bwd(q, k, gq, gk, workspace=ws, **how)]
        graphs.append((g, out))
    for _ in range(2):
        for g, out in graphs:
            for t in out:
                t.zero_()
            ws.fill_(255)
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_another_device(monkeypatch):
    """Tensors that are not on the current device are refused (the current one is made out to be another)."""
    q, k, wq, wk, gq, gk = make(5, 2, 1, 64, "bf16")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        gdr.qk_norm_rope(q, k)
    with pytest.raises(ValueError, match="current device"):
        gdr.qk_norm_rope_bwd(q, k, gq, gk)
    monkeypatch.undo()
    with pytest.raises(TypeError):
        gdr.qk_norm_rope(q, k, q_weight=wq.cpu())


def test_offsets_past_32_bits():
    """A tensor of more than 2^31 values, in place: its last tokens as they are alone."""
    H, D, extra = 32, 128, 70
    T = 2 ** 31 // (H * D) + extra
    x = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    x[-extra:] = torch.randn((extra, H, D), device="cuda")
    x[:extra] = torch.randn((extra, H, D), device="cuda")
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), freq_of(D)
    ends = [gdr.qk_norm_rope(x[s].clone(), positions=pos[s].clone(), freq=freq)[0] for s in (slice(0, extra), slice(T - extra, T))]
    g = [torch.randn((extra, H, D), device="cuda").bfloat16() for _ in range(2)]
    dx = [gdr.qk_norm_rope_bwd(x[s].clone(), None, y, None, positions=pos[s].clone(), freq=freq)[0]
          for s, y in zip((slice(0, extra), slice(T - extra, T)), g)]
    d = torch.zeros_like(x)
    d[:extra], d[-extra:] = g
    gdr.qk_norm_rope_bwd(x, None, d, None, positions=pos, freq=freq, d_q=d)
    assert torch.equal(d[:extra], dx[0]) and torch.equal(d[-extra:], dx[1]) and (d[extra:-extra] == 0).all()
    gdr.qk_norm_rope(x, positions=pos, freq=freq, q_out=x)
    assert torch.equal(x[:extra], ends[0]) and torch.equal(x[-extra:], ends[1]) and (x[extra:-extra] == 0).all()
