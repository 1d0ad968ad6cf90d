"""What the documentation of the norms with rotation allows besides: gradients written over the inputs, and the
weights' gradients held to the number of additions that the work's division gives.

A weight's gradient (u = 2^-24).  A term g x r: r 13.5 u, as in the forward, and 1 u for the product x r; g 3 u for
the rotation and 2^-23 for sine and cosine (bf16 2^-20): 19.5 u, 34.5 u with bf16, of max |g| sqrt(2) |x r|.  The
sum: a warp takes 512 / D rows at once (a pass), so a lane adds a term a pass; with P passes a warp, then
log2(512 / D) steps of lanes, 8 warps in turn, and of C CTAs' sums one of 32 warps adds every 32nd, in turn, then 5
steps: P + log2(512 / D) + 8 + ceil(C / 32) + 5 additions at most, each off by u of the terms' magnitudes."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
from test_norm_rope_gpu import CASES, backward, f64, freq_of, prepare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    yield
    torch.cuda.synchronize()
    assert gdr.last_device_error() == 0


def additions(T, heads, D, rot, which):
    """The most additions between a term and its weight's gradient: the CTAs go by four passes a warp while two
    CTAs an SM are enough for that, else they are shared out by cost, a pass and half a one where tokens begin."""
    rows = 512 // D
    passes = [-(-T * h // rows) for h in heads]
    ctas = [-(-p // 32) for p in passes]
    most = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    if sum(ctas) > most:
        cost = [2 * p + (min(p, T) if rot else 0) for p in passes]
        q = min(max((most * cost[0] + sum(cost) // 2) // sum(cost), 1), most - 1)
        ctas = [q, most - q]
    n = ctas[which]
    return -(-passes[which] // (8 * n)) + int(math.log2(rows)) + 8 + -(-n // 32) + 5


LONG = [
    (9000, 32, 8, 128, 128, "half", "rms", "bf16", True),
    (20000, 3, 1, 64, 32, "adjacent", "rms", "f32", True),
    (5000, 16, 16, 512, 0, "half", "l2", "f32", True),
]


@pytest.mark.parametrize("case", [c for c in CASES if c[-1]] + LONG, ids=lambda c: "-".join(map(str, c)))
def test_weights_gradients(case):
    T, Hq, Hk, D, rot, pairs, norm, dtype, _ = case
    q, k, gq, gk, how, cs = prepare(*case, seed=7)
    got = gdr.qk_norm_rope_bwd(q, k, gq, gk, **how)
    term = 34.5 if dtype == "bf16" and rot else 19.5
    for which, (x, g, w, dw) in enumerate(((q, gq, how["q_weight"], got[2]), (k, gk, how["k_weight"], got[3]))):
        _, want, _, size = backward(f64(x), f64(w), f64(g), norm, 1e-6, cs, pairs, rot)
        tol = (term + additions(T, (Hq, Hk), D, rot, which)) * 2.0 ** -24 * size
        assert (np.abs(f64(dw) - want) <= tol).all(), (which, (np.abs(f64(dw) - want) / tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(300, 6, 2, 64, 64), (3000, 32, 8, 128, 128), (777, 5, 3, 256, 0), (41, 3, 1, 16, 16)])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("onto", ["inputs", "gradients"])
def test_gradients_over_what_they_are_of(dtype, T, Hq, Hk, D, rot, weights, onto):
    """d_q, d_k over q and k themselves, or over d_q_out and d_k_out: slices of wider tensors, whose other columns
    stay.  The same bits as into tensors of their own."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x, y = (torch.randn((T, Hq + 2 * Hk + 1, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    sides = slice(1, 1 + Hq), slice(1 + Hq, 1 + Hq + Hk)
    pos = torch.randint(-3, 70000, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[::11] = -1
    how = dict(positions=pos, freq=freq_of(rot))
    if weights:
        how.update({n: torch.rand(D, generator=g, device="cuda") for n in ("q_weight", "k_weight")})
    a, b = x.clone(), y.clone()
    want = gdr.qk_norm_rope_bwd(*(x[:, s] for s in sides), *(y[:, s] for s in sides), **how)
    assert torch.equal(a, x) and torch.equal(b, y)
    over, kept = (x, a) if onto == "inputs" else (y, b)
    got = gdr.qk_norm_rope_bwd(*(x[:, s] for s in sides), *(y[:, s] for s in sides), d_q=over[:, sides[0]],
                               d_k=over[:, sides[1]], **how)
    assert all(torch.equal(over[:, s], w) for s, w in zip(sides, want))
    assert all((p is None and q is None) or torch.equal(p, q) for p, q in zip(got[2:], want[2:]))
    assert torch.equal(over[:, :1], kept[:, :1]) and torch.equal(over[:, 1 + Hq + Hk:], kept[:, 1 + Hq + Hk:])
