"""Pins of the paged cache's oracle (CPU): facts that do not come from its own formulas."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import kv8 as O


def test_e4m3_values_and_rounding():
    v = O.e4m3_values()
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, ref, equal_nan=True)
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-10, 8, 4000), v[~np.isnan(v)],
                        (_mid := (O._POS[1:] + O._POS[:-1]) / 2), -_mid])
    y = np.clip(y, -448, 448).astype(np.float32)
    ref = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.encode(y.astype(np.float64), "e4m3"), ref)
    assert O.encode(np.array([math.inf, -math.inf, math.nan]), "e4m3").tolist() == [0x7e, 0xfe, 0]


def test_int8_rounding():
    y = np.array([0.5, 1.5, -0.5, -2.5, 126.6, 1e9, -1e9, math.nan])
    assert O.encode(y, "int8").view(np.int8).tolist() == [0, 2, 0, -2, 127, 127, -127, 0]


@pytest.mark.parametrize("kv,q", [("e4m3", 448.0), ("int8", 127.0)])
def test_scale_is_the_least_power_of_two(kv, q):
    for amax in (1e-30, 1e-3, 0.9, 1.0, q, q * 2, np.nextafter(q, 1e9), 12345.0):
        s = O.scale_for(amax, kv)
        assert math.frexp(s)[0] == 0.5 and amax <= q * s
        assert s == 2.0 ** -40 or amax > q * s / 2
    assert O.scale_for(0.0, kv) == 2.0 ** -40 and O.scale_for(1e30, kv) == 2.0 ** 40


def test_plan_by_hand():
    # pages of 16: request 0 has 15 tokens (1 page), 2 new cross into a page; request 1 is
    # finished with 2 pages; request 2 is new with 33 tokens (3 pages)
    table = np.full((3, 4), -1)
    table[0, 0], table[1, :2] = 7, (5, 6)
    ring = np.array([-1, -1, 0, 1, 2, 3, -1, -1])
    kv, cu, slots, pos, ok, st, tab, rg = O.plan([15, 20, 0], [2, -1, 33], table, ring, [2, 4], 16, 40)
    assert kv == [17, 0, 33] and cu == [0, 2, 2, 35] and ok == [1, 1, 1]
    assert slots[:2].tolist() == [7 * 16 + 15, 0 * 16]
    assert slots[2] == 1 * 16 and slots[18] == 2 * 16 and slots[34] == 3 * 16 and slots[35] == -1
    assert pos[:3].tolist() == [15, 16, 0] and st == [6, 2]
    assert rg.tolist() == [-1, -1, 0, 1, 2, 3, 5, 6] and tab[2].tolist() == [1, 2, 3, -1]
    # one page short: request 2 gets nothing, request 0 keeps its grant
    kv, cu, slots, pos, ok, st, _, _ = O.plan([15, 20, 0], [2, -1, 33], table, ring, [2, 3], 16, 40)
    assert ok == [1, 1, 0] and kv == [17, 0, 0] and st == [3, 4] and (slots[2:] == -1).all()


def test_attention_limits():
    rng = np.random.default_rng(1)
    N, H, P, D = 4, 1, 16, 64
    kc = O.encode(rng.normal(size=(N, H, P, D)), "e4m3")
    vc = O.encode(rng.normal(size=(N, H, P, D)), "e4m3")
    ks, vs = np.full((N, H), 2.0), np.full((N, H), 0.5)
    table = np.array([[2, 0, -1]])
    # zero queries: the mean of the visible values; lse = ln(count)
    out, lse = O.attention(np.zeros((2, 2, D)), kc, vc, ks, vs, table, [20], [0, 2], 0.125, "e4m3")
    v = 0.5 * np.concatenate([O.decode(vc[2, 0], "e4m3"), O.decode(vc[0, 0, :4], "e4m3")])
    assert np.allclose(out[1], v.mean(0)) and np.allclose(out[0], v[:19].mean(0))
    assert np.allclose(lse, np.log([[19, 19], [20, 20]]))
    # one visible key: its value exactly, lse its score
    q = rng.normal(size=(1, 1, D))
    out, lse = O.attention(q, kc, vc, ks, vs, table, [1], [0, 1], 0.125, "e4m3")
    assert np.allclose(out[0, 0], v[0])
    assert np.isclose(lse[0, 0], 0.125 * 2.0 * O.decode(kc[2, 0, 0], "e4m3") @ q[0, 0])
    # nothing visible: more queries than keys, and a page that is gone
    out, lse = O.attention(np.ones((3, 1, D)), kc, vc, ks, vs, table, [1], [0, 3], 1.0, "e4m3")
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all() and np.isfinite(lse[2])
    out, lse = O.attention(np.ones((1, 1, D)), kc, vc, ks, vs, np.array([[-1, 9]]), [18], [0, 1], 1.0, "e4m3")
    assert (out == 0).all() and (lse == -math.inf).all()


def test_append_restarts_and_rescales():
    codes = O.encode(np.full((2, 1, 16, 64), 4.0), "int8")
    scale = np.ones((2, 1))
    x = np.full((3, 1, 64), 1.0)
    x[2] = 1000.0                                            # needs 2^3 (127 * 8 >= 1000)
    O.append(x, [2, 3, 16], codes, scale, 16, "int8")
    assert scale[:, 0].tolist() == [1.0, 8.0]                # page 0 keeps its larger scale
    assert codes[0, 0, :4, 0].tolist() == [4, 4, 1, 1] and codes[1, 0, 0, 0] == 125
    O.append(np.full((1, 1, 64), 500.0), [4], codes, scale, 16, "int8")
    assert scale[0, 0] == 4.0 and codes[0, 0, :5, 0].tolist() == [1, 1, 0, 0, 125]
