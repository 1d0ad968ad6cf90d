"""Pins of the plan's oracle (CPU), by hand: gone pages, lengths beyond the table, held pages."""
from __future__ import annotations

import numpy as np

from oracle import kv8 as O


def test_gone_pages_stay_out_of_the_ring():
    table, ring = np.array([[5, -1, 6, 9], [-1] * 4]), np.array([0, 1, 2, 3, -1, -1, -1, -1])
    kv, _, slots, _, ok, state, tab, rg = O.plan([64, 0], [-1, 20], table, ring, [0, 4], 16, 20)
    assert kv == [0, 20] and ok == [1, 1] and state == [2, 4]              # 9 is no page of 8
    assert rg.tolist() == [0, 1, 2, 3, 5, 6, -1, -1] and tab[1].tolist() == [0, 1, -1, -1]
    assert slots.tolist() == list(range(20))


def test_tokens_of_a_gone_page_have_no_place():
    _, _, slots, pos, ok, _, _, _ = O.plan([10], [8], np.array([[1 << 26, -1]]), np.array([1, 0]), [0, 1], 16, 8)
    assert ok == [1] and slots.tolist() == [-1] * 6 + [16, 17] and pos.tolist() == [-1] * 6 + [16, 17]


def test_lengths_beyond_the_table():
    kv, _, _, _, ok, state, _, rg = O.plan([33, 40, 32], [0, -1, 0], np.array([[0, 1], [2, 3], [4, 5]]), np.full(6, -1),
                                           [0, 0], 16, 4)
    assert kv == [33, 0, 32] and ok == [0, 1, 1] and state == [0, 2] and rg[:2].tolist() == [2, 3]


def test_held_pages():
    table, ring = np.array([[3, 7, -1], [1, 2, 0]]), np.array([4, 5, 6, -1, -1, -1, -1, -1])
    out = O.plan([15, 1], [3, -1], table, ring, [0, 3], 16, 3, held=[2, 3])
    assert out[2].tolist() == [63, 112, 113] and out[5] == [0, 6] and out[8] == [2, 0]
    assert out[7].tolist() == [4, 5, 6, 1, 2, 0, -1, -1] and out[6][0].tolist() == [3, 7, -1]
    out = O.plan([15, 1], [20, 0], table, ring, [0, 3], 16, 20, held=[2, 0])     # 35 tokens: a third page
    assert out[6][0].tolist() == [3, 7, 4] and out[8] == [3, 1] and out[5] == [1, 2]
