"""Refusals of gdr_page_plan_ex: host-only checks, nothing is launched."""
from __future__ import annotations

import ctypes

import pytest

import gated_delta_rule_gdr_gb300 as gdr
from gated_delta_rule_gdr_gb300 import build as gbuild

A, B, C = (ctypes.c_void_p(0x1000 * i) for i in (1, 2, 3))
ARGS = (("kv", A), ("q", A), ("held", A), ("table", A), ("ring", A), ("state", A), ("kvo", B), ("cu", A), ("slots", A),
        ("pos", A), ("ok", A), ("heldo", B), ("sto", B), ("S", 4), ("W", 8), ("page", 16), ("N", 100), ("T", 64),
        ("stream", None))


@pytest.mark.parametrize("kw,code", [
    (dict(heldo=None), 1), (dict(heldo=A), 1), (dict(held=B), 1), (dict(held=C, heldo=C), 1),
    (dict(kv=None), 1), (dict(q=None), 1), (dict(sto=A), 1), (dict(S=-1), 1), (dict(page=24), 2), (dict(S=8193), 2),
])
def test_page_plan_ex_rejects(kw, code):
    gbuild.build()
    assert gdr.load().gdr_page_plan_ex(*(kw.get(n, d) for n, d in ARGS)) == code
