"""Refusals of the attention of requests that share a prefix and of its plan: host-only checks."""
from __future__ import annotations

import ctypes

import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
from gated_delta_rule_gdr_gb300 import build as gbuild

P, P2, P3, ODD = (ctypes.c_void_p(0x1000 * i) for i in (1, 2, 3, 1))
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdr.load()


def call(fn, names, **kw):
    return fn(*(kw.get(n, d) for n, d in names))


PLAN = (("table", P), ("kv", P), ("cu", P), ("group", P), ("shared", P2), ("lead", P3), ("S", 4), ("NG", 2), ("W", 8),
        ("page", 16), ("stream", None))


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(NG=-1), 1), (dict(W=-1), 1), (dict(S=0), 1), (dict(NG=0), 1), (dict(W=0), 1), (dict(S=0, NG=0), 0),
    (dict(page=8), 2), (dict(page=48), 2), (dict(S=8193), 2), (dict(NG=8193), 2), (dict(W=2 ** 27), 2),
    (dict(table=None), 1), (dict(kv=None), 1), (dict(group=None), 1), (dict(shared=None), 1), (dict(lead=None), 1),
    (dict(shared=P), 1), (dict(lead=P), 1), (dict(lead=P2), 1),
])
def test_plan_rejects(lib, kw, code):
    assert call(lib.gdr_kv8_shared_plan, PLAN, **kw) == code


ATTN = (("q", P), ("qs", 1024), ("kc", P), ("vc", P), ("ksc", P), ("vsc", P), ("table", P), ("kvl", P), ("cu", P),
        ("group", P), ("shared", P), ("lead", P), ("scale", 0.1), ("out", P), ("lse", None), ("S", 4), ("max_q", 3),
        ("NG", 2), ("mg", 6), ("T", 12), ("Hq", 8), ("Hkv", 2), ("D", 128), ("W", 8), ("page", 16), ("N", 100),
        ("dtype", 1), ("kv", 0), ("ws", P), ("wsb", 1 << 40), ("stream", None))


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(max_q=-1), 1), (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(W=-1), 1), (dict(N=-1), 1),
    (dict(NG=-1), 1), (dict(mg=-1), 1), (dict(NG=0), 1), (dict(mg=0), 1), (dict(NG=8193), 2),
    (dict(scale=float("nan")), 1), (dict(D=32), 2), (dict(page=20), 2), (dict(dtype=5), 2), (dict(kv=3), 2),
    (dict(S=8193), 2), (dict(T=2 ** 28), 2), (dict(W=2 ** 27), 2), (dict(N=2 ** 26), 2), (dict(Hq=7), 1), (dict(Hkv=0), 1),
    (dict(W=0), 1), (dict(N=0), 1), (dict(cu=None), 1), (dict(cu=None, max_q=1, T=5), 1),
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vsc=None), 1), (dict(table=None), 1), (dict(kvl=None), 1),
    (dict(group=None), 1), (dict(shared=None), 1), (dict(lead=None), 1), (dict(out=None), 1), (dict(qs=1023), 1),
    (dict(qs=1028), 1), (dict(q=ODD), 1), (dict(kc=ODD), 1), (dict(out=ODD), 1), (dict(ws=None), 1), (dict(ws=ODD), 1),
    (dict(wsb=0), 1), (dict(S=0), 0), (dict(T=0), 0), (dict(Hq=0), 0), (dict(max_q=0), 0),
])
def test_attention_rejects(lib, kw, code):
    assert call(lib.gdr_kv8_attn_shared, ATTN, **kw) == code


def test_workspace_size(lib):
    f = lib.gdr_kv8_attn_shared_workspace_size
    assert f(0, 1, 1, 1, 1, 8, 2, 128, 1) == 0 and f(4, 1, 0, 4, 4, 8, 2, 128, 1) == 0 and f(4, 1, 1, 4, 4, 7, 2, 128, 1) == 0
    need = f(4, 3, 2, 6, 12, 8, 2, 128, 1)
    assert need >= 12 * 8 * 130 * 4 and need % 16 == 0
    assert call(lib.gdr_kv8_attn_shared, ATTN, wsb=need - 1) == 1


def test_binding_refuses(lib):
    i = torch.zeros(3, dtype=torch.int32)
    c = torch.zeros((4, 2, 16, 64), dtype=torch.int8)
    s, x = torch.ones((4, 2)), torch.zeros((3, 2, 64))
    with pytest.raises(TypeError):
        gdr.kv8_shared_plan(i[None], i[:1], i[:2], 16)                       # not on the GPU
    with pytest.raises(ValueError):
        gdr.kv8_attn_shared(x, c, c, s, s, i[None], i[:1], 0.1, i[:2], i[:1], i[:1], max_group_q=1)
