"""Refusals of the paged cache's entry points: host-only checks, nothing is launched."""
from __future__ import annotations

import ctypes

import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
from gated_delta_rule_gdr_gb300 import build as gbuild

P, P2 = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdr.load()


def call(fn, names, **kw):
    return fn(*(kw.get(n, d) for n, d in names))


PLAN = (("kv", P), ("q", P), ("table", P), ("ring", P), ("state", P), ("kvo", P2), ("cu", P), ("slots", P),
        ("pos", P), ("ok", P), ("sto", P2), ("S", 4), ("W", 8), ("page", 16), ("N", 100), ("T", 64), ("stream", None))


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(T=-1), 1), (dict(W=0), 1), (dict(N=0), 1),
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(S=8193), 2), (dict(T=2 ** 30 + 1), 2),
    (dict(N=2 ** 27, page=16), 2), (dict(W=2 ** 27), 2), (dict(S=8192, W=2 ** 19), 2),
    (dict(kv=None), 1), (dict(q=None), 1), (dict(table=None), 1), (dict(ring=None), 1), (dict(state=None), 1),
    (dict(kvo=None), 1), (dict(cu=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(ok=None), 1),
    (dict(sto=None), 1), (dict(kvo=P), 1), (dict(sto=P), 1),
])
def test_page_plan_rejects(lib, kw, code):
    assert call(lib.gdr_page_plan, PLAN, **kw) == code


APPEND = (("k", P), ("v", P), ("ks", 512), ("vs", 512), ("slots", P), ("kc", P), ("vc", P), ("ksc", P), ("vsc", P),
          ("T", 4), ("H", 4), ("D", 128), ("page", 16), ("N", 100), ("dtype", 1), ("kv", 0), ("stream", None))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=-1), 1), (dict(N=-1), 1), (dict(D=96), 2), (dict(D=256), 2), (dict(page=24), 2),
    (dict(dtype=2), 2), (dict(kv=2), 2), (dict(kv=-1), 2), (dict(N=2 ** 25, H=4), 2), (dict(H=4097), 2),
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(kc=None), 1), (dict(vsc=None), 1),
    (dict(ks=511), 1), (dict(vs=516), 1), (dict(ks=-512), 1), (dict(k=ODD), 1), (dict(vc=ODD), 1),
    (dict(T=0), 0), (dict(H=0), 0), (dict(N=0), 0),
])
def test_kv8_append_rejects(lib, kw, code):
    assert call(lib.gdr_kv8_append, APPEND, **kw) == code


ATTN = (("q", P), ("qs", 1024), ("kc", P), ("vc", P), ("ksc", P), ("vsc", P), ("table", P), ("kvl", P), ("cu", P),
        ("scale", 0.1), ("out", P), ("lse", None), ("S", 4), ("max_q", 3), ("T", 12), ("Hq", 8), ("Hkv", 2), ("D", 128),
        ("W", 8), ("page", 16), ("N", 100), ("dtype", 1), ("kv", 0), ("ws", P), ("wsb", 1 << 40), ("stream", None))


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), 1), (dict(max_q=-1), 1), (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(W=-1), 1), (dict(N=-1), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(D=32), 2), (dict(page=20), 2),
    (dict(dtype=5), 2), (dict(kv=3), 2), (dict(S=8193), 2), (dict(T=2 ** 28), 2), (dict(W=2 ** 27), 2),
    (dict(N=2 ** 26), 2), (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(W=0), 1), (dict(N=0), 1),
    (dict(cu=None), 1),                                        # one query a request wants max_q 1, total_q S
    (dict(cu=None, max_q=1, T=5), 1),
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ksc=None), 1), (dict(vsc=None), 1),
    (dict(table=None), 1), (dict(kvl=None), 1), (dict(out=None), 1), (dict(qs=1023), 1), (dict(qs=1028), 1),
    (dict(q=ODD), 1), (dict(kc=ODD), 1), (dict(out=ODD), 1),
    (dict(S=0), 0), (dict(T=0), 0), (dict(Hq=0), 0), (dict(max_q=0), 0),
])
def test_kv8_attn_rejects(lib, kw, code):
    assert call(lib.gdr_kv8_attn, ATTN, **kw) == code


def test_workspace_size(lib):
    f = lib.gdr_kv8_attn_workspace_size
    assert f(0, 1, 1, 8, 2, 128, 1) == 0 and f(1, 1, 1, 7, 2, 128, 1) == 0 and f(1, 1, 1, 8, 2, 96, 1) == 0
    need = f(4, 3, 12, 8, 2, 128, 1)
    assert need % 16 == 0
    if need:
        assert call(lib.gdr_kv8_attn, ATTN, wsb=need - 1) == 1
        assert call(lib.gdr_kv8_attn, ATTN, ws=None) == 1
        assert call(lib.gdr_kv8_attn, ATTN, ws=ODD) == 1


def test_binding_refuses(lib):
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        gdr.page_plan(i, i, torch.zeros((3, 4), dtype=torch.int32), i, i[:2], 16, 8)      # not on the GPU
    c = torch.zeros((4, 2, 16, 64), dtype=torch.int8)
    s = torch.ones((4, 2))
    x = torch.zeros((3, 2, 64))
    with pytest.raises(ValueError):
        gdr.kv8_append(x, x, i, c, c, s, s)
    with pytest.raises(TypeError):
        gdr.kv8_append(x, x, i, c.float(), c.float(), s, s)
    with pytest.raises(ValueError):
        gdr.kv8_attn(x, c, c, s, s, i[None], i, 0.1)
