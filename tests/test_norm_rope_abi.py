"""Refusals of the norms with rotation: host-only checks, nothing is launched."""
from __future__ import annotations

import ctypes

import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
from gated_delta_rule_gdr_gb300 import build as gbuild

P, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdr.load()


def call(fn, names, **kw):
    return fn(*(kw.get(n, d) for n, d in names))


HEAD = (("q", P), ("qs", 1024), ("k", P), ("ks", 256), ("qw", P), ("kw", P), ("eps", 1e-6), ("norm", 1), ("pos", P),
        ("freq", P), ("rot", 128), ("pairs", 0))
FWD = HEAD + (("qo", P), ("qos", 1024), ("ko", P), ("kos", 256), ("T", 4), ("Hq", 8), ("Hk", 2), ("D", 128),
              ("dtype", 1), ("stream", None))
BWD = HEAD + (("gq", P), ("gqs", 1024), ("gk", P), ("gks", 256), ("qo", P), ("qos", 1024), ("ko", P), ("kos", 256),
              ("dqw", P), ("dkw", P), ("T", 4), ("Hq", 8), ("Hk", 2), ("D", 128), ("dtype", 1), ("ws", P),
              ("wsb", 1 << 40), ("stream", None))

BOTH = [
    (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(Hk=-1), 1), (dict(rot=-16), 1), (dict(eps=-1e-6), 1), (dict(eps=NAN), 1),
    (dict(eps=INF), 1), (dict(norm=3), 1), (dict(norm=-1), 1), (dict(pairs=2), 1), (dict(pairs=-1), 1),
    (dict(D=96), 2), (dict(D=8), 2), (dict(D=1024), 2), (dict(D=0), 2), (dict(dtype=2), 2), (dict(Hq=65537), 2),
    (dict(rot=144), 2), (dict(rot=8), 2), (dict(rot=40), 2), (dict(pos=None), 1), (dict(freq=None), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(q=ODD), 1), (dict(ko=ODD), 1),
    (dict(qs=1023), 1), (dict(qs=1028), 1), (dict(ks=255), 1), (dict(qos=-1024), 1), (dict(kos=252), 1),
    (dict(qs=2 ** 40), 1), (dict(T=2 ** 30 + 1), 2),
]


@pytest.mark.parametrize("kw,code", BOTH + [(dict(T=0), 0), (dict(Hq=0, Hk=0), 0)])
def test_forward_rejects(lib, kw, code):
    assert call(lib.gdr_qk_norm_rope, FWD, **kw) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(gq=None), 1), (dict(gk=ODD), 1), (dict(gqs=1000), 1), (dict(ws=None), 1), (dict(ws=ODD), 1), (dict(wsb=0), 1),
    (dict(dkw=None, ws=None), 1), (dict(dqw=None, dkw=None, T=0, ws=None), 0),
    (dict(dqw=None, dkw=None, Hq=0, Hk=0, ws=None), 0),
])
def test_backward_rejects(lib, kw, code):
    assert call(lib.gdr_qk_norm_rope_bwd, BWD, **kw) == code


def test_workspace_size(lib):
    f = gdr.qk_norm_rope_bwd_workspace_size
    assert f(96) == 0 and f(8) == 0 and f(1024) == 0
    assert f(128) == 2 * f(64) > 0


def test_binding_refuses(lib):
    x = torch.zeros((3, 2, 64))
    with pytest.raises(ValueError):
        gdr.qk_norm_rope(x)                                   # not on the GPU
    with pytest.raises(TypeError):
        gdr.qk_norm_rope(x.half())
    with pytest.raises(ValueError):
        gdr.qk_norm_rope_bwd(x, None, x, None)
