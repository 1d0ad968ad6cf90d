"""kv8_attn on the GPU, row by row: a row's result depends on no other row, on no bound that the
caller gives for the lengths, and holds where the largest weight's value is nothing.

Tolerances.  A bf16 output is rounded once (uniform in half a unit of the last of 8 bits: at
most 2^-7 / sqrt(12) = 2.26e-3 in relative L2) and its weights to 11 bits (at most 2^-11): 3e-3,
of every row; fp32: 1e-5, the library's."""
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
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    yield
    assert gdr.last_device_error() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def case(lens, qs, Hq, Hkv, D, page, dtype, kv, seed):
    """Normal queries over caches of any codes but NaN; scores of standard deviation about 1."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    N = sum(need)
    order, at = torch.randperm(N, generator=g).to(torch.int32), 0
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    codes = []
    for _ in range(2):
        c = torch.randint(0, 256, (N, Hkv, page, D), dtype=torch.uint8, generator=g)
        c[(c & 0x7f) == 0x7f] = 0x30
        codes.append(c)
    ks = torch.full((N, Hkv), 2.0 ** -6 if kv == "int8" else 2.0 ** -7)
    vs = torch.exp2(torch.randint(-1, 2, (N, Hkv), generator=g).float())
    return dict(q=torch.randn((sum(qs), Hq, D), generator=g).to(dtype), kc=codes[0], vc=codes[1], ks=ks, vs=vs,
                table=table, lens=lens, cu=[sum(qs[:i]) for i in range(len(qs) + 1)], kv=kv, scale=1 / math.sqrt(D))


def attend(x, **kw):
    a = [x[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "table")]
    a[1:3] = [t.view(CODE[x["kv"]]) for t in a[1:3]]
    out = torch.full_like(a[0], math.nan)
    return gdr.kv8_attn(*a, i32(x["lens"]), x["scale"], cu_q=i32(x["cu"]), want_lse=True, out=out, **kw)


def want(x):
    return O.attention(x["q"].double().numpy(), x["kc"].numpy(), x["vc"].numpy(), x["ks"].double().numpy(),
                       x["vs"].double().numpy(), x["table"].numpy(), x["lens"], x["cu"], x["scale"], x["kv"])


def worst_row(out, ref, keep=None):
    a, b = out.double().cpu().numpy().reshape(-1, out.shape[-1]), ref.reshape(-1, out.shape[-1])
    err = np.linalg.norm(a - b, axis=1) / np.maximum(np.linalg.norm(b, axis=1), 1e-300)
    return float(err.max() if keep is None else err[keep.reshape(-1)].max())


# ------------------------------------------------------------------ a small max_q
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,qs,Hq,Hkv,max_q", [
    ([4000], [5], 8, 1, 1),                       # items of 8 rows, five of them, all divided
    ([3000, 2000, 1], [40, 7, 1], 4, 2, 1), ([5000, 300], [70, 30], 8, 2, 4), ([2500, 900], [90, 3], 8, 1, 3),
    ([3000], [200], 8, 1, 8), ([4000, 128], [300, 128], 4, 1, 20), ([2000, 50], [5, 2], 16, 2, 0),
    ([2000] * 50, [9] * 50, 8, 1, 1),
])
def test_a_small_max_q_costs_time_only(dtype, lens, qs, Hq, Hkv, max_q):
    x = case(lens, qs, Hq, Hkv, 128, 16, dtype, "e4m3", 1)
    out, lse = attend(x, max_q=max_q)
    ro, rl = want(x)
    assert worst_row(out, ro) <= TOL[dtype]
    assert np.abs(lse.double().cpu().numpy() - rl).max() <= 1e-5 * max(1.0, np.abs(rl).max())


def test_lengths_want_a_max_q():
    x = case([40], [5], 2, 1, 64, 16, BF16, "int8", 2)
    with pytest.raises(ValueError):
        attend(x)


# ------------------------------------------------------------------ rows far apart
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("qs,Hq,Hkv,D", [([1, 1], 8, 1, 128), ([2, 2], 8, 1, 64), ([3, 5], 8, 1, 128), ([7, 6], 8, 1, 64),
                                         ([13, 16], 8, 1, 128), ([100, 60], 8, 2, 128), ([40, 70], 10, 1, 64)])
def test_rows_far_apart(kv, qs, Hq, Hkv, D):
    """Every third row 2^40 or 2^120 times larger than the others, one infinite and one NaN: the
    others' results stay as exact as alone."""
    x = case([400, 333], qs, Hq, Hkv, D, 32, BF16, kv, 3)
    rows = torch.arange(sum(qs) * Hq).reshape(sum(qs), Hq)
    ro, _ = want(x)
    x["q"] = torch.where((rows % 3 == 1)[..., None], x["q"] * 2.0 ** 40, x["q"])
    x["q"] = torch.where((rows % 9 == 4)[..., None], x["q"] * 2.0 ** 80, x["q"])
    x["q"].view(-1, D)[1, 5], x["q"].view(-1, D)[4, 6] = math.inf, math.nan
    out, _ = attend(x, max_q=max(qs))
    assert worst_row(out, ro, (rows % 3 != 1).numpy()) <= TOL[BF16]


# ------------------------------------------------------------------ a largest weight whose value is nothing
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,gap", [(BF16, 12.0), (BF16, 16.0), (BF16, 20.0), (F32, 12.0), (F32, 20.0), (F32, 60.0)])
@pytest.mark.parametrize("qs,Hq,Hkv,D", [([1], 8, 1, 128), ([1], 8, 2, 64), ([2], 8, 1, 128), ([4], 8, 1, 128),
                                         ([8], 8, 1, 64), ([15], 8, 1, 128), ([150], 4, 1, 128)])
def test_a_dominant_key_without_a_value(kv, dtype, gap, qs, Hq, Hkv, D):
    """The first key scores `gap` nats above the other thousand and its value codes are zero (an
    attention sink), so the output is what the small weights give.  bf16: the weights stand
    2^13 .. 2^14 for the row's largest, so 20 nats below (2^-28.9) they are 2^-15.9 or more, in
    steps of 2^-24: off by 2^-25.8 at most in rms, 2^-9.9 = 1.0e-3 of the weight, which with the
    output's rounding is 2.5e-3 of 3e-3.  fp32 keeps 24 bits of every weight."""
    x = case([1001], qs, Hq, Hkv, D, 16, dtype, kv, 4)
    one = 0x38 if kv == "e4m3" else 1                     # the code of 1
    big, value = (0x78, 256.0) if kv == "e4m3" else (100, 100.0)
    first = int(x["table"][0, 0])
    x["kc"][..., 0] = one                                 # dimension 0: the gap alone
    x["kc"][first, :, 0] = 0
    x["kc"][first, :, 0, 0] = big
    x["vc"][first, :, 0] = 0
    x["q"] = x["q"] * 0.25
    x["q"][..., 0] = gap / ((value - 1) * float(x["ks"][0, 0]) * x["scale"])
    ro, rl = want(x)
    out, lse = attend(x, max_q=max(qs))
    assert worst_row(out, ro) <= TOL[dtype]
    assert np.abs(lse.double().cpu().numpy() - rl).max() <= 1e-5 * max(1.0, np.abs(rl).max())
