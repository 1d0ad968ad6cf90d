"""Where the buffers of gdr_kv8_attn_shared lie: outputs and workspaces on 16-byte boundaries that are on no
wider one, workspaces of exactly the stated size, sums of more than 2^31 values.  The arithmetic does not depend
on any of these, so results are equal bit for bit; nothing around the buffers changes."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
from test_kv8_shared_gpu import BF16, F32, attend, case, check, i32, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    with gdr.option(shared_least=1):        # both passes
        yield
    torch.cuda.synchronize()
    assert gdr.last_device_error() == 0


CASES = [
    # groups, Hq, Hkv, D, page: the first pass's form / the second's
    ([(20, [(300, 200), (180, 150)])], 8, 2, 128, 64),              # pairs of tiles / pairs
    ([(12, [(40, 20), (30, 15)]), (3, [(25, 20), (9, 4)])], 8, 2, 128, 16),     # pairs / one tile
    ([(70, [(20, 12), (15, 6)])], 8, 2, 64, 16),                    # one tile / two copies
    ([(30, [(9, 5), (9, 5)])], 8, 2, 128, 32),                      # two copies / four copies
    ([(50, [(9, 5)] * 2)], 4, 2, 128, 16),                          # four copies / 16 rows of the split kernel
    ([(75, [(3, 1)] * 33)], 28, 4, 64, 16),                         # pairs of many parts / 8 rows
    ([(64, [(700, 70), (65, 65)])], 5, 1, 128, 128),                # pairs / pairs, both of many parts
    ([(90, [(2, 1)] * 4)], 8, 2, 128, 16),                          # 16 rows and more, single tokens
]


def offset(n, dtype, by):
    """A tensor of n values that begins `by` bytes behind an allocation's start, and what lies around it."""
    size = torch.empty(0, dtype=dtype).element_size()
    whole = torch.full((n * size + 512,), 0x55, dtype=torch.uint8, device="cuda")
    assert whole.data_ptr() % 256 == 0
    inside = whole[by:by + n * size]
    return inside.view(dtype), lambda: bool((whole[:by] == 0x55).all()) and bool((whole[by + n * size:] == 0x55).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kv", ["e4m3", "int8"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_on_16_bytes(dtype, kv, i):
    x = case(*CASES[i], dtype, kv, seed=40 + i)
    d = on_gpu(x)
    want, lse = attend(x, d, packed=True)
    check(x, (want, lse))
    need = gdr.kv8_attn_shared_workspace_size(
        len(x["lens"]), max(x["qs"]), len(x["ends"]) - 1,
        max(x["cu"][b] - x["cu"][a] for a, b in zip(x["ends"], x["ends"][1:])), *want.shape[:2], x["kc"].shape[1],
        want.shape[2], dtype)
    for at_out, at_ws in ((16, 0), (0, 16), (16, 16), (48, 80)):
        out, out_kept = offset(want.numel(), dtype, at_out)
        ws, ws_kept = offset(need, torch.uint8, at_ws)
        got = attend(x, d, packed=True, out=out.view(want.shape), workspace=ws)
        assert torch.equal(got[0], want) and torch.equal(got[1], lse), (at_out, at_ws)
        assert out_kept() and ws_kept(), (at_out, at_ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_kv8_attn_on_16_bytes(dtype, n):
    """gdr_kv8_attn likewise, whose kernels these are."""
    x = case([(30, [(n + 50, n), (n, n), (n + 900, n)])], 8, 2, 128, 16, dtype, "e4m3", seed=60)
    d = on_gpu(x)
    call = lambda **kw: gdr.kv8_attn(d["q"], *d["cache"], d["table"], d["kv_len"], x["scale"], cu_q=d["cu"], max_q=n,  # noqa: E731
                                     want_lse=True, **kw)
    want, lse = call()
    need = gdr.kv8_attn_workspace_size(3, n, *want.shape[:2], 2, 128, dtype)
    for at in (16, 48):
        out, out_kept = offset(want.numel(), dtype, at)
        ws, ws_kept = offset(need, torch.uint8, at)
        got = call(out=out.view(want.shape), workspace=ws)
        assert torch.equal(got[0], want) and torch.equal(got[1], lse)
        assert out_kept() and ws_kept()


def test_offsets_past_32_bits():
    """The sums of the first pass, queries and outputs of more than 2^31 values: the last requests as they are
    in a batch of their own."""
    S, n, Hq, Hkv, D, page = 8192, 33, 64, 1, 128, 16
    last = 7                                            # requests; the others share pages, these are a group
    g = torch.Generator(device="cuda").manual_seed(1)
    pages = 12 + 3 * last
    cache = [torch.randint(-127, 128, (pages, Hkv, page, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
    scale = [torch.full((pages, Hkv), 2.0 ** -6, device="cuda") for _ in range(2)]
    table = torch.arange(5, dtype=torch.int32, device="cuda").repeat(S, 1)
    for r in range(last):
        table[S - last + r] = i32([6, 7, 12 + 3 * r, 13 + 3 * r, 14 + 3 * r])
    kv = torch.full((S,), 5 * page - 3, dtype=torch.int32, device="cuda")
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
    group = i32([0, S - last, S])
    assert S * n * Hq * D > 2 ** 31
    q = torch.empty((S * n, Hq, D), dtype=BF16, device="cuda").normal_(generator=g)
    plan = gdr.kv8_shared_plan(table, kv, group, page, cu_q=cu)
    # whole pages that all 33 queries of a request see: 77 - 33 + 1 = 45 tokens, two pages
    assert plan[0].unique().tolist() == [32] and plan[1].tolist() == [0, S - last]
    out, lse = gdr.kv8_attn_shared(q, *cache, *scale, table, kv, 0.1, group, *plan, cu_q=cu, max_q=n,
                                   max_group_q=(S - last) * n, want_lse=True)
    for a, b in ((0, last), (S - last, S)):
        t, k, c = table[a:b].contiguous(), kv[a:b].contiguous(), cu[:last + 1].contiguous()
        one = i32([0, last])
        p = gdr.kv8_shared_plan(t, k, one, page, cu_q=c)
        ref, ref_lse = gdr.kv8_attn_shared(q[a * n:b * n], *cache, *scale, t, k, 0.1, one, *p, cu_q=c, max_q=n,
                                           max_group_q=last * n, want_lse=True)
        # other parts, so other orders of sums: two roundings of a value at most, 2^-8 each, and the weights' bits
        rel = (out[a * n:b * n].double() - ref.double()).norm() / ref.double().norm()
        assert rel <= 6e-3, float(rel)
        assert (lse[a * n:b * n] - ref_lse).abs().max() <= 2e-5 * max(1.0, float(ref_lse.abs().max()))
    assert torch.isfinite(lse).all()
