"""Waits of the cache attention that run out, in every kernel (no fault, no hang): with a limit of
zero each CTA's first wait fails, whether its data is there or not, so the error word always says
so and the way out (copies, products and weights in flight) is always taken."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 64)])
@pytest.mark.parametrize("lens", [[1], [17, 0], [700, 33, 0, 1290], [60000, 33]])
@pytest.mark.parametrize("rows", [8, 16, 24, 56, 96, 320])
def test_every_form_gives_up_and_recovers(dtype, D, page, lens, rows):
    gdr.load(build_if_missing=True)
    g = torch.Generator().manual_seed(rows)
    S, H, q = len(lens), 2, rows // 8
    need = [-(-n // page) for n in lens]
    N, W = sum(need), max(need)
    table = torch.full((S, W), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        table[s, :n] = torch.arange(sum(need[:s]), sum(need[:s]) + n)
    kc, vc = (torch.randint(-127, 128, (N, H, page, D), generator=g).to(torch.int8).cuda() for _ in range(2))
    ks, vs = torch.full((N, H), 2.0 ** -6, device="cuda"), torch.ones((N, H), device="cuda")
    x = torch.randn((S * q, 8 * H, D), generator=g).to(dtype).cuda()
    cu = torch.arange(0, S * q + 1, q, dtype=torch.int32, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert gdr.last_device_error() == 0

    def call():
        return gdr.kv8_attn(x, kc, vc, ks, vs, table.cuda(), kv, 1 / math.sqrt(D), cu_q=cu, max_q=q, want_lse=True)

    before = call()
    assert gdr.last_device_error() == 0
    with gdr.option(wait_limit_ns=0):
        call()
        assert gdr.last_device_error() == 5          # GDR_ERR_TIMEOUT
    after = call()
    assert gdr.last_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(before, after))
