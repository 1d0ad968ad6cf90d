"""Workspaces that a caller gives: tensors whose bytes do not lie in a row are refused before anything is
launched (an expanded byte has as many elements as any size wants, and no memory behind it)."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    yield
    torch.cuda.synchronize()
    assert gdr.last_device_error() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def calls():
    q = torch.ones((2, 2, 64), device="cuda")
    cache = [torch.ones((4, 1, 16, 64), dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.ones((4, 1), device="cuda") for _ in range(2)]
    table, kv, group = i32([[0, 1], [0, 2]]), i32([20, 20]), i32([0, 2])
    plan = gdr.kv8_shared_plan(table, kv, group, 16)
    w = torch.ones(64, device="cuda")
    return [
        (gdr.kv8_attn_workspace_size(2, 1, 2, 2, 1, 64, q.dtype),
         lambda ws: gdr.kv8_attn(q, *cache, *scale, table, kv, 0.1, workspace=ws)),
        (gdr.kv8_attn_shared_workspace_size(2, 1, 1, 2, 2, 2, 1, 64, q.dtype),
         lambda ws: gdr.kv8_attn_shared(q, *cache, *scale, table, kv, 0.1, group, *plan, max_group_q=2, workspace=ws)),
        (gdr.qk_norm_rope_bwd_workspace_size(64),
         lambda ws: gdr.qk_norm_rope_bwd(q, q, q, q, q_weight=w, k_weight=w, workspace=ws)),
    ]


@pytest.mark.parametrize("i", range(3))
def test_workspaces_that_are_not_in_a_row(i):
    need, call = calls()[i]
    assert need > 0
    whole = torch.empty(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (whole[:1].expand(need), whole[::2], whole.view(2, need).t(), whole[:need - 1], whole.view(torch.int8)):
        with pytest.raises(ValueError, match="contiguous uint8"):
            call(ws)
    call(whole[:need])
