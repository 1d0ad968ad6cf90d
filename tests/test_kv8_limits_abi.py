"""gdr_kv8_attn's limits of size: host-only checks, nothing is launched."""
from __future__ import annotations

import ctypes

import pytest

import gated_delta_rule_gdr_gb300 as gdr
from gated_delta_rule_gdr_gb300 import build as gbuild

P = ctypes.c_void_p(0x1000)


@pytest.mark.parametrize("page,width", [(16, 2 ** 27 - 1), (32, 2 ** 26 - 2), (128, 2 ** 24 - 1), (64, 2 ** 25)])
def test_a_table_of_almost_2_31_tokens_is_refused(page, width):
    """A unit's end past the last token would not fit 32 bits."""
    gbuild.build()
    code = gdr.load().gdr_kv8_attn(P, 1024, P, P, P, P, P, P, P, 0.1, P, None, 4, 3, 12, 8, 2, 128, width, page, 100, 1, 0,
                                   P, 1 << 40, None)
    assert code == 2
