"""The norms around a training step of an incremental layer, run together: slices of a projection ->
gdr_qk_norm_rope (unit length) -> gdr_chunk_fwd_train -> gdr_chunk_bwd_saved -> gdr_qk_norm_rope_bwd onto the
projection's gradient.  The layer takes [B, H, T, d], so transposing copies stand between.

Reference: the fp64 oracle's gradients at the same rounded unit rows, times the norm's Jacobian r (1 - y y^T) in 64
bits.  The layer's gradients are within 5e-3 of the oracle's in relative L2, then rounded once more to bf16 (2^-8 /
sqrt(3) of the value).  The Jacobian can only shorten what it is applied to, so the difference is held against r times
the oracle's gradient, not against the projected one; rows' r differ by a factor of 1.5 from their mean at most
(128 values): (5e-3 + 2.3e-3) 1.5 < 1.1e-2."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
import oracle

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    yield
    torch.cuda.synchronize()
    assert gdr.last_device_error() == 0


def heads_first(x, B):
    """[B T, H, D] -> [B, H, T, D]"""
    return x.unflatten(0, (B, -1)).transpose(1, 2).contiguous()


def tokens_first(x):
    return x.transpose(1, 2).flatten(0, 1)


@pytest.mark.parametrize("B,H,T", [(1, 2, 130), (2, 3, 64), (2, 1, 333)])
def test_projection_to_projection(B, H, T):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((B * T, 3 * H, D), generator=g, device="cuda").bfloat16()       # q, k, v side by side
    gate, beta = torch.randn((2, B, H, T), generator=g, device="cuda")
    beta = beta.sigmoid()
    d_out = torch.randn((B, H, T, D), generator=g, device="cuda").bfloat16()
    q, k, v = x.split(H, 1)
    yq, yk = gdr.qk_norm_rope(q, k, norm="l2", eps=1e-24)
    args = *(heads_first(t, B) for t in (yq, yk, v)), gate, beta, 0.95
    _, _, saved = gdr.chunk_fwd_train(*args)
    grads = gdr.chunk_bwd_saved(*args, None, d_out, saved, want_dinit=False)
    dx = torch.full_like(x, 7.0)
    gdr.qk_norm_rope_bwd(q, k, *(tokens_first(t).contiguous() for t in grads[:2]), norm="l2", eps=1e-24,
                         d_q=dx[:, :H], d_k=dx[:, H:2 * H])
    dx[:, 2 * H:] = tokens_first(grads[2])
    ref = oracle.bwd(*(t.cpu() for t in args[:5]), 0.95, None, d_out.cpu())
    for t, y, got, want in ((q, yq, dx[:, :H], ref[0]), (k, yk, dx[:, H:2 * H], ref[1])):
        t, y, got = (a.double().cpu().numpy() for a in (t, y, got))
        r = 1 / np.linalg.norm(t, axis=-1, keepdims=True)
        assert r.max() / r.mean() < 1.5 and r.min() / r.mean() > 1 / 1.5
        want = np.swapaxes(want, 1, 2).reshape(t.shape)
        u = t * r                                                # |u| = 1; y is u rounded
        assert np.linalg.norm(y - u) <= 2.0 ** -8 * np.linalg.norm(u)
        exact = r * (want - u * (u * want).sum(-1, keepdims=True))
        assert np.linalg.norm(got - exact) <= 1.1e-2 * np.linalg.norm(r * want)
    assert oracle.rel_l2(dx[:, 2 * H:], np.swapaxes(ref[2], 1, 2).reshape(B * T, H, D)) <= 5e-3
