"""The serving example with norms, rotation and a common prefix, run together: its logits against the
same decoder evaluated a whole sequence (the prefix's tokens first) at once, with unquantised keys and
values, norms and rotation in fp32 and 64-bit angles.

Tolerance: the codes' rounding, as in the example's test without these: 6e-2 in relative L2 (a code is off by
2^-4 / sqrt(3) of the value at most, keys and values; the norms and the rotation are bf16 roundings, 2^-8)."""
from __future__ import annotations

import math
import os
import sys

import pytest
import torch
import torch.nn.functional as F

import oracle
import gated_delta_rule_gdr_gb300 as gdr

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import hybrid_serving as hs  # noqa: E402

pytestmark = pytest.mark.gpu
D = hs.D


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    yield
    assert gdr.last_device_error() == 0


def turned(x, w, freq):
    """x [heads, T, D] fp32: root-mean-square norm, weights, rotation by the place in the sequence."""
    x = F.rms_norm(x, x.shape[-1:], eps=1e-6) * w
    a = torch.arange(x.shape[1], dtype=torch.float64, device="cuda")[:, None] * freq
    c, s = a.cos().float(), a.sin().float()
    u, v = x.chunk(2, -1)
    return torch.cat([u * c - v * s, u * s + v * c], -1)


def whole(m, tokens):
    """Logits after the last of `tokens`, no cache."""
    x = m.embedding[torch.tensor(tokens, device="cuda")]
    T, H = x.shape[0], m.heads
    for b in range(m.blocks):
        y = F.rms_norm(x, x.shape[-1:]) @ m.w_delta[b]
        q, k, v = (t.view(T, H, D).transpose(0, 1)[None] for t in y[:, :3 * H * D].split(H * D, 1))
        gate, beta = (t.t()[None].contiguous() for t in y[:, 3 * H * D:].float().split(H, 1))
        q, k = (F.normalize(t.float(), dim=-1).bfloat16().contiguous() for t in (q, k))
        o, _ = gdr.chunk_fwd(q, k, v.contiguous(), gate, beta.sigmoid(), hs.A_MIN)
        x = x + o[0].transpose(0, 1).reshape(T, -1) @ m.w_delta_out[b]
        y = (F.rms_norm(x, x.shape[-1:]) @ m.w_qkv[b]).view(T, -1, D).float().transpose(0, 1)
        q, k, v = y.split([m.q_heads, m.kv_heads, m.kv_heads])
        if m.freq is not None:
            q, k = turned(q, m.q_norm[b], m.freq), turned(k, m.k_norm[b], m.freq)
        k, v = (t.repeat_interleave(m.q_heads // m.kv_heads, 0) for t in (k, v))
        s = (q @ k.transpose(1, 2)) / math.sqrt(D)
        s = s.masked_fill(torch.ones((T, T), dtype=torch.bool, device="cuda").triu(1), -math.inf)
        x = x + (s.softmax(-1) @ v).transpose(0, 1).reshape(T, -1).bfloat16() @ m.w_attn_out[b]
    return F.rms_norm(x[-1], x.shape[-1:]) @ m.unembedding


@pytest.mark.parametrize("least", [0, 1])
@pytest.mark.parametrize("codes", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("theta", [None, 10000.0])
@pytest.mark.parametrize("prefix", [0, 150])
def test_steps_equal_whole_sequences(codes, theta, prefix, least):
    m = hs.HybridDecoder(3, 80, 24, codes=codes, theta=theta)
    g = torch.Generator().manual_seed(5)
    common = torch.randint(0, 1000, (prefix,), generator=g).tolist()
    with gdr.option(shared_least=least):
        m.share(common)
        common = common[:m.prefix]
        assert len(common) == prefix // 32 * 32
        seqs = [[], [], []]
        for n in ([70, 33, 1], [1, 1, 1], [200, 0, 64], [1, 1, 1], [2, 3, 4]):
            new = [torch.randint(0, 1000, (i,), generator=g).tolist() for i in n]
            seqs = [s + t for s, t in zip(seqs, new)]
            logits = m.step(new)
            for s in range(3):
                if n[s]:
                    assert oracle.rel_l2(logits[s].cpu(), whole(m, common + seqs[s]).cpu()) <= 6e-2
    assert m.kv_len.tolist() == [m.prefix + len(s) for s in seqs]


def test_requests_come_and_go():
    """More requests than slots after one prefix: every page comes back but the prefix's own."""
    m = hs.HybridDecoder(4, 44, 12, theta=10000.0)
    m.share(list(range(140)))
    assert m.prefix == 128 and m.ring_state[1].item() == 40
    prompts = [[7 * i + j for j in range(n)] for i, n in enumerate([1, 90, 200, 33, 64, 5, 150])]
    with gdr.option(shared_least=1):
        answers = hs.serve(m, prompts, 6, 64)
    assert [len(a) for a in answers] == [6] * 7
    assert m.ring_state[1].item() == 40 and m.kv_len.tolist() == [0] * 4
    free = m.ring.tolist()
    head = m.ring_state[0].item()
    pages = [free[(head + i) % 44] for i in range(40)]
    assert sorted(pages + m.prefix_pages.tolist()) == list(range(44))
    with pytest.raises(RuntimeError):
        m.share([1] * 32)
