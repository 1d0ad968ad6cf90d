"""The serving example on the GPU: the incremental layers, the page plan, the 8-bit cache and
the attention over it, run together.  Its logits against the same decoder evaluated a whole
sequence at once with unquantised keys and values in fp32.

Tolerance.  An e4m3 code is off by at most 2^-4 of the value, uniformly within half a step:
2^-4 / sqrt(3) = 3.6e-2 in relative L2 at most.  Values carry it to the output as it is; keys
change the scores (standard deviation about 1) by as much, so the weights and the output by
3.6e-2 again: 5.1e-2 together for an exact layer's output, which is one of two parts that each
block adds to its input.  6e-2 is asked of the logits, and of int8 the same (its step, at most
1/127 of a page's largest value, is finer for the bulk of normal values)."""
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
        k, v = (t.repeat_interleave(m.q_heads // m.kv_heads, 0) for t in (k, v))
        s = (q @ k.transpose(1, 2)) / math.sqrt(D)
        s = s.masked_fill(torch.ones((T, T), dtype=torch.bool, device="cuda").triu(1), -math.inf)
        x = x + (s.softmax(-1) @ v).transpose(0, 1).reshape(T, -1).bfloat16() @ m.w_attn_out[b]
    return F.rms_norm(x[-1], x.shape[-1:]) @ m.unembedding


@pytest.mark.parametrize("codes", [torch.float8_e4m3fn, torch.int8])
def test_steps_equal_whole_sequences(codes):
    m = hs.HybridDecoder(3, 60, 20, codes=codes)
    g = torch.Generator().manual_seed(5)
    seqs = [[], [], []]
    for n in ([70, 33, 1], [1, 1, 1], [200, 0, 64], [1, 1, 1], [2, 3, 4]):
        new = [torch.randint(0, 1000, (i,), generator=g).tolist() for i in n]
        seqs = [s + t for s, t in zip(seqs, new)]
        logits = m.step(new)
        for s in range(3):
            if n[s]:
                assert oracle.rel_l2(logits[s].cpu(), whole(m, seqs[s]).cpu()) <= 6e-2
    assert m.kv_len.tolist() == [len(s) for s in seqs]


def test_requests_come_and_go():
    """More requests than slots: each answer has its length, and every page comes back."""
    m = hs.HybridDecoder(4, 40, 8)
    prompts = [[7 * i + j for j in range(n)] for i, n in enumerate([1, 90, 200, 33, 64, 5, 150])]
    answers = hs.serve(m, prompts, 6, 64)
    assert [len(a) for a in answers] == [6] * 7
    assert m.ring_state[1].item() == 40 and m.kv_len.tolist() == [0] * 4
