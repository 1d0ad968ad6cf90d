"""Serving a hybrid decoder: incremental (gated delta rule) layers and exact-attention layers
with a paged 8-bit cache, side by side, under continuous batching.

A slot holds one request: its row of the block table (shared by all exact layers), its
state of every incremental layer and its sequence length.  A step takes each slot's new
tokens (a prompt, a chunk of one, one decoded token, none, or "finished") and runs

    page_plan                                   places for the new tokens, once a step
    incremental layer:  chunk_fwd_varlen, or decode_step where every slot has one token
    exact layer:        kv8_append, kv8_attn

Weights are random; the linear maps around the layers are plain matrix products.

    python examples/hybrid_serving.py --slots 32 --prompt 2000 --new 64
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_delta_rule_gdr_gb300 as gdr  # noqa: E402

A_MIN, D = 0.95, 128


class HybridDecoder:
    """Blocks of one incremental and one exact-attention layer each, with their caches."""

    def __init__(self, slots, pages, table_width, *, blocks=2, vocab=1000, width=512, heads=4,
                 q_heads=8, kv_heads=2, page=32, codes=torch.float8_e4m3fn, device="cuda", seed=0):
        self.slots, self.pages, self.page, self.blocks = slots, pages, page, blocks
        self.heads, self.q_heads, self.kv_heads = heads, q_heads, kv_heads
        self.device = device
        g = torch.Generator().manual_seed(seed)

        def matrix(rows, cols):
            return (torch.randn((rows, cols), generator=g) / math.sqrt(rows)).bfloat16().to(device)

        self.embedding = torch.randn((vocab, width), generator=g).bfloat16().to(device)
        self.unembedding = matrix(width, vocab)
        self.w_delta = [matrix(width, heads * (3 * D + 2)) for _ in range(blocks)]
        self.w_delta_out = [matrix(heads * D, width) for _ in range(blocks)]
        self.w_qkv = [matrix(width, (q_heads + 2 * kv_heads) * D) for _ in range(blocks)]
        self.w_attn_out = [matrix(q_heads * D, width) for _ in range(blocks)]

        # what a request leaves behind between steps
        self.state = [torch.zeros((slots, heads, D, D), device=device) for _ in range(blocks)]
        shape = (pages, kv_heads, page, D)
        self.cache = [[torch.zeros(shape, device=device).to(codes) for _ in range(2)] for _ in range(blocks)]
        self.scale = [[torch.ones(shape[:2], device=device) for _ in range(2)] for _ in range(blocks)]
        self.table = torch.full((slots, table_width), -1, dtype=torch.int32, device=device)
        self.ring = torch.arange(pages, dtype=torch.int32, device=device)
        self.ring_state = torch.tensor([0, pages], dtype=torch.int32, device=device)
        self.kv_len = torch.zeros(slots, dtype=torch.int32, device=device)
        # one workspace for every exact layer of any step up to this size, kept by the caller
        self.workspace = torch.empty(0, dtype=torch.uint8, device=device)

    def _delta(self, b, x, cu, single):
        """The incremental layer: q and k of unit length, beta in (0, 1)."""
        y = x @ self.w_delta[b]
        T, H = x.shape[0], self.heads
        q, k, v = (t.view(T, H, D) for t in y[:, :3 * H * D].split(H * D, 1))
        gate, beta = y[:, 3 * H * D:].float().split(H, 1)
        q, k = F.normalize(q.float(), dim=-1).bfloat16(), F.normalize(k.float(), dim=-1).bfloat16()
        args = (q, k, v.contiguous(), gate.contiguous(), beta.sigmoid(), A_MIN)
        if single:
            out = gdr.decode_step(*args, self.state[b])
        else:
            out, self.state[b] = gdr.chunk_fwd_varlen(*args, cu, self.state[b])
        return out.view(T, H * D) @ self.w_delta_out[b]

    def _attention(self, b, x, cu, slots, kv_len, longest, single):
        """The exact layer: the new keys and values into the cache, then attention over it."""
        y = (x @ self.w_qkv[b]).view(x.shape[0], -1, D)      # q, k, v stay where the product put them
        q, k, v = y.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        gdr.kv8_append(k, v, slots, *self.cache[b], *self.scale[b])
        out = gdr.kv8_attn(q, *self.cache[b], *self.scale[b], self.table, kv_len, 1 / math.sqrt(D),
                           cu_q=None if single else cu, max_q=longest, workspace=self.workspace)
        return out.view(x.shape[0], -1) @ self.w_attn_out[b]

    def step(self, tokens):
        """tokens: per slot the new token ids (a list), [] for none, None where the request is
        finished (its pages return to the ring and its states to zero).  Returns the logits
        [slots, vocab] after each slot's last new token (rows of slots without: of no use)."""
        n = [-1 if t is None else len(t) for t in tokens]
        flat = [i for t in tokens if t for i in t]
        total, longest = len(flat), max(n)
        q_len = torch.tensor(n, dtype=torch.int32, device=self.device)
        kv_len, cu, slots, _, granted, ring_state = gdr.page_plan(
            self.kv_len, q_len, self.table, self.ring, self.ring_state, self.page, total)
        self.kv_len, self.ring_state = kv_len, ring_state
        for s, t in enumerate(tokens):
            if t is None:
                for state in self.state:
                    state[s].zero_()
        if total == 0:
            return None
        if not bool(granted.all()):
            raise RuntimeError("no pages left: admit fewer requests")
        single = longest == 1 and min(n) == 1
        size = gdr.kv8_attn_workspace_size(self.slots, longest, total, self.q_heads, self.kv_heads, D)
        if self.workspace.numel() < size:
            self.workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
        x = self.embedding[torch.tensor(flat, device=self.device)]
        for b in range(self.blocks):
            x = x + self._delta(b, F.rms_norm(x, x.shape[-1:]), cu, single)
            x = x + self._attention(b, F.rms_norm(x, x.shape[-1:]), cu, slots, kv_len, longest, single)
        last = (cu[1:] - 1).clamp_min(0).long()
        return F.rms_norm(x[last], x.shape[-1:]) @ self.unembedding


def serve(model, prompts, new, chunk):
    """Greedy continuations of the prompts, `new` tokens each: prompts enter free slots in
    chunks of at most `chunk` tokens beside the other slots' single tokens; a finished request
    gives its pages back and the next prompt takes its slot."""
    waiting = list(range(len(prompts)))[::-1]
    live = [None] * model.slots                # request, tokens of the prompt taken
    answers = [[] for _ in prompts]
    given_back = [False] * model.slots
    while waiting or any(given_back) or any(r is not None for r in live):
        tokens = []
        for s in range(model.slots):
            if live[s] is None and waiting and not given_back[s]:
                live[s] = [waiting.pop(), 0]
            if given_back[s]:
                tokens.append(None)
                given_back[s] = False
            elif live[s] is None:
                tokens.append([])
            else:
                r, at = live[s]
                take = prompts[r][at:at + chunk] if at < len(prompts[r]) else answers[r][-1:]
                live[s][1] = at + len(take)
                tokens.append(take)
        logits = model.step(tokens)
        if logits is None:
            continue
        best = logits.argmax(-1).tolist()
        for s, t in enumerate(tokens):
            if not t:
                continue
            r, at = live[s]
            if at >= len(prompts[r]):
                answers[r].append(best[s])
                if len(answers[r]) == new:
                    live[s], given_back[s] = None, True
    return answers


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--slots", type=int, default=32)
    p.add_argument("--requests", type=int, default=40)
    p.add_argument("--prompt", type=int, default=2000, help="longest prompt")
    p.add_argument("--new", type=int, default=64, help="tokens to decode per request")
    p.add_argument("--chunk", type=int, default=512, help="most prompt tokens of a request in a step")
    p.add_argument("--codes", choices=["e4m3", "int8"], default="e4m3")
    a = p.parse_args(argv)
    gdr.load(build_if_missing=True)
    page = 32
    width = -(-(a.prompt + a.new) // page)
    model = HybridDecoder(a.slots, 2 * a.slots * width, width, page=page,
                          codes=torch.float8_e4m3fn if a.codes == "e4m3" else torch.int8)
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(1, a.prompt + 1, (a.requests,), generator=g).tolist()
    prompts = [torch.randint(0, 1000, (n,), generator=g).tolist() for n in lengths]
    torch.cuda.synchronize()
    start = time.perf_counter()
    answers = serve(model, prompts, a.new, a.chunk)
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    if gdr.last_device_error():
        raise RuntimeError("a device wait gave up")
    print(f"{a.requests} requests, {sum(lengths)} prompt and {a.requests * a.new} new tokens in {took:.2f} s; "
          f"first answer {answers[0][:8]} ...; free pages {model.ring_state[1].item()} of {model.pages}")
    return answers


if __name__ == "__main__":
    main()
