"""A step of a server kept as a CUDA graph: norms with rotation, append, plan and attention over shared prefixes
captured once and replayed as the requests grow, take other pages and other groups; two such calls at once on two
streams; two graphs over one workspace.  Every kernel's result repeats, so replayed and eager steps are equal bit for
bit."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
from test_kv8_shared_gpu import BF16, F32, attend, case, check, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    with gdr.option(shared_least=1):
        yield
    torch.cuda.synchronize()
    assert gdr.last_device_error() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    """S requests of single tokens with Hq and Hkv heads; the prefix's pages are the first ones."""

    def __init__(self, S, prefix_pages, dtype, codes, Hq=8, Hkv=2, D=128, page=16, width=40):
        g = torch.Generator(device="cuda").manual_seed(3)
        self.S, self.page, self.Hq, self.Hkv, self.D = S, page, Hq, Hkv, D
        pages = prefix_pages + S * (width - prefix_pages)
        self.cache = [torch.zeros((pages, Hkv, page, D), device="cuda").to(codes) for _ in range(2)]
        self.scale = [torch.ones((pages, Hkv), device="cuda") for _ in range(2)]
        self.table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        n = prefix_pages * page
        k, v = torch.randn((2, n, Hkv, D), generator=g, device="cuda").to(dtype)
        gdr.kv8_append(k, v, torch.arange(n, dtype=torch.int32, device="cuda"), *self.cache, *self.scale)
        self.table[:, :prefix_pages] = torch.arange(prefix_pages, device="cuda", dtype=torch.int32)
        self.kv = torch.full((S,), n, dtype=torch.int32, device="cuda")
        self.ring = torch.arange(pages, dtype=torch.int32, device="cuda").roll(-prefix_pages)
        self.state = i32([0, pages - prefix_pages])
        self.q_len = torch.ones(S, dtype=torch.int32, device="cuda")
        self.group = i32([0, S])
        self.freq = (10000.0 ** (-2 * torch.arange(D // 2, dtype=torch.float64) / D)).cuda()
        self.x = torch.zeros((S, Hq + 2 * Hkv, D), device="cuda", dtype=dtype)
        self.workspace = torch.zeros(gdr.kv8_attn_shared_workspace_size(S, 1, 1, S, S, Hq, Hkv, D, dtype),
                                     dtype=torch.uint8, device="cuda")

    def step(self):
        kv, _, slots, pos, _, state = gdr.page_plan(self.kv, self.q_len, self.table, self.ring, self.state, self.page, self.S)
        q, k, v = self.x.split([self.Hq, self.Hkv, self.Hkv], 1)
        q, k = gdr.qk_norm_rope(q, k, positions=pos, freq=self.freq)
        gdr.kv8_append(k, v, slots, *self.cache, *self.scale)
        plan = gdr.kv8_shared_plan(self.table, kv, self.group, self.page)
        out, lse = gdr.kv8_attn_shared(q, *self.cache, *self.scale, self.table, kv, 1 / math.sqrt(self.D), self.group,
                                       *plan, max_group_q=self.S, want_lse=True, workspace=self.workspace)
        self.kv.copy_(kv)
        self.state.copy_(state)
        return out, lse, *plan, pos


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S", [3, 40])
def test_a_step_kept_as_a_graph(dtype, S):
    codes = torch.float8_e4m3fn if dtype is BF16 else torch.int8
    eager, kept = (Server(S, 20, dtype, codes) for _ in range(2))
    warm = Server(S, 20, dtype, codes)
    warm.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):               # captured, not run: nothing of `kept` moves on
        got = kept.step()
    g = torch.Generator(device="cuda").manual_seed(5)
    for i in range(40):
        x = torch.randn(eager.x.shape, generator=g, device="cuda").to(dtype)
        for s in (eager, kept):
            s.x.copy_(x)
            if i == 15:                         # a request leaves the prefix: its first page is a copy elsewhere
                s.table[S - 1, 0] = s.table[S - 1, 21]
            if i == 25:                         # other groups, of which one is empty
                s.group.copy_(i32([0, S // 2]))
        want = eager.step()
        kept.workspace.fill_(255)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i
        shared = [320] * S if i < 15 else [0] * S if i < 25 or S == 3 else [320] * (S // 2) + [0] * (S - S // 2)
        assert want[2].tolist() == shared and want[4].tolist() == [320 + i] * S
    assert torch.equal(eager.kv, kept.kv) and torch.equal(eager.table, kept.table)
    assert torch.equal(eager.cache[0].view(torch.uint8), kept.cache[0].view(torch.uint8))


def test_two_at_once():
    """Two batches on two streams, each with a workspace of its own, many times over."""
    xs = [case([(60, [(20, 1)] * 40)], 16, 2, 128, 16, BF16, "e4m3", seed=71),
          case([(30, [(9, 3), (40, 5), (8, 8)] * 3), (9, [(5, 1)] * 7)], 8, 2, 128, 32, BF16, "int8", seed=72)]
    ds = [on_gpu(x) for x in xs]
    want = [attend(x, d) for x, d in zip(xs, ds)]
    for x, w in zip(xs, want):
        check(x, w)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(attend(xs[i], ds[i]))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert all(torch.equal(a, w[0]) and torch.equal(b, w[1]) for a, b in many)


def test_two_graphs_over_one_workspace():
    xs = [case([(60, [(20, 1)] * 40)], 16, 2, 128, 16, BF16, "e4m3", seed=73),
          case([(30, [(9, 3), (40, 5), (8, 8)] * 3)], 8, 2, 128, 32, BF16, "e4m3", seed=74)]
    ds = [on_gpu(x) for x in xs]
    want = [attend(x, d) for x, d in zip(xs, ds)]
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for x, d in zip(xs, ds):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(attend(x, d, workspace=ws))
        graphs.append(g)
    for _ in range(5):
        for g, o, w in zip(graphs, got, want):
            o[0].zero_()
            g.replay()
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
