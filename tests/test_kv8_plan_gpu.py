"""gdr_page_plan on the GPU where requests do not hold plain rows of pages, against the integer
oracle: pages that are gone, lengths beyond the table, pages held beyond the length.  All
outputs are whole numbers: equal."""
from __future__ import annotations

import random
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_gdr_gb300 as gdr
from oracle import kv8 as O

pytestmark = pytest.mark.gpu
NAMES = ("kv", "cu", "slots", "pos", "granted", "state", "table", "ring")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load(build_if_missing=True)
    yield
    assert gdr.last_device_error() == 0


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def check_plan(kv, q, table, ring, state, page, T):
    t, r = i32(table), i32(ring)
    got = gdr.page_plan(i32(kv), i32(q), t, r, i32(state), page, T)
    want = O.plan(kv, q, table, ring, state, page, T)
    for g, w, name in zip((*got, t, r), want, NAMES):
        assert np.array_equal(g.cpu().numpy(), np.asarray(w)), name
    return [np.asarray(w) for w in want]


def pool(S, W, page, seed, *, kv_max, q_max, finished, free, markers, gone):
    """Requests over a shuffled pool whose entries are `markers` here and there."""
    r = random.Random(seed)
    kv = [r.randint(0, kv_max) for _ in range(S)]
    q = [-1 if r.random() < finished else r.randint(0, q_max) for _ in range(S)]
    N = sum(-(-k // page) for k in kv) + free
    perm = list(range(N))
    r.shuffle(perm)
    table, it = np.full((S, W), -7), iter(perm)
    for s, k in enumerate(kv):
        for i in range(-(-k // page)):
            table[s, i] = next(it)
            if r.random() < gone:
                table[s, i] = r.choice(markers) if r.random() < 0.9 else N
    head, ring = r.randrange(N), np.full(N, -3)
    for i, p in enumerate(it):
        ring[(head + i) % N] = p
    return kv, q, table, ring, [head, free], sum(n for n in q if n > 0) + 5


# ------------------------------------------------------------------ pages that are gone
def test_a_finished_request_gives_back_the_pages_it_has():
    """Pages of 16.  Request 0 ends with the pages 5, gone, 6; request 1 takes four free ones.
    The next call hands out 5 and 6, and then there are no more."""
    table, ring = i32([[5, -1, 6, -1, -1], [-1] * 5]), i32([0, 1, 2, 3, -1, -1, -1, -1])
    kv, _, slots, _, ok, state = gdr.page_plan(i32([48, 0]), i32([-1, 64]), table, ring, i32([0, 4]), 16, 64)
    assert ok.tolist() == [1, 1] and kv.tolist() == [0, 64]
    assert slots.tolist() == list(range(64)) and table[1].tolist() == [0, 1, 2, 3, -1]
    assert state.tolist() == [4, 2] and ring.tolist()[4:6] == [5, 6]
    kv, _, slots, _, ok, state = gdr.page_plan(kv, i32([32, 0]), table, ring, state, 16, 32)
    assert ok.tolist() == [1, 1] and slots.tolist() == list(range(80, 112)) and state.tolist() == [6, 0]
    _, _, slots, _, ok, _ = gdr.page_plan(kv, i32([1, 0]), table, ring, state, 16, 1)
    assert ok.tolist() == [0, 1] and slots.tolist() == [-1]


@pytest.mark.parametrize("S,W,page,kv_max,finished,gone", [
    (1, 40, 16, 640, 1.0, 0.3), (7, 1500, 16, 24000, 0.6, 0.02), (300, 40, 64, 2500, 0.3, 0.1),
    (1500, 20, 32, 600, 0.5, 0.3), (9, 700, 128, 89000, 1.0, 1.0), (60, 300, 16, 4800, 0.5, 0.0),
    (8192, 3, 16, 48, 0.4, 0.2), (300, 2000, 16, 3000, 0.5, 0.1), (8192, 70, 16, 100, 0.3, 0.2), (600, 900, 32, 9000, 0.3, 0.0),
])
def test_gone_pages_do_not_come_back(S, W, page, kv_max, finished, gone):
    check_plan(*pool(S, W, page, S + W, kv_max=kv_max, q_max=0, finished=finished, free=50,
                     markers=[-1, -2 ** 31, 2 ** 31 - 1], gone=gone)[:5], page, 5)


@pytest.mark.parametrize("marker", [-1, 40, 1 << 26, -(1 << 26), 2 ** 31 - 1])
def test_tokens_of_a_gone_page_have_no_slot(marker):
    """Request 0's partly filled page is gone: its next tokens have no place (1 << 26 times 64
    would wrap to slot 0 of another request's page), those past it do."""
    table = np.full((2, 4), -1)
    table[0, :2], table[1, 0] = (3, marker), 0
    got = check_plan([70, 10], [60, 2], table, np.arange(40) % 7 + 10, [0, 7], 64, 64)
    slots, pos = got[2], got[3]
    assert (slots[:58] == -1).all() and (pos[:58] == -1).all()
    assert slots[58:62].tolist() == [640, 641, 10, 11] and pos[58:62].tolist() == [128, 129, 10, 11]


@pytest.mark.parametrize("S,W,page", [(5, 30, 16), (200, 40, 32), (1000, 12, 64)])
def test_gone_pages_at_random(S, W, page):
    check_plan(*(x := pool(S, W, page, S, kv_max=(W - 3) * page, q_max=3 * page, finished=0.1, free=2 * S,
                           markers=[-1, 1 << 26, -(1 << 26)], gone=0.3))[:5], page, x[5])


# ------------------------------------------------------------------ lengths beyond the table
def test_a_length_beyond_the_table_is_not_granted():
    """Two columns of pages of 16.  A request whose length is past them is refused and keeps its
    length, even without new tokens; at its end the pages of its row return."""
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 7]])
    got = check_plan([33, 40, 100, 32], [0, 3, -1, 0], table, np.full(12, 8), [0, 4], 16, 8)
    assert got[0].tolist() == [33, 40, 0, 32] and got[4].tolist() == [0, 0, 1, 1] and got[5].tolist() == [0, 6]
    assert (got[2] == -1).all()
    check_plan([2 ** 31 - 1, 5], [2 ** 31 - 1, 1], table[:2], np.full(12, 8), [3, 4], 16, 8)


# ------------------------------------------------------------------ calls of several threads
def test_threads_plan_batches_of_different_sizes():
    """A launch's shared-memory limit belongs to the kernel, not to the call: one thread's small
    batch does not take it from another's large one."""
    lib, codes = gdr.load(), set()

    def work(S):
        z = torch.zeros(S, dtype=torch.int32, device="cuda")
        table, ring = torch.full((S, 1), -1, dtype=torch.int32, device="cuda"), i32([0, 1])
        out = [torch.zeros(S + 8, dtype=torch.int32, device="cuda") for _ in range(4)]
        state, stream = i32([0, 2]), torch.cuda.Stream()
        ptr = [t.data_ptr() for t in (z, z, table, ring, state, out[0], out[1], z, z, out[2], out[3])]
        torch.cuda.synchronize()
        start.wait()
        for i in range(4000):
            codes.add(lib.gdr_page_plan(*ptr, S, 1, 16, 2, 0, stream.cuda_stream))
            if i % 500 == 0:
                stream.synchronize()
        stream.synchronize()

    start = threading.Barrier(2)
    threads = [threading.Thread(target=work, args=(S,)) for S in (8192, 2000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert codes == {0}


# ------------------------------------------------------------------ pages held beyond the length
def test_refused_drafts_keep_their_pages():
    """15 tokens in pages of 16 and three drafts a step that are refused each time: the page that
    the first drafts crossed into stays the request's, and returns at its end."""
    kv, held, state = i32([15]), i32([1]), i32([0, 3])
    table, ring = i32([[3, -1, -1]]), i32([0, 1, 2, -1])
    for _ in range(5):
        out = gdr.page_plan(kv, i32([3]), table, ring, state, 16, 3, held)
        assert out[0].tolist() == [18] and out[2].tolist() == [63, 0, 1] and out[4].tolist() == [1]
        state, held = out[5], out[6]
        assert state.tolist() == [1, 2] and held.tolist() == [2] and table.tolist() == [[3, 0, -1]]
    out = gdr.page_plan(kv, i32([-1]), table, ring, state, 16, 3, held)
    assert out[5].tolist() == [1, 4] and out[6].tolist() == [0] and ring.tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("S,W,page,seed", [(1, 9, 16, 1), (40, 30, 16, 2), (300, 40, 32, 3), (1300, 16, 128, 4), (270, 2000, 16, 5)])
def test_held_pages_equal_oracle(S, W, page, seed):
    r = random.Random(seed)
    used, kv, q, held = 0, [], [], []
    for _ in range(S):
        has = r.randint(0, min(W, 60))
        kv.append(r.randint(0, has * page) if r.random() < 0.9 else W * page + 3)
        held.append(has if r.random() < 0.9 else r.choice([0, W + 5, -4]))
        q.append(-1 if r.random() < 0.2 else r.randint(0, 4 * page))
        used += W
    N = used + 2 * S
    perm = r.sample(range(N), N)
    table, ring, head = np.array(perm[:used]).reshape(S, W), np.full(N, -3), r.randrange(N)
    for i, p in enumerate(perm[used:]):
        ring[(head + i) % N] = p
    T = sum(n for n in q if n > 0)
    t, g = i32(table), i32(ring)
    got = gdr.page_plan(i32(kv), i32(q), t, g, i32([head, 2 * S]), page, T, i32(held))
    want = O.plan(kv, q, table, ring, [head, 2 * S], page, T, held)
    for a, b, name in zip((*got[:6], t, g, got[6]), want, (*NAMES, "held")):
        assert np.array_equal(a.cpu().numpy(), np.asarray(b)), name


def test_no_page_is_lost_while_drafts_are_refused():
    """Forty steps of twenty requests that draft up to eight tokens, keep some, end and return:
    the free pages and the held ones are all the pages, each once, after every step."""
    r = random.Random(9)
    S, W, page, N = 20, 12, 16, 150
    kv, held, state = i32([0] * S), i32([0] * S), i32([5, N])
    table, ring = torch.full((S, W), -1, dtype=torch.int32, device="cuda"), i32(r.sample(range(N), N))
    for _ in range(40):
        q = [-1 if r.random() < 0.06 else r.randint(0, 8) if r.random() < 0.8 else r.randint(0, 40) for _ in range(S)]
        before = kv.tolist()
        kv, _, _, _, ok, state, held = gdr.page_plan(kv, i32(q), table, ring, state, page, sum(n for n in q if n > 0), held)
        h, (head, count) = held.tolist(), state.tolist()
        pages = [p for s in range(S) for p in table[s, :h[s]].tolist()] + [ring[(head + i) % N].item() for i in range(count)]
        assert sorted(pages) == list(range(N))
        kept = [r.randint(b, max(a, b)) if n >= 0 else 0 for a, b, n in zip(kv.tolist(), before, q)]
        kv = i32(kept)
