"""gdr_last_device_error reads the words of the attention kernels that a process has used, no others: a word
that is read loads its kernels' code, and every one is a copy of its own.  The copies are told by their time,
the least of many, in a process of its own: at first no word of the five units of attention kernels over the
8-bit cache is read, after two passes over a shared prefix two are, of ten in all.  Ten equal copies and a
stream's synchronisation against eight: 0.8 to 1; 0.95 leaves room for noise in the least of 40 rounds."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import time
import torch
import gated_delta_rule_gdr_gb300 as gdr

def least():
    best = 1.0
    for _ in range(40):
        begin = time.perf_counter()
        for _ in range(20):
            assert gdr.last_device_error() == 0
        best = min(best, (time.perf_counter() - begin) / 20)
    return best

def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")

torch.zeros(1, device="cuda")
before = least()
S = 20
cache = [torch.ones((2 + S, 1, 16, 64), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
scale = [torch.ones((2 + S, 1), device="cuda") for _ in range(2)]
table, kv, group = i32([[0, 1, 2 + s] for s in range(S)]), i32([40] * S), i32([0, S])
q = torch.ones((S, 2, 64), device="cuda").bfloat16()
with gdr.option(shared_least=1):
    plan = gdr.kv8_shared_plan(table, kv, group, 16)
    call = lambda: gdr.kv8_attn_shared(q, *cache, *scale, table, kv, 0.1, group, *plan, max_group_q=S)
    call()
    after = least()
    with gdr.option(wait_limit_ns=0):
        call()
    assert gdr.last_device_error() == 5 and gdr.last_device_error() == 0
print(before, after)
"""


def test_words_of_kernels_that_have_not_run_are_not_read():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_gdr_gb300 as gdr
    gdr.load(build_if_missing=True)
    out = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    before, after = map(float, out.stdout.split())
    assert before <= 0.95 * after, (before, after)
