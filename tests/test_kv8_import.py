"""The binding can be imported on a torch build without CUDA."""
from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_the_cuda_bindings():
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_getCurrentRawStream')]:\n"
            "    delattr(torch._C, n)\n"
            "import gated_delta_rule_gdr_gb300 as gdr\n"
            "assert gdr.kv8_attn and gdr.chunk_fwd\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
