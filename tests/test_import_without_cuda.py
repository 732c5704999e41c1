"""The binding imports, and answers what needs no GPU, on a torch built without
CUDA (its C module then lacks the lookups of the current stream)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import sys
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
sys.path.insert(0, sys.argv[1])
from block_scaled_fp4_tcgen05_gb300 import qfp4
print(len(qfp4.SIGNATURES), qfp4._stream(5), end="")
"""


def test_import():
    r = subprocess.run([sys.executable, "-c", PROGRAM, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    from block_scaled_fp4_tcgen05_gb300 import qfp4
    assert r.stdout == f"{len(qfp4.SIGNATURES)} 5"
