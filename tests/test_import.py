"""The package imports, and refuses as everywhere, under a PyTorch build without CUDA's
private functions (a CPU-only one has none of them)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import torch
for n in [n for n in dir(torch._C) if n.startswith("_cuda_") or n.startswith("_Cuda")]:
    delattr(torch._C, n)
from test_sequence_layers_gb300 import abi, rotary
assert rotary.rope_table(4, 8, device="cpu").shape == (4, 4, 2)
try:
    abi.ttt_rope(torch.zeros(1, 1, 4, 8), None, None, rotary.rope_table(4, 8, device="cpu"))
except ValueError as e:
    print("refused:", e)
"""


def test_import_without_cuda_functions():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused: q must be a CUDA tensor" in r.stdout, r.stderr
