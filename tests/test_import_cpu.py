"""The package imports beside a torch without CUDA's private names (a build for CPUs)."""
import os
import subprocess
import sys

import rotational_w4a4_quantization_gb300 as rq

CODE = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import rotational_w4a4_quantization_gb300 as rq
turns, _ = rq.rope_turns(64, device="cpu")
try:
    rq.rope(torch.zeros(1, 1, 64), None, torch.zeros(1, dtype=torch.int64), turns)
except (ValueError, ImportError) as e:
    print("refused:", e)
"""


def test_import_without_private_names():
    root = os.path.dirname(os.path.dirname(rq.__file__))
    r = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused:" in r.stdout, r.stderr
