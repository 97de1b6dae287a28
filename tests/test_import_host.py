"""The package imports on a torch built without CUDA."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_training_operators_import_on_a_torch_without_cuda():
    code = """
import torch
for n in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, n)
from spherical_disco_convolution_b200 import conv, muon, norm
try:
    norm.layer_norm(torch.zeros(1, 2, 3, 4))
except ValueError as e:
    print("refused", e)
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.startswith("refused"), run.stderr[-2000:]
