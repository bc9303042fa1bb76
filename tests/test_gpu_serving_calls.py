"""The serving operators' calls as a program makes them: under transforms, from several threads, in several graphs and
among calls that overlap."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_tensor_without_data_raises():
    """Tensors inside torch.vmap have no address: an error, after which the process goes on."""
    code = """
import torch
import bit_quantized_gemv_dequant_gb300 as qg
x = torch.ones(3, 4, 256, device="cuda")
for i in range(2):
    try:
        torch.vmap(lambda x: qg.quantize_fp8_b128(x))(x)
    except RuntimeError:
        print("raised")
codes, scales = qg.quantize_fp8_b128(x[0])
assert (codes.float() == 448).all() and qg.device_error() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["raised", "raised"], (r.returncode, r.stdout, r.stderr[-2000:])
