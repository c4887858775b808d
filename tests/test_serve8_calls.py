"""Calls of the 8-bit serving wrappers that have to be refused or answered before anything runs on a GPU."""
import os
import subprocess
import sys

import pytest
import torch

from semi_structured_sparsity_online_b200 import ss24

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def int8_rows(rows, k):
    return {"values": torch.zeros(rows, k, dtype=torch.int8), "scales": torch.ones(rows, 1)}


def test_gemm_int8_refuses_a_sparse_operand():
    """A 2:4 or 4:8 INT8 pass has int8 values of k / 2 columns and one scale per row too; its metadata says which
    columns they are."""
    sparse = {**int8_rows(4, 64), "meta": torch.zeros(4, 16, dtype=torch.uint8)}
    for a, b in ((sparse, sparse), (sparse, int8_rows(4, 64)), (int8_rows(4, 64), sparse)):
        with pytest.raises(ValueError, match="dense"):
            ss24.gemm_int8(a, b)


def test_the_binding_imports_without_a_cuda_build_of_torch():
    """A torch that was built without CUDA lacks the private functions that read the current stream and device; the
    module imports there and its host-side checks answer."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from semi_structured_sparsity_online_b200 import ss24
i8 = {"values": torch.zeros(4, 64, dtype=torch.int8), "scales": torch.ones(4, 1)}
try:
    ss24.gemm_int8(i8, {"values": torch.zeros(4, 32, dtype=torch.int8), "scales": torch.ones(4, 1)})
except ValueError as e:
    assert "differ in k" in str(e)
else:
    raise AssertionError("accepted")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_attention_refuses_a_scale_that_overflows(scale):
    """The kernels take the scale times log2(e) in binary32."""
    from test_serve8_host import ARG, attend
    assert attend(scale=scale) == ARG
