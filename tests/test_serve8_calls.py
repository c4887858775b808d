"""Calls of the 8-bit serving wrappers that have to be refused or answered before anything runs on a GPU."""
import pytest
import torch

from semi_structured_sparsity_online_b200 import ss24


def int8_rows(rows, k):
    return {"values": torch.zeros(rows, k, dtype=torch.int8), "scales": torch.ones(rows, 1)}


def test_gemm_int8_refuses_a_sparse_operand():
    """A 2:4 or 4:8 INT8 pass has int8 values of k / 2 columns and one scale per row too; its metadata says which
    columns they are."""
    sparse = {**int8_rows(4, 64), "meta": torch.zeros(4, 16, dtype=torch.uint8)}
    for a, b in ((sparse, sparse), (sparse, int8_rows(4, 64)), (int8_rows(4, 64), sparse)):
        with pytest.raises(ValueError, match="dense"):
            ss24.gemm_int8(a, b)
