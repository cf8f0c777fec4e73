"""GPU tests of the norm's, the routing's and the 4-bit operators' edges."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, f64, note, require_gpu
from oracle import expert_block_oracle as O

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.mark.parametrize("M,N,K", [(20, 32, 608), (400, 2000, 608), (12288, 4096, 608)])
def test_products_by_expert_of_no_rows(M, N, K):
    """Every index lies outside a left operand without rows: rows of zeros, several steps of K, each kernel."""
    require_gpu()
    note(f"mx grouped without rows of a {M}x{N}x{K}")
    b = torch.randint(0, 256, (3, N, K // 2), generator=torch.Generator().manual_seed(0)).to(U8).to(DEV)
    sb = torch.full((3, N, K // 32), 127, dtype=U8, device=DEV)
    rows = (torch.arange(M) % 7 - 3).int().to(DEV)
    offsets = torch.tensor([0, M // 4, M // 2, M - 2], dtype=torch.int32, device=DEV)
    out = torch.full((M, N), 5.0, device=DEV)
    a, sa = torch.empty(0, K // 2, dtype=U8, device=DEV), torch.empty(0, K // 32, dtype=U8, device=DEV)
    E.mxfp4_grouped_matmul(a, sa, b, sb, offsets, rows=rows, out=out)
    assert not out[:M - 2].any() and (out[M - 2:] == 5).all()
