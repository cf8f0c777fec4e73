"""GPU parity of the 4-bit values with a power of two per 32 elements: codes, exponents
and values are defined to the bit and compared so."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, note, require_gpu
from oracle import expert_block_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _x(rows, cols, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.7 * torch.randn(cols, generator=g))
    if kind == "wide":      # from subnormals of float32 to the largest values, blocks of zeros
        x = torch.sign(x) * torch.exp2(torch.randint(-149, 128, (rows, cols), generator=g).float()) * \
            (1 + torch.randint(0, 2, (rows, cols), generator=g) * 0.75)
        x[:, :32] = 0
    if kind == "ties":      # at and beside the middles between neighbouring values
        x = torch.randint(-32, 33, (rows, cols), generator=g).float() / 4
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (128, 128), (37, 2048), (300, 1056), (5, 5504), (2049, 512)])
def test_codes_and_values(rows, cols, dtype):
    require_gpu()
    for kind in ("normal", "wide", "ties"):
        note(f"mxfp4 {rows}x{cols} {dtype} {kind}")
        x = _x(rows, cols, dtype, rows + cols, kind)
        q, s = E.mxfp4_quantize(x.to(DEV))
        codes, e = O.mx_quantize(x.float().numpy())
        assert q.shape == (rows, cols // 2) and s.shape == (rows, cols // 32)
        assert np.array_equal(s.cpu().numpy(), e)
        assert np.array_equal(q.cpu().numpy(), O.mx_pack(codes))
        want = O.mx_values(O.mx_pack(codes), e)
        for out in (F32, BF):
            v = E.mxfp4_dequantize(q, s, out)
            assert v.dtype == out and np.array_equal(v.double().cpu().numpy(), want)
        assert np.array_equal(E.mxfp4_dequantize(q, s).double().cpu().numpy(), want)


def test_every_code_and_exponent():
    require_gpu()
    note("mxfp4 all codes and exponents")
    q = (torch.arange(16, dtype=torch.uint8).repeat(256, 1)) * 17    # each code twice a byte, 32 of a block
    s = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(256, 1)
    for out in (F32, BF):
        v = E.mxfp4_dequantize(q.to(DEV), s.to(DEV), out).cpu()
        assert torch.isnan(v[255]).all()
        want = O.mx_values(q[:255].numpy(), s[:255].numpy())
        with np.errstate(over="ignore"):
            want = np.where(np.abs(want) > 3.4e38, np.copysign(np.inf, want), want)
        assert np.array_equal(v[:255].double().numpy(), want)


def test_non_finite_blocks_only():
    require_gpu()
    note("mxfp4 non-finite")
    for dtype in (F32, BF):
        x = _x(6, 128, dtype, 3)
        clean = E.mxfp4_quantize(x.to(DEV))
        x[1, 40], x[2, 0], x[3, 127] = float("nan"), float("inf"), float("-inf")
        q, s = E.mxfp4_quantize(x.to(DEV))
        bad = torch.zeros(6, 4, dtype=torch.bool)
        bad[1, 1] = bad[2, 0] = bad[3, 3] = True
        assert torch.equal(s.cpu() == 255, bad)
        assert torch.equal(s.cpu()[~bad], clean[1].cpu()[~bad])
        qb, cb = q.cpu().view(6, 4, 16), clean[0].cpu().view(6, 4, 16)
        assert torch.equal(qb[~bad], cb[~bad]) and not qb[bad].any()
        assert torch.equal(torch.isnan(E.mxfp4_dequantize(q, s)).cpu().view(6, 4, 32).all(-1), bad)


def test_leading_shapes_and_empty():
    require_gpu()
    note("mxfp4 shapes")
    x = _x(24, 64, BF, 1).to(DEV)
    q, s = E.mxfp4_quantize(x)
    q3, s3 = E.mxfp4_quantize(x.view(2, 3, 4, 64))
    assert q3.shape == (2, 3, 4, 32) and torch.equal(q3.view(24, 32), q) and torch.equal(s3.view(24, 2), s)
    assert torch.equal(E.mxfp4_dequantize(q3, s3).view(24, 64), E.mxfp4_dequantize(q, s))
    q0, s0 = E.mxfp4_quantize(x[:0])
    assert q0.shape == (0, 32) and E.mxfp4_dequantize(q0, s0).shape == (0, 64)
