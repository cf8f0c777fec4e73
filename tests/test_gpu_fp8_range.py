"""The 8-bit product over the whole range of its scales, against the fp64 oracle.

Tolerances as for ordinary scales: float32 results (KB + 32) 2^-24 of the sum of
|terms|, bfloat16 results 2^-8 of the value and 2^-13 of that sum; blocks whose
products are exactly zero add nothing to either.  Below float32's normal range
the product of two scales is rounded within 2^-150 and multiplies a block sum
of at most 128 * 448^2 < 2^24.7, so each block may add 2^-125."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, f64, note, require_gpu
from oracle import fp8_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# few rows with tiles of one to four row fragments, in chunks, K split; 128 x 128 tiles whole and K split; large tiles
SHAPES = [(1, 16, 128), (5, 300, 400), (40, 77, 272), (64, 48, 16400), (130, 512, 400), (300, 1700, 272),
          (300, 1700, 4112), (4133, 4366, 272)]


def _check(a, b, form, out, KB):
    av = O.values(f64(a[0]), a[1].cpu().numpy(), 1, 128)
    bv = O.values(f64(b[0]), b[1].cpu().numpy(), 128 if form == "tiles" else 1, 128)
    y = f64(E.fp8_matmul(*a, *b, out_dtype=out))
    ref, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    tol = (KB + 32) * 2.0 ** -24 * mag if out == F32 else 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * mag
    assert np.isfinite(ref).all() and np.isfinite(y).all()
    assert np.all(np.abs(y - ref) <= tol + KB * 2.0 ** -125), np.max(np.abs(y - ref) / (tol + KB * 2.0 ** -125))
    return ref


def _quantized(a, b, form):
    return E.fp8_quantize(a.to(DEV)), (E.fp8_quantize_weight if form == "tiles" else E.fp8_quantize)(b.to(DEV))


@pytest.mark.parametrize("form", ["tiles", "rows"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_large_blocks_that_do_not_meet(M, N, K, out, form):
    """The first block of both sides is large, in columns that the other side leaves empty: it adds exactly nothing."""
    require_gpu()
    g = torch.Generator().manual_seed(M + K)
    for ea, eb in ((76, 76), (120, 40)):
        note(f"range disjoint {M}x{N}x{K} {form} {out} 2^{ea} 2^{eb}")
        a, b = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
        a[:, :64] *= 2.0 ** ea
        a[:, 64:128] = 0
        b[:, :64] = 0
        b[:, 64:128] *= 2.0 ** eb
        _check(*_quantized(a, b, form), form, out, (K + 127) // 128)


@pytest.mark.parametrize("form", ["tiles", "rows"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_small_values_of_large_blocks(M, N, K, out, form):
    """Values far below their block's largest, whose products are within float32 though the product of the scales is not."""
    require_gpu()
    note(f"range finite {M}x{N}x{K} {form} {out}")
    g = torch.Generator().manual_seed(M + K)
    a, b = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    a[:, :64] *= 2.0 ** 74
    a[:, 64:128] = 0
    b[:, :63] = 0
    b[:, 64:128] *= 2.0 ** 75
    a[:, 63], b[:, 63] = 2.0 ** 62, 2.0 ** 63
    ref = _check(*_quantized(a, b, form), form, out, (K + 127) // 128)
    assert np.abs(ref).min() > 2.0 ** 120


@pytest.mark.parametrize("form", ["tiles", "rows"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(5, 300, 400), (300, 1700, 272)])
def test_small_scales(M, N, K, out, form):
    require_gpu()
    g = torch.Generator().manual_seed(M + K)
    for ea, eb in ((-60, -58), (-90, -40), (-101, 90), (-130, 0)):
        note(f"range small {M}x{N}x{K} {form} {out} 2^{ea} 2^{eb}")
        a, b = torch.randn(M, K, generator=g) * 2.0 ** ea, torch.randn(N, K, generator=g) * 2.0 ** eb
        a[0], b[:128] = 0, 0
        _check(*_quantized(a, b, form), form, out, (K + 127) // 128)


@pytest.mark.parametrize("form", ["tiles", "rows"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(5, 300, 400), (300, 1700, 272), (4133, 4366, 272)])
def test_rows_with_infinities_beside_large_blocks(M, N, K, out, form):
    """A block that holds an infinity or NaN makes its row NaN, whatever the size of the others' scales."""
    require_gpu()
    note(f"range non-finite {M}x{N}x{K} {form} {out}")
    g = torch.Generator().manual_seed(M)
    a, b = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    a[:, :64] *= 2.0 ** 76
    a[:, 64:128] = 0
    b[:, :64] = 0
    b[:, 64:128] *= 2.0 ** 76
    a[1, 3], a[M - 1, K - 1] = float("inf"), float("nan")
    aq, bq = _quantized(a, b, form)
    y = E.fp8_matmul(*aq, *bq, out_dtype=out)
    bad = torch.zeros(M, dtype=torch.bool, device=DEV)
    bad[1] = bad[M - 1] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("form", ["tiles", "rows"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(40, 300, 400), (300, 1700, 272)])
def test_one_large_row_beside_an_infinite_one(M, N, K, out, form):
    """Rows 17 and 33 hold large finite blocks, row 1 an infinity: the first two are still the formula's."""
    require_gpu()
    note(f"range one row {M}x{N}x{K} {form} {out}")
    g = torch.Generator().manual_seed(M)
    a, b = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    for r in (17, 33):
        a[r, :64] *= 2.0 ** 120
        a[r, 64:128] = 0
    a[1, 5] = float("inf")
    b[:, :64] = 0
    b[:, 64:128] *= 2.0 ** 30
    (aq, sa), bq = _quantized(a, b, form)
    y = E.fp8_matmul(aq, sa, *bq, out_dtype=out)
    assert torch.isnan(y[1]).all()
    keep = torch.arange(M, device=DEV) != 1
    assert torch.isfinite(y[keep]).all()
    _check((aq[keep].contiguous(), sa[keep].contiguous()), bq, form, out, (K + 127) // 128)
    clean = E.fp8_matmul(aq[keep].contiguous(), sa[keep].contiguous(), *bq, out_dtype=out)
    av = O.values(f64(aq[keep]), sa[keep].cpu().numpy(), 1, 128)
    assert np.all(np.abs(f64(y[keep]) - f64(clean)) <= 2.0 ** -7 * np.abs(f64(clean)) + 2.0 ** -12 * (
        np.abs(av) @ np.abs(O.values(f64(bq[0]), bq[1].cpu().numpy(), 128 if form == "tiles" else 1, 128)).T))
