"""GPU parity of the 4-bit products against float64 products of the values.

A block of 32 sums exactly and 128 elements are added to the accumulator with an error
of at most 2^-22 of the sum of their |terms| and its own (measured: 2^-22.5), over
K/128 of them and at most 24 additions of parts: |error| <= (K / 128 + 24) 2^-22 of the
sum of all |terms|; a bfloat16 result adds its rounding, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, note, require_gpu
from oracle import expert_block_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _operand(rows, K, seed, spread=6):
    """Random codes (all of them) and exponents."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (rows, K // 2), generator=g).to(torch.uint8)
    s = torch.randint(127 - spread, 128 + spread, (rows, K // 32), generator=g).to(torch.uint8)
    return q, s


def _vals(q, s):
    return torch.from_numpy(O.mx_values(q.numpy(), s.numpy()))


def _close(y, want, mag, K, dtype):
    got = y.double().cpu()
    tol = (K / 128 + 24) * 2.0 ** -22 * mag + (2.0 ** -8 * want.abs() if dtype == BF else 2.0 ** -24 * want.abs())
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((got - want).abs().max()))


SHAPES = [(1, 16, 32), (1, 11008, 2048), (3, 40, 96), (16, 16, 128), (17, 100, 160), (33, 72, 512), (37, 2048, 5504),
          (49, 17, 1056), (64, 64, 4096), (65, 256, 544), (100, 33, 64), (200, 300, 1376), (129, 4096, 288),
          (300, 4097, 320), (513, 2049, 256), (640, 2056, 800), (1000, 4608, 2080), (2050, 8200, 256), (4096, 4100, 608),
          (2500, 5504, 608), (6000, 8201, 160), (6000, 8204, 32), (6000, 8200, 96),
          (130, 1500, 4128), (2, 48, 65536), (64, 512, 16384), (33, 77, 40032), (300, 1024, 8192), (513, 701, 7200), (700, 1001, 9696)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K, dtype):
    require_gpu()
    note(f"mx matmul {M}x{N}x{K} {dtype}")
    a, b = _operand(M, K, M + K), _operand(N, K, N + K + 1)
    d = [t.to(DEV) for t in (*a, *b)]
    ws = {}
    y = E.mxfp4_matmul(*d, out_dtype=dtype, workspace=ws)
    av, bv = _vals(*a), _vals(*b)
    _close(y, av @ bv.t(), av.abs() @ bv.abs().t(), K, dtype)
    again = E.mxfp4_matmul(*d, out_dtype=dtype, workspace=ws)
    assert torch.equal(y, again)


def test_quantised_operands_and_out():
    require_gpu()
    note("mx matmul of quantised data")
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(70, 768, generator=g), torch.randn(512, 768, generator=g)
    (aq, sa), (bq, sb) = E.mxfp4_quantize(x.to(DEV)), E.mxfp4_quantize(w.to(DEV).bfloat16())
    out = torch.full((72, 512), 7.0, device=DEV)
    E.mxfp4_matmul(aq, sa, bq, sb, out=out[:70])
    av, bv = E.mxfp4_dequantize(aq, sa, F32).double().cpu(), E.mxfp4_dequantize(bq, sb, F32).double().cpu()
    _close(out[:70], av @ bv.t(), av.abs() @ bv.abs().t(), 768, F32)
    assert (out[70:] == 7).all()
    # the quantised product is the product, to a few per cent
    assert ((out[:70].cpu() - x @ w.t()).norm() / (x @ w.t()).norm()) < 0.2


def test_wide_exponents_and_nan_blocks():
    require_gpu()
    for M, N in ((20, 48), (500, 3000), (2500, 5504)):
        note(f"mx matmul wide exponents {M}x{N}")
        K = 416
        a, b = _operand(M, K, 1, 40), _operand(N, K, 2, 40)
        av, bv = _vals(*a), _vals(*b)
        y = E.mxfp4_matmul(*(t.to(DEV) for t in (*a, *b)), out_dtype=F32)
        _close(y, av @ bv.t(), av.abs() @ bv.abs().t(), K, F32)
        a[1][3, 5] = 255
        b[1][7, K // 32 - 1] = 255          # the last block, beside the next row's first
        z = E.mxfp4_matmul(*(t.to(DEV) for t in (*a, *b)), out_dtype=F32)
        bad = torch.zeros(M, N, dtype=torch.bool)
        bad[3] = True
        bad[:, 7] = True
        assert torch.equal(torch.isnan(z).cpu(), bad)
        assert torch.equal(z.cpu()[~bad], y.cpu()[~bad])


def test_nan_of_the_next_row_stays_there():
    """Exponent rows start at any byte and are read in dwords: none of a neighbour's reaches a row."""
    require_gpu()
    note("mx matmul neighbours")
    for M, N, K in ((40, 64, 32), (40, 64, 96), (700, 1600, 160), (6000, 8192, 160)):
        a, b = _operand(M, K, 1), _operand(N, K, 2)
        y = E.mxfp4_matmul(*(t.to(DEV) for t in (*a, *b)), out_dtype=F32).cpu()
        a[1][1::2] = 255
        b[1][0::2] = 255
        z = E.mxfp4_matmul(*(t.to(DEV) for t in (*a, *b)), out_dtype=F32).cpu()
        assert torch.equal(z[0::2, 1::2], y[0::2, 1::2])
        assert torch.isnan(z[1::2]).all() and torch.isnan(z[:, 0::2]).all()


GROUPED = [(1, 16, 32, [1]), (5, 40, 96, [0, 5, 0]), (7, 48, 160, [3, 0, 4]), (64, 128, 512, [1] * 64),
           (384, 272, 1024, None), (300, 100, 288, [70, 0, 17, 1, 49, 33, 64, 65]), (1000, 520, 352, [129, 600, 0, 1, 127, 128]),
           (2000, 1032, 544, [300, 256, 1400]), (2100, 136, 256, [2, 2000, 3]), (700, 77, 96, [0, 0, 690, 0]),
           (1000, 2056, 352, [129, 600, 0, 1, 127, 128]), (700, 1501, 96, [0, 0, 690, 0]), (2100, 1500, 416, [2, 2000, 3])]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("M,N,K,counts", GROUPED)
def test_grouped(M, N, K, counts, gather):
    require_gpu()
    g = torch.Generator().manual_seed(M + N)
    if counts is None:
        counts = torch.bincount(torch.randint(0, 70, (M,), generator=g), minlength=70).tolist()
    note(f"mx grouped {M}x{N}x{K} {len(counts)} experts gather={gather}")
    n_e, used = len(counts), sum(counts)
    offsets = torch.tensor([0] + counts).cumsum(0).int()
    R = max(1, M // 3) if gather else M
    a, b = _operand(R, K, 3), _operand(n_e * N, K, 4)
    rows = torch.randint(0, R, (M,), generator=g).int() if gather else None
    d = [t.to(DEV) for t in (*a, b[0].view(n_e, N, -1), b[1].view(n_e, N, -1), offsets)]
    av, bv = _vals(*a), _vals(*b).view(n_e, N, K)
    x = av if rows is None else av[rows.long()]
    for dtype in (BF, F32):
        out = torch.full((M, N), 5.0, dtype=dtype, device=DEV)
        y = E.mxfp4_grouped_matmul(*d, rows=None if rows is None else rows.to(DEV), out=out)
        assert y is out and (y[used:] == 5).all()          # rows behind the last expert's stay
        for e in range(n_e):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            _close(y[lo:hi], x[lo:hi] @ bv[e].t(), x[lo:hi].abs() @ bv[e].abs().t(), K, dtype)


def test_grouped_bad_rows_and_offsets():
    require_gpu()
    note("mx grouped bad rows, offsets past the ends")
    for M, N in ((20, 32), (400, 32), (400, 2000)):        # few rows in chunks of 16 and 64, tiles
        a, b = _operand(10, 64, 1), _operand(3 * N, 64, 2)
        rows = torch.arange(M).int() % 10
        rows[3], rows[4], rows[5] = -1, 10, 2 ** 31 - 1
        offsets = torch.tensor([-4, 6, M + 100, M + 100]).int()
        out = torch.full((M, N), 5.0, device=DEV)
        d = [t.to(DEV) for t in (*a, b[0].view(3, N, 32), b[1].view(3, N, 2))]
        E.mxfp4_grouped_matmul(*d, offsets.to(DEV), rows=rows.to(DEV), out=out)
        x = _vals(*a)[rows.long().clamp(0, 9)]
        x[3:6] = 0
        bv = _vals(*b).view(3, N, 64)
        want = torch.cat((x[:6] @ bv[0].t(), x[6:] @ bv[1].t()))
        assert torch.allclose(out.double().cpu(), want, rtol=1e-5, atol=1e-5)
        out.fill_(5.0)                                     # no rows at all
        E.mxfp4_grouped_matmul(*d, torch.zeros(4).int().to(DEV), rows=rows.to(DEV), out=out)
        assert (out == 5).all()


def test_empty():
    require_gpu()
    note("mx empty")
    u8 = dict(dtype=torch.uint8, device=DEV)
    y = E.mxfp4_matmul(torch.empty(0, 32, **u8), torch.empty(0, 2, **u8), torch.zeros(8, 32, **u8), torch.zeros(8, 2, **u8))
    assert y.shape == (0, 8)
    y = E.mxfp4_grouped_matmul(torch.zeros(4, 32, **u8), torch.zeros(4, 2, **u8), torch.zeros(2, 8, 32, **u8),
                               torch.zeros(2, 8, 2, **u8), torch.zeros(3, dtype=torch.int32, device=DEV),
                               rows=torch.empty(0, dtype=torch.int32, device=DEV))
    assert y.shape == (0, 8)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("counts,N,K", [([1024] * 8, 3000, 160), ([4000, 0, 300, 1, 255, 2049], 4100, 96),
                                        ([2100, 256, 4200, 3, 700], 4001, 544), ([5000, 3300], 3080, 1184)])
def test_large_tiles_by_expert(counts, N, K, gather):
    """Tiles of 256, several for a workgroup, exponents that start at any byte, rows outside a and behind the last expert's."""
    require_gpu()
    note(f"mx grouped large tiles {counts} {N} {K} gather={gather}")
    n_e, used = len(counts), sum(counts)
    M = used + 60
    assert E.mxfp4_grouped_matmul_workspace_size(M, N, K, n_e) > 0
    offsets = torch.tensor([0] + counts).cumsum(0).int()
    R = 777 if gather else M
    a, b = _operand(R, K, 3), _operand(n_e * N, K, 4)
    rows = torch.randint(0, R, (M,), generator=torch.Generator().manual_seed(N)).int() if gather else None
    if gather:
        rows[5], rows[used - 1] = -1, R
    d = [t.to(DEV) for t in (*a, b[0].view(n_e, N, -1), b[1].view(n_e, N, -1), offsets)]
    av, bv = _vals(*a), _vals(*b).view(n_e, N, K)
    x = av if rows is None else av[rows.long().clamp(0, R - 1)]
    if gather:
        x[5] = x[used - 1] = 0
    ws = {}
    for dtype in (BF, F32):
        out = torch.full((M, N), 5.0, dtype=dtype, device=DEV)
        E.mxfp4_grouped_matmul(*d, rows=None if rows is None else rows.to(DEV), out=out, workspace=ws)
        assert (out[used:] == 5).all()
        for e in range(n_e):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            _close(out[lo:hi], x[lo:hi] @ bv[e].t(), x[lo:hi].abs() @ bv[e].abs().t(), K, dtype)


@pytest.mark.parametrize("M,N,K,counts", [(60, 100, 288, [0, 50, 0, 10]), (64, 64, 96, [0, 0, 0, 64]), (160, 48, 544, [3] * 4 + [145] + [0] * 5 + [1] * 3),
                                          (1000, 4112, 64, [0] * 60 + [17, 900, 16, 33] + [0] * 10)])
def test_few_rows_with_a_crowded_expert(M, N, K, counts):
    """At most 16 rows for each expert on average, and more for some."""
    require_gpu()
    note(f"mx crowded expert {M} {N} {K}")
    n_e, used = len(counts), sum(counts)
    offsets = torch.tensor([0] + counts).cumsum(0).int()
    a, b = _operand(M, K, 3), _operand(n_e * N, K, 4)
    d = [t.to(DEV) for t in (*a, b[0].view(n_e, N, -1), b[1].view(n_e, N, -1), offsets)]
    av, bv = _vals(*a), _vals(*b).view(n_e, N, K)
    out = torch.full((M, N), 5.0, dtype=F32, device=DEV)
    E.mxfp4_grouped_matmul(*d, out=out)
    assert (out[used:] == 5).all()
    for e in range(n_e):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        _close(out[lo:hi], av[lo:hi] @ bv[e].t(), av[lo:hi].abs() @ bv[e].abs().t(), K, F32)


@pytest.mark.parametrize("M,N,K", [(5, 40, 96), (130, 700, 160), (130, 700, 256), (6000, 8192, 128), (6000, 8192, 160)])
def test_slices_of_rows(M, N, K):
    """Rows from the middle of larger operands: their exponents start at any byte."""
    require_gpu()
    note(f"mx matmul of slices {M}x{N}x{K}")
    (a, sa), (b, sb) = ([t.to(DEV) for t in _operand(n + 7, K, n)] for n in (M, N))
    buf = torch.empty(sa.numel() + 3, dtype=torch.uint8, device=DEV)
    for at in (0, 1, 3):
        sa_ = buf[at:at + sa.numel()].view(sa.shape).copy_(sa)
        got = E.mxfp4_matmul(a[3:3 + M], sa_[3:3 + M], b[1:1 + N], sb[1:1 + N], out_dtype=F32)
        want = E.mxfp4_matmul(*(t.clone() for t in (a[3:3 + M], sa[3:3 + M], b[1:1 + N], sb[1:1 + N])), out_dtype=F32)
        assert torch.equal(got, want)
        off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
        got = E.mxfp4_grouped_matmul(a[3:3 + M], sa_[3:3 + M], b[1:1 + N][None], sb[1:1 + N][None], off, out_dtype=F32)
        again = E.mxfp4_grouped_matmul(*(t.clone() for t in (a[3:3 + M], sa[3:3 + M], b[1:1 + N][None], sb[1:1 + N][None])), off,
                                       out_dtype=F32)
        assert torch.equal(got, again)
    av, bv = _vals(a[3:3 + M].cpu(), sa[3:3 + M].cpu()), _vals(b[1:1 + N].cpu(), sb[1:1 + N].cpu())
    _close(want, av @ bv.t(), av.abs() @ bv.abs().t(), K, F32)
    _close(got, av @ bv.t(), av.abs() @ bv.abs().t(), K, F32)


def test_shapes_reach_every_kernel():
    size = E.mxfp4_matmul_workspace_size
    large = [s for s in SHAPES if size(*s) > 0]
    assert {N % 8 == 0 for _, N, _ in large} == {True, False} and {K % 128 == 0 for _, _, K in SHAPES} == {True, False}
    assert size(6000, 8192, 160) > 0 and size(2500, 5504, 416) > 0 and size(700, 1600, 160) == 0
    assert {min((K + 127) // 128, 4) for _, _, K in large} >= {1, 2, 4}     # fewer steps than stages too
    # K in parts: few rows and tiles
    assert size(64, 512, 16384) == 8 * 64 * 512 * 4 and size(300, 1024, 8192) % (300 * 1024 * 4) == 0 < size(300, 1024, 8192)
    assert all(size(*s) > 0 for s in SHAPES[-6:])


@pytest.mark.parametrize("M,N,K", [(5, 40, 96), (900, 1700, 160), (6000, 8192, 160)])
def test_exponents_at_the_ends(M, N, K):
    """2^-127 on one side, 2^127 on the other; the largest sums leave float32's range and are infinite."""
    require_gpu()
    note(f"mx matmul end exponents {M}x{N}x{K}")
    a, b = _operand(M, K, 1, 2), _operand(N, K, 2, 2)
    g = torch.Generator().manual_seed(3)
    a[1].copy_(torch.randint(0, 3, a[1].shape, generator=g))
    b[1].copy_(torch.randint(252, 255, b[1].shape, generator=g))
    av, bv = _vals(*a), _vals(*b)
    d = [t.to(DEV) for t in (*a, *b)]
    _close(E.mxfp4_matmul(*d, out_dtype=F32), av @ bv.t(), av.abs() @ bv.abs().t(), K, F32)
    a[1][0] = 250
    y = E.mxfp4_matmul(*(t.to(DEV) for t in (*a, *b)), out_dtype=F32).cpu()
    want = _vals(*a)[:1] @ bv.t()
    over = want.abs() > 2.0 ** 130
    assert over.any() and not torch.isfinite(y[:1][over]).any() and torch.isfinite(y[1:]).all()
