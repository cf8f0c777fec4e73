"""GPU parity of the 4-bit products' large tiles where a workgroup takes several one after the other, and which kernel
each shape of the products' tests reaches.

Everything is compared with float64 products of the values, with the bound of the products' other tests: an error of at
most (K / 128 + 24) 2^-22 of the sum of all |terms|, and the result's rounding."""
import pytest
import torch

import group_sparse_swiglu_amd as E
import test_gpu_mx_matmul as X
from gpu_common import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
CUS = 256


def _ceil(a, b):
    return -(-a // b)


def _near(got, av, bv, K):
    bt = bv.t().contiguous()
    want, mag = av @ bt, av.abs() @ bt.abs()
    tol = (K / 128 + 24) * 2.0 ** -22 * mag + (2.0 ** -8 if got.dtype == BF else 2.0 ** -24) * want.abs()
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


# steps of 128 elements: 3 (all of a tile's loads are the next tile's), 4, 6, 7, 16; two and three tiles of a workgroup
CARRIED = [(5000, 5400, 320), (5000, 5400, 384), (5001, 5403, 512), (5000, 5400, 768), (4900, 5397, 864), (8200, 5400, 384),
           (8197, 5405, 416), (8200, 5400, 512), (5000, 5400, 2048), (8200, 5400, 2048)]


@pytest.mark.parametrize("M,N,K", CARRIED)
def test_tile_after_tile(M, N, K):
    require_gpu()
    a, b = X._operand(M, K, M + K), X._operand(N, K, N + K + 1)
    assert E.mxfp4_matmul_workspace_size(M, N, K) == (M + N) * _ceil(K, 128) * 4          # words: large tiles
    assert _ceil(M, 256) * _ceil(N, 256) > CUS * (2 if M > 8000 else 1)
    d = [t.to(DEV) for t in (*a, *b)]
    av, bv = (X._vals(*t).to(DEV) for t in (a, b))
    for dtype in (BF, F32):
        note(f"mx matmul tile after tile {M}x{N}x{K} {dtype}")
        _near(E.mxfp4_matmul(*d, out_dtype=dtype), av, bv, K)


CARRIED_BY_EXPERT = [([2600, 300, 0, 4100, 513, 1, 2500], 5400, 384), ([1100] * 9, 5403, 352), ([5000, 5000], 5400, 512),
                     ([3000, 700, 0, 0, 6000, 4000], 5400, 832), ([2600, 300, 0, 4100, 513, 1, 2500], 5400, 2048),
                     ([9000, 4, 7500], 5000, 384)]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("counts,N,K", CARRIED_BY_EXPERT)
def test_tile_after_tile_by_expert(counts, N, K, gather):
    require_gpu()
    n_e, used = len(counts), sum(counts)
    M = used + 37
    assert E.mxfp4_grouped_matmul_workspace_size(M, N, K, n_e) == (M + n_e * N) * _ceil(K, 128) * 4
    assert sum(_ceil(c, 256) for c in counts) * _ceil(N, 256) > CUS * (2 if used > 16000 else 1)   # tiles that have rows
    offsets = torch.tensor([0] + counts).cumsum(0).int()
    R = 1999 if gather else M
    a, b = X._operand(R, K, 3), X._operand(n_e * N, K, 4)
    rows = torch.randint(0, R, (M,), generator=torch.Generator().manual_seed(N)).int() if gather else None
    d = [t.to(DEV) for t in (*a, b[0].view(n_e, N, -1), b[1].view(n_e, N, -1), offsets)]
    av, bv = X._vals(*a).to(DEV), X._vals(*b).to(DEV).view(n_e, N, K)
    if gather:
        rows = rows.to(DEV)
        av = av[rows.long()]
    for dtype in (BF, F32):
        note(f"mx grouped tile after tile {counts} {N} {K} {dtype} gather={gather}")
        out = torch.full((M, N), 5.0, dtype=dtype, device=DEV)
        E.mxfp4_grouped_matmul(*d, rows=rows, out=out)
        assert (out[used:] == 5).all()
        for e in range(n_e):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            if hi > lo:
                _near(out[lo:hi], av[lo:hi], bv[e], K)


KERNELS = ["mx_rows_2_16", "mx_rows_4_16", "mx_rows_8_16", "mx_rows_4_64", "mx_rows_8_64", "mx_tile_128", "mx_tile_256",
           "mx_words", "mx_parts"]


def _launched(call):
    E.timing_enable()
    E.timing_reset()
    try:
        call()
        return {k for k in KERNELS if E.timing_read(k)[1] > 0}
    finally:
        E.timing_reset()
        E.timing_enable(False)


def _zeros(*shape):
    return torch.zeros(*shape, dtype=U8, device=DEV)


def _product(M, N, K):
    return _launched(lambda: E.mxfp4_matmul(_zeros(M, K // 2), _zeros(M, K // 32), _zeros(N, K // 2), _zeros(N, K // 32)))


def _by_expert(counts, N, K):
    n_e, offsets = len(counts), torch.tensor([0] + counts).cumsum(0).int().to(DEV)
    M = sum(counts)
    return _launched(lambda: E.mxfp4_grouped_matmul(_zeros(M, K // 2), _zeros(M, K // 32), _zeros(n_e, N, K // 2),
                                                    _zeros(n_e, N, K // 32), offsets))


@pytest.mark.parametrize("want,shape", [
    ({"mx_rows_8_16"}, (1, 16, 32)), ({"mx_rows_4_16"}, (1, 11008, 2048)), ({"mx_rows_8_64"}, (64, 64, 4096)),
    ({"mx_rows_4_64"}, (64, 8192, 256)), ({"mx_rows_8_64"}, (200, 300, 1376)), ({"mx_rows_4_64"}, (129, 4096, 288)),
    ({"mx_tile_128"}, (300, 4097, 320)), ({"mx_tile_128"}, (640, 2056, 800)), ({"mx_words", "mx_tile_256"}, (2500, 5504, 608)),
    ({"mx_words", "mx_tile_256"}, (6000, 8204, 32)), ({"mx_rows_8_64", "mx_parts"}, (64, 512, 16384)),
    ({"mx_tile_128", "mx_parts"}, (300, 1024, 8192))])
def test_kernel_of_a_product(want, shape):
    require_gpu()
    note(f"mx kernels of {shape}")
    assert _product(*shape) == want


@pytest.mark.parametrize("want,counts,N,K", [
    ({"mx_rows_8_16"}, [0, 5, 0], 40, 96), ({"mx_rows_4_16"}, [6] * 64, 272, 1024), ({"mx_rows_2_16"}, [6] * 64, 1400, 256),
    ({"mx_rows_8_64"}, [70, 0, 17, 1, 49, 33, 64, 65], 100, 288), ({"mx_rows_4_64"}, [129, 600, 0, 1, 127, 128], 520, 352),
    ({"mx_tile_128"}, [129, 600, 0, 1, 127, 128], 2056, 352), ({"mx_words", "mx_tile_256"}, [4000, 0, 300, 1, 255, 2049], 4100, 96)])
def test_kernel_of_a_product_by_expert(want, counts, N, K):
    require_gpu()
    note(f"mx kernels by expert of {counts} {N} {K}")
    assert _by_expert(counts, N, K) == want


def test_the_tests_reach_every_kernel():
    require_gpu()
    note("mx kernels of all shapes of the tests")
    seen = set().union(*(_product(*s) for s in X.SHAPES))
    assert seen == set(KERNELS) - {"mx_rows_2_16"}         # by expert only
    counts = [c if c is not None else [6] * 64 for *_, c in X.GROUPED]
    seen = set().union(*(_by_expert(c, N, K) for (_, N, K, _), c in zip(X.GROUPED, counts)))
    assert seen >= {"mx_rows_8_16", "mx_rows_8_64", "mx_rows_4_64", "mx_tile_128"}
