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


def test_gradients_through_saved_tensor_hooks():
    """Tensors saved on the host, or given back strided: the same gradients; of another type or device: refused."""
    require_gpu()
    note("norm and routing through saved-tensor hooks")
    hooks = torch.autograd.graph.saved_tensors_hooks
    x, r, w, z = (torch.randn(*s, device=DEV).to(t).requires_grad_() for s, t in (((37, 528), BF), ((37, 528), BF), ((528,), F32), ((37, 43), BF)))

    def gradients():
        y, h = E.rms_norm(x, w, r)
        p, _ = E.topk_routing(z, 5)
        gy, gp = (torch.arange(t.numel(), device=DEV).remainder(7).to(t.dtype).view(t.shape) - 3 for t in (y, p))
        return lambda: (*torch.autograd.grad((y, h), (x, r, w), (gy, gy)), *torch.autograd.grad(p, z, gp))

    want = gradients()()
    for pack, unpack in ((lambda t: t.cpu(), lambda t: t.to(DEV)), (lambda t: t.clone(), lambda t: torch.stack((t, t), -1)[..., 0])):
        with hooks(pack, unpack):
            again = gradients()
        assert all(torch.equal(a, b) for a, b in zip(again(), want))
    for unpack in (lambda t: t, lambda t: t.to(DEV).double()):
        with hooks(lambda t: t.cpu(), unpack):
            again = gradients()
        with pytest.raises(E.EsgError, match="of the backward"):
            again()


@pytest.mark.parametrize("Ex,k", [(40, 4), (256, 8), (43, 20), (1000, 5)])
def test_routing_gradient_of_non_finite_rows(Ex, k):
    """A logit that makes its row's weights NaN makes all of the row's gradient NaN, whatever dprobs are; no other row's."""
    require_gpu()
    for dtype in (F32, BF):
        for scoring in ("softmax", "sigmoid"):
            for normalize in (True, False):
                note(f"route backward non-finite {Ex} {k} {dtype} {scoring} {normalize}")
                z = torch.randn(7, Ex, generator=torch.Generator().manual_seed(Ex)).to(dtype)
                clean = z.clone()
                z[1, 3] = float("nan")
                z[2, Ex - 1] = float("inf")
                z[3] = float("nan")
                z[4, k:] = float("-inf")
                z[6, 0] = float("nan")
                bad = [1, 3, 6] + ([2] if scoring == "softmax" else [])
                fine = [t for t in range(7) if t not in bad]
                zd = z.to(DEV).requires_grad_()
                p, idx = E.topk_routing(zd, k, scoring, normalize=normalize)
                assert torch.isnan(p[bad]).all() and torch.isfinite(p[fine]).all()
                dp = torch.randn(7, k, generator=torch.Generator().manual_seed(1)).to(DEV)
                dz, = torch.autograd.grad(p, zd, dp)
                assert torch.isnan(dz[bad]).all() and torch.isfinite(dz[fine]).all()
                want = E.topk_routing_bwd(dp, clean.to(DEV), idx, scoring, normalize)
                assert torch.equal(dz[[0, 5]], want[[0, 5]])


@pytest.mark.parametrize("Ex,groups,keep,k", [(32, 4, 2, 4), (256, 8, 3, 8), (60, 6, 2, 3), (384, 6, 1, 2), (512, 32, 4, 6)])
def test_groups_of_a_forced_and_masked_experts(Ex, groups, keep, k):
    """A group whose largest keys are +infinity and -infinity (a NaN bias is one) counts as +infinity: it stays, before
    finite groups and after equal ones of lower number, and no more than topk_groups stay."""
    require_gpu()
    per = Ex // groups
    for scoring in ("softmax", "sigmoid"):
        for dtype in (F32, BF):
            for masked in (float("-inf"), float("nan")):
                note(f"route forced and masked {Ex} {groups}/{keep} {k} {scoring} {dtype} {masked}")
                z = torch.randn(9, Ex, generator=torch.Generator().manual_seed(Ex)).to(dtype)
                bias = 0.1 * torch.randn(Ex, generator=torch.Generator().manual_seed(1))
                for g in range(1, groups, 2):              # every other group, more than may stay for the larger shapes
                    bias[g * per:(g + 1) * per] = masked
                    bias[g * per + g % per] = float("inf")
                _, idx = E.topk_routing(z.to(DEV), k, scoring, bias.to(DEV), groups, keep)
                key = O.scores(f64(z), scoring).astype(np.float32) + bias.nan_to_num(nan=-np.inf, posinf=np.inf, neginf=-np.inf).numpy()
                two = np.sort(key.reshape(9, groups, per), axis=2)[:, :, ::-1][:, :, :2]
                with np.errstate(invalid="ignore"):
                    rank = two[:, :, 0] + two[:, :, 1]
                rank[np.isnan(rank)] = np.inf
                best = np.argsort(-rank, axis=1, kind="stable")[:, :keep]
                for t in range(9):
                    allowed = np.concatenate([np.arange(g * per, (g + 1) * per) for g in sorted(best[t])])
                    want = np.sort(allowed[np.argsort(-key[t, allowed], kind="stable")[:k]])
                    assert np.array_equal(idx[t].cpu().numpy(), want)


U = 2.0 ** -24  # one float32 rounding


@pytest.mark.parametrize("d", [16, 144, 528, 1024, 2048, 5504, 16384])
def test_norm_of_tiny_rows(d):
    """Squares below float32's range and an eps that does not cover them: the bounds of the norm's other tests (45 roundings
    of y, 225 of the sum of dx's terms), whatever the size of h; dw is not looked at where r is past float32."""
    require_gpu()
    g = torch.Generator().manual_seed(d)
    size = torch.tensor([1e-16, 1e-19, 1e-22, 1e-25, 1e-30, 1e-36, 1e-42, 1.0], dtype=torch.float64)[:, None]
    w = 1 + 0.3 * torch.randn(d, generator=g)
    for dtype in (F32, BF):
        x = (torch.randn(8, d, generator=g).double() * size).to(dtype)
        half = 2.0 ** -8 if dtype == BF else U
        for eps in (0.0, 1e-44, 1e-40, 1e-35, 1e-30, 1e-12):
            note(f"norm of tiny rows {d} {dtype} eps={eps}")
            e = float(torch.tensor(eps, dtype=F32))
            with np.errstate(divide="ignore", invalid="ignore"):
                want, r = O.rms_norm(f64(x), f64(w), e)
            y, _, rstd = E.rms_norm_fwd(x.to(DEV), w.to(DEV), eps=eps)
            zero = ~f64(x).any(1) & (e == 0)               # 1e-42 is zero in bf16, and 0 / 0 is NaN
            assert np.isnan(f64(y)[zero]).all()
            assert (np.abs(f64(y) - want) <= (half + 45 * U) * np.abs(want) + 2.0 ** -149)[~zero].all()
            past = r[:, 0] > 2.0 ** 127.999
            assert (np.abs(f64(rstd)[~past] - r[~past, 0]) <= 41 * U * r[~past, 0]).all() and np.isinf(f64(rstd)[past]).all()
            q, s = E.rms_norm_quantize(x.to(DEV), w.to(DEV), eps=eps)
            top = np.stack([np.abs(want[:, i:i + 128]).max(1) for i in range(0, d, 128)], 1)
            big = top > 2.0 ** -90                         # below, the scale of an empty block
            assert (np.abs(f64(s) - top / 448)[big] <= 48 * U * f64(s)[big]).all()
            v, unit = f64(q) * np.repeat(f64(s), 128, 1)[:, :d], np.repeat(f64(s), 128, 1)[:, :d]
            near = np.abs(v - want) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * unit) + 100 * U * np.abs(want)
            assert near[np.repeat(big, 128, 1)[:, :d]].all()
            keep = r[:, 0] < 1e30
            dy = torch.randn(8, d, generator=g).to(dtype)
            dx, _ = E.rms_norm_bwd(dy.to(DEV), x.to(DEV), w.to(DEV), rstd)
            with np.errstate(divide="ignore", invalid="ignore"):
                wx, _, mx, _ = O.rms_norm_backward(f64(dy), f64(x), f64(w), e)
            assert (np.abs(f64(dx) - wx)[keep] <= (half * np.abs(wx) + 225 * U * mx)[keep]).all()
