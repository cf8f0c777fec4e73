"""An 8-bit feed-forward stack, from training to serving, on one MI355X.

    python examples/fp8_experts.py [--steps N]

1. A gated feed-forward layer is trained for a few steps with fp8_linear (every
   product of the forward and the backward in e4m3 with block scales) on float32
   master weights, beside the same layer in plain float32.
2. Its trained projections are quantised once (fp8_quantize_weight) and serve a
   prompt through fp8_quantize and fp8_matmul.
3. An expert layer's weights are quantised the same way and answer token by token
   and in small batches through moe_decode, beside the same call on the bfloat16
   weights.

Prints what each part reached; every number is relative to the plain form."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import group_sparse_swiglu_amd as E  # noqa: E402

DEV, BF = "cuda", torch.bfloat16


def swiglu(x, w_gate, w_up, w_down, linear):
    g = linear(x, w_gate)
    return linear((torch.nn.functional.silu(g.float()) * linear(x, w_up).float()).to(x.dtype), w_down)


def rel(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def train(steps: int, T=512, d=256, ff=768):
    """Fit a fixed random layer; returns the losses of the 8-bit and the plain run and the 8-bit run's weights."""
    g = torch.Generator(device=DEV).manual_seed(0)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    target = [rand(ff, d) * d ** -0.5, rand(ff, d) * d ** -0.5, rand(d, ff) * ff ** -0.5]
    start = [w + 0.5 * w.std() * rand(*w.shape) for w in target]
    plain = lambda x, w: (x.float() @ w.t()).to(x.dtype)  # noqa: E731
    out = []
    for linear in (E.fp8_linear, plain):
        ws = [w.clone().requires_grad_() for w in start]
        opt = torch.optim.Adam(ws, lr=2e-3)
        data = torch.Generator(device=DEV).manual_seed(1)
        losses = []
        for _ in range(steps):
            x = torch.randn(T, d, device=DEV, generator=data).to(BF)
            with torch.no_grad():
                want = swiglu(x, *target, plain).float()
            loss = (swiglu(x, *ws, linear).float() - want).square().mean()
            opt.zero_grad()
            loss.backward()
            opt.step()
            losses.append(loss.item())
        out.append((losses, [w.detach() for w in ws]))
    return out


def serve_dense(weights, T=333):
    """A prompt through the trained layer with its projections quantised once."""
    x = torch.randn(T, weights[0].shape[1], device=DEV).to(BF)
    q = [E.fp8_quantize_weight(w) for w in weights]
    product = lambda x, w: E.fp8_matmul(*E.fp8_quantize(x), *w)  # noqa: E731
    return rel(swiglu(x, *q, product), swiglu(x.float(), *weights, lambda x, w: x @ w.t()))


def serve_experts(T, experts=64, k=6, d=1024, ff=512):
    """y of the 8-bit experts against the bfloat16 ones, same routing."""
    g = torch.Generator(device=DEV).manual_seed(2)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    x, router = rand(T, d).to(BF), (rand(experts, d) * d ** -0.5).to(BF)
    bias = torch.zeros(experts, device=DEV)
    ws = [(rand(experts, *s) * s[1] ** -0.5).to(BF) for s in ((ff, d), (ff, d), (d, ff))]
    q = [E.fp8_quantize_weight(w) for w in ws]
    workspace = {}
    y, probs, idx = E.moe_decode(x, router, bias, *ws, k, scaling_factor=2.5, workspace=workspace)
    y8, probs8, idx8 = E.moe_decode(x, router, bias, *(p[0] for p in q), k, scaling_factor=2.5,
                                    scales=tuple(p[1] for p in q), workspace=workspace)
    assert torch.equal(idx, idx8) and torch.equal(probs, probs8)
    return rel(y8, y)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args(argv)
    (l8, w8), (lp, _) = train(a.steps)
    print(f"training: loss {l8[0]:.4f} -> {l8[-1]:.4f} in 8 bits, {lp[0]:.4f} -> {lp[-1]:.4f} in float32")
    dense = serve_dense(w8)
    print(f"prompt through the quantised layer: {dense:.3f} off the float32 one (relative norm)")
    experts = {T: serve_experts(T) for T in (1, 8, 64)}
    for T, e in experts.items():
        print(f"expert layer, {T} tokens: 8-bit weights {e:.3f} off the bfloat16 ones")
    return l8, lp, dense, experts


if __name__ == "__main__":
    main()
