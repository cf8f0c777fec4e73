"""What is measured of the 8-bit feed-forward operators and of the whole
mixture-of-experts layer for a few tokens.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and as a user calls it from ``group_sparse_swiglu_amd``:

- ``quant``: bfloat16 or float32 rows to 8-bit floating point (e4m3) with one
  float32 scale per 1 x 128 block; optionally the transposed form with one
  scale per 128 rows of a column as well; or, for weights, one scale per
  128 x 128 block and the transposed copy.  With a the largest magnitude of a
  block (at least 2^-100): scale = a / 448, q = e4m3(x * (448 / a)), every
  operation rounded once to float32.
- ``matmul``: y[m, n] = sum_k a[m, k] sa[m, k/128] b[n, k] sb[n or n/128, k/128].
- ``linear``: y = x W^T with both sides quantised as above, and the gradients
  of x and W from the quantised dy, W and x.
- ``moe``: router logits, sigmoid top-k with an expert bias, the chosen
  experts' SwiGLU and their weighted sum, for up to 64 tokens.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
TOP = 448.0            # largest e4m3 value
FLOOR = 2.0 ** -100    # smallest block magnitude a scale is taken from
E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's activations before an 8-bit projection: latency
        dict(name="quant_decode64", op="quant", form="rows", M=64, K=2048, dtype="bf16"),
        # a training step's activations at the 1.3B width, both directions in one pass
        dict(name="quant_train_both", op="quant", form="both", M=32768, K=2048, dtype="bf16"),
        # gate and up projections stacked (2 x 5504), one token
        dict(name="matmul_token1", op="matmul", form="tiles", M=1, N=11008, K=2048, out="bf16"),
        # down projection for an odd decode batch, float32 result
        dict(name="matmul_batch37", op="matmul", form="tiles", M=37, N=2048, K=5504, out="f32"),
        # the 1.3B layer's gate projection over a whole training batch
        dict(name="matmul_train", op="matmul", form="tiles", M=32768, N=5504, K=2048, out="bf16"),
        # a weight gradient: both sides quantised along the tokens, odd token count
        dict(name="matmul_wgrad", op="matmul", form="rows", M=2688, N=1024, K=16400, out="f32"),
        # forward and backward of one projection at the 1.3B shape, float32 master weights
        dict(name="linear_8192", op="linear", T=8192, K=2048, N=5504, wdtype="f32"),
        # a small ragged batch at the 128M shape, bfloat16 weights
        dict(name="linear_333", op="linear", T=333, K=768, N=2048, wdtype="bf16"),
        # single-token serving of a wide bfloat16 expert layer
        dict(name="moe_token1", op="moe", T=1, E=256, k=8, d=2048, ff=1024, weights="bf16", scaling=2.5),
        # the 1.3B layer's 43 groups of 128 as experts, 11 active, a small batch
        dict(name="moe_e43_batch8", op="moe", T=8, E=43, k=11, d=2048, ff=128, weights="bf16", scaling=0.0),
        # an odd speculative-decoding batch on 8-bit experts of a ragged width
        dict(name="moe_fp8_batch5", op="moe", T=5, E=256, k=8, d=2048, ff=1008, weights="fp8", scaling=2.5),
        # the largest batch of the decode path on 8-bit experts
        dict(name="moe_fp8_batch64", op="moe", T=64, E=64, k=6, d=2048, ff=1408, weights="fp8", scaling=1.0),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["quant", "matmul", "matmul", "linear", "moe", "moe"])
    while True:
        if op == "quant":
            c = dict(op=op, form=rng.choice(["rows", "both", "weight"]), M=_log(rng, 1, 32768), K=_log(rng, 16, 8192, 16),
                     dtype=rng.choice(["bf16", "f32"]))
            if c["M"] * c["K"] * (2 if c["dtype"] == "f32" else 1) <= 32768 * 2048:
                return c
        elif op == "matmul":
            c = dict(op=op, form=rng.choice(["tiles", "tiles", "rows"]), M=_log(rng, 1, 32768), N=_log(rng, 16, 16384),
                     K=_log(rng, 64, 16384, 16), out=rng.choice(["bf16", "f32"]))
            if c["M"] * c["N"] * c["K"] <= 32768 * 5504 * 2048 and c["M"] * c["N"] <= 32768 * 5504 // 2:
                return c
        elif op == "linear":
            c = dict(op=op, T=_log(rng, 1, 16384), K=_log(rng, 128, 8192, 16), N=_log(rng, 128, 8192, 16),
                     wdtype=rng.choice(["bf16", "f32"]))
            if c["T"] * c["K"] * c["N"] <= 8192 * 2048 * 5504:
                return c
        else:
            E = _log(rng, 8, 256)
            c = dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(E, 12)), d=_log(rng, 256, 4096, 16),
                     ff=_log(rng, 64, 4096, 16), weights=rng.choice(["bf16", "fp8"]), scaling=rng.choice([0.0, 1.0, 2.5]))
            if E * c["d"] * c["ff"] <= 256 * 2048 * 1024 and c["T"] * c["k"] * c["d"] * c["ff"] <= 64 * 6 * 2048 * 1408:
                return c


# ------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, cols, dtype=torch.bfloat16):
    """Normal values whose channels differ in size, a few of them by much."""
    size = torch.exp(0.7 * torch.randn(cols, device=DEV, generator=g))
    return (torch.randn(rows, cols, device=DEV, generator=g) * size).to(dtype)


def _weights(g, *shape, dtype=torch.bfloat16):
    return (torch.randn(*shape, device=DEV, generator=g, dtype=torch.bfloat16 if dtype == torch.bfloat16 else None)
            * shape[-1] ** -0.5).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quant":
        x = _activations(g, case["M"], case["K"], TYPES[case["dtype"]])
        return dict(case=case, x=x)
    if op == "matmul":
        a, sa = _quant_rows(_activations(g, case["M"], case["K"]))
        if case["form"] == "tiles":
            b, sb = _quant_tiles(_weights(g, case["N"], case["K"]))
        else:
            b, sb = _quant_rows(_activations(g, case["N"], case["K"]))
        return dict(case=case, a=a, sa=sa, b=b, sb=sb, workspace={})
    if op == "linear":
        x = _activations(g, case["T"], case["K"])
        w = _weights(g, case["N"], case["K"], dtype=TYPES[case["wdtype"]])
        dy = _activations(g, case["T"], case["N"]) * 1e-3
        return dict(case=case, x=x.requires_grad_(), w=w.requires_grad_(), dy=dy)
    T, E, d, ff = case["T"], case["E"], case["d"], case["ff"]
    x = _activations(g, T, d)
    router = _weights(g, E, d)
    bias = 0.1 * torch.rand(E, device=DEV, generator=g) - 0.05
    scales, ws = None, []
    for shape in ((E, ff, d), (E, ff, d), (E, d, ff)):
        ws.append(_weights(g, *shape))
    if case["weights"] == "fp8":
        pairs = [_quant_tiles(w) for w in ws]
        ws, scales = [p[0] for p in pairs], tuple(p[1] for p in pairs)
    return dict(case=case, x=x, router=router, bias=bias, ws=ws, scales=scales, workspace={})


# -------------------------------------------------------------- plain forms
def _blocks(n):
    return -(-n // BLOCK)


def _pad(x, rows, cols):
    if x.shape[-2:] == (rows, cols):
        return x
    out = x.new_zeros(*x.shape[:-2], rows, cols)
    out[..., : x.shape[-2], : x.shape[-1]] = x
    return out


def _scale_of(amax):
    amax = amax.clamp(min=FLOOR)
    top = torch.full_like(amax, TOP)  # two tensors: a division by a number may go by its rounded reciprocal
    return amax / top, top / amax


def _quant_rows(x):
    """[M, K] -> e4m3 [M, K], float32 [M, ceil(K/128)]."""
    M, K = x.shape
    xb = _pad(x.float(), M, _blocks(K) * BLOCK).view(M, _blocks(K), BLOCK)
    scale, inv = _scale_of(xb.abs().amax(-1))
    return (xb * inv[..., None]).view(M, -1)[:, :K].to(E4M3).contiguous(), scale


def _quant_cols(x):
    """The row form of x^T, its length padded with zeros to a multiple of 16."""
    M, K = x.shape
    return _quant_rows(_pad(x, -(-M // 16) * 16, K).t().contiguous())


def _quant_tiles(w):
    """[..., N, K] -> e4m3, float32 [..., ceil(N/128), ceil(K/128)]."""
    N, K = w.shape[-2:]
    nb, kb = _blocks(N), _blocks(K)
    wb = _pad(w.float(), nb * BLOCK, kb * BLOCK).view(*w.shape[:-2], nb, BLOCK, kb, BLOCK)
    scale, inv = _scale_of(wb.abs().amax((-3, -1)))
    q = (wb * inv[..., :, None, :, None]).view(*w.shape[:-2], nb * BLOCK, kb * BLOCK)
    return q[..., :N, :K].to(E4M3).contiguous(), scale


def _transposed_tiles(q, scale):
    N, K = q.shape
    qt = _pad(q.view(torch.uint8), -(-N // 16) * 16, K).t().contiguous().view(E4M3)
    return qt, scale.t().contiguous()


def _values(q, scale, rows_of_scale=1):
    """The float32 values that q and its scales stand for."""
    s = scale.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]
    if rows_of_scale > 1:
        s = s.repeat_interleave(rows_of_scale, -2)[..., : q.shape[-2], :]
    return q.float() * s


def _plain_linear(x, w, dy):
    xq, wq, dq = _quant_rows(x), _quant_tiles(w), _quant_rows(dy)
    wv = _values(*wq, BLOCK)
    y = _values(*xq) @ wv.t()
    dx = _values(*dq) @ wv
    dw = _values(*_quant_cols(dy)) @ _values(*_quant_cols(x)).t()
    return y.to(x.dtype), dx.to(x.dtype), dw.to(w.dtype)


def _plain_topk(score, bias, k):
    """Experts above the k-th largest key in ascending order, then its equals."""
    key = score + bias
    kth = key.sort(dim=-1, descending=True).values[:, k - 1 : k]
    rank = 2 - 2 * (key > kth).int() - (key == kth).int()
    return rank.sort(dim=-1, stable=True).indices[:, :k].contiguous()


def _plain_moe(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    x = s["x"].float()
    score = 1.0 / (1.0 + torch.exp(-(x @ s["router"].float().t())))
    idx = _plain_topk(score, s["bias"], k)
    p = score.gather(1, idx)
    p = p / (p.sum(-1, keepdim=True) + 1e-20)
    if c["scaling"]:
        p = p * c["scaling"]
    e = idx.reshape(-1)

    def chosen(i):
        w = s["ws"][i]
        if s["scales"] is None:
            return w[e].float()
        return _values(w.view(torch.uint8)[e].view(E4M3), s["scales"][i][e], BLOCK)

    xr = x.repeat_interleave(k, 0).unsqueeze(-1)
    hg, hu = torch.bmm(chosen(0), xr), torch.bmm(chosen(1), xr)
    h = hg / (1.0 + torch.exp(-hg)) * hu * p.reshape(-1, 1, 1)
    y = torch.bmm(chosen(2), h).view(T, k, -1).sum(1)
    return y.to(s["x"].dtype), p, idx


# ----------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import group_sparse_swiglu_amd as E
    if op == "quant":
        x = s["x"]
        if c["form"] == "rows":
            return E.fp8_quantize(x) if own else _quant_rows(x)
        if c["form"] == "both":
            return E.fp8_quantize(x, transposed=True) if own else (*_quant_rows(x), *_quant_cols(x))
        if own:
            return E.fp8_quantize_weight(x, transposed=True)
        q, scale = _quant_tiles(x)
        return (q, scale, *_transposed_tiles(q, scale))
    if op == "matmul":
        if own:
            return E.fp8_matmul(s["a"], s["sa"], s["b"], s["sb"], out_dtype=TYPES[c["out"]], workspace=s["workspace"])
        b = _values(s["b"], s["sb"], BLOCK if c["form"] == "tiles" else 1)
        return (_values(s["a"], s["sa"]) @ b.t()).to(TYPES[c["out"]])
    if op == "linear":
        if own:
            y = E.fp8_linear(s["x"], s["w"])
            return (y, *torch.autograd.grad(y, (s["x"], s["w"]), s["dy"]))
        with torch.no_grad():
            return _plain_linear(s["x"], s["w"], s["dy"])
    if own:
        return E.moe_decode(s["x"], s["router"], s["bias"], *s["ws"], c["k"], scaling_factor=c["scaling"] or None,
                            scales=s["scales"], workspace=s["workspace"])
    return _plain_moe(s)


def work(case):
    op = case["op"]
    if op == "quant":
        M, K = case["M"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        nb, kb = _blocks(M), _blocks(K)
        out = {"rows": M * K + 4 * M * kb, "both": 2 * M * K + 4 * (M * kb + K * nb),
               "weight": 2 * M * K + 8 * nb * kb}[case["form"]]
        return {"bytes": M * K * size + out, "flops": 3 * M * K}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * _blocks(K) * (M + (N if case["form"] == "rows" else _blocks(N)))
        return {"bytes": (M + N) * K + scales + M * N * (4 if case["out"] == "f32" else 2), "flops": 2 * M * N * K}
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        size = 4 if case["wdtype"] == "f32" else 2
        return {"bytes": 4 * T * K + 4 * T * N + 2 * N * K * size, "flops": 6 * T * N * K}
    T, E, k, d, ff = (case[n] for n in ("T", "E", "k", "d", "ff"))
    active = E * (1.0 - (1.0 - k / E) ** T)  # distinct experts of T tokens
    size = 2 if case["weights"] == "bf16" else 1 + 4 / BLOCK ** 2
    return {"bytes": active * 3 * d * ff * size + 2 * E * d + 4 * T * d + 12 * T * k,
            "flops": 6 * T * k * d * ff + 2 * T * E * d}


# ------------------------------------------------------------------ 64 bits
def _e4m3_64(v):
    """v (float64) to the nearest e4m3 value, ties to even, as float64."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _split64(x, rows, cols):
    """Each row's or tile's 64-bit quantised values, scale by blocks of rows x cols."""
    R, C = x.shape
    nr, nc = -(-R // rows), -(-C // cols)
    big = torch.zeros(nr * rows, nc * cols, dtype=torch.float64, device=x.device)
    big[:R, :C] = x.double()
    b = big.reshape(nr, rows, nc, cols)
    top = b.abs().amax(dim=(1, 3)).clamp(min=FLOOR)
    # reciprocal, scale and product are 32-bit values by definition: with 8-bit significands in x many
    # products lie at or next to a tie of e4m3, so that their rounding decides
    inv = (TOP / top).float().double()
    scale = (top / TOP).float().double()
    q = _e4m3_64((b * inv[:, None, :, None]).float().double()).reshape(nr * rows, nc * cols)[:R, :C]
    return q, scale


def _times64(q, scale, rows, cols):
    s = torch.repeat_interleave(torch.repeat_interleave(scale, rows, 0), cols, 1)
    return q.double() * s[: q.shape[0], : q.shape[1]]


def _padded_t(x):
    M = x.shape[0]
    xt = torch.zeros(x.shape[1], (M + 15) // 16 * 16, dtype=x.dtype, device=x.device)
    xt[:, :M] = x.t()
    return xt


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op == "quant":
            x = s["x"]
            if case["form"] == "rows":
                return _split64(x, 1, BLOCK)
            if case["form"] == "both":
                return (*_split64(x, 1, BLOCK), *_split64(_padded_t(x), 1, BLOCK))
            q, scale = _split64(x, BLOCK, BLOCK)
            return q, scale, _padded_t(q), scale.t()
        if op == "matmul":
            a = _times64(s["a"], s["sa"].double(), 1, BLOCK)
            b = _times64(s["b"], s["sb"].double(), BLOCK if case["form"] == "tiles" else 1, BLOCK)
            return torch.matmul(a, b.t().contiguous())
        if op == "linear":
            x, w, dy = s["x"], s["w"], s["dy"]
            wv = _times64(*_split64(w, BLOCK, BLOCK), BLOCK, BLOCK)
            y = torch.matmul(_times64(*_split64(x, 1, BLOCK), 1, BLOCK), wv.t().contiguous())
            dx = torch.matmul(_times64(*_split64(dy, 1, BLOCK), 1, BLOCK), wv)
            dyt = _times64(*_split64(_padded_t(dy), 1, BLOCK), 1, BLOCK)
            xt = _times64(*_split64(_padded_t(x), 1, BLOCK), 1, BLOCK)
            return y, dx, torch.matmul(dyt, xt.t().contiguous())
        return _exact_moe(s)


def _exact_moe(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["x"].double()
    score = torch.sigmoid(torch.matmul(x, s["router"].double().t().contiguous()))
    order = torch.argsort(score + s["bias"].double(), dim=1, descending=True, stable=True)
    # ascending, the one with the k-th largest key last (no ties are expected in these inputs)
    idx = torch.cat((torch.sort(order[:, : k - 1], dim=1).values, order[:, k - 1 : k]), dim=1)
    p = torch.gather(score, 1, idx)
    p = p / p.sum(dim=1, keepdim=True)
    if c["scaling"]:
        p = p * c["scaling"]
    y = torch.zeros(T, c["d"], dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        if s["scales"] is None:
            g, u, d = (w[e].double() for w in s["ws"])
        else:
            g, u, d = (_times64(w[e], sc[e].double(), BLOCK, BLOCK) for w, sc in zip(s["ws"], s["scales"]))
        hg = torch.matmul(x[t], g.t().contiguous())
        h = hg * torch.sigmoid(hg) * torch.matmul(x[t], u.t().contiguous())
        y[t] += torch.matmul(h * p[t, j, None], d.t().contiguous())
    return y, p, None
