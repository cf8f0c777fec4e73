"""Oracle of the operators around and inside an expert block: norm, routing with
groups, 4-bit values and products.  CPU, numpy, float64, plain loops where the
definition has them; what the definition rounds to float32 is rounded there."""
from __future__ import annotations

import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])  # e2m1 codes 0 .. 7
BLOCK = 32


# ------------------------------------------------------------------ norm
def rms_norm(h: np.ndarray, w: np.ndarray, eps: float):
    """(y, r) of rows h."""
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h * r * w, r


def rms_norm_backward(dy, h, w, eps, dh=None):
    """(dx, dw) and the sums of |terms| of each."""
    _, r = rms_norm(h, w, eps)
    g = dy * w
    mean = lambda v: np.mean(v, axis=1, keepdims=True)
    add = 0.0 if dh is None else dh
    dx = add + r * (g - h * r ** 2 * mean(g * h))
    mag = np.abs(add) + r * (np.abs(g) + np.abs(h) * r ** 2 * mean(np.abs(g * h)))
    return dx, np.sum(dy * h * r, axis=0), mag, np.sum(np.abs(dy * h * r), axis=0)


# --------------------------------------------------------------- routing
def scores(z: np.ndarray, scoring: str) -> np.ndarray:
    """float64 scores of finite or -infinite logits."""
    with np.errstate(over="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
    top = np.max(z, axis=1, keepdims=True)
    e = np.exp(z - np.where(np.isinf(top), 0.0, top))
    total = e.sum(1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route(z, k, scoring, bias=None, groups=1, topk_groups=1):
    """int [T, k]: chosen experts in ascending order."""
    T, E = z.shape
    key = scores(z, scoring).astype(np.float32)
    if bias is not None:
        key = key + bias.astype(np.float32)
    per = E // groups
    out = np.empty((T, k), np.int64)
    for t in range(T):
        allowed = np.arange(E)
        if topk_groups < groups:
            rank = []
            for g in range(groups):
                two = np.sort(key[t, g * per:(g + 1) * per])[::-1][:2]
                rank.append(two[0] + two[1] if per > 1 else two[0])
            best = np.argsort(-np.array(rank), kind="stable")[:topk_groups]
            allowed = np.concatenate([np.arange(g * per, (g + 1) * per) for g in sorted(best)])
        order = np.argsort(-key[t, allowed], kind="stable")[:k]
        out[t] = np.sort(allowed[order])
    return out


def weights(z, idx, scoring, normalize, scaling):
    s = np.take_along_axis(scores(z, scoring), idx, 1)
    return s / (s.sum(1, keepdims=True) + 1e-20) * scaling if normalize else s * scaling


def weights_backward(dp, z, idx, scoring, normalize, scaling):
    """dz and the sums of |terms| of its elements."""
    s = scores(z, scoring)
    sel = np.take_along_axis(s, idx, 1)
    if normalize:
        total = sel.sum(1, keepdims=True) + 1e-20
        ds = scaling / total * (dp - (dp * sel).sum(1, keepdims=True) / total)
        mag = scaling / total * (np.abs(dp) + (np.abs(dp) * sel).sum(1, keepdims=True) / total)
    else:
        ds, mag = dp * scaling, np.abs(dp) * scaling
    full, full_mag = np.zeros_like(s), np.zeros_like(s)
    np.put_along_axis(full, idx, ds, 1)
    np.put_along_axis(full_mag, idx, mag, 1)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            rest = 1.0 / (1.0 + np.exp(z))
        return full * s * rest, full_mag * s * rest
    # sum of s ds: with normalised weights, total - sum(sel) being 1e-20 by definition,
    #   c / total (g - g sum(sel) / total) = c g 1e-20 / total^2  for g = sum(dp sel),
    # in which nothing cancels (float64 would leave 1e-17 of it)
    if normalize:
        dot = scaling * (dp * sel).sum(1, keepdims=True) * 1e-20 / total ** 2
    else:
        dot = (s * full).sum(1, keepdims=True)
    dz = s * (full - dot)
    return dz, s * (full_mag + (0.0 if normalize else (s * full_mag).sum(1, keepdims=True)))


# ------------------------------------------------------------- 4 bits
def e2m1(u: np.ndarray) -> np.ndarray:
    """Codes of the nearest of the eight magnitudes (ties: the even code), with the sign bit."""
    code = np.zeros(u.shape, np.uint8)
    a = np.abs(u)
    for i in range(1, 8):
        mid = (MAGS[i - 1] + MAGS[i]) / 2
        code[a >= mid if i % 2 == 0 else a > mid] = i
    return code | (np.signbit(u).astype(np.uint8) << 3)


def mx_quantize(x: np.ndarray):
    """Finite float32 [rows, K] -> (codes uint8 [rows, K], biased exponents uint8 [rows, K/32])."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    b = x.reshape(rows, K // BLOCK, BLOCK)
    biased = np.abs(b).max(-1).view(np.uint32).astype(np.int64) >> 23
    e = np.maximum(biased - 2, 0)
    return e2m1(b.astype(np.float64) * 2.0 ** (127 - e)[..., None]).reshape(rows, K), e.astype(np.uint8)


def mx_pack(codes: np.ndarray) -> np.ndarray:
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def mx_values(q: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """float64 values of packed codes and exponent bytes below 255."""
    codes = np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)
    v = MAGS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(2.0 ** (scale.astype(np.float64) - 127), BLOCK, -1)
