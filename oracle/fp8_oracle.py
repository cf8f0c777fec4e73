"""Oracle of the 8-bit block-scaled operators: CPU, numpy, plain loops over
blocks.  Scales, reciprocals and products that the definition rounds to float32
are rounded there; sums of products are float64."""
from __future__ import annotations

import numpy as np

BLOCK = 128
TOP = np.float32(448.0)
FLOOR = np.float32(2.0 ** -100)


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """float32 values to the nearest e4m3 value (ties to even; finite, |v| < 464)."""
    v = np.asarray(v, dtype=np.float64)
    exp = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = 2.0 ** (exp - 3)  # 3 fraction bits; below 2^-6 the spacing stays 2^-9
    return np.rint(v / step) * step


def quantize(x: np.ndarray, rows: int, cols: int):
    """(values as float64, scale float32) of blocks of rows x cols."""
    x = np.asarray(x, dtype=np.float32)
    R, C = x.shape
    nr, nc = -(-R // rows), -(-C // cols)
    q = np.zeros((R, C))
    scale = np.zeros((nr, nc), np.float32)
    for i in range(nr):
        for j in range(nc):
            blk = x[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols]
            a = max(np.max(np.abs(blk)), FLOOR)
            scale[i, j] = a / TOP
            q[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols] = e4m3_round(blk * (TOP / a))
    return q, scale


def values(q: np.ndarray, scale: np.ndarray, rows: int, cols: int) -> np.ndarray:
    """What q and its scales stand for, float64."""
    s = np.repeat(np.repeat(scale.astype(np.float64), rows, 0), cols, 1)
    return np.asarray(q, np.float64) * s[: q.shape[0], : q.shape[1]]


def linear(x: np.ndarray, w: np.ndarray, dy: np.ndarray):
    """y, dx, dW of the quantised linear layer and the sums of |terms| of each."""
    xv = values(*quantize(x, 1, BLOCK), 1, BLOCK)
    wv = values(*quantize(w, BLOCK, BLOCK), BLOCK, BLOCK)
    dv = values(*quantize(dy, 1, BLOCK), 1, BLOCK)
    xt = values(*quantize(x.T, 1, BLOCK), 1, BLOCK)
    dt = values(*quantize(dy.T, 1, BLOCK), 1, BLOCK)
    outs = (xv @ wv.T, dv @ wv, dt @ xt.T)
    mags = (np.abs(xv) @ np.abs(wv).T, np.abs(dv) @ np.abs(wv), np.abs(dt) @ np.abs(xt).T)
    return outs, mags
