"""Plain statement of the microscaled 4-bit float operators, in NumPy and 64 bits.

Shares no code with the kernels.  Format (OCP Microscaling Formats, MXFP4):
32 consecutive elements of a row share one scale byte b standing for
2^(b - 127); an element is a 4-bit float e2m1 with magnitudes GRID; codes are
packed two to a byte, even k in the low nibble.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_SCALE = 255


def quantize(x: np.ndarray):
    """x [M, K] (float64 values of 16-bit floats) -> (codes, scales) uint8."""
    M, K = x.shape
    v = np.asarray(x, dtype=np.float64).reshape(M, K // BLOCK, BLOCK)
    scales = np.zeros((M, K // BLOCK), dtype=np.uint8)
    codes = np.zeros(v.shape, dtype=np.uint8)
    for m in range(M):
        for b in range(K // BLOCK):
            blk = v[m, b]
            if not np.all(np.isfinite(blk)):
                scales[m, b] = NAN_SCALE
                continue
            top = float(np.max(np.abs(blk)))
            if top > 0:
                scales[m, b] = min(254, max(0, int(np.frexp(top)[1]) - 1 - 2 + 127))
            u = np.abs(blk) / 2.0 ** (int(scales[m, b]) - 127)
            dist = np.abs(u[:, None] - GRID[None, :])
            near = np.argmin(dist, axis=1)  # the lower code of two equally near
            tie = (near < 7) & (dist[np.arange(BLOCK), near] == dist[np.arange(BLOCK), np.minimum(near + 1, 7)])
            near = np.where(tie & (near % 2 == 1), near + 1, near)  # ties to the even code
            codes[m, b] = near + 8 * np.signbit(blk)
    flat = codes.reshape(M, K // 2, 2)
    return flat[..., 0] | (flat[..., 1] << 4), scales


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The float64 values [..., K] of codes [..., K/2] and scales [..., K/32]."""
    low, high = codes & 15, codes >> 4
    n = np.stack([low, high], axis=-1).reshape(*codes.shape[:-1], -1)
    v = GRID[n & 7] * np.where(n >> 3, -1.0, 1.0)
    s = np.where(scales == NAN_SCALE, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, BLOCK, axis=-1)


def top_k(logits: np.ndarray, k: int) -> np.ndarray:
    """Indices [T, k] by descending logit, the lower index first among equals."""
    return np.argsort(-logits, axis=1, kind="stable")[:, :k]


def moe(x: np.ndarray, router: np.ndarray, up: np.ndarray, down: np.ndarray, k: int):
    """y [T, H] and the choice [T, k] for x [T, H], router [E, H], up [E, 2 I, H], down [E, H, I]."""
    logits = x @ router.T
    ids = top_k(logits, k)
    chosen = np.take_along_axis(logits, ids, 1)
    p = np.exp(chosen - chosen.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    I = up.shape[1] // 2
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(k):
            gu = up[ids[t, j]] @ x[t]
            h = gu[:I] / (1.0 + np.exp(-gu[:I])) * gu[I:]
            y[t] += p[t, j] * (down[ids[t, j]] @ h)
    return y, ids
