"""The root-mean-square norm and its gradients in 64 bits, row by row, and the INT8 codes
by the same binary32 steps that define them.  numpy only; shares no code with the kernels."""
from __future__ import annotations

import numpy as np


def inverse(h: np.ndarray, eps: float) -> np.ndarray:
    """(rows, 1): 1 / sqrt(mean of squares + eps)."""
    with np.errstate(all="ignore"):
        return 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + np.float64(np.float32(eps)))


def forward(h: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    with np.errstate(all="ignore"):
        return h * inverse(h, eps) * w


def codes(h: np.ndarray, w: np.ndarray, eps: float):
    """(q, scale): q from t = h w and 127 * (1 / max |t|) in binary32, scale in 64 bits."""
    with np.errstate(all="ignore"):
        t = h.astype(np.float32) * w.astype(np.float32)
        m = np.abs(t).max(axis=1, keepdims=True)
        fine = np.isfinite(t).all(axis=1, keepdims=True)
        # (a power of two keeps 1 / m in binary32's normal range)
        d = np.where(m < 2.0 ** -64, 2.0 ** 64, np.where(m > 2.0 ** 64, 2.0 ** -64, 1.0)).astype(np.float32)
        q = np.rint((t * d) * (np.float32(127) * (np.float32(1) / (m * d))))
        scale = np.abs(h * w).max(axis=1, keepdims=True) * inverse(h, eps) / 127.0
    q = np.where(fine & (m > 0), q, 0.0)
    return q, np.where(fine, np.where(m > 0, scale, 0.0), np.nan)[:, 0]


def backward(dy: np.ndarray, h: np.ndarray, w: np.ndarray, eps: float, dh: np.ndarray | None = None):
    """(dx, dw), and the magnitudes that their roundings are relative to."""
    r = inverse(h, eps)
    n, g = h * r, dy * w
    dx = r * (g - n * np.mean(g * n, axis=1, keepdims=True))
    size = r * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), axis=1, keepdims=True))
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    return dx, (dy * n).sum(axis=0), size, np.abs(dy * n).sum(axis=0)
