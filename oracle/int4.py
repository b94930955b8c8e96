"""Group-scaled INT4 weights in 64 bits: packing, values, products, and a
mixture-of-experts layer of them.  numpy only; shares no code with the kernels."""
from __future__ import annotations

import numpy as np


def pack(codes: np.ndarray) -> np.ndarray:
    """Signed codes (..., K) in [-8, 7] -> bytes (..., ceil(K/2)), the even k in the low nibble."""
    if codes.shape[-1] % 2:
        codes = np.concatenate([codes, np.zeros(codes.shape[:-1] + (1,), codes.dtype)], axis=-1)
    u = (codes.astype(np.int64) % 16).astype(np.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def values(codes: np.ndarray, scales: np.ndarray, group: int) -> np.ndarray:
    """codes (N, K) times scales (groups, N), stored by group."""
    q = np.arange(codes.shape[1]) // group
    return codes.astype(np.float64) * scales.astype(np.float64)[q].T


def product(a: np.ndarray, w: np.ndarray):
    """(a w^T, the sums of magnitudes)."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def route(logits: np.ndarray, top: int):
    """(ids, weights): the largest logits of each row, ties to the lower index, and their softmax among
    themselves; -inf is not taken (id -1, weight 0).  A row with a NaN or +inf has weights NaN where taken, a NaN
    counting as the largest."""
    T, E = logits.shape
    ids, weights = np.full((T, top), -1, np.int64), np.zeros((T, top))
    for t in range(T):
        key = [(0 if np.isnan(v) else 1, -v if not np.isnan(v) else 0.0, e) for e, v in enumerate(logits[t])]
        order = [k[2] for k in sorted(key) if not logits[t, k[2]] == -np.inf][:top]
        if not order:
            continue
        v = logits[t, order].astype(np.float64)
        with np.errstate(invalid="ignore"):
            p = np.exp(v - v[0])
            ids[t, :len(order)], weights[t, :len(order)] = order, p / p.sum()
    return ids, weights


def experts(x, ids, weights, w13, w2, m13=None, m2=None):
    """y (T, H) for lists of dense expert weights w13[e] (2I, H), w2[e] (H, I), and what its errors are relative to: the
    sum of its terms' magnitudes; what changes of the first product's sums of |m13| |x| do to it; the sums of |m2| times
    the gated activations; and of |w2| (one unit of such an activation).  m13, m2: magnitudes in the place of the
    weights' (their scales', say).  An id outside the list adds nothing."""
    m13 = w13 if m13 is None else m13
    m2 = w2 if m2 is None else m2
    y, size, act_size, second, mass = (np.zeros_like(x) for _ in range(5))
    for t in range(x.shape[0]):
        for slot, e in enumerate(ids[t]):
            if not 0 <= e < len(w13):
                continue
            I = w2[e].shape[1]
            both = w13[e] @ x[t]
            mag = np.abs(m13[e]) @ np.abs(x[t])
            g, u = both[:I], both[I:]
            s = 1.0 / (1.0 + np.exp(-g))
            act = g * s * u
            # a change of g or u changes act by so much: |d silu| <= 1.1
            change = 1.1 * mag[:I] * np.abs(u) + np.abs(g * s) * mag[I:]
            wt = np.abs(weights[t, slot])
            y[t] += weights[t, slot] * (w2[e] @ act)
            size[t] += wt * (np.abs(w2[e]) @ np.abs(act))
            act_size[t] += wt * (np.abs(w2[e]) @ change)
            second[t] += wt * (np.abs(m2[e]) @ np.abs(act))
            mass[t] += np.abs(w2[e]).sum(axis=1)
    return y, size, act_size, second, mass
