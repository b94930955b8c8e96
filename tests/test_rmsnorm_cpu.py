"""CPU checks of the norm: the oracle against the formulas differently put, and the C ABI's
and the binding's refusals (dummy pointers that are never dereferenced)."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

import oracle.norm as rn
from tests.test_abi_cpu import LIB, codes

built = pytest.mark.skipif(not os.path.exists(LIB), reason="libpdgemm.so not built")


def test_oracle_rows_by_hand():
    h = np.array([[3.0, -4.0, 0.0, 0.0]])
    y = rn.forward(h, np.array([1.0, 2.0, 5.0, 1.0]), 0.0)             # mean of squares 25 / 4
    assert np.allclose(y, [[1.2, -3.2, 0.0, 0.0]], rtol=1e-15)
    q, s = rn.codes(h, np.array([1.0, 2.0, 5.0, 1.0]), 0.0)
    assert q.tolist() == [[48.0, -127.0, 0.0, 0.0]] and np.allclose(s, 3.2 / 127, rtol=1e-15)   # 3 * (127 / 8) = 47.6


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(1)
    h, g, w = rng.standard_normal((2, 5)), rng.standard_normal((2, 5)), rng.standard_normal(5)
    dx, dw, _, _ = rn.backward(g, h, w, 1e-3)
    loss = lambda h, w: (rn.forward(h, w, 1e-3) * g).sum()  # noqa: E731
    for i in range(2):
        for j in range(5):
            d = np.zeros((2, 5))
            d[i, j] = 1e-6
            assert abs((loss(h + d, w) - loss(h - d, w)) / 2e-6 - dx[i, j]) < 1e-8
    for j in range(5):
        d = np.zeros(5)
        d[j] = 1e-6
        assert abs((loss(h, w + d) - loss(h, w - d)) / 2e-6 - dw[j]) < 1e-8


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(LIB)
    i64, p, i, f = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.pdgemm_rms_norm.argtypes = [i64, i64, p, i64, i, p, i64, p, i64, p, i, f, p, i64, i, p, p]
    L.pdgemm_rms_norm_backward.argtypes = [i64, i64, p, i64, p, i64, p, i64, i, p, i, f, p, i64, p, p, i64, p]
    L.pdgemm_rms_norm_backward_workspace_size.argtypes = [i64, i64]
    L.pdgemm_rms_norm_backward_workspace_size.restype = i64
    return L


P = {n: 0x10000 * (k + 1) for k, n in enumerate(("x", "res", "sum", "w", "out", "scale", "dy", "h", "dh", "dx", "dw", "ws"))}


def norm(L, rows=4, cols=64, ldx=64, type=2, ldr=64, lds=64, wtype=2, eps=1e-5, ldo=64, otype=3, **ptr):
    p = {**P, **ptr}
    return L.pdgemm_rms_norm(rows, cols, p["x"], ldx, type, p["res"], ldr, p["sum"], lds, p["w"], wtype, eps, p["out"], ldo,
                             otype, p["scale"], None)


def grad(L, rows=4, cols=64, lddy=64, ldh=64, lddh=64, type=2, wtype=2, eps=1e-5, lddx=64, ws_bytes=1 << 20, **ptr):
    p = {**P, **ptr}
    return L.pdgemm_rms_norm_backward(rows, cols, p["dy"], lddy, p["h"], ldh, p["dh"], lddh, type, p["w"], wtype, eps, p["dx"],
                                      lddx, p["dw"], p["ws"], ws_bytes, None)


NAN = float("nan")
REFUSED = [
    (norm, "EINVAL_CFG", dict(type=3)), (norm, "EINVAL_CFG", dict(type=-1)), (norm, "EINVAL_CFG", dict(wtype=3)),
    (norm, "EINVAL_CFG", dict(otype=4)), (norm, "EINVAL_CFG", dict(eps=-1e-9)), (norm, "EINVAL_CFG", dict(eps=NAN)),
    (norm, "EINVAL_CFG", dict(eps=float("inf"))), (norm, "EINVAL_DIM", dict(rows=-1)), (norm, "EINVAL_DIM", dict(cols=-1)),
    (norm, "EINVAL_DIM", dict(cols=32769, ldx=32769, ldr=32769, lds=32769, ldo=32769)),
    (norm, "EINVAL_DIM", dict(rows=2 ** 30 + 1)), (norm, "EINVAL_LD", dict(ldx=63)), (norm, "EINVAL_LD", dict(ldr=63)),
    (norm, "EINVAL_LD", dict(lds=63)), (norm, "EINVAL_LD", dict(ldo=63)), (norm, "EINVAL_LD", dict(ldx=2 ** 21 + 1)),
    (norm, "EINVAL_LD", dict(ldo=2 ** 22 + 1)), (norm, "ENULL", dict(x=None)), (norm, "ENULL", dict(res=None)),
    (norm, "ENULL", dict(sum=None)), (norm, "ENULL", dict(w=None)), (norm, "ENULL", dict(out=None)),
    (norm, "ENULL", dict(scale=None)), (norm, "EALIGN", dict(x=P["x"] + 1)), (norm, "EALIGN", dict(res=P["res"] + 1)),
    (norm, "EALIGN", dict(sum=P["sum"] + 1)), (norm, "EALIGN", dict(w=P["w"] + 2, wtype=0)),
    (norm, "EALIGN", dict(out=P["out"] + 2, otype=0)), (norm, "EALIGN", dict(scale=P["scale"] + 2)),
    (grad, "EINVAL_CFG", dict(type=3)), (grad, "EINVAL_CFG", dict(wtype=-1)), (grad, "EINVAL_CFG", dict(eps=NAN)),
    (grad, "EINVAL_DIM", dict(rows=-1)), (grad, "EINVAL_DIM", dict(cols=32769, lddy=32769, ldh=32769, lddh=32769, lddx=32769)),
    (grad, "EINVAL_LD", dict(lddy=63)), (grad, "EINVAL_LD", dict(ldh=63)), (grad, "EINVAL_LD", dict(lddh=63)),
    (grad, "EINVAL_LD", dict(lddx=63)), (grad, "ENULL", dict(dy=None)), (grad, "ENULL", dict(h=None)),
    (grad, "ENULL", dict(w=None)), (grad, "ENULL", dict(dx=None)), (grad, "ENULL", dict(dw=None)),
    (grad, "ENULL", dict(ws=None)), (grad, "EWORKSPACE", dict(ws=P["ws"] + 8)), (grad, "EWORKSPACE", dict(ws_bytes=64 * 4)),
    (grad, "EWORKSPACE", dict(ws_bytes=-1)), (grad, "EALIGN", dict(dy=P["dy"] + 1)), (grad, "EALIGN", dict(dw=P["dw"] + 2)),
    (grad, "EALIGN", dict(dh=P["dh"] + 1)), (grad, "EALIGN", dict(dx=P["dx"] + 1)),
]


@built
@pytest.mark.parametrize("fn,code,bad", REFUSED, ids=[f"{f.__name__}-{c}-{n}" for n, (f, c, b) in enumerate(REFUSED)])
def test_refusals(lib, fn, code, bad):
    if fn is grad and "rows" not in bad and "cols" not in bad:
        bad = {"rows": 40, **bad}                       # (several workgroups: a workspace is needed)
    assert fn(lib, **bad) == codes()["PDGEMM_" + code]


@built
def test_empty_calls_and_workspace_sizes(lib):
    none = {k: None for k in P}
    assert norm(lib, rows=0, **none) == 0 and norm(lib, cols=0, **none) == 0 and grad(lib, cols=0, **none) == 0
    size = lib.pdgemm_rms_norm_backward_workspace_size
    assert size(1, 8192) == 0 and size(0, 8192) == 0 and size(-1, 5) == 0 and size(5, 40000) == 0
    assert size(2, 8192) == 2 * 8192 * 4 and size(10 ** 6, 8192) == 256 * 8192 * 4


@built
def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    x, w = torch.zeros(4, 32), torch.zeros(32)
    for error, call in [
        (TypeError, lambda: pd.rms_norm(x.double(), w)), (TypeError, lambda: pd.rms_norm(x, w.double())),
        (TypeError, lambda: pd.rms_norm(x, None)), (TypeError, lambda: pd.rms_norm(x, w, residual=x.half())),
        (TypeError, lambda: pd.rms_norm(x, w, out_dtype=torch.int8)), (ValueError, lambda: pd.rms_norm(x, w[:31])),
        (ValueError, lambda: pd.rms_norm(x, torch.zeros(64)[::2])), (ValueError, lambda: pd.rms_norm(x[0], w)),
        (ValueError, lambda: pd.rms_norm(x.t(), torch.zeros(4))), (ValueError, lambda: pd.rms_norm(x, w, sum_out=x)),
        (ValueError, lambda: pd.rms_norm(x, w, residual=x[:3])), (ValueError, lambda: pd.rms_norm(x, w, out=x[:3])),
        (ValueError, lambda: pd.rms_norm(x, w)),                                   # not on a GPU
        (TypeError, lambda: pd.rms_norm_i8(x, w, out=(x, w))), (ValueError, lambda: pd.rms_norm_i8(x, w)),
        (ValueError, lambda: pd.rms_norm_i8(x, w, out=(x.to(torch.int8), torch.zeros(3)))),
        (TypeError, lambda: pd.rms_norm_backward(x.half(), x, w)), (TypeError, lambda: pd.rms_norm_backward(x, x, w, out=x.half())),
        (ValueError, lambda: pd.rms_norm_backward(x, x[:3], w)), (ValueError, lambda: pd.rms_norm_backward(x, x, w)),
        (ValueError, lambda: pd.rms_norm_backward(x, x, w, dweight=torch.zeros(31))),
    ]:
        with pytest.raises(error):
            call()
