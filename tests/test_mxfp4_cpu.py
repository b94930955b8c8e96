"""CPU checks of MXFP4: the oracle against independent restatements of the format, and the
C ABI's and the binding's refusals (dummy pointers that are never dereferenced)."""
from __future__ import annotations

import ctypes
import os
from fractions import Fraction

import numpy as np
import pytest

import oracle.mxfp4 as mx
from tests.test_abi_cpu import LIB, codes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libpdgemm.so not built")


# ---- the oracle ----

def test_e2m1_values_from_their_bits():
    for code in range(8):
        e, m = code >> 1, code & 1
        assert mx.E2M1[code] == (m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))


def test_rounding_is_to_nearest_and_ties_to_even():
    xs = np.concatenate([np.arange(0, 1025) / 128.0, np.nextafter(np.arange(0, 65) / 8.0, 0),
                         np.nextafter(np.arange(0, 65) / 8.0, 100)])
    for x, c in zip(xs, mx.nearest_code(xs)):
        d = [abs(Fraction(float(v)) - min(Fraction(float(x)), Fraction(6))) for v in mx.E2M1]
        best = [i for i in range(8) if d[i] == min(d)]
        assert int(c) == (best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)), x


@pytest.mark.parametrize("rule", ["floor", "fit"])
def test_scale_rule_by_search(rule):
    # the exponent by trying them all, for magnitudes around every power of two of interest
    mags = []
    for p in (-149, -130, -127, -126, -125, -124, -1, 0, 1, 100, 127):
        for f in (1.0, np.nextafter(1.0, 2, dtype=np.float32), 1.25, 1.5,
                  np.nextafter(np.float32(1.5), np.float32(2)), 1.75, 2 - 2.0 ** -23):
            mags.append(np.float32(np.ldexp(float(f), p)))
    mags = np.array([m for m in mags if 0 < m < np.inf], np.float32)
    _, scales = mx.quantize(mags[:, None], rule)
    for m, byte in zip(mags, scales[0]):
        m = Fraction(float(m))
        fits = (lambda e: m < 8 * Fraction(2) ** e) if rule == "floor" else (lambda e: m <= 6 * Fraction(2) ** e)
        assert int(byte) - 127 == next(e for e in range(-127, 128) if fits(e)), float(m)


def test_special_blocks():
    x = np.ones((5, 64))
    x[0, 3], x[1, 40], x[2, 0] = np.nan, np.inf, -np.inf
    x[3, :32] = 0.0
    x[4, :] = -0.0
    q, s = mx.quantize(x)
    assert s[:, 0].tolist() == [255, 125] and s[:, 1].tolist() == [125, 255] and s[0, 2] == 255
    assert not q[0, :16].any() and not q[1, 16:].any() and not q[2, :16].any()
    assert s[0, 3] == 0 and not q[3, :16].any()
    assert (q[4] == 0x88).all()                       # the sign of a zero is kept
    v = mx.values(q, s, 64)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()


def test_values_and_packing_order():
    codes_ = np.array([[0x21, 0x43, 0x65, 0x87] + [0] * 12], np.uint8)
    v = mx.values(codes_, np.array([[128]], np.uint8), 8)
    assert v.tolist() == [[1.0, 2.0, 3.0, 4.0, 6.0, 8.0, 12.0, -0.0]]
    q, s = mx.quantize(v)
    assert (q[:, :4] == codes_[:, :4]).all() and s[0, 0] == 128
    assert mx.quantize(np.zeros((3, 33)))[0].shape == (3, 32)


def test_product_is_the_plain_sum():
    rng = np.random.default_rng(5)
    a, b = rng.standard_normal((5, 70)), rng.standard_normal((4, 70))
    qa, qb = mx.quantize(a), mx.quantize(b)
    va, vb = mx.values(*qa, 70), mx.values(*qb, 70)
    R, S = mx.product(va, vb)
    for i in range(5):
        for j in range(4):
            exact = sum(Fraction(x) * Fraction(y) for x, y in zip(va[i].tolist(), vb[j].tolist()))
            mag = sum(abs(Fraction(x) * Fraction(y)) for x, y in zip(va[i].tolist(), vb[j].tolist()))
            assert abs(exact - Fraction(R[i, j])) <= Fraction(1, 2 ** 40) * mag
            assert abs(mag - Fraction(S[i, j])) <= Fraction(1, 2 ** 40) * mag
    va[2, 5] = np.nan
    R, _ = mx.product(va, vb)
    assert np.isnan(R[2]).all() and np.isfinite(np.delete(R, 2, 0)).all()


# ---- refusals of the C ABI ----

P = dict(src=0x10000, q=0x20000, s=0x30000, qt=0x40000, st=0x50000, dst=0x60000, A=0x70000, sa=0x80000, B=0x90000,
         sb=0xA0000, C=0xB0000)


@pytest.fixture(scope="module")
def lib():
    L = ctypes.CDLL(LIB)
    i64, p, i = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    L.pdgemm_mxf4_quantize.argtypes = [i64, i64, p, i64, i, p, i64, p, i64, p, i64, p, i64, i, p]
    L.pdgemm_mxf4_dequantize.argtypes = [i64, i64, p, i64, p, i64, p, i64, i, p]
    L.gemm_mxf4.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p, i64, i, p]
    L.gemm_a16_mxf4.argtypes = [i64, i64, i64, p, i64, i, p, i64, p, i64, p, i64, i, p]
    return L


def quantize(L, rows=64, K=96, ld=96, type=0, ldq=96, lds=64, ldqt=64, ldst=96, rule=0, **ptrs):
    a = {**P, **ptrs}
    return L.pdgemm_mxf4_quantize(rows, K, a["src"], ld, type, a["q"], ldq, a["s"], lds, a["qt"], ldqt, a["st"], ldst,
                                  rule, None)


def dequantize(L, rows=64, K=96, ldq=96, lds=64, ldd=96, type=0, **ptrs):
    a = {**P, **ptrs}
    return L.pdgemm_mxf4_dequantize(rows, K, a["q"], ldq, a["s"], lds, a["dst"], ldd, type, None)


def product(L, M=64, N=80, K=96, lda=96, ldsa=64, ldb=96, ldsb=80, ldc=80, type=0, **ptrs):
    a = {**P, **ptrs}
    return L.gemm_mxf4(M, N, K, a["A"], lda, a["sa"], ldsa, a["B"], ldb, a["sb"], ldsb, a["C"], ldc, type, None)


def a16(L, M=64, N=80, K=96, lda=96, a_type=1, ldb=96, ldsb=80, ldc=80, type=0, **ptrs):
    a = {**P, **ptrs}
    return L.gemm_a16_mxf4(M, N, K, a["A"], lda, a_type, a["B"], ldb, a["sb"], ldsb, a["C"], ldc, type, None)


REFUSED = [
    (quantize, "EINVAL_CFG", dict(type=3)), (quantize, "EINVAL_CFG", dict(type=-1)),
    (quantize, "EINVAL_CFG", dict(rule=2)), (quantize, "EINVAL_CFG", dict(rule=2, rows=-1)),
    (quantize, "EINVAL_DIM", dict(rows=-1)), (quantize, "EINVAL_DIM", dict(K=-1)),
    (quantize, "EINVAL_DIM", dict(K=2 ** 30 + 1)), (quantize, "EINVAL_DIM", dict(rows=2 ** 31)),
    (quantize, "EINVAL_LD", dict(ld=95)), (quantize, "EINVAL_LD", dict(ldq=64)), (quantize, "EINVAL_LD", dict(lds=48)),
    (quantize, "EINVAL_LD", dict(ldqt=32)), (quantize, "EINVAL_LD", dict(ldst=80)),
    (quantize, "ENULL", dict(src=None)), (quantize, "ENULL", dict(q=None)), (quantize, "ENULL", dict(s=None)),
    (quantize, "ENULL", dict(qt=None)), (quantize, "ENULL", dict(st=None)),
    (quantize, "ENULL", dict(q=None, s=None, qt=None, st=None)),
    (quantize, "EINVAL_LD", dict(ld=2 ** 20 + 1)), (quantize, "EINVAL_LD", dict(ld=2 ** 21 + 1, type=1)),
    (quantize, "EINVAL_LD", dict(ldq=2 ** 23 + 32)), (quantize, "EINVAL_LD", dict(lds=2 ** 22 + 16)),
    (quantize, "EALIGN", dict(src=P["src"] + 2)), (quantize, "EALIGN", dict(src=P["src"] + 1, type=2)),
    (quantize, "EALIGN", dict(q=P["q"] + 8)), (quantize, "EALIGN", dict(s=P["s"] + 4)),
    (quantize, "EALIGN", dict(ldq=112)), (quantize, "EALIGN", dict(lds=72)), (quantize, "EALIGN", dict(ldqt=80)),
    (quantize, "EALIGN", dict(ldst=104)), (quantize, "EALIGN", dict(qt=P["qt"] + 1)),
    (dequantize, "EINVAL_CFG", dict(type=3)), (dequantize, "EINVAL_DIM", dict(rows=-1)),
    (dequantize, "EINVAL_LD", dict(ldq=64)), (dequantize, "EINVAL_LD", dict(lds=48)),
    (dequantize, "EINVAL_LD", dict(ldd=95)), (dequantize, "ENULL", dict(q=None)), (dequantize, "ENULL", dict(s=None)),
    (dequantize, "ENULL", dict(dst=None)), (dequantize, "EALIGN", dict(dst=P["dst"] + 2)),
    (dequantize, "EINVAL_LD", dict(ldd=2 ** 20 + 1)), (dequantize, "EALIGN", dict(ldq=112)),
    (product, "EINVAL_CFG", dict(type=3)), (product, "EINVAL_DIM", dict(M=-1)), (product, "EINVAL_DIM", dict(N=-1)),
    (product, "EINVAL_DIM", dict(K=-1)), (product, "EINVAL_LD", dict(lda=64)), (product, "EINVAL_LD", dict(ldb=64)),
    (product, "EINVAL_LD", dict(ldsa=48)), (product, "EINVAL_LD", dict(ldsb=64)), (product, "EINVAL_LD", dict(ldc=79)),
    (product, "ENULL", dict(A=None)), (product, "ENULL", dict(sa=None)), (product, "ENULL", dict(B=None)),
    (product, "ENULL", dict(sb=None)), (product, "ENULL", dict(C=None)), (product, "EALIGN", dict(A=P["A"] + 8)),
    (product, "EALIGN", dict(sb=P["sb"] + 8)), (product, "EALIGN", dict(lda=112)), (product, "EALIGN", dict(ldsb=88)),
    (product, "EALIGN", dict(C=P["C"] + 2)), (product, "EALIGN", dict(C=P["C"] + 1, type=2)),
    (product, "EINVAL_LD", dict(ldc=2 ** 20 + 1)), (product, "EINVAL_LD", dict(ldsa=2 ** 22 + 16)),
    (a16, "EINVAL_CFG", dict(a_type=0)), (a16, "EINVAL_CFG", dict(type=3)), (a16, "EINVAL_DIM", dict(M=-1)),
    (a16, "EINVAL_LD", dict(lda=95)), (a16, "EINVAL_LD", dict(ldb=64)), (a16, "EINVAL_LD", dict(ldc=79)),
    (a16, "EINVAL_LD", dict(lda=2 ** 21 + 8)), (a16, "ENULL", dict(A=None)), (a16, "ENULL", dict(sb=None)),
    (a16, "EALIGN", dict(A=P["A"] + 8)), (a16, "EALIGN", dict(lda=100)), (a16, "EALIGN", dict(ldb=112)),
]


@built
@pytest.mark.parametrize("fn,code,bad", REFUSED, ids=[f"{f.__name__}-{c}-{'-'.join(map(str, b))}-{n}"
                                                      for n, (f, c, b) in enumerate(REFUSED)])
def test_refusals(lib, fn, code, bad):
    assert fn(lib, **bad) == codes()["PDGEMM_" + code]


@built
def test_empty_calls_succeed_without_pointers(lib):
    none = {k: None for k in P}
    assert quantize(lib, rows=0, **none) == 0 and quantize(lib, K=0, **none) == 0
    assert dequantize(lib, rows=0, **none) == 0 and dequantize(lib, K=0, **none) == 0
    assert product(lib, M=0, **none) == 0 and product(lib, N=0, **none) == 0
    assert a16(lib, M=0, **none) == 0 and a16(lib, N=0, **none) == 0


@built
def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    x = torch.zeros((8, 32))
    u = torch.zeros((8, 16), dtype=torch.uint8)
    with pytest.raises(TypeError):
        pd.mxf4_quantize(x.double())
    with pytest.raises(ValueError):
        pd.mxf4_quantize(x, scale_rule="nearest")
    with pytest.raises(ValueError):
        pd.mxf4_quantize(x)                              # not on a GPU
    with pytest.raises(TypeError):
        pd.gemm_a16_mxf4(x, u, u)                        # float32 activations
    with pytest.raises(TypeError):
        pd.gemm_mxf4(x, u, u, u)
    with pytest.raises(TypeError):
        pd.mxf4_dequantize(u, x)


@pytest.mark.parametrize("K, width, agree", [(32, 16, True), (33, 17, True), (33, 32, True), (64, 33, False),
                                             (32, 32, False), (33, 16, False), (0, 1, False)])
def test_a16_refuses_another_length(K, width, agree):
    """Weights of another K than the activations' are refused by name, not cut to fit; those that
    agree come as far as the check that wants tensors on a GPU."""
    torch = pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    a, codes = torch.zeros((4, K), dtype=torch.float16), torch.zeros((8, width), dtype=torch.uint8)
    scales = torch.zeros((4, 16), dtype=torch.uint8)[:, :8]
    with pytest.raises(ValueError, match="GPU" if agree else "disagree on K|fewer than K"):
        pd.gemm_a16_mxf4(a, codes, scales)


def test_a_single_row_has_no_stride(monkeypatch):
    """The last token of a sequence, h[:, -1, :], is one row that torch strides by the whole
    sequence (and calls contiguous, so that a copy would not mend it).  The library takes rows of
    at most 4 MiB, so the stride of a single row is not passed on."""
    torch = pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    called = []
    monkeypatch.setattr(pd, "_mx_call", lambda fn, args, tensors, stream: called.append(args))

    def row(n, dtype):
        t = torch.empty_strided((1, n), ((1 << 24) + 1, 1), dtype=dtype)
        assert t.is_contiguous()
        return t

    K, N = 90, 50
    x, x16 = row(K, torch.float32), row(K, torch.float16)
    codes, scales = row(45, torch.uint8), torch.zeros((3, 16), dtype=torch.uint8)[:, :1]
    one_block = row(N, torch.uint8)                      # scales of a K of one block
    wide = torch.zeros((N, 48), dtype=torch.uint8)[:, :45], torch.zeros((3, 64), dtype=torch.uint8)[:, :N]
    out = row(N, torch.float32)
    room = torch.as_strided(torch.zeros(48, dtype=torch.uint8), (1, 45), (1 << 24, 1))
    pd.mxf4_quantize(x, out=(room, scales))
    assert called.pop()[3] == K                          # (rows, K, src, ld, type, q, ldq, ...)
    pd.mxf4_quantize(x, out=(room, scales))
    assert called.pop()[6] == 96
    pd.mxf4_dequantize(codes, scales, K, out=row(K, torch.float32))
    args = called.pop()                                  # (rows, K, q, ldq, scales, lds, dst, ldd, type)
    assert (args[3], args[5], args[7]) == (96, 16, K)
    pd.gemm_mxf4(codes, scales, *wide, K, out=out)
    args = called.pop()                                  # (M, N, K, A, lda, sa, ldsa, B, ldb, sb, ldsb, C, ldc, type)
    assert (args[4], args[6], args[8], args[10], args[12]) == (96, 16, 96, 64, N)
    pd.gemm_a16_mxf4(x16, *wide, out=out)
    args = called.pop()                                  # (M, N, K, A, lda, type, B, ldb, sb, ldsb, C, ldc, type)
    assert (args[4], args[7], args[9], args[11]) == (96, 96, 64, N)
    pd.mxf4_dequantize(torch.zeros((N, 16), dtype=torch.uint8), one_block, 32)
    assert called.pop()[5] == 64


@pytest.mark.parametrize("K, width, agree", [(32, 16, True), (33, 17, True), (33, 32, True), (64, 33, False),
                                             (32, 32, False), (33, 16, False), (0, 1, False)])
def test_every_operand_refuses_another_length(K, width, agree):
    """Codes of another K than the call's (in a layer step M, N and K each stand in for another)
    are refused by name by every call that is told K, not cut to fit."""
    torch = pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    fits = -(-K // 32) * 16
    blocks = torch.zeros((4, 16), dtype=torch.uint8)
    good, bad = (torch.zeros((8, w), dtype=torch.uint8) for w in (fits, width))
    scales = blocks[:, :8]
    calls = [lambda: pd.gemm_mxf4(bad, scales, good, scales, K), lambda: pd.gemm_mxf4(good, scales, bad, scales, K)]
    if K:                                                # (nothing to read back or to quantise: no call to the library)
        calls += [lambda: pd.mxf4_dequantize(bad, scales, K),
                  lambda: pd.mxf4_quantize(torch.zeros((8, K)), out=(torch.zeros((9, 64), dtype=torch.uint8)[:8, :width], scales)),
                  lambda: pd.mxf4_quantize(torch.zeros((K, 8)), transpose=True,
                                           out=(torch.zeros((9, 64), dtype=torch.uint8)[:8, :width], scales))]
    for call in calls:
        with pytest.raises(ValueError, match="GPU" if agree else "disagree on K|fewer than K"):
            call()


@built
def test_alignment_message_names_the_operands():
    # scales of 4 bits' blocks have a stricter rule than the dequantizing epilogue's
    L = ctypes.CDLL(LIB)
    L.pdgemm_strerror.restype = ctypes.c_char_p
    message = L.pdgemm_strerror(codes()["PDGEMM_EALIGN"]).decode()
    assert "MXFP4 codes and scales" in message and "rows of a multiple of 16 bytes" in message
