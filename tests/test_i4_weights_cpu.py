"""CPU checks of the operators with group-scaled INT4 weights: the oracle against its
definition differently put, and the C ABI's and the binding's refusals (dummy pointers that
are never dereferenced)."""
from __future__ import annotations

import os

import numpy as np
import pytest

import oracle.int4 as i4
from tests.test_abi_cpu import LIB, codes

built = pytest.mark.skipif(not os.path.exists(LIB), reason="libpdgemm.so not built")


# ---- the oracle ----

def test_packing_order_and_signs():
    assert i4.pack(np.array([[0, 1, 7, -8, -1]])).tolist() == [[0x10, 0x87, 0x0F]]
    every = np.arange(-8, 8)[None, :]
    b = i4.pack(every)
    low, high = b & 15, b >> 4
    back = np.stack([low, high], axis=-1).reshape(1, 16).astype(int)
    assert (np.where(back > 7, back - 16, back) == every).all()


def test_values_take_their_groups_scale():
    v = i4.values(np.array([[2, -3, 5]]), np.array([[0.5], [4.0]]), 2)
    assert v.tolist() == [[1.0, -1.5, 20.0]]


def test_route_by_hand():
    ids, w = i4.route(np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4]), 3)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1]]
    e = np.exp(-2.0)
    assert np.allclose(w, [[1 / (2 + e), 1 / (2 + e), e / (2 + e)], [0, 0, 0]])


def test_experts_by_hand():
    w13 = [np.array([[1.0, 0.0], [0.0, 2.0]])]           # gate reads x0, up reads 2 x1
    w2 = [np.array([[3.0], [-1.0]])]
    y = i4.experts(np.array([[1.0, 5.0], [1.0, 5.0]]), np.array([[0, -1], [0, 0]]), np.array([[0.5, 9.0], [0.25, 0.5]]), w13, w2)[0]
    act = 10.0 / (1 + np.exp(-1.0))
    assert np.allclose(y, [[1.5 * act, -0.5 * act], [2.25 * act, -0.75 * act]])


# ---- refusals ----

@pytest.fixture(scope="module")
def lib():
    pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    return pd.lib


P = {n: 0x10000 * (k + 1) for k, n in enumerate(
    ("A", "B", "s", "C", "x", "ids", "w", "w13", "s13", "w2", "s2", "y", "ws", "logits"))}


def product(L, M=4, N=80, K=96, lda=96, a_type=2, ldb=96, ldsb=80, stype=0, group=32, ldc=80, type=0, cfg=None, ws_bytes=1 << 30,
            **ptr):
    p = {**P, **ptr}
    args = (M, N, K, p["A"], lda, a_type, p["B"], ldb, p["s"], ldsb, stype, group, p["C"], ldc, type, p["ws"], ws_bytes, None)
    return L.gemm_a16_i4(*args) if cfg is None else L.pdgemm_a16_i4_cfg(cfg, *args)


def experts(L, T=4, H=96, I=64, E=8, top=2, ldx=96, type=2, ld13=96, e13=96 * 128, lds13=128, es13=384, ld2=64, e2=64 * 96,
            lds2=96, es2=192, stype=0, group=32, ldy=96, ws_bytes=1 << 20, **ptr):
    p = {**P, **ptr}
    return L.pdgemm_moe_a16_i4(T, H, I, E, top, p["x"], ldx, type, p["ids"], p["w"], p["w13"], ld13, e13, p["s13"], lds13, es13,
                               p["w2"], ld2, e2, p["s2"], lds2, es2, stype, group, p["y"], ldy, p["ws"], ws_bytes, None)


def route(L, T=4, E=16, top=2, ld=16, type=0, **ptr):
    p = {**P, **ptr}
    return L.pdgemm_moe_route(T, E, top, p["logits"], ld, type, 1, p["ids"], p["w"], None)


REFUSED = [
    (product, "EINVAL_CFG", dict(a_type=0)), (product, "EINVAL_CFG", dict(type=3)), (product, "EINVAL_CFG", dict(stype=3)),
    (product, "EINVAL_CFG", dict(group=0)), (product, "EINVAL_CFG", dict(group=-32)), (product, "EINVAL_CFG", dict(group=48)),
    (product, "EINVAL_CFG", dict(cfg=-1)), (product, "EINVAL_CFG", dict(cfg=99)), (product, "EINVAL_DIM", dict(M=-1)),
    (product, "EINVAL_DIM", dict(N=-1)), (product, "EINVAL_DIM", dict(K=-1)),
    (product, "EINVAL_DIM", dict(K=2 ** 30 + 1, lda=2 ** 31, ldb=2 ** 31)), (product, "EINVAL_LD", dict(lda=95)),
    (product, "EINVAL_LD", dict(ldb=64)), (product, "EINVAL_LD", dict(ldsb=79)), (product, "EINVAL_LD", dict(ldc=79)),
    (product, "EINVAL_LD", dict(lda=2 ** 21 + 8)), (product, "EINVAL_LD", dict(ldb=2 ** 23 + 32)),
    (product, "EINVAL_LD", dict(ldsb=2 ** 20 + 1)), (product, "EINVAL_LD", dict(ldc=2 ** 20 + 1)),
    (product, "ENULL", dict(A=None)), (product, "ENULL", dict(B=None)), (product, "ENULL", dict(s=None)),
    (product, "ENULL", dict(C=None)), (product, "EALIGN", dict(A=P["A"] + 8)), (product, "EALIGN", dict(B=P["B"] + 8)),
    (product, "EALIGN", dict(s=P["s"] + 2)), (product, "EALIGN", dict(C=P["C"] + 2)), (product, "EALIGN", dict(lda=100)),
    (product, "EALIGN", dict(ldb=112)),
    (experts, "EINVAL_CFG", dict(type=0)), (experts, "EINVAL_CFG", dict(stype=-1)), (experts, "EINVAL_CFG", dict(group=33)),
    (experts, "EINVAL_DIM", dict(T=-1)), (experts, "EINVAL_DIM", dict(H=0)), (experts, "EINVAL_DIM", dict(I=0)),
    (experts, "EINVAL_DIM", dict(E=0)), (experts, "EINVAL_DIM", dict(E=1025)), (experts, "EINVAL_DIM", dict(top=0)),
    (experts, "EINVAL_DIM", dict(top=65)), (experts, "EINVAL_DIM", dict(T=2049)),
    (experts, "EINVAL_DIM", dict(I=2 ** 20, T=2000, ld13=2 ** 20)), (experts, "EINVAL_LD", dict(ldx=88)),
    (experts, "EINVAL_LD", dict(ldy=95)), (experts, "EINVAL_LD", dict(ld13=64)), (experts, "EINVAL_LD", dict(lds13=127)),
    (experts, "EINVAL_LD", dict(ld2=32)), (experts, "EINVAL_LD", dict(lds2=95)), (experts, "EINVAL_LD", dict(e13=-32)),
    (experts, "EINVAL_LD", dict(es2=-1)), (experts, "EINVAL_LD", dict(T=2000, ldx=2 ** 20)),
    (experts, "EINVAL_LD", dict(ld2=2 ** 23 + 32)), (experts, "ENULL", dict(x=None)), (experts, "ENULL", dict(ids=None)),
    (experts, "ENULL", dict(w=None)), (experts, "ENULL", dict(w13=None)), (experts, "ENULL", dict(s13=None)),
    (experts, "ENULL", dict(w2=None)), (experts, "ENULL", dict(s2=None)), (experts, "ENULL", dict(y=None)),
    (experts, "ENULL", dict(ws=None)), (experts, "EALIGN", dict(x=P["x"] + 8)), (experts, "EALIGN", dict(ldx=100)),
    (experts, "EALIGN", dict(w13=P["w13"] + 4)), (experts, "EALIGN", dict(ld13=112)), (experts, "EALIGN", dict(e2=64 * 96 + 16)),
    (experts, "EALIGN", dict(s2=P["s2"] + 2)), (experts, "EALIGN", dict(ids=P["ids"] + 2)), (experts, "EALIGN", dict(y=P["y"] + 1)),
    (experts, "EWORKSPACE", dict(ws_bytes=64)), (experts, "EWORKSPACE", dict(ws=P["ws"] + 8)),
    (experts, "EWORKSPACE", dict(ws_bytes=-1)),
    (route, "EINVAL_CFG", dict(type=3)), (route, "EINVAL_DIM", dict(T=-1)), (route, "EINVAL_DIM", dict(E=0)),
    (route, "EINVAL_DIM", dict(E=1025, ld=1025)), (route, "EINVAL_DIM", dict(top=0)), (route, "EINVAL_DIM", dict(top=17)),
    (route, "EINVAL_DIM", dict(E=100, ld=100, top=65)), (route, "EINVAL_LD", dict(ld=15)), (route, "ENULL", dict(logits=None)),
    (route, "ENULL", dict(ids=None)), (route, "ENULL", dict(w=None)), (route, "EALIGN", dict(logits=P["logits"] + 2)),
    (route, "EALIGN", dict(ids=P["ids"] + 2)),
]


@built
@pytest.mark.parametrize("fn,code,bad", REFUSED, ids=[f"{f.__name__}-{c}-{n}" for n, (f, c, b) in enumerate(REFUSED)])
def test_refusals(lib, fn, code, bad):
    assert fn(lib, **bad) == codes()["PDGEMM_" + code]


@built
def test_empty_calls_succeed_without_pointers(lib):
    none = {k: None for k in P}
    assert product(lib, M=0, **none) == 0 and product(lib, N=0, **none) == 0
    assert experts(lib, T=0, **none) == 0 and route(lib, T=0, **none) == 0
    assert lib.pdgemm_moe_a16_i4_workspace_size(0, 96, 64, 8, 2) == 0
    assert lib.pdgemm_moe_a16_i4_workspace_size(5, 96, 64, 2000, 2) == 0
    assert lib.pdgemm_moe_a16_i4_workspace_size(5, 96, 60, 8, 2) == 10 * 128 + 48 + 48 + 32 + 2 * 4 * 5 * 96


@built
def test_every_pick_is_a_configuration(lib):
    n = lib.pdgemm_a16_i4_num_configs()
    for M in (1, 3, 8, 9, 16, 17, 32, 33, 64, 65, 100, 128, 129, 500, 2048, 100000):
        for N in (1, 64, 1000, 4096, 8192, 65536):
            for K in (0, 1, 128, 4096, 65536):
                for group in (32, 128):
                    assert 0 <= lib.pdgemm_a16_i4_pick(M, N, K, group) < n


@built
def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    a, b, s = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(2, 8)
    x, ids, w = a, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w13, s13 = torch.zeros(3, 32, 32, dtype=torch.uint8), torch.zeros(3, 2, 32)
    w2, s2 = torch.zeros(3, 64, 16, dtype=torch.uint8)[:, :, :8], torch.zeros(3, 1, 64)
    logits = torch.zeros(4, 3)
    for error, call in [
        (TypeError, lambda: pd.gemm_a16_i4(a.float(), b, s, 32)), (TypeError, lambda: pd.gemm_a16_i4(a, b.to(torch.int8), s, 32)),
        (TypeError, lambda: pd.gemm_a16_i4(a, b, s.double(), 32)), (TypeError, lambda: pd.gemm_a16_i4(a, b, None, 32)),
        (TypeError, lambda: pd.gemm_a16_i4(a, b, s, 32, out_dtype=torch.int32)),
        (ValueError, lambda: pd.gemm_a16_i4(a, b, s, 48)), (ValueError, lambda: pd.gemm_a16_i4(a, b, s, 0)),
        (ValueError, lambda: pd.gemm_a16_i4(a, b[:, :31], s, 32)), (ValueError, lambda: pd.gemm_a16_i4(a, b, s[:1], 32)),
        (ValueError, lambda: pd.gemm_a16_i4(a, b, s.t(), 32)), (ValueError, lambda: pd.gemm_a16_i4(a, b, s[:, :7], 32)),
        (ValueError, lambda: pd.gemm_a16_i4(a, b, s, 32, out=torch.zeros(4, 7))), (ValueError, lambda: pd.gemm_a16_i4(a, b, s, 32)),
        (TypeError, lambda: pd.moe_route(logits.double(), 2)), (ValueError, lambda: pd.moe_route(logits, 2)),
        (TypeError, lambda: pd.moe_route(logits, 2, out=(ids.long(), w))), (ValueError, lambda: pd.moe_route(logits, 1, out=(ids, w))),
        (TypeError, lambda: pd.moe_a16_i4(x.float(), ids, w, w13, s13, w2, s2, 32)),
        (TypeError, lambda: pd.moe_a16_i4(x, ids.long(), w, w13, s13, w2, s2, 32)),
        (TypeError, lambda: pd.moe_a16_i4(x, ids, w.half(), w13, s13, w2, s2, 32)),
        (TypeError, lambda: pd.moe_a16_i4(x, ids, w, w13, s13, w2, s2.half(), 32)),
        (TypeError, lambda: pd.moe_a16_i4(x, ids, w, w13, s13, w2, s2, 32, out=torch.zeros(4, 64))),
        (ValueError, lambda: pd.moe_a16_i4(x, ids[:3], w, w13, s13, w2, s2, 32)),
        (ValueError, lambda: pd.moe_a16_i4(x, ids, w[:, :1], w13, s13, w2, s2, 32)),
        (ValueError, lambda: pd.moe_a16_i4(x, ids, w[:, :1].contiguous(), w13, s13, w2, s2, 32)),
        (ValueError, lambda: pd.moe_a16_i4(x, ids, w, w13[:, :31], s13, w2, s2, 32)),
        (ValueError, lambda: pd.moe_a16_i4(x, ids, w, w13, s13[:2], w2, s2, 32)),
        (ValueError, lambda: pd.moe_a16_i4(x, ids, w, w13, s13, w2[:, :63], s2, 32)),
        (ValueError, lambda: pd.moe_a16_i4(x, ids, w, w13, s13, w2, s2, 64)),
        (ValueError, lambda: pd.moe_a16_i4(x, ids, w, w13, s13, w2, s2, 32)),       # not on a GPU
    ]:
        with pytest.raises(error):
            call()


def test_a_single_row_or_expert_has_no_stride(monkeypatch):
    torch = pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    called = []
    monkeypatch.setattr(pd, "_mx_call", lambda fn, args, tensors, stream: called.append(args))
    far = 1 << 24

    def row(n, dtype):
        return torch.empty_strided((1, n), (far + 1, 1), dtype=dtype)

    pd.gemm_a16_i4(row(90, torch.float16), row(45, torch.uint8), row(1, torch.float32), 96, out=row(1, torch.float32))
    args = called.pop()      # (M, N, K, A, lda, type, B, ldb, s, lds, type, group, C, ldc, type)
    assert (args[4], args[7], args[9], args[13]) == (96, 96, 1, 1)
    codes = torch.empty_strided((1, 2, 45), (far + 1, 48, 1), dtype=torch.uint8)
    scales = torch.empty_strided((1, 1, 2), (far + 1, far + 1, 1))
    codes2 = torch.empty_strided((1, 90, 1), (far + 1, 16, 1), dtype=torch.uint8)
    scales2 = torch.empty_strided((1, 1, 90), (far + 1, far + 1, 1))
    pd.moe_a16_i4(row(90, torch.float16), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1), codes, scales, codes2, scales2, 96)
    args = called.pop()      # (T, H, I, E, top, x, ldx, type, ids, weights, w13, ld, expert, s13, ld, expert, w2, ...
    assert (args[6], args[11:13], args[14:16], args[17:19], args[20:22]) == (96, (96, 0), (2, 0), (32, 0), (90, 0))
