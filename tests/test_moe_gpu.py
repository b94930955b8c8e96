"""GPU parity of the expert layer and its routing with the 64-bit oracle.

Tolerance of the layer.  The first product's sums are within (512 + H / 12) * 2^-22 of the sum of
|x| |scale| (as in the products' own tests), which silu(g) * u carries on with slopes of 1.1 |u| and
|silu(g)|.  silu's exponential takes its argument in binary32: a relative 2^-16 covers |g| < 128 and the
few roundings after it.  The gated activation is rounded to 16 bits: half a unit of it (2^-11,
2^-8), or half the type's smallest subnormal.  The second product sums over all experts that have a token:
(512 + experts * I / 12) * 2^-22 of the sum of |activation| |scale|.  y is rounded once more.
"""
from __future__ import annotations

import numpy as np
import pytest

import oracle.int4 as i4
import oracle.norm as rn
from tests import gpu_util as gu
from tests.test_a16_i4_gpu import HALF_TINY, HALF_UNIT, TYPES, held, placed, placed_activations

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_dense_gemm_amd as pd
    return pd


def expert_weights(E, N, K, group, seed, kind):
    """(codes on the GPU (E, N, ceil(K/2)) among 0x77, scales (E, groups, N) among NaN, the lists of dense values
    and of their scales' magnitudes)."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(-8, 8, (E, N, K))
    width = (K + 1) // 2
    packed = i4.pack(codes)
    if K % 2:
        packed[..., -1] |= 0x70
    buf = torch.full((E + 1, N + 1, gu.round_up(width, 16) + 16), 0x77, dtype=torch.uint8)
    buf[:E, :N, :width] = torch.from_numpy(packed)
    groups = -(-K // group)
    scales, sv = held(np.exp2(rng.uniform(-2, 1, (E, groups, N))) / np.sqrt(K), kind)
    sb = torch.full((E + 1, groups + 1, N + 3), float("nan"), dtype=scales.dtype)
    sb[:E, :groups, :N] = scales
    dense = [i4.values(codes[e], sv[e], group) for e in range(E)]
    size = [np.abs(i4.values(np.ones_like(codes[e]), sv[e], group)) for e in range(E)]
    return buf.cuda()[:E, :N, :width], sb.cuda()[:E, :groups, :N], (dense, size)


def layer(T, H, I, E, group, seed, kind, s_kind):
    rng = np.random.default_rng(seed)
    x, xv = held(rng.standard_normal((T, H)), kind)
    w13, s13, d13 = expert_weights(E, 2 * I, H, group, seed + 1, s_kind)
    w2, s2, d2 = expert_weights(E, H, I, group, seed + 2, s_kind)
    return placed_activations(x), xv, (w13, s13, w2, s2), d13, d2


def check_layer(got, edge, xv, ids, weights, first, second, kind, what):
    """got: the output's buffer with `edge` sentinel rows and columns around y."""
    T, H = xv.shape
    (d13, m13), (d2, m2) = first, second
    I = d2[0].shape[1]
    R, size, act_size, second, mass = i4.experts(xv, ids, weights, d13, d2, m13, m2)
    full = got.cpu().double().numpy()
    y = full[1:-1, :H] if edge else full
    if edge:
        rim = np.ones(full.shape, bool)
        rim[1:-1, :H] = False
        assert (full[rim] == float(torch.tensor(-777.0, dtype=TYPES[kind]))).all(), f"{what}: stores beside the result"
    live = len({e for row in ids for e in row if 0 <= e < len(d2)})
    tol = act_size * (512 + H / 12) * 2.0 ** -22 + mass * HALF_TINY[kind]
    tol += (size + tol) * (HALF_UNIT[kind] + 2.0 ** -16) + (second + tol) * (512 + live * I / 12) * 2.0 ** -22
    tol += (np.abs(R) + tol) * HALF_UNIT[kind] + HALF_TINY[kind]
    bad = ~(np.abs(y - R) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {np.argwhere(bad)[0]}: {y[bad][0]} for {R[bad][0]}"


def run_layer(pd, T, H, I, E, top, group, kind, s_kind, seed=0, ids=None):
    what = f"T {T} H {H} I {I} E {E} top {top} group {group} {kind} scales {s_kind}"
    gu.note(what)
    x, xv, w, d13, d2 = layer(T, H, I, E, group, seed, kind, s_kind)
    rng = np.random.default_rng(seed + 5)
    if ids is None:
        ids = np.stack([rng.permutation(E)[:top] for _ in range(T)])
    weights = rng.uniform(0.05, 1.0, (T, top)).astype(np.float32)
    buf = torch.full((T + 2, H + 3), -777.0, dtype=TYPES[kind], device="cuda")
    pd.moe_a16_i4(x, torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(weights).cuda(), *w, group, out=buf[1:-1, :H])
    check_layer(buf, True, xv, ids, weights.astype(np.float64), d13, d2, kind, what)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,I,E,top,group", [
    (1, 1, 1, 1, 1, 32), (1, 256, 128, 4, 2, 128), (2, 100, 33, 3, 3, 32), (5, 333, 129, 7, 2, 64), (16, 512, 257, 33, 4, 64),
    (17, 200, 300, 5, 5, 96), (32, 128, 640, 40, 3, 128), (33, 130, 65, 6, 2, 32), (64, 64, 100, 3, 1, 32), (70, 96, 40, 9, 3, 64),
    (130, 40, 64, 2, 2, 32), (3, 512, 1100, 4, 1, 256), (40, 64, 32, 200, 8, 32), (1, 64, 2200, 40, 8, 64)])
def test_layer(pd, T, H, I, E, top, group, kind):
    for n, s_kind in enumerate(("f32", kind)):
        run_layer(pd, T, H, I, E, top, group, kind, s_kind, seed=100 * n + T)


def test_many_experts_of_many_tokens(pd):
    """More active experts than the largest tile's table holds, and ids at the end of the range."""
    rng = np.random.default_rng(3)
    ids = np.stack([rng.permutation(1024)[:16] for _ in range(60)])
    ids[0, :2] = 1023, 0
    run_layer(pd, 60, 32, 16, 1024, 16, 32, "f16", "f16", ids=ids)


def test_ids_that_name_no_expert_or_one_twice(pd):
    ids = np.array([[0, -1, 2], [-1, -1, -1], [1, 1, 1], [2, 5, 2], [6, 1 << 30, -(1 << 31)], [4, 4, 3], [3, 0, 3]])
    run_layer(pd, 7, 200, 100, 6, 3, 64, "bf16", "f32", ids=ids)
    none = np.full((20, 2), -1)
    run_layer(pd, 20, 64, 64, 4, 2, 32, "f16", "f16", ids=none)
    run_layer(pd, 50, 64, 64, 4, 4, 32, "f16", "f16", ids=np.full((50, 4), 3))      # all pairs on one expert


def test_broken_expert_stays_with_its_tokens(pd):
    x, xv, w, d13, d2 = layer(20, 160, 96, 4, 32, 9, "bf16", "f32")
    w13, s13, w2, s2 = w
    s2[1, 0, 5] = float("inf")
    s2[1, 2, 7] = float("nan")
    s13[2, 1, 11] = float("nan")
    ids = np.random.default_rng(4).integers(0, 4, (20, 1))
    weights = np.ones((20, 1), np.float32)
    y = pd.moe_a16_i4(x, torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(weights).cuda(), *w, 32).cpu()
    for t, e in enumerate(ids[:, 0]):
        if e == 2:
            assert torch.isnan(y[t]).all()
        else:
            bad = {5, 7} if e == 1 else set()
            assert {int(j) for j in torch.nonzero(~torch.isfinite(y[t]))[:, 0]} == bad, (t, e)


def test_bad_token_stays_alone(pd):
    x, xv, w, d13, d2 = layer(20, 160, 96, 4, 32, 9, "f16", "f32")
    x[3, 4], x[8, 159] = float("nan"), float("inf")
    ids = torch.randint(0, 4, (20, 2), dtype=torch.int32, device="cuda")
    y = pd.moe_a16_i4(x, ids, torch.ones(20, 2, device="cuda"), *w, 32).cpu()
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[8]).any()
    keep = [t for t in range(20) if t not in (3, 8)]
    assert torch.isfinite(y[keep]).all()


def test_bad_tokens_leave_the_others_bits(pd):
    """Thirty tokens of one expert, in whatever order they reach its tiles: with some of them not finite, the
    others' results keep their bits."""
    x, xv, w, d13, d2 = layer(30, 300, 96, 2, 32, 9, "bf16", "f32")
    ids, ones = torch.zeros(30, 1, dtype=torch.int32, device="cuda"), torch.ones(30, 1, device="cuda")
    want = pd.moe_a16_i4(x, ids, ones, *w, 32).cpu()
    x[4, 7], x[13, 280], x[21, 0] = float("nan"), float("-inf"), 3e38
    keep = [t for t in range(30) if t not in (4, 13, 21)]
    for _ in range(5):
        assert torch.equal(pd.moe_a16_i4(x, ids, ones, *w, 32).cpu()[keep], want[keep])


@pytest.mark.parametrize("T,E,top", [(4096, 3, 1), (512, 20, 8), (64, 1024, 64)])
def test_most_pairs(pd, T, E, top):
    run_layer(pd, T, 32, 16, E, top, 32, "f16", "f16")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (3, 7, 7), (5, 64, 8), (9, 65, 4), (4, 128, 64), (6, 200, 16), (2, 257, 3), (7, 1024, 64)])
def test_route(pd, T, E, top, kind):
    rng = np.random.default_rng(T * E + top)
    logits, lv = held(np.round(rng.standard_normal((T, E)) * 4) / 4, kind)      # many ties
    if T > 2:
        lv[1, rng.permutation(E)[:E // 2 + 1]] = -np.inf
        lv[2, :] = -np.inf
        logits = torch.from_numpy(lv).to(TYPES[kind])
    for normalize in (True, False):
        what = f"route T {T} E {E} top {top} {kind} normalize {normalize}"
        gu.note(what)
        out = (torch.full((T + 1, top), 77, dtype=torch.int32, device="cuda"), torch.full((T + 1, top), 77.0, device="cuda"))
        pd.moe_route(placed(logits, 5, float("nan")), top, normalize, out=(out[0][:T], out[1][:T]))
        ids, weights = i4.route(lv, top)
        if not normalize:
            with np.errstate(invalid="ignore"):
                p = np.exp(lv - lv.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
            weights = np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), axis=1), 0.0)
        assert np.array_equal(out[0][:T].cpu().numpy(), ids), what
        # an exponential of a difference below 64 (2^-18 of its argument's rounding), and sums of up to 1024 in order
        assert np.allclose(out[1][:T].cpu().double().numpy(), weights, rtol=2.0 ** -17, atol=2.0 ** -126), what
        assert (out[0][T] == 77).all() and (out[1][T] == 77).all(), what


def test_route_of_nan_and_infinity(pd):
    x = torch.zeros(4, 10)
    x[0, 6], x[1, 3], x[1, 5] = float("nan"), float("inf"), 2.0
    x[2, 9], x[2, 4] = float("nan"), float("nan")
    ids, weights = pd.moe_route(x.cuda(), 3)
    want, _ = i4.route(x.double().numpy(), 3)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert torch.isnan(weights[:3]).all() and torch.allclose(weights[3].cpu(), torch.full((3,), 1 / 3))


def test_norm_route_and_experts_together(pd):
    """A decoder layer's feed-forward half, as a program runs it: the norm with the residual, the router's product, the
    choice, the experts; then the shared expert's product on the same norm.  Checked step by step."""
    T, H, I, E, top, group = 9, 256, 160, 12, 3, 64
    rng = np.random.default_rng(8)
    x, _ = held(rng.standard_normal((T, H)), "f16")
    res, _ = held(rng.standard_normal((T, H)), "f16")
    wn, wv = held(1 + 0.1 * rng.standard_normal(H), "f16")
    router, rv = held(0.2 * rng.standard_normal((E, H)), "f16")
    _, _, w, d13, d2 = layer(T, H, I, E, group, 20, "f16", "f16")
    ws = torch.empty(pd.moe_a16_i4_workspace_size(T, H, I, E, top), dtype=torch.uint8, device="cuda")
    y, h = pd.rms_norm(x.cuda(), wn.cuda(), 1e-5, residual=res.cuda())
    logits = pd.gemm_f16(y, router.cuda())
    ids, weights = pd.moe_route(logits, top)
    out = pd.moe_a16_i4(y, ids, weights, *w, group, workspace=ws)
    shared = pd.gemm_a16_i4(y, w[0][0], w[1][0], group)
    hv = (x.float() + res.float()).half().double().numpy()
    assert np.array_equal(h.cpu().double().numpy(), hv)
    want = rn.forward(hv, wv, 1e-5)
    assert np.allclose(y.cpu().double().numpy(), want, rtol=2.0 ** -11 + 2.0 ** -18, atol=2.0 ** -25)
    yv = y.cpu().double().numpy()
    assert np.all(np.abs(logits.cpu().double().numpy() - yv @ rv.T) <= 1e-3 * (np.abs(yv) @ np.abs(rv).T))
    wi, ww = i4.route(logits.cpu().double().numpy(), top)
    assert np.array_equal(ids.cpu().numpy(), wi) and np.allclose(weights.cpu().numpy(), ww, rtol=2.0 ** -17)
    check_layer(out, False, yv, wi, weights.cpu().double().numpy(), d13, d2, "f16", "together")
    R, A = i4.product(yv, d13[0][0])[0], np.abs(yv) @ d13[1][0].T
    assert (np.abs(shared.cpu().double().numpy() - R) <= (512 + H / 12) * 2.0 ** -22 * A).all()


def test_same_bits_again_on_streams_and_in_replayed_graphs(pd):
    T, H, I, E, top = 20, 256, 200, 16, 4
    x, _, w, _, _ = layer(T, H, I, E, 64, 30, "bf16", "f32")
    logits = torch.randn(T, E, device="cuda")

    def step(stream=None, ws=None):
        ids, weights = pd.moe_route(logits, top, stream=stream)
        return ids, weights, pd.moe_a16_i4(x, ids, weights, *w, 64, workspace=ws, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    size = pd.moe_a16_i4_workspace_size(T, H, I, E, top)
    ws = [torch.full((size,), 0xEE, dtype=torch.uint8, device="cuda") for _ in range(2)]
    graphs = []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step(ws=ws[k])))
    for turn in range(3):
        logits.normal_()
        x.copy_(torch.randn(T, H, device="cuda"))
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = step()
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(want, got)), turn
