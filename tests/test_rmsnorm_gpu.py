"""GPU parity of the root-mean-square norm and its gradients with the 64-bit oracle.

Tolerances, in u = 2^-24 (half a step of binary32), for rows of at most 32768 values.  A
thread adds at most 32 squares one after another, then 6 exchanges of lanes and at most 15
additions of waves: the sum of squares is within 54 u, its square root's inverse within
27 u + 4 u (mean, eps, root, division), and y, three products later, within 40 u.  A
gradient's mean of g n is within 54 u + 40 u of the mean of magnitudes, so dx within 128 u of
r (|g| + |n| mean |g n|) + |dh|; a weight's gradient adds up to rows / blocks + 16 + parts / 16
+ 16 terms that are within 43 u each.  A result in 16 bits is half a unit more (2^-11, 2^-8).
INT8 codes are equal.
"""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import oracle.norm as rn
from tests import gpu_util as gu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_UNIT = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
HALF_TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
EPS = 1e-5


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_dense_gemm_amd as pd
    return pd


def values(rows, cols, seed, kind, scale=1.0):
    """(CPU tensor of the type, its values in 64 bits): rows and columns of unequal size."""
    rng = np.random.default_rng(seed)
    x = scale * rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-3, 4, (rows, 1))) * np.exp2(
        rng.integers(-2, 3, (1, cols)))
    t = torch.from_numpy(x).to(TYPES[kind])
    return t, t.double().numpy()


def weights(cols, seed, kind):
    t = torch.from_numpy(1.0 + 0.3 * np.random.default_rng(seed).standard_normal(cols)).to(TYPES[kind])
    return t, t.double().numpy()


def placed(t, pad=3, fill=float("nan")):
    """t on the GPU between NaN: rows `pad` elements apart, a row before and one after."""
    buf = torch.full((t.shape[0] + 2, t.shape[1] + pad), fill, dtype=t.dtype)
    buf[1:-1, :t.shape[1]] = t
    return buf.cuda()[1:-1, :t.shape[1]]


class Guarded:
    """An output among sentinel bytes, and the check that nothing beside it was written."""

    def __init__(self, rows, cols, dtype, pad=3):
        size = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full(((rows + 2) * (cols + pad) * size,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all = self.raw.view(dtype).view(rows + 2, cols + pad)
        self.view = self.all[1:-1, :cols]

    def check(self, what):
        left = self.all.clone()
        left[1:-1, :self.view.shape[1]] = 0
        want = torch.full_like(self.raw, 0xA5).view(self.all.dtype).view(self.all.shape)
        want[1:-1, :self.view.shape[1]] = 0
        assert torch.equal(left.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)), f"{what}: stores beside the result"


def assert_near(got, want, size, kind, what, units=40):
    got = got.cpu().double().numpy()
    tol = units * U * size
    tol = tol + (np.abs(want) + tol) * HALF_UNIT[kind] + HALF_TINY[kind]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


SHAPES = [(1, 1), (3, 7), (17, 64), (5, 65), (33, 127), (16, 128), (9, 129), (6, 512), (2, 513), (4, 1000), (3, 4096),
          (2, 8191), (1, 8193), (2, 16385), (1, 32768)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(pd, rows, cols, kind):
    for seed, (out_kind, w_kind, residual) in enumerate([("f32", "f32", True), (kind, kind, True), ("f16", "bf16", False),
                                                         ("bf16", "f16", True)]):
        what = f"norm {rows}x{cols} {kind} -> {out_kind}, weight {w_kind}, residual {residual}"
        gu.note(what)
        x, xv = values(rows, cols, seed, kind)
        w, wv = weights(cols, seed + 1, w_kind)
        out = Guarded(rows, cols, TYPES[out_kind])
        h = xv
        if residual:
            res, resv = values(rows, cols, seed + 2, kind)
            h = (torch.from_numpy(xv).float() + torch.from_numpy(resv).float()).to(TYPES[kind]).double().numpy()
            hs = Guarded(rows, cols, TYPES[kind], pad=5)
            y, hg = pd.rms_norm(placed(x), w.cuda(), EPS, residual=placed(res, 1), out=out.view, sum_out=hs.view)
            assert np.array_equal(hg.cpu().double().numpy(), h), what
            hs.check(what)
        else:
            y = pd.rms_norm(placed(x), w.cuda(), EPS, out=out.view)
        want = rn.forward(h, wv, EPS)
        assert_near(y, want, np.abs(want), out_kind, what)
        out.check(what)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_int8(pd, rows, cols, kind):
    for residual in (False, True):
        what = f"norm {rows}x{cols} {kind} -> int8, residual {residual}"
        gu.note(what)
        x, h = values(rows, cols, 11, kind)
        w, wv = weights(cols, 12, "f32" if residual else kind)
        q, scale = Guarded(rows, cols, torch.int8, pad=7), Guarded(1, rows, torch.float32)
        more = {}
        if residual:
            res, resv = values(rows, cols, 13, kind)
            h = (torch.from_numpy(h).float() + torch.from_numpy(resv).float()).to(TYPES[kind]).double().numpy()
            more = {"residual": placed(res)}
        got = pd.rms_norm_i8(placed(x), w.cuda(), EPS, out=(q.view, scale.view[0]), **more)
        want, s = rn.codes(h, wv, EPS)
        assert np.array_equal(got[0].cpu().numpy(), want.astype(np.int8)), what
        assert_near(got[1], s, s, "f32", what)
        q.check(what)
        scale.check(what)
        if residual:
            assert np.array_equal(got[2].cpu().double().numpy(), h), what


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES + [(0, 100), (600, 200), (1025, 8), (515, 1030)])
def test_gradients(pd, rows, cols, kind):
    for with_dh in (False, True):
        what = f"gradient {rows}x{cols} {kind}, dh {with_dh}"
        gu.note(what)
        hx, h = values(rows, cols, 21, kind)
        gx, g = values(rows, cols, 22, kind, 0.01)
        w, wv = weights(cols, 23, "f32" if with_dh else kind)
        dhx, dh = values(rows, cols, 24, kind, 0.01)
        dx = Guarded(rows, cols, TYPES[kind])
        dw = Guarded(1, cols, torch.float32)
        _, got = pd.rms_norm_backward(placed(gx), placed(hx, 1), w.cuda(), EPS, dh=placed(dhx) if with_dh else None,
                                      out=dx.view, dweight=dw.view[0])
        want, wdw, size, wsize = rn.backward(g, h, wv, EPS, dh if with_dh else None)
        assert_near(dx.view, want, size, kind, what, 128)
        assert_near(got, wdw, wsize, "f32", what, 43 + 2 * 16 + rows // 512 + 32)
        dx.check(what)
        dw.check(what)


def test_gradient_against_differences(pd):
    """Of the loss sum(y * dy), by central differences of the oracle's norm, whose own error at a step of 1e-5 of a
    value is some 1e-10 of the terms it adds."""
    rows, cols = 3, 9
    hx, h = values(rows, cols, 31, "f32")
    gx, g = values(rows, cols, 32, "f32")
    w, wv = weights(cols, 33, "f32")
    dx, dw = (t.cpu().double().numpy() for t in pd.rms_norm_backward(gx.cuda(), hx.cuda(), w.cuda(), EPS))
    _, _, size, wsize = rn.backward(g, h, wv, EPS)
    loss = lambda h, w: (rn.forward(h, w, EPS) * g).sum()  # noqa: E731
    terms = np.abs(rn.forward(h, wv, EPS) * g).sum()
    for i in range(rows):
        for j in range(cols):
            step = 1e-5 * np.sqrt(np.mean(h[i] ** 2))
            d = np.zeros_like(h)
            d[i, j] = step
            want = (loss(h + d, wv) - loss(h - d, wv)) / (2 * step)
            assert abs(dx[i, j] - want) <= 129 * U * size[i, j] + 1e-13 * terms / step
    for j in range(cols):
        d = np.zeros_like(wv)
        d[j] = 1e-5
        want = (loss(h, wv + d) - loss(h, wv - d)) / 2e-5
        assert abs(dw[j] - want) <= 76 * U * wsize[j] + 1e-8 * terms


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [40, 300, 700, 5000, 20000])
def test_rows_outside_the_range_of_squares(pd, kind, cols):
    """Squares that overflow or vanish in binary32, among ordinary rows."""
    for eps in (EPS, 0.0):
        x, _ = values(8, cols, 41, "f32")
        x = x.double()
        for row, factor in ((1, 2.0 ** 100), (2, 2.0 ** -100), (4, 2.0 ** 119), (5, 2.0 ** -70), (6, 2.0 ** 62)):
            x[row] *= factor
        x = x.to(TYPES[kind])
        h = x.double().numpy()
        w, wv = weights(cols, 42, "f32")
        want = rn.forward(h, wv, eps)
        what = f"{kind} {cols} eps {eps}"
        gu.note(what)
        assert_near(pd.rms_norm(x.cuda(), w.cuda(), eps, out_dtype=torch.float32), want, np.abs(want), "f32", what)
        q, scale = pd.rms_norm_i8(x.cuda(), w.cuda(), eps)
        fine = np.abs(h * wv).max(axis=1) < 2.0 ** 127          # (t itself within binary32)
        wq, ws = rn.codes(h, wv, eps)
        assert np.array_equal(q.cpu().numpy()[fine], wq.astype(np.int8)[fine]), what
        assert_near(scale[torch.from_numpy(fine)], ws[fine], ws[fine], "f32", what)
        g, gv = values(8, cols, 43, kind)
        dx, _ = pd.rms_norm_backward(g.cuda(), x.cuda(), w.cuda(), eps)
        wdx, _, size, _ = rn.backward(gv, h, wv, eps)
        # (a factor r below binary32's normal range has fewer bits: half a step of 2^-149 of it)
        size = size + (np.abs(gv * wv) + np.abs(h * rn.inverse(h, eps))) * 2.0 ** -149 / U
        top = np.abs(wdx) < float(torch.finfo(TYPES[kind]).max) / 2
        got = dx.cpu().double().numpy()
        tol = 128 * U * size
        tol += (np.abs(wdx) + tol) * HALF_UNIT[kind] + HALF_TINY[kind]
        assert (np.abs(got - wdx) <= tol)[top].all(), what


@pytest.mark.parametrize("rows,cols", [(5000, 300), (9000, 40), (3000, 200)])
def test_odd_rows_leave_the_others_bits(pd, rows, cols):
    """More rows than the groups of threads: rows outside the range of squares, each time beside others."""
    x, g, dh = (values(rows, cols, 60 + k, "f32")[0].cuda() for k in range(3))
    w = weights(cols, 63, "f32")[0].cuda()
    want, _ = pd.rms_norm_backward(g, x, w, EPS, dh=dh)
    odd = torch.zeros(rows, dtype=torch.bool)
    odd[::7], odd[rows // 2] = True, True
    x[odd] *= 2.0 ** 70
    h = x.cpu().double().numpy()
    got, _ = pd.rms_norm_backward(g, x, w, EPS, dh=dh)
    assert torch.equal(got[~odd], want[~odd])
    wdx, _, size, _ = rn.backward(g.cpu().double().numpy(), h, w.cpu().double().numpy(), EPS, dh.cpu().double().numpy())
    assert (np.abs(got.cpu().double().numpy() - wdx) <= 129 * U * size).all()
    x[odd] = float("nan")
    got, _ = pd.rms_norm_backward(g, x, w, EPS, dh=dh)
    assert torch.equal(got[~odd], want[~odd]) and got[odd].isnan().all()


@pytest.mark.parametrize("cols", [48, 500, 3000])
def test_rows_of_zeros_infinities_and_nan(pd, cols):
    x = torch.ones(6, cols)
    x[1] = 0.0
    x[2, cols // 2] = float("inf")
    x[3, 1] = float("nan")
    x[4, cols - 1] = -float("inf")
    w = torch.full((cols,), 0.5)
    w[0] = 2.0
    y = pd.rms_norm(x.cuda(), w.cuda(), EPS).cpu()
    want = torch.from_numpy(rn.forward(x.double().numpy(), w.double().numpy(), EPS))
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.allclose(y[ok].double(), want[ok], rtol=40 * U, atol=0)
    q, s = pd.rms_norm_i8(x.cuda(), w.cuda(), EPS)
    q, s = q.cpu(), s.cpu()
    assert torch.isnan(s[[2, 3, 4]]).all() and not q[[1, 2, 3, 4]].any() and s[1] == 0
    assert (q[[0, 5], 0] == 127).all() and (q[[0, 5], 1:] == 32).all()     # 0.5 * (127 / 2) = 31.75
    _, dw = pd.rms_norm_backward(torch.ones_like(x).cuda()[:2], x.cuda()[:2], w.cuda(), 0.0)
    assert dw.isnan().all()                  # (a row of zeros has no norm without eps)
    dx, dw = pd.rms_norm_backward(torch.ones_like(x).cuda()[:1], x.cuda()[:1], w.cuda(), 0.0)
    assert dx.isfinite().all() and dw.isfinite().all()


def test_in_place(pd):
    for cols in (100, 700, 9000, 20000, 32768):
        x, _ = values(5, cols, 51, "bf16")
        r, _ = values(5, cols, 52, "bf16")
        w, _ = weights(cols, 53, "bf16")
        y0, h0 = pd.rms_norm(x.cuda(), w.cuda(), EPS, residual=r.cuda())
        a, b = x.cuda(), r.cuda()
        y1, h1 = pd.rms_norm(a, w.cuda(), EPS, residual=b, out=a, sum_out=b)
        assert torch.equal(y1, y0) and torch.equal(h1, h0) and h1 is b and y1 is a
        dx0, dw0 = pd.rms_norm_backward(x.cuda(), h0, w.cuda(), EPS, dh=r.cuda())
        g = x.cuda()
        dx1, dw1 = pd.rms_norm_backward(g, h0, w.cuda(), EPS, dh=r.cuda(), out=g)
        assert torch.equal(dx1, dx0) and torch.equal(dw1, dw0)
        d = r.cuda()
        dx2, _ = pd.rms_norm_backward(x.cuda(), h0, w.cuda(), EPS, dh=d, out=d)
        assert torch.equal(dx2, dx0)


def test_codes_feed_the_int8_product(pd):
    """norm -> gemm_i8_dequant, as a layer runs them, for a K that is no multiple of 16."""
    rows, cols, n = 37, 1000, 200
    x, _ = values(rows, cols, 61, "bf16")
    r, _ = values(rows, cols, 62, "bf16")
    w, wv = weights(cols, 63, "bf16")
    rng = np.random.default_rng(64)
    b = rng.integers(-127, 128, (n, cols)).astype(np.int8)
    sb = rng.uniform(0.5, 2.0, n).astype(np.float32)
    bd = torch.zeros(n, 1008, dtype=torch.int8)
    bd[:, :cols] = torch.from_numpy(b)
    q, s, h = pd.rms_norm_i8(x.cuda(), w.cuda(), EPS, residual=r.cuda())
    c = pd.gemm_i8_dequant(q, bd.cuda()[:, :cols], s, torch.from_numpy(sb).cuda())
    hv = h.cpu().double().numpy()
    wq, ws = rn.codes(hv, wv, EPS)
    want = oracle.gemm_i8(wq.astype(np.int8), b).astype(np.float64) * ws[:, None] * sb[None, :]
    assert_near(c, want, np.abs(want), "f32", "norm and product", 44)


def test_streams_and_a_replayed_graph(pd):
    x, _ = values(40, 2000, 71, "bf16")
    r, _ = values(40, 2000, 72, "bf16")
    w, _ = weights(2000, 73, "bf16")
    x, r, w = x.cuda(), r.cuda(), w.cuda()
    want = pd.rms_norm_i8(x, w, EPS, residual=r)
    grads = pd.rms_norm_backward(x, r, w, EPS, dh=x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pd.rms_norm_i8(x, w, EPS, residual=r, stream=side)
    gg = pd.rms_norm_backward(x, r, w, EPS, dh=x, stream=side)
    side.synchronize()
    for a, b in zip(want + grads, got + gg):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pd.rms_norm_i8(x, w, EPS, residual=r)
        gg = pd.rms_norm_backward(x, r, w, EPS, dh=x)
    for turn in range(3):
        x.copy_(values(40, 2000, 80 + turn, "bf16")[0])
        graph.replay()
        torch.cuda.synchronize()
        want = pd.rms_norm_i8(x, w, EPS, residual=r) + pd.rms_norm_backward(x, r, w, EPS, dh=x)
        for a, b in zip(want, got + gg):
            assert torch.equal(a, b), turn
