"""GPU parity of the MXFP4 entry points against the 64-bit oracle: codes and scales bit for
bit, values exactly, products within the rounding of binary32 sums.

Every buffer is wider than the operand and holds poison outside it (NaN, 0x77 codes, 0xFF
scales), every output sits among sentinels, and each case prints its name before it touches
the GPU.

Tolerance of a product: each matrix instruction adds at least 32 products to a binary32
sum; its result is taken to be within four half units (2^-22) of the magnitudes it adds, so
a sum of K products is within ceil(K / 64) * 2^-22 of the sum of magnitudes (steps of 32
values: ceil(K / 32) half of that each for the a16 product, whose partial sums are scaled
exactly).  Rounding to a 16-bit type adds half a unit of the result (2^-11, 2^-8), or half
its smallest subnormal.
"""
from __future__ import annotations

import numpy as np
import pytest

import oracle.mxfp4 as mx
from tests import gpu_util as gu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_UNIT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
HALF_TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
SENTINEL = 0xA5


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_dense_gemm_amd as pd
    return pd


@pytest.fixture(scope="module")
def dev(pd):
    return torch.device("cuda:0")


def to_type(x, kind):
    """float64 host values -> (CPU tensor of the type, the float64 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[kind])
    return t, t.double().numpy()


def source(t, dev, pad=5, fill=float("nan")):
    """t on the GPU with rows `pad` elements apart that hold `fill`, and rows after the last."""
    buf = torch.full((t.shape[0] + 2, t.shape[1] + pad), fill, dtype=t.dtype)
    buf[:t.shape[0], :t.shape[1]] = t
    return buf.to(dev)[:t.shape[0], :t.shape[1]]


def blank_operand(rows, K, dev):
    """(codes, scales) views into sentinel-filled buffers, and the buffers."""
    nb = mx.blocks_of(K)
    cb = torch.full((rows + 2, 16 * nb + 32), SENTINEL, dtype=torch.uint8, device=dev)
    sb = torch.full((nb + 2, gu.round_up(rows, 16) + 16), SENTINEL, dtype=torch.uint8, device=dev)
    return (cb[:rows, :(K + 1) // 2], sb[:nb, :rows]), (cb, sb)


def check_operand(buffers, rows, K, want, what):
    """The written operand equals the oracle's, and nothing else was written."""
    cb, sb = (b.cpu().numpy() for b in buffers)
    codes, scales = want
    wc, ws = np.full_like(cb, SENTINEL), np.full_like(sb, SENTINEL)
    wc[:rows, :codes.shape[1]], ws[:scales.shape[0], :rows] = codes, scales
    assert np.array_equal(sb, ws), f"{what}: scales differ at {np.argwhere(sb != ws)[:5].tolist()}"
    assert np.array_equal(cb, wc), f"{what}: codes differ at {np.argwhere(cb != wc)[:5].tolist()}"


def stored(codes, scales, K, dev):
    """An oracle operand on the GPU among poison: codes of 0x77 after the last value's byte
    and in the high nibble of an odd K, scales of 0xFF after the last row and block."""
    rows, nb = codes.shape[0], scales.shape[0]
    cb = np.full((rows + 1, gu.round_up(16 * nb, 16) + 32), 0x77, np.uint8)
    cb[:rows, :(K + 1) // 2] = codes[:, :(K + 1) // 2]
    if K % 2:
        cb[:rows, K // 2] = (cb[:rows, K // 2] & 0x0F) | 0x70
    sb = np.full((nb + 1, gu.round_up(rows, 16) + 16), 0xFF, np.uint8)
    sb[:nb, :rows] = scales
    c, s = torch.from_numpy(cb).to(dev), torch.from_numpy(sb).to(dev)
    return c[:rows, :(K + 1) // 2], s[:nb, :rows]


def random_operand(rows, K, seed, lo=120, hi=134):
    """Random codes and scales (bytes lo .. hi), as the oracle's arrays."""
    rng = np.random.default_rng(seed)
    nb = mx.blocks_of(K)
    return (rng.integers(0, 256, (rows, 16 * nb), dtype=np.uint8),
            rng.integers(lo, hi + 1, (nb, rows), dtype=np.uint8))


def spread(rows, K, seed):
    """Values of many magnitudes: normal, times a power of two of the row and of the column."""
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((rows, K)) * np.exp2(rng.integers(-6, 7, (rows, 1)))
            * np.exp2(rng.integers(-4, 5, (1, K))))


def assert_close(C, R, S, steps, kind, what):
    """C (a GPU tensor of the kind) against the 64-bit product R and the sum of magnitudes S."""
    got = C.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(R)), f"{what}: NaN where there is none, or none where one is"
    top = float(torch.finfo(TYPES[kind]).max)
    tol = steps * 2.0 ** -22 * S
    tol = tol + (np.abs(R) + tol) * HALF_UNIT[kind] + HALF_TINY[kind]
    with np.errstate(invalid="ignore"):
        clear = np.abs(R) + tol < top                # far enough from the type's overflow
        over = np.abs(R) - tol > top * (1 + 2 * HALF_UNIT[kind] + 2.0 ** -23)
        bad = clear & ~(np.abs(got - R) <= tol)
        bad |= over & (got != np.sign(R) * np.inf)
    assert not bad.any(), (f"{what}: {int(bad.sum())} off, first {tuple(np.argwhere(bad)[0])}: got "
                           f"{got[tuple(np.argwhere(bad)[0])]} want {R[tuple(np.argwhere(bad)[0])]}")


# ---- quantising ----

QSHAPES = [(1, 1), (1, 31), (1, 33), (3, 4096), (17, 515), (64, 256), (65, 130), (257, 127), (300, 1029), (513, 64)]


@pytest.mark.parametrize("form", ["rows", "transpose", "both"])
@pytest.mark.parametrize("rule", ["floor", "fit"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", QSHAPES, ids=[f"{r}x{k}" for r, k in QSHAPES])
def test_quantize(pd, dev, shape, kind, rule, form):
    rows, K = shape
    gu.note(f"[case] quantize {rows}x{K} {kind} {rule} {form}")
    t, x = to_type(spread(rows, K, 100 + rows + K), kind)
    x_dev = source(t, dev)
    out, bufs = blank_operand(rows, K, dev)
    out_t, bufs_t = blank_operand(K, rows, dev)
    if form == "rows":
        pd.mxf4_quantize(x_dev, scale_rule=rule, out=out)
    elif form == "transpose":
        pd.mxf4_quantize(x_dev, transpose=True, scale_rule=rule, out=out_t)
    else:
        pd.mxf4_quantize_both(x_dev, scale_rule=rule, out=(out, out_t))
    torch.cuda.synchronize()
    if form != "transpose":
        check_operand(bufs, rows, K, mx.quantize(x, rule), "rows")
    if form != "rows":
        check_operand(bufs_t, K, rows, mx.quantize(x.T, rule), "transpose")


def special_rows(kind):
    """Rows of one block: its first value sets the scale, the other 31 run over every value of
    the 16-bit types that is not larger (fp32: ties and their neighbours at many scales)."""
    rng = np.random.default_rng(3)
    if kind == "f32":
        tops = [np.ldexp(m, e) for e in (-149, -140, -127, -126, -125, -124, -20, 0, 1, 60, 125, 127)
                for m in (1.0, 1.25, 1.5, 1.5 + 2.0 ** -23, 1.75, 2 - 2.0 ** -23)]
        tops = np.array(tops, np.float32)
        rows = []
        for top in tops[(tops > 0) & np.isfinite(tops)]:
            f = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6], np.float64) / 8
            e = np.floor(np.log2(float(top)))
            v = np.ldexp(f * 2, int(e)).astype(np.float32)
            v = np.concatenate([v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(0))])
            v = np.minimum(v, top)[:31]
            rows.append(np.concatenate([[top], v, np.zeros(31 - len(v), np.float32)]) * rng.choice([-1, 1], 32))
        return torch.from_numpy(np.array(rows, np.float32))
    bits = np.arange(0, 0x7C00 if kind == "f16" else 0x7F80, dtype=np.uint16)
    every = torch.from_numpy(bits.view(np.int16)).view(TYPES[kind])
    vals = every.double().numpy()
    rows = []
    for top in vals[len(vals) % 31::977]:
        if top == 0:
            continue
        below = vals[vals <= top][-31 * 40:]
        below = below[:len(below) // 31 * 31].reshape(-1, 31)
        rows.append(np.hstack([np.full((len(below), 1), top), below]))
    rows = np.vstack(rows) if rows else np.zeros((0, 32))
    rows = rows * np.where(np.random.default_rng(4).random(rows.shape) < 0.5, -1, 1)
    return torch.from_numpy(rows).to(TYPES[kind])


@pytest.mark.parametrize("rule", ["floor", "fit"])
@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_values(pd, dev, kind, rule):
    t = special_rows(kind)
    gu.note(f"[case] quantize values {kind} {rule} {tuple(t.shape)}")
    want = mx.quantize(t.double().numpy(), rule)
    q, s = pd.mxf4_quantize(t.to(dev), scale_rule=rule)
    qt, st = pd.mxf4_quantize(t.t().contiguous().to(dev), transpose=True, scale_rule=rule)
    (b, sb), (bt, sbt) = pd.mxf4_quantize_both(torch.cat([t, t], 1).contiguous().to(dev), scale_rule=rule)
    torch.cuda.synchronize()
    for name, codes, scales in (("rows", q, s), ("transpose", qt, st)):
        assert np.array_equal(scales.cpu().numpy(), want[1]), name
        assert np.array_equal(codes.cpu().numpy(), want[0]), name
    assert np.array_equal(b.cpu().numpy(), np.hstack([want[0], want[0]]))
    assert np.array_equal(sb.cpu().numpy(), np.vstack([want[1], want[1]]))
    again = mx.quantize(torch.cat([t, t], 1).double().numpy().T, rule)
    assert np.array_equal(bt.cpu().numpy(), again[0][:, :bt.shape[1]]) and np.array_equal(sbt.cpu().numpy(), again[1])


@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_special_blocks(pd, dev, kind):
    gu.note(f"[case] quantize special blocks {kind}")
    x = spread(40, 100, 9)
    x[0, 5], x[1, 40], x[2, 99], x[39, 70] = np.nan, np.inf, -np.inf, np.nan
    x[3, :], x[4:, 64:96] = 0.0, -0.0
    t, x = to_type(x, kind)
    (q, s), (qt, st) = pd.mxf4_quantize_both(t.to(dev))
    q1, s1 = pd.mxf4_quantize(t.to(dev))
    torch.cuda.synchronize()
    want, want_t = mx.quantize(x), mx.quantize(x.T)
    for got, ref in (((q, s), want), ((q1, s1), want), ((qt, st), want_t)):
        assert np.array_equal(got[1].cpu().numpy(), ref[1])
        assert np.array_equal(got[0].cpu().numpy(), ref[0][:, :got[0].shape[1]])
    v = pd.mxf4_dequantize(q, s, 100).cpu().double().numpy()
    assert np.array_equal(v, mx.values(*want, 100), equal_nan=True)


# ---- reading back ----

@pytest.mark.parametrize("kind", list(TYPES))
def test_dequantize_every_code_and_scale(pd, dev, kind):
    gu.note(f"[case] dequantize every code and scale {kind}")
    codes = np.tile(np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2, np.uint8), (256, 1))
    scales = np.arange(256, dtype=np.uint8)[None, :]
    out = pd.mxf4_dequantize(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), out_dtype=TYPES[kind])
    want = torch.from_numpy(mx.values(codes, scales, 32))
    want = want.float().to(TYPES[kind])              # exact in binary32 (or infinite), then rounded once
    got = out.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(torch.where(nan, torch.zeros_like(got), got), torch.where(nan, torch.zeros_like(want), want))
    assert torch.equal(torch.signbit(got)[~nan], torch.signbit(want)[~nan])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", QSHAPES, ids=[f"{r}x{k}" for r, k in QSHAPES])
def test_dequantize_shapes(pd, dev, shape, kind):
    rows, K = shape
    gu.note(f"[case] dequantize {rows}x{K} {kind}")
    codes, scales = random_operand(rows, K, rows + K)
    buf = torch.full((rows + 2, K + 3), 7.0, dtype=TYPES[kind], device=dev)
    pd.mxf4_dequantize(*stored(codes, scales, K, dev), K, out=buf[:rows, :K])
    want = torch.full((rows + 2, K + 3), 7.0, dtype=torch.float64)
    want[:rows, :K] = torch.from_numpy(mx.values(codes, scales, K))
    assert torch.equal(buf.cpu().double(), want)     # few significant bits: exact in every type


# ---- products ----

PSHAPES = [(1, 1, 1), (1, 33, 31), (2, 3, 32), (5, 17, 33), (16, 32, 64), (17, 31, 255), (33, 65, 256), (64, 64, 257),
           (65, 63, 513), (100, 130, 1000), (127, 257, 640), (129, 128, 384), (255, 300, 1030), (520, 260, 2049),
           (1, 600, 8192), (31, 100, 8191)]


def operands(M, N, K, seed, lo=120, hi=134):
    a, b = random_operand(M, K, seed, lo, hi), random_operand(N, K, seed + 1, lo, hi)
    R, S = mx.product(mx.values(*a, K), mx.values(*b, K))
    return a, b, R, S


def guarded(M, N, kind, dev):
    """An output of odd row stride among sentinels."""
    buf = torch.full((M + 2, N + 3), 7.0, dtype=TYPES[kind], device=dev)
    return buf, buf[:M, :N]


def check_rest(buf, M, N):
    rest = buf.clone()
    rest[:M, :N] = 7.0
    assert bool((rest == 7.0).all()), "stores outside the M x N block"


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", PSHAPES, ids=[f"{m}x{n}x{k}" for m, n, k in PSHAPES])
def test_product(pd, dev, shape, kind):
    M, N, K = shape
    gu.note(f"[case] gemm_mxf4 {M}x{N}x{K} {kind}")
    a, b, R, S = operands(M, N, K, 1000 + M + 3 * N + K)
    buf, out = guarded(M, N, kind, dev)
    pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K, out=out)
    torch.cuda.synchronize()
    check_rest(buf, M, N)
    assert_close(out, R, S, -(-K // 64), kind, f"{shape} {kind}")


TILE_SHAPES = [(1, 1, 1), (33, 65, 256), (65, 63, 513), (255, 257, 1030), (260, 130, 640), (520, 260, 2049),
               (300, 520, 8191), (129, 300, 300)]


@pytest.mark.parametrize("cfg", range(10))
@pytest.mark.parametrize("shape", TILE_SHAPES, ids=[f"{m}x{n}x{k}" for m, n, k in TILE_SHAPES])
def test_product_every_tile(pd, dev, shape, cfg):
    M, N, K = shape
    kind = list(TYPES)[(M + cfg) % 3]
    gu.note(f"[case] gemm_mxf4 {M}x{N}x{K} cfg={cfg} {kind}")
    a, b, R, S = operands(M, N, K, 4000 + M + N + K, 110, 140)
    buf, out = guarded(M, N, kind, dev)
    pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K, out=out, cfg=cfg)
    torch.cuda.synchronize()
    check_rest(buf, M, N)
    assert_close(out, R, S, -(-K // 64), kind, f"{shape} cfg {cfg} {kind}")


@pytest.mark.parametrize("bits", [(127, 127), (100, 150), (64, 190), (1, 253)])
@pytest.mark.parametrize("shape", [(5, 40, 300), (150, 140, 700)], ids=["5x40x300", "150x140x700"])
def test_product_wide_scales(pd, dev, shape, bits):
    M, N, K = shape
    gu.note(f"[case] gemm_mxf4 scales {bits} {shape}")
    a, b, R, S = operands(M, N, K, 77, *bits)
    C = pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K)
    if bits == (1, 253):
        # sums that leave binary32's range on the way may end infinite or NaN: those whose
        # magnitudes stay inside have to be right
        got = C.cpu().double().numpy()
        inside = S < 2.0 ** 126
        tol = -(-K // 64) * 2.0 ** -22 * S + K * 2.0 ** -149
        assert (np.abs(got - R)[inside] <= tol[inside]).all()
    else:
        assert_close(C, R, S, -(-K // 64), "f32", f"{shape} {bits}")


@pytest.mark.parametrize("shape", [(3, 50, 100), (200, 150, 600)], ids=["3x50x100", "200x150x600"])
def test_product_nan_scales(pd, dev, shape):
    M, N, K = shape
    gu.note(f"[case] gemm_mxf4 NaN scales {shape}")
    a, b, _, _ = operands(M, N, K, 5)
    a[1][0, 1] = a[1][-1, M - 1] = 255          # first and last (short) block
    a[0][M - 1, :] = 0                          # a NaN scale over zero codes is NaN too
    b[1][1, 7] = 255
    R, S = mx.product(mx.values(*a, K), mx.values(*b, K))
    assert_close(pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K), R, S, -(-K // 64), "f32", "NaN scales")


def test_product_overflow_of_16_bit_outputs(pd, dev):
    gu.note("[case] gemm_mxf4 overflow")
    M, N, K = 40, 50, 128
    codes = np.full((M, 64), 0x77, np.uint8)
    a = (codes, np.full((4, M), 140, np.uint8))
    b = (np.full((N, 64), 0xF7, np.uint8), np.full((4, N), 130, np.uint8))
    b[0][:, :] = 0x77
    R, S = mx.product(mx.values(*a, K), mx.values(*b, K))
    assert R.min() > 65504
    for kind in TYPES:
        assert_close(pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K, out_dtype=TYPES[kind]), R, S, 2, kind, kind)


@pytest.mark.parametrize("kind", list(TYPES))
def test_product_empty(pd, dev, kind):
    gu.note(f"[case] gemm_mxf4 empty {kind}")
    u = lambda r, c: torch.zeros((r, c), dtype=torch.uint8, device=dev)  # noqa: E731
    for M, N in ((3, 5), (300, 70)):
        buf, out = guarded(M, N, kind, dev)
        pd.gemm_mxf4(u(M, 0), u(0, M), u(N, 0), u(0, N), 0, out=out)
        check_rest(buf, M, N)
        assert not bool(out.any())
        pd.gemm_a16_mxf4(torch.zeros((M, 0), dtype=torch.float16, device=dev), u(N, 0), u(0, N), out=out.fill_(3))
        assert not bool(out.any())
    assert pd.gemm_mxf4(u(0, 16), u(1, 0), u(5, 16), u(1, 5), 32).shape == (0, 5)
    assert pd.mxf4_quantize(torch.zeros((0, 40), device=dev))[0].shape == (0, 20)
    assert pd.mxf4_dequantize(u(4, 0), u(0, 4)).shape == (4, 0)


@pytest.mark.parametrize("a_kind", ["f16", "bf16"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", PSHAPES, ids=[f"{m}x{n}x{k}" for m, n, k in PSHAPES])
def test_a16(pd, dev, shape, kind, a_kind):
    M, N, K = shape
    gu.note(f"[case] gemm_a16_mxf4 {M}x{N}x{K} {a_kind} {kind}")
    t, x = to_type(spread(M, K, 2000 + M + K), a_kind)
    b = random_operand(N, K, 3000 + N + K)
    R, S = mx.product(x, mx.values(*b, K))
    buf, out = guarded(M, N, kind, dev)
    pd.gemm_a16_mxf4(source(t, dev, gu.round_up(K, 8) - K + 8), *stored(*b, K, dev), out=out)
    torch.cuda.synchronize()
    check_rest(buf, M, N)
    assert_close(out, R, S, -(-K // 64) + 1, kind, f"{shape} {a_kind} {kind}")


@pytest.mark.parametrize("a_kind", ["f16", "bf16"])
@pytest.mark.parametrize("cfg", range(13))
@pytest.mark.parametrize("shape", TILE_SHAPES, ids=[f"{m}x{n}x{k}" for m, n, k in TILE_SHAPES])
def test_a16_every_tile(pd, dev, shape, cfg, a_kind):
    M, N, K = shape
    kind = list(TYPES)[(N + cfg) % 3]
    gu.note(f"[case] gemm_a16_mxf4 {M}x{N}x{K} cfg={cfg} {a_kind} {kind}")
    t, x = to_type(spread(M, K, 5000 + M + K), a_kind)
    b = random_operand(N, K, 6000 + N + K, 110, 140)
    R, S = mx.product(x, mx.values(*b, K))
    buf, out = guarded(M, N, kind, dev)
    pd.gemm_a16_mxf4(source(t, dev, gu.round_up(K, 8) - K + 8), *stored(*b, K, dev), out=out, cfg=cfg)
    torch.cuda.synchronize()
    check_rest(buf, M, N)
    assert_close(out, R, S, -(-K // 64) + 1, kind, f"{shape} cfg {cfg} {a_kind} {kind}")


@pytest.mark.parametrize("a_kind", ["f16", "bf16"])
@pytest.mark.parametrize("M", [5, 150])
def test_a16_wide_and_nan_scales(pd, dev, M, a_kind):
    N, K = 70, 500
    gu.note(f"[case] gemm_a16_mxf4 wide scales M={M} {a_kind}")
    t, x = to_type(spread(M, K, 8), a_kind)
    for lo, hi in ((60, 190), (0, 20), (200, 240)):
        b = random_operand(N, K, lo, lo, hi)
        R, S = mx.product(x, mx.values(*b, K))
        C = pd.gemm_a16_mxf4(source(t, dev, 12), *stored(*b, K, dev))
        got = C.cpu().double().numpy()
        tol = (-(-K // 64) + 1) * 2.0 ** -22 * S + K * 2.0 ** -149
        # every partial sum of an element is at most S (1 + 2^-19) in magnitude: below 2^128,
        # binary32's overflow, where S < 2^127; the largest S here is 1.78 * 2^128
        inside = S < 2.0 ** 127
        assert inside.mean() > 0.9 and (np.abs(got - R)[inside] <= tol[inside]).all(), (lo, hi)
    b = random_operand(N, K, 1)
    b[1][0, 3] = b[1][-1, 69] = 255
    x[1, 2], x[2, 499] = np.nan, np.inf
    t = torch.from_numpy(x).to(TYPES[a_kind])
    got = pd.gemm_a16_mxf4(source(t, dev, 12), *stored(*b, K, dev)).cpu().double().numpy()
    nan_b = np.zeros(N, bool)
    nan_b[[3, 69]] = True
    assert np.isnan(got[1]).all() and np.isnan(got[:, nan_b]).all()
    assert not np.isfinite(got[2]).any()             # infinity times zero, or an infinity
    rest = np.delete(np.delete(got, [1, 2], 0), np.flatnonzero(nan_b), 1)
    assert np.isfinite(rest).all()


def test_products_are_reproducible(pd, dev):
    gu.note("[case] repeated products")
    for M, N, K in ((7, 200, 4000), (300, 500, 1000)):
        a, b, _, _ = operands(M, N, K, 31)
        A, B = stored(*a, K, dev), stored(*b, K, dev)
        x = source(to_type(spread(M, K, 3), "bf16")[0], dev, gu.round_up(K, 8) - K)
        first = pd.gemm_mxf4(*A, *B, K), pd.gemm_a16_mxf4(x, *B)
        for _ in range(3):
            assert torch.equal(pd.gemm_mxf4(*A, *B, K), first[0])
            assert torch.equal(pd.gemm_a16_mxf4(x, *B), first[1])


# ---- used together ----

def layer_step(pd, x, w, g, out_dtype):
    """Forward product and both gradients of Y = X W^T with every product in MXFP4."""
    (xq, xs), (xt, xst) = pd.mxf4_quantize_both(x)
    (wq, ws), (wt, wst) = pd.mxf4_quantize_both(w)
    (gq, gs), (gt, gst) = pd.mxf4_quantize_both(g)
    M, K, N = x.shape[0], x.shape[1], w.shape[0]
    return (pd.gemm_mxf4(xq, xs, wq, ws, K, out_dtype=out_dtype), pd.gemm_mxf4(gq, gs, wt, wst, N, out_dtype=out_dtype),
            pd.gemm_mxf4(gt, gst, xt, xst, M))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 64, 96), (77, 130, 200), (300, 257, 515)], ids=["1x64x96", "77x130x200", "300x257x515"])
def test_layer_step(pd, dev, shape, kind):
    M, N, K = shape
    gu.note(f"[case] layer step {shape} {kind}")
    (xt, x), (wt, w), (gt, g) = (to_type(spread(*s, 40 + n), kind) for n, s in enumerate(((M, K), (N, K), (M, N))))
    y, dx, dw = layer_step(pd, source(xt, dev), source(wt, dev), source(gt, dev), TYPES[kind])
    val = lambda t: mx.values(*mx.quantize(t), t.shape[1])  # noqa: E731
    for name, got, a, b, k, out in (("y", y, x, w, K, kind), ("dx", dx, g, w.T, N, kind), ("dw", dw, g.T, x.T, M, "f32")):
        R, S = mx.product(val(a), val(b))
        assert_close(got, R, S, -(-k // 64), out, f"{name} {shape}")


def test_gradients_by_differences(pd, dev):
    """With operands that MXFP4 holds exactly along both axes (one magnitude per tensor, so
    every block's scale is the same), dX and dW are the differences of the loss sum(G * Y)
    itself: it is linear in each element of X and W, and its every term is a dyadic number
    that binary32 holds exactly."""
    gu.note("[case] gradients by differences")
    M, N, K = 33, 40, 65
    rng = np.random.default_rng(17)
    grid = np.array([-6, -4, -3, -2, -1.5, -1, -.5, 0, .5, 1, 1.5, 2, 3, 4, 6])

    def exact(rows, cols):
        v = rng.choice(grid, (rows, cols))
        # every 32-block along either axis holds a 4 or 6, so that its scale is 1
        for i in range(rows):
            for b in range(0, cols, 32):
                v[i, b + (i % min(32, cols - b))] = 4.0
        for j in range(cols):
            for b in range(0, rows, 32):
                v[b + (j % min(32, rows - b)), j] = 6.0
        return v

    x, w, g = exact(M, K), exact(N, K), exact(M, N)
    for t in (x, w, g):
        for u in (t, t.T):
            assert np.array_equal(mx.values(*mx.quantize(u), u.shape[1]), u)
    put = lambda v: torch.from_numpy(v).half().to(dev)  # noqa: E731
    y, dx, dw = (t.cpu().double().numpy() for t in layer_step(pd, put(x), put(w), put(g), torch.float32))
    assert np.array_equal(y, x @ w.T) and np.array_equal(dx, g @ w) and np.array_equal(dw, g.T @ x)

    def loss(xv, wv):
        q = pd.mxf4_quantize(put(xv)), pd.mxf4_quantize(put(wv))
        return float((pd.gemm_mxf4(*q[0], *q[1], K).cpu().double().numpy() * g).sum())

    base = loss(x, w)
    for i, k in ((0, 0), (32, 64), (17, 31), (5, 40)):
        for t, grad, which in ((x, dx, 0), (w, dw, 1)):
            v = t.copy()
            old = v[i, k]
            v[i, k] = 2.0 if old != 2.0 else 3.0
            if not np.array_equal(mx.values(*mx.quantize(v), K), v):
                continue                             # the only 4 or 6 of its block: the scale would move
            moved = loss(v, w) if which == 0 else loss(x, v)
            assert moved - base == grad[i, k] * (v[i, k] - old)


def test_captured_step_replays(pd, dev):
    """Quantising and the products recorded into a graph, beside an eager run of the same
    call; each replay follows eager work that overwrites the outputs."""
    gu.note("[case] graph of a layer step")
    M, N, K = 130, 200, 330
    x, w, g = (source(to_type(spread(*s, 60 + n), "bf16")[0], dev) for n, s in enumerate(((M, K), (N, K), (M, N))))
    ops = [pd.mxf4_quantize_both(t) for t in (x, w, g)]
    outs = [torch.empty((M, N), device=dev), torch.empty((M, K), device=dev), torch.empty((N, K), device=dev),
            torch.empty((M, K), device=dev)]
    a16_out = torch.empty((M, N), device=dev)
    x16 = source(to_type(spread(M, K, 60), "bf16")[0], dev, gu.round_up(K, 8) - K)

    def call():
        for t, o in zip((x, w, g), ops):
            pd.mxf4_quantize_both(t, out=o)
        (xq, xt), (wq, wt), (gq, gt) = ops
        pd.gemm_mxf4(*xq, *wq, K, out=outs[0])
        pd.gemm_mxf4(*gq, *wt, N, out=outs[1])
        pd.gemm_mxf4(*gt, *xt, M, out=outs[2])
        pd.mxf4_dequantize(*xq, K, out=outs[3])
        pd.gemm_a16_mxf4(x16, *wq, out=a16_out)

    call()
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs + [a16_out]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for replay in range(3):
        for t in outs + [a16_out]:
            t.fill_(float("nan"))
        for pair in ops:
            for codes, scales in pair:
                codes.fill_(0x55)
                scales.fill_(0x7F)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, (t, e) in enumerate(zip(outs + [a16_out], eager)):
            assert torch.equal(t, e), f"replay {replay}, output {n}"
    del graph


def test_another_stream(pd, dev):
    gu.note("[case] another stream")
    M, N, K = 200, 300, 520
    t, x = to_type(spread(M, K, 71), "f16")
    b = random_operand(N, K, 72)
    R, S = mx.product(mx.values(*mx.quantize(x), K), mx.values(*b, K))
    B = stored(*b, K, dev)
    xd = t.to(dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s = pd.mxf4_quantize(xd, stream=side)
    C = pd.gemm_mxf4(q, s, *B, K, stream=side)
    v = pd.mxf4_dequantize(q, s, K, stream=side)
    side.synchronize()
    assert_close(C, R, S, -(-K // 64), "f32", "side stream")
    assert np.array_equal(v.cpu().double().numpy(), mx.values(*mx.quantize(x), K))


# ---- large sizes, long rows ----

@pytest.mark.parametrize("a_kind", [None, "f16", "bf16"], ids=["mxf4", "a16-f16", "a16-bf16"])
@pytest.mark.parametrize("shape", [(4096, 4096, 256), (8192, 4096, 96), (2560, 2304, 520), (1024, 8192, 320)],
                         ids=["one-window", "two-windows", "bands", "wide"])
def test_many_tiles(pd, dev, shape, a_kind):
    """Grids of whole 16 x 16 windows of tiles, and of bands: every element, against the
    product in 64 bits of the oracle's values."""
    M, N, K = shape
    gu.note(f"[case] many tiles {shape} {a_kind}")
    b = random_operand(N, K, 82, 124, 130)
    vb = torch.from_numpy(mx.values(*b, K)).to(dev)
    if a_kind is None:
        a = random_operand(M, K, 81, 124, 130)
        va = torch.from_numpy(mx.values(*a, K)).to(dev)
        C = pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K)
    else:
        t, x = to_type(spread(M, K, 83), a_kind)
        va = torch.from_numpy(x).to(dev)
        C = pd.gemm_a16_mxf4(source(t, dev, gu.round_up(K, 8) - K + 8), *stored(*b, K, dev))
    R, S = va @ vb.t(), va.abs() @ vb.t().abs()
    bad = (C.double() - R).abs() > (-(-K // 64) + 1) * 2.0 ** -22 * S
    assert not bool(bad.any()), f"{int(bad.sum())} off, first at {torch.nonzero(bad)[0].tolist()}"


@pytest.mark.parametrize("cfg", [0, 1, 2, 3, 9])
def test_rows_of_4_mib(pd, dev, cfg):
    """The longest rows the library takes: codes, scales, activations and C 4 MiB apart."""
    M, N, K = (260, 70, 300) if cfg < 2 else (70, 40, 300)
    gu.note(f"[case] rows of 4 MiB cfg={cfg}")
    row = 1 << 22
    a, b, R, S = operands(M, N, K, 91)

    def far(host):
        buf = torch.empty((host.shape[0], row), dtype=torch.uint8, device=dev)
        buf[:, :host.shape[1]] = torch.from_numpy(host).to(dev)
        return buf[:, :host.shape[1]]

    A, sa, B, sb = far(a[0]), far(a[1]), far(b[0]), far(b[1])
    out = torch.empty((M, row // 4), device=dev)[:, :N]
    pd.gemm_mxf4(A, sa, B, sb, K, out=out, cfg=cfg)
    assert_close(out, R, S, -(-K // 64), "f32", f"4 MiB cfg {cfg}")
    t, x = to_type(spread(M, K, 92), "bf16")
    x16 = torch.empty((M, row // 2), dtype=torch.bfloat16, device=dev)[:, :K]
    x16.copy_(t)
    R, S = mx.product(x, mx.values(*b, K))
    pd.gemm_a16_mxf4(x16, B, sb, out=out, cfg=cfg)
    assert_close(out, R, S, -(-K // 64) + 1, "f32", f"4 MiB a16 cfg {cfg}")


def test_offsets_past_32_bits(pd, dev):
    """A tensor of more than 2^31 elements (and bytes past 2^32): its last rows, and rows in
    between, quantise and read back as those rows alone do."""
    rows, K = 33000, 65600
    gu.note(f"[case] past 32 bits {rows}x{K}")
    x = torch.empty((rows, K), dtype=torch.bfloat16, device=dev)
    part = torch.from_numpy(spread(96, K, 97)).to(torch.bfloat16).to(dev)
    for first in range(0, rows, 96):
        x[first:first + 96] = part[:min(96, rows - first)] * 2.0 ** (first % 7)
    (q, s), (qt, st) = pd.mxf4_quantize_both(x)
    for first in (0, 16384, rows - 96):
        alone, scales = pd.mxf4_quantize(x[first:first + 96])
        assert torch.equal(q[first:first + 96], alone) and torch.equal(s[:, first:first + 96], scales)
        v = pd.mxf4_dequantize(q[first:first + 96], s[:, first:first + 112][:, :96].contiguous(), K)
        assert torch.equal(v, pd.mxf4_dequantize(alone, scales, K))
    last = rows // 32 * 32 - 64
    alone, scales = pd.mxf4_quantize(x[last:].contiguous(), transpose=True)
    assert torch.equal(qt[:, last // 2:], alone) and torch.equal(st[last // 32:], scales)
    v = pd.mxf4_dequantize(q, s, K, out_dtype=torch.bfloat16)
    assert torch.equal(v[-5:], pd.mxf4_dequantize(*pd.mxf4_quantize(x[-5:]), K, out_dtype=torch.bfloat16))


def test_out_needs_room_for_whole_blocks(pd, dev):
    gu.note("[case] out without room")
    x = torch.randn((1, 40), device=dev)
    scales = torch.empty((2, 16), dtype=torch.uint8, device=dev)[:, :1]
    with pytest.raises(ValueError):
        pd.mxf4_quantize(x, out=(torch.empty((1, 20), dtype=torch.uint8, device=dev), scales))
    codes = torch.empty((1, 32), dtype=torch.uint8, device=dev)[:, :20]
    pd.mxf4_quantize(x, out=(codes, scales))
    want = mx.quantize(x.cpu().double().numpy())
    assert np.array_equal(codes.cpu().numpy(), want[0][:, :20]) and np.array_equal(scales.cpu().numpy(), want[1])


def test_two_streams_at_once(pd, dev):
    gu.note("[case] two streams at once")
    M, N, K = 300, 400, 2000
    cases = [operands(M, N, K, 51 + n) for n in range(2)]
    devs = [(stored(*a, K, dev), stored(*b, K, dev)) for a, b, _, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for n, st in enumerate(streams):
            outs[n].append(pd.gemm_mxf4(*devs[n][0], *devs[n][1], K, stream=st))
    torch.cuda.synchronize()
    for n, (_, _, R, S) in enumerate(cases):
        assert_close(outs[n][0], R, S, -(-K // 64), "f32", f"stream {n}")
        assert all(torch.equal(o, outs[n][0]) for o in outs[n])


@pytest.mark.parametrize("a_kind", ["f16", "bf16"])
@pytest.mark.parametrize("cfg", range(13))
@pytest.mark.parametrize("K", [1, 41, 300])
def test_a16_largest_scales_beside_the_operand(pd, dev, K, cfg, a_kind):
    """Codes of 6 right after the last value, in a block whose scale makes them 2^129: a column's
    result holds only the values inside, +-2^126."""
    M, N = 20, 37
    gu.note(f"[case] gemm_a16_mxf4 largest scales K={K} cfg={cfg} {a_kind}")
    rng = np.random.default_rng(K)
    t, x = to_type(rng.standard_normal((M, K)) * 2.0 ** -10, a_kind)
    codes = np.where(rng.integers(0, 2, (N, 16 * mx.blocks_of(K))) == 1, 0x91, 0x19).astype(np.uint8)
    b = codes, np.full((mx.blocks_of(K), N), 254, np.uint8)
    R, S = mx.product(x, mx.values(*b, K))
    C = pd.gemm_a16_mxf4(source(t, dev, gu.round_up(K, 8) - K + 8), *stored(*b, K, dev), cfg=cfg)
    assert_close(C, R, S, -(-K // 64) + 1, "f32", f"K={K} cfg {cfg} {a_kind}")


@pytest.mark.parametrize("cfg", range(10))
@pytest.mark.parametrize("K", [41, 300])
def test_product_of_zeros_at_the_largest_scales(pd, dev, K, cfg):
    M, N = 20, 37
    gu.note(f"[case] gemm_mxf4 zeros at the largest scales K={K} cfg={cfg}")
    a = random_operand(M, K, 1)
    a[0][:, 16:], a[1][1:] = 0, 254               # zero codes from the second block on
    b = random_operand(N, K, 2)
    b[1][1:] = 254
    R, S = mx.product(mx.values(*a, K), mx.values(*b, K))
    C = pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K, cfg=cfg)
    assert_close(C, R, S, -(-K // 64), "f32", f"K={K} cfg {cfg}")


@pytest.mark.parametrize("a_kind", ["mxf4", "f16", "bf16"])
@pytest.mark.parametrize("cfg", [0, 1])
def test_large_outputs_whose_rows_share_lines(pd, dev, cfg, a_kind):
    """More than 28 MB of C with an odd row stride: stored through the L2."""
    M, N, K = 2700, 2701, 40
    gu.note(f"[case] large C {M}x{N}x{K} cfg={cfg} {a_kind}")
    a, b, R, S = operands(M, N, K, 60 + cfg)
    buf, out = guarded(M, N, "f32", dev)
    assert out.stride(0) % 32 and M * N * 4 > 28_000_000
    if a_kind == "mxf4":
        pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K, out=out, cfg=cfg)
    else:
        t, x = to_type(spread(M, K, 61), a_kind)
        R, S = mx.product(x, mx.values(*b, K))
        pd.gemm_a16_mxf4(source(t, dev, 8), *stored(*b, K, dev), out=out, cfg=cfg)
    torch.cuda.synchronize()
    check_rest(buf, M, N)
    assert_close(out, R, S, -(-K // 64) + 1, "f32", f"{a_kind} cfg {cfg}")


@pytest.mark.parametrize("K, stride", [(40, 32), (2048, 1024), (2080, 1152), (2500, 1280)])
def test_strides_of_new_operands(pd, dev, K, stride):
    """Rows of more than 1 KB of codes start on whole lines; the values are the same."""
    gu.note(f"[case] new operand K={K}")
    x = torch.randn((40, K), device=dev)
    want = mx.quantize(x.cpu().double().numpy())
    (codes, scales), (codes_t, _) = pd.mxf4_quantize_both(x)
    assert codes.shape == (40, (K + 1) // 2) and codes.stride() == (stride, 1) and codes_t.stride() == (32, 1)
    assert np.array_equal(codes.cpu().numpy(), want[0][:, :(K + 1) // 2]) and np.array_equal(scales.cpu().numpy(), want[1])
    v = pd.mxf4_dequantize(codes, scales, K)
    assert np.array_equal(v.cpu().double().numpy(), mx.values(*want, K))
    R, S = mx.product(mx.values(*want, K), mx.values(*want, K))
    assert_close(pd.gemm_mxf4(codes, scales, codes, scales, K), R, S, -(-K // 64), "f32", f"K={K}")


def test_one_row_of_a_long_tensor(pd, dev):
    """h[:, -1, :] of one sequence: one row, strided by the whole sequence, as every operand."""
    gu.note("[case] one row of a long tensor")
    K, N, far = 1030, 300, (1 << 22) + 16

    def put(host):
        buf = torch.full((2, far), 0, dtype=host.dtype, device=dev)
        buf[1, :host.shape[1]] = host[0].to(dev)
        return buf.view(1, 2, far)[:, -1, :host.shape[1]]

    t, x = to_type(spread(1, K, 5), "bf16")
    xd = put(t)
    assert xd.stride(0) * xd.element_size() > 1 << 22 and xd.is_contiguous()
    want = mx.quantize(x)
    out = put(torch.zeros((1, (K + 1) // 2), dtype=torch.uint8)), torch.zeros((33, 16), dtype=torch.uint8, device=dev)[:, :1]
    q, s = pd.mxf4_quantize(xd, out=out)
    (b, sb), (bt, sbt) = pd.mxf4_quantize_both(xd)
    for codes, scales in ((q, s), (b, sb)):
        assert np.array_equal(codes.cpu().numpy(), want[0][:, :(K + 1) // 2])
        assert np.array_equal(scales.cpu().numpy(), want[1])
    want_t = mx.quantize(x.T)
    assert np.array_equal(bt.cpu().numpy(), want_t[0][:, :1]) and np.array_equal(sbt.cpu().numpy(), want_t[1])
    v = pd.mxf4_dequantize(q, s, K, out=put(torch.zeros((1, K))))
    assert np.array_equal(v.cpu().double().numpy(), mx.values(*want, K))
    w = random_operand(N, K, 6)
    W = stored(*w, K, dev)
    for got, a in ((pd.gemm_mxf4(q, s, *W, K, out=put(torch.zeros((1, N)))), mx.values(*want, K)),
                   (pd.gemm_a16_mxf4(xd, *W, out=put(torch.zeros((1, N)))), x)):
        assert_close(got, *mx.product(a, mx.values(*w, K)), -(-K // 64) + 1, "f32", "one row")


@pytest.mark.parametrize("N", [48, 50])
def test_scales_of_a_checkpoint(pd, dev, N):
    """Scales kept by row, (N, K / 32): their transpose, in rows of a multiple of 16 bytes.  As
    it comes, packed, it is refused where N is not such a multiple."""
    M, K = 20, 320
    gu.note(f"[case] scales of a checkpoint N={N}")
    t, x = to_type(spread(M, K, 5), "bf16")
    codes, by_block = random_operand(N, K, 6)
    B, by_row = torch.from_numpy(codes).to(dev), torch.from_numpy(by_block.T.copy()).to(dev)
    packed = by_row.t().contiguous()
    if N % 16:
        with pytest.raises(pd.PdgemmError, match="MXFP4 codes and scales .* 16"):
            pd.gemm_a16_mxf4(t.to(dev), B, packed)
    scales = torch.empty((K // 32, gu.round_up(N, 16)), dtype=torch.uint8, device=dev)[:, :N]
    scales.copy_(by_row.t())
    R, S = mx.product(x, mx.values(codes, by_block, K))
    assert_close(pd.gemm_a16_mxf4(t.to(dev), B, scales), R, S, -(-K // 64) + 1, "f32", f"N={N}")


def test_results_carry_no_graph(pd, dev):
    """The calls are not differentiable operations: results of tensors that require gradients do
    not, and the documentation says so."""
    gu.note("[case] no graph")
    x = torch.randn((20, 64), device=dev, dtype=torch.float16, requires_grad=True)
    q, s = pd.mxf4_quantize(x)
    for out in (pd.mxf4_dequantize(q, s, 64), pd.gemm_mxf4(q, s, q, s, 64), pd.gemm_a16_mxf4(x, q, s)):
        assert not out.requires_grad and out.grad_fn is None
    assert "gradient" in pd.__doc__


@pytest.mark.parametrize("rule", ["floor", "fit"])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_quantize_every_16_bit_value(pd, dev, kind, rule):
    """Every value of a 16-bit type under scales from one end of its range to the other: in
    each row the first value sets the scale, and the 31 others run over all that are not larger."""
    bits = np.arange(0, 0x7C00 if kind == "f16" else 0x7F80, dtype=np.uint16)
    vals = torch.from_numpy(bits.view(np.int16)).view(TYPES[kind]).double().numpy()
    rows = []
    for top in vals[[1, 5, len(vals) // 5, len(vals) // 3, len(vals) // 2, 3 * len(vals) // 4, -700, -200, -1]]:
        below = vals[vals <= top]
        below = np.concatenate([below, np.full(-len(below) % 31, top)]).reshape(-1, 31)
        rows.append(np.hstack([np.full((len(below), 1), top), below]))
    rows = np.vstack(rows)
    t = torch.from_numpy(rows * np.where(np.random.default_rng(4).random(rows.shape) < 0.5, -1, 1)).to(TYPES[kind])
    gu.note(f"[case] quantize every 16-bit value {kind} {rule} {tuple(t.shape)}")
    want = mx.quantize(t.double().numpy(), rule)
    assert set(np.unique(np.concatenate([want[0] & 15, want[0] >> 4]))) == set(range(16))
    q, s = pd.mxf4_quantize(t.to(dev), scale_rule=rule)
    qt, st = pd.mxf4_quantize(t.t().contiguous().to(dev), transpose=True, scale_rule=rule)
    (b, sb), _ = pd.mxf4_quantize_both(t.to(dev), scale_rule=rule)
    for name, codes, scales in (("rows", q, s), ("transpose", qt, st), ("both", b, sb)):
        assert np.array_equal(scales.cpu().numpy(), want[1]), name
        assert np.array_equal(codes.cpu().numpy(), want[0]), name


# ---- the corners of what the header allows ----

def off_by_one(rows, cols, kind, dev, value=7.0):
    """A view whose first element has only its own alignment, in rows of an odd stride."""
    ld = cols + 3 + (cols % 2)                       # odd
    flat = torch.full((rows * ld + ld + 1,), value, dtype=TYPES[kind], device=dev)
    return flat, torch.as_strided(flat, (rows, cols), (ld, 1), 1)


@pytest.mark.parametrize("kind", list(TYPES))
def test_elements_aligned_sources_and_results(pd, dev, kind):
    """Dense arrays need only their element's alignment, the first element's too."""
    gu.note(f"[case] element alignment {kind}")
    rows, K = 300, 1029
    t, x = to_type(spread(rows, K, 21), kind)
    _, src = off_by_one(rows, K, kind, dev, float("nan"))
    src.copy_(t)
    assert src.data_ptr() % 16 == TYPES[kind].itemsize
    want, want_t = mx.quantize(x), mx.quantize(x.T)
    (q, s), (qt, st) = pd.mxf4_quantize_both(src)
    q1, s1 = pd.mxf4_quantize(src)
    for codes, scales, ref in ((q, s, want), (q1, s1, want), (qt, st, want_t)):
        assert np.array_equal(codes.cpu().numpy(), ref[0][:, :codes.shape[1]])
        assert np.array_equal(scales.cpu().numpy(), ref[1])
    flat, out = off_by_one(rows, K, kind, dev)
    pd.mxf4_dequantize(q, s, K, out=out)
    # (a value of few bits is exact in each type; spread's are far from the types' ends)
    assert np.array_equal(out.cpu().double().numpy(), mx.values(*want, K))
    out.fill_(7.0)
    assert bool((flat == 7.0).all())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("cfg", range(13))
def test_elements_aligned_products(pd, dev, cfg, kind):
    M, N, K = 261, 135, 328
    gu.note(f"[case] element-aligned C cfg={cfg} {kind}")
    a, b, R, S = operands(M, N, K, 22)
    for what, steps in (("mxf4", -(-K // 64)), ("f16", -(-K // 64) + 1), ("bf16", -(-K // 64) + 1)):
        flat, out = off_by_one(M, N, kind, dev)
        if what == "mxf4":
            if cfg >= pd.mxf4_num_configs():
                continue
            pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K, out=out, cfg=cfg)
        else:
            t, x = to_type(spread(M, K, 23), what)
            R, S = mx.product(x, mx.values(*b, K))
            pd.gemm_a16_mxf4(source(t, dev, 8), *stored(*b, K, dev), out=out, cfg=cfg)
        assert_close(out, R, S, steps, kind, f"{what} cfg {cfg}")
        out.fill_(7.0)
        assert bool((flat == 7.0).all()), "stores outside the M x N block"


def on_gpu(codes, scales, K, dev):
    """float64 values on the GPU of codes and scales there (no NaN scales)."""
    table = torch.tensor(list(mx.E2M1) + [-v for v in mx.E2M1], dtype=torch.float64, device=dev)
    nib = torch.stack((codes & 15, codes >> 4), dim=2).view(codes.shape[0], -1)[:, :K]
    scale = ((scales.t().to(torch.int64) - 127 + 1023) << 52).view(torch.float64)
    return table[nib.to(torch.int64)] * scale.repeat_interleave(32, dim=1)[:, :K]


def random_on_gpu(rows, K, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    nb = mx.blocks_of(K)
    codes = torch.randint(0, 256, (rows, 16 * nb), dtype=torch.uint8, device=dev, generator=g)
    scales = torch.randint(122, 132, (nb, gu.round_up(rows, 16)), dtype=torch.uint8, device=dev, generator=g)
    return codes, scales[:, :rows]


def assert_close_on_gpu(C, va, vb, steps, what):
    R, S = va @ vb.t(), va.abs() @ vb.abs().t()
    bad = ~((C.double() - R).abs() <= steps * 2.0 ** -22 * S)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, first at {torch.nonzero(bad)[0].tolist()}"


@pytest.mark.parametrize("M, N", [((1 << 22), 5), (9, 1 << 20)], ids=["rows", "columns"])
def test_most_rows(pd, dev, M, N):
    """Operands of 4 Mi rows (their scales' rows are 4 MiB) and C's rows of 4 MiB."""
    K = 40
    gu.note(f"[case] most rows {M}x{N}x{K}")
    a, b = random_on_gpu(M, K, 1, dev), random_on_gpu(N, K, 2, dev)
    va, vb = on_gpu(*a, K, dev), on_gpu(*b, K, dev)
    assert_close_on_gpu(pd.gemm_mxf4(a[0], a[1], b[0], b[1], K), va, vb, 1, "mxf4")
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=dev).copy_(va)      # (two significant bits: exact)
    assert_close_on_gpu(pd.gemm_a16_mxf4(x, *b), va, vb, 2, "a16")
    with pytest.raises(pd.PdgemmError):
        pd.mxf4_quantize(torch.zeros(((1 << 22) + 1, 1), device=dev))        # scales' rows past 4 MiB


def test_more_rows_of_activations(pd, dev):
    """16-bit activations have no scales: more rows than an MXFP4 operand may have."""
    M, N, K = 5_000_001, 3, 8
    gu.note(f"[case] more rows of activations {M}x{N}x{K}")
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    x = torch.randn((M, K), device=dev, generator=g).half()
    b = random_on_gpu(N, K, 3, dev)
    assert_close_on_gpu(pd.gemm_a16_mxf4(x, *b), x.double(), on_gpu(*b, K, dev), 2, "a16")


def test_tallest_transpose(pd, dev):
    """8 Mi rows quantised along themselves: a row of the transpose is 4 MiB of codes."""
    rows, K = 1 << 23, 3
    gu.note(f"[case] tallest transpose {rows}x{K}")
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    x = torch.randn((rows, K), device=dev, generator=g).bfloat16()
    qt, st = pd.mxf4_quantize(x, transpose=True)
    assert qt.shape == (K, rows // 2)
    # a row along K of the copied transpose, in pieces of 2 MiB of values, which are rows of their own
    pieces = x.t().contiguous().view(4 * K, rows // 4)
    q, s = pd.mxf4_quantize(pieces)
    assert torch.equal(qt.reshape(4 * K, rows // 8), q)
    blocks = rows // 32
    assert torch.equal(st.t().reshape(K, 4, blocks // 4), s.t().reshape(K, 4, blocks // 4))
    v = pd.mxf4_dequantize(qt[:, :rows // 16], st[:rows // 256], rows // 8, out_dtype=torch.bfloat16)
    assert torch.equal(v, pd.mxf4_dequantize(q, s, rows // 4, out_dtype=torch.bfloat16)[::4, :rows // 8])


@pytest.mark.parametrize("cfg", [None, 0, 1, 2])
def test_longest_rows(pd, dev, cfg):
    """Rows of 4 MiB: 8 Mi values of K in MXFP4, 2 Mi of 16-bit activations."""
    M, N, K = 3, 5, 1 << 23
    gu.note(f"[case] longest rows {M}x{N}x{K} cfg={cfg}")
    a, b = random_on_gpu(M, K, 6, dev), random_on_gpu(N, K, 7, dev)
    assert_close_on_gpu(pd.gemm_mxf4(*a, *b, K, cfg=cfg), on_gpu(*a, K, dev), on_gpu(*b, K, dev), K // 64, "mxf4")
    K = 1 << 21
    b = random_on_gpu(N, K, 7, dev)
    g = torch.Generator(device=dev)
    g.manual_seed(8)
    for dtype in (torch.float16, torch.bfloat16):
        x = torch.randn((M, K), device=dev, generator=g).to(dtype)
        assert_close_on_gpu(pd.gemm_a16_mxf4(x, *b, cfg=cfg), x.double(), on_gpu(*b, K, dev), K // 64 + 1, f"a16 {dtype}")


@pytest.mark.parametrize("a_kind", ["mxf4", "f16", "bf16"])
@pytest.mark.parametrize("cfg", range(13))
def test_nan_and_infinity_stay_in_their_rows(pd, dev, cfg, a_kind):
    """On every tile: NaN blocks and non-finite activations reach their row or column of C, and
    the rest is as without them."""
    M, N, K = 70, 75, 300
    gu.note(f"[case] NaN on every tile cfg={cfg} {a_kind}")
    a, b, _, _ = operands(M, N, K, 33)
    b[1][0, 3] = b[1][-1, N - 1] = b[1][4, 40] = 255
    b[0][3, :16] = 0                                 # a NaN scale over zero codes is NaN too
    vb = mx.values(*b, K)
    if a_kind == "mxf4":
        if cfg >= pd.mxf4_num_configs():
            return
        a[1][0, 1] = a[1][-1, M - 1] = 255
        va = mx.values(*a, K)
        C = pd.gemm_mxf4(*stored(*a, K, dev), *stored(*b, K, dev), K, cfg=cfg)
    else:
        x = spread(M, K, 34)
        x[1, 2], x[M - 1, K - 1], x[17, 130] = np.nan, np.inf, -np.inf
        t, va = to_type(x, a_kind)
        C = pd.gemm_a16_mxf4(source(t, dev, gu.round_up(K, 8) - K + 8), *stored(*b, K, dev), cfg=cfg)
    got = C.cpu().double().numpy()
    rows, cols = ~np.isfinite(va).all(axis=1), np.isnan(vb).any(axis=1)
    assert not np.isfinite(got[rows]).any() and np.isnan(got[:, cols]).all()
    R, S = mx.product(va[~rows], vb[~cols])
    tol = (-(-K // 64) + 1) * 2.0 ** -22 * S
    assert (np.abs(got[~rows][:, ~cols] - R) <= tol).all()
