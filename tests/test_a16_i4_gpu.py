"""GPU parity of products with group-scaled INT4 weights against the 64-bit oracle.

Every buffer is wider than the operand and holds poison outside it, every output sits among
sentinels, and each case prints its name before it touches the GPU.

Tolerance, with A the sum of |a| |scale| over K.  A matrix instruction adds at least 32 products to
a binary32 sum, and its result is taken to be within four half units (2^-22) of the magnitudes it adds.
The codes may enter with a bias (16 to 31 in the place of -8 to 7, after 24 times the activations
were taken off), so those are at most 55 |a| of a step of 128 values, for which at most 8 instructions
follow one another: 440 * 2^-22 A in all.  Each sum of a group is then scaled and added to a sum below 8
A, at most 1.25 K / 32 times, and up to 16 waves' and 16 splits' sums are added: another (1.25 K / 32 + 32) * 8
* 2^-24 A.  (512 + K / 12) * 2^-22 A bounds both.  Rounding to a 16-bit type adds half a unit of the
result, or half its smallest subnormal.
"""
from __future__ import annotations

import numpy as np
import pytest

import oracle.int4 as i4
from tests import gpu_util as gu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_UNIT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
HALF_TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_dense_gemm_amd as pd
    return pd


def held(x, kind):
    """float64 host values -> (CPU tensor of the type, the float64 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[kind])
    return t, t.double().numpy()


def placed(t, pad, fill):
    """t on the GPU in rows `pad` elements longer that hold `fill`, with a row of it before and after."""
    buf = torch.full((t.shape[0] + 2, t.shape[1] + pad), fill, dtype=t.dtype)
    buf[1:-1, :t.shape[1]] = t
    return buf.cuda()[1:-1, :t.shape[1]]


def activations(M, K, seed, kind):
    rng = np.random.default_rng(seed)
    return held(rng.standard_normal((M, K)) * np.exp2(rng.integers(-4, 5, (M, 1))) * np.exp2(rng.integers(-3, 4, (1, K))), kind)


def placed_activations(t):
    K = t.shape[1]
    return placed(t, gu.round_up(K, 8) - K + 8, float("nan"))


def weights(N, K, group, seed, kind, lo=-8, hi=7):
    """(codes, scales as a CPU tensor, values in 64 bits, the magnitudes of their scales)."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(lo, hi + 1, (N, K))
    scales, sv = held(np.exp2(rng.uniform(-6, 2, (-(-K // group), N))) * rng.choice([-1.0, 1.0], (1, N)), kind)
    return codes, scales, i4.values(codes, sv, group), np.abs(i4.values(np.ones_like(codes), sv, group))


def placed_codes(codes):
    """Packed codes on the GPU among 0x77, also in the high nibble of an odd K."""
    N, K = codes.shape
    packed = i4.pack(codes)
    if K % 2:
        packed[:, -1] |= 0x70
    t = torch.from_numpy(packed)
    buf = torch.full((N + 2, gu.round_up(t.shape[1], 16) + 16), 0x77, dtype=torch.uint8)
    buf[1:-1, :t.shape[1]] = t
    return buf.cuda()[1:-1, :t.shape[1]]


def guarded(M, N, kind, pad=3):
    buf = torch.full((M + 2, N + pad), -777.0, dtype=TYPES[kind], device="cuda")
    return buf, buf[1:-1, :N]


def check(buf, M, N, R, A, K, kind, what):
    got = buf.cpu().double().numpy()
    edge = np.ones(got.shape, bool)
    edge[1:-1, :N] = False
    sentinel = float(torch.tensor(-777.0, dtype=TYPES[kind]))
    assert (got[edge] == sentinel).all(), f"{what}: stores beside the result"
    got = got[1:-1, :N]
    tol = (512 + K / 12) * 2.0 ** -22 * A
    tol = tol + (np.abs(R) + tol) * HALF_UNIT[kind] + HALF_TINY[kind]
    bad = ~(np.abs(got - R) <= tol) & (np.abs(R) + tol < float(torch.finfo(TYPES[kind]).max))
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {np.argwhere(bad)[0]}: {got[bad][0]} for {R[bad][0]}"


def run_case(pd, M, N, K, group, kind, s_kind, out, seed=0, cfg=None):
    what = f"{M}x{N}x{K} group {group} {kind} scales {s_kind} -> {out} cfg {cfg}"
    gu.note(what)
    a, av = activations(M, K, seed, kind)
    codes, scales, w, m = weights(N, K, group, seed + 1, s_kind)
    R, A = i4.product(av, w)[0], np.abs(av) @ m.T
    buf, view = guarded(M, N, out)
    pd.gemm_a16_i4(placed_activations(a), placed_codes(codes), placed(scales, 3, float("nan")), group, out=view, cfg=cfg)
    check(buf, M, N, R, A, K, out, what)


def configs(pd, group):
    """The tile configurations that serve a group: the last one multiples of 128."""
    return range(pd.a16_i4_num_configs() - (1 if group % 128 else 0))


@pytest.mark.parametrize("cfg", range(11))
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_every_tile(pd, cfg, kind):
    assert pd.a16_i4_num_configs() == 11
    for n, (M, N, K, group) in enumerate([(1, 1, 1, 32), (3, 17, 129, 32), (16, 64, 256, 64), (17, 65, 333, 64), (33, 130, 640, 128),
                                          (67, 70, 1337, 96), (65, 100, 2048, 256), (130, 33, 5000, 160), (2, 40, 96, 4096),
                                          (260, 270, 1500, 128), (129, 513, 257, 256)]):
        if cfg not in configs(pd, group):
            with pytest.raises(pd.PdgemmError):
                run_case(pd, M, N, K, group, kind, "f32", "f32", 0, cfg)
            continue
        run_case(pd, M, N, K, group, kind, ("f32", kind)[n % 2], ("f32", "f16", "bf16")[n % 3], 7 * n, cfg)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 64, 65, 200, 300])
def test_shapes(pd, M):
    for n, (N, K) in enumerate([(1, 4096), (255, 31), (1000, 1000), (4099, 65), (600, 3001)]):
        for group in (32, 64, 128):
            run_case(pd, M, N, K, group, ("f16", "bf16")[(n + M) % 2], ("f32", "f16", "bf16")[(n + group // 32) % 3],
                     ("f32", "bf16", "f16")[n % 3], n + M)


def test_every_code_exactly(pd):
    """One-hot activations read the weights back: code times scale, exact in binary32."""
    K = 160
    codes = (np.arange(16 * K).reshape(16, K) + np.arange(16)[:, None]) % 16 - 8
    for kind in ("f16", "bf16"):
        for group in (32, 64, 128):
            scales, sv = held(np.exp2(np.arange(16) - 8.0)[None, :] * (1 + np.arange(-(-K // group)))[:, None], kind)
            eye = torch.eye(K, dtype=TYPES[kind])
            for cfg in configs(pd, group):
                got = pd.gemm_a16_i4(eye.cuda(), placed_codes(codes), scales.cuda(), group, cfg=cfg)
                assert np.array_equal(got.cpu().double().numpy(), i4.values(codes, sv, group).T), (kind, group, cfg)


def test_infinities_and_nan(pd):
    K, N = 200, 24
    codes, scales, w, m = weights(N, K, 64, 5, "f32", lo=1)
    for kind in ("f16", "bf16"):
        a, av = activations(4, K, 6, kind)
        a[1, 7], a[2, 190], a[3, 0] = float("inf"), float("nan"), -float("inf")
        with np.errstate(invalid="ignore"):
            R = a.double().numpy() @ w.T                         # no code is zero: infinite, of either sign
        for cfg in configs(pd, 64):
            got = pd.gemm_a16_i4(placed_activations(a), placed_codes(codes), scales.cuda(), 64, cfg=cfg).cpu().double().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(R)), (kind, cfg)
            assert np.array_equal(got[1], R[1]) and np.array_equal(got[3], R[3]), (kind, cfg)
    s = scales.clone()
    s[-1, 3] = float("inf")                                      # of the last, short group
    a, av = activations(2, K, 6, "bf16")
    got = pd.gemm_a16_i4(placed_activations(a), placed_codes(codes), s.cuda(), 64).cpu()
    assert torch.isinf(got[:, 3]).all() and torch.isfinite(got[:, 4:]).all() and torch.isfinite(got[:, :3]).all()


def test_large_activations_and_scales_stay_finite(pd):
    """Products of 2^120 activations with small scales, and the other way round."""
    K = 256
    codes, scales, w, m = weights(32, K, 128, 8, "f32")
    for up, down in ((2.0 ** 120, 2.0 ** -100), (2.0 ** -100, 2.0 ** 118)):
        a, av = held(np.random.default_rng(1).uniform(-1, 1, (3, K)) * up, "bf16")
        R, A = i4.product(av, w * down)[0], np.abs(av) @ m.T * down
        buf, view = guarded(3, 32, "f32")
        pd.gemm_a16_i4(a.cuda(), placed_codes(codes), (scales.double() * down).float().cuda(), 128, out=view)
        check(buf, 3, 32, R, A, K, "f32", f"{up}")


def test_empty(pd):
    s = torch.zeros(0, 5, device="cuda")
    out = pd.gemm_a16_i4(torch.zeros(3, 0, dtype=torch.float16, device="cuda"), torch.zeros(5, 0, dtype=torch.uint8, device="cuda"), s, 32,
                         out=torch.ones(3, 5, device="cuda"))
    assert not out.any()
    a = torch.zeros(0, 32, dtype=torch.float16, device="cuda")
    assert pd.gemm_a16_i4(a, torch.zeros(5, 16, dtype=torch.uint8, device="cuda"), torch.zeros(1, 5, device="cuda"), 32).shape == (0, 5)


def test_a_sequences_last_token(pd):
    """h[:, -1, :] of one sequence: a row whose stride says nothing."""
    h, hv = activations(9, 512, 3, "bf16")
    codes, scales, w, m = weights(100, 512, 128, 4, "bf16")
    last = h.cuda().view(1, 9, 512)[:, -1, :]
    R, A = i4.product(hv[-1:], w)[0], np.abs(hv[-1:]) @ m.T
    buf, view = guarded(1, 100, "f32")
    pd.gemm_a16_i4(last, placed_codes(codes), scales.cuda(), 128, out=view)
    check(buf, 1, 100, R, A, 512, "f32", "last token")


def test_long_rows_of_scales_and_codes(pd):
    """Rows at the longest strides: offsets of a tile's last row, and of the last group, past 32 bits."""
    N, K, group = 40, 4096, 32
    codes, scales, w, m = weights(N, K, group, 9, "f32")
    wide = torch.zeros(N, 1 << 22, dtype=torch.uint8, device="cuda")
    wide[:, :K // 2] = torch.from_numpy(i4.pack(codes))
    s = torch.zeros(K // group, 1 << 20, device="cuda")
    s[:, :N] = scales
    many = torch.zeros(70, 1 << 21, dtype=torch.bfloat16, device="cuda")
    a, av = activations(70, K, 10, "bf16")
    many[:, :K] = a
    R, A = i4.product(av, w)[0], np.abs(av) @ m.T
    for cfg in configs(pd, group):
        buf, view = guarded(70, N, "f32")
        pd.gemm_a16_i4(many[:, :K], wide[:, :K // 2], s[:, :N], group, out=view, cfg=cfg)
        check(buf, 70, N, R, A, K, "f32", f"cfg {cfg}")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_what_is_not_finite_leaves_the_other_sums_bits(pd, kind):
    """A row of A and a column's scale that are not finite change their own row and column alone, to the bit."""
    M, N, K, group = 40, 100, 700, 64
    a, _ = activations(M, K, 2, kind)
    codes, scales, _, _ = weights(N, K, group, 3, "f32")
    rows, cols = [i for i in range(M) if i % 5 != 1], [j for j in range(N) if j != 17]
    bad, bad_scales = a.clone(), scales.clone()
    bad[1::5, 333] = float("inf")
    bad_scales[2, 17] = float("nan")
    for m in (2, 7, 16, 40):
        what = f"{m} rows of {kind}"
        gu.note(what)
        want, got = (pd.gemm_a16_i4(placed_activations(x[:m]), placed_codes(codes), s.cuda(), group, out_dtype=torch.float32).cpu()
                     for x, s in ((a, scales), (bad, bad_scales)))
        keep = [i for i in rows if i < m]
        assert torch.equal(got[keep][:, cols], want[keep][:, cols]), what
        assert torch.isnan(got[:, 17]).all() and not torch.isfinite(got[1]).any(), what


def test_same_bits_again_on_streams_and_in_a_replayed_graph(pd):
    codes, scales, w, m = weights(300, 1000, 64, 12, "f16")
    b, s = placed_codes(codes), scales.cuda()
    a = activations(20, 1000, 13, "f16")[0].cuda()
    want = pd.gemm_a16_i4(a, b, s, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pd.gemm_a16_i4(a, b, s, 64, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pd.gemm_a16_i4(a, b, s, 64)
    for turn in range(3):
        a.copy_(activations(20, 1000, 20 + turn, "f16")[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, pd.gemm_a16_i4(a, b, s, 64)), turn
