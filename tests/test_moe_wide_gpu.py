"""GPU parity of what passes between the expert layer's two products with the 64-bit oracle.

Tolerance.  As in test_moe_gpu.py up to the gated activation: the first product's sums are within
(512 + H / 12) * 2^-22 of the sum of |x| |scale|, carried on with slopes of 1.1 |u| and |silu(g)|, and silu's
exponential and roundings are within 2^-16 of the value.  The activation then is the sum of two bf16 values: the first
is within 2^-8 of it (2^-7 where it is cut off at bfloat16's largest value), the second within 2^-8 of what is left, or half
of bfloat16's smallest subnormal, so the two are within 2^-16 (2^-15 there).  Their sums of the second product are within
(512 + experts * I / 12) * 2^-22 of the sum of the parts' magnitudes times |scale|, at most 1 + 2^-7 times the values'.
y is rounded once.
"""
from __future__ import annotations

import numpy as np
import pytest

import oracle.int4 as i4
from tests import gpu_util as gu
from tests.test_a16_i4_gpu import HALF_TINY, HALF_UNIT, TYPES
from tests.test_moe_gpu import check_layer, layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_dense_gemm_amd as pd
    return pd


def check_wide(y, xv, ids, weights, first, second, kind, what, parts=2.0 ** -16):
    (d13, m13), (d2, m2) = first, second
    H, I = xv.shape[1], d2[0].shape[1]
    R, size, act_size, second, mass = i4.experts(xv, ids, weights, d13, d2, m13, m2)
    live = len({e for row in ids for e in row if 0 <= e < len(d2)})
    tol = act_size * (512 + H / 12) * 2.0 ** -22 + mass * 2.0 ** -134
    tol += (size + tol) * (parts + 2.0 ** -16) + (1 + 2.0 ** -7) * (second + tol) * (512 + live * I / 12) * 2.0 ** -22
    tol += (np.abs(R) + tol) * HALF_UNIT[kind] + HALF_TINY[kind]
    got = y.cpu().double().numpy()
    bad = ~(np.abs(got - R) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {np.argwhere(bad)[0]}: {got[bad][0]} for {R[bad][0]}"


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,I,E,top,group", [
    (1, 500, 1, 8, 4, 32), (1, 256, 300, 4, 2, 128), (2, 700, 1, 3, 3, 32), (2, 512, 2, 40, 8, 64), (4, 600, 1, 30, 2, 64),
    (9, 333, 3, 7, 2, 64), (16, 512, 257, 33, 4, 64), (40, 512, 1, 4, 2, 128), (64, 300, 2, 9, 3, 32), (70, 96, 40, 9, 3, 64),
    (130, 40, 1, 2, 2, 32), (3, 512, 1100, 4, 1, 256)])
def test_gated_activations_are_not_rounded_to_16_bits(pd, T, H, I, E, top, group, kind):
    """Few activations to a sum: the rounding of one would show beside that of y."""
    for n, s_kind in enumerate(("f32", kind)):
        what = f"T {T} H {H} I {I} E {E} top {top} group {group} {kind} scales {s_kind}"
        gu.note(what)
        x, xv, w, d13, d2 = layer(T, H, I, E, group, 40 + T + n, kind, s_kind)
        rng = np.random.default_rng(n)
        ids = np.stack([rng.permutation(E)[:top] for _ in range(T)])
        weights = rng.uniform(0.05, 1.0, (T, top)).astype(np.float32)
        y = pd.moe_a16_i4(x, torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(weights).cuda(), *w, group)
        check_wide(y, xv, ids, weights.astype(np.float64), d13, d2, kind, what)


@pytest.mark.parametrize("T", [1, 2, 5, 40])
def test_large_gated_activations_of_f16_stay_finite(pd, T):
    """Gates and up projections of some hundreds, whose product passes 65504, and second weights that bring it back."""
    H, I, E, top, group = 256, 160, 4, 2, 64
    x, xv, w, (d13, m13), (d2, m2) = layer(T, H, I, E, group, 3, "f16", "f32")
    w[1].mul_(2.0 ** 9)
    w[3].mul_(2.0 ** -12)
    d13, m13 = ([2.0 ** 9 * d for d in ds] for ds in (d13, m13))
    d2, m2 = ([2.0 ** -12 * d for d in ds] for ds in (d2, m2))
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:top] for _ in range(T)])
    weights = rng.uniform(0.2, 1.0, (T, top))
    weights = weights.astype(np.float32)
    largest = max(np.abs(d13[e][:I] @ xv[t] * (d13[e][I:] @ xv[t])).max() for t in range(T) for e in ids[t])
    assert largest > 2 * 65504
    y = pd.moe_a16_i4(x, torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(weights).cuda(), *w, group)
    assert torch.isfinite(y).all()
    check_wide(y, xv, ids, weights.astype(np.float64), (d13, m13), (d2, m2), "f16", f"T {T}")


def test_gated_activations_near_the_largest_binary32(pd):
    """One activation a token, the largest near binary32's largest and past bfloat16's."""
    T, H, I, E = 6, 32, 1, 1
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 1.0
    x[:, 1] = torch.tensor([1.0, 0.5, 1.0 - 2.0 ** -8, 2.0 ** -60, 2.0 ** -120, -1.0])
    c13, s13 = np.zeros((1, 2, H), np.int64), np.zeros((1, 1, 2), np.float32)
    c13[0, 0, 0], c13[0, 1, 1] = 7, 1                   # gate from x0, up projection from x1
    s13[0, 0] = 2.0 ** 40 / 7 * (1 + 2.0 ** -20), 2.0 ** 88 * (1 - 2.0 ** -15)
    c2, s2 = np.arange(-8, 8).repeat(2).reshape(1, H, 1), np.full((1, 1, H), 2.0 ** -100, np.float32)
    d13 = [i4.values(c13[0], s13[0].astype(np.float64), 32)]
    d2 = [i4.values(c2[0], s2[0].astype(np.float64), 32)]
    gate, up = d13[0] @ x.double().numpy().T
    assert 2.0 ** 128 * (1 - 2.0 ** -9) < gate[0] * up[0] < 2.0 ** 128 * (1 - 2.0 ** -16)   # bfloat16 rounds it up
    w13 = torch.zeros(1, 2, 16, dtype=torch.uint8)
    w13[:] = torch.from_numpy(i4.pack(c13))
    w2 = torch.zeros(1, H, 16, dtype=torch.uint8)
    w2[:, :, :1] = torch.from_numpy(i4.pack(c2))
    for rows in (1, 2, T):
        ids, weights = np.zeros((rows, 1), np.int64), np.ones((rows, 1), np.float32)
        y = pd.moe_a16_i4(x[:rows].cuda(), torch.zeros(rows, 1, dtype=torch.int32, device="cuda"), torch.ones(rows, 1, device="cuda"),
                          w13.cuda(), torch.from_numpy(s13).cuda(), w2.cuda()[:, :, :1], torch.from_numpy(s2).cuda(), 32)
        assert torch.isfinite(y).all()
        # (the bound's magnitudes are the scales', at every k: a code of zero enters with its bias, so that beside x0 = 1 an
        # x1 of 2^-60 is below half a unit of the sum 24 x0, 2^-20)
        m13, m2 = [np.repeat(s13[0].T.astype(np.float64), H, axis=1)], [np.full_like(d2[0], 2.0 ** -100)]
        check_wide(y, x[:rows].double().numpy(), ids, weights.astype(np.float64), (d13, m13), (d2, m2), "bf16", f"{rows} rows", 2.0 ** -15)


def test_infinite_gated_activations_reach_their_own_rows(pd):
    """A first product that overflows binary32: its token's results are not finite, the others keep their bits."""
    T, H, I, E, group = 20, 160, 96, 3, 32
    x, xv, w, d13, d2 = layer(T, H, I, E, group, 9, "bf16", "f32")
    ids = torch.from_numpy(np.random.default_rng(2).integers(0, E, (T, 2)).astype(np.int32)).cuda()
    ones = torch.ones(T, 2, device="cuda")
    want = pd.moe_a16_i4(x, ids, ones, *w, group)
    x[7, 3] = 3e38
    got = pd.moe_a16_i4(x, ids, ones, *w, group)
    keep = [t for t in range(T) if t != 7]
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[7]).any()


def c_call(pd, x, ids, weights, w, group, y, ws, ws_bytes):
    T, H = x.shape
    w13, s13, w2, s2 = w
    E, I = w13.shape[0], w13.shape[1] // 2
    kinds = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    return pd.lib.pdgemm_moe_a16_i4(T, H, I, E, ids.shape[1], x.data_ptr(), x.stride(0), kinds[x.dtype], ids.data_ptr(),
                                    weights.data_ptr(), *pd._moe_weights(w13, s13, E, 2 * I, H, group, "w13"),
                                    *pd._moe_weights(w2, s2, E, H, I, group, "w2"), kinds[s13.dtype], group, y.data_ptr(), y.stride(0),
                                    ws.data_ptr(), ws_bytes, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("T,E,top", [(1, 5, 3), (2, 5, 3), (12, 40, 4), (30, 4, 2)])
def test_the_workspace_says_which_form(pd, T, E, top, kind):
    """Of the narrow size and up to the wide one, the activations are rounded to the type and nothing past the size given
    is written; of the wide size and more, they are not.  The binding takes the wide size alone."""
    H, I, group = 200, 100, 32
    what = f"T {T} {kind}"
    gu.note(what)
    x, xv, w, d13, d2 = layer(T, H, I, E, group, 5, kind, "f32")
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:top] for _ in range(T)])
    weights = rng.uniform(0.2, 1.0, (T, top)).astype(np.float32)
    on = torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(weights).cuda()
    least, wide = pd.lib.pdgemm_moe_a16_i4_workspace_size(T, H, I, E, top), pd.moe_a16_i4_workspace_size(T, H, I, E, top)
    want = pd.moe_a16_i4(x, *on, *w, group)
    for size in (least, wide - 16, wide, wide + 4096):
        ws = torch.full((wide + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        buf = torch.full((T + 2, H + 3), -777.0, dtype=TYPES[kind], device="cuda")
        y = buf[1:-1, :H]
        assert c_call(pd, x, *on, w, group, y, ws, size) == 0
        assert (ws[size:] == 0xA5).all(), what
        check_layer(buf, True, xv, ids, weights.astype(np.float64), d13, d2, kind, f"{what} workspace {size}")
        if size >= wide:
            assert torch.equal(y, want), what
    assert c_call(pd, x, *on, w, group, torch.empty_like(want), ws, least - 16) == -7
    with pytest.raises(pd.PdgemmError, match="workspace"):
        pd.moe_a16_i4(x, *on, *w, group, workspace=ws[:wide - 16])
    assert torch.equal(pd.moe_a16_i4(x, *on, *w, group, workspace=ws[:wide]), want)
