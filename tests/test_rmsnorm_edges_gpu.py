"""GPU tests of the root-mean-square norm at the ends of its ranges."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.norm as rn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_dense_gemm_amd as pd
    yield pd
    torch.cuda.empty_cache()


def test_rows_of_one_value_past_a_launch_of_32_bits(pd):
    """More rows than 2^32 work-items have, sixteen to a row."""
    rows = (1 << 28) + 17
    x = torch.full((rows, 1), 2.0, dtype=torch.float16, device="cuda")
    x[1::2] = -0.5
    x[-3:] = torch.tensor([[1.0], [0.0], [-4.0]])
    w = torch.tensor([3.0], dtype=torch.float16, device="cuda")
    few = torch.cat([x[:2], x[-3:]])
    y, (q, scale) = pd.rms_norm(few, w, EPS), pd.rms_norm_i8(few, w, EPS)
    got, (gq, gs) = pd.rms_norm(x, w, EPS), pd.rms_norm_i8(x, w, EPS)
    for all_rows, of_few in ((got[:, 0], y[:, 0]), (gq[:, 0], q[:, 0]), (gs, scale)):
        assert torch.equal(all_rows[-3:], of_few[2:])
        assert (all_rows[:-3:2] == of_few[0]).all() and (all_rows[1:-3:2] == of_few[1]).all()


def test_workgroups_of_a_row_past_a_launch_of_32_bits(pd):
    """128 threads to a row, in place."""
    rows, cols, last = (1 << 25) + 5, 513, 100
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    x[-last:] = torch.randn(last, cols, device="cuda", generator=g).bfloat16()
    w = torch.randn(cols, device="cuda", generator=g).bfloat16()
    first, end = pd.rms_norm(x[:1], w, EPS), pd.rms_norm(x[-last:], w, EPS)
    pd.rms_norm(x, w, EPS, out=x)
    assert torch.equal(x[-last:], end)
    for part in x[:-last].split(1 << 21):
        assert (part == first).all()


def test_scales_of_rows_without_values(pd):
    """cols = 0: no code, and a scale for every row all the same (a product over K = 0 takes it)."""
    for rows in (1, 5, 300, 2_000_000):
        scale = torch.full((rows + 1,), float("nan"), device="cuda")
        x = torch.empty(rows, 0, dtype=torch.bfloat16, device="cuda")
        w = torch.empty(0, dtype=torch.bfloat16, device="cuda")
        q, s = pd.rms_norm_i8(x, w, EPS, out=(torch.empty(rows, 0, dtype=torch.int8, device="cuda"), scale[:rows]))
        assert q.shape == (rows, 0) and not s.any() and scale[rows].isnan()
        assert pd.rms_norm(x, w, EPS).shape == (rows, 0)
    assert pd.rms_norm_i8(x[:0], w, EPS)[1].shape == (0,)


@pytest.mark.parametrize("cols", [40, 300, 700, 5000, 20000])
def test_codes_of_rows_out_of_the_range_of_squares_under_weights_that_bring_them_back(pd, cols):
    """Squares below and above binary32's range, weights that make t = h w ordinary, small or large: the oracle's codes, and
    its scales to 44 units of 2^-24 (as in test_rmsnorm_gpu.py, 40, and the product with the power of two)."""
    rng = np.random.default_rng(cols)
    for row, weight in ((-52, 120), (-52, 40), (-60, 60), (-75, 20), (60, -122), (60, -60), (75, -30), (100, 20), (120, -120)):
        # (values of magnitude 1/2 to 2, so that all of t are normal)
        h, w = (np.ldexp(rng.uniform(0.5, 2.0, n) * rng.choice([-1.0, 1.0], n), e).astype(np.float32) for n, e in
                (((3, cols), row), (cols, weight)))
        q, scale = pd.rms_norm_i8(torch.from_numpy(h).cuda(), torch.from_numpy(w).cuda(), 0.0)
        want, s = rn.codes(h.astype(np.float64), w.astype(np.float64), 0.0)
        assert np.isfinite(s).all() and np.array_equal(q.cpu().numpy(), want.astype(np.int8)), (row, weight)
        assert (np.abs(scale.cpu().double().numpy() - s) <= 44 * 2.0 ** -24 * s + 2.0 ** -149).all(), (row, weight)


def test_rows_past_32_bits_keep_their_bits(pd):
    """Rows 4 MiB apart, the last ones past 2^32 bytes: norm, codes and gradients as of the same rows beside each other."""
    rows, cols = 1100, 300
    g = torch.Generator("cuda").manual_seed(3)
    x, r, dy, dh = (torch.randn(rows, cols, device="cuda", generator=g) for _ in range(4))
    w = torch.randn(cols, device="cuda", generator=g)

    def far(t, dtype=torch.float32):
        buf = torch.empty(rows, (1 << 22) // torch.empty(0, dtype=dtype).element_size(), dtype=dtype, device="cuda")
        if t is not None:
            buf[:, :cols] = t
        return buf[:, :cols]

    y, h = pd.rms_norm(x, w, EPS, residual=r)
    fy, fh = pd.rms_norm(far(x), w, EPS, residual=far(r), out=far(None), sum_out=far(None))
    assert torch.equal(y, fy) and torch.equal(h, fh)
    q, s = pd.rms_norm_i8(x, w, EPS)
    fq, fs = pd.rms_norm_i8(far(x), w, EPS, out=(far(None, torch.int8), torch.empty_like(s)))
    assert torch.equal(q, fq) and torch.equal(s, fs)
    dx, dw = pd.rms_norm_backward(dy, h, w, EPS, dh=dh)
    fdx, fdw = pd.rms_norm_backward(far(dy), fh, w, EPS, dh=far(dh), out=far(None))
    assert torch.equal(dx, fdx) and torch.equal(dw, fdw)
