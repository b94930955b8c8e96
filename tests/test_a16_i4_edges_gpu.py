"""GPU tests of products with group-scaled INT4 weights, and of the expert layer, at the ends of their ranges."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.int4 as i4
from tests import gpu_util as gu
from tests.test_a16_i4_gpu import activations, placed_activations, placed_codes, weights
from tests.test_moe_gpu import check_layer, layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_dense_gemm_amd as pd
    yield pd
    torch.cuda.empty_cache()


# ---- the scale of a value beside a border of two very long groups ----
#
# The longest rows of 16-bit activations, 2^21 values, in two groups; the quotient of the first group's last block of 32
# was 1 with a reciprocal of 31 bits.  One value of a row is 1: its weight comes back exactly.

LONG = [32 * 46779, 32 * 46410, 32 * 46568]     # of multiples of 32, 64 and 128 values


def one_hot_rows(K, group):
    at = [group - 1, group, group - 32, 0, K - 1]
    x = torch.zeros(len(at), K, dtype=torch.bfloat16, device="cuda")
    for row, k in enumerate(at):
        x[row, k] = 1.0
    return at, x


@pytest.mark.parametrize("group", LONG)
def test_scales_of_very_long_groups(pd, group):
    K, N = 1 << 21, 3
    at, x = one_hot_rows(K, group)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    codes |= 0x11                                               # (no code of zero)
    scales = torch.tensor([[1.0, 2.0, 4.0], [16.0, 32.0, 64.0]], device="cuda")
    want = np.empty((len(at), N))
    for row, k in enumerate(at):
        nibble = codes[:, k // 2].cpu().numpy().astype(int) >> (4 * (k % 2)) & 15
        want[row] = np.where(nibble > 7, nibble - 16, nibble) * scales[k // group].cpu().numpy()
    for cfg in range(pd.a16_i4_num_configs() - (1 if group % 128 else 0)):
        gu.note(f"group {group} cfg {cfg}")
        got = pd.gemm_a16_i4(x, codes, scales, group, cfg=cfg)
        assert np.array_equal(got.cpu().double().numpy(), want), cfg


@pytest.mark.parametrize("group", LONG)
def test_experts_scales_of_very_long_groups(pd, group):
    """The first product's rows that long: gates of 1, up projections of the groups' scales, every column of the second
    product's code 1.  (The second product's rows end at 2^20 values, half the longest row of scales.)"""
    H, I = 1 << 21, 1
    at, x = one_hot_rows(H, group)
    w13 = torch.full((1, 2, H // 2), 0x11, dtype=torch.uint8, device="cuda")
    s13 = torch.tensor([[[1.0, 2.0], [1.0, 32.0]]], dtype=torch.bfloat16, device="cuda")
    w2 = torch.ones(1, H, 16, dtype=torch.uint8, device="cuda")[:, :, :1]
    s2 = torch.ones(1, 1, H, dtype=torch.bfloat16, device="cuda")
    for rows in (1, 2, len(at)):
        y = pd.moe_a16_i4(x[:rows], torch.zeros(rows, 1, dtype=torch.int32, device="cuda"), torch.ones(rows, 1, device="cuda"),
                          w13, s13, w2, s2, group)
        up = torch.tensor([2.0 if k < group else 32.0 for k in at[:rows]], dtype=torch.float64)
        want = up / (1 + np.exp(-1.0))                          # (two groups differ 16 times; one rounding, 2^-8)
        assert torch.allclose(y.cpu().double(), want[:, None].expand(rows, H), rtol=2.0 ** -8 + 2.0 ** -14, atol=0), rows


def test_routing_of_tokens_past_a_launch_of_32_bits(pd):
    """More tokens than 2^32 work-items have, 64 to a token."""
    T = (1 << 26) + 3
    logits = torch.zeros(T, 2, dtype=torch.float16, device="cuda")
    logits[::2, 1] = 1.0
    logits[-1] = torch.tensor([0.0, 2.0])
    ids, weights = pd.moe_route(logits, 1, normalize=False)
    assert (ids[:-1:2] == 1).all() and (ids[1:-1:2] == 0).all() and ids[-1, 0] == 1
    few, share = pd.moe_route(torch.cat([logits[:2], logits[-1:]]), 1, normalize=False)
    assert torch.equal(weights[-1], share[2]) and (weights[:-1:2] == share[0]).all() and (weights[1:-1:2] == share[1]).all()


# ---- offsets of more than 32 bits ----

FAR = 1100          # rows of 4 MiB: the last ones begin past 2^32 bytes


def within(got, R, A, K, what):
    """The bound of every configuration (its derivation: test_a16_i4_gpu.py)."""
    err = np.abs(got.cpu().double().numpy() - R)
    assert (err <= (512 + K / 12) * 2.0 ** -22 * A).all(), what


def test_activations_and_results_past_32_bits(pd):
    N, K, group = 40, 200, 128
    codes, scales, w, m = weights(N, K, group, 1, "f32")
    a, av = activations(FAR, K, 2, "bf16")
    wide = torch.full((FAR, 1 << 21), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = a
    out = torch.full((FAR, 1 << 20), -777.0, device="cuda")
    R, A = i4.product(av, w)[0], np.abs(av) @ m.T
    for cfg in [None, *range(pd.a16_i4_num_configs())]:
        gu.note(f"cfg {cfg}")
        out[:, :N] = -777.0
        pd.gemm_a16_i4(wide[:, :K], placed_codes(codes), scales.cuda(), group, out=out[:, :N], cfg=cfg)
        within(out[:, :N], R, A, K, cfg)
        assert (out[:, N] == -777.0).all()


def test_codes_past_32_bits(pd):
    N, K, group = FAR, 200, 128
    codes, scales, w, m = weights(N, K, group, 3, "bf16")
    wide = torch.full((N, 1 << 22), 0x77, dtype=torch.uint8, device="cuda")
    wide[:, :K // 2] = torch.from_numpy(i4.pack(codes))
    for M in (3, 40):
        a, av = activations(M, K, 4, "f16")
        R, A = i4.product(av, w)[0], np.abs(av) @ m.T
        for cfg in [None, *range(pd.a16_i4_num_configs())]:
            gu.note(f"M {M} cfg {cfg}")
            within(pd.gemm_a16_i4(placed_activations(a), wide[:, :K // 2], scales.cuda(), group, cfg=cfg), R, A, K, (M, cfg))


def test_scales_past_32_bits(pd):
    N, group = 40, 32
    K = group * FAR - 5
    codes, scales, w, m = weights(N, K, group, 5, "f32")
    wide = torch.full((FAR, 1 << 20), float("nan"), device="cuda")
    wide[:, :N] = scales
    for M in (1, 3, 40):
        a, av = activations(M, K, 6, "bf16")
        R, A = i4.product(av, w)[0], np.abs(av) @ m.T
        for cfg in [None, *range(pd.a16_i4_num_configs() - 1)]:
            gu.note(f"M {M} cfg {cfg}")
            within(pd.gemm_a16_i4(placed_activations(a), placed_codes(codes), wide[:, :N], group, cfg=cfg), R, A, K, (M, cfg))


@pytest.mark.parametrize("T", [1, 2, 12, FAR])
def test_experts_past_32_bits(pd, T):
    """Experts 2.2 GB apart in codes and in scales of both products; rows of y 4 MiB apart."""
    H, I, E, group, apart = 96, 40, 3, 32, 2_200_000_000
    x, xv, w, d13, d2 = layer(T, H, I, E, group, 7, "bf16", "f32")
    far = []
    for t in w:
        size, (n, k) = t.element_size(), t.shape[1:]
        ld = gu.round_up(k, 16)
        buf = torch.empty((E - 1) * apart + n * ld * size, dtype=torch.uint8, device="cuda").view(t.dtype)
        view = buf.as_strided((E, n, k), (apart // size, ld, 1))
        view.copy_(t)
        far.append(view)
    ids = (np.arange(T)[:, None] + np.array([[2, 1]])) % E
    weights = np.random.default_rng(T).uniform(0.2, 1.0, (T, 2)).astype(np.float32)
    out = torch.full((T, 1 << 21), -777.0, dtype=torch.bfloat16, device="cuda")
    pd.moe_a16_i4(x, torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(weights).cuda(), *far, group, out=out[:, :H])
    check_layer(out[:, :H], False, xv, ids, weights.astype(np.float64), d13, d2, "bf16", f"T {T}")
    assert (out[:, H] == -777.0).all()


# ---- the tile kernel's own bound ----

@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("cfg", range(6, 11))
def test_tile_kernel_within_its_own_bound(pd, cfg, kind):
    """No code of the tile kernel enters with a bias.  With B the sum of |a code scale|: the one to four matrix instructions
    of a scale's sum add 32 products each, to within 2^-22 of the magnitudes they add: 4 * 2^-22 B.  A step of 128 values
    takes at most four multiply-adds, K / 32 + 8 in all (units are 256 values), each half a unit of a sum below B, so
    (K / 128 + 2) * 2^-22 B; up to 4 groups' and 16 splits' sums, 5 * 2^-22 B more.  (12 + K / 128) * 2^-22 B bounds them, a
    fortieth of the bound that holds for every configuration."""
    for n, (M, N, K, group) in enumerate([(16, 64, 256, 64), (33, 130, 640, 128), (67, 70, 1337, 96), (65, 100, 2048, 256), (1, 40, 31, 32),
                                          (130, 33, 5000, 160), (260, 270, 1500, 128), (37, 65, 8192, 32), (129, 513, 257, 256)]):
        if cfg == pd.a16_i4_num_configs() - 1 and group % 128:
            continue
        gu.note(f"{M}x{N}x{K} group {group} {kind} cfg {cfg}")
        a, av = activations(M, K, 30 + n, kind)
        codes, scales, w, _ = weights(N, K, group, 60 + n, ("f32", kind)[n % 2])
        R, B = i4.product(av, w)
        got = pd.gemm_a16_i4(placed_activations(a), placed_codes(codes), scales.cuda(), group, cfg=cfg).cpu().double().numpy()
        bad = ~(np.abs(got - R) <= (12 + K / 128) * 2.0 ** -22 * B)
        assert not bad.any(), (M, N, K, group, int(bad.sum()), float((np.abs(got - R) / B).max() * 2.0 ** 22))
