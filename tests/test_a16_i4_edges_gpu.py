"""GPU tests of products with group-scaled INT4 weights, and of the expert layer, at the ends of their ranges."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.int4 as i4
from tests import gpu_util as gu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_dense_gemm_amd as pd
    return pd


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
