"""CPU checks of size queries and choices of the norm, INT4-weight and expert operators at the ends of their ranges."""
from __future__ import annotations

import os

import pytest

from tests.test_abi_cpu import LIB

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libpdgemm.so not built")


@pytest.fixture(scope="module")
def pd():
    pytest.importorskip("torch")
    import precision_dense_gemm_amd as pd
    return pd


def test_the_wide_workspace_holds_the_activations_twice(pd):
    for T, H, I, E, top in [(1, 1, 1, 1, 1), (5, 96, 60, 8, 2), (16, 2048, 768, 128, 8), (4096, 8, 100, 3, 1), (64, 64, 2 ** 16, 1024, 64)]:
        least = pd.lib.pdgemm_moe_a16_i4_workspace_size(T, H, I, E, top)
        wide = pd.lib.pdgemm_moe_a16_i4_wide_workspace_size(T, H, I, E, top)
        assert least > 0 and wide == least + T * top * ((2 * I + 15) // 16 * 16)
        assert pd.moe_a16_i4_workspace_size(T, H, I, E, top) == wide
    for sizes in [(0, 96, 64, 8, 2), (-1, 96, 64, 8, 2), (5, 96, 64, 2000, 2), (5, 0, 64, 8, 2), (5, 96, 64, 8, 0), (5, 96, 64, 8, 65)]:
        assert pd.lib.pdgemm_moe_a16_i4_wide_workspace_size(*sizes) == 0


def test_a_choice_for_empty_and_refused_sizes(pd):
    """(a quotient by their tiles would end the process)"""
    for M in (-2 ** 62, -33, -1, 0, 1, 16, 17, 32, 500, 2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 62):
        for N in (-2 ** 62, -7, 0, 1, 4096, 2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 62):
            for K in (-1, 0, 1, 8192, 2 ** 30, 2 ** 62):
                for group in (-32, 0, 32, 128, 2 ** 62):
                    c = pd.a16_i4_pick(M, N, K, group)
                    assert 0 <= c < pd.a16_i4_num_configs(), (M, N, K, group)
                    if M <= 0 or N <= 0 or K < 0 or max(M, N) >= 2 ** 31 or K > 2 ** 30:
                        assert c == 0 and pd.a16_i4_workspace_size(M, N, K, group) == 0
                    for cfg in (-1, 0, 8, 10, 11):
                        assert pd.a16_i4_workspace_size(M, N, K, group, cfg) >= 0


def test_rows_without_values_need_no_pointers(pd):
    """(the scales of a norm to INT8 are set where they are given, so their alignment is looked at)"""
    def norm(out_type, scale):
        return pd.lib.pdgemm_rms_norm(5, 0, None, 0, 2, None, 0, None, 0, None, 2, 1e-5, None, 0, out_type, scale, None)
    assert norm(0, 0x10002) == 0 and norm(3, None) == 0 and norm(3, 0x10002) == -5
