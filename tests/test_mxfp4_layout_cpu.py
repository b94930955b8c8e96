"""The MXFP4 kernels' layouts, restated: LDS placement, fragment reads, the shares of K, result
registers, the quantiser's exchange, and the tile choices."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest

from tests.test_abi_cpu import LIB
from tests.test_layout_cpu import extra_cycles, swizzle16, swizzle8

LANES = range(64)


def swizzle_bf16(r):
    return (r & 7) ^ ((r >> 3) & 1)


@pytest.mark.parametrize("rows,wave_rows", [(256, 128), (256, 64), (128, 64)])
def test_tile_rows_interleave_over_fragments(rows, wave_rows):
    # LDS row cr of an operand holds row cr / W * W + F (cr % 32) + cr % W / 32 of the tile (W rows
    # a wave, F = W / 32 fragments): fragment i of a wave, LDS rows 32 i + r, then holds rows F r + i
    F = wave_rows // 32
    held = [cr // wave_rows * wave_rows + F * (cr % 32) + cr % wave_rows // 32 for cr in range(rows)]
    assert sorted(held) == list(range(rows))
    for w0 in range(0, rows, wave_rows):
        for i in range(F):
            for r in range(32):
                assert held[w0 + 32 * i + r] == w0 + F * r + i
                # the lane's scales of its F fragments lie in one dword, fragment i in byte i of its share
                assert held[w0 + 32 * i + r] // 4 == (w0 + F * r) // 4
                assert held[w0 + 32 * i + r] % 4 == (F * r) % 4 + i


@pytest.mark.parametrize("F", [1, 2, 4])
def test_few_rows_interleave_over_fragments(F):
    held = [F * (cr % 16) + cr // 16 for cr in range(16 * F)]
    assert sorted(held) == list(range(16 * F))
    assert all(held[16 * i + r] == F * r + i for i in range(F) for r in range(16))


def test_fragment_reads_have_no_bank_conflicts():
    for base in range(0, 512, 32):
        for s in range(4):       # 32 x 32 tiles: lane l reads row l % 32, chunk 2 s + l / 32
            assert extra_cycles(lambda l: (base + l % 32, 2 * s + l // 32), swizzle8) == 0
    for base in range(0, 256, 16):
        for u in (0, 1):
            # few rows and f16 activations: chunk 4 u + l / 16 (bf16 activations read chunk
            # 2 (l / 16) + u, whose swizzle was chosen by the counters of four)
            assert extra_cycles(lambda l: (base + l % 16, 4 * u + l // 16), swizzle16) == 0
    for r in range(64):
        assert sorted(c ^ swizzle_bf16(r) for c in range(8)) == list(range(8))
        # a wave's copies are whole 16-row groups apart, and take one chunk offset for all
        assert swizzle_bf16(r) == swizzle_bf16(r % 16) and swizzle16(r) == swizzle16(r % 16)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_a16_shares_of_a_step(kind):
    # MFMA u, lane group g: eight values of A (a 16-byte chunk) and one dword of B's codes, which
    # have to be the same values of K; every value of the 64 once
    seen = []
    for u in (0, 1):
        for g in range(4):
            if kind == "bf16":
                a = 8 * (2 * g + u)
                block, dword = g >> 1, 2 * (g & 1) + u
            else:
                a = 8 * (4 * u + g)
                block, dword = u, g
            assert 32 * block + 8 * dword == a
            seen += range(a, a + 8)
    assert sorted(seen) == list(range(64))


@pytest.mark.parametrize("FM,FN", [(4, 2), (2, 2)])
def test_tile_results_cover_the_wave_tile(FM, FN):
    cells = [(FM * (8 * (e // 4) + 4 * (l // 32) + e % 4) + i, FN * (l % 32) + j)
             for l in LANES for i in range(FM) for j in range(FN) for e in range(16)]
    assert sorted(cells) == [(r, c) for r in range(32 * FM) for c in range(32 * FN)]


@pytest.mark.parametrize("FM,FN,mixed", [(1, 1, True), (2, 4, True), (4, 4, True), (1, 4, False), (3, 2, False)])
def test_join_reads_every_partial_sum(FM, FN, mixed):
    # written: register e of lane l in block (i, j); read back by row and column of the tile
    written = {}
    for i in range(FM):
        for j in range(FN):
            for e in range(4):
                for l in LANES:
                    rr = 4 * (l // 16) + e
                    cell = (FM * rr + i if mixed else 16 * i + rr, FN * (l % 16) + j)
                    written[((i * FN + j) * 4 + e) * 64 + l] = cell
    for x in range(16 * FM * 16 * FN):
        row, n, j = x // (16 * FN), x % (16 * FN) // FN, x % FN
        i, rr = (row % FM, row // FM) if mixed else (row // 16, row % 16)
        assert written[((i * FN + j) * 4 + (rr & 3)) * 64 + (rr >> 2) * 16 + n] == (row, FN * n + j)


def test_quantiser_exchange_leaves_two_rows_a_lane():
    # each step a lane keeps the half of its rows that its bit names, against its partner's
    rng = np.random.default_rng(3)
    start = rng.integers(0, 1 << 31, (16, 32))
    v = [list(map(int, row)) for row in start]
    for n, bit, partner in ((16, 8, lambda l: 15 - l), (8, 4, lambda l: l ^ 7), (4, 2, lambda l: l ^ 2), (2, 1, lambda l: l ^ 1)):
        give = [[v[l][p] if l & bit else v[l][p + n] for p in range(n)] for l in range(16)]
        keep = [[v[l][p + n] if l & bit else v[l][p] for p in range(n)] for l in range(16)]
        assert all((partner(l) & bit) != (l & bit) for l in range(16))
        v = [[max(keep[l][p], give[partner(l)][p]) for p in range(n)] for l in range(16)]
    most = start.max(axis=0)
    assert all(v[l] == [most[2 * l], most[2 * l + 1]] for l in range(16))


@pytest.mark.skipif(not os.path.exists(LIB), reason="libpdgemm.so not built")
def test_tile_choices_are_configurations():
    L = ctypes.CDLL(LIB)
    i64 = ctypes.c_int64
    L.pdgemm_mxf4_pick.argtypes = [i64] * 3
    L.pdgemm_a16_mxf4_pick.argtypes = [ctypes.c_int] + [i64] * 3
    n_mx, n_a16 = L.pdgemm_mxf4_num_configs(), L.pdgemm_a16_mxf4_num_configs()
    rng = np.random.default_rng(9)
    taken = {"mx": set(), "f16": set(), "bf16": set()}
    shapes = [[int(2 ** rng.uniform(0, hi)) for hi in (14, 15, 14)] for _ in range(4000)]
    for M, N, K in shapes + [[1, 1, 0], [2 ** 22, 2 ** 22, 2 ** 23], [2 ** 31 - 1, 1, 8]]:
        taken["mx"].add(L.pdgemm_mxf4_pick(M, N, K))
        taken["f16"].add(L.pdgemm_a16_mxf4_pick(1, M, N, K))
        taken["bf16"].add(L.pdgemm_a16_mxf4_pick(2, M, N, K))
    # every configuration serves some call, and no other number is returned
    assert taken["mx"] == set(range(n_mx))
    assert taken["f16"] | taken["bf16"] == set(range(n_a16))
    assert L.pdgemm_a16_mxf4_pick(0, 64, 64, 64) == -1
