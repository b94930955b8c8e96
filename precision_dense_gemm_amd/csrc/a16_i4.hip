// a16_i4.hip -- products of 16-bit activations with group-scaled INT4 weights for gfx950
// (MI355X), behind the C ABI declared in include/pdgemm.h.
#include "i4_core.h"

namespace {

struct A16I4Args {
    const uint8_t *A;
    const uint8_t *B;
    void *C;
    float *part;        // the splits' sums, M x N each
    I4Scales s;
    int64_t lda, ldb;   // bytes
    int64_t ldc;        // elements
    int M, N, K;
    int tiles_m, tiles_n;
    int splits;
    int group, out_type;
    uint32_t group_magic;
};

__device__ __forceinline__ void store_as(void *C, int type, int64_t at, float v) {
    if (type == kF32)
        static_cast<float *>(C)[at] = v;
    else if (type == kF16)
        static_cast<_Float16 *>(C)[at] = (_Float16)v;
    else
        static_cast<__bf16 *>(C)[at] = (__bf16)v;
}
// the first n of N neighbours
template <int N>
__device__ __forceinline__ void store_as(void *C, int type, int64_t at, const float (&v)[N], int n) {
    if (type == kF32) {
        store_some<N>(static_cast<float *>(C) + at, v, n);
    } else if (type == kF16) {
        _Float16 e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = (_Float16)v[i];
        store_some<N>(static_cast<_Float16 *>(C) + at, e, n);
    } else {
        __bf16 e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = (__bf16)v[i];
        store_some<N>(static_cast<__bf16 *>(C) + at, e, n);
    }
}

// Few rows: a tile of RA rows and 16 NT columns of C to a workgroup, K split over its W waves,
// whose sums meet in LDS and are added in wave order.  The stream of the codes bounds it: one row of
// bf16 against 8192 x 8192 in groups of 128 takes 8.4 us, 34.6 MB at 4.1 TB/s with the launch's start and end, 8 rows
// 10.3, 16 rows 11.4, one row against 4096 x 4096 4.3 to 4.6.
template <int T, int RA, int NT, int W, int Q, bool kS32, bool kAhead>
__global__ __launch_bounds__(W *kWave) void a16_i4_few_kernel(A16I4Args args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Wave = I4Wave<T, RA, NT, 1, Q, kS32, kAhead>;
    constexpr int kTile = NT * 256;
    __shared__ union {
        typename Wave::Lds wave[W];
        float part[W][kTile];
    } lds;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int m0 = (blockIdx.x / args.tiles_n) * RA, n0 = (blockIdx.x % args.tiles_n) * 16 * NT;
    const int M = args.M, N = args.N, K = args.K;

    typename Wave::Source src;
    src.a = args.A + (int64_t)m0 * args.lda;
    src.a_end = (int)((min(RA, M - m0) - 1) * args.lda) + ((2 * K + 15) & ~15);
    src.b[0] = args.B + (int64_t)n0 * args.ldb;
    src.b_end[0] = (int)((min(16 * NT, N - n0) - 1) * args.ldb) + (((K + 1) / 2 + 15) & ~15);
#pragma unroll
    for (int j = 0; j < Wave::kX; ++j) {
        const int row = Wave::copied_row(j);
        src.xa[j] = row < RA && row < M - m0 ? (uint32_t)row * (uint32_t)args.lda + 16 * Wave::copied_chunk() : kOutside;
    }
    const int size = kS32 ? 4 : 2;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = 16 * t + Wave::code_row();
        src.vb[t] = row < N - n0 ? (uint32_t)row * (uint32_t)args.ldb + 16 * Wave::code_chunk() : kOutside;
        src.vs[t] = (uint32_t)(n0 + min(16 * t + lane % 16, N - n0 - 1)) * size;
    }
    src.s[0] = args.s;
    src.K = K, src.group_magic = args.group_magic, src.groups = (K + args.group - 1) / args.group;

    // The workgroups of an XCD begin at different places of their rows, or all of them would ask
    // the same memory channels at a time where a row is a power of two long.
    const int units = (K + 2 * kStep - 1) / (2 * kStep);
    const int turned = units > 0 ? (int)(blockIdx.x / 8 * W % units) : 0;
    int next = wave;
    Wave w;
    w.run(
        src, lds.wave[wave],
        [&](auto &, auto &) {
            if (next >= units) return -1;
            const int unit = next + turned;
            next += W;
            return unit < units ? unit : unit - units;
        },
        [](auto &) {});
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) lds.part[wave][(t * 4 + e) * kWave + lane] = w.acc[t][e];
    __syncthreads();
    // fragment t holds, in register e of lane l, row 4 (l / 16) + e and column 16 t + l % 16
    for (int x = tid; x < RA * 16 * NT; x += W * kWave) {
        const int row = x / (16 * NT), col = x % (16 * NT);
        if (m0 + row >= M || n0 + col >= N) continue;
        const int at = (col / 16 * 4 + row % 4) * kWave + row / 4 * 16 + col % 16;
        float sum = lds.part[0][at];
#pragma unroll
        for (int v = 1; v < W; ++v) sum += lds.part[v][at];
        store_as(args.C, args.out_type, (int64_t)(m0 + row) * args.ldc + n0 + col, sum);
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// Chunk c (16 bytes) of row r of a step of activations lies at c ^ turn_of(r).  The LDS takes a wave's 16-byte reads in
// four turns of 16 lanes, of which four by four rows have the same lane group g and the others the next one,
// whose chunk differs by 1 or 4: the turns keep all sixteen in different banks for either (r % 8 in its place: 2048 x
// 8192 x 8192 3 to 6% slower).
__device__ __forceinline__ int turn_of(int r) { return (r & 3) | (r >> 1 & 4) | ((r << 1 ^ r) & 8); }

// More rows: a tile of 16 MT rows to a workgroup, whose W waves have 16 NT columns each, so that a
// code is converted once per tile.  Activations go through LDS, a step of 128 values of K at a time
// and two deep, for all waves; codes are loaded whole lines to four lanes, a unit of 256 values ahead,
// and pass through LDS to the lanes that convert them.  Fragment t holds columns NT n + t (n = l % 16) of
// the wave's: a lane's results are neighbours in C.  G such groups of W waves share out the units of K,
// and their sums meet in LDS.  With `splits`, K is split over that many workgroups too, which write
// binary32 sums for split_join_kernel; what they write and the second launch cost 37 x 4096 x 8192
// 7 of 19 us with 16 splits and G = 1, so G is 4 and 2 for the tiles of few rows (14.4 us).
// Up to some hundred rows the stream of codes bounds it.  Past that no unit is full: of the cycles of 2048 x 8192 x 8192
// the matrix instructions take 44%, vector instructions issue in as many (a code takes an instruction and a half, each sum
// of a scale's values a multiply-add), the LDS works in a third, and the two waves that a SIMD has between barriers
// overlap these little.  bf16 or f16 in groups of 128: 252 to 264 us in a steady stream of calls (290 to 340 for the
// first dozens after a pause, whose clock still rises), 1.04 to 1.09 PFLOP/s; of 64: 363 to 371 us; of 32: 464 to 485 us.
template <int T, int MT, int NT, int W, int G, int Q, bool kS32>
__global__ __launch_bounds__(G *W *kWave) void a16_i4_tile_kernel(A16I4Args args) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int BM = 16 * MT, BN = 16 * NT * W, kThreads = W * kWave;   // (threads of a group)
    constexpr int kX = BM * 16 / kThreads, kSc = 4 / Q;
    static_assert(BM * 16 % kThreads == 0, "a step of activations in whole runs");
    __shared__ union {
        uint4 xs[G][2][BM][16];
        float part[G][G == 1 ? 1 : BM * BN];
    } lds;
    __shared__ uint4 codes[G * W][2][NT][16][4];   // a unit's, each wave its own
    const int tid = threadIdx.x % kThreads, lane = tid % kWave;
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane % 16, g = lane / 16;
    const int M = args.M, N = args.N, K = args.K;
    const int tile = blockIdx.x / args.splits, split = blockIdx.x % args.splits;
    const int m0 = tile % args.tiles_m * BM, n0 = tile / args.tiles_m * BN + wave * 16 * NT;
    const int units = (K + 2 * kStep - 1) / (2 * kStep);
    const int first = (int)((int64_t)units * split / args.splits), last = (int)((int64_t)units * (split + 1) / args.splits);

    const uint8_t *const a = args.A + (int64_t)m0 * args.lda;
    const int a_end = (int)((min(BM, M - m0) - 1) * args.lda) + ((2 * K + 15) & ~15);
    const int cols = min(max(N - n0, 0), 16 * NT);   // (a wave may have no column)
    const uint8_t *const b = args.B + (int64_t)(cols > 0 ? n0 : 0) * args.ldb;
    const int b_end = cols > 0 ? (int)((cols - 1) * args.ldb) + (((K + 1) / 2 + 15) & ~15) : 0;
    uint32_t xa[kX], vb[NT], vs[NT];
#pragma unroll
    for (int j = 0; j < kX; ++j) {
        const int row = (tid + j * kThreads) / 16;
        xa[j] = row < M - m0 ? (uint32_t)row * (uint32_t)args.lda + 16 * (tid % 16) : kOutside;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = NT * r + t;
        const int copied = NT * (lane / 4) + t;
        vb[t] = copied < cols ? (uint32_t)copied * (uint32_t)args.ldb + 16 * (lane % 4) : kOutside;
        vs[t] = (uint32_t)(cols > 0 ? n0 + min(col, cols - 1) : 0) * (kS32 ? 4 : 2);
    }
    const int groups = (K + args.group - 1) / args.group;

    uint4 xr[kX];
    auto load_x = [&](int step) __attribute__((always_inline)) {
        const int left = step < 2 * last ? a_end - step * 256 : 0;
        const auto ra = rsrc(a + (int64_t)step * 256, left > 0 ? left : 0);
#pragma unroll
        for (int j = 0; j < kX; ++j) xr[j] = load16(ra, xa[j]);
    };
    auto store_x = [&](int step) __attribute__((always_inline)) {
        if (step * kStep + kStep > K) {
            // activations at and past K may be anything, a NaN too: they become zeros
            const int n = K - step * kStep - tid % 16 * 8;
            uint32_t m[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) m[d] = n >= 2 * d + 2 ? 0xFFFFFFFFu : n == 2 * d + 1 ? 0xFFFFu : 0u;
#pragma unroll
            for (int j = 0; j < kX; ++j) xr[j] = make_uint4(xr[j].x & m[0], xr[j].y & m[1], xr[j].z & m[2], xr[j].w & m[3]);
        }
#pragma unroll
        for (int j = 0; j < kX; ++j) {
            const int row = (tid + j * kThreads) / 16;
            lds.xs[group][step & 1][row][(tid % 16) ^ turn_of(row)] = xr[j];
        }
    };
    struct Codes {
        uint4 b[NT][2];
        uint32_t s[NT][2 * kSc];
    };
    auto load_codes = [&](Codes &c, int unit) __attribute__((always_inline)) {
        const int left = unit < last ? b_end - unit * 128 : 0;
        const auto rb = rsrc(b + (int64_t)unit * 128, left > 0 ? left : 0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            c.b[t][0] = load16(rb, vb[t]);
            c.b[t][1] = load16(rb, vb[t] + 64);
        }
#pragma unroll
        for (int u = 0; u < 2 * kSc; ++u) {
            const int q = I4Groups::of<Q>(unit * 8 + u * Q, args.group_magic, groups);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint8_t *const p = args.s.p + q * args.s.ld + vs[t];
                if constexpr (kS32)
                    c.s[t][u] = *reinterpret_cast<const uint32_t *>(p);
                else
                    c.s[t][u] = *reinterpret_cast<const uint16_t *>(p);
            }
        }
    };
    floatx4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[i][t] = floatx4_t{0, 0, 0, 0};

    if (first < last) {
        Codes next;
        // (a group past its last unit sums zeros until all are there)
        const int mine = first + group, turns = (last - first + G - 1) / G;
        load_codes(next, mine);
        load_x(2 * mine);
        store_x(2 * mine);
        load_x(2 * mine + 1);
        for (int i = 0; i < turns; ++i) {
            const int unit = mine + i * G;
            float scale[NT][2 * kSc];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int h = 0; h < 2; ++h) write_codes(codes[group * W + wave][h][t], next.b[t][h]);
#pragma unroll
                for (int v = 0; v < 2 * kSc; ++v) {
                    const float f = scale_value<kS32>(next.s[t][v], args.s.half);
                    scale[t][v] = unit * 2 * kStep + v * Q * kBlock < K && unit < last ? f * 16.0f : 0.0f;   // (no scale past K)
                }
            }
            load_codes(next, unit + G);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int step = 2 * unit + h;
                __syncthreads();
                store_x(h ? 2 * (unit + G) : step + 1);
                load_x(2 * (unit + G) + h);
                // the step's codes converted once, then four fragments of rows at a time, as the registers hold
                uint4 c[NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    uint32_t w[4];
                    read_codes<Q>(w, codes[group * W + wave][h][t]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) c[t][u] = widen<T>(w[u]);
                }
                constexpr int kRows = MT < 4 ? MT : 4;
#pragma unroll
                for (int i0 = 0; i0 < MT; i0 += kRows) {
                    uint4 x[kRows][4];
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            x[i][u] = lds.xs[group][h][16 * (i0 + i) + r][position<Q>(u, g) ^ turn_of(r)];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int v = 0; v < kSc; ++v) {
                            floatx4_t p[kRows];
#pragma unroll
                            for (int u = v * Q; u < v * Q + Q; ++u)
#pragma unroll
                                for (int i = 0; i < kRows; ++i)
                                    p[i] = mfma16<T>(x[i][u], c[t][u], u == v * Q ? floatx4_t{0, 0, 0, 0} : p[i]);
#pragma unroll
                            for (int i = 0; i < kRows; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    acc[i0 + i][t][e] = __builtin_fmaf(p[i][e], scale[t][h * kSc + v], acc[i0 + i][t][e]);
                        }
                }
            }
        }
    }
    float *const part = args.splits > 1 ? args.part + (int64_t)split * M * N : nullptr;
    if constexpr (G > 1) {
        constexpr int kTile = MT * NT * 256;   // of a wave
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) lds.part[group][wave * kTile + ((i * NT + t) * 4 + e) * kWave + lane] = acc[i][t][e];
        __syncthreads();
        // group k adds up every G-th fragment's row
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = m0 + 16 * i + 4 * g + e, n = cols - NT * r;
                if ((i * 4 + e) % G != group || row >= M || n <= 0) continue;
                float v[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int at = wave * kTile + ((i * NT + t) * 4 + e) * kWave + lane;
                    v[t] = lds.part[0][at];
#pragma unroll
                    for (int k = 1; k < G; ++k) v[t] += lds.part[k][at];
                }
                if (part)
                    store_some<NT>(part + (int64_t)row * N + n0 + NT * r, v, n);
                else
                    store_as<NT>(args.C, args.out_type, (int64_t)row * args.ldc + n0 + NT * r, v, n);
            }
        return;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = m0 + 16 * i + 4 * g + e;
            if (row >= M) continue;
            float v[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) v[t] = acc[i][t][e];
            const int n = cols - NT * r;
            if (n <= 0) continue;
            if (part)
                store_some<NT>(part + (int64_t)row * N + n0 + NT * r, v, n);
            else
                store_as<NT>(args.C, args.out_type, (int64_t)row * args.ldc + n0 + NT * r, v, n);
        }
#endif  // __HIP_DEVICE_COMPILE__
}


constexpr int kMaxSplits = 16;

// C from the splits' sums, added in their order.
__global__ __launch_bounds__(256) void split_join_kernel(A16I4Args args) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)args.M * args.N;
    if (x >= all) return;
    // (all loads before the first sum)
    float v[kMaxSplits], sum = 0;
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k) v[k] = k < args.splits ? args.part[k * all + x] : 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k)
        if (k < args.splits) sum += v[k];
    store_as(args.C, args.out_type, x / args.N * args.ldc + x % args.N, sum);
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// host side

// few: rows of a tile 2, 8 or 16; else 16 MT
struct Config {
    bool few;
    int rows, nt, waves, groups;
};
constexpr Config kConfigs[] = {{true, 2, 1, 8, 1},   {true, 2, 2, 8, 1},   {true, 8, 1, 8, 1},   {true, 8, 2, 8, 1},
                               {true, 16, 1, 8, 1},  {true, 16, 2, 8, 1},  {false, 32, 1, 4, 4}, {false, 48, 1, 4, 4},
                               {false, 64, 2, 4, 2}, {false, 64, 2, 8, 1}, {false, 128, 2, 8, 1}};
constexpr int kNumConfigs = sizeof(kConfigs) / sizeof(kConfigs[0]);
// The last one is for groups of whole steps: with more scales its values leave the registers (2048 x 8192 x 8192 of
// f16 in groups of 64 takes 806 us on it, 381 on the one before).
bool serves(int c, int64_t group) { return c < kNumConfigs - 1 || group % kStep == 0; }

template <int T, int C, int Q, bool kS32>
const void *a16_i4_ptr() {
    constexpr Config c = kConfigs[C];
    if constexpr (c.few)
        return reinterpret_cast<const void *>(&a16_i4_few_kernel<T, c.rows, c.nt, c.waves, Q, kS32, c.rows != 16>);
    else if constexpr (C == kNumConfigs - 1 && Q != 4)
        return nullptr;
    else
        return reinterpret_cast<const void *>(&a16_i4_tile_kernel<T, c.rows / 16, c.nt, c.waves, c.groups, Q, kS32>);
}
template <int T, int Q, int C = 0>
const void *a16_i4_ptr(int cfg, bool s32) {
    if constexpr (C < kNumConfigs)
        return cfg != C ? a16_i4_ptr<T, Q, C + 1>(cfg, s32) : s32 ? a16_i4_ptr<T, C, Q, true>() : a16_i4_ptr<T, C, Q, false>();
    return nullptr;
}
template <int T>
const void *a16_i4_ptr(int cfg, int group, bool s32) {
    return group % 128 == 0 ? a16_i4_ptr<T, 4>(cfg, s32)
           : group % 64 == 0 ? a16_i4_ptr<T, 2>(cfg, s32)
                             : a16_i4_ptr<T, 1>(cfg, s32);
}

int64_t tiles_m(int c, int64_t M) { return cdiv(M, kConfigs[c].rows); }
int64_t tiles_n(int c, int64_t N) { return cdiv(N, 16 * kConfigs[c].nt * (kConfigs[c].few ? 1 : kConfigs[c].waves)); }

// Ranges of K of a tile configuration: as many as make a workgroup for each CU, of a unit or more for each
// of its groups.
int splits_of(int cfg, int64_t M, int64_t N, int64_t K) {
    if (kConfigs[cfg].few) return 1;
    int64_t s = 256 / (tiles_m(cfg, M) * tiles_n(cfg, N)), most = cdiv(K, 2 * kStep) / kConfigs[cfg].groups;
    if (s > most) s = most;
    return s < 2 ? 1 : s > kMaxSplits ? kMaxSplits : (int)s;
}
// To 16 rows, the tile of the least rows that holds them, and the wider one where that makes a workgroup
// for each CU (one row, us, of width 32 and 16: 8192 x 8192 8.4 and 9.1, 4096 x 4096 5.4 and 4.3).  Past
// that, the least of a model of time: rounds of the CUs, each K / S values at a configuration's rate (us for
// 1000 values of K), and where K is split the second launch and what the splits write and read.  Its
// constants are fitted to all configurations' times at 88 shapes, 20 to 2048 rows against 1024 x 4096 to 14336 x
// 8192 in groups of 64 and 128: it takes the fastest in 82 of them, and one within 6% of it in the others.
int pick_a16_i4(int64_t M, int64_t N, int64_t K, int64_t group) {
    if (M <= 2) return tiles_n(1, N) >= 256 ? 1 : 0;
    if (M <= 8) return tiles_n(3, N) >= 256 ? 3 : 2;
    if (M <= 16) return tiles_n(5, N) >= 256 ? 5 : 4;
    constexpr double kRate[] = {1.1, 2.48, 3.35, 5.93, 9.08, 14.3};
    int best = 5;
    double least = 0;
    for (int c = 5; c < kNumConfigs; ++c) {
        if (!serves(c, group)) continue;
        const int64_t s = splits_of(c, M, N, K);
        double us = (double)cdiv(tiles_m(c, M) * tiles_n(c, N) * s, 256) * (double)K / (double)s * kRate[c - 5] * 1e-3;
        if (s > 1) us += 2.76 + (double)(s * M * N) * 2.7e-6;
        if (c == 5 || us < least) best = c, least = us;
    }
    return best;
}

int64_t split_bytes(int cfg, int64_t M, int64_t N, int64_t K) {
    const int s = splits_of(cfg, M, N, K);
    return s > 1 ? 4 * s * M * N : 0;
}

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 0 && N >= 0 && K >= 0 && M <= INT32_MAX && N <= INT32_MAX && K <= (int64_t(1) << 30);
}

int launch_a16_i4(int cfg, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type, const uint8_t *B,
                  int64_t ldb, const void *scale_b, int64_t ldsb, int scale_type, int64_t group, void *C, int64_t ldc,
                  int out_type, void *workspace, int64_t workspace_bytes, void *stream) {
    if (cfg >= kNumConfigs || (a_type != kF16 && a_type != kBF16) || !known_type(scale_type) || !known_type(out_type) ||
        group <= 0 || group % kBlock || group > (int64_t(1) << 30) || (cfg >= 0 && !serves(cfg, group)))
        return PDGEMM_EINVAL_CFG;
    if (!sizes_ok(M, N, K)) return PDGEMM_EINVAL_DIM;
    if (lda < K || ldb < K || ldsb < N || ldc < N) return PDGEMM_EINVAL_LD;
    if (M == 0 || N == 0) return PDGEMM_OK;
    int rc = check_plain(C, ldc, out_type);
    if (rc == PDGEMM_OK && K > 0) rc = check_plain(A, lda, a_type);
    if (rc == PDGEMM_OK && K > 0 && !B) rc = PDGEMM_ENULL;
    if (rc == PDGEMM_OK && K > 0) rc = check_plain(scale_b, ldsb, scale_type);
    if (rc == PDGEMM_OK && K > 0 && ldb > 2 * kMaxRowBytes) rc = PDGEMM_EINVAL_LD;
    if (rc == PDGEMM_OK && K > 0 && (lda % 8 || ldb % 32 || ((uintptr_t)A & 15) || ((uintptr_t)B & 15))) rc = PDGEMM_EALIGN;
    if (rc != PDGEMM_OK) return rc;
    if (cfg < 0) cfg = pick_a16_i4(M, N, K, group);
    const int splits = splits_of(cfg, M, N, K);
    if (splits > 1) {
        if (!workspace) return PDGEMM_ENULL;
        if (workspace_bytes < split_bytes(cfg, M, N, K) || ((uintptr_t)workspace & 15)) return PDGEMM_EWORKSPACE;
    }
    const Config &c = kConfigs[cfg];
    // with K = 0 no operand is read: the kernels form addresses from C instead
    const uint8_t *const p = static_cast<const uint8_t *>(C);
    A16I4Args args = {K ? static_cast<const uint8_t *>(A) : p,
                      K ? B : p,
                      C,
                      static_cast<float *>(workspace),
                      {K ? static_cast<const uint8_t *>(scale_b) : p, K ? ldsb * elem_size(scale_type) : 0, scale_type == kF16 ? ~0u : 0u},
                      K ? 2 * lda : 0,
                      K ? ldb / 2 : 0,
                      ldc,
                      (int)M,
                      (int)N,
                      (int)K,
                      (int)tiles_m(cfg, M),
                      (int)tiles_n(cfg, N),
                      splits,
                      (int)group,
                      out_type,
                      I4Groups::magic(group)};
    const bool s32 = scale_type == kF32;
    const void *fn = a_type == kF16 ? a16_i4_ptr<kF16>(cfg, (int)group, s32) : a16_i4_ptr<kBF16>(cfg, (int)group, s32);
    rc = run(fn, (int64_t)args.tiles_m * args.tiles_n * splits, c.waves * c.groups * kWave, &args, stream);
    if (rc != PDGEMM_OK || splits == 1) return rc;
    return run(reinterpret_cast<const void *>(&split_join_kernel), cdiv(M * N, 256), 256, &args, stream);
}

}  // namespace

extern "C" {

int64_t pdgemm_a16_i4_workspace_size(int64_t M, int64_t N, int64_t K, int64_t group) {
    return sizes_ok(M, N, K) && M > 0 && N > 0 ? split_bytes(pick_a16_i4(M, N, K, group), M, N, K) : 0;
}

int gemm_a16_i4(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type, const uint8_t *B, int64_t ldb,
                const void *scale_b, int64_t ldsb, int scale_type, int64_t group, void *C, int64_t ldc, int out_type,
                void *workspace, int64_t workspace_bytes, void *stream) {
    return launch_a16_i4(-1, M, N, K, A, lda, a_type, B, ldb, scale_b, ldsb, scale_type, group, C, ldc, out_type, workspace,
                         workspace_bytes, stream);
}

int64_t pdgemm_a16_i4_cfg_workspace_size(int cfg, int64_t M, int64_t N, int64_t K) {
    return cfg >= 0 && cfg < kNumConfigs && sizes_ok(M, N, K) && M > 0 && N > 0 ? split_bytes(cfg, M, N, K) : 0;
}

int pdgemm_a16_i4_cfg(int cfg, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type, const uint8_t *B,
                      int64_t ldb, const void *scale_b, int64_t ldsb, int scale_type, int64_t group, void *C, int64_t ldc,
                      int out_type, void *workspace, int64_t workspace_bytes, void *stream) {
    if (cfg < 0) return PDGEMM_EINVAL_CFG;
    return launch_a16_i4(cfg, M, N, K, A, lda, a_type, B, ldb, scale_b, ldsb, scale_type, group, C, ldc, out_type, workspace,
                         workspace_bytes, stream);
}

int pdgemm_a16_i4_num_configs(void) { return kNumConfigs; }

int pdgemm_a16_i4_pick(int64_t M, int64_t N, int64_t K, int64_t group) {
    // (with no tiles there is nothing to choose by)
    return sizes_ok(M, N, K) && M > 0 && N > 0 ? pick_a16_i4(M, N, K, group) : 0;
}

}  // extern "C"
