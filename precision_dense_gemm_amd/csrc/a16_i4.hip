// a16_i4.hip -- products of 16-bit activations with group-scaled INT4 weights for gfx950
// (MI355X), behind the C ABI declared in include/pdgemm.h.
#include "i4_core.h"

namespace {

struct A16I4Args {
    const uint8_t *A;
    const uint8_t *B;
    void *C;
    I4Scales s;
    int64_t lda, ldb;   // bytes
    int64_t ldc;        // elements
    int M, N, K;
    int tiles_n;
    int group, out_type;
};

__device__ __forceinline__ void store_as(void *C, int type, int64_t at, float v) {
    if (type == kF32)
        static_cast<float *>(C)[at] = v;
    else if (type == kF16)
        static_cast<_Float16 *>(C)[at] = (_Float16)v;
    else
        static_cast<__bf16 *>(C)[at] = (__bf16)v;
}

// A tile of 16 MT rows and 16 NT columns of C to a workgroup, K split over its W waves, whose
// sums meet in LDS and are added in wave order.
template <int T, int MT, int NT, int W, int Q, bool kS32>
__global__ __launch_bounds__(W *kWave) void a16_i4_kernel(A16I4Args args) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int kTile = MT * NT * 256;
    __shared__ float part[W][kTile];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane % 16, g = lane / 16;
    const int m0 = (blockIdx.x / args.tiles_n) * 16 * MT, n0 = (blockIdx.x % args.tiles_n) * 16 * NT;
    const int M = args.M, N = args.N, K = args.K;

    I4Source<MT, NT, 1> src;
    src.a = args.A + (int64_t)m0 * args.lda;
    src.a_end = (int)((min(16 * MT, M - m0) - 1) * args.lda) + ((2 * K + 15) & ~15);
    src.b[0] = args.B + (int64_t)n0 * args.ldb;
    src.b_end[0] = (int)((min(16 * NT, N - n0) - 1) * args.ldb) + (((K + 1) / 2 + 15) & ~15);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = 16 * i + r;
        src.va[i] = row < M - m0 ? (uint32_t)row * (uint32_t)args.lda + 16 * g : kOutside;
    }
    const int size = kS32 ? 4 : 2;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = 16 * t + r;
        src.vb[t] = row < N - n0 ? (uint32_t)row * (uint32_t)args.ldb + 16 * g : kOutside;
        src.vs[t] = (uint32_t)(n0 + min(row, N - n0 - 1)) * size;
    }
    src.s[0] = args.s;
    src.K = K, src.group = args.group;

    I4Wave<T, MT, NT, 1, Q, kS32, MT == 4 ? 2 : 4> w;
    // pairs of steps, which are whole 128-byte lines of the codes' rows
    const int steps = (K + kStep - 1) / kStep, pairs = (steps + 1) / 2;
    const int mine = wave < pairs ? (pairs - wave + W - 1) / W : 0;
    const int odd = mine > 0 && wave + (mine - 1) * W == pairs - 1 ? steps % 2 : 0;   // the last pair may be half of one
    w.run(src, 2 * mine - odd, [&](int i, auto &) { return 2 * (wave + (i >> 1) * W) + (i & 1); });
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[wave][((i * NT + t) * 4 + e) * kWave + lane] = w.acc[i][t][e];
    __syncthreads();
    // fragment (i, t) holds, in register e of lane l, row 16 i + 4 (l / 16) + e and column 16 t + l % 16
    for (int x = tid; x < kTile; x += W * kWave) {
        const int row = x / (16 * NT), col = x % (16 * NT);
        if (m0 + row >= M || n0 + col >= N) continue;
        const int at = ((row / 16 * NT + col / 16) * 4 + row % 4) * kWave + row % 16 / 4 * 16 + col % 16;
        float sum = part[0][at];
#pragma unroll
        for (int v = 1; v < W; ++v) sum += part[v][at];
        store_as(args.C, args.out_type, (int64_t)(m0 + row) * args.ldc + n0 + col, sum);
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// host side

struct Config {
    int mt, nt, waves;
};
constexpr Config kConfigs[] = {{1, 1, 8}, {1, 2, 8}, {1, 4, 8}, {2, 1, 8}, {2, 2, 8}, {4, 2, 4}, {4, 4, 4}};
constexpr int kNumConfigs = sizeof(kConfigs) / sizeof(kConfigs[0]);

template <int T, int C, int Q>
const void *a16_i4_ptr(bool s32) {
    constexpr Config c = kConfigs[C];
    return s32 ? reinterpret_cast<const void *>(&a16_i4_kernel<T, c.mt, c.nt, c.waves, Q, true>)
               : reinterpret_cast<const void *>(&a16_i4_kernel<T, c.mt, c.nt, c.waves, Q, false>);
}
template <int T, int Q, int C = 0>
const void *a16_i4_ptr(int cfg, bool s32) {
    if constexpr (C < kNumConfigs) return cfg == C ? a16_i4_ptr<T, C, Q>(s32) : a16_i4_ptr<T, Q, C + 1>(cfg, s32);
    return nullptr;
}
template <int T>
const void *a16_i4_ptr(int cfg, int group, bool s32) {
    return group % 128 == 0 ? a16_i4_ptr<T, 4>(cfg, s32)
           : group % 64 == 0 ? a16_i4_ptr<T, 2>(cfg, s32)
                             : a16_i4_ptr<T, 1>(cfg, s32);
}

// The widest tile of the rows that still makes a workgroup for each CU.
int pick_a16_i4(int64_t M, int64_t N, int64_t K) {
    (void)K;
    auto tiles = [&](int c) { return cdiv(M, 16 * kConfigs[c].mt) * cdiv(N, 16 * kConfigs[c].nt); };
    if (M <= 16) return tiles(2) >= 256 ? 2 : tiles(1) >= 256 ? 1 : 0;
    if (M <= 32) return tiles(4) >= 256 ? 4 : 3;
    return tiles(6) >= 256 ? 6 : tiles(5) >= 256 ? 5 : tiles(4) >= 256 ? 4 : 3;
}

int launch_a16_i4(int cfg, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type, const uint8_t *B,
                  int64_t ldb, const void *scale_b, int64_t ldsb, int scale_type, int64_t group, void *C, int64_t ldc,
                  int out_type, void *stream) {
    if (cfg >= kNumConfigs || (a_type != kF16 && a_type != kBF16) || !known_type(scale_type) || !known_type(out_type) ||
        group <= 0 || group % kBlock || group > (int64_t(1) << 30))
        return PDGEMM_EINVAL_CFG;
    if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > (int64_t(1) << 30)) return PDGEMM_EINVAL_DIM;
    if (lda < K || ldb < K || ldsb < N || ldc < N) return PDGEMM_EINVAL_LD;
    if (M == 0 || N == 0) return PDGEMM_OK;
    int rc = check_plain(C, ldc, out_type);
    if (rc == PDGEMM_OK && K > 0) rc = check_plain(A, lda, a_type);
    if (rc == PDGEMM_OK && K > 0 && !B) rc = PDGEMM_ENULL;
    if (rc == PDGEMM_OK && K > 0) rc = check_plain(scale_b, ldsb, scale_type);
    if (rc == PDGEMM_OK && K > 0 && ldb > 2 * kMaxRowBytes) rc = PDGEMM_EINVAL_LD;
    if (rc == PDGEMM_OK && K > 0 && (lda % 8 || ldb % 32 || ((uintptr_t)A & 15) || ((uintptr_t)B & 15))) rc = PDGEMM_EALIGN;
    if (rc != PDGEMM_OK) return rc;
    if (cfg < 0) cfg = pick_a16_i4(M, N, K);
    const Config &c = kConfigs[cfg];
    // with K = 0 no operand is read: the kernels form addresses from C instead
    const uint8_t *const p = static_cast<const uint8_t *>(C);
    A16I4Args args = {K ? static_cast<const uint8_t *>(A) : p,
                      K ? B : p,
                      C,
                      {K ? static_cast<const uint8_t *>(scale_b) : p, K ? ldsb * elem_size(scale_type) : 0, scale_type},
                      K ? 2 * lda : 0,
                      K ? ldb / 2 : 0,
                      ldc,
                      (int)M,
                      (int)N,
                      (int)K,
                      (int)cdiv(N, 16 * c.nt),
                      (int)group,
                      out_type};
    const bool s32 = scale_type == kF32;
    const void *fn = a_type == kF16 ? a16_i4_ptr<kF16>(cfg, (int)group, s32) : a16_i4_ptr<kBF16>(cfg, (int)group, s32);
    return run(fn, cdiv(M, 16 * c.mt) * args.tiles_n, c.waves * kWave, &args, stream);
}

}  // namespace

extern "C" {

int gemm_a16_i4(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type, const uint8_t *B, int64_t ldb,
                const void *scale_b, int64_t ldsb, int scale_type, int64_t group, void *C, int64_t ldc, int out_type,
                void *stream) {
    return launch_a16_i4(-1, M, N, K, A, lda, a_type, B, ldb, scale_b, ldsb, scale_type, group, C, ldc, out_type, stream);
}

int pdgemm_a16_i4_cfg(int cfg, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type, const uint8_t *B,
                      int64_t ldb, const void *scale_b, int64_t ldsb, int scale_type, int64_t group, void *C, int64_t ldc,
                      int out_type, void *stream) {
    if (cfg < 0) return PDGEMM_EINVAL_CFG;
    return launch_a16_i4(cfg, M, N, K, A, lda, a_type, B, ldb, scale_b, ldsb, scale_type, group, C, ldc, out_type, stream);
}

int pdgemm_a16_i4_num_configs(void) { return kNumConfigs; }

int pdgemm_a16_i4_pick(int64_t M, int64_t N, int64_t K) { return pick_a16_i4(M, N, K); }

}  // extern "C"
