// mxfp4.hip -- microscaled 4-bit floating point (MXFP4) for gfx950 (MI355X):
// quantising, reading back, and the products, behind the C ABI declared in
// include/pdgemm.h.
//
// An MXFP4 operand holds `rows` rows of K values.  32 consecutive values of K
// share a block scale: value = e2m1(code) * 2^(byte - 127), byte 255 = NaN.
// The codes are packed two per byte (even k in the low nibble), so a block is
// one 16-byte chunk of its row.  The scales are stored by block: scale of block b
// of row i at scales[b * lds + i].  A tile of rows then reads its scales of one
// block as one contiguous run (with a row's scales side by side instead, a tile's
// scales of one stage would be a few bytes of each of its rows' lines, and the L2
// returns whole lines).
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <type_traits>

#include "pdgemm.h"

namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx2_t __attribute__((ext_vector_type(2)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef int intx8_t __attribute__((ext_vector_type(8)));
typedef unsigned int uintx2_t __attribute__((ext_vector_type(2)));
typedef unsigned int uintx4_t __attribute__((ext_vector_type(4)));
typedef unsigned short ushortx2_t __attribute__((ext_vector_type(2)));

constexpr int kF32 = PDGEMM_F32;
constexpr int kF16 = PDGEMM_F16;
constexpr int kBF16 = PDGEMM_BF16;

constexpr int kWave = 64;
constexpr int kBlock = 32;   // values per scale

// Buffer resource word 3 for raw (untyped) buffer loads on gfx9-family parts.
constexpr int kRsrcWord3 = 0x00020000;

template <int T> struct ElemOf { using type = float; };
template <> struct ElemOf<kF16> { using type = _Float16; };
template <> struct ElemOf<kBF16> { using type = __bf16; };
constexpr int elem_size(int t) { return t == kF32 ? 4 : 2; }

// f(std::integral_constant<int, i>) for i = 0 .. N-1, in order
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F &&f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        static_for<N, I + 1>(f);
    }
}

// ---------------------------------------------------------------------------
// Block scales
//
// With a = the largest magnitude of a block and E = floor(log2 a), the scale is
// 2^e, e = max(E - 2, -127): the largest power of two of e2m1 is 2^2, so a lies in
// [4, 8) of it and what exceeds 6 saturates (PDGEMM_SCALE_FLOOR, the rule of the
// OCP microscaling formats).  PDGEMM_SCALE_FIT takes e one higher where a > 6 * 2^e,
// so nothing saturates.  A block of zeros takes byte 0; one that holds an infinity
// or a NaN takes byte 255, which makes the whole block NaN, and zero codes.

// what is added to the bits of a before its exponent is read: FIT carries into the
// exponent where the mantissa is above 1.5
__host__ __device__ constexpr uint32_t rule_bias(int rule) { return rule == PDGEMM_SCALE_FIT ? 0x3FFFFFu : 0u; }

// the scale's byte from the binary32 bits of a
__device__ __forceinline__ uint32_t scale_byte(uint32_t a, uint32_t bias) {
    const int b = max((int)((a + bias) >> 23) - 2, 0);
    return a >= 0x7F800000u ? 255u : (uint32_t)b;
}

// binary32 2^(byte - 127) of a byte below 255 (byte 0: the subnormal 2^-127)
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __builtin_bit_cast(float, max(byte << 23, 0x00400000u));
}

// binary32 bits of the magnitude whose 16-bit pattern (f16 or bf16) is h
template <int T>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t h) {
    if constexpr (T == kBF16) return h << 16;
    return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)h));
}

// Two values of a pair (16-bit types: packed in `x`) over `scale`, rounded to nearest
// even and saturated at 6, as byte kSel of `old`.
template <int T, int kSel>
__device__ __forceinline__ uint32_t codes16(uint32_t old, uint32_t x, float scale) {
    if constexpr (T == kF16)
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(half2_t, x), scale, kSel);
    else
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_t, x), scale, kSel);
}
template <int kSel>
__device__ __forceinline__ uint32_t codes32(uint32_t old, float x, float y, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, x, y, scale, kSel);
}

// maximum over groups of 4 or 8 lanes (in every lane); every lane is active
template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));                            // quad_perm 1 0 3 2
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));                            // quad_perm 2 3 0 1
    if constexpr (kLanes >= 8) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));   // row_half_mirror
    return v;
}

// Orders a wave's LDS accesses before and after it, across its lanes.  The LDS serves one wave's
// accesses in the order they are issued, so this costs no instruction: it keeps the compiler,
// which sees one lane alone, from moving a read above the other lanes' store.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One exchange of a maximum over lanes: of 2 n values v, the lanes without `kBit` keep the
// first n and the others the last n, each with what its partner (DPP control kDpp, which
// flips that bit) has there.
template <int n, int kBit, int kDpp>
__device__ __forceinline__ void halve(uint32_t (&v)[32], int lane) {
    const bool upper = lane & kBit;
#pragma unroll
    for (int p = 0; p < n; ++p) {
        const uint32_t keep = upper ? v[p + n] : v[p], give = upper ? v[p] : v[p + n];
        v[p] = max(keep, (uint32_t)__builtin_amdgcn_mov_dpp((int)give, kDpp, 0xF, 0xF, true));
    }
}

struct QuantArgs {
    const void *src;
    uint8_t *q;    // packed along K (NULL: not written)
    uint8_t *s;
    uint8_t *qt;   // the transpose: packed along the rows (NULL: not written)
    uint8_t *st;
    int64_t ld;    // elements
    int64_t ldq;   // bytes
    int64_t lds;
    int64_t ldqt;  // bytes
    int64_t ldst;
    int rows, K;
    int tiles_k;   // workgroups along K
    uint32_t bias;
};

// Rows along K only.  A lane takes 16 bytes of a row, a wave a span of 64 of them,
// so every load instruction reads 1 KB of one row, and a block is 4 (fp32: 8)
// neighbouring lanes.  A workgroup of 4 waves takes 4 * kRpw rows of one span; the
// scales go through LDS so that a block's scales of those rows are written as one run.
// Bound by memory: 8192 x 8192 takes 24.2 us from f16 (7.0 TB/s of reads and writes) and
// 46.4 us from fp32 (6.6); a copy of as many bytes runs at 5 to 8.5.
template <int T, int kRpw>
__global__ __launch_bounds__(256) void mx_quant_rows_kernel(QuantArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    constexpr int kVals = 16 / elem_size(T);      // values per lane
    constexpr int kLanes = kBlock / kVals;        // lanes per block
    constexpr int kSpan = kWave * kVals;
    constexpr int kBlocks = kSpan / kBlock;       // blocks per span
    constexpr int kRows = 4 * kRpw;
    __shared__ uint8_t sc[kBlocks][kRows];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int tile_m = blockIdx.x / args.tiles_k, tile_k = blockIdx.x % args.tiles_k;
    const int row0 = tile_m * kRows + wave * kRpw;
    const int k0 = tile_k * kSpan + lane * kVals;
    const int K = args.K;

    uint32_t v[kRpw][4];
    const Elem *const src = static_cast<const Elem *>(args.src) + (int64_t)row0 * args.ld + k0;
    if (row0 + kRpw <= args.rows && (tile_k + 1) * kSpan <= K) {
        // (rows need only the element's alignment)
#pragma unroll
        for (int r = 0; r < kRpw; ++r) __builtin_memcpy(v[r], src + r * args.ld, 16);
    } else {
#pragma unroll
        for (int r = 0; r < kRpw; ++r) {
            Elem e[kVals] = {};
            if (row0 + r < args.rows) {
#pragma unroll
                for (int x = 0; x < kVals; ++x)
                    if (k0 + x < K) e[x] = src[r * args.ld + x];
            }
            __builtin_memcpy(v[r], e, 16);
        }
    }
#pragma unroll
    for (int r = 0; r < kRpw; ++r) {
        uint32_t a;
        if constexpr (T == kF32) {
            a = max(max(v[r][0] & 0x7FFFFFFFu, v[r][1] & 0x7FFFFFFFu), max(v[r][2] & 0x7FFFFFFFu, v[r][3] & 0x7FFFFFFFu));
            a = group_max<kLanes>(a);
        } else {
            // magnitudes of either 16-bit type order as their bit patterns
            ushortx2_t m = __builtin_bit_cast(ushortx2_t, v[r][0] & 0x7FFF7FFFu);
#pragma unroll
            for (int d = 1; d < 4; ++d)
                m = __builtin_elementwise_max(m, __builtin_bit_cast(ushortx2_t, v[r][d] & 0x7FFF7FFFu));
            a = magnitude_bits<T>(group_max<kLanes>(max((uint32_t)m[0], (uint32_t)m[1])));
        }
        const uint32_t byte = scale_byte(a, args.bias);
        const float scale = scale_value(byte);
        uint32_t c = 0;
        if constexpr (T == kF32) {
            c = codes32<0>(c, __builtin_bit_cast(float, v[r][0]), __builtin_bit_cast(float, v[r][1]), scale);
            c = codes32<1>(c, __builtin_bit_cast(float, v[r][2]), __builtin_bit_cast(float, v[r][3]), scale);
        } else {
            c = codes16<T, 0>(c, v[r][0], scale);
            c = codes16<T, 1>(c, v[r][1], scale);
            c = codes16<T, 2>(c, v[r][2], scale);
            c = codes16<T, 3>(c, v[r][3], scale);
        }
        if (byte == 255) c = 0;
        if (lane % kLanes == 0) sc[lane / kLanes][wave * kRpw + r] = (uint8_t)byte;
        // the chunk that holds the row's last value is written whole
        if (row0 + r < args.rows && k0 - k0 % kBlock < K) {
            uint8_t *const q = args.q + (int64_t)(row0 + r) * args.ldq + k0 / 2;
            if constexpr (T == kF32)
                *reinterpret_cast<uint16_t *>(q) = (uint16_t)c;
            else
                *reinterpret_cast<uint32_t *>(q) = c;
        }
    }
    __syncthreads();
    const int blocks = (K + kBlock - 1) / kBlock;
    for (int x = tid; x < kBlocks * kRows; x += 256) {
        const int b = tile_k * kBlocks + x / kRows, i = tile_m * kRows + x % kRows;
        if (b < blocks && i < args.rows) args.s[(int64_t)b * args.lds + i] = sc[x / kRows][x % kRows];
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// The transpose, and with kBoth the rows along K too, from one read.  A lane takes two
// neighbouring columns of 32 rows, so a load instruction of a wave reads a run of 128
// columns of one row; a column's block is in one lane's registers and a row's block in
// 16 neighbouring lanes.  A workgroup of 8 waves takes 256 rows x 128 columns, and the
// codes (4 bits a value) go through LDS so that both forms are written in runs of whole
// chunks: 128 bytes per column, 64 bytes per row.  Both forms of 4096 x 8192 bf16 take 18.2 us
// (5.6 TB/s), the transpose alone 14.4: bound by memory and, for both, by the conversions, two
// for every value.
template <int T, bool kBoth>
__global__ __launch_bounds__(512) void mx_quant_cols_kernel(QuantArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    constexpr int kRows = 256, kCols = 128;
    constexpr int kD = T == kF32 ? 2 : 1;         // dwords per pair of columns
    __shared__ uint4 lqt[kCols][8];               // chunk w of column c at w ^ ((c / 2) % 8)
    __shared__ __align__(16) uint8_t lq[kBoth ? kRows : 1][64];
    __shared__ uint8_t sct[8][kCols];
    __shared__ __align__(16) uint8_t scr[4][kBoth ? kRows : 16];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int tile_m = blockIdx.x / args.tiles_k, tile_k = blockIdx.x % args.tiles_k;
    const int m0 = tile_m * kRows, c0 = tile_k * kCols;
    const int row0 = m0 + wave * 32;
    const int k = c0 + 2 * lane;
    const int rows = args.rows, K = args.K;

    uint32_t v[32][kD];
    const Elem *const src = static_cast<const Elem *>(args.src) + (int64_t)row0 * args.ld + k;
    if (row0 + 32 <= rows && c0 + kCols <= K) {
        // (rows need only the element's alignment)
#pragma unroll
        for (int r = 0; r < 32; ++r) __builtin_memcpy(v[r], src + r * args.ld, 4 * kD);
    } else {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            Elem e[2] = {};
            if (row0 + r < rows && k < K) e[0] = src[r * args.ld];
            if (row0 + r < rows && k + 1 < K) e[1] = src[r * args.ld + 1];
            __builtin_memcpy(v[r], e, 4 * kD);
        }
    }

    if constexpr (kBoth) {
        // The 32 rows' largest magnitudes over 16 lanes: each exchange leaves a lane half of its
        // rows, so that lane l ends with rows 2 (l % 16) and + 1 of its block, and one lane
        // makes a row's scale for all 16.
        uint32_t a[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            if constexpr (T == kF32)
                a[r] = max(v[r][0] & 0x7FFFFFFFu, v[r][1] & 0x7FFFFFFFu);
            else
                a[r] = max(v[r][0] & 0x7FFFu, (v[r][0] >> 16) & 0x7FFFu);
        }
        halve<16, 8, 0x140>(a, lane);   // row_mirror: lane 15 - l
        halve<8, 4, 0x141>(a, lane);    // row_half_mirror: 7 - l
        halve<4, 2, 0x4E>(a, lane);     // quad_perm 2 3 0 1
        halve<2, 1, 0xB1>(a, lane);     // quad_perm 1 0 3 2
        uint32_t b[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) b[x] = scale_byte(T == kF32 ? a[x] : magnitude_bits<T>(a[x]), args.bias);
        // (copied as bytes both ways: a 16-bit store and a 32-bit read of it would be taken not to
        // overlap)
        uint8_t *const sr = static_cast<uint8_t *>(__builtin_assume_aligned(&scr[lane / 16][wave * 32], 16));
        const uint16_t pair_of_scales = (uint16_t)(b[0] | b[1] << 8);
        __builtin_memcpy(__builtin_assume_aligned(sr + 2 * (lane & 15), 2), &pair_of_scales, 2);
        wave_lds_order();   // the block's 32 scales come from its 16 lanes
        const bool special = __builtin_amdgcn_ballot_w64(max(b[0], b[1]) == 255u) != 0;   // of any block of the wave
        uint32_t w[8];
        __builtin_memcpy(w, sr, 32);
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            const uint32_t byte = (w[r / 4] >> (8 * (r & 3))) & 255u;
            const float scale = scale_value(byte);
            uint32_t c;
            if constexpr (T == kF32)
                c = codes32<0>(0, __builtin_bit_cast(float, v[r][0]), __builtin_bit_cast(float, v[r][1]), scale);
            else
                c = codes16<T, 0>(0, v[r][0], scale);
            lq[wave * 32 + r][lane] = special && byte == 255 ? 0 : (uint8_t)c;
        }
    }

    uint32_t a0 = 0, a1 = 0;   // the two columns' magnitudes
    if constexpr (T == kF32) {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            a0 = max(a0, v[r][0] & 0x7FFFFFFFu);
            a1 = max(a1, v[r][1] & 0x7FFFFFFFu);
        }
    } else {
        ushortx2_t m = {0, 0};
#pragma unroll
        for (int r = 0; r < 32; ++r)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(ushortx2_t, v[r][0] & 0x7FFF7FFFu));
        a0 = magnitude_bits<T>(m[0]);
        a1 = magnitude_bits<T>(m[1]);
    }
    const uint32_t b0 = scale_byte(a0, args.bias), b1 = scale_byte(a1, args.bias);
    const float s0 = scale_value(b0), s1 = scale_value(b1);
    uint32_t w0[4], w1[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t x = 0, y = 0;
        const auto pair = [&](auto sel_c) __attribute__((always_inline)) {
            constexpr int kSel = decltype(sel_c)::value;
            const int r = 8 * d + 2 * kSel;
            if constexpr (T == kF32) {
                x = codes32<kSel>(x, __builtin_bit_cast(float, v[r][0]), __builtin_bit_cast(float, v[r + 1][0]), s0);
                y = codes32<kSel>(y, __builtin_bit_cast(float, v[r][kD - 1]), __builtin_bit_cast(float, v[r + 1][kD - 1]), s1);
            } else {
                x = codes16<T, kSel>(x, __builtin_amdgcn_perm(v[r + 1][0], v[r][0], 0x05040100u), s0);
                y = codes16<T, kSel>(y, __builtin_amdgcn_perm(v[r + 1][0], v[r][0], 0x07060302u), s1);
            }
        };
        pair(std::integral_constant<int, 0>{});
        pair(std::integral_constant<int, 1>{});
        pair(std::integral_constant<int, 2>{});
        pair(std::integral_constant<int, 3>{});
        w0[d] = b0 == 255 ? 0 : x;
        w1[d] = b1 == 255 ? 0 : y;
    }
    const int pos = wave ^ (lane & 7);
    lqt[2 * lane][pos] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
    lqt[2 * lane + 1][pos] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
    sct[wave][2 * lane] = (uint8_t)b0;
    sct[wave][2 * lane + 1] = (uint8_t)b1;
    __syncthreads();

    const int blocks_k = (K + kBlock - 1) / kBlock, blocks_m = (rows + kBlock - 1) / kBlock;
#pragma unroll
    for (int x = tid; x < kCols * 8; x += 512) {
        const int c = x / 8, w = x % 8;
        if (c0 + c < K && m0 + 32 * w < rows)
            *reinterpret_cast<uint4 *>(args.qt + (int64_t)(c0 + c) * args.ldqt + m0 / 2 + 16 * w) =
                lqt[c][w ^ ((c >> 1) & 7)];
    }
    for (int x = tid; x < 8 * kCols; x += 512) {
        const int w = x / kCols, c = x % kCols;
        if (c0 + c < K && m0 / 32 + w < blocks_m) args.st[(int64_t)(m0 / 32 + w) * args.ldst + c0 + c] = sct[w][c];
    }
    if constexpr (kBoth) {
#pragma unroll
        for (int x = tid; x < kRows * 4; x += 512) {
            const int r = x / 4, w = x % 4;
            if (m0 + r < rows && c0 + 32 * w < K)
                *reinterpret_cast<uint4 *>(args.q + (int64_t)(m0 + r) * args.ldq + c0 / 2 + 16 * w) =
                    *reinterpret_cast<const uint4 *>(&lq[r][16 * w]);
        }
        for (int x = tid; x < 4 * kRows; x += 512) {
            const int w = x / kRows, r = x % kRows;
            if (m0 + r < rows && c0 / 32 + w < blocks_k) args.s[(int64_t)(c0 / 32 + w) * args.lds + m0 + r] = scr[w][r];
        }
    }
#endif  // __HIP_DEVICE_COMPILE__
}

struct DequantArgs {
    const uint8_t *q;
    const uint8_t *s;
    void *dst;
    int64_t ldq;   // bytes
    int64_t lds;
    int64_t ldd;   // elements
    int rows, K;
    int tiles_k;
};

// Values back from codes and scales.  A lane makes 16 bytes of a row (4 or 8 values), so every
// store of a wave is a run of 1 KB; a workgroup of 4 waves takes 4 * kRpw rows of that span,
// whose scales it first reads into LDS, a run of rows per block.  The stores are non-temporal
// where they fill whole lines (8192 x 8192 to f16 24.8 us and not 25.6, 3000 x 5120 to fp32
// 11.1 and not 11.7); rows that start inside a line share it, and such pieces are left to the L2
// to join (2999 x 5003 to fp32 12.9 and not 16.8, to bf16 8.3 and not 9.0).
// (kLines: dst's rows start on 128-byte lines.)
template <int T, int kRpw, bool kLines>
__global__ __launch_bounds__(256) void mx_dequant_kernel(DequantArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    constexpr int kVals = 16 / elem_size(T), kSpan = kWave * kVals, kBlocks = kSpan / kBlock, kRows = 4 * kRpw;
    using Codes = typename std::conditional<kVals == 8, uint32_t, uint16_t>::type;
    __shared__ uint8_t sc[kBlocks][kRows];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int tile_m = blockIdx.x / args.tiles_k, tile_k = blockIdx.x % args.tiles_k;
    const int row0 = tile_m * kRows + wave * kRpw;
    const int k0 = tile_k * kSpan + lane * kVals;
    const int K = args.K;
    const int blocks = (K + kBlock - 1) / kBlock;

    uint32_t w[kRpw];
#pragma unroll
    for (int r = 0; r < kRpw; ++r) {
        w[r] = 0;
        if (row0 + r < args.rows && k0 < K)
            w[r] = *reinterpret_cast<const Codes *>(args.q + (int64_t)(row0 + r) * args.ldq + k0 / 2);
    }
    for (int x = tid; x < kBlocks * kRows; x += 256) {
        const int b = tile_k * kBlocks + x / kRows, i = tile_m * kRows + x % kRows;
        sc[x / kRows][x % kRows] = b < blocks && i < args.rows ? args.s[(int64_t)b * args.lds + i] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRpw; ++r) {
        if (row0 + r >= args.rows || k0 >= K) continue;
        // (the conversion reads the scale's exponent alone: 0 is 2^-127 and 255 gives NaN)
        const float scale = __builtin_bit_cast(float, (uint32_t)sc[lane / (kBlock / kVals)][wave * kRpw + r] << 23);
        Elem e[kVals];
        static_for<kVals / 2>([&](auto sel_c) __attribute__((always_inline)) {
            constexpr int kSel = decltype(sel_c)::value;
            const floatx2_t p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r], scale, kSel);
            e[2 * kSel] = (Elem)p[0];
            e[2 * kSel + 1] = (Elem)p[1];
        });
        Elem *const p = static_cast<Elem *>(args.dst) + (int64_t)(row0 + r) * args.ldd + k0;
        if (k0 + kVals <= K) {
            typedef Elem vec_t __attribute__((ext_vector_type(kVals)));
            typedef vec_t packed_t __attribute__((aligned(sizeof(Elem))));   // the element's alignment only
            vec_t v;
            __builtin_memcpy(&v, e, 16);
            if constexpr (kLines)
                __builtin_nontemporal_store(v, reinterpret_cast<packed_t *>(p));
            else
                *reinterpret_cast<packed_t *>(p) = v;
        } else {
#pragma unroll
            for (int x = 0; x < kVals; ++x)
                if (k0 + x < K) p[x] = e[x];
        }
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// Products
//
// C[i][j] = sum over blocks b of 2^(sa + sb - 254) * sum over k in b of a * b: the
// scaled MFMA v_mfma_scale_f32_16x16x128_f8f6f4 with e2m1 operands.  Lane l of a
// 16-row fragment holds the 32 values of block l / 16 of row l % 16, one 16-byte chunk,
// and that block's scale in a byte of a scale register.

struct MxArgs {
    const uint8_t *A;    // packed e2m1, or 16-bit values (the a16 product)
    const uint8_t *SA;
    const uint8_t *B;
    const uint8_t *SB;
    void *C;
    int64_t lda, ldb;    // bytes
    int64_t ldsa, ldsb;
    int64_t ldc;         // elements
    int M, N, K;
    int tiles_m, tiles_n;
    bool plain;          // C through the L2 (the tile kernels; see plain_stores)
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, int range) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, range, kRsrcWord3);
}

// Byte offset of row `row` of a tile (a row spans at most 4 MiB and a tile 256 rows) that
// has `rows` rows; rows past them get an offset outside every range, so that zeros arrive and
// no memory is read.
constexpr uint32_t kOutside = 0x80000000u;
__device__ __forceinline__ uint32_t row_offset(int row, int rows, int64_t ld) {
    return row < rows ? (uint32_t)row * (uint32_t)ld : kOutside;
}

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    const uintx4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// v at byte offset off, not stored where that is outside the range; kAux: cache control
template <int kAux, typename V>
__device__ __forceinline__ void store_bytes(__amdgpu_buffer_rsrc_t r, uint32_t off, const V &v) {
    static_assert(sizeof(V) == 2 || sizeof(V) == 4 || sizeof(V) == 8, "an element of C, or two");
    if constexpr (sizeof(V) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), r, off, 0, kAux);
    if constexpr (sizeof(V) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, off, 0, kAux);
    if constexpr (sizeof(V) == 8) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uintx2_t, v), r, off, 0, kAux);
}

// n (1, 2 or 4) bytes, zero-extended
template <int n>
__device__ __forceinline__ uint32_t load_bytes(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (n == 1) return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
    if constexpr (n == 2) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    if constexpr (n == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}

template <int kOpA, int kOpB>
__device__ __forceinline__ floatx4_t mfma_fp4(const uint4 &a, const uint4 &b, const floatx4_t &c, uint32_t sa, uint32_t sb) {
    const intx8_t a8 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w};
    const intx8_t b8 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w};
    // format 4 of both operands: e2m1
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, kOpA, (int)sa, kOpB, (int)sb);
}

// Sum of the waves' partial tiles (each wave summed its own range of K) in wave order,
// rounded once to C's type and stored.  acc[i][j] of a wave holds, in register e of lane
// l, row FM * (4 (l / 16) + e) + i (with kMixed; else 16 i + 4 (l / 16) + e) and column
// FN * (l % 16) + j of the tile, of which BM rows are stored.  `part` is LDS of kStride floats
// per wave, each wave's part free for it to write; where it does not hold a wave's tile, the
// column blocks j go through it in two halves.
template <int FM, int FN, int W, int OT, int kStride, int BM, bool kMixed>
__device__ __forceinline__ void join_and_store(floatx4_t (&acc)[FM][FN], float *part, const MxArgs &args, int m0, int n0,
                                               int tid, int lane, int wave) {
    using Out = typename ElemOf<OT>::type;
    constexpr int kTile = FM * FN * 4 * kWave;
    constexpr int kParts = kStride >= kTile ? 1 : 2, FG = FN / kParts;
    static_assert(kStride * kParts >= kTile && FN % kParts == 0, "a wave's tile, or half of it");
    Out *const C = static_cast<Out *>(args.C);
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
        if (h > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FG; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    part[wave * kStride + ((i * FG + j) * 4 + e) * kWave + lane] = acc[i][h * FG + j][e];
        __syncthreads();
        for (int x = tid; x < BM * 16 * FG; x += W * kWave) {
            const int row = x / (16 * FG), n = x % (16 * FG) / FG, j = x % FG;
            const int col = FN * n + h * FG + j;
            if (m0 + row >= args.M || n0 + col >= args.N) continue;
            const int i = kMixed ? row % FM : row / 16, rr = kMixed ? row / FM : row % 16;
            const int at = ((i * FG + j) * 4 + (rr & 3)) * kWave + (rr >> 2) * 16 + n;
            float sum = part[at];
#pragma unroll
            for (int w = 1; w < W; ++w) sum += part[w * kStride + at];
            C[(int64_t)(m0 + row) * args.ldc + n0 + col] = (Out)sum;
        }
    }
}

// Block id -> tile, the order of the other GEMM kernels: workgroups are dispatched
// round-robin over the 8 XCDs, so each XCD takes a contiguous range of tiles, in bands
// of GM block rows, whose operands its L2 then shares; a grid of whole 16 x 16 windows
// of tiles goes window by window (one round of the 256 CUs each, serpentine), 4 x 8
// tiles to an XCD.
template <int GM, bool kWindows>
__device__ __forceinline__ void tile_of(int tiles_m, int tiles_n, int &tile_m, int &tile_n) {
    const int nb = gridDim.x, bid = blockIdx.x;
    const int xcd = bid & 7, loc = bid >> 3;
    if (kWindows && ((tiles_m | tiles_n) & 15) == 0) {
        const int w = loc >> 5, k = loc & 31;   // window; this XCD's k-th tile in it
        const int wcols = tiles_n >> 4;
        const int wm = w / wcols, wi = w - wm * wcols;
        const int wn = (wm & 1) ? wcols - 1 - wi : wi;
        tile_m = wm * 16 + (xcd & 3) * 4 + (k & 3);
        tile_n = wn * 16 + (xcd >> 2) * 8 + (k >> 2);
        return;
    }
    const int q = nb >> 3, r = nb & 7;
    const int id = (xcd < r) ? xcd * (q + 1) + loc : r * (q + 1) + (xcd - r) * q + loc;
    const int band = id / (GM * tiles_n);
    const int first_m = band * GM;
    const int rows = min(tiles_m - first_m, GM);
    const int in_band = id - band * GM * tiles_n;
    tile_m = first_m + in_band % rows;
    tile_n = in_band / rows;
}

typedef float floatx16_t __attribute__((ext_vector_type(16)));
typedef int intx4_t __attribute__((ext_vector_type(4)));

template <int kOpA, int kOpB>
__device__ __forceinline__ floatx16_t mfma32_fp4(const uint4 &a, const uint4 &b, const floatx16_t &c, uint32_t sa, uint32_t sb) {
    const intx4_t a4 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w}, b4 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w};
    // format 4 reads four of an operand's eight registers
    const intx8_t a8 = __builtin_shufflevector(a4, a4, 0, 1, 2, 3, -1, -1, -1, -1);
    const intx8_t b8 = __builtin_shufflevector(b4, b4, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, kOpA, (int)sa, kOpB, (int)sb);
}

#define LDS_PTR(p) ((__attribute__((address_space(3))) void *)(p))

// LDS position of 16-byte chunk c of the 128-byte stage row r is c ^ swizzle8(r): the
// 16 lanes of a phase of a fragment read (16 consecutive rows, one chunk) fall in
// distinct bank groups.
__device__ __forceinline__ int swizzle8(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Many rows: a BM x BN tile of C per workgroup of (BM / WM) x (BN / WN) waves on
// v_mfma_scale_f32_32x32x64_f8f6f4 (one instruction, 64 values of K: twice the work per
// instruction of the 16 x 16 form; a loop of nothing but MFMAs on random operands ran at
// 6.5 PFLOP/s, of the 16 x 16 form at 5.9).
//
// A stage is one 128-byte line (256 values) of K of the tile's BM rows of A and BN of B,
// copied from memory straight into LDS, two stages deep, and its scales.  Fragment i of a
// wave holds rows FM r + i (r = 0 .. 31) of the wave's WM rows, which the copy places at
// LDS rows 32 i + r: so a lane's scales of its FM fragments are neighbouring bytes of a
// dword, which one MFMA operand register takes whole (the instruction picks the byte), and
// a lane's results of FN fragments are neighbouring columns of C, stored together.  A
// stage's scales are copied by the first waves, 16 rows of a block per lane.
//
// 8192^3 to fp32 takes 242 to 260 us by GPU (4.2 to 4.5 PFLOP/s), 1024 x 8192 x 8192 34 to 37.
// Counters of the former: MFMAs busy 58% of the cycles, LDS 25%, no bank conflicts, operands
// fetched past the L2s 6 times (428 MB), C written once; the clock falls to 1.7 GHz under
// the MFMAs' load, and the stores of C at each tile's end are a tenth of the time.
template <int BM, int BN, int WM, int WN, int OT>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * kWave, 2) void mx_tile_kernel(MxArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Out = typename ElemOf<OT>::type;
    constexpr int NW = (BM / WM) * (BN / WN);
    constexpr int kWavesN = BN / WN;
    constexpr int FM = WM / 32, FN = WN / 32;
    constexpr int kRows = BM + BN;
    constexpr int kDma = kRows / 8 / NW;           // copies of 1 KB (8 rows) per wave per stage
    constexpr int kDmaA = BM / 8 / NW;
    constexpr int kSc = kRows / 128;               // waves that copy 1 KB of scales too
    constexpr int kAll = kDma + 1;
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "a stage's rows split evenly over the waves");
    static_assert(BM % 128 == 0 && BN % 128 == 0 && kSc <= NW, "a wave copies scales of one operand");
    static_assert((FM == 1 || FM == 2 || FM == 4) && (FN == 1 || FN == 2 || FN == 4), "scales of a lane in one dword");
    struct Stage {
        uint4 rows[kRows][8];
        uint4 sc[kRows / 2 + 64];   // bytes: [A: 8 blocks of BM rows | B: 8 blocks of BN rows | unused]
    };
    __shared__ Stage l0, l1;

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int M = args.M, N = args.N, K = args.K;
    int tile_m, tile_n;
    tile_of<4, true>(args.tiles_m, args.tiles_n, tile_m, tile_n);
    const int m0 = tile_m * BM, n0 = tile_n * BN;
    const int blocks = (K + kBlock - 1) / kBlock;
    const int n_st = (blocks + 7) / 8;

    const uint8_t *const a_base = args.A + (int64_t)m0 * args.lda;
    const uint8_t *const b_base = args.B + (int64_t)n0 * args.ldb;
    const int a_end = (int)((min(BM, M - m0) - 1) * args.lda) + blocks * 16;
    const int b_end = (int)((min(BN, N - n0) - 1) * args.ldb) + blocks * 16;
    // a block's scales are read up to the 16-byte granule that holds the last row's
    const int sa_cols = min(((M + 15) & ~15) - m0, BM), sb_cols = min(((N + 15) & ~15) - n0, BN);

    // copy j of this wave fills LDS rows (j NW + wave) 8 .. + 7, lane l chunk position l % 8
    // of row l / 8
    uint32_t voff[kDma];
#pragma unroll
    for (int j = 0; j < kDma; ++j) {
        const int cr = (j * NW + wave) * 8 + (lane >> 3);
        const int chunk = (lane & 7) ^ swizzle8(cr);
        if (j < kDmaA) {
            const int row = cr / WM * WM + FM * (cr % 32) + cr % WM / 32;
            voff[j] = row_offset(row, M - m0, args.lda) + chunk * 16;
        } else {
            const int cb = cr - BM;
            const int row = cb / WN * WN + FN * (cb % 32) + cb % WN / 32;
            voff[j] = row_offset(row, N - n0, args.ldb) + chunk * 16;
        }
    }
    // scale copy `wave`, 16 rows of one block per lane.  The waves beyond copy nothing (an
    // empty range: zeros into a kilobyte nobody reads), so that a stage is straight-line code
    // and every wave counts its copies alike
    const bool sc_a = wave < BM / 128, sc_none = wave >= kSc;
    const int sd = (sc_a ? wave : wave - BM / 128) * 64 + lane, sq = (sc_a ? BM : BN) / 16;
    const int sc_ld = sc_none ? 0 : (int)(sc_a ? args.ldsa : args.ldsb);
    const int sc_cols = sc_none ? 0 : sc_a ? sa_cols : sb_cols;
    const uint8_t *const sc_base = sc_a ? args.SA + m0 : args.SB + n0;
    const uint32_t soff = (uint32_t)(sd / sq * sc_ld) + sd % sq * 16;
    auto stage = [&](int st, Stage &buf) __attribute__((always_inline)) {
        const int nb = min(blocks - st * 8, 8);   // at most 0 past K: nothing is read, zeros arrive
        const bool live = nb > 0;
        const auto ra = rsrc(a_base + st * 128, live ? a_end - st * 128 : 0);
        const auto rb = rsrc(b_base + st * 128, live ? b_end - st * 128 : 0);
#pragma unroll
        for (int j = 0; j < kDma; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(j < kDmaA ? ra : rb, LDS_PTR(&buf.rows[(j * NW + wave) * 8][0]), 16,
                                                     voff[j], 0, 0, 0);
        // (a scale row holds at least the tile's columns, so the range of no blocks is not positive)
        const auto rs = rsrc(sc_base + (int64_t)st * 8 * sc_ld, max((nb - 1) * sc_ld + sc_cols, 0));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, LDS_PTR(&buf.sc[sc_none ? kSc * 64 : wave * 64]), 16, soff, 0, 0, 0);
    };

    const int wm0 = (wave / kWavesN) * WM, wn0 = (wave % kWavesN) * WN;
    const int r = lane & 31, h = lane >> 5;
    // fragment rows start at multiples of 32, so the swizzle of row r applies
    auto read_frags = [&](const Stage &buf, int s, uint4 (&fa)[FM], uint4 (&fb)[FN]) __attribute__((always_inline)) {
        const int ch = (2 * s + h) ^ swizzle8(r);
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = buf.rows[BM + wn0 + j * 32 + r][ch];
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[i] = buf.rows[wm0 + i * 32 + r][ch];
    };
    // this lane's dwords of a stage's four k-steps: block 2 s + h, the rows around its own
    const int ia = h * BM + (wm0 + FM * r), ib = 8 * BM + h * BN + (wn0 + FN * r);
    auto read_scales = [&](const Stage &buf, uint32_t (&sa)[4], uint32_t (&sb)[4]) __attribute__((always_inline)) {
        const uint32_t *const sc = reinterpret_cast<const uint32_t *>(&buf.sc[0]);
#pragma unroll
        for (int s = 0; s < 4; ++s) sa[s] = sc[(ia + 2 * s * BM) / 4];
#pragma unroll
        for (int s = 0; s < 4; ++s) sb[s] = sc[(ib + 2 * s * BN) / 4];
    };
    // a lane's bytes to the bottom of each dword
    const int sha = 8 * ((FM * r) & 3), shb = 8 * ((FN * r) & 3);

    floatx16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    auto mma = [&](const uint4 (&fa)[FM], const uint4 (&fb)[FN], uint32_t sa, uint32_t sb) __attribute__((always_inline)) {
        if constexpr (FM < 4) sa >>= sha;
        if constexpr (FN < 4) sb >>= shb;
        static_for<FM>([&](auto i_c) __attribute__((always_inline)) {
            static_for<FN>([&](auto j_c) __attribute__((always_inline)) {
                constexpr int i = decltype(i_c)::value, j = decltype(j_c)::value;
                acc[i][j] = mfma32_fp4<i, j>(fa[i], fb[j], acc[i][j], sa, sb);
            });
        });
    };
    // issue order of a k-step: its MFMAs, the next one's fragment reads and (after the
    // stage barrier) the copies of a later stage slotted between them
    constexpr int kMfma = FM * FN;
    auto interleave = [&](auto reads_c, auto dma_c) __attribute__((always_inline)) {
        constexpr int reads = decltype(reads_c)::value, dma = decltype(dma_c)::value;
        constexpr int rper = (reads + kMfma - 1) / kMfma, dper = (dma + kMfma - 1) / kMfma;
#pragma unroll
        for (int i = 0; i < kMfma; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                    // MFMA
            if (i * rper < reads) __builtin_amdgcn_sched_group_barrier(0x100, rper, 0);           // LDS reads
            if (i * dper < dma) __builtin_amdgcn_sched_group_barrier(0x020, dper, 0);             // copies
        }
    };
    using kNone = std::integral_constant<int, 0>;
    using kFrags = std::integral_constant<int, FM + FN>;
    using kFragsScales = std::integral_constant<int, FM + FN + 8>;
    using kCopies = std::integral_constant<int, kAll>;

    // fragments of the even (0) and odd (1) k-steps; the scales of the current and next stage
    uint4 fa0[FM], fb0[FN], fa1[FM], fb1[FN];
    uint32_t sa[4], sb[4], sa_next[4], sb_next[4];
    // stage st (not the last) from `cur`, whose k-step 0 is in fa0 / fb0 and scales in sa / sb;
    // refills `cur` with stage st + 2 and reads the same of stage st + 1 from `nxt`
    auto full_stage = [&](Stage &cur, const Stage &nxt, int st) __attribute__((always_inline)) {
        read_frags(cur, 1, fa1, fb1);
        mma(fa0, fb0, sa[0], sb[0]);
        interleave(kFrags{}, kNone{});
        read_frags(cur, 2, fa0, fb0);
        mma(fa1, fb1, sa[1], sb[1]);
        interleave(kFrags{}, kNone{});
        read_frags(cur, 3, fa1, fb1);
        mma(fa0, fb0, sa[2], sb[2]);
        interleave(kFrags{}, kNone{});
        // this wave's copies of stage st + 1 have landed and its reads of `cur` are done; after
        // the barrier the same holds for every wave
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        stage(st + 2, cur);
        read_scales(nxt, sa_next, sb_next);
        read_frags(nxt, 0, fa0, fb0);
        mma(fa1, fb1, sa[3], sb[3]);
        interleave(kFragsScales{}, kCopies{});
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            sa[s] = sa_next[s];
            sb[s] = sb_next[s];
        }
    };
    // A's values at and beyond K become zeros: what is beside them in B is finite (e2m1
    // holds nothing else), and scales past the last block are zero
    auto mask = [&](int st, int s, uint4 (&f)[FM]) __attribute__((always_inline)) {
        const int n = K - (st * 256 + s * 64 + h * kBlock);
        uint32_t m[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int left = n - 8 * d;
            m[d] = left >= 8 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (4 * left)) - 1u;
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            f[i].x &= m[0];
            f[i].y &= m[1];
            f[i].z &= m[2];
            f[i].w &= m[3];
        }
    };
    auto last_stage = [&](const Stage &cur, int st) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s > 0) read_frags(cur, s, fa0, fb0);
            mask(st, s, fa0);
            mma(fa0, fb0, sa[s], sb[s]);
        }
    };
    if (n_st > 0) {
        stage(0, l0);
        stage(1, l1);
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kAll) : "memory");
        read_frags(l0, 0, fa0, fb0);
        read_scales(l0, sa, sb);
        int st = 0;
        for (; st + 2 < n_st; st += 2) {
            full_stage(l0, l1, st);
            full_stage(l1, l0, st + 1);
        }
        if (st + 1 < n_st) full_stage(l0, l1, st++);
        last_stage((st & 1) ? l1 : l0, st);
        // no copy may still be writing this workgroup's LDS when it exits
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    // C.  Register e of lane l in block (i, j): row FM (8 (e / 4) + 4 h + e % 4)
    // + i, column FN (l % 32) + j of the wave's tile, so a store of a lane's FN columns by 32
    // lanes is a run of WN columns of one row.
    typedef Out vec_t __attribute__((ext_vector_type(FN)));
    typedef vec_t packed_t __attribute__((aligned(sizeof(Out))));
    const int row0 = m0 + wm0 + FM * 4 * h, col0 = n0 + wn0 + FN * r;
    Out *const c_lane = static_cast<Out *>(args.C) + (int64_t)row0 * args.ldc + col0;
    const int cols_left = N - col0;
    if (!args.plain && m0 + BM <= M && n0 + BN <= N) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                vec_t v;
#pragma unroll
                for (int j = 0; j < FN; ++j) v[j] = (Out)acc[i][j][e];
                Out *const p = c_lane + (FM * (8 * (e >> 2) + (e & 3)) + i) * args.ldc;
                __builtin_nontemporal_store(v, reinterpret_cast<packed_t *>(p));
            }
    } else {
        // An edge tile (or stores through the L2): offsets from the tile's first element, of which
        // those past row M are outside the range, and lanes without whole FN columns are sent
        // there.  (Tests at every store cost each such tile 1 to 2 us: 768 x 1000 x 1024 5.9 us, not
        // 5.5, 768 x 1001 x 1024 7.2, not 5.9.)  A lane that holds C's last columns and some beyond
        // stores them one by one afterwards.
        constexpr int kSize = sizeof(Out), kNonTemporal = 2;
        const auto rc = rsrc(static_cast<Out *>(args.C) + (int64_t)m0 * args.ldc + n0,
                             (int)(((min(BM, M - m0) - 1) * args.ldc + min(BN, N - n0)) * kSize));
        const uint32_t ldc = (uint32_t)args.ldc * kSize;
        const uint32_t off = (uint32_t)(row0 - m0) * ldc + (uint32_t)(col0 - n0) * kSize;
        const uint32_t whole = FN <= cols_left ? off : kOutside;
        const auto store_edge = [&](auto aux_c) __attribute__((always_inline)) {
            constexpr int kAux = decltype(aux_c)::value;
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    vec_t v;
#pragma unroll
                    for (int j = 0; j < FN; ++j) v[j] = (Out)acc[i][j][e];
                    store_bytes<kAux>(rc, whole + (FM * (8 * (e >> 2) + (e & 3)) + i) * ldc, v);
                }
            const bool some = cols_left > 0 && cols_left < FN;
            if (__builtin_amdgcn_ballot_w64(some) != 0) {
#pragma unroll
                for (int j = 0; j < FN - 1; ++j) {
                    const uint32_t one = some && j < cols_left ? off + j * kSize : kOutside;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
#pragma unroll
                        for (int i = 0; i < FM; ++i)
                            store_bytes<kAux>(rc, one + (FM * (8 * (e >> 2) + (e & 3)) + i) * ldc, (Out)acc[i][j][e]);
                }
            }
        };
        if (args.plain)
            store_edge(std::integral_constant<int, 0>{});
        else
            store_edge(std::integral_constant<int, kNonTemporal>{});
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// Few rows: a tile of 16 FM x 16 FN of C per workgroup, whose W waves take the 128-byte lines
// of K in turn, on 16 x 16 x 128 MFMAs, and join their sums at the end.  Every wave has its own
// three slots of a line of the tile's rows in LDS, filled two lines ahead, so the loop has
// no barrier.  (A fragment's lanes 0 .. 15 are 16 rows: read from memory straight into
// registers it touches 16 lines per instruction, at about 16 bytes a clock per CU; copied in
// whole lines, 8 lanes each, and read from LDS, 64 x 8192 x 8192 took 9.5 us and not 14.3,
// 1 x 8192 x 8192 7.5 and not 7.7.)  Fragment i holds rows FM r + i (r = 0 .. 15), so that a lane's scales of
// its fragments are neighbouring bytes.  One row is bound by reading B (4.7 TB/s, a launch's
// start and end included).  333 x 2081 x 4133 takes 11.6 us on 64 x 64 tiles, 198 workgroups that
// copy 278 KB each, every operand once per tile of the other; its counters show no unit near its
// rate (MFMAs busy 6% of the SIMD cycles, LDS 8%, the waves waiting 32% of theirs): three waves
// a CU, each with its own chain of copies.
template <int FM, int FN, int W, int OT>
__global__ __launch_bounds__(W *kWave) void mx_few_kernel(MxArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int BM = 16 * FM, BN = 16 * FN;
    constexpr int kRows = BM + BN;
    constexpr int kDma = kRows / 8;                // copies of 1 KB (8 rows) per line
    constexpr int kAll = kDma + 4;                 // ... and 4 loads of scales
    struct Slot {
        uint4 rows[kRows][8];
    };
    struct Scales {
        uint32_t a[2], b[2];
    };
    __shared__ Slot s0[W], s1[W], s2[W];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int m0 = (blockIdx.x / args.tiles_n) * BM, n0 = (blockIdx.x % args.tiles_n) * BN;
    const int M = args.M, N = args.N, K = args.K;
    const int blocks = (K + kBlock - 1) / kBlock;
    const int lines = (blocks + 7) / 8;

    const uint8_t *const a_base = args.A + (int64_t)m0 * args.lda;
    const uint8_t *const b_base = args.B + (int64_t)n0 * args.ldb;
    const int a_end = (int)((min(BM, M - m0) - 1) * args.lda) + blocks * 16;
    const int b_end = (int)((min(BN, N - n0) - 1) * args.ldb) + blocks * 16;
    // fragment i's row r of a tile (FM r + i) at LDS row 16 i + r; chunk c at c ^ swizzle16(row)
    auto swizzle16 = [](int row) __attribute__((always_inline)) { return ((row ^ (row >> 1)) & 1) | ((row >> 2) & 2) | (row & 4); };
    uint32_t voff[kDma];
#pragma unroll
    for (int j = 0; j < kDma; ++j) {
        const int cr = j * 8 + (lane >> 3);
        const int chunk = (lane & 7) ^ swizzle16(cr);
        if (j < BM / 8)
            voff[j] = row_offset(FM * (cr % 16) + cr / 16, M - m0, args.lda) + chunk * 16;
        else
            voff[j] = row_offset(FN * ((cr - BM) % 16) + (cr - BM) / 16, N - n0, args.ldb) + chunk * 16;
    }
    // a block's scales are read up to the 16-byte granule that holds the last row's
    const int sa_cols = min(((M + 15) & ~15) - m0, BM), sb_cols = min(((N + 15) & ~15) - n0, BN);
    const int ldsa = (int)args.ldsa, ldsb = (int)args.ldsb;

    // a line past K reads nothing: zeros arrive
    auto copy = [&](int line, Slot &slot, Scales &sc) __attribute__((always_inline)) {
        const int nb = min(blocks - line * 8, 8);
        const auto ra = rsrc(a_base + line * 128, nb > 0 ? a_end - line * 128 : 0);
        const auto rb = rsrc(b_base + line * 128, nb > 0 ? b_end - line * 128 : 0);
        const auto rsa = rsrc(args.SA + (int64_t)line * 8 * args.ldsa + m0, max((nb - 1) * ldsa + sa_cols, 0));
        const auto rsb = rsrc(args.SB + (int64_t)line * 8 * args.ldsb + n0, max((nb - 1) * ldsb + sb_cols, 0));
#pragma unroll
        for (int j = 0; j < kDma; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(j < BM / 8 ? ra : rb, LDS_PTR(&slot.rows[j * 8][0]), 16, voff[j], 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            sc.a[q] = load_bytes<FM>(rsa, (4 * q + g) * ldsa + FM * r);
            sc.b[q] = load_bytes<FN>(rsb, (4 * q + g) * ldsb + FN * r);
        }
    };

    floatx4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = floatx4_t{0, 0, 0, 0};

    auto turn = [&](int line, Slot &slot, Scales &sc) __attribute__((always_inline)) {
        // this line's copies have landed; the two lines' after it may be in flight
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kAll) : "memory");
        uint4 fa[2][FM], fb[2][FN];
        const uint32_t sa[2] = {sc.a[0], sc.a[1]}, sb[2] = {sc.b[0], sc.b[1]};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int ch = (4 * q + g) ^ swizzle16(r);
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[q][i] = slot.rows[16 * i + r][ch];
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[q][j] = slot.rows[BM + 16 * j + r][ch];
        }
        // the slot is read: it takes the line after the next two
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        copy(line + 3 * W, slot, sc);
        if (line * 256 + 256 > K) {
            // A's values at and beyond K become zeros: what is beside them in B is finite (e2m1
            // holds nothing else), and scales past the last block are zero
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int n = K - (line * 256 + q * 128 + g * kBlock);
                uint32_t m[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int left = n - 8 * d;
                    m[d] = left >= 8 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (4 * left)) - 1u;
                }
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    uint4 &v = fa[q][i];
                    v = make_uint4(v.x & m[0], v.y & m[1], v.z & m[2], v.w & m[3]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
            static_for<FM>([&](auto i_c) __attribute__((always_inline)) {
                static_for<FN>([&](auto j_c) __attribute__((always_inline)) {
                    constexpr int i = decltype(i_c)::value, j = decltype(j_c)::value;
                    acc[i][j] = mfma_fp4<i, j>(fa[q][i], fb[q][j], acc[i][j], sa[q], sb[q]);
                });
            });
    };
    if (wave < lines) {
        Scales c0, c1, c2;
        copy(wave, s0[wave], c0);
        copy(wave + W, s1[wave], c1);
        copy(wave + 2 * W, s2[wave], c2);
        for (int line = wave; line < lines; line += 3 * W) {
            turn(line, s0[wave], c0);
            if (line + W >= lines) break;
            turn(line + W, s1[wave], c1);
            if (line + 2 * W >= lines) break;
            turn(line + 2 * W, s2[wave], c2);
        }
        // no copy may still be writing this workgroup's LDS when it exits
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    join_and_store<FM, FN, W, OT, sizeof(Slot) / 4, BM, true>(acc, reinterpret_cast<float *>(&s0[0]), args, m0, n0, tid, lane, wave);
#endif  // __HIP_DEVICE_COMPILE__
}

// 16-bit activations times MXFP4 weights.  The codes become the 16-bit type exactly
// (e2m1 values need two significant bits); an MFMA of 32 values of K covers one block,
// and its result is scaled by the block's 2^(byte - 127) as it is added to the sum, in
// binary32.  (With the scale in an f16 operand instead, weights are exact for scales of
// 2^-23 .. 2^13, bytes 104 .. 140, only: half of 2^-23 is f16's least value, and 6 * 2^14 is
// above its largest.  The kernels take any byte and have one path.)
template <int T>
__device__ __forceinline__ floatx4_t mfma16(const uint4 &a, const uint4 &b, const floatx4_t &c) {
    if constexpr (T == kF16) {
        half8_t x, y;
        __builtin_memcpy(&x, &a, 16);
        __builtin_memcpy(&y, &b, 16);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
    } else {
        bf16x8_t x, y;
        __builtin_memcpy(&x, &a, 16);
        __builtin_memcpy(&y, &b, 16);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
    }
}

// the eight values of a dword of codes, exact: as f16, or times a power of two as bf16
__device__ __forceinline__ uint4 widen_f16(uint32_t w) {
    uint32_t x[4];
    static_for<4>([&](auto s_c) __attribute__((always_inline)) {
        constexpr int s = decltype(s_c)::value;
        const half2_t h = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, s);
        x[s] = __builtin_bit_cast(uint32_t, h);
    });
    return make_uint4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ uint4 widen_bf16(uint32_t w, float scale) {
    uint32_t x[4];
    static_for<4>([&](auto s_c) __attribute__((always_inline)) {
        constexpr int s = decltype(s_c)::value;
        const bf16x2_t h = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, s);
        x[s] = __builtin_bit_cast(uint32_t, h);
    });
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// Byte j of v moved to where a binary32 has its exponent, which is all that the conversions read
// of a scale (0 is 2^-127 there and 255 gives NaN): what is left beside it does not matter.
__device__ __forceinline__ float scale_bits(uint32_t v, int j) {
    return __builtin_bit_cast(float, j < 3 ? v << (23 - 8 * j) : v >> 1);
}

// binary32 of that scale, NaN included: a code of 1.0 converted with it
__device__ __forceinline__ float scale_f32(float bits) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(0x22u, bits, 0)[0];
}

// How a step of 64 values of K (a line of a row of A, two blocks of B) is shared out over the
// four lane groups g = l / 16 of two MFMAs u.
//
// bf16: its exponents reach the weights' (a code times 2^(byte - 127) is exact, subnormals
// included, which the MFMA keeps), so the scale goes into the operand: group g takes half a
// block, values 16 g .. + 15 of the step, and MFMA u its values 8 u .. + 7.
// f16: group g takes dword g of a block, MFMA u covers block u alone, and its result is scaled
// as it is added: 4 vector instructions per MFMA, as many cycles as it takes itself.
template <int T> struct A16Map;
template <> struct A16Map<kBF16> {
    static __device__ __forceinline__ int chunk(int u, int g) { return 2 * g + u; }       // of A's 8
    static __device__ __forceinline__ int swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }
};
template <> struct A16Map<kF16> {
    static __device__ __forceinline__ int chunk(int u, int g) { return 4 * u + g; }
    static __device__ __forceinline__ int swizzle(int r) { return ((r ^ (r >> 1)) & 1) | ((r >> 2) & 2) | (r & 4); }
};

// Few rows of 16-bit activations: the scheme of mx_few_kernel in steps of a line of A, W
// waves with S slots each (as many as LDS holds: what is on its way bounds the rate), so W
// neighbouring waves share a line of B.  RA: the rows of A that are staged; with eight
// (M <= 8) a fragment's rows repeat them and LDS holds more steps.  One row is bound by reading
// B (8192 x 8192 9.3 us, 3.8 TB/s; steps of a whole line of B, 128 bytes a row, took 9.9 there,
// 4.0 instead of 4.7 for 4096 x 4096, and 20 instead of 12.4 for 37 rows of f16).  37 x 4096 x
// 8192 takes 9.8 us in bf16 and 12.4 in f16, whose widening and scaling need 1.8 times the vector
// instructions; B is copied three times, once per tile of 16 rows, and the waves wait 37 and 41%
// of their cycles.
template <int T, int RA, int FN, int W, int S, int OT>
__global__ __launch_bounds__(W *kWave) void a16_few_kernel(MxArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Map = A16Map<T>;
    constexpr int FM = (RA + 15) / 16, BN = 16 * FN;
    constexpr int kDmaA = RA / 8, kDmaB = (BN + 31) / 32;   // copies of 1 KB (8 rows of A, 32 of B) per step
    constexpr int kSc = T == kBF16 ? 1 : 2;                 // loads of scales per step
    constexpr int kAll = kDmaA + kDmaB + kSc;
    static_assert(RA == 8 || RA % 16 == 0, "rows of A");
    static_assert(S >= 2 && S <= 6 && (S - 1) * kAll <= 63, "vmcnt holds at most 63 outstanding loads");
    struct Slot {
        uint4 a[RA][8];             // chunk c of row r at c ^ Map::swizzle(r)
        uint4 b[32 * kDmaB][2];     // chunk c of row r at c ^ ((r / 8) % 2)
    };
    struct Scales {
        uint32_t v[kSc];
    };
    // separate objects: a read of one slot does not wait for the copies into the others
    __shared__ Slot s0[W], s1[W];
    __shared__ typename std::conditional<(S > 2), Slot, char>::type s2[S > 2 ? W : 1];
    __shared__ typename std::conditional<(S > 3), Slot, char>::type s3[S > 3 ? W : 1];
    __shared__ typename std::conditional<(S > 4), Slot, char>::type s4[S > 4 ? W : 1];
    __shared__ typename std::conditional<(S > 5), Slot, char>::type s5[S > 5 ? W : 1];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int m0 = (blockIdx.x / args.tiles_n) * RA, n0 = (blockIdx.x % args.tiles_n) * BN;
    const int M = args.M, N = args.N, K = args.K;
    const int blocks = (K + kBlock - 1) / kBlock;
    const int steps = (blocks + 1) / 2;

    const uint8_t *const a_base = args.A + (int64_t)m0 * args.lda;
    const uint8_t *const b_base = args.B + (int64_t)n0 * args.ldb;
    const int a_end = (int)((min(RA, M - m0) - 1) * args.lda) + ((2 * K + 15) & ~15);
    const int b_end = (int)((min(BN, N - n0) - 1) * args.ldb) + blocks * 16;
    const int sb_cols = min(((N + 15) & ~15) - n0, BN), ldsb = (int)args.ldsb;
    uint32_t va[kDmaA], vb[kDmaB];
#pragma unroll
    for (int j = 0; j < kDmaA; ++j) {
        const int cr = j * 8 + (lane >> 3);
        va[j] = row_offset(cr, M - m0, args.lda) + ((lane & 7) ^ Map::swizzle(cr)) * 16;
    }
#pragma unroll
    for (int j = 0; j < kDmaB; ++j) {
        const int cr = j * 32 + (lane >> 1);   // column FN n + j at LDS row 16 j + n
        vb[j] = row_offset(FN * (cr % 16) + cr / 16, cr < BN ? N - n0 : 0, args.ldb) + ((lane & 1) ^ ((cr >> 3) & 1)) * 16;
    }
    // a step past K reads nothing: zeros arrive
    auto copy = [&](int step, Slot &slot, Scales &sc) __attribute__((always_inline)) {
        const int nb = min(blocks - step * 2, 2);
        const auto ra = rsrc(a_base + step * 128, nb > 0 ? a_end - step * 128 : 0);
        const auto rb = rsrc(b_base + step * 32, nb > 0 ? b_end - step * 32 : 0);
        const auto rs = rsrc(args.SB + (int64_t)step * 2 * args.ldsb + n0, max((nb - 1) * ldsb + sb_cols, 0));
#pragma unroll
        for (int j = 0; j < kDmaB; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, LDS_PTR(&slot.b[j * 32][0]), 16, vb[j], 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kDmaA; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, LDS_PTR(&slot.a[j * 8][0]), 16, va[j], 0, 0, 0);
#pragma unroll
        for (int u = 0; u < kSc; ++u) sc.v[u] = load_bytes<FN>(rs, (T == kBF16 ? g >> 1 : u) * ldsb + FN * r);
    };

    floatx4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = floatx4_t{0, 0, 0, 0};

    auto turn = [&](int step, Slot &slot, Scales &sc) __attribute__((always_inline)) {
        // this step's copies have landed; those of the S - 1 after it may be in flight
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * kAll) : "memory");
        uint4 fa[2][FM];
        uint32_t w[FN][2];
        const int ra = RA == 8 ? r & 7 : r, flip = (r >> 3) & 1;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t *const row = reinterpret_cast<const uint32_t *>(&slot.b[16 * j + r][0]);
            if constexpr (T == kBF16) {
                w[j][0] = row[((g >> 1) ^ flip) * 4 + 2 * (g & 1)];
                w[j][1] = row[((g >> 1) ^ flip) * 4 + 2 * (g & 1) + 1];
            } else {
                w[j][0] = row[flip * 4 + g];
                w[j][1] = row[(1 ^ flip) * 4 + g];
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[u][i] = slot.a[16 * i + ra][Map::chunk(u, g) ^ Map::swizzle(ra)];
        // (the scales leave the registers that the copy loads into, or the compiler would load
        // into others and wait at once to move them)
        uint32_t sb[kSc];
#pragma unroll
        for (int u = 0; u < kSc; ++u) {
            sb[u] = sc.v[u];
            asm volatile("" : "+v"(sb[u]));
        }
        // the slot is read: it takes the step after the next S - 1
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        copy(step + S * W, slot, sc);
        if (step * 64 + 64 > K) {
            // A's values at and beyond K may be anything, a NaN too: they become zeros, and in bf16,
            // where a code times a scale of 2^126 or 2^127 may be infinite, B's codes too (scales
            // past the last block are zero)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = K - step * 64 - 8 * Map::chunk(u, g);
                uint32_t m[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) m[d] = n >= 2 * d + 2 ? 0xFFFFFFFFu : n == 2 * d + 1 ? 0xFFFFu : 0u;
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    uint4 &v = fa[u][i];
                    v = make_uint4(v.x & m[0], v.y & m[1], v.z & m[2], v.w & m[3]);
                }
                if constexpr (T == kBF16) {
#pragma unroll
                    for (int j = 0; j < FN; ++j) w[j][u] &= n >= 8 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (4 * n)) - 1u;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (T == kBF16) {
                    const uint4 b = widen_bf16(w[j][u], scale_bits(sb[0], j));
#pragma unroll
                    for (int i = 0; i < FM; ++i) acc[i][j] = mfma16<T>(fa[u][i], b, acc[i][j]);
                } else {
                    const uint4 b = widen_f16(w[j][u]);
                    const float scale = scale_f32(scale_bits(sb[u], j));
#pragma unroll
                    for (int i = 0; i < FM; ++i) {
                        const floatx4_t p = mfma16<T>(fa[u][i], b, floatx4_t{0, 0, 0, 0});
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], scale, acc[i][j][e]);
                    }
                }
            }
    };
    if (wave < steps) {
        Scales c0, c1, c2, c3, c4, c5;
        copy(wave, s0[wave], c0);
        copy(wave + W, s1[wave], c1);
        if constexpr (S > 2) copy(wave + 2 * W, s2[wave], c2);
        if constexpr (S > 3) copy(wave + 3 * W, s3[wave], c3);
        if constexpr (S > 4) copy(wave + 4 * W, s4[wave], c4);
        if constexpr (S > 5) copy(wave + 5 * W, s5[wave], c5);
        for (int step = wave; step < steps; step += S * W) {
            turn(step, s0[wave], c0);
            if (step + W >= steps) break;
            turn(step + W, s1[wave], c1);
            if constexpr (S > 2) {
                if (step + 2 * W >= steps) break;
                turn(step + 2 * W, s2[wave], c2);
            }
            if constexpr (S > 3) {
                if (step + 3 * W >= steps) break;
                turn(step + 3 * W, s3[wave], c3);
            }
            if constexpr (S > 4) {
                if (step + 4 * W >= steps) break;
                turn(step + 4 * W, s4[wave], c4);
            }
            if constexpr (S > 5) {
                if (step + 5 * W >= steps) break;
                turn(step + 5 * W, s5[wave], c5);
            }
        }
        // no copy may still be writing this workgroup's LDS when it exits
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    join_and_store<FM, FN, W, OT, sizeof(Slot) / 4, RA, false>(acc, reinterpret_cast<float *>(&s0[0]), args, m0, n0, tid, lane, wave);
#endif  // __HIP_DEVICE_COMPILE__
}

// Many rows of 16-bit activations: a BM x BN tile of C per workgroup on 16 x 16 x 32
// MFMAs.  A is staged in lines of 128 bytes (64 values of K), two deep, as the FP16 GEMM
// does; B in lines of 128 bytes too, which are 256 values of K, two deep, so a line of B
// serves four steps of A and is copied a quarter per step.  The codes become the 16-bit
// type in registers, once per wave and step.
//
// Fragment j holds columns FN n + j (n = l % 16) of the wave's, so a lane's scales of its
// fragments are one dword and its results neighbouring columns of C.
//
// 2048 x 8192 x 8192 takes 172 to 182 us by GPU in bf16 (1.5 to 1.6 PFLOP/s; the FP16 GEMM of
// this library reaches 1.24 at 8192^3) and 262 to 275 in f16 (1.0).  Counters: MFMAs busy 72% of
// the cycles in bf16, at 1.9 GHz, the waves waiting 28% of theirs, and 43% in f16, whose scaled
// sums cost as many cycles of vector instructions as of MFMAs.  Both spend 0.8 cycles per LDS
// instruction on bank conflicts; another swizzle of B's lines did not move them.  A loop of
// nothing but these MFMAs on normal values runs at 1.70 PFLOP/s in bf16 and 1.60 in f16.
template <int T, int BM, int BN, int WM, int WN, int OT>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * kWave, 2) void a16_tile_kernel(MxArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Out = typename ElemOf<OT>::type;
    using Map = A16Map<T>;
    constexpr int NW = (BM / WM) * (BN / WN);
    constexpr int kWavesN = BN / WN;
    constexpr int FM = WM / 16, FN = WN / 16, FH = FM / 2;
    constexpr int kDmaA = BM / 8 / NW;             // copies of 1 KB (8 rows) per wave per step
    constexpr int kDmaB = BN / 8 / NW / 4;         // ... of a quarter of B's line
    constexpr int kSc = BN / 128;                  // waves that copy 1 KB of scales
    static_assert(BM % (8 * NW) == 0 && BN % (32 * NW) == 0 && BN % 128 == 0 && FM % 2 == 0 && FN == 4, "tile");
    struct LineB {
        uint4 rows[BN][8];
        uint4 sc[BN / 2 + 64];   // bytes: [8 blocks of BN columns | unused]
    };
    __shared__ uint4 la0[BM][8], la1[BM][8];
    __shared__ LineB lb0, lb1;
    using LineA = uint4[BM][8];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int M = args.M, N = args.N, K = args.K;
    int tile_m, tile_n;
    tile_of<4, true>(args.tiles_m, args.tiles_n, tile_m, tile_n);
    const int m0 = tile_m * BM, n0 = tile_n * BN;
    const int blocks = (K + kBlock - 1) / kBlock;
    const int n_ln = (blocks + 7) / 8;             // lines of B; four steps each
    const int whole16 = 2 * (K & ~7);              // bytes of a row's whole chunks of A

    const uint8_t *const a_base = args.A + (int64_t)m0 * args.lda;
    const uint8_t *const b_base = args.B + (int64_t)n0 * args.ldb;
    const int a_end = (int)((min(BM, M - m0) - 1) * args.lda) + ((2 * K + 15) & ~15);
    const int b_end = (int)((min(BN, N - n0) - 1) * args.ldb) + blocks * 16;
    const int sb_cols = min(((N + 15) & ~15) - n0, BN);

    uint32_t va[kDmaA], vb[4 * kDmaB];
    // (rows of a lane's copies differ by multiples of 16, so their swizzles are the same)
    static_assert(NW % 2 == 0, "copies of a wave are whole 16-row groups apart");
    const int a_chunk = ((lane & 7) ^ Map::swizzle(wave * 8 + (lane >> 3))) * 16;
#pragma unroll
    for (int j = 0; j < kDmaA; ++j) {
        const int cr = (j * NW + wave) * 8 + (lane >> 3);
        va[j] = row_offset(cr, M - m0, args.lda) + a_chunk;
    }
#pragma unroll
    for (int j = 0; j < 4 * kDmaB; ++j) {
        const int cr = (j * NW + wave) * 8 + (lane >> 3);
        const int col = cr / WN * WN + FN * (cr % 16) + cr % WN / 16;   // column FN n + j at LDS row 16 j + n
        vb[j] = row_offset(col, N - n0, args.ldb) + ((lane & 7) ^ swizzle8(cr)) * 16;
    }
    const bool sc_none = wave >= kSc;
    const int sd = wave * 64 + lane;
    const int sc_ld = sc_none ? 0 : (int)args.ldsb, sc_cols = sc_none ? 0 : sb_cols;
    const uint32_t soff = (uint32_t)(sd / (BN / 16) * sc_ld) + sd % (BN / 16) * 16;

    // step `step` of A; a chunk that reaches past K becomes zeros (its lane's offset leaves the
    // range), as what lies there, a NaN say, is not to enter a sum
    auto copy_a = [&](int step, LineA &buf) __attribute__((always_inline)) {
        const int kb = step * 128;
        const auto ra = rsrc(a_base + kb, max(a_end - kb, 0));
#pragma unroll
        for (int j = 0; j < kDmaA; ++j) {
            const uint32_t off = kb + a_chunk < whole16 ? va[j] : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, LDS_PTR(&buf[(j * NW + wave) * 8][0]), 16, off, 0, 0, 0);
        }
    };
    // quarter q of line ln of B; with the first one, the line's scales
    auto copy_b = [&](int ln, auto q_c, LineB &buf) __attribute__((always_inline)) {
        constexpr int q = decltype(q_c)::value;
        const int nb = min(blocks - ln * 8, 8);   // at most 0 past K: nothing is read, zeros arrive
        const auto rb = rsrc(b_base + ln * 128, nb > 0 ? b_end - ln * 128 : 0);
#pragma unroll
        for (int j = q * kDmaB; j < (q + 1) * kDmaB; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, LDS_PTR(&buf.rows[(j * NW + wave) * 8][0]), 16, vb[j], 0, 0, 0);
        if constexpr (q == 0) {
            // (a scale row holds at least the tile's columns, so the range of no blocks is not positive)
            const auto rs = rsrc(args.SB + n0 + (int64_t)ln * 8 * sc_ld, max((nb - 1) * sc_ld + sc_cols, 0));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, LDS_PTR(&buf.sc[sc_none ? kSc * 64 : wave * 64]), 16, soff, 0, 0, 0);
        }
    };

    const int wm0 = (wave / kWavesN) * WM, wn0 = (wave % kWavesN) * WN;
    const int r = lane & 15, g = lane >> 4;
    auto read_a = [&](const LineA &buf, int u, int half, uint4 (&fa)[FH]) __attribute__((always_inline)) {
        const int ch = Map::chunk(u, g) ^ Map::swizzle(r);
#pragma unroll
        for (int i = 0; i < FH; ++i) fa[i] = buf[wm0 + (half * FH + i) * 16 + r][ch];
    };
    // the codes and scales of step t of a line: bf16 the half block of this group, f16 dword g
    // of the step's two blocks
    struct Codes {
        uint32_t w[FN][2];
        uint32_t s[T == kBF16 ? 1 : 2];
    };
    auto read_b = [&](const LineB &buf, int t, Codes &c) __attribute__((always_inline)) {
        const uint32_t *const sc = reinterpret_cast<const uint32_t *>(&buf.sc[0]) + (wn0 + FN * r) / 4;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t *const row = reinterpret_cast<const uint32_t *>(&buf.rows[wn0 + j * 16 + r][0]);
            if constexpr (T == kBF16) {
                const uint32_t *const half = &row[((2 * t + (g >> 1)) ^ swizzle8(r)) * 4 + 2 * (g & 1)];
                c.w[j][0] = half[0];
                c.w[j][1] = half[1];
            } else {
                c.w[j][0] = row[((2 * t) ^ swizzle8(r)) * 4 + g];
                c.w[j][1] = row[((2 * t + 1) ^ swizzle8(r)) * 4 + g];
            }
        }
        if constexpr (T == kBF16) {
            c.s[0] = sc[(2 * t + (g >> 1)) * (BN / 4)];
        } else {
            c.s[0] = sc[2 * t * (BN / 4)];
            c.s[1] = sc[(2 * t + 1) * (BN / 4)];
        }
    };
    // B fragments of MFMA u of a step, and (f16) the columns' scales of its block
    struct FragB {
        uint4 f[FN];
        float s[T == kBF16 ? 1 : FN];
    };
    // (bf16: where A's chunk has been zeroed, `live` is false and the scale is 2^-127, or a code
    // times 2^126 or 2^127 could be infinite there)
    auto make_b = [&](const Codes &c, int u, bool live, FragB &b) __attribute__((always_inline)) {
        const uint32_t sc = T != kBF16 ? c.s[u] : live ? c.s[0] : 0;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if constexpr (T == kBF16) {
                b.f[j] = widen_bf16(c.w[j][u], scale_bits(sc, j));
            } else {
                b.f[j] = widen_f16(c.w[j][u]);
                b.s[j] = scale_f32(scale_bits(sc, j));
            }
        }
    };

    floatx4_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = floatx4_t{0, 0, 0, 0};
    auto mma = [&](int half, const uint4 (&fa)[FH], const FragB &b) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FH; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                floatx4_t &c = acc[half * FH + i][j];
                if constexpr (T == kBF16) {
                    c = mfma16<T>(fa[i], b.f[j], c);
                } else {
                    const floatx4_t p = mfma16<T>(fa[i], b.f[j], floatx4_t{0, 0, 0, 0});
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = __builtin_fmaf(p[e], b.s[j], c[e]);
                }
            }
    };
    // The last K % 8 values, which the loop leaves out, first: one MFMA per block, from memory,
    // in which lane group 0 holds that chunk and the others zeros
    if (K % 8 != 0) {
        const int kt = K & ~7;
        const auto ra = rsrc(a_base, a_end), rb = rsrc(b_base, b_end);
        const auto rs = rsrc(args.SB + n0 + (int64_t)(kt / kBlock) * args.ldsb, sb_cols);
        Codes c;
        FragB b;
        uint4 fa[FH];
        const uint32_t sc = load_bytes<4>(rs, wn0 + FN * r);
        const uint32_t inside = g == 0 ? (1u << (4 * (K % 8))) - 1u : 0u;
#pragma unroll
        for (int j = 0; j < FN; ++j)
            c.w[j][0] = load_bytes<4>(rb, row_offset(wn0 + FN * r + j, N - n0, args.ldb) + kt / 2) & inside;
        c.s[0] = sc;
        make_b(c, 0, true, b);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int i = 0; i < FH; ++i) {
                const int row = wm0 + (half * FH + i) * 16 + r;
                uint4 v = load16(ra, g == 0 ? row_offset(row, M - m0, args.lda) + 2 * kt : kOutside);
                uint32_t m[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) m[d] = K % 8 >= 2 * d + 2 ? 0xFFFFFFFFu : K % 8 == 2 * d + 1 ? 0xFFFFu : 0u;
                fa[i] = make_uint4(v.x & m[0], v.y & m[1], v.z & m[2], v.w & m[3]);
            }
            if (half == 0)
                mma(0, fa, b);
            else
                mma(1, fa, b);
        }
    }

    // whether this lane's half of MFMA u of the step `step` lies before K & ~7
    auto live = [&](int step, int u) __attribute__((always_inline)) { return (K & ~7) - step * 64 - 8 * u > 16 * g; };
    uint4 fl[FH], fu[FH];
    Codes codes;
    FragB b0, b1;
    // step 4 ln + t from `cur`, whose first lower half is in fl, codes in `codes` and first B
    // fragments in b0; afterwards the same of the next step, from `nxt` and, past the line's last step, from the other
    // line.  Copies step + 2 of A into `cur` and the next quarter of the line after the next
    // step's into the buffer that is free
    auto step = [&](LineA &cur, const LineA &nxt, LineB &line, LineB &other, int ln, auto t_c)
        __attribute__((always_inline)) {
        constexpr int t = decltype(t_c)::value;
        read_a(cur, 0, 1, fu);
        mma(0, fl, b0);
        __builtin_amdgcn_sched_barrier(0);
        make_b(codes, 1, live(4 * ln + t, 1), b1);
        read_a(cur, 1, 0, fl);
        mma(1, fu, b0);
        __builtin_amdgcn_sched_barrier(0);
        read_a(cur, 1, 1, fu);
        mma(0, fl, b1);
        // this wave's copies have landed and its reads of `cur` (and, after a line's last step,
        // of `line`) are done; after the barrier the same holds for every wave
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        copy_a(4 * ln + t + 2, cur);
        if constexpr (t < 3)
            copy_b(ln + 1, std::integral_constant<int, (t + 1) & 3>{}, other);
        else
            copy_b(ln + 2, std::integral_constant<int, 0>{}, line);
        read_a(nxt, 0, 0, fl);
        read_b(t < 3 ? line : other, (t + 1) & 3, codes);
        mma(1, fu, b1);
        make_b(codes, 0, live(4 * ln + t + 1, 0), b0);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto whole_line = [&](LineB &line, LineB &other, int ln) __attribute__((always_inline)) {
        step(la0, la1, line, other, ln, std::integral_constant<int, 0>{});
        step(la1, la0, line, other, ln, std::integral_constant<int, 1>{});
        step(la0, la1, line, other, ln, std::integral_constant<int, 2>{});
        step(la1, la0, line, other, ln, std::integral_constant<int, 3>{});
    };
    if (n_ln > 0) {
        copy_a(0, la0);
        copy_a(1, la1);
        static_for<4>([&](auto q_c) __attribute__((always_inline)) { copy_b(0, q_c, lb0); });
        copy_b(1, std::integral_constant<int, 0>{}, lb1);
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        read_a(la0, 0, 0, fl);
        read_b(lb0, 0, codes);
        make_b(codes, 0, live(0, 0), b0);
        int ln = 0;
        for (; ln + 1 < n_ln; ln += 2) {
            whole_line(lb0, lb1, ln);
            whole_line(lb1, lb0, ln + 1);
        }
        if (ln < n_ln) whole_line(lb0, lb1, ln);
        // no copy may still be writing this workgroup's LDS when it exits
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    // C.  Register e of lane l in block (i, j): row 16 i + 4 (l / 16) + e, column
    // FN (l % 16) + j of the wave's tile: a store writes runs of WN columns of four rows
    typedef Out vec_t __attribute__((ext_vector_type(FN)));
    typedef vec_t packed_t __attribute__((aligned(sizeof(Out))));
    const int row0 = m0 + wm0 + 4 * g, col0 = n0 + wn0 + FN * r;
    Out *const c_lane = static_cast<Out *>(args.C) + (int64_t)row0 * args.ldc + col0;
    const int rows_left = M - row0, cols_left = N - col0;
    auto store_all = [&](auto interior_c, auto plain_c) __attribute__((always_inline)) {
        constexpr bool kInterior = decltype(interior_c)::value, kPlain = decltype(plain_c)::value;
        const int whole = FN <= cols_left ? rows_left : 0;   // rows that this lane stores FN columns of
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 16 * i + e;
                Out *const p = c_lane + row * args.ldc;
                vec_t v;
#pragma unroll
                for (int j = 0; j < FN; ++j) v[j] = (Out)acc[i][j][e];
                if (kInterior || row < whole) {
                    if constexpr (kPlain)
                        *reinterpret_cast<packed_t *>(p) = v;
                    else
                        __builtin_nontemporal_store(v, reinterpret_cast<packed_t *>(p));
                }
            }
        // a lane that holds C's last columns and some beyond: one by one, in a pass of their own
        // (tested at every store they cost each edge tile 1 us more; the offsets of mx_tile_kernel
        // need more registers than the 256 x 256 tile has left: 2048 x 8192 x 8192 bf16 190 us, not
        // 178)
        const bool some = cols_left > 0 && cols_left < FN;
        if (!kInterior && __builtin_amdgcn_ballot_w64(some) != 0) {
#pragma unroll
            for (int j = 0; j < FN - 1; ++j) {
                const int last = some && j < cols_left ? rows_left : 0;
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (16 * i + e < last) c_lane[(16 * i + e) * args.ldc + j] = (Out)acc[i][j][e];
            }
        }
    };
    if (args.plain) {
        // (the markers keep the compiler from joining these stores with the others')
        asm volatile("; C through the L2" ::: "memory");
        store_all(std::false_type{}, std::true_type{});
        asm volatile("; C through the L2, end" ::: "memory");
    } else if (m0 + BM <= M && n0 + BN <= N) {
        store_all(std::true_type{}, std::false_type{});
    } else {
        store_all(std::false_type{}, std::false_type{});
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// host side

constexpr int64_t kMaxRowBytes = int64_t(1) << 22;  // 4 MiB, as for the other operands

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int finish(hipError_t e, hipStream_t s) {
    // PDGEMM_SYNC_CHECK=1 at the first call: every call waits for its kernel
    static const bool check = [] {
        const char *v = getenv("PDGEMM_SYNC_CHECK");
        return v && strcmp(v, "1") == 0;
    }();
    if (e == hipSuccess && check) e = hipStreamSynchronize(s);
    return (int)e;
}

int run(const void *fn, int64_t blocks, int threads, void *args, void *stream) {
    // a launch counts its work-items in 32 bits
    if (blocks * threads > (int64_t)UINT32_MAX) return PDGEMM_EINVAL_DIM;
    void *kargs[] = {args};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(hipLaunchKernel(fn, dim3((unsigned)blocks), dim3((unsigned)threads), kargs, 0, s), s);
}

bool known_type(int t) { return t == kF32 || t == kF16 || t == kBF16; }

// The checks of one MXFP4 operand of `rows` x K, in two steps, so that a call's size
// errors come before its pointer errors whichever operand has them.
int check_mx_sizes(int64_t rows, int64_t K, int64_t ldq, int64_t lds) {
    if (rows < 0 || K < 0 || rows > INT32_MAX || K > (int64_t(1) << 30)) return PDGEMM_EINVAL_DIM;
    if (ldq < K || lds < rows) return PDGEMM_EINVAL_LD;
    return PDGEMM_OK;
}
int check_mx_memory(const void *q, int64_t ldq, const void *s, int64_t lds) {
    if (!q || !s) return PDGEMM_ENULL;
    if (ldq > 2 * kMaxRowBytes || lds > kMaxRowBytes) return PDGEMM_EINVAL_LD;
    if (ldq % 32 || lds % 16 || ((uintptr_t)q & 15) || ((uintptr_t)s & 15)) return PDGEMM_EALIGN;
    return PDGEMM_OK;
}

// rows of a dense matrix with only its element's alignment
int check_plain(const void *p, int64_t ld, int type) {
    if (!p) return PDGEMM_ENULL;
    if (ld > kMaxRowBytes / elem_size(type)) return PDGEMM_EINVAL_LD;
    if ((uintptr_t)p & (elem_size(type) - 1)) return PDGEMM_EALIGN;
    return PDGEMM_OK;
}

template <int T>
int launch_quant(const QuantArgs &base, void *stream) {
    QuantArgs args = base;
    if (args.qt) {
        args.tiles_k = (int)cdiv(args.K, 128);
        const void *fn = args.q ? reinterpret_cast<const void *>(&mx_quant_cols_kernel<T, true>)
                                : reinterpret_cast<const void *>(&mx_quant_cols_kernel<T, false>);
        return run(fn, cdiv(args.rows, 256) * args.tiles_k, 512, &args, stream);
    }
    args.tiles_k = (int)cdiv(args.K, 64 * 16 / elem_size(T));
    return run(reinterpret_cast<const void *>(&mx_quant_rows_kernel<T, 2>), cdiv(args.rows, 8) * args.tiles_k, 256, &args,
               stream);
}

template <int T>
const void *dequant_ptr(bool lines) {
    return lines ? reinterpret_cast<const void *>(&mx_dequant_kernel<T, 4, true>)
                 : reinterpret_cast<const void *>(&mx_dequant_kernel<T, 4, false>);
}

struct Config {
    int bm, bn, threads;
};

constexpr Config kMxConfigs[] = {
    {256, 256, 512}, {128, 128, 256},                // 0-1: tiles
    {64, 64, 192}, {64, 32, 256},                    // 2-3: K split over the waves
    {32, 64, 256}, {32, 32, 256}, {32, 16, 256},     // 4-6
    {16, 64, 256}, {16, 32, 256}, {16, 16, 256},     // 7-9
};
constexpr int kNumMxConfigs = sizeof(kMxConfigs) / sizeof(kMxConfigs[0]);

template <int C, int OT>
const void *mx_few_ptr() {
    constexpr Config c = kMxConfigs[C];
    return reinterpret_cast<const void *>(&mx_few_kernel<c.bm / 16, c.bn / 16, c.threads / 64, OT>);
}

template <int OT>
const void *mx_ptr(int cfg) {
    switch (cfg) {
    case 0: return reinterpret_cast<const void *>(&mx_tile_kernel<256, 256, 128, 64, OT>);
    case 1: return reinterpret_cast<const void *>(&mx_tile_kernel<128, 128, 64, 64, OT>);
    case 2: return mx_few_ptr<2, OT>();
    case 3: return mx_few_ptr<3, OT>();
    case 4: return mx_few_ptr<4, OT>();
    case 5: return mx_few_ptr<5, OT>();
    case 6: return mx_few_ptr<6, OT>();
    case 7: return mx_few_ptr<7, OT>();
    case 8: return mx_few_ptr<8, OT>();
    default: return mx_few_ptr<9, OT>();
    }
}

constexpr Config kA16Configs[] = {
    {256, 256, 512}, {128, 128, 256},                         // 0-1: tiles
    {64, 32, 512}, {48, 32, 512},                             // 2-3: K split over the waves
    {32, 64, 256}, {32, 32, 512},                             // 4-5
    {16, 64, 512}, {16, 32, 512}, {16, 16, 512},              // 6-8
    {8, 64, 512}, {8, 32, 1024}, {8, 16, 512},                // 9-11
    {64, 64, 512},                                            // 12
};
constexpr int kNumA16Configs = sizeof(kA16Configs) / sizeof(kA16Configs[0]);

template <int T, int C, int S, int OT>
const void *a16_few_ptr() {
    constexpr Config c = kA16Configs[C];
    return reinterpret_cast<const void *>(&a16_few_kernel<T, c.bm, c.bn / 16, c.threads / 64, S, OT>);
}

template <int T, int OT>
const void *a16_ptr(int cfg) {
    switch (cfg) {
    case 0: return reinterpret_cast<const void *>(&a16_tile_kernel<T, 256, 256, 128, 64, OT>);
    case 1: return reinterpret_cast<const void *>(&a16_tile_kernel<T, 128, 128, 64, 64, OT>);
    case 2: return a16_few_ptr<T, 2, 2, OT>();
    case 3: return a16_few_ptr<T, 3, 2, OT>();
    case 4: return a16_few_ptr<T, 4, 5, OT>();
    case 5: return a16_few_ptr<T, 5, 3, OT>();
    case 6: return a16_few_ptr<T, 6, 4, OT>();
    case 7: return a16_few_ptr<T, 7, 5, OT>();
    case 8: return a16_few_ptr<T, 8, 5, OT>();
    case 9: return a16_few_ptr<T, 9, 5, OT>();
    case 10: return a16_few_ptr<T, 10, 4, OT>();
    case 11: return a16_few_ptr<T, 11, 5, OT>();
    default: return a16_few_ptr<T, 12, 2, OT>();
    }
}
template <int T>
const void *a16_ptr(int cfg, int ot) {
    return ot == kF32 ? a16_ptr<T, kF32>(cfg) : ot == kF16 ? a16_ptr<T, kF16>(cfg) : a16_ptr<T, kBF16>(cfg);
}

// The tile of a product of many rows: 0 (256 x 256, one workgroup per CU) or 1 (128 x 128,
// two).  A round of the CUs costs the tiles' area; a last round that is not full 0.35 + 0.65
// of its share (fewer CUs clock higher and get more of the L2); and the area of 128 x 128
// tiles costs `dearer` times that of 256 x 256 ones (twice the bytes through the L2 per
// product).  Timed at 14 shapes from 1500^3 to 8192^3 the choice is the faster one: e.g. (MXFP4,
// us, 0 against 1) 8192^3 248 and 287, 7000 x 7001 x 2000 86 and 88, 3000^3 24.6 and 28.0,
// 2500^3 20.7 and 15.4, 1024 x 8192 x 8192 40.8 and 35.6.
int pick_tile(int64_t M, int64_t N, double dearer) {
    auto rounds = [](int64_t tiles, int64_t slots) {
        const double part = double(tiles % slots) / double(slots);
        return double(tiles / slots) + (part > 0 ? 0.35 + 0.65 * part : 0.0);
    };
    const double large = rounds(cdiv(M, 256) * cdiv(N, 256), 256) * 256 * 256;
    const double small = rounds(cdiv(M, 128) * cdiv(N, 128), 512) * 2 * 128 * 128 * dearer;
    return large <= small ? 0 : 1;
}

// How the tile kernels store C.  Non-temporal stores leave the L2 to A and B (4096^3 to bf16
// 33.8 us and not 34.3) and are not held up in it at the kernel's end.  Rows that share lines
// make them pieces of lines, which cost more the more there are: past 28 MB of C, about what the
// L2s hold, such rows go through the L2, which joins them (us, plain against non-temporal:
// 2000 x 4001 x 4096 to fp32, 32 MB, 24.1 and 26.3; 7000 x 7001 x 2000 to fp32 90 and 110; but
// 2500^3 to fp32, 25 MB, 18.0 and 16.9).
bool plain_stores(const void *C, int64_t M, int64_t N, int64_t ldc, int type) {
    const bool lines = ldc * elem_size(type) % 128 == 0 && ((uintptr_t)C & 127) == 0;
    return !lines && M * N * elem_size(type) > 28'000'000;
}

int64_t tiles(const Config &c, int64_t M, int64_t N) { return cdiv(M, c.bm) * cdiv(N, c.bn); }

// gemm_mxf4.  While one round of the CUs takes all of them, small tiles, whose workgroups read
// the least (us: 251 x 90 x 2911 16 x 16 3.1, 64 x 32 4.5; 256 x 1024 x 8192 64 x 32 7.4,
// 128 x 128 16.3), 64 x 64 where K is long enough to pay for its start (256 x 4096 x 8192
// 13.4 against 16.9 on 128 x 128 tiles, at K = 2048 8.2 against 6.6); to 32 rows a wider tile
// over a long K, where 128 workgroups are enough (one row by width 64 / 32 / 16: 8192 x 8192
// 7.5 / 8.6 / 11.5, 4096 x 14336 9.0 / 7.3 / 8.8, 4096 x 4096 4.2 / 3.5 / 3.1).
int pick_mx(int64_t M, int64_t N, int64_t K) {
    if (M <= 32) {
        const int64_t least = K <= 4096 ? 256 : 128;
        return (M <= 16 ? 7 : 4) + (cdiv(N, 64) >= least ? 0 : cdiv(N, 32) >= least ? 1 : 2);
    }
    for (int c : {9, 6, 8, 5, 3})
        if (tiles(kMxConfigs[c], M, N) <= 256) return c;
    if (K > 4096 && tiles(kMxConfigs[2], M, N) <= 256) return 2;
    return pick_tile(M, N, 1.15);
}

int launch_mx(int cfg, int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const uint8_t *scale_a,
              int64_t ldsa, const uint8_t *B, int64_t ldb, const uint8_t *scale_b, int64_t ldsb, void *C, int64_t ldc,
              int out_type, void *stream) {
    if (cfg >= kNumMxConfigs || !known_type(out_type)) return PDGEMM_EINVAL_CFG;
    int rc = check_mx_sizes(M, K, lda, ldsa);
    if (rc == PDGEMM_OK) rc = check_mx_sizes(N, K, ldb, ldsb);
    if (rc != PDGEMM_OK) return rc;
    if (ldc < N) return PDGEMM_EINVAL_LD;
    if (M == 0 || N == 0) return PDGEMM_OK;
    rc = check_plain(C, ldc, out_type);
    if (rc == PDGEMM_OK && K > 0) rc = check_mx_memory(A, lda, scale_a, ldsa);
    if (rc == PDGEMM_OK && K > 0) rc = check_mx_memory(B, ldb, scale_b, ldsb);
    if (rc != PDGEMM_OK) return rc;
    if (cfg < 0) cfg = pick_mx(M, N, K);
    const Config &c = kMxConfigs[cfg];
    // with K = 0 no operand is read: the kernels form addresses from C instead
    const uint8_t *const p = static_cast<const uint8_t *>(C);
    MxArgs args = {K ? A : p, K ? scale_a : p, K ? B : p, K ? scale_b : p, C, K ? lda / 2 : 0, K ? ldb / 2 : 0,
                   K ? ldsa : 0, K ? ldsb : 0, ldc, (int)M, (int)N, (int)K, (int)cdiv(M, c.bm), (int)cdiv(N, c.bn),
                   plain_stores(C, M, N, ldc, out_type)};
    const void *fn = out_type == kF32 ? mx_ptr<kF32>(cfg) : out_type == kF16 ? mx_ptr<kF16>(cfg) : mx_ptr<kBF16>(cfg);
    return run(fn, (int64_t)args.tiles_m * args.tiles_n, c.threads, &args, stream);
}

// gemm_a16_mxf4.  The same, with A's 16-bit rows four times as dear as B's: the tile that
// reads the least and makes one round of workgroups (us: 152 x 68 x 4562 f16 8 x 16 5.5,
// 64 x 32 13.0; one row by width 64 / 32 / 16 16384 x 4096 8.4 / 9.7 / 14.1, 8192 x 8192
// 11.2 / 9.3 / 12.9, 4096 x 4096 6.0 / 5.1 / 4.7).  Past that, to 32 rows the widest.  A round
// of 64 x 64 takes two fifths of one of 128 x 128 tiles, a third for f16, whose products are
// scaled by vector instructions (K = 8192: 24 us against 61, 31 against 106), so it is taken
// for so many rounds of a K that is not short (1086 x 1004 x 456 12.4 against 8.6).
int pick_a16(int a_type, int64_t M, int64_t N, int64_t K) {
    for (int c : {11, 10, 8, 7, 9, 6, 5, 3, 4, 2, 12})
        if (tiles(kA16Configs[c], M, N) <= 256) return c;
    if (M <= 32) return M <= 8 ? 9 : M <= 16 ? 6 : 4;
    if (K >= 2048 && tiles(kA16Configs[12], M, N) <= 256 * (a_type == kF16 ? 3 : 2)) return 12;
    return pick_tile(M, N, 1.23);
}

int launch_a16(int cfg, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type, const uint8_t *B,
               int64_t ldb, const uint8_t *scale_b, int64_t ldsb, void *C, int64_t ldc, int out_type, void *stream) {
    if (cfg >= kNumA16Configs || (a_type != kF16 && a_type != kBF16) || !known_type(out_type)) return PDGEMM_EINVAL_CFG;
    if (M < 0 || M > INT32_MAX) return PDGEMM_EINVAL_DIM;
    int rc = check_mx_sizes(N, K, ldb, ldsb);
    if (rc != PDGEMM_OK) return rc;
    if (lda < K || ldc < N) return PDGEMM_EINVAL_LD;
    if (M == 0 || N == 0) return PDGEMM_OK;
    rc = check_plain(C, ldc, out_type);
    if (rc == PDGEMM_OK && K > 0) rc = check_plain(A, lda, a_type);
    if (rc == PDGEMM_OK && K > 0) rc = check_mx_memory(B, ldb, scale_b, ldsb);
    if (rc == PDGEMM_OK && K > 0 && (lda % 8 || ((uintptr_t)A & 15))) rc = PDGEMM_EALIGN;
    if (rc != PDGEMM_OK) return rc;
    if (cfg < 0) cfg = pick_a16(a_type, M, N, K);
    const Config &c = kA16Configs[cfg];
    const uint8_t *const p = static_cast<const uint8_t *>(C);
    MxArgs args = {K ? static_cast<const uint8_t *>(A) : p, nullptr, K ? B : p, K ? scale_b : p, C, K ? 2 * lda : 0,
                   K ? ldb / 2 : 0, 0, K ? ldsb : 0, ldc, (int)M, (int)N, (int)K, (int)cdiv(M, c.bm), (int)cdiv(N, c.bn),
                   plain_stores(C, M, N, ldc, out_type)};
    const void *fn = a_type == kF16 ? a16_ptr<kF16>(cfg, out_type) : a16_ptr<kBF16>(cfg, out_type);
    return run(fn, (int64_t)args.tiles_m * args.tiles_n, c.threads, &args, stream);
}

}  // namespace

extern "C" {

int pdgemm_mxf4_quantize(int64_t rows, int64_t K, const void *src, int64_t ld, int src_type, uint8_t *q, int64_t ldq,
                         uint8_t *scales, int64_t lds, uint8_t *qt, int64_t ldqt, uint8_t *scales_t, int64_t ldst,
                         int scale_rule, void *stream) {
    if (!known_type(src_type) || (scale_rule != PDGEMM_SCALE_FLOOR && scale_rule != PDGEMM_SCALE_FIT))
        return PDGEMM_EINVAL_CFG;
    const bool along_k = q || scales, along_rows = qt || scales_t;
    if (rows < 0 || K < 0 || rows > (int64_t(1) << 30) || K > (int64_t(1) << 30)) return PDGEMM_EINVAL_DIM;
    if (ld < K) return PDGEMM_EINVAL_LD;
    int rc = along_k ? check_mx_sizes(rows, K, ldq, lds) : PDGEMM_OK;
    if (rc == PDGEMM_OK && along_rows) rc = check_mx_sizes(K, rows, ldqt, ldst);
    if (rc != PDGEMM_OK) return rc;
    if (rows == 0 || K == 0) return PDGEMM_OK;
    if (!along_k && !along_rows) return PDGEMM_ENULL;
    rc = check_plain(src, ld, src_type);
    if (rc == PDGEMM_OK && along_k) rc = check_mx_memory(q, ldq, scales, lds);
    if (rc == PDGEMM_OK && along_rows) rc = check_mx_memory(qt, ldqt, scales_t, ldst);
    if (rc != PDGEMM_OK) return rc;
    const QuantArgs args = {src, q, scales, qt, scales_t, ld, ldq / 2, lds, ldqt / 2, ldst, (int)rows, (int)K, 0,
                            rule_bias(scale_rule)};
    return src_type == kF32 ? launch_quant<kF32>(args, stream)
                            : src_type == kF16 ? launch_quant<kF16>(args, stream) : launch_quant<kBF16>(args, stream);
}

int pdgemm_mxf4_dequantize(int64_t rows, int64_t K, const uint8_t *q, int64_t ldq, const uint8_t *scales, int64_t lds,
                           void *dst, int64_t ldd, int dst_type, void *stream) {
    if (!known_type(dst_type)) return PDGEMM_EINVAL_CFG;
    int rc = check_mx_sizes(rows, K, ldq, lds);
    if (rc != PDGEMM_OK) return rc;
    if (ldd < K) return PDGEMM_EINVAL_LD;
    if (rows == 0 || K == 0) return PDGEMM_OK;
    rc = check_mx_memory(q, ldq, scales, lds);
    if (rc == PDGEMM_OK) rc = check_plain(dst, ldd, dst_type);
    if (rc != PDGEMM_OK) return rc;
    const int size = elem_size(dst_type);
    DequantArgs args = {q, scales, dst, ldq / 2, lds, ldd, (int)rows, (int)K, (int)cdiv(K, 64 * 16 / size)};
    const bool lines = (ldd * size) % 128 == 0 && ((uintptr_t)dst & 127) == 0;
    const void *fn = dst_type == kF32   ? dequant_ptr<kF32>(lines)
                     : dst_type == kF16 ? dequant_ptr<kF16>(lines)
                                        : dequant_ptr<kBF16>(lines);
    return run(fn, cdiv(rows, 16) * args.tiles_k, 256, &args, stream);
}

int gemm_mxf4(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const uint8_t *scale_a, int64_t ldsa,
              const uint8_t *B, int64_t ldb, const uint8_t *scale_b, int64_t ldsb, void *C, int64_t ldc, int out_type,
              void *stream) {
    return launch_mx(-1, M, N, K, A, lda, scale_a, ldsa, B, ldb, scale_b, ldsb, C, ldc, out_type, stream);
}

int pdgemm_mxf4_cfg(int cfg, int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const uint8_t *scale_a,
                    int64_t ldsa, const uint8_t *B, int64_t ldb, const uint8_t *scale_b, int64_t ldsb, void *C,
                    int64_t ldc, int out_type, void *stream) {
    if (cfg < 0) return PDGEMM_EINVAL_CFG;
    return launch_mx(cfg, M, N, K, A, lda, scale_a, ldsa, B, ldb, scale_b, ldsb, C, ldc, out_type, stream);
}

int pdgemm_mxf4_num_configs(void) { return kNumMxConfigs; }

int pdgemm_mxf4_pick(int64_t M, int64_t N, int64_t K) { return pick_mx(M, N, K); }

int gemm_a16_mxf4(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type, const uint8_t *B, int64_t ldb,
                  const uint8_t *scale_b, int64_t ldsb, void *C, int64_t ldc, int out_type, void *stream) {
    return launch_a16(-1, M, N, K, A, lda, a_type, B, ldb, scale_b, ldsb, C, ldc, out_type, stream);
}

int pdgemm_a16_mxf4_cfg(int cfg, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int a_type,
                        const uint8_t *B, int64_t ldb, const uint8_t *scale_b, int64_t ldsb, void *C, int64_t ldc,
                        int out_type, void *stream) {
    if (cfg < 0) return PDGEMM_EINVAL_CFG;
    return launch_a16(cfg, M, N, K, A, lda, a_type, B, ldb, scale_b, ldsb, C, ldc, out_type, stream);
}

int pdgemm_a16_mxf4_num_configs(void) { return kNumA16Configs; }

int pdgemm_a16_mxf4_pick(int a_type, int64_t M, int64_t N, int64_t K) {
    if (a_type != kF16 && a_type != kBF16) return -1;
    return pick_a16(a_type, M, N, K);
}

}  // extern "C"
