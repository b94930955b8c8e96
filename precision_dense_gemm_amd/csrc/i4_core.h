// i4_core.h -- a wave's part of a product of 16-bit activations with group-scaled INT4
// weights, for the kernels that read such weights.
//
// C[i][j] = sum over groups q of scale[q][j] * sum over k in q of a[i][k] * code[j][k]
//
// A step is 128 values of K: 64 bytes of a row of codes, 16 to a lane, so lane l of a
// fragment of 16 rows first holds block l / 16 (32 values) of row l % 16.  The matrix
// instruction wants 8 values of one block in each of the four lane groups instead, which a
// 4 x 4 transpose over the groups gives (four swaps of lanes): instruction u then covers
// block u alone, whatever the group's size, and its sum is scaled as it is added, in
// binary32.  A code becomes the 16-bit type exactly: v / 16 by the conversion of 4-bit
// integers, and the scale takes the 16 back.
#ifndef PDGEMM_I4_CORE_H
#define PDGEMM_I4_CORE_H

#include "common.h"

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int kStep = 128;    // values of K per step
constexpr int kBlock = 32;    // ... per matrix instruction; groups are multiples of it

// Buffer resource word 3 for raw (untyped) buffer loads on gfx9-family parts.
constexpr int kRsrcWord3 = 0x00020000;
constexpr uint32_t kOutside = 0x80000000u;   // an offset outside every range: zeros arrive

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, int range) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, range, kRsrcWord3);
}
__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    const uintx4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
    return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int T>
__device__ __forceinline__ floatx4_t mfma16(const uint4 &a, const uint4 &b, const floatx4_t &c) {
    if constexpr (T == kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// the pair of 16-bit values of two floats that the type holds exactly
template <int T>
__device__ __forceinline__ uint32_t pair_of(float x, float y) {
    if constexpr (T == kF16) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(x, y));
    } else {
        const bf16x2_t v = {(__bf16)x, (__bf16)y};
        return __builtin_bit_cast(uint32_t, v);
    }
}

// a sixteenth of the eight signed codes of a dword, in order
template <int T>
__device__ __forceinline__ uint4 widen(uint32_t w) {
    const uint32_t h = w >> 4;   // (the conversion reads the low four bits of a byte)
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = pair_of<T>(__builtin_amdgcn_cvt_off_f32_i4(w >> (8 * i)), __builtin_amdgcn_cvt_off_f32_i4(h >> (8 * i)));
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// v[u] of lane group g becomes v[g] of lane group u
__device__ __forceinline__ void transpose_groups(uint32_t (&v)[4]) {
    const uintx2_t a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const uintx2_t b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    const uintx2_t c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const uintx2_t d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    v[0] = c[0], v[1] = c[1], v[2] = d[0], v[3] = d[1];
}

// Scales of one matrix of weights: of group q and row j at p + q * ld + j * size
struct I4Scales {
    const uint8_t *p;
    int64_t ld;    // bytes
    int type;
};

// Where a wave reads: MT fragments of 16 rows of activations, NT of weights, whose tile t
// has its codes in matrix t % NB (the gate's and the up projection's, say).
template <int MT, int NT, int NB>
struct I4Source {
    const uint8_t *a;          // activations; K values a row
    int a_end;                 // bytes that may be read
    uint32_t va[MT];           // this lane's row l % 16 of each fragment, plus 16 (l / 16); kOutside: no row
    const uint8_t *b[NB];      // codes
    int b_end[NB];
    uint32_t vb[NT];           // likewise
    I4Scales s[NB];
    uint32_t vs[NT];           // byte offset of this lane's row's scale
    int K, group;
};

// Q: blocks that share a scale (4: groups of whole steps, 2: of multiples of 64 values, 1:
// any).  kS32: binary32 scales.  D: items whose loads are on their way.  kAbsent: rows of
// activations may be absent from a step, and a scale that is not finite stays out of them.
template <int T, int MT, int NT, int NB, int Q, bool kS32, int D, bool kAbsent = false>
struct I4Wave {
    static constexpr int kSc = 4 / Q;
    using Source = I4Source<MT, NT, NB>;
    struct Stage {
        uint4 b[NT];
        uint4 a[MT][4];
        uint32_t s[NT][kSc];
        int step;
    };
    floatx4_t acc[MT][NT];

    __device__ __forceinline__ void load(Stage &st, const Source &src, int step) {
        const bool any = step >= 0;
        const int at = any ? step : 0;   // (no step: nothing is read but a scale, which is not used)
        st.step = step;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const auto rb = rsrc(src.b[t % NB] + at * 64, any ? src.b_end[t % NB] - at * 64 : 0);
            st.b[t] = load16(rb, src.vb[t]);
        }
        const auto ra = rsrc(src.a + (int64_t)at * 256, any ? src.a_end - at * 256 : 0);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) st.a[i][u] = load16(ra, src.va[i] + u * 64);
        const int groups = (src.K + src.group - 1) / src.group;
#pragma unroll
        for (int u = 0; u < kSc; ++u) {
            const int q = min((at * kStep + u * Q * kBlock) / src.group, groups - 1);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint8_t *const p = src.s[t % NB].p + q * src.s[t % NB].ld + src.vs[t];
                if constexpr (kS32)
                    st.s[t][u] = *reinterpret_cast<const uint32_t *>(p);
                else
                    st.s[t][u] = *reinterpret_cast<const uint16_t *>(p);
            }
        }
    }

    __device__ __forceinline__ void add(Stage &st, const Source &src) {
        const int step = st.step;
        if (step * kStep + kStep > src.K) {
            // activations at and past K may be anything, a NaN too: they become zeros
            const int g = (threadIdx.x % kWave) / 16;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int n = src.K - step * kStep - u * kBlock - g * 8;
                uint32_t m[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) m[d] = n >= 2 * d + 2 ? 0xFFFFFFFFu : n == 2 * d + 1 ? 0xFFFFu : 0u;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint4 &v = st.a[i][u];
                    v = make_uint4(v.x & m[0], v.y & m[1], v.z & m[2], v.w & m[3]);
                }
            }
            // and so do the scales of groups past it, which may not be there
#pragma unroll
            for (int u = 0; u < kSc; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (step * kStep + u * Q * kBlock >= src.K) st.s[t][u] = 0;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t w[4] = {st.b[t].x, st.b[t].y, st.b[t].z, st.b[t].w};
            transpose_groups(w);
            uint4 b[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) b[u] = widen<T>(w[u]);
#pragma unroll
            for (int v = 0; v < kSc; ++v) {
                float s;
                if constexpr (kS32)
                    s = as_float(st.s[t][v]);
                else
                    s = src.s[0].type == kF16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)st.s[t][v])
                                              : as_float(st.s[t][v] << 16);
                s *= 16.0f;
                const bool odd = kAbsent && __builtin_expect(__any(!(__builtin_fabsf(s) <= 3.4e38f)), 0);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    floatx4_t p = {0, 0, 0, 0};
#pragma unroll
                    for (int u = 0; u < Q; ++u) p = mfma16<T>(st.a[i][v * Q + u], b[v * Q + u], p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (kAbsent && odd && p[e] == 0.0f) continue;
                        acc[i][t][e] = __builtin_fmaf(p[e], s, acc[i][t][e]);
                    }
                }
            }
        }
    }

    // The wave's items 0 .. count - 1: item(i, src) gives item i's step, and its source in src; it
    // is called for i = 0, 1, 2, ... once each, D items ahead of the sums.
    template <typename F>
    __device__ __forceinline__ void run(Source &src, int count, F &&item) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[i][t] = floatx4_t{0, 0, 0, 0};
        if (count <= 0) return;   // (there may be no scale to load)
        Stage st[D];
#pragma unroll
        for (int d = 0; d < D; ++d) load(st[d], src, d < count ? item(d, src) : -1);
        for (int i = 0; i < count; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (i + d < count) add(st[d], src);
                load(st[d], src, i + d + D < count ? item(i + d + D, src) : -1);
            }
        }
    }
};

}  // namespace

#endif  // PDGEMM_I4_CORE_H
