// i4_core.h -- a wave's part of a product of 16-bit activations with group-scaled INT4
// weights, for the kernels that read such weights.
//
// C[i][j] = sum over groups q of scale[q][j] * sum over k in q of a[i][k] * code[j][k]
//
// A step is 128 values of K: 64 bytes of a row of codes, 16 to a lane, so lane l of a
// fragment of 16 rows holds dwords 0 .. 3 (8 values each) of block l / 16 (32 values) of row
// l % 16.  A matrix instruction takes a dword from each of the four lane groups.  Instruction
// u's sum is scaled as it is added, in binary32, so its dwords must lie in one group of values: in
// groups of whole steps any dwords do (u of every block); shorter groups want them exchanged
// between the lane groups first, two swaps of lanes for groups of 64 values (instruction u then
// covers dwords of blocks 2 (u / 2) and 2 (u / 2) + 1), four for 32 (block u alone).  A code
// becomes the 16-bit type exactly: v / 16 by the conversion of 4-bit integers, and the scale
// takes the 16 back.
#ifndef PDGEMM_I4_CORE_H
#define PDGEMM_I4_CORE_H

#include "common.h"

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
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
__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off, int base = 0) {
    const uintx4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, off, base, 0);
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
    uint32_t h = w >> 4;   // (the conversion reads the low four bits of a byte)
    asm("" : "+v"(h));     // (kept whole, so that the conversions select its bytes themselves)
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = pair_of<T>(__builtin_amdgcn_cvt_off_f32_i4((w >> (8 * i)) & 0xFF),
                          __builtin_amdgcn_cvt_off_f32_i4((h >> (8 * i)) & 0xFF));
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// The same in the order 0 4 1 5 2 6 3 7, in which a dword's halves hold them
template <int T>
__device__ __forceinline__ uint4 widen_spread(uint32_t w) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = pair_of<T>(__builtin_amdgcn_cvt_off_f32_i4(w >> (4 * i)), __builtin_amdgcn_cvt_off_f32_i4(w >> (4 * i + 16)));
    return make_uint4(x[0], x[1], x[2], x[3]);
}
// eight 16-bit values in that order
__device__ __forceinline__ uint4 spread(const uint4 &x) {
    return make_uint4(__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
                      __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u));
}

// The same codes with a bias, in a shift and a bit operation for two.  bf16: code + 24, a code's four bits (their
// sign flipped) on top of the mantissa of 16.  f16: 2^-18 (code + 8), as a subnormal, which the
// matrix instructions keep.  Operand kBiasPair, the bias with the other sign in all places, takes it
// off again: the sums of activations it makes are the same for every column.  Activations that
// are infinite, or whose sums with the bias overflow, leave infinities or NaN, and the unit is summed
// again with widen_spread() (I4Wave).  f of Biased: what a sum is short of.
template <int T> struct Biased;
template <> struct Biased<kBF16> {
    static constexpr uint32_t kMask = 0x00780078u, kFlip = 0x41C041C0u, kBiasPair = 0xC1C0C1C0u;
    static constexpr int kShift = 3;   // the first pair's, to the left; 4 less for each pair after it
    static constexpr float f = 1.0f;
};
template <> struct Biased<kF16> {
    static constexpr uint32_t kMask = 0x03C003C0u, kFlip = 0x02000200u, kBiasPair = 0x82008200u;
    static constexpr int kShift = 6;
    static constexpr float f = 0x1p18f;
};
template <int T>
__device__ __forceinline__ uint4 widen_biased(uint32_t w) {
    using B = Biased<T>;
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = B::kShift - 4 * i;
        x[i] = ((s >= 0 ? w << (s >= 0 ? s : 0) : w >> (s < 0 ? -s : 0)) & B::kMask) ^ B::kFlip;
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// Dwords v of a lane's block to those of matrix instructions 0 .. 3, and (position) where
// instruction u's dword of lane group g lies in the step, in dwords.
template <int Q>
__device__ __forceinline__ void share_out(uint32_t (&v)[4]) {
    if constexpr (Q == 4) return;
    const uintx2_t a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const uintx2_t b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    v[0] = a[0], v[1] = b[0], v[2] = a[1], v[3] = b[1];
    if constexpr (Q == 2) return;
    const uintx2_t c = __builtin_amdgcn_permlane16_swap(v[0], v[1], false, false);
    const uintx2_t d = __builtin_amdgcn_permlane16_swap(v[2], v[3], false, false);
    v[0] = c[0], v[1] = c[1], v[2] = d[0], v[3] = d[1];
}
template <int Q>
__device__ __forceinline__ int position(int u, int g) {
    if constexpr (Q == 4) return 4 * g + u;
    if constexpr (Q == 2) return 8 * (u >> 1) + 4 * (g & 1) + 2 * (g >> 1) + (u & 1);
    return 4 * u + g;
}

// The same of a step's codes of a fragment in LDS: chunk c (16 bytes) of row r at c ^ (r / 2 % 4), so that rows that
// are read together lie in different banks.  A lane that copies has 16 bytes, chunk l % 4 of row l / 4.
__device__ __forceinline__ void write_codes(uint4 (*b)[4], const uint4 &v) {
    const int lane = threadIdx.x % kWave, r = lane / 4;
    b[r][(lane % 4) ^ (r / 2 % 4)] = v;
}
template <int Q>
__device__ __forceinline__ void read_codes(uint32_t (&w)[4], const uint4 (*b)[4]) {
    const int lane = threadIdx.x % kWave, g = lane / 16, r = lane % 16, swap = r / 2 % 4;
    if constexpr (Q == 4) {
        const uint4 v = b[r][g ^ swap];
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (Q == 2) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const uint2 x = reinterpret_cast<const uint2 *>(&b[r][(2 * v + (g & 1)) ^ swap])[g >> 1];
            w[2 * v] = x.x, w[2 * v + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = reinterpret_cast<const uint32_t *>(&b[r][u ^ swap])[g];
    }
}

// Orders a wave's LDS accesses before and after it, across its lanes.  The LDS serves one wave's
// accesses in the order they are issued, so this costs no instruction: it keeps the compiler,
// which sees one lane alone, from moving a read above the other lanes' store.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// binary32 of a scale as it was loaded: 32 bits, or 16 of f16 (half all ones) or bf16 (half 0), without a branch
template <bool kS32>
__device__ __forceinline__ float scale_value(uint32_t bits, uint32_t half) {
    if constexpr (kS32) return as_float(bits);
    const uint32_t f = bits_of((float)__builtin_bit_cast(_Float16, (uint16_t)bits));
    return as_float((f & half) | ((bits << 16) & ~half));
}

// Scales of one matrix of weights: of group q and row j at p + q * ld + j * size
struct I4Scales {
    const uint8_t *p;
    int64_t ld;    // bytes
    uint32_t half; // of scale_value
};

// Where a wave reads: up to 16 rows of activations, and NT fragments of 16 rows of weights,
// whose tile t has its codes in matrix t % NB (the gate's and the up projection's, say).  xa, vb: byte offsets of
// the rows that this lane copies and its 16 bytes of them (see I4Wave), kOutside: no row.
template <int kX, int NT, int NB>
struct I4Source {
    const uint8_t *a;          // activations; K values a row
    const uint8_t *a2;         // kParts 2: their second parts (kDirect: xa takes a lane to its part)
    int a_end;                 // bytes that may be read
    uint32_t xa[kX];
    const uint8_t *b[NB];      // codes
    int b_end[NB];
    uint32_t vb[NT];
    I4Scales s[NB];
    uint32_t vs[NT];           // byte offset of the scale of this lane's row l % 16
    int K;
    uint32_t group_magic;      // of I4Groups
    int groups;
};

// The group of a block of 32 values: block / g with g = group / 32, by one multiplication with magic =
// (2^32 + e) / g, 0 <= e < g.  A row of 16-bit activations has at most 2^21 values, 2^16 blocks, so that block * e <
// 2^32 wherever there is more than one group, and what e adds, block * e / (2^32 g), is below the 1 / g that a quotient
// lacks at least of the next one: it is exact (a last group's overshoot is cut).  2^32 itself, for g = 1, is passed as 0.
struct I4Groups {
    static uint32_t magic(int64_t group) { return (uint32_t)(((int64_t(1) << 32) + group / 32 - 1) / (group / 32)); }
    template <int Q>
    static __device__ __forceinline__ int of(int block, uint32_t magic, int groups) {
        int q = (int)__umulhi((uint32_t)block, magic);
        if (Q == 1 && magic == 0) q = block;   // (groups of 64 values and more have another magic)
        return min(q, groups - 1);
    }
};

// A wave's sums over units of 256 values of K: a whole 128-byte line of each row of codes, two
// steps.  Everything is loaded in runs of a row, 4 lanes to 64 bytes of codes and 16 to 256 of activations, and goes
// through LDS of the wave's own, a step at a time, to the lanes that want it.  (Codes loaded by the lanes
// that convert them, 16 rows to an instruction, ask the L1 for four times as many lines: 16 rows against 8192 x
// 8192 took 12.1 us and not 10.9.)  RA rows of activations: 2, 8 or 16; a fragment's further rows repeat
// them.  With RA = 2 there is little but the codes, and they do go straight to their lanes (kDirect): one row
// against 8192 x 8192 takes 8.3 us so, and 9.5 through LDS.  Q: blocks that share a scale (4: groups of whole steps, 2: of multiples of 64 values, 1: any).
// kS32: binary32 scales.  kAhead: see run.  kParts 2: activation row p is the sum of rows 2 p and 2 p + 1 of the RA,
// whose sums the caller adds.
template <int T, int RA, int NT, int NB, int Q, bool kS32, bool kAhead, int kParts = 1>
struct I4Wave {
    static constexpr int kSc = 4 / Q;                 // scales per step
    static constexpr bool kDirect = RA == 2;
    static constexpr int kRows = RA / kParts;         // activations' rows
    static constexpr int kX = kDirect ? 1 : RA / 4;   // loads of four rows of a step of activations (two of a unit)
    static constexpr int kXs = kDirect ? 1 : 2;       // ... each for every step
    static constexpr int kRun = kDirect ? 32 : 16;    // chunks of a row of x
    static constexpr int kLoads = Q == 1 ? 2 : 1;     // loads of scales of four groups
    using Source = I4Source<kX, NT, NB>;
    // chunk c (16 bytes) of row r of x at c ^ (r % 8): rows that are read together lie in different banks; the values
    // in the order of widen_biased
    struct Lds {
        uint4 x[RA][kRun];
        uint4 b[kDirect ? 1 : NT][kDirect ? 1 : 16][4];
        float s[NT][16][2 * kSc];
    };
    struct Stage {
        uint4 b[NT][2];
        uint4 x[kX][kXs];
        uint32_t s[NT][kLoads];
        int unit;
        int tag, left;   // the item's own
    };
    floatx4_t acc[NT];

    // which of the RA rows this lane copies in load j (two parts: four rows of one of them to a load), and its 16
    // bytes of the run
    static __device__ __forceinline__ int copied_row(int j) {
        const int sub = (threadIdx.x % kWave) / kRun;
        if constexpr (kParts == 1 || kDirect) return kWave / kRun * j + sub;
        return 2 * (kWave / kRun * (j % (kX / 2)) + sub) + j / (kX / 2);
    }
    static __device__ __forceinline__ int copied_chunk() { return threadIdx.x % kRun; }
    // and of a fragment of codes
    static __device__ __forceinline__ int code_row() { return kDirect ? threadIdx.x % 16 : threadIdx.x % kWave / 4; }
    static __device__ __forceinline__ int code_chunk() { return kDirect ? threadIdx.x % kWave / 16 : threadIdx.x % 4; }

    __device__ __forceinline__ void load(Stage &st, const Source &src, int unit) {
        st.unit = unit;
        if (unit < 0) return;
        // (a unit's offset is below the range: it begins inside its rows)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const auto rb = rsrc(src.b[t % NB], src.b_end[t % NB]);
            st.b[t][0] = load16(rb, src.vb[t], unit * 128);
            st.b[t][1] = load16(rb, src.vb[t] + 64, unit * 128);
        }
#pragma unroll
        for (int j = 0; j < kX; ++j) {
            const auto ra = rsrc(kParts == 2 && !kDirect && j >= kX / 2 ? src.a2 : src.a, src.a_end);
            st.x[j][0] = load16(ra, src.xa[j], unit * 512);
            if constexpr (!kDirect) st.x[j][1] = load16(ra, src.xa[j] + 256, unit * 512);
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int i = 4 * k + threadIdx.x % kWave / 16, block = unit * 8 + i * Q;
            // (scales past K are zeros: they may not be there)
            const bool in = i < 2 * kSc && block * kBlock < src.K;
            const int64_t q = I4Groups::of<Q>(block, src.group_magic, src.groups);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                st.s[t][k] = 0;
                const uint8_t *const p = src.s[t % NB].p + q * src.s[t % NB].ld + src.vs[t];
                if (in) st.s[t][k] = kS32 ? *reinterpret_cast<const uint32_t *>(p) : *reinterpret_cast<const uint16_t *>(p);
            }
        }
    }

    __device__ __forceinline__ void add(Stage &st, const Source &src, Lds &lds) {
        const int lane = threadIdx.x % kWave;
        if (__builtin_expect(st.unit * 2 * kStep + 2 * kStep > src.K, 0)) {
            // activations at and past K may be anything, a NaN too: they become zeros
#pragma unroll
            for (int h = 0; h < kXs; ++h) {
                const int n = src.K - (st.unit * 2 + h) * kStep - copied_chunk() * 8;
                uint32_t m[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) m[d] = n >= 2 * d + 2 ? 0xFFFFFFFFu : n == 2 * d + 1 ? 0xFFFFu : 0u;
#pragma unroll
                for (int j = 0; j < kX; ++j) {
                    uint4 &x = st.x[j][h];
                    x = make_uint4(x.x & m[0], x.y & m[1], x.z & m[2], x.w & m[3]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            if (4 * k + lane / 16 < 2 * kSc)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    lds.s[t][lane % 16][4 * k + lane / 16] = scale_value<kS32>(st.s[t][k], src.s[0].half);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (!kDirect)
#pragma unroll
                for (int t = 0; t < NT; ++t) write_codes(lds.b[t], st.b[t][h]);
            if (h < kXs)
#pragma unroll
                for (int j = 0; j < kX; ++j)
                    lds.x[copied_row(j)][copied_chunk() ^ (copied_row(j) % 8)] = spread(st.x[j][h < kXs ? h : 0]);
            if (h < kXs) wave_lds_order();
            floatx4_t d[NT];
            sum_step<true>(d, st, lds, h);
            float odd = 0;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) odd = __builtin_fmaf(d[t][e], 0.0f, odd);
            if (__builtin_expect(__any(!(odd == 0.0f)), 0)) {   // (NaN: infinity or NaN in d)
                // (only those sums change: the others' bits are the same beside them as without them)
                floatx4_t whole[NT];
                sum_step<false>(whole, st, lds, h);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[t][e] = d[t][e] * 0.0f == 0.0f ? d[t][e] : whole[t][e];
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] += d[t];
            if (!kDirect || h == 1) wave_lds_order();
        }
    }

    // the dwords of matrix instructions 0 .. 3 of step h of fragment t
    static __device__ __forceinline__ void codes(uint32_t (&w)[4], const Stage &st, const Lds &lds, int t, int h) {
        if constexpr (kDirect) {
            w[0] = st.b[t][h].x, w[1] = st.b[t][h].y, w[2] = st.b[t][h].z, w[3] = st.b[t][h].w;
            share_out<Q>(w);
        } else {
            read_codes<Q>(w, lds.b[t]);
        }
    }

    // step h's sums
    template <bool kBiased>
    static __device__ __forceinline__ void sum_step(floatx4_t (&d)[NT], const Stage &st, const Lds &lds, int h) {
        const int lane = threadIdx.x % kWave, g = lane / 16, row = lane % RA % 16;
        constexpr uint32_t kB = Biased<T>::kBiasPair;
        uint4 a[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) a[u] = lds.x[row][((kDirect ? 16 * h : 0) + position<Q>(u, g)) ^ (row % 8)];
        floatx4_t bias[kSc];
#pragma unroll
        for (int v = 0; v < kSc; ++v) {
            bias[v] = floatx4_t{0, 0, 0, 0};
            if constexpr (kBiased)
#pragma unroll
                for (int u = 0; u < Q; ++u) bias[v] = mfma16<T>(a[v * Q + u], make_uint4(kB, kB, kB, kB), bias[v]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t w[4];
            codes(w, st, lds, t, h);
            d[t] = floatx4_t{0, 0, 0, 0};
#pragma unroll
            for (int v = 0; v < kSc; ++v) {
                floatx4_t p = bias[v];
#pragma unroll
                for (int u = 0; u < Q; ++u)
                    p = mfma16<T>(a[v * Q + u], kBiased ? widen_biased<T>(w[v * Q + u]) : widen_spread<T>(w[v * Q + u]), p);
                const float s = lds.s[t][lane % 16][h * kSc + v] * (kBiased ? Biased<T>::f : 16.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[t][e] = __builtin_fmaf(p[e], s, d[t][e]);
            }
        }
    }

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = floatx4_t{0, 0, 0, 0};
    }

    // The wave's units in turn: item(st, src) gives the next one, and its source in src, or -1 after
    // the last; done(st) is called after each unit's sums.
    // The next unit's loads are on their way while one is summed (kAhead), or not.  One copy of the code,
    // and registers moved: with the loop unrolled so that none are, two to four units ahead, one row
    // against 8192 x 8192 took 9.1 to 10.2 us instead of 8.1, for a launch fetches its code anew.
    template <typename F, typename G>
    __device__ __forceinline__ void run(Source &src, Lds &lds, F &&item, G &&done) {
        clear();
        Stage next;
        load(next, src, item(next, src));
        while (next.unit >= 0) {
            Stage st = next;
            if constexpr (kAhead) load(next, src, item(next, src));
            add(st, src, lds);
            done(st);
            if constexpr (!kAhead) load(next, src, item(next, src));
        }
    }
};

}  // namespace

#endif  // PDGEMM_I4_CORE_H
