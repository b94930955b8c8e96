// common.h -- what the kernels around the products share: element types, cross-lane
// sums, launches and argument checks.
#ifndef PDGEMM_COMMON_H
#define PDGEMM_COMMON_H

#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <type_traits>

#include "pdgemm.h"

namespace {

typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef unsigned int uintx2_t __attribute__((ext_vector_type(2)));
typedef unsigned int uintx4_t __attribute__((ext_vector_type(4)));

constexpr int kF32 = PDGEMM_F32;
constexpr int kF16 = PDGEMM_F16;
constexpr int kBF16 = PDGEMM_BF16;
constexpr int kI8 = PDGEMM_I8;

constexpr int kWave = 64;

template <int T> struct ElemOf { using type = float; };
template <> struct ElemOf<kF16> { using type = _Float16; };
template <> struct ElemOf<kBF16> { using type = __bf16; };
template <> struct ElemOf<kI8> { using type = int8_t; };
constexpr int elem_size(int t) { return t == kF32 ? 4 : t == kI8 ? 1 : 2; }

// N elements at their own alignment, as one access
template <int N, typename E>
__device__ __forceinline__ void load_run(E (&v)[N], const E *p) {
    __builtin_memcpy(v, p, N * sizeof(E));
}
template <int N, typename E>
__device__ __forceinline__ void store_run(E *p, const E (&v)[N]) {
    typedef E vec_t __attribute__((ext_vector_type(N)));
    typedef vec_t packed_t __attribute__((aligned(sizeof(E))));
    vec_t x;
    __builtin_memcpy(&x, v, N * sizeof(E));
    *reinterpret_cast<packed_t *>(p) = x;
}

// The first `n` of a run of N elements (all of them, or few at a row's end); zeros in the others.
template <int N, typename E>
__device__ __forceinline__ void load_some(E (&v)[N], const E *p, int n) {
    if (n >= N) {
        load_run<N>(v, p);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? p[i] : (E)0;
}
template <int N, typename E>
__device__ __forceinline__ void store_some(E *p, const E (&v)[N], int n) {
    if (n >= N) {
        store_run<N>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n) p[i] = v[i];
}

// The same of elements of a type known at run time, as binary32
template <int N>
__device__ __forceinline__ void load_some_as_float(float (&v)[N], const void *p, int type, int64_t at, int n) {
    if (type == kF32) {
        load_some<N>(v, static_cast<const float *>(p) + at, n);
    } else if (type == kF16) {
        _Float16 e[N];
        load_some<N>(e, static_cast<const _Float16 *>(p) + at, n);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = (float)e[i];
    } else {
        __bf16 e[N];
        load_some<N>(e, static_cast<const __bf16 *>(p) + at, n);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = (float)e[i];
    }
}

__device__ __forceinline__ float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }

// v of the lane whose number differs by the bit `kBit`
template <int kBit>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
    if constexpr (kBit == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
    if constexpr (kBit == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
    return (uint32_t)__shfl_xor((int)v, kBit);
}
// f over the 2 kBit neighbouring lanes, the same bits in each of them (f is commutative); every lane is active
template <int kLanes, int kBit = 1, typename F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v, F &&f) {
    if constexpr (kBit < kLanes) return over_lanes<kLanes, 2 * kBit>(f(v, partner<kBit>(v)), f);
    return v;
}
template <int kLanes>
__device__ __forceinline__ float sum_over_lanes(float v) {
    return as_float(over_lanes<kLanes>(bits_of(v), [](uint32_t a, uint32_t b) { return bits_of(as_float(a) + as_float(b)); }));
}
template <int kLanes>
__device__ __forceinline__ uint32_t max_over_lanes(uint32_t v) {
    return over_lanes<kLanes>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int kLanes, int kBit = 1>
__device__ __forceinline__ double sum_over_lanes64(double v) {
    if constexpr (kBit < kLanes) return sum_over_lanes64<kLanes, 2 * kBit>(v + __shfl_xor(v, kBit));
    return v;
}

// ---- host side ----

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

// The same of more work-items: in rows of `across` workgroups, which the kernel counts by block_of()
int run_rows(const void *fn, int64_t blocks, int across, int threads, void *args, void *stream) {
    void *kargs[] = {args};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(hipLaunchKernel(fn, dim3((unsigned)across, (unsigned)cdiv(blocks, across)), dim3((unsigned)threads), kargs, 0, s), s);
}
int blocks_across(int64_t blocks, int threads) {
    const int64_t most = (int64_t(1) << 31) / threads;
    return (int)(blocks < most ? blocks : most);
}
// (the last row's workgroups may pass the last block)
__device__ __forceinline__ int block_of(int across) { return blockIdx.y * across + blockIdx.x; }

bool known_type(int t) { return t == kF32 || t == kF16 || t == kBF16; }

// rows of a dense matrix with only its element's alignment
int check_plain(const void *p, int64_t ld, int type) {
    if (!p) return PDGEMM_ENULL;
    if (ld > kMaxRowBytes / elem_size(type)) return PDGEMM_EINVAL_LD;
    if ((uintptr_t)p & (elem_size(type) - 1)) return PDGEMM_EALIGN;
    return PDGEMM_OK;
}

}  // namespace

#endif  // PDGEMM_COMMON_H
