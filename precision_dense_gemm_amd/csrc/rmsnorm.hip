// rmsnorm.hip -- the root-mean-square norm for gfx950 (MI355X), with the residual's
// addition before it and INT8 codes with row scales after it, and its gradients, behind
// the C ABI declared in include/pdgemm.h.
//
//   h = x + residual (rounded to x's type),  r = (mean h^2 + eps)^(-1/2),  y = h r w
//   INT8: t = h w, m = max |t| of the row, q = rint(t * (127 * (1 / m))), scale = m r / 127
//
// r is the row's, so it cancels in the codes: they and the sum of squares come from one
// look at the row.
#include "common.h"

namespace {

struct NormArgs {
    const void *x, *res;    // res NULL: no residual
    void *sum;
    const void *w;
    void *out;
    float *scale;
    int64_t ldx, ldr, ldsum, ldo;   // elements
    int rows, cols;
    int across;             // of block_of()
    int w_type;
    float eps;
};

// A row's factor: y = (h * c) * r * w, with c a power of two that is 1 unless squares
// leave binary32's range.
struct Inverse {
    float c, r;
};

// from the mean of squares plus eps
__device__ __forceinline__ Inverse inverse_of(double e) {
    const double c = e > 0x1p100 ? 0x1p-64 : e < 0x1p-100 ? 0x1p64 : 1.0;
    return {(float)c, (float)(1.0 / sqrt(e) / c)};
}
// whether binary32 sums of squares serve: neither overflown nor lost below its range
__device__ __forceinline__ bool in_range(float ss, float mean_eps) { return ss <= 0x1p126f && mean_eps >= 0x1p-100f; }

// Sum and maximum over the threads of a row: kLanes neighbouring lanes, or (0) waves
// first .. first + waves - 1 of the workgroup, which meet in `part`.  The waves' sums are added in wave order.
template <int kLanes>
__device__ __forceinline__ void over_row(float &a, float &b, float (*part)[2], int first, int waves) {
    a = sum_over_lanes<kLanes ? kLanes : kWave>(a);
    b = sum_over_lanes<kLanes ? kLanes : kWave>(b);
    if constexpr (kLanes == 0) {
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave][0] = a, part[threadIdx.x / kWave][1] = b;
        __syncthreads();
        a = part[first][0], b = part[first][1];
        for (int i = 1; i < waves; ++i) a += part[first + i][0], b += part[first + i][1];
    }
}
template <int kLanes>
__device__ __forceinline__ void sum_and_max_over_row(float &a, uint32_t &m, float (*part)[2]) {
    a = sum_over_lanes<kLanes ? kLanes : kWave>(a);
    m = max_over_lanes<kLanes ? kLanes : kWave>(m);
    if constexpr (kLanes == 0) {
        const int waves = blockDim.x / kWave;
        if (waves == 1) return;
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave][0] = a, part[threadIdx.x / kWave][1] = as_float(m);
        __syncthreads();
        a = part[0][0], m = bits_of(part[0][1]);
        for (int i = 1; i < waves; ++i) a += part[i][0], m = max(m, bits_of(part[i][1]));
    }
}
template <int kLanes>
__device__ __forceinline__ double sum_over_row64(double a, double *part, int first, int waves) {
    a = sum_over_lanes64<kLanes ? kLanes : kWave>(a);
    if constexpr (kLanes == 0) {
        __syncthreads();   // (the part may be read still)
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = a;
        __syncthreads();
        a = part[first];
        for (int i = 1; i < waves; ++i) a += part[first + i];
    }
    return a;
}

// A row per workgroup, or (kLanes) per group of lanes.  A thread holds V runs of 16 bytes of
// it in registers from the one read to the store, so each value moves once: memory bounds it.  8192 x
// 8192 of f16 with a residual, to codes: 85 to 87 us, 470 MB at 5.4 TB/s (a large copy reaches 5.1); 2999 x 5003 of
// fp32 to bf16, whose rows begin anywhere: 20.7 us, 90 MB at 4.3 TB/s; one row of 8192 3.8 us.
template <int T, int OUT, int V, int kLanes>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void rms_norm_kernel(NormArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    using Out = typename ElemOf<OUT>::type;
    constexpr int N = 16 / elem_size(T);
    __shared__ float part[16][2];
    __shared__ double part64[16];

    const int tid = threadIdx.x;
    const int step = kLanes ? kLanes : (int)blockDim.x, t = kLanes ? tid % (kLanes ? kLanes : 1) : tid;
    const int block = block_of(args.across);
    const int row = kLanes ? block * (256 / (kLanes ? kLanes : 1)) + tid / (kLanes ? kLanes : 1) : block;
    const int cols = row < args.rows ? args.cols : 0;   // (lanes of no row take part in the sums' exchanges)

    Elem h[V][N];
    float w[V][N];
    const Elem *const x = static_cast<const Elem *>(args.x) + row * args.ldx;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at = (v * step + t) * N;
        load_some<N>(h[v], x + at, cols - at);
    }
    if (args.res) {
        const Elem *const res = static_cast<const Elem *>(args.res) + row * args.ldr;
        Elem *const sum = static_cast<Elem *>(args.sum) + row * args.ldsum;
        Elem add[V][N];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
            load_some<N>(add[v], res + at, cols - at);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
#pragma unroll
            for (int i = 0; i < N; ++i) h[v][i] = (Elem)((float)h[v][i] + (float)add[v][i]);
            store_some<N>(sum + at, h[v], cols - at);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at = (v * step + t) * N;
        load_some_as_float<N>(w[v], args.w, args.w_type, at, cols - at);
    }
    float ss = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) ss = __builtin_fmaf((float)h[v][i], (float)h[v][i], ss);

    auto inverse = [&](float ss) __attribute__((always_inline)) -> Inverse {
        const float e = ss / (float)args.cols + args.eps;
        if (in_range(ss, e)) return {1.0f, 1.0f / sqrtf(e)};
        // (for kLanes the lanes of a wave may differ in this, those of a row do not)
        double s64 = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) s64 += (double)h[v][i] * (double)h[v][i];
        return inverse_of(sum_over_row64<kLanes>(s64, part64, 0, blockDim.x / kWave) / args.cols + (double)args.eps);
    };

    Out *const out = static_cast<Out *>(args.out) + row * args.ldo;
    if constexpr (OUT == kI8) {
        // magnitudes order as their bits, NaN above infinity
        auto largest = [&](float c) __attribute__((always_inline)) {
            uint32_t m = 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i) m = max(m, bits_of((float)h[v][i] * c * w[v][i]) & 0x7FFFFFFFu);
            return m;
        };
        uint32_t top = largest(1.0f);
        sum_and_max_over_row<kLanes>(ss, top, part);
        const Inverse f = inverse(ss);
        // (a row out of the range of squares takes t times c, where t is out there too: the weights may have brought it back)
        float c = 1.0f, rest = f.c;
        if ((f.c > 1.0f && top < bits_of(0x1p-64f)) || (f.c < 1.0f && top > bits_of(0x1p64f))) {
            float none = 0;
            c = f.c, rest = 1.0f;
            top = largest(c);
            if constexpr (kLanes == 0) __syncthreads();
            sum_and_max_over_row<kLanes>(none, top, part);
        }
        const bool fine = top < 0x7F800000u;
        const float m = as_float(top);
        const float d = m < 0x1p-64f ? 0x1p64f : m > 0x1p64f ? 0x1p-64f : 1.0f;   // 1 / m in binary32's normal range
        const float inv = top && fine ? 127.0f * (1.0f / (m * d)) : 0.0f;
        if (t == 0 && row < args.rows) args.scale[row] = !fine ? __builtin_nanf("") : top ? m * f.r / 127.0f * rest : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
            Out q[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                q[i] = fine ? (Out)(int)rintf((float)h[v][i] * c * w[v][i] * d * inv) : (Out)0;
            store_some<N>(out + at, q, cols - at);
        }
    } else {
        float none = 0;
        over_row<kLanes>(ss, none, part, 0, blockDim.x / kWave);
        const Inverse f = inverse(ss);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
            Out y[N];
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = (Out)((float)h[v][i] * f.c * f.r * w[v][i]);
            store_some<N>(out + at, y, cols - at);
        }
    }
#endif  // __HIP_DEVICE_COMPILE__
}

struct GradArgs {
    const void *dy, *h, *dh;   // dh NULL: no gradient of the residual stream
    const void *w;
    void *dx;
    float *dw;                 // a row of cols per workgroup
    int64_t lddy, ldh, lddh, lddx;
    int rows, cols;
    int step;                  // threads of a row
    int w_type;
    float eps;
};

// 16 bytes of a row, held as they are: converted, 16-bit values take twice the registers
struct Run {
    uint32_t d[4];
};
template <int T>
__device__ __forceinline__ Run load_packed(const typename ElemOf<T>::type *p, int n) {
    using Elem = typename ElemOf<T>::type;
    constexpr int N = 16 / elem_size(T);
    Run r = {{0, 0, 0, 0}};
    if (n >= N) {
        Elem e[N];
        load_run<N>(e, p);
        __builtin_memcpy(&r, e, 16);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) {
                if constexpr (T == kF32)
                    r.d[i] = bits_of(p[i]);
                else
                    r.d[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (i % 2 * 16);
            }
    }
    return r;
}
template <int T>
__device__ __forceinline__ float value_of(const Run &r, int i) {
    if constexpr (T == kF32) return as_float(r.d[i]);
    if constexpr (T == kBF16) return as_float(i % 2 ? r.d[i / 2] & 0xFFFF0000u : r.d[i / 2] << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(r.d[i / 2] >> (i % 2 * 16)));
}
__device__ __forceinline__ void as_it_is(Run &r) { asm volatile("" : "+v"(r.d[0]), "+v"(r.d[1]), "+v"(r.d[2]), "+v"(r.d[3])); }

// With n = h r and g = dy w: dx = r (g - n mean(g n)) + dh, and dw is the sum over the rows of
// dy n.  kLanes lanes, or (0) args.step threads of whole waves, have a row, a workgroup as many rows at a time as
// it has such groups.  It takes every gridDim.x-th row of groups, keeps its share of dw in registers, and
// writes it for join_kernel.  Memory bounds it: 4096 x 8192 of bf16 with dh takes 65 us, 268 MB at 4.1 TB/s
// (shares of dw 17 MB more, join_kernel 4 us), 8192 x 4096 58 us.  A thread's values stay in registers up to two runs:
// with four and eight they spill, and reading the row again from the caches is faster (1024 x 32768 of bf16 121 us
// against 149, of f32 169 against 341).
template <int T, int V, int kLanes>
__global__ __launch_bounds__(1024, 4) void rms_norm_backward_kernel(GradArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    constexpr int N = 16 / elem_size(T);
    __shared__ float part[2][16][2];
    __shared__ double part64[16];
    __shared__ int odd[3];
    __shared__ float join[V == 1 ? 256 * N : 1];   // a row of step * N for each group

    const int tid = threadIdx.x;
    const int step = kLanes ? kLanes : args.step, group = tid / step, t = tid - group * step, groups = blockDim.x / step;
    const int first_wave = kLanes ? 0 : group * (step / kWave), waves = kLanes ? 0 : step / kWave;

    constexpr bool kKeep = V * N <= 8;      // the weights stay in registers
    constexpr int kTurns = V <= 2 ? V : 1;   // runs at a time
    float w[kKeep ? V : 1][N], dw[V][N];
    auto load_w = [&](int v) __attribute__((always_inline)) {
        const int at = (v * step + t) * N;
        load_some_as_float<N>(w[kKeep ? v : 0], args.w, args.w_type, at, args.cols - at);
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (kKeep) load_w(v);
#pragma unroll
        for (int i = 0; i < N; ++i) dw[v][i] = 0;
    }
    if (kLanes == 0 && V == 1) {
        if (tid < 3) odd[tid] = 0;
        __syncthreads();
    }
    int turn = 0, mark = 0;
    for (int64_t first = (int64_t)blockIdx.x * groups; first < args.rows; first += (int64_t)gridDim.x * groups, ++turn) {
        const int64_t row = first + group;
        const int cols = row < args.rows ? args.cols : 0;
        Run h[V <= 2 ? V : 1], dy[V <= 2 ? V : 1], dh[V <= 2 ? V : 1];
        const Elem *const ph = static_cast<const Elem *>(args.h) + row * args.ldh;
        const Elem *const pdy = static_cast<const Elem *>(args.dy) + row * args.lddy;
        const Elem *const pdh = static_cast<const Elem *>(args.dh) + row * args.lddh;
        // (of more runs than two the later passes read the row again, from the caches)
        auto load = [&](int v, bool all) __attribute__((always_inline)) {
            const int at = (v * step + t) * N, own = V <= 2 ? v : 0;
            h[own] = load_packed<T>(ph + at, cols - at);
            dy[own] = load_packed<T>(pdy + at, cols - at);
            if (all && args.dh) dh[own] = load_packed<T>(pdh + at, cols - at);
        };
        if (V <= 2)
#pragma unroll
            for (int v = 0; v < V; ++v) load(v, true);
        float ss = 0, dot = 0;
#pragma unroll kTurns
        for (int x = 0; x < V; ++x) {
            const int v = V <= 2 ? x : 0;
            if (V > 2) load(x, false);
            if (!kKeep) load_w(x);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float value = value_of<T>(h[v], i);
                ss = __builtin_fmaf(value, value, ss);
                dot = __builtin_fmaf(value_of<T>(dy[v], i) * w[kKeep ? v : 0][i], value, dot);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (V == 2 && !kKeep) as_it_is(h[v]), as_it_is(dy[v]);
        // A row whose sums leave binary32's range is summed in 64 bits.  All waves take part, each for its own
        // row, and rows in range keep their sums; so that one barrier will do, each wave says before it whether
        // its share may be of such a row (three marks in turn: one is cleared while others are read and set).
        const bool several = kLanes == 0 && V == 1 && groups > 1;
        if (several) {
            const float a = sum_over_lanes<kWave>(ss), b = sum_over_lanes<kWave>(dot);
            if (tid % kWave == 0 && row < args.rows &&
                !(a <= 0x1p120f && a / (float)args.cols + args.eps >= 0x1p-100f && fabsf(b) <= 0x1p120f))
                odd[mark] = 1;
        }
        // (two parts in turn: a wave writes the next row's while another reads this one's)
        over_row<kLanes>(ss, dot, part[turn & 1], first_wave, waves);
        float mean = 0;    // of g n
        Inverse f = {1.0f, 1.0f};
        const float e = ss / (float)args.cols + args.eps;
        float r = 0;
        const bool fine = in_range(ss, e) && fabsf(dot) <= 0x1p126f;
        if (fine) {
            r = f.r = 1.0f / sqrtf(e);
            mean = dot * r / (float)args.cols;
        }
        bool sum64 = !fine;
        if (several) {
            sum64 = odd[mark];
            mark = mark < 2 ? mark + 1 : 0;
            if (tid == 0) odd[mark < 2 ? mark + 1 : 0] = 0;
        }
        if (sum64) {
            double s64 = 0, d64 = 0;
#pragma unroll kTurns
            for (int x = 0; x < V; ++x) {
                const int v = V <= 2 ? x : 0;
                if (V > 2) load(x, false);
                if (!kKeep) load_w(x);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const double value = value_of<T>(h[v], i);
                    s64 += value * value;
                    d64 += (double)value_of<T>(dy[v], i) * (double)w[kKeep ? v : 0][i] * value;
                }
            }
            s64 = sum_over_row64<kLanes>(s64, part64, first_wave, waves);
            d64 = sum_over_row64<kLanes>(d64, part64, first_wave, waves);
            if (!fine) {
                const double e64 = s64 / args.cols + (double)args.eps;
                f = inverse_of(e64);
                r = (float)(1.0 / sqrt(e64));
                mean = (float)(d64 / sqrt(e64) / args.cols);
            }
        }
        Elem *const pdx = static_cast<Elem *>(args.dx) + row * args.lddx;
#pragma unroll
        for (int x = 0; x < V; ++x) {
            const int v = V <= 2 ? x : 0, at = (x * step + t) * N;
            if (V > 2) load(x, true);
            if (!kKeep) load_w(x);
            Elem dx[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float n = value_of<T>(h[v], i) * f.c * f.r, g = value_of<T>(dy[v], i);
                float d = r * __builtin_fmaf(-n, mean, g * w[kKeep ? v : 0][i]);
                if (args.dh) d += value_of<T>(dh[v], i);
                dx[i] = (Elem)d;
                if (cols) dw[x][i] = __builtin_fmaf(g, n, dw[x][i]);   // (lanes of no row: n may be NaN)
            }
            store_some<N>(pdx + at, dx, cols - at);
        }
    }
    float *const out = args.dw + (int64_t)blockIdx.x * args.cols;
    if (V > 1 || groups == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
            store_some<N>(out + at, dw[v], args.cols - at);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) join[tid * N + i] = dw[0][i];
        __syncthreads();
        for (int j = tid; j < args.cols; j += blockDim.x) {
            float s = join[j];
            for (int k = 1; k < groups; ++k) s += join[k * step * N + j];
            out[j] = s;
        }
    }
#endif  // __HIP_DEVICE_COMPILE__
}

struct JoinArgs {
    const float *part;
    float *dw;
    int parts, cols;
};

// dw from the workgroups' shares, in a fixed order: 64 columns to a workgroup, whose 16 waves
// each add every 16th share.
__global__ __launch_bounds__(1024) void join_kernel(JoinArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ float s[16][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int col = blockIdx.x * kWave + lane;
    float a = 0;
    if (col < args.cols)
#pragma unroll 8
        for (int p = wave; p < args.parts; p += 16) a += args.part[(int64_t)p * args.cols + col];
    s[wave][lane] = a;
    __syncthreads();
    if (wave == 0 && col < args.cols) {
        for (int i = 1; i < 16; ++i) a += s[i][lane];
        args.dw[col] = a;
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// host side

constexpr int64_t kMaxCols = 32768;

// How a row's `cols` values are shared out: V runs of 16 bytes for each of `threads` threads
// of one workgroup, or of kLanes lanes of one of 256.
struct Share {
    int v, lanes, threads;
};

Share share_of(int64_t cols, int type) {
    const int64_t runs = cdiv(cols * elem_size(type), 16);
    if (runs <= 16) return {1, 16, 256};
    if (runs <= 64) return {1, 64, 256};
    const int v = runs <= 1024 ? 1 : runs <= 2048 ? 2 : runs <= 4096 ? 4 : 8;
    return {v, 0, (int)cdiv(cdiv(runs, v), kWave) * kWave};
}

template <int T, int OUT>
const void *norm_ptr(const Share &s) {
    if (s.lanes == 16) return reinterpret_cast<const void *>(&rms_norm_kernel<T, OUT, 1, 16>);
    if (s.lanes == 64) return reinterpret_cast<const void *>(&rms_norm_kernel<T, OUT, 1, 64>);
    if (s.v == 1) return reinterpret_cast<const void *>(&rms_norm_kernel<T, OUT, 1, 0>);
    if (s.v == 2) return reinterpret_cast<const void *>(&rms_norm_kernel<T, OUT, 2, 0>);
    if constexpr (T == kF32)
        if (s.v == 8) return reinterpret_cast<const void *>(&rms_norm_kernel<T, OUT, 8, 0>);
    return reinterpret_cast<const void *>(&rms_norm_kernel<T, OUT, 4, 0>);
}
template <int T>
const void *norm_ptr(const Share &s, int out_type) {
    return out_type == kI8    ? norm_ptr<T, kI8>(s)
           : out_type == kF32 ? norm_ptr<T, kF32>(s)
           : out_type == kF16 ? norm_ptr<T, kF16>(s)
                              : norm_ptr<T, kBF16>(s);
}

template <int T>
const void *grad_ptr(const Share &s) {
    if (s.lanes == 16) return reinterpret_cast<const void *>(&rms_norm_backward_kernel<T, 1, 16>);
    if (s.lanes == 64) return reinterpret_cast<const void *>(&rms_norm_backward_kernel<T, 1, 64>);
    if (s.v == 1) return reinterpret_cast<const void *>(&rms_norm_backward_kernel<T, 1, 0>);
    if (s.v == 2) return reinterpret_cast<const void *>(&rms_norm_backward_kernel<T, 2, 0>);
    if constexpr (T == kF32)
        if (s.v == 8) return reinterpret_cast<const void *>(&rms_norm_backward_kernel<T, 8, 0>);
    return reinterpret_cast<const void *>(&rms_norm_backward_kernel<T, 4, 0>);
}

// n zeros, by a kernel: a graph may hold it
__global__ __launch_bounds__(256) void zeros_kernel(float *p, int n) {
#if defined(__HIP_DEVICE_COMPILE__)
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
#endif  // __HIP_DEVICE_COMPILE__
}

int check_norm_sizes(int64_t rows, int64_t cols) {
    return rows < 0 || cols < 0 || rows > (int64_t(1) << 30) || cols > kMaxCols ? PDGEMM_EINVAL_DIM : PDGEMM_OK;
}

// The gradient's share: as many groups of threads with a row each as 256 threads have, and 1024 threads on
// each CU, what the registers allow.  (Workgroups of 512 and 1024 threads with more rows each, which wait for one
// another at every sum: 16384 x 2048 of bf16 7 and 12% slower.)
struct GradShare {
    Share s;
    int groups;
    int64_t blocks;
};
GradShare grad_share_of(int64_t rows, int64_t cols, int type) {
    GradShare g = {share_of(cols, type), 1, 0};
    const int step = g.s.lanes ? g.s.lanes : g.s.threads;
    if (g.s.v == 1) g.groups = step < 256 ? 256 / step : 1;
    g.s.threads = step * g.groups;
    const int64_t turns = cdiv(rows, g.groups), most = 256 * (g.s.threads < 1024 ? 1024 / g.s.threads : 1);
    g.blocks = turns < most ? turns : most;
    return g;
}

}  // namespace

extern "C" {

int pdgemm_rms_norm(int64_t rows, int64_t cols, const void *x, int64_t ldx, int type, const void *residual, int64_t ldr,
                    void *sum, int64_t lds, const void *weight, int weight_type, float eps, void *out, int64_t ldo,
                    int out_type, float *scale, void *stream) {
    if (!known_type(type) || !known_type(weight_type) || (!known_type(out_type) && out_type != kI8) ||
        !(eps >= 0.0f && eps <= 3.4e38f))
        return PDGEMM_EINVAL_CFG;
    int rc = check_norm_sizes(rows, cols);
    if (rc != PDGEMM_OK) return rc;
    const bool add = residual || sum;
    if (ldx < cols || ldo < cols || (add && (ldr < cols || lds < cols))) return PDGEMM_EINVAL_LD;
    if (rows == 0 || (cols == 0 && (out_type != kI8 || !scale))) return PDGEMM_OK;
    if (cols == 0) {
        rc = check_plain(scale, 1, kF32);
        if (rc != PDGEMM_OK) return rc;
        int n = (int)rows;
        void *kargs[] = {&scale, &n};
        hipStream_t s = static_cast<hipStream_t>(stream);
        const int64_t blocks = cdiv(rows, 256);
        return finish(hipLaunchKernel(reinterpret_cast<const void *>(&zeros_kernel), dim3(blocks < 4096 ? (unsigned)blocks : 4096u),
                                      dim3(256), kargs, 0, s), s);
    }
    rc = check_plain(x, ldx, type);
    if (rc == PDGEMM_OK && add) rc = check_plain(residual, ldr, type);
    if (rc == PDGEMM_OK && add) rc = check_plain(sum, lds, type);
    if (rc == PDGEMM_OK) rc = check_plain(weight, cols, weight_type);
    if (rc == PDGEMM_OK) rc = check_plain(out, ldo, out_type);
    if (rc == PDGEMM_OK && out_type == kI8) rc = check_plain(scale, 1, kF32);
    if (rc != PDGEMM_OK) return rc;
    const Share s = share_of(cols, type);
    const int64_t blocks = s.lanes ? cdiv(rows, 256 / s.lanes) : rows;
    const int across = blocks_across(blocks, s.threads);
    NormArgs args = {x, residual, sum, weight, out, scale, ldx, ldr, lds, ldo, (int)rows, (int)cols, across, weight_type, eps};
    const void *fn = type == kF32   ? norm_ptr<kF32>(s, out_type)
                     : type == kF16 ? norm_ptr<kF16>(s, out_type)
                                    : norm_ptr<kBF16>(s, out_type);
    return run_rows(fn, blocks, across, s.threads, &args, stream);
}

int64_t pdgemm_rms_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (check_norm_sizes(rows, cols) != PDGEMM_OK) return 0;
    const int64_t a = grad_share_of(rows, cols, kF32).blocks, b = grad_share_of(rows, cols, kF16).blocks;
    return a > 1 || b > 1 ? (a > b ? a : b) * cols * 4 : 0;
}

int pdgemm_rms_norm_backward(int64_t rows, int64_t cols, const void *dy, int64_t lddy, const void *h, int64_t ldh,
                             const void *dh, int64_t lddh, int type, const void *weight, int weight_type, float eps,
                             void *dx, int64_t lddx, float *dweight, void *workspace, int64_t workspace_bytes,
                             void *stream) {
    if (!known_type(type) || !known_type(weight_type) || !(eps >= 0.0f && eps <= 3.4e38f)) return PDGEMM_EINVAL_CFG;
    int rc = check_norm_sizes(rows, cols);
    if (rc != PDGEMM_OK) return rc;
    if (lddy < cols || ldh < cols || lddx < cols || (dh && lddh < cols)) return PDGEMM_EINVAL_LD;
    if (cols == 0) return PDGEMM_OK;
    rc = check_plain(dweight, 1, kF32);
    if (rc == PDGEMM_OK && rows > 0) {
        rc = check_plain(dy, lddy, type);
        if (rc == PDGEMM_OK) rc = check_plain(h, ldh, type);
        if (rc == PDGEMM_OK && dh) rc = check_plain(dh, lddh, type);
        if (rc == PDGEMM_OK) rc = check_plain(weight, cols, weight_type);
        if (rc == PDGEMM_OK) rc = check_plain(dx, lddx, type);
    }
    if (rc != PDGEMM_OK) return rc;
    const int64_t need = pdgemm_rms_norm_backward_workspace_size(rows, cols);
    if (need > 0) {
        if (!workspace) return PDGEMM_ENULL;
        if (workspace_bytes < need || ((uintptr_t)workspace & 15)) return PDGEMM_EWORKSPACE;
    }
    const GradShare g = grad_share_of(rows, cols, type);
    if (rows > 0) {
        GradArgs args = {dy, h, dh, weight, dx, need ? static_cast<float *>(workspace) : dweight, lddy, ldh, lddh, lddx,
                         (int)rows, (int)cols, g.s.threads / g.groups, weight_type, eps};
        const void *fn = type == kF32 ? grad_ptr<kF32>(g.s) : type == kF16 ? grad_ptr<kF16>(g.s) : grad_ptr<kBF16>(g.s);
        rc = run(fn, g.blocks, g.s.threads, &args, stream);
        if (rc != PDGEMM_OK || !need) return rc;
    }
    JoinArgs args = {static_cast<const float *>(workspace), dweight, (int)(rows > 0 ? g.blocks : 0), (int)cols};
    return run(reinterpret_cast<const void *>(&join_kernel), cdiv(cols, kWave), 1024, &args, stream);
}

}  // extern "C"
