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

// Sum and maximum over the threads of a row: kLanes neighbouring lanes, or (0) the whole
// workgroup, whose waves meet in `part`.  The waves' sums are added in wave order.
template <int kLanes>
__device__ __forceinline__ void over_row(float &a, float &b, float (*part)[2]) {
    a = sum_over_lanes<kLanes ? kLanes : kWave>(a);
    b = sum_over_lanes<kLanes ? kLanes : kWave>(b);
    if constexpr (kLanes == 0) {
        const int waves = blockDim.x / kWave;
        if (waves == 1) return;
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave][0] = a, part[threadIdx.x / kWave][1] = b;
        __syncthreads();
        a = part[0][0], b = part[0][1];
        for (int i = 1; i < waves; ++i) a += part[i][0], b += part[i][1];
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
__device__ __forceinline__ double sum_over_row64(double a, double *part) {
    a = sum_over_lanes64<kLanes ? kLanes : kWave>(a);
    if constexpr (kLanes == 0) {
        const int waves = blockDim.x / kWave;
        __syncthreads();   // (the part may be read still)
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = a;
        __syncthreads();
        a = part[0];
        for (int i = 1; i < waves; ++i) a += part[i];
    }
    return a;
}

// A row per workgroup, or (kLanes) per group of lanes.  A thread holds V runs of 16 bytes of
// it in registers from the one read to the store.
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
    const int row = kLanes ? blockIdx.x * (256 / (kLanes ? kLanes : 1)) + tid / (kLanes ? kLanes : 1) : blockIdx.x;
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
        return inverse_of(sum_over_row64<kLanes>(s64, part64) / args.cols + (double)args.eps);
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
        if (f.c != 1.0f) {
            float none = 0;
            top = largest(f.c);
            if constexpr (kLanes == 0) __syncthreads();
            sum_and_max_over_row<kLanes>(none, top, part);
        }
        const bool fine = top < 0x7F800000u;
        const float m = as_float(top);
        const float d = m < 0x1p-64f ? 0x1p64f : m > 0x1p64f ? 0x1p-64f : 1.0f;   // 1 / m in binary32's normal range
        const float inv = top && fine ? 127.0f * (1.0f / (m * d)) : 0.0f;
        if (t == 0 && row < args.rows) args.scale[row] = !fine ? __builtin_nanf("") : top ? m * f.r / 127.0f : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
            Out q[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                q[i] = fine ? (Out)(int)rintf((float)h[v][i] * f.c * w[v][i] * d * inv) : (Out)0;
            store_some<N>(out + at, q, cols - at);
        }
    } else {
        float none = 0;
        over_row<kLanes>(ss, none, part);
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
    int w_type;
    float eps;
};

// With n = h r and g = dy w: dx = r (g - n mean(g n)) + dh, and dw is the sum over the rows of
// dy n.  A workgroup takes every gridDim.x-th row (kLanes: a group of lanes every such row
// of groups), keeps its share of dw in registers, and writes it for join_kernel.
template <int T, int V, int kLanes>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void rms_norm_backward_kernel(GradArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    constexpr int N = 16 / elem_size(T);
    constexpr int kGroups = kLanes ? 256 / (kLanes ? kLanes : 1) : 1;
    __shared__ float part[2][16][2];
    __shared__ double part64[16];
    __shared__ float join[kLanes ? kGroups : 1][kLanes ? kLanes * N * V : 1];

    const int tid = threadIdx.x;
    const int step = kLanes ? kLanes : (int)blockDim.x, t = kLanes ? tid % (kLanes ? kLanes : 1) : tid;
    const int group = kLanes ? tid / (kLanes ? kLanes : 1) : 0;

    float w[V][N], dw[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int at = (v * step + t) * N;
        load_some_as_float<N>(w[v], args.w, args.w_type, at, args.cols - at);
#pragma unroll
        for (int i = 0; i < N; ++i) dw[v][i] = 0;
    }
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * kGroups; first < args.rows; first += (int64_t)gridDim.x * kGroups, ++turn) {
        const int64_t row = first + group;
        const int cols = row < args.rows ? args.cols : 0;
        Elem h[V][N], dy[V][N], dh[V][N];
        const Elem *const ph = static_cast<const Elem *>(args.h) + row * args.ldh;
        const Elem *const pdy = static_cast<const Elem *>(args.dy) + row * args.lddy;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
            load_some<N>(h[v], ph + at, cols - at);
            load_some<N>(dy[v], pdy + at, cols - at);
        }
        if (args.dh) {
            const Elem *const pdh = static_cast<const Elem *>(args.dh) + row * args.lddh;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int at = (v * step + t) * N;
                load_some<N>(dh[v], pdh + at, cols - at);
            }
        }
        float ss = 0, dot = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                ss = __builtin_fmaf((float)h[v][i], (float)h[v][i], ss);
                dot = __builtin_fmaf((float)dy[v][i] * w[v][i], (float)h[v][i], dot);
            }
        // (two parts in turn: a wave writes the next row's while another reads this one's)
        over_row<kLanes>(ss, dot, part[turn & 1]);
        float mean;        // of g n
        Inverse f = {1.0f, 1.0f};
        const float e = ss / (float)args.cols + args.eps;
        float r;
        if (in_range(ss, e) && fabsf(dot) <= 0x1p126f) {
            r = f.r = 1.0f / sqrtf(e);
            mean = dot * r / (float)args.cols;
        } else {
            double s64 = 0, d64 = 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    s64 += (double)h[v][i] * (double)h[v][i];
                    d64 += (double)dy[v][i] * (double)w[v][i] * (double)h[v][i];
                }
            const double e64 = sum_over_row64<kLanes>(s64, part64) / args.cols + (double)args.eps;
            f = inverse_of(e64);
            r = (float)(1.0 / sqrt(e64));
            mean = (float)(sum_over_row64<kLanes>(d64, part64) / sqrt(e64) / args.cols);
        }
        Elem *const pdx = static_cast<Elem *>(args.dx) + row * args.lddx;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
            Elem dx[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float n = (float)h[v][i] * f.c * f.r;
                float d = r * __builtin_fmaf(-n, mean, (float)dy[v][i] * w[v][i]);
                if (args.dh) d += (float)dh[v][i];
                dx[i] = (Elem)d;
                if (cols) dw[v][i] = __builtin_fmaf((float)dy[v][i], n, dw[v][i]);   // (lanes of no row: n may be NaN)
            }
            store_some<N>(pdx + at, dx, cols - at);
        }
    }
    float *const out = args.dw + (int64_t)blockIdx.x * args.cols;
    if constexpr (kLanes == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int at = (v * step + t) * N;
            store_some<N>(out + at, dw[v], args.cols - at);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) join[group][(v * step + t) * N + i] = dw[v][i];
        __syncthreads();
        for (int j = tid; j < args.cols; j += 256) {
            float s = join[0][j];
            for (int k = 1; k < kGroups; ++k) s += join[k][j];
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

int check_norm_sizes(int64_t rows, int64_t cols) {
    return rows < 0 || cols < 0 || rows > (int64_t(1) << 30) || cols > kMaxCols ? PDGEMM_EINVAL_DIM : PDGEMM_OK;
}

// workgroups of the gradient: two of 1024 threads fit a CU
int64_t grad_blocks(int64_t rows, int64_t cols) {
    const Share s = share_of(cols, kF32);
    const int64_t groups = s.lanes ? cdiv(rows, 256 / s.lanes) : rows;
    return groups < 512 ? groups : 512;
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
    if (rows == 0 || cols == 0) return PDGEMM_OK;
    rc = check_plain(x, ldx, type);
    if (rc == PDGEMM_OK && add) rc = check_plain(residual, ldr, type);
    if (rc == PDGEMM_OK && add) rc = check_plain(sum, lds, type);
    if (rc == PDGEMM_OK) rc = check_plain(weight, cols, weight_type);
    if (rc == PDGEMM_OK) rc = check_plain(out, ldo, out_type);
    if (rc == PDGEMM_OK && out_type == kI8) rc = check_plain(scale, 1, kF32);
    if (rc != PDGEMM_OK) return rc;
    NormArgs args = {x, residual, sum, weight, out, scale, ldx, ldr, lds, ldo, (int)rows, (int)cols, weight_type, eps};
    const Share s = share_of(cols, type);
    const void *fn = type == kF32   ? norm_ptr<kF32>(s, out_type)
                     : type == kF16 ? norm_ptr<kF16>(s, out_type)
                                    : norm_ptr<kBF16>(s, out_type);
    return run(fn, s.lanes ? cdiv(rows, 256 / s.lanes) : rows, s.threads, &args, stream);
}

int64_t pdgemm_rms_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (check_norm_sizes(rows, cols) != PDGEMM_OK) return 0;
    const int64_t blocks = grad_blocks(rows, cols);
    return blocks > 1 ? blocks * cols * 4 : 0;
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
    const int64_t blocks = grad_blocks(rows, cols);
    if (rows > 0) {
        GradArgs args = {dy, h, dh, weight, dx, need ? static_cast<float *>(workspace) : dweight, lddy, ldh, lddh, lddx,
                         (int)rows, (int)cols, weight_type, eps};
        const Share s = share_of(cols, type);
        const void *fn = type == kF32 ? grad_ptr<kF32>(s) : type == kF16 ? grad_ptr<kF16>(s) : grad_ptr<kBF16>(s);
        // (a 16-bit row may have fewer groups of lanes than the workspace's size allows for)
        rc = run(fn, blocks, s.threads, &args, stream);
        if (rc != PDGEMM_OK || !need) return rc;
    }
    JoinArgs args = {static_cast<const float *>(workspace), dweight, (int)(rows > 0 ? blocks : 0), (int)cols};
    return run(reinterpret_cast<const void *>(&join_kernel), cdiv(cols, kWave), 1024, &args, stream);
}

}  // extern "C"
