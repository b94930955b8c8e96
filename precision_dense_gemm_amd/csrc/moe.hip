// moe.hip -- a mixture-of-experts layer of group-scaled INT4 weights for a few tokens, for
// gfx950 (MI355X): the choice of experts from the router's logits, and the chosen experts'
// gated feed-forward products with their weighted sum, behind the C ABI declared in
// include/pdgemm.h.
//
//   y[t] = sum over the token's slots s of weight[t][s] * W2[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])),  e = ids[t][s]
#include "i4_core.h"

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 64;
constexpr int kMaxPairs = 4096;
constexpr uint32_t kNone = 0xFFFFu;   // no pair

// ---------------------------------------------------------------------------
// routing

struct RouteArgs {
    const void *logits;
    int32_t *ids;
    float *weights;
    int64_t ld;
    int T, E, top, type;
    bool normalize;
};

// A wave per token, V logits to a lane.  Logits are compared as whole numbers in their order,
// NaN above all; -infinity is 0, which is never taken.
template <int V>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = threadIdx.x % kWave;
    const int t = blockIdx.x * 4 + threadIdx.x / kWave;
    if (t >= args.T) return;
    float x[V];
    uint32_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = j * kWave + lane;
        float v[1] = {-__builtin_inff()};
        if (e < args.E) load_some_as_float<1>(v, args.logits, args.type, t * args.ld + e, 1);
        x[j] = v[0];
        const uint32_t u = bits_of(v[0] + 0.0f);   // (-0 ties with 0)
        key[j] = v[0] != v[0] ? 0xFFFFFFFFu : u == 0xFF800000u ? 0u : u >> 31 ? ~u : u | 0x80000000u;
    }
    int id = -1;           // of slot `lane`
    float mine = 0, first = 0;
    int taken = 0;
    for (int s = 0; s < args.top; ++s) {
        uint32_t m = key[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = max(m, key[j]);
        m = max_over_lanes<kWave>(m);
        if (m == 0) break;
        int at = -1;       // the lowest index that has it
#pragma unroll
        for (int j = V - 1; j >= 0; --j) {
            const uint64_t who = __ballot(key[j] == m);
            if (who) at = j * kWave + __builtin_ctzll(who);
        }
        float v = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (at / kWave == j) {
                v = x[j];
                if (at % kWave == lane) key[j] = 0;
            }
        v = __shfl(v, at % kWave);
        if (s == 0) first = v;
        if (s == lane) id = at, mine = v;
        ++taken;
    }
    float e = lane < taken ? expf(mine - first) : 0.0f;
    float sum = e;
    if (!args.normalize) {
        sum = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (x[j] != -__builtin_inff()) sum += expf(x[j] - first);
    }
    sum = sum_over_lanes<kWave>(sum);
    if (lane < args.top) {
        args.ids[(int64_t)t * args.top + lane] = id;
        args.weights[(int64_t)t * args.top + lane] = lane < taken ? e / sum : 0.0f;
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// experts
//
// A pair is a token and one of its slots, p = t * top + s.  The first kernel computes the
// gated activations of every pair, times the pair's weight, in 16 bits: a row of `act` per
// pair.  The second adds the experts up: a tile of y's columns to a workgroup, whose waves
// share out all (expert, range of I), so no sum leaves the workgroup and their order is fixed.

struct MoeArgs {
    const uint8_t *x;
    const int32_t *ids;
    const float *weights;
    const uint8_t *w13, *w2;
    const uint8_t *s13, *s2;
    uint8_t *act;
    int32_t *active;        // how many experts have a token, then which
    uint16_t *table;        // of each of them: its pair for every token, or kNone
    uint8_t *y;
    int64_t ldx, ldact;     // bytes
    int64_t ld13, e13, ld2, e2;         // bytes: a row, an expert
    int64_t lds13, es13, lds2, es2;     // bytes
    int64_t ldy;            // elements
    int T, H, I, E, top;
    int most;               // of active experts
    int tiles;
    int group, s_type;
};

// The experts that some pair names, as bits, and their count; the a-th of them.
struct Active {
    uint32_t bits[kMaxExperts / 32];
    int count[kMaxExperts / 32];   // in the words before
    int total;
};
__device__ __forceinline__ void find_active(Active &act, const int32_t *ids, int pairs, int E) {
    const int tid = threadIdx.x;
    if (tid < kMaxExperts / 32) act.bits[tid] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += blockDim.x) {
        const int e = ids[p];
        if ((uint32_t)e < (uint32_t)E) atomicOr(&act.bits[e / 32], 1u << (e % 32));
    }
    __syncthreads();
    if (tid < kWave) {
        const int own = tid < kMaxExperts / 32 ? __builtin_popcount(act.bits[tid]) : 0;
        int n = own;
#pragma unroll
        for (int d = 1; d < kMaxExperts / 32; d *= 2) {
            const int before = __shfl_up(n, d);
            if (tid >= d) n += before;
        }
        if (tid < kMaxExperts / 32) act.count[tid] = n - own;
        if (tid == kMaxExperts / 32 - 1) act.total = n;
    }
    __syncthreads();
}
__device__ __forceinline__ int nth_active(const Active &act, int a) {
    int word = 0;
#pragma unroll
    for (int d = kMaxExperts / 64; d > 0; d /= 2)
        if (act.count[word + d] <= a) word += d;
    uint32_t left = act.bits[word];
    for (int n = a - act.count[word]; n > 0; --n) left &= left - 1;
    return word * 32 + __builtin_ctz(left);
}

// Gate and up rows of one active expert: 8 NT rows of each (tile t of the wave has the gate's
// rows where t is even, else the up projection's).
template <int T, int MT, int NT, int W, int Q, bool kS32, int D>
__global__ __launch_bounds__(W *kWave) void moe_up_kernel(MoeArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    constexpr int kCols = 8 * NT, kTile = MT * NT * 256;
    __shared__ Active active;
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int listed;
    __shared__ float part[W][kTile];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane % 16, g = lane / 16;
    const int a = blockIdx.x / args.tiles, tile = blockIdx.x % args.tiles;
    const int H = args.H, I = args.I, top = args.top, pairs = args.T * top;

    if (tid == 0) listed = 0;
    find_active(active, args.ids, pairs, args.E);
    if (blockIdx.x == 0 && tid == 0) args.active[0] = active.total;
    if (a >= active.total) return;
    const int e = __builtin_amdgcn_readfirstlane(nth_active(active, a));
    if (tile == 0) {
        if (tid == 0) args.active[1 + a] = e;
        for (int t = tid; t < args.T; t += W * kWave) {
            int p = kNone;
            for (int s = top - 1; s >= 0; --s)
                if (args.ids[t * top + s] == e) p = t * top + s;
            args.table[(int64_t)a * args.T + t] = (uint16_t)p;
        }
    }
    for (int p = tid; p < pairs; p += W * kWave)
        if (args.ids[p] == e) {
            bool again = false;   // an expert that a token names twice is computed once, with the weights' sum
            for (int q = p - p % top; q < p; ++q) again |= args.ids[q] == e;
            if (!again) list[atomicAdd(&listed, 1)] = (uint16_t)p;
        }
    __syncthreads();
    const int rows = listed;

    const int i0 = tile * kCols;
    const int cols = min(kCols, I - i0);
    using Wave = I4Wave<T, MT, NT, 2, Q, kS32, D>;
    typename Wave::Source src;
    src.a = args.x;
    src.a_end = (int)((args.T - 1) * args.ldx) + ((2 * H + 15) & ~15);
    const int size = kS32 ? 4 : 2;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        src.b[b] = args.w13 + e * args.e13 + (int64_t)(b * I + i0) * args.ld13;
        src.b_end[b] = (int)((cols - 1) * args.ld13) + (((H + 1) / 2 + 15) & ~15);
        src.s[b] = {args.s13 + e * args.es13 + (int64_t)(b * I + i0) * size, args.lds13, args.s_type};
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = 16 * (t / 2) + r;
        src.vb[t] = row < cols ? (uint32_t)row * (uint32_t)args.ld13 + 16 * g : kOutside;
        src.vs[t] = (uint32_t)min(row, cols - 1) * size;
    }
    src.K = H, src.group = args.group;
    const int steps = (H + kStep - 1) / kStep, lines = (steps + 1) / 2;
    const int mine = wave < lines ? (lines - wave + W - 1) / W : 0;
    const int odd = mine > 0 && wave + (mine - 1) * W == lines - 1 ? steps % 2 : 0;
    for (int first = 0; first < rows; first += 16 * MT) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int at = first + 16 * i + r;
            src.va[i] = at < rows ? (uint32_t)(list[at] / top) * (uint32_t)args.ldx + 16 * g : kOutside;
        }
        Wave w;
        w.run(src, 2 * mine - odd, [&](int i, auto &) { return 2 * (wave + (i >> 1) * W) + (i & 1); });
        if (first > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) part[wave][((i * NT + t) * 4 + k) * kWave + lane] = w.acc[i][t][k];
        __syncthreads();
        for (int x = tid; x < 16 * MT * kCols; x += W * kWave) {
            const int row = x / kCols, col = x % kCols;
            if (first + row >= rows || col >= cols) continue;
            const int at = ((row / 16 * NT + col / 16 * 2) * 4 + row % 4) * kWave + row % 16 / 4 * 16 + col % 16;
            float gate = part[0][at], up = part[0][at + 4 * kWave];
#pragma unroll
            for (int v = 1; v < W; ++v) gate += part[v][at], up += part[v][at + 4 * kWave];
            const int p = list[first + row];
            float weight = args.weights[p];
            for (int q = p + 1; q < p - p % top + top; ++q)
                if (args.ids[q] == e) weight += args.weights[q];
            // (rounded to the type that the second product's matrix instructions take)
            reinterpret_cast<Elem *>(args.act + (int64_t)p * args.ldact)[i0 + col] =
                (Elem)(gate / (1.0f + __expf(-gate)) * up * weight);
        }
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// Columns of y.  Row t of a fragment of activations is token t's, for every expert: its pair's
// row of `act`, or nothing, so the experts add up in the accumulators.
template <int T, int MT, int NT, int W, int Q, bool kS32, int D>
__global__ __launch_bounds__(W *kWave) void moe_down_kernel(MoeArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    constexpr int kCols = 16 * NT, kRows = 16 * MT, kTile = MT * NT * 256;
    extern __shared__ uint8_t lds[];   // the pairs of each expert, then the waves' sums
    uint16_t *const pair = reinterpret_cast<uint16_t *>(lds);
    float(*const part)[kTile] = reinterpret_cast<float(*)[kTile]>(lds);
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane % 16, g = lane / 16;
    const int t0 = blockIdx.x / args.tiles * kRows, n0 = blockIdx.x % args.tiles * kCols;
    const int H = args.H, I = args.I;
    const int experts = __builtin_amdgcn_readfirstlane(min(args.active[0], args.most));

    for (int x = tid; x < experts * kRows; x += W * kWave) {
        const int t = t0 + x % kRows;
        pair[x] = t < args.T ? args.table[(int64_t)(x / kRows) * args.T + t] : (uint16_t)kNone;
    }
    __syncthreads();

    using Wave = I4Wave<T, MT, NT, 1, Q, kS32, D, true>;
    typename Wave::Source src;
    src.a = args.act;
    src.a_end = (int)((args.T * args.top - 1) * args.ldact) + ((2 * I + 15) & ~15);
    const int cols = min(kCols, H - n0), size = kS32 ? 4 : 2;
    src.b_end[0] = (int)((cols - 1) * args.ld2) + (((I + 1) / 2 + 15) & ~15);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = 16 * t + r;
        src.vb[t] = row < cols ? (uint32_t)row * (uint32_t)args.ld2 + 16 * g : kOutside;
        src.vs[t] = (uint32_t)min(row, cols - 1) * size;
    }
    src.K = I, src.group = args.group;
    // unit u: a pair of steps of one expert, wave u % W's
    const int steps = (I + kStep - 1) / kStep, lines = (steps + 1) / 2;
    const int units = experts * lines, mine = wave < units ? (units - wave + W - 1) / W : 0;
    const int by_expert = W / lines, by_line = W % lines;
    int at = wave / lines, line = wave % lines;   // of the next unit
    Wave w;
    w.run(src, 2 * mine, [&](int i, auto &src) -> int {
        if (i % 2) {   // the second step of the unit, which an odd number of steps leaves out
            const int step = 2 * line + 1;
            at += by_expert, line += by_line;
            if (line >= lines) line -= lines, ++at;
            return step < steps ? step : -1;
        }
        const int e = __builtin_amdgcn_readfirstlane(args.active[1 + at]);
        src.b[0] = args.w2 + e * args.e2 + (int64_t)n0 * args.ld2;
        src.s[0] = {args.s2 + e * args.es2 + (int64_t)n0 * size, args.lds2, args.s_type};
#pragma unroll
        for (int k = 0; k < MT; ++k) {
            const uint32_t p = pair[at * kRows + 16 * k + r];
            src.va[k] = p != kNone ? p * (uint32_t)args.ldact + 16 * g : kOutside;
        }
        return 2 * line;
    });
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) part[wave][((i * NT + t) * 4 + k) * kWave + lane] = w.acc[i][t][k];
    __syncthreads();
    for (int x = tid; x < kTile; x += W * kWave) {
        const int row = x / kCols, col = x % kCols;
        if (t0 + row >= args.T || col >= cols) continue;
        const int from = ((row / 16 * NT + col / 16) * 4 + row % 4) * kWave + row % 16 / 4 * 16 + col % 16;
        float sum = part[0][from];
#pragma unroll
        for (int v = 1; v < W; ++v) sum += part[v][from];
        reinterpret_cast<Elem *>(args.y)[(int64_t)(t0 + row) * args.ldy + n0 + col] = (Elem)sum;
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// host side

int64_t round_up(int64_t x, int64_t m) { return cdiv(x, m) * m; }

// The workspace: act, then the active experts, then the table of pairs
struct Workspace {
    int64_t ldact, active, table, bytes;   // bytes: a row of act; where the others begin; in all
};
Workspace workspace_of(int64_t T, int64_t top, int64_t I, int64_t E) {
    const int64_t pairs = T * top, most = E < pairs ? E : pairs;
    Workspace w;
    w.ldact = round_up(2 * I, 16);
    w.active = pairs * w.ldact;
    w.table = w.active + round_up(4 * (1 + most), 16);
    w.bytes = w.table + round_up(2 * most * T, 16);
    return w;
}

bool moe_sizes_ok(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top) {
    const int64_t row = kMaxRowBytes;
    return T >= 0 && H > 0 && I > 0 && E > 0 && E <= kMaxExperts && top > 0 && top <= kMaxTop && T <= kMaxPairs / top &&
           H <= row / 2 && I <= row / 2 && T * top * (2 * I + 16) <= INT32_MAX;
}

template <int T, int Q, bool kS32>
int launch_moe(MoeArgs args, void *stream) {
    // (a token's experts are few of many: a fragment's 16 rows hold an expert's pairs)
    args.tiles = (int)cdiv(args.I, 16);
    int rc = run(reinterpret_cast<const void *>(&moe_up_kernel<T, 1, 2, 8, Q, kS32, 4>), (int64_t)args.most * args.tiles, 512,
                 &args, stream);
    if (rc != PDGEMM_OK) return rc;
    int mt = args.T <= 16 ? 1 : args.T <= 32 ? 2 : 4;
    while (mt > 1 && 32 * mt * args.most > 64 * 1024) mt /= 2;
    args.tiles = (int)cdiv(args.H, 16);
    const int waves = mt == 4 ? 8 : 16;
    const int join = waves * mt * 1024, table = 32 * mt * args.most, bytes = join > table ? join : table;
    const void *fn = mt == 1   ? reinterpret_cast<const void *>(&moe_down_kernel<T, 1, 1, 16, Q, kS32, 4>)
                     : mt == 2 ? reinterpret_cast<const void *>(&moe_down_kernel<T, 2, 1, 16, Q, kS32, 2>)
                               : reinterpret_cast<const void *>(&moe_down_kernel<T, 4, 1, 8, Q, kS32, 2>);
    void *kargs[] = {&args};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return finish(hipLaunchKernel(fn, dim3((unsigned)(cdiv(args.T, 16 * mt) * args.tiles)), dim3(waves * kWave), kargs, bytes, s), s);
}
template <int T, bool kS32>
int launch_moe(const MoeArgs &args, void *stream) {
    return args.group % 128 == 0  ? launch_moe<T, 4, kS32>(args, stream)
           : args.group % 64 == 0 ? launch_moe<T, 2, kS32>(args, stream)
                                  : launch_moe<T, 1, kS32>(args, stream);
}

// the codes and scales of E experts of N rows of K values
int check_expert_sizes(int64_t N, int64_t K, int64_t ld, int64_t expert, int64_t lds, int64_t expert_s) {
    return ld < K || lds < N || expert < 0 || expert_s < 0 ? PDGEMM_EINVAL_LD : PDGEMM_OK;
}
int check_expert_memory(const uint8_t *w, int64_t ld, int64_t expert, const void *s, int64_t lds, int scale_type) {
    if (!w) return PDGEMM_ENULL;
    const int rc = check_plain(s, lds, scale_type);
    if (rc != PDGEMM_OK) return rc;
    if (ld > 2 * kMaxRowBytes) return PDGEMM_EINVAL_LD;
    return ld % 32 || expert % 32 || ((uintptr_t)w & 15) ? PDGEMM_EALIGN : PDGEMM_OK;
}

}  // namespace

extern "C" {

int pdgemm_moe_route(int64_t T, int64_t E, int64_t top, const void *logits, int64_t ld, int type, int normalize, int32_t *ids,
                     float *weights, void *stream) {
    if (!known_type(type)) return PDGEMM_EINVAL_CFG;
    if (T < 0 || T > (int64_t(1) << 30) || E <= 0 || E > kMaxExperts || top <= 0 || top > kMaxTop || top > E)
        return PDGEMM_EINVAL_DIM;
    if (ld < E) return PDGEMM_EINVAL_LD;
    if (T == 0) return PDGEMM_OK;
    int rc = check_plain(logits, ld, type);
    if (rc == PDGEMM_OK) rc = check_plain(ids, 1, kF32);
    if (rc == PDGEMM_OK) rc = check_plain(weights, 1, kF32);
    if (rc != PDGEMM_OK) return rc;
    RouteArgs args = {logits, ids, weights, ld, (int)T, (int)E, (int)top, type, normalize != 0};
    const void *fn = E <= 64    ? reinterpret_cast<const void *>(&moe_route_kernel<1>)
                     : E <= 128 ? reinterpret_cast<const void *>(&moe_route_kernel<2>)
                     : E <= 256 ? reinterpret_cast<const void *>(&moe_route_kernel<4>)
                                : reinterpret_cast<const void *>(&moe_route_kernel<16>);
    return run(fn, cdiv(T, 4), 256, &args, stream);
}

int64_t pdgemm_moe_a16_i4_workspace_size(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top) {
    return moe_sizes_ok(T, H, I, E, top) && T > 0 ? workspace_of(T, top, I, E).bytes : 0;
}

int pdgemm_moe_a16_i4(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top, const void *x, int64_t ldx, int type,
                      const int32_t *ids, const float *weights, const uint8_t *w13, int64_t ld13, int64_t expert13,
                      const void *s13, int64_t lds13, int64_t expert_s13, const uint8_t *w2, int64_t ld2, int64_t expert2,
                      const void *s2, int64_t lds2, int64_t expert_s2, int scale_type, int64_t group, void *y, int64_t ldy,
                      void *workspace, int64_t workspace_bytes, void *stream) {
    if ((type != kF16 && type != kBF16) || !known_type(scale_type) || group <= 0 || group % kBlock || group > (int64_t(1) << 30))
        return PDGEMM_EINVAL_CFG;
    if (!moe_sizes_ok(T, H, I, E, top)) return PDGEMM_EINVAL_DIM;
    if (ldx < H || ldy < H) return PDGEMM_EINVAL_LD;
    int rc = check_expert_sizes(2 * I, H, ld13, expert13, lds13, expert_s13);
    if (rc == PDGEMM_OK) rc = check_expert_sizes(H, I, ld2, expert2, lds2, expert_s2);
    if (rc != PDGEMM_OK) return rc;
    if (T == 0) return PDGEMM_OK;
    rc = check_plain(y, ldy, type);
    if (rc == PDGEMM_OK) rc = check_plain(x, ldx, type);
    if (rc == PDGEMM_OK) rc = check_plain(ids, 1, kF32);
    if (rc == PDGEMM_OK) rc = check_plain(weights, 1, kF32);
    if (rc == PDGEMM_OK) rc = check_expert_memory(w13, ld13, expert13, s13, lds13, scale_type);
    if (rc == PDGEMM_OK) rc = check_expert_memory(w2, ld2, expert2, s2, lds2, scale_type);
    if (rc == PDGEMM_OK && T * ldx * 2 > INT32_MAX) rc = PDGEMM_EINVAL_LD;
    if (rc == PDGEMM_OK && (ldx % 8 || ((uintptr_t)x & 15))) rc = PDGEMM_EALIGN;
    if (rc == PDGEMM_OK && !workspace) rc = PDGEMM_ENULL;
    const Workspace w = workspace_of(T, top, I, E);
    if (rc == PDGEMM_OK && (workspace_bytes < w.bytes || ((uintptr_t)workspace & 15))) rc = PDGEMM_EWORKSPACE;
    if (rc != PDGEMM_OK) return rc;
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    const int size = elem_size(scale_type);
    const int64_t pairs = T * top;
    const MoeArgs args = {static_cast<const uint8_t *>(x), ids, weights, w13, w2, static_cast<const uint8_t *>(s13),
                          static_cast<const uint8_t *>(s2), ws, reinterpret_cast<int32_t *>(ws + w.active),
                          reinterpret_cast<uint16_t *>(ws + w.table), static_cast<uint8_t *>(y), 2 * ldx, w.ldact, ld13 / 2,
                          expert13 / 2, ld2 / 2, expert2 / 2, lds13 * size, expert_s13 * size, lds2 * size, expert_s2 * size, ldy,
                          (int)T, (int)H, (int)I, (int)E, (int)top, (int)(E < pairs ? E : pairs), 0, (int)group, scale_type};
    const bool s32 = scale_type == kF32;
    if (type == kF16) return s32 ? launch_moe<kF16, true>(args, stream) : launch_moe<kF16, false>(args, stream);
    return s32 ? launch_moe<kBF16, true>(args, stream) : launch_moe<kBF16, false>(args, stream);
}

}  // extern "C"
