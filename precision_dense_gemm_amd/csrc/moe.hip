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
constexpr int kMaxSplits = 8;
constexpr int kUpWaves = 4;   // of a workgroup of the first product

// ---------------------------------------------------------------------------
// routing

struct RouteArgs {
    const void *logits;
    int32_t *ids;
    float *weights;
    int64_t ld;
    int T, E, top, type;
    int across;             // of block_of()
    bool normalize;
};

// A wave per token, V logits to a lane.  Logits are compared as whole numbers in their order,
// NaN above all; -infinity is 0, which is never taken.  One maximum over the lanes for each slot, one after the
// other, bounds it: 8 of 128 take 4.6 us (the shortest kernel here 2.3).
template <int V>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = threadIdx.x % kWave;
    const int t = block_of(args.across) * 4 + threadIdx.x / kWave;
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
// A pair is a token and one of its slots, p = t * top + s; an expert that a token names twice is
// computed for the first of the slots, with the weights' sum.  The first kernel computes the gated
// activations of every pair, times its weight: a row of `act` per pair, which the second product's matrix
// instructions take in 16 bits.  A value of two bf16 parts (wide) keeps binary32's range and is within 2^-16 of
// itself, a 32nd of the rounding of an f16 y; rounded to x's type it would add an error as large as y's own
// rounding, and in f16 end at 65504.  The parts are two rows of one matrix instruction, which few pairs leave
// room for.  Where the caller's workspace holds one part only, it is of x's type.  The second kernel adds
// the experts up: 16 columns of y to a workgroup, whose waves share out all (expert, line of
// its rows), each with sums of its own for every token, so no sum leaves the workgroup and
// their order is fixed.  Both read an expert's codes once (once for 1 to 16 of its pairs), and their stream
// bounds them: 16 tokens through 8 of 128 experts (H 2048, I 768, f16, groups of 64), 206 MB of codes and
// scales, take 75 us with the routing, 38 to 42 for the first kernel (137 MB) and 28 to 29 for the second (69 MB, one
// workgroup to a CU: 2.4 TB/s); one token through 4 of 32 (H 4096, I 2048, bf16, groups of 128), 52 MB, 24.
// Past 64 tokens a workgroup of the second kernel goes through all experts' pairs for its 64, so its time grows with the
// square: through 8 of 32 experts (H 2048, I 1024) 64 tokens take 85 us, 128 192, 256 570 and 512 1980.

struct MoeArgs {
    const uint8_t *x;
    const int32_t *ids;
    const float *weights;
    const uint8_t *w13, *w2;
    const uint8_t *s13, *s2;
    uint8_t *act;
    int64_t act2;           // bytes from a value to its second part (0: one part)
    int32_t *active;        // how many experts have a token, and which
    int32_t *offset;        // where the pairs of each of them begin in `order`, and their end
    uint16_t *order;        // the pairs by expert
    float *part;            // the splits' sums, T x H each
    uint8_t *y;
    int64_t ldx, ldact;     // bytes
    int64_t ld13, e13, ld2, e2;         // bytes: a row, an expert
    int64_t lds13, es13, lds2, es2;     // bytes
    int64_t ldy;            // elements
    int T, H, I, E, top;
    int type;               // of x and y
    int most;               // of active experts
    int tiles;              // workgroups along an expert's rows
    int wk;                 // waves that share a tile's K
    int splits;             // workgroups that share a tile of y
    int group;
    uint32_t s_half;        // of I4Scales
    uint32_t group_magic;
};

// The experts that some pair names, as bits, and their count; the a-th of them, and which one e is.
struct Active {
    uint32_t bits[kMaxExperts / 32];
    int count[kMaxExperts / 32];   // in the words before
    int total;
};
__device__ __forceinline__ void find_active(Active &act, const int *ids, int pairs, int E) {   // (ids in LDS)
    const int tid = threadIdx.x;
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
__device__ __forceinline__ int rank_of(const Active &act, int e) {
    return act.count[e / 32] + __builtin_popcount(act.bits[e / 32] & ((1u << (e % 32)) - 1));
}

// whether an earlier slot of pair p's token names the same expert (ids in LDS)
__device__ __forceinline__ bool named_before(const int *ids, int p, int top) {
    bool found = false;
    for (int q = p - p % top; q < p; ++q) found |= ids[q] == ids[p];
    return found;
}

// active, offset and order, by one workgroup; ids, n: LDS, n of kMaxExperts
__device__ __forceinline__ void sort_pairs(const MoeArgs &args, const Active &act, const int *ids, int *n) {
    const int tid = threadIdx.x, pairs = args.T * args.top;
    for (int a = tid; a < act.total; a += blockDim.x) {
        n[a] = 0;
        args.active[1 + a] = nth_active(act, a);
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += blockDim.x)
        if ((uint32_t)ids[p] < (uint32_t)args.E && !named_before(ids, p, args.top)) atomicAdd(&n[rank_of(act, ids[p])], 1);
    __syncthreads();
    if (tid < kWave) {
        constexpr int kEach = kMaxExperts / kWave;
        int own = 0;
        for (int i = 0; i < kEach; ++i) own += tid * kEach + i < act.total ? n[tid * kEach + i] : 0;
        int sum = own;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int before = __shfl_up(sum, d);
            if (tid >= d) sum += before;
        }
        int at = sum - own;
        for (int i = 0; i < kEach; ++i) {
            const int a = tid * kEach + i;
            if (a >= act.total) break;
            const int c = n[a];
            n[a] = args.offset[a] = at;
            at += c;
        }
        if (tid == kWave - 1) {
            args.active[0] = act.total;
            args.offset[act.total] = sum;
        }
    }
    __syncthreads();
    // (the order within an expert is whichever comes first: nothing is added up along it)
    for (int p = tid; p < pairs; p += blockDim.x)
        if ((uint32_t)ids[p] < (uint32_t)args.E && !named_before(ids, p, args.top))
            args.order[atomicAdd(&n[rank_of(act, ids[p])], 1)] = (uint16_t)p;
    __syncthreads();
}

// 16 gate rows of an active expert and the up projection's 16 beside them to args.wk waves, which
// split K; RA pairs at a time.
template <int T, int RA, int Q, bool kS32>
__global__ __launch_bounds__(kUpWaves *kWave) void moe_up_kernel(MoeArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Elem = typename ElemOf<T>::type;
    using Wave = I4Wave<T, RA, 2, 2, Q, kS32, true>;
    constexpr int W = kUpWaves;
    // all pairs' experts and weights, then the expert's own pairs and their weights
    extern __shared__ int ids[];
    float *const weights = reinterpret_cast<float *>(ids + args.T * args.top), *const own_weight = weights + args.T * args.top;
    uint16_t *const own = reinterpret_cast<uint16_t *>(own_weight + args.T);
    __shared__ Active active;
    __shared__ int listed;
    __shared__ union {
        int n[kMaxExperts];
        typename Wave::Lds wave[W];
        floatx4_t part[W][2][kWave];
    } lds;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane % 16, g = lane / 16;
    const int a = blockIdx.x / args.tiles;
    const int H = args.H, I = args.I, top = args.top, pairs = args.T * top;

    if (tid == 0) listed = 0;
    if (tid < kMaxExperts / 32) active.bits[tid] = 0;
    for (int p = tid; p < pairs; p += W * kWave) {
        ids[p] = args.ids[p];
        weights[p] = args.weights[p];
    }
    __syncthreads();
    find_active(active, ids, pairs, args.E);
    if (blockIdx.x == 0) sort_pairs(args, active, ids, lds.n);
    if (a >= active.total) return;
    const int e = __builtin_amdgcn_readfirstlane(nth_active(active, a));
    for (int p = tid; p < pairs; p += W * kWave)
        if (ids[p] == e && !named_before(ids, p, top)) {
            float weight = weights[p];
            for (int q = p + 1; q < p - p % top + top; ++q) weight += ids[q] == e ? weights[q] : 0.0f;
            const int at = atomicAdd(&listed, 1);
            own[at] = (uint16_t)p;
            own_weight[at] = weight;
        }
    __syncthreads();
    const int rows = listed;

    const int wk = args.wk, k0 = wave % wk;
    const int i0 = (blockIdx.x % args.tiles * (W / wk) + wave / wk) * 16;
    const int cols = min(16, I - i0);   // (a wave may have none)
    typename Wave::Source src;
    src.a = args.x;
    src.a_end = (int)((args.T - 1) * args.ldx) + ((2 * H + 15) & ~15);
    const int size = kS32 ? 4 : 2;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int64_t row = b * I + i0;
        src.b[b] = args.w13 + e * args.e13 + row * args.ld13;
        src.b_end[b] = (int)((cols - 1) * args.ld13) + (((H + 1) / 2 + 15) & ~15);
        src.s[b] = {args.s13 + e * args.es13 + row * size, args.lds13, args.s_half};
        const int at = Wave::code_row();
        src.vb[b] = at < cols ? (uint32_t)at * (uint32_t)args.ld13 + 16 * Wave::code_chunk() : kOutside;
        src.vs[b] = (uint32_t)min(r, cols - 1) * size;
    }
    src.K = H, src.group_magic = args.group_magic, src.groups = (H + args.group - 1) / args.group;
    const int units = cols > 0 ? (H + 2 * kStep - 1) / (2 * kStep) : 0;
    for (int first = 0; first < rows; first += RA) {
#pragma unroll
        for (int j = 0; j < Wave::kX; ++j) {
            const int at = first + Wave::copied_row(j);
            src.xa[j] = Wave::copied_row(j) < RA && at < rows ? (uint32_t)(own[at] / top) * (uint32_t)args.ldx + 16 * Wave::copied_chunk() : kOutside;
        }
        int next = k0;
        Wave w;
        w.run(
            src, lds.wave[wave],
            [&](auto &, auto &) {
                if (next >= units) return -1;
                const int unit = next;
                next += wk;
                return unit;
            },
            [](auto &) {});
        if (wk > 1) {
            __syncthreads();   // (the sums take the activations' place)
            lds.part[wave][0][lane] = w.acc[0];
            lds.part[wave][1][lane] = w.acc[1];
            __syncthreads();
            if (k0 == 0)
                for (int k = 1; k < wk; ++k) {
                    w.acc[0] += lds.part[wave + k][0][lane];
                    w.acc[1] += lds.part[wave + k][1][lane];
                }
            __syncthreads();
        }
        if (k0 != 0 || r >= cols) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = first + 4 * g + k;
            if (4 * g + k >= RA || at >= rows) break;
            const float gate = w.acc[0][k], up = w.acc[1][k];
            const float v = gate / (1.0f + __expf(-gate)) * up * own_weight[at];
            uint8_t *const row = args.act + (int64_t)own[at] * args.ldact;
            if (args.act2) {
                // (the first part of the largest finite values is cut off: rounded, it would be infinite)
                const float most = __builtin_copysignf(0x1.FEp127f, v);
                const bool finite = v * 0.0f == 0.0f;
                const __bf16 one = (__bf16)(finite && __builtin_fabsf(v) > 0x1.FEp127f ? most : v);
                reinterpret_cast<__bf16 *>(row)[i0 + r] = one;
                reinterpret_cast<__bf16 *>(row + args.act2)[i0 + r] = (__bf16)(finite ? v - (float)one : 0.0f);
            } else {
                reinterpret_cast<Elem *>(row)[i0 + r] = (Elem)v;
            }
        }
    }
#endif  // __HIP_DEVICE_COMPILE__
}

__device__ __forceinline__ void store_y(const MoeArgs &args, int t, int col, float v) {
    uint16_t *const at = reinterpret_cast<uint16_t *>(args.y) + (int64_t)t * args.ldy + col;
    if (args.type == kF16)
        *reinterpret_cast<_Float16 *>(at) = (_Float16)v;
    else
        *reinterpret_cast<__bf16 *>(at) = (__bf16)v;
}

// 16 columns of y for TT tokens.  Where there are few such tiles, args.splits workgroups share
// the (expert, line) pairs of one, and their sums are added up by moe_join_kernel.  (With the last of them to
// finish adding up what the others wrote, ordered by fences of the device's scope, 16 tokens through 8 of 128
// experts took 180 us instead of 50: such a fence writes back and drops a whole L2.)
// T: the activations' type, kParts of them to a value.
template <int T, int RA, int TT, int W, int Q, bool kS32, int kParts>
__global__ __launch_bounds__(W *kWave) void moe_down_kernel(MoeArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Wave = I4Wave<T, RA, 1, 1, Q, kS32, true, kParts>;
    constexpr int kPairs = Wave::kRows;   // at a time
    __shared__ int expert[kMaxExperts], offset[kMaxExperts + 1];
    __shared__ uint16_t pair[kMaxPairs], token[kMaxPairs];
    __shared__ typename Wave::Lds own[W];
    __shared__ float sums[W][TT][16];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane % 16, g = lane / 16;
    const int tile = blockIdx.x / args.splits, split = blockIdx.x % args.splits;
    const int t0 = tile / args.tiles * TT, n0 = tile % args.tiles * 16;
    const int H = args.H, I = args.I;

    // (whole lists, so that no load waits for another's count: what lies past the counts is not looked at)
    const int experts = __builtin_amdgcn_readfirstlane(args.active[0]);
    for (int a = tid; a <= args.most; a += W * kWave) {
        if (a < args.most) expert[a] = args.active[1 + a];
        offset[a] = args.offset[a];
    }
    for (int i = tid; i < args.T * args.top; i += W * kWave) {
        const int p = args.order[i];
        pair[i] = (uint16_t)p;
        token[i] = (uint16_t)(p / args.top);
    }
    for (int i = lane; i < TT * 16; i += kWave) (&sums[wave][0][0])[i] = 0.0f;
    __syncthreads();

    const int cols = min(16, H - n0), size = kS32 ? 4 : 2;
    typename Wave::Source src;
    src.a = args.act, src.a2 = args.act + args.act2;
    // (a lane of kDirect has a part of its own: both are below 2^31 where T <= 2)
    const uint32_t second = kParts == 2 && Wave::kDirect ? (uint32_t)args.act2 : 0u;
    src.a_end = (int)second + (int)((args.T * args.top - 1) * args.ldact) + ((2 * I + 15) & ~15);
    src.b_end[0] = (int)((cols - 1) * args.ld2) + (((I + 1) / 2 + 15) & ~15);
    src.vb[0] = Wave::code_row() < cols ? (uint32_t)Wave::code_row() * (uint32_t)args.ld2 + 16 * Wave::code_chunk() : kOutside;
    src.vs[0] = (uint32_t)min(r, cols - 1) * size;
    src.K = I, src.group_magic = args.group_magic, src.groups = (I + args.group - 1) / args.group;
    // (expert, line) number i is wave i's of the splits' waves, round and round; an expert of more than kPairs
    // pairs takes a turn for every kPairs
    const int lines = (I + 2 * kStep - 1) / (2 * kStep);
    const int stride = W * args.splits, by_expert = stride / lines, by_line = stride % lines;
    int at = (split * W + wave) / lines, line = (split * W + wave) % lines, first = 0;
    Wave w;
    w.run(
        src, own[wave],
        [&](auto &st, auto &src) {
            if (at >= experts) return -1;
            const int e = __builtin_amdgcn_readfirstlane(expert[at]);
            const int from = __builtin_amdgcn_readfirstlane(offset[at]), to = __builtin_amdgcn_readfirstlane(offset[at + 1]);
            st.tag = from + first;
            st.left = min(to - st.tag, kPairs);
            src.b[0] = args.w2 + e * args.e2 + (int64_t)n0 * args.ld2;
            src.s[0] = {args.s2 + e * args.es2 + (int64_t)n0 * size, args.lds2, args.s_half};
#pragma unroll
            for (int j = 0; j < Wave::kX; ++j) {
                const int row = Wave::copied_row(j) / kParts, i = st.tag + min(row, st.left - 1);
                const bool in = row < st.left && (uint32_t)(token[i] - t0) < (uint32_t)TT;
                src.xa[j] = in ? (uint32_t)pair[i] * (uint32_t)args.ldact + 16 * Wave::copied_chunk() : kOutside;
                if (Wave::copied_row(j) % kParts == 1) src.xa[j] += second;
            }
            const int unit = line;
            first += kPairs;
            if (from + first >= to) {
                first = 0, at += by_expert, line += by_line;
                if (line >= lines) line -= lines, ++at;
            }
            return unit;
        },
        [&](auto &st) {
            // a token has one pair of an expert: the lanes add to different sums
#pragma unroll
            for (int k = 0; k < 4; k += kParts) {
                const int row = (4 * g + k) / kParts;
                const int t = token[st.tag + min(row, st.left - 1)] - t0;
                const float sum = kParts == 1 ? w.acc[0][k] : w.acc[0][k] + w.acc[0][k + kParts - 1];
                if (row < st.left && (uint32_t)t < (uint32_t)TT) sums[wave][t][r] += sum;
            }
            wave_lds_order();
            w.clear();
        });
    __syncthreads();
    for (int x = tid; x < TT * 16; x += W * kWave) {
        const int t = x / 16, col = x % 16;
        if (t0 + t >= args.T || col >= cols) continue;
        float sum = sums[0][t][col];
#pragma unroll
        for (int v = 1; v < W; ++v) sum += sums[v][t][col];
        if (args.splits == 1)
            store_y(args, t0 + t, n0 + col, sum);
        else
            args.part[((int64_t)split * args.T + t0 + t) * H + n0 + col] = sum;
    }
#endif  // __HIP_DEVICE_COMPILE__
}

// y from the splits' sums, added in their order.
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs args) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int x = blockIdx.x * 256 + threadIdx.x, t = x / args.H, col = x % args.H;
    if (t >= args.T) return;
    float v[kMaxSplits], sum = 0;
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k) v[k] = k < args.splits ? args.part[(int64_t)k * args.T * args.H + x] : 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxSplits; ++k)
        if (k < args.splits) sum += v[k];
    store_y(args, t, col, sum);
#endif  // __HIP_DEVICE_COMPILE__
}

// ---------------------------------------------------------------------------
// host side

int64_t round_up(int64_t x, int64_t m) { return cdiv(x, m) * m; }

// Tiles of y, of 16 columns for up to 64 tokens, and how many workgroups share one: as many as make
// 256, one for each CU, each of a few experts.  (With 128, 256 and 512 workgroups the layer takes, us: 16 tokens through 8
// of 128 experts, H 2048, I 768, 88, 71 and 67; 32 of them 114, 89 and 95; 64 through 4 of 64, H 1024, I 512, 42, 35 and
// 39; 61 through 6 of 60, H 2000, I 1001, 132, 102 and 110.  Two, four or eight experts to a workgroup at least: no
// difference in any of twelve shapes.)
int64_t y_tiles(int64_t T, int64_t H) { return cdiv(T, 64) * cdiv(H, 16); }
int splits_of(int64_t T, int64_t H, int64_t most) {
    int64_t s = 256 / y_tiles(T, H);
    if (s > most / 4) s = most / 4;
    return s < 2 ? 1 : s > kMaxSplits ? kMaxSplits : (int)s;
}

// The workspace: act (its parts one after the other), the active experts, their offsets, the order of pairs, the
// splits' sums
struct Workspace {
    int64_t ldact, act2, active, offset, order, part, bytes;   // bytes: a row of act; where the others begin; in all
    int most, splits;
};
Workspace workspace_of(int64_t T, int64_t top, int64_t H, int64_t I, int64_t E, int parts) {
    const int64_t pairs = T * top;
    Workspace w;
    w.most = (int)(E < pairs ? E : pairs);
    w.splits = splits_of(T, H, w.most);
    const int64_t list = round_up(4 * (1 + w.most), 16);
    w.ldact = round_up(2 * I, 16);
    w.act2 = (parts - 1) * pairs * w.ldact;
    w.active = w.act2 + pairs * w.ldact;
    w.offset = w.active + list;
    w.order = w.offset + list;
    w.part = w.order + round_up(2 * pairs, 16);
    w.bytes = w.part + (w.splits > 1 ? round_up(4 * w.splits * T * H, 16) : 0);
    return w;
}

bool moe_sizes_ok(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top) {
    const int64_t row = kMaxRowBytes;
    return T >= 0 && H > 0 && I > 0 && E > 0 && E <= kMaxExperts && top > 0 && top <= kMaxTop && T <= kMaxPairs / top &&
           H <= row / 2 && I <= row / 2 && T * top * (2 * I + 16) <= INT32_MAX;
}

template <int T, int RA, int Q, bool kS32, int kParts>
int launch_down(MoeArgs &args, void *stream) {
    constexpr int W = RA == 2 ? 16 : 8;   // (as registers and LDS allow)
    const int64_t blocks = y_tiles(args.T, args.H) * args.splits;
    if constexpr (RA > 2)   // (2 serve up to two tokens)
        if (args.T > 16)
            return run(reinterpret_cast<const void *>(&moe_down_kernel<T, RA, 64, W, Q, kS32, kParts>), blocks, W * kWave, &args, stream);
    return run(reinterpret_cast<const void *>(&moe_down_kernel<T, RA, 16, W, Q, kS32, kParts>), blocks, W * kWave, &args, stream);
}

template <int T, int RA, int Q, bool kS32>
int launch_moe(MoeArgs args, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t tiles = cdiv(args.I, 16);
    // waves that share a tile: as many as make 2048 of them, eight for each CU (with 1024, 2048 and 4096 the layer takes, us:
    // one token through 8 of 32 experts, H 4096, I 2048, 37, 30 and 30; the same of 4 experts 22, 19 and 19; 61 through 6
    // of 60, H 2000, I 1001, 102, 102 and 110)
    args.wk = 1;
    while (args.wk < kUpWaves && args.most * tiles * args.wk < 2048) args.wk *= 2;
    args.tiles = (int)cdiv(tiles * args.wk, kUpWaves);
    if ((int64_t)args.most * args.tiles * kUpWaves * kWave > (int64_t)UINT32_MAX) return PDGEMM_EINVAL_DIM;   // (as run())
    void *kargs[] = {&args};
    int rc = finish(hipLaunchKernel(reinterpret_cast<const void *>(&moe_up_kernel<T, RA, Q, kS32>),
                                    dim3((unsigned)(args.most * args.tiles)), dim3(kUpWaves * kWave), kargs,
                                    8 * args.T * args.top + 6 * args.T, s), s);
    if (rc != PDGEMM_OK) return rc;
    args.tiles = (int)cdiv(args.H, 16);
    // Of two parts, 1, 4 or 8 pairs at a time.  The layer, us, with 4 and with 8: experts of 2 pairs on average
    // (128 experts, H 2048, I 768, groups of 64) 90 and 96, of 3 104 and 105, of 4 123 and 118; (64, 2048, 1024, 128) 66 and
    // 70, 75 and 75, 85 and 82.  Two tokens (H 4096, I 2048) with 1 and with 4: of 32 experts 30 and 32, of 4 22 and 21.
    rc = args.act2 == 0                        ? launch_down<T, RA, Q, kS32, 1>(args, stream)
         : args.T <= 2                         ? launch_down<kBF16, 2, Q, kS32, 2>(args, stream)
         : args.T * args.top <= 3 * args.most ? launch_down<kBF16, 8, Q, kS32, 2>(args, stream)
                                               : launch_down<kBF16, 16, Q, kS32, 2>(args, stream);
    if (rc != PDGEMM_OK || args.splits == 1) return rc;
    return run(reinterpret_cast<const void *>(&moe_join_kernel), cdiv((int64_t)args.T * args.H, 256), 256, &args, stream);
}
// Pairs that the first product's rows of codes are read for at once: 8, or 16 where there are more than 4 for each expert
// (of all, or of as many as there are pairs; the host cannot tell which pairs name none).  The layer, us, with 8 and with
// 16, at 3, 4, 5, 6 and 8 pairs an expert: 64 experts (H 2048, I 1024, groups of 128) 74 and 77, 80 and 81, 87 and 84, 99
// and 91, 111 and 98; 60 (H 2000, I 1001, groups of 32) 86 and 91, 94 and 94, 104 and 100, 111 and 104, 168 and 153.
template <int T, int Q, bool kS32>
int launch_moe(const MoeArgs &args, void *stream) {
    const int pairs = args.T * args.top;
    return args.T <= 2              ? launch_moe<T, 2, Q, kS32>(args, stream)
           : pairs <= 4 * args.most ? launch_moe<T, 8, Q, kS32>(args, stream)
                                    : launch_moe<T, 16, Q, kS32>(args, stream);
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
    const int64_t blocks = cdiv(T, 4);
    const int across = blocks_across(blocks, 256);
    RouteArgs args = {logits, ids, weights, ld, (int)T, (int)E, (int)top, type, across, normalize != 0};
    const void *fn = E <= 64    ? reinterpret_cast<const void *>(&moe_route_kernel<1>)
                     : E <= 128 ? reinterpret_cast<const void *>(&moe_route_kernel<2>)
                     : E <= 256 ? reinterpret_cast<const void *>(&moe_route_kernel<4>)
                                : reinterpret_cast<const void *>(&moe_route_kernel<16>);
    return run_rows(fn, blocks, across, 256, &args, stream);
}

int64_t pdgemm_moe_a16_i4_workspace_size(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top) {
    return moe_sizes_ok(T, H, I, E, top) && T > 0 ? workspace_of(T, top, H, I, E, 1).bytes : 0;
}

int64_t pdgemm_moe_a16_i4_wide_workspace_size(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top) {
    return moe_sizes_ok(T, H, I, E, top) && T > 0 ? workspace_of(T, top, H, I, E, 2).bytes : 0;
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
    const Workspace wide = workspace_of(T, top, H, I, E, 2);
    const Workspace w = workspace_bytes >= wide.bytes ? wide : workspace_of(T, top, H, I, E, 1);
    if (rc == PDGEMM_OK && (workspace_bytes < w.bytes || ((uintptr_t)workspace & 15))) rc = PDGEMM_EWORKSPACE;
    if (rc != PDGEMM_OK) return rc;
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    const int size = elem_size(scale_type);
    const MoeArgs args = {static_cast<const uint8_t *>(x), ids, weights, w13, w2, static_cast<const uint8_t *>(s13),
                          static_cast<const uint8_t *>(s2), ws, w.act2, reinterpret_cast<int32_t *>(ws + w.active),
                          reinterpret_cast<int32_t *>(ws + w.offset), reinterpret_cast<uint16_t *>(ws + w.order), reinterpret_cast<float *>(ws + w.part), static_cast<uint8_t *>(y), 2 * ldx, w.ldact, ld13 / 2,
                          expert13 / 2, ld2 / 2, expert2 / 2, lds13 * size, expert_s13 * size, lds2 * size, expert_s2 * size, ldy,
                          (int)T, (int)H, (int)I, (int)E, (int)top, type, w.most, 0, 1, w.splits, (int)group,
                          scale_type == kF16 ? ~0u : 0u, I4Groups::magic(group)};
    const bool s32 = scale_type == kF32;
    if (type == kF16) return s32 ? launch_moe<kF16, true>(args, stream) : launch_moe<kF16, false>(args, stream);
    return s32 ? launch_moe<kBF16, true>(args, stream) : launch_moe<kBF16, false>(args, stream);
}

}  // extern "C"
