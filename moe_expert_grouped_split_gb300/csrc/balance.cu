// balance.cu: the router's losses and gradients: per sequence the experts'
// counts, their mean share of the scores and two losses (dwdp_balance_loss),
// and the logits' gradient from those losses and from the chosen experts'
// weights (dwdp_route_scored_grad).  Memory-bound: one pass over the logits.
//
// A token's logits lie in LANES lanes of a warp (32 / LANES tokens a warp at
// once), 4 V of them in a lane.  Shares and log-sum-exp come without a pass
// for the largest logit: with exp(z) (softmax) or s = 1 / (1 + exp(-z))
// (sigmoid) as they are, the sum says whether binary32 held them, and only a
// token whose sum lies outside [kLeast, kMost] is taken again relative to its
// largest logit.  (An exponential's relative error goes with its argument: so
// that is at most 32 more than the logits' spread.)  For the sigmoid with c = min(that, 0), else 0:
//   t = exp(z - c),  r = 16 / (1 + t exp(c)) = 16 (1 - s),  u = t r = 16 exp(-c) s,
//   p = u / sum u
// (16: the reciprocal of the largest t would be subnormal, and taken for 0) so neither small scores nor scores next to 1 lose their digits, and sum t
// serves the log-sum-exp as well.
#include <math_constants.h>

#include <algorithm>

#include "dwdp_internal.h"
#include "row_ops.h"

namespace dwdp {
namespace {

constexpr int kWarps = 16, kGradWarps = 8;  // of a block: the losses', the gradients'
// A token's choices in each of its lanes, for the most that E experts can have.
__host__ __device__ constexpr int choices_a_lane(int lanes) { return lanes >= 32 ? 1 : lanes == 16 ? 2 : 4; }
// (kMost: the sums times gradients of up to 2^90, a loss' scale in them, stay in binary32's range)
constexpr float kLeast = 0x1p-36f, kMost = 0x1p36f;
// exp(kTop) is 2^125.99, the most whose reciprocal is no subnormal: a sigmoid's
// exponents stop there where exp(z) would pass binary32's range.
constexpr float kTop = 87.33f;
constexpr float kSigmoidUnit = 16.0f;  // of u and r above
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// exp by the approximate power of two: its argument's rounding makes the
// relative error |x| 2^-23 or 2^-22, whichever is more; 0 below 2^-126.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / x, 0 below 2^-126.
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp_fast(float x) { return exp2_fast(x * kLog2e); }
// Sums and maxima over the LANES lanes of a token.
template <int LANES>
__device__ __forceinline__ float token_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ float token_max(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Four sums over the LANES lanes of a token: halves, then quarters of the lanes
// go on with some of the values each, and everybody gets all at the end.
template <int LANES>
__device__ __forceinline__ float4 token_sums(float a, float b, float c, float d) {
    constexpr uint32_t all = 0xffffffffu;
    const int lane = threadIdx.x % LANES;
    const bool upper = lane & (LANES / 2), odd = lane & (LANES / 4);
    const float u = (upper ? c : a) + __shfl_xor_sync(all, upper ? a : c, LANES / 2);
    const float v = (upper ? d : b) + __shfl_xor_sync(all, upper ? b : d, LANES / 2);
    float s = (odd ? v : u) + __shfl_xor_sync(all, odd ? u : v, LANES / 4);
#pragma unroll
    for (int o = LANES / 8; o > 0; o >>= 1) s += __shfl_xor_sync(all, s, o);
    return make_float4(__shfl_sync(all, s, 0, LANES), __shfl_sync(all, s, LANES / 4, LANES),
                       __shfl_sync(all, s, LANES / 2, LANES), __shfl_sync(all, s, 3 * LANES / 4, LANES));
}

// Two of them.
template <int LANES>
__device__ __forceinline__ float2 token_sums(float a, float b) {
    constexpr uint32_t all = 0xffffffffu;
    const bool upper = threadIdx.x % LANES & (LANES / 2);
    float s = (upper ? b : a) + __shfl_xor_sync(all, upper ? a : b, LANES / 2);
#pragma unroll
    for (int o = LANES / 4; o > 0; o >>= 1) s += __shfl_xor_sync(all, s, o);
    return make_float2(__shfl_sync(all, s, 0, LANES), __shfl_sync(all, s, LANES / 2, LANES));
}

// How rows lie: any E; a multiple of 4 (16-byte aligned rows); every column of
// every lane there.
enum Rows : int { ROWS_ANY, ROWS_VEC, ROWS_FULL };

// A token's lanes' place in shared memory: tokens on their way (depth() of them),
// each with its logits, columns 4 (v LANES + lane) .. + 3 of a lane, its choices
// and, for the gradients, their weights' gradients.  Every lane copies what it
// reads itself, but for the chosen logits.
template <int LANES, int V, bool DW>
struct Ring {
    static constexpr int kCols = 4 * V * LANES, kPer = choices_a_lane(LANES), kChoices = kPer * LANES;
    static constexpr int kDepth = 2;
    static constexpr int kStage = kCols + kChoices * (DW ? 2 : 1);  // 4-byte values
    static constexpr int kFloats = kDepth * kStage;
    float* at;  // of this token's lanes

    // -inf where there is no column; nothing is copied there
    __device__ __forceinline__ void clear(int E, int lane) const {
        for (int s = 0; s < kDepth; ++s)
#pragma unroll
            for (int i = 0; i < 4 * V; ++i) {
                const int c = 4 * (i / 4 * LANES + lane) + i % 4;
                if (c >= E) at[s * kStage + c] = -CUDART_INF_F;
            }
    }
    template <int ROWS>
    __device__ __forceinline__ void fetch(int s, const float* logits, const int32_t* ids, const float* dw, int64_t t, int E, int k,
                                          int lane) const {
        float* const to = at + s * kStage;
        const float* const row = logits + t * E;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 4 * (v * LANES + lane);
            if constexpr (ROWS != ROWS_ANY) {
                if (ROWS == ROWS_FULL || c < E) copy_async<16>(to + c, row + c);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < E) copy_async<4>(to + c + i, row + c + i);
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = lane + j * LANES;
            if (i >= k || !ids) continue;
            copy_async<4>(to + kCols + i, ids + t * k + i);
            if constexpr (DW) copy_async<4>(to + kCols + kChoices + i, dw + t * k + i);
        }
    }
    __device__ __forceinline__ void take(int s, int lane, float (&z)[4 * V]) const {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float4 q = reinterpret_cast<const float4*>(at + s * kStage)[v * LANES + lane];
            z[4 * v] = q.x;
            z[4 * v + 1] = q.y;
            z[4 * v + 2] = q.z;
            z[4 * v + 3] = q.w;
        }
    }
    __device__ __forceinline__ int choice(int s, int i) const { return __float_as_int(at[s * kStage + kCols + i]); }
    __device__ __forceinline__ float dw(int s, int i) const { return at[s * kStage + kCols + kChoices + i]; }
};

// A token's exp(z - c) and their sum.
template <int LANES, int V>
__device__ __forceinline__ float soft_terms(const float (&z)[4 * V], float (&e)[4 * V], float& c) {
    float sum = 0.0f;
    c = 0.0f;
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) {
        e[i] = exp_fast(z[i]);
        sum += e[i];
    }
    sum = token_sum<LANES>(sum);
    const bool lost = !(sum >= kLeast && sum <= kMost);
    if (__any_sync(0xffffffffu, lost)) {
        float m = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) m = max_nan(m, z[i]);
        m = token_max<LANES>(m);
        if (lost) c = m;
        // from the difference itself: of large logits, their product with
        // kLog2e alone would be off by more than 1
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) e[i] = exp_fast(z[i] - c);
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) sum += e[i];
        sum = token_sum<LANES>(sum);
    }
    return sum;
}

// 16 / (1 + t one)
__device__ __forceinline__ float sigmoid_rest(float t, float one) {
    return rcp_fast(fmaf(t, one * (1.0f / kSigmoidUnit), 1.0f / kSigmoidUnit));
}

// A token's u and r and the sum of u; z_sum, where asked for, gets sum t, and
// z_c its c.  Columns beyond E get u = 0.
template <int LANES, int V>
__device__ __forceinline__ float sigmoid_terms(const float (&z)[4 * V], float (&u)[4 * V], float (&r)[4 * V], float& c,
                                               bool want_z, float& z_sum, float& z_c) {
    c = 0.0f;
    float sum;
    // far: relative to c, from the difference itself (as in soft_terms)
    auto terms = [&](bool far, float one) {
        sum = z_sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) {
            const float t = far ? exp_fast(min_nan(z[i] - c, kTop)) : exp_fast(z[i]);
            r[i] = sigmoid_rest(t, one);
            u[i] = t * r[i];
            sum += u[i];
            z_sum += t;
        }
        if (want_z) {
            const float2 both = token_sums<LANES>(sum, z_sum);
            sum = both.x;
            z_sum = both.y;
        } else {
            sum = token_sum<LANES>(sum);
        }
    };
    terms(false, 1.0f);
    const bool lost = !(sum >= kSigmoidUnit * kLeast);  // too small, or a logit so large that u is inf 0
    if (__any_sync(0xffffffffu, lost)) {
        float m = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) m = max_nan(m, z[i]);
        m = token_max<LANES>(m);
        if (lost) c = min_nan(m, 0.0f);
        terms(true, exp_fast(c));
    }
    z_c = c;
    if (want_z && __any_sync(0xffffffffu, !(z_sum <= kMost))) {
        float e[4 * V];
        z_sum = soft_terms<LANES, V>(z, e, z_c);
    }
    return sum;
}

__device__ __forceinline__ float log_of(float sum, float c) { return c + __log2f(sum) * kLn2; }

__device__ __forceinline__ int seq_begin(const BalanceArgs& p, int b) {
    return p.offsets ? min(max(p.offsets[b], 0), p.T) : 0;
}
__device__ __forceinline__ int seq_end(const BalanceArgs& p, int b) {
    return p.offsets ? min(max(p.offsets[b + 1], 0), p.T) : p.T;
}

// A sequence's outputs from its sums, by the whole block.  sum_p(e), count(e):
// over the sequence.
template <class SumP, class Count>
__device__ __forceinline__ void finish_sequence(const BalanceArgs& p, int b, int tokens, float z_sum, SumP sum_p,
                                                Count count, float* red) {
    const float per_token = tokens > 0 ? 1.0f / (float)tokens : 0.0f;
    float loss = 0.0f, none = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        const float m = sum_p(e) * per_token;
        const int n = count(e);
        p.mean_p[(int64_t)b * p.E + e] = m;
        p.counts[(int64_t)b * p.E + e] = n;
        loss = fmaf((float)n, m, loss);
    }
    warp_sum_max<false>(loss, none);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = loss;
    __syncthreads();
    if (warp == 0) {
        loss = lane < nw ? red[lane] : 0.0f;
        warp_sum_max<false>(loss, none);
        if (lane == 0) {
            p.balance[b] = loss * ((float)p.E / (float)p.k) * per_token;
            if (p.z) p.z[b] = z_sum * per_token;
        }
    }
    __syncthreads();
}

// What a lane has summed up over its tokens.
template <int V>
struct TokenSums {
    float p[4 * V];
    float z;
};

// Adds up tokens `first`, first + step, ... below `to` for a warp (first: of
// its first LANES lanes, the next tokens for the others), and counts their
// choices in hist.  asked: the first tokens are on their way already.
template <int LANES, int V, int ROWS>
__device__ __forceinline__ void add_tokens(const BalanceArgs& p, const Ring<LANES, V, false>& ring, bool asked, int first, int to,
                                           int step, int* hist, TokenSums<V>& sums) {
    using R = Ring<LANES, V, false>;
    const int lane = threadIdx.x % LANES, sub = (threadIdx.x & 31) / LANES;
    auto fetch = [&](int64_t t0, int s) {  // a token of the warp at least is there
        if (t0 < to) ring.template fetch<ROWS>(s, p.logits, p.ids, nullptr, min((int)t0 + sub, to - 1), p.E, p.k, lane);
        end_copies();
    };
    if (!asked) {
#pragma unroll
        for (int s = 0; s < R::kDepth; ++s) fetch(first + (int64_t)s * step, s);
    }
    int s = 0;
    for (int t0 = first; t0 < to; t0 += step) {  // whole warps together
        wait_copies<R::kDepth - 1>();
        const bool in = t0 + sub < to;
        float z[4 * V], e[4 * V], c, sum;
        ring.take(s, lane, z);
#pragma unroll
        for (int j = 0; j < R::kPer; ++j) {
            if (!in || lane + j * LANES >= p.k) continue;
            const int id = ring.choice(s, lane + j * LANES);
            if (id >= 0 && id < p.E)
                atomicAdd(hist + id, 1);
            else
                atomicOr(p.err, DERR_BAD_INDEX);
        }
        fetch(t0 + (int64_t)R::kDepth * step, s);
        s = s + 1 == R::kDepth ? 0 : s + 1;
        float z_sum, z_c;
        if (p.sigmoid) {
            float r[4 * V];
            sum = sigmoid_terms<LANES, V>(z, e, r, c, p.z != nullptr, z_sum, z_c);
        } else {
            z_sum = sum = soft_terms<LANES, V>(z, e, c);
            z_c = c;
        }
        const float f = in ? rcp_fast(sum) : 0.0f;
        if (in) {
#pragma unroll
            for (int i = 0; i < 4 * V; ++i) sums.p[i] = fmaf(e[i], f, sums.p[i]);
            if (p.z) {
                const float l = log_of(z_sum, z_c);
                sums.z = fmaf(l, l, sums.z);
            }
        }
    }
    wait_copies<0>();
}

// A lane's sums to its token's first stage; afterwards (a barrier on)
// total_p(rings, e) is the block's sum of column e.
template <int LANES, int V>
__device__ __forceinline__ void leave(const TokenSums<V>& sums, const Ring<LANES, V, false>& ring, float* z_rows) {
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
#pragma unroll
    for (int v = 0; v < V; ++v)
        reinterpret_cast<float4*>(ring.at)[v * LANES + lane] =
            make_float4(sums.p[4 * v], sums.p[4 * v + 1], sums.p[4 * v + 2], sums.p[4 * v + 3]);
    if (lane == 0) z_rows[slot] = sums.z;
}
template <int LANES, int V>
__device__ __forceinline__ float total_p(const float* rings, int e) {
    float s = 0.0f;
#pragma unroll 8
    for (int i = 0; i < 32 / LANES * kWarps; ++i) s += rings[i * Ring<LANES, V, false>::kFloats + e];
    return s;
}

// Many tokens: a block takes tokens [blockIdx.x chunk, + chunk), sequence by
// sequence.  A sequence whose tokens are all here is finished here; one that
// began before leaves its sums in slot 0, one that goes on in slot 1.
template <int LANES, int V, int ROWS>
__global__ void __launch_bounds__(32 * kWarps) balance_kernel(const __grid_constant__ BalanceArgs p) {
    extern __shared__ __align__(16) float smem[];
    constexpr int kTokens = 32 / LANES * kWarps;  // at once
    using R = Ring<LANES, V, false>;
    const R ring{smem + threadIdx.x / LANES * R::kFloats};
    int* hist = reinterpret_cast<int*>(smem + kTokens * R::kFloats);  // [kCols]
    __shared__ float red[32], z_rows[kTokens];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tid = threadIdx.x, warp = tid >> 5;
    const int lo = blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.T);
    // the block's first tokens, before it is known which sequence they are in
    ring.clear(p.E, tid % LANES);
#pragma unroll
    for (int s = 0; s < R::kDepth; ++s) {
        const int t0 = lo + warp * (32 / LANES) + s * kTokens;
        if (t0 < hi)
            ring.template fetch<ROWS>(s, p.logits, p.ids, nullptr, min(t0 + (tid & 31) / LANES, hi - 1), p.E, p.k, tid % LANES);
        end_copies();
    }
    bool asked = true;
    int b = p.offsets ? max(last_not_above(p.offsets, p.n_seqs + 1, lo), 0) : 0;
    for (; b < p.n_seqs; ++b) {
        const int begin = seq_begin(p, b), end = seq_end(p, b);
        if (begin >= hi) break;
        const int from = max(begin, lo), to = min(end, hi);
        if (from >= to) continue;
        for (int e = tid; e < p.E; e += blockDim.x) hist[e] = 0;
        if (!asked || from != lo) {
            wait_copies<0>();
            ring.clear(p.E, tid % LANES);
            asked = false;
        }
        __syncthreads();
        TokenSums<V> sums{};
        add_tokens<LANES, V, ROWS>(p, ring, asked, from + warp * (32 / LANES), to, kTokens, hist, sums);
        asked = false;
        leave<LANES, V>(sums, ring, z_rows);
        __syncthreads();
        float z_all = 0.0f;
        if (tid == 0)
            for (int i = 0; i < kTokens; ++i) z_all += z_rows[i];
        auto sum_of = [&](int e) { return total_p<LANES, V>(smem, e); };
        if (begin >= lo && end <= hi) {
            finish_sequence(p, b, end - begin, z_all, sum_of, [&](int e) { return hist[e]; }, red);
        } else {
            const int64_t at = (int64_t)blockIdx.x * 2 + (begin < lo ? 0 : 1);
            for (int e = tid; e < p.E; e += blockDim.x) {
                p.part_p[at * p.E + e] = sum_of(e);
                p.part_counts[at * p.E + e] = hist[e];
            }
            if (tid == 0) p.part_z[at] = z_all;
            __syncthreads();
        }
    }
}

// Few tokens: a cluster of 8 blocks takes a sequence, adds its blocks' sums up
// through shared memory and finishes it, in one kernel.
constexpr int kFewBlocks = 8;
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();  // the barrier is the whole warp's; lanes took more or fewer columns
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t from_rank(const void* own, int rank) {
    uint32_t at = (uint32_t)__cvta_generic_to_shared(own), v;
    asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
// finish_sequence by a cluster whose blocks have their sums in total [E], hist
// [E] and *z each.
__device__ __forceinline__ void finish_cluster(const BalanceArgs& p, int b, int tokens, const float* total, const int* hist,
                                               const float* z, int rank, float* red) {
    cluster_sync();
    if (rank == 0) {
        float z_sum = 0.0f;
        if (threadIdx.x == 0 && p.z)
            for (int i = 0; i < kFewBlocks; ++i) z_sum += __uint_as_float(from_rank(z, i));
        finish_sequence(
            p, b, max(tokens, 0), z_sum,
            [&](int e) {
                float v[kFewBlocks], s = 0.0f;
#pragma unroll
                for (int i = 0; i < kFewBlocks; ++i) v[i] = __uint_as_float(from_rank(total + e, i));
#pragma unroll
                for (int i = 0; i < kFewBlocks; ++i) s += v[i];
                return s;
            },
            [&](int e) {
                int v[kFewBlocks], s = 0;
#pragma unroll
                for (int i = 0; i < kFewBlocks; ++i) v[i] = (int)from_rank(hist + e, i);
#pragma unroll
                for (int i = 0; i < kFewBlocks; ++i) s += v[i];
                return s;
            },
            red);
    }
    cluster_sync();  // the others' shared memory stays until it has been read
}
template <int LANES, int V, int ROWS>
__global__ void __cluster_dims__(kFewBlocks, 1, 1) __launch_bounds__(32 * kWarps)
    balance_few_kernel(const __grid_constant__ BalanceArgs p) {
    extern __shared__ __align__(16) float smem[];
    using R = Ring<LANES, V, false>;
    constexpr int kTokens = 32 / LANES * kWarps;
    const R ring{smem + threadIdx.x / LANES * R::kFloats};
    int* hist = reinterpret_cast<int*>(smem + kTokens * R::kFloats);
    float* total = smem + kTokens * R::kFloats + R::kCols;  // [kCols]
    __shared__ float red[32], z_rows[kTokens];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tid = threadIdx.x, warp = tid >> 5, b = blockIdx.x / kFewBlocks, rank = blockIdx.x % kFewBlocks;
    const int begin = seq_begin(p, b), end = seq_end(p, b);
    for (int e = tid; e < p.E; e += blockDim.x) hist[e] = 0;
    ring.clear(p.E, tid % LANES);
    __syncthreads();
    TokenSums<V> sums{};
    add_tokens<LANES, V, ROWS>(p, ring, false, begin + (rank * kWarps + warp) * (32 / LANES), end, kFewBlocks * kTokens, hist, sums);
    leave<LANES, V>(sums, ring, z_rows);
    __syncthreads();
    for (int e = tid; e < p.E; e += blockDim.x) total[e] = total_p<LANES, V>(smem, e);
    if (tid == 0) {
        float z = 0.0f;
        for (int i = 0; i < kTokens; ++i) z += z_rows[i];
        z_rows[0] = z;
    }
    finish_cluster(p, b, end - begin, total, hist, z_rows, rank, red);
}

// The sequences that no block finished alone: those of several blocks, and
// those without tokens.  A block each (CLUSTER: 8, where a sequence has many
// blocks' sums: an SM takes in 600 KB in 6 us); 4 threads a column at most.
template <bool CLUSTER>
__global__ void __launch_bounds__(1024, 1) balance_finish_kernel(const __grid_constant__ BalanceArgs p) {
    __shared__ float sums[4][DWDP_MAX_EXPERTS];
    __shared__ int counts[4][DWDP_MAX_EXPERTS];
    __shared__ float red[32], z_all;
    constexpr int kBlocks = CLUSTER ? kFewBlocks : 1;
    // (the kernel before let this one start when everything before it was done)
    const int b = blockIdx.x / kBlocks, rank = blockIdx.x % kBlocks;
    const int begin = seq_begin(p, b), end = seq_end(p, b);
    int first = 0, last = -1;
    if (begin < end) {
        first = begin / p.chunk;
        last = (end - 1) / p.chunk;
    }
    // (before any return: who comes next waits for this kernel only)
    wait_for_previous_kernel();
    let_next_kernel_start();
    if (first == last) return;  // finished already; the whole cluster
    const int parts = min(4, 1024 / p.E), part = threadIdx.x / p.E, e = threadIdx.x % p.E;
    if (part < parts) {
        float s = 0.0f;
        int n = 0;
        constexpr int kLoads = 6;  // of each on their way
        for (int i0 = first + rank * parts + part; i0 <= last; i0 += kLoads * kBlocks * parts) {
            float v[kLoads];
            int m[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int i = i0 + j * kBlocks * parts;
                const int64_t at = ((int64_t)i * 2 + (i == first ? 1 : 0)) * p.E + e;
                v[j] = i <= last ? p.part_p[at] : 0.0f;
                m[j] = i <= last ? p.part_counts[at] : 0;
            }
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                s += v[j];
                n += m[j];
            }
        }
        sums[part][e] = s;
        counts[part][e] = n;
    }
    if (p.z && threadIdx.x < 32) {
        float z = 0.0f, none = 0.0f;
        for (int i = first + rank * 32 + threadIdx.x; i <= last; i += 32 * kBlocks)
            z += p.part_z[(int64_t)i * 2 + (i == first ? 1 : 0)];
        warp_sum_max<false>(z, none);
        if (threadIdx.x == 0) z_all = z;
    }
    __syncthreads();
    auto own_p = [&](int c) {
        float s = 0.0f;
        for (int i = 0; i < parts; ++i) s += sums[i][c];
        return s;
    };
    auto own_count = [&](int c) {
        int n = 0;
        for (int i = 0; i < parts; ++i) n += counts[i][c];
        return n;
    };
    if constexpr (CLUSTER) {
        for (int c = threadIdx.x; c < p.E; c += blockDim.x) {
            const float s = own_p(c);
            const int n = own_count(c);
            sums[0][c] = s;
            counts[0][c] = n;
        }
        finish_cluster(p, b, end - begin, sums[0], counts[0], &z_all, rank, red);
    } else {
        finish_sequence(p, b, max(end - begin, 0), p.z ? z_all : 0.0f, own_p, own_count, red);
    }
}

// ------------------------------------------------------------ gradients --

__device__ __forceinline__ void store4(void* out, bool half, int64_t at, float a, float b, float c, float d) {
    if (half) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
        uint2 q;
        q.x = *reinterpret_cast<const uint32_t*>(&lo);
        q.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) = q;
    } else {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(a, b, c, d);
    }
}

// LANES lanes a token; a block takes tokens [blockIdx.x chunk, + chunk), its
// warps in turn.  The next token's logits, choices and weights are on their way
// while one is worked on.
template <int LANES, int V, int ROWS, bool SIGMOID>
__global__ void __launch_bounds__(32 * kGradWarps, V <= 2 ? 3 : 1) router_grad_kernel(const __grid_constant__ RouterGradArgs p) {
    using R = Ring<LANES, V, true>;
    constexpr int kTokens = 32 / LANES * kGradWarps, kCols = R::kCols, KPL = R::kPer;
    extern __shared__ __align__(16) float smem[];  // [kTokens][kCols]: what the choices add, zero between tokens; the rings
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tid = threadIdx.x, lane = tid % LANES, slot = tid / LANES;
    float* mine = smem + slot * kCols;
    const R ring{smem + kTokens * kCols + slot * R::kFloats};
    ring.clear(p.E, lane);
#pragma unroll
    for (int v = 0; v < V; ++v) reinterpret_cast<float4*>(mine)[v * LANES + lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
    const int lo = blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.T);
    const bool losses = p.dbalance || p.dz, direct = p.renorm || SIGMOID;
    auto fetch = [&](int64_t t0, int s) {
        if (t0 < hi)
            ring.template fetch<ROWS>(s, p.logits, p.dw ? p.ids : nullptr, p.dw, min((int)t0 + slot, hi - 1), p.E, p.k, lane);
        end_copies();
    };
#pragma unroll
    for (int s = 0; s < R::kDepth; ++s) fetch(lo + s * kTokens, s);
    int s = 0;
    // the sequence at hand, and where its tokens end; none yet
    int seq = losses && p.offsets ? last_not_above(p.offsets, p.n_seqs + 1, lo) : 0, to = 0;
    float by_p = 0.0f, by_z = 0.0f;
    float of_counts[V <= 2 ? 4 * V : 1] = {};  // d loss / d p of its balance loss, where registers allow
    const int32_t* counts = p.counts;
    for (int t0 = lo; t0 < hi; t0 += kTokens) {  // whole warps together
        const int t = min(t0 + slot, hi - 1);
        const bool in = t0 + slot < hi;
        float z[4 * V], e[4 * V], r[4 * V], g[4 * V], d[4 * V], dw[KPL], chosen_z[KPL];
        int id[KPL];
        wait_copies<R::kDepth - 1>();
        __syncwarp();  // the chosen logits are other lanes' copies
        ring.take(s, lane, z);
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
            const int i = lane + j * LANES;
            id[j] = -1;
            dw[j] = 0.0f;
            if (p.dw && i < p.k) {
                id[j] = ring.choice(s, i);
                if (id[j] < 0 || id[j] >= p.E) {
                    atomicOr(p.err, DERR_BAD_INDEX);
                    id[j] = -1;
                } else if (p.bias && __ldg(p.bias + id[j]) == -CUDART_INF_F) {
                    id[j] = -1;  // taken out: its weight is 0 whatever its logit
                } else {
                    dw[j] = ring.dw(s, i);
                }
            }
            chosen_z[j] = id[j] >= 0 ? ring.at[s * R::kStage + id[j]] : -CUDART_INF_F;
        }
        __syncwarp();  // everybody has read this stage
        fetch(t0 + (int64_t)R::kDepth * kTokens, s);
        s = s + 1 == R::kDepth ? 0 : s + 1;
        // what the choices have left in shared memory; then none of it is there
        auto gather = [&](float (&v)[4 * V]) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 q = reinterpret_cast<const float4*>(mine)[i * LANES + lane];
                v[4 * i] = q.x;
                v[4 * i + 1] = q.y;
                v[4 * i + 2] = q.z;
                v[4 * i + 3] = q.w;
            }
            __syncwarp();
        };
        auto clear = [&]() {
#pragma unroll
            for (int j = 0; j < KPL; ++j)
                if (id[j] >= 0) mine[id[j]] = 0.0f;
            __syncwarp();
        };
        if (losses && t >= to) {  // another sequence
            int from = 0;
            to = p.T;
            if (p.offsets) {
                while (seq < p.n_seqs && p.offsets[seq + 1] <= t) ++seq;
                from = seq >= 0 ? max(p.offsets[seq], 0) : 0;
                to = seq < p.n_seqs ? min(p.offsets[seq + 1], p.T) : p.T;
            }
            by_p = by_z = 0.0f;
            if (seq >= 0 && seq < p.n_seqs) {
                const float per_token = 1.0f / (float)(to - from);
                if (p.dbalance) by_p = p.dbalance[seq] * ((float)p.E / (float)p.k) * per_token * per_token;
                if (p.dz) by_z = 2.0f * p.dz[seq] * per_token;
                counts = p.counts + (int64_t)seq * p.E;
            }
            if constexpr (V <= 2) {
#pragma unroll
                for (int i = 0; i < 4 * V; ++i) {
                    const int c = 4 * (i / 4 * LANES + lane) + i % 4;
                    of_counts[i] = by_p != 0.0f && c < p.E ? by_p * (float)__ldg(counts + c) : 0.0f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) {
            if constexpr (V <= 2) {
                g[i] = of_counts[i];
            } else {
                const int c = 4 * (i / 4 * LANES + lane) + i % 4;
                g[i] = by_p != 0.0f && c < p.E ? by_p * (float)__ldg(counts + c) : 0.0f;
            }
        }
        // softmax over all: the weights' gradients go through the shares, with the losses' part
        if (p.dw && !direct) {
#pragma unroll
            for (int j = 0; j < KPL; ++j)
                if (id[j] >= 0) mine[id[j]] = p.scale * dw[j];
            gather(d);
#pragma unroll
            for (int i = 0; i < 4 * V; ++i) g[i] += d[i];
            clear();
        }
        // u = exp(-c) s and r = 1 - s (softmax: r = 1) of every expert, each times 16,
        // and of the chosen ones, as they are; and all sums at once: of u, u g, and
        // the chosen ones' u, u dw
        float c = 0.0f, chosen_c = 0.0f, chosen_u[KPL], chosen_r[KPL], chosen_one;
        float4 sums;
        auto terms = [&](bool far) {
            const float one = far && SIGMOID ? exp_fast(c) : 1.0f;
            chosen_one = far && SIGMOID ? exp_fast(chosen_c) : 1.0f;
            float a = 0.0f, b = 0.0f, chosen_a = 0.0f, chosen_b = 0.0f;
#pragma unroll
            for (int i = 0; i < 4 * V; ++i) {
                e[i] = far ? exp_fast(min_nan(z[i] - c, kTop)) : exp_fast(z[i]);
                if constexpr (SIGMOID) {
                    r[i] = sigmoid_rest(e[i], one);
                    e[i] *= r[i];
                }
                a += e[i];
                b = fmaf(e[i], g[i], b);
            }
#pragma unroll
            for (int j = 0; j < KPL; ++j) {
                chosen_u[j] = exp_fast(min_nan(chosen_z[j] - chosen_c, kTop));
                if constexpr (SIGMOID) {
                    chosen_r[j] = rcp_fast(fmaf(chosen_u[j], chosen_one, 1.0f));
                    chosen_u[j] *= chosen_r[j];
                }
                chosen_a += chosen_u[j];
                chosen_b = fmaf(chosen_u[j], dw[j], chosen_b);
            }
            sums = token_sums<LANES>(a, b, chosen_a, chosen_b);
        };
        terms(false);
        {
            const bool lost = !(sums.x >= (SIGMOID ? kSigmoidUnit : 1.0f) * kLeast && sums.x <= kMost);  // a sigmoid's u is inf 0 of a large logit
            const bool chosen_lost = p.dw && p.renorm && !(sums.z >= kLeast && sums.z <= kMost);
            if (__any_sync(0xffffffffu, lost || chosen_lost)) {
                float m = -CUDART_INF_F, chosen_m = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < 4 * V; ++i) m = max_nan(m, z[i]);
#pragma unroll
                for (int j = 0; j < KPL; ++j) chosen_m = max_nan(chosen_m, chosen_z[j]);
                m = token_max<LANES>(m);
                chosen_m = token_max<LANES>(chosen_m);
                if (lost) c = SIGMOID ? min_nan(m, 0.0f) : m;
                if (chosen_lost) chosen_c = SIGMOID ? min_nan(chosen_m, 0.0f) : chosen_m;
                terms(true);
            }
        }
        const float one_sum = rcp_fast(sums.x);
        if (p.dw && direct) {
            const float by = p.renorm ? p.scale * rcp_fast(sums.z) : p.scale * chosen_one;
            const float mean = p.renorm ? sums.w * rcp_fast(sums.z) : 0.0f;
#pragma unroll
            for (int j = 0; j < KPL; ++j)
                if (id[j] >= 0) mine[id[j]] = by * chosen_u[j] * (dw[j] - mean) * (SIGMOID ? chosen_r[j] : 1.0f);
            gather(d);
            clear();
        } else {
#pragma unroll
            for (int i = 0; i < 4 * V; ++i) d[i] = 0.0f;
        }
        if (p.dbalance || !direct) {
            // (shares first: one_sum twice could pass binary32's range)
            const float mean = sums.y * one_sum, by_sum = SIGMOID ? one_sum * (1.0f / kSigmoidUnit) : one_sum;
#pragma unroll
            for (int i = 0; i < 4 * V; ++i) {
                const float p_i = SIGMOID ? e[i] * r[i] : e[i];
                d[i] = fmaf(p_i * by_sum, g[i] - mean, d[i]);
            }
        }
        if (p.dz) {
            float z_c;
            const float z_sum = soft_terms<LANES, V>(z, e, z_c), by = by_z * log_of(z_sum, z_c) * rcp_fast(z_sum);
#pragma unroll
            for (int i = 0; i < 4 * V; ++i) d[i] = fmaf(by, e[i], d[i]);
        }
        if (in) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = 4 * (v * LANES + lane);
                const int64_t at = (int64_t)t * p.E + col;
                if constexpr (ROWS != ROWS_ANY) {
                    if (ROWS == ROWS_FULL || col < p.E)
                        store4(p.dlogits, p.half, at, d[4 * v], d[4 * v + 1], d[4 * v + 2], d[4 * v + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (col + i >= p.E) continue;
                        if (p.half)
                            static_cast<__nv_bfloat16*>(p.dlogits)[at + i] = __float2bfloat16_rn(d[4 * v + i]);
                        else
                            static_cast<float*>(p.dlogits)[at + i] = d[4 * v + i];
                    }
                }
            }
        }
    }
}

// kTokens, kGradTokens: of a block at once, the losses' and the gradients' kernel.
template <int L, int N, int W>
struct Form {
    static constexpr int LANES = L, V = N, kCols = 4 * V * LANES, kTokens = 32 / LANES * kWarps,
                         kGradTokens = 32 / LANES * kGradWarps;
    static constexpr int ROWS = W;
};

template <int L, int V, class F>
cudaError_t by_rows(int E, F f) {
    return E == 4 * V * L ? f(Form<L, V, ROWS_FULL>()) : E % 4 == 0 ? f(Form<L, V, ROWS_VEC>()) : f(Form<L, V, ROWS_ANY>());
}
// f(Form) for E experts.
template <class F>
cudaError_t by_experts(int E, F f) {
    if (E <= 16) return by_rows<4, 1>(E, f);
    if (E <= 32) return by_rows<8, 1>(E, f);
    if (E <= 64) return by_rows<16, 1>(E, f);
    if (E <= 128) return by_rows<32, 1>(E, f);
    if (E <= 256) return by_rows<32, 2>(E, f);
    if (E <= 512) return by_rows<32, 4>(E, f);
    return by_rows<32, 8>(E, f);
}

// Few tokens: one kernel of a cluster a sequence.  us for 256 experts, sigmoid, z
// loss, one kernel / two: 256 tokens in 1 sequence 4.4 / 6.6, 768 in 1 6.5 / 8.1, 1024
// in 1 7.6 / 6.7, 2048 in 1 12.2 / 7.6, in 4 5.7 / 7.0, 8192 in 16 7.4 / 8.8, 16384 in
// 64 11.0 / 10.5.
bool balance_is_few(int64_t T, int n_seqs) { return T <= 8192 && T <= 768 * (int64_t)n_seqs && n_seqs <= 4096; }
// Tokens of a block of the losses' kernel: two blocks an SM of a GB300's 152,
// whole rounds of a block's warps.
int balance_chunk(int64_t T, int E) {
    int at_once = 0;
    by_experts(E, [&](auto form) {
        at_once = decltype(form)::kTokens;
        return cudaSuccess;
    });
    const int64_t want = (T + 152 * 2 - 1) / (152 * 2);
    return (int)std::max<int64_t>(at_once, (want + at_once - 1) / at_once * at_once);
}

struct BalanceLayout {
    int64_t blocks, p, counts, z, bytes;
};
BalanceLayout balance_layout(int64_t T, int E) {
    BalanceLayout L;
    const int64_t chunk = balance_chunk(T, E);
    L.blocks = std::max<int64_t>(1, (T + chunk - 1) / chunk);
    L.p = 0;
    L.counts = L.blocks * 2 * E * 4;
    L.z = L.counts * 2;
    L.bytes = L.z + L.blocks * 2 * 4;
    return L;
}

}  // namespace

size_t balance_bytes(int64_t T, int E) { return (size_t)balance_layout(T, E).bytes; }

cudaError_t launch_balance(BalanceArgs& p, void* ws, cudaStream_t s) {
    const BalanceLayout L = balance_layout(p.T, p.E);
    p.chunk = balance_chunk(p.T, p.E);
    char* base = static_cast<char*>(ws);
    p.part_p = reinterpret_cast<float*>(base + L.p);
    p.part_counts = reinterpret_cast<int32_t*>(base + L.counts);
    p.part_z = reinterpret_cast<float*>(base + L.z);
    if (balance_is_few(p.T, p.n_seqs))
        return by_experts(p.E, [&](auto form) {
            using F = decltype(form);
            const auto kernel = balance_few_kernel<F::LANES, F::V, F::ROWS>;
            const size_t smem = (F::kTokens * Ring<F::LANES, F::V, false>::kFloats + 2 * F::kCols) * sizeof(float);
            cudaError_t e = smem > (48 << 10) ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                                              : cudaSuccess;
            return e != cudaSuccess ? e : launch_dependent(kernel, p, dim3((unsigned)p.n_seqs * kFewBlocks), 32 * kWarps, smem, s);
        });
    const cudaError_t e = by_experts(p.E, [&](auto form) {
        using F = decltype(form);
        const auto kernel = balance_kernel<F::LANES, F::V, F::ROWS>;
        const size_t smem = (F::kTokens * Ring<F::LANES, F::V, false>::kFloats + F::kCols) * sizeof(float);
        cudaError_t e = smem > (48 << 10) ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                                          : cudaSuccess;
        return e != cudaSuccess ? e : launch_dependent(kernel, p, dim3((unsigned)L.blocks), 32 * kWarps, smem, s);
    });
    if (e != cudaSuccess) return e;
    if (L.blocks / p.n_seqs >= 64)
        return launch_dependent(balance_finish_kernel<true>, p, dim3((unsigned)p.n_seqs * kFewBlocks), 1024, 0, s, kFewBlocks);
    return launch_dependent(balance_finish_kernel<false>, p, dim3((unsigned)p.n_seqs), 1024, 0, s);
}

cudaError_t launch_router_grad(RouterGradArgs& p, cudaStream_t s) {
    if (p.T <= 0) return cudaSuccess;
    return by_experts(p.E, [&](auto form) {
        using F = decltype(form);
        // three blocks an SM, whole rounds of their warps
        const int64_t want = (p.T + 152 * 3 - 1) / (152 * 3);
        p.chunk = (int)std::max<int64_t>(F::kGradTokens, (want + F::kGradTokens - 1) / F::kGradTokens * F::kGradTokens);
        const dim3 grid((unsigned)((p.T + p.chunk - 1) / p.chunk));
        const size_t smem = F::kGradTokens * (F::kCols + Ring<F::LANES, F::V, true>::kFloats) * sizeof(float);
        const auto kernel = p.sigmoid ? router_grad_kernel<F::LANES, F::V, F::ROWS, true> : router_grad_kernel<F::LANES, F::V, F::ROWS, false>;
        const cudaError_t e = smem > (48 << 10)
                                  ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                                  : cudaSuccess;
        return e != cudaSuccess ? e : launch_dependent(kernel, p, grid, 32 * kGradWarps, smem, s);
    });
}

}  // namespace dwdp
