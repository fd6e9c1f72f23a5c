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
// largest logit.  For the sigmoid with c = min(that, 0):
//   a = exp(c - z),  u = 1 / (a + exp(c)) = exp(-c) s,  p = u / sum u,
//   1 - s = a u
// so neither small scores nor scores next to 1 lose their digits.
#include <math_constants.h>

#include <algorithm>

#include "dwdp_internal.h"
#include "row_ops.h"

namespace dwdp {
namespace {

constexpr int kWarps = 8;  // of a block
constexpr float kLeast = 1e-20f, kMost = 1e35f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// exp by the approximate power of two: its argument's rounding makes the
// relative error |x| 2^-23 or 2^-22, whichever is more.
__device__ __forceinline__ float exp_fast(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x * kLog2e));
    return r;
}

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

// A lane's logits of one token: columns 4 (v LANES + lane) .. + 3, -inf beyond E.
// VEC: E is a multiple of 4, so rows are 16-byte aligned.
template <int LANES, int V, bool VEC>
__device__ __forceinline__ void load_token(const float* row, int E, int lane, float (&z)[4 * V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = 4 * (v * LANES + lane);
        if constexpr (VEC) {
            const float4 q = c < E ? __ldg(reinterpret_cast<const float4*>(row + c))
                                   : make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
            z[4 * v] = q.x;
            z[4 * v + 1] = q.y;
            z[4 * v + 2] = q.z;
            z[4 * v + 3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[4 * v + i] = c + i < E ? __ldg(row + c + i) : -CUDART_INF_F;
        }
    }
}

template <int LANES, int V>
__device__ __forceinline__ bool column(int v, int i, int lane, int E) {
    return 4 * (v * LANES + lane) + i < E;
}

// A token's exp(z - c) and their sum.
template <int LANES, int V>
__device__ __forceinline__ float soft_terms(const float (&z)[4 * V], float (&e)[4 * V], float& c) {
    c = 0.0f;
    float sum = 0.0f;
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
        float again = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) {
            e[i] = exp_fast(z[i] - c);
            again += e[i];
        }
        sum = token_sum<LANES>(again);
    }
    return sum;
}

// A token's u and their sum (a u = 1 - s).  Columns beyond E get u = 0.
template <int LANES, int V>
__device__ __forceinline__ float sigmoid_terms(const float (&z)[4 * V], int lane, int E, float (&a)[4 * V],
                                               float (&u)[4 * V], float& c) {
    c = 0.0f;
    float sum = 0.0f, one = 1.0f;
    auto terms = [&]() {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) {
            a[i] = exp_fast(min_nan(c - z[i], 87.0f));
            u[i] = column<LANES, V>(i / 4, i % 4, lane, E) ? rcp(a[i] + one) : 0.0f;
            sum += u[i];
        }
        sum = token_sum<LANES>(sum);
    };
    terms();
    const bool lost = !(sum >= kLeast);
    if (__any_sync(0xffffffffu, lost)) {
        float m = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) m = max_nan(m, z[i]);
        m = token_max<LANES>(m);
        if (lost) c = min_nan(m, 0.0f);
        one = exp_fast(c);
        terms();
    }
    return sum;
}

__device__ __forceinline__ float log_of(float sum, float c) { return c + __log2f(sum) * kLn2; }

// The last sequence whose tokens start at t or before; -1 or n_seqs - 1 and
// beyond it where t is in none.  One thread.
__device__ __forceinline__ int seq_of(const int32_t* offsets, int n_seqs, int t) {
    int lo = 0, hi = n_seqs + 1;  // offsets[lo - 1] <= t < offsets[hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= t)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo - 1 < n_seqs ? lo - 1 : -1;
}

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

// A block takes tokens [blockIdx.x chunk, + chunk), sequence by sequence.  A
// sequence whose tokens are all here is finished here; one that began before
// leaves its sums in slot 0, one that goes on in slot 1.
template <int LANES, int V, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) balance_kernel(const __grid_constant__ BalanceArgs p) {
    extern __shared__ float smem[];
    constexpr int kTokens = 32 / LANES * kWarps;  // at once
    constexpr int kCols = 4 * V * LANES;
    float* sums = smem;                                     // [kTokens][kCols]
    int* hist = reinterpret_cast<int*>(smem + kTokens * kCols);  // [kCols]
    __shared__ float red[32], z_red[kTokens];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tid = threadIdx.x, lane = tid % LANES, slot = tid / LANES;
    const int lo = blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.T);
    int b = p.offsets ? seq_of(p.offsets, p.n_seqs, lo) : 0;
    if (b < 0) b = p.offsets[0] > lo ? 0 : p.n_seqs;
    for (; b < p.n_seqs; ++b) {
        const int begin = seq_begin(p, b), end = seq_end(p, b);
        if (begin >= hi) break;
        const int from = max(begin, lo), to = min(end, hi);
        if (from >= to) continue;
        for (int e = tid; e < p.E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
        for (int64_t i = (int64_t)from * p.k + tid; i < (int64_t)to * p.k; i += blockDim.x) {
            const int id = p.ids[i];
            if (id >= 0 && id < p.E)
                atomicAdd(hist + id, 1);
            else
                atomicOr(p.err, DERR_BAD_INDEX);
        }
        float sum_p[4 * V] = {}, z_sum = 0.0f;
        for (int t0 = from; t0 < to; t0 += kTokens) {  // whole warps together
            const int t = t0 + slot;
            const bool in = t < to;
            float z[4 * V], e[4 * V], c;
            load_token<LANES, V, VEC>(p.logits + (int64_t)(in ? t : to - 1) * p.E, p.E, lane, z);
            float sum;
            if (p.sigmoid) {
                float u[4 * V];
                sum = sigmoid_terms<LANES, V>(z, lane, p.E, e, u, c);
                const float f = in ? 1.0f / sum : 0.0f;
                if (in) {
#pragma unroll
                    for (int i = 0; i < 4 * V; ++i) sum_p[i] = fmaf(u[i], f, sum_p[i]);
                }
                if (p.z) sum = soft_terms<LANES, V>(z, e, c);
            } else {
                sum = soft_terms<LANES, V>(z, e, c);
                const float f = 1.0f / sum;
                if (in) {
#pragma unroll
                    for (int i = 0; i < 4 * V; ++i) sum_p[i] = fmaf(e[i], f, sum_p[i]);
                }
            }
            if (p.z && in) {
                const float l = log_of(sum, c);
                z_sum = fmaf(l, l, z_sum);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            reinterpret_cast<float4*>(sums + slot * kCols)[v * LANES + lane] =
                make_float4(sum_p[4 * v], sum_p[4 * v + 1], sum_p[4 * v + 2], sum_p[4 * v + 3]);
        if (lane == 0) z_red[slot] = z_sum;
        __syncthreads();
        auto sum_of = [&](int e) {
            float s = 0.0f;
            for (int i = 0; i < kTokens; ++i) s += sums[i * kCols + e];
            return s;
        };
        float z_all = 0.0f;
        if (tid == 0)
            for (int i = 0; i < kTokens; ++i) z_all += z_red[i];
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

// The sequences that no block finished alone: those of several blocks, and
// those without tokens.  A block each; 4 threads a column at most.
__global__ void __launch_bounds__(1024) balance_finish_kernel(const __grid_constant__ BalanceArgs p) {
    __shared__ float sums[4][DWDP_MAX_EXPERTS];
    __shared__ int counts[4][DWDP_MAX_EXPERTS];
    __shared__ float red[32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int b = blockIdx.x;
    const int begin = seq_begin(p, b), end = seq_end(p, b);
    int first = 0, last = -1;
    if (begin < end) {
        first = begin / p.chunk;
        last = (end - 1) / p.chunk;
        if (first == last) return;
    }
    const int parts = min(4, 1024 / p.E), part = threadIdx.x / p.E, e = threadIdx.x % p.E;
    if (part < parts) {
        float s = 0.0f;
        int n = 0;
        for (int i = first + part; i <= last; i += parts) {
            const int64_t at = ((int64_t)i * 2 + (i == first ? 1 : 0)) * p.E + e;
            s += p.part_p[at];
            n += p.part_counts[at];
        }
        sums[part][e] = s;
        counts[part][e] = n;
    }
    float z = 0.0f;
    if (p.z && threadIdx.x < 32) {
        float none = 0.0f;
        for (int i = first + threadIdx.x; i <= last; i += 32) z += p.part_z[(int64_t)i * 2 + (i == first ? 1 : 0)];
        warp_sum_max<false>(z, none);
    }
    __syncthreads();
    finish_sequence(
        p, b, max(end - begin, 0), z,
        [&](int c) {
            float s = 0.0f;
            for (int i = 0; i < parts; ++i) s += sums[i][c];
            return s;
        },
        [&](int c) {
            int n = 0;
            for (int i = 0; i < parts; ++i) n += counts[i][c];
            return n;
        },
        red);
}

// ------------------------------------------------------------ gradients --

template <bool HALF>
__device__ __forceinline__ void store4(void* out, int64_t at, float a, float b, float c, float d) {
    if constexpr (HALF) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
        uint2 q;
        q.x = *reinterpret_cast<const uint32_t*>(&lo);
        q.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) = q;
    } else {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(a, b, c, d);
    }
}

// The gradients of a token's chosen logits from those of its weights: lane
// holds choices lane, lane + LANES, ... (KPL of them).  direct: added to the
// chosen logits; through: d loss / d s of the chosen, to go through all
// shares (softmax over all, not renormalized).
template <int LANES, int KPL>
__device__ __forceinline__ void choice_terms(const RouterGradArgs& p, const float* row, const int (&id)[KPL],
                                             const float (&dw)[KPL], float c, float (&direct)[KPL]) {
    float e[KPL], a[KPL];
    float sum = 0.0f, m = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < KPL; ++j) {
        const float z = id[j] >= 0 ? __ldg(row + id[j]) : -CUDART_INF_F;
        e[j] = z;
        m = max_nan(m, z);
    }
    if (p.renorm) m = token_max<LANES>(m);
    const float shift = !p.renorm ? c : p.sigmoid ? min_nan(m, 0.0f) : m, one = exp_fast(shift);
#pragma unroll
    for (int j = 0; j < KPL; ++j) {
        if (p.sigmoid) {
            a[j] = exp_fast(min_nan(shift - e[j], 87.0f));
            e[j] = id[j] >= 0 ? rcp(a[j] + one) : 0.0f;  // exp(-shift) s
            a[j] *= e[j];                                // 1 - s
        } else {
            e[j] = id[j] >= 0 ? exp_fast(e[j] - shift) : 0.0f;
            a[j] = 1.0f;
        }
        sum += e[j];
    }
    if (p.renorm) {
        sum = 1.0f / token_sum<LANES>(sum);
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
            e[j] *= sum;
            dot = fmaf(e[j], dw[j], dot);
        }
        dot = token_sum<LANES>(dot);
#pragma unroll
        for (int j = 0; j < KPL; ++j) direct[j] = p.scale * a[j] * e[j] * (dw[j] - dot);
    } else {
        // sigmoid, each on its own
#pragma unroll
        for (int j = 0; j < KPL; ++j) direct[j] = p.scale * a[j] * e[j] * one * dw[j];
    }
}

// LANES lanes a token; a block takes tokens [blockIdx.x chunk, + chunk), its
// warps in turn.
template <int LANES, int V, bool VEC, bool HALF>
__global__ void __launch_bounds__(32 * kWarps) router_grad_kernel(const __grid_constant__ RouterGradArgs p) {
    constexpr int kTokens = 32 / LANES * kWarps, kCols = 4 * V * LANES;
    constexpr int KPL = LANES >= 32 ? 1 : LANES == 16 ? 2 : 4;
    extern __shared__ float smem[];  // [kTokens][kCols]: what the choices add, zero between tokens
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tid = threadIdx.x, lane = tid % LANES, slot = tid / LANES;
    float* mine = smem + slot * kCols;
#pragma unroll
    for (int v = 0; v < V; ++v) reinterpret_cast<float4*>(mine)[v * LANES + lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
    const int lo = blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.T);
    for (int t0 = lo; t0 < hi; t0 += kTokens) {  // whole warps together
        const int t = min(t0 + slot, hi - 1);
        const bool in = t0 + slot < hi;
        const float* row = p.logits + (int64_t)t * p.E;
        float z[4 * V], e[4 * V], a[4 * V], g[4 * V] = {};
        load_token<LANES, V, VEC>(row, p.E, lane, z);
        int b = -1, tokens = 0;
        if (p.dbalance || p.dz) {
            b = p.offsets ? seq_of(p.offsets, p.n_seqs, t) : 0;
            if (b >= 0) tokens = p.offsets ? min(p.offsets[b + 1], p.T) - max(p.offsets[b], 0) : p.T;
        }
        const float per_token = b >= 0 ? 1.0f / (float)tokens : 0.0f;
        // d loss / d p: the balance losses' part
        float by_p = 0.0f;
        if (p.dbalance && b >= 0) {
            by_p = p.dbalance[b] * ((float)p.E / (float)p.k) * per_token * per_token;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = 4 * (v * LANES + lane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < p.E) g[4 * v + i] = by_p * (float)__ldg(p.counts + (int64_t)b * p.E + c + i);
            }
        }
        float c = 0.0f, sum;
        if (p.sigmoid) {
            sum = sigmoid_terms<LANES, V>(z, lane, p.E, a, e, c);
        } else {
            sum = soft_terms<LANES, V>(z, e, c);
        }
        const float one_sum = 1.0f / sum;
        // the chosen experts' weights
        int id[KPL];
        float dw[KPL];
        bool direct_terms = false;
        if (p.dw) {
#pragma unroll
            for (int j = 0; j < KPL; ++j) {
                const int i = lane + j * LANES;
                id[j] = i < p.k ? p.ids[(int64_t)t * p.k + i] : -1;
                dw[j] = i < p.k ? p.dw[(int64_t)t * p.k + i] : 0.0f;
                if (i < p.k && (id[j] < 0 || id[j] >= p.E)) {
                    atomicOr(p.err, DERR_BAD_INDEX);
                    id[j] = -1;
                }
                if (id[j] < 0) dw[j] = 0.0f;
            }
            direct_terms = p.renorm || p.sigmoid;
            float add[KPL];
            if (direct_terms) {
                choice_terms<LANES, KPL>(p, row, id, dw, c, add);
            } else {
#pragma unroll
                for (int j = 0; j < KPL; ++j) add[j] = p.scale * dw[j];
            }
#pragma unroll
            for (int j = 0; j < KPL; ++j)
                if (id[j] >= 0) mine[id[j]] = add[j];
            __syncwarp();
        }
        float chosen[4 * V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float4 q = reinterpret_cast<const float4*>(mine)[v * LANES + lane];
            chosen[4 * v] = q.x;
            chosen[4 * v + 1] = q.y;
            chosen[4 * v + 2] = q.z;
            chosen[4 * v + 3] = q.w;
        }
        if (p.dw) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < KPL; ++j)
                if (id[j] >= 0) mine[id[j]] = 0.0f;
        }
        // softmax over all: the weights' gradients go through the shares too
        if (!direct_terms) {
#pragma unroll
            for (int i = 0; i < 4 * V; ++i) {
                g[i] += chosen[i];
                chosen[i] = 0.0f;
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) {
            e[i] *= one_sum;
            dot = fmaf(e[i], g[i], dot);
        }
        dot = token_sum<LANES>(dot);
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) {
            float d = e[i] * (g[i] - dot);
            if (p.sigmoid) d *= a[i] * (e[i] * sum);  // 1 - s
            chosen[i] += d;
        }
        if (p.dz) {
            if (p.sigmoid) {
                sum = soft_terms<LANES, V>(z, e, c);
#pragma unroll
                for (int i = 0; i < 4 * V; ++i) e[i] *= 1.0f / sum;
            }
            if (b >= 0) {
                const float by = 2.0f * p.dz[b] * per_token * log_of(sum, c);
#pragma unroll
                for (int i = 0; i < 4 * V; ++i) chosen[i] = fmaf(by, e[i], chosen[i]);
            }
        }
        if (in) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = 4 * (v * LANES + lane);
                const int64_t at = (int64_t)t * p.E + col;
                if constexpr (VEC) {
                    if (col < p.E)
                        store4<HALF>(p.dlogits, at, chosen[4 * v], chosen[4 * v + 1], chosen[4 * v + 2], chosen[4 * v + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (col + i >= p.E) continue;
                        if constexpr (HALF)
                            static_cast<__nv_bfloat16*>(p.dlogits)[at + i] = __float2bfloat16_rn(chosen[4 * v + i]);
                        else
                            static_cast<float*>(p.dlogits)[at + i] = chosen[4 * v + i];
                    }
                }
            }
        }
    }
}

template <int L, int N, bool W>
struct Form {
    static constexpr int LANES = L, V = N, kCols = 4 * V * LANES, kTokens = 32 / LANES * kWarps;
    static constexpr bool VEC = W;
};

// f(Form) for E experts.
template <class F>
cudaError_t by_experts(int E, F f) {
    const bool vec = E % 4 == 0;
    if (E <= 16) return vec ? f(Form<4, 1, true>()) : f(Form<4, 1, false>());
    if (E <= 32) return vec ? f(Form<8, 1, true>()) : f(Form<8, 1, false>());
    if (E <= 64) return vec ? f(Form<16, 1, true>()) : f(Form<16, 1, false>());
    if (E <= 128) return vec ? f(Form<32, 1, true>()) : f(Form<32, 1, false>());
    if (E <= 256) return vec ? f(Form<32, 2, true>()) : f(Form<32, 2, false>());
    if (E <= 512) return vec ? f(Form<32, 4, true>()) : f(Form<32, 4, false>());
    return vec ? f(Form<32, 8, true>()) : f(Form<32, 8, false>());
}

// Tokens of a block of the losses' kernel: few enough to give every SM of a
// GB300 (152) a block, whole rounds of the block's warps, 16 rounds at most.
int balance_chunk(int64_t T, int E) {
    const int at_once = kWarps * std::max(1, 32 / std::max(4, (E + 3) / 4));
    const int64_t want = (T + 152 * 4 - 1) / (152 * 4);
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
    if (p.T > 0) {
        const cudaError_t e = by_experts(p.E, [&](auto form) {
            using F = decltype(form);
            return launch_dependent(balance_kernel<F::LANES, F::V, F::VEC>, p, dim3((unsigned)L.blocks), 32 * kWarps,
                                    (F::kTokens + 1) * F::kCols * sizeof(float), s);
        });
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(balance_finish_kernel, p, dim3((unsigned)p.n_seqs), 1024, 0, s);
}

cudaError_t launch_router_grad(RouterGradArgs& p, cudaStream_t s) {
    if (p.T <= 0) return cudaSuccess;
    return by_experts(p.E, [&](auto form) {
        using F = decltype(form);
        const int64_t want = (p.T + 152 * 8 - 1) / (152 * 8);
        p.chunk = (int)std::max<int64_t>(F::kTokens, (want + F::kTokens - 1) / F::kTokens * F::kTokens);
        const dim3 grid((unsigned)((p.T + p.chunk - 1) / p.chunk));
        const size_t smem = F::kTokens * F::kCols * sizeof(float);
        if (p.half)
            return launch_dependent(router_grad_kernel<F::LANES, F::V, F::VEC, true>, p, grid, 32 * kWarps, smem, s);
        return launch_dependent(router_grad_kernel<F::LANES, F::V, F::VEC, false>, p, grid, 32 * kWarps, smem, s);
    });
}

}  // namespace dwdp
