// route_scored.cu: the choice of dwdp_route_scored from the router's logits:
// scores, choice values, groups of experts, top-k and weights, one warp per
// token.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "dwdp_internal.h"

namespace dwdp {
namespace {

constexpr int kNoExpert = 0x7fffffff;
constexpr unsigned kFull = 0xffffffffu;

// Order-preserving keys: a > b iff key(a) > key(b); -0 folds into +0, every
// NaN is above +inf, and no value has key 0, which marks "not a candidate".
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint64_t kSign64 = 0x8000000000000000ull;
__device__ __forceinline__ uint64_t order_key(double x) {
    if (x != x) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(x == 0.0 ? 0.0 : x);
    return (u & kSign64) ? ~u : (u | kSign64);
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __longlong_as_double((long long)((k & kSign64) ? (k & ~kSign64) : ~k));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kFull, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <class V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Which experts a lane holds.  A group of gs experts is shared by L lanes (a
// power of two), each with PL consecutive ones, so lane order is expert
// order, a lane's experts are one run in memory and a group's best two are
// merged over log2 L shuffles.  Lane l: group g = l / L (none if g >= G).
struct Lane {
    int g, first, n;  // group, first expert, experts held
    __device__ Lane(const ScoredArgs& p, int lane) {
        g = lane / p.lanes;
        const int at = (lane % p.lanes) * p.per_lane;
        n = g < p.n_groups ? max(0, min(p.per_lane, p.group_size - at)) : 0;
        first = g * p.group_size + at;
    }
};

// z[j] = the token's logit of expert first + j: the partial-sum planes of a
// K-split router GEMM added in plane order.  Whole runs in 16-byte loads.
template <int P>
__device__ __forceinline__ void load_logits(const ScoredArgs& p, int64_t t, const Lane& ln, float (&z)[P]) {
    const float* src = p.logits + t * p.E + ln.first;
    if (P >= 4 && p.vector_loads) {
#pragma unroll
        for (int j = 0; j < P; j += 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < ln.n) {
                v = *reinterpret_cast<const float4*>(src + j);
                for (int q = 1; q < p.parts; ++q) {
                    const float4 u = *reinterpret_cast<const float4*>(src + q * p.part_stride + j);
                    v.x += u.x;
                    v.y += u.y;
                    v.z += u.z;
                    v.w += u.w;
                }
            }
            z[j] = v.x;
            if (P >= 4) {
                z[(j + 1) % P] = v.y;
                z[(j + 2) % P] = v.z;
                z[(j + 3) % P] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            z[j] = 0.0f;
            if (j < ln.n) {
                z[j] = src[j];
                for (int q = 1; q < p.parts; ++q) z[j] += src[q * p.part_stride + j];
            }
        }
    }
}

__device__ __forceinline__ float logit_of(const ScoredArgs& p, int64_t t, int e) {
    float v = p.logits[t * p.E + e];
    for (int q = 1; q < p.parts; ++q) v += p.logits[q * p.part_stride + t * p.E + e];
    return v;
}

// The choice among the keys of the choice values (0: no expert).  Lane s < k
// ends up with the s-th pick's id.  `close` is set when a decision lies within
// the tolerance: between the last kept and the first dropped group, or
// between the k-th pick and the best one left.  rel and ref describe the
// error of a choice value v: at most (rel * (ref or |v|) + 2^-22 |v|) / 2.
template <class K, int P>
__device__ __forceinline__ int choose(const ScoredArgs& p, K (&key)[P], const Lane& ln, int lane, float rel,
                                      float ref, bool& close) {
    close = false;
    // a difference of infinities is NaN and never close: ties go by id
    auto near = [&](K a, K b, float times) {
        const float va = (float)key_value(a), d = (float)(key_value(a) - key_value(b));
        return d <= times * (rel * (ref > 0.0f ? ref : fabsf(va)) + 0x1p-22f * fabsf(va));
    };
    if (p.top_groups < p.n_groups) {
        K k1 = 0, k2 = 0;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const K c = key[j];
            k2 = max(k2, min(k1, c));
            k1 = max(k1, c);
        }
        for (int o = 1; o < p.lanes; o <<= 1) {
            const K o1 = __shfl_xor_sync(kFull, k1, o), o2 = __shfl_xor_sync(kFull, k2, o);
            k2 = max(min(k1, o1), max(k2, o2));
            k1 = max(k1, o1);
        }
        K gk = k1;
        if (p.group_top2 && k2 != 0) gk = order_key(key_value(k1) + key_value(k2));
        const bool is_group = ln.g < p.n_groups;
        if (!is_group) gk = 0;
        int rank = 0;
        for (int g = 0; g < p.n_groups; ++g) {
            const K other = __shfl_sync(kFull, gk, g * p.lanes);
            rank += (other > gk) || (other == gk && g < ln.g);
        }
        const bool kept = is_group && rank < p.top_groups;
        const K worst_kept = ~warp_max(kept ? (K)~gk : (K)0);
        const K best_dropped = warp_max((is_group && !kept) ? gk : (K)0);
        close = near(worst_kept, best_dropped, 2.0f);
        if (!kept) {
#pragma unroll
            for (int j = 0; j < P; ++j) key[j] = 0;
        }
    }
    K lk;
    int li;
    auto best = [&] {  // this lane's best remaining, the lowest id on ties
        lk = 0;
        li = kNoExpert;
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (key[j] > lk) {
                lk = key[j];
                li = ln.first + j;
            }
    };
    best();
    int my_id = -1;
    K last = 0;
    for (int s = 0; s < p.k; ++s) {
        const K gk = warp_max(lk);
        if (gk == 0) break;  // fewer than k candidates (refused on the host)
        const int gi = __reduce_min_sync(kFull, lk == gk ? li : kNoExpert);
        last = gk;
        if (lane == s) my_id = gi;
        if (lk == gk && li == gi) {
#pragma unroll
            for (int j = 0; j < P; ++j)  // (a constant index keeps key[] in registers)
                if (ln.first + j == gi) key[j] = 0;
            best();
        }
    }
    const K next = warp_max(lk);
    if (next != 0) close = close || near(last, next, 1.0f);
    return my_id;
}

// The same decision from the same logits in binary64: for the few tokens
// whose choice binary32 cannot tell apart.
template <int P>
__device__ __noinline__ int choose_in_64(const ScoredArgs& p, int64_t t, int lane) {
    const Lane ln(p, lane);
    float z[P];
    load_logits<P>(p, t, ln, z);
    float zm = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < P; ++j)
        if (j < ln.n) zm = fmaxf(zm, z[j]);
    zm = warp_max(zm);
    double total = 1.0;
    if (!p.sigmoid) {
        double sum = 0.0;
        for (int j = 0; j < P; ++j)
            if (j < ln.n) sum += exp((double)z[j] - (double)zm);
        total = warp_sum(sum);
    }
    uint64_t key[P];
    for (int j = 0; j < P; ++j) {
        key[j] = 0;
        if (j < ln.n) {
            double s;
            if (p.sigmoid) {
                const double e = exp(-fabs((double)z[j]));
                s = (z[j] >= 0.0f ? 1.0 : e) / (1.0 + e);
            } else {
                s = exp((double)z[j] - (double)zm) / total;
            }
            key[j] = order_key(p.bias ? s + (double)p.bias[ln.first + j] : s);
        }
    }
    bool close;
    return choose<uint64_t, P>(p, key, ln, lane, 0.0f, 0.0f, close);
}

// One token by one warp.
template <int P>
__device__ __forceinline__ void route_token(const ScoredArgs& p, int64_t t, int lane) {
    const Lane ln(p, lane);
    float z[P];
    load_logits<P>(p, t, ln, z);
    bool finite = true;
    float zm = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < P; ++j)
        if (j < ln.n) {
            if (p.z_out) p.z_out[t * p.E + ln.first + j] = z[j];
            finite = finite && isfinite(z[j]);
            zm = fmaxf(zm, z[j]);
        }
    // s, in z's place
    float total = 1.0f, top = 0.0f;
    if (!p.sigmoid) {
        zm = warp_max(zm);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (j < ln.n) {
                z[j] = expf(z[j] - zm);
                sum += z[j];
            }
        total = warp_sum(sum);
    }
    uint32_t key[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        key[j] = 0u;
        if (j < ln.n) {
            float s;
            if (p.sigmoid) {
                const float e = expf(-fabsf(z[j]));
                s = (z[j] >= 0.0f ? 1.0f : e) / (1.0f + e);
            } else {
                s = z[j] / total;
            }
            top = fmaxf(top, s);
            if (p.bias) {
                const float b = __ldg(p.bias + ln.first + j);
                finite = finite && b < CUDART_INF_F;  // false for NaN too
                s += b;
            }
            key[j] = order_key(s);
        }
    }
    finite = __all_sync(kFull, finite);
    if (!finite && lane == 0) atomicOr(p.err, DERR_NONFINITE_LOGIT);
    bool close;
    // binary32 scores are off by at most 4 units (sigmoid), or the rounding of
    // a sum of up to 64 + 5 terms more (softmax); rel is twice that, rounded up
    int my_id = choose<uint32_t, P>(p, key, ln, lane, p.sigmoid ? 0x1p-19f : 0x1p-16f,
                                    p.bias ? warp_max(top) : 0.0f, close);
    if (close && finite) my_id = choose_in_64<P>(p, t, lane);

    // weights, by lane s < k for its own pick
    const bool mine = lane < p.k && my_id >= 0;
    const float zc = mine ? logit_of(p, t, my_id) : -CUDART_INF_F;
    const bool out = !mine || (p.bias && p.bias[my_id] == -CUDART_INF_F);  // taken out: weight 0
    float w = 0.0f;
    if (p.renorm) {
        // relative to the largest chosen score, so nothing underflows
        const float top_z = warp_max(out ? -CUDART_INF_F : zc);
        if (!out)
            w = p.sigmoid ? expf(fminf(zc, 0.0f) - fminf(top_z, 0.0f)) / (1.0f + expf(-fabsf(zc)))
                          : expf(zc - top_z);
        const float sum = warp_sum(w);
        w = sum > 0.0f ? w / sum * p.scale : 0.0f;
    } else if (!out) {
        const float e = expf(-fabsf(zc));
        w = p.scale * (p.sigmoid ? (zc >= 0.0f ? 1.0f : e) / (1.0f + e) : expf(zc - zm) / total);
    }
    // rank of my id among the chosen ids -> ascending-id slot
    int rank = 0;
    for (int s = 0; s < p.k; ++s) {
        const int other = __shfl_sync(kFull, my_id, s);
        rank += other >= 0 && other < my_id;
    }
    if (mine) {
        p.ids[t * p.k + rank] = my_id;
        p.w[t * p.k + rank] = w;
    }
}

template <int P>
__global__ void __launch_bounds__(256) scored_topk_kernel(const __grid_constant__ ScoredArgs p) {
    const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t < p.T) route_token<P>(p, t, threadIdx.x & 31);
}

}  // namespace

void scored_layout(ScoredArgs& p) {
    int lanes = 1;
    while (lanes * 2 * p.n_groups <= 32) lanes *= 2;
    p.lanes = lanes;
    p.group_size = p.E / p.n_groups;
    p.per_lane = (p.group_size + lanes - 1) / lanes;
    p.vector_loads = p.group_size % 4 == 0 && p.per_lane % 4 == 0;
}

cudaError_t launch_scored_topk(const ScoredArgs& p, cudaStream_t s) {
    if (p.T <= 0) return cudaSuccess;
    const int warps = 8, grid = (p.T + warps - 1) / warps;
    if (p.per_lane <= 1) scored_topk_kernel<1><<<grid, 32 * warps, 0, s>>>(p);
    else if (p.per_lane <= 2) scored_topk_kernel<2><<<grid, 32 * warps, 0, s>>>(p);
    else if (p.per_lane <= 4) scored_topk_kernel<4><<<grid, 32 * warps, 0, s>>>(p);
    else if (p.per_lane <= 8) scored_topk_kernel<8><<<grid, 32 * warps, 0, s>>>(p);
    else if (p.per_lane <= 16) scored_topk_kernel<16><<<grid, 32 * warps, 0, s>>>(p);
    else if (p.per_lane <= 32) scored_topk_kernel<32><<<grid, 32 * warps, 0, s>>>(p);
    else scored_topk_kernel<64><<<grid, 32 * warps, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace dwdp
