// route_scored.cu: what dwdp_route_scored does with the router's logits:
// scores, choice values, groups of experts, top-k and weights, one warp per
// token, and the grouping of the pairs by expert.  Latency- and
// instruction-bound (a few bytes a token).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "dwdp_internal.h"

namespace dwdp {
namespace {

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

// A lane's two best keys with their places in its run (the lowest on ties).
template <class K>
struct Best2 {
    K k1 = 0, k2 = 0;
    int i1 = 0, i2 = 0;
    __device__ __forceinline__ void add(K c, int j) {
        if (c > k1) {
            k2 = k1;
            i2 = i1;
            k1 = c;
            i1 = j;
        } else if (c > k2) {
            k2 = c;
            i2 = j;
        }
    }
};

// The error of a binary32 choice value v against the formula's is at most half
// of rel (ref or |v|) + 2^-22 |v|: two values further apart than that are in
// the right order.  A sigmoid s is off by at most s (1 - s) 2^-23 (expf) +
// 2^-24 s (the sum) + 2^-24 s (the quotient) < 2^-22 s; a softmax term by the
// roundings of its sum of per_lane + 5 terms as well, 2^-24 each.  Without a
// bias the value is the score (softmax: unnormalised) and ref is 0.
struct Tolerance {
    float rel, ref;
    __device__ __forceinline__ float operator()(float v) const {
        return rel * (ref > 0.0f ? ref : fabsf(v)) + 0x1p-22f * fabsf(v);
    }
};

// Keys of the choice values (0: no expert) from the logits in z.  zm is the
// largest logit, total the softmax denominator; both 1 and unused for sigmoid.
template <int P>
__device__ __forceinline__ Tolerance choice_keys(const ScoredArgs& p, const Lane& ln, float (&z)[P],
                                                 uint32_t (&key)[P], float& zm, float& total, bool& finite) {
    finite = true;
    zm = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < P; ++j)
        if (j < ln.n) {
            finite = finite && isfinite(z[j]);
            zm = fmaxf(zm, z[j]);
        }
    total = 1.0f;
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
    const float inv = 1.0f / total;
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < P; ++j) {
        key[j] = 0u;
        if (j < ln.n) {
            float s = z[j];
            if (p.sigmoid) {
                const float e = expf(-fabsf(z[j]));
                s = (z[j] >= 0.0f ? 1.0f : e) / (1.0f + e);
            }
            if (p.bias) {
                if (!p.sigmoid) s *= inv;
                top = fmaxf(top, s);
                const float b = __ldg(p.bias + ln.first + j);
                finite = finite && b < CUDART_INF_F;  // false for NaN too
                s += b;
            }
            key[j] = order_key(s);
        }
    }
    finite = __all_sync(kFull, finite);
    return Tolerance{p.sigmoid ? 0x1p-21f : (float)(p.per_lane + 12) * 0x1p-23f, p.bias ? warp_max(top) : 0.0f};
}

// The value itself in binary64 (softmax: total is the denominator with a
// bias, 1 without).
__device__ __forceinline__ double choice_in_64(const ScoredArgs& p, float z, int expert, float zm, double total) {
    double s;
    if (p.sigmoid) {
        const double e = exp(-fabs((double)z));
        s = (z >= 0.0f ? 1.0 : e) / (1.0 + e);
    } else {
        s = exp((double)z - (double)zm) / total;
    }
    return p.bias ? s + (double)p.bias[expert] : s;
}

// A group's best two (by all its lanes) and its score.
template <class K>
__device__ __forceinline__ K group_score(const ScoredArgs& p, const Lane& ln, K& k1, K& k2) {
    for (int o = 1; o < p.lanes; o <<= 1) {
        const K o1 = __shfl_xor_sync(kFull, k1, o), o2 = __shfl_xor_sync(kFull, k2, o);
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
    }
    const K score = p.group_top2 && k2 != 0 ? order_key(key_value(k1) + key_value(k2)) : k1;
    return ln.g < p.n_groups ? score : (K)0;
}

// How many groups come before this lane's: larger, or as large and lower.
template <class K>
__device__ __forceinline__ int group_rank(const ScoredArgs& p, const Lane& ln, K score) {
    int rank = 0;
    for (int g = 0; g < p.n_groups; ++g) {
        const K other = __shfl_sync(kFull, score, g * p.lanes);
        rank += (other > score) || (other == score && g < ln.g);
    }
    return rank;
}

// The k best of the lanes' keys.  Lane s < k gets the s-th pick's id; last is
// the k-th pick's key, next the best left (0: none).  A lane offers its best
// key; after a pick it falls back on its second, and looks through its run
// again only when that is gone too.  Lane order is expert order, so the
// lowest lane offering the largest key holds the lowest id.
template <class K, int P>
__device__ __forceinline__ int pick(const ScoredArgs& p, const K (&key)[P], const Best2<K>& best, const Lane& ln,
                                    int lane, K& last, K& next) {
    K offer = best.k1, second = best.k2;
    int at = best.i1, at2 = best.i2, my_id = -1;
    last = 0;
    for (int s = 0; s < p.k; ++s) {
        const K gk = warp_max(offer);
        if (gk == 0) break;  // fewer than k candidates (refused on the host)
        last = gk;
        const int owner = __ffs(__ballot_sync(kFull, offer == gk)) - 1;
        const int id = __shfl_sync(kFull, ln.first + at, owner);
        if (lane == s) my_id = id;
        if (lane == owner) {
            if (second != 0) {
                offer = second;
                at = at2;
                second = 0;
            } else {  // the best of what comes after (offer, at) in order
                Best2<K> rest;
#pragma unroll
                for (int j = 0; j < P; ++j)
                    if (key[j] < offer || (key[j] == offer && j > at)) rest.add(key[j], j);
                offer = rest.k1;
                at = rest.i1;
                second = rest.k2;
                at2 = rest.i2;
            }
        }
    }
    next = warp_max(offer);
    return my_id;
}

// Shared memory of one warp for choose_close: the choice values' keys, and
// the values in doubt with their keys in binary64.
struct Scratch {
    uint64_t* exact;  // [E], by place in the list
    uint32_t* key;    // [E]
    int* list;        // [E]
    static constexpr int kBytes = 16;  // per expert
    __device__ Scratch(void* base, int E, int warp) {
        char* at = static_cast<char*>(base) + (size_t)warp * E * kBytes;
        exact = reinterpret_cast<uint64_t*>(at);
        key = reinterpret_cast<uint32_t*>(at + 8 * (size_t)E);
        list = reinterpret_cast<int*>(at + 12 * (size_t)E);
    }
};

// The entry that follows (last, last_at) in the order of keys, largest first
// and the lowest place among equals, of n keys in shared memory that `use`
// admits; 0 if none.  Start with (all ones, -1).
template <class K, class F>
__device__ __forceinline__ void next_in_order(const K* keys, int n, int lane, K& last, int& last_at, F use) {
    K best = 0;
    int at = 0x7fffffff;
#pragma unroll 1
    for (int i = lane; i < n; i += 32) {
        const K c = keys[i];
        if (c > best && (c < last || (c == last && i > last_at)) && use(i)) {
            best = c;
            at = i;
        }
    }
    const K top = warp_max(best);
    last_at = (int)__reduce_min_sync(kFull, best == top ? (unsigned)at : 0x7fffffffu);
    last = top;
}

// The choice where binary32 cannot tell.  What lies further from a decision
// than the tolerance is settled; the values within it are listed and taken in
// binary64, 32 at a time (binary64 runs at 1/64 of binary32's rate or less,
// so the whole choice in it would take a warp some 30 us).  Rare, so small:
// loops over shared memory, nothing unrolled.  s.key holds the keys.
__device__ __forceinline__ int choose_close(const ScoredArgs& p, int64_t t, int lane, const Scratch& s,
                                            const Tolerance& tol, float zm) {
    const int E = p.E, G = p.n_groups, gs = p.group_size;
    double total = 1.0;
    if (!p.sigmoid && p.bias) {
        double sum = 0.0;
#pragma unroll 1
        for (int e = lane; e < E; e += 32) sum += exp((double)logit_of(p, t, e) - (double)zm);
        total = warp_sum(sum);
    }
    auto take_in_64 = [&](int n) {
        __syncwarp();
#pragma unroll 1
        for (int i = lane; i < n; i += 32) {
            const int e = s.list[i];
            s.exact[i] = order_key(choice_in_64(p, logit_of(p, t, e), e, zm, total));
        }
        __syncwarp();
    };
    uint32_t groups = kFull;  // the groups a token may choose from
    if (p.top_groups < G) {
        // lane g: group g
        const bool is_group = lane < G;
        uint32_t k1 = 0, k2 = 0;
        if (is_group)
#pragma unroll 1
            for (int e = lane * gs; e < (lane + 1) * gs; ++e) {
                const uint32_t c = s.key[e];
                k2 = max(k2, min(k1, c));
                k1 = max(k1, c);
            }
        const bool two = p.group_top2 && k2 != 0;
        const float v = two ? key_value(k1) + key_value(k2) : key_value(k1);
        const uint32_t score = is_group ? order_key(v) : 0u;
        int rank = 0;
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
            const uint32_t o = __shfl_sync(kFull, score, g);
            rank += o > score || (o == score && g < lane);
        }
        const float edge = key_value(~warp_max(is_group && rank < p.top_groups ? ~score : 0u)), wide = 2.0f * tol(edge);
        const bool sure = is_group && v > edge && !(v - edge <= wide);
        const bool open = is_group && !sure && !(edge - v > wide);
        const uint32_t sures = __ballot_sync(kFull, sure);
        const uint32_t opens = __ballot_sync(kFull, open);
        // the values that the open groups' scores may consist of
        const float low = key_value(two ? k2 : k1), floor_of = low - tol(low);
        int n = 0;
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
            if (!((opens >> g) & 1u)) continue;
            const float floor_g = __shfl_sync(kFull, floor_of, g);
#pragma unroll 1
            for (int i = 0; i < gs; i += 32) {
                const int e = g * gs + i + lane;
                const bool in = i + lane < gs && !(key_value(s.key[e]) < floor_g);
                const uint32_t ins = __ballot_sync(kFull, in);
                if (in) s.list[n + __popc(ins & ((1u << lane) - 1u))] = e;
                n += __popc(ins);
            }
        }
        take_in_64(n);
        uint64_t m1 = 0, m2 = 0;
#pragma unroll 1
        for (int i = 0; i < n; ++i)
            if (open && s.list[i] / gs == lane) {
                const uint64_t c = s.exact[i];
                m2 = max(m2, min(m1, c));
                m1 = max(m1, c);
            }
        const uint64_t exact = open ? (p.group_top2 && m2 != 0 ? order_key(key_value(m1) + key_value(m2)) : m1) : 0;
        rank = 0;
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
            const uint64_t o = __shfl_sync(kFull, exact, g);
            rank += o > exact || (o == exact && g < lane);
        }
        groups = sures | __ballot_sync(kFull, open && rank < p.top_groups - __popc(sures));
    }
    auto allowed = [&](int e) { return ((groups >> (e / gs)) & 1u) != 0; };
    // the k-th value, then what is above it beyond doubt and what is near it
    uint32_t last = 0xffffffffu;
    int at = -1;
#pragma unroll 1
    for (int i = 0; i < p.k; ++i) next_in_order(s.key, E, lane, last, at, allowed);
    const float edge = key_value(last), wide = tol(edge);
    int my_id = -1, n_sure = 0, n = 0;
#pragma unroll 1
    for (int i = 0; i < E; i += 32) {
        const int e = i + lane;
        const bool in = e < E && allowed(e);
        const float v = in ? key_value(s.key[e]) : 0.0f;
        const bool sure = in && v > edge && !(v - edge <= wide);
        const bool open = in && !sure && !(edge - v > wide);
        uint32_t sures = __ballot_sync(kFull, sure);
        const uint32_t opens = __ballot_sync(kFull, open);
        for (; sures != 0; sures &= sures - 1, ++n_sure)
            if (lane == n_sure) my_id = i + __ffs(sures) - 1;
        if (open) s.list[n + __popc(opens & ((1u << lane) - 1u))] = e;
        n += __popc(opens);
    }
    take_in_64(n);
    uint64_t last64 = ~0ull;
    at = -1;
#pragma unroll 1
    for (int i = n_sure; i < p.k; ++i) {
        next_in_order(s.exact, n, lane, last64, at, [](int) { return true; });
        if (lane == i && at < n) my_id = s.list[at];
    }
    __syncwarp();
    return my_id;
}

// One token by one warp: lane s < k gets the s-th pick's id, the slot it has
// in ascending order of ids, and its weight.
struct Pick {
    int id, slot;
    float w;
};
template <int P>
__device__ __forceinline__ Pick route_token(const ScoredArgs& p, int64_t t, int lane, const Scratch& scratch) {
    const Lane ln(p, lane);
    float z[P];
    load_logits<P>(p, t, ln, z);
    if (p.z_out) {
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (j < ln.n) p.z_out[t * p.E + ln.first + j] = z[j];
    }
    uint32_t key[P];
    float zm, total;
    bool finite;
    const Tolerance tol = choice_keys<P>(p, ln, z, key, zm, total, finite);
    if (!finite && lane == 0) atomicOr(p.err, DERR_NONFINITE_LOGIT);
    // close: a difference of infinities is NaN and never close, ties go by id
    auto close = [&](uint32_t a, uint32_t b, float times) {
        return key_value(a) - key_value(b) <= times * tol(key_value(a));
    };
    Best2<uint32_t> best;
#pragma unroll
    for (int j = 0; j < P; ++j) best.add(key[j], j);
    bool again = false;
    if (p.top_groups < p.n_groups) {
        uint32_t k1 = best.k1, k2 = best.k2;
        const uint32_t score = group_score(p, ln, k1, k2);
        const int rank = group_rank(p, ln, score);  // by every lane: it shuffles
        const bool is_group = ln.g < p.n_groups, kept = is_group && rank < p.top_groups;
        again = close(~warp_max(kept ? ~score : 0u), warp_max(is_group && !kept ? score : 0u), 2.0f);
        if (!kept) best.k1 = best.k2 = 0;
    }
    uint32_t last, next;
    int my_id = pick<uint32_t, P>(p, key, best, ln, lane, last, next);
    again = again || (next != 0 && close(last, next, 1.0f));
    if (again && finite) {
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (j < ln.n) scratch.key[ln.first + j] = key[j];
        __syncwarp();
        my_id = choose_close(p, t, lane, scratch, tol, zm);
    }

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
    return Pick{my_id, rank, w};
}

// ------------------------------------------------------------- grouping --
// The pairs are taken in chunks of whole tokens, at most kChunk pairs each:
//   select   a cluster of 8 blocks per chunk chooses, and counts its pairs
//            by expert in its first block's shared memory: hist[chunk][e]
//   place    a block per chunk adds up the counts of all chunks (its base is
//            what lies before it), and ranks its own pairs
// or, with one chunk, the cluster's first block does both.  Each pair's row is the stable one
// (ascending flat index within an expert).
constexpr int kChunk = 1024;
constexpr int kSelectCluster = 8;
constexpr int kSelectWarps = 8;
// Above this many chunks the sums over all of them, in every chunk's block,
// cost more than a scan kernel between the two.
constexpr int kSelfScanChunks = 128;

__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive scan of one value per thread over a block of up to 1024; `tmp`
// holds 32, zero where the block has no warp.
__device__ __forceinline__ int block_scan(int v, int* tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) tmp[warp] = s;
    __syncthreads();
    int w = tmp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += u;
    }
    const int before = __shfl_sync(kFull, w, warp > 0 ? warp - 1 : 0);
    return s - v + (warp > 0 ? before : 0);
}

// Rows of a chunk's n pairs (thread i: pair first + i of expert e, or none)
// from the row of each expert's first pair in the chunk, base[e].
// wc: [32 warps][E] bytes, zeroed; the block is past a barrier since then.
__device__ __forceinline__ void place_pairs(const ScoredArgs& p, int first, int n, int e, const int* base,
                                            uint8_t* wc) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool valid = (int)threadIdx.x < n;
    const uint32_t same = __match_any_sync(kFull, valid ? e : -1);
    const int in_warp = __popc(same & ((1u << lane) - 1u));
    if (valid && in_warp == 0) wc[warp * p.E + e] = (uint8_t)__popc(same);
    __syncthreads();
    if (valid) {
        int r = base[e] + in_warp;
        for (int w = 0; w < warp; ++w) r += wc[w * p.E + e];
        p.perm[r] = first + threadIdx.x;
        p.inv_perm[first + threadIdx.x] = r;
    }
}

// hist holds the chunks' counts; with SCANNED, the chunks' bases (and counts
// and offsets are written already).
template <bool SCANNED>
__global__ void __launch_bounds__(kChunk) scored_place_kernel(const __grid_constant__ ScoredArgs p, int n_chunks) {
    extern __shared__ int base[];  // [E], then wc
    __shared__ int part[2][kChunk];
    __shared__ int tmp[32];
    uint8_t* wc = reinterpret_cast<uint8_t*>(base + p.E);
    const int chunk = blockIdx.x, tid = threadIdx.x;
    for (int i = tid; i < 8 * p.E; i += kChunk) reinterpret_cast<int*>(wc)[i] = 0;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int first = chunk * p.chunk_tokens * p.k;
    const int n = min(p.T * p.k - first, p.chunk_tokens * p.k);
    const int e = tid < n ? p.ids[first + tid] : 0;
    if constexpr (SCANNED) {
        for (int i = tid; i < p.E; i += kChunk) base[i] = p.hist[(int64_t)chunk * p.E + i];
        __syncthreads();
    } else {
        // 1024 / ep threads per expert, each a part of the chunks
        int ep = 1;
        while (ep < p.E) ep <<= 1;
        const int parts = kChunk / ep, x = tid % ep, q = tid / ep;
        int all = 0, before = 0;
        if (x < p.E)
#pragma unroll 4
            for (int c = q; c < n_chunks; c += parts) {
                const int h = p.hist[(int64_t)c * p.E + x];
                all += h;
                before += c < chunk ? h : 0;
            }
        part[0][tid] = all;
        part[1][tid] = before;
        __syncthreads();
        all = before = 0;
        if (tid < p.E)
            for (int i = 0; i < parts; ++i) {
                all += part[0][tid + i * ep];
                before += part[1][tid + i * ep];
            }
        const int offset = block_scan(all, tmp);
        if (tid < p.E) {
            base[tid] = offset + before;
            if (chunk == 0) {
                p.counts[tid] = all;
                p.offsets[tid] = offset;
                if (tid == p.E - 1) p.offsets[p.E] = offset + all;
            }
        }
        __syncthreads();
    }
    place_pairs(p, first, n, e, base, wc);
}

// The cluster's choice for chunk `chunk`: ids and weights written, its pairs
// counted by expert in `count` of the cluster's first block.  Dynamic shared
// memory: Scratch of every warp.
template <int P>
__device__ __forceinline__ void select_chunk(const ScoredArgs& p, int chunk, int rank, void* smem, int* count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Scratch scratch(smem, p.E, warp);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) count[e] = 0;
    wait_for_previous_kernel();
    let_next_kernel_start();
    cluster_sync();
    const int end = min(p.T, (chunk + 1) * p.chunk_tokens);
    for (int t = chunk * p.chunk_tokens + rank * kSelectWarps + warp; t < end; t += kSelectCluster * kSelectWarps) {
        const Pick pick = route_token<P>(p, t, lane, scratch);
        if (lane < p.k && pick.id >= 0) {
            uint32_t at;
            asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                         : "=r"(at)
                         : "r"((uint32_t)__cvta_generic_to_shared(count + pick.id)));
            asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], 1;" ::"r"(at) : "memory");
        }
        __syncwarp();
    }
    __syncwarp();
    cluster_sync();
}

template <int P>
__global__ void __launch_bounds__(32 * kSelectWarps) __cluster_dims__(kSelectCluster, 1, 1)
    scored_select_kernel(const __grid_constant__ ScoredArgs p) {
    extern __shared__ __align__(16) char smem[];
    __shared__ int count[DWDP_MAX_EXPERTS];
    const int chunk = blockIdx.x / kSelectCluster, rank = blockIdx.x % kSelectCluster;
    select_chunk<P>(p, chunk, rank, smem, count);
    if (rank == 0)
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[(int64_t)chunk * p.E + e] = count[e];
}

// One chunk: the cluster's first block also places the pairs, a round of 256
// at a time; base[e] moves on by the round's pairs.
template <int P>
__global__ void __launch_bounds__(32 * kSelectWarps) __cluster_dims__(kSelectCluster, 1, 1)
    scored_one_kernel(const __grid_constant__ ScoredArgs p) {
    constexpr int kThreads = 32 * kSelectWarps, kPer = DWDP_MAX_EXPERTS / kThreads;
    extern __shared__ __align__(16) char smem[];
    __shared__ int base[DWDP_MAX_EXPERTS];
    __shared__ int tmp[32];
    select_chunk<P>(p, 0, blockIdx.x, smem, base);
    if (blockIdx.x != 0) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* wc = reinterpret_cast<uint8_t*>(smem);  // [warps][E]; the scratch is done with
    int mine[kPer], sum = 0;                         // experts kPer tid ...
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        mine[j] = kPer * tid + j < p.E ? base[kPer * tid + j] : 0;
        sum += mine[j];
    }
    if (tid < 32) tmp[tid] = 0;
    __syncthreads();
    int offset = block_scan(sum, tmp);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = kPer * tid + j;
        if (e < p.E) {
            base[e] = offset;
            p.counts[e] = mine[j];
            p.offsets[e] = offset;
            offset += mine[j];
            if (e == p.E - 1) p.offsets[p.E] = offset;
        }
    }
    const int n = p.T * p.k;
    for (int first = 0; first < n; first += kThreads) {
        for (int i = tid; i < kSelectWarps * p.E; i += kThreads) wc[i] = 0;
        __syncthreads();
        const int f = first + tid;
        const int e = f < n ? p.ids[f] : -1;
        const uint32_t same = __match_any_sync(kFull, e);
        const int in_warp = __popc(same & ((1u << lane) - 1u));
        if (e >= 0 && in_warp == 0) wc[warp * p.E + e] = (uint8_t)__popc(same);
        __syncthreads();
        int r = 0;
        if (e >= 0) {
            r = base[e] + in_warp;
            for (int w = 0; w < warp; ++w) r += wc[w * p.E + e];
            p.perm[r] = f;
            p.inv_perm[f] = r;
        }
        __syncthreads();
        if (e >= 0 && in_warp == 0) atomicAdd(&base[e], (int)__popc(same));
    }
}

template <class F, class... A>
cudaError_t launch(F kernel, int grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

template <int P>
cudaError_t launch_per_lane(const ScoredArgs& p, int n_chunks, cudaStream_t s) {
    const size_t smem = (size_t)kSelectWarps * p.E * Scratch::kBytes;
    auto kernel = n_chunks == 1 ? scored_one_kernel<P> : scored_select_kernel<P>;
    if (smem > 40 << 10) {  // beside the static part, beyond what a launch gets unasked
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch(kernel, n_chunks * kSelectCluster, 32 * kSelectWarps, smem, s, p);
    if (e != cudaSuccess || n_chunks == 1) return e;
    if (n_chunks <= kSelfScanChunks)
        return launch(scored_place_kernel<false>, n_chunks, kChunk, (size_t)p.E * 36, s, p, n_chunks);
    e = launch_chunk_scan(p.hist, n_chunks, p.E, p.counts, p.offsets, s);
    if (e != cudaSuccess) return e;
    return launch(scored_place_kernel<true>, n_chunks, kChunk, (size_t)p.E * 36, s, p, n_chunks);
}

}  // namespace

size_t scored_scratch_bytes(int64_t T, int64_t E, int64_t k) {
    const int64_t tokens = kChunk / k;
    return (size_t)((T + tokens - 1) / tokens * E * 4);
}

cudaError_t launch_scored_choice(ScoredArgs& p, cudaStream_t s) {
    if (p.T <= 0) return cudaSuccess;
    p.lanes = 1;
    while (p.lanes * 2 * p.n_groups <= 32) p.lanes *= 2;
    p.group_size = p.E / p.n_groups;
    p.per_lane = (p.group_size + p.lanes - 1) / p.lanes;
    p.vector_loads = p.group_size % 4 == 0 && p.per_lane % 4 == 0;
    p.chunk_tokens = kChunk / p.k;
    const int n_chunks = (p.T + p.chunk_tokens - 1) / p.chunk_tokens;
    if (p.per_lane <= 1) return launch_per_lane<1>(p, n_chunks, s);
    if (p.per_lane <= 2) return launch_per_lane<2>(p, n_chunks, s);
    if (p.per_lane <= 4) return launch_per_lane<4>(p, n_chunks, s);
    if (p.per_lane <= 8) return launch_per_lane<8>(p, n_chunks, s);
    if (p.per_lane <= 16) return launch_per_lane<16>(p, n_chunks, s);
    if (p.per_lane <= 32) return launch_per_lane<32>(p, n_chunks, s);
    return launch_per_lane<64>(p, n_chunks, s);
}

}  // namespace dwdp
