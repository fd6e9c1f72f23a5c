// route_scored.cu: what dwdp_route_scored does with the router's logits:
// scores, choice values, groups of experts, top-k and weights, one warp per
// token, and the grouping of the pairs by expert.  A few bytes a token: bound
// by latency for few tokens and by instructions (about 1000 a token of 256
// experts) for many.  8 of 256 experts in 4 of 8 groups, with the router GEMM
// of H = 7168: 1 token 7.5 us, 256 tokens 17.9, 8192 tokens 47.7, of which the
// GEMM about 28, the choice 13 and the grouping 6.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "dwdp_internal.h"

namespace dwdp {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// Order-preserving keys: a > b iff key(a) > key(b).  Made of results of
// arithmetic only: a sum never gives -0 here (scores are not negative), and a
// NaN is the positive one, above +inf.  No value has key 0, which marks "not
// a candidate".
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ (((k >> 31) - 1u) | 0x80000000u));
}
// Keys of a lane's run: the value's last log2 P bits, cut towards zero, make
// room for the place j (lower places larger), so that no two keys of a lane
// are alike and a pick needs no index beside it.  What the cut costs is part
// of the tolerance below.
template <int P>
__device__ __forceinline__ uint32_t place_key(float x, int j) {
    return (order_key(__uint_as_float(__float_as_uint(x) & ~(P - 1u))) & ~(P - 1u)) | (P - 1u - j);
}
template <int P>
__device__ __forceinline__ float place_value(uint32_t k) {
    return __uint_as_float(__float_as_uint(key_value(k)) & ~(P - 1u));
}
constexpr uint64_t kSign64 = 0x8000000000000000ull;
__device__ __forceinline__ uint64_t order_key(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    return u ^ ((uint64_t)((int64_t)u >> 63) | kSign64);
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __longlong_as_double((long long)(k ^ (((k >> 63) - 1ull) | kSign64)));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kFull, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((uint64_t)hi << 32) | lo;
}
// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 2^x, and 1 / x: a few units in the last place, results below the normal
// range are 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.44269504f;

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
        first = g * p.group_size + at;  // (beyond the experts where there are none)
    }
};

// The kernels come in two forms.  FULL: every lane holds exactly P experts
// (32 P = E and whole groups), so nothing asks whether expert j exists; and
// runs are read in 16-byte pieces (8 for P = 2).  In the other form a lane
// holds n <= P of them.
template <int P, bool FULL>
__device__ __forceinline__ bool has(const Lane& ln, int j) {
    return FULL || j < ln.n;
}

// v[j] = src[first + j]
template <int P, bool FULL>
__device__ __forceinline__ void load_run(const float* src, const Lane& ln, float (&v)[P]) {
    src += ln.first;
    if constexpr (FULL && P >= 4) {
#pragma unroll
        for (int j = 0; j < P; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(src + j);
            v[j] = f.x;
            v[j + 1] = f.y;
            v[j + 2] = f.z;
            v[j + 3] = f.w;
        }
    } else if constexpr (FULL && P == 2) {
        const float2 f = *reinterpret_cast<const float2*>(src);
        v[0] = f.x;
        v[1] = f.y;
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = has<P, FULL>(ln, j) ? src[j] : 0.0f;
    }
}

// z[j] = the token's logit of expert first + j: the partial-sum planes of a
// K-split router GEMM added in plane order.
template <int P, bool FULL>
__device__ __forceinline__ void load_logits(const ScoredArgs& p, int64_t t, const Lane& ln, float (&z)[P]) {
    load_run<P, FULL>(p.logits + t * p.pitch, ln, z);
#pragma unroll 1
    for (int q = 1; q < p.parts; ++q) {
        float u[P];
        load_run<P, FULL>(p.logits + (q * (int64_t)p.T + t) * p.pitch, ln, u);
#pragma unroll
        for (int j = 0; j < P; ++j) z[j] += u[j];
    }
}

__device__ __forceinline__ float logit_of(const ScoredArgs& p, int64_t t, int e) {
    float v = p.logits[t * p.pitch + e];
    for (int q = 1; q < p.parts; ++q) v += p.logits[(q * (int64_t)p.T + t) * p.pitch + e];
    return v;
}

// A lane's three best keys.
struct Best3 {
    uint32_t k1 = 0, k2 = 0, k3 = 0;
    __device__ __forceinline__ void add(uint32_t c) {
        k3 = max(k3, min(k2, c));
        k2 = max(k2, min(k1, c));
        k1 = max(k1, c);
    }
};

// Two choice values further apart than (*this)(v) are in the right order.  A
// binary32 value's error is at most half of rel (ref or |v|) + 2^-22 |v|, and
// its key is cut by less than P - 1 units of 2^-23 |v|, always towards zero.
// Two groups' sums of two values are in the right order where they are further
// apart than twice (*this)(m), m the larger of |first| + |second| of the two
// groups: four values' errors, and cuts that go both ways where the signs differ.
// With ex2.approx and its argument's rounding, |z| <= most:
//   sigmoid      s (1 - s) (1.7 |z| 2^-24 + 2^-22) + s 2^-22: 2^-21 of 1 at
//                most, or (most 2^-23 + 2^-21) of s
//   softmax term e (2.7 |z - max| 2^-24 + 2^-22): with a bias 2^-21 of the
//                largest and the roundings of the sum of per_lane + 5; without
//                one unnormalised, so (most 2^-21 + 2^-22) of e
struct Tolerance {
    float rel, ref, own;
    __device__ __forceinline__ float operator()(float v) const {
        return rel * (ref > 0.0f ? ref : fabsf(v)) + own * fabsf(v);
    }
};

// Keys of the choice values (0: no expert) from the logits in z and the bias
// in b.  Without a bias the value is the score (softmax: unnormalised).  zm is the largest
// logit, total the softmax denominator (neither set for sigmoid).
template <int P, bool FULL>
__device__ __forceinline__ Tolerance choice_keys(const ScoredArgs& p, const Lane& ln, float (&z)[P],
                                                 const float (&b)[P], uint32_t (&key)[P], float& zm, float& total, bool& finite) {
    float most = 0.0f, worst = 0.0f;
#pragma unroll
    for (int j = 0; j < P; ++j) most = max_nan(most, fabsf(z[j]));  // (0 where there is no expert)
    finite = most < CUDART_INF_F;
    zm = total = 0.0f;
    float factor = 1.0f;
    if (p.sigmoid) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float e = exp2_fast(-kLog2e * fabsf(z[j]));
            z[j] = (z[j] >= 0.0f ? 1.0f : e) * rcp_fast(1.0f + e);
        }
    } else {
        zm = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (has<P, FULL>(ln, j)) zm = fmaxf(zm, z[j]);
        zm = warp_max(zm);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            z[j] = has<P, FULL>(ln, j) ? exp2_fast(kLog2e * (z[j] - zm)) : 0.0f;
            total += z[j];
        }
        total = warp_sum(total);
        if (p.bias) factor = 1.0f / total;
    }
    if (p.bias) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            z[j] = fmaf(z[j], factor, b[j]);
            worst = max_nan(worst, z[j]);  // +inf or NaN where the bias is
        }
    }
#pragma unroll
    for (int j = 0; j < P; ++j) key[j] = has<P, FULL>(ln, j) ? place_key<P>(z[j], j) : 0u;
    finite = __all_sync(kFull, finite && worst < CUDART_INF_F);
    most = __uint_as_float(warp_max(__float_as_uint(most)));
    constexpr float own = 0x1p-22f + (P - 1) * 0x1p-23f;
    if (p.bias) return p.sigmoid ? Tolerance{0x1p-20f, 1.0f, own} : Tolerance{0x1p-18f + p.per_lane * 0x1p-23f, factor, own};
    return Tolerance{p.sigmoid ? 0x1p-20f + most * 0x1p-22f : 0x1p-21f + most * 0x1p-20f, 0.0f, own};
}

// The k best of the lanes' keys.  Lane s < k gets the s-th pick's id; last is
// the k-th pick's key, next the best left (0: none); a pick's own key goes to
// its lane.  A lane offers its best key, and after a pick the next of its
// three; a lane picked three times (one token in five has one, at 8 of 16
// lanes' 128) looks through its run again.  Lane order is expert order, so
// the lowest lane offering the largest key holds the lowest id.
template <int P>
__device__ __forceinline__ int pick(const ScoredArgs& p, const uint32_t (&key)[P], Best3 best, const Lane& ln,
                                    int lane, uint32_t& my_key, uint32_t& last, uint32_t& next) {
    int my_owner = 0;
    last = my_key = 0;
#pragma unroll 1
    for (int s = 0; s < p.k; ++s) {
        const uint32_t gk = last = warp_max(best.k1);  // never 0: the host refuses fewer than k candidates
        const int owner = __ffs(__ballot_sync(kFull, best.k1 == gk)) - 1;
        my_owner = lane == s ? owner : my_owner;
        my_key = lane == s ? gk : my_key;
        if (lane == owner) {
            best.k1 = best.k2;
            best.k2 = best.k3;
            best.k3 = 0;
            if (P > 3 && best.k1 == 0) {  // what comes after gk in order
#pragma unroll
                for (int j = 0; j < P; ++j) best.add(key[j] < gk ? key[j] : 0u);
            }
        }
        __syncwarp();
    }
    next = warp_max(best.k1);
    const int first = __shfl_sync(kFull, ln.first, my_owner);
    return lane < p.k ? first + (int)(P - 1u - (my_key & (P - 1u))) : -1;
}

// --------------------------------------------------- what is too close --
// Where binary32 cannot tell, what lies further from the decision than the
// tolerance is settled, and only the values within it are listed and taken in
// binary64 (which runs at 1/64 of binary32's rate or less: the whole choice
// in it took a warp 30 us).

// Shared memory of one warp: the listed experts and their values' keys.
struct Scratch {
    uint64_t* exact;  // [E], by place in the list
    int* list;        // [E], ascending
    static constexpr int kBytes = 12;  // per expert
    __device__ Scratch(void* base, int E, int warp) {
        char* at = static_cast<char*>(base) + (size_t)warp * ((E + 1) & ~1) * kBytes;
        exact = reinterpret_cast<uint64_t*>(at);
        list = reinterpret_cast<int*>(at + 8 * (size_t)((E + 1) & ~1));
    }
    static size_t bytes(int E, int warps) { return (size_t)warps * ((E + 1) & ~1) * kBytes; }
};

// The list's values in binary64.  zm: the largest logit (softmax).  No
// exchange between lanes but the denominator's.
__device__ __noinline__ void take_in_64(const ScoredArgs& p, int64_t t, int lane, const Scratch& s, int n, float zm) {
    double total = 1.0;
    if (!p.sigmoid && p.bias) {
        total = 0.0;
#pragma unroll 1
        for (int e = lane; e < p.E; e += 32) total += exp((double)logit_of(p, t, e) - (double)zm);
        total = warp_sum(total);
    }
#pragma unroll 1
    for (int i = lane; i < n; i += 32) {
        const int e = s.list[i];
        const float z = logit_of(p, t, e);
        double v = exp(p.sigmoid ? -fabs((double)z) : (double)z - (double)zm);
        v = p.sigmoid ? (z >= 0.0f ? 1.0 : v) / (1.0 + v) : v / total;
        if (p.bias) v += (double)p.bias[e];
        s.exact[i] = order_key(v);
    }
    __syncwarp();
}

// Lists the marked experts of all lanes (bit j: first + j) and takes them in
// binary64; returns their number.
__device__ __forceinline__ int list_in_64(const ScoredArgs& p, int64_t t, int lane, const Lane& ln, uint64_t bits,
                                          const Scratch& s, float zm) {
    const int mine = __popcll(bits);
    int at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += u;
    }
    const int n = __shfl_sync(kFull, at, 31);
    at -= mine;
    __syncwarp();
    for (; bits != 0; bits &= bits - 1) s.list[at++] = ln.first + __ffsll((long long)bits) - 1;
    __syncwarp();
    take_in_64(p, t, lane, s, n, zm);
    return n;
}

// The largest of the warp's magnitudes (their order is their bits').
__device__ __forceinline__ float warp_max_magnitude(float v) { return __uint_as_float(warp_max(__float_as_uint(v))); }

// Whether this lane's group stays (kept: by the keys), where the edge between
// kept and dropped groups is too close.  k1, k2: the group's best two; score,
// edge, dropped: its score, that of the last one kept and of the first one
// not; size: the magnitudes of what its score is the sum of; wide: the
// tolerance by the largest size.
template <int P>
__device__ __forceinline__ bool keep_close_group(const ScoredArgs& p, int64_t t, int lane, const Lane& ln,
                                                 const uint32_t (&key)[P], uint32_t k1, uint32_t k2, uint32_t score,
                                                 float edge, float dropped, float size, float wide, bool kept,
                                                 const Tolerance& tol, const Scratch& s, float zm) {
    const float v = key_value(score);
    const bool is_group = ln.g < p.n_groups;
    // Groups further from the edge than the largest size allows are settled;
    // among the others only their own sizes count.
    const bool near = is_group && !(v - edge > wide) && !(edge - v > wide);
    wide = 2.0f * tol(warp_max_magnitude(near ? size : 0.0f));
    if (edge - dropped > wide) return kept;
    const bool sure = is_group && v > edge && !(v - edge <= wide);
    const bool open = is_group && !sure && !(edge - v > wide);
    const float low = place_value<P>(p.group_top2 && k2 != 0 ? k2 : k1), floor = low - tol(low);
    uint64_t bits = 0;  // the values an open group's score may consist of
#pragma unroll
    for (int j = 0; j < P; ++j)
        if (open && key[j] != 0 && !(place_value<P>(key[j]) < floor)) bits |= 1ull << j;
    const int n = list_in_64(p, t, lane, ln, bits, s, zm);
    uint64_t m1 = 0, m2 = 0;
    for (int i = 0; i < n; ++i)
        if (open && s.list[i] / p.group_size == ln.g) {
            const uint64_t c = s.exact[i];
            m2 = max(m2, min(m1, c));
            m1 = max(m1, c);
        }
    const uint64_t exact = !open ? 0 : p.group_top2 && m2 != 0 ? order_key(key_value(m1) + key_value(m2)) : m1;
    int rank = 0;
    for (int g = 0; g < p.n_groups; ++g) {
        const uint64_t o = __shfl_sync(kFull, exact, g * p.lanes);
        rank += o > exact || (o == exact && g < ln.g);
    }
    const int slots = p.top_groups - __popc(__ballot_sync(kFull, sure && lane % p.lanes == 0));
    return sure || (open && rank < slots);
}

// The k picks where the edge between the k-th and the next is too close:
// my_id and my_key as pick() left them (the picks beyond doubt come first).
template <int P>
__device__ __forceinline__ int pick_close(const ScoredArgs& p, int64_t t, int lane, const Lane& ln,
                                          const uint32_t (&key)[P], bool kept, int my_id, uint32_t my_key,
                                          uint32_t edge_key, const Tolerance& tol, const Scratch& s, float zm) {
    const float edge = place_value<P>(edge_key), wide = tol(edge);
    auto above = [&](uint32_t k) { return place_value<P>(k) > edge && !(place_value<P>(k) - edge <= wide); };
    uint64_t bits = 0;
#pragma unroll
    for (int j = 0; j < P; ++j)
        if (kept && key[j] != 0 && !above(key[j]) && !(edge - place_value<P>(key[j]) > wide)) bits |= 1ull << j;
    const int n_sure = __popc(__ballot_sync(kFull, my_id >= 0 && above(my_key)));
    const int n = list_in_64(p, t, lane, ln, bits, s, zm);
    uint64_t last = ~0ull;
    int last_at = -1;
    for (int i = n_sure; i < p.k; ++i) {
        // what follows (last, last_at): largest first, the lowest on ties
        uint64_t best = 0;
        int at = 0x7fffffff;
        for (int q = lane; q < n; q += 32) {
            const uint64_t c = s.exact[q];
            if (c > best && (c < last || (c == last && q > last_at))) {
                best = c;
                at = q;
            }
        }
        last = warp_max(best);
        last_at = (int)__reduce_min_sync(kFull, best == last ? (unsigned)at : 0x7fffffffu);
        if (lane == i) my_id = last_at < n ? s.list[last_at] : -1;
    }
    __syncwarp();
    return my_id;
}

// The k picks where the last of them are experts taken out (-inf): those go
// by id, but keys of different lanes order equal values by place first, and
// a difference of infinities is no measure of closeness.
template <int P>
__device__ __forceinline__ int pick_taken_out(const ScoredArgs& p, int lane, const Lane& ln, const uint32_t (&key)[P],
                                              bool kept, int my_id, uint32_t my_key, const Scratch& s) {
    auto is_out = [](uint32_t k) { return place_value<P>(k) == -CUDART_INF_F; };
    uint64_t bits = 0;
#pragma unroll
    for (int j = 0; j < P; ++j)
        if (kept && key[j] != 0 && is_out(key[j])) bits |= 1ull << j;
    const int n_left = __popc(__ballot_sync(kFull, my_id >= 0 && !is_out(my_key)));
    const int mine = __popcll(bits);
    int at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += u;
    }
    at -= mine;
    for (; bits != 0 && at < p.k; bits &= bits - 1) s.list[at++] = ln.first + __ffsll((long long)bits) - 1;
    __syncwarp();
    if (lane >= n_left && lane < p.k) my_id = s.list[lane - n_left];
    __syncwarp();
    return my_id;
}

// One token by one warp: lane s < k gets the s-th pick's id, the slot it has
// in ascending order of ids, and its weight.
struct Pick {
    int id, slot;
    float w;
};
template <int P, bool FULL>
__device__ __forceinline__ Pick route_token(const ScoredArgs& p, int64_t t, int lane, const Lane& ln,
                                            const float (&b)[P], const Scratch& scratch) {
    float z[P];
    load_logits<P, FULL>(p, t, ln, z);
    if (p.z_out) {
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (has<P, FULL>(ln, j)) p.z_out[t * p.E + ln.first + j] = z[j];
    }
    uint32_t key[P];
    float zm, total;
    bool finite;
    const Tolerance tol = choice_keys<P, FULL>(p, ln, z, b, key, zm, total, finite);
    if (!finite && lane == 0) atomicOr(p.err, DERR_NONFINITE_LOGIT);
    // (a difference of infinities is NaN and never close)
    auto close = [&](float a, float b) { return finite && a - b <= tol(a); };
    Best3 best;
#pragma unroll
    for (int j = 0; j < P; ++j) best.add(key[j]);
    bool kept = true;
    if (p.top_groups < p.n_groups) {
        // the group's best two and score, by all its lanes
        uint32_t k1 = best.k1, k2 = best.k2;
        for (int o = 1; o < p.lanes; o <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(kFull, k1, o), o2 = __shfl_xor_sync(kFull, k2, o);
            k2 = max(min(k1, o1), max(k2, o2));
            k1 = max(k1, o1);
        }
        const bool is_group = ln.g < p.n_groups;
        const float top = place_value<P>(k1), second = p.group_top2 && k2 != 0 ? place_value<P>(k2) : 0.0f;
        uint32_t score = order_key(p.group_top2 && k2 != 0 ? top + second : top);
        // a sum is as uncertain as its terms are large, but one of -inf is certain
        float size = fabsf(top) + fabsf(second);
        if (!is_group) score = 0;
        if (!is_group || top == -CUDART_INF_F || second == -CUDART_INF_F) size = 0.0f;
        int rank = 0;  // groups before this one: larger, or as large and lower
        for (int g0 = 0; g0 < p.n_groups; g0 += 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // (0 beyond the last group)
                const int g = g0 + i;
                const uint32_t other = g * p.lanes < 32 ? __shfl_sync(kFull, score, g * p.lanes) : 0u;
                rank += other > score || (other == score && g < ln.g);
            }
        }
        kept = is_group && rank < p.top_groups;
        const uint32_t edge_key = ~warp_max(kept ? ~score : 0u), first_out = warp_max(is_group && !kept ? score : 0u);
        const float edge = key_value(edge_key), dropped = key_value(first_out);
        const float wide = 2.0f * tol(warp_max_magnitude(size));
        if (first_out != 0 && finite && edge - dropped <= wide)
            kept = keep_close_group<P>(p, t, lane, ln, key, k1, k2, score, edge, dropped, size, wide, kept, tol, scratch, zm);
        if (!kept) best.k1 = best.k2 = best.k3 = 0;
    }
    uint32_t my_key, last, next;
    int my_id = pick<P>(p, key, best, ln, lane, my_key, last, next);
    if (place_value<P>(last) == -CUDART_INF_F)
        my_id = pick_taken_out<P>(p, lane, ln, key, kept, my_id, my_key, scratch);
    else if (next != 0 && close(place_value<P>(last), place_value<P>(next)))
        my_id = pick_close<P>(p, t, lane, ln, key, kept, my_id, my_key, last, tol, scratch, zm);

    // weights, by lane s < k for its own pick
    const bool mine = lane < p.k && my_id >= 0;
    const float zc = mine ? logit_of(p, t, my_id) : -CUDART_INF_F;
    const bool out = !mine || (p.bias && p.bias[my_id] == -CUDART_INF_F);  // taken out: weight 0
    float top_z = zm, sum = total;
    if (p.renorm) top_z = warp_max(out ? -CUDART_INF_F : zc);
    // sigmoid: e^min(z, 0) / (1 + e^-|z|).  Renormalised, both kinds relative
    // to the largest chosen one, so that nothing underflows.
    const float shift = p.sigmoid ? (p.renorm ? fminf(top_z, 0.0f) : 0.0f) : top_z;
    float w = out ? 0.0f : exp2_fast(kLog2e * ((p.sigmoid ? fminf(zc, 0.0f) : zc) - shift));
    if (p.sigmoid) w *= rcp_fast(1.0f + exp2_fast(-kLog2e * fabsf(zc)));
    if (p.renorm) sum = warp_sum(w);
    if (p.renorm || !p.sigmoid) w *= sum > 0.0f ? rcp_fast(sum) : 0.0f;
    w *= p.scale;
    // rank of my id among the chosen ids -> ascending-id slot
    int slot = 0;
    const unsigned order = mine ? (unsigned)my_id : 0xffffffffu;
    for (int s0 = 0; s0 < p.k; s0 += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) slot += __shfl_sync(kFull, order, s0 + i) < order;
    }
    if (mine) {
        p.ids[t * p.k + slot] = my_id;
        p.w[t * p.k + slot] = w;
    }
    return Pick{my_id, slot, w};
}

// ------------------------------------------------------------- grouping --
// The pairs are taken in chunks of whole tokens, at most kChunk pairs each:
//   select   a warp per token chooses, and counts its pairs by chunk and
//            expert: hist[chunk][e], zeroed by the router GEMM's kernel
//   place    a block per chunk adds up the counts of all chunks (its base is
//            what lies before it), and ranks its own pairs
// or, for up to 64 tokens, one kernel for both: a block that chooses and
// places, a warp per token, and above 8 tokens a cluster of 8 blocks that
// choose and send their counts and ids to the first block, which places.
// Each pair's row is the stable one (ascending flat index within an expert).
constexpr int kChunk = 1024;
constexpr int kSelectWarps = 8;
constexpr int kOneCluster = 8;  // blocks of the one-chunk kernel
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
#pragma unroll 8
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
#pragma unroll 16
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

// The lane's bias, before the kernel before this one (the router GEMM) is
// done: it lets this one start only after everything before it is.
template <int P, bool FULL>
__device__ __forceinline__ void early_bias(const ScoredArgs& p, const Lane& ln, float (&b)[P]) {
    if (p.bias) load_run<P, FULL>(p.bias, ln, b);
}

template <int P, bool FULL>
__global__ void __launch_bounds__(32 * kSelectWarps, P <= 8 ? 3 : P <= 16 ? 2 : 1)
    scored_select_kernel(const __grid_constant__ ScoredArgs p) {
    extern __shared__ __align__(16) char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Lane ln(p, lane);
    float bias[P];
    early_bias<P, FULL>(p, ln, bias);
    wait_for_previous_kernel();
    const int t = blockIdx.x * kSelectWarps + warp;
    if (t >= p.T) return;
    const Pick pick = route_token<P, FULL>(p, t, lane, ln, bias, Scratch(smem, p.E, warp));
    // not earlier: the placing blocks would take slots from waiting tokens
    // (8192 tokens of 256 experts: 0.3 to 3 us of 48)
    let_next_kernel_start();
    if (lane < p.k && pick.id >= 0) atomicAdd(p.hist + (int64_t)(t / p.chunk_tokens) * p.E + pick.id, 1);
}

// One chunk.  The blocks of a cluster (up to 8 tokens: a single block, ALONE)
// send their picks to the first one's shared memory, which places the pairs,
// a round of 256 at a time; base[e] moves on by the round's pairs.
template <int P, bool FULL, bool ALONE>
__global__ void __launch_bounds__(32 * kSelectWarps, P <= 16 ? 2 : 1)
    scored_one_kernel(const __grid_constant__ ScoredArgs p) {
    constexpr int kThreads = 32 * kSelectWarps, kPer = DWDP_MAX_EXPERTS / kThreads;
    extern __shared__ __align__(16) char smem[];
    __shared__ int base[DWDP_MAX_EXPERTS], sid[kChunk];
    __shared__ int tmp[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int e = tid; e < p.E; e += kThreads) base[e] = 0;
    const Lane ln(p, lane);
    float bias[P];
    early_bias<P, FULL>(p, ln, bias);
    wait_for_previous_kernel();
    let_next_kernel_start();
    __syncwarp();  // the cluster's barrier is the whole warp's; lanes zeroed more or fewer counts
    if constexpr (ALONE) __syncthreads();
    else cluster_sync();
    for (int t = blockIdx.x * kSelectWarps + warp; t < p.T; t += gridDim.x * kSelectWarps) {
        const Pick pick = route_token<P, FULL>(p, t, lane, ln, bias, Scratch(smem, p.E, warp));
        if (lane < p.k && pick.id >= 0) {
            if constexpr (ALONE) {
                atomicAdd(base + pick.id, 1);
                sid[t * p.k + pick.slot] = pick.id;
            } else {
                uint32_t count_at, id_at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                             : "=r"(count_at)
                             : "r"((uint32_t)__cvta_generic_to_shared(base + pick.id)));
                asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                             : "=r"(id_at)
                             : "r"((uint32_t)__cvta_generic_to_shared(sid + t * p.k + pick.slot)));
                asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], 1;" ::"r"(count_at) : "memory");
                asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(id_at), "r"(pick.id) : "memory");
            }
        }
        __syncwarp();
    }
    __syncwarp();
    if constexpr (ALONE) __syncthreads();
    else cluster_sync();
    if (blockIdx.x != 0) return;
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
        const int e = f < n ? sid[f] : -1;
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

// most: what any call of the kernel may ask for.  The limit belongs to the
// kernel, not to the launch: set to this call's size it could refuse another
// host thread's larger launch.
template <class F, class... A>
cudaError_t launch(F kernel, int grid, int threads, size_t smem, size_t most, bool cluster, cudaStream_t s, A... args) {
    if (smem > 36 << 10) {  // beside the static part, beyond what a launch gets unasked
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;  // the whole grid
    at[1].val.clusterDim.x = grid;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

template <int P, bool FULL>
cudaError_t launch_form(const ScoredArgs& p, cudaStream_t s) {
    constexpr int threads = 32 * kSelectWarps;
    const size_t smem = Scratch::bytes(p.E, kSelectWarps), most = Scratch::bytes(DWDP_MAX_EXPERTS, kSelectWarps);
    if (p.in_one && p.T <= kSelectWarps)
        return launch(scored_one_kernel<P, FULL, true>, 1, threads, smem, most, false, s, p);
    if (p.in_one) return launch(scored_one_kernel<P, FULL, false>, kOneCluster, threads, smem, most, true, s, p);
    const int n_chunks = p.chunks;
    cudaError_t e =
        launch(scored_select_kernel<P, FULL>, (p.T + kSelectWarps - 1) / kSelectWarps, threads, smem, most, false, s, p);
    if (e != cudaSuccess) return e;
    const size_t place_smem = (size_t)p.E * 36, place_most = (size_t)DWDP_MAX_EXPERTS * 36;
    if (n_chunks <= kSelfScanChunks)
        return launch(scored_place_kernel<false>, n_chunks, kChunk, place_smem, place_most, false, s, p, n_chunks);
    e = launch_chunk_scan(p.hist, n_chunks, p.E, p.counts, p.offsets, s);
    if (e != cudaSuccess) return e;
    return launch(scored_place_kernel<true>, n_chunks, kChunk, place_smem, place_most, false, s, p, n_chunks);
}

template <int P>
cudaError_t launch_per_lane(const ScoredArgs& p, cudaStream_t s) {
    if constexpr (P <= 32)
        if (p.per_lane == P && 32 * P == p.E && p.lanes * P == p.group_size) return launch_form<P, true>(p, s);
    return launch_form<P, false>(p, s);
}

}  // namespace

int scored_chunks(int64_t T, int64_t k) {
    const int64_t tokens = kChunk / k;
    return (int)((T + tokens - 1) / tokens);
}

// One kernel chooses and places: one chunk, one plane, and a token for each of
// the cluster's 64 warps at most.  Routing to 8 of 256 experts, H = 7168, one
// kernel / two, us: 32 tokens 9.5 / 9.7, 64 11.4 / 11.6, 128 16.9 / 14.3 (with
// 8 planes 24); 2 of 16: 64 7.2 / 7.7, 512 18.1 / 9.0.
bool scored_in_one(int64_t T, int64_t k, int parts) {
    return parts == 1 && T <= kSelectWarps * kOneCluster && scored_chunks(T, k) == 1;
}

cudaError_t launch_scored_choice(ScoredArgs& p, cudaStream_t s) {
    if (p.T <= 0) return cudaSuccess;
    p.lanes = 1;
    while (p.lanes * 2 * p.n_groups <= 32) p.lanes *= 2;
    p.group_size = p.E / p.n_groups;
    p.per_lane = (p.group_size + p.lanes - 1) / p.lanes;
    p.chunk_tokens = kChunk / p.k;
    if (p.per_lane <= 1) return launch_per_lane<1>(p, s);
    if (p.per_lane <= 2) return launch_per_lane<2>(p, s);
    if (p.per_lane <= 4) return launch_per_lane<4>(p, s);
    if (p.per_lane <= 8) return launch_per_lane<8>(p, s);
    if (p.per_lane <= 16) return launch_per_lane<16>(p, s);
    if (p.per_lane <= 32) return launch_per_lane<32>(p, s);
    return launch_per_lane<64>(p, s);
}

}  // namespace dwdp
