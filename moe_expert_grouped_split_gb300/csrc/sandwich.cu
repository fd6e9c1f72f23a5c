// sandwich.cu: the norms after and before a block with the block's gate and
// the residual's scale (dwdp_sandwich_norm) and their gradients
// (dwdp_sandwich_norm_grad), memory-bound.
//
// Forward, per row: x stays in registers for its sum of squares, h for its
// own; two reductions a row, which also carry the largest magnitudes that the
// E4M3 rows' scales need.  Backward, per row: one reduction; the weights' and
// gates' gradients are sums over rows, which each block keeps in registers for
// the rows it takes, one after the other, and a second kernel adds up in the
// blocks' order: the same bits from run to run.
#include <math_constants.h>

#include <algorithm>

#include "dwdp_internal.h"
#include "row_ops.h"
#include "tc_ops.h"

namespace dwdp {
namespace {

// As in norm.cu: a sum of squares beyond the limit is taken again on values
// scaled by 2^-80.  (1 / rms is then below 2^-40; 2^-128 at its least, whose
// subnormal binary32 still has 21 bits.)
constexpr float kSquaresLimit = 1e38f;
constexpr float kDownScale = 0x1p-80f;
constexpr float kMinCodeMax = 0x1p-100f;

// The group of `row`: offsets[g] <= row < offsets[g + 1], the last such g; -1
// where there is none.  The whole warp together.
__device__ __forceinline__ int group_of(const int32_t* offsets, int n_groups, int64_t row) {
    const int g = last_not_above(offsets, n_groups + 1, row);
    return g < n_groups ? g : -1;
}

// (sum, max, max) over the block; every thread gets them.  `turn` alternates
// between two buffers, so one barrier is enough.
__device__ __forceinline__ float3 block_sum_max2(float s, float a, float b, float4 (*red)[32], int& turn) {
    warp_sum_max<false>(s, a);
    a = warp_max(a);
    b = warp_max(b);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return make_float3(s, a, b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float4* r = red[turn];
    turn ^= 1;
    if (lane == 0) r[warp] = make_float4(s, a, b, 0.0f);
    __syncthreads();
    const float4 v = lane < nw ? r[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    s = v.x;
    warp_sum_max<false>(s, a);
    return make_float3(s, warp_max(v.y), warp_max(v.z));
}

// Two binary32 values in one 64-bit register, one instruction for both.
using pair = unsigned long long;
__device__ __forceinline__ pair two(float a, float b) {
    pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ pair two(float a) { return two(a, a); }
__device__ __forceinline__ float2 apart(pair v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ pair fma2(pair a, pair b, pair c) {
    pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ pair mul2(pair a, pair b) {
    pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
using four = pair[4];  // a vector's 8 elements
__device__ __forceinline__ void unpack4(uint4 q, four& f) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = two(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack4(const four& f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = apart(f[i]);
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load4(const ulonglong2* at, int far, four& f) {
    const ulonglong2 a = at[0], b = at[far];
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}
__device__ __forceinline__ float sum_of(pair v) {
    const float2 f = apart(v);
    return f.x + f.y;
}
__device__ __forceinline__ float max_of(const four& v, float m) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float2 f = apart(v[c]);
        m = max_nan(max_nan(m, fabsf(f.x)), fabsf(f.y));
    }
    return m;
}

__device__ __forceinline__ uint2 codes8(const four& v, float inv) {
    uint32_t q[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) q[c] = __nv_cvt_float2_to_fp8x2(apart(mul2(v[c], two(inv))), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}

// 448 / the largest magnitude (0 for zeros), and the scale that goes with it.
__device__ __forceinline__ float code_factor(float m) { return m == 0.0f ? 0.0f : 448.0f * rcp(max_nan(m, kMinCodeMax)); }
__device__ __forceinline__ float code_scale(float m) { return m == 0.0f ? 1.0f : max_nan(m, kMinCodeMax) / 448.0f; }

// What is asked of a forward call (the rest are pointers that may be null).
template <bool POST_, bool PRE_, bool CODES_, bool KEPT_>
struct Asked {
    static constexpr bool POST = POST_, PRE = PRE_, CODES = CODES_, KEPT = KEPT_;
};

// Waits for the bulk copies of row r of `rows`, in stage `stage`, 2 s at most.
// A thread whose wait ran out gets a `poison` of NaN, else 0: it waits for no
// other row, all that it writes from there on is NaN (these calls have no error
// word), and the one that asks for rows asks for no more.  That one also gives
// those that are on their way 2 s to land, as the shared memory goes to another block
// after this one.
template <int STAGES>
__device__ __forceinline__ void wait_row(uint32_t full, int r, int rows, int stage, uint32_t parity, float& poison) {
    if (poison != 0.0f || mbar_try_wait(full + 8 * stage, parity)) return;
    uint64_t since = global_timer();
    while (!mbar_try_wait(full + 8 * stage, parity)) {
        if (global_timer() - since <= kWaitLimitNs) continue;
        poison = CUDART_NAN_F;
        if (threadIdx.x != 0) return;
        since = global_timer();
        for (const int to = min(r + STAGES, rows); r < to; ++r) {
            while (!mbar_try_wait(full + 8 * stage, parity) && global_timer() - since <= kWaitLimitNs) {
            }
            if (++stage == STAGES) {
                stage = 0;
                parity ^= 1;
            }
        }
        return;
    }
}

// c gate post of a vector's elements.
__device__ __forceinline__ void block_factor(const SandwichArgs& p, const uint4* gate, const uint4* post, int i, four& f) {
#pragma unroll
    for (int c = 0; c < 4; ++c) f[c] = two(p.block_scale);
    four w;
    if (gate) {
        unpack4(__ldg(gate + i), w);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = mul2(f[c], w[c]);
    }
    if (post) {
        unpack4(__ldg(post + i), w);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = mul2(f[c], w[c]);
    }
}

// One row of which the thread has VPT vectors: x and the residual (zeros where
// there is nothing), factor(j, f) = c gate post and pre.  vec: the first
// one's place among all vectors, the others n on each; held[j]: to be stored.
// poison: 0, or NaN for all outputs.
template <class ASK, int VPT, class Factor>
__device__ __forceinline__ void sandwich_row(const SandwichArgs& p, int64_t row, int64_t vec, int n, const bool (&held)[VPT],
                                             const uint4 (&x)[VPT], const uint4 (&r)[VPT], const uint4 (&pre)[VPT],
                                             Factor factor, float4 (*red)[32], int& turn, float poison = 0.0f) {
    float rx = 1.0f, x_inv = 0.0f;
    const bool first = threadIdx.x == 0;
    // 1 / rms from the sum of squares; where that passes the limit it is taken
    // again on scaled values, squares(by): rare, and the whole block agrees
    auto rms = [&](float ss, auto squares) {
        float scaled = 1.0f;
        if (!(ss < kSquaresLimit)) {
            scaled = kDownScale;
            pair again = two(poison);
            squares(two(scaled), again);
            ss = block_sum_max2(sum_of(again), 0.0f, 0.0f, red, turn).x;
        }
        return rsqrtf(fmaf(ss, p.one_nth, p.eps * scaled * scaled)) * scaled;
    };
    if constexpr (ASK::POST || ASK::KEPT) {
        pair ss = two(poison);
        float ax = poison;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            four f;
            unpack4(x[j], f);
            if constexpr (ASK::POST) {
#pragma unroll
                for (int c = 0; c < 4; ++c) ss = fma2(f[c], f[c], ss);
            }
            if constexpr (ASK::KEPT) ax = max_of(f, ax);
        }
        const float3 sums = block_sum_max2(sum_of(ss), ax, 0.0f, red, turn);
        if constexpr (ASK::POST)
            rx = rms(sums.x, [&](pair by, pair& again) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    four f;
                    unpack4(x[j], f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        f[c] = mul2(f[c], by);
                        again = fma2(f[c], f[c], again);
                    }
                }
            });
        if constexpr (ASK::KEPT) {
            x_inv = code_factor(sums.y);
            if (first && p.x_scale) p.x_scale[row] = code_scale(sums.y);
        }
    }
    const pair by_residual = two(p.residual_scale + poison);
    four h[VPT];
    pair ss = 0;
    float ah = 0.0f, ay = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        four f, w;
        unpack4(x[j], f);
        if (ASK::KEPT && p.x_codes && held[j]) p.x_codes[vec + j * n] = codes8(f, x_inv);
        factor(j, w);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = mul2(f[c], ASK::POST ? mul2(two(rx), w[c]) : w[c]);
        unpack4(r[j], w);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            h[j][c] = fma2(by_residual, w[c], f[c]);
            if constexpr (ASK::PRE) ss = fma2(h[j][c], h[j][c], ss);
        }
        if constexpr (ASK::KEPT) ah = max_of(h[j], ah);
        if constexpr (ASK::CODES) {
            unpack4(pre[j], w);
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = mul2(h[j][c], w[c]);
            ay = max_of(w, ay);
        }
        if (p.residual_out && held[j]) p.residual_out[vec + j * n] = pack4(h[j]);
    }
    float rh = 1.0f, h_inv = 0.0f, y_inv = 0.0f;
    if constexpr (ASK::PRE || ASK::KEPT) {
        const float3 sums = block_sum_max2(sum_of(ss), ah, ay, red, turn);
        if constexpr (ASK::PRE)
            rh = rms(sums.x, [&](pair by, pair& again) {
#pragma unroll
                for (int j = 0; j < VPT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const pair v = mul2(h[j][c], by);
                        again = fma2(v, v, again);
                    }
            });
        if constexpr (ASK::KEPT) {
            h_inv = code_factor(sums.y);
            if (first && p.h_scale) p.h_scale[row] = code_scale(sums.y);
        }
        if constexpr (ASK::CODES) {
            y_inv = code_factor(sums.z);
            if (first) p.row_scale[row] = sums.z == 0.0f ? 1.0f : code_scale(sums.z) * rh;
        }
    }
    if (first && p.rstd) p.rstd[row] = make_float2(rx, rh);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (ASK::KEPT && p.h_codes && held[j]) p.h_codes[vec + j * n] = codes8(h[j], h_inv);
        if constexpr (ASK::PRE) {
            four w, y;
            unpack4(pre[j], w);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[c] = mul2(w[c], h[j][c]);
                y[c] = mul2(w[c], two(rh));
            }
            if (held[j]) p.out[vec + j * n] = pack4(y);
            if (ASK::CODES && held[j]) p.codes[vec + j * n] = codes8(w, y_inv);
        }
    }
}

// One block per row; thread i holds the row's vectors i, i + blockDim.x, ...
template <class ASK, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 448 ? 2 : 1) sandwich_norm_kernel(const __grid_constant__ SandwichArgs p) {
    __shared__ float4 red[2][32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int64_t row = blockIdx.x;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 x[VPT], r[VPT], pre[VPT];
    bool held[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        held[j] = i < p.nv;
        x[j] = held[j] ? p.x[row * p.x_vecs + i] : zero;
        r[j] = held[j] && p.residual ? p.residual[row * p.nv + i] : zero;
        pre[j] = ASK::PRE && held[j] ? __ldg(p.pre + i) : zero;
    }
    const uint4* gate = p.gate;
    if (p.row_offsets) {
        const int g = group_of(p.row_offsets, p.n_groups, row);
        if (g < 0) return;  // the whole block
        gate += (int64_t)g * p.nv;
    }
    auto factor = [&](int j, four& f) {
        if (held[j]) {
            block_factor(p, gate, ASK::POST ? p.post : nullptr, threadIdx.x + j * blockDim.x, f);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) f[c] = 0;
        }
    };
    int turn = 0;
    sandwich_row<ASK, VPT>(p, row, row * p.nv + threadIdx.x, blockDim.x, held, x, r, pre, factor, red, turn);
}

// Many wide rows: a block stays and takes rows [blockIdx.x chunk, + chunk) in order.
// One thread asks for whole rows, STAGES - 1 ahead, into shared memory, where c
// gate post of the group lies too; what is never fetched is zero there.
constexpr int kNormVecs = 2, kNormSmem = (228 << 10) / 2 - 2048;  // of a block: two fit an SM
template <class ASK, int STAGES>
__global__ void __launch_bounds__(512, 2) sandwich_stream_kernel(const __grid_constant__ SandwichArgs p) {
    constexpr int VPT = kNormVecs;
    extern __shared__ __align__(16) char smem[];
    __shared__ float4 red[2][32];  // 16 warps at most: its end holds the stages' barriers, that their rows have come
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tid = threadIdx.x, n = blockDim.x;
    const int64_t lo = (int64_t)blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.rows);
    const bool held[VPT] = {tid < p.nv, tid + n < p.nv};
    const int stage_bytes = 2 * VPT * n * 16;
    char* const own = smem + tid * 16;
    ulonglong2* const factors = reinterpret_cast<ulonglong2*>(smem + STAGES * stage_bytes) + tid;
    const uint32_t full = smem_u32(&red[1][30]);
    float poison = 0.0f;
    auto fetch = [&](int64_t row, int stage) {
        if (tid != 0 || row >= hi || poison != 0.0f) return;
        const uint32_t to = smem_u32(smem) + stage * stage_bytes, bar = full + 8 * stage, bytes = p.nv * 16;
        mbar_arrive_expect_tx(bar, p.residual ? 2 * bytes : bytes);
        bulk_load(to, p.x + row * p.x_vecs, bytes, bar);
        if (p.residual) bulk_load(to + VPT * n * 16, p.residual + row * p.nv, bytes, bar);
    };
    uint4 pre[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        pre[j] = ASK::PRE && held[j] ? __ldg(p.pre + tid + j * n) : zero;
        if (held[j] && p.residual) continue;
        for (int at = 0; at < STAGES * stage_bytes; at += stage_bytes) {
            *reinterpret_cast<uint4*>(own + at + (VPT + j) * n * 16) = zero;
            if (!held[j]) *reinterpret_cast<uint4*>(own + at + j * n * 16) = zero;
        }
        if (!held[j]) factors[2 * j * n] = factors[(2 * j + 1) * n] = make_ulonglong2(0, 0);
    }
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(full + 8 * s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STAGES; ++s) fetch(lo + s, s);
    auto open_group = [&](int group) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (!held[j]) continue;
            four f;
            block_factor(p, p.gate ? p.gate + (int64_t)group * p.nv : nullptr, ASK::POST ? p.post : nullptr, tid + j * n, f);
            factors[2 * j * n] = make_ulonglong2(f[0], f[1]);
            factors[(2 * j + 1) * n] = make_ulonglong2(f[2], f[3]);
        }
    };
    bool open = !p.row_offsets;
    if (open) open_group(0);
    const int rows = (int)(hi - lo);
    int change = open ? rows : 0, stage = 0, parity = 0, turn = 0;
    for (int i = 0; i < rows; ++i) {
        wait_row<STAGES>(full, i, rows, stage, parity, poison);
        if (i == change) {
            const int group = group_of(p.row_offsets, p.n_groups, lo + i);
            open = group >= 0;
            change = i + 1;
            if (open) {
                change = (int)min(max((int64_t)p.row_offsets[group + 1] - lo, (int64_t)change), (int64_t)rows);
                open_group(group);
            }
        }
        if (open) {
            const char* const in = own + stage * stage_bytes;
            uint4 x[VPT], r[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                x[j] = *reinterpret_cast<const uint4*>(in + j * n * 16);
                r[j] = *reinterpret_cast<const uint4*>(in + (VPT + j) * n * 16);
            }
            sandwich_row<ASK, VPT>(
                p, lo + i, (lo + i) * p.nv + tid, n, held, x, r, pre, [&](int j, four& f) { load4(factors + 2 * j * n, n, f); }, red,
                turn, poison);
        }
        // everybody has taken his part of the stage: they were at a barrier of
        // the row since, where it has one (and nobody is a phase of the stage's
        // own barrier behind)
        if (!open || !(ASK::POST || ASK::PRE || ASK::KEPT))
            __syncthreads();
        else
            __syncwarp();  // a block of one warp
        fetch(lo + i + STAGES, stage);
        if (++stage == STAGES) {
            stage = 0;
            parity ^= 1;
        }
    }
}

// ------------------------------------------------------------ gradients --
// As wait_row above for the gradients' rows, in two parts and without a value to
// poison with: one form for both kernels costs either the norm 8% (8192 x 7168,
// rows kept: 107 us for 99) or the gradients 20% (138 for 113, spills).
__device__ __forceinline__ void wait_row(uint32_t bar, uint32_t parity, bool& lost) {
    if (lost || mbar_try_wait(bar, parity)) return;
    const uint64_t since = global_timer();
    while (!lost && !mbar_try_wait(bar, parity)) lost = global_timer() - since > kWaitLimitNs;
}
// For the thread that asked for them, at the end: rows `from` .. `to` - 1 were never seen.
__device__ __forceinline__ void wait_lost_rows(uint32_t full, int stages, int from, int to) {
    const uint64_t since = global_timer();
    for (int r = from; r < to; ++r)
        while (!mbar_try_wait(full + 8 * (r % stages), r / stages & 1) && global_timer() - since <= kWaitLimitNs) {
        }
}

// How a row was kept.
enum Kept : int { KEPT_NOT, KEPT_BF16, KEPT_E4M3 };
__host__ __device__ constexpr int kept_bytes(int k) { return k == KEPT_E4M3 ? 8 : k == KEPT_BF16 ? 16 : 0; }

// 8 elements of a kept row times `by`.
template <int K>
__device__ __forceinline__ void values(const char* at, pair by, four& f) {
    if constexpr (K == KEPT_E4M3) {
        const uint2 q = *reinterpret_cast<const uint2*>(at);
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw v =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> ((i & 1) * 16)), __NV_E4M3);
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&v));
            f[i] = two(t.x, t.y);
        }
    } else {
        unpack4(*reinterpret_cast<const uint4*>(at), f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], by);
}

// The sums of a, b and c over the `size` blocks (4 at most) that share a row,
// for every thread.  A warp's three sums together: half of the lanes go on
// with each value, and eight lanes end with each, one of them for each block.
// Rows take the two halves of red ([2][size][warps][4]) in turn, so one
// barrier is enough.  16 warps at most.
template <bool SHARED>
__device__ __forceinline__ float3 row_sums(float a, float b, float c, float* red, int& turn, int size) {
    constexpr uint32_t all = 0xffffffffu;
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const bool upper = lane & 16, odd = lane & 8;
    float u = (upper ? c : a) + __shfl_xor_sync(all, upper ? a : c, 16);
    float v = (upper ? 0.0f : b) + __shfl_xor_sync(all, upper ? b : 0.0f, 16);
    float s = (odd ? v : u) + __shfl_xor_sync(all, odd ? u : v, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(all, s, o);
    // lanes 8 i .. 8 i + 7: value i
    const int warp = threadIdx.x >> 5, w = lane & 7, i = lane >> 3;
    if (SHARED) {
        float* r = red + turn * size * nw * 4;
        turn ^= 1;
        if (w < size) {
            uint32_t at = (uint32_t)__cvta_generic_to_shared(r + (cluster_ctarank() * nw + warp) * 4 + i);
            asm("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(w));
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(s) : "memory");
        }
        __syncwarp();  // the cluster's barrier is the whole warp's
        cluster_sync();
        s = 0.0f;
        for (int e = w; e < size * nw; e += 8) s += r[e * 4 + i];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(all, s, o);
    } else if (nw > 1) {
        float* r = red + turn * 64;
        turn ^= 1;
        if (w == 0) r[warp * 4 + i] = s;
        __syncthreads();
        s = (w < nw ? r[w * 4 + i] : 0.0f) + (w + 8 < nw ? r[(w + 8) * 4 + i] : 0.0f);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(all, s, o);
    }
    return make_float3(__shfl_sync(all, s, 0), __shfl_sync(all, s, 8), __shfl_sync(all, s, 16));
}

__device__ __forceinline__ void store4(float* to, const four& f) {
    reinterpret_cast<ulonglong2*>(to)[0] = make_ulonglong2(f[0], f[1]);
    reinterpret_cast<ulonglong2*>(to)[1] = make_ulonglong2(f[2], f[3]);
}

constexpr int kGradVecs = 2, kGradStages = 3, kGradSmem = (227 << 10) - 1024;

// A block takes rows [unit chunk, + chunk) in order; thread i holds the row's
// vectors i and i + blockDim.x and their columns' sums.  Rows of more than
// 8192 elements are shared by a cluster of blocks, each with its part of the
// columns (SHARED).  Of the weights' gradients only two sums a column have to
// be kept while rows go by (HBM bounds this only if a row costs a warp few
// enough instructions: 128 registers a thread leave an SM 16 warps): dout hhat, and S = dh xhat since the group began, as dgate = c post S and
// dpost_weight = sum over groups of c gate S.  The rows kGradStages ahead are
// on their way into shared memory.  One reduction a row: with e = dres + rh gy
// and q = c gate post xhat,
//   mean(gn xhat) = mean(q e) - rh mean(gy hhat) mean(q hhat).
// partial [units][4][H]: the sums for pre and post, and S of the group that
// was begun before the unit's rows and of the one that goes on after them
// (a group whose rows are all here goes to dgate at once).  With one group
// for all rows its S takes post's place.
// X, HK: how x and h were kept (HK KEPT_NOT: no pre norm); POST: a post norm;
// THREADS at most (448: the compiler's order of things is 5% faster than for 512).
// BULK: one thread asks for whole rows (16-byte addresses and sizes: bf16, or
// codes of H a multiple of 16), at the end of the row whose stage they take; else
// every thread copies what it will read itself, as soon as it has taken its
// part of that row.
template <int X, int HK, bool POST, int THREADS, bool SHARED, bool BULK>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 2 : 1) sandwich_grad_kernel(const __grid_constant__ SandwichGradArgs p) {
    constexpr int VPT = kGradVecs, kX = kept_bytes(X), kH = kept_bytes(HK);
    constexpr bool PRE = HK != KEPT_NOT;
    extern __shared__ __align__(16) char smem[];
    __shared__ uint64_t full_bars[kGradStages];  // BULK: of the stages, when their rows have come
    const int tid = threadIdx.x, n = blockDim.x, lane = tid & 31;
    const int size = SHARED ? p.size : 1, rank = SHARED ? (int)cluster_ctarank() : 0, unit = blockIdx.x / size;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int64_t lo = (int64_t)unit * p.chunk, hi = min(lo + p.chunk, p.rows);
    const int H = p.nv * 8, own_vecs = SHARED ? min(p.nv - rank * p.share, p.share) : p.nv;
    const int first = SHARED ? rank * p.share + tid : tid;  // this thread's first vector
    // a stage: vectors of dout, dres, x and h; behind the stages c gate post
    const int vecs = n * VPT, stage_bytes = vecs * (kX + kH + 32), all_stages = kGradStages * stage_bytes;
    char* const own = smem + tid * 16;
    char* const own_x = smem + vecs * 32 + tid * kX;
    char* const own_h = smem + vecs * (32 + kX) + tid * kH;
    // (vector j's two halves n 16 bytes apart: no two lanes on one bank)
    ulonglong2* const gw = reinterpret_cast<ulonglong2*>(smem + all_stages) + tid;
    float* const red = reinterpret_cast<float*>(smem + all_stages + vecs * 32);
    const bool held[VPT] = {tid < own_vecs, tid + n < own_vecs};
    const uint32_t full = smem_u32(full_bars);
    const int row_bytes = p.nv * (kX + kH + (PRE ? 16 : 0) + (p.dres ? 16 : 0));
    bool lost = false;
    int lost_at = 0;
    // asks for a row into stage `stage`, which begins at `at`
    auto fetch = [&](int64_t row, int stage, int at) {
        if (BULK) {
            if (tid != 0 || row >= hi || lost) return;
            const uint32_t to = smem_u32(smem) + at, bar = full + 8 * stage;
            mbar_arrive_expect_tx(bar, row_bytes);
            if constexpr (X != KEPT_NOT)
                bulk_load(to + vecs * 32, static_cast<const char*>(p.x) + row * p.x_vecs * kX, p.nv * kX, bar);
            if constexpr (PRE) {
                bulk_load(to + vecs * (32 + kX), static_cast<const char*>(p.h) + row * p.nv * kH, p.nv * kH, bar);
                bulk_load(to, p.dout + row * p.nv, p.nv * 16, bar);
            }
            if (p.dres) bulk_load(to + vecs * 16, p.dres + row * p.nv, p.nv * 16, bar);
            return;
        }
        if (row < hi) {
            const char* const x = static_cast<const char*>(p.x) + row * p.x_vecs * kX;
            const char* const h = static_cast<const char*>(p.h) + row * p.nv * kH;
            const char* const dout = reinterpret_cast<const char*>(p.dout) + row * p.nv * 16;
            const char* const dres = reinterpret_cast<const char*>(p.dres) + row * p.nv * 16;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (!held[j]) continue;
                const uint32_t place = first + j * n;
                if constexpr (X != KEPT_NOT) copy_async<kX>(own_x + at + j * n * kX, x + place * kX);
                if constexpr (PRE) {
                    copy_async<kH>(own_h + at + j * n * kH, h + place * kH);
                    copy_async<16>(own + at + j * n * 16, dout + place * 16);
                }
                if (p.dres) copy_async<16>(own + at + (VPT + j) * n * 16, dres + place * 16);
            }
        }
        end_copies();
    };
    // what is never fetched is zero, so that the arithmetic need not ask
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        if (held[j] && p.dres) continue;
        for (int at = 0; at < all_stages; at += stage_bytes) {
            *reinterpret_cast<uint4*>(own + at + (VPT + j) * n * 16) = zero;
            if (held[j]) continue;
            *reinterpret_cast<uint4*>(own + at + j * n * 16) = zero;
            if (kX == 16) *reinterpret_cast<uint4*>(own_x + at + j * n * kX) = zero;
            if (kX == 8) *reinterpret_cast<uint2*>(own_x + at + j * n * kX) = make_uint2(0, 0);
            if (kH == 16) *reinterpret_cast<uint4*>(own_h + at + j * n * kH) = zero;
            if (kH == 8) *reinterpret_cast<uint2*>(own_h + at + j * n * kH) = make_uint2(0, 0);
        }
        if (!held[j]) gw[2 * j * n] = gw[(2 * j + 1) * n] = make_ulonglong2(0, 0);
    }
    // what a row has once: 1 / rms of both norms, and what x's and h's values are to be multiplied by
    auto row_factors = [&](int64_t row) {
        if (row >= hi) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float2 r = p.rstd ? p.rstd[row] : make_float2(1.0f, 1.0f);
        return make_float4(r.x, r.y, X == KEPT_E4M3 ? p.x_scale[row] * r.x : r.x, HK == KEPT_E4M3 ? p.h_scale[row] * r.y : r.y);
    };
    if (BULK) {
        if (tid == 0) {
            for (int s = 0; s < kGradStages; ++s) mbar_init(full + 8 * s, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < kGradStages; ++s) fetch(lo + s, s, s * stage_bytes);
    float4 mine = row_factors(lo + lane), later = row_factors(lo + 32 + lane);  // of 32 rows, a lane each
    four dpre[VPT] = {}, sum[VPT] = {};
    uint4 pre[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) pre[j] = PRE && held[j] ? __ldg(p.pre + first + j * n) : make_uint4(0, 0, 0, 0);
    float* partial = p.partial + (int64_t)unit * 4 * H;
    const bool to_dx[VPT] = {held[0] && p.dx, held[1] && p.dx};
    const bool to_dresidual[VPT] = {held[0] && p.dresidual, held[1] && p.dresidual};
    int group = 0, in = 0, turn = 0, stage = 0, parity = 0;
    int64_t begin = 0, end = p.rows, next_end = 0;  // of the group; of the one behind it
    bool open = !p.row_offsets, any = false;
    // block_scale times a weight's or gate's elements (1 where there is none)
    auto scaled = [&](const uint4* w, int64_t vec, four& f) {
        if (w) {
            unpack4(__ldg(w + vec), f);
#pragma unroll
            for (int c = 0; c < 4; ++c) f[c] = mul2(f[c], two(p.block_scale));
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) f[c] = two(p.block_scale);
        }
    };
    auto open_group = [&]() {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * n;
            if (!held[j]) continue;
            four g;
            scaled(p.gate, (int64_t)group * p.nv + i, g);
            if constexpr (POST) {
                four w;
                unpack4(__ldg(p.post + i), w);
#pragma unroll
                for (int c = 0; c < 4; ++c) g[c] = mul2(g[c], w[c]);
            }
            gw[2 * j * n] = make_ulonglong2(g[0], g[1]);
            gw[(2 * j + 1) * n] = make_ulonglong2(g[2], g[3]);
        }
    };
    auto close_group = [&]() {
        if (!p.row_offsets) {  // one group: S is all that both gradients need
            if (p.dpost || p.dgate) {
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (held[j]) store4(partial + H + 8 * (first + j * n), sum[j]);
            }
            return;
        }
        const bool whole = begin >= lo && end <= hi;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * n;
            if (!held[j]) continue;
            if (POST && p.dpost) {
                four g, before = {};
                scaled(p.gate, (int64_t)group * p.nv + i, g);
                float* to = partial + H + 8 * i;
                if (any) load4(reinterpret_cast<const ulonglong2*>(to), 1, before);
#pragma unroll
                for (int c = 0; c < 4; ++c) before[c] = fma2(g[c], sum[j][c], before[c]);
                store4(to, before);
            }
            if (p.dgate) {
                if (whole) {
                    four w;
                    scaled(POST ? p.post : nullptr, i, w);
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum[j][c] = mul2(sum[j][c], w[c]);
                }
                store4((whole ? p.dgate + (int64_t)group * H : partial + (begin < lo ? 2 : 3) * H) + 8 * i, sum[j]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[j][c] = 0;
        }
        any = true;
    };
    if (open) open_group();
    if (SHARED) {
        __syncwarp();
        cluster_sync();  // all blocks are there to be written to
    }
    const int rows = (int)(hi - lo);
    int change = open ? rows : 0;  // the row at which the group has to be looked up again
    for (int r = 0; r < rows; ++r) {
        const int at = r & 31;
        if (at == 0 && r != 0) {
            mine = later;
            later = row_factors(lo + r + 32 + lane);
        }
        if (BULK) {
            wait_row(full + 8 * stage, parity, lost);
            lost_at += !lost;
        } else {
            wait_copies<kGradStages - 1>();
        }
        if (r == change) {
            if (open) close_group();
            const int64_t row = lo + r;
            if (open && row == end && row < next_end) {  // the next group
                ++group;
            } else {
                group = group_of(p.row_offsets, p.n_groups, row);
                open = group >= 0;
                next_end = open ? min((int64_t)p.row_offsets[group + 1], p.rows) : 0;
            }
            change = r + 1;
            if (open) {
                begin = any ? row : max(p.row_offsets[group], 0);
                end = next_end;
                next_end = min((int64_t)p.row_offsets[min(group + 2, p.n_groups)], p.rows);
                change = (int)min(max(end - lo, (int64_t)change), (int64_t)rows);
                open_group();
                if (group + 1 < p.n_groups && end < hi) {  // its gate on its way
#pragma unroll
                    for (int j = 0; j < VPT; ++j)
                        if (held[j])
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.gate + (int64_t)(group + 1) * p.nv + first + j * n));
                }
            }
        }
        if (open) {
            const float rx = __shfl_sync(0xffffffffu, mine.x, at), rh = __shfl_sync(0xffffffffu, mine.y, at);
            const float x_by = __shfl_sync(0xffffffffu, mine.z, at), h_by = __shfl_sync(0xffffffffu, mine.w, at);
            four e[VPT], hh[VPT], xx[VPT];
            pair by_h = 0, q_e = 0, q_h = 0;  // the sums of gy hhat, q e and q hhat
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                unpack4(*reinterpret_cast<const uint4*>(own + in + (VPT + j) * n * 16), e[j]);
                if constexpr (BULK && !PRE) {
                    if (lost) e[j][0] = e[j][1] = e[j][2] = e[j][3] = two(CUDART_NAN_F);
                }
                if constexpr (PRE) {
                    four w, dy;
                    values<HK>(own_h + in + j * n * kH, two(h_by), hh[j]);
                    unpack4(*reinterpret_cast<const uint4*>(own + in + j * n * 16), dy);
                    unpack4(pre[j], w);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        dpre[j][c] = fma2(dy[c], hh[j][c], dpre[j][c]);
                        const pair gy = mul2(dy[c], w[c]);
                        by_h = fma2(gy, hh[j][c], by_h);
                        e[j][c] = fma2(two(rh), gy, e[j][c]);
                    }
                }
                if constexpr (X != KEPT_NOT) values<X>(own_x + in + j * n * kX, two(x_by), xx[j]);
                if constexpr (POST) {
                    four w;
                    load4(gw + 2 * j * n, n, w);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const pair t = mul2(w[c], xx[j][c]);
                        q_e = fma2(t, e[j][c], q_e);
                        if constexpr (PRE) q_h = fma2(t, hh[j][c], q_h);
                    }
                }
            }
            if (!BULK) fetch(lo + r + kGradStages, stage, in);
            float m = 0.0f, m2 = 0.0f;
            const int64_t vec = (lo + r) * p.nv + first;
            if constexpr (PRE || POST) {
                const float2 s0 = apart(by_h), s1 = apart(q_e), s2 = apart(q_h);
                // (lost: m and m2 of the whole block, and with m e below)
                const float3 sums = row_sums<SHARED>(BULK && lost ? CUDART_NAN_F : s0.x + s0.y, s1.x + s1.y, s2.x + s2.y, red, turn, size);
                m = rh * sums.x * p.one_nth;
                m2 = rx * (sums.y - m * sums.z) * p.one_nth;
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                four t;
                if constexpr (PRE) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) e[j][c] = fma2(two(-m), hh[j][c], e[j][c]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) t[c] = mul2(two(p.residual_scale), e[j][c]);
                if (to_dresidual[j]) p.dresidual[vec + j * n] = pack4(t);
                if constexpr (X != KEPT_NOT) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum[j][c] = fma2(e[j][c], xx[j][c], sum[j][c]);
                }
                load4(gw + 2 * j * n, n, t);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    t[c] = mul2(t[c], e[j][c]);
                    if constexpr (POST) t[c] = fma2(two(rx), t[c], mul2(two(-m2), xx[j][c]));
                }
                if (to_dx[j]) p.dx[vec + j * n] = pack4(t);
            }
        }
        if (BULK) {
            // everybody has taken his part of the stage: they were at the row's
            // barrier since, where it has one (and nobody is a phase of the
            // stage's own barrier behind)
            if (!open || !(PRE || POST))
                __syncthreads();
            else
                __syncwarp();  // a block of one warp
        }
        if (BULK || !open) fetch(lo + r + kGradStages, stage, in);
        in += stage_bytes;
        if (++stage == kGradStages) {
            stage = in = 0;
            parity ^= 1;
        }
    }
    if (BULK && lost) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) dpre[j][c] = two(CUDART_NAN_F);
    }
    if (open) close_group();
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = first + j * n;
        if (!held[j]) continue;
        const four none = {};
        if (PRE && p.dpre) store4(partial + 8 * i, dpre[j]);
        if (POST && p.dpost && p.row_offsets && !any) store4(partial + H + 8 * i, none);
    }
    if (BULK && lost && tid == 0) wait_lost_rows(full, kGradStages, lost_at, min(lost_at + kGradStages, rows));
    if (SHARED) {
        __syncwarp();
        cluster_sync();  // no block leaves while another may write to it
    }
}

// Adds up the units' sums, 64 columns a block of 16 warps.  blockIdx.y 0: pre,
// 1: post (with one group for all rows, its S: post and the gate); beyond, the groups' gates, p.sum_warps warps a group.  A sum's units
// are dealt to its warps, kSumLoads of each on their way.
constexpr int kSumWarps = 16, kSumLoads = 12;
__global__ void __launch_bounds__(32 * kSumWarps) sandwich_sums_kernel(const __grid_constant__ SandwichGradArgs p) {
    __shared__ float2 red[kSumWarps][32];
    const int H = p.nv * 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 64 + 2 * lane;
    const bool gates = blockIdx.y >= 2;
    const uint32_t warps = gates ? p.sum_warps : kSumWarps, part = warp % warps;
    const int group = gates ? (blockIdx.y - 2) * (kSumWarps / warps) + warp / warps : 0;
    float* to = gates ? p.dgate + (int64_t)group * H : blockIdx.y == 0 ? p.dpre : p.dpost;
    // (the kernel before let this one start when everything before it was done)
    uint32_t first = 0, last = (uint32_t)p.units;  // one behind the last unit
    const bool single = blockIdx.y == 1 && !p.row_offsets;
    bool wanted = col < H && (to != nullptr || (single && p.dgate));
    if (gates) {
        if (group >= p.n_groups) {
            wanted = false;
        } else {
            const uint32_t begin = max(p.row_offsets[group], 0), chunk = (uint32_t)p.chunk;
            const uint32_t end = min((uint32_t)max(p.row_offsets[group + 1], 0), (uint32_t)p.rows);
            first = begin / chunk;
            last = begin < end ? (end - 1) / chunk + 1 : 0;
        }
        if (last == first + 1) wanted = false;  // written already
    }
    // (before any return: who comes next waits for this kernel only)
    wait_for_previous_kernel();
    let_next_kernel_start();
    float2 s = make_float2(0.0f, 0.0f);
    if (wanted) {
        const float* from = p.partial + (gates ? 2 : blockIdx.y) * (int64_t)H + col;
        for (uint32_t b0 = first + part; b0 < last; b0 += kSumLoads * warps) {
            float2 v[kSumLoads];
#pragma unroll
            for (int i = 0; i < kSumLoads; ++i) {
                const uint32_t b = b0 + i * warps;
                // the group begun in its first unit lies in the slot behind
                v[i] = b < last ? *reinterpret_cast<const float2*>(from + ((int64_t)b * 4 + (gates && b == first)) * H)
                                : make_float2(0.0f, 0.0f);
            }
#pragma unroll
            for (int i = 0; i < kSumLoads; ++i) {
                s.x += v[i].x;
                s.y += v[i].y;
            }
        }
    }
    red[warp][lane] = s;
    __syncthreads();
    if (part != 0 || !wanted) return;
    for (int w = warp + 1; w < warp + (int)warps; ++w) {
        s.x += red[w][lane].x;
        s.y += red[w][lane].y;
    }
    auto times = [&](const uint4* w) {  // c w S
        const float2 f = w ? __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(w)[col / 2]) : make_float2(1.0f, 1.0f);
        return make_float2(s.x * p.block_scale * f.x, s.y * p.block_scale * f.y);
    };
    if (single) {
        if (p.dpost) *reinterpret_cast<float2*>(p.dpost + col) = times(p.gate);
        if (p.dgate) *reinterpret_cast<float2*>(p.dgate + col) = times(p.post);
        return;
    }
    if (gates && first < last) s = times(p.post);  // (a group without rows: zeros)
    *reinterpret_cast<float2*>(to + col) = s;
}

// How the gradients' kernel is launched for rows of nv vectors.
struct GradShape {
    int size, share, threads;  // blocks that share a row, vectors a block, threads
    explicit GradShape(int nv)
        : size((nv + 1023) / 1024), share((nv + size - 1) / size), threads(((share + kGradVecs - 1) / kGradVecs + 31) / 32 * 32) {}
    size_t smem(int x_bytes, int h_bytes) const {  // 226 KB at most
        return (size_t)threads * kGradVecs * (kGradStages * (x_bytes + h_bytes + 32) + 32) + std::max(size * threads, 512);
    }
    // As many units (rows at once) as a GB300's 152 SMs hold at 128 registers
    // a thread and `smem` bytes a block (the workspace: 0), but no more than one
    // an SM for less than rows / 3 units (1003 x 2048, 11 gates, 8 bits: four rows
    // each 16.3 us; two 18.2, seven 18.7).
    int64_t units(int64_t rows, size_t smem) const {
        const int64_t blocks = std::min<int64_t>(512 / threads, (228 << 10) / (smem + 1024));
        return std::max<int64_t>(1, std::min({rows, 152 * blocks / size, std::max<int64_t>(152 / size, rows / 3)}));
    }
};

template <int X, int HK, bool POST, int THREADS, bool SHARED, bool BULK>
cudaError_t launch_grad(const SandwichGradArgs& p, const GradShape& g, size_t smem, cudaStream_t s) {
    const auto kernel = sandwich_grad_kernel<X, HK, POST, THREADS, SHARED, BULK>;
    // the kernel's limit, not this call's size (norm.cu)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, p, dim3((unsigned)(p.units * g.size)), g.threads, smem, s, g.size);
}
template <int X, int HK, bool POST>
cudaError_t launch_grad(SandwichGradArgs& p, cudaStream_t s) {
    const GradShape g(p.nv);
    const size_t smem = g.smem(kept_bytes(X), kept_bytes(HK));
    p.size = g.size;
    p.share = g.share;
    p.units = g.units(p.rows, smem);
    p.chunk = (p.rows + p.units - 1) / p.units;
    p.units = (p.rows + p.chunk - 1) / p.chunk;
    if (g.size > 1) return launch_grad<X, HK, POST, 512, true, false>(p, g, smem, s);
    if constexpr (X == KEPT_E4M3 || HK == KEPT_E4M3)
        if (p.nv % 2 || (X == KEPT_E4M3 && p.x_vecs % 2)) return launch_grad<X, HK, POST, 512, false, false>(p, g, smem, s);
    return g.threads <= 256   ? launch_grad<X, HK, POST, 256, false, true>(p, g, smem, s)
           : g.threads <= 448 ? launch_grad<X, HK, POST, 448, false, true>(p, g, smem, s)
                              : launch_grad<X, HK, POST, 512, false, true>(p, g, smem, s);
}
template <int X, bool POST>
cudaError_t launch_grad(SandwichGradArgs& p, cudaStream_t s) {
    return !p.pre        ? launch_grad<X, KEPT_NOT, POST>(p, s)
           : !p.h_scale ? launch_grad<X, KEPT_BF16, POST>(p, s)
                        : launch_grad<X, KEPT_E4M3, POST>(p, s);
}

// Which kernel.  us with a post norm, kept rows and no codes: a block a row, one
// vector a thread / the same, two a thread / staying blocks.
//   rows   H 512               2048                4096                7168
//    152   2.3 / 2.6 /  3.4    2.5 / 2.8 /  3.6    2.8 / 3.1 /  3.8     3.7 /  3.7 /  4.4
//    608   2.5 / 2.7 /  3.4    3.6 / 4.3 /  5.0    8.2 / 8.4 /  9.0    15.5 / 11.2 / 11.3
//   1216   2.8 / 3.1 /  3.7    7.7 / 7.6 /  9.1   14.7 / 13.0 / 13.4   29.4 / 19.8 / 19.0
//   4864   7.4 / 6.8 /  8.8   24.2 / 19.0 / 22.4  49.4 / 39.5 / 37.0    107 / 65.3 / 61.1
//  16384  19.1 / 17.5 / 19.1  72.7 / 55.4 / 60.5   157 / 121 / 113      355 / 209 / 190
// So one vector a thread while all rows' blocks are on the SMs at once (64
// registers a thread), then two; staying blocks for many wide rows (16384 x
// 7168: 92% of the copy rate).  Wider rows than 8192 are read by a block a row:
// 4864 x 12288 143 us (62%), x 16384 177 (67%), x 32768 359 (66%).
template <class ASK>
cudaError_t launch_norm(SandwichArgs& p, cudaStream_t s) {
    const int nv = p.nv, threads1 = (nv + 31) / 32 * 32, threads2 = ((nv + 1) / 2 + 31) / 32 * 32;
    const dim3 grid((unsigned)p.rows);
    if (nv <= 1024 && p.rows <= 152 * (1024 / threads1))
        return launch_dependent(sandwich_norm_kernel<ASK, 1, 1024>, p, grid, threads1, 0, s);
    if (nv <= 896 && (nv <= 448 || p.rows < 8 * 152))
        return launch_dependent(sandwich_norm_kernel<ASK, 2, 448>, p, grid, threads2, 0, s);
    if (nv <= 1024) {
        // two an SM
        auto bytes = [&](int stages) { return (size_t)threads2 * kNormVecs * (stages * 32 + 32); };
        const int stages = bytes(3) <= kNormSmem ? 3 : 2;
        const int64_t most = 152 * std::min<int64_t>(1024 / threads2, (228 << 10) / (bytes(stages) + 2048));
        p.chunk = (p.rows + most - 1) / most;
        const dim3 blocks((unsigned)((p.rows + p.chunk - 1) / p.chunk));
        const auto kernel = stages == 3 ? sandwich_stream_kernel<ASK, 3> : sandwich_stream_kernel<ASK, 2>;
        // the kernel's limit, not this call's size (norm.cu)
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
        return e != cudaSuccess ? e : launch_dependent(kernel, p, blocks, threads2, bytes(stages), s);
    }
    if (nv <= 2048) return launch_dependent(sandwich_norm_kernel<ASK, 2, 1024>, p, grid, threads2, 0, s);
    return launch_dependent(sandwich_norm_kernel<ASK, 4, 1024>, p, grid, ((nv + 3) / 4 + 31) / 32 * 32, 0, s);
}

template <bool POST, bool KEPT>
cudaError_t launch_norm(SandwichArgs& p, cudaStream_t s) {
    if (!p.pre) return launch_norm<Asked<POST, false, false, KEPT>>(p, s);
    return p.codes ? launch_norm<Asked<POST, true, true, KEPT>>(p, s) : launch_norm<Asked<POST, true, false, KEPT>>(p, s);
}

}  // namespace

cudaError_t launch_sandwich_norm(SandwichArgs& p, cudaStream_t s) {
    if (p.rows <= 0) return cudaSuccess;
    const bool kept = p.x_codes || p.h_codes;
    if (p.post) return kept ? launch_norm<true, true>(p, s) : launch_norm<true, false>(p, s);
    return kept ? launch_norm<false, true>(p, s) : launch_norm<false, false>(p, s);
}

size_t sandwich_grad_bytes(int64_t rows, int H) {
    return (size_t)GradShape(H / 8).units(rows, 0) * 4 * H * sizeof(float);
}

cudaError_t launch_sandwich_grad(SandwichGradArgs& p, cudaStream_t s) {
    const int H = p.nv * 8;
    if (p.rows == 0) {
        const size_t row = H * sizeof(float);
        cudaError_t e = cudaSuccess;
        if (p.dpre) e = cudaMemsetAsync(p.dpre, 0, row, s);
        if (p.dpost && e == cudaSuccess) e = cudaMemsetAsync(p.dpost, 0, row, s);
        if (p.dgate && e == cudaSuccess) e = cudaMemsetAsync(p.dgate, 0, row * p.n_groups, s);
        return e;
    }
    const cudaError_t e = !p.x         ? launch_grad<KEPT_NOT, false>(p, s)
                          : !p.x_scale ? (p.post ? launch_grad<KEPT_BF16, true>(p, s) : launch_grad<KEPT_BF16, false>(p, s))
                                       : (p.post ? launch_grad<KEPT_E4M3, true>(p, s) : launch_grad<KEPT_E4M3, false>(p, s));
    if (e != cudaSuccess || (!p.dpre && !p.dpost && !p.dgate)) return e;
    // a warp for every 8 units of a group, on average
    int blocks = 2;
    p.sum_warps = 1;
    if (p.dgate && p.row_offsets) {
        while (p.sum_warps < kSumWarps && (int64_t)p.sum_warps * 8 * p.n_groups < p.units) p.sum_warps *= 2;
        blocks += (p.n_groups * p.sum_warps + kSumWarps - 1) / kSumWarps;
    }
    return launch_dependent(sandwich_sums_kernel, p, dim3((H + 63) / 64, blocks), 32 * kSumWarps, 0, s);
}

}  // namespace dwdp
