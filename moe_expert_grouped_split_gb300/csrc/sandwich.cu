// sandwich.cu: the norms after and before a block with the block's gate and
// the residual's scale (dwdp_sandwich_norm) and their gradients
// (dwdp_sandwich_norm_grad), memory-bound.
//
// Forward, per row: x stays in registers for its sum of squares, h for its
// own; two reductions a row, which also carry the largest magnitudes that the
// E4M3 rows' scales need.  Backward, per row: two reductions, the means of
// (dout pre) h and of (dn post) x; the weights' and gates' gradients are sums
// over rows, which each block keeps in registers for the rows it takes, one
// after the other, and a second kernel adds up in the blocks' order: the same
// bits from run to run.
#include <math_constants.h>

#include <algorithm>

#include "dwdp_internal.h"
#include "row_ops.h"

namespace dwdp {
namespace {

// As in norm.cu: a sum of squares beyond the limit is taken again on values
// scaled by 2^-80.  (1 / rms is then below 2^-40; 2^-128 at its least, whose
// subnormal binary32 still has 21 bits.)
constexpr float kSquaresLimit = 1e38f;
constexpr float kDownScale = 0x1p-80f;
constexpr float kMinCodeMax = 0x1p-100f;

// The group of `row`: offsets[g] <= row < offsets[g + 1], the last such g; -1
// where there is none.  The whole warp together: 32 offsets a step.
__device__ __forceinline__ int group_of(const int32_t* offsets, int n_groups, int64_t row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_groups + 1;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const uint32_t at = __ballot_sync(0xffffffffu, i < n && (int64_t)offsets[lo + i] <= row);
        if (at == 0) return -1;
        const int j = (31 - __clz(at)) * step;
        lo += j;
        n = min(step, n - j);
    }
    return lo < n_groups ? lo : -1;
}

// (sum, max, max) over the block; every thread gets them.
__device__ __forceinline__ float3 block_sum_max2(float s, float a, float b, float4* red) {
    warp_sum_max<false>(s, a);
    a = warp_max(a);
    b = warp_max(b);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = make_float4(s, a, b, 0.0f);
    __syncthreads();
    const float4 v = lane < nw ? red[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    s = v.x;
    a = v.y;
    warp_sum_max<false>(s, a);
    a = warp_max(a);
    b = warp_max(v.z);
    __syncthreads();  // red may be written again
    return make_float3(s, a, b);
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    uint32_t q[2] = {0u, 0u};
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
        const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(v[c] * inv, v[c + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        q[c >> 2] |= two << ((c & 2) * 8);
    }
    return make_uint2(q[0], q[1]);
}

// 448 / the largest magnitude, and the scale that goes with it (1 for zeros).
__device__ __forceinline__ float code_factor(float m, float& scale) {
    if (m == 0.0f) {
        scale = 1.0f;
        return 0.0f;
    }
    m = max_nan(m, kMinCodeMax);
    scale = m / 448.0f;
    return 448.0f * rcp(m);
}

// One block per row; thread i holds the row's 16-byte vectors i, i + blockDim.x,
// ... (VPT of them at most).
template <int VPT>
__global__ void __launch_bounds__(1024) sandwich_norm_kernel(const __grid_constant__ SandwichArgs p) {
    __shared__ float4 red[32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int64_t row = blockIdx.x;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 x[VPT], r[VPT], post[VPT];
    int held = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        if (i < p.nv) {
            x[j] = p.x[row * p.x_vecs + i];
            r[j] = p.residual ? p.residual[row * p.nv + i] : zero;
            post[j] = p.post ? __ldg(p.post + i) : zero;
            held = j + 1;
        }
    }
    const uint4* gate = p.gate;
    if (p.row_offsets) {
        const int g = group_of(p.row_offsets, p.n_groups, row);
        if (g < 0) return;  // the whole block
        gate += (int64_t)g * p.nv;
    }
    float rx = 1.0f;
    const bool keep_x = p.x_codes != nullptr;
    if (p.post || keep_x) {
        float ss = 0.0f, ax = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (j >= held) continue;
            float f[8];
            unpack8(x[j], f);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                ss = fmaf(f[c], f[c], ss);
                ax = max_nan(ax, fabsf(f[c]));
            }
        }
        float3 sums = block_sum_max2(ss, ax, 0.0f, red);
        float scaled = 1.0f;
        if (p.post && !(sums.x < kSquaresLimit)) {  // rare; the whole block agrees
            scaled = kDownScale;
            ss = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (j >= held) continue;
                float f[8];
                unpack8(x[j], f);
#pragma unroll
                for (int c = 0; c < 8; ++c) ss = fmaf(f[c] * scaled, f[c] * scaled, ss);
            }
            sums.x = block_sum_max2(ss, 0.0f, 0.0f, red).x;
        }
        if (p.post) rx = rsqrtf(fmaf(sums.x, p.one_nth, p.eps * scaled * scaled)) * scaled;
        if (keep_x) {
            float scale;
            const float inv = code_factor(sums.y, scale);
            if (threadIdx.x == 0) p.x_scale[row] = scale;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (j >= held) continue;
                float f[8];
                unpack8(x[j], f);
                p.x_codes[row * p.nv + threadIdx.x + j * blockDim.x] = codes8(f, inv);
            }
        }
    }
    float h[VPT][8];
    uint4 pre[VPT];
    float ss = 0.0f, ah = 0.0f, ay = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (j >= held) continue;
        const int i = threadIdx.x + j * blockDim.x;
        float f[8], w[8];
        unpack8(x[j], f);
        if (p.post) {
            unpack8(post[j], w);
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = f[c] * rx * w[c];
        }
        if (gate) {
            unpack8(__ldg(gate + i), w);
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] *= w[c];
        }
        unpack8(r[j], w);
        pre[j] = p.pre ? __ldg(p.pre + i) : zero;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            h[j][c] = fmaf(p.block_scale, f[c], p.residual_scale * w[c]);
            ss = fmaf(h[j][c], h[j][c], ss);
            ah = max_nan(ah, fabsf(h[j][c]));
        }
        unpack8(pre[j], w);
#pragma unroll
        for (int c = 0; c < 8; ++c) ay = max_nan(ay, fabsf(h[j][c] * w[c]));
        if (p.residual_out) p.residual_out[row * p.nv + i] = pack8(h[j]);
    }
    if (!p.pre && !p.h_codes) {
        if (p.rstd && threadIdx.x == 0) p.rstd[row] = make_float2(rx, 1.0f);
        return;
    }
    float3 sums = block_sum_max2(ss, ah, ay, red);
    float rh = 1.0f;
    if (p.pre) {
        float scaled = 1.0f;
        if (!(sums.x < kSquaresLimit)) {
            scaled = kDownScale;
            ss = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (j >= held) continue;
#pragma unroll
                for (int c = 0; c < 8; ++c) ss = fmaf(h[j][c] * scaled, h[j][c] * scaled, ss);
            }
            sums.x = block_sum_max2(ss, 0.0f, 0.0f, red).x;
        }
        rh = rsqrtf(fmaf(sums.x, p.one_nth, p.eps * scaled * scaled)) * scaled;
    }
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = make_float2(rx, rh);
    float h_scale, y_scale;
    const float h_inv = code_factor(sums.y, h_scale), y_inv = code_factor(sums.z, y_scale);
    if (threadIdx.x == 0) {
        if (p.h_codes) p.h_scale[row] = h_scale;
        if (p.codes) p.row_scale[row] = sums.z == 0.0f ? 1.0f : y_scale * rh;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (j >= held) continue;
        const int64_t at = row * p.nv + threadIdx.x + j * blockDim.x;
        if (p.h_codes) p.h_codes[at] = codes8(h[j], h_inv);
        if (p.pre) {
            float w[8], y[8];
            unpack8(pre[j], w);
#pragma unroll
            for (int c = 0; c < 8; ++c) y[c] = h[j][c] * rh * w[c];
            p.out[at] = pack8(y);
            if (p.codes) {
#pragma unroll
                for (int c = 0; c < 8; ++c) y[c] = h[j][c] * w[c];
                p.codes[at] = codes8(y, y_inv);
            }
        }
    }
}

// ------------------------------------------------------------ gradients --

__device__ __forceinline__ void values8(uint2 q, float scale, float (&f)[8]) {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw v =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> ((i & 1) * 16)), __NV_E4M3);
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&v));
        f[2 * i] = t.x * scale;
        f[2 * i + 1] = t.y * scale;
    }
}

// 8 elements of a kept row, bf16 or E4M3 codes, times `by`.
template <bool K8>
__device__ __forceinline__ void kept8(const void* base, int vec, float by, float (&f)[8]) {
    if constexpr (K8) {
        values8(static_cast<const uint2*>(base)[vec], by, f);
    } else {
        unpack8(static_cast<const uint4*>(base)[vec], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] *= by;
    }
}

// Copies 16 bytes (8 for codes) of this thread's into shared memory; nobody
// else reads them, so nothing is waited for but the thread's own copies.
template <bool K8>
__device__ __forceinline__ void fetch8(void* to, const void* base, int64_t vec) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (K8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(static_cast<const uint2*>(base) + vec)
                     : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(static_cast<const uint4*>(base) + vec)
                     : "memory");
}

// The block's sum of s, for every thread; `turn` alternates between two
// buffers, so one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float s, float (*red)[32], int& turn) {
    float none = 0.0f;
    warp_sum_max<false>(s, none);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return s;
    float* r = red[turn];
    turn ^= 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) r[warp] = s;
    __syncthreads();
    s = (lane & 15) < nw ? r[lane & 15] : 0.0f;  // 16 warps at most
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

__device__ __forceinline__ void store8(float* to, const float (&f)[8]) {
    reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void load8(const float* from, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(from)[0], b = reinterpret_cast<const float4*>(from)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

constexpr int kGradStages = 3, kGradVecs = 2;

// A block takes rows [blockIdx.x chunk, + chunk) in order; thread i holds the
// row's vectors i and i + blockDim.x and their columns' sums.  Of the weights'
// gradients only two sums a column have to be kept while rows go by: dout
// hhat, and S = dh xhat since the group began, as dgate = c post S and
// dpost_weight = sum over groups of c gate S.  The rows kGradStages ahead are
// on their way into shared memory.
// partial [blocks][4][H]: the sums for pre and post, and S of the group that
// was begun before the block's rows and of the one that goes on after them
// (a group whose rows are all here goes to dgate at once).
template <bool X8, bool H8>
__global__ void __launch_bounds__(512, 1) sandwich_grad_kernel(const __grid_constant__ SandwichGradArgs p) {
    constexpr int VPT = kGradVecs;
    extern __shared__ __align__(16) char smem[];
    __shared__ float red[2][32];
    const int tid = threadIdx.x, n = blockDim.x, lane = tid & 31;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int64_t lo = (int64_t)blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.rows);
    const int H = p.nv * 8;
    // the stages, each x, h, dout and dres of a row; then c gate post
    const int x_bytes = X8 ? 8 : 16, h_bytes = H8 ? 8 : 16, stage_bytes = n * VPT * (x_bytes + h_bytes + 32);
    // (vector j's two halves n 16 bytes apart: no two lanes on one bank)
    float4* gw = reinterpret_cast<float4*>(smem + kGradStages * stage_bytes) + tid;
    auto fetch = [&](int64_t row, int stage) {
        if (row < hi) {
            char* at = smem + stage * stage_bytes;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = tid + j * n;
                if (i >= p.nv) continue;
                if (p.x) fetch8<X8>(at + i * x_bytes, p.x, row * p.x_vecs + i);
                if (p.pre) {
                    fetch8<H8>(at + n * VPT * x_bytes + i * h_bytes, p.h, row * p.nv + i);
                    fetch8<false>(at + n * VPT * (x_bytes + h_bytes) + i * 16, p.dout, row * p.nv + i);
                }
                if (p.dres) fetch8<false>(at + n * VPT * (x_bytes + h_bytes + 16) + i * 16, p.dres, row * p.nv + i);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // what a row has once: 1 / rms of both norms, and what x's and h's values are to be multiplied by
    auto row_factors = [&](int64_t row) {
        if (row >= hi) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float2 r = p.rstd ? p.rstd[row] : make_float2(1.0f, 1.0f);
        return make_float4(r.x, r.y, X8 ? p.x_scale[row] * r.x : r.x, H8 ? p.h_scale[row] * r.y : r.y);
    };
#pragma unroll
    for (int s = 0; s < kGradStages; ++s) fetch(lo + s, s);
    float4 mine = row_factors(lo + lane), later = row_factors(lo + 32 + lane);  // of 32 rows, a lane each
    float dpre[VPT][8] = {}, sum[VPT][8] = {};
    uint4 pre[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) pre[j] = p.pre && tid + j * n < p.nv ? __ldg(p.pre + tid + j * n) : make_uint4(0, 0, 0, 0);
    float* partial = p.partial + (int64_t)blockIdx.x * 4 * H;
    int group = 0, stage = 0, turn = 0;
    int64_t begin = 0, end = p.rows;  // of the group
    bool open = !p.row_offsets, any = false;
    auto weight_of = [&](const uint4* w, int64_t vec, float (&f)[8]) {
        if (w) {
            unpack8(__ldg(w + vec), f);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = 1.0f;
        }
    };
    auto open_group = [&]() {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * n;
            if (i >= p.nv) continue;
            float g[8], w[8];
            weight_of(p.gate, (int64_t)group * p.nv + i, g);
            weight_of(p.post, i, w);
#pragma unroll
            for (int c = 0; c < 8; ++c) g[c] *= p.block_scale * w[c];
            gw[2 * j * n] = make_float4(g[0], g[1], g[2], g[3]);
            gw[(2 * j + 1) * n] = make_float4(g[4], g[5], g[6], g[7]);
        }
    };
    auto close_group = [&]() {
        const bool whole = begin >= lo && end <= hi;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * n;
            if (i >= p.nv) continue;
            if (p.dpost) {
                float g[8], before[8] = {};
                weight_of(p.gate, (int64_t)group * p.nv + i, g);
                if (any) load8(partial + H + 8 * i, before);
#pragma unroll
                for (int c = 0; c < 8; ++c) before[c] = fmaf(p.block_scale * g[c], sum[j][c], before[c]);
                store8(partial + H + 8 * i, before);
            }
            if (p.dgate) {
                if (whole) {
                    float w[8];
                    weight_of(p.post, i, w);
#pragma unroll
                    for (int c = 0; c < 8; ++c) sum[j][c] *= p.block_scale * w[c];
                }
                store8((whole ? p.dgate + (int64_t)group * H : partial + (begin < lo ? 2 : 3) * H) + 8 * i, sum[j]);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) sum[j][c] = 0.0f;
        }
        any = true;
    };
    if (open) open_group();
    for (int64_t row = lo; row < hi; ++row) {
        const int at = (int)(row - lo) & 31;
        if (at == 0 && row != lo) {
            mine = later;
            later = row_factors(row + 32 + lane);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kGradStages - 1) : "memory");
        if (p.row_offsets && (!open || row >= end)) {
            if (open) close_group();
            group = group_of(p.row_offsets, p.n_groups, row);
            open = group >= 0;
            if (open) {
                begin = max(p.row_offsets[group], 0);
                end = min((int64_t)p.row_offsets[group + 1], p.rows);
                open_group();
            }
        }
        const char* in = smem + stage * stage_bytes;
        if (open) {
            const float rx = __shfl_sync(0xffffffffu, mine.x, at), rh = __shfl_sync(0xffffffffu, mine.y, at);
            const float x_by = __shfl_sync(0xffffffffu, mine.z, at), h_by = __shfl_sync(0xffffffffu, mine.w, at);
            float gy[VPT][8] = {}, hh[VPT][8] = {};
            float dot = 0.0f;
            if (p.pre) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int i = tid + j * n;
                    if (i >= p.nv) continue;
                    float w[8], dy[8];
                    kept8<H8>(in + n * VPT * x_bytes, i, h_by, hh[j]);
                    unpack8(*reinterpret_cast<const uint4*>(in + n * VPT * (x_bytes + h_bytes) + i * 16), dy);
                    unpack8(pre[j], w);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        dpre[j][c] = fmaf(dy[c], hh[j][c], dpre[j][c]);
                        gy[j][c] = dy[c] * w[c];
                        dot = fmaf(gy[j][c], hh[j][c], dot);
                    }
                }
                dot = block_sum(dot, red, turn) * p.one_nth * rh;
            }
            float xx[VPT][8];
            float dot2 = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = tid + j * n;
                if (i >= p.nv) continue;
                float d[8] = {}, w[8];
                if (p.dres) unpack8(*reinterpret_cast<const uint4*>(in + n * VPT * (x_bytes + h_bytes + 16) + i * 16), d);
                if (p.pre) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) d[c] = fmaf(rh, gy[j][c], fmaf(-dot, hh[j][c], d[c]));
                }
                if (p.dresidual) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) w[c] = p.residual_scale * d[c];
                    p.dresidual[row * p.nv + i] = pack8(w);
                }
                {
                    const float4 a = gw[2 * j * n], b = gw[(2 * j + 1) * n];
                    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
                }
                if (p.x) kept8<X8>(in, i, x_by, xx[j]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    gy[j][c] = d[c] * w[c];
                    if (p.x) {
                        sum[j][c] = fmaf(d[c], xx[j][c], sum[j][c]);
                        dot2 = fmaf(gy[j][c], xx[j][c], dot2);
                    }
                }
            }
            if (p.post) dot2 = block_sum(dot2, red, turn) * p.one_nth * rx;
            if (p.dx) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int i = tid + j * n;
                    if (i >= p.nv) continue;
                    if (p.post) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) gy[j][c] = fmaf(rx, gy[j][c], -dot2 * xx[j][c]);
                    }
                    p.dx[row * p.nv + i] = pack8(gy[j]);
                }
            }
        }
        fetch(row + kGradStages, stage);
        if (++stage == kGradStages) stage = 0;
    }
    if (open) close_group();
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = tid + j * n;
        if (i >= p.nv) continue;
        const float none[8] = {};
        if (p.dpre) store8(partial + 8 * i, dpre[j]);
        if (p.dpost && !any) store8(partial + H + 8 * i, none);
    }
}

// Adds up the blocks' sums: blockIdx.y 0 pre, 1 post, 2 + g group g's gate;
// 32 columns a block, the row blocks dealt to 8 warps.
__global__ void __launch_bounds__(256) sandwich_sums_kernel(const __grid_constant__ SandwichGradArgs p) {
    __shared__ float red[8][32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int H = p.nv * 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    const int what = blockIdx.y;
    int64_t first = 0, last = p.blocks - 1;
    float* to;
    if (what < 2) {
        to = what == 0 ? p.dpre : p.dpost;
        if (!to) return;
    } else {
        if (!p.dgate) return;
        const int g = what - 2;
        to = p.dgate + (int64_t)g * H;
        if (p.row_offsets) {
            const int64_t begin = max(p.row_offsets[g], 0), end = min((int64_t)p.row_offsets[g + 1], p.rows);
            if (begin < end) {
                first = begin / p.chunk;
                last = (end - 1) / p.chunk;
                if (first == last) return;  // written already
            } else {
                last = -1;
            }
        } else if (p.blocks == 1) {
            return;
        }
    }
    float s = 0.0f;
    if (col < H) {
#pragma unroll 8
        for (int64_t b = first + warp; b <= last; b += 8) {
            const int slot = what < 2 ? what : b == first ? 3 : 2;
            s += p.partial[(b * 4 + slot) * H + col];
        }
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < H) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s += red[w][lane];
        if (what >= 2) {
            s *= p.block_scale;
            if (p.post) s *= __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.post)[col]);
        }
        to[col] = s;
    }
}

// The gradients' kernel: threads of a block, its shared memory with kept rows
// of x_bytes and h_bytes a vector, and how many blocks.
int grad_threads(int nv) { return ((nv + kGradVecs - 1) / kGradVecs + 31) / 32 * 32; }
size_t grad_smem(int nv, int x_bytes, int h_bytes) {
    return (size_t)grad_threads(nv) * kGradVecs * (kGradStages * (x_bytes + h_bytes + 32) + 32);
}
// As many blocks as a GB300's 152 SMs hold at 128 registers a thread and
// `smem` bytes a block (the workspace: 0).
int64_t grad_blocks(int64_t rows, int nv, size_t smem) {
    const int64_t by_smem = (228 << 10) / (smem + 1024 + 256), most = 152 * std::min<int64_t>(512 / grad_threads(nv), by_smem);
    return std::max<int64_t>(1, std::min(rows, most));
}

template <bool X8, bool H8>
cudaError_t launch_grad(const SandwichGradArgs& p, cudaStream_t s) {
    const auto kernel = sandwich_grad_kernel<X8, H8>;
    // the kernel's limit, not this call's size (norm.cu)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)grad_smem(1024, X8 ? 8 : 16, H8 ? 8 : 16));
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, p, dim3((unsigned)p.blocks), grad_threads(p.nv),
                            grad_smem(p.nv, X8 ? 8 : 16, H8 ? 8 : 16), s);
}

}  // namespace

cudaError_t launch_sandwich_norm(const SandwichArgs& p, cudaStream_t s) {
    if (p.rows <= 0) return cudaSuccess;
    const int nv = p.nv;
    if (nv <= 1024)
        return launch_dependent(sandwich_norm_kernel<1>, p, dim3((unsigned)p.rows), (nv + 31) / 32 * 32, 0, s);
    return launch_dependent(sandwich_norm_kernel<4>, p, dim3((unsigned)p.rows), ((nv + 3) / 4 + 31) / 32 * 32, 0, s);
}

size_t sandwich_grad_bytes(int64_t rows, int H) { return (size_t)grad_blocks(rows, H / 8, 0) * 4 * H * sizeof(float); }

cudaError_t launch_sandwich_grad(SandwichGradArgs& p, cudaStream_t s) {
    const int H = p.nv * 8;
    const bool x8 = p.x_scale != nullptr, h8 = p.h_scale != nullptr;
    p.blocks = grad_blocks(p.rows, p.nv, grad_smem(p.nv, x8 ? 8 : 16, h8 ? 8 : 16));
    p.chunk = std::max<int64_t>(1, (p.rows + p.blocks - 1) / p.blocks);
    p.blocks = std::max<int64_t>(1, (p.rows + p.chunk - 1) / p.chunk);  // none without rows, but for one
    const cudaError_t e = x8 ? (h8 ? launch_grad<true, true>(p, s) : launch_grad<true, false>(p, s))
                             : (h8 ? launch_grad<false, true>(p, s) : launch_grad<false, false>(p, s));
    if (e != cudaSuccess || (!p.dpre && !p.dpost && !p.dgate)) return e;
    const dim3 grid((unsigned)((H + 31) / 32), (unsigned)(2 + (p.dgate ? p.n_groups : 0)));
    return launch_dependent(sandwich_sums_kernel, p, grid, 256, 0, s);
}

}  // namespace dwdp
