// norm.cu: residual addition + root-mean-square norm + E4M3 rows
// (dwdp_add_rmsnorm), memory-bound.
//
// Per row, in one pass over the data: h = x + r stays in registers; its sum
// of squares and max|h w| are reduced together, which is all that both
// outputs need: y = h rs w with rs = 1 / sqrt(mean + eps), max|y| =
// max|h w| rs, and the code's argument y / (max|y| / 448) = h w (448 /
// max|h w|), in which rs cancels.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include <atomic>

#include "dwdp_internal.h"

namespace dwdp {
namespace {

// A row's sum of squares beyond this is taken again on values scaled by
// 2^-80 (bf16 values reach 2^128, so 32768 squares then stay below 2^112).
constexpr float kSquaresLimit = 1e38f;
constexpr float kDownScale = 0x1p-80f;
constexpr float kMinCodeMax = 0x1p-100f;
// With an eps from here on squares that binary32 loses do not count.  Below it
// (TINY, forms of their own: in the others this costs 8192 rows of 7168 with a
// residual and codes 2%, of 8200 6%) a row whose mean + eps is lower is taken on
// values scaled by 2^80 (bf16's least value is 2^-133); a row's sum then loses
// at most 2^-30 of itself, 32768 additions to within 2^-150.
constexpr float kEpsEnough = 0x1p-120f;
constexpr float kUpScale = 0x1p80f;

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float rcp(float a) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}

__device__ __forceinline__ void unpack8(uint4 q, float (&f)[8]) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __bfloat1622float2(h[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint4 q;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return q;
}

__device__ __forceinline__ void copy16(uint4* to, const uint4* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
}

// m: magnitudes, whose order as floats is their bits' (a NaN is above +inf).
template <bool MAX>
__device__ __forceinline__ void warp_sum_max(float& s, float& m) {
    if constexpr (MAX) m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
}

// (sum, max) over the block; every thread gets them.
template <bool MAX>
__device__ __forceinline__ float2 block_sum_max(float s, float m, float2* red) {
    warp_sum_max<MAX>(s, m);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = make_float2(s, m);
    __syncthreads();
    const float2 v = lane < nw ? red[lane] : make_float2(0.0f, 0.0f);
    s = v.x;
    m = v.y;
    warp_sum_max<MAX>(s, m);
    __syncthreads();  // red may be written again
    return make_float2(s, m);
}

__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

struct NormArgs {
    const uint4* x;
    int64_t x_vecs;  // 16-byte vectors between x's rows
    const uint4* residual;
    uint4* residual_out;
    const uint4* weight;
    float eps;
    float least;  // TINY: the least sum of squares that is taken as it is
    int64_t rows;
    int nv;         // vectors a row
    float one_nth;  // 1 / H
    uint4* out;
    uint2* codes;
    float* row_scale;
};

// 8 elements of a row: h = x + r, its squares' sum and max|h w|.
template <bool RES, bool CODES>
__device__ __forceinline__ void take(const NormArgs& p, int64_t at, uint4 x, uint4 r, uint4 w, float (&h)[8], float& ss,
                                     float& mx) {
    unpack8(x, h);
    if constexpr (RES) {
        float t[8];
        unpack8(r, t);
#pragma unroll
        for (int c = 0; c < 8; ++c) h[c] += t[c];
        p.residual_out[at] = pack8(h);
    }
    float f[8];
    unpack8(w, f);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        ss = fmaf(h[c], h[c], ss);
        if constexpr (CODES) mx = max_nan(mx, fabsf(h[c] * f[c]));
    }
}

// The same 8 elements' outputs, from 1 / rms and 448 / max|h w|.
template <bool CODES>
__device__ __forceinline__ void give(const NormArgs& p, int64_t at, const float (&h)[8], uint4 w, float rs, float inv) {
    float f[8], y[8];
    unpack8(w, f);
#pragma unroll
    for (int c = 0; c < 8; ++c) y[c] = h[c] * rs * f[c];
    p.out[at] = pack8(y);
    if constexpr (CODES) {
        uint32_t q[2] = {0u, 0u};
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
            const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(h[c] * f[c] * inv, h[c + 1] * f[c + 1] * inv),
                                                          __NV_SATFINITE, __NV_E4M3);
            q[c >> 2] |= two << ((c & 2) * 8);
        }
        p.codes[at] = make_uint2(q[0], q[1]);
    }
}

// A row's two factors from its sums; `first` writes the row's scale.  Every
// thread does this, so by the approximate instructions: a few units in the
// last place, where the roundings to come are 2^-8 and 2^-4.
template <bool CODES>
__device__ __forceinline__ void factors(const NormArgs& p, int64_t row, float ss, float mx, float eps, bool first,
                                        float& rs, float& inv) {
    rs = rsqrtf(fmaf(ss, p.one_nth, eps));
    inv = 0.0f;
    if constexpr (CODES) {
        const float m = mx == 0.0f ? 0.0f : max_nan(mx, kMinCodeMax);
        inv = m == 0.0f ? 0.0f : 448.0f * rcp(m);
        if (first) p.row_scale[row] = m == 0.0f ? 1.0f : m * rs / 448.0f;
    }
}

// The sums again on values scaled down, for a row whose squares pass
// binary32's range.
template <int VPT, bool CODES>
__device__ __forceinline__ void take_scaled(float (&h)[VPT][8], const uint4 (&w)[VPT], int held, float& ss, float& mx) {
    ss = mx = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (j >= held) continue;
        float f[8];
        unpack8(w[j], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            h[j][c] *= kDownScale;
            ss = fmaf(h[j][c], h[j][c], ss);
            if constexpr (CODES) mx = max_nan(mx, fabsf(h[j][c] * f[c]));
        }
    }
}

// TINY: whether binary32 holds a row's squares and its products with the weight.
template <bool CODES>
__device__ __forceinline__ bool in_range(const NormArgs& p, float ss, float mx) {
    return ss < kSquaresLimit && ss >= p.least && (!CODES || mx < CUDART_INF_F);
}

// TINY: a row that is not in range (or holds a NaN): h normalized in place,
// from the squares of scaled values, and sums that say so: a mean of 1, no eps,
// mx = max|y|.  An all-zero row keeps its zeros and its eps.  reduce(s, m):
// over the row.
template <int VPT, bool CODES, class Reduce>
__device__ __forceinline__ void normalize(const NormArgs& p, float (&h)[VPT][8], const uint4 (&w)[VPT], int held, float& ss,
                                          float& mx, float& eps, Reduce reduce) {
    const float scale = !(ss < kSquaresLimit) ? kDownScale : ss < p.least ? kUpScale : 1.0f;
    ss = mx = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (j >= held) continue;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            h[j][c] *= scale;
            ss = fmaf(h[j][c], h[j][c], ss);
        }
    }
    reduce(ss, mx);
    eps = eps * scale * scale;
    const float rs = ss == 0.0f ? 1.0f : rsqrtf(fmaf(ss, p.one_nth, eps));
    mx = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (j >= held) continue;
        float f[8];
        unpack8(w[j], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            h[j][c] *= rs;
            if constexpr (CODES) mx = max_nan(mx, fabsf(h[j][c] * f[c]));
        }
    }
    float none = 0.0f;
    if constexpr (CODES) reduce(none, mx);
    if (ss != 0.0f) {
        ss = (float)(p.nv * 8);
        eps = 0.0f;
    }
}

// One block per row; thread i holds the row's 16-byte vectors i, i + blockDim.x,
// ... (VPT of them at most).
template <int VPT, bool RES, bool CODES, bool TINY>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const __grid_constant__ NormArgs p) {
    __shared__ float2 red[32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int64_t row = blockIdx.x;
    float h[VPT][8];
    uint4 w[VPT];
    float ss = 0.0f, mx = 0.0f;
    int held = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        if (i < p.nv) {
            w[j] = __ldg(p.weight + i);
            const uint4 r = RES ? p.residual[row * p.nv + i] : make_uint4(0, 0, 0, 0);
            take<RES, CODES>(p, row * p.nv + i, p.x[row * p.x_vecs + i], r, w[j], h[j], ss, mx);
            held = j + 1;
        }
    }
    float2 sums = block_sum_max<CODES>(ss, mx, red);
    float eps = p.eps;
    if constexpr (TINY) {
        if (!in_range<CODES>(p, sums.x, sums.y))
            normalize<VPT, CODES>(p, h, w, held, sums.x, sums.y, eps,
                                  [&](float& s, float& m) {
                                      const float2 v = block_sum_max<CODES>(s, m, red);
                                      s = v.x;
                                      m = v.y;
                                  });
    } else if (!(sums.x < kSquaresLimit)) {  // rare; the whole block agrees
        take_scaled<VPT, CODES>(h, w, held, ss, mx);
        eps = p.eps * kDownScale * kDownScale;
        sums = block_sum_max<CODES>(ss, mx, red);
    }
    float rs, inv;
    factors<CODES>(p, row, sums.x, sums.y, eps, threadIdx.x == 0, rs, inv);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (j < held) give<CODES>(p, row * p.nv + threadIdx.x + j * blockDim.x, h[j], w[j], rs, inv);
}

// One warp per row, 8 rows a block: rows of up to 32 VPT vectors.
template <int VPT, bool RES, bool CODES, bool TINY>
__global__ void __launch_bounds__(256) add_rmsnorm_warp_kernel(const __grid_constant__ NormArgs p) {
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= p.rows) return;
    float h[VPT][8];
    uint4 w[VPT], x[VPT], r[VPT];
    int held = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = lane + 32 * j;
        if (i < p.nv) {
            x[j] = p.x[row * p.x_vecs + i];
            r[j] = RES ? p.residual[row * p.nv + i] : make_uint4(0, 0, 0, 0);
            w[j] = __ldg(p.weight + i);
            held = j + 1;
        }
    }
    float ss = 0.0f, mx = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (j < held) take<RES, CODES>(p, row * p.nv + lane + 32 * j, x[j], r[j], w[j], h[j], ss, mx);
    warp_sum_max<CODES>(ss, mx);
    float eps = p.eps;
    if constexpr (TINY) {
        if (!in_range<CODES>(p, ss, mx))
            normalize<VPT, CODES>(p, h, w, held, ss, mx, eps, [](float& s, float& m) { warp_sum_max<CODES>(s, m); });
    } else if (!(ss < kSquaresLimit)) {
        take_scaled<VPT, CODES>(h, w, held, ss, mx);
        eps = p.eps * kDownScale * kDownScale;
        warp_sum_max<CODES>(ss, mx);
    }
    float rs, inv;
    factors<CODES>(p, row, ss, mx, eps, lane == 0, rs, inv);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (j < held) give<CODES>(p, row * p.nv + lane + 32 * j, h[j], w[j], rs, inv);
}

// Many rows without a residual: a block stays and takes rows blockIdx.x, + gridDim.x, ...; each
// thread fetches its own vectors of the rows STAGES ahead into shared memory
// (cp.async: nobody else reads them, so nothing is waited for but the
// thread's own copies), and keeps its part of the weight.
template <int STAGES, bool CODES, bool TINY>
__global__ void __launch_bounds__(1024, 1) rmsnorm_stream_kernel(const __grid_constant__ NormArgs p) {
    extern __shared__ uint4 ring[];  // [STAGES][blockDim.x]
    __shared__ float2 red[2][32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tid = threadIdx.x, n = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = n >> 5;
    const int held = tid < p.nv ? 1 : 0;
    uint4 w[1] = {held ? __ldg(p.weight + tid) : make_uint4(0, 0, 0, 0)};
    auto fetch = [&](int64_t row, int stage) {
        if (held && row < p.rows) copy16(ring + stage * n + tid, p.x + row * p.x_vecs + tid);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < STAGES; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
    int stage = 0, half = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        float h[1][8], ss = 0.0f, mx = 0.0f;
        if (held)
            take<false, CODES>(p, row * p.nv + tid, ring[stage * n + tid], make_uint4(0, 0, 0, 0), w[0], h[0], ss, mx);
        fetch(row + (int64_t)STAGES * gridDim.x, stage);
        auto block_sums = [&](float& s, float& m) {
            warp_sum_max<CODES>(s, m);
            if (lane == 0) red[half][warp] = make_float2(s, m);
            __syncthreads();
            const float2 v = lane < nw ? red[half][lane] : make_float2(0.0f, 0.0f);
            s = v.x;
            m = v.y;
            warp_sum_max<CODES>(s, m);
            half ^= 1;  // the next sums go to the other half: one barrier is enough
        };
        block_sums(ss, mx);
        float eps = p.eps;
        if constexpr (TINY) {
            if (!in_range<CODES>(p, ss, mx)) normalize<1, CODES>(p, h, w, held, ss, mx, eps, block_sums);
        } else if (!(ss < kSquaresLimit)) {
            take_scaled<1, CODES>(h, w, held, ss, mx);
            eps = p.eps * kDownScale * kDownScale;
            block_sums(ss, mx);
        }
        float rs, inv;
        factors<CODES>(p, row, ss, mx, eps, tid == 0, rs, inv);
        if (held) give<CODES>(p, row * p.nv + tid, h[0], w[0], rs, inv);
        if (++stage == STAGES) stage = 0;
    }
}

// Programmatic dependent launch: the block's start overlaps the end of the
// kernel before it (0.1 to 0.4 us of a small call).
template <class K>
cudaError_t launch(K kernel, const NormArgs& p, int64_t grid, int threads, size_t smem, cudaStream_t s) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, p);
}

// SMs of the current device, looked up once per device.
int current_sms() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <bool RES, bool CODES, bool TINY>
cudaError_t launch_form(const NormArgs& p, cudaStream_t s) {
    const int nv = p.nv, sms = current_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Which kernel, us at 8192 rows (a warp / a block per row / the staying
    // blocks).  Residual and codes: H = 512 5.1 / 8.7 / -, 1000 12.8 / 10.7 / -,
    // 4096 - / 44.8 / 48.4, 7168 - / 84.5 / 85.1 (92% of the copy rate), 8192 -
    // / 94.3 / 99.7.  Neither: 512 3.2 / 8.7 / -, 1000 4.7 / 8.8 / -, 4096 - /
    // 27.7 / 29.5, 7168 - / 60 / 43.8.  512 x 64 rows, both: 1.9 / 1.6 / -.
    // Wider rows, both: 8200 147 (60%), 16384 265 (67%), 32768 554 (64%); with
    // codes that kernel spills 72 bytes a thread at its 64 registers.
    if (nv <= 64 && p.rows >= 8 * sms)
        return launch(add_rmsnorm_warp_kernel<2, RES, CODES, TINY>, p, (p.rows + 7) / 8, 256, 0, s);
    if constexpr (!RES)
        if (nv <= 128 && p.rows >= 8 * sms)
            return launch(add_rmsnorm_warp_kernel<4, RES, CODES, TINY>, p, (p.rows + 7) / 8, 256, 0, s);
    const int threads = (nv + 31) / 32 * 32;
    if constexpr (!RES)
        if (nv > 768 && nv <= 1024 && p.rows >= 12 * sms) {
            constexpr int kStages = 3;
            const size_t smem = (size_t)kStages * threads * 16;  // 48 KB at most, and the static part
            // the kernel's limit, not this call's size: another host thread
            // may be about to launch a wider row
            const cudaError_t e =
                cudaFuncSetAttribute(rmsnorm_stream_kernel<kStages, CODES, TINY>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * 1024 * 16);
            return e != cudaSuccess ? e : launch(rmsnorm_stream_kernel<kStages, CODES, TINY>, p, sms, threads, smem, s);
        }
    if (nv <= 1024) return launch(add_rmsnorm_kernel<1, RES, CODES, TINY>, p, p.rows, threads, 0, s);
    return launch(add_rmsnorm_kernel<4, RES, CODES, TINY>, p, p.rows, ((nv + 3) / 4 + 31) / 32 * 32, 0, s);
}

template <bool RES, bool CODES>
cudaError_t launch_form(const NormArgs& p, cudaStream_t s) {
    return p.eps < kEpsEnough ? launch_form<RES, CODES, true>(p, s) : launch_form<RES, CODES, false>(p, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* x, int64_t x_stride, const void* residual, void* residual_out,
                               const void* weight, float eps, int64_t rows, int H, void* out, void* codes,
                               float* row_scale, cudaStream_t s) {
    if (rows <= 0) return cudaSuccess;
    const NormArgs p{static_cast<const uint4*>(x),      x_stride / 8, static_cast<const uint4*>(residual),
                     static_cast<uint4*>(residual_out), static_cast<const uint4*>(weight),
                     eps, (kEpsEnough - eps) * (float)H,
                     rows, H / 8, 1.0f / (float)H,
                     static_cast<uint4*>(out),          static_cast<uint2*>(codes), row_scale};
    if (residual && codes) return launch_form<true, true>(p, s);
    if (residual) return launch_form<true, false>(p, s);
    if (codes) return launch_form<false, true>(p, s);
    return launch_form<false, false>(p, s);
}

}  // namespace dwdp
