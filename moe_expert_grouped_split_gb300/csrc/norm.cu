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

#include "dwdp_internal.h"

namespace dwdp {
namespace {

// A row's sum of squares beyond this is taken again on values scaled by
// 2^-80 (bf16 values reach 2^128, so 32768 squares then stay below 2^112).
constexpr float kSquaresLimit = 1e38f;
constexpr float kDownScale = 0x1p-80f;
constexpr float kMinCodeMax = 0x1p-100f;

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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

// (sum, max) over the block; every thread gets them.  red holds 2 x 32 floats.
__device__ __forceinline__ float2 block_sum_max(float s, float m, float2* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = make_float2(s, m);
    __syncthreads();
    const float2 v = lane < nw ? red[lane] : make_float2(0.0f, 0.0f);
    s = v.x;
    m = v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    __syncthreads();  // red may be written again
    return make_float2(s, m);
}

// One block per row; thread i holds the row's 16-byte vectors i, i + blockDim.x,
// ... (VPT of them at most).
template <int VPT, bool RES, bool CODES>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const uint4* x, int64_t x_vecs, const uint4* residual,
                                                           uint4* residual_out, const uint4* __restrict__ weight,
                                                           float eps, int nv, uint4* out,
                                                           uint2* __restrict__ codes,
                                                           float* __restrict__ row_scale) {
    __shared__ float2 red[32];
    const int64_t r = blockIdx.x;
    float h[VPT][8];
    uint4 w[VPT];
    float ss = 0.0f, mx = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        if (i < nv) {
            unpack8(x[r * x_vecs + i], h[j]);
            w[j] = __ldg(weight + i);
            if constexpr (RES) {
                float t[8];
                unpack8(residual[r * nv + i], t);
#pragma unroll
                for (int c = 0; c < 8; ++c) h[j][c] += t[c];
                residual_out[r * nv + i] = pack8(h[j]);
            }
            float f[8];
            unpack8(w[j], f);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                ss = fmaf(h[j][c], h[j][c], ss);
                if constexpr (CODES) mx = max_nan(mx, fabsf(h[j][c] * f[c]));
            }
        }
    }
    float2 red_v = block_sum_max(ss, mx, red);
    float e = eps;
    if (!(red_v.x < kSquaresLimit)) {  // rare; the whole block agrees
        ss = mx = 0.0f;
        e = eps * kDownScale * kDownScale;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (threadIdx.x + j * blockDim.x >= nv) continue;
            float f[8];
            unpack8(w[j], f);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                h[j][c] *= kDownScale;
                ss = fmaf(h[j][c], h[j][c], ss);
                if constexpr (CODES) mx = max_nan(mx, fabsf(h[j][c] * f[c]));
            }
        }
        red_v = block_sum_max(ss, mx, red);
    }
    const float rs = 1.0f / sqrtf(red_v.x / (float)(8 * nv) + e);
    float inv = 0.0f;
    if constexpr (CODES) {
        const float m = red_v.y == 0.0f ? 0.0f : max_nan(red_v.y, kMinCodeMax);
        inv = m == 0.0f ? 0.0f : 448.0f / m;
        if (threadIdx.x == 0) row_scale[r] = m == 0.0f ? 1.0f : m * rs / 448.0f;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        if (i < nv) {
            float f[8], y[8];
            unpack8(w[j], f);
#pragma unroll
            for (int c = 0; c < 8; ++c) y[c] = h[j][c] * rs * f[c];
            out[r * nv + i] = pack8(y);
            if constexpr (CODES) {
                uint32_t q[2] = {0u, 0u};
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    const uint32_t p = __nv_cvt_float2_to_fp8x2(
                        make_float2(h[j][c] * f[c] * inv, h[j][c + 1] * f[c + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                    q[c >> 2] |= p << ((c & 2) * 8);
                }
                codes[r * nv + i] = make_uint2(q[0], q[1]);
            }
        }
    }
}

template <int VPT>
cudaError_t launch_vpt(const uint4* x, int64_t xv, const uint4* res, uint4* res_out, const uint4* w, float eps,
                       int64_t rows, int nv, uint4* out, uint2* codes, float* row_scale, cudaStream_t s) {
    const int threads = ((nv + VPT - 1) / VPT + 31) / 32 * 32;
    const unsigned grid = (unsigned)rows;
#define DWDP_NORM(R, C) \
    add_rmsnorm_kernel<VPT, R, C><<<grid, threads, 0, s>>>(x, xv, res, res_out, w, eps, nv, out, codes, row_scale)
    if (res && codes) DWDP_NORM(true, true);
    else if (res) DWDP_NORM(true, false);
    else if (codes) DWDP_NORM(false, true);
    else DWDP_NORM(false, false);
#undef DWDP_NORM
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* x, int64_t x_stride, const void* residual, void* residual_out,
                               const void* weight, float eps, int64_t rows, int H, void* out, void* codes,
                               float* row_scale, cudaStream_t s) {
    if (rows <= 0) return cudaSuccess;
    const uint4* xv = static_cast<const uint4*>(x);
    const uint4* rv = static_cast<const uint4*>(residual);
    const uint4* wv = static_cast<const uint4*>(weight);
    uint4* ro = static_cast<uint4*>(residual_out);
    uint4* ov = static_cast<uint4*>(out);
    uint2* cv = static_cast<uint2*>(codes);
    const int nv = H / 8;
    if (nv <= 1024) return launch_vpt<1>(xv, x_stride / 8, rv, ro, wv, eps, rows, nv, ov, cv, row_scale, s);
    return launch_vpt<4>(xv, x_stride / 8, rv, ro, wv, eps, rows, nv, ov, cv, row_scale, s);
}

}  // namespace dwdp
