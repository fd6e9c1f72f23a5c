// lora.cu: low-rank adapters of many requests beside a shared projection
// (dwdp_lora_add): out[t] = base[t] + s_i (x[t] A_i^T) B_i^T, i the token's
// adapter.  Memory-bound: x, base, out and the used adapters once.
#include <cuda_bf16.h>

#include "dwdp_internal.h"

namespace dwdp {
namespace {

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float acc) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&a);
    const __nv_bfloat162* q = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = __bfloat1622float2(p[i]), v = __bfloat1622float2(q[i]);
        acc = fmaf(u.x, v.x, acc);
        acc = fmaf(u.y, v.y, acc);
    }
    return acc;
}

// v[t][r] = bf16(s_i x[t] . A_i[r]); one block per token, one warp per r.
__global__ void __launch_bounds__(256) lora_shrink_kernel(const uint4* __restrict__ x, int64_t x_vecs, int kv,
                                                          const uint4* __restrict__ a,
                                                          const float* __restrict__ scale, int n, int R,
                                                          const int32_t* __restrict__ ids,
                                                          __nv_bfloat16* __restrict__ v, int* __restrict__ err) {
    const int64_t t = blockIdx.x;
    const int id = ids[t];
    if (id < 0 || id >= n) {
        if (id != -1 && threadIdx.x == 0) atomicOr(err, DERR_BAD_INDEX);
        return;
    }
    const int lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < R; r += blockDim.x >> 5) {
        const uint4* ar = a + ((int64_t)id * R + r) * kv;
        float acc = 0.0f;
        for (int i = lane; i < kv; i += 32) acc = dot8(x[t * x_vecs + i], __ldg(ar + i), acc);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane == 0) v[t * R + r] = __float2bfloat16_rn(acc * scale[id]);
    }
}

// out[t][c] = base[t][c] + v[t] . B_i[c]; a thread takes 8 columns.
__global__ void __launch_bounds__(128) lora_expand_kernel(const uint4* __restrict__ v, const uint4* __restrict__ b,
                                                          int n, int rv, const int32_t* __restrict__ ids, int nvecs,
                                                          const uint4* base, int64_t base_vecs, uint4* out,
                                                          int64_t out_vecs) {
    const int64_t t = blockIdx.x;
    const int i = blockIdx.y * blockDim.x + threadIdx.x;
    if (i >= nvecs) return;
    const int id = ids[t];
    uint4 q = base[t * base_vecs + i];
    if (id >= 0 && id < n) {
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float2 f = __bfloat1622float2(h[c]);
            const uint4* b0 = b + ((int64_t)id * nvecs * 8 + i * 8 + 2 * c) * rv;
            float d0 = 0.0f, d1 = 0.0f;
            for (int j = 0; j < rv; ++j) {
                const uint4 w = __ldg(v + t * rv + j);
                d0 = dot8(w, __ldg(b0 + j), d0);
                d1 = dot8(w, __ldg(b0 + rv + j), d1);
            }
            h[c] = __floats2bfloat162_rn(f.x + d0, f.y + d1);
        }
    }
    out[t * out_vecs + i] = q;
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t, int64_t, int64_t R) {
    return ((size_t)(T * R) * 2 + 255) / 256 * 256;
}

cudaError_t launch_lora_add(const LoraArgs& p, cudaStream_t s) {
    if (p.T <= 0) return cudaSuccess;
    lora_shrink_kernel<<<p.T, 256, 0, s>>>(static_cast<const uint4*>(p.x), p.x_stride / 8, p.K / 8,
                                           static_cast<const uint4*>(p.a), p.scale, p.n_adapters, p.R, p.ids,
                                           static_cast<__nv_bfloat16*>(p.ws), p.err);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const dim3 grid(p.T, (p.N / 8 + 127) / 128);
    lora_expand_kernel<<<grid, 128, 0, s>>>(static_cast<const uint4*>(p.ws), static_cast<const uint4*>(p.b),
                                            p.n_adapters, p.R / 8, p.ids, p.N / 8, static_cast<const uint4*>(p.base),
                                            p.base_stride / 8, static_cast<uint4*>(p.out), p.out_stride / 8);
    return cudaGetLastError();
}

}  // namespace dwdp
