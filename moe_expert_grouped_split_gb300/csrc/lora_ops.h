// lora_ops.h: what the two forms of dwdp_lora_add (lora.cu, lora_tc.cu) share.
#pragma once

#include <cuda_bf16.h>

#include "dwdp_internal.h"

namespace dwdp {

constexpr uint32_t kNoAdapter = 0xffffffffu;

// The order of k inside a step is free as long as both operands use it:
// thread q of a row's four takes 4 (expand) or 8 (shrink: two steps)
// consecutive elements instead of the MMA's 2 + 2, one vector load a row.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Stores v at this CTA's address `p` in another CTA of the cluster.
__device__ __forceinline__ void store_to_rank(float* p, uint32_t rank, float v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// A token's adapter as the kernels use it; what is not one is kNoAdapter.
__device__ __forceinline__ uint32_t adapter_of(const LoraArgs& p, int t, bool in_tile) {
    if (!in_tile) return kNoAdapter;
    const int id = p.ids[t];
    return id >= 0 && id < p.n_adapters ? (uint32_t)id : kNoAdapter;
}

// out = base + v B_i^T for 16 tokens and 32 columns by one warp.  Column
// 2 q + e of n8 tile j is the warp's column 8 q + 2 j + e, so a thread's
// results for a row are 8 neighbours: one 16-byte load and store.
template <int KS>
struct Expand {
    // B_i's rows of the warp's columns (columns beyond N read the last one)
    static __device__ __forceinline__ void load_b(const LoraArgs& p, uint32_t i, int c0, int lane, uint2 (&f)[KS][4]) {
        const int g = lane >> 2, q = lane & 3, rv = p.R / 4, c = c0 + 8 * (g >> 1) + (g & 1);
        const uint2* b = static_cast<const uint2*>(p.b) + (int64_t)(i == kNoAdapter ? 0 : i) * p.N * rv + q;
        if (c0 + 32 <= p.N) {
            b += (int64_t)c * rv;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    f[s][j] = s < KS / 2 || s * 4 + q < rv ? __ldg(b + 2 * j * rv + s * 4) : make_uint2(0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    f[s][j] = s * 4 + q < rv ? __ldg(b + (int64_t)min(c + 2 * j, p.N - 1) * rv + s * 4) : make_uint2(0, 0);
        }
    }
    // base (two rows' 8 columns) + v B
    static __device__ __forceinline__ void product(const uint4 (&base)[2], const uint2 (&v)[2][KS], const uint2 (&b)[KS][4],
                                                   float (&d)[4][4]) {
        const __nv_bfloat162* lo = reinterpret_cast<const __nv_bfloat162*>(&base[0]);
        const __nv_bfloat162* hi = reinterpret_cast<const __nv_bfloat162*>(&base[1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 l = __bfloat1622float2(lo[j]), h = __bfloat1622float2(hi[j]);
            d[j][0] = l.x;
            d[j][1] = l.y;
            d[j][2] = h.x;
            d[j][3] = h.y;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                mma16816(d[j], v[0][s].x, v[1][s].x, v[0][s].y, v[1][s].y, b[s][j].x, b[s][j].y);
        }
    }
    static __device__ __forceinline__ uint4 round(const float (&d)[4][4], int h) {
        uint4 o;
        __nv_bfloat162* w = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __floats2bfloat162_rn(d[j][2 * h], d[j][2 * h + 1]);
        return o;
    }
};

}  // namespace dwdp
