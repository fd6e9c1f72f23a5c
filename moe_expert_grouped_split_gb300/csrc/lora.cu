// lora.cu: low-rank adapters of many requests beside a shared projection
// (dwdp_lora_add): out[t] = base[t] + s_i (x[t] A_i^T) B_i^T, i the token's
// adapter.  Memory-bound: x, base, out and the used adapters once.
//
// Two kernels, v = bf16(s_i x A_i^T) [T][R] between them:
//   shrink  clusters of 8 CTAs per token tile, each CTA a part of K; the
//           parts meet in distributed shared memory, in rank order
//   expand  token tile x 256 columns per CTA, base and out in 16-byte vectors
// Both take 16 tokens at a time against each adapter that occurs among them
// (mma m16n8k16) and give every row its own adapter's result, so tokens may
// come in any order, and values of one adapter never meet another's rows.
// A step is at most 2 R flops a byte of x: far from the tensor rate, so the
// warp-level MMA on operands straight from global memory is enough.
#include <cuda_bf16.h>

#include <algorithm>

#include "dwdp_internal.h"

namespace dwdp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kNone = 0xffffffffu;  // a row without an adapter
constexpr int kThreads = 256;
constexpr int kCluster = 8;

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

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// A float of another CTA of the cluster, at this CTA's address `p`.
__device__ __forceinline__ float load_of_rank(const float* p, uint32_t rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// A token's adapter as the kernels use it; what is not one is kNone.
__device__ __forceinline__ uint32_t adapter_of(const LoraArgs& p, int t, bool in_tile) {
    if (!in_tile) return kNone;
    const int id = p.ids[t];
    return id >= 0 && id < p.n_adapters ? (uint32_t)id : kNone;
}

// x rows of one warp against A_i: TW x KW warps, MT m16 tiles a warp; NT
// n8 tiles hold the rank.  G adapters share a pass over the warp's x.
template <int NT, int TW, int KW, int MT>
struct Shrink {
    static constexpr int kRows = TW * MT * 16;
    static constexpr int kSmem = KW * kRows * NT * 8 * 4;

    template <int G, int U>
    static __device__ __forceinline__ void pass(const LoraArgs& p, const uint4* const (&xr)[2 * MT],
                                                const uint32_t (&cur)[G], int step0, int step1, int lane,
                                                const uint32_t (&id)[2 * MT], float* part) {
        const int g = lane >> 2, q = lane & 3, kv = p.K / 8;
        float acc[G][MT][NT][4] = {};
        const uint4* ar[G];
#pragma unroll
        for (int s = 0; s < G; ++s)
            ar[s] = static_cast<const uint4*>(p.a) + (int64_t)(cur[s] == kNone ? 0 : cur[s]) * p.R * kv + (int64_t)g * kv;
        for (int st = step0; st < step1; st += U) {
            uint4 xv[U][2 * MT], av[U][G][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (st + u) * 4 + q;
                const bool in = st + u < step1 && k < kv;
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i)
                    xv[u][i] = in && xr[i] ? __ldg(xr[i] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int s = 0; s < G; ++s)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        av[u][s][j] = in && cur[s] != kNone && j * 8 + g < p.R ? __ldg(ar[s] + (int64_t)j * 8 * kv + k)
                                                                                  : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < G; ++s)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const uint4 &lo = xv[u][2 * m], &hi = xv[u][2 * m + 1], &b = av[u][s][j];
                            mma16816(acc[s][m][j], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
                            mma16816(acc[s][m][j], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
                        }
        }
#pragma unroll
        for (int s = 0; s < G; ++s)
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
                if (id[i] != kNone && id[i] == cur[s]) {
                    float* row = part + ((i >> 1) * 16 + (i & 1) * 8 + g) * NT * 8 + 2 * q;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        *reinterpret_cast<float2*>(row + j * 8) =
                            make_float2(acc[s][i >> 1][j][2 * (i & 1)], acc[s][i >> 1][j][2 * (i & 1) + 1]);
                }
    }
};

template <int NT, int TW, int KW, int MT>
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
    lora_shrink_kernel(const __grid_constant__ LoraArgs p, int tile_rows) {
    static_assert(TW * KW * 32 == kThreads, "one warp per (token part, K part)");
    using S = Shrink<NT, TW, KW, MT>;
    constexpr int G = NT <= 2 ? 4 : NT <= 4 ? 2 : 1;        // adapters a mixed pass takes at once
    constexpr int U = MT * NT <= 4 ? 4 : MT * NT <= 16 ? 2 : 1;  // steps in flight
    extern __shared__ float part[];                         // [KW][rows][NT * 8]
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const int tw = warp % TW, kw = warp / TW;
    const int t0 = (int)(blockIdx.x / kCluster) * tile_rows;
    const uint32_t rank = cluster_rank();
    // this warp's rows
    uint32_t id[2 * MT], left[2 * MT];
    const uint4* xr[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        const int r = tw * MT * 16 + (i >> 1) * 16 + (i & 1) * 8 + g, t = t0 + r;
        const bool in = r < tile_rows && t < p.T;
        left[i] = id[i] = adapter_of(p, t, in);
        xr[i] = id[i] != kNone ? static_cast<const uint4*>(p.x) + (int64_t)t * (p.x_stride / 8) : nullptr;
        if (rank == 0 && kw == 0 && in && id[i] == kNone && p.ids[t] != -1) atomicOr(p.err, DERR_BAD_INDEX);
    }
    const int steps = (p.K + 31) / 32, at = (int)rank * KW + kw;
    const int step0 = steps * at / (kCluster * KW), step1 = steps * (at + 1) / (kCluster * KW);
    float* mine = part + (kw * S::kRows + tw * MT * 16) * NT * 8;
    // the lowest adapter among the rows not done yet
    auto next = [&] {
        uint32_t m = kNone;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) m = min(m, left[i]);
        m = __reduce_min_sync(kFull, m);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            if (left[i] == m) left[i] = kNone;
        return m;
    };
    uint32_t a0 = next();
    while (a0 != kNone) {
        const uint32_t a1 = next();
        if (G == 1 || a1 == kNone) {
            const uint32_t cur[1] = {a0};
            S::template pass<1, U>(p, xr, cur, step0, step1, lane, id, mine);
            a0 = a1;
        } else {
            uint32_t cur[G];
            cur[0] = a0;
#pragma unroll
            for (int s = 1; s < G; ++s) cur[s] = s == 1 ? a1 : next();
            S::template pass<G, (MT * NT <= 2 ? 2 : 1)>(p, xr, cur, step0, step1, lane, id, mine);
            a0 = next();
        }
    }
    __syncthreads();
    const int n = S::kRows * NT * 8;
    if constexpr (KW > 1) {
        for (int e = threadIdx.x; e < n; e += kThreads) {
            float s = part[e];
#pragma unroll
            for (int w = 1; w < KW; ++w) s += part[w * n + e];
            part[e] = s;
        }
    }
    cluster_sync();
    // each rank finishes an eighth of the tile's rows
    __nv_bfloat16* v = static_cast<__nv_bfloat16*>(p.ws);
    for (int e = (int)rank * kThreads + threadIdx.x; e < n; e += kCluster * kThreads) {
        const int r = e / (NT * 8), c = e % (NT * 8), t = t0 + r;
        if (r >= tile_rows || c >= p.R) continue;
        const uint32_t i = adapter_of(p, t, t < p.T);
        if (i == kNone) continue;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kCluster; ++k) s += load_of_rank(part + e, k);
        v[(int64_t)t * p.R + c] = __float2bfloat16_rn(s * p.scale[i]);
    }
    cluster_sync();  // nobody leaves while another rank may still read its shared memory
}

// out = base + v B_i^T: a warp takes MT m16 tiles and 32 columns.  Column
// 2 q + e of n8 tile j is the warp's column 8 q + 2 j + e, so a thread's
// results for a row are 8 neighbours: one 16-byte load and store.
template <int KS, int MT>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(const __grid_constant__ LoraArgs p, int tile_rows) {
    constexpr int G = MT > 1 ? 1 : KS <= 1 ? 4 : KS <= 2 ? 2 : 1;  // adapters whose B is loaded together
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int t0 = (int)blockIdx.x * tile_rows, c0 = ((int)blockIdx.y * (kThreads / 32) + warp) * 32;
    const bool col_in = c0 + 8 * q < p.N;
    // base and the ids do not come from the kernel before this one, which
    // lets this one start only after everything before it is done
    uint32_t id[MT][2];
    uint4 bs[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = m * 16 + h * 8 + g, t = t0 + r;
            const bool in = r < tile_rows && t < p.T;
            id[m][h] = adapter_of(p, t, in);
            if (in && col_in)
                bs[m][h] = *(static_cast<const uint4*>(p.base) + (int64_t)t * (p.base_stride / 8) + c0 / 8 + q);
        }
    const uint2* bw = static_cast<const uint2*>(p.b);
    const int rv = p.R / 4;
    auto load_b = [&](uint32_t i, uint2 (&f)[KS][4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
            for (int s = 0; s < KS; ++s)
                f[s][j] = i != kNone && c < p.N && s * 4 + q < rv
                              ? __ldg(bw + ((int64_t)i * p.N + c) * rv + s * 4 + q) : make_uint2(0, 0);
        }
    };
    wait_for_previous_kernel();
    uint2 bf[G][KS][4];
    uint32_t held = kNone;  // G == 1: the adapter bf holds
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        uint2 vf[2][KS];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < KS; ++s)
                vf[h][s] = id[m][h] != kNone && s * 4 + q < rv
                               ? *(static_cast<const uint2*>(p.ws) + (int64_t)(t0 + m * 16 + h * 8 + g) * rv + s * 4 + q)
                               : make_uint2(0, 0);
        uint32_t left[2] = {id[m][0], id[m][1]};
        float d[4][4];
        for (;;) {
            uint32_t cur[G];
#pragma unroll
            for (int s = 0; s < G; ++s) {
                cur[s] = __reduce_min_sync(kFull, min(left[0], left[1]));
                if (left[0] == cur[s]) left[0] = kNone;
                if (left[1] == cur[s]) left[1] = kNone;
            }
            if (cur[0] == kNone) break;
            if (G > 1 || cur[0] != held) {
#pragma unroll
                for (int s = 0; s < G; ++s) load_b(cur[s], bf[s]);
                held = cur[0];
            }
#pragma unroll
            for (int s = 0; s < G; ++s) {
                if (cur[s] == kNone) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        mma16816(e, vf[0][ks].x, vf[1][ks].x, vf[0][ks].y, vf[1][ks].y, bf[s][ks][j].x, bf[s][ks][j].y);
                    if (id[m][0] == cur[s]) {
                        d[j][0] = e[0];
                        d[j][1] = e[1];
                    }
                    if (id[m][1] == cur[s]) {
                        d[j][2] = e[2];
                        d[j][3] = e[3];
                    }
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = m * 16 + h * 8 + g, t = t0 + r;
            if (r >= tile_rows || t >= p.T || !col_in) continue;
            uint4 o = bs[m][h];
            if (id[m][h] != kNone) {
                __nv_bfloat162* w = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = __bfloat1622float2(w[j]);
                    w[j] = __floats2bfloat162_rn(f.x + d[j][2 * h], f.y + d[j][2 * h + 1]);
                }
            }
            *(static_cast<uint4*>(p.out) + (int64_t)t * (p.out_stride / 8) + c0 / 8 + q) = o;
        }
    }
}

cudaError_t launch(const void* kernel, dim3 grid, size_t smem, cudaStream_t s, const LoraArgs& p, int tile_rows) {
    if (smem > 48 << 10) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    void* args[] = {const_cast<LoraArgs*>(&p), &tile_rows};
    return cudaLaunchKernelExC(&c, kernel, args);
}

template <int NT>
cudaError_t launch_rank(const LoraArgs& p, cudaStream_t s) {
    constexpr int KS = NT / 2;
    const int cols = (p.N + 255) / 256;
    cudaError_t e;
    if (p.T >= 2048) {
        using S = Shrink<NT, 4, 2, 2>;
        e = launch((const void*)lora_shrink_kernel<NT, 4, 2, 2>, dim3((p.T + S::kRows - 1) / S::kRows * kCluster),
                   S::kSmem, s, p, S::kRows);
        if (e != cudaSuccess) return e;
        return launch((const void*)lora_expand_kernel<KS, 4>, dim3((p.T + 63) / 64, cols), 0, s, p, 64);
    }
    // few tokens: tiles of 1 to 16 tokens, so that the clusters fill the GPU
    int rows = 1;
    while (rows < 16 && (int64_t)((p.T + rows - 1) / rows) * kCluster > p.n_sms) rows *= 2;
    using S = Shrink<NT, 1, 8, 1>;
    e = launch((const void*)lora_shrink_kernel<NT, 1, 8, 1>, dim3((p.T + rows - 1) / rows * kCluster), S::kSmem, s, p,
               rows);
    if (e != cudaSuccess) return e;
    return launch((const void*)lora_expand_kernel<KS, 1>, dim3((p.T + rows - 1) / rows, cols), 0, s, p, rows);
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t, int64_t, int64_t R) {
    return ((size_t)(T * R) * 2 + 255) / 256 * 256;
}

cudaError_t launch_lora_add(const LoraArgs& p, cudaStream_t s) {
    if (p.T <= 0) return cudaSuccess;
    if (p.R <= 16) return launch_rank<2>(p, s);
    if (p.R <= 32) return launch_rank<4>(p, s);
    if (p.R <= 64) return launch_rank<8>(p, s);
    return launch_rank<16>(p, s);
}

}  // namespace dwdp
