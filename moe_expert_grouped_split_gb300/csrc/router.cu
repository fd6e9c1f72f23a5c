// router.cu: the router's logits for few tokens (dwdp_route_scored):
// z [T][E] = x W^T, fp32.
//
// Few tokens read W once and little else, so what counts is that the whole
// GPU loads at once and how few round trips a launch needs: a tile of 16
// or 32 tokens x 16 to 64 experts is a cluster of 8 CTAs of 8 warps that share
// K, operands straight from global memory, several steps' loads in flight;
// the parts meet in shared memory, then across the cluster, in order.
#include <cuda_bf16.h>

#include "dwdp_internal.h"

namespace dwdp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// MW x NW x KW warps, each MT m16 tiles of tokens x NT n8 tiles of experts x
// its part of K.  A step is 32 elements of K: thread q of a row's four takes
// 8 neighbours, 16 bytes, as the operands of two MMAs (the order of k is free
// as long as both operands share it).
template <int MW, int NW, int KW, int MT, int NT, int U>
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1)
    router_small_kernel(const uint4* __restrict__ x, const uint4* __restrict__ w, int T, int E, int H,
                        float* __restrict__ z, int32_t* __restrict__ zero, int64_t n_zero) {
    static_assert(MW * NW * KW == kWarps, "");
    constexpr int kRows = MW * MT * 16, kCols = NW * NT * 8, kTile = kRows * kCols;
    constexpr int kShare = kTile / kCluster;
    __shared__ __align__(16) float part[KW][kTile];
    __shared__ float sent[kCluster][kShare];  // what the cluster's ranks send of this one's share
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int mw = warp % MW, nw = warp / MW % NW, kw = warp / (MW * NW);
    const int rank = blockIdx.x % kCluster;
    const int t0 = (int)(blockIdx.x / kCluster) * kRows, e0 = (int)blockIdx.y * kCols;
    const int tw = t0 + mw * MT * 16, ew = e0 + nw * NT * 8;  // this warp's first token and expert
    const int hv = H / 8, steps = H / 32;
    const int at = rank * KW + kw;
    const int step0 = steps * at / (kCluster * KW), step1 = steps * (at + 1) / (kCluster * KW);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const int64_t blocks = (int64_t)gridDim.x * gridDim.y, block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    for (int64_t i = block * kThreads + threadIdx.x; i < n_zero; i += blocks * kThreads) zero[i] = 0;
    float acc[MT][NT][4] = {};
    for (int st = step0; st < step1; st += U) {
        uint4 xv[U][2 * MT], wv[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (st + u) * 4 + q;
            const bool in = st + u < step1;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int e = ew + j * 8 + g;
                wv[u][j] = in && e < E ? __ldg(w + (int64_t)e * hv + k) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                const int t = tw + i * 8 + g;
                xv[u][i] = in && t < T ? __ldg(x + (int64_t)t * hv + k) : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 &lo = xv[u][2 * m], &hi = xv[u][2 * m + 1], &b = wv[u][j];
                    mma16816(acc[m][j], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
                    mma16816(acc[m][j], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
                }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2*>(&part[kw][(tw - t0 + m * 16 + h * 8 + g) * kCols + ew - e0 + j * 8 + 2 * q]) =
                    make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // everybody runs: may be written to
    for (int i = threadIdx.x; i < kTile; i += kThreads) {
        float s = part[0][i];
#pragma unroll
        for (int v = 1; v < KW; ++v) s += part[v][i];
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at)
                     : "r"((uint32_t)__cvta_generic_to_shared(&sent[rank][i % kShare])), "r"(i / kShare));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(s) : "memory");
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int i = threadIdx.x; i < kShare; i += kThreads) {
        float s = sent[0][i];
#pragma unroll
        for (int c = 1; c < kCluster; ++c) s += sent[c][i];
        const int at = rank * kShare + i, t = t0 + at / kCols, e = e0 + at % kCols;
        if (t < T && e < E) z[(int64_t)t * E + e] = s;
    }
}

template <int MW, int NW, int KW, int MT, int NT, int U>
cudaError_t launch(const void* x, const void* w, int T, int E, int H, float* z, int32_t* zero, int64_t n_zero,
                   cudaStream_t s) {
    constexpr int kRows = MW * MT * 16, kCols = NW * NT * 8;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((T + kRows - 1) / kRows * kCluster, (E + kCols - 1) / kCols);
    c.blockDim = dim3(kThreads);
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, router_small_kernel<MW, NW, KW, MT, NT, U>, static_cast<const uint4*>(x),
                              static_cast<const uint4*>(w), T, E, H, z, zero, n_zero);
}

}  // namespace

// Where the tensor-core pairs (router_pair.cu) take over.  Routing to 8 of 256
// experts, H = 7168, here / there, us: 192 tokens 17.1 / 19.1, 256 17.2 / 18.9,
// 384 23.3 / 19.4, 512 21.9 / 19.0.
bool router_is_small(int64_t T, int64_t E) { return T * E <= 64 << 10 && T <= 1 << 10; }

// The tile by the size of z: small tiles spread W over all SMs, larger ones
// read x and W fewer times.  7168 x 256, us at 1 / 64 / 128 / 256 / 512
// tokens: 16 x 16 3.1 / 5.2 / 9.5 / 18 / 34, 32 x 32 4.3 / 6.2 / 6.5 / 12 / 24,
// 32 x 64 5.9 / 7.1 / 8.7 / 9.2 / 18.
cudaError_t launch_router_small(const void* x, const void* w, int T, int E, int H, float* z, int32_t* zero,
                                int64_t n_zero, cudaStream_t s) {
    const int64_t n = (int64_t)T * E;
    if (n <= 16 << 10) return launch<1, 1, 8, 1, 2, 4>(x, w, T, E, H, z, zero, n_zero, s);
    if (n <= 32 << 10) return launch<1, 1, 8, 2, 4, 2>(x, w, T, E, H, z, zero, n_zero, s);
    return launch<1, 2, 4, 2, 4, 2>(x, w, T, E, H, z, zero, n_zero, s);
}

}  // namespace dwdp
