// router_pair.cu: the router's logits for many tokens (dwdp_route_scored):
// planes z[part] [T][pitch] = x W^T over the part's K, fp32 (zeros from expert
// E on, so that a row is whole 32-byte sectors).
//
// What bounds it: 8192 x 7168 x 256 is 30 GFLOP, 16 us at the measured bf16
// rate, and x comes from HBM once, 117 MB, 17 us; it takes about 28 us.  The
// tensor pipe of the 128 SMs in use is busy 67% of that; the rest is start,
// first loads and epilogue.  (W shared by two pairs through multicast loads
// changed nothing: 47.9 us of routing against 47.7, so L2 is not the limit.)
// Every token tile needs all of W again, from L2.  So the tile is as
// tall as it can be: a pair of CTAs (cta_group::2) multiplies 256 tokens by
// up to 256 experts, each CTA loading its 128 token rows and half of the
// experts' rows.  A 64-element slice of K is 32 KB a CTA; six are in flight.
//   warp 0      TMA producer of its CTA; all loads complete on the leader's
//               barrier
//   warp 1      allocates TMEM; the leader's issues the pair's MMAs
//   warps 2..5  epilogue: 32 TMEM lanes each, a thread one token's row, stored
//               in whole sectors of 32 bytes
// K is cut into parts so that the pairs fill the GPU; the choice adds the
// planes in order.
#include <cuda_bf16.h>

#include <algorithm>

#include "dwdp_internal.h"
#include "tc_ops.h"

namespace dwdp {
namespace {

constexpr int kThreads = 192;
constexpr int kSlice = 64;                      // elements of K per stage
constexpr int kPairStages = 6;
constexpr int kRowsBytes = 128 * kSlice * 2;    // a CTA's token rows of one slice

// half of N experts' rows per CTA
template <int N>
struct PairSmem {
    static constexpr int kWBytes = N / 2 * kSlice * 2;
    static constexpr int kStage = kRowsBytes + kWBytes;
    static constexpr int kBars = kPairStages * kStage;         // full[S], empty[S], done
    static constexpr int kMisc = kBars + 8 * (2 * kPairStages + 1);
    static constexpr int kBytes = 1024 + kMisc + 16;           // base aligned to 1024 inside
};

// The address of `addr` in the pair's first CTA.
__device__ __forceinline__ uint32_t at_leader(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

// A box into this CTA's shared memory, completing on a barrier of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// D [256 x N] (+)= A [256 x 16] B [N x 16]^T over the pair.
template <int N>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate) {
    // D fp32, A and B bf16, both K-major, N / 8 at bits 17-22, M / 16 at 24-28
    constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (16u << 24);
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)0x3)
        : "memory");
}

__device__ __forceinline__ void store8(float* to, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    router_pair_kernel(const __grid_constant__ RouterPairArgs p) {
    using S = PairSmem<N>;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* mem = raw + (base - smem_u32(raw));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(mem + S::kMisc + 8);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mem + S::kMisc);
    const uint32_t full0 = base + S::kBars, empty0 = full0 + 8 * kPairStages, done = empty0 + 8 * kPairStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1;
    const int tile = pair / p.parts, part = pair - tile * p.parts;
    const int row0 = tile * 256 + (int)rank * 128, e0 = (int)blockIdx.y * N;
    const int slices = p.H / kSlice;
    const int s0 = (int)((int64_t)slices * part / p.parts), s1 = (int)((int64_t)slices * (part + 1) / p.parts);

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&p.tm_x);
        prefetch_map(&p.tm_w);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(N < 32 ? 32 : N)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and TMEM are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp >= 2) {  // the epilogue's warps have nothing else to do yet
        const int64_t blocks = (int64_t)gridDim.x * gridDim.y, block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
        for (int64_t i = block * 128 + threadIdx.x - 64; i < p.n_zero; i += blocks * 128) p.zero[i] = 0;
    }

    if (warp == 0) {
        if (lane == 0) {
            uint32_t phase = 0;
            int stage = 0;
            for (int s = s0; s < s1; ++s) {
                if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.err, DERR_PRODUCER_WAIT)) {
                    // loads still on their way land before this CTA may leave
                    const uint64_t t = global_timer();
                    while (global_timer() - t < 1000000ull) {}
                    break;
                }
                if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * S::kStage);  // both CTAs' loads
                const uint32_t bar = at_leader(full0 + 8 * stage), dst = base + stage * S::kStage;
                tma_load_pair(dst, &p.tm_x, s * kSlice, row0, bar);
                tma_load_pair(dst + kRowsBytes, &p.tm_w, s * kSlice, e0 + (int)rank * (N / 2), bar);
                if (++stage == kPairStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            uint32_t phase = 0;
            int stage = 0;
            for (int s = s0; s < s1; ++s) {
                if (!mbar_wait(full0 + 8 * stage, phase, abort_flag, p.err, DERR_MMA_FULL_WAIT)) break;
                tc_fence_after();
                const uint64_t a = smem_desc(base + stage * S::kStage), b = smem_desc(base + stage * S::kStage + kRowsBytes);
#pragma unroll
                for (int k = 0; k < kSlice / 16; ++k)  // 32 bytes of K further: + 2 in the start address
                    mma_pair<N>(tmem, a + 2 * k, b + 2 * k, s > s0 || k > 0);
                commit_pair(empty0 + 8 * stage);
                if (++stage == kPairStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            commit_pair(done);
        }
    } else {
        const int q = warp & 3;  // the TMEM lane quarter this warp may read
        if (__all_sync(0xffffffffu, mbar_wait(done, 0, abort_flag, p.err, DERR_EPI_WAIT))) {
            tc_fence_after();
            const int t = row0 + 32 * q + lane;
            float* row = p.z + ((int64_t)part * p.T + t) * p.pitch + e0;
            const bool wide = (uint64_t)p.z % 32 == 0;  // whole sectors
#pragma unroll 1
            for (int c = 0; c < N; c += 32) {
                uint32_t v[32];
                __syncwarp();  // the load is the whole warp's; lanes beyond T are ahead here
                tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + c, v);
                tmem_wait_ld();
                if (t >= p.T) continue;
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    if (e0 + c + j >= p.pitch) break;
                    if (wide) {
                        store8(row + c + j, v + j);
                    } else {
                        *reinterpret_cast<uint4*>(row + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                        *reinterpret_cast<uint4*>(row + c + j + 4) = make_uint4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // neither CTA leaves while the other may still load for it, read its
    // shared memory or arrive on its barriers
    cluster_sync();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(N < 32 ? 32 : N) : "memory");
}

template <int N>
cudaError_t launch_n(const RouterPairArgs& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(router_pair_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PairSmem<N>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(2 * ((p.T + 255) / 256) * p.parts, (p.E + N - 1) / N);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = PairSmem<N>::kBytes;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, router_pair_kernel<N>, p);
}

}  // namespace

int router_pair_cols(int E) { return E <= 64 ? 64 : E <= 128 ? 128 : 256; }

// Parts of K: as many pairs as fill whole rounds of the GPU's 76 pairs of SMs
// best, in passes over all of K; a round costs 10% of one beside its work
// (start and epilogue), a part's plane 1.5% (written and read again).  Of 7168
// x 256, us of routing at 384 / 1024 / 2048 tokens: 8 parts 19.4 / 20.2 / 25.1,
// 14 or as many as fit 20.3 / 22.4 / 24.8 (5 at 2048: 26.8).  From the sizes
// alone, so the logits depend on nothing else.
int router_pair_parts(int64_t T, int64_t E, int64_t H) {
    const int n = router_pair_cols((int)E);
    const int64_t tiles = (T + 255) / 256 * ((E + n - 1) / n);
    int best = 1;
    double least = 1e30;
    for (int s = 1; s == 1 || (s <= kRouterPairMaxParts && s * 4 <= H / kSlice); ++s) {
        if (s > 4 && tiles * s > 76) break;  // (what router_pair_plane_rows counts on)
        const double cost = (double)((tiles * s + 75) / 76) * (1.0 / s + 0.1) + 0.015 * s;
        if (cost < least - 1e-9) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// More than 4 parts only where 256-token tiles x parts <= 76.
int64_t router_pair_plane_rows(int64_t T) {
    return std::max<int64_t>(4 * T, std::min<int64_t>(kRouterPairMaxParts * T, 76 * 256));
}

cudaError_t launch_router_pair(const RouterPairArgs& p, cudaStream_t s) {
    switch (router_pair_cols(p.E)) {
        case 64: return launch_n<64>(p, s);
        case 128: return launch_n<128>(p, s);
        default: return launch_n<256>(p, s);
    }
}

}  // namespace dwdp
