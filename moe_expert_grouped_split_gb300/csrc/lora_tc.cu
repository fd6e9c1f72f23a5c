// lora_tc.cu: dwdp_lora_add for many tokens (lora_is_long), fed by TMA.
//
// Both halves stream: x once (shrink), base in and out once (expand); the
// adapters stay in L2.  What counts is bytes in flight and their order, so the
// loads are bulk copies into rings in shared memory, 100 KB and more an SM, and
// the arithmetic is whatever keeps up: tcgen05 on the x tiles, warp MMAs on
// the base tiles.
//   shrink  a cluster shares a tile of 128 tokens, each CTA a part of K; the
//           parts meet in the owner's shared memory, in rank order
//   expand  staying CTAs walk stages of 16 tokens x 512 columns: load, add
//           v B^T in place, store
// 8192 tokens, 7168 x 7168, rank 16: 73.5 us for 360 MB, 4.9 TB/s (72% of the
// copy rate): shrink 25 us, expand 46 us.
// A tile's tokens may have any adapters: shrink multiplies the tile by each
// that occurs (4 at a time up to rank 16, else one) and keeps a row's own; so
// does expand.  Every such step reads x again: 16 adapters at random instead of
// in order, 8192 tokens, 7168 x 7168: rank 16 273 us (71), rank 64 865 (107).
#include <cuda_bf16.h>

#include <algorithm>

#include "dwdp_internal.h"
#include "lora_ops.h"
#include "tc_ops.h"

namespace dwdp {
namespace {

// ---------------------------------------------------------------- shrink --
constexpr int kTokens = 128;    // tokens of a tile
constexpr int kSlice = 64;      // elements of K per stage
constexpr int kXBytes = kTokens * kSlice * 2;
constexpr int kShrinkThreads = 192;

// NR: the rank rounded up to 16 or a power of two (columns of one adapter's
// accumulator); a pass takes kGroup adapters, kCols columns of TMEM.  Two CTAs
// fit an SM up to NR = 64.
template <int NR>
struct ShrinkSmem {
    static constexpr int kGroup = NR == 16 ? 4 : 1;
    static constexpr int kStages = NR == 64 ? 3 : 4;
    static constexpr int kCols = NR * kGroup < 32 ? 32 : NR * kGroup;
    static constexpr int kABytes = NR * kSlice * 2;  // one adapter's rows of a slice
    static constexpr int kStage = kXBytes + kGroup * kABytes;
    static constexpr int kPart = kStages * kStage;         // float [128][NR]: this CTA's part of K
    static constexpr int kList = kPart + kTokens * NR * 4;  // uint32 ids[128], distinct[128]
    static constexpr int kBars = kList + 2 * kTokens * 4;   // full[S], empty[S], done
    static constexpr int kMisc = kBars + 8 * (2 * kStages + 1);
    static constexpr int kBytes = 1024 + kMisc + 32;
    // what the cluster sends, float [C][128 / C][NR], goes where the stages were
    static_assert(kTokens * NR * 4 <= kPart, "");
    static_assert(NR == 128 || 2 * (kBytes + 1024) <= 227 << 10, "two CTAs an SM");
};

__device__ __forceinline__ void mma_rank(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

template <int NR>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_tc_kernel(const __grid_constant__ LoraTcArgs p) {
    using S = ShrinkSmem<NR>;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* mem = raw + (base - smem_u32(raw));
    float* part = reinterpret_cast<float*>(mem + S::kPart);
    float* sent = reinterpret_cast<float*>(mem);
    uint32_t* ids = reinterpret_cast<uint32_t*>(mem + S::kList);
    uint32_t* distinct = ids + kTokens;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mem + S::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(mem + S::kMisc + 8);
    int* n_distinct = reinterpret_cast<int*>(mem + S::kMisc + 16);
    const uint32_t full0 = base + S::kBars, empty0 = full0 + 8 * S::kStages, done = empty0 + 8 * S::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = p.parts;  // CTAs of the cluster
    const uint32_t rank = C > 1 ? cluster_ctarank() : 0;
    const int t0 = (int)(blockIdx.x / C) * kTokens;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&p.tm_x);
        prefetch_map(&p.tm_a);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(S::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    wait_for_previous_kernel();
    let_next_kernel_start();
    if (warp == 0) {
        // the tile's adapters, and which occur, ascending
        uint32_t left[kTokens / 32];
#pragma unroll
        for (int i = 0; i < kTokens / 32; ++i) {
            const int r = 32 * i + lane, t = t0 + r;
            left[i] = adapter_of(p.lora, t, t < p.lora.T);
            ids[r] = left[i];
            if (rank == 0 && t < p.lora.T && left[i] == kNoAdapter && p.lora.ids[t] != -1)
                atomicOr(p.lora.err, DERR_BAD_INDEX);
        }
        int n = 0;
        for (;; ++n) {
            uint32_t m = kNoAdapter;
#pragma unroll
            for (int i = 0; i < kTokens / 32; ++i) m = min(m, left[i]);
            m = __reduce_min_sync(0xffffffffu, m);
            if (m == kNoAdapter) break;
#pragma unroll
            for (int i = 0; i < kTokens / 32; ++i)
                if (left[i] == m) left[i] = kNoAdapter;
            if (lane == 0) distinct[n] = m;
        }
        if (lane == 0) *n_distinct = n;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int n = *n_distinct;
    const int slices = (p.lora.K + kSlice - 1) / kSlice;
    const int s0 = slices * (int)rank / C, s1 = slices * ((int)rank + 1) / C;
    // D fp32, A and B bf16, both K-major, N / 8 at bits 17-22, M / 16 at 24-28
    constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NR >> 3) << 17) | (8u << 24);

    int stage = 0;  // of this thread's role; they go round together
    uint32_t phase = 0, pass = 0;
    bool ok = true;
    for (int d0 = 0; d0 < n; d0 += S::kGroup, ++pass) {
        const int group = min(S::kGroup, n - d0);
        if (warp == 0 && lane == 0) {
            for (int s = s0; s < s1 && ok; ++s) {
                ok = mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.lora.err, DERR_PRODUCER_WAIT);
                if (!ok) break;
                const uint32_t bar = full0 + 8 * stage, dst = base + stage * S::kStage;
                mbar_arrive_expect_tx(bar, kXBytes + group * p.lora.R * kSlice * 2);
                tma_load_2d(dst, &p.tm_x, s * kSlice, t0, bar);
                for (int a = 0; a < group; ++a)
                    tma_load_2d(dst + kXBytes + a * S::kABytes, &p.tm_a, s * kSlice, (int)distinct[d0 + a] * p.lora.R, bar);
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) {  // loads still on their way land before this CTA may leave
                const uint64_t t = global_timer();
                while (global_timer() - t < 1000000ull) {}
            }
        } else if (warp == 1 && lane == 0) {
            for (int s = s0; s < s1; ++s) {
                if (!mbar_wait(full0 + 8 * stage, phase, abort_flag, p.lora.err, DERR_MMA_FULL_WAIT)) break;
                tc_fence_after();
                const uint32_t at = base + stage * S::kStage;
                const uint64_t x = smem_desc(at);
                for (int a = 0; a < group; ++a) {
                    const uint64_t w = smem_desc(at + kXBytes + a * S::kABytes);
#pragma unroll
                    for (int k = 0; k < kSlice / 16; ++k)  // 32 bytes of K further: + 2 in the start address
                        mma_rank(tmem + a * NR, x + 2 * k, w + 2 * k, idesc, s > s0 || k > 0);
                }
                tc_commit(empty0 + 8 * stage);
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            tc_commit(done);
        } else if (warp >= 2) {
            const int q = warp & 3, r = 32 * q + lane;  // the TMEM lanes this warp may read; this thread's token
            const bool got = s1 > s0 && __all_sync(0xffffffffu, mbar_wait(done, pass & 1u, abort_flag, p.lora.err, DERR_EPI_WAIT));
            tc_fence_after();
            for (int a = 0; a < group; ++a) {
                const bool own = ids[r] == distinct[d0 + a];
#pragma unroll
                for (int c = 0; c < NR; c += 16) {
                    uint32_t v[16];
                    __syncwarp();  // the load is the whole warp's; lanes of other adapters are ahead here
                    if (got) {
                        tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + a * NR + c, v);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = 0u;
                    }
                    if (own) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<uint4*>(part + r * NR + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    }
                }
            }
            tc_fence_before();
        }
        __syncwarp();
        __syncthreads();  // the accumulators may be written again
        tc_fence_after();
    }
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");

    // the cluster's parts: rank o finishes rows o * 128 / C ...
    const int rows = kTokens / C, n_own = rows * NR;
    if (C > 1) {
        cluster_arrive();
        cluster_wait();  // nobody uses its stages any more
        for (int e = threadIdx.x; e < kTokens * NR; e += kShrinkThreads)
            store_to_rank(sent + rank * n_own + e % n_own, e / n_own, part[e]);
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    __nv_bfloat16* v = static_cast<__nv_bfloat16*>(p.lora.ws);
    for (int i = threadIdx.x; i < n_own; i += kShrinkThreads) {
        const int r = (int)rank * rows + i / NR, c = i % NR;
        const uint32_t a = ids[r];
        if (c >= p.lora.R || a == kNoAdapter) continue;
        float s = C > 1 ? sent[i] : part[i];
        for (int k = 1; k < C; ++k) s += sent[k * n_own + i];
        v[(int64_t)(t0 + r) * p.lora.R + c] = __float2bfloat16_rn(s * p.lora.scale[a]);
    }
}

template <int NR>
cudaError_t launch_shrink(const LoraTcArgs& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(lora_shrink_tc_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         ShrinkSmem<NR>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.parts;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((p.lora.T + kTokens - 1) / kTokens * p.parts);
    c.blockDim = dim3(kShrinkThreads);
    c.dynamicSmemBytes = ShrinkSmem<NR>::kBytes;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 2;
    return cudaLaunchKernelEx(&c, lora_shrink_tc_kernel<NR>, p);
}

// ---------------------------------------------------------------- expand --
// A stage holds 16 rows of base, kCols columns of each, fetched and put back
// row by row (bulk copies of up to 896 bytes; a multiple of 16, since rows and
// N are).  The pitch of 64 bytes more keeps a warp's 16-byte accesses to
// neighbouring rows in different banks.
// 7 warps of arithmetic and 1 of copies: with two CTAs an SM 128 registers a
// thread, which the arithmetic needs (8 + 1 warps spill at 96: 51 us for
// 8192 x 7168 instead of 46; the copies alone take 40).
constexpr int kExpandWarps = 7;
constexpr int kExpandThreads = 32 * (kExpandWarps + 1);

template <int KS>
struct ExpandSmem {
    static constexpr int kHalves = KS <= 4 ? 2 : 1;  // 32-column halves a warp holds B for
    static constexpr int kCols = kExpandWarps * 32 * kHalves;
    static constexpr int kPitch = kCols * 2 + 64;
    static constexpr int kStage = 16 * kPitch;
    static constexpr int kPerSm = KS <= 2 ? 2 : 1;
    static constexpr int kStages = KS <= 2 ? 6 : 12;
    static constexpr int kBars = kStages * kStage;  // full[S], ready[S]
    static constexpr int kBytes = kBars + 16 * kStages + 16;
};
// Staying CTAs: the grid is groups of as many CTAs as stages lie across a row;
// CTA c of group j takes column c of the group's row tiles, one after the
// other, so that what a group works on at one time lies together in memory and
// B stays in registers while the adapter does.
template <int KS>
__global__ void __launch_bounds__(kExpandThreads, ExpandSmem<KS>::kPerSm)
    lora_expand_tc_kernel(const __grid_constant__ LoraArgs p) {
    using S = ExpandSmem<KS>;
    constexpr int NH = S::kHalves;
    extern __shared__ __align__(128) uint8_t mem[];
    const uint32_t base = smem_u32(mem), full0 = base + S::kBars, ready0 = full0 + 8 * S::kStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(mem + S::kBars + 16 * S::kStages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int across = (p.N + S::kCols - 1) / S::kCols, tiles = (p.T + 15) / 16;
    const int groups = gridDim.x / across, group = blockIdx.x / across, col = blockIdx.x % across;
    const int tile0 = (int)((int64_t)tiles * group / groups), tile1 = (int)((int64_t)tiles * (group + 1) / groups);
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(ready0 + 8 * s, kExpandWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (warp == kExpandWarps) {
        // lane r < 16 copies row r of a tile
        const int bytes = 2 * min(S::kCols, p.N - col * S::kCols);
        const uint8_t* src = static_cast<const uint8_t*>(p.base) + 2 * (lane * p.base_stride + (int64_t)col * S::kCols);
        uint8_t* dst = static_cast<uint8_t*>(p.out) + 2 * (lane * p.out_stride + (int64_t)col * S::kCols);
        int load_s = 0, s = 0;
        uint32_t phase = 0;
        auto load = [&](int tile) {
            if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * load_s, bytes * min(16, p.T - tile * 16));
            __syncwarp();
            if (lane < 16 && tile * 16 + lane < p.T)
                bulk_load(base + load_s * S::kStage + lane * S::kPitch, src + 32 * tile * p.base_stride, bytes,
                          full0 + 8 * load_s);
            if (++load_s == S::kStages) load_s = 0;
        };
        // base does not come from the kernel before this one, which lets
        // this one start only after everything before it is done
        for (int tile = tile0; tile < min(tile1, tile0 + S::kStages); ++tile) load(tile);
        bool ok = true;
        for (int tile = tile0; tile < tile1; ++tile) {
            ok = __all_sync(0xffffffffu, mbar_wait(ready0 + 8 * s, phase, abort_flag, p.err, DERR_EPI_WAIT));
            if (!ok) break;
            if (lane < 16 && tile * 16 + lane < p.T)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + 32 * tile * p.out_stride),
                             "r"(base + s * S::kStage + lane * S::kPitch), "r"(bytes)
                             : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            // this lane's row of the tile before has left its stage: fill it again
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            if (tile > tile0 && tile - 1 + S::kStages < tile1) load(tile - 1 + S::kStages);
            if (++s == S::kStages) {
                s = 0;
                phase ^= 1u;
            }
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok) {  // loads still on their way land before this CTA may leave
            const uint64_t t = global_timer();
            while (global_timer() - t < 1000000ull) {}
        }
    } else {
        const int rv = p.R / 4;
        // this thread's first row and its chunk of the warp's first half
        uint8_t* const chunk = mem + g * S::kPitch + warp * 64 * NH + q * 16;
        const int n0 = col * S::kCols + warp * 32 * NH;  // this warp's first column
        wait_for_previous_kernel();
        int s = 0;
        uint32_t phase = 0, held = kNoAdapter;
        uint2 bf[NH][KS][4];
        uint32_t id_next[2];
        uint2 v_next[2][KS];
        auto fetch = [&](int tile) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = tile * 16 + 8 * h + g;
                const bool in = t < p.T;
                id_next[h] = adapter_of(p, t, in);
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    v_next[h][k] = in && k * 4 + q < rv ? static_cast<const uint2*>(p.ws)[(int64_t)t * rv + q + k * 4]
                                                        : make_uint2(0, 0);
            }
        };
        fetch(tile0);
        for (int tile = tile0; tile < tile1; ++tile) {
            uint32_t id[2], left[2];
            uint2 v[2][KS];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                left[h] = id[h] = id_next[h];
#pragma unroll
                for (int k = 0; k < KS; ++k) v[h][k] = v_next[h][k];
            }
            if (tile + 1 < tile1) fetch(tile + 1);
            auto next = [&] {
                const uint32_t m = __reduce_min_sync(0xffffffffu, min(left[0], left[1]));
                if (left[0] == m) left[0] = kNoAdapter;
                if (left[1] == m) left[1] = kNoAdapter;
                return m;
            };
            auto hold = [&](uint32_t a) {  // a's B in registers
                if (a != kNoAdapter && a != held) {
#pragma unroll
                    for (int h = 0; h < NH; ++h) Expand<KS>::load_b(p, a, n0 + 32 * h, lane, bf[h]);
                    held = a;
                }
            };
            uint32_t cur = next();
            hold(cur);
            if (!__all_sync(0xffffffffu, mbar_wait(full0 + 8 * s, phase, abort_flag, p.err, DERR_MMA_FULL_WAIT))) break;
            uint4* at = reinterpret_cast<uint4*>(chunk + s * S::kStage);
            constexpr int kRow8 = 8 * S::kPitch / 16;
            uint4 bs[NH][2];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                bs[h][0] = at[4 * h];
                bs[h][1] = at[4 * h + kRow8];
            }
            while (cur != kNoAdapter) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float d[4][4];
                    __syncwarp();  // the products are the whole warp's; lanes of other adapters are ahead here
                    Expand<KS>::product(bs[h], v, bf[h], d);
                    if (id[0] == cur) at[4 * h] = Expand<KS>::round(d, 0);
                    if (id[1] == cur) at[4 * h + kRow8] = Expand<KS>::round(d, 1);
                }
                cur = next();
                hold(cur);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(ready0 + 8 * s);
            if (++s == S::kStages) {
                s = 0;
                phase ^= 1u;
            }
        }
    }
}

template <int KS>
cudaError_t launch_expand(const LoraArgs& p, cudaStream_t s) {
    using S = ExpandSmem<KS>;
    cudaError_t e = cudaFuncSetAttribute(lora_expand_tc_kernel<KS>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    const int across = (p.N + S::kCols - 1) / S::kCols;
    const int groups = std::min((p.T + 15) / 16, std::max(1, S::kPerSm * p.n_sms / across));
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(groups * across);
    c.blockDim = dim3(kExpandThreads);
    c.dynamicSmemBytes = S::kBytes;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, lora_expand_tc_kernel<KS>, p);
}

}  // namespace

// Parts of K per tile of 128 tokens: as many (at most 8) as the SMs' two CTAs
// (one beyond rank 64) hold at once.
int lora_tc_parts(int64_t T, int R, int n_sms) {
    const int64_t tiles = (T + kTokens - 1) / kTokens;
    int parts = 8;
    while (parts > 1 && tiles * parts > (R > 64 ? 1 : 2) * n_sms) parts /= 2;
    return parts;
}

// Where these kernels take over from lora.cu's (here / there, us, 20 requests).
// 2048 x 1536, rank 64: 2048 tokens 20.7 / 18.5, 3000 22.7 / 28.5; 520 x 6000,
// rank 8: 18.7 / 16.5, 21.7 / 24.3; 7168 x 7168, rank 16: 1024 tokens 20.7 /
// 23.1, 1300 22.4 / 25.3, 2048 25.5 / 31.0.
bool lora_is_long(int64_t T, int64_t K, int64_t N) {
    return T > 2048 || (T >= kLoraMapTokens && T * (K + N) > 16 << 20);
}

cudaError_t launch_lora_tc(const LoraTcArgs& p, cudaStream_t s) {
    const int R = p.lora.R;
    const cudaError_t e = R <= 16 ? launch_shrink<16>(p, s) : R <= 32 ? launch_shrink<32>(p, s)
                          : R <= 64 ? launch_shrink<64>(p, s) : launch_shrink<128>(p, s);
    if (e != cudaSuccess) return e;
    return R <= 16 ? launch_expand<1>(p.lora, s) : R <= 32 ? launch_expand<2>(p.lora, s)
           : R <= 64 ? launch_expand<4>(p.lora, s) : launch_expand<8>(p.lora, s);
}

}  // namespace dwdp
