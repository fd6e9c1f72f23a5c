// lora.cu: low-rank adapters of many requests beside a shared projection
// (dwdp_lora_add): out[t] = base[t] + s_i (x[t] A_i^T) B_i^T, i the token's
// adapter.  Memory-bound: x, base, out and the used adapters once.
//
// A handful of tokens: one kernel (lora_one_kernel).  More, up to where
// lora_tc.cu takes over: two kernels, v = bf16(s_i x A_i^T) [T][R] between them:
//   shrink  a cluster of 2 to 8 CTAs per tile of up to 16 tokens, each warp a
//           part of K; the parts meet in distributed shared memory, in order
//   expand  token tile x 256 columns per CTA, base and out in 16-byte vectors
// Both take 16 tokens at a time against each adapter that occurs among them
// (mma m16n8k16) and give every row its own adapter's result, so tokens may
// come in any order, and values of one adapter never meet another's rows.
// v is rounded to bf16 because it is the second product's operand on bf16
// matrix instructions, whose other operand, B, is bf16 as given: the error of
// the result against 64 bits is 0.0018 of it instead of 0.0017 with v in
// binary32, of which the result's own rounding is most.
// A step is at most 2 R flops a byte of x: far from the tensor rate, so the
// warp-level MMA on operands straight from global memory is enough.
// 64 tokens of 64 adapters, 7168 x 7168, rank 16 (32 MB): 9.6 us, 3.3 TB/s;
// 517 tokens of 11 requests, 2048 x 1536, rank 64: 10.7 us.  What bounds both is
// the chain load, multiply, exchange in the cluster, launch, load, store.
#include <cuda_bf16.h>

#include <algorithm>

#include "dwdp_internal.h"
#include "lora_ops.h"

namespace dwdp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kNone = kNoAdapter;  // a row without an adapter
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ------------------------------------------------------ tokens by adapter --
// A batch whose tokens' adapters change from token to token costs a tile as
// many products as it has adapters.  So where they change at half of 32 places
// or more, tiles of more than 4 tokens take the tokens in the order of their
// adapters (stable, those without one last): every block finds the same order
// and keeps its own tile's part.  A row's result does not depend on its tile.
// 16 adapters at random, us without / with it: 7168 x 7168, rank 16: 128
// tokens 12.8 / 11.6, 256 17.7 / 12.1, 1000 60 / 31; 2048 x 1536, rank 64: 256
// 31 / 11.4, 1000 56 / 20.  Looking costs tokens that are in order 0.5 us (256
// of 20 requests 8.1 / 8.6).  The look takes the pairs 2 i, 2 i + 1, so a batch
// of two neighbouring tokens a request counts as in order (256 tokens of 16
// adapters, 7168 x 7168, rank 16: 13.8 us, at random 12.0, in order 6.5).
constexpr int kOrderTokens = 2048;  // at most
constexpr int kOrderLeast = 5;      // fewer have nothing to gain
constexpr int kOrderBins = 256;  // adapters, and one for tokens without
constexpr int kOrderRows = 64;   // of a tile at most

// Shared memory: start[bins], count[bins], sums[warps], then the pairs by chunk
// of 32 tokens and adapter, a byte each.
__host__ __device__ inline int order_pitch(const LoraArgs& p) { return (p.n_adapters + 4) / 4 * 4; }
bool may_order(const LoraArgs& p, int rows) {
    return rows > 4 && p.T >= kOrderLeast && p.T <= kOrderTokens && p.n_adapters < kOrderBins;
}
// Lane l looks at ids 2 i and 2 i + 1, i = order_place(T, l): with 2 tokens or
// more never beyond the last.
__host__ __device__ constexpr int order_place(int T, int lane) { return (int)((int64_t)lane * (T / 2) / 32); }
constexpr bool order_places_exist(int least, int most) {
    for (int T = least; T <= most; ++T)
        if (2 * order_place(T, 31) + 1 >= T) return false;
    return true;
}
static_assert(order_places_exist(kOrderLeast, kOrderTokens), "");
static_assert(!order_places_exist(1, 1) && order_places_exist(2, 2), "one token has no pair");
size_t order_bytes(const LoraArgs& p) {
    return (2 * kOrderBins + kWarps) * 4 + (size_t)((p.T + 31) / 32) * order_pitch(p);
}

// Whether the tile at t0 takes tokens order[0 .. rows) (p.T: none) instead of
// t0, t0 + 1, ...  Called by the whole block.
__device__ __forceinline__ bool order_tile(const LoraArgs& p, int t0, int rows, void* mem, int* order) {
    constexpr int kMine = kOrderTokens / kThreads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // neighbours at 32 places of the batch, the same for every warp; and the
    // tile's own ids on their way
    const int2 two = reinterpret_cast<const int2*>(p.ids)[order_place(p.T, lane)];
    const int own = p.ids[min(t0 + lane, p.T - 1)];
    asm volatile("" ::"r"(own));
    if (__popc(__ballot_sync(kFull, two.x != two.y)) < 16) return false;
    int bin[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        bin[i] = -1;
        if (i * kThreads >= p.T) continue;
        const int t = (warp + kWarps * i) * 32 + lane;
        bin[i] = t < p.T ? (int)min(adapter_of(p, t, true), (uint32_t)p.n_adapters) : -1;
    }
    int *const start = static_cast<int*>(mem), *const count = start + kOrderBins, *const sums = count + kOrderBins;
    uint8_t* const in_chunk = reinterpret_cast<uint8_t*>(sums + kWarps);
    const int pitch = order_pitch(p), words = (p.T + 31) / 32 * pitch / 4;
    count[tid] = 0;
    for (int i = tid; i < words; i += kThreads) reinterpret_cast<uint32_t*>(in_chunk)[i] = 0;
    if (tid < rows) order[tid] = p.T;
    __syncthreads();
    int before[kMine] = {};  // of the same adapter in the chunk
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        if (i * kThreads >= p.T) continue;
        const uint32_t same = __match_any_sync(kFull, bin[i]);
        before[i] = __popc(same & ((1u << lane) - 1u));
        if (bin[i] >= 0 && before[i] == 0) {
            in_chunk[(warp + kWarps * i) * pitch + bin[i]] = (uint8_t)__popc(same);
            atomicAdd(count + bin[i], __popc(same));
        }
    }
    __syncthreads();
    int at = count[tid];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += u;
    }
    if (lane == 31) sums[warp] = at;
    __syncthreads();
    at -= count[tid];
    for (int w = 0; w < warp; ++w) at += sums[w];
    start[tid] = at;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int b = max(bin[i], 0), chunk = warp + kWarps * i;
        int r = start[b] - t0;
        if (bin[i] >= 0 && r < rows && r + count[b] > 0) {
            r += before[i];
            for (int c = 0; c < chunk; ++c) r += in_chunk[c * pitch + b];
            if (r >= 0 && r < rows) order[r] = chunk * 32 + lane;
        }
    }
    __syncthreads();
    return true;
}

// 16 rows of x against A_i: a cluster of C blocks of 8 warps, each warp a part
// of K; NT n8 tiles hold the rank.  A step is 32 elements of K.
template <int NT, int C>
struct Shrink {
    static constexpr int kTile = 16 * NT * 8;
    static constexpr int kSmem = (kWarps + 1) * kTile * 4;

    // G adapters against the warp's rows, one reading of x, U steps' loads in
    // flight.  Loads are in bounds without a predicate: a row without an
    // adapter (or beyond the batch) reads some row of x, an adapter that is
    // none adapter 0, a row of A beyond R the last one, and nothing of them
    // is used.
    template <int G, int U>
    static __device__ __forceinline__ void pass(const LoraArgs& p, const uint4* const (&xr)[2],
                                                const uint32_t (&cur)[G], int step0, int step1, int lane,
                                                const uint32_t (&id)[2], float* part) {
        const int g = lane >> 2, q = lane & 3, kv = p.K / 8;
        float acc[G][NT][4] = {};
        const uint4* xp[2];
        const uint4* ap[G][NT];
#pragma unroll
        for (int i = 0; i < 2; ++i) xp[i] = xr[i] + step0 * 4 + q;
#pragma unroll
        for (int s = 0; s < G; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                ap[s][j] = static_cast<const uint4*>(p.a) +
                           ((int64_t)(cur[s] == kNone ? 0 : cur[s]) * p.R + min(j * 8 + g, p.R - 1)) * kv + step0 * 4 + q;
        // U steps from `at`; `last`: the part's or the row's end may lie within them
        auto steps = [&](int at, bool last) {
            uint4 xv[U][2], av[U][G][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = !last || (at + u < step1 && (at + u) * 4 + q < kv);
#pragma unroll
                for (int s = 0; s < G; ++s)
#pragma unroll
                    for (int j = 0; j < NT; ++j) av[u][s][j] = in ? __ldg(ap[s][j] + 4 * u) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 2; ++i) xv[u][i] = in ? __ldg(xp[i] + 4 * u) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < G; ++s)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint4 &lo = xv[u][0], &hi = xv[u][1], &b = av[u][s][j];
                        mma16816(acc[s][j], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
                        mma16816(acc[s][j], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
                    }
#pragma unroll
            for (int i = 0; i < 2; ++i) xp[i] += 4 * U;
#pragma unroll
            for (int s = 0; s < G; ++s)
#pragma unroll
                for (int j = 0; j < NT; ++j) ap[s][j] += 4 * U;
        };
        const int whole = min(step1, kv / 4);  // steps that lie wholly in the part and the row
#pragma unroll 1
        for (int st = step0; st < step1; st += U) steps(st, st + U > whole);
#pragma unroll
        for (int s = 0; s < G; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (id[i] != kNone && id[i] == cur[s]) {
                    float* row = part + (i * 8 + g) * NT * 8 + 2 * q;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        *reinterpret_cast<float2*>(row + j * 8) = make_float2(acc[s][j][2 * i], acc[s][j][2 * i + 1]);
                }
    }
};

// The tile's partial sums over this block's part of K in part[0] ([16][NT * 8]
// floats of shared memory for every warp); rows without an adapter hold
// anything.  token(r): the tile's r-th token, p.T or more: none.  Ends with the
// block in step.
template <int NT, int C, class Token>
__device__ __forceinline__ void shrink_tile(const LoraArgs& p, Token token, int tile_rows, uint32_t rank, float* part) {
    using S = Shrink<NT, C>;
    // adapters a mixed pass takes at once, and steps in flight with one and
    // with several: what the registers hold
    constexpr int G = NT <= 2 ? 4 : NT <= 4 ? 2 : 1;
    constexpr int U1 = NT <= 2 ? 4 : NT <= 8 ? 2 : 1, UG = 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    uint32_t id[2], left[2];
    const uint4* xr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = i * 8 + g, t = r < tile_rows ? token(r) : p.T;
        const bool in = t < p.T;
        left[i] = id[i] = adapter_of(p, t, in);
        xr[i] = static_cast<const uint4*>(p.x) + (int64_t)(in ? t : 0) * (p.x_stride / 8);
        if (rank == 0 && warp == 0 && in && id[i] == kNone && p.ids[t] != -1) atomicOr(p.err, DERR_BAD_INDEX);
    }
    const int steps = (p.K + 31) / 32, at = (int)rank * kWarps + warp;
    const int step0 = steps * at / (C * kWarps), step1 = steps * (at + 1) / (C * kWarps);
    float* mine = part + warp * S::kTile;
    // the lowest adapter among the rows not done yet
    auto next = [&] {
        const uint32_t m = __reduce_min_sync(kFull, min(left[0], left[1]));
        if (left[0] == m) left[0] = kNone;
        if (left[1] == m) left[1] = kNone;
        return m;
    };
    uint32_t a0 = next();
    while (a0 != kNone) {
        const uint32_t a1 = next();
        if (G == 1 || a1 == kNone) {
            const uint32_t cur[1] = {a0};
            S::template pass<1, U1>(p, xr, cur, step0, step1, lane, id, mine);
            a0 = a1;
        } else {
            uint32_t cur[G];
            cur[0] = a0;
#pragma unroll
            for (int s = 1; s < G; ++s) cur[s] = s == 1 ? a1 : next();
            S::template pass<G, UG>(p, xr, cur, step0, step1, lane, id, mine);
            a0 = next();
        }
    }
    __syncthreads();
}

template <int NT, int C, bool ORDER>
__global__ void __launch_bounds__(kThreads, NT <= 8 ? 2 : 1) __cluster_dims__(C, 1, 1)
    lora_shrink_kernel(const __grid_constant__ LoraArgs p, int tile_rows) {
    using S = Shrink<NT, C>;
    extern __shared__ float part[];  // [warps][16][NT * 8], then what the cluster sends [C][this rank's share]
    __shared__ int order[kOrderRows];
    wait_for_previous_kernel();
    let_next_kernel_start();
    cluster_arrive();
    const int t0 = (int)(blockIdx.x / C) * tile_rows;
    const uint32_t rank = cluster_rank();
    const bool ordered = ORDER && order_tile(p, t0, tile_rows, part, order);
    auto token = [&](int r) { return ordered ? order[r] : t0 + r; };
    shrink_tile<NT, C>(p, token, tile_rows, rank, part);
    // the K parts of the block, then of the cluster: rank e / share gets
    // element e of every rank, and adds them in order
    const int n = tile_rows * NT * 8, share = n / C;
    float* sent = part + kWarps * S::kTile;
    cluster_wait();  // everybody runs: its shared memory may be written
    for (int e = threadIdx.x; e < n; e += kThreads) {
        float s = part[e];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s += part[w * S::kTile + e];
        store_to_rank(sent + rank * share + e % share, e / share, s);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    __nv_bfloat16* v = static_cast<__nv_bfloat16*>(p.ws);
    for (int i = threadIdx.x; i < share; i += kThreads) {
        const int e = (int)rank * share + i, r = e / (NT * 8), c = e % (NT * 8), t = token(r);
        if (c >= p.R) continue;
        const uint32_t a = adapter_of(p, t, t < p.T);
        if (a == kNone) continue;
        float s = sent[i];
#pragma unroll
        for (int k = 1; k < C; ++k) s += sent[k * share + i];
        v[(int64_t)t * p.R + c] = __float2bfloat16_rn(s * p.scale[a]);
    }
}

// A handful of tokens in one kernel: a cluster of 8 blocks takes one token and
// 2048 columns.  Its blocks share K for the first product, send every partial
// sum to every block, and each goes on with 256 of the columns, whose base and
// B it fetched at the start.  Other clusters compute the same v for other
// columns.  One token, 7168 x 7168, rank 16: 3.4 us against the two kernels'
// 4.4, and one launch less (2 us of a call from Python).  Latency-bound: the
// bytes alone would take 0.07 us.
template <int NT>
__global__ void __launch_bounds__(kThreads) __cluster_dims__(8, 1, 1)
    lora_one_kernel(const __grid_constant__ LoraArgs p, int) {
    constexpr int C = 8, KS = NT / 2, kRank = NT * 8;
    using X = Expand<KS>;
    extern __shared__ float part[];  // [warps][16][NT * 8]
    __shared__ float sent[C * kRank];  // what the cluster sends
    __shared__ __align__(8) __nv_bfloat16 vs[kRank];
    wait_for_previous_kernel();
    let_next_kernel_start();
    cluster_arrive();
    const uint32_t rank = cluster_rank();
    const int wide = (p.N + 2047) / 2048, cluster = blockIdx.x / C, t = cluster / wide;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int c0 = ((cluster % wide) * C + (int)rank) * 256 + warp * 32;
    const bool mine = g == 0 && c0 + 8 * q < p.N;  // the MMA's first row is the token's
    const uint32_t id = adapter_of(p, t, true);
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint4 bs[2] = {mine ? *(static_cast<const uint4*>(p.base) + t * (p.base_stride / 8) + c0 / 8 + q) : none, none};
    uint2 bf[KS][4];
    X::load_b(p, id, min(c0, p.N - 8), lane, bf);
    shrink_tile<NT, C>(p, [&](int) { return t; }, 1, rank, part);
    cluster_wait();  // everybody runs: its shared memory may be written
    for (int e = threadIdx.x; e < kRank; e += kThreads) {
        float s = part[e];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s += part[w * Shrink<NT, C>::kTile + e];
#pragma unroll
        for (int c = 0; c < C; ++c) store_to_rank(sent + rank * kRank + e, c, s);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (int e = threadIdx.x; e < kRank; e += kThreads) {
        float s = sent[e];
#pragma unroll
        for (int k = 1; k < C; ++k) s += sent[k * kRank + e];
        vs[e] = __float2bfloat16_rn(id != kNone && e < p.R ? s * p.scale[id] : 0.0f);
    }
    __syncthreads();
    uint2 vf[2][KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        vf[0][s] = g == 0 ? *reinterpret_cast<const uint2*>(vs + s * 16 + 4 * q) : make_uint2(0, 0);
        vf[1][s] = make_uint2(0, 0);
    }
    float d[4][4];
    X::product(bs, vf, bf, d);
    // a token without an adapter keeps base's bits
    if (mine) *(static_cast<uint4*>(p.out) + t * (p.out_stride / 8) + c0 / 8 + q) = id != kNone ? X::round(d, 0) : bs[0];
}

// A warp takes MT m16 tiles and 32 columns.  base is the accumulator's start,
// so a row's result does not depend on the tile's other rows.
template <int KS, int MT, bool ORDER>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(const __grid_constant__ LoraArgs p, int tile_rows) {
    using X = Expand<KS>;
    constexpr int G = MT > 1 || KS > 1 ? 1 : 2;  // adapters whose B is loaded together
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int t0 = (int)blockIdx.x * tile_rows, c0 = ((int)blockIdx.y * (kThreads / 32) + warp) * 32;
    __shared__ int order[kOrderRows];
    extern __shared__ int order_mem[];
    const bool col_in = c0 + 8 * q < p.N;
    const int rv = p.R / 4;
    // base and the ids do not come from the kernel before this one, which
    // lets this one start only after everything before it is done
    uint32_t id[MT][2], most = 0, least = kNone;
    uint4 bs[MT][2];
    int token[MT][2];  // p.T: none
    const uint4* base = static_cast<const uint4*>(p.base) + c0 / 8 + q;
    auto fetch = [&](auto of) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = m * 16 + h * 8 + g, t = token[m][h] = r < tile_rows ? of(r) : p.T;
                bs[m][h] = t < p.T && col_in ? base[t * (p.base_stride / 8)] : make_uint4(0, 0, 0, 0);
                id[m][h] = adapter_of(p, t, t < p.T);
            }
    };
    fetch([&](int r) { return min(t0 + r, p.T); });
    if (ORDER && order_tile(p, t0, tile_rows, order_mem, order)) fetch([&](int r) { return order[r]; });
    if (c0 >= p.N) return;  // a whole warp beyond the columns
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            most = max(most, id[m][h]);
            least = min(least, id[m][h]);
        }
    least = __reduce_min_sync(kFull, least);
    most = __reduce_max_sync(kFull, most);
    const uint2* v = static_cast<const uint2*>(p.ws) + q;
    uint4* out = static_cast<uint4*>(p.out) + c0 / 8 + q;
    uint2 bf[G][KS][4];
    if (MT > 1 && least == most && least != kNone) {  // one adapter, every row in use
        X::load_b(p, least, c0, lane, bf[0]);
        wait_for_previous_kernel();
        uint2 vf[MT][2][KS];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    vf[m][h][s] = s * 4 + q < rv ? v[(int64_t)token[m][h] * rv + s * 4] : make_uint2(0, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float d[4][4];
            X::product(bs[m], vf[m], bf[0], d);
            if (col_in) {
                out[token[m][0] * (p.out_stride / 8)] = X::round(d, 0);
                out[token[m][1] * (p.out_stride / 8)] = X::round(d, 1);
            }
        }
        return;
    }
    uint32_t held = kNone;  // G == 1: the adapter bf holds
    bool waited = false;
#pragma unroll 1
    for (int m = 0; m < MT; ++m) {
        uint32_t mid[2] = {id[0][0], id[0][1]};
        uint4 mb[2] = {bs[0][0], bs[0][1]};
        int mt[2] = {token[0][0], token[0][1]};
#pragma unroll
        for (int i = 1; i < MT; ++i)  // (constant indexes keep the arrays in registers)
            if (i == m) {
                mid[0] = id[i][0];
                mid[1] = id[i][1];
                mb[0] = bs[i][0];
                mb[1] = bs[i][1];
                mt[0] = token[i][0];
                mt[1] = token[i][1];
            }
        uint32_t left[2] = {mid[0], mid[1]};
        uint2 vf[2][KS];
        uint4 o[2] = {mb[0], mb[1]};  // a row without an adapter keeps base's bits
        for (bool first = true;; first = false) {
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
                for (int s = 0; s < G; ++s)
                    if (s == 0 || cur[s] != kNone) X::load_b(p, cur[s], c0, lane, bf[s]);
                held = cur[0];
            }
            if (!waited) wait_for_previous_kernel();
            waited = true;
            if (first)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int s = 0; s < KS; ++s)
                        vf[h][s] = mid[h] != kNone && s * 4 + q < rv ? v[(int64_t)mt[h] * rv + s * 4]
                                                                     : make_uint2(0, 0);
#pragma unroll
            for (int s = 0; s < G; ++s) {
                if (cur[s] == kNone) continue;
                float d[4][4];
                X::product(mb, vf, bf[s], d);
                if (mid[0] == cur[s]) o[0] = X::round(d, 0);
                if (mid[1] == cur[s]) o[1] = X::round(d, 1);
            }
        }
        // a tile without adapters has waited for nothing: out may be base,
        // which only this thread reads
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (mt[h] < p.T && col_in) out[mt[h] * (p.out_stride / 8)] = o[h];
    }
    if (!waited) wait_for_previous_kernel();
}

cudaError_t launch(const void* kernel, dim3 grid, size_t smem, cudaStream_t s, const LoraArgs& p, int tile_rows) {
    if (smem > 40 << 10) {  // beside the static part, beyond what a launch gets unasked
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

template <int NT, int C>
cudaError_t launch_shrink(const LoraArgs& p, int rows, cudaStream_t s) {
    const bool order = may_order(p, rows);
    const size_t smem = std::max((size_t)Shrink<NT, C>::kSmem, order ? order_bytes(p) : 0);
    const void* kernel = order ? (const void*)lora_shrink_kernel<NT, C, true> : (const void*)lora_shrink_kernel<NT, C, false>;
    return launch(kernel, dim3((p.T + rows - 1) / rows * C), smem, s, p, rows);
}

template <int KS, int MT>
cudaError_t launch_expand(const LoraArgs& p, int rows, int cols, cudaStream_t s) {
    const bool order = may_order(p, rows);
    const void* kernel = order ? (const void*)lora_expand_kernel<KS, MT, true> : (const void*)lora_expand_kernel<KS, MT, false>;
    return launch(kernel, dim3((p.T + rows - 1) / rows, cols), order ? order_bytes(p) : 0, s, p, rows);
}

template <int NT>
cudaError_t launch_rank(const LoraArgs& p, cudaStream_t s) {
    if constexpr (NT <= 8) {
        // one kernel while its clusters fit the GPU at once (rank 128 is slower so)
        const int64_t blocks = (int64_t)p.T * ((p.N + 2047) / 2048) * 8;
        if (p.T <= 16 && blocks <= p.n_sms * 4 / 5)
            return launch((const void*)lora_one_kernel<NT>, dim3((unsigned)blocks),
                          (size_t)kWarps * Shrink<NT, 8>::kTile * 4, s, p, 1);
    }
    // shrink: the smallest tiles, then the fewest parts of K, whose clusters
    // fit the GPU at once with a block per SM (a cluster that has to wait for
    // another one's end costs more: 128 tokens of one adapter, rank 16, 8.0 us
    // so, 5.1 us in one round).  Blocks of 8-block clusters that cannot share
    // an SM (rank above 64) leave a fifth of the SMs in the gaps.
    auto fits = [&](int rows, int C) {
        return (int64_t)((p.T + rows - 1) / rows) * C <= p.n_sms * (NT == 16 && C == 8 ? 4 : 5) / 5;
    };
    int rows = 1;
    while (rows < 16 && !fits(rows, 8)) rows *= 2;
    const cudaError_t e = fits(rows, 8) ? launch_shrink<NT, 8>(p, rows, s)
                          : fits(rows, 4) ? launch_shrink<NT, 4>(p, rows, s) : launch_shrink<NT, 2>(p, rows, s);
    if (e != cudaSuccess) return e;
    // expand: 64 tokens a warp where that leaves every SM two blocks
    constexpr int KS = NT / 2;
    const int cols = (p.N + 255) / 256;
    if ((int64_t)((p.T + 63) / 64) * cols >= 2 * p.n_sms)
        return launch_expand<KS, 4>(p, 64, cols, s);
    return launch_expand<KS, 1>(p, rows, cols, s);
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
