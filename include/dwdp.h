/*
 * dwdp.h: C ABI of libdwdp.so, the single-rank hot path of DWDP
 * (Distributed Weight Data Parallelism) on one GB300 (sm_103a).
 *
 * Sources, cited by page title and section:
 *   [DWDP] "DWDP: Distributed Weight Data Parallelism for High-Performance LLM
 *          Inference on NVL72" (arXiv 2604.01621), as summarised on its
 *          summary pages;
 *   [news] the thecoregrid.dev news summary of the same paper.
 *
 * One rank runs one MoE block per layer.  Some experts of each layer are
 * resident ("local"); the others live on peers and are pulled into one of the
 * staging buffers (two by default: double buffering) by asynchronous copies
 * while the previous layer computes ([DWDP] §2 Methodology Overview).  The grouped GEMM reads each expert from
 * whichever buffer holds it through a per-expert table, with no merge copy
 * ([DWDP] §4.2).  Copies are cut into fixed-size slices issued round-robin
 * over the sources ([DWDP] §4.3.2; [news]).  On one GPU the peers are emulated
 * by separate device-memory pools.
 *
 * Conventions for every call:
 *   - bf16 tensors are raw 16-bit IEEE bfloat16; every matrix is row-major
 *     with no padding between rows.
 *   - "device" pointers point into the current CUDA device's global memory
 *     and must be 16-byte aligned; the caller owns every buffer it passes and
 *     keeps it alive until the work enqueued on it has finished.  Buffers
 *     the GEMMs read through TMA tensor maps (x, the workspace, the router
 *     weight, the local pool, the shared expert, the staging buffers) are
 *     checked to be device memory of the context's (current) device, else
 *     INVALID_ARG: the kernels never read another GPU's or the host's memory
 *     through a tensor map.  Only peer pools, which are copied from and
 *     never read by a kernel, may live elsewhere.
 *   - The context owns its CUDA events, tensor-map descriptors, its small
 *     device tables and error word, and the copy plans.  Use one context from
 *     one host thread at a time.
 *   - Every call validates its arguments on the host first.  A negative
 *     return means nothing was enqueued; dwdp_last_error() says why.
 *     Asynchronous CUDA faults surface as DWDP_ERR_CUDA from a later call.
 *   - Kernels never trap.  A bounded wait inside a kernel that runs out sets
 *     the context's device error word and returns; dwdp_device_status()
 *     reports it as DWDP_ERR_DEVICE_CHECK.
 *
 * Weight layouts:
 *   w13 of one expert : [2I][H]  rows 0..I-1 = W_gate^T, rows I..2I-1 = W_up^T
 *   w2  of one expert : [H][I]   = W_down^T
 *   a pool            : w13 [n_slots][2I][H] and w2 [n_slots][H][I]
 *   router weight     : [E][H]   row e = column e of the H x E gate matrix
 * Expert weights are bf16, 1-byte E4M3 codes in an E4M3 context, or NVFP4
 * slots (see DWDP_DTYPE_NVFP4) in an NVFP4 context; the router weight and
 * the activations passed in and out are always bf16.
 */
#ifndef DWDP_H_
#define DWDP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DWDP_ABI_VERSION 5
#define DWDP_MAX_EXPERTS 1024
#define DWDP_MAX_TOPK 32
#define DWDP_MAX_LAYERS 256
#define DWDP_MAX_PEERS 64
#define DWDP_MAX_GROUPS 32
#define DWDP_MAX_LORA_RANK 128

typedef struct dwdp_ctx dwdp_ctx;
/* Same object as cudaStream_t; NULL = the legacy default stream. */
typedef struct CUstream_st* dwdp_stream_t;

typedef enum {
    DWDP_OK = 0,
    DWDP_ERR_INVALID_ARG = -1,  /* bad pointer, size, index or alignment */
    DWDP_ERR_NOT_MAPPED = -2,   /* layer has no expert map, or stage holds another layer */
    DWDP_ERR_CUDA = -3,         /* a CUDA runtime call failed */
    DWDP_ERR_TIMEOUT = -4,      /* dwdp_wait_stage ran out of time */
    DWDP_ERR_UNSUPPORTED = -5,  /* shape outside what the kernels handle */
    DWDP_ERR_DEVICE_CHECK = -6  /* a kernel reported a failed check or wait */
} dwdp_status;

typedef struct {
    int32_t hidden;       /* H: multiple of 64 (NVFP4: of 256) */
    int32_t inter;        /* I: expert intermediate size, multiple of 64 (NVFP4: of 256) */
    int32_t n_experts;    /* E: routed experts, 1..DWDP_MAX_EXPERTS */
    int32_t top_k;        /* k: 1..min(E, DWDP_MAX_TOPK) */
    int32_t n_shared;     /* always-on shared experts: 0 or 1 */
    int32_t max_tokens;   /* largest T any call will pass */
    int32_t n_layers;     /* layers that get an expert map: 1..DWDP_MAX_LAYERS */
    int32_t stage_slots;  /* experts each staging buffer holds (0 = no staging) */
    int32_t weight_dtype; /* DWDP_DTYPE_BF16, DWDP_DTYPE_E4M3 or DWDP_DTYPE_NVFP4 */
    int32_t n_stages;     /* staging buffers: 0 = 2 (the pages' double buffering); 1..DWDP_MAX_STAGES */
    int32_t flags;        /* DWDP_FLAG_* (0 = defaults) */
} dwdp_config;

/* NVFP4 contexts: the gate/up GEMM drains its one TMEM accumulator with
 * eight epilogue warps (two per lane quarter) instead of four, so the next
 * tile's MMAs start sooner.  Faster when the GEMM runs alone; on one GPU a
 * copy-engine prefetch running beside it then gets much less of the memory
 * system (the copy, and with it the overlapped layer, takes longer), so it
 * is off by default.  Ignored by bf16 and E4M3 contexts. */
#define DWDP_FLAG_WIDE_EPILOGUE 1

#define DWDP_MAX_STAGES 4

/* Expert weight types.  DWDP_DTYPE_E4M3 (an FP8 variant of the layer; the
 * pages run NVFP4 expert weights, DWDP §5.1): pools and stage buffers hold
 * 1-byte E4M3 codes (w = code * scale, one scale per expert tensor, given by
 * dwdp_set_expert_scales); the layer quantizes its activations per row to
 * E4M3 (scale = row amax / 448, binary32, round-to-nearest-even,
 * saturating) before each expert GEMM, and the GEMMs run on FP8 tensor
 * cores.  Routing stays bf16. */
#define DWDP_DTYPE_BF16 0
#define DWDP_DTYPE_E4M3 1
/* DWDP_DTYPE_NVFP4 (the format the pages run DeepSeek-R1's MoE weights in,
 * DWDP §5.1): a weight is an E2M1 code (4 bits) times an E4M3 scale shared by
 * 16 consecutive elements along K, times one binary32 scale per expert tensor
 * (dwdp_set_expert_scales).  One pool slot of a [rows][K] tensor (w13: rows =
 * 2I, K = H; w2: rows = H, K = I) is rows * K * 9 / 16 bytes:
 *   - codes [rows][K / 2] bytes, element 2i of a row in the low nibble of
 *     byte i, 2i + 1 in the high nibble;
 *   - then the block scales in 512-byte chunks, one per (row block rb of 128
 *     rows, K step ks of 64 elements), chunk (rb, ks) at (rb * K / 64 + ks) *
 *     512; in it the scale of row 128 rb + 32 m1 + m0 and 16-element block kb
 *     of the step is byte 16 m0 + 4 m1 + kb.
 * The layer quantizes its activations per row to NVFP4 before each expert
 * GEMM (row scale = row amax / 2688 in binary32; block scale = E4M3 of block
 * amax / (6 * row scale); code = E2M1 of v / (block scale * row scale), round
 * to nearest even, saturating) and the GEMMs run on the block-scaled FP4
 * tensor cores.  H and I must be multiples of 256. */
#define DWDP_DTYPE_NVFP4 2

/* One buffer of experts: w13 [n_slots][2I][H], w2 [n_slots][H][I] (device;
 * NVFP4: n_slots slots of the sizes given at DWDP_DTYPE_NVFP4). */
typedef struct {
    const void* w13;
    const void* w2;
    int32_t n_slots;
} dwdp_pool;

/* Routing results (all device pointers, written by dwdp_route).
 *   topk_ids [T][k]  chosen experts of each token, ascending expert id
 *   topk_w   [T][k]  their weights: softmax renormalised over the chosen k
 *   counts   [E]     (token, slot) pairs routed to each expert
 *   offsets  [E+1]   exclusive scan of counts; offsets[E] = T*k
 *   perm     [T*k]   flat index t*k+j of the pair at grouped row r; within an
 *                    expert, rows keep ascending flat index
 *   inv_perm [T*k]   grouped row of pair t*k+j
 *   logits   [T][E]  fp32 router logits x.Wr (+ bias); NULL = not returned.
 *                    With few tokens the router GEMM splits K into up to 4
 *                    parts summed in order: the logits are the ones the
 *                    choice was made on, deterministic for a given device
 *                    and shape. */
typedef struct {
    int32_t* topk_ids;
    float* topk_w;
    int32_t* counts;
    int32_t* offsets;
    int32_t* perm;
    int32_t* inv_perm;
    float* logits;
} dwdp_route_out;

/* One slice of a prefetch copy plan.  tensor 0 = w13, 1 = w2; offsets are in
 * bytes from the start of the peer pool's tensor and the stage buffer's
 * tensor. */
typedef struct {
    int32_t peer;
    int32_t tensor;
    int64_t src_offset;
    int64_t dst_offset;
    int64_t nbytes;
} dwdp_copy_slice;

/* ABI version of the loaded library (DWDP_ABI_VERSION). */
int32_t dwdp_version(void);

/* Create a context on the current CUDA device.  stage_w13[s] / stage_w2[s]
 * (s = 0 .. n_stages - 1, n_stages = cfg->n_stages or 2 when that is 0) are
 * the caller's staging buffers ([DWDP] §2: double buffering; a third stage
 * lets the copy of layer l + 2 start while layer l computes, so the copy
 * stream can run back to back), each [stage_slots][2I][H] /
 * [stage_slots][H][I] in the weight format; they may be NULL when
 * cfg->stage_slots == 0.  On success *out owns the events and descriptors
 * listed above.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_create(const dwdp_config* cfg, void* const stage_w13[], void* const stage_w2[],
                    dwdp_ctx** out);

/* Destroy a context (waits for nothing; the caller synchronises first). */
void dwdp_destroy(dwdp_ctx* ctx);

/* Text of the last error on this context (or of the last failed
 * dwdp_create / host helper when ctx is NULL).  Never NULL. */
const char* dwdp_last_error(const dwdp_ctx* ctx);

/* Device workspace, in bytes, that dwdp_route, dwdp_route_scored and
 * dwdp_moe_layer (_codes) need for T tokens (the largest of them; they may
 * share one buffer when they run in order on one stream). */
size_t dwdp_workspace_bytes(const dwdp_ctx* ctx, int32_t T);

/* Where dwdp_moe_layer keeps each intermediate of a T-token layer in its
 * workspace (instrumentation: after the layer has run, and until the next
 * call that uses the workspace, the caller may read them back).  Regions,
 * with rows_r = T k routed rows in expert order (dwdp_route's grouped rows)
 * and rows_all = T (k + n_shared) (the shared expert's rows after them):
 *   DWDP_WS_XP  [rows_r][H] x in expert order (bf16, E4M3 or NVFP4 codes)
 *   DWDP_WS_A   [rows_all][I] bf16 a = SiLU(gate) * up
 *   DWDP_WS_Y   [rows_all][H] bf16 expert outputs y
 *   DWDP_WS_XQ  [T][H] x's codes (E4M3 / NVFP4 contexts)
 *   DWDP_WS_SX, DWDP_WS_SXP  fp32 row scales of x by token / in expert order
 *   DWDP_WS_AQ  [rows_all][I] a's codes; DWDP_WS_SA [rows_all] fp32 a's row scales
 *   DWDP_WS_SFX, DWDP_WS_SFA  NVFP4 block scales of the gate/up and down
 *     GEMMs' A operands in the 512-byte chunk layout, chunk (tile, ks) at
 *     (tile * K / 64 + ks) * 512, where the A tiles are numbered expert by
 *     expert (ceil(rows_e / 128) tiles each, in expert order), then the
 *     shared expert's ceil(T / 128) tiles.
 * Writes the byte offset from ws and the region's size (0 when the context's
 * weight type has no such region).  Errors: INVALID_ARG. */
#define DWDP_WS_XP 0
#define DWDP_WS_A 1
#define DWDP_WS_Y 2
#define DWDP_WS_XQ 3
#define DWDP_WS_SX 4
#define DWDP_WS_SXP 5
#define DWDP_WS_AQ 6
#define DWDP_WS_SA 7
#define DWDP_WS_SFX 8
#define DWDP_WS_SFA 9
int32_t dwdp_workspace_region(const dwdp_ctx* ctx, int32_t T, int32_t region, size_t* offset, size_t* bytes);

/* Placement of layer `layer` ([DWDP] §2: experts partitioned across peers,
 * placement need not be disjoint; a redundant expert is read from its local
 * copy).  For each routed expert e:
 *   local_slot[e] >= 0  -> resident in `local` at that slot;
 *   otherwise peer_id[e] in [0, n_peers) and peer_slot[e] name its copy in
 *   peers[peer_id[e]], and it is staged by dwdp_prefetch_layer.
 * local_slot, peer_id, peer_slot are host arrays [E]; local and peers are host
 * structs describing device buffers (a peer pool may instead be pinned host
 * memory: its slices then cross the host link, and only their writes land in
 * this GPU's memory).  shared_w13 [2I][H] / shared_w2 [H][I]
 * (device) are the layer's shared expert, required iff n_shared == 1.  The
 * non-resident experts take stage slots 0, 1, ... in ascending id, at most
 * stage_slots of them.  Replaces any earlier map of the layer (the caller
 * makes sure no enqueued work still uses it).  Errors: INVALID_ARG, CUDA. */
int32_t dwdp_set_expert_map(dwdp_ctx* ctx, int32_t layer, const dwdp_pool* local,
                            const dwdp_pool* peers, int32_t n_peers, const int32_t* local_slot,
                            const int32_t* peer_id, const int32_t* peer_slot,
                            const void* shared_w13, const void* shared_w2);

/* Per-expert-tensor weight scales of layer `layer` for DWDP_DTYPE_E4M3 and
 * DWDP_DTYPE_NVFP4 contexts: expert e's gate/up weights are the w13 codes'
 * values * w13_scale[e], its down weights the w2 codes' values * w2_scale[e]
 * (host arrays [E]; NVFP4: on top of the block scales); shared_* for the
 * shared expert (ignored when n_shared == 0).  Required before
 * dwdp_moe_layer on such a context; kept until replaced.  Errors:
 * INVALID_ARG (bf16 context, bad layer, non-finite or non-positive scale). */
int32_t dwdp_set_expert_scales(dwdp_ctx* ctx, int32_t layer, const float* w13_scale, const float* w2_scale,
                               float shared_w13_scale, float shared_w2_scale);

/* Top-k routing with a deterministic grouping of the (token, slot) pairs by
 * expert.  x [T][H] bf16 and w_router [E][H] bf16 are device pointers;
 * logit_bias [E] fp32 (device) or NULL is added to every logit before the
 * choice.  The chosen experts are the k largest logits (softmax is
 * monotone), ties to the lower id, decided on the fp32 logits; weights are
 * exp(z_j - z_max) / sum over the chosen set.  ws (device, ws_bytes >=
 * dwdp_workspace_bytes) is scratch.  Enqueued on `stream`.  A token with
 * a logit that is not finite (NaN or +-inf, e.g. from a NaN in x) has no
 * defined choice: it still gets k distinct experts, but its ids and weights
 * are unspecified and the device error word is set (dwdp_device_status:
 * DEVICE_CHECK).  x and w_router must be device memory of the context's
 * device (they are read through TMA tensor maps).
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_route(dwdp_ctx* ctx, const void* x, int32_t T, const void* w_router,
                   const float* logit_bias, const dwdp_route_out* out, void* ws, size_t ws_bytes,
                   dwdp_stream_t stream);

/* Pull layer `layer`'s non-resident experts from their peer pools into stage
 * buffer `stage` ([DWDP] §2: asynchronous prefetch of layer l+1 during layer
 * l, double-buffered; §4.3.2: fixed-size slices, round-robin over sources).
 * Each slice is one memcpy node (copy engine, no SMs) of at
 * most chunk_bytes in a CUDA graph that the context builds on first use for
 * this (chunk_bytes, stage, n_copy_streams) and keeps until the layer's map
 * is replaced; slices from peer p form chain p % n_copy_streams of the graph
 * (chains may run on separate copy engines), each chain in plan order.  The
 * graph is launched on copy_streams[0] (the other streams are not used)
 * after that stream waits until the last dwdp_moe_layer that read this
 * stage has finished reading it; completion is recorded as the stage's
 * "ready" event.  Errors: INVALID_ARG, NOT_MAPPED, CUDA. */
int32_t dwdp_prefetch_layer(dwdp_ctx* ctx, int32_t layer, int32_t stage, size_t chunk_bytes,
                            dwdp_stream_t const* copy_streams, int32_t n_copy_streams);

/* One MoE layer for T tokens on `stream` ([DWDP] §2 and §4.2):
 *   xp  = x rows copied into expert order (row route->inv_perm[t*k+j] = x[t])
 *   a   = SiLU(xp W_gate) * (xp W_up)          per expert, bf16
 *   y   = a W_down                             per expert, bf16
 *   out[t] = sum_j topk_w[t][j] y[inv_perm[t*k+j]] + y_shared[t]  (fp32 sum, bf16)
 * Each expert's weights come from the local pool or from stage `stage`, per
 * the layer's map; before the gate/up GEMM the stream waits for that stage's
 * "ready" event when the layer has non-resident experts (per-layer arrival,
 * [DWDP] §2).  route
 * holds dwdp_route's outputs for the same x (offsets, inv_perm and topk_w are
 * read; NVFP4 contexts also read topk_ids).  In E4M3 and NVFP4 contexts x
 * and a are quantized per row first (see DWDP_DTYPE_*) and the GEMMs run on
 * the codes.  out [T][H] bf16 (device).  An inv_perm entry outside
 * [0, T*k) is not followed: the kernels skip it (the token's output then
 * lacks that expert) and set the device error word, which
 * dwdp_device_status reports as DEVICE_CHECK.
 * Errors: INVALID_ARG, NOT_MAPPED, UNSUPPORTED, CUDA. */
int32_t dwdp_moe_layer(dwdp_ctx* ctx, int32_t layer, int32_t stage, const void* x, int32_t T,
                       const dwdp_route_out* route, void* out, void* ws, size_t ws_bytes,
                       dwdp_stream_t stream);

/* Activation quantization on its own, the same kernels and decisions as
 * dwdp_moe_layer applies to x and to a: x [rows][K] bf16 (device) to
 *   DWDP_DTYPE_E4M3: codes [rows][K] E4M3 bytes, row_scale [rows] fp32
 *     (amax / 448; block_scales unused);
 *   DWDP_DTYPE_NVFP4: codes [rows][K / 2] (two E2M1 codes per byte, element
 *     2i in the low nibble), row_scale [rows] fp32 (amax / 2688) and
 *     block_scales in the 512-byte chunk layout of DWDP_DTYPE_NVFP4 for a
 *     tensor of ceil(rows / 128) * 128 rows (bytes of rows past `rows` are
 *     not written).
 * K a multiple of 64; rows < 2^31.  All pointers device, 16-byte aligned.
 * Enqueued on `stream`; needs no context.  Errors: INVALID_ARG, CUDA. */
int32_t dwdp_quantize_rows(int32_t weight_dtype, const void* x, int64_t rows, int32_t K, void* codes,
                           void* block_scales, float* row_scale, dwdp_stream_t stream);

/* Host-side bounded wait for stage `stage`'s last prefetch: returns OK when
 * it has finished, TIMEOUT after timeout_ms (>= 0), CUDA on a fault. */
int32_t dwdp_wait_stage(dwdp_ctx* ctx, int32_t stage, int32_t timeout_ms);

/* Layer whose experts stage `stage` holds (or is being filled with), -1 if
 * none.  Host-side bookkeeping only. */
int32_t dwdp_stage_layer(const dwdp_ctx* ctx, int32_t stage);

/* Read and clear the device error word (synchronises the device).  OK, or
 * DEVICE_CHECK with the failing check described by dwdp_last_error: bits
 * 0-5 a bounded wait inside the grouped GEMM ran out, bit 6 an index outside
 * its buffer was skipped, bit 7 a router logit was not finite, bit 8 the
 * wait of dwdp_selftest_bounded_wait ran out (as that call intends). */
int32_t dwdp_device_status(dwdp_ctx* ctx);

/* Diagnostic (the pages have no counterpart): enqueues on `stream` one
 * one-thread kernel that waits, with the same bounded mbarrier wait every
 * grouped-GEMM role uses, for a barrier phase that nothing completes.  The
 * wait gives up after limit_us microseconds, sets bit 8 of the context's
 * device error word and the kernel returns: no trap, no hang, the context
 * stays usable.  The next dwdp_device_status then returns DEVICE_CHECK
 * (and clears the word).  limit_us in [1, 1000000].  Errors: INVALID_ARG,
 * CUDA. */
int32_t dwdp_selftest_bounded_wait(dwdp_ctx* ctx, uint32_t limit_us, dwdp_stream_t stream);

/* Optional phase timing.  events is a host array of DWDP_PHASE_EVENTS
 * caller-owned cudaEvent_t (or NULL to stop).  While set, dwdp_route records
 * events[0] at its start and events[1] at its end on its stream, and
 * dwdp_moe_layer records events[2] once x is in expert order (E4M3 / NVFP4:
 * quantized), events[3] after waiting for its stage (the layer puts x in
 * expert order before it waits: only the GEMMs read staged weights),
 * events[4] after the gate/up GEMM, events[5] after the down GEMM and
 * events[6] after the combine.  The context keeps the pointers
 * until the next call; the caller keeps the events alive.  Errors:
 * INVALID_ARG (a NULL event or a wrong count; the previous events, or
 * none, stay in effect). */
#define DWDP_PHASE_EVENTS 7
int32_t dwdp_set_phase_events(dwdp_ctx* ctx, void* const* events, int32_t n_events);

/* Split-pointer grouped GEMM on its own ([DWDP] §4.2: one kernel over several
 * weight buffers, no merge).  For each group g in [0, G):
 *   rows r in [row_offsets[g], row_offsets[g+1]) of a [rows][K] bf16:
 *   d[r][n] = sum_k a[r][k] * B_g[n][k],  B_g = slot buf_slot[2g+1] of
 *   buffer bufs[buf_slot[2g]] (each buffer [n_slots][N_b][K] bf16).
 * epilogue 0: d bf16 [rows][N], B_g has N rows.
 * epilogue 1: d bf16 [rows][N] = SiLU(gate) * up with gate = rows 0..N-1 and
 *             up = rows N..2N-1 of B_g (B_g has 2N rows).
 * epilogue 2: d fp32 [rows][N], B_g has N rows.
 * row_offsets is a DEVICE array [G+1] (non-decreasing, row_offsets[G] <=
 * a_rows; rows outside [0, a_rows) are not stored and raise DEVICE_CHECK);
 * buf_slot is a HOST array [2G]; bufs is a host array of n_bufs <= 3 buffers
 * of which only .w13 (the base) and .n_slots are read.
 * K and N multiples of 64 (epilogue 2: N any value >= 1).  Enqueued on
 * `stream`; uses no workspace.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_grouped_gemm(dwdp_ctx* ctx, int32_t epilogue, const void* a, int64_t a_rows, int32_t K,
                          int32_t N, const int32_t* row_offsets, int32_t G, const dwdp_pool* bufs,
                          int32_t n_bufs, const int32_t* buf_slot, void* d, dwdp_stream_t stream);

/* Routing that allocates no device memory (the paper has no counterpart: it
 * serves callers that cannot call cudaMalloc where they route tokens, e.g. a
 * framework whose caching allocator owns all device memory, a latency-bound
 * serving loop that cannot afford the synchronisation cudaMalloc may imply,
 * or a host with a memory budget fixed at start-up).
 * Computes exactly what dwdp_route computes (same kernels, same results) for
 * x [T][hidden], w_router [n_experts][hidden], logit_bias [n_experts] or
 * NULL, without a context or workspace; out->logits is ignored (the logits
 * stay in the scratch).  Its scratch is one file-scope device array of
 * 32 MiB + 256 bytes: DWDP_STATIC_SCRATCH_BYTES (16 MiB) of fp32 logits, as
 * much again for the router GEMM's partial sums (its K may be split into
 * parts as in dwdp_route, which always fit on GPUs with up to 256 SMs) and a
 * 256-byte error word, held by every GPU that loads this library until the
 * process exits, so T * n_experts * 4 must not exceed
 * DWDP_STATIC_SCRATCH_BYTES (else INVALID_ARG, nothing enqueued).  The first
 * call on each device (of this entry point or of dwdp_route_static_status)
 * looks up the array's device address (cudaGetSymbolAddress) with that
 * device current and keeps it for the life of the process; make that first
 * call before any stream capture, and do not use these two calls on a
 * device after cudaDeviceReset (the address belonged to the context the
 * reset destroyed).  Every call on a device shares the one array and it
 * keeps the last call's contents (the error word is cleared on `stream` at
 * the start of each call): calls whose work overlaps on the GPU (other
 * streams, other threads) race on it.  Device-side failures (a non-finite
 * logit as in dwdp_route, a bounded wait that ran out) set the array's
 * error word: read it with dwdp_route_static_status.  Calls no cudaMalloc,
 * cudaFree or other allocating routine.  Errors (text in
 * dwdp_last_error(NULL)): INVALID_ARG, UNSUPPORTED, CUDA. */
#define DWDP_STATIC_SCRATCH_BYTES (16u << 20)
int32_t dwdp_route_static(const void* x, int32_t T, int32_t hidden, int32_t n_experts, int32_t top_k,
                          const void* w_router, const float* logit_bias, const dwdp_route_out* out,
                          dwdp_stream_t stream);

/* The device error word of dwdp_route_static on the current device (no
 * counterpart in the paper; dwdp_route_static has no context whose
 * dwdp_device_status could report it).  Waits for the work already enqueued
 * on `stream` (not allowed while `stream` is being captured), reads the word
 * and, when it is non-zero, clears it on `stream`.  *bits (may be NULL)
 * receives the raw bits (as for dwdp_device_status).  Returns OK for a zero
 * word, DEVICE_CHECK otherwise (text in dwdp_last_error(NULL)).  Allocates
 * nothing.  Errors: CUDA, UNSUPPORTED. */
int32_t dwdp_route_static_status(dwdp_stream_t stream, int32_t* bits);

/* Host-only (no GPU needed): the prefetch copy plan dwdp_prefetch_layer
 * issues for a map ([DWDP] §4.3.2).  The non-resident experts (local_slot <
 * 0) take stage slots in ascending id; each peer's work is its w13 copies then
 * its w2 copies in ascending expert id, merged where contiguous in both
 * source and destination, cut into slices of chunk_bytes (the last one
 * short); slices are emitted round-robin over peers 0..n_peers-1.  Writes up
 * to max_out slices to out (may be NULL when max_out == 0) and the full count
 * to *n_out.  weight_dtype (DWDP_DTYPE_*) sets the bytes of one expert
 * tensor.  Errors: INVALID_ARG (bad map or a non-resident expert with no
 * peer copy). */
int32_t dwdp_plan_prefetch(int32_t n_experts, int32_t hidden, int32_t inter, int32_t weight_dtype,
                           const int32_t* local_slot, const int32_t* peer_id,
                           const int32_t* peer_slot, int32_t n_peers, size_t chunk_bytes,
                           dwdp_copy_slice* out, int64_t max_out, int64_t* n_out);

/* Host-only (no GPU needed): the expert map of rank `rank` in a DWDP group
 * of n_ranks ranks ([DWDP] §2: each rank keeps a partition of the experts
 * and pulls the rest from its peers; §4.3.1-§4.3.2: the pulls of several
 * destinations from one source contend, so slices are issued round-robin).
 * Rank q hosts experts [floor(q E / N), floor((q + 1) E / N)) in slots
 * 0, 1, ... of its pool.  Fills local_slot [E] (the slot for this rank's own
 * experts, else -1), and for the others peer_id [E] and peer_slot [E] (-1 for
 * own experts), numbering this rank's peers from the next rank on: peer p
 * is rank (rank + 1 + p) mod n_ranks, so the peers array given to
 * dwdp_set_expert_map lists the other ranks' pools in that order.  With this
 * numbering the round-robin of dwdp_plan_prefetch has every rank, at the
 * same step of its plan, pulling from a different source (when every rank
 * hosts the same number of experts), so no source serves two destinations
 * at once.  A map for placement only: the pulls themselves are copy-engine
 * memcpy nodes whose source may be any memory the copy engine reaches.
 * Errors: INVALID_ARG. */
int32_t dwdp_group_map(int32_t n_experts, int32_t n_ranks, int32_t rank, int32_t* local_slot, int32_t* peer_id,
                       int32_t* peer_slot);

/* ---- the rest of a decoder block's second half --------------------------
 * The three calls below surround dwdp_moe_layer in a decoder block: the
 * adapters of the attention's output projection (the projection itself is
 * dwdp_grouped_gemm with one group), the residual addition with the norm, and
 * the router of the R1 models.  They serve, for one token as
 * for many, and can be captured into CUDA graphs. */

/* Residual addition and root-mean-square norm, optionally also as E4M3 rows
 * for dwdp_moe_layer_codes.  Per row of H elements, with h = x + residual
 * (h = x when residual is NULL):
 *   residual_out = bf16(h)                        (iff residual is given)
 *   y   = h / sqrt(mean(h^2) + eps) * weight      binary32, from the unrounded h
 *   out = bf16(y)
 *   row_scale = max|y| / 448 (1 for an all-zero row),
 *   codes = E4M3(y / row_scale)                   (iff codes is given)
 * The codes come from the unrounded y: one rounding, to nearest even (of
 * y / row_scale by approximate reciprocals, so that a value next to the middle
 * of two codes may take either).  A row whose largest |h weight| is below 2^-100
 * is quantized as if it were 2^-100.
 * The squares are summed in binary32, on scaled values where they would pass
 * its range, or vanish below it with an eps that does not make up for them (eps
 * below 2^-120, e.g. 0; an all-zero row of out is then NaN, 0 / 0).  The codes
 * ask for weights of ordinary size: with an eps of 2^-120 or more, |h weight| has
 * to stay in binary32's range, and a row whose squares pass it (|h| beyond 2^55)
 * is quantized as if its largest |h weight| were at least 2^-20.
 * A NaN makes its row of out, and its row_scale, NaN.
 * x: bf16, row r at x + r * x_stride elements (x_stride >= H, a multiple of
 * 8); residual, residual_out, out: bf16 [rows][H]; weight: bf16 [H]; codes:
 * E4M3 bytes [rows][H]; row_scale: fp32 [rows].  Either of residual and
 * residual_out NULL means both are; likewise codes and row_scale.
 * residual_out may be residual, and out may be x when x_stride == H; no other
 * overlap.  H a multiple of 8, 8 <= H <= 32768; eps >= 0 and finite; rows in
 * [0, 2^31).  All pointers device, 16-byte aligned.  Enqueued on `stream`;
 * needs no context.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_add_rmsnorm(const void* x, int64_t x_stride, const void* residual, void* residual_out,
                         const void* weight, float eps, int64_t rows, int32_t H, void* out, void* codes,
                         float* row_scale, dwdp_stream_t stream);

/* How dwdp_route_scored scores, chooses and weighs.
 *   score        DWDP_SCORE_SOFTMAX (over all E) or DWDP_SCORE_SIGMOID
 *   n_groups     experts e / (E / n_groups) form a group; divides E, 1 = none
 *   top_groups   groups a token may choose from, 1..n_groups
 *   group_score  DWDP_GROUP_MAX: a group's largest choice value;
 *                DWDP_GROUP_TOP2: the sum of its two largest (of its one)
 *   renormalize  1: the k weights are divided by their sum; 0: as scored
 *   scale        factor on the weights, finite and > 0 */
#define DWDP_SCORE_SOFTMAX 0
#define DWDP_SCORE_SIGMOID 1
#define DWDP_GROUP_MAX 0
#define DWDP_GROUP_TOP2 1
typedef struct {
    int32_t score;
    int32_t n_groups;
    int32_t top_groups;
    int32_t group_score;
    int32_t renormalize;
    float scale;
} dwdp_scoring;

/* Routing as the R1 models do it, with dwdp_route's outputs.  With the fp32
 * logits z = x W^T:
 *   s = softmax(z) or sigmoid(z);  c = s + choice_bias (NULL = 0)
 *   the top_groups groups with the largest group score of c stay;
 *   the k largest c in them are chosen; topk_w = s of the chosen
 *   (divided by their sum if renormalize) * scale.
 * Ties go to the lowest group and expert id.  choice_bias [E] fp32 (device)
 * steers the choice only, not the weights; -inf takes an expert out: it is
 * chosen only where fewer than k others are left, the lowest ids first, and
 * then has weight 0.  Weights are right to a few units in the last place
 * (approximate exponentials and reciprocals; 0 below 2^-126).  The
 * choice is the one these formulas give in binary64 on the fp32 logits (a
 * token whose decision binary32 cannot tell apart is decided again in
 * binary64), so it depends on the logits alone.  The logits are deterministic
 * for a given device and shape; out->logits (NULL = not returned) gets them.
 * A token with a logit that is not finite, or a bias that is NaN or +inf, is
 * treated as in dwdp_route: k distinct experts, DEVICE_CHECK.
 * x, w_router, out, ws, T as for dwdp_route; k <= top_groups * E / n_groups;
 * n_groups <= DWDP_MAX_GROUPS.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_route_scored(dwdp_ctx* ctx, const void* x, int32_t T, const void* w_router,
                          const float* choice_bias, const dwdp_scoring* scoring, const dwdp_route_out* out,
                          void* ws, size_t ws_bytes, dwdp_stream_t stream);

/* Low-rank adapters of many requests beside a shared projection.  For token t
 * with adapter i = adapter_ids[t]:
 *   out[t] = bf16(base[t] + adapter_scale[i] * (x[t] A_i^T) B_i^T)
 * and out[t] = base[t] where i is -1 (no adapter).  The inner product is
 * summed in fp32, scaled and rounded once to bf16 (it is the second product's
 * operand); the second is summed in fp32 on top of base, rounded once.
 * a: bf16 [n_adapters][R][K]; b: bf16 [n_adapters][N][R]; adapter_scale fp32
 * [n_adapters]; adapter_ids int32 [T] (all device).  Adapters of a smaller
 * rank are padded with zero rows (columns).  Tokens may come in any order;
 * tokens of one adapter next to each other are the cheap case.  Where adapters
 * change from token to token (in half of 32 pairs of ids 2 i, 2 i + 1 spread
 * over the batch), up to 2048 tokens, from 1024 on with T (K + N) up to 2^24,
 * of a bank of up to 255 adapters are taken in the adapters' order; other such
 * batches read x again for every few adapters of a tile of 16 to 128 tokens.
 * x: row t at
 * x + t * x_stride elements, K of them; base and out: row t at t *
 * base_stride / t * out_stride, N of them; every stride a multiple of 8 and
 * no smaller than the row.  out may be base (equal strides); no other
 * overlap.  K, N multiples of 8, at most 2^20; R a multiple of 8,
 * 8..DWDP_MAX_LORA_RANK; T at most 2^30; n_adapters * R below 2^31.  An id
 * outside [-1, n_adapters) is not followed: the token gets base and the device
 * error word reports a bad index (DEVICE_CHECK).  ws: at least
 * dwdp_lora_workspace_bytes(T, K, N, R) bytes, device.  All pointers 16-byte
 * aligned; from 1024 tokens on x and a must be device memory of the context's
 * device (they are read through tensor maps).  Enqueued on `stream`.  Errors:
 * INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_lora_add(dwdp_ctx* ctx, const void* x, int64_t x_stride, int32_t T, int32_t K, int32_t N,
                      const void* a, const void* b, const float* adapter_scale, int32_t n_adapters, int32_t R,
                      const int32_t* adapter_ids, const void* base, int64_t base_stride, void* out,
                      int64_t out_stride, void* ws, size_t ws_bytes, dwdp_stream_t stream);

/* Workspace of dwdp_lora_add; 0 for sizes it refuses. */
size_t dwdp_lora_workspace_bytes(int32_t T, int32_t K, int32_t N, int32_t R);

/* dwdp_moe_layer of an E4M3 context on rows that are E4M3 already: xq [T][H]
 * codes and sx [T] fp32 row scales (x = code * scale), e.g. those of
 * dwdp_add_rmsnorm, which are the more exact ones (rounded once, from the
 * norm's unrounded rows).  Everything else is as for dwdp_moe_layer; xq must
 * be device memory of the context's device.  The workspace regions XQ and SX
 * stay unwritten.  Errors: INVALID_ARG (also: the context is not E4M3),
 * NOT_MAPPED, UNSUPPORTED, CUDA. */
int32_t dwdp_moe_layer_codes(dwdp_ctx* ctx, int32_t layer, int32_t stage, const void* xq, const float* sx,
                             int32_t T, const dwdp_route_out* route, void* out, void* ws, size_t ws_bytes,
                             dwdp_stream_t stream);

/* ---- training the block's norms and its router ---------------------------
 * The calls below add what a decoder block's second half needs around
 * dwdp_moe_layer when its norms, gates or router are trained or tuned: the
 * norms before and after a block in one pass, with their gradients and with
 * rows kept in 8 bits for them, the router's losses, and the gradient of its
 * logits.  dwdp_sandwich_norm serves single tokens too.  All can be captured
 * into CUDA graphs, and give the same bits from run to run. */

/* What dwdp_sandwich_norm and its gradients share.
 *   pre_weight, post_weight  bf16 [H] (device) or NULL: no such norm
 *   gate          bf16 [n_groups][H] (device), or NULL (n_groups 0): 1
 *   row_offsets   int32 [n_groups + 1] (device), non-decreasing: gate g is for
 *                 rows row_offsets[g] .. row_offsets[g + 1] - 1, and rows outside
 *                 [row_offsets[0], row_offsets[n_groups]) are left alone: not
 *                 written, no part of any sum, whatever they hold (they may be
 *                 read, so every array has all its rows)
 *                 NULL: one gate for all rows (n_groups 1)
 *   block_scale, residual_scale  finite constants
 *   eps           of both norms, finite and at least 2^-100 */
typedef struct {
    const void* pre_weight;
    const void* post_weight;
    const void* gate;
    const int32_t* row_offsets;
    int32_t n_groups;
    float block_scale;
    float residual_scale;
    float eps;
} dwdp_sandwich;
#define DWDP_MAX_GATES 32768

/* The norm after a block, its gate, the residual addition and the next
 * block's norm.  Per row of H elements, in binary32:
 *   n = x rx post_weight,  rx = 1 / sqrt(mean(x^2) + eps)   (n = x without post_weight)
 *   h = residual_scale residual + block_scale gate n        (residual NULL: 0)
 *   residual_out = bf16(h)                                  (iff given)
 *   y = h rh pre_weight,   rh = 1 / sqrt(mean(h^2) + eps)   from the unrounded h
 *   out = bf16(y)                                           (iff pre_weight is given)
 *   codes, row_scale: y as E4M3 rows, as in dwdp_add_rmsnorm (iff given)
 * and what dwdp_sandwich_norm_grad takes (each iff given):
 *   x_codes, x_scale: x as E4M3 rows, scale = max|x| / 448 (1 for a row of zeros)
 *   h_codes, h_scale: the unrounded h, likewise
 *   rstd [rows][2]: rx and rh (1 for a norm that is not there)
 * The E4M3 rows are rounded once, to nearest even, by approximate reciprocals: a
 * value next to the middle of two codes may take either; a row whose largest
 * magnitude (codes: of h pre_weight) is below 2^-100 is quantized as if it were
 * 2^-100.  h and h pre_weight have to stay in binary32's range; squares may pass
 * it.  A NaN makes its row NaN where it goes.
 * x: bf16, row r at x + r * x_stride elements (x_stride >= H, a multiple of 8);
 * residual, residual_out, out bf16 [rows][H]; codes, x_codes, h_codes E4M3
 * bytes [rows][H]; row_scale, x_scale, h_scale fp32 [rows]; rstd fp32.  Codes
 * and their scale go together; out and codes need pre_weight.  residual_out may
 * be residual, and out may be x when x_stride == H; no other overlap.  H a
 * multiple of 8, 8 <= H <= 32768; rows in [0, 2^31); at most DWDP_MAX_GATES
 * groups.  All pointers device, 16-byte aligned.  Enqueued on `stream`; needs no
 * context.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_sandwich_norm(const dwdp_sandwich* how, const void* x, int64_t x_stride, const void* residual,
                           int64_t rows, int32_t H, void* residual_out, void* out, void* codes, float* row_scale,
                           void* x_codes, float* x_scale, void* h_codes, float* h_scale, float* rstd,
                           dwdp_stream_t stream);

/* The gradients of dwdp_sandwich_norm (without post_weight and gate: of
 * dwdp_add_rmsnorm).  From x and h (bf16 rows, or E4M3 codes where x_scale /
 * h_scale is given), rstd as the forward call wrote it, and the gradients of
 * out (dout) and residual_out (dresidual_out; NULL = 0), both bf16 [rows][H]:
 *   hhat = h rh,  gy = dout pre_weight
 *   dh = dresidual_out + rh (gy - hhat mean(gy hhat))       (dh = dresidual_out without pre_weight)
 *   dresidual = residual_scale dh,  dn = block_scale gate dh
 *   xhat = x rx,  gn = dn post_weight
 *   dx = rx (gn - xhat mean(gn xhat))                       (dx = dn without post_weight)
 *   dpre_weight = sum over rows of dout hhat,  dpost_weight = sum of dn xhat
 *   dgate[g] = sum over its rows of block_scale dh xhat post_weight
 * in binary32; dx and dresidual are rounded once to bf16 [rows][H], the sums
 * are fp32 ([H], [H], [n_groups][H]), written whole (zeros where there are no
 * rows).  Each output may be NULL.  x may be NULL without post_weight and
 * dgate, and h without pre_weight, which also has no dout.  x_stride (in
 * elements) holds for x's codes too; h is dense.  dresidual may be
 * dresidual_out and dx may be dout; no other overlap.  The rest as for
 * dwdp_sandwich_norm.  ws: dwdp_sandwich_grad_workspace_bytes(rows,
 * H) bytes (device), needed for the sums only; calls that may overlap, replays of
 * captured ones too, need one each.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_sandwich_norm_grad(const dwdp_sandwich* how, const void* x, int64_t x_stride, const float* x_scale,
                                const void* h, const float* h_scale, const float* rstd, const void* dout,
                                const void* dresidual_out, int64_t rows, int32_t H, void* dx, void* dresidual,
                                float* dpost_weight, float* dpre_weight, float* dgate, void* ws, size_t ws_bytes,
                                dwdp_stream_t stream);

/* Workspace of dwdp_sandwich_norm_grad; 0 for sizes it refuses. */
size_t dwdp_sandwich_grad_workspace_bytes(int64_t rows, int32_t H);

/* How evenly the experts were used, per sequence.  Sequence b has tokens
 * seq_offsets[b] .. seq_offsets[b + 1] - 1, T_b of them (seq_offsets: int32
 * [n_seqs + 1], device, non-decreasing; NULL: one sequence of all T tokens);
 * tokens outside [seq_offsets[0], seq_offsets[n_seqs]) are in none.  From the
 * router's logits z [T][E] fp32 and choices topk_ids [T][k]
 * (dwdp_route_scored's logits and topk_ids), with the token's shares p =
 * softmax(z), or s / sum(s) with s = sigmoid(z):
 *   counts [n_seqs][E]  tokens of the sequence that chose the expert (int32)
 *   mean_p [n_seqs][E]  mean of p over the sequence
 *   balance [n_seqs]    E / (k T_b) sum_e counts mean_p (1 when all is even)
 *   z [n_seqs]          mean of logsumexp(z)^2; NULL = not computed
 * all zero for a sequence without tokens.  Sums are binary32; a share is right
 * to (2 m + 24) 2^-23 of itself, m the logits' spread where the sum of exp(z)
 * (softmax) or s lies outside 2^-36 .. 2^36, else at most 32 more (approximate
 * exponentials of the logits as they are).  Of `scoring` only score is used.  A
 * NaN or infinite logit may make its sequence's mean_p, balance and z NaN; -inf
 * is a share of 0 where the token has a finite one.  An id outside [0, E) is not
 * counted; the device error word reports it (DEVICE_CHECK).  T at most
 * max_tokens and 2^30.  ws: dwdp_balance_workspace_bytes(T, E, n_seqs) bytes,
 * device, one for each of calls that may overlap.  All pointers 16-byte aligned.  Enqueued on `stream`.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_balance_loss(dwdp_ctx* ctx, const float* logits, const int32_t* topk_ids, int32_t T,
                          const int32_t* seq_offsets, int32_t n_seqs, const dwdp_scoring* scoring, int32_t* counts,
                          float* mean_p, float* balance, float* z, void* ws, size_t ws_bytes, dwdp_stream_t stream);

/* Workspace of dwdp_balance_loss; 0 for sizes it refuses. */
size_t dwdp_balance_workspace_bytes(int32_t T, int32_t E, int32_t n_seqs);

/* The gradient of dwdp_route_scored's logits, from that of its weights and
 * from dwdp_balance_loss's losses:
 *   dlogits = d/dz ( sum dtopk_w topk_w + sum_b dbalance[b] balance[b] + dz[b] z[b] )
 * with the choice and the counts held fixed, for a routing without choice_bias or
 * with one that took no expert out (-inf; else dwdp_route_scored_biased_grad).
 * dtopk_w fp32 [T][k], dbalance and
 * dz fp32 [n_seqs] (device): each NULL = 0.  counts as dwdp_balance_loss wrote them
 * (needed with dbalance; counts added up over several devices, with dbalance to
 * match, serve as well).  Tokens in no sequence get the weights' part only.
 * score, renormalize and scale of `scoring` are used.  The ids of a token are distinct.
 * dlogits [T][E]: fp32, or bf16 when dlogits_bf16 is 1; every element is written.
 * A NaN or infinite logit may make its token's gradient NaN; -inf has a gradient
 * of 0 where the token, and with renormalize its choice, has a finite one; an id outside [0,
 * E) is skipped and reported as above.  Other arguments as for dwdp_balance_loss;
 * dlogits overlaps none of them.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int32_t dwdp_route_scored_grad(dwdp_ctx* ctx, const float* logits, const int32_t* topk_ids, const float* dtopk_w,
                               int32_t T, const int32_t* seq_offsets, int32_t n_seqs, const dwdp_scoring* scoring,
                               const int32_t* counts, const float* dbalance, const float* dz, void* dlogits,
                               int32_t dlogits_bf16, dwdp_stream_t stream);

/* The same where choice_bias (fp32 [E], device, or NULL), as dwdp_route_scored
 * got it, takes experts out: one that filled a choice up has the weight 0, no
 * part of the sum that the others are divided by, and no gradient from its
 * weight.  (In counts, and so in the balance loss, it is a chosen one.) */
int32_t dwdp_route_scored_biased_grad(dwdp_ctx* ctx, const float* logits, const int32_t* topk_ids,
                                      const float* dtopk_w, const float* choice_bias, int32_t T,
                                      const int32_t* seq_offsets, int32_t n_seqs, const dwdp_scoring* scoring,
                                      const int32_t* counts, const float* dbalance, const float* dz, void* dlogits,
                                      int32_t dlogits_bf16, dwdp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DWDP_H_ */
