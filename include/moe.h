/*
 * moe.h -- C ABI of the fused MoE layer forward on one GB300 (sm_103a).
 *
 * One call runs the whole layer on the GPU:
 *   RMSNorm -> router GEMV + top-k softmax -> expert align (histogram,
 *   prefix sum, padded permutation) -> gather -> gate/up grouped GEMM with a
 *   SwiGLU epilogue -> down grouped GEMM -> top-k weighted combine.
 *
 * Definitions the calls implement:
 *   RMSNorm      h_j = bf16( x_j / sqrt(mean_i x_i^2 + eps) * g_j ), fp32
 *                accumulation -- "4 · La fusion de noyaux", §4.2
 *                "Réduction + élémentaire"; eps inside the square root and
 *                the cast back to the input type as in "CuTeDSL chez
 *                Perplexity", section "Norme QK".
 *   Router       fp32 logits l_e = sum_j h_j Wr[e,j] (+ b_e); the top_k
 *                largest (ties to the lower expert index), weights =
 *                softmax over all E taken at the selected experts, divided
 *                by their sum when renormalize != 0.
 *   Dispatch     per-expert counts, a unique slot per routed token in its
 *                expert's list, lists copied into padded per-expert buffers
 *                -- "CuTeDSL chez Perplexity", MoE dispatch/combine, "Local".
 *   Experts      SwiGLU(x) = (SiLU(x W_gate) (.) (x W_up)) W_down with gate
 *                and up in one concatenated weight -- "4 · La fusion de
 *                noyaux", §4.2 "GEMM + GEMM"; SiLU(gate)*up is applied to
 *                the accumulators before the only store ("GEMM + épilogue").
 *   Combine      y_t = bf16( sum_j w_tj * o_tj ) -- "CuTeDSL chez
 *                Perplexity", MoE dispatch/combine, "Local".
 *
 * Conventions for every call:
 *   - bf16 tensors are passed as raw bfloat16 bits (moe_bf16).
 *   - All tensor pointers are DEVICE pointers of the current CUDA device,
 *     row-major and contiguous, 16-byte aligned; the workspace is 256-byte
 *     aligned.  The caller owns every buffer; the library allocates no
 *     device memory on any call.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default
 *     stream).  Outputs are valid once the stream has reached the end of
 *     the call.  Inputs are never modified.
 *   - A call can be captured into a CUDA graph (stream capture on `stream`)
 *     and replayed: it makes no host synchronisation and no allocation, and
 *     it reads the pointed-to data when the kernels run.  The shape, the
 *     pointers and the tensor maps built from them are fixed at capture;
 *     new inputs go into the same buffers between replays.  Make one call
 *     outside capture first on each device (it sets per-device kernel
 *     attributes, which are not stream work).  A replay gives the same bits
 *     as the direct call.
 *   - Argument and shape errors are reported synchronously, before anything
 *     is enqueued.  A failed launch returns MOE_ERR_CUDA.  Errors found on
 *     the device (a routing index out of range, a bounded wait that ran out)
 *     are written to an error word at the start of the workspace and are
 *     returned by moe_device_status().
 *   - The library keeps no state between calls except per-device kernel
 *     attributes set once; it is reentrant as long as concurrent calls use
 *     different workspaces.  One exception: moe_forward_static_scratch keeps
 *     its scratch in one device array per GPU that every call of it on that
 *     GPU shares (and caches that array's address), so its callers must
 *     serialise their calls although they pass no workspace.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* raw bfloat16 bits */
typedef uint16_t moe_bf16;
/* a cudaStream_t */
typedef struct CUstream_st* moe_stream_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1, /* null pointer, bad alignment, bad shape value */
  MOE_ERR_UNSUPPORTED = 2, /* a shape outside the supported set (see moe_shape) */
  MOE_ERR_WORKSPACE = 3,   /* workspace smaller than moe_workspace_size() */
  MOE_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
  MOE_ERR_TIMEOUT = 5,     /* a device-side bounded wait ran out (reported by moe_device_status) */
  MOE_ERR_DEVICE = 6       /* the device found bad data, e.g. an expert index >= E */
} moe_status;

/* Layer shape and routing options.
 *   T            tokens (>= 0; moe_forward with T = 0 returns MOE_OK at once and
 *                touches no pointer)
 *   H            hidden size, a multiple of 128 (the down GEMM's weight tile
 *                is 128 output features), <= 16384 (the router keeps its
 *                tokens' rows of h in shared memory)
 *   I            expert intermediate size, a multiple of 64 (the gate/up
 *                GEMM's unit is 64 features, the down GEMM's K block 64
 *                elements; 128 for the block-scaled layers, whose scale tiles
 *                cover 128 elements of K), <= 16384
 *   E            experts, 1..1024
 *   top_k        experts per token, 1..min(E, 32) (one lane of the selecting
 *                warp per selected expert)
 *   renormalize  nonzero: the top_k weights are divided by their sum
 *   eps          RMSNorm epsilon (>= 0, finite)                              */
typedef struct {
  int32_t T, H, I, E, top_k;
  int32_t renormalize;
  float eps;
} moe_shape;

/* Bytes of device workspace moe_forward() needs for this shape.  Host only:
 * makes no CUDA call.  Returns MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED for
 * a bad shape. */
MOE_API moe_status moe_workspace_size(const moe_shape* shape, size_t* bytes);

/* The layer forward.
 *   x          [T, H]        bf16 token activations
 *   g_norm     [H]           bf16 RMSNorm gain
 *   w_router   [E, H]        fp32 router weight
 *   router_bias[E]           fp32 logit bias, or NULL for none
 *   w13        [E, 2I, H]    bf16; rows [0, I) of expert e are W_gate
 *                            (transposed, K-major), rows [I, 2I) are W_up
 *   w2         [E, H, I]     bf16; W_down of expert e (transposed, K-major)
 *   y          [T, H]        bf16 output (must not alias the inputs)
 *   workspace  device scratch of at least moe_workspace_size() bytes; its
 *              contents on entry do not matter; it holds the intermediate
 *              tensors (see moe_workspace_views) after the call.
 * Ownership: all buffers belong to the caller.  Errors: as above. */
MOE_API moe_status moe_forward(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                       const float* w_router, const float* router_bias, const moe_bf16* w13,
                       const moe_bf16* w2, moe_bf16* y, void* workspace, size_t workspace_bytes,
                       moe_stream_t stream);

/* The steps of one moe_forward call, in order:
 *   1 RMSNorm + router logits, 2 top-k + softmax, 3 expert align, 4 gather,
 *   5 gate/up grouped GEMM + SwiGLU, 6 down grouped GEMM, 7 weighted combine.
 * For T <= MOE_FUSED_TOPK_MAX_T and E <= MOE_FUSED_TOPK_MAX_E, steps 2 and 3
 * run as one single-CTA kernel; otherwise step 2 is one multi-CTA kernel
 * (top-k with per-block expert counts) and step 3 two (scan, scatter).
 * So 6 launches per call (8 with the multi-CTA top-k and align);
 * moe_kernels_per_call_of gives the count for each entry point. */
#define MOE_NUM_KERNELS 7
#define MOE_FUSED_TOPK_MAX_T 256
#define MOE_FUSED_TOPK_MAX_E 256

/* Number of kernels one moe_forward call with this shape launches on the
 * current device (0 for T = 0).  Host-only apart from querying the device. */
MOE_API moe_status moe_kernels_per_call(const moe_shape* shape, int32_t* count);

/* The same for each entry point: call = MOE_CALL_FORWARD (moe_forward,
 * moe_forward_events, moe_forward_static_scratch), MOE_CALL_FORWARD_FUSED_FRONT
 * (moe_forward_fused_front), MOE_CALL_FORWARD_MX (moe_forward_mx),
 * MOE_CALL_FORWARD_FUSED_COMBINE (moe_forward_fused_combine),
 * MOE_CALL_FORWARD_MXFP4 (moe_forward_mxfp4), MOE_CALL_FORWARD_MXFP4A4
 * (moe_forward_mxfp4a4), MOE_CALL_FORWARD_NVFP4 (moe_forward_nvfp4) or
 * MOE_CALL_FORWARD_FUSED_MLP (moe_forward_fused_mlp; MOE_ERR_UNSUPPORTED for
 * shapes it refuses).  Another value of call: MOE_ERR_INVALID_ARG.  Host-only. */
#define MOE_CALL_FORWARD 0
#define MOE_CALL_FORWARD_FUSED_FRONT 1
#define MOE_CALL_FORWARD_MX 2
#define MOE_CALL_FORWARD_FUSED_COMBINE 3
#define MOE_CALL_FORWARD_MXFP4 4
#define MOE_CALL_FORWARD_MXFP4A4 5
#define MOE_CALL_FORWARD_NVFP4 6
#define MOE_CALL_FORWARD_FUSED_MLP 7
MOE_API moe_status moe_kernels_per_call_of(const moe_shape* shape, int32_t call, int32_t* count);

/* moe_forward, plus CUDA events recorded on `stream` around the kernels:
 * events[0] before kernel 1 and events[i] right after kernel i (i = 1..7),
 * so cudaEventElapsedTime(events[i-1], events[i]) is kernel i's time on the
 * stream (with top-k fused into the align kernel, events[2] follows events[1]
 * at once and the align interval includes the top-k; otherwise events[2] ends
 * the top-k/count kernel and events[3] the scan and scatter kernels; with the
 * single-launch front end, events[1] ends it and events[2..4] follow at once).  `events` holds n_events >= MOE_NUM_KERNELS + 1 cudaEvent_t
 * handles created by the caller (cudaEventCreate); the library records them
 * and does not create, wait on or destroy them.  Everything else is as for
 * moe_forward; with T = 0 no event is recorded. */
MOE_API moe_status moe_forward_events(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                      const float* w_router, const float* router_bias, const moe_bf16* w13,
                                      const moe_bf16* w2, moe_bf16* y, void* workspace, size_t workspace_bytes,
                                      moe_stream_t stream, void* const* events, int32_t n_events);

/* moe_forward with steps 1-4 (norm, router, top-k, align, gather) run as one
 * launch of one thread-block cluster: the decode dispatch as a single kernel
 * with a grid-wide barrier ("CuTeDSL chez Perplexity", "Synchronisation de la
 * grille"), here the cluster's hardware barrier (4 launches per call).  For
 * T <= MOE_FRONT_MAX_T and E <= MOE_FRONT_MAX_E on a device that runs a
 * cluster of at least 8 such CTAs; other shapes return MOE_ERR_UNSUPPORTED
 * before anything is enqueued.  Results are the same bits as moe_forward's;
 * the padding rows of the gathered input (moe_views.xg) are not written.
 * `events` is NULL, or as for moe_forward_events (the front end's time falls
 * in events[0]..events[1]).  moe_forward stays the faster choice on GB300:
 * there the expert GEMM cannot start its weight loads until the whole front
 * end has finished, and 16 SMs read the router weights more slowly than the
 * multi-launch router's grid. */
#define MOE_FRONT_MAX_T 64
#define MOE_FRONT_MAX_E 256
MOE_API moe_status moe_forward_fused_front(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                           const float* w_router, const float* router_bias, const moe_bf16* w13,
                                           const moe_bf16* w2, moe_bf16* y, void* workspace, size_t workspace_bytes,
                                           moe_stream_t stream, void* const* events, int32_t n_events);

/* moe_forward with step 7 (the top-k weighted combine) in the epilogue of
 * step 6, the down GEMM ("4 · La fusion de noyaux", §4.2 "GEMM + épilogue",
 * with one counter per piece of output as in §4.2 "GEMM + GEMM"): a unit of
 * the down GEMM that has stored its output rows of a 128-feature tile counts
 * one arrival per routed row in a per-(tile, token) counter of the workspace
 * (zeroed by the gather kernel), and the arrival that completes a token's k
 * rows sums them in routing-slot order j = 0..k-1 into y, with the separate
 * combine kernel's arithmetic: the same output bits as moe_forward, 5 launches
 * (7 with the multi-CTA top-k and align).  No thread ever waits on a counter.
 * `events` is NULL, or as for moe_forward_events (events[7] then follows
 * events[6] at once).  moe_forward stays the faster choice on GB300: the
 * epilogue's chain of store, fence, counter atomic and reads of the other
 * rows is as long as the kernel boundary it saves in decode, and in prefill
 * the epilogue waits on rows read back from DRAM and holds up the tensor
 * cores. */
MOE_API moe_status moe_forward_fused_combine(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                             const float* w_router, const float* router_bias, const moe_bf16* w13,
                                             const moe_bf16* w2, moe_bf16* y, void* workspace,
                                             size_t workspace_bytes, moe_stream_t stream, void* const* events,
                                             int32_t n_events);

/* moe_forward with both expert GEMMs in one persistent launch (the GEMM ->
 * GEMM fusion of "4 · La fusion de noyaux", §4.2 "GEMM + GEMM", grown into
 * the megakernel of §4.6): every CTA runs its stream-K share of the gate/up
 * GEMM, then its share of the down GEMM; a down-GEMM unit loads its
 * activation rows once every gate/up unit of its expert and token chunk has
 * counted the stores of its four epilogue warps in a per-chunk counter of the
 * workspace (zeroed by the align kernel; release add, acquire poll, proxy
 * fence before the TMA reads), while its weight tiles stream in ahead.  Same
 * K split as moe_forward, so the same output bits.  Decode tile plan only
 * (T * top_k <= 16 * E), else MOE_ERR_UNSUPPORTED before anything is
 * enqueued.  `events` as for moe_forward_events (events[6] then follows
 * events[5] at once).  moe_forward stays the faster choice on GB300: the
 * launch boundary saved (~4 us) is lost again because the fused kernel's
 * gate/up phase runs slower than the separate gate/up kernel. */
MOE_API moe_status moe_forward_fused_mlp(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                         const float* w_router, const float* router_bias, const moe_bf16* w13,
                                         const moe_bf16* w2, moe_bf16* y, void* workspace, size_t workspace_bytes,
                                         moe_stream_t stream, void* const* events, int32_t n_events);

/* Routing front end only (RMSNorm, router, top-k, align with `pad_rows`
 * rows of padding granularity), with the results copied out:
 *   topk_ids       [T, top_k] int32   selected experts, best first
 *   topk_w         [T, top_k] fp32    their weights
 *   expert_offsets [E + 1]    int32   start row of each expert's padded list;
 *                                     expert_offsets[E] = total rows P
 *   sorted_ids     [sorted_capacity] int32: rows [0, P) hold the flat index
 *                  t*top_k + j routed there (increasing within an expert),
 *                  padding rows hold T*top_k; entries in [P, T*top_k + E*(pad_rows-1))
 *                  are unspecified, entries beyond that are not written.
 * sorted_capacity must be >= T*top_k + E*(pad_rows - 1).  pad_rows: 1..256.
 * The workspace must be sized by moe_workspace_size() for the same shape. */
MOE_API moe_status moe_route_debug(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                           const float* w_router, const float* router_bias, int32_t pad_rows,
                           int32_t* topk_ids, float* topk_w, int32_t* expert_offsets,
                           int32_t* sorted_ids, int64_t sorted_capacity, void* workspace,
                           size_t workspace_bytes, moe_stream_t stream);

/* Bytes of the fixed device scratch array used by moe_forward_static_scratch. */
#define MOE_STATIC_SCRATCH_BYTES (64ull << 20)

/* moe_forward without a caller-provided workspace and without allocating.
 * The pages have no counterpart of this call; it exists for callers that
 * cannot allocate device memory: hosts that give all device memory to their
 * own pool or run under a fixed budget, callers without a device allocator
 * (plain C, plug-ins), and latency-critical loops that avoid cudaMalloc /
 * cudaFree because those can block and synchronise the device.
 * The scratch is a file-scope __device__ array of MOE_STATIC_SCRATCH_BYTES
 * (64 MiB) inside the library; every GPU that loads the library holds it
 * until the process exits.  The caller still passes inputs and output, as
 * for moe_forward.
 *   - Shapes whose moe_workspace_size() exceeds MOE_STATIC_SCRATCH_BYTES are
 *     rejected with MOE_ERR_WORKSPACE before anything is enqueued (e.g. the
 *     decode layer H = I = 4096, E = 64, top_k = 8 fits for T <= 128: at
 *     T = 129 its tile plan changes and it needs 117 MB).
 *   - The first call on a device (with that device current) looks up the
 *     array's device address once (cudaGetSymbolAddress) and keeps it; make
 *     that first call before any stream capture.
 *   - Every call on a device shares the one array, which keeps the last
 *     call's contents; each call rewrites everything it reads, so nothing
 *     has to be cleared between calls.  Calls whose work overlaps on the GPU
 *     (other streams, other host threads) race on the array: serialise them.
 *   - The intermediate tensors are not exposed (no moe_workspace_views).
 *     Device-detected errors go to the error word at the start of the array;
 *     moe_static_scratch_device_status() reads it.
 *   - No cudaMalloc, cudaFree or allocating library routine is called. */
MOE_API moe_status moe_forward_static_scratch(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                              const float* w_router, const float* router_bias, const moe_bf16* w13,
                                              const moe_bf16* w2, moe_bf16* y, moe_stream_t stream);

/* The size of that array as compiled into the library (the value of
 * MOE_STATIC_SCRATCH_BYTES the library was built with), for bindings that
 * cannot read the macro.  Host-only; makes no CUDA call. */
MOE_API moe_status moe_static_scratch_bytes(size_t* bytes);

/* moe_device_status for moe_forward_static_scratch: waits for `stream`, then
 * reads the error word of the current device's static array (the one the
 * last moe_forward_static_scratch call on this device used; it is cleared by
 * the first kernel of every such call).  Returns MOE_OK, MOE_ERR_TIMEOUT or
 * MOE_ERR_DEVICE as moe_device_status does; `detail` (int32[4] or NULL)
 * receives the word.  Like the first moe_forward_static_scratch call, the
 * first call of either on a device looks up the array's address. */
MOE_API moe_status moe_static_scratch_device_status(moe_stream_t stream, int32_t* detail);

/* Device pointers to the intermediate tensors inside a workspace, valid for
 * the shape it was sized for (layout only; makes no CUDA call). */
typedef struct {
  void* error_word;   /* int32[4]: code, kernel id, detail, detail */
  void* h;            /* [T, H] bf16 RMSNorm output */
  void* logits;       /* [T, E] fp32 router logits (bias included) */
  void* topk_ids;     /* [T, top_k] int32 */
  void* topk_w;       /* [T, top_k] fp32 */
  void* counts;       /* [E] int32 tokens per expert */
  void* offsets;      /* [E + 1] int32 padded row offsets (16-row padding) */
  void* sorted_ids;   /* [P_max] int32 */
  void* slot_of;      /* [T * top_k] int32 row of each routed token */
  void* xg;           /* [P_max, H] bf16 gathered, padded expert inputs; written
                       * only where a gather kernel runs: moe_forward's decode
                       * tile plan (T * top_k <= 16 E) reads the rows of h in
                       * the gate/up GEMM instead (unless the combine is fused) */
  void* act;          /* [P_max, I] bf16 SwiGLU activations */
  void* out_rows;     /* [P_max, H] bf16 per-row expert outputs */
  int64_t P_max;      /* T*top_k + E*15: the most padded rows any routing can need */
} moe_views;

/* Device addresses of the block-scaled layers' extra intermediates (MXFP8,
 * MXFP4 and NVFP4; their token codes are in moe_views.xg, two per byte for the
 * FP4 layers).  Scales in the layouts described below. */
typedef struct {
  void* x_codes;    /* [P_max, H] E4M3 codes of the gathered token rows */
  void* x_scales;   /* their scales */
  void* act_codes;  /* [P_max, I] E4M3 codes of the SwiGLU activations */
  void* act_scales; /* their scales */
  int32_t x_chunk_rows;    /* token rows per scale chunk of x_scales (the gate/up GEMM's unit) */
  int32_t act_chunk_rows;  /* the same for act_scales (the down GEMM's unit) */
  void* x_gscale;          /* NVFP4 layer: [P_max] fp32 tensor scale of each gathered token row */
  void* act_gscale;        /* NVFP4 layer: [P_max] fp32 tensor scale of each activation row */
  int32_t nv_chunk_rows;   /* NVFP4 layer: token rows per scale chunk, both GEMMs (one CTA per unit) */
} moe_mx_views;

MOE_API moe_status moe_workspace_views_mx(const moe_shape* shape, void* workspace, size_t workspace_bytes,
                                          moe_views* views, moe_mx_views* mx_views);

MOE_API moe_status moe_workspace_views(const moe_shape* shape, void* workspace, size_t workspace_bytes,
                               moe_views* views);

/* Waits for `stream`, then reads the workspace's error word: MOE_OK, or the
 * device-side error of the last call that used this workspace
 * (MOE_ERR_TIMEOUT / MOE_ERR_DEVICE).  detail (may be NULL) receives the
 * four raw int32 words: the code, the id of the kernel that recorded it
 * (1 norm/router, 2 top-k, 3 align, 4 gather, 5 gate/up GEMM, 6 down GEMM,
 * 7 combine, 8 self-test, 9 grouped products' tables, 10 grouped GEMM,
 * 11 grouped 4-bit GEMM, 12 grouped 8-bit GEMM), for the expert GEMMs a bit mask of the waits that
 * ran out (bit 1 producer: ring slot free; 2 MMA: accumulator free; 3 MMA:
 * ring slot loaded; 4 epilogue: accumulator complete; 5 epilogue: stream-K
 * partial sums; 6 epilogue: fused-combine rendezvous; 7 MMA: a stage's scales
 * written to TMEM; 8 scale warps: ring slot loaded; 10 a CTA pair's next unit), and the index of the CTA
 * that recorded the timeout. */
MOE_API moe_status moe_device_status(const void* workspace, size_t workspace_bytes, moe_stream_t stream,
                             int32_t* detail);

/* Static text for a status code. */
/* ---- FP8 expert weights (MXFP8) --------------------------------------
 * Block-scaled FP8 ("CuTeDSL chez Perplexity", "Prise en charge de Blackwell":
 * MXFP8, an absolute maximum over 32 elements): every 32 consecutive elements
 * along the reduction dimension share a power-of-two scale X = 2^E (one E8M0
 * byte, E + 127) with E = floor(log2(amax)) - 8 clamped to [-127, 127] (-127 for
 * an all-zero block); each element is stored as the E4M3 code of x / X, rounded
 * to nearest even and clamped to +-448.
 * Codes keep the matrix layout (one byte per element).  Scales are stored for
 * the block-scaled tensor-core MMA: per 128-row group and 128-element chunk of
 * the reduction dimension a 512-byte tile, byte r*16 + 4*j + b holding the
 * scale of row 32*j + r of the group and 32-element block b of the chunk.  For
 * W13 the rows of a group are the gate/up GEMM's tile rows: group e*(I/64) + t
 * holds features [64t, 64t+64) of expert e as, for g = 0..3, the 16 gate rows
 * 64t+16g .. +15 then the 16 matching up rows.  W2 groups are 128 consecutive
 * rows. */

/* Byte sizes of the MXFP8 copies of W13 and W2 for this shape. */
MOE_API moe_status moe_mx_weight_sizes(const moe_shape* shape, size_t* w13_codes, size_t* w13_scales,
                                       size_t* w2_codes, size_t* w2_scales);

/* Quantize the bf16 expert weights (layouts as for moe_forward) to MXFP8 on
 * the device (asynchronous on `stream`).  All pointers device, 16-byte aligned,
 * sized by moe_mx_weight_sizes. */
MOE_API moe_status moe_mx_quantize_weights(const moe_shape* shape, const moe_bf16* w13, const moe_bf16* w2,
                                           uint8_t* w13_codes, uint8_t* w13_scales, uint8_t* w2_codes,
                                           uint8_t* w2_scales, moe_stream_t stream);

/* Workspace bytes of moe_forward_mx (larger than moe_workspace_size's). */
MOE_API moe_status moe_workspace_size_mx(const moe_shape* shape, size_t* bytes);

/* The layer with MXFP8 expert weights: the same norm, router, top-k and
 * combine as moe_forward; each expert's input rows (the bf16 h) and its bf16
 * SwiGLU activations are quantized to MXFP8 the same way and the two expert
 * GEMMs run on the block-scaled tensor cores (tcgen05.mma kind::mxf8f6f4,
 * fp32 accumulation), in work units of 32 token rows (T * top_k / E <= 16)
 * or else 128, or 256 on CTA pairs where an expert's weight tiles come in
 * pairs (the tile plans of moe_forward).  Expert lists are padded to
 * 32 rows.  E <= 256 (else MOE_ERR_UNSUPPORTED).  events: NULL
 * or as for moe_forward_events (events[1] ends routing and align, events[4]
 * the gather + quantize, events[6] the activation quantize + down GEMM). */
MOE_API moe_status moe_forward_mx(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                  const float* w_router, const float* router_bias, const uint8_t* w13_codes,
                                  const uint8_t* w13_scales, const uint8_t* w2_codes, const uint8_t* w2_scales,
                                  moe_bf16* y, void* workspace, size_t workspace_bytes, moe_stream_t stream,
                                  void* const* events, int32_t n_events);

/* ---- FP4 expert weights (MXFP4) --------------------------------------
 * Block-scaled 4-bit weights (the same pages list Blackwell's block-scaled
 * FP4 formats beside MXFP8, "CuTeDSL chez Perplexity", "Prise en charge de
 * Blackwell"; the OCP Microscaling rule with E2M1 elements): every 32
 * consecutive elements along the reduction dimension share X = 2^E (one E8M0
 * byte, E + 127) with E = floor(log2(amax)) - 2 clamped to [-127, 127] (-127
 * for an all-zero block); each element is the E2M1 code of x / X (magnitudes
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6; sign in bit 3) rounded to nearest with ties to
 * the even code and clamped to +-6.  Codes: the matrix layout with two codes
 * per byte, element 2i in the low nibble of byte i ([rows, K/2] bytes).
 * Scales: the MXFP8 layout above (the same tiles, the same W13 row order). */

/* Byte sizes of the MXFP4 copies of W13 and W2 for this shape (codes: half
 * the MXFP8 sizes; scales: the same). */
MOE_API moe_status moe_mxfp4_weight_sizes(const moe_shape* shape, size_t* w13_codes, size_t* w13_scales,
                                          size_t* w2_codes, size_t* w2_scales);

/* Quantize the bf16 expert weights (layouts as for moe_forward) to MXFP4 on
 * the device (asynchronous on `stream`).  All pointers device, sized by
 * moe_mxfp4_weight_sizes; codes 32-byte aligned (the tensor maps' rule for
 * packed 4-bit data), the rest 16-byte aligned; else MOE_ERR_INVALID_ARG. */
MOE_API moe_status moe_mxfp4_quantize_weights(const moe_shape* shape, const moe_bf16* w13, const moe_bf16* w2,
                                              uint8_t* w13_codes, uint8_t* w13_scales, uint8_t* w2_codes,
                                              uint8_t* w2_scales, moe_stream_t stream);

/* The layer with MXFP4 expert weights (W4A8): as moe_forward_mx (the same
 * routing, MXFP8 token rows and activations, tile plans, workspace
 * moe_workspace_size_mx and views moe_workspace_views_mx, events), with the
 * weights as E2M1 codes in the block-scaled MMA (tcgen05.mma
 * kind::mxf8f6f4, A = E2M1 weights, B = E4M3 tokens, fp32 accumulation).
 * Weight codes 32-byte aligned, else MOE_ERR_INVALID_ARG. */
MOE_API moe_status moe_forward_mxfp4(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                     const float* w_router, const float* router_bias, const uint8_t* w13_codes,
                                     const uint8_t* w13_scales, const uint8_t* w2_codes, const uint8_t* w2_scales,
                                     moe_bf16* y, void* workspace, size_t workspace_bytes, moe_stream_t stream,
                                     void* const* events, int32_t n_events);

/* The MXFP4 layer (W4A4): as moe_forward_mxfp4 (the same MXFP4 weights from
 * moe_mxfp4_quantize_weights, workspace, views and events), with each expert's
 * input rows and its SwiGLU activations quantized to MXFP4 by the same rule
 * as the weights, and both expert GEMMs on packed E2M1 operands (tcgen05.mma
 * kind::mxf4, two E8M0 scales per row per MMA of K = 64, fp32 accumulation).
 * H and I multiples of 128 like every block-scaled layer (else
 * MOE_ERR_UNSUPPORTED; a GEMM stage covers 256 elements of K, and an odd
 * multiple of 128 ends half way into the last one); weight codes 32-byte
 * aligned. */
MOE_API moe_status moe_forward_mxfp4a4(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                       const float* w_router, const float* router_bias, const uint8_t* w13_codes,
                                       const uint8_t* w13_scales, const uint8_t* w2_codes, const uint8_t* w2_scales,
                                       moe_bf16* y, void* workspace, size_t workspace_bytes, moe_stream_t stream,
                                       void* const* events, int32_t n_events);

/* ---- NVFP4 (E2M1 codes, E4M3 scales per 16, fp32 tensor scales) ---------
 * NVFP4 (the same pages name it beside MXFP8 / MXFP4, with an absolute
 * maximum over 16 elements; its published two-level form): every 16
 * consecutive elements along the reduction dimension share an E4M3 scale s
 * (sign 0), every tensor an fp32 scale g = amax_tensor / (448 * 6) (1 for an
 * all-zero tensor); s = E4M3(amax_16 / (6 g)) (nearest even, saturating to
 * 448) and each element the E2M1 code of x / (value(s) * g) (0 where that is
 * 0), each step one fp32 operation in this order.  The tensor of a weight is
 * one expert matrix (W13_e, W2_e); that of the token rows and activations one
 * row.  Codes: two per byte as for MXFP4.  Scales: 512-byte tiles per 128
 * rows and 64 elements of K, byte r*16 + 4*j + b = the scale of row 32*j + r
 * and 16-element block b of the 64 (W13 rows in the gate/up tile-row order as
 * for MXFP8). */

/* Byte sizes of the NVFP4 copies of W13 and W2 (their tensor scales: E floats
 * each, caller-sized). */
MOE_API moe_status moe_nvfp4_weight_sizes(const moe_shape* shape, size_t* w13_codes, size_t* w13_scales,
                                          size_t* w2_codes, size_t* w2_scales);

/* Quantize the bf16 expert weights to NVFP4 on the device (asynchronous on
 * `stream`): codes and block scales sized by moe_nvfp4_weight_sizes, tensor
 * scales w13_gscale[E], w2_gscale[E] (fp32; they hold the absolute maxima
 * until the last kernel of the call has run).  Codes 32-byte aligned, scales
 * 16-byte, tensor scales 4-byte aligned; else MOE_ERR_INVALID_ARG. */
MOE_API moe_status moe_nvfp4_quantize_weights(const moe_shape* shape, const moe_bf16* w13, const moe_bf16* w2,
                                              uint8_t* w13_codes, uint8_t* w13_scales, float* w13_gscale,
                                              uint8_t* w2_codes, uint8_t* w2_scales, float* w2_gscale,
                                              moe_stream_t stream);

/* The NVFP4 layer: as moe_forward_mxfp4a4 with NVFP4 weights, token rows and
 * activations (tcgen05.mma kind::mxf4nvf4, scale_vec::4X: four E4M3 scales per
 * row per MMA of K = 64; the fp32 tensor scales of the expert matrix and of the
 * token row multiply each accumulator in the epilogue), one CTA per work unit
 * in every tile plan.  H and I multiples of 128 (else MOE_ERR_UNSUPPORTED). */
MOE_API moe_status moe_forward_nvfp4(const moe_shape* shape, const moe_bf16* x, const moe_bf16* g_norm,
                                     const float* w_router, const float* router_bias, const uint8_t* w13_codes,
                                     const uint8_t* w13_scales, const float* w13_gscale, const uint8_t* w2_codes,
                                     const uint8_t* w2_scales, const float* w2_gscale, moe_bf16* y, void* workspace,
                                     size_t workspace_bytes, moe_stream_t stream, void* const* events,
                                     int32_t n_events);

/* QK-norm, in place: RMSNorm of every attention head of Q and of K
 * ("CuTeDSL chez Perplexity", "Norme QK"):
 *   out_j = bf16((w_j + weight_bias) * (x_j * rstd)),  rstd = 1/sqrt(mean_j x_j^2 + eps),
 * over the D elements of each head, with q_weight[D] applied to every head of Q
 * and k_weight[D] to every head of K.  Computed in fp32 in one fixed order
 * (see k_qk_norm.cu), so the result is within one bf16 ulp of the exact value.
 *   q [T, Hq, D] bf16, k [T, Hk, D] bf16: device, contiguous, 16-byte aligned,
 *   overwritten with the result; q_weight / k_weight [D] bf16.
 *   D: 64, 128 or 256.  Hq or Hk may be 0 (its pointers are then unused).
 * Errors: MOE_ERR_INVALID_ARG for a bad D, negative sizes, null or misaligned
 * pointers of a non-empty tensor, or a non-finite eps / weight_bias;
 * MOE_ERR_UNSUPPORTED for T * (Hq + Hk) >= 2^31 heads; T = 0 is a no-op.
 * Asynchronous on `stream`; no workspace. */
MOE_API moe_status moe_qk_norm(int64_t T, int32_t Hq, int32_t Hk, int32_t D, moe_bf16* q, moe_bf16* k,
                               const moe_bf16* q_weight, const moe_bf16* k_weight, float weight_bias, float eps,
                               moe_stream_t stream);

/* ---- Products grouped by expert, and their gradients ------------------
 * The experts' matrix products on their own, for callers that bring their own
 * routing or train the experts: rows of the token matrices belong to groups
 * (experts), group g holding rows [offsets[g], offsets[g] + counts[g]), any
 * number of them, none included; w is [groups, N, K] (K-major like W13 and W2).
 *   forward          y[p, :]  = x[p, :] w_g^T                    (p in group g)
 *   input gradient   dx[p, :] = dy[p, :] w_g
 *   weight gradient  dw_g     = sum over the group's p of dy[p, :]^T x[p, :]
 * The lists moe_route_debug and moe_views give (offsets with padding between
 * the groups, counts) are such groups.  Products are summed in fp32 and each
 * output is rounded once.  The order of the sums follows the shape, the lists
 * and the device: calls with the same ones repeat bit for bit.  A row's last bits
 * can change with other groups' counts: forward and input gradient of at most 24
 * rows a group on average split the sums wherever the lists make the work even.
 * The tensor core cuts an fp32 sum towards zero once for every 16 products (4
 * bits: 64), by at most 17 * 2^-23 (65 * 2^-23) of the sum of their magnitudes;
 * measured, some 2^-24.
 *   offsets  [groups + 1] int32, device: offsets[g] + counts[g] <= offsets[g+1]
 *            and offsets[groups] <= rows; or NULL: equal groups of
 *            rows / groups rows (rows a multiple of groups, else
 *            MOE_ERR_INVALID_ARG)
 *   counts   [groups] int32, device, or NULL: offsets[g + 1] - offsets[g]
 * Rows that belong to no group are not written, and what they hold (NaN
 * included) reaches no output.  Offsets that break the rules above are found on
 * the device: nothing is written then, and moe_device_status() returns MOE_ERR_DEVICE with
 * kernel id 9 and the first such group's index (detail[2]).
 *   type     of x, w, y, dy, dx: MOE_TYPE_BF16 or MOE_TYPE_FP16
 *   ldx ...  row strides in elements: >= the row's width, multiples of 8
 *   N, K     multiples of 8, <= 2^20; groups <= 1024; rows <= 2^31 - 512
 *            (others: MOE_ERR_UNSUPPORTED)
 *   workspace  moe_grouped_workspace_size() bytes of the shape (of as many rows as
 *            any call brings), 256-byte aligned; contents on entry do not matter;
 *            one call at a time uses it (two graphs that share one are replayed
 *            one after the other).
 * Matrices 16-byte aligned, outputs apart from the inputs.  Asynchronous on
 * `stream`, capturable like every call.  rows = 0 is a no-op (the weight
 * gradient still writes its zeros, unless it accumulates): nothing is enqueued, and
 * moe_device_status() goes on to say what the call before reported, or on a workspace
 * that no call has used, whatever its memory holds. */
#define MOE_TYPE_BF16 0
#define MOE_TYPE_FP16 1
#define MOE_TYPE_FP32 2

typedef struct {
  int32_t groups, N, K;
  int32_t type;
  int64_t rows; /* rows of the token matrices, those of no group included */
} moe_grouped_shape;

/* Host only; makes no CUDA call. */
MOE_API moe_status moe_grouped_workspace_size(const moe_grouped_shape* shape, size_t* bytes);

/* y [rows, N] from x [rows, K]. */
MOE_API moe_status moe_grouped_gemm(const moe_grouped_shape* shape, const void* x, int64_t ldx, const void* w,
                                    const int32_t* offsets, const int32_t* counts, void* y, int64_t ldy,
                                    void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* dx [rows, K] from dy [rows, N]; w as in the forward (no transposed copy). */
MOE_API moe_status moe_grouped_gemm_dgrad(const moe_grouped_shape* shape, const void* dy, int64_t lddy, const void* w,
                                          const int32_t* offsets, const int32_t* counts, void* dx, int64_t lddx,
                                          void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* dw [groups, N, K] of dw_type (the operands' type, or MOE_TYPE_FP32): written
 * whole, zeros for an empty group; or, with accumulate != 0 (MOE_TYPE_FP32
 * only, else MOE_ERR_INVALID_ARG), added to what dw holds.  The tensor core (which
 * cuts, see above) accumulates 768 rows of a group at most, or 3840 for a dw of 16
 * bits, where the cuts stay below half an fp16 step of the sum of |dy x|; the sums
 * of such segments are added in fp32, rounded to nearest, and dw is rounded once.
 * Into 16 bits: rows <= 2^26 (else MOE_ERR_UNSUPPORTED); more than 3840 rows want
 * the workspace that moe_grouped_workspace_size() gives for them, 29 MB more. */
MOE_API moe_status moe_grouped_gemm_wgrad(const moe_grouped_shape* shape, const void* dy, int64_t lddy, const void* x,
                                          int64_t ldx, const int32_t* offsets, const int32_t* counts, void* dw,
                                          int32_t dw_type, int32_t accumulate, void* workspace,
                                          size_t workspace_bytes, moe_stream_t stream);

/* ---- Rows in 4 bits, and their grouped product -------------------------
 * MXFP4 and NVFP4 of any rows (the formats of the layer's weights, above; here
 * in plain row order), back, and the forward product of the grouped products
 * on such operands (tcgen05.mma kind::mxf4 / kind::mxf4nvf4, fp32 accumulation).
 *   codes   [rows, K / 2] bytes, two E2M1 codes each, element 2i in the low nibble
 *   scales  512-byte tiles of 128 rows x 4 blocks of K (128 elements for MXFP4, 64
 *           for NVFP4): byte r*16 + 4*j + b = the scale of row 32*j + r, block b;
 *           the ceil(K / 128) (ceil(K / 64)) tiles of one tile row adjacent, blocks past K
 *           zero.  A group's rows start a tile row of their own: for equal
 *           groups of R rows (offsets NULL; weights [groups, N, K] are groups
 *           of N rows) group g starts at tile row g * ceil(R / 128), for listed
 *           ones at floor(offsets[g] / 128) + g.
 *   gscale  NVFP4's fp32 scales: one per row (MOE_SCALE_PER_ROW, [rows]) or
 *           one per group (MOE_SCALE_PER_GROUP, [groups]); unused (NULL) for MXFP4
 * MXFP4: a block with a NaN or an infinity gets the NaN scale 255; NVFP4: a row
 * (group) with one gets a NaN gscale; what they stand for is NaN.
 * offsets, counts, rows, groups, strides and alignment as for the grouped
 * products; K a multiple of 32 (else MOE_ERR_UNSUPPORTED); codes and scales
 * 16-byte aligned.  Rows of no group are skipped; lists that break the rules
 * are not reported by these two calls (rows they misplace are skipped), but by
 * the product. */
#define MOE_FORMAT_MXFP4 0
#define MOE_FORMAT_NVFP4 1
#define MOE_SCALE_PER_ROW 0
#define MOE_SCALE_PER_GROUP 1

typedef struct {
  int32_t format;
  int32_t groups;
  int64_t rows;
  int32_t K;
} moe_fp4_shape;

/* Byte sizes of codes and scales, enough for any lists.  Host only. */
MOE_API moe_status moe_fp4_sizes(const moe_fp4_shape* shape, size_t* codes, size_t* scales);

/* src [rows, K] of src_type (MOE_TYPE_*) -> codes, scales, gscale. */
MOE_API moe_status moe_fp4_quantize(const moe_fp4_shape* shape, int32_t src_type, const void* src, int64_t ldsrc,
                                    const int32_t* offsets, const int32_t* counts, uint8_t* codes, uint8_t* scales,
                                    float* gscale, int32_t gscale_per, moe_stream_t stream);

/* The values the codes stand for, rounded to dst_type, into dst [rows, K]. */
MOE_API moe_status moe_fp4_dequantize(const moe_fp4_shape* shape, const uint8_t* codes, const uint8_t* scales,
                                      const float* gscale, int32_t gscale_per, const int32_t* offsets,
                                      const int32_t* counts, int32_t dst_type, void* dst, int64_t lddst,
                                      moe_stream_t stream);

/* y[p, :] = x[p, :] w_g^T as moe_grouped_gemm (lists, workspace of
 * moe_grouped_workspace_size(), errors; GEMM kernel id 11), with x quantized
 * for the same lists (NVFP4: x_gscale per row) and w as groups of N rows without
 * lists (NVFP4: w_gscale per group).  shape->type: y's type. */
MOE_API moe_status moe_fp4_gemm(const moe_grouped_shape* shape, int32_t format, const uint8_t* x_codes,
                                const uint8_t* x_scales, const float* x_gscale, const uint8_t* w_codes,
                                const uint8_t* w_scales, const float* w_gscale, const int32_t* offsets,
                                const int32_t* counts, void* y, int64_t ldy, void* workspace,
                                size_t workspace_bytes, moe_stream_t stream);

/* ---- Rows in 8 bits with scales of 128, and their grouped products ------
 * E4M3 codes under fp32 scales: 128 consecutive elements of a row share one, or
 * (weights) a block of 128 x 128:
 *   s = (largest magnitude) / 448, or 1 where that is 0;  code = E4M3(x / s)
 * each division one fp32 operation, codes to nearest with ties to the even one;
 * a block that holds a NaN or an infinity gets a NaN scale (what it stands for is
 * NaN).  The products sum each block's codes on the tensor core (kind::f8f6f4)
 * and add sx sw times that sum in fp32, so the scales may be any numbers: where sx sw
 * is no normal fp32 number, the sum is multiplied by the larger scale, then by the smaller.
 *   codes   [rows, K] bytes
 *   scales  MOE_SCALE_PER_ROW: [rows][lds] fp32, block b of row p at p * lds + b
 *           (lds >= ceil(K / 128), a multiple of 4; what lies between them is unspecified);
 *           MOE_SCALE_PER_BLOCK: `groups` matrices of N = rows / groups rows each,
 *           [groups][ceil(N / 128)][ceil(K / 128)] (lds unused, blocks at the edges smaller)
 * K a multiple of 16 and <= 2^20; rows <= 2^31 - 512; row strides in elements,
 * multiples of 8; src, dst, codes and scales 16-byte aligned.  No lists:
 * all rows are quantized, those of no group reach no product. */
#define MOE_SCALE_PER_BLOCK 2

typedef struct {
  int32_t scale_per; /* MOE_SCALE_PER_ROW or MOE_SCALE_PER_BLOCK */
  int32_t groups;    /* MOE_SCALE_PER_BLOCK: matrices, 1 .. 1024, rows a multiple of it (else unused) */
  int64_t rows;
  int32_t K;
} moe_fp8_shape;

/* Byte sizes of codes and scales (lds = ceil(K / 128) rounded up to 4).  Host only. */
MOE_API moe_status moe_fp8_sizes(const moe_fp8_shape* shape, size_t* codes, size_t* scales);

/* src [rows, K] of src_type (MOE_TYPE_*) -> codes, scales. */
MOE_API moe_status moe_fp8_quantize(const moe_fp8_shape* shape, int32_t src_type, const void* src, int64_t ldsrc,
                                    uint8_t* codes, float* scales, int64_t lds, moe_stream_t stream);

/* The values the codes stand for (code * s), rounded to dst_type, into dst [rows, K]. */
MOE_API moe_status moe_fp8_dequantize(const moe_fp8_shape* shape, const uint8_t* codes, const float* scales,
                                      int64_t lds, int32_t dst_type, void* dst, int64_t lddst, moe_stream_t stream);

/* y[p, :] = x[p, :] w_g^T and dx[p, :] = dy[p, :] w_g as moe_grouped_gemm and its
 * input gradient (lists, workspace of moe_grouped_workspace_size(), errors; GEMM
 * kernel id 12), with x [rows, K] (dy [rows, N]) quantized per row and w
 * [groups, N, K] quantized per block, once for both products.  N and K multiples
 * of 16 (else MOE_ERR_UNSUPPORTED).  shape->type: the type of y (dx).  The host does
 * not see the lists, so the tile plan follows the mean, rows / groups (rows of no group
 * count): where a few of many groups hold nearly all rows, a mean of up to 16 costs
 * these groups three to four times what they need.  (The weight
 * gradient sums over rows, whose scales differ: moe_grouped_gemm_wgrad takes 16 bits.) */
MOE_API moe_status moe_fp8_gemm(const moe_grouped_shape* shape, const uint8_t* x_codes, const float* x_scales,
                                int64_t ldxs, const uint8_t* w_codes, const float* w_scales, const int32_t* offsets,
                                const int32_t* counts, void* y, int64_t ldy, void* workspace,
                                size_t workspace_bytes, moe_stream_t stream);
MOE_API moe_status moe_fp8_gemm_dgrad(const moe_grouped_shape* shape, const uint8_t* dy_codes,
                                      const float* dy_scales, int64_t ldds, const uint8_t* w_codes,
                                      const float* w_scales, const int32_t* offsets, const int32_t* counts, void* dx,
                                      int64_t lddx, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* SwiGLU of separate rows, between the gate/up and the down product: h
 * [rows, 2I] holds gate in columns [0, I) and up in [I, 2I) (the order of a
 * W13 product), act [rows, I] = SiLU(gate) * up; and its gradient,
 * dh [rows, 2I] from dact [rows, I].  dh may be h itself (lddh = ldh).  type, strides,
 * alignment and rows as above; I a multiple of 8, rows * I < 2^34. */
MOE_API moe_status moe_swiglu(int32_t type, int64_t rows, int32_t I, const void* h, int64_t ldh, void* act,
                              int64_t ldact, moe_stream_t stream);
MOE_API moe_status moe_swiglu_grad(int32_t type, int64_t rows, int32_t I, const void* h, int64_t ldh,
                                   const void* dact, int64_t lddact, void* dh, int64_t lddh, moe_stream_t stream);

/* ---- The norm of rows, and its gradient --------------------------------
 * What the layer does to its tokens first, on its own, with the layer norm
 * beside it and the gradients of both:
 *   n = (x - m) r,  r = 1 / sqrt(mean((x - m)^2) + eps),  y = n weight + bias
 * over the H elements of each row, m the row's mean (MOE_NORM_LAYER) or 0
 * (MOE_NORM_RMS, no bias); and with e = dy weight
 *   dx = r (e - mean(e) - n mean(e n))       (MOE_NORM_RMS: without mean(e))
 *   dweight = sum over the rows of dy n,  dbias = sum over the rows of dy
 * fp32 inside, one rounding per output; a row's results depend on the row alone,
 * and calls repeat bit for bit.  Squares and sums are fp32 numbers: rows whose
 * squares do not fit them (|x| above some 1e17) get r = 0, rows of the layer norm whose
 * sum does not (|x| above some 1e34) a NaN; with eps = 0, rows whose squares vanish (|x|
 * below some 1e-23) r = infinity.
 *   type         of x, y, dy, dx: MOE_TYPE_*
 *   weight_type  of weight and bias: type, or MOE_TYPE_FP32
 *   weight, bias [H], NULL for ones and zeros
 *   mean, rstd   [rows] fp32: m and r, written by moe_norm (NULL: not kept) and
 *                read by the gradient; MOE_NORM_RMS has no mean (NULL)
 *   dweight, dbias  [H] of dweight_type (weight_type or MOE_TYPE_FP32), NULL where not
 *                wanted; or, with accumulate != 0 (MOE_TYPE_FP32 only), added to
 *                what they hold; MOE_NORM_RMS has no dbias (NULL)
 *   workspace    moe_norm_grad_workspace_size() bytes, 256-byte aligned, contents on entry
 *                do not matter, one call at a time uses it; unused (NULL) without dweight and dbias
 * H a multiple of 8, <= 16384; rows <= 2^31 - 512; row strides in elements,
 * multiples of 8; matrices, weight, bias and their gradients 16-byte aligned.  y may be x, and dx
 * dy or x, with the same row stride.  rows = 0 is a no-op, but the gradient still writes
 * zeros into dweight and dbias, unless it accumulates.  Asynchronous on `stream`. */
#define MOE_NORM_RMS 0
#define MOE_NORM_LAYER 1

typedef struct {
  int32_t kind;
  int32_t type, weight_type;
  int32_t H;
  int64_t rows;
  float eps; /* >= 0, finite */
} moe_norm_shape;

MOE_API moe_status moe_norm(const moe_norm_shape* shape, const void* x, int64_t ldx, const void* weight,
                            const void* bias, void* y, int64_t ldy, float* mean, float* rstd, moe_stream_t stream);

/* Host only; makes no CUDA call. */
MOE_API moe_status moe_norm_grad_workspace_size(const moe_norm_shape* shape, size_t* bytes);

MOE_API moe_status moe_norm_grad(const moe_norm_shape* shape, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                 const void* weight, const float* mean, const float* rstd, void* dx, int64_t lddx,
                                 void* dweight, void* dbias, int32_t dweight_type, int32_t accumulate,
                                 void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* ---- The norm of all gradients, and clipping ---------------------------
 *   norm = sqrt(sum of the squares of all elements of all tensors)
 *   out = data * min(1, max_norm / (norm + eps))
 * `tensors` is a host array that the call reads before it returns: any number of
 * tensors of any size (n = 0 too; n <= 2^40) and type, n contiguous elements each, aligned
 * to their elements (16-byte borders are faster).  Squares are summed in fp32 for 64
 * elements at most, in fp64 beyond, in a fixed order; no finite element overflows or
 * vanishes, and a norm above fp32's range is infinity.
 *   norm   fp32, device: written by moe_grad_norm and moe_grad_norm_clip, read by
 *          moe_grad_clip (one already known, such as that of these tensors and others)
 *   out    of out_type; may be data itself (with the same type), else apart from
 *          every tensor, and each apart from the others: a tensor given twice would
 *          be clipped twice, or in part.  Unused by moe_grad_norm.
 * Where an element is a NaN or infinite, nothing is clipped (the factor is 1).  Finite
 * elements whose norm passes fp32's range (`norm` is infinity) are clipped by its fp64
 * value in moe_grad_norm_clip; moe_grad_clip, which reads the fp32 number, clips
 * nothing by an infinite or NaN one.  A
 * factor of 1 leaves a tensor in place untouched.  max_norm >= 0 (infinity: never
 * clip), eps >= 0 and finite.  No tensors: the norm is 0.
 *   workspace  moe_grad_norm_workspace_size() bytes for as many tensors, 256-byte aligned,
 *              contents on entry do not matter, one call at a time uses it
 * Asynchronous on `stream`, capturable like every call. */
typedef struct {
  const void* data;
  void* out;
  int64_t n;
  int32_t type, out_type; /* MOE_TYPE_* */
} moe_grad_tensor;

/* Host only; makes no CUDA call. */
MOE_API moe_status moe_grad_norm_workspace_size(int32_t n_tensors, size_t* bytes);
MOE_API moe_status moe_grad_norm(const moe_grad_tensor* tensors, int32_t n_tensors, float* norm, void* workspace,
                                 size_t workspace_bytes, moe_stream_t stream);
MOE_API moe_status moe_grad_clip(const moe_grad_tensor* tensors, int32_t n_tensors, const float* norm,
                                 double max_norm, double eps, moe_stream_t stream);
/* moe_grad_norm and moe_grad_clip by its norm, with less to launch. */
MOE_API moe_status moe_grad_norm_clip(const moe_grad_tensor* tensors, int32_t n_tensors, double max_norm, double eps,
                                      float* norm, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* Self-test of the failure path of the library's bounded device waits (no
 * counterpart on the pages): enqueues one small kernel whose two waits -- on
 * an mbarrier phase that nothing completes and on a flag in the workspace's
 * error area that nothing sets -- give up after timeout_ns (1 .. 1e9) and
 * record MOE_ERR_TIMEOUT, with kernel id 8 in detail[1], in the workspace's
 * error word, then return normally.  moe_device_status() afterwards returns
 * MOE_ERR_TIMEOUT; the CUDA context stays usable, and the next moe_forward on
 * that workspace clears the word.  workspace: >= 64 bytes, 256-byte aligned;
 * its first 64 bytes are overwritten. */
MOE_API moe_status moe_selftest_wait_timeout(void* workspace, size_t workspace_bytes, int64_t timeout_ns,
                                             moe_stream_t stream);

MOE_API const char* moe_status_string(moe_status status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
