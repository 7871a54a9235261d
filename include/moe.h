/*
 * moe.h -- C ABI of the single-GPU MoE-layer forward for GB300 (sm_103a).
 *
 * The operation (from "Mixture-of-Kittens: MoE Megakernel for NVL72s",
 * Sec. 2.1, Eq. "MoE", and the vendor blog's E_i(x) with SiLU):
 *
 *   MoE(x) = f_shared(x) + sum_{i in E(x)} g_i f_i(x),   g_i = s_i / sum_{j in E(x)} s_j,
 *   f_i(x) = W_down^(i) ( SiLU(W_gate^(i) x) * W_up^(i) x ),
 *
 * E(x) = the k routed experts with the highest router score s = score(W_r x + b)
 * (score = sigmoid, or softmax over all experts).  All experts are on this GPU:
 * the paper's cross-GPU dispatch/combine become an on-device gather into a
 * fixed-size ring of minibatches and a scatter back to token order.
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are CUDA device pointers on the plan's device;
 *     the caller owns all memory (inputs, outputs, workspace) and the stream.
 *   - Matrices are row-major; every weight is K-major (its contraction
 *     dimension contiguous), exactly the shapes of Sec. 2.1: W_up, W_gate in
 *     R^{I x D}, W_down in R^{D x I}; expert e's matrix is block e of the
 *     stacked [E, ...] array.
 *   - bf16 = IEEE bfloat16 bit patterns (2 bytes).
 *   - Calls are asynchronous on `stream`, allocate nothing on the device, do
 *     not synchronise the host, and never read device memory on the host;
 *     device-side failures are reported through moe_get_status().
 *   - Return value: MOE_OK (0) or a negative moe_error; no C++ exception
 *     crosses this interface.
 *   - Plans are immutable after creation and may be shared by threads; one
 *     workspace must not be used by two forwards that overlap on the GPU.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* moe_stream_t; /* identical to cudaStream_t */

typedef enum moe_error {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,        /* null pointer, T > T_max, bad enum value */
  MOE_ERR_UNSUPPORTED_SHAPE = -2,  /* shape outside the limits listed at moe_config */
  MOE_ERR_WORKSPACE_TOO_SMALL = -3,
  MOE_ERR_CUDA = -4,               /* a CUDA runtime call failed (launch, copy, attribute) */
  MOE_ERR_UNSUPPORTED_DEVICE = -5, /* the current device is not sm_103 */
  MOE_ERR_STATIC_SCRATCH_TOO_SMALL = -6 /* moe_route_static: request exceeds its fixed scratch */
} moe_error;

typedef enum moe_device_status {
  MOE_STATUS_OK = 0,
  MOE_STATUS_TIMEOUT = 1,          /* a device-side wait exceeded its limit; outputs are invalid */
  MOE_STATUS_SCHEDULE_INVALID = 2, /* an expert index out of range or route counts inconsistent
                                      (moe_fwd_routed: an index out of range or given twice for a token;
                                      a backward: its forward was of the other kind) */
  MOE_STATUS_STAGING_OVERFLOW = 3  /* the forward completed, but an expert output left the fp16 range of
                                      the staging rows (|v| > 65504, or NaN) and was saturated: the
                                      output is finite but not the layer's value */
} moe_device_status;

typedef enum moe_score_fn { MOE_SCORE_SIGMOID = 0, MOE_SCORE_SOFTMAX = 1 } moe_score_fn;
typedef enum moe_precision { MOE_PREC_BF16 = 0, MOE_PREC_MXFP8 = 1 } moe_precision;
typedef enum moe_dispatch { MOE_DISPATCH_RING = 0, MOE_DISPATCH_DIRECT = 1, MOE_DISPATCH_SPREAD = 2 } moe_dispatch;

/*
 * Layer shape and execution knobs.
 *   T_max  largest token count a forward will be called with (>= 1)
 *   D      hidden size, multiple of 256
 *   I      routed-expert intermediate size, multiple of 128
 *   E      routed experts, 1..512
 *   k      experts per token, 1..min(16, E)
 *   I_s    shared-expert intermediate size, multiple of 128, or 0 (no shared expert)
 *   score_fn   moe_score_fn
 *   precision  moe_precision of the routed experts (the router and the shared
 *              expert always run in bf16, Sec. 3.4 "MXFP8 Support")
 *   minibatch  b: routes per minibatch of the dispatch ring, multiple of 128,
 *              128..32768 (Sec. 3.2 sweeps 512..32768)
 *   ring_slots minibatch slots in the ring (>= lag + 1); ring_slots * minibatch
 *              >= T*k gives the over-allocated (no wrap) buffer of Sec. 3.3
 *   dispatch   MOE_DISPATCH_RING: gather CTAs copy the routed tokens into the
 *              ring of minibatches (the pages' communication SMs);
 *              MOE_DISPATCH_DIRECT: the GEMM CTAs' TMA producers fetch each
 *              tile's token rows straight from x (tile::gather4), no gather
 *              CTAs and no x ring (MXFP8: from the router pass's x codes);
 *              MOE_DISPATCH_SPREAD: the same ring as MOE_DISPATCH_RING, filled
 *              by two otherwise idle warps of every GEMM CTA (each takes the
 *              minibatch's M-tiles c, c + gemm CTAs, ...), so every SM runs
 *              expert tiles; gather_ctas is ignored
 *   gather_ctas  ring dispatch: CTAs (one per SM) that only gather tokens, >= 1
 *              (Sec. 3.4 "Computation-Communication SM Tuning"); ignored for
 *              direct dispatch
 *   gemm_ctas  CTAs that run expert GEMMs; 0 = all remaining SMs
 *   lag        0: down projections of minibatch m follow its up/gate tiles;
 *              1: they follow the up/gate tiles of minibatch m + 1
 *   timeout_ms limit of every device-side wait (0 = 2000 ms)
 *   l2_prefetch  K steps ahead that the GEMM producers prefetch operand tiles
 *              into L2 (0 = off, the default: on DSV3 it measured slower)
 *   mma_pair   1: the GEMM CTAs run as pairs (clusters of 2) and each expert
 *              tile is one tcgen05.mma.cta_group::2 of 256 rows, the pair's
 *              two 128-row M-tiles sharing the weight tile, each CTA loading
 *              half of it (half the operand bytes per SM of the one-CTA tile);
 *              a segment with an odd number of M-tiles pads its last pair.
 *              With mxfp8 the scale blocks of both CTAs' rows travel with the
 *              pair's loads and every CTA holds the weight tile's scales for
 *              all 256 columns.  Ring or spread dispatch (direct gives
 *              MOE_ERR_INVALID_ARG); gather_ctas must be even.  Results are
 *              bitwise those of the one-CTA tiles.  0: one CTA per tile.
 *   clc        1: the GEMM CTAs take their work tokens from cluster launch
 *              control (MoK Sec. 3.4 "RDMA Overlap via Cluster Launch
 *              Control"): the kernel is launched with one CTA per task beyond
 *              the gather CTAs, not cooperatively; each running CTA cancels
 *              the launch of a CTA that has not started and takes its token,
 *              so when the hardware declines (a higher-priority stream wants
 *              the SM) the CTA finishes its unit and leaves, and CTAs launched
 *              later take the remaining units.  Which unit a token buys still
 *              comes from the global counter in task order, so results are
 *              bitwise those of the default scheduling.  One CTA per tile only
 *              (mma_pair = 1 gives MOE_ERR_INVALID_ARG).  0: the persistent
 *              cooperative grid claims units from the counter alone.
 *   test_unfilled_minibatch  test hook for the bounded waits, 0 in normal
 *              use: n >= 1 makes the ring fill never mark minibatch n - 1 as
 *              gathered, so the expert tiles waiting for it give up after
 *              timeout_ms and the forward ends with MOE_STATUS_TIMEOUT (the
 *              kernels return normally, the stream stays usable).  Ring or
 *              spread dispatch only (direct gives MOE_ERR_INVALID_ARG).
 *   pad_odd_tiles  CTA pairs: 1 pairs an expert segment's odd last M-tile with
 *              an empty partner (one M = 256 MMA, 128 of its rows zero); 0 =
 *              the default: with bf16 precision the tile is split over the
 *              pair instead (one M = 128 MMA, 64 rows per CTA: half the A
 *              bytes and half the tensor time of the padded form).  MXFP8
 *              pairs always pad.  Results are bitwise the same either way.
 *   plain_launch  profiling aid, 0 in normal use: 1 launches the persistent
 *              kernel without the cooperative attribute (profilers that replay
 *              kernels cannot launch a cooperative cluster kernel).  Its CTAs
 *              still wait on each other, so the grid (sized to what fits on
 *              the GPU at once) must all be resident, which it is when nothing
 *              else runs on the GPU; every wait is bounded, so a grid that
 *              did not fit ends the forward with MOE_STATUS_TIMEOUT.  Ignored
 *              with clc (never cooperative).
 *   raster     order of an expert segment's up/gate tiles: groups of `raster`
 *              M-tiles, each group sweeping all I/128 column tiles (so a
 *              group's token rows are re-read from L2 while its weight
 *              slices stream); 0 = the library default, >= the segment's
 *              M-tile count = column-tile major over the whole segment.  With
 *              mma_pair it is rounded up to even.  Results do not depend on it.
 * Zero for minibatch / ring_slots / gather_ctas / lag picks the defaults
 * (8192 / 4 / 8 / 1).
 */
typedef struct moe_config {
  int64_t T_max;
  int64_t D;
  int64_t I;
  int64_t E;
  int64_t k;
  int64_t I_s;
  int32_t score_fn;
  int32_t precision;
  int32_t minibatch;
  int32_t ring_slots;
  int32_t gather_ctas;
  int32_t gemm_ctas;
  int32_t lag;
  int32_t timeout_ms;
  int32_t dispatch;
  int32_t l2_prefetch;
  int32_t mma_pair;
  int32_t raster;
  int32_t test_unfilled_minibatch;
  int32_t clc;
  int32_t plain_launch;
  int32_t pad_odd_tiles;
} moe_config;

/*
 * Layer parameters (device pointers).
 *   W_router [E, D] bf16;  b_router [E] fp32 or NULL (no bias; the bias is
 *   added to the logits before the score function)
 *   bf16 precision:  W_up, W_gate [E, I, D] bf16;  W_down [E, D, I] bf16;
 *                    the *_scale pointers are ignored
 *   MXFP8 precision: W_up, W_gate [E, I, D] and W_down [E, D, I] E4M3 codes
 *                    (1 byte), and *_scale the E8M0 block scales written by
 *                    moe_quantize_mxfp8 for the same matrices
 *   Ws_up, Ws_gate [I_s, D] bf16; Ws_down [D, I_s] bf16; all three NULL = no
 *   shared expert in this call (required when I_s = 0)
 */
typedef struct moe_weights {
  const void* W_router;
  const float* b_router;
  const void* W_up;
  const void* W_gate;
  const void* W_down;
  const uint8_t* W_up_scale;
  const uint8_t* W_gate_scale;
  const uint8_t* W_down_scale;
  const void* Ws_up;
  const void* Ws_gate;
  const void* Ws_down;
} moe_weights;

/*
 * Outputs (device pointers).  `out` is required; every other field may be
 * NULL (not exported).
 *   out            [T, D] bf16: MoE(x)
 *   topk_idx       [T, k] int32: selected experts, ascending id per token
 *   topk_w         [T, k] fp32: g, same order
 *   expert_counts  [E] int32: M_e, routes per expert (Algorithm 1)
 *   expert_offsets [E + 1] int32: S_e, exclusive prefix of M (S_E = T*k)
 *   sched          [T*k, 3] int32: schedule table row P = {src_index t,
 *                  expert e, dst_index j = t*k + slot}, rows sorted by expert
 *                  then token (Algorithm 1 with one rank)
 *   route_row      [T*k] int32: inverse of sched, route j -> row P
 */
typedef struct moe_outputs {
  void* out;
  int32_t* topk_idx;
  float* topk_w;
  int32_t* expert_counts;
  int32_t* expert_offsets;
  int32_t* sched;
  int32_t* route_row;
} moe_outputs;

typedef struct moe_plan moe_plan;

/*
 * Validate `cfg` for the current CUDA device and create a plan.
 * Errors: MOE_ERR_INVALID_ARG (null), MOE_ERR_UNSUPPORTED_SHAPE,
 * MOE_ERR_UNSUPPORTED_DEVICE, MOE_ERR_CUDA.  *out is NULL on failure.
 * Host memory only; the caller releases it with moe_plan_destroy.
 */
int moe_plan_create(const moe_config* cfg, moe_plan** out);

/* Release a plan (NULL is accepted).  Returns MOE_OK. */
int moe_plan_destroy(moe_plan* plan);

/* Bytes of device workspace a forward of T tokens needs (0 on bad input).
 * The workspace holds the routing results, the schedule, the task list, the
 * dispatch ring, the gated activations and the token-order staging rows. */
size_t moe_workspace_bytes(const moe_plan* plan, int64_t T);

/*
 * MXFP8 weight pre-quantisation (Sec. 3.4 "MXFP8 Support", OCP MX v1.0):
 * W [rows, K] bf16 (device), rows and K multiples of 128 -> q [rows, K] E4M3
 * codes and scales (E8M0, one per 32 consecutive K elements),
 * moe_mxfp8_scale_bytes(rows, K) = rows * K / 32 bytes.  Block scale
 * X = 2^(floor(log2 amax) - 8), elements rounded to nearest-even and saturated
 * at +-448; an all-zero block gets X = 2^-127.  Scale layout: 512-byte blocks
 * ordered [rows/128][K/128], each holding 128 rows x 4 blocks of 32 with the
 * scale of (row r, block kb) at byte (r % 32) * 16 + ((r % 128) / 32) * 4 + kb
 * (the layout the block-scaled tensor-core MMA reads).  A stacked [E, I, D]
 * weight is quantised as rows = E * I.  Asynchronous on `stream`.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED_SHAPE, MOE_ERR_CUDA.
 */
int moe_quantize_mxfp8(const moe_plan* plan, const void* W, int64_t rows, int64_t K, uint8_t* q,
                       uint8_t* scales, moe_stream_t stream);
size_t moe_mxfp8_scale_bytes(int64_t rows, int64_t K);

/*
 * The forward pass for T tokens (0 <= T <= T_max; T = 0 does nothing).
 *   x          [T, D] bf16 (device)
 *   w          layer parameters, see moe_weights
 *   o          outputs, see moe_outputs
 *   workspace  device memory of at least moe_workspace_bytes(plan, T) bytes,
 *              256-byte aligned; its contents need no initialisation
 * Launches, in order on `stream`: router + top-k (for MXFP8 it also
 * quantises x per token), schedule, persistent forward kernel -- three
 * kernels, no host synchronisation.  Two calls on identical
 * inputs give bitwise-identical outputs, also across minibatch, ring_slots,
 * gather_ctas, gemm_ctas and lag settings.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA.
 */
int moe_fwd(const moe_plan* plan, int64_t T, const void* x, const moe_weights* w, const moe_outputs* o,
            void* workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * The forward pass with the routing given instead of made by the built-in
 * router (moe_route makes one):
 *   topk_idx [T, k] int32, topk_w [T, k] fp32 (device): expert and router
 *   weight g of every slot; an index of -1 is an empty slot.
 *   out = f_shared(x) + sum over the slots of g f_idx(x).
 * W_router and b_router are ignored (may be NULL).  Every token takes up k
 * routes: an empty slot runs the lowest expert that the token does not use,
 * with weight 0 (it shows as such in o->topk_idx, o->topk_w, the counts and
 * the schedule; what it makes reaches neither out nor the status).  For
 * moe_bwd_routed x must be finite in tokens without experts too.  An index
 * out of [-1, E), or a second slot of a token with the same expert, is run as
 * an empty slot and reported as MOE_STATUS_SCHEDULE_INVALID.
 * Otherwise as moe_fwd (bf16 and MXFP8 plans).
 */
int moe_fwd_routed(const moe_plan* plan, int64_t T, const void* x, const moe_weights* w, const int32_t* topk_idx,
                   const float* topk_w, const moe_outputs* o, void* workspace, size_t workspace_bytes,
                   moe_stream_t stream);

/*
 * Read the device status of the last forward that used `workspace` (a
 * moe_device_status: a failure if one was recorded, else
 * MOE_STATUS_STAGING_OVERFLOW if that warning was raised, else MOE_STATUS_OK).
 * This call waits for `stream` to finish: it is the one host synchronisation
 * point, taken only when the caller asks.
 */
int moe_get_status(const moe_plan* plan, const void* workspace, int* device_status, moe_stream_t stream);

/*
 * Optional per-launch timing for profiling harnesses: with events != NULL,
 * every later moe_fwd with this plan records events[0] (cudaEvent_t) on its
 * stream before the router launch, events[1] after it, events[2] after the
 * schedule launch and events[3] after the persistent kernel; events == NULL
 * turns it off.  The caller owns the events.  Not to be called while another
 * thread runs moe_fwd with the same plan.
 */
int moe_plan_set_timing_events(moe_plan* plan, void* const* events);

/*
 * Optional phase timing for profiling harnesses: the persistent kernel of the
 * last forward that used `workspace` stamps, with the GPU's global timer, when
 * its first CTA started, when the last minibatch was marked gathered (ring or
 * spread dispatch), and when the final combine pass began (the first CTA to
 * start it) and ended (the last CTA to finish it).  times_ms[0..2] receive the
 * last three as milliseconds after the start (-1 where a phase did not
 * happen).  Like moe_get_status, this call waits for `stream` to finish.
 */
int moe_get_phase_times(const moe_plan* plan, const void* workspace, double* times_ms, moe_stream_t stream);

/*
 * Routing stage without any device allocation -- no counterpart in the paper.
 *
 * For callers that cannot call cudaMalloc themselves and cannot hand over a
 * workspace: code embedded in a framework whose allocator owns all device
 * memory, or latency-critical loops where an allocation (which can
 * synchronise the device) is not allowed.  It runs the same router + top-k
 * and schedule kernels as moe_fwd, but their scratch (per-chunk expert
 * histograms, counters, status word, schedule-builder lists) lives in one
 * fixed array inside the library, moe_route_static_scratch_bytes() bytes
 * (512 KiB), that every GPU which loads the library keeps until the process
 * exits.  Limits: T <= MOE_ROUTE_STATIC_MAX_TOKENS (and <= the plan's T_max);
 * larger requests return MOE_ERR_STATIC_SCRATCH_TOO_SMALL and launch nothing.
 *   x [T, D] bf16, W_router [E, D] bf16, b_router [E] fp32 or NULL (device)
 *   outputs (device, all required): topk_idx [T, k] int32, topk_w [T, k] fp32,
 *   expert_counts [E], expert_offsets [E + 1], sched [T*k, 3], route_row [T*k]
 *   (int32, same meaning as in moe_outputs); device_status: optional device
 *   int32 that receives the call's moe_device_status.
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture.  All calls share the one array, which keeps the previous call's
 * contents (the kernels clear what must start at zero): calls that overlap on
 * the GPU -- on two streams, or from two threads -- race with each other.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_STATIC_SCRATCH_TOO_SMALL, MOE_ERR_CUDA.
 */
#define MOE_ROUTE_STATIC_MAX_TOKENS 16384
int moe_route_static(const moe_plan* plan, int64_t T, const void* x, const void* W_router, const float* b_router,
                     int32_t* topk_idx, float* topk_w, int32_t* expert_counts, int32_t* expert_offsets,
                     int32_t* sched, int32_t* route_row, int32_t* device_status, moe_stream_t stream);
size_t moe_route_static_scratch_bytes(void);

/*
 * Gradients of the layer (device pointers), written by moe_bwd.
 *   dx        [T, D] bf16: dL/dx (required)
 *   dW_router [E, D] fp32: dL/dW_r (required)
 *   db_router [E] fp32: dL/db, or NULL (not exported)
 *   dW_up, dW_gate [E, I, D] bf16; dW_down [E, D, I] bf16 (required)
 *   dWs_up, dWs_gate [I_s, D] bf16; dWs_down [D, I_s] bf16: the shared
 *   expert's, required when the forward had a shared expert, else NULL
 */
typedef struct moe_grads {
  void* dx;
  float* dW_router;
  float* db_router;
  void* dW_up;
  void* dW_gate;
  void* dW_down;
  void* dWs_up;
  void* dWs_gate;
  void* dWs_down;
} moe_grads;

/* Bytes of device workspace moe_bwd needs for T tokens (0 on bad input or a
 * shape the backward does not support: I and I_s must be multiples of 256). */
size_t moe_bwd_workspace_bytes(const moe_plan* plan, int64_t T);

/*
 * The backward pass ("Mixture-of-Kittens: MoE Megakernel for NVL72s",
 * Sec. 3.3 "Ring-Aware Forward Replay" and Sec. 3.4 "Router Weight Gradient
 * Computation"): given dO = dL/d out for the forward that moe_fwd computed on
 * the same x and weights with `fwd_workspace` (its routing and schedule are
 * reused, unmodified, from that workspace), writes every gradient of
 * moe_grads by the chain rule on Eq. MoE:
 *   dy_j = g_j dO;  dg_j = <W_down[e]^T dO, h>  (the SonicMoE form: the
 *   expert output is never materialised);  dh = g_j W_down[e]^T dO;
 *   da_u = dh * SiLU(a_g);  da_g = dh * a_u * SiLU'(a_g);
 *   dW_down[e] = sum dy h^T;  dW_up[e] = sum da_u x^T;  dW_gate[e] = sum da_g x^T;
 *   dx = sum_j (W_up[e]^T da_u + W_gate[e]^T da_g) + shared expert + W_r^T dl,
 *   with dl from g = s_sel / sum s_sel through the score function.
 * The gated activations are recomputed (the forward replay): every route's
 * up/gate projections run again from the gathered x rows.  BF16 routed
 * experts only (MOE_ERR_UNSUPPORTED_SHAPE for an MXFP8 plan).  No
 * floating-point atomics: every gradient element is produced by one tile with
 * a fixed K order or by a fixed-order sum, so two calls give the same bits.
 *   dO         [T, D] bf16 (device)
 *   workspace  at least moe_bwd_workspace_bytes(plan, T) bytes, 256-byte aligned
 * Launches eight kernels on `stream`; no host synchronisation; device-side
 * failures are reported through moe_get_status on `workspace`.  After a forward
 * whose routing was given (moe_fwd_routed) there is no router gradient: the
 * status is MOE_STATUS_SCHEDULE_INVALID, and dW_router, db_router and dx are NaN.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED_SHAPE,
 * MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA.
 */
int moe_bwd(const moe_plan* plan, int64_t T, const void* x, const moe_weights* w, const void* dO,
            const void* fwd_workspace, const moe_grads* grads, void* workspace, size_t workspace_bytes,
            moe_stream_t stream);

/*
 * The backward pass after moe_fwd_routed: every gradient of moe_grads but the
 * router's (dW_router and db_router are ignored, dx is without the router's
 * term), and instead
 *   dtopk_w [T, k] fp32 (device, required): dL/d topk_w; 0 in an empty slot
 * which moe_route_bwd takes on to the logits.  After a forward that routed by
 * itself (moe_fwd) the status is MOE_STATUS_SCHEDULE_INVALID and dtopk_w NaN.
 * Otherwise as moe_bwd; launches six kernels.
 */
int moe_bwd_routed(const moe_plan* plan, int64_t T, const void* x, const moe_weights* w, const void* dO,
                   const void* fwd_workspace, const moe_grads* grads, float* dtopk_w, void* workspace,
                   size_t workspace_bytes, moe_stream_t stream);

/*
 * Optional per-phase timing of moe_bwd for profiling harnesses: with events
 * != NULL, every later moe_bwd with this plan records events[0] before its
 * first launch, events[1] after the gather of the routes' x and dO rows,
 * events[2] after the replay + activation-gradient GEMMs, events[3] after the
 * input- and weight-gradient GEMMs and events[4] after its last launch;
 * NULL turns it off.  The caller owns the events (cudaEvent_t).
 */
int moe_plan_set_bwd_timing_events(moe_plan* plan, void* const* events);

/* ------------------------------------------------------------------ routing from given logits
 *
 * The general router: scores of given logits, an optional balance bias that
 * takes part in the selection only, expert groups, top-k, and weights that may
 * or may not be renormalised; with its gradient.  (moe_fwd's built-in router
 * multiplies x by W_router itself, adds its bias to the logits and always
 * renormalises; moe_fwd_routed runs the experts on the routing made here.)
 */
typedef enum moe_dtype { MOE_DTYPE_FP32 = 0, MOE_DTYPE_BF16 = 1, MOE_DTYPE_FP16 = 2 } moe_dtype;

/*
 *   E            experts, 1..512
 *   k            experts per token, 1..16, at most topk_group * E / n_group
 *   n_group      groups of E / n_group consecutive experts, 1..32, dividing E; 1 = no groups
 *   topk_group   groups kept per token, 1..n_group
 *   score_fn     moe_score_fn: s = sigmoid(x), or softmax over the E logits
 *   logits_dtype moe_dtype of the logits and of their gradient
 *   group_top    a group's score is the sum of its group_top (1 or 2) largest keys
 *   renormalize  1: w_i = scale s_i / (sum of the selected s); 0: w_i = scale s_i
 *   scale        factor of the weights, finite
 */
typedef struct moe_route_config {
  int64_t E;
  int64_t k;
  int64_t n_group;
  int64_t topk_group;
  int32_t score_fn;
  int32_t logits_dtype;
  int32_t group_top;
  int32_t renormalize;
  float scale;
} moe_route_config;

typedef struct moe_route_plan moe_route_plan;

/* Validate `cfg` for the current CUDA device and create a plan (host memory
 * only).  Errors as moe_plan_create. */
int moe_route_plan_create(const moe_route_config* cfg, moe_route_plan** out);
int moe_route_plan_destroy(moe_route_plan* plan);

/* Device workspace of moe_route for T tokens, needed only when expert_counts
 * or prob_sum is asked for (0 on bad input). */
size_t moe_route_workspace_bytes(const moe_route_plan* plan, int64_t T);

/*
 * Route T tokens (T = 0: only the sums are written, as zeros).
 *   logits        [T, E] of logits_dtype, rows logits_stride elements apart (0 = E)
 *   bias          [E] fp32 or NULL: the selection ranks s + bias (without it the
 *                 logits' own order); the weights do not see it
 *   topk_idx      [T, k] int32: the selected experts, ascending id; -1 in the
 *                 slots of a token with fewer than k experts to select
 *   topk_w        [T, k] fp32: the weights, same order, 0 in an empty slot
 *   expert_counts [E] int32 or NULL: routes per expert
 *   prob_sum      [E] fp32 or NULL: sum over the tokens of s_e / sum_f s_f, the
 *                 mean score that a load-balance loss is made of
 * An expert whose logit is -inf or NaN is never selected (a row of them has no
 * experts).  A NaN makes the row's softmax weights, and prob_sum, NaN.  Ties
 * go to the lower id, of groups to the lower group.  The selection is that of
 * keys and groups' scores computed in fp64 from the logits and biases: where
 * they lie closer than fp32 resolves they are, elsewhere fp32 gives the same.
 * So keys that fp64 does not tell apart are ties -- sigmoid scores of logits
 * above 37 (all 1), or scores added to a bias some 1e16 times their size -- also
 * with a bias of zeros, whereas without a bias the logits themselves decide.
 * No floating-point atomics: two calls give the same bits.
 * One launch, and a second one for the sums of more than 8 tokens.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA.
 */
int moe_route(const moe_route_plan* plan, int64_t T, const void* logits, int64_t logits_stride, const float* bias,
              int32_t* topk_idx, float* topk_w, int32_t* expert_counts, float* prob_sum, void* workspace,
              size_t workspace_bytes, moe_stream_t stream);

/*
 * The gradient of the logits, from dtopk_w = dL/d topk_w [T, k] fp32 and
 * dprob_sum = dL/d prob_sum [E] fp32 or NULL, for the selection topk_idx that
 * moe_route wrote (the selection itself has no gradient; a slot outside
 * [0, E) is empty).  dlogits [T, E] of logits_dtype, every element written.
 * dlogits must not overlap logits.  One launch, no workspace.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA.
 */
int moe_route_bwd(const moe_route_plan* plan, int64_t T, const void* logits, int64_t logits_stride,
                  const int32_t* topk_idx, const float* dtopk_w, const float* dprob_sum, void* dlogits,
                  int64_t dlogits_stride, moe_stream_t stream);

/* ------------------------------------------------------------------ momentum and orthogonalised updates
 *
 * The update of a stack of weight matrices as the Muon optimiser makes it from
 * moe_bwd's gradients:
 *   M = mu M + G;  U = G + mu M (nesterov) or M;  X = U / |U|_F;
 *   steps times:  A = X X^T,  X = a X + (b A + c A^2) X     (rows <= cols;
 *                 A = X^T X,  X = a X + X (b A + c A^2)      otherwise)
 *   update = scale X
 * Products run in fp16 operands with fp32 sums; see moe_muon_update.
 */
/*
 *   count, rows, cols  the stack [count, rows, cols]; count 1..65536, rows and cols
 *                      1..65536, rows * cols up to 2^30
 *   steps              Newton-Schulz steps, 1..32 (0 = 5)
 *   grad_dtype         moe_dtype of the gradient
 *   a, b, c            the step's coefficients, finite (all 0 = 3.4445, -4.7750, 2.0315).
 *                      Iterates, A and b A + c A^2 are held in fp16 and must stay
 *                      below 16: coefficients with which the singular values 0..1
 *                      of X can lead out of that (or within 1% a step of it) are
 *                      refused (MOE_ERR_INVALID_ARG)
 *   timeout_ms         limit of every device-side wait (0 = 2000 ms)
 */
typedef struct moe_muon_config {
  int64_t count;
  int64_t rows;
  int64_t cols;
  int32_t steps;
  int32_t grad_dtype;
  float a;
  float b;
  float c;
  int32_t timeout_ms;
} moe_muon_config;

typedef struct moe_muon_plan moe_muon_plan;

/* Validate `cfg` for the current CUDA device and create a plan (host memory
 * only).  Errors as moe_plan_create. */
int moe_muon_plan_create(const moe_muon_config* cfg, moe_muon_plan** out);
int moe_muon_plan_destroy(moe_muon_plan* plan);

/* Device workspace of moe_muon_update (0 on bad input). */
size_t moe_muon_workspace_bytes(const moe_muon_plan* plan);

/*
 * One update.
 *   grad      [count, rows, cols] of grad_dtype, rows grad_row_stride elements
 *             apart (0 = cols), matrices grad_stride apart (0 = rows * row stride)
 *   momentum  [count, rows, cols] fp32, updated in place; NULL = no momentum
 *             (U = G; mu and nesterov are ignored)
 *   update    [count, rows, cols] bf16
 *   workspace at least moe_muon_workspace_bytes(plan) bytes, 256-byte aligned,
 *             no initialisation needed
 * A matrix of zeros gives zeros; a matrix with an infinity or a NaN gives NaN,
 * without touching the others.  Two calls on the same inputs give the same
 * bits.  No host synchronisation; a device-side wait that ran out is reported by
 * moe_muon_get_status.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA.
 */
int moe_muon_update(const moe_muon_plan* plan, const void* grad, int64_t grad_row_stride, int64_t grad_stride,
                    float* momentum, float mu, int32_t nesterov, float scale, void* update, void* workspace,
                    size_t workspace_bytes, moe_stream_t stream);

/* The device status of the last update that used `workspace` (MOE_STATUS_OK or
 * MOE_STATUS_TIMEOUT); waits for `stream`, as moe_get_status does. */
int moe_muon_get_status(const moe_muon_plan* plan, const void* workspace, int* device_status, moe_stream_t stream);

/* ------------------------------------------------------------------ the layer for a few tokens
 *
 * moe_fwd's layer for T <= MOE_DECODE_MAX_TOKENS tokens (the decode steps of a
 * server), in one launch that streams the weights of the experts that have a
 * token, each once: the router, the selected experts, the shared expert and the
 * weighted sum.  The same plan and weights as moe_fwd (the ring, gather, pair and
 * raster settings do not matter here); for MXFP8 plans x and h are quantised as
 * there.  Products are summed in fp32 and h is held in bf16 (or MXFP8) as there,
 * but the experts' outputs stay fp32 (moe_fwd holds them in fp16), so
 * results agree with moe_fwd's up to roundings, not bit for bit.
 */
#define MOE_DECODE_MAX_TOKENS 64

/* Device workspace of moe_decode and moe_decode_routed for T tokens (0 on bad
 * input); what is enough for T is enough for fewer. */
size_t moe_decode_workspace_bytes(const moe_plan* plan, int64_t T);

/*
 *   x          [T, D] bf16 (device), 0 <= T <= min(T_max, MOE_DECODE_MAX_TOKENS); T = 0 does nothing
 *   out        [T, D] bf16
 *   topk_idx   [T, k] int32 or NULL: the selected experts, ascending id per token
 *   topk_w     [T, k] fp32 or NULL: their weights g
 *   workspace  at least moe_decode_workspace_bytes(plan, T) bytes, 256-byte
 *              aligned, no initialisation needed; not to be shared by calls that overlap
 * The selection is that of exact logits (with the bias; ties to the lower id):
 * where fp32 sums cannot tell the k-th logit from the next, fp64 sums decide.
 * (Logits or partial sums of 2^128 and more are infinities or NaN here.)  The weights
 * are those of logits off by 2^-6 at most, in truth a small part of it (10^-6 for unit
 * tokens): where parts cancel so far that fp32 sums may miss a selected one by more, fp64
 * sums take their place.
 * The launch is cooperative.  Two calls on the same inputs give the same bits; a
 * token's last bits may depend on which other tokens are in the call.  moe_get_status reads
 * the call's status from `workspace` (MOE_STATUS_TIMEOUT: a wait inside ran out).
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA.
 */
int moe_decode(const moe_plan* plan, int64_t T, const void* x, const moe_weights* w, void* out, int32_t* topk_idx,
               float* topk_w, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * The same on a routing that is given: topk_idx [T, k] int32, topk_w [T, k] fp32
 * (device) as moe_route writes them.  W_router and b_router are ignored.  An
 * empty slot (-1) costs nothing and its weight is not looked at; an index out of
 * [-1, E), or a second slot of a token with the same expert, is taken for an empty
 * slot and reported as MOE_STATUS_SCHEDULE_INVALID.  A token without experts gets the shared
 * expert's output, or zeros.
 */
int moe_decode_routed(const moe_plan* plan, int64_t T, const void* x, const moe_weights* w, const int32_t* topk_idx,
                      const float* topk_w, void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------ norms around a block
 *
 * What stands between two blocks of a decoder, in one pass over the rows:
 *   z = N(o; post_weight, post_bias)        norm of the block's output
 *   y = x_scale x + o_scale (gate * z)      gate and scaled residual
 *   h = N(y; pre_weight, pre_bias)          norm of the next block's input
 * with N(v) = (v - m) / sqrt(mean((v - m)^2) + eps) * (weight_offset + weight) + bias
 * over the D elements of a row, m = 0 (MOE_NORM_RMS) or the row's mean
 * (MOE_NORM_LAYER).  Either norm may be left out of the plan (z = o; no h), the
 * gate, the residual x or the block's output o out of a call.
 */
typedef enum moe_norm_kind { MOE_NORM_RMS = 0, MOE_NORM_LAYER = 1 } moe_norm_kind;

/*
 *   D             elements of a row, 1..16384
 *   kind          moe_norm_kind
 *   post, pre     1: with the norm of the block's output, of the next block's input
 *   stream_dtype  moe_dtype of the residual stream x, y and of dy, dx
 *   branch_dtype  moe_dtype of o, h, a gate per row, do and dh: the stream's, or
 *                 any beside an fp32 stream
 *   param_dtype   moe_dtype of the weights, biases and a gate per channel
 *   eps           > 0;  weight_offset, x_scale, o_scale  finite
 */
typedef struct moe_norm_config {
  int64_t D;
  int32_t kind;
  int32_t post;
  int32_t pre;
  int32_t stream_dtype;
  int32_t branch_dtype;
  int32_t param_dtype;
  float eps;
  float weight_offset;
  float x_scale;
  float o_scale;
} moe_norm_config;

typedef struct moe_norm_plan moe_norm_plan;

/*
 * Parameters (device pointers), each may be NULL.
 *   post_weight, pre_weight  [D]: NULL = ones (weight_offset is not added then)
 *   post_bias, pre_bias      [D]: layer norms only
 *   gate         [D] of param_dtype (gate_stride 0), or [T, D] of branch_dtype with
 *                rows gate_stride elements apart; NULL = 1
 */
typedef struct moe_norm_params {
  const void* post_weight;
  const void* post_bias;
  const void* pre_weight;
  const void* pre_bias;
  const void* gate;
  int64_t gate_stride;
} moe_norm_params;

/* Validate `cfg` for the current CUDA device and create a plan (host memory
 * only).  Errors as moe_plan_create. */
int moe_norm_plan_create(const moe_norm_config* cfg, moe_norm_plan** out);
int moe_norm_plan_destroy(moe_norm_plan* plan);

/*
 * The forward (T = 0 does nothing).  Rows [T, D] lie `_stride` elements apart (0 = D);
 * what is between D and the stride is not written and has no effect (a row that does
 * not start on 16 bytes may be fetched from that boundary on).
 *   x      the residual stream, or NULL: y = o_scale (gate * z)
 *   o      the block's output, or NULL: y = x_scale x (a plan without a post norm, no gate)
 *   y      the new residual stream, or NULL: not written (with a pre norm only).
 *          It may be x itself (the same pointer and stride)
 *   h      the next block's input, with a pre norm (else NULL).  It may be o itself
 *   stats  [T, 4] fp32 or NULL: m and 1 / sqrt(mean((v - m)^2) + eps) of o, then of y, for
 *          moe_norm_bwd; 0 where a norm is left out
 * h is the norm of y as it is written, so the fused call gives the bits of the
 * separate ones.  Sums are fp32; rows whose squares leave fp32's range come out
 * as zeros or NaN.  A row's result does not depend on the other rows.  One launch.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA.
 */
int moe_norm(const moe_norm_plan* plan, int64_t T, const moe_norm_params* params, const void* x, int64_t x_stride,
             const void* o, int64_t o_stride, void* y, int64_t y_stride, void* h, int64_t h_stride, float* stats,
             moe_stream_t stream);

/*
 * Gradients of the parameters, written by moe_norm_bwd (device pointers, each
 * may be NULL): fp32 [D], summed over the T rows; of a gate per row [T, D] of
 * branch_dtype, rows gate_stride elements apart (0 = D).
 */
typedef struct moe_norm_grads {
  float* post_weight;
  float* post_bias;
  float* pre_weight;
  float* pre_bias;
  void* gate;
  int64_t gate_stride;
} moe_norm_grads;

/* Device workspace of moe_norm_bwd for T rows (0 on bad input). */
size_t moe_norm_workspace_bytes(const moe_norm_plan* plan, int64_t T);

/*
 * The gradients, from dy = dL/dy (the part that reaches y past the pre norm) and
 * dh = dL/dh, for a forward on the same o and parameters that wrote y and stats.
 *   o    needed with a post norm or for the gate's gradient;  y, dh  with a pre norm
 *   dy   or NULL: 0 (with a pre norm only)
 *   dx   or NULL: not written; it may be dy itself
 *   d_o  or NULL: not written; it may be dh itself
 *   workspace  at least moe_norm_workspace_bytes(plan, T) bytes, 256-byte aligned,
 *              no initialisation needed; not to be shared by calls that overlap
 * With T = 0 the summed gradients are zeros.  No floating-point atomics: two
 * calls give the same bits.  One launch, and a second one for the sums.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA.
 */
int moe_norm_bwd(const moe_norm_plan* plan, int64_t T, const moe_norm_params* params, const float* stats, const void* o,
                 int64_t o_stride, const void* y, int64_t y_stride, const void* dy, int64_t dy_stride, const void* dh,
                 int64_t dh_stride, void* dx, int64_t dx_stride, void* d_o, int64_t d_o_stride,
                 const moe_norm_grads* grads, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* Static description of an error code. */
const char* moe_error_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
