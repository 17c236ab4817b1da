/*
 * rf.h — C ABI of librf.so: the RidgeFill upper-layer KV fill, its calibration
 * statistics and closed-form ridge solve, the cross-model per-head ridge
 * mapper, and the operators that decode from a filled cache (norms and rotation of
 * queries and keys, attention of drafted trees over one sequence's cache or a shared
 * prefix, sampling, verification, eviction), for one NVIDIA GB300 (sm_103a).
 *
 * Sources cited below:
 *   [RF] RidgeFill review (jaehun.me, English edition of the review of arXiv
 *        2611.09709): "Two numbers set the skip range", "Ridge map: predict the
 *        input, and the original projection runs unchanged", Table 3.
 *   [XM] "Cross-Model KV Cache Transfer in LLM Families: A Closed-Form Linear
 *        Mapping for Prefill Reuse" (digest): per-head ridge regression,
 *        cross-layer source selection, content-space mapping equation.
 *
 * Conventions shared by every call
 *   - Tensor arguments are DEVICE pointers owned by the caller, unless a comment
 *     says "host". bf16 values are passed as their 16-bit patterns (rf_bf16).
 *   - Every call is asynchronous on the caller's stream (a cudaStream_t passed
 *     as rf_stream_t; NULL is the legacy default stream). No call synchronises
 *     the host unless its comment says so.
 *   - The library allocates no device memory. Calls that need scratch memory
 *     take a caller workspace of at least rf_*_workspace_bytes(...) bytes,
 *     256-byte aligned; its contents are undefined after the call. Calls that
 *     share one workspace must be ordered on one stream.
 *   - Argument errors are detected on the host before any launch and return a
 *     status other than RF_OK; nothing is written then. rf_last_error() gives a
 *     thread-local text for the last failing call on the calling thread.
 *   - Errors found on the device (a bounded wait that gave up, a non-positive
 *     Cholesky pivot) are written to the optional device int32 *dev_status
 *     (first error wins; the caller zeroes it). A kernel that gives up returns
 *     without touching the outputs it had not written yet.
 *   - Functions are thread-safe; no call aborts the process or throws.
 *   - Rows of every matrix are contiguous; "ld" arguments are row strides in
 *     elements. Pointers must be 16-byte aligned and row/layer strides multiples
 *     of 8 elements, else RF_ERR_ALIGN.
 */
#ifndef RIDGE_MAP_KV_RF_H
#define RIDGE_MAP_KV_RF_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rf_status {
  RF_OK = 0,
  RF_ERR_INVALID_ARG = 1,  /* null pointer, negative size, unknown mode        */
  RF_ERR_SHAPE = 2,        /* sizes the kernels do not support                */
  RF_ERR_ALIGN = 3,        /* pointer or stride alignment                      */
  RF_ERR_CUDA = 4,         /* CUDA runtime error; text in rf_last_error()      */
  RF_ERR_NOT_SPD = 5,      /* device status: Cholesky pivot <= 0               */
  RF_ERR_TIMEOUT = 6,      /* device status: a bounded device wait gave up      */
  RF_ERR_UNSUPPORTED = 7,  /* current device is not sm_100-family (tcgen05)    */
  RF_ERR_WORKSPACE = 8     /* workspace missing, too small or misaligned       */
} rf_status;

typedef uint16_t rf_bf16;   /* bfloat16 bit pattern                             */
typedef void* rf_stream_t;  /* cudaStream_t                                     */

/* Library version (major*10000 + minor*100 + patch). */
int rf_version(void);
/* Static text for a status code (never NULL). */
const char* rf_status_string(int status);
/* Thread-local text describing the last failing call on this thread ("" if none). */
const char* rf_last_error(void);
/* 1 if `device` has tcgen05 tensor cores (compute capability 10.x), else 0. */
int rf_device_supported(int device);
/* Bounded device waits give up after this many milliseconds (default 4000). Host
 * setting, read at each launch; values < 1 restore the default. */
void rf_set_wait_timeout_ms(int64_t ms);

/* Optional per-kernel timing. Between rf_profile_start and rf_profile_stop every
 * kernel the library launches (on any thread) is bracketed by two CUDA events
 * recorded on its launching stream, up to `max_records` kernels; later launches
 * are not recorded. rf_profile_stop waits for the recorded events, writes up to
 * `capacity` (stage id, milliseconds) pairs in launch order (host arrays) and
 * returns how many it wrote (-1 on a CUDA error). Recording adds two event
 * records per launch and no synchronisation. */
enum rf_stage {
  RF_STAGE_COMPACT = 1,      /* exact-row mask -> fill_idx                    */
  RF_STAGE_GATHER = 2,       /* x_S rows -> dense operand                      */
  RF_STAGE_ROPE_TABLE = 3,   /* (unused: RoPE angles are computed in the kernels) */
  RF_STAGE_MAP_GEMM = 4,     /* x̂ = x_S A_lᵀ + b_l, all upper layers           */
  RF_STAGE_KV_GEMM = 5,      /* K/V projection + norm scale + RoPE + scatter   */
  RF_STAGE_FOLD = 6,         /* gain fold into W_k / W_v                       */
  RF_STAGE_CALIB_GEMM = 7,   /* XᵀX and XᵀY_l                                  */
  RF_STAGE_COLSUM = 8,       /* Σx, Σy, n                                      */
  RF_STAGE_SOLVE = 9,        /* ridge solve: centring, Cholesky, H^-1          */
  RF_STAGE_UNROPE = 10,      /* RoPE / inverse RoPE on cache rows              */
  RF_STAGE_XMODEL_GEMM = 11, /* cross-model mapper GEMM                        */
  RF_STAGE_RESCALE = 12,     /* value rescale: value norms and their ratios   */
  RF_STAGE_EXPAND = 13,      /* int8 map codes -> bf16 before a layer's GEMM   */
  RF_STAGE_QUANTIZE = 14,    /* bf16 maps -> int8 codes and row scales         */
  RF_STAGE_SOLVE_PRODUCT = 15, /* solve: A_p = Cc_pᵀ H^-1 (split tensor-core GEMM) */
  RF_STAGE_SOLVE_REFINE = 16,  /* solve: fp64 residual and correction, per sweep */
  RF_STAGE_ROW_RMS = 17,       /* fill: per-row RMS scale from the map GEMM's sums */
  RF_STAGE_SELECT_GEMM = 18,   /* source selection: split tensor-core products    */
  RF_STAGE_SELECT_FACTOR = 19, /* source selection: batched Cholesky and inverse  */
  RF_STAGE_SELECT_SCORE = 20,  /* source selection: set-up, scores, argmax, copies */
  RF_STAGE_SELECT_SPLIT = 21,  /* source selection: fp32 -> three bf16 planes      */
  RF_STAGE_ROPE = 22,          /* rf_rope                                          */
  RF_STAGE_TREE_BUILD = 23,    /* rf_tree_build                                    */
  RF_STAGE_ATTENTION = 24,     /* rf_tree_attention, rf_prefix_attention: the attention kernel */
  RF_STAGE_ATTN_COMBINE = 25,  /* the same: joining of split sequences, or of a prefix's and others' parts */
  RF_STAGE_VERIFY = 26,        /* rf_verify_draft                                  */
  RF_STAGE_COMMIT = 27,        /* rf_commit_draft                                  */
  RF_STAGE_ATTN_WEIGHTS = 28,  /* rf_attn_weights                                  */
  RF_STAGE_EVICT_SELECT = 29,  /* rf_evict: which rows stay                        */
  RF_STAGE_EVICT_MOVE = 30,    /* rf_evict: rows into the holes                    */
  RF_STAGE_NORM_ROPE = 31,     /* rf_norm_rope, rf_norm_rope_backward              */
  RF_STAGE_SAMPLE = 32         /* rf_sample                                        */
};
rf_status rf_profile_start(int max_records);
/* Diagnostic: runs the tensor-core GEMM kernel on a problem whose operand copies
 * are never issued, so its MMA thread's bounded wait runs out after the wait limit
 * (rf_set_wait_timeout_ms). The kernel then drains, frees its TMEM and writes
 * RF_ERR_TIMEOUT to *dev_status (device int32, must be 0 before the call). It
 * tests the library's failure path without faulting the GPU: nothing is ever in
 * flight, and the context stays usable.
 *   mode  bit 0: the CTA-pair kernel (else the single-CTA one); bit 1: the dynamic
 *         unit order (units posted through the shared-memory ring, from a counter
 *         inside the library's device code), else round-robin. */
rf_status rf_selftest_wait_timeout(int mode, int32_t* dev_status, rf_stream_t stream);
int rf_profile_stop(int32_t* stage_ids, float* ms, int capacity);
const char* rf_stage_name(int stage_id);

/* ===================================================================== *
 * Fill  ([RF] "Two numbers set the skip range"; "Ridge map", first equation
 * x̂_l = A_l x_S + b_l; the layer's own norm and K/V projections and RoPE)
 * ===================================================================== */
typedef struct rf_fill_desc {
  int64_t d;           /* hidden size: map output width, projection input; also the */
                       /* map input width unless d_in is set                        */
  int64_t L;           /* number of layers                                          */
  int64_t S;           /* split layer: maps exist for layers S .. L-1 (P = L - S)    */
  int64_t N;           /* prompt rows                                               */
  int64_t T;           /* tail rows: rows N-T .. N-1 are never filled (0 <= T <= N)  */
  int64_t n_kv_heads;  /* H                                                         */
  int64_t head_dim;    /* hd; KV = H*hd                                              */
  double rope_theta;   /* RoPE base (rotate-half pairs (i, i+hd/2), θ^(-2i/hd))      */
  double rms_eps;      /* RMSNorm ε: y = g ⊙ x / sqrt(mean(x²) + ε)                   */
  int64_t pos_offset;  /* RoPE position of row 0                                     */
  uint64_t flags;      /* RF_FLAG_* (0 = defaults)                                   */
  const float* v_scale;/* [P][H] device fp32 or NULL: the value rescale. Filled V of  */
                       /* layer S+p, head h is multiplied by v_scale[p*H + h] before */
                       /* rounding (see rf_value_scale). NULL = no rescale.         */
  const rf_bf16* k_norm_gain; /* [P][hd] device bf16 or NULL: key normalisation.      */
                       /* Each key head becomes g_p * k_h / sqrt(mean(k_h²) + ε)      */
                       /* (ε = rms_eps) before RoPE ("Qwen models normalize keys").  */
  int64_t d_in;        /* width of x_S rows and of the maps' input; 0 = d (square).  */
                       /* Non-square maps A_p [d][d_in] read a wider split state,    */
                       /* e.g. parallel residual streams ([RF] "Ridge map": 10,240 */
                       /* -> 2,560 for Flash-Next). Must be a multiple of 256.       */
} rf_fill_desc;

/* Flags of rf_fill_desc, rf_calib_desc and rf_xmodel_desc: which tensor-core GEMM
 * kernel runs. RF_FLAG_SINGLE_CTA: one CTA per 128 x 256 output tile
 * (cta_group::1). RF_FLAG_CTA_PAIR: a CTA pair per 256 x 256 tile (cta_group::2,
 * each CTA holding half of B). With neither bit set every operation runs on
 * CTA pairs, the measured-faster kernel. Results agree up to the order of fp32
 * additions. */
#define RF_FLAG_SINGLE_CTA 1u
#define RF_FLAG_CTA_PAIR 2u
/* Flag of rf_fill_desc: the K and V projections passed to the fill already hold
 * the RMSNorm gain, Wk[p][j][i] = W_k,p[j][i] g_p[i] (likewise Wv), for example
 * from rf_fold_kv_weights; `gain` is then ignored and may be NULL. Without it the
 * fill folds the gain into its workspace on every call. */
#define RF_WEIGHTS_PREFOLDED 4u
/* Flag of rf_calib_desc for rf_solve: the refinement's residual cuts its operands
 * into 7-bit digits at every width. By default it takes 8-bit digits up to
 * d_in = 21845 and 7-bit ones above, where the int32 sums of 8-bit digit products
 * could overflow; the flag runs the wider widths' arithmetic at any size (the
 * result meets the same accuracy, with more digit products). */
#define RF_SOLVE_DIGITS7 8u

/* Supported fill shapes: d % 256 == 0, head_dim in {64, 128}, KV % 128 == 0,
 * N - T <= 2^24. */

/* Workspace bytes rf_fill_kv needs for `desc` (0 on invalid desc). Without
 * RF_WEIGHTS_PREFOLDED in desc->flags this includes 2*P*KV*d bf16 for the folded
 * projections. */
size_t rf_fill_workspace_bytes(const rf_fill_desc* desc);

/* Weight preparation for the fill (run once per weight set, then pass the results
 * with RF_WEIGHTS_PREFOLDED): folds each layer's RMSNorm gain into its K and V
 * projections,
 *   Wk_folded[p][j][i] = bf16(Wk[p][j][i] * gain[p][i]),
 *   Wv_folded[p][j][i] = bf16(Wv[p][j][i] * gain[p][i]),
 * gain [P][d], Wk, Wv, Wk_folded, Wv_folded [P][KV][d] (row = output channel),
 * all device. The bf16 x bf16 product is exact in fp32, so the only rounding is
 * the last one. In place (Wk_folded == Wk, Wv_folded == Wv) is allowed. */
rf_status rf_fold_kv_weights(const rf_fill_desc* desc, const rf_bf16* gain,
                             const rf_bf16* Wk, const rf_bf16* Wv,
                             rf_bf16* Wk_folded, rf_bf16* Wv_folded, rf_stream_t stream);

/* The fill. For every filled row t (t < N-T, exact_mask[t] == 0, ascending) and
 * every layer l = S + p:
 *   x̂ = A_p x_S[t] + b_p;  r = (mean(x̂²) + ε)^-1/2;
 *   k = r · (Wk_p ⊙ g_p) x̂,  v = r · (Wv_p ⊙ g_p) x̂   (g_p scales the input channels);
 *   k_h <- g_k,p ⊙ k_h / sqrt(mean(k_h²) + ε)   when desc->k_norm_gain is set;
 *   v_h <- v_scale[p][h] · v_h                  when desc->v_scale is set;
 *   k_h <- RoPE(k_h, t + pos_offset) per head;
 *   k_cache[l][t][h][:] = bf16(k_h),  v_cache[l][t][h][:] = bf16(v_h).
 * Nothing else in the caches is written: not the tail, not exact rows, not
 * layers < S ([RF] Table 3). x̂ is rounded to bf16 before the projection.
 *   x_S        [N][ld_x] bf16 rows of width d_in (d if d_in = 0), the state entering layer S
 *   exact_mask [N-T] uint8, nonzero = exact row (never filled); NULL = none
 *   A          [P][d][d_in] bf16, A_p[o][i] (row = output)
 *   b          [P][d] fp32
 *   gain       [P][d] bf16, the layers' RMSNorm gains (ignored with RF_WEIGHTS_PREFOLDED)
 *   Wk, Wv     [P][KV][d] bf16, the layers' K and V projections (row = output
 *              channel); with RF_WEIGHTS_PREFOLDED they already include the gain
 *              (rf_fold_kv_weights), else the call folds it into its workspace
 *   k_cache, v_cache: element (l, t, h, c) at l*layer_stride + t*row_stride + h*hd + c
 *   n_fill_out device int32 (may be NULL): number of filled rows
 * Kernels: the gain fold (unless prefolded), row compaction + gather, one tcgen05
 * GEMM for all maps (bias, bf16 x̂ and per-row sum-of-squares in its epilogue), one
 * tcgen05 GEMM for all K/V projections (RMS scale, RoPE and cache scatter in its
 * epilogue). */
rf_status rf_fill_kv(const rf_fill_desc* desc,
                     const rf_bf16* x_S, int64_t ld_x,
                     const uint8_t* exact_mask,
                     const rf_bf16* A, const float* b,
                     const rf_bf16* gain, const rf_bf16* Wk, const rf_bf16* Wv,
                     rf_bf16* k_cache, rf_bf16* v_cache,
                     int64_t layer_stride, int64_t row_stride,
                     int32_t* n_fill_out, int32_t* dev_status,
                     void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* Fill for callers that cannot allocate device memory (the pages have no
 * counterpart; this is a library convenience). Some callers have no way to get
 * scratch memory on the GPU: a plugin inside a serving engine whose device memory
 * all belongs to the engine's own pool, or a latency-critical path where a
 * cudaMalloc would synchronise the device. This call computes exactly what
 * rf_fill_kv computes, with the same arguments minus the workspace: its scratch
 * (including the gain fold, unless the weights are prefolded) is a fixed 256-byte
 * aligned array of RF_STATIC_SCRATCH_BYTES inside the
 * library's device code, which every GPU that loads the library keeps until the
 * process exits. It makes no allocating call.
 *   - Fills whose rf_fill_workspace_bytes(desc) exceeds RF_STATIC_SCRATCH_BYTES
 *     are rejected with RF_ERR_WORKSPACE before anything runs.
 *   - Every call looks up the array's device address in the current context (a
 *     host call; the first one in a context may load the library's device code
 *     there), so a cudaDeviceReset or another context never sees a stale address.
 *     Make the first call in each context before any stream capture.
 *   - All calls on a device share the array, which keeps the previous call's
 *     contents; nothing in it needs clearing between calls. Calls that overlap
 *     on the GPU race on it: order them on one stream. */
#define RF_STATIC_SCRATCH_BYTES (64u * 1024u * 1024u)
rf_status rf_fill_kv_static(const rf_fill_desc* desc,
                            const rf_bf16* x_S, int64_t ld_x,
                            const uint8_t* exact_mask,
                            const rf_bf16* A, const float* b,
                            const rf_bf16* gain, const rf_bf16* Wk, const rf_bf16* Wv,
                            rf_bf16* k_cache, rf_bf16* v_cache,
                            int64_t layer_stride, int64_t row_stride,
                            int32_t* n_fill_out, int32_t* dev_status, rf_stream_t stream);

/* Value rescale ([RF] "Hybrid layers and two corrections", value rescale; the
 * 27B deployment uses it with c = 512, "Two numbers set the skip range"). For
 * each upper layer l = S + p and KV head h:
 *   v_scale[p*H + h] = mean over t in [0, c) of ||v_exact_h(t)|| / ||v_pred_h(t)||
 *   v_pred(t)  = r(x̂) · Wv'_p x̂,  x̂ = bf16(A_p x_S[N-T+t] + b_p)   (as in the fill)
 *   v_exact(t) = r(x)  · Wv'_p x,  x  = x_exact[p][t]
 * where Wv'_p = bf16(Wv_p ⊙ g_p) is the gain-folded V projection (Wv as given with
 * RF_WEIGHTS_PREFOLDED in desc->flags, else folded into the workspace from `gain`
 * and `Wv`, both [P][KV][d] / [P][d] bf16), r(x) = (mean(x²) + ε)^-1/2 and
 * ||.|| is the L2 norm of the head's hd values. Rows whose predicted norm is 0 are
 * left out of a head's mean (scale 1 if none is left). The result is meant for
 * rf_fill_desc.v_scale.
 *   c         number of tail rows used, 1 <= c <= T (rows N-T .. N-T+c-1)
 *   x_S, ld_x as for rf_fill_kv (only rows N-T .. N-T+c-1 are read)
 *   x_exact   [P][c][ld_e] bf16 (device): the exact inputs of layers S .. L-1
 *             at those rows (the tail runs every layer exactly)
 *   A, b, gain, Wv as for rf_fill_kv;  v_scale  [P][H] fp32 (device), written
 * Requires d % 256 == 0, head_dim 64 or 128, KV % 128 == 0, S < L. Kernels: the
 * fill's map GEMM on the c tail rows, one tcgen05 GEMM for the V projections of
 * the predicted and the exact rows with per-head norms in its epilogue, and a
 * small reduction. The workspace is rf_value_scale_workspace_bytes(desc, c). */
size_t rf_value_scale_workspace_bytes(const rf_fill_desc* desc, int64_t c);
rf_status rf_value_scale(const rf_fill_desc* desc, int64_t c,
                         const rf_bf16* x_S, int64_t ld_x,
                         const rf_bf16* x_exact, int64_t ld_e,
                         const rf_bf16* A, const float* b,
                         const rf_bf16* gain, const rf_bf16* Wv,
                         float* v_scale, int32_t* dev_status,
                         void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* ===================================================================== *
 * Map storage ([RF] "Ridge map": the 27B maps "in int8 total 1.2 GiB"; "maps can
 * be kept resident in GPU memory or streamed from host memory one layer at a time")
 * ===================================================================== */
/* int8 code of the maps, symmetric per output row (the pages give no scheme):
 *   s[p][o] = max_i |A[p][o][i]| / 127,  q[p][o][i] = rint(A[p][o][i] / s[p][o])
 * (ties to even; both in fp32; a zero row gives s = 0 and q = 0), so that
 * A[p][o][i] ≈ s[p][o] q[p][o][i]. A [P][d][d_in] bf16, q [P][d][d_in] int8,
 * s [P][d] fp32, all device. */
rf_status rf_quantize_maps_int8(const rf_fill_desc* desc, const rf_bf16* A, int8_t* q, float* s,
                                rf_stream_t stream);

#define RF_MAPS_BF16 0 /* A is [P][d][d_in] bf16                                   */
#define RF_MAPS_INT8 1 /* A is q [P][d][d_in] int8 with row_scale s [P][d] fp32    */
typedef struct rf_map_source {
  int32_t kind;           /* RF_MAPS_BF16 or RF_MAPS_INT8                               */
  int32_t on_host;        /* nonzero: A is in host memory. Page-locked memory lets the */
                          /* copy of layer p+1 overlap the GEMMs of layer p; pageable  */
                          /* memory works but its copies may block the calling thread. */
  const void* A;          /* the maps, layer after layer (p = 0 .. P-1)                 */
  const float* row_scale; /* RF_MAPS_INT8: [P][d] fp32 on the device; else unused       */
} rf_map_source;

/* The fill of rf_fill_kv, a few layers at a time: for each step of up to 4
 * layers the map GEMM of those layers and then their K/V GEMM, so x̂ exists for
 * 4 layers only (workspace 4*M_pad*d instead of P*M_pad*d bf16). Maps on the host
 * or in int8 pass through a two-slot bf16 ring in the workspace: the library's
 * copy stream copies the next step's maps (and expands int8 codes to bf16, exact
 * for |q| <= 127) while the caller's stream computes the current step; int8 row
 * scales are applied to the map GEMM's output
 * columns with the bias. Device bf16 maps are read in place. The results equal
 * rf_fill_kv's bit for bit when the maps are the same bf16 values (same kernels,
 * same summation order). Arguments as for rf_fill_kv, with `maps` replacing A
 * (gain, Wk, Wv and RF_WEIGHTS_PREFOLDED as there); the workspace is
 * rf_fill_layered_workspace_bytes(desc, maps). Everything is asynchronous on
 * `stream`. */
size_t rf_fill_layered_workspace_bytes(const rf_fill_desc* desc, const rf_map_source* maps);
rf_status rf_fill_kv_layered(const rf_fill_desc* desc,
                             const rf_bf16* x_S, int64_t ld_x,
                             const uint8_t* exact_mask,
                             const rf_map_source* maps, const float* b,
                             const rf_bf16* gain, const rf_bf16* Wk, const rf_bf16* Wv,
                             rf_bf16* k_cache, rf_bf16* v_cache,
                             int64_t layer_stride, int64_t row_stride,
                             int32_t* n_fill_out, int32_t* dev_status,
                             void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* ===================================================================== *
 * Calibration statistics ([RF] "Ridge map": only XᵀX, XᵀY_l and the two means
 * are accumulated in one pass; [XM]: XᵀX is the dominant fitting cost)
 * ===================================================================== */
typedef struct rf_calib_desc {
  int64_t d_in;    /* width of x (map input)        */
  int64_t d_out;   /* width of each y_p (map output) */
  int64_t n_maps;  /* P                              */
  uint64_t flags;  /* RF_FLAG_* (0 = defaults)       */
} rf_calib_desc;

/* Raw one-pass sums, all device fp64 (n as int64), caller-owned.
 *   G   [d_in][d_in]          Σ x xᵀ   (both triangles)
 *   C   [n_maps][d_in][d_out] Σ x y_pᵀ
 *   sx  [d_in]                Σ x
 *   sy  [n_maps][d_out]       Σ y_p
 *   n   [1]                   rows seen
 *   syy [n_maps][d_out]       Σ y_p² per column (optional, NULL = not kept; the
 *                             total sums of squares that rf_select_sources needs)
 * Zero them to start; saved and reloaded sums resume accumulation. */
typedef struct rf_calib_stats {
  double* G;
  double* C;
  double* sx;
  double* sy;
  int64_t* n;
  double* syy;
} rf_calib_stats;

/* Supported: d_in % 128 == 0, d_out % 256 == 0 (or n_maps == 0), n_rows % 8 == 0.
 * The workspace is optional (see rf_calib_accumulate); this is its size (256). */
size_t rf_calib_workspace_bytes(const rf_calib_desc* desc, int64_t n_rows);

/* Adds one batch of rows: G += XᵀX, C_p += XᵀY_p, sx += Σx, sy_p += Σy_p, n += n_rows
 * (and syy_p += Σy_p² when stats->syy is set).
 *   X [n_rows][ld_x] bf16; Y_p at Y + p*y_map_stride, [n_rows][ld_y] bf16.
 * Products are exact in fp32, summed in fp32 over chunks of rows on the tensor
 * cores and added to the fp64 totals.
 *   workspace  NULL, or rf_calib_workspace_bytes(...) bytes, 256-byte aligned: with
 *              it the GEMM takes its output tiles in dynamic order (a device
 *              counter), which keeps the CTAs that share operand rows together in
 *              L2; without it, in a fixed round-robin order. The sums are the same
 *              bit for bit either way (each tile is added to the totals once per
 *              16 chunks of rows, in stream order). */
rf_status rf_calib_accumulate(const rf_calib_desc* desc,
                              const rf_bf16* X, int64_t ld_x,
                              const rf_bf16* Y, int64_t ld_y, int64_t y_map_stride,
                              int64_t n_rows, const rf_calib_stats* stats,
                              int32_t* dev_status,
                              void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* ===================================================================== *
 * Ridge solve ([RF] "Ridge map": A_l = Y_lᵀX (XᵀX + αI)^-1, b_l = μ_l − A_l μ_S,
 * α = λ·tr(XᵀX)/d_in on centred X; a new λ only needs a re-solve)
 * ===================================================================== */
enum { RF_ALPHA_TRACE = 0, RF_ALPHA_ABSOLUTE = 1 };

size_t rf_solve_workspace_bytes(const rf_calib_desc* desc);

/* Solves every map from the statistics (read only, so re-solving at another λ
 * is legal):
 *   Gc = G − n μ_x μ_xᵀ, Cc_p = C_p − n μ_x μ_pᵀ, α = λ tr(Gc)/d_in (TRACE) or λ,
 *   Gc + αI = L Lᵀ (fp32 Cholesky), A_p = Cc_pᵀ (Gc + αI)^-1 (fp32), then
 *   `refine_iters` sweeps of A_p += (Cc_pᵀ − A_p (Gc + αI)) (Gc + αI)^-1 with the
 *   residual computed beyond fp32 accuracy (exact integer digit products on the
 *   tensor cores); b_p = μ_p − A_p μ_x (compensated, to about 2^-44 of Σ|A||μ|,
 *   rounded to fp32). How accurate the residual and the correction are is chosen on
 *   the device from κ(Gc + αI), estimated once by power iteration (24 steps, whose
 *   estimate is taken twice over): accurate enough for a sweep to bring A to fp32
 *   accuracy, the residual to at least 2^-(25 + log2 2κ) of Σ|A||Gc + αI| (with
 *   8-bit digits 2^-31.7 for κ up to about 51, 2^-39.4 up to about 10,800, else
 *   2^-47.2, its limit; with 7-bit digits, above d_in = 21845 or under
 *   RF_SOLVE_DIGITS7, 2^-27.7 up to about 3, 2^-34.4 up to about 330, else 2^-41.2),
 *   the correction to fp32 when 4κ > 2^10, else to about 2^-16 of its terms.
 *   A [n_maps][d_out][d_in] fp32, b [n_maps][d_out] fp32,
 *   A_bf16 (may be NULL) bf16 copy of A for rf_fill_kv, alpha_out (device, may be NULL).
 * A non-positive pivot sets RF_ERR_NOT_SPD in *dev_status. */
rf_status rf_solve(const rf_calib_desc* desc, const rf_calib_stats* stats,
                   double lambda, int alpha_mode, int refine_iters,
                   float* A, float* b, rf_bf16* A_bf16, double* alpha_out,
                   int32_t* dev_status,
                   void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* ===================================================================== *
 * Cross-model mapper ([XM] content-space mapping
 *   K̂_t = (K_s R_s^-1(t) W_K + b_K) R_t(t), V mapped without RoPE;
 * the k source layers chosen for a target layer are concatenated, all heads)
 * ===================================================================== */
typedef struct rf_xmodel_desc {
  int64_t L_src;       /* source layers                                  */
  int64_t L_tgt;       /* target layers                                  */
  int64_t k;           /* source layers concatenated per target layer     */
  int64_t n_kv_heads;  /* H (same on both sides: KV-matched pair)         */
  int64_t head_dim;    /* hd                                             */
  int64_t N;           /* rows (tokens)                                  */
  double theta_src;    /* source RoPE base                                */
  double theta_tgt;    /* target RoPE base                                */
  int64_t pos_offset;  /* position of row 0                               */
  uint64_t flags;      /* RF_FLAG_* (0 = defaults)                        */
} rf_xmodel_desc;

/* Supported: head_dim in {64, 128}, KV % 256 == 0, N >= 1. */
size_t rf_xmodel_workspace_bytes(const rf_xmodel_desc* desc);

/* For every target layer l and row t:
 *   F_K = [RoPE_src^-1(k_src[s_j][t]) for j < k] (feature order: j, head, dim),
 *   F_V = [v_src[s_j][t] for j < k],  s_j = src_layers[l*k + j],
 *   k_tgt[l][t] = bf16(RoPE_tgt(F_K Wk_lᵀ + bk_l)),  v_tgt[l][t] = bf16(F_V Wv_lᵀ + bv_l).
 *   src_layers  device int32 [L_tgt][k], each in [0, L_src) (e.g. rf_select_sources'
 *               output, used with no host round trip). The table is checked on the
 *               device: an entry outside [0, L_src) writes RF_ERR_INVALID_ARG to
 *               *dev_status and the call then writes no target entry.
 *   k_src, v_src [L_src][N][KV] bf16;  k_tgt, v_tgt [L_tgt][N][KV] bf16
 *   Wk, Wv [L_tgt][KV][k*KV] bf16 (row = output);  bk, bv [L_tgt][KV] fp32 */
rf_status rf_xmodel_map(const rf_xmodel_desc* desc, const int32_t* src_layers,
                        const rf_bf16* k_src, const rf_bf16* v_src,
                        const rf_bf16* Wk, const float* bk,
                        const rf_bf16* Wv, const float* bv,
                        rf_bf16* k_tgt, rf_bf16* v_tgt, int32_t* dev_status,
                        void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* RoPE (inverse = 0) or its inverse (inverse = 1) on rows of heads, out of place
 * or in place: out[t][h][:] = R^{±1}(t + pos_offset) in[t][h][:]. The angle
 * (t + pos_offset)·θ^(-2i/hd) is reduced mod 2π exactly in 64-bit fixed point,
 * then its sine and cosine are taken in fp32 (absolute error about 2^-21); the
 * fill and the mapper rotate the same way.
 * in, out [n_rows][ld] bf16 with H*hd <= ld. Used to build cross-model
 * calibration features (un-roped keys). [XM] content-space mapping. */
rf_status rf_rope_rows(const rf_bf16* in, rf_bf16* out, int64_t n_rows, int64_t ld,
                       int64_t n_heads, int64_t head_dim, double theta,
                       int64_t pos_offset, int inverse, rf_stream_t stream);

/* Side-by-side features of several layers, for cross-model calibration:
 *   out[t][l*W + j] = f(src[l*layer_stride + t*ld_src + j]),  W = n_heads*head_dim,
 *   f = inverse RoPE at position t + pos_offset with base theta (theta > 0: keys)
 *   or the identity (theta == 0: values), for l < n_layers, t < n_rows, j < W.
 * src, out bf16 device; ld_src >= W, ld_out >= n_layers*W, strides multiples of 8.
 * [XM] "층 교차 소스 선택": a target layer's features are all heads of its source
 * layers side by side; content-space mapping: keys are un-roped first. */
rf_status rf_concat_layers(const rf_bf16* src, int64_t n_layers, int64_t layer_stride,
                           int64_t n_rows, int64_t ld_src, int64_t n_heads, int64_t head_dim,
                           double theta, int64_t pos_offset,
                           rf_bf16* out, int64_t ld_out, rf_stream_t stream);

/* ===================================================================== *
 * Cross-layer source selection ([XM] "소스 층은 몇 개가 필요한가": greedy
 * forward selection adding the source layer that raises the head-mean R² most;
 * "층 교차 소스 선택": k layers per target layer, chosen by the head-mean R² of
 * the un-roped keys and of the values, shared by all heads of the target layer)
 * ===================================================================== */
typedef struct rf_select_desc {
  int64_t L_src;      /* candidate source layers                                       */
  int64_t F;          /* features per source layer (the statistics' d_in = L_src * F)  */
  int64_t n_targets;  /* target layers (the statistics' n_maps)                        */
  int64_t d_out;      /* columns per target layer                                      */
  int64_t head_dim;   /* columns per target head; R² is averaged over d_out/head_dim   */
  int64_t k;          /* layers chosen per target layer, 1 <= k <= L_src               */
  int64_t n_kinds;    /* statistics sets scored together: 1, or 2 (keys and values)    */
  int64_t group;      /* target layers per pass, 0 = all; the workspace grows with it  */
  uint64_t flags;     /* RF_FLAG_* (0 = defaults)                                      */
} rf_select_desc;

/* Supported: F % 256 == 0, d_out % 256 == 0, d_out % head_dim == 0,
 * L_src * F <= 65536, n_targets <= 65535. */
size_t rf_select_workspace_bytes(const rf_select_desc* desc);

/* Greedy forward selection for every target layer t, from calibration sums
 * (stats[kind], one set per kind, each with d_in = L_src*F, d_out, n_maps =
 * n_targets and syy set):
 *   per kind: Gc, Cc_t centred as in rf_solve, TSS_t[o] = syy_t[o] − n μ_t[o]²,
 *   α = λ·tr(Gc)/(L_src*F) (RF_ALPHA_TRACE, over ALL source features) or λ;
 *   the score of a layer set S for target t and kind: the mean over heads h of
 *     R²_h = Σ_{o∈h} Cc_t[S,o]ᵀ (Gc[S,S] + αI)^-1 Cc_t[S,o] / Σ_{o∈h} TSS_t[o],
 *   i.e. 1 − (RSS + α‖w‖²)/TSS of the ridge fit (the least-squares R² at λ = 0);
 *   a head with TSS = 0 counts as R² = 0;
 *   step j adds the layer s not yet chosen whose set S ∪ {s} has the highest mean
 *   score over kinds (the lowest index among equal scores).
 * Outputs (device): src_layers [n_targets][k] int32, the layer chosen at each step;
 * r2 [n_kinds][n_targets][k][L_src] fp32 (may be NULL): each candidate's score at
 * each step, NaN for layers already chosen (step 0 is the single-layer R² table).
 * Arithmetic: the Gram and cross terms in fp32, products as fp32-accurate split
 * bf16 tensor-core GEMMs, Schur blocks factored in fp32; scores in fp64.
 * A non-positive pivot sets RF_ERR_NOT_SPD in *dev_status. */
rf_status rf_select_sources(const rf_select_desc* desc, const rf_calib_stats* stats,
                            double lambda, int alpha_mode,
                            int32_t* src_layers, float* r2, int32_t* dev_status,
                            void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* ===================================================================== *
 * Decoding from a filled cache: rotation, attention of drafted trees,
 * verification of drafted tokens, eviction.
 *
 * A decoding step drafts a tree of n_nodes tokens per sequence. Node 0 is its root
 * (the last token accepted, whose K and V are not in the cache yet), every other
 * node's parent has a lower index. The drafted rows' K and V stay in buffers of
 * their own until the tokens are verified; only accepted rows join the cache. With
 * n_nodes = 1 a step is plain decoding of one token.
 * A cache of one layer holds, for sequence b, row t, KV head h, channel c, element
 * b*seq_stride + t*row_stride + h*head_dim + c; lens[b] rows are in use. What lies
 * in rows beyond lens[b] is never used, whatever its bits are.
 * ===================================================================== */

/* Element types and channel pairings of rf_rope; frequency scalings for contexts
 * longer than the model was trained on. */
#define RF_BF16 0
#define RF_F32 1
#define RF_ROPE_HALF 0        /* channel i turns with i + rot_dim/2                     */
#define RF_ROPE_INTERLEAVED 1 /* channel 2i turns with 2i + 1                           */
#define RF_ROPE_SCALE_NONE 0
#define RF_ROPE_SCALE_LINEAR 1
#define RF_ROPE_SCALE_BASE 2
#define RF_ROPE_SCALE_WAVELENGTH 3
#define RF_ROPE_SCALE_RAMP 4

typedef struct rf_rope_desc {
  int64_t n_rows;       /* tokens, at most 2^24                                         */
  int64_t n_heads;      /* heads of a row, head_dim channels each, one after another    */
                        /* (at most 65535)                                              */
  int64_t head_dim;     /* a multiple of 8, at most 256                                 */
  int64_t rot_dim;      /* the first rot_dim channels of a head turn (even, at most     */
                        /* head_dim); the others are copied                             */
  int64_t ld_in;        /* row strides                                                  */
  int64_t ld_out;
  int64_t pos_offset;   /* position of row 0 when no positions are given                */
  double theta;         /* base                                                         */
  double factor;        /* s >= 1: how many times longer the context is (see below)     */
  double original_rows; /* R: context the model was trained on (WAVELENGTH, RAMP)       */
  double low_turns;     /* turns within R rows below which a frequency is divided by s  */
  double high_turns;    /* turns within R rows above which a frequency stays            */
  double amplitude;     /* the rotation is multiplied by it; 0 = 1                      */
  int32_t layout;       /* RF_ROPE_HALF or RF_ROPE_INTERLEAVED                          */
  int32_t dtype;        /* RF_BF16 or RF_F32, of in and out                             */
  int32_t transpose;    /* nonzero: the transposed rotation, which is the gradient's    */
                        /* (and the inverse where amplitude is 1)                       */
  int32_t scaling;      /* RF_ROPE_SCALE_*                                              */
} rf_rope_desc;

/* out[t][h] = amplitude * R(p_t) in[t][h], with p_t = positions[t] (device int32) or
 * t + pos_offset when positions is NULL. Pair i of a head turns by p_t f_i,
 *   f_i = theta^(-2i/rot_dim)                                          (NONE)
 *   f_i / s                                                            (LINEAR)
 *   (theta s^(rot_dim/(rot_dim-2)))^(-2i/rot_dim)                      (BASE, rot_dim > 2)
 *   f_i (w + (1-w)/s), w = clamp((R f_i/2pi - low)/(high - low), 0, 1)  (WAVELENGTH)
 *   f_i ((1-w) + w/s), w = clamp((i - lo)/(hi - lo), 0, 1),            (RAMP)
 *     lo = max(floor(d(high)), 0), hi = min(ceil(d(low)), rot_dim - 1),
 *     d(x) = rot_dim ln(R/(2 pi x)) / (2 ln theta).
 * The angle is reduced mod 2 pi in 64-bit fixed point; bf16 rows take their sine and
 * cosine to about 2^-21, fp32 rows to fp32. in and out 16-byte aligned, strides
 * multiples of 8 elements; out may be in (with ld_out = ld_in). No workspace. */
rf_status rf_rope(const rf_rope_desc* desc, const void* in, void* out, const int32_t* positions,
                  rf_stream_t stream);

/* Rotation of normalised queries and keys ("Qwen models normalize keys": a cache filled with
 * rf_fill_desc.k_norm_gain is decoded from with these). A row holds n_q_heads query heads, then
 * key heads, rope.n_heads in all. */
typedef struct rf_norm_rope_desc {
  rf_rope_desc rope;    /* rows, heads, strides, types and rotation as for rf_rope; transpose 0 */
  int64_t n_q_heads;    /* 0 .. rope.n_heads: these take q_gain, the others k_gain             */
  double eps;           /* > 0 (a normal number in fp32)                                        */
} rf_norm_rope_desc;

/* out[t][h] = amplitude * R(p_t) (g * x / sqrt(mean(x^2) + eps)) for every head x = in[t][h], with
 * the means over the head's channels, the rotation R and the positions of rf_rope, and g = q_gain
 * or k_gain, [head_dim] values of the rows' type (16-byte aligned; NULL: ones). Squares, means and
 * products are fp32 (a head's squares must add up to less than 2^128); there is one rounding, at
 * the end. A gain that is not finite stays within its channel, or, if that turns, its pair of channels.
 * out may be in (with ld_out = ld_in). No workspace. */
rf_status rf_norm_rope(const rf_norm_rope_desc* desc, const void* in, const void* q_gain, const void* k_gain,
                       void* out, const int32_t* positions, rf_stream_t stream);

/* The gradient of rf_norm_rope, from d_out (laid out as out):
 *   d_in     (laid out as in; only the heads are written) the rows' gradient. It may be in, or
 *            d_out (with ld_out = ld_in).
 *   d_q_gain, d_k_gain  [head_dim] fp32 (either may be NULL), written, not added to: the sums over all
 *            rows and query heads, or key heads, of the gains' gradients; zero where there are none
 * in, gains, positions and desc as for the call whose gradient it is. What is not finite in d_out stays within
 * its head's gradient, and in the gains' within its channel or pair of channels. Sums are fp32, in an order that
 * depends on the sizes and the GPU alone. The workspace is needed for the gains' gradients only. */
size_t rf_norm_rope_backward_workspace_bytes(const rf_norm_rope_desc* desc);
rf_status rf_norm_rope_backward(const rf_norm_rope_desc* desc, const void* in, const void* q_gain,
                                const void* k_gain, const void* d_out, const int32_t* positions, void* d_in,
                                float* d_q_gain, float* d_k_gain, void* workspace, size_t workspace_bytes,
                                rf_stream_t stream);

/* Words of a node's mask: bit j % 64 of word j / 64 says whether it sees node j. */
#define RF_TREE_WORDS(n_nodes) (((n_nodes) + 63) / 64)
#define RF_TREE_MAX_NODES 1024

/* From each sequence's parents (device int32 [n_seqs][n_nodes]; parents[0] = -1, else
 * 0 <= parents[i] < i):
 *   mask       [n_seqs][n_nodes][RF_TREE_WORDS(n_nodes)] uint64: a node sees itself
 *              and its ancestors (may be NULL)
 *   positions  [n_seqs][n_nodes] int32: next_pos[b] + the node's depth (may be NULL)
 *   next_pos   [n_seqs] int32: position of node 0 (not read when positions is NULL)
 * n_nodes <= RF_TREE_MAX_NODES. A sequence with other parents records
 * RF_ERR_INVALID_ARG in *dev_status and its outputs are not written. */
rf_status rf_tree_build(int64_t n_seqs, int64_t n_nodes, const int32_t* parents, const int32_t* next_pos,
                        uint64_t* mask, int32_t* positions, int32_t* dev_status, rf_stream_t stream);

typedef struct rf_attn_desc {
  int64_t n_seqs;           /* sequences, at most 2^20                                  */
  int64_t n_q_heads;        /* query heads, a multiple of n_kv_heads; query head i reads */
                            /* KV head i / (n_q_heads/n_kv_heads); at most 128 per KV head */
  int64_t n_kv_heads;
  int64_t head_dim;         /* 64 or 128                                                */
  int64_t n_nodes;          /* queries (drafted rows) per sequence                      */
  int64_t capacity;         /* cache rows per sequence, 0 <= lens[b] <= capacity <= 2^30 */
  int64_t q_row_stride;     /* q: element b*q_seq_stride + i*q_row_stride + head*head_dim + c */
  int64_t q_seq_stride;
  int64_t draft_row_stride; /* k_draft, v_draft, likewise                               */
  int64_t draft_seq_stride;
  int64_t cache_row_stride; /* k_cache, v_cache, likewise                               */
  int64_t cache_seq_stride;
  int64_t out_row_stride;   /* out, likewise                                            */
  int64_t out_seq_stride;
  double scale;             /* scores are scale * q.k; > 0, scale / ln 2 finite in fp32 */
  uint64_t flags;           /* 0                                                        */
} rf_attn_desc;

/* Attention of the drafted rows over the cache and over each other. For sequence b,
 * node i, query head a (KV head h):
 *   S = {cache rows t < lens[b]} + {drafted rows j that node i sees},
 *   lse = ln sum_{j in S} exp(scale q.k_j),  out = sum_{j in S} exp(scale q.k_j - lse) v_j.
 *   tree_mask  [n_seqs][n_nodes][RF_TREE_WORDS(n_nodes)] uint64 (device), any bits (n_nodes
 *              <= RF_TREE_MAX_NODES; bits beyond n_nodes are ignored), or NULL: node i
 *              sees drafted rows j <= i (rows in order, n_nodes <= 2^20; < 2^20 with more
 *              than 64 query heads per KV head)
 *   lens       [n_seqs] int32 (device); a length outside [0, capacity] records
 *              RF_ERR_INVALID_ARG in *dev_status and that sequence is not written
 *   out bf16;  lse [n_seqs][n_nodes][n_q_heads] fp32 (may be NULL)
 * A row that sees nothing gives out = 0 and lse = -inf. Rows that are not seen have no
 * influence, NaN and infinities among them. Scores, statistics and sums are fp32; a
 * weight is rounded to bf16 for its product with v. The keys are split over the GPU in
 * equal shares whatever the lengths are, and split rows are joined in a fixed order. */
size_t rf_attn_workspace_bytes(const rf_attn_desc* desc);
rf_status rf_tree_attention(const rf_attn_desc* desc, const rf_bf16* q,
                            const rf_bf16* k_cache, const rf_bf16* v_cache, const int32_t* lens,
                            const rf_bf16* k_draft, const rf_bf16* v_draft, const uint64_t* tree_mask,
                            rf_bf16* out, float* lse, int32_t* dev_status,
                            void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* A batch whose sequences all continue one prompt, for example one that rf_fill_kv has filled. */
typedef struct rf_prefix_attn_desc {
  rf_attn_desc attn;          /* queries, the sequences' own caches, drafted rows and output, as for */
                              /* rf_tree_attention; n_seqs * n_nodes * n_q_heads <= 2^28             */
  int64_t prefix_capacity;    /* rows of k_prefix and v_prefix, 1 .. 2^30                            */
  int64_t prefix_row_stride;  /* element t*prefix_row_stride + h*head_dim + c                        */
} rf_prefix_attn_desc;

/* rf_tree_attention over a prefix that all sequences share, each one's own cache rows and the drafted
 * rows:
 *   S = {prefix rows t < *prefix_len} + {cache rows t < lens[b]} + {drafted rows j that node i sees}.
 * The prefix is held once and read once for all sequences, whose rows make up its matrix products, so a
 * prefix costs a batch about what it costs one sequence, up to 256 query rows per KV head. Own caches may
 * be empty (lens[b] = 0), and so may the prefix.
 *   prefix_len  device int32; outside [0, prefix_capacity] it records RF_ERR_INVALID_ARG and nothing is
 *               written
 * All other arguments, masks, what is not seen, refusals and the status of lengths as for
 * rf_tree_attention; an infinity in a V row that is seen may come out as NaN. Scores, statistics and sums are
 * fp32, joined in a fixed order; a weight is rounded to bf16 for its product with v. */
size_t rf_prefix_attn_workspace_bytes(const rf_prefix_attn_desc* desc);
rf_status rf_prefix_attention(const rf_prefix_attn_desc* desc, const rf_bf16* q,
                              const rf_bf16* k_prefix, const rf_bf16* v_prefix, const int32_t* prefix_len,
                              const rf_bf16* k_cache, const rf_bf16* v_cache, const int32_t* lens,
                              const rf_bf16* k_draft, const rf_bf16* v_draft, const uint64_t* tree_mask,
                              rf_bf16* out, float* lse, int32_t* dev_status,
                              void* workspace, size_t workspace_bytes, rf_stream_t stream);

typedef struct rf_verify_desc {
  int64_t n_seqs;     /* at most 2^24                                                  */
  int64_t n_nodes;    /* 1 .. RF_TREE_MAX_NODES                                        */
  int64_t vocab;      /* V <= 2^31 - 65536                                             */
  int64_t ld_target;  /* row strides, >= vocab (any value)                              */
  int64_t ld_draft;
  int64_t ld_noise;
} rf_verify_desc;

/* Verifies each sequence's drafted tokens against the target's probabilities, so that
 * the tokens kept are distributed as the target's own. From node c = 0, with
 * r = target row of c and Z = 1: c's children x are tried in index order; child x (its
 * token t) is accepted when u[x] q(t) Z < r(t), and then c = x starts over. A refused
 * one leaves r <- max(r/Z - q, 0) and Z <- sum r (r and Z stay when that sum is 0).
 * With no child left the next token is the lowest argmax of r(t)/noise(t) over r > 0.
 *   target   [n_seqs*n_nodes][ld_target] fp32: probabilities after each node
 *   draft    [n_seqs*n_nodes][ld_draft] fp32: q, the distribution that each node's
 *            children were drawn from; NULL: children were chosen outright, q(t) = 1 at
 *            the child's own token and 0 elsewhere (a refused one leaves r without its
 *            token)
 *   tokens   [n_seqs][n_nodes] int32 (node 0's is not read), parents as for rf_tree_build
 *   u        [n_seqs][n_nodes] fp32 uniform in [0, 1) (node 0's is not read)
 *   noise    [n_seqs][ld_noise] fp32, exponentially distributed, > 0
 * Outputs: path [n_seqs][n_nodes] int32, the accepted nodes in order (node 0 first),
 * then -1; n_path [n_seqs] int32; next_token [n_seqs] int32. A sequence with wrong
 * parents or tokens outside [0, vocab) records RF_ERR_INVALID_ARG and gets n_path 0,
 * next_token -1. Sums are fp32; r/Z, its difference to q and r/noise are rounded one by
 * one (IEEE), u q Z from the left. No workspace. */
rf_status rf_verify_draft(const rf_verify_desc* desc, const float* target, const float* draft,
                          const int32_t* tokens, const int32_t* parents, const float* u, const float* noise,
                          int32_t* path, int32_t* n_path, int32_t* next_token, int32_t* dev_status,
                          rf_stream_t stream);

typedef struct rf_sample_desc {
  int64_t n_rows;     /* at most 2^24                                                  */
  int64_t vocab;      /* 1 .. 2^20                                                     */
  int64_t ld_logits;  /* row strides, >= vocab (any value up to 2^36)                   */
  int64_t ld_noise;
  int64_t ld_probs;
  int32_t dtype;      /* RF_BF16 or RF_F32, of the logits                               */
  int32_t reserved;   /* 0                                                             */
} rf_sample_desc;

/* Draws a token from each row of logits, or gives the probabilities to draw it from (for example
 * rf_verify_draft's target and draft, for logits after each node).
 * With w_i = exp((x_i - max x) / temperature) and the tokens by falling logit, the lowest token first
 * among equals, those that stay are, one filter after another,
 *   top_k   the first k (0: all);
 *   top_p   of those the fewest first ones whose weights add up to p times the sum of theirs or more
 *           (1 or more: all; 0: the first);
 *   min_p   of those the ones with w_i >= min_p (0: all).
 *   probs[i] = w_i / (sum of the weights that stay), 0 for the others;
 *   token    = the lowest argmax of w_i / noise[i] of those that stay; logprob = ln probs[token]
 * temperature 0 is greedy: the lowest argmax of x, with probability 1. Logits of -inf or NaN never
 * stay; where some are +inf, they alone do, with equal weights.
 *   logits       [n_rows][ld_logits] bf16 or fp32
 *   temperature  [n_rows] fp32, 0 or 2^-100 .. 2^100 (NULL: 1);  top_k [n_rows] int32 >= 0 (NULL: 0);
 *                top_p [n_rows] fp32 >= 0 (NULL: 1);  min_p [n_rows] fp32 in [0, 1] (NULL: 0)
 *   noise        [n_rows][ld_noise] fp32, exponentially distributed, > 0; used where tokens stay. Needed
 *                with token, NULL without
 *   probs        [n_rows][ld_probs] fp32, NULL: not wanted. May be the logits (fp32, the same stride), but
 *                not the noise
 *   token, logprob, n_kept  [n_rows] int32, fp32, int32; each may be NULL, but not token and probs both.
 *                n_kept is how many tokens stay
 * A row with nothing to choose from gives token -1, logprob -inf, n_kept 0 and probabilities 0, and so
 * does a row with a setting out of range, which also records RF_ERR_INVALID_ARG in *dev_status. So does a row
 * without noise above 0 at any token that stays, whose token is -1 and logprob -inf.
 * What stays is decided by sums of integers, in which a weight counts to 2^-29 of itself (of those below
 * 2^-32 to 2^-53), and the weights of each 1/64 octave together to 2^-42; weights, probabilities and scores are
 * fp32, and weights below 2^-126 are 0. Equal inputs give equal results. No workspace. */
rf_status rf_sample(const rf_sample_desc* desc, const void* logits, const float* temperature, const int32_t* top_k,
                    const float* top_p, const float* min_p, const float* noise, float* probs, int32_t* token,
                    float* logprob, int32_t* n_kept, int32_t* dev_status, rf_stream_t stream);

/* A cache of all layers: element l*layer_stride + b*seq_stride + t*row_stride + h*head_dim + c.
 * Layers, sequences and rows may be nested in any order; no two rows may overlap. */
typedef struct rf_cache_desc {
  int64_t n_layers;     /* at most 65535, as n_seqs and n_kv_heads                      */
  int64_t n_seqs;
  int64_t n_kv_heads;
  int64_t head_dim;     /* a multiple of 8, at most 256                                 */
  int64_t capacity;     /* rows per sequence, at most 2^24                              */
  int64_t row_stride;
  int64_t seq_stride;
  int64_t layer_stride;
} rf_cache_desc;

/* Appends the accepted rows of every layer to the cache: for j < n_path[b],
 *   cache row lens[b] + j <- drafted row path[b][j],
 *   score[l][b][h][lens[b]+j] <- 0, pos[l][b][h][lens[b]+j] <- next_pos[b] + j,
 *   new_lens[b] = lens[b] + n_path[b], new_next_pos[b] = next_pos[b] + n_path[b].
 * score, pos [n_layers][n_seqs][n_kv_heads][capacity] (either may be NULL); k_draft,
 * v_draft: element l*draft_layer_stride + b*draft_seq_stride + i*draft_row_stride +
 * h*head_dim + c. new_lens may be lens and new_next_pos next_pos; either may be any of lens,
 * next_pos and n_path, but not overlap them in part, nor path. next_pos may be NULL together
 * with new_next_pos and pos. A sequence whose rows do not fit, or whose path or
 * counts are out of range, records RF_ERR_INVALID_ARG and keeps its lengths and rows. */
rf_status rf_commit_draft(const rf_cache_desc* desc, int64_t n_nodes, int64_t draft_row_stride,
                          int64_t draft_seq_stride, int64_t draft_layer_stride,
                          const int32_t* path, const int32_t* n_path,
                          const int32_t* lens, const int32_t* next_pos,
                          const rf_bf16* k_draft, const rf_bf16* v_draft,
                          rf_bf16* k_cache, rf_bf16* v_cache, float* score, int32_t* pos,
                          int32_t* new_lens, int32_t* new_next_pos, int32_t* dev_status, rf_stream_t stream);

/* Adds the attention weights that each cached row received. The queries are the nodes
 * path[b][0 .. n_path[b]-1] (all n_nodes rows in order when path and n_path are NULL);
 * their own rows are the last of the cache's lens[b] rows (after rf_commit_draft). For
 * every cache row t < lens[b] and KV head h:
 *   score_out[b][h][t] = decay score_in[b][h][t]
 *       + sum over j with t <= lens[b] - n + j, and the KV head's query heads a, of
 *         exp(scale q[path[j]][a].k_t - lse[path[j]][a]),   n = n_path[b] or n_nodes.
 * q, lse, desc as for rf_tree_attention, with n_seqs <= 1024; score
 * [n_seqs][n_kv_heads][capacity] fp32, score_out may be score_in; entries t >= lens[b] are
 * not written. A query whose lse is -inf adds nothing. decay 0 does not read score_in (which
 * may be NULL then). A sequence with a length, count or path out of range records
 * RF_ERR_INVALID_ARG and is not written (n <= lens[b] is required). Sums are fp32, in an
 * order that depends on the sizes alone. The workspace (256 bytes) is required, though
 * nothing is kept in it at present. */
size_t rf_attn_weights_workspace_bytes(const rf_attn_desc* desc);
rf_status rf_attn_weights(const rf_attn_desc* desc, const rf_bf16* q, const float* lse,
                          const int32_t* path, const int32_t* n_path,
                          const rf_bf16* k_cache, const int32_t* lens, double decay,
                          const float* score_in, float* score_out, int32_t* dev_status,
                          void* workspace, size_t workspace_bytes, rf_stream_t stream);

/* Evicts rows of little weight: in every layer, sequence and KV head, min(lens[b], keep)
 * rows stay. Rows whose position is below n_sink or at least next_pos[b] - n_recent rank
 * as +inf, the others by score (NaN as -inf); the highest ranks stay, the lowest row
 * index first among equals. Rows that stay and lie below `keep` do not move; the i-th
 * (ascending) that lies beyond moves into the i-th (ascending) hole below, so each head
 * moves as few rows as can be. Attention does not depend on the rows' order; `pos`
 * holds each row's position.
 *   score_in, pos_in, score_out, pos_out  [n_layers][n_seqs][n_kv_heads][capacity]; out
 *       may be in; entries beyond new_lens[b] are not written
 *   new_lens [n_seqs] int32: lens itself (or next_pos), or apart from lens
 * A length outside [0, capacity] records RF_ERR_INVALID_ARG and that sequence stays as
 * it is. keep >= 1, n_layers * n_seqs * n_kv_heads <= 65535. */
size_t rf_evict_workspace_bytes(const rf_cache_desc* desc, int64_t keep);
rf_status rf_evict(const rf_cache_desc* desc, int64_t keep, int64_t n_sink, int64_t n_recent,
                   const int32_t* lens, const int32_t* next_pos, rf_bf16* k_cache, rf_bf16* v_cache,
                   const float* score_in, const int32_t* pos_in, float* score_out, int32_t* pos_out,
                   int32_t* new_lens, int32_t* dev_status,
                   void* workspace, size_t workspace_bytes, rf_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* RIDGE_MAP_KV_RF_H */
