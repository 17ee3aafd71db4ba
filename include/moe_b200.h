/*
 * moe_b200.h -- C ABI of the B200 (sm_100a) sparse-MoE layer forward pass.
 *
 * The layer is the gpt-oss-style Mixture-of-Experts feed-forward block:
 *
 *   s_e   = W_r[e] . x_t + b_r[e]                          (router logits)
 *   S_t   = the k largest s_e (ties: lower expert index first)
 *   p_j   = exp(s_j) / sum_{l in S_t} exp(s_l)             (softmax over S_t)
 *   E_e(x)= W_down[e] (silu(W_gate[e] x) * (W_up[e] x))    (SwiGLU expert)
 *   out_t = sum_{j in S_t} p_j E_j(x_t)
 *
 * Sources: "llm-surgery-dark-arts-gpt-oss-40b-64a8-init", section 2, "Proof"
 * (the forward pass, the router logits and the softmax over the selected set);
 * field guide "gpt-oss 20B", "03 Sparse Mixture of Experts" (score all experts,
 * keep the top k, normalise those scores, weighted sum of SwiGLU experts);
 * "gpt-oss-20b and gpt-oss-120b", "Four-bit expert weights" (MXFP4 experts,
 * 4.25 bits per parameter); "shrink/gpt_oss-mic", "Preserved properties"
 * (hidden_act silu).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers named *_dev are CUDA device pointers; *_host are host pointers.
 *   Every device pointer must be 16-byte aligned. Inputs are read-only.
 * - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *   stream). All device work is enqueued on it; no entry point synchronises
 *   the stream except moe_forward_hostio and moe_sync_status, which say so.
 * - The library allocates no device memory. The caller owns every buffer,
 *   including the workspace, whose size moe_workspace_size() returns.
 *   Concurrent calls must not share a workspace.
 * - Errors are returned as moe_status; nothing is thrown or printed.
 *   Arguments are checked before anything is launched; on an argument error
 *   no work is enqueued. Device-side timeouts (a bounded wait in a kernel
 *   that gave up) are recorded in a status word inside the workspace and
 *   reported by moe_sync_status() or by the next call on that workspace.
 *
 * Data layout (row-major, C order)
 * --------------------------------
 *   x           [T][d]        bf16 (raw 16-bit patterns)
 *   W_r         [E][d]        float32
 *   b_r         [E]           float32
 *   Wgu_codes   [E][2I][d/2]  uint8  MXFP4 E2M1 codes; rows 0..I-1 are the
 *                                    gate projection, rows I..2I-1 the up
 *                                    projection; byte b of a row holds
 *                                    element 2b in its low nibble and
 *                                    element 2b+1 in its high nibble
 *   Wgu_scales  [E][2I][d/32] uint8  E8M0 scale 2^(S-127) of each group of
 *                                    32 consecutive elements along d
 *   Wd_codes    [E][d][I/2]   uint8  down projection codes (contraction on I)
 *   Wd_scales   [E][d][I/32]  uint8
 *   out         [T][d]        bf16
 *   topk_idx    [T][k]        int32  experts of token t, logit descending,
 *                                    then expert index ascending
 *   topk_w      [T][k]        float32 selected-set softmax weights
 *
 * Supported range: 1 <= E <= 256, 1 <= k <= min(E, 32), T >= 0,
 * d and I multiples of 32 with 32 <= d, I <= 16384. Decoded weight
 * magnitudes must be below 2^128 (E8M0 bytes up to 252), the range bf16
 * represents; within it every decoded weight is exact.
 */
#ifndef MOE_B200_H
#define MOE_B200_H

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

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,   /* null pointer, misaligned pointer, bad shape  */
  MOE_ERR_UNSUPPORTED = 2,   /* shape outside the supported range            */
  MOE_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required   */
  MOE_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed            */
  MOE_ERR_TIMEOUT = 5,       /* a kernel's bounded wait expired              */
  MOE_ERR_NO_DEVICE = 6      /* no sm_100 device is current                  */
} moe_status;

/* Human-readable name of a status code (static storage, never NULL). */
MOE_API const char* moe_status_string(moe_status s);

/* Library version as major*10000 + minor*100 + patch. */
MOE_API int moe_version(void);

/*
 * Tile policy of the grouped GEMMs, process-wide: 0 (default) picks by shape
 * from the average number of routed rows per expert, P/E with P = T*k:
 *   P/E < 32        block-scaled tiles (policy 4 below) where the shape allows
 *                   them, else swapped-operand tiles (128 weight rows x 64
 *                   tokens, the decoded weights as the UMMA A operand),
 *   32 <= P/E < 192 single-CTA tiles (256 x 128, the second 128-row half
 *                   skipped for short expert tails),
 *   P/E >= 192      CTA-pair tiles: the block-scaled ones (policy 5 below)
 *                   where the shape allows them, else bf16 CTA-pair tiles (a
 *                   2-CTA cluster computes 256 x 240 tiles with tcgen05
 *                   cta_group::2).
 * 1, 2 and 3 force single-CTA, CTA-pair and swapped-operand tiles; these
 * decode the MXFP4 weights to bf16 in shared memory or TMEM and run bf16
 * UMMAs on bf16 activations.
 * 4 selects the block-scaled tiles: tcgen05.mma .kind::mxf8f6f4 with the E2M1
 * codes widened to 8-bit containers by TMA, the E8M0 weight scales applied by
 * the tensor core, and each bf16 activation (and H) row split per 32 elements
 * into two E4M3 terms (hi and lo) with E8M0 scales; the split is exact for
 * elements of at least 2^-13 of their group's max |x|, smaller ones keep an
 * error below 2^-21 of it. 128 weight rows x 16 tokens per tile, two CTAs
 * per SM with two UMMA-issuing threads each (120-token tiles, one CTA per SM,
 * when experts average 64 rows or more).
 * 5 selects the block-scaled tiles on a CTA pair: a 2-CTA cluster computes
 * 256-token tiles with tcgen05.mma.cta_group::2 (M = 256 token rows, the two
 * E4M3 terms issued as two UMMAs into one accumulator; N = 192 weight rows for
 * gate/up, 240 for down).
 * 4 and 5 need d and I multiples of 64 in [128, 3072] and 32-byte aligned
 * code arrays; otherwise they pick as policy 0 does.
 * All policies compute the same function within the output tolerance.
 * This sets the process default that the entry points without an options
 * argument use; a change takes effect for calls made after it, from any
 * thread. Callers that share a process and want a policy of their own pass
 * it per call through moe_forward_ex instead. MOE_ERR_INVALID_ARG for other
 * values.
 */
MOE_API moe_status moe_set_tile_policy(int policy);

/*
 * Precision of the activations that enter the expert GEMMs (the expert inputs
 * x and the SwiGLU rows H), per call through moe_forward_opts.act_quant.
 *   MOE_ACT_BF16   the layer as the pages define it: bf16 activations used at
 *                  full precision (the block-scaled tiles split each value
 *                  exactly into two E4M3 terms); output within 2e-2 x RMS.
 * The two others change the function ("gpt-oss-20b and gpt-oss-120b",
 * "Four-bit expert weights" puts only the expert weights in MXFP4; field
 * guide "gpt-oss 20B": MXFP4 is "not every path"): the activations are
 * rounded to an MX block format, per group of 32 along the contraction, with
 * the OCP Microscaling conversion (shared scale 2^(floor(log2 max|v|) - emax),
 * elements rounded to nearest even, magnitudes above the largest normal
 * clamped to it):
 *   MOE_ACT_MXFP8  E4M3 elements (emax 8): the w4a8 layer;
 *   MOE_ACT_MXFP4  E2M1 elements (emax 2): the w4a4 layer.
 */
typedef enum { MOE_ACT_BF16 = 0, MOE_ACT_MXFP8 = 1, MOE_ACT_MXFP4 = 2 } moe_act_quant;

/*
 * Per-call options of moe_forward_ex. Zero-initialise and set what you need.
 *   tile_policy    -1: the process default (moe_set_tile_policy); 0: pick by
 *                  shape; 1..5: force a tile family (as moe_set_tile_policy).
 *                  0 is what a zeroed struct asks for.
 *   act_quant      a moe_act_quant value (0 = MOE_ACT_BF16).
 *   gu_bias_dev, down_bias_dev   the experts' biases as in
 *                  moe_forward_biased; NULL for none.
 */
typedef struct {
  int tile_policy;
  int act_quant;
  const float* gu_bias_dev;
  const float* down_bias_dev;
} moe_forward_opts;

/*
 * Bytes of device workspace moe_forward needs for this shape (0 for invalid
 * shapes). The workspace holds the router's logits and top-k, the routing
 * tables, the permuted activations, the SwiGLU hidden rows H [T*k][I] bf16,
 * the weighted per-slot expert outputs [T*k][d] fp32, and the down weights'
 * scale factors re-laid out for the CTA-pair tiles (E * ceil(d/224) *
 * ceil(I/128) KiB).
 */
MOE_API size_t moe_workspace_size(int E, int k, int T, int d, int I);

/*
 * Forward pass of the MoE layer (the whole path: router, top-k, selected-set
 * softmax, permutation, gate/up grouped GEMM with SwiGLU, down grouped GEMM
 * with the weighted un-permute, and the per-token sum).
 * "llm-surgery-dark-arts-gpt-oss-40b-64a8-init", section 2, "Proof".
 *
 * Writes out_dev [T][d] bf16 completely. Asynchronous on `stream`.
 */
MOE_API moe_status moe_forward(const void* x_dev, const float* W_r_dev, const float* b_r_dev,
                       const uint8_t* Wgu_codes_dev, const uint8_t* Wgu_scales_dev,
                       const uint8_t* Wd_codes_dev, const uint8_t* Wd_scales_dev,
                       int E, int k, int T, int d, int I, void* out_dev,
                       void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * moe_forward with per-expert projection biases, as a gpt-oss expert carries
 * them (the parameter totals of "gpt-oss-20b and gpt-oss-120b" count 2I + d
 * bias values per expert):
 *   H = silu(x Wgate^T + b_gate) * (x Wup^T + b_up),  y = H Wdown^T + b_down,
 * and the layer output sum_j p_j y_j as in moe_forward.
 * gu_bias_dev [E][2I] f32: row e holds expert e's gate biases (0..I-1), then
 * its up biases (I..2I-1). down_bias_dev [E][d] f32. Either may be NULL (no
 * bias on that projection; with both NULL this is moe_forward); each given
 * one is 16-byte aligned device memory, read-only and the caller's. The
 * biases are added to the fp32 accumulators in the GEMM epilogues (no extra
 * launches). Errors, workspace and stream semantics are those of moe_forward.
 */
MOE_API moe_status moe_forward_biased(const void* x_dev, const float* W_r_dev, const float* b_r_dev,
                                      const uint8_t* Wgu_codes_dev, const uint8_t* Wgu_scales_dev,
                                      const float* gu_bias_dev, const uint8_t* Wd_codes_dev,
                                      const uint8_t* Wd_scales_dev, const float* down_bias_dev,
                                      int E, int k, int T, int d, int I, void* out_dev,
                                      void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * moe_forward with per-call options (opts may be NULL: the process default
 * tile policy, bf16 activations, no biases). Everything else -- arguments,
 * workspace size (moe_workspace_size), errors, stream semantics -- is as in
 * moe_forward. MOE_ERR_INVALID_ARG for a tile_policy outside -1..5 or an
 * unknown act_quant; MOE_ERR_UNSUPPORTED for an act_quant the shape cannot
 * run (the quantised modes need the block-scaled tiles' shapes: d and I
 * multiples of 64 in [128, 3072], 32-byte aligned code arrays).
 * The quantised modes always run the block-scaled tiles (E2M1 weights x E4M3
 * or E2M1 activations, one term): 16-token tiles when experts average under
 * 64 rows; 256-token tiles on a CTA pair with tile_policy 5, or with 0 when
 * experts average 192 rows or more (w4a4 there runs kind::mxf4 when d and I
 * are at least 256); else 128-token tiles on one CTA.
 * Their intermediates in the workspace: the converted x rows in the xp region
 * and the converted H rows in the h region, in the padded token layout the
 * block-scaled tiles read, their scales at x_scales and h_scales.
 */
MOE_API moe_status moe_forward_ex(const void* x_dev, const float* W_r_dev, const float* b_r_dev,
                                  const uint8_t* Wgu_codes_dev, const uint8_t* Wgu_scales_dev,
                                  const uint8_t* Wd_codes_dev, const uint8_t* Wd_scales_dev,
                                  int E, int k, int T, int d, int I, void* out_dev,
                                  void* workspace_dev, size_t workspace_bytes,
                                  const moe_forward_opts* opts, void* stream);

/*
 * Same as moe_forward, instrumented: records a CUDA event on `stream` at the
 * boundaries of the pass's stages and one after the last, waits for the last
 * event, and writes to stage_ms_host[0..11] (host memory, 12 floats) the
 * device time in milliseconds of each stage, in order -- router (its weight
 * split, logits and top-k/softmax launches; for at most 256 tokens also the
 * permutation), top-k/softmax (0: inside the router stage), expert histogram,
 * scan, scatter, activation gather, the two scale transposes (gate/up, down),
 * gate/up GEMM + SwiGLU, down GEMM + weighted un-permute (on the CTA-pair
 * tiles with the launch before it that lays out the down weights' scale
 * atoms), per-token sum --
 * and in stage_ms_host[11] the span from the first launch to the end of the
 * last. A stage the pass does not launch reads as the cost of its two events.
 * Blocks the calling thread until the pass has finished.
 */
MOE_API moe_status moe_forward_timed(const void* x_dev, const float* W_r_dev, const float* b_r_dev,
                                     const uint8_t* Wgu_codes_dev, const uint8_t* Wgu_scales_dev,
                                     const uint8_t* Wd_codes_dev, const uint8_t* Wd_scales_dev,
                                     int E, int k, int T, int d, int I, void* out_dev,
                                     void* workspace_dev, size_t workspace_bytes, void* stream,
                                     float* stage_ms_host);

/*
 * moe_forward_timed with only some launch boundaries recorded, for timing
 * with less interference: each event recorded between two launches delays
 * the second by a few microseconds, which is visible on decode-sized steps.
 * Bit i of event_mask (i = 0..11) records boundary i, the event before launch
 * i in the order of moe_forward_timed (bit 11: after the last launch); bits 0
 * and 11 are always recorded, bits above 11 are an error (MOE_ERR_INVALID_ARG).
 * stage_ms_host[i] for a recorded boundary i < 11 is the device time to the
 * next recorded boundary, 0 for the others; stage_ms_host[11] is the whole
 * span. Example: bits 0, 8, 9, 11 give the gate/up GEMM alone in [8] and the
 * whole pass in [11]. Blocks the calling thread until the pass has finished.
 */
MOE_API moe_status moe_forward_timed_events(const void* x_dev, const float* W_r_dev,
                                            const float* b_r_dev, const uint8_t* Wgu_codes_dev,
                                            const uint8_t* Wgu_scales_dev,
                                            const uint8_t* Wd_codes_dev,
                                            const uint8_t* Wd_scales_dev, int E, int k, int T,
                                            int d, int I, void* out_dev, void* workspace_dev,
                                            size_t workspace_bytes, void* stream,
                                            unsigned int event_mask, float* stage_ms_host);

/*
 * moe_forward_timed_events with per-call options (opts as in moe_forward_ex;
 * NULL: the defaults). Same timing semantics, errors and blocking.
 */
MOE_API moe_status moe_forward_timed_ex(const void* x_dev, const float* W_r_dev,
                                        const float* b_r_dev, const uint8_t* Wgu_codes_dev,
                                        const uint8_t* Wgu_scales_dev, const uint8_t* Wd_codes_dev,
                                        const uint8_t* Wd_scales_dev, int E, int k, int T, int d,
                                        int I, void* out_dev, void* workspace_dev,
                                        size_t workspace_bytes, const moe_forward_opts* opts,
                                        void* stream, unsigned int event_mask,
                                        float* stage_ms_host);

/*
 * Same as moe_forward with the activations in host memory: copies x_host
 * (T*d*2 bytes; pinned memory gives asynchronous copies) to the workspace,
 * runs the forward pass and copies the result to out_host, then synchronises
 * `stream`. Expert and router weights stay on the device (the layer's
 * resident parameters). moe_workspace_size_hostio() gives the workspace size.
 * Batches of at least 2048 tokens are processed as 4 chunks of tokens (each
 * token's output depends on that token alone, so the result is the same):
 * the copy in, the forward and the copy out of neighbouring chunks overlap on
 * two copy streams the library creates once per device, ordered after the
 * caller's earlier work on `stream`. Host threads may call it concurrently on
 * one device (with separate workspaces): they take turns at enqueueing and
 * share the copy streams. If a launch or a copy fails, the call waits for the
 * copies it had enqueued before it returns the error. The call returns the
 * device status of the pass itself: each chunk keeps its own status word
 * (chunk c uses 32-bit word c of the 16-byte status block at the workspace's
 * start), so a timeout in any chunk is returned. moe_workspace_size_hostio()
 * is at least moe_workspace_size(), so one workspace serves both calls.
 */
MOE_API size_t moe_workspace_size_hostio(int E, int k, int T, int d, int I);
MOE_API moe_status moe_forward_hostio(const void* x_host, const float* W_r_dev, const float* b_r_dev,
                              const uint8_t* Wgu_codes_dev, const uint8_t* Wgu_scales_dev,
                              const uint8_t* Wd_codes_dev, const uint8_t* Wd_scales_dev,
                              int E, int k, int T, int d, int I, void* out_host,
                              void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * Router and permutation only (the first two steps of the path): router
 * logits in fp32, top-k with the lower-index tie rule, selected-set softmax
 * ("Proof", s_i and p_i), then the stable grouping of the T*k (token, slot)
 * pairs by expert.
 *
 * Precision of the choice: the logits are fp32 dot products on the tensor
 * cores (the fp32 router weights as three bf16 terms, exactly). Where two
 * neighbouring logits of a token's top-k list, or the k-th and a runner-up,
 * lie within tau_t = 2^-17 ||x_t||_2 max_e ||W_r[e]||_2 of each other, their
 * order is decided on fp64 dot products of the same inputs; so the experts
 * and their order are those of the exact logits, equal exact logits going to
 * the lower index. The softmax uses the fp32 logits (the fp64 ones where
 * they were computed). moe_forward leaves the fp32 logits in its workspace
 * (moe_workspace_layout's logits, [T][E]).
 *
 *   topk_idx_dev [T][k] int32, topk_w_dev [T][k] float32
 *   counts_dev   [E]    int32  pairs routed to each expert
 *   offsets_dev  [E+1]  int32  exclusive prefix sum of counts
 *   perm_dev     [T*k]  int32  pair ids (t*k + j) grouped by expert, in
 *                              ascending pair id inside each expert
 * Any of counts/offsets/perm may be NULL to skip the permutation outputs
 * (all three NULL, or none). workspace size: moe_route_workspace_size().
 */
MOE_API size_t moe_route_workspace_size(int E, int k, int T, int d);
MOE_API moe_status moe_route(const void* x_dev, const float* W_r_dev, const float* b_r_dev,
                     int E, int k, int T, int d,
                     int32_t* topk_idx_dev, float* topk_w_dev,
                     int32_t* counts_dev, int32_t* offsets_dev, int32_t* perm_dev,
                     void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * moe_route without a workspace, for callers that cannot allocate device
 * memory: code that is handed only its inputs, outputs and a stream (plugin
 * hooks of inference runtimes, serving threads that must not call cudaMalloc,
 * which can synchronise the device and can fail under memory pressure). The
 * pages have no counterpart to this entry point; it is a deployment aid.
 *
 * Same arguments, outputs and results as moe_route (all five outputs are
 * required here), minus the workspace; it makes the same launches as
 * moe_route, so its results are bit-identical to moe_route's. The scratch it
 * needs (router logits, the router's split weights and small routing tables)
 * lives in one device array owned by the library: 32.1 MiB that every GPU
 * which loads the library holds until the process exits. Limit: T * E <= 1,048,576 (e.g. T = 8192 tokens at E = 128,
 * or T = 4096 at E = 248); larger calls return MOE_ERR_UNSUPPORTED and
 * launch nothing. Every call looks up the array's device address on the
 * current device (cudaGetSymbolAddress; no address is cached, so a new
 * primary context or a device reset needs nothing from the caller); the
 * first call on a device also loads the library's device code there, so
 * make that first call before any stream capture. All calls on a device share the array and
 * it keeps the last call's contents (each call rewrites what it reads), so
 * calls whose device work overlaps -- concurrent streams, or several host
 * threads -- race on it; serialise them.
 */
MOE_API moe_status moe_route_noalloc(const void* x_dev, const float* W_r_dev, const float* b_r_dev,
                                     int E, int k, int T, int d, int32_t* topk_idx_dev,
                                     float* topk_w_dev, int32_t* counts_dev,
                                     int32_t* offsets_dev, int32_t* perm_dev, void* stream);

/*
 * Where moe_forward keeps its intermediates inside the workspace (byte
 * offsets from the workspace base), so that a caller can read them after a
 * call for inspection: logits [T][E] f32, topk_idx [T][k] i32, topk_w [T][k]
 * f32, counts [E] i32, offsets [E+1] i32, perm [T*k] i32 (pair id at each
 * permuted row), xp [T*k][d] bf16 (permuted activations), h [T*k][I] bf16
 * (SwiGLU hidden rows in permuted order), yw [T*k][d] fp32 (p-weighted expert
 * outputs in pair order t*k+j). Rows of xp and h keep each run of 8
 * consecutive elements in the order 0,4,1,5,2,6,3,7 (the operand order of the
 * grouped GEMMs). Returns MOE_ERR_INVALID_ARG for bad shapes.
 */
typedef struct {
  size_t logits, topk_idx, topk_w, counts, offsets, perm, xp, h, yw, status, total;
  /* the block-scaled tiles' B-scale blocks of the x rows and of the H rows
   * (E8M0 bytes in the layout the GEMMs copy into tensor memory) */
  size_t x_scales, h_scales;
} moe_ws_layout;
MOE_API moe_status moe_workspace_layout(int E, int k, int T, int d, int I, moe_ws_layout* layout);

/*
 * The activation split of the block-scaled tiles (tile policy 4), on plain
 * rows: x_dev [rows][K] bf16 -> hi_dev, lo_dev [rows][K] E4M3 bytes and
 * scales_dev [rows][K/32][2] E8M0 bytes (hi, lo) such that, per group of 32,
 * x = 2^(s_hi-127) e4m3(hi) + 2^(s_lo-127) e4m3(lo), exactly for every
 * element of at least 2^-13 of the group's max |x| and within 2^-21 of that
 * max otherwise (for groups whose max |x| is at least 2^-116). The pages have no counterpart: the split only lets bf16
 * activations enter the tensor core's block-scaled MMA kind next to E2M1
 * weights ("Four-bit expert weights"). K a multiple of 32; x_dev, hi_dev and
 * lo_dev 16-byte aligned. All buffers are the caller's.
 */
MOE_API moe_status moe_mx_split_e4m3(const void* x_dev, int rows, int K, uint8_t* hi_dev,
                                     uint8_t* lo_dev, uint8_t* scales_dev, void* stream);

/*
 * The activation conversion of the quantised modes (moe_forward_opts.act_quant)
 * on plain rows, with the kernels the layer uses: x_dev [rows][K] bf16 ->
 * q_dev [rows][K] E4M3 bytes (MOE_ACT_MXFP8) or [rows][K/2] packed E2M1 codes
 * (MOE_ACT_MXFP4; byte b holds element 2b in its low nibble, as the weights),
 * and scales_dev [rows][K/32] E8M0 bytes, per group of 32: the OCP
 * Microscaling conversion (v1.0, section 6.3) with shared scale
 * 2^(floor(log2 max|x|) - emax), emax 8 (E4M3) or 2 (E2M1), elements rounded
 * to nearest even and clamped to the largest normal. A group whose max|x| is
 * below 2^(emax - 127) keeps the smallest scale byte, 0; an all-zero group
 * gets byte 127 and zero codes. The pages have no counterpart: they put only
 * the expert weights in MXFP4 ("Four-bit expert weights"). K a multiple of 32;
 * x_dev and q_dev 16-byte aligned; all buffers the caller's.
 */
MOE_API moe_status moe_mx_quantize(const void* x_dev, int rows, int K, int act_quant,
                                   uint8_t* q_dev, uint8_t* scales_dev, void* stream);

/*
 * Decode MXFP4 rows to bf16 on the device with the same decoder the grouped
 * GEMMs use ("Four-bit expert weights"). codes_dev [rows][K/2], scales_dev
 * [rows][K/32] -> out_dev [rows][K] bf16. K must be a multiple of 32.
 */
MOE_API moe_status moe_mxfp4_to_bf16(const uint8_t* codes_dev, const uint8_t* scales_dev,
                             int rows, int K, void* out_dev, void* stream);

/*
 * Synchronise `stream`, then read and clear the device status word in the
 * workspace. Returns MOE_OK, or MOE_ERR_TIMEOUT when a kernel gave up a wait.
 */
MOE_API moe_status moe_sync_status(void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * Failure-detection self-test: enqueues one kernel whose only thread waits,
 * with the same bounded wait the GEMM roles use, on an mbarrier that nothing
 * completes. After about two seconds the wait gives up and stores
 * MOE_ERR_TIMEOUT in the status word at the start of workspace_dev (16 bytes
 * suffice), which moe_sync_status() then returns. Nothing hangs or faults.
 */
MOE_API moe_status moe_selftest_wait_timeout(void* workspace_dev, void* stream);

/*
 * The MoE sublayer of a decoder block with its pre-norm and residual add
 * (field guide "gpt-oss 20B", "04 One decoder block": RMSNorm is applied
 * before the MoE and the sublayer is added back to the residual stream):
 *   x   = bf16((h / sqrt(mean(h^2) + eps)) * g)   per row (moe_rms_norm)
 *   out = bf16(h + sum_j p_j E_j(x))              (one rounding, after the add)
 * h_dev [T][d] bf16 (the residual stream), g_dev [d] f32 (the norm's gain),
 * eps >= 0 (the pages give no value; gpt-oss configurations commonly use
 * 1e-5); gu_bias_dev and down_bias_dev (each may be NULL) are the experts'
 * biases as in moe_forward_biased. All other arguments, the result, the errors
 * and the stream semantics are those of moe_forward; the workspace must hold
 * moe_workspace_size_block(...) bytes (moe_forward's, plus the x rows).
 * moe_forward_launch_count(...) + 1 launches.
 */
MOE_API size_t moe_workspace_size_block(int E, int k, int T, int d, int I);
MOE_API moe_status moe_forward_block(const void* h_dev, const float* g_dev, float eps,
                                     const float* W_r_dev, const float* b_r_dev,
                                     const uint8_t* Wgu_codes_dev, const uint8_t* Wgu_scales_dev,
                                     const float* gu_bias_dev, const uint8_t* Wd_codes_dev,
                                     const uint8_t* Wd_scales_dev, const float* down_bias_dev,
                                     int E, int k, int T, int d, int I, void* out_dev,
                                     void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * The pre-MoE RMSNorm alone: x_dev[t] = bf16((h[t] / sqrt(mean(h[t]^2) + eps)) * g),
 * h_dev and x_dev [T][d] bf16, g_dev [d] f32; d a multiple of 32; all three
 * 16-byte aligned and the caller's. Per row: fp32 sum of squares (a fixed
 * lane-strided order), IEEE sqrt and division, one rounding to bf16.
 */
MOE_API moe_status moe_rms_norm(const void* h_dev, const float* g_dev, float eps, int T, int d,
                                void* x_dev, void* stream);

/*
 * Number of kernel launches one moe_forward call enqueues for this shape
 * under the current tile policy (0 for T = 0), assuming 32-byte aligned code
 * arrays. Used to count device work per step.
 */
MOE_API int moe_forward_launch_count(int E, int k, int T, int d, int I);

/*
 * ------------------------------------------------------ training the router
 * The gradients a user needs to train the router (W_r, b_r) around frozen MXFP4
 * experts, next to the forward pass that leaves what they read:
 * moe_workspace_layout's logits, topk_idx, topk_w and yw, or moe_route's outputs;
 * and the norm's, for what reaches it. Order of a backward pass for the sublayer
 * out = h + MoE(RMSNorm(h)), given dout [T][d]:
 *   moe_gate_backward           dlogits from dout and the weighted expert rows
 *   moe_balance_loss(_backward) the auxiliary loss, added to dlogits
 *   moe_router_backward         dW_r, db_r and dx = dlogits W_r (+ dx_in)
 *   moe_rms_norm_backward       dg and dh = dh_in + d/dh of the norm
 * dW_r, db_r and the auxiliary loss need nothing else. The gradient that reaches x
 * through the frozen experts is not computed: dg, and dh beyond dh_in, are the
 * sublayer's only if the caller passes that share as dx_in; without it they hold
 * the path through the logits alone, and the gain and what lies before the
 * sublayer cannot be trained on them.
 *
 * Shared by these entry points:
 * - T tokens, E, k and d within the range above (1 <= E <= 256, k <= min(E, 32),
 *   d a multiple of 32 up to 16384). Arrays whose size is a multiple of T may
 *   be NULL when T is 0; sums over no tokens are zero.
 * - token_mask_dev [T] uint8, or NULL: a token whose byte is 0 (padding) is
 *   left out of every sum and count, and none of its floating-point inputs
 *   (logits, rows, gradients) changes a result, whatever they hold.
 * - accumulate (0 or 1): add to the output instead of overwriting it.
 * - A workspace needs no initialisation and may be shared by calls that run one
 *   after another. Its first word is moe_router_backward's status (0, or
 *   MOE_ERR_TIMEOUT if one of its bounded waits gave up: moe_sync_status); no
 *   other call writes it.
 * - A call reads and writes nothing but its arguments: calls on different
 *   streams with workspaces of their own may run at the same time, and each may
 *   be captured into a CUDA graph.
 * - A NaN or an infinity in a live token's inputs shows as NaN (or infinity) in
 *   the outputs that depend on it; a logits' gradient beyond bf16's largest value
 *   (3.39e38) may count as an infinity in moe_router_backward's dW.
 * - Every sum over tokens has a fixed order: the same call gives the same bits.
 */

/*
 * Load-balance and z loss of a batch's router logits, with the per-expert
 * counts. (Even routing has balance 1 whatever k is; a coefficient chosen for a loss
 * with f_e = counts_e / n is to be multiplied by k here.)
 * Over the n live tokens, with p_t = softmax(logits_t) over all E:
 *   f_e = counts_e / (n k),  P_e = (1/n) sum_t p_{t,e},
 *   balance = E sum_e f_e P_e,  z = (1/n) sum_t lse(logits_t)^2,
 *   loss = balance_coef * balance + z_coef * z.
 *   logits_dev     [T][E] f32    topk_idx_dev [T][k] i32
 *   stats_dev      [4]    f32    loss, balance, z, n
 *   counts_dev     [E]    i32    live (token, slot) pairs of each expert
 *   mean_probs_dev [E]    f32    P
 *   lse_dev        [T]    f32    log sum exp of each row (0 for padded tokens)
 * An index outside 0..E-1 (a dropped pair, say -1) is not counted. A logit of
 * -inf has probability 0; a row of nothing but -inf adds nothing to P and z
 * (its lse is -inf) and gets no gradient. NaN and +inf in a live row give NaN.
 * Sums over tokens: of p T / 4096 + 32 terms at most in fp32, their sums and those of
 * lse^2 in fp64; balance and z enter the loss unrounded (a z beyond fp32's range is an
 * infinity in stats, and no NaN in the loss where z_coef is 0).
 */
MOE_API size_t moe_balance_loss_workspace_size(int E, int k, int T);
MOE_API moe_status moe_balance_loss(const float* logits_dev, const int32_t* topk_idx_dev,
                                    const uint8_t* token_mask_dev, int E, int k, int T,
                                    float balance_coef, float z_coef, float* stats_dev,
                                    int32_t* counts_dev, float* mean_probs_dev, float* lse_dev,
                                    void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * Gradient of that loss to the logits (the counts are constants):
 *   dlogits[t,e] (+)= (dloss / n) p_{t,e} (balance_coef E (f_e - sum_e' f_e' p_{t,e'})
 *                                          + 2 z_coef lse_t)
 * lse, counts and stats as moe_balance_loss left them (n is stats[3]), the same
 * mask and coefficients; dloss_dev: one f32, the gradient of the loss itself,
 * or NULL for 1. dlogits_dev [T][E] f32; rows of padded tokens are set to 0
 * (left alone with accumulate).
 */
MOE_API moe_status moe_balance_loss_backward(const float* logits_dev, const float* lse_dev,
                                             const int32_t* counts_dev, const float* stats_dev,
                                             const uint8_t* token_mask_dev, int E, int k, int T,
                                             float balance_coef, float z_coef,
                                             const float* dloss_dev, int accumulate,
                                             float* dlogits_dev, void* stream);

/*
 * Gradient to the logits through the selected-set softmax and the weighted sum
 * out_t = sum_j p_j y_j: with A_j = <dout_t, p_j y_j> (fp32),
 *   dlogits[t, topk_idx_j] (+)= A_j - p_j sum_l A_l,   0 for the other experts,
 * formed as sum_l (p_l A_j - p_j A_l), the same since a token's weights sum to 1: off
 * by roundings of these products only, however close to 1 a weight is.
 *   dout_dev [T][d] bf16   gradient of the layer's output
 *   yw_dev   [T*k][d] f32  p-weighted expert rows in pair order t*k+j, as a
 *                          forward call leaves them (moe_workspace_layout's yw)
 *   topk_idx_dev [T][k] i32, topk_w_dev [T][k] f32 (p)
 * p enters only as a factor, so weights that underflowed to 0 are no case of
 * their own. Pairs whose index lies outside 0..E-1 get no gradient of their
 * own; an index that a row holds twice collects both.
 */
MOE_API moe_status moe_gate_backward(const void* dout_dev, const float* yw_dev,
                                     const int32_t* topk_idx_dev, const float* topk_w_dev,
                                     const uint8_t* token_mask_dev, int E, int k, int T, int d,
                                     int accumulate, float* dlogits_dev, void* stream);

/*
 * Gradients of the router product s = x W_r^T + b_r:
 *   dW[e] (+)= sum_t dlogits[t,e] x_t,  db[e] (+)= sum_t dlogits[t,e],
 *   dx[t] = bf16(sum_e dlogits[t,e] W_r[e] + dx_in[t])     (one rounding)
 * The rows come as x_dev [T][d] bf16, or (x_dev NULL) are rebuilt from the
 * checkpoint of moe_rms_norm_checkpoint as q 2^(s-127) rstd_t g: q_dev [T][d]
 * E4M3, scales_dev [T][d/32] E8M0, rstd_dev [T] f32, g_dev [d] f32 (all four,
 * or all four NULL).
 * dW_dev [E][d] f32, db_dev [E] f32, dx_dev [T][d] bf16: each may be NULL (not
 * computed; without dW no rows are read). dx_in_dev [T][d] bf16 or NULL, may
 * be dx_dev itself (no other output may overlap an input); accumulate concerns
 * dW and db. A padded token's dx row is its dx_in row (0 without one), whatever
 * W_r holds.
 * dW and db: fp32 products and sums (above 96 to 144 tokens on the tensor cores,
 * dlogits in three bf16 terms: nothing of its 24 bits is lost above 2^-110; of 8-bit
 * rows that holds for the product dlogits rstd, which is rounded to fp32 first).
 * dx: below that an fp32 product; on the tensor cores dlogits and W_r enter as two
 * fp16 terms, 22 bits. Before its rounding to bf16 it is off by at most
 * (2^-20 + 3 E 2^-27) sum_e |dlogits W_r|, the second part for the additions, plus
 * what values far below their neighbours lose: of a token's dlogits 2^-39 of the
 * largest (or 2^-151) times |W_r|, of W_r as much of its largest times |dlogits|.
 */
MOE_API size_t moe_router_backward_workspace_size(int E, int T, int d);
MOE_API moe_status moe_router_backward(const float* dlogits_dev, const float* W_r_dev,
                                       const void* x_dev, const uint8_t* q_dev,
                                       const uint8_t* scales_dev, const float* rstd_dev,
                                       const float* g_dev, const uint8_t* token_mask_dev, int E,
                                       int T, int d, const void* dx_in_dev, int accumulate,
                                       float* dW_dev, float* db_dev, void* dx_dev,
                                       void* workspace_dev, size_t workspace_bytes, void* stream);

/*
 * moe_rms_norm that keeps what its backward pass and moe_router_backward read:
 * the input rows as an 8-bit checkpoint instead of h and x in bf16 (1.03 bytes
 * per element instead of 4).
 *   x_dev [T][d] bf16: as moe_rms_norm, bit for bit; NULL: not written
 *   q_dev [T][d] E4M3, scales_dev [T][d/32] E8M0: h as moe_mx_quantize with
 *         MOE_ACT_MXFP8 converts it, byte for byte
 *   rstd_dev [T] f32: 1 / sqrt(mean(h_t^2) + eps)
 * A NaN in a row makes its rstd NaN, and with it all that is computed from the
 * checkpoint. Where the sum of squares is infinite in fp32 (an infinity in h, or
 * values above 1.8e19) rstd is 0 and x moe_rms_norm's, q holds the largest code for
 * an infinity, and the row counts as zeros to the backward pass.
 */
MOE_API moe_status moe_rms_norm_checkpoint(const void* h_dev, const float* g_dev, float eps, int T,
                                           int d, void* x_dev, uint8_t* q_dev,
                                           uint8_t* scales_dev, float* rstd_dev, void* stream);

/*
 * Backward of the norm, n = h rstd:
 *   dh[t] = bf16(dh_in[t] + rstd_t (g dx_t - n_t mean(n_t g dx_t)))
 *   dg    (+)= sum_t dx_t n_t
 * dx_dev [T][d] bf16; rows h_dev [T][d] bf16, or (h_dev NULL) the checkpoint's
 * q_dev and scales_dev; dh_in_dev [T][d] bf16 (the residual's gradient) or
 * NULL. dh_dev [T][d] bf16 may be dx_dev or dh_in_dev; dg_dev [d] f32. A
 * padded token's dh row is its dh_in row (0 without one).
 */
MOE_API size_t moe_rms_norm_backward_workspace_size(int T, int d);
MOE_API moe_status moe_rms_norm_backward(const void* dx_dev, const void* h_dev,
                                         const uint8_t* q_dev, const uint8_t* scales_dev,
                                         const float* rstd_dev, const float* g_dev,
                                         const uint8_t* token_mask_dev, int T, int d,
                                         const void* dh_in_dev, int accumulate, void* dh_dev,
                                         float* dg_dev, void* workspace_dev,
                                         size_t workspace_bytes, void* stream);

/*
 * moe_forward_block whose norm also leaves the checkpoint (q_dev, scales_dev,
 * rstd_dev as moe_rms_norm_checkpoint): the training form of the sublayer.
 * Same arguments, output bits, errors and launches otherwise (no array may be
 * NULL, T = 0 or not, as there); the logits,
 * choices, weights and weighted rows that the backward pass reads stay in the
 * workspace (moe_workspace_layout) until its next use.
 */
MOE_API moe_status moe_forward_block_checkpoint(
    const void* h_dev, const float* g_dev, float eps, const float* W_r_dev, const float* b_r_dev,
    const uint8_t* Wgu_codes_dev, const uint8_t* Wgu_scales_dev, const float* gu_bias_dev,
    const uint8_t* Wd_codes_dev, const uint8_t* Wd_scales_dev, const float* down_bias_dev, int E,
    int k, int T, int d, int I, void* out_dev, uint8_t* q_dev, uint8_t* scales_dev,
    float* rstd_dev, void* workspace_dev, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_B200_H */
