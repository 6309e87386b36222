/*
 * xp.h -- C ABI of the GB300 (sm_103a) XPress Jacobi refinement pass.
 *
 * One pass over a batch of N draft blocks of B slots (slot 0 = the verified
 * anchor) computes, for every slot b:
 *   latent   x[b] = xh[b] + W_lat w1[prev[b]],  prev[0] = am1, prev[b] = blk[b-1]
 *            u[b] = sum_{j<=b} mix[c,b,j] x[j]  (per channel c, folded mixer)
 *            lat[b] = u[b] + W_down (silu(W_gate u[b]) * (W_up u[b]))
 *   readout  logits[b, v] = base[b, v] + lat[b] . w2[v]
 *   argmax   blk[b] = argmax_v logits[b, v], written in place for the next pass
 * for the draft slots b = 1..B-1, and repeats that K times (Jacobi iteration).
 *
 * Sources: the vLLM API page of vllm.model_executor.models.qwen3_xpress
 * ("qwen3_xpress page": XPressRefinerHead and its methods) and the vLLM API
 * page of vllm.v1.worker.gpu.spec_decode.xpress.kernels ("xpress kernels
 * page": the docstrings of the per-pass kernels).
 *
 * Conventions (all entry points):
 *  - Memory is owned by the caller.  The library never allocates device
 *    memory; pointers marked "device" must be device (or managed) memory,
 *    pointers marked "host" host memory.  Sizes are element counts unless
 *    stated otherwise.
 *  - Every call is asynchronous on the given stream (0 = legacy default) and
 *    performs no host synchronisation, except xp_get_error and
 *    xp_head_create/xp_head_refill (which synchronise nothing either, but
 *    read device properties).  Host-side validation runs before any launch;
 *    a call that returns an error has launched nothing.
 *  - A head belongs to the device that was current when it was created.  Every
 *    call that takes a head refuses (XP_EINVAL) while another device is current.
 *  - Calls that take a workspace also take its size in bytes; a workspace smaller
 *    than the call needs (xp_workspace_bytes for that N and topc) is refused with
 *    XP_ECAPACITY before anything is launched.
 *  - Token ids are int64 at the boundary.  A token id outside [0, V) read by
 *    a kernel is clamped into range and raises XP_EBADTOKEN in the head's
 *    device error word (read with xp_get_error); kernels never trap.
 *  - Dtypes: the head's weights, base logits, h and latents all share the
 *    head dtype (XP_BF16 or XP_F32); accumulation is fp32 throughout.
 *  - Argmax ties go to the lowest vocabulary id (full vocabulary, init and
 *    top-C alike); -0 compares equal to +0.  Inputs are assumed finite.
 */
#ifndef XP_H_
#define XP_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  XP_OK = 0,
  XP_EINVAL = 1,        /* null pointer, bad shape, bad stride or alignment            */
  XP_ECAPACITY = 2,     /* N above the head's max_N, or a buffer too small             */
  XP_ENOTPREPARED = 3,  /* head missing (the weights were never prepared)              */
  XP_ECUDA = 4,         /* a CUDA runtime call failed (launch, copy, attribute)        */
  XP_EBADTOKEN = 5,     /* device flag: a token id outside [0, V) was clamped          */
  XP_ETIMEOUT = 6,      /* device flag: a bounded wait inside a kernel gave up         */
  XP_EUNSUPPORTED = 7,  /* shape not supported by this build                           */
  XP_ERANGE = 8,        /* device flag: a latent-stage value left the fp16 range of the
                           tensor-core latent's exchanges (saturated; results unreliable), or a
                           row written to a quantised cache held NaN or more than it can hold   */
  XP_EBADPAGE = 9,      /* device flag: a page id outside the pool (clamped when read, ignored
                           when freed) or a page freed more often than it was held        */
  XP_ENOPAGES = 10,     /* device flag: the pool ran out of free pages; rows were cut short */
  XP_ESHARED = 11,      /* device flag: a resize would have ended inside a shared page; the
                           row was left as it was                                          */
  XP_ELENGTH = 12,      /* device flag: a length or a row number outside its range was clamped */
  XP_EEMPTY = 13        /* device flag: a target row left no token to draw (token -1)      */
} xp_status;

/* XP_Q8 and XP_Q4 are types of paged caches alone (see xp_cache_desc). */
typedef enum { XP_BF16 = 0, XP_F32 = 1, XP_Q8 = 2, XP_Q4 = 3 } xp_dtype;

/* Head weights, torch layouts ([out, in] row-major for linear maps).  All
 * pointers are device pointers, read only during xp_head_create /
 * xp_head_refill (they are copied into the head's prepared memory).
 * qwen3_xpress page, XPressRefinerHead.__init__. */
typedef struct {
  int V;          /* vocabulary size                                   */
  int hidden;     /* target-model hidden size                          */
  int r;          /* refiner rank (latent width)                       */
  int H;          /* SwiGLU hidden size (mlp_hidden)                   */
  int B;          /* block size (slots per draft block, >= 2)          */
  int max_N;      /* most blocks any call will pass (max_num_reqs)     */
  xp_dtype dtype; /* storage type of every tensor below                */
  const void* w1;       /* [V, r]       token embedding                     */
  const void* down_h;   /* [r, hidden]                                      */
  const void* down_g;   /* [r, hidden]                                      */
  const void* in_proj;  /* [r, 3r]      columns: down_h | down_g | embedding */
  const void* mix_L;    /* [r, B, B]    FOLDED mixer (raw*tril + I), index  */
                        /*              [channel, out slot, in slot]        */
  const void* w_gate;   /* [H, r]                                           */
  const void* w_up;     /* [H, r]                                           */
  const void* w_down;   /* [r, H]                                           */
  const void* w2;       /* [V, r]       readout                             */
} xp_weights;

typedef struct xp_head xp_head; /* opaque, host-side */

/* Device bytes the head's prepared copies need (caller allocates them once).
 * Beyond copies of the weights (about 2 * V * r * es for w1 and w2), a bf16 head with
 * r = 256 and H = 512 also keeps the projected embedding table E = w1 . W_lat^T in
 * fp32, V * r * 4 bytes (155 MB at V = 151936), so that each pass gathers one row of
 * it per slot instead of multiplying W_lat; and the folded hidden-cache projection
 * as two bf16 planes, 2 * 2r * hidden * 2 bytes (8 MB at hidden = 4096). */
size_t xp_head_prep_bytes(const xp_weights* w);

/* Device bytes of the per-call workspace for up to N blocks; topc > 0 adds
 * the candidate buffers of the top-C path for C = min(topc, V): cand and base_c,
 * plus w2c only where xp_jacobi_refine copies the candidates' w2 rows (while
 * N*(B-1)*C <= V; beyond that each pass reads them by id from w2). */
size_t xp_workspace_bytes(const xp_weights* w, int N, int topc);

/* Zero a workspace once after allocating it.  The argmax finish keeps its
 * counters at zero between calls; after XP_ETIMEOUT, zero it again. */
xp_status xp_workspace_init(void* ws, size_t ws_bytes, cudaStream_t stream);

/* Copy and lay out the weights into prep_dev (device, prep_bytes >=
 * xp_head_prep_bytes) and return a host handle.  qwen3_xpress page,
 * process_weights_after_loading: prepared copies the kernels index directly. */
xp_status xp_head_create(const xp_weights* w, void* prep_dev, size_t prep_bytes,
                         cudaStream_t stream, xp_head** out);

/* Refill the prepared copies in place from new weights of the same shapes, so
 * that captured CUDA graphs keep their addresses (process_weights_after_loading
 * on a reload). */
xp_status xp_head_refill(xp_head* head, const xp_weights* w, cudaStream_t stream);

void xp_head_destroy(xp_head* head);

/* mix_L[c,b,j] = raw_L[c,b,j] * [j <= b] + [j == b], evaluated in fp64 and
 * rounded once to dtype.  raw_L, mix_L: device [r, B, B].
 * qwen3_xpress page, XPressRefinerHead.fold_from_raw_. */
xp_status xp_fold_mix(const void* raw_L, void* mix_L, int r, int B, xp_dtype dtype,
                      cudaStream_t stream);

/* Pass-invariant hidden half of in_proj, once per draft step:
 *   xh[n,b] = in_proj[:, :2r] . [down_h h[n,b] ; down_g mean_b' h[n,b']]
 * h_full: device [N, B, hidden] (head dtype); xh: device [N, B, r] fp32.
 * ws: workspace of ws_bytes >= xp_workspace_bytes(w, N, 0).
 * qwen3_xpress page, hidden_cache and the xh hoist in jacobi_refine_greedy. */
xp_status xp_hidden_cache(const xp_head* head, const void* h_full, int N, float* xh,
                          void* ws, size_t ws_bytes, cudaStream_t stream);

/* Latent stage of one pass (all slots), written for slots 1..B-1:
 * blk: device [N, B] int64; am1: device [N] int64; xh: device [N, B, r] fp32;
 * lat: device [N, B-1, r] head dtype (written).
 * Precision of the bf16 tensor-core path (r = 256, H = 512): the mixed latent u
 * and the down projection's partial sums cross between CTAs as fp16 (relative
 * error 2^-11, about a quarter of the bf16 output rounding); the SwiGLU
 * activations are carried as bf16 hi + lo pairs; everything else is fp32.  A value
 * outside the fp16 range saturates and raises XP_ERANGE.
 * xpress kernels page, _xpress_latent_kernel; qwen3_xpress page, _refine_latent. */
xp_status xp_latent_pass(const xp_head* head, const int64_t* blk, const int64_t* am1,
                         const float* xh, int N, void* lat, cudaStream_t stream);

/* Readout + argmax straight into the block:
 *   blk[n, 1+b] = argmax_v (base[n,b,v] + lat[n,b] . w2[v]),  b = 0..B-2
 * lat: device [N, B-1, r] head dtype.  base: device, draft row (n, b) starts
 * at base + n*stride_n + b*stride_b (elements), unit stride over v.  blk:
 * device [N, B] int64, slots 1..B-1 written.  win_val: device [N*(B-1)]
 * fp32 winning logits, or NULL.  ws: workspace of ws_bytes >=
 * xp_workspace_bytes(w, N, 0) (argmax partials).
 * The [N*(B-1), V] logits are never written to memory.
 * xpress kernels page, fused_add_argmax_to_blk; qwen3_xpress page, refine_bias. */
xp_status xp_readout_argmax(const xp_head* head, const void* lat, const void* base,
                            int64_t stride_n, int64_t stride_b, int N, int64_t* blk,
                            float* win_val, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Unfused readout: the draft rows' logits (or the refiner bias alone) instead of
 * their argmax, for callers that sample or otherwise need the distribution:
 *   out[n*(B-1) + b, v] = base[n,b,v] + lat[n,b] . w2[v]   (base given)
 *   out[n*(B-1) + b, v] = lat[n,b] . w2[v]                 (base == NULL)
 * for b = 0..B-2 (the draft slots 1..B-1; slot 0 holds the anchor, whose bias
 * the method never reads).  lat and base as for xp_readout_argmax; base may be
 * NULL.  out: device fp32, row r of the N*(B-1) rows at out + r*ld_out, ld_out
 * >= V elements; the caller owns it (N*(B-1)*ld_out*4 bytes).  Products are
 * accumulated in fp32 and the base value is added in fp32: out is the exact
 * logit up to fp32 rounding, not rounded to the head dtype.  No workspace.
 * XP_EINVAL: null lat/out, ld_out < V, negative N or strides.
 * qwen3_xpress page, refine_bias (w2 applied to the refined latent) and the
 * base + bias sum that fused_add_argmax_to_blk reduces. */
xp_status xp_refine_logits(const xp_head* head, const void* lat, const void* base,
                           int64_t stride_n, int64_t stride_b, int N, float* out,
                           int64_t ld_out, cudaStream_t stream);

/* xp_readout_argmax for callers that cannot allocate device memory -- no
 * counterpart on the pages; the refinement method itself says nothing about
 * where scratch lives.  Same arguments and results as xp_readout_argmax,
 * without the workspace: the cross-CTA argmax scratch (48 KB) is a fixed array
 * in the library's device memory, present on every GPU that loads the library
 * until the process exits.  Meant for callers that run inside a memory pool
 * they do not own, or on a path where cudaMalloc and the synchronisation it can
 * bring are not acceptable.  Limit: N*(B-1) <= 4096 draft rows, else
 * XP_ECAPACITY.  The first call on a device looks the array up (once per
 * device, on the current device); make that first call before any stream
 * capture.  All calls share the one array, so calls that overlap on the GPU
 * (other streams, other threads) race; each call clears it before use. */
xp_status xp_readout_argmax_noalloc(const xp_head* head, const void* lat, const void* base,
                                    int64_t stride_n, int64_t stride_b, int N, int64_t* blk,
                                    float* win_val, cudaStream_t stream);

/* Initial block: blk[n,0] = anchor[n], blk[n,1+b] = argmax_v base[n,b,v].
 * Same base addressing and workspace as xp_readout_argmax.  anchor: device [N] int64.
 * qwen3_xpress page, jacobi_refine_greedy (before the passes). */
xp_status xp_init_argmax(const xp_head* head, const void* base, int64_t stride_n,
                         int64_t stride_b, const int64_t* anchor, int N, int64_t* blk,
                         float* win_val, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Top-C candidates, once per draft step.  Per draft row: the C largest base
 * values (ties at the boundary to the lower id), stored in ascending id order:
 * cand: device [N, B-1, C] int64; base_c: device [N, B-1, C] head dtype;
 * w2c: device [N, B-1, C, r] head dtype = w2[cand] rows, or NULL to have the
 * top-C readout gather w2 rows itself each pass.  blk: device [N, B] int64 or
 * NULL; when given, slots 1..B-1 receive the base argmax (the init).
 * 1 <= C <= V.  qwen3_xpress page, jacobi_refine_greedy top-C branch. */
xp_status xp_topc_gather(const xp_head* head, const void* base, int64_t stride_n,
                         int64_t stride_b, int N, int C, int64_t* cand, void* base_c,
                         void* w2c, int64_t* blk, cudaStream_t stream);

/* Top-C readout + argmax, per pass:
 *   blk[n, 1+b] = cand[n,b,k*],  k* = argmax_k (base_c[n,b,k] + w2c[n,b,k] . lat[n,b])
 * ties to the lowest vocabulary id.  w2c may be NULL (rows gathered from the
 * head's w2 through cand).  win_val: device [N*(B-1)] fp32 or NULL.
 * xpress kernels page, _xpress_topc_argmax_to_blk_kernel. */
xp_status xp_topc_readout_argmax(const xp_head* head, const void* lat, const void* base_c,
                                 const int64_t* cand, const void* w2c, int N, int C,
                                 int64_t* blk, float* win_val, cudaStream_t stream);

/* Whole draft step: hidden cache, init argmax (or top-C gather when topc > 0),
 * then K passes of latent + readout-argmax.  blk: device [N, B] int64 (out;
 * slot 0 = anchor).  topc >= V scores the full vocabulary through the top-C
 * path with C = V.  ws: workspace of ws_bytes >= xp_workspace_bytes(w, N, topc).
 * Top-C: the candidates' w2 rows are copied once per step while N*(B-1)*C <= V
 * (the copy is no larger than w2); for larger batches every pass reads them by id
 * from w2 instead.  Both give the same blk.
 * qwen3_xpress page, XPressRefinerHead.jacobi_refine_greedy. */
xp_status xp_jacobi_refine(const xp_head* head, const void* base, int64_t stride_n,
                           int64_t stride_b, const void* h_full, const int64_t* anchor,
                           const int64_t* am1, int N, int K, int topc, int64_t* blk,
                           void* ws, size_t ws_bytes, cudaStream_t stream);

/* The K passes of xp_jacobi_refine alone, for callers that prepare the pass-invariant
 * inputs themselves: blk (device [N, B] int64) holds the initial block (slot 0 = anchor,
 * slots 1..B-1 the initial tokens, e.g. from xp_init_argmax) and is refined in place; xh
 * (device [N, B, r] fp32) is the hidden cache of xp_hidden_cache; am1 and the base
 * addressing as for xp_jacobi_refine; ws of ws_bytes >= xp_workspace_bytes(w, N, 0).
 * Full-vocabulary scoring.  Each pass is one latent and one readout launch, or, under
 * XP_PASSES_PERSISTENT with a bf16 head of r = 256, H = 512 and B <= 16, all K passes run
 * in one persistent launch (one CTA per SM, every CTA resident at once).  Both give the
 * same blk up to the latent's rounding (see xp_latent_pass).
 * qwen3_xpress page, XPressRefinerHead.jacobi_refine_greedy (the loop over passes). */
xp_status xp_jacobi_passes(const xp_head* head, const void* base, int64_t stride_n,
                           int64_t stride_b, const float* xh, const int64_t* am1, int N, int K,
                           int64_t* blk, void* ws, size_t ws_bytes, cudaStream_t stream);

/* How xp_jacobi_refine and xp_jacobi_passes run the passes (full vocabulary):
 *  XP_PASSES_AUTO        the faster of the two for the shapes; on GB300 that has been the
 *                        per-stage launches at every measured shape (single request,
 *                        batched decode, max batch), so AUTO runs them
 *  XP_PASSES_PERSISTENT  the persistent launch wherever the shapes allow it
 *  XP_PASSES_PER_STAGE   one latent and one readout launch per pass
 * The choice changes the launches, not the method: blocks agree up to the latent's
 * rounding.  Default XP_PASSES_AUTO.  XP_EINVAL for another value. */
enum { XP_PASSES_AUTO = 0, XP_PASSES_PERSISTENT = 1, XP_PASSES_PER_STAGE = 2 };
xp_status xp_set_pass_mode(xp_head* head, int mode);

/* The tensor-core argmax readout (xp_readout_argmax, the per-stage passes, the
 * workspace-free readout) takes up to 128 draft rows per CTA.  When the row tiles come in
 * an even number, on = 1 runs them as 2-CTA clusters whose two CTAs share every MMA and
 * stage half of each w2 tile each; on = 0 (the default) keeps one CTA per row tile.  Both
 * compute the same fp32 dot products over the same k order.  The readout's vocabulary
 * loop is bound by the HBM stream of base rather than by shared-memory traffic, so pairs
 * have not been faster on GB300; the setting is there for shapes where w2 traffic
 * dominates.  XP_EINVAL for another value.  Host only. */
xp_status xp_set_readout_pairs(xp_head* head, int on);

/* 1 when an argmax readout of N blocks would run as 2-CTA pairs under the head's
 * setting, else 0.  Host only. */
int xp_readout_pairs(const xp_head* head, int N);

/* 1 when a full-vocabulary refine of N blocks over this base addressing would run its
 * passes in the persistent launch under the head's pass mode, else 0.  Host only. */
int xp_passes_persistent(const xp_head* head, const void* base, int64_t stride_n,
                         int64_t stride_b, int N);

/* Synchronise `stream`, read and clear the head's device error word: XP_OK, XP_EBADTOKEN,
 * XP_ELENGTH, XP_EEMPTY, XP_ERANGE or XP_ETIMEOUT (precedence in reverse order). */
xp_status xp_get_error(const xp_head* head, cudaStream_t stream);

/* Failure-path self-test (no counterpart on the pages): launches one kernel whose
 * mbarrier wait nothing will ever complete.  Like every wait in this library it
 * gives up after about half a second and records XP_ETIMEOUT in the head's error
 * word (read it with xp_get_error); no trap, no fault, the context stays usable.
 * Returns XP_OK when the launch succeeded. */
xp_status xp_selftest_wait_timeout(const xp_head* head, cudaStream_t stream);

/* Measurement aid (no counterpart on the pages): where xp_jacobi_refine runs all K passes
 * in its persistent kernel (bf16 head, r = 256, H = 512, B <= 16, full vocabulary), it can
 * record when each CTA reached each phase of each pass.  With buf (device) set, later
 * refines of at most K passes write, per CTA c and pass k, twelve globaltimer stamps (ns) at
 * buf[(c * K + k) * 12 + slot]: 0 the CTA's latent work of the pass starts (its tokens are
 * final; 0 if it has none), 1 its latent work is done, 2 its readout starts (its row tile's
 * latent is complete), 3 its readout's winners are merged; within its first latent group
 * of the pass, 8 its tokens are read, 9 its first gathered rows have landed, 4 every CTA of
 * its team has written its slice of the mixed latent u, 5 its SwiGLU activations are
 * written, 6 its down-projection partials are written, 7 every CTA of its team has
 * written its partials; in its readout, 10 its latent tile is in tensor memory, 11 its
 * first vocabulary tile is reduced.  Slots a CTA never reaches stay as they were.  *needed (nullable) receives
 * the bytes K passes need.  buf = NULL turns the recording off.  The work done is the same
 * either way.  XP_ECAPACITY when bytes is below *needed. */
xp_status xp_profile_timeline(xp_head* head, void* buf, size_t bytes, int K, size_t* needed);

/* Name of the readout kernel the head uses for its shape (for profiling). */
const char* xp_readout_kernel_name(const xp_head* head);

/* ---------------------------------------------------------------------------------------
 * After the refinement: the drafted blocks are scored by the target model over a paged
 * cache, verified, and the cache is cut back to what was accepted.  None of these calls has
 * a counterpart on the pages; they are the target's side of the same draft step.
 * An empty batch (no rows, sequences or children) is XP_OK, and the pointers that belong to it may
 * be NULL.
 * ------------------------------------------------------------------------------------- */

/* Verification of drafted blocks against the target's probabilities, from given random
 * numbers.  With D = n_draft[n] drafted tokens x_b = blk[n, 1+b] (b = 0..D-1) per block:
 *   p_b = softmax(target[n, b] / t[n])      b = 0..D (row b is the target after slot b)
 *   q_b = softmax(draft[n, b] / t[n]), or one-hot at x_b when draft == NULL (the refinement's
 *         own greedy drafts)
 *   slot b is accepted while u[n, b] * q_b(x_b) < p_b(x_b); the first slot a that is not ends
 *   the block with one token drawn from the normalised residual max(p_a - q_a, 0); when all D
 *   are accepted, a = D and the token is drawn from p_D.
 * The draw is a race: argmax_v w(v) / noise[n, v], which draws from w when the noise is
 * exponential; equal ratios go to the lowest id.  (Where rounding leaves no positive
 * residual, p_a itself is drawn from.)  t[n] = 0 makes block n greedy: p_b is one-hot at the
 * lowest argmax, a draft is accepted when it is that id, and no noise is read.
 * The emitted tokens then follow the target's own distribution, whatever the draft's, provided that
 * each x_b was drawn from q_b.  So the refinement's own blocks, which are argmaxes, go with
 * draft == NULL; draft logits go with tokens drawn from their softmax at the block's temperature.  An
 * argmax given with the logits it was taken from, proposed with certainty but tested as if with
 * probability q, would be refused too often: the tokens emitted would not follow the target.
 *
 * target: device [N, B, V] head dtype, row (n, b) at target + n*stride_n + b*stride_b, unit
 * stride over v.  draft: device fp32, row n*(B-1) + b at draft + (n*(B-1) + b)*ld_draft (the
 * layout xp_refine_logits writes), or NULL.  blk: device [N, B] int64.  n_draft: device [N]
 * int32 (clamped to [0, B-1], XP_ELENGTH), or NULL for B-1.  temperature: device [N] fp32, or
 * NULL for 1; one below the least normal float (1.1755e-38), negative or NaN counts as 0.
 * u: device [N, B-1] fp32 in [0, 1).  noise: device fp32 > 0, row n at noise + n*ld_noise.
 * tokens (out): device [N, B] int64: the accepted drafts, then the drawn token, then -1.
 * counts (out): device [N] int32, tokens emitted (accepted + 1).  prob (out): device
 * [N, B-1] fp32 = min(1, p_b(x_b) / q_b(x_b)) for the slots tested, 0 behind them, or NULL.
 * Logits are read as: NaN like -inf (never drawn), +inf like the largest finite value.  A
 * target row with nothing above -inf accepts nothing, and a block that ends there, or whose
 * race no id wins (noise that is NaN or infinite), gets token -1 (XP_EEMPTY).  A drafted id outside [0, V) is rejected (XP_EBADTOKEN).
 * Rows behind a block's first rejection cannot change the result and are mostly not read.
 * B, V, dtype: what the buffers were made for; XP_EINVAL unless they are the head's.
 * ws: xp_verify_workspace_bytes, zeroed once with xp_workspace_init (again after XP_ETIMEOUT);
 * calls that overlap on the GPU need a workspace each. */
size_t xp_verify_workspace_bytes(const xp_head* head, int N);
xp_status xp_verify_drafts(const xp_head* head, const void* target, int64_t stride_n,
                           int64_t stride_b, const float* draft, int64_t ld_draft,
                           const int64_t* blk, const int32_t* n_draft, int N, int B, int V,
                           xp_dtype dtype, const float* temperature, const float* u, const float* noise,
                           int64_t ld_noise, int64_t* tokens, int32_t* counts, float* prob,
                           void* ws, size_t ws_bytes, cudaStream_t stream);

/* Log probabilities of given tokens under the rows they were drawn from, with the entropy of the
 * distribution, the token's rank and the best alternatives.  With x = tokens[n, b], l = logits[n, b] and
 * t = temperature[n], p = softmax(l / t):
 *   logprob[n, b] = log p(x),  entropy[n, b] = -sum_v p(v) log p(v),
 *   rank[n, b] = 1 + the number of ids ahead of x in order of l, ties to the lower id,
 *   top_ids[n, b, 0..top-1], top_logprobs: the first ids in that order (-1 and -inf where there are not
 *   as many ids above -inf), and their log p.
 * tokens: the layout that xp_verify_drafts writes (its token of slot b was drawn from target row b).  A row
 * whose token is -1 is not read: logprob, entropy, rank and top_logprobs 0, top_ids -1; so is one whose
 * token lies outside [-1, V) (XP_EBADTOKEN).  temperature as for xp_verify_drafts: t = 0 makes p one-hot at
 * the lowest argmax.  Logits are read as there: NaN like -inf, +inf like the largest finite value; a
 * row with nothing above -inf has logprob -inf, entropy 0, rank x + 1 and no alternatives (XP_EEMPTY).
 * logits: device, bf16 or fp32 as `dtype` says (not the head's necessarily), row (n, b) at
 * n*stride_n + b*stride_b, unit stride over v; V: XP_EINVAL unless the head's.  tokens: device [N, B] int64;
 * B is any number of rows a block.  Outputs: device [N, B] (logprob, entropy fp32, rank int32) and
 * [N, B, top] (int64, fp32), each may be NULL; 0 <= top <= 32 (the top pointers are not used at 0).
 * Sums are fp32 of the differences from the row's maximum.  N*B rows below 2^31 / 64.
 * ws: xp_logprobs_workspace_bytes, zeroed once with xp_workspace_init; calls that overlap on the GPU need
 * a workspace each. */
size_t xp_logprobs_workspace_bytes(const xp_head* head, int rows, int top);
xp_status xp_token_logprobs(const xp_head* head, const void* logits, int64_t stride_n, int64_t stride_b,
                            const int64_t* tokens, int N, int B, int V, xp_dtype dtype,
                            const float* temperature, int top, float* logprob, float* entropy,
                            int32_t* rank, int64_t* top_ids, float* top_logprobs, void* ws,
                            size_t ws_bytes, cudaStream_t stream);

/* A paged key/value cache.  K and V are pools of `pages` pages of `page_size` tokens in each
 * of `layers` layers; a sequence is a row of page ids (its table) and a length, and a page
 * that several rows hold is counted in `refs`.  The pools belong to the caller; element
 * (layer, page, token, head, i) of either is at
 *   layer*stride_layer + page*stride_page + token*stride_token + head*stride_head + i
 * (elements).  A page is one dense block in either order: tokens outside
 * (stride_token = kv_heads*head_dim, stride_head = head_dim) or heads outside
 * (stride_head = page_size*head_dim, stride_token = head_dim). */
typedef struct {
  int pages, page_size, layers, kv_heads, head_dim;
  int max_seqs;    /* most rows any table call will pass */
  xp_dtype dtype;
  int64_t stride_layer, stride_page, stride_token, stride_head;
  void* k;
  void* v;
} xp_cache_desc;

/* Quantised caches: dtype XP_Q8 or XP_Q4.  16 consecutive dims of a token's head share a scale s and are
 * held as whole numbers c of 8 or 4 bits that stand for c*s, |c| <= 127 or 7.  s is an 8-bit float without a
 * sign, 5 bits of exponent and 3 of mantissa: the 16-bit float whose bits are the byte << 7.  It is the least
 * one for which 127*s or 7*s reaches the largest magnitude of the 16, at most 512 or 7680; c is the element
 * over s, rounded to nearest, ties to even.  So every value held is exact in 16-bit floats (and those of 4
 * bits in bf16), and an element is off by at most s/2.  A NaN is held as 0, and what lies beyond
 * 127*512 or 7*7680 as the nearest value that can be held; both raise XP_ERANGE.
 * All strides are in bytes, and heads lie outside the tokens of a page.  A head of a page is
 * xp_quant_head_bytes: the codes of its tokens, head_dim*8/8 or head_dim*4/8 bytes each, then their scales,
 * head_dim/16 bytes each, padded to a multiple of 4; the whole is padded to a multiple of 16.  8-bit codes
 * are c + 128, a byte a dim.  4-bit codes are c + 8; those of 8 dims are a 32-bit word (lowest byte first),
 * dim 2j + e of the 8 in the bits from 4*(j + 4*e) on.  head_dim: a multiple of 16; stride_token: the bytes
 * of a token's codes; stride_head: xp_quant_head_bytes; pools on 16-byte boundaries; stride_page and
 * stride_layer: multiples of 16.  Every call on caches takes them.  The rows of xp_cache_append and
 * xp_cache_read are bf16 or fp32, queries and results of xp_prefix_attention bf16; where the calls below
 * copy part of a page, they copy a quantised one whole. */

/* Bytes of one head of a page of a quantised cache (0: not XP_Q8 or XP_Q4, or sizes it cannot have).
 * Host only. */
size_t xp_quant_head_bytes(int page_size, int head_dim, xp_dtype dtype);

typedef struct xp_cache xp_cache; /* opaque, host-side */

/* Device bytes of the cache's error word and of the table calls' scratch. */
size_t xp_cache_prep_bytes(const xp_cache_desc* d);

/* Host handle of a cache.  prep_dev: device, 256-byte aligned, cleared by the call.  The
 * pools stay the caller's and must outlive the handle.  head_dim <= 256. */
xp_status xp_cache_create(const xp_cache_desc* d, void* prep_dev, size_t prep_bytes,
                          cudaStream_t stream, xp_cache** out);
void xp_cache_destroy(xp_cache* cache);

/* Synchronise `stream`, read and clear the cache's device error word: XP_OK or one of XP_ERANGE,
 * XP_EBADPAGE, XP_ENOPAGES, XP_ESHARED, XP_ELENGTH, XP_ETIMEOUT (the last named first). */
xp_status xp_cache_get_error(const xp_cache* cache, cudaStream_t stream);

/* Write the keys and values of the T newest tokens of N sequences: token t of row n goes to
 * position lens[n] - T + t (lens counts them already; positions below 0 are skipped).
 * k, v: device, element (n, t, head, i) at n*stride_n + t*stride_t + head*stride_h + i.
 * heads, head_dim, dtype: theirs; XP_EINVAL unless they are the cache's (of a quantised one: dtype
 * XP_BF16 or XP_F32).  table: device
 * int32, row n at table + n*ld_table; lens: device [N] int32.  Positions behind a row's columns are
 * skipped (XP_ELENGTH): xp_cache_append takes ld_table as their number, xp_cache_append_columns
 * has `width` of them (a table that is some columns of a wider one). */
xp_status xp_cache_append(const xp_cache* cache, int layer, const void* k, const void* v,
                          int64_t stride_n, int64_t stride_t, int64_t stride_h,
                          int heads, int head_dim, xp_dtype dtype, const int32_t* table,
                          int64_t ld_table, const int32_t* lens, int N, int T,
                          cudaStream_t stream);
xp_status xp_cache_append_columns(const xp_cache* cache, int layer, const void* k, const void* v,
                                  int64_t stride_n, int64_t stride_t, int64_t stride_h,
                                  int heads, int head_dim, xp_dtype dtype, const int32_t* table,
                                  int64_t ld_table, int width, const int32_t* lens, int N, int T,
                                  cudaStream_t stream);

/* Read back T positions of N sequences as dense rows: row (n, t) is position first[n] + t, its keys and
 * values where it lies in [0, lens[n]) and zeros where it does not.  first: device [N] int32, or NULL for
 * 0 (lens[n] - T gives what xp_cache_append wrote last).  k, v (out): device, element (n, t, head, i) at
 * n*stride_n + t*stride_t + head*stride_h + i, of type `dtype`, XP_BF16 or XP_F32, whatever the cache's
 * (rounded to nearest once where it cannot hold the cache's value).  table, ld_table, width, lens as for
 * xp_cache_append_columns; positions behind a row's columns are zeros (XP_ELENGTH). */
xp_status xp_cache_read(const xp_cache* cache, int layer, const int32_t* table, int64_t ld_table, int width,
                        const int32_t* lens, const int32_t* first, int N, int T, void* k, void* v,
                        int64_t stride_n, int64_t stride_t, int64_t stride_h, int heads, int head_dim,
                        xp_dtype dtype, cudaStream_t stream);

/* The table calls below change page tables, lengths and reference counts (and, where they
 * say so, move pages of K and V in every layer).  Each output may be the matching input
 * itself.  Page ids of a table behind ceil(length / page_size) are not read and are written
 * as -1.  `width`: columns of the tables (width*page_size, and resize's N*width, below 2^31);
 * `pages`: entries of refs, refs_out and map, XP_EINVAL unless the pool's.  They share the
 * handle's scratch: calls on one cache must not overlap on the GPU. */

/* Copy whole pages src[i] -> dst[i] (device int32, `count` of them), K and V, every layer.
 * A negative id skips the pair; no page may be the target of one pair and in another. */
xp_status xp_cache_copy(const xp_cache* cache, const int32_t* src, const int32_t* dst, int count,
                        cudaStream_t stream);

/* Lengths old -> new: pages behind the new length are let go (refs - 1), missing ones taken
 * (refs = 1): the lowest free ids, after all releases, in row and then in column order.
 * new_lens is clamped to [0, width*page_size] (XP_ELENGTH).  Where the pool runs out, rows
 * end at the last page they got (XP_ENOPAGES).  A row whose old or new length, the smaller
 * of the two, ends inside a page that is held more than once stays as it was (XP_ESHARED):
 * fork it instead. */
xp_status xp_cache_resize(const xp_cache* cache, const int32_t* table, int64_t ld_table,
                          const int32_t* lens, const int32_t* new_lens, const int32_t* refs,
                          int pages, int N, int width, int32_t* table_out, int64_t ld_out, int32_t* lens_out,
                          int32_t* refs_out, cudaStream_t stream);

/* M children: child i continues row parent[i] of a table of `rows` rows at length
 * min(lens[parent[i]], cut[i]) (cut may be NULL).  Its full pages are shared (refs + 1); of a
 * partly filled last page it gets a copy of its own, the tokens it holds only (a quantised one whole): the lowest
 * free id, in child order.  Without one it ends at its last full page (XP_ENOPAGES).  A
 * parent outside [0, rows) gives an empty child (XP_ELENGTH).  child_table may be rows of the
 * same table, parents among them: all parents are read before any child is written (XP_EINVAL
 * where entries of different columns overlap, or the rows lie at strides too unlike to tell).
 * What a child's row held before is not let go: its pages stay counted. */
xp_status xp_cache_fork(const xp_cache* cache, const int32_t* table, int64_t ld_table,
                        const int32_t* lens, int rows, const int32_t* parent, const int32_t* cut,
                        int M, int width, const int32_t* refs, int pages, int32_t* child_table,
                        int64_t ld_child, int32_t* child_lens, int32_t* refs_out,
                        cudaStream_t stream);

/* Pack the pages in use (refs > 0) to ids 0..live-1: the i-th of those with an id >= live
 * moves to the i-th free id < live.  Every table row, refs and the pools follow; map (device
 * [pages] int32, may be NULL) receives each page's new id, -1 for a free one, for tables
 * kept elsewhere; live (device [1] int32, may be NULL) their number. */
xp_status xp_cache_compact(const xp_cache* cache, const int32_t* table, int64_t ld_table,
                           const int32_t* lens, int N, int width, const int32_t* refs, int pages,
                           int32_t* table_out, int64_t ld_out, int32_t* refs_out, int32_t* map,
                           int32_t* live, cudaStream_t stream);

/* Attention of N sequences of T new tokens (T = 1: plain decoding; T = B: a drafted block)
 * that share a prefix of prefix_len tokens and each have a tail of their own.  Query (n, t)
 * of head h sees the whole prefix and the tail's positions below lens[n] - T + t + 1 (the
 * new tokens' keys and values are in the tail already), through kv head
 * h / (heads / kv_heads):
 *   out = sum_j softmax_j(scale * q . k_j) v_j,   lse = log sum_j exp(scale * q . k_j).
 * The prefix is read once for the whole batch, not once a sequence.  A query that sees
 * nothing, or only scores of -inf, gets out = 0 and lse = -inf.  Tokens behind the lengths may
 * hold anything, and an infinite or NaN key or value reaches the queries that see it and no others.
 * q, out: cache dtype, element (n, t, h, i) at n*stride_n + t*stride_t + h*stride_h + i.
 * prefix_table: device int32, prefix_pages >= ceil(prefix_len / page_size) entries.  table:
 * device int32, row n at table + n*ld_table, width >= ceil(max_len / page_size) columns.
 * lens: device [N] int32; lengths above max_len are clamped (XP_ELENGTH).  lse: device fp32
 * [N, T, heads] or NULL.  scale: positive and finite.  Scores, softmax and sums are fp32 (bf16:
 * each weight is rounded to bf16 before it multiplies v, as the tensor cores take it).
 * bf16 caches of head_dim 64 or 128 and pages of a multiple of 8 tokens, with pools on 16-byte
 * boundaries and strides that are multiples of 8, run on the tensor cores (scores there: below 2^29; the
 * rounding of larger ones leaves what a weight can be); all others run on CUDA
 * cores, at a small part of that rate (an fp32 cache keeps the weights in 32 bits).  On tensor cores
 * queries on 16-byte boundaries with one stride from token to token, across sequences too, are
 * loaded fastest: a slice of the last T tokens of longer rows costs half the call's time again.
 * Quantised caches: q and out are bf16, any head_dim and page size, on tensor cores; values are those held,
 * in 16-bit floats, and each weight is rounded to one of those.  Where many queries share a key (head_dim 64
 * or 128) keys and values are written out in 16 bits to the workspace, which is as much larger: 4 kv_heads
 * head_dim bytes a token.  A prefix is from 256 rows of N T heads/kv_heads on, whatever its length (a million
 * tokens of 8 heads of 128: 4.3 GB).  Tails are, to 1 GiB together: without a prefix from 64 rows of T
 * heads/kv_heads on; beside a prefix that is, from 32, and at any number where they have at most twice its pages
 * of 128 tokens.  Rows there with scores past 2^17 are right but slow.  scale times a query's largest
 * magnitude: below 2e38. */
typedef struct {
  int layer, N, T, heads;
  int head_dim;      /* head_dim and dtype: those of q and out, which must be the cache's */
  xp_dtype dtype;
  int prefix_len, max_len;
  float scale;
  int64_t q_stride_n, q_stride_t, q_stride_h;
  int64_t o_stride_n, o_stride_t, o_stride_h;
} xp_attn;

/* Device bytes of the attention's workspace (need not be cleared). */
size_t xp_attention_workspace_bytes(const xp_cache* cache, const xp_attn* a);
xp_status xp_prefix_attention(const xp_cache* cache, const xp_attn* a, const void* q,
                              const int32_t* prefix_table, int prefix_pages, const int32_t* table,
                              int64_t ld_table, int width, const int32_t* lens, void* out, float* lse,
                              void* ws, size_t ws_bytes, cudaStream_t stream);

const char* xp_status_str(xp_status s);

#ifdef __cplusplus
}
#endif

#endif /* XP_H_ */
