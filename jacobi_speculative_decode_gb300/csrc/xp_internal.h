// Internal declarations shared by the host API and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "xp.h"

// Host-side head: shapes, the prepared device copies, device facts.
struct xp_head {
  int V, hidden, r, H, B, max_N;
  xp_dtype dtype;
  int device, num_sms;
  char* prep;            // caller-owned device memory holding everything below
  size_t prep_bytes;
  uint32_t* err;         // device error word (XP_ERR_* bits)
  void *w1, *down_hg, *w_hc, *w_lat, *mix, *w_gate, *w_up, *w_down, *w2;  // down_hg = [down_h ; down_g]
  void* wgu16;           // [w_gate ; w_up] as fp16 in cluster row order (tensor-core latent only)
  void* mixT;            // folded mixer laid out [out slot][in slot][channel]
  float* E;              // w1 . in_proj[:, 2r:]^T, fp32 [V, r] (tensor-core latent only)
  void* hfold;           // [in_proj[:, :r] . down_h ; in_proj[:, r:2r] . down_g] as bf16 hi, lo planes
  int hidden_tc;         // tcgen05 hidden cache usable for this head's shapes
  CUtensorMap tm_hfold;  // hfold viewed as [4r, hidden] (hi rows, then lo rows)
  int readout_tc;        // tcgen05 readout usable for this head's shapes
  int latent_mma;        // cluster tensor-core latent usable for this head's shapes
  CUtensorMap tm_w2;     // W2 [V, r] tiled map for the tcgen05 readout
  CUtensorMap tm_w2_half;  // the same with half-tile boxes (one CTA of a readout pair)
  int readout_pair_ok;   // tm_w2_half could be encoded
  int readout_pairs;     // xp_set_readout_pairs: 2-CTA readout when the row tiles pair up
  CUtensorMap tm_wgu, tm_wd, tm_mixT;  // [w_gate ; w_up] fp16 rows, w_down, mixer slices (TMA)
  void* timeline;        // optional per-CTA per-pass phase timestamps of the persistent refine
  size_t timeline_bytes;
  int pass_mode;         // XP_PASSES_AUTO / _PERSISTENT / _PER_STAGE
};

// device error word bits
enum : uint32_t {
  XP_ERR_BADTOKEN = 1u, XP_ERR_TIMEOUT = 2u, XP_ERR_RANGE = 4u, XP_ERR_BADPAGE = 8u,
  XP_ERR_NOPAGES = 16u, XP_ERR_SHARED = 32u, XP_ERR_LENGTH = 64u, XP_ERR_EMPTY = 128u
};

// Workspace layout.  Regions that must stay zero between calls come first and
// are sized by the head's max_N so that the layout never moves with N.
struct xp_ws_layout {
  size_t ro_packed, ro_ticket;        // readout argmax partials, per-row-tile tickets
  size_t in_packed, in_ticket;        // init argmax partials, per-row tickets
  size_t pk1, cnt;                    // persistent refine: odd passes' argmax words, counters
  size_t zero_end;                    // [0, zero_end) must be zero between calls
  size_t xh, lat, part, hc;           // pass data and hidden-cache scratch
  size_t xbuf;                        // persistent refine: latent partial-sum exchange
  int part_rows;                      // rows of fp32 split-K partials the scratch holds
  size_t cand, base_c, w2c;           // top-C tail (sized by the call's N and C)
  size_t total;
};
xp_ws_layout xp_layout(int V, int hidden, int r, int H, int B, int max_N, xp_dtype dt, int N,
                       int C);

// bytes of an element; of a quantised cache, whose sizes and strides are bytes, 1
static inline size_t xp_elem(xp_dtype d) { return d == XP_BF16 ? 2 : d == XP_F32 ? 4 : 1; }

// true when the current device is the one the head was created on
bool xp_on_head_device(const xp_head* h);

// ---- launchers (return cudaGetLastError() after launching) -----------------
cudaError_t xp_launch_fold(const void* raw, void* mix, int r, int B, xp_dtype dt, cudaStream_t s);
cudaError_t xp_launch_mix_transpose(const void* mix, void* mixT, int r, int B, xp_dtype dt,
                                    cudaStream_t s);

// E = w1 . w_lat^T, the projected embedding table of the tensor-core latent
cudaError_t xp_launch_embed_table(const xp_head* h, cudaStream_t s);

cudaError_t xp_launch_hidden(const xp_head* h, const void* h_full, int N, float* xh, float* part,
                             float* hc, int part_rows, cudaStream_t s);
// tcgen05 hidden cache over the folded projection (bf16 heads, 2r a multiple of 256)
bool xp_hidden_tc_ok(int r, int hidden, xp_dtype dt);
bool xp_hidden_tc_map(xp_head* h);
cudaError_t xp_launch_hidden_fold(const xp_head* h, const void* in_proj, cudaStream_t s);
bool xp_hidden_tc_call_ok(const xp_head* h, const void* h_full);
// returns cudaErrorNotSupported when h_full cannot be tiled by TMA
cudaError_t xp_launch_hidden_tc(const xp_head* h, const void* h_full, int N, float* xh,
                                float* part, int part_rows, cudaStream_t s);
// the same in two launches, so that independent work can run between them: the GEMM
// lets a programmatically dependent launch start early; the reduce (pdl = true) waits
// for its predecessor before reading the partials
cudaError_t xp_launch_hidden_tc_gemm(const xp_head* h, const void* h_full, int N, float* part,
                                     int part_rows, cudaStream_t s, int* splits_out);
cudaError_t xp_launch_xh_reduce(const xp_head* h, int N, float* xh, const float* part, int splits,
                                cudaStream_t s, bool pdl);

// overlap_prev: launch with a programmatic dependency on the previous kernel, which
// must touch none of base, blk, win or the argmax scratch; the kernel waits for that
// kernel only at its end, so whatever follows sees both completed
cudaError_t xp_launch_init_argmax(const xp_head* h, const void* base, int64_t sn, int64_t sb,
                                  const int64_t* anchor, int N, int64_t* blk, float* win,
                                  unsigned long long* packed, unsigned* ticket, cudaStream_t s,
                                  bool overlap_prev = false);

cudaError_t xp_launch_latent_simt(const xp_head* h, const int64_t* blk, const int64_t* am1,
                                  const float* xh, int N, void* lat, cudaStream_t s);
bool xp_latent_mma_ok(int r, int H, int B, xp_dtype dt);
bool xp_latent_mma_maps(xp_head* h);
// w_gate / w_up copied to fp16 for the tensor-core latent (saturating; XP_ERR_RANGE)
cudaError_t xp_launch_gu_to_f16(const xp_head* h, const void* w_gate, const void* w_up,
                                cudaStream_t s);
cudaError_t xp_launch_latent_mma(const xp_head* h, const int64_t* blk, const int64_t* am1,
                                 const float* xh, int N, void* lat, cudaStream_t s);

cudaError_t xp_launch_readout_simt(const xp_head* h, const void* lat, const void* base,
                                   int64_t sn, int64_t sb, int N, int64_t* blk, float* win,
                                   unsigned long long* packed, unsigned* ticket, cudaStream_t s);
// returns cudaErrorNotSupported when the call's base addressing cannot be tiled by TMA
cudaError_t xp_launch_readout_tc(const xp_head* h, const void* lat, const void* base,
                                 int64_t sn, int64_t sb, int N, int64_t* blk, float* win,
                                 unsigned long long* packed, unsigned* ticket, cudaStream_t s);
int xp_readout_tc_tile();   // vocabulary ids per tile of the tcgen05 readout (w2 map box rows)
// true when the argmax readout of N blocks runs as 2-CTA pairs (even number of row tiles)
bool xp_readout_paired(const xp_head* h, int N);
bool xp_readout_tc_call_ok(const xp_head* h, const void* lat, const void* base, int64_t sn,
                           int64_t sb, int N);
// logits base + lat.w2 (bias alone when base is null) as fp32 rows of out (row stride ldo)
cudaError_t xp_launch_logits_simt(const xp_head* h, const void* lat, const void* base, int64_t sn,
                                  int64_t sb, int N, float* out, int64_t ldo, cudaStream_t s);
// returns cudaErrorNotSupported when the tcgen05 path cannot take the call
cudaError_t xp_launch_logits_tc(const xp_head* h, const void* lat, const void* base, int64_t sn,
                                int64_t sb, int N, float* out, int64_t ldo, cudaStream_t s);
bool xp_logits_tc_call_ok(const xp_head* h, const void* lat, const void* base, int64_t sn,
                          int64_t sb, int N, const float* out, int64_t ldo);

// All K passes in one persistent cooperative launch (bf16, r = 256, H = 512, B <= 16).
bool xp_persist_ok(int r, int H, int B, xp_dtype dt);
size_t xp_persist_xbuf_bytes(int B, int max_N);
size_t xp_persist_counter_words(int max_N);
size_t xp_persist_timeline_bytes(const xp_head* h, int K);
bool xp_persist_call_ok(const xp_head* h, const void* base, int64_t sn, int64_t sb, int N);
// the automatic choice between the persistent and the per-stage passes for N blocks
bool xp_persist_preferred(const xp_head* h, int N);
// returns cudaErrorNotSupported (nothing launched) when the call cannot take this path
cudaError_t xp_launch_persist(const xp_head* h, const void* base, int64_t sn, int64_t sb, int N,
                              int K, const float* xh, const int64_t* am1, int64_t* blk, void* lat,
                              unsigned long long* packed0, unsigned long long* packed1,
                              void* xbuf, unsigned* counters, cudaStream_t s);

cudaError_t xp_launch_topc_gather(const xp_head* h, const void* base, int64_t sn, int64_t sb,
                                  int N, int C, int64_t* cand, void* base_c, void* w2c,
                                  int64_t* blk, const int64_t* anchor, cudaStream_t s);
cudaError_t xp_launch_topc_readout(const xp_head* h, const void* lat, const void* base_c,
                                   const int64_t* cand, const void* w2c, int N, int C,
                                   int64_t* blk, float* win, cudaStream_t s);

// Verification of drafted blocks.  packed, marks and tickets must be zero between calls.
struct xp_verify_ws {
  size_t marks, tickets, packed, draw_ticket, next;   // zero between calls
  size_t part, row;                             // softmax statistics: per chunk, per row
  size_t total;
};
xp_verify_ws xp_verify_layout(const xp_head* h, int N);
struct xp_verify_args {
  const void* target;
  int64_t sn, sb;
  const float* draft;
  int64_t ld_draft;
  const int64_t* blk;
  const int32_t* n_draft;
  const float* temperature;
  const float* u;
  const float* noise;
  int64_t ld_noise;
  int64_t* tokens;
  int32_t* counts;
  float* prob;
  int N, B, V;
  uint32_t* err;
  // workspace
  unsigned* marks;
  unsigned* tickets;
  unsigned long long* packed;
  unsigned* draw_ticket;
  unsigned* next;
  float* part;
  float* row;
};
cudaError_t xp_launch_verify(const xp_head* h, const xp_verify_args& a, cudaStream_t s);

// Log probabilities of given tokens.  tickets must be zero between calls.
struct xp_logprobs_ws {
  size_t tickets, stat, best, total;
};
xp_logprobs_ws xp_logprobs_layout(const xp_head* h, int rows, int top);
struct xp_logprobs_args {
  const void* logits;
  int64_t sn, sb;
  const int64_t* tokens;
  const float* temperature;
  int N, B, top;
  xp_dtype dtype;
  float *logprob, *entropy;
  int32_t* rank;
  int64_t* top_ids;
  float* top_logprobs;
  unsigned* tickets;
  void* stat;
  unsigned long long* best;
};
cudaError_t xp_launch_logprobs(const xp_head* h, const xp_logprobs_args& a, cudaStream_t s);

// Host-side cache: the caller's pools, the prepared scratch, device facts.
struct xp_cache {
  xp_cache_desc d;
  int device, num_sms;
  bool heads_outside;      // page order: [head][token][dim] instead of [token][head][dim]
  uint32_t* err;           // device error word (XP_ERR_* bits)
  int32_t *src, *dst, *cnt;  // page moves: source, target, tokens (scratch, `pages` each)
  int32_t* n_moves;        // their number
  int32_t* map;            // compaction: new id of every page (scratch)
  int32_t *row_a, *row_b, *row_c, *row_d;  // per-row scratch of the table calls (max_seqs each)
  int attn_tc;             // tokens of a TMA box of the tensor-core attention, 0: not usable (of a
                           // quantised cache: of what is widened for it)
  CUtensorMap tm_k, tm_v;  // the pools as (dim, token, head, page, layer)
};

cudaError_t xp_launch_append(const xp_cache* c, int layer, const void* k, const void* v, int64_t sn,
                             int64_t st, int64_t sh, const int32_t* table, int64_t ld,
                             int64_t width, const int32_t* lens, int N, int T, cudaStream_t s);
// rows: their type, XP_BF16 or XP_F32
cudaError_t xp_launch_append_quant(const xp_cache* c, int layer, const void* k, const void* v, int64_t sn,
                                   int64_t st, int64_t sh, xp_dtype rows, const int32_t* table, int64_t ld,
                                   int64_t width, const int32_t* lens, int N, int T, cudaStream_t s);
cudaError_t xp_launch_cache_read(const xp_cache* c, int layer, const int32_t* table, int64_t ld,
                                 int64_t width, const int32_t* lens, const int32_t* first, int N, int T,
                                 void* k, void* v, int64_t sn, int64_t st, int64_t sh, xp_dtype rows,
                                 cudaStream_t s);
// moves given by the caller (n on the host) or left by a table kernel (n_moves on the device);
// tokens == nullptr copies whole pages
cudaError_t xp_launch_copy_pages(const xp_cache* c, const int32_t* src, const int32_t* dst,
                                 const int32_t* tokens, int n, const int32_t* n_dev,
                                 cudaStream_t s);
cudaError_t xp_launch_resize(const xp_cache* c, const int32_t* table, int64_t ld,
                             const int32_t* lens, const int32_t* new_lens, const int32_t* refs,
                             int N, int width, int32_t* table_out, int64_t ld_out,
                             int32_t* lens_out, int32_t* refs_out, cudaStream_t s);
// in_place: children may be rows of their parents' table
cudaError_t xp_launch_fork(const xp_cache* c, const int32_t* table, int64_t ld,
                           const int32_t* lens, int rows, const int32_t* parent,
                           const int32_t* cut, int M, int width, const int32_t* refs,
                           bool in_place, int32_t* child, int64_t ld_child, int32_t* child_lens,
                           int32_t* refs_out, cudaStream_t s);
cudaError_t xp_launch_compact(const xp_cache* c, const int32_t* table, int64_t ld,
                              const int32_t* lens, int N, int width, const int32_t* refs,
                              int32_t* table_out, int64_t ld_out, int32_t* refs_out, int32_t* map,
                              int32_t* live, cudaStream_t s);

// How one attention call is split: `prefix_splits` ranges of prefix_keys keys, then
// `tail_splits` ranges of tail_keys keys; every range leaves one partial result a row.
struct xp_attn_plan {
  bool tc;                       // the tensor-core form
  int rows_tile;                 // query rows of one work item
  int prefix_tiles, tail_tiles;  // row tiles: over the batch, of one sequence
  bool prefix_few, tail_few;     // tensor-core form: few rows in the last of them
  int prefix_blocks, tail_blocks;   // tensor-core form: the same in blocks of 32 rows
  int64_t second_blocks;            // and those of the second stream's own results
  int prefix_splits, prefix_keys, tail_splits, tail_keys;
  int parts;
  // quantised form: what is widened to fp16 first, in pages of kWidePage tokens (0: nothing), where its
  // pools and its table are, elements of a head there; tc: then all of the call, else the prefix
  int wide_prefix, wide_tail;
  int64_t wide_plane;
  size_t wide_k, wide_v, wide_table, wide_q, wide_factor;
  size_t wide_stat, wide_acc, wide_line;   // the tcgen05 form's own workspace
  size_t part_stat, part_acc;              // and what it leaves of the prefix
  int64_t units;                           // row tiles of kv heads, of the prefix and of all tails
  // workspace: (max, sum) pairs, accumulators; tensor-core form: where each sequence's work begins
  size_t stat_off, acc_off, line_off, total;
};
struct xp_attn_args {
  xp_attn a;
  int group, kv_heads, dim, page_size, pages;
  const void *q, *k, *v;         // k, v: this layer's pools
  int64_t kv_page, kv_token, kv_head;
  const int32_t *prefix_table, *table, *lens;
  int64_t ld_table;
  void* out;
  float* lse;
  float* stat;                   // CUDA-core form: [parts][N*T*heads][2]
  float* acc;                    //                 [parts][N*T*heads][dim]
  int* line;
  // tcgen05 form: not null where q, k and v are fp16: what a product of query row r (rows of a kv head
  // together, [kv_heads][N*T*group]) is multiplied by to be a score in base 2
  const float* q_factor;
  // tcgen05 form: not null where the joined rows are not the call's results but one range of it, and
  // left as such: (max, sum) and weighted values, in the layout of stat and acc above
  float *part_stat, *part_acc;
  char* ws;
  uint32_t* err;
  xp_attn_plan plan;
};
xp_attn_plan xp_attn_simt_plan(const xp_cache* c, const xp_attn* a);
int xp_attn_tc_maps(xp_cache* c);   // tokens of a TMA box, 0 where the kernel cannot run
xp_attn_plan xp_attn_tc_plan(const xp_cache* c, const xp_attn* a);
cudaError_t xp_launch_attn_tc(const xp_cache* c, const xp_attn_args& g, cudaStream_t s);
cudaError_t xp_launch_attn_simt(const xp_cache* c, const xp_attn_args& g, cudaStream_t s);
cudaError_t xp_launch_attn_combine(const xp_attn_args& g, cudaStream_t s);
cudaError_t xp_launch_widen(const xp_cache* c, const xp_attn_args& g, int prefix_pages, int tail_pages,
                            void* k, void* v, int64_t plane, int32_t* table, void* q, float* q_factor,
                            cudaStream_t s);
xp_attn_plan xp_attn_quant_plan(const xp_cache* c, const xp_attn* a);
cudaError_t xp_launch_attn_quant(const xp_cache* c, const xp_attn_args& g, cudaStream_t s);

// Read and clear an error word behind what the stream holds, and wait for both.
inline cudaError_t xp_take_error(uint32_t* err, cudaStream_t s, uint32_t* word) {
  cudaError_t e = cudaMemcpyAsync(word, err, sizeof(*word), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(err, 0, sizeof(*word), s);
  const cudaError_t done = cudaStreamSynchronize(s);
  return e == cudaSuccess ? done : e;
}

// Let a kernel use `bytes` of dynamic shared memory: asked of the runtime once a device.
inline cudaError_t xp_allow_smem(const void* kernel, size_t bytes, unsigned long long* devices) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (__atomic_load_n(devices, __ATOMIC_RELAXED) >> dev & 1)) return cudaSuccess;
  const cudaError_t f =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (f == cudaSuccess && dev < 64) __atomic_fetch_or(devices, 1ull << dev, __ATOMIC_RELAXED);
  return f;
}

// Launch with a programmatic dependency on the previous kernel in the stream:
// the kernel's prologue may overlap that kernel's tail; the kernel itself must
// call griddepcontrol.wait before it touches anything the predecessor writes.
template <typename... KArgs, typename... Args>
cudaError_t xp_launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// tensor-map encoder fetched from the driver at run time (no -lcuda link)
typedef CUresult (*xp_encode_tiled_fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                       const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                       const cuuint32_t*, CUtensorMapInterleave,
                                       CUtensorMapSwizzle, CUtensorMapL2promotion,
                                       CUtensorMapFloatOOBfill);
xp_encode_tiled_fn xp_get_encode_tiled();
