/*
 * kda.h -- C ABI of the KDA (Kimi Delta Attention) prefill hot path for
 * AMD Instinct MI355X (gfx950).
 *
 * The prefill step has three stages:
 *   1. kda_state_gather   -- copy each request's initial recurrent state out
 *                            of indexed rows of a state cache;
 *   2. kda_chunk_prefill  -- run the chunkwise gated delta rule (chunk size
 *                            64) over a varlen batch delimited by cu_seqlens;
 *   3. kda_state_scatter  -- copy the final states back into cache rows.
 * Decode has one: kda_recurrent_decode advances each sequence by one token
 * with its state updated in place in its cache row.  Checkpoints can be
 * parked compressed: kda_ckpt_quantize_scatter / kda_ckpt_dequantize_gather
 * move states between packed buffers and an INT8 checkpoint store.
 * Hybrid models interleave KDA layers with latent-attention layers over the
 * same packed batch: kda_latent_prefill and kda_latent_decode are those
 * layers' attention, and kda_page_fork / kda_page_compact / kda_page_free keep
 * the pages of a latent cache (and the rows of a state cache) shared, dense
 * and reclaimed.  kda_latent_quantize_scatter / kda_latent_dequantize_gather write
 * and read a latent cache in 8 bits, kda_latent_decode_fp8 attends to it, and
 * kda_latent_decode_shared computes a prefix that sequences share (as after a
 * fork) once for all of them.
 *
 * Sources (web pages, cited by title and section):
 *  [P1] "vllm-ascend 的 KDA 状态复制 Triton 集成：PR 17301 对齐的预编译 worker
 *       生命周期方案": section "背景" (gather -> chunk math -> scatter around
 *       an unchanged chunk kernel with chunk size 64), section "数值契约"
 *       (the copy contract), section "自动分发" (the layout admissibility
 *       rule), section "启动准备" (index dtype kept as given).
 *  [P2] "【轻量化复刻大模型 / KIMI K3】KDA 对 AI Infra 的挑战与各家应对",
 *       section 1.1 (S_t = M_t S_{t-1} + b_t) and the varlen row of the
 *       table in section 0x00 (cu_seqlens, every sequence advances its own
 *       state).
 *  [P3] "PR #33465 完整报告" (SGLang Kimi-K3 on NPU), section "关键源码片段":
 *       the prefill decomposition l2norm -> chunk-local cumulative gate sum
 *       (scaled by log2 e) -> gated K K^T -> triangular solve -> W/U
 *       recompute -> inter-chunk state recurrence -> chunk output, with scale
 *       K^-1/2 and the output allowed to reuse v's buffer.
 *
 * Conventions shared by every entry point:
 *  - Ownership: the library owns no memory (except the static scratch of
 *    kda_chunk_prefill_noalloc).  The caller allocates every buffer (device
 *    memory unless stated) and passes the HIP stream on each call; no buffer
 *    or per-call state is retained between calls (the library looks up each
 *    device's CU count, and the scratch's address, once).
 *  - stream: a hipStream_t passed as void* (NULL = the default stream).  All
 *    work is enqueued on it; no entry point synchronises the device or reads
 *    device memory on the host.
 *  - Validation is host-only and fail-closed: a bad argument returns an error
 *    status and enqueues nothing.
 *  - Errors from the HIP runtime return KDA_E_HIP; kda_last_error_detail()
 *    then names the failing call (thread-local, valid until the next call on
 *    the same thread).
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { KDA_F32 = 0, KDA_BF16 = 1, KDA_E4M3 = 2 } kda_dtype_t; /* E4M3: codes of the 8-bit latent cache alone */
typedef enum { KDA_I32 = 0, KDA_I64 = 1 } kda_index_t;

typedef enum {
  KDA_OK = 0,
  KDA_E_NULL = 1,        /* a required pointer is NULL                                   */
  KDA_E_DTYPE = 2,       /* dtype / index type outside the supported set                 */
  KDA_E_SHAPE = 3,       /* negative or zero size where a positive one is required       */
  KDA_E_LAYOUT = 4,      /* cache inner dims [H,V,K] are not dense                       */
  KDA_E_OVERLAP = 5,     /* cache row stride smaller than the row payload (pages overlap) */
  KDA_E_UNSUPPORTED = 6, /* a size the library has no kernel for (e.g. K > 128)          */
  KDA_E_WORKSPACE = 7,   /* workspace missing or smaller than kda_chunk_prefill_workspace_size */
  KDA_E_ALIAS = 8,       /* an output overlaps an input or another output               */
  KDA_E_HIP = 9          /* the HIP runtime reported an error                           */
} kda_status_t;

/*
 * A view of one layer's recurrent-state cache: a 4-D tensor [num_rows, H, V, K].
 * Element (r, h, v, c) is S_h[c][v] of cache row r, where S_h is the K x V
 * state of head h (state rows are laid out [H][V][K], K fastest; [P1] section
 * "自动分发" gives the [N,H,V,K] shape).
 *  data      -- address of element (0,0,0,0): the storage offset is already
 *               applied (a tensor's data_ptr()).
 *  dtype     -- KDA_F32 or KDA_BF16.
 *  stride[4] -- element strides of the four dims.
 * Admissible layouts ([P1] section "自动分发"): num_rows > 0, H, V, K > 0;
 * reading the inner dims from the back, each has size 1 or a stride equal to
 * the running payload (stride[3] = 1, stride[2] = K, stride[1] = V*K); and
 * stride[0] >= H*V*K, so rows never overlap.  The gap between a row's payload
 * and the next row is never read or written, nor is anything before data.
 */
typedef struct {
  void* data;
  kda_dtype_t dtype;
  int64_t num_rows, H, V, K;
  int64_t stride[4];
} kda_state_cache_t;

/*
 * kda_state_gather -- [P1] section "数值契约", gather side.
 * For i in [0, num_selected):
 *   packed[i] = cache row indices[i]   if 0 <= indices[i] < num_rows and
 *                                       (flags == NULL or flags[i] != 0),
 *   packed[i] = all-zero bits           otherwise.
 *  indices     -- device array of num_selected int32 (KDA_I32) or int64
 *                 (KDA_I64) values, read in their own width (no conversion).
 *                 Duplicates are allowed.
 *  flags       -- device array of num_selected bytes, or NULL (all true).
 *  packed      -- device output [num_selected, H, V, K], contiguous, in the
 *                 cache dtype; every row is written.
 * Bits are copied unchanged.  num_selected == 0 validates the cache view and
 * enqueues nothing.  Preconditions (not checked): packed does not overlap the
 * cache.  Errors: KDA_E_NULL, KDA_E_DTYPE, KDA_E_SHAPE, KDA_E_LAYOUT,
 * KDA_E_OVERLAP, KDA_E_HIP.
 */
kda_status_t kda_state_gather(const kda_state_cache_t* cache, const void* indices, kda_index_t index_type,
                              int64_t num_selected, const uint8_t* flags, void* packed, void* stream);

/*
 * kda_state_scatter -- [P1] section "数值契约", scatter side.
 * For i in [0, num_selected): if 0 <= indices[i] < num_rows, cache row
 * indices[i] = packed[i]; other entries are skipped.  Initial-state flags
 * play no part: a valid target is always written.
 *  packed      -- device input [num_selected, H, V, K], contiguous, cache
 *                 dtype (convert final states to the cache dtype first).
 * Preconditions (not checked, no device-to-host scan): valid targets are
 * unique; packed does not overlap the cache.  num_selected == 0 enqueues
 * nothing.  Errors as for kda_state_gather.
 */
kda_status_t kda_state_scatter(const kda_state_cache_t* cache, const void* indices, kda_index_t index_type,
                               int64_t num_selected, const void* packed, void* stream);

/*
 * Arguments of kda_chunk_prefill.  All pointers are device pointers to
 * contiguous row-major arrays.
 *  T, N, H, K, V   -- tokens, sequences, heads, key dim (1..128), value dim (>= 1);
 *                     H * max(K, V) <= 2^22 (else KDA_E_UNSUPPORTED).
 *  q, k            -- [T, H, K] in qkv_dtype.           v -- [T, H, V] in qkv_dtype.
 *  g               -- [T, H, K] fp32: natural-log decay per key channel; the
 *                     state is multiplied by exp(g) (g <= 0 for a decay).
 *  beta            -- [T, H] in beta_dtype (fp32 or bf16).
 *  cu_seqlens      -- [N+1] int32 token offsets; sequence n is tokens
 *                     [cu_seqlens[n], cu_seqlens[n+1]).  Precondition (not
 *                     checked on the host): cu_seqlens[0] = 0, non-decreasing,
 *                     cu_seqlens[N] = T; the kernels clamp so that bad
 *                     offsets cannot address outside [0, T).
 *  initial_state   -- [N, H, V, K] in initial_dtype, element (n,h,v,c) =
 *                     S[c][v]; or NULL for zero initial states.
 *  out             -- [T, H, V] in qkv_dtype.  It may be exactly v (the
 *                     output then overwrites v, [P3]).
 *  final_state     -- [N, H, V, K] in final_dtype, or NULL.  fp32 states are
 *                     rounded to bf16 to nearest even when final_dtype is bf16.
 *                     It may be exactly initial_state with the same dtype
 *                     (the states are then updated in place).
 *  scale           -- read-out scale ([P3] uses K^-1/2).
 *  use_qk_l2norm   -- nonzero: q and k rows are divided by sqrt(|x|^2 + 1e-6).
 *  workspace       -- device scratch of at least
 *                     kda_chunk_prefill_workspace_size(T, N, H, K, V) bytes
 *                     (may be NULL when that size is 0).
 * Aliasing (checked on the host, KDA_E_ALIAS): the outputs -- out,
 * final_state, ckpt_states and the workspace's first
 * kda_chunk_prefill_workspace_size bytes -- overlap neither each other nor
 * any input (q, k, v, g, beta, cu_seqlens, initial_state, ckpt_cu), except
 * for the two exact aliases above.
 * Per sequence n and head h, with S the K x V fp32 state, this computes for
 * each token t in order ([P2] section 1.1 and the gated delta rule):
 *   S <- (I - beta_t k_t k_t^T) Diag(exp g_t) S + beta_t k_t v_t^T
 *   out_t = scale * S^T q_t
 * evaluated chunkwise in chunks of 64 tokens aligned to each sequence start
 * ([P3]).  Sequences of length 0 pass their initial state through.
 * Precision: the state, the gate sums, the row norms, the triangular
 * inverse's diagonal blocks and every accumulation are fp32; the operands of
 * the matrix products (the gated q/k tiles, the inverse, W, U, V_new and the
 * state as a right-hand operand) are rounded to bf16 -- for fp32 q/k/v too.
 * Against an fp64 evaluation of the recurrence this gives a relative L2
 * error of about 4e-3 on outputs and final states for bf16 and fp32 inputs
 * alike (tolerance 2e-2).
 */
typedef struct {
  int64_t T, N, H, K, V;
  const void* q;
  const void* k;
  const void* v;
  kda_dtype_t qkv_dtype;
  const float* g;
  const void* beta;
  kda_dtype_t beta_dtype;
  const int32_t* cu_seqlens;
  const void* initial_state;
  kda_dtype_t initial_dtype;
  void* out;
  void* final_state;
  kda_dtype_t final_dtype;
  float scale;
  int use_qk_l2norm;
  void* workspace;
  size_t workspace_bytes;
  /* Optional chunk-boundary checkpoints (prefix states that a cache can keep
   * and later resume from; [P2] section 1.3 and section 5.2's checkpoints at
   * chunk boundaries).  With ckpt_states != NULL, for sequence n the j-th
   * checkpoint (j = 0 .. ckpt_cu[n+1]-ckpt_cu[n]-1) is the state after
   * (j+1)*ckpt_interval tokens of that sequence, written to row ckpt_cu[n]+j
   * of ckpt_states ([num_ckpt, H, V, K], ckpt_dtype, same element order as
   * final_state, rounded like final_state).  Positions past the sequence's
   * length and rows outside [0, num_ckpt) are not written; the natural
   * choice is ckpt_cu[n+1]-ckpt_cu[n] = floor(len_n / ckpt_interval).
   * Chunks never straddle a multiple of 64 tokens of a sequence, so the
   * checkpoint states are exact chunk-boundary states, and requesting them
   * does not change out or final_state.
   *  ckpt_interval -- positive multiple of 64 (ignored when ckpt_states is NULL).
   *  ckpt_cu       -- [N+1] int32 device array of checkpoint row offsets,
   *                   non-decreasing (not checked).
   *  ckpt_states   -- device output, num_ckpt rows, or NULL for none.  It must
   *                   not overlap any other argument (checked, KDA_E_ALIAS). */
  int64_t ckpt_interval;
  const int32_t* ckpt_cu;
  void* ckpt_states;
  int64_t num_ckpt;
  kda_dtype_t ckpt_dtype;
} kda_prefill_args_t;

/* Bytes of device workspace kda_chunk_prefill needs for these sizes. */
size_t kda_chunk_prefill_workspace_size(int64_t T, int64_t N, int64_t H, int64_t K, int64_t V);

/*
 * kda_chunk_prefill -- the chunkwise gated delta rule of [P3] over a varlen
 * batch; see kda_prefill_args_t for arguments and semantics.
 * N == 0 enqueues nothing.  Errors: KDA_E_NULL, KDA_E_DTYPE, KDA_E_SHAPE,
 * KDA_E_UNSUPPORTED, KDA_E_WORKSPACE, KDA_E_ALIAS, KDA_E_HIP.
 */
kda_status_t kda_chunk_prefill(const kda_prefill_args_t* args, void* stream);

/*
 * Bytes of device scratch that kda_chunk_prefill_noalloc keeps on each device
 * it runs on: 256 MiB, more than kda_chunk_prefill_workspace_size returns for
 * any sizes kda_chunk_prefill accepts.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)

/*
 * kda_chunk_prefill_noalloc -- kda_chunk_prefill for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  Same arguments, semantics, validation and
 * kernels as kda_chunk_prefill, except that args->workspace and
 * args->workspace_bytes are ignored: the workspace is a static device array of
 * KDA_NOALLOC_SCRATCH_BYTES inside the library, one copy per device, created
 * when the library's code is loaded on that device and held until the process
 * ends.  The call allocates and frees nothing (no hipMalloc, no hipFree, no
 * allocating library routine) and enqueues no memset.  The first call on a
 * device looks up that device's copy (hipGetSymbolAddress) with the device
 * current.
 * Calls on one device share that device's array: two calls that can overlap
 * in time on one device (different streams, or different host threads with
 * no ordering between them) race on it and give undefined results; order
 * them on one stream or with events.  Calls on different devices do not
 * interact.  Nothing is carried from one call to the next.
 * Errors: as kda_chunk_prefill, with KDA_E_WORKSPACE when
 * kda_chunk_prefill_workspace_size(T, N, H, K, V) exceeds
 * KDA_NOALLOC_SCRATCH_BYTES (no accepted size does), and KDA_E_HIP if the
 * scratch array cannot be located on the current device.
 */
kda_status_t kda_chunk_prefill_noalloc(const kda_prefill_args_t* args, void* stream);

/*
 * Arguments of kda_recurrent_decode: one new token for each of N sequences.
 * All pointers are device pointers to contiguous row-major arrays.
 *  N, H, K, V      -- sequences (= tokens), heads, key dim (1..128), value dim (>= 1);
 *                     H, V, K must equal the cache's.
 *  q, k            -- [N, H, K] in qkv_dtype.       v -- [N, H, V] in qkv_dtype.
 *  g               -- [N, H, K] fp32 natural-log decays (state multiplied by exp(g)).
 *  beta            -- [N, H] in beta_dtype.
 *  state_indices   -- [N] int32 (KDA_I32) or int64 (KDA_I64): the cache row
 *                     holding sequence n's state, read in its own width.
 *  out             -- [N, H, V] in qkv_dtype; may be exactly v.
 *  scale, use_qk_l2norm -- as for kda_chunk_prefill.
 */
typedef struct {
  int64_t N, H, K, V;
  const void* q;
  const void* k;
  const void* v;
  kda_dtype_t qkv_dtype;
  const float* g;
  const void* beta;
  kda_dtype_t beta_dtype;
  const void* state_indices;
  kda_index_t index_type;
  void* out;
  float scale;
  int use_qk_l2norm;
} kda_decode_args_t;

/*
 * kda_recurrent_decode -- one step of the gated delta rule per sequence with
 * the state updated in place in its cache row ([P2] section 1.1 for one
 * token; decode runs its own recurrent kernel on the indexed state rows, [P1]
 * section "背景" and [P3] section "实现拆解").  For each n with
 * r = state_indices[n] in [0, num_rows) and each head h, with S the K x V
 * state of cache row r, head h (element (r,h,v,c) = S[c][v]):
 *   S <- (I - beta k^ k^T) Diag(exp g) S + beta k^ v^T   (written back to row r,
 *                                                       rounded to the cache dtype)
 *   out[n,h,:] = scale * S^T q^
 * computed in fp32.  An index outside [0, num_rows) marks a padding slot: its
 * output is zero and no cache row is read or written.
 * Preconditions (not checked, no device-to-host scan): valid indices are
 * unique within one call (rows are updated concurrently).  Aliasing (checked
 * on the host, KDA_E_ALIAS): neither the cache's address span nor out
 * overlaps q, k, v, g, beta, state_indices or the other, except that out may
 * be exactly v.
 * N == 0 validates the cache view and enqueues nothing.
 * Errors: KDA_E_NULL, KDA_E_DTYPE, KDA_E_SHAPE, KDA_E_LAYOUT, KDA_E_OVERLAP,
 * KDA_E_UNSUPPORTED, KDA_E_ALIAS, KDA_E_HIP.
 */
kda_status_t kda_recurrent_decode(const kda_state_cache_t* cache, const kda_decode_args_t* args, void* stream);

/*
 * A compressed (INT8) checkpoint store for one layer ([P2] section 5.3: parked
 * checkpoints compressed to INT8 and dequantised into a fresh active slot on
 * a hit; section 6.6.2: qdata [slots, heads, d_v, d_k] int8 and scale
 * [slots, heads, 1, d_k]).
 *  qdata         -- int8 codes; element (s, h, v, c) at qdata[s*qdata_stride0 + (h*V + v)*K + c].
 *  scale         -- fp32 scales; element (s, h, c) at scale[s*scale_stride0 + h*K + c].
 *  num_slots, H, V, K -- num_slots > 0, 1 <= K <= 128, H, V > 0.
 *  qdata_stride0 >= H*V*K and scale_stride0 >= H*K (slots never overlap); the
 *  qdata and scale address ranges must be disjoint.
 */
typedef struct {
  int8_t* qdata;
  float* scale;
  int64_t num_slots, H, V, K;
  int64_t qdata_stride0, scale_stride0;
} kda_int8_store_t;

/*
 * kda_ckpt_quantize_scatter -- for i in [0, num_selected): if
 * 0 <= indices[i] < num_slots, slot indices[i] receives packed[i] quantised
 * per (head, key channel c):
 *   amax_c  = max over v of |x[v][c]|,   scale_c = amax_c / 127   (fp32 division)
 *   code    = clamp(rint(x[v][c] / scale_c), -127, 127)            (fp32 division,
 *             ties to even), code = 0 where scale_c == 0.
 * Other entries are skipped.  packed: [num_selected, H, V, K] in packed_dtype
 * (fp32 or bf16), contiguous.  Preconditions (not checked): valid slots are
 * unique; finite inputs.  The store's qdata and scale ranges must not overlap
 * packed or indices (checked, KDA_E_ALIAS).  num_selected == 0 enqueues
 * nothing.
 * Errors: KDA_E_NULL, KDA_E_DTYPE, KDA_E_SHAPE, KDA_E_OVERLAP, KDA_E_UNSUPPORTED,
 * KDA_E_ALIAS, KDA_E_HIP.
 */
kda_status_t kda_ckpt_quantize_scatter(const kda_int8_store_t* store, const void* indices, kda_index_t index_type,
                                       int64_t num_selected, const void* packed, kda_dtype_t packed_dtype,
                                       void* stream);

/*
 * kda_ckpt_dequantize_gather -- for i in [0, num_selected):
 *   packed[i][h][v][c] = code * scale_c (fp32, then rounded to packed_dtype)
 *       if 0 <= indices[i] < num_slots and (flags == NULL or flags[i] != 0),
 *   packed[i] = zeros otherwise.
 * Every row of packed is written; the result can seed kda_chunk_prefill's
 * initial_state or go to active cache rows through kda_state_scatter.  packed
 * must not overlap the store, indices or flags (checked, KDA_E_ALIAS).
 * Errors as for kda_ckpt_quantize_scatter.
 */
kda_status_t kda_ckpt_dequantize_gather(const kda_int8_store_t* store, const void* indices, kda_index_t index_type,
                                        int64_t num_selected, const uint8_t* flags, void* packed,
                                        kda_dtype_t packed_dtype, void* stream);

/*
 * Arguments of kda_latent_prefill: attention with keys and values expanded per
 * head from one latent vector a token, over a packed batch.  All pointers are
 * device pointers; every tensor's last dim is dense and its other dims have
 * the element strides given.
 *  T, S, N, H      -- query tokens, key tokens, sequences, heads (T, S and N at
 *                     most 2^31 - 256, H at most 65535, and fewer than 2^24
 *                     workgroups, of which a head has (T + 127 N) / 128).
 *  D, R, E         -- key dim per head (8..128), rotary key dim shared by the
 *                     heads (0..64), value dim (8..128); multiples of 8.
 *  dtype           -- of q, k, k_rope, v and out: KDA_BF16.
 *  q               -- [T, H, D+R]; q_stride = {token, head}.
 *  k               -- [S, H, D];   k_stride = {token, head}.
 *  k_rope          -- [S, R], one row a token for all heads; k_rope_stride =
 *                     token stride (NULL with R == 0).
 *  v               -- [S, H, E];   v_stride = {token, head}.
 *                     q, k, k_rope and v are 16-byte aligned and their strides
 *                     are multiples of 8 elements, not negative (0: a broadcast
 *                     dim); the token strides of k, k_rope and v are at most 2^24.
 *  cu_seqlens_q    -- [N+1] int32 offsets of the sequences' queries in q.
 *  cu_seqlens_k    -- [N+1] int32 offsets of their keys in k, k_rope and v.
 *                     Both non-decreasing (not checked: the kernel clamps them
 *                     to the tensors and raises a query offset to the largest
 *                     before it, so bad offsets address nothing outside and no
 *                     query belongs to two sequences).
 *  out             -- [T, H, E] contiguous, 8-byte aligned.
 *  lse             -- [T, H] fp32, or NULL.
 *  scale           -- factor of the scores, positive, at most 2^127.
 *  causal          -- nonzero: query i of a sequence with Lq queries and Lk
 *                     keys sees keys j < Lk - (Lq - 1 - i), so its queries are
 *                     the last Lq of Lk positions; zero: it sees all Lk keys.
 *  workspace       -- device scratch, 16-byte aligned, of at least
 *                     kda_latent_prefill_workspace_size(T, S, N, H, E) bytes
 *                     (may be NULL when that size is 0).
 * For query i and head h of a sequence, over the keys j it sees:
 *   s_j = scale (q_i[:D] . k_j + q_i[D:] . k_rope_j)
 *   out_i = sum_j exp(s_j - lse_i) v_j,   lse_i = log sum_j exp(s_j)
 * A query that sees no key (or only keys whose score is -inf, as an infinite
 * component of a key can make it) gets out 0 and lse -inf.  Rows of q that
 * belong to no sequence have their out and lse rows left as they were.
 * Precision: products of bf16 operands with fp32 sums; scores (and their
 * products with log2 e, which count as infinite beyond fp32), the running
 * maximum and sum and the output accumulate in fp32; the softmax weights are
 * rounded to bf16 as operands of the second product.  The weights are taken against a
 * maximum that may be 2^8 too small, and the output is divided by their sum at the end:
 * where the keys that a query sees times the largest magnitude of a value pass 2^119, it
 * can be infinite or NaN although the formula's result is not.
 * A NaN or infinite value row v_j can reach queries that do not see key j but
 * see another key of the same 64 (their weight 0 multiplies it); keys and
 * rotary keys that a query does not see never reach it.
 */
typedef struct {
  int64_t T, S, N, H, D, R, E;
  kda_dtype_t dtype;
  const void* q;
  int64_t q_stride[2];
  const void* k;
  int64_t k_stride[2];
  const void* k_rope;
  int64_t k_rope_stride;
  const void* v;
  int64_t v_stride[2];
  const int32_t* cu_seqlens_q;
  const int32_t* cu_seqlens_k;
  void* out;
  float* lse;
  float scale;
  int causal;
  void* workspace;
  size_t workspace_bytes;
} kda_latent_prefill_args_t;

/* Bytes of device workspace kda_latent_prefill needs for these sizes: 0 unless
 * there are few queries and many keys, which are then split. */
size_t kda_latent_prefill_workspace_size(int64_t T, int64_t S, int64_t N, int64_t H, int64_t E);

/*
 * kda_latent_prefill -- see kda_latent_prefill_args_t.  Aliasing (checked on
 * the host, KDA_E_ALIAS): out, lse and the workspace overlap neither each
 * other nor any input.  Calls that can run at the same time need workspaces of
 * their own.  T == 0 or N == 0 enqueues nothing.
 * Errors: KDA_E_NULL, KDA_E_DTYPE, KDA_E_SHAPE, KDA_E_LAYOUT (alignment or
 * strides), KDA_E_UNSUPPORTED, KDA_E_WORKSPACE, KDA_E_ALIAS, KDA_E_HIP.
 */
kda_status_t kda_latent_prefill(const kda_latent_prefill_args_t* args, void* stream);

/*
 * Arguments of kda_latent_decode: Q new tokens for each of N sequences against
 * a paged cache of latent rows, in the absorbed form (the key up-projection
 * folded into q, the value up-projection applied to out by the caller).
 *  N, Q, H         -- sequences (<= 65535), new tokens a sequence (>= 1), heads;
 *                     Q * H <= 1024.
 *  L, R            -- latent dim (8..512), rotary key dim (0..64); multiples of 8.
 *  dtype           -- of the cache, q, q_rope and out: KDA_BF16.
 *  cache           -- [num_pages, page_size, L+R], dense inner dims, page_stride
 *                     elements (>= page_size (L+R), multiple of 8) from page to
 *                     page; 16-byte aligned.  Row = one token's latent vector,
 *                     then its rotary key.
 *  page_table      -- [N, max_pages] int32, rows table_stride apart; entry j of
 *                     row n is the page of sequence n's tokens j page_size ...
 *  lengths         -- [N] int32 tokens in the cache, the Q new ones included.
 *  q, q_rope       -- [N, Q, H, L], [N, Q, H, R] with strides {n, query, head}
 *                     (multiples of 8 elements), last dim dense, 16-byte
 *                     aligned; q_rope NULL with R == 0.
 *  out             -- [N, Q, H, L] contiguous, 16-byte aligned.
 *  lse             -- [N, Q, H] fp32, or NULL.
 *  scale           -- factor of the scores, positive, at most 2^127.
 *  workspace       -- device scratch, 16-byte aligned, of at least
 *                     kda_latent_decode_workspace_size(N, Q, H, L) bytes.
 * Query i of sequence n sees the rows j < lengths[n] - (Q - 1 - i):
 *   s_j = scale (q . row_j[:L] + q_rope . row_j[L:]),  out = sum_j softmax(s)_j row_j[:L]
 * A query that sees no row gets out 0 and lse -inf.  Rows whose page_table
 * entry lies outside [0, num_pages) are not seen; lengths are clamped to
 * [0, max_pages * page_size] (which may not exceed 2^30, nor 2^40 / N).
 * Rows of a page behind a sequence's length are not read.  The result does not
 * depend on the order of workgroups; how a sequence is split depends on the
 * whole batch's lengths, so its rounding may change with its neighbours'.
 * Precision as kda_latent_prefill; partial results of split sequences are fp32.
 * A non-finite row a later query of the same call sees can reach its earlier
 * queries, as in kda_latent_prefill.
 */
typedef struct {
  int64_t N, Q, H, L, R;
  kda_dtype_t dtype;
  const void* cache;
  int64_t num_pages, page_size, page_stride;
  const int32_t* page_table;
  int64_t table_stride, max_pages;
  const int32_t* lengths;
  const void* q;
  int64_t q_stride[3];
  const void* q_rope;
  int64_t q_rope_stride[3];
  void* out;
  float* lse;
  float scale;
  void* workspace;
  size_t workspace_bytes;
} kda_latent_decode_args_t;

/* Bytes of device workspace kda_latent_decode needs for these sizes. */
size_t kda_latent_decode_workspace_size(int64_t N, int64_t Q, int64_t H, int64_t L);

/*
 * kda_latent_decode -- see kda_latent_decode_args_t.  Aliasing (checked,
 * KDA_E_ALIAS): out, lse and the workspace overlap neither each other nor any
 * input.  Calls that can run at the same time need workspaces of their own.
 * N == 0 enqueues nothing.  The call can be captured: its work follows the
 * lengths and the table that each replay finds.
 * Errors: KDA_E_NULL, KDA_E_DTYPE, KDA_E_SHAPE, KDA_E_LAYOUT, KDA_E_OVERLAP,
 * KDA_E_UNSUPPORTED, KDA_E_WORKSPACE, KDA_E_ALIAS, KDA_E_HIP.
 */
kda_status_t kda_latent_decode(const kda_latent_decode_args_t* args, void* stream);

/*
 * An 8-bit latent cache: token rows in pages, a row as L e4m3 codes (1 sign, 4
 * exponent and 3 mantissa bits, largest 448, no infinity) with one fp32 scale, and
 * R rotary key components in bf16.  Its value is code * scale, and the rotary key.
 *  codes   -- [num_pages, page_size, L] bytes, 16-byte aligned.
 *  scales  -- [num_pages, page_size] fp32.
 *  rope    -- [num_pages, page_size, R] bf16, 16-byte aligned (NULL with R == 0).
 *             Pages are dense inside; from page to page lie codes_page_stride
 *             bytes (a multiple of 16), scales_page_stride fp32 and
 *             rope_page_stride bf16 (a multiple of 8).
 *             The three byte ranges, first page to last, lie apart (arrays that take turns
 *             page by page in one block of memory are refused, as by kda_page_fork).
 *  num_pages, page_size -- positive, num_pages * page_size below 2^31.
 *  L, R    -- latent dim (16..512, a multiple of 16), rotary key dim (0..64, a
 *             multiple of 8).
 * The three arrays are three stores for kda_page_fork and kda_page_compact.
 */
typedef struct {
  void* codes;
  float* scales;
  void* rope;
  int64_t num_pages, page_size, L, R;
  int64_t codes_page_stride, scales_page_stride, rope_page_stride;
} kda_latent_store_t;

/*
 * kda_latent_quantize_scatter -- for t in [0, num_rows): if 0 <= slots[t] <
 * num_pages * page_size, token row slots[t] (page slots[t] / page_size, place
 * slots[t] % page_size) receives row t:
 *   scale = 2^e with the smallest e >= -126 for which max |c| <= 448 2^e,
 *   code  = c / scale rounded to e4m3 (ties to even),
 *   rope  = k_rope rounded to bf16 (ties to even).
 * A row whose c holds an infinity or a NaN gets the scale NaN and codes 0: what
 * reads it gets NaN, and nothing else does.  Other entries are skipped.
 *  c       -- [num_rows, L], c_stride elements from row to row; k_rope
 *             [num_rows, R] with k_rope_stride (NULL with R == 0); both in dtype
 *             (KDA_F32 or KDA_BF16), dense last dim, 16-byte aligned, strides
 *             multiples of 8 elements, not negative.
 *  slots   -- [num_rows] int32 or int64; num_rows below 2^28.
 * Preconditions (not checked): valid slots are unique.  Aliasing (checked,
 * KDA_E_ALIAS): codes, scales and rope overlap neither each other nor c, k_rope or
 * slots.  num_rows == 0 enqueues nothing.
 * Errors: KDA_E_NULL, KDA_E_DTYPE, KDA_E_SHAPE, KDA_E_LAYOUT, KDA_E_OVERLAP,
 * KDA_E_UNSUPPORTED, KDA_E_ALIAS, KDA_E_HIP.
 */
kda_status_t kda_latent_quantize_scatter(const kda_latent_store_t* store, const void* c, int64_t c_stride,
                                         const void* k_rope, int64_t k_rope_stride, kda_dtype_t dtype,
                                         const void* slots, kda_index_t index_type, int64_t num_rows, void* stream);

/*
 * kda_latent_dequantize_gather -- out[t] = the value of token row slots[t], its L
 * latent components (code * scale in fp32, then rounded to dtype) and its R rotary
 * ones, or zeros where slots[t] lies outside [0, num_pages * page_size).
 *  out     -- [num_rows, L + R] in dtype (KDA_F32 or KDA_BF16), contiguous, 16-byte
 *             aligned: the layout of a 16-bit latent cache's rows.
 * Slots may repeat.  out overlaps neither the store nor slots (checked).
 * num_rows == 0 enqueues nothing.  Errors as for kda_latent_quantize_scatter.
 */
kda_status_t kda_latent_dequantize_gather(const kda_latent_store_t* store, const void* slots, kda_index_t index_type,
                                          int64_t num_rows, void* out, kda_dtype_t dtype, void* stream);

/*
 * Arguments of kda_latent_decode_fp8 and kda_latent_decode_shared: those of
 * kda_latent_decode with a cache in 16 or in 8 bits and with groups of
 * sequences that share their first tokens.
 *  cache_dtype     -- KDA_BF16: cache is [num_pages, page_size, L+R] bf16 and
 *                     page_stride in elements, as for kda_latent_decode; scales
 *                     and rope play no part.  KDA_E4M3: cache, scales and rope
 *                     are the three arrays of a kda_latent_store_t, with
 *                     page_stride (bytes), scales_page_stride and
 *                     rope_page_stride, and L is a multiple of 16.
 *  G               -- groups, 0 .. 65535 (0: no sharing).
 *  cu_groups       -- [G+1] int32: group g is the sequences cu_groups[g] ..
 *                     cu_groups[g+1] - 1.  Non-decreasing (not checked: the
 *                     kernel clamps offsets to [0, N] and raises one to the largest
 *                     before it).  Sequences of no group share nothing.
 *  shared          -- [G] int32: the first shared[g] tokens of the group's
 *                     sequences are the same rows.  They are read through the
 *                     table of the group's first sequence, up to its length;
 *                     the others' tables are read behind that.  Any number of
 *                     tokens, whole pages or not; negative: 0.
 *  The rest        -- as for kda_latent_decode, N Q H times max_pages *
 *                     page_size may not exceed 2^48, and with several pages the
 *                     page strides lie below 2^32 bytes.
 *  workspace       -- device scratch, 16-byte aligned, of at least
 *                     kda_latent_shared_workspace_size(N, Q, H, L, G) bytes.
 *                     (With groups it holds at least a block of 16, 32 or, above 32 query rows in
 *                     the batch, 64 rows of fp32 outputs for each sequence and group.)
 * When to share: a prefix is read once for 64 query rows and not once a sequence,
 * but the products stay the same and joining costs a launch's time.  On MI355X it
 * pays from about 64 sequences of up to 32 query rows (Q H) behind 4096 to 8192 tokens on (64
 * of 8 rows behind 32768 in one group: 86 us against 220), and does not for few sequences,
 * short prefixes (64 of 32 rows behind 1024: 43 against 37) and 128 rows and more, where
 * products bound both.  A shared length that is no multiple of 8, and pages of no multiple
 * of 8 tokens, cost up to a sixth more (tokens are then looked up one by one).
 * The result is that of kda_latent_decode, whose rules on lengths, pages, empty
 * rows and order of workgroups hold.  With a shared prefix, query rows see the
 * first rows through the first sequence's table: where that has no page, no sequence
 * of the group sees the row.
 * Precision: as kda_latent_decode; in 8 bits the codes enter both products as
 * bf16, which holds them whole, a token's scale multiplies its latent score in fp32,
 * and the softmax weight times the scale is rounded to bf16 once (below 2^-126 it
 * may count as 0).  Infinite results by large values are as there (2^119), in 8 bits by a
 * row's scale of 2^119 and more too.
 * Codes must not be NaN (0x7f, 0xff): such a code can reach all queries of a tile of
 * 64 tokens.  A NaN or infinite scale, or a NaN in a rotary key, reaches the queries
 * that see its row and no others.
 */
typedef struct {
  int64_t N, Q, H, L, R, G;
  kda_dtype_t cache_dtype;
  const void* cache;
  const float* scales;
  const void* rope;
  int64_t num_pages, page_size;
  int64_t page_stride, scales_page_stride, rope_page_stride;
  const int32_t* page_table;
  int64_t table_stride, max_pages;
  const int32_t* lengths;
  const int32_t* cu_groups;
  const int32_t* shared;
  const void* q;
  int64_t q_stride[3];
  const void* q_rope;
  int64_t q_rope_stride[3];
  void* out;
  float* lse;
  float scale;
  void* workspace;
  size_t workspace_bytes;
} kda_latent_shared_args_t;

/* Bytes of device workspace kda_latent_decode_fp8 (G = 0) and
 * kda_latent_decode_shared need for these sizes. */
size_t kda_latent_shared_workspace_size(int64_t N, int64_t Q, int64_t H, int64_t L, int64_t G);

/*
 * kda_latent_decode_fp8 -- latent decode over an 8-bit cache: cache_dtype is
 * KDA_E4M3 and G is 0.  kda_latent_decode_shared -- either cache, any G.
 * Aliasing (checked, KDA_E_ALIAS): out, lse and the workspace overlap neither each
 * other nor any input.  Calls that can run at the same time need workspaces of
 * their own.  N == 0 enqueues nothing.  The calls can be captured: their work
 * follows the lengths, the tables and the groups that each replay finds.
 * Errors: as for kda_latent_decode.
 */
kda_status_t kda_latent_decode_fp8(const kda_latent_shared_args_t* args, void* stream);
kda_status_t kda_latent_decode_shared(const kda_latent_shared_args_t* args, void* stream);

/*
 * The bookkeeping of a cache's pages, all on the device: sequence slot s holds
 * lengths[s] tokens in the pages table[s * table_stride + j],
 * j < ceil(lengths[s] / page_size); refs[p] says how many slots hold page p,
 * and a page is free when refs[p] <= 0.  A slot of length 0 is empty.  A state
 * cache is a pool with page_size 1, one page a slot and lengths 0 or 1.
 *  num_seqs, max_pages, num_pages, page_size -- positive; num_seqs <= 2^24,
 *   max_pages <= 2^20, num_pages <= 2^30, page_size <= 2^30.
 *   table_stride >= max_pages.
 */
typedef struct {
  int32_t* table;
  int64_t table_stride, num_seqs, max_pages;
  int32_t* lengths;
  int32_t* refs;
  int64_t num_pages, page_size;
} kda_page_pool_t;

/*
 * One layer's pages: page p is the page_bytes bytes at data + p * page_stride
 * (bytes; page_stride >= page_bytes > 0).  The gap between pages is never
 * read or written.  A pool serves any number of stores; layers that lie side
 * by side in one page are one store.
 */
typedef struct {
  void* data;
  int64_t page_stride, page_bytes;
} kda_page_store_t;

/*
 * kda_page_fork -- slot dst[i] becomes a child of slot src[i], i < num_forks.
 *  share != 0: the child holds the parent's full pages too (refs + 1) and
 *   takes one free page for a copy of a partly filled last page.  For pages
 *   that are only appended to.
 *  share == 0: the child takes as many free pages as the parent has and all
 *   are copied.  For pages that are updated in place (recurrent states).
 * Entries are served in order, and free pages are taken in ascending order.
 * status[i] receives
 *  2 if src[i] or dst[i] is no slot, both are the same, dst[i] is not empty or
 *    is an earlier entry's dst too, the parent's length is negative or above
 *    max_pages * page_size, or one of the parent's pages is outside
 *    [0, num_pages) or has refs <= 0;
 *  1 if the pages of this entry and the served or unserved sound ones before
 *    it are not all free;
 *  0 if it was served: table row dst[i] holds the child's pages and -1 behind
 *    them, lengths[dst[i]] = lengths[src[i]], the pages taken have refs 1 and
 *    every store's copies are done.
 * Unserved entries change nothing.  All entries see the pool as it was before
 * the call.
 *  src, dst  -- [num_forks] int32 or int64 device arrays; num_forks <= 65536.
 *  stores    -- host array of num_stores stores (0 .. 4096; NULL with 0).
 *  status    -- [num_forks] int32 device output.
 *  workspace -- device scratch (4-byte aligned) of
 *               kda_page_fork_workspace_size bytes.
 * Aliasing (checked, KDA_E_ALIAS): table, lengths, refs, status, the workspace
 * and the stores' spans are disjoint from each other and from src and dst.
 * num_forks == 0 enqueues nothing.  Errors: KDA_E_NULL, KDA_E_DTYPE,
 * KDA_E_SHAPE, KDA_E_OVERLAP, KDA_E_UNSUPPORTED, KDA_E_WORKSPACE, KDA_E_ALIAS,
 * KDA_E_HIP.
 */
kda_status_t kda_page_fork(const kda_page_pool_t* pool, const kda_page_store_t* stores, int64_t num_stores,
                           const void* src, const void* dst, kda_index_t index_type, int64_t num_forks, int share,
                           int32_t* status, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace kda_page_fork needs for these sizes. */
size_t kda_page_fork_workspace_size(int64_t num_forks, int64_t max_pages, int64_t num_pages, int share);

/*
 * kda_page_compact -- moves the pages in use to the front.  With n pages in
 * use (refs > 0), the k-th page in use of index >= n goes to the k-th free
 * page of index < n: every store's page is copied, refs moves along and the
 * slots' table entries are renamed (those within a slot's length).  Pages
 * below n that are in use stay where they are; afterwards pages [0, n) are in
 * use and all others free.
 *  live      -- device output, one int32: n; or NULL.
 *  workspace -- device scratch (4-byte aligned) of
 *               kda_page_compact_workspace_size(num_pages) bytes.
 * Aliasing and errors as for kda_page_fork.
 */
kda_status_t kda_page_compact(const kda_page_pool_t* pool, const kda_page_store_t* stores, int64_t num_stores,
                              int32_t* live, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace kda_page_compact needs. */
size_t kda_page_compact_workspace_size(int64_t num_pages);

/*
 * kda_page_free -- for every slot s with release[s] != 0 ([num_seqs] bytes on
 * the device): refs - 1 for each of its pages (entries outside
 * [0, num_pages) are passed over), its entries -1, its length 0.  Page
 * contents stay.  Aliasing (checked): table, lengths, refs and release are
 * disjoint.
 * Errors: KDA_E_NULL, KDA_E_SHAPE, KDA_E_OVERLAP, KDA_E_UNSUPPORTED,
 * KDA_E_ALIAS, KDA_E_HIP.
 */
kda_status_t kda_page_free(const kda_page_pool_t* pool, const uint8_t* release, void* stream);

/* Static, human-readable name of a status code. */
const char* kda_status_string(kda_status_t status);

/* Detail of the last KDA_E_HIP on this thread ("" if none). */
const char* kda_last_error_detail(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
