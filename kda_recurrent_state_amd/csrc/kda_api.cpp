// Host entry points of libkda: argument validation and kernel dispatch.
//
// Validation is host-only and fail-closed, as the copy contract of the page
// "vllm-ascend 的 KDA 状态复制 Triton 集成：PR 17301 对齐的预编译 worker 生命周期方案"
// asks (sections "数值契约" and "启动准备"): no device reads, no
// synchronisation, no environment scan, no conversion of int32 indices; a bad
// layout returns an error and enqueues nothing; an empty selection validates
// the cache view and enqueues nothing.
#include <string.h>

#include "internal.h"

namespace {

thread_local char g_detail[256] = "";

void set_detail(const char* what, hipError_t e) {
  const char* s = hipGetErrorString(e);
  size_t n = strlen(what);
  if (n > 100) n = 100;
  memcpy(g_detail, what, n);
  g_detail[n] = ':';
  g_detail[n + 1] = ' ';
  strncpy(g_detail + n + 2, s ? s : "?", sizeof(g_detail) - n - 3);
  g_detail[sizeof(g_detail) - 1] = 0;
}

kda_status_t hip_status(const char* what, hipError_t e) {
  if (e == hipSuccess) return KDA_OK;
  set_detail(what, e);
  return KDA_E_HIP;
}

int64_t dtype_bytes(kda_dtype_t d) { return d == KDA_F32 ? 4 : (d == KDA_BF16 ? 2 : 0); }

bool valid_dtype(kda_dtype_t d) { return d == KDA_F32 || d == KDA_BF16; }

// Layout admissibility: 4-D, num_rows > 0, positive inner sizes, inner dims
// dense from the back (size 1 or stride = running payload), rows disjoint.
kda_status_t check_cache(const kda_state_cache_t* c, int64_t* payload_elems) {
  if (!c) return KDA_E_NULL;
  if (!valid_dtype(c->dtype)) return KDA_E_DTYPE;
  if (c->num_rows <= 0 || c->H <= 0 || c->V <= 0 || c->K <= 0) return KDA_E_SHAPE;
  const int64_t sizes[3] = {c->H, c->V, c->K};
  int64_t run = 1;
  for (int d = 2; d >= 0; --d) {
    if (sizes[d] != 1 && c->stride[d + 1] != run) return KDA_E_LAYOUT;
    if (run > ((int64_t)1 << 40) / sizes[d]) return KDA_E_SHAPE;
    run *= sizes[d];
  }
  if (c->stride[0] < run) return KDA_E_OVERLAP;
  if (c->stride[0] > ((int64_t)1 << 46) / c->num_rows) return KDA_E_SHAPE;
  if (!c->data) return KDA_E_NULL;
  *payload_elems = run;
  return KDA_OK;
}

kda_status_t copy_common(bool gather, const kda_state_cache_t* cache, const void* indices, kda_index_t it,
                         int64_t num_selected, const uint8_t* flags, void* packed, void* stream) {
  int64_t payload = 0;
  kda_status_t st = check_cache(cache, &payload);
  if (st != KDA_OK) return st;
  if (it != KDA_I32 && it != KDA_I64) return KDA_E_DTYPE;
  if (num_selected < 0) return KDA_E_SHAPE;
  if (num_selected == 0) return KDA_OK;
  if (!indices || !packed) return KDA_E_NULL;
  const int64_t eb = dtype_bytes(cache->dtype);
  hipError_t e = kda::launch_state_copy(gather, static_cast<char*>(cache->data), cache->stride[0] * eb,
                                        cache->num_rows, payload * eb, indices, it == KDA_I64, num_selected,
                                        gather ? flags : nullptr, static_cast<char*>(packed),
                                        static_cast<hipStream_t>(stream));
  return hip_status(gather ? "kda_state_gather launch" : "kda_state_scatter launch", e);
}

bool ranges_overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

// A device byte range; an absent argument has p == NULL or bytes == 0.
struct Span {
  const void* p;
  int64_t bytes;
};

bool spans_overlap(const Span& a, const Span& b) {
  return a.p && b.p && a.bytes > 0 && b.bytes > 0 && ranges_overlap(a.p, a.bytes, b.p, b.bytes);
}

// Every output must be disjoint from every input and from the other outputs,
// except for the pairs (outs[i], ins[same[i]]) that are the very same range
// (same[i] < 0: no such exception).
bool alias_error(const Span* outs, const int* same, int nouts, const Span* ins, int nins) {
  for (int i = 0; i < nouts; ++i) {
    for (int j = 0; j < nins; ++j) {
      if (!spans_overlap(outs[i], ins[j])) continue;
      if (same[i] == j && outs[i].p == ins[j].p && outs[i].bytes == ins[j].bytes) continue;
      return true;
    }
    for (int j = i + 1; j < nouts; ++j)
      if (spans_overlap(outs[i], outs[j])) return true;
  }
  return false;
}

kda_status_t int8_common(bool quantize, const kda_int8_store_t* st, const void* indices, kda_index_t it,
                         int64_t num_selected, const uint8_t* flags, void* packed, kda_dtype_t pdt, void* stream) {
  if (!st) return KDA_E_NULL;
  if (st->num_slots <= 0 || st->H <= 0 || st->V <= 0 || st->K <= 0) return KDA_E_SHAPE;
  if (st->K > 128) return KDA_E_UNSUPPORTED;
  if (st->H * st->V > ((int64_t)1 << 40) / st->K) return KDA_E_SHAPE;
  const int64_t qpay = st->H * st->V * st->K, spay = st->H * st->K;
  if (st->qdata_stride0 < qpay || st->scale_stride0 < spay) return KDA_E_OVERLAP;
  if (st->qdata_stride0 > ((int64_t)1 << 46) / st->num_slots || st->scale_stride0 > ((int64_t)1 << 46) / st->num_slots)
    return KDA_E_SHAPE;
  if (!st->qdata || !st->scale) return KDA_E_NULL;
  if (ranges_overlap(st->qdata, (st->num_slots - 1) * st->qdata_stride0 + qpay, st->scale,
                     ((st->num_slots - 1) * st->scale_stride0 + spay) * 4))
    return KDA_E_OVERLAP;
  if (!valid_dtype(pdt)) return KDA_E_DTYPE;
  if (it != KDA_I32 && it != KDA_I64) return KDA_E_DTYPE;
  if (num_selected < 0) return KDA_E_SHAPE;
  if (num_selected > ((int64_t)1 << 40) / qpay) return KDA_E_SHAPE;
  if (num_selected == 0) return KDA_OK;
  if (!indices || !packed) return KDA_E_NULL;
  {
    const Span qd{st->qdata, (st->num_slots - 1) * st->qdata_stride0 + qpay};
    const Span sc{st->scale, ((st->num_slots - 1) * st->scale_stride0 + spay) * 4};
    const Span pk{packed, num_selected * qpay * dtype_bytes(pdt)};
    const Span ix{indices, num_selected * (it == KDA_I64 ? 8 : 4)};
    const Span fl{quantize ? nullptr : flags, num_selected};
    const int none[2] = {-1, -1};
    if (quantize) {
      const Span outs[2] = {qd, sc}, ins[2] = {pk, ix};
      if (alias_error(outs, none, 2, ins, 2)) return KDA_E_ALIAS;
    } else {
      const Span outs[1] = {pk}, ins[4] = {qd, sc, ix, fl};
      if (alias_error(outs, none, 1, ins, 4)) return KDA_E_ALIAS;
    }
  }
  hipError_t e = kda::launch_int8_ckpt(quantize, *st, indices, it == KDA_I64, num_selected, quantize ? nullptr : flags,
                                       packed, pdt == KDA_BF16, static_cast<hipStream_t>(stream));
  return hip_status(quantize ? "kda_ckpt_quantize_scatter launch" : "kda_ckpt_dequantize_gather launch", e);
}

}  // namespace

extern "C" {

kda_status_t kda_state_gather(const kda_state_cache_t* cache, const void* indices, kda_index_t index_type,
                              int64_t num_selected, const uint8_t* flags, void* packed, void* stream) {
  return copy_common(true, cache, indices, index_type, num_selected, flags, packed, stream);
}

kda_status_t kda_state_scatter(const kda_state_cache_t* cache, const void* indices, kda_index_t index_type,
                               int64_t num_selected, const void* packed, void* stream) {
  return copy_common(false, cache, indices, index_type, num_selected, nullptr, const_cast<void*>(packed), stream);
}

size_t kda_chunk_prefill_workspace_size(int64_t T, int64_t N, int64_t H, int64_t K, int64_t V) {
  return kda::chunk_prefill_workspace_bytes(T, N, H, K, V);
}

}  // extern "C"

namespace {

// Validation shared by kda_chunk_prefill and kda_chunk_prefill_noalloc: every
// check but the caller's workspace.  *need receives the workspace bytes the
// call uses; KDA_OK with a->N == 0 means there is nothing to enqueue.
kda_status_t check_prefill(const kda_prefill_args_t* a, size_t* need) {
  *need = 0;
  if (!a) return KDA_E_NULL;
  if (a->T < 0 || a->N < 0 || a->H <= 0 || a->K <= 0 || a->V <= 0) return KDA_E_SHAPE;
  if (a->N == 0 && a->T != 0) return KDA_E_SHAPE;
  if (!valid_dtype(a->qkv_dtype) || !valid_dtype(a->beta_dtype)) return KDA_E_DTYPE;
  if (a->initial_state && !valid_dtype(a->initial_dtype)) return KDA_E_DTYPE;
  if (a->final_state && !valid_dtype(a->final_dtype)) return KDA_E_DTYPE;
  if (a->K > 128) return KDA_E_UNSUPPORTED;
  if (a->H * (a->K > a->V ? a->K : a->V) > ((int64_t)1 << 22)) return KDA_E_UNSUPPORTED;  // 32-bit chunk offsets
  if (a->ckpt_states) {
    if (a->ckpt_interval <= 0 || a->ckpt_interval % 64 != 0 || a->num_ckpt < 0) return KDA_E_SHAPE;
    if (!a->ckpt_cu) return KDA_E_NULL;
    if (!valid_dtype(a->ckpt_dtype)) return KDA_E_DTYPE;
  }
  if (a->T > ((int64_t)1 << 40) / (a->H * (a->K > a->V ? a->K : a->V))) return KDA_E_SHAPE;
  if (a->N > ((int64_t)1 << 40) / (a->H * a->V * a->K)) return KDA_E_SHAPE;
  if (a->ckpt_states && a->num_ckpt > ((int64_t)1 << 40) / (a->H * a->V * a->K)) return KDA_E_SHAPE;
  if (a->N == 0) return KDA_OK;
  if (!a->cu_seqlens) return KDA_E_NULL;
  if (a->T > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->out)) return KDA_E_NULL;
  *need = kda::chunk_prefill_workspace_bytes(a->T, a->N, a->H, a->K, a->V);
  {
    // out may be exactly v and final_state exactly initial_state (same
    // dtype); any other overlap between an output and an argument is an error
    const int64_t eb = dtype_bytes(a->qkv_dtype), TH = a->T * a->H, NHVK = a->N * a->H * a->V * a->K;
    const Span vin{a->v, TH * a->V * eb};
    const Span init{a->initial_state, a->initial_state ? NHVK * dtype_bytes(a->initial_dtype) : 0};
    const Span ins[8] = {{a->q, TH * a->K * eb},
                         {a->k, TH * a->K * eb},
                         vin,
                         {a->g, TH * a->K * 4},
                         {a->beta, TH * dtype_bytes(a->beta_dtype)},
                         {a->cu_seqlens, (a->N + 1) * 4},
                         init,
                         {a->ckpt_states ? a->ckpt_cu : nullptr, (a->N + 1) * 4}};
    const Span outs[4] = {{a->out, TH * a->V * eb},
                          {a->final_state, a->final_state ? NHVK * dtype_bytes(a->final_dtype) : 0},
                          {a->ckpt_states, a->ckpt_states ? a->num_ckpt * a->H * a->V * a->K * dtype_bytes(a->ckpt_dtype) : 0},
                          {*need > 0 ? a->workspace : nullptr, (int64_t)*need}};
    const int same[4] = {2, 6, -1, -1};
    if (alias_error(outs, same, 4, ins, 8)) return KDA_E_ALIAS;
  }
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_chunk_prefill(const kda_prefill_args_t* a, void* stream) {
  size_t need = 0;
  const kda_status_t st = check_prefill(a, &need);
  if (st != KDA_OK || a->N == 0) return st;
  if (need > 0 && (!a->workspace || a->workspace_bytes < need)) return KDA_E_WORKSPACE;
  hipError_t e = kda::launch_chunk_prefill(*a, static_cast<hipStream_t>(stream));
  return hip_status("kda_chunk_prefill launch", e);
}

kda_status_t kda_chunk_prefill_noalloc(const kda_prefill_args_t* a, void* stream) {
  kda_prefill_args_t b;
  size_t need = 0;
  if (a) {
    // the caller's workspace fields play no part
    b = *a;
    b.workspace = nullptr;
    b.workspace_bytes = 0;
  }
  const kda_status_t st = check_prefill(a ? &b : nullptr, &need);
  if (st != KDA_OK || b.N == 0) return st;
  if (need > KDA_NOALLOC_SCRATCH_BYTES) return KDA_E_WORKSPACE;
  if (need > 0) {
    // this device's copy of the library's scratch array (set up on the first
    // call on each device)
    hipError_t e = kda::noalloc_scratch(&b.workspace);
    if (e != hipSuccess) return hip_status("kda_chunk_prefill_noalloc scratch lookup", e);
    b.workspace_bytes = KDA_NOALLOC_SCRATCH_BYTES;
  }
  hipError_t e = kda::launch_chunk_prefill(b, static_cast<hipStream_t>(stream));
  return hip_status("kda_chunk_prefill_noalloc launch", e);
}

kda_status_t kda_recurrent_decode(const kda_state_cache_t* cache, const kda_decode_args_t* a, void* stream) {
  int64_t payload = 0;
  kda_status_t st = check_cache(cache, &payload);
  if (st != KDA_OK) return st;
  if (!a) return KDA_E_NULL;
  if (a->N < 0 || a->H <= 0 || a->K <= 0 || a->V <= 0) return KDA_E_SHAPE;
  if (a->H != cache->H || a->V != cache->V || a->K != cache->K) return KDA_E_SHAPE;
  if (!valid_dtype(a->qkv_dtype) || !valid_dtype(a->beta_dtype)) return KDA_E_DTYPE;
  if (a->index_type != KDA_I32 && a->index_type != KDA_I64) return KDA_E_DTYPE;
  if (a->K > 128) return KDA_E_UNSUPPORTED;
  if (a->V * a->K * 4 >= ((int64_t)1 << 31)) return KDA_E_UNSUPPORTED;  // 32-bit offsets within a head's state
  if (a->N > ((int64_t)1 << 40) / (a->H * (a->K > a->V ? a->K : a->V))) return KDA_E_SHAPE;
  if (a->N == 0) return KDA_OK;
  if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->state_indices || !a->out) return KDA_E_NULL;
  {
    // the cache rows are updated in place; out may be exactly v; any other
    // overlap between the cache or out and an argument is an error
    const int64_t eb = dtype_bytes(a->qkv_dtype), NH = a->N * a->H;
    const Span ins[6] = {{a->q, NH * a->K * eb},
                         {a->k, NH * a->K * eb},
                         {a->v, NH * a->V * eb},
                         {a->g, NH * a->K * 4},
                         {a->beta, NH * dtype_bytes(a->beta_dtype)},
                         {a->state_indices, a->N * (a->index_type == KDA_I64 ? 8 : 4)}};
    const Span outs[2] = {{a->out, NH * a->V * eb},
                          {cache->data, ((cache->num_rows - 1) * cache->stride[0] + payload) * dtype_bytes(cache->dtype)}};
    const int same[2] = {2, -1};
    if (alias_error(outs, same, 2, ins, 6)) return KDA_E_ALIAS;
  }
  hipError_t e = kda::launch_recurrent_decode(*cache, *a, static_cast<hipStream_t>(stream));
  return hip_status("kda_recurrent_decode launch", e);
}

kda_status_t kda_ckpt_quantize_scatter(const kda_int8_store_t* store, const void* indices, kda_index_t index_type,
                                       int64_t num_selected, const void* packed, kda_dtype_t packed_dtype,
                                       void* stream) {
  return int8_common(true, store, indices, index_type, num_selected, nullptr, const_cast<void*>(packed),
                     packed_dtype, stream);
}

kda_status_t kda_ckpt_dequantize_gather(const kda_int8_store_t* store, const void* indices, kda_index_t index_type,
                                        int64_t num_selected, const uint8_t* flags, void* packed,
                                        kda_dtype_t packed_dtype, void* stream) {
  return int8_common(false, store, indices, index_type, num_selected, flags, packed, packed_dtype, stream);
}

}  // extern "C"

namespace {

constexpr int64_t kMaxSpan = (int64_t)1 << 46;  // elements a tensor may span

bool aligned(const void* p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

// Span in elements of a tensor with a dense last dim of ``last`` elements and
// ``n`` outer dims; false if a stride is negative or no multiple of 8, or the
// span passes kMaxSpan.
bool outer_span(const int64_t* size, const int64_t* stride, int n, int64_t last, int64_t* span) {
  int64_t end = last;
  for (int i = 0; i < n; ++i) {
    if (size[i] == 1) continue;  // its stride plays no part
    if (stride[i] < 0 || stride[i] % 8 != 0) return false;
    if (stride[i] > 0 && size[i] - 1 > (kMaxSpan - end) / stride[i]) return false;
    end += (size[i] - 1) * stride[i];
  }
  *span = end;
  return true;
}

// Factor of the scores: its product with log2 e is finite.
constexpr float kMostScale = 0x1p127f;

// Tokens of a packed batch of latent attention: the kernel counts in 31 bits to
// the end of the last tile (of 128 queries, of 64 keys).
constexpr int64_t kMostTokens = 0x7fffff00;

bool dim8(int64_t x, int64_t lo, int64_t hi) { return x >= lo && x <= hi && x % 8 == 0; }

kda_status_t check_latent_prefill(const kda_latent_prefill_args_t* a) {
  if (!a) return KDA_E_NULL;
  if (a->T < 0 || a->S < 0 || a->N < 0 || a->H <= 0 || a->D <= 0 || a->R < 0 || a->E <= 0) return KDA_E_SHAPE;
  if (a->N == 0 && a->T != 0) return KDA_E_SHAPE;
  if (a->dtype != KDA_BF16) return KDA_E_DTYPE;
  if (!dim8(a->D, 8, 128) || !dim8(a->R, 0, 64) || !dim8(a->E, 8, 128)) return KDA_E_UNSUPPORTED;
  if (!(a->scale > 0.f && a->scale <= kMostScale)) return KDA_E_UNSUPPORTED;
  if (a->T > kMostTokens || a->S > kMostTokens || a->N > kMostTokens || a->H > 65535) return KDA_E_UNSUPPORTED;
  // (HIP launches fewer than 2^32 threads a grid dimension; a workgroup has 256)
  if (a->N > 0 && kda::latent_prefill_workgroups(a->T, a->S, a->N, a->H) >= (int64_t)1 << 24) return KDA_E_UNSUPPORTED;
  if (a->T == 0 || a->N == 0) return KDA_OK;
  if (!a->q || !a->cu_seqlens_q || !a->cu_seqlens_k || !a->out) return KDA_E_NULL;
  if (a->S > 0 && (!a->k || !a->v || (a->R > 0 && !a->k_rope))) return KDA_E_NULL;
  int64_t qn = 0, kn = 0, rn = 0, vn = 0;
  const int64_t th[2] = {a->T, a->H}, sh[2] = {a->S > 0 ? a->S : 1, a->H};
  if (!outer_span(th, a->q_stride, 2, a->D + a->R, &qn) || !outer_span(sh, a->k_stride, 2, a->D, &kn) ||
      !outer_span(sh, a->v_stride, 2, a->E, &vn) || (a->R > 0 && !outer_span(sh, &a->k_rope_stride, 1, a->R, &rn)))
    return KDA_E_LAYOUT;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || (a->R > 0 && !aligned(a->k_rope, 16)) ||
      !aligned(a->out, 8))
    return KDA_E_LAYOUT;
  // (the kernel's offsets within a tile of 64 keys are 32-bit)
  const int64_t far = (int64_t)1 << 24;
  if (a->S > 1 && (a->k_stride[0] > far || a->v_stride[0] > far || (a->R > 0 && a->k_rope_stride > far)))
    return KDA_E_UNSUPPORTED;
  if (a->S == 0) kn = vn = rn = 0;
  const size_t need = kda::latent_prefill_workspace_bytes(a->T, a->S, a->N, a->H, a->E);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need)) return KDA_E_WORKSPACE;
  if (need > 0 && !aligned(a->workspace, 16)) return KDA_E_LAYOUT;
  const Span ins[6] = {{a->q, qn * 2},
                       {a->k, kn * 2},
                       {a->R > 0 ? a->k_rope : nullptr, rn * 2},
                       {a->v, vn * 2},
                       {a->cu_seqlens_q, (a->N + 1) * 4},
                       {a->cu_seqlens_k, (a->N + 1) * 4}};
  const Span outs[3] = {{a->out, a->T * a->H * a->E * 2},
                        {a->lse, a->T * a->H * 4},
                        {need > 0 ? a->workspace : nullptr, (int64_t)need}};
  const int same[3] = {-1, -1, -1};
  return alias_error(outs, same, 3, ins, 6) ? KDA_E_ALIAS : KDA_OK;
}

kda_status_t check_latent_decode(const kda_latent_decode_args_t* a) {
  if (!a) return KDA_E_NULL;
  if (a->N < 0 || a->Q <= 0 || a->H <= 0 || a->L <= 0 || a->R < 0) return KDA_E_SHAPE;
  if (a->num_pages <= 0 || a->page_size <= 0 || a->max_pages <= 0) return KDA_E_SHAPE;
  if (a->dtype != KDA_BF16) return KDA_E_DTYPE;
  if (!dim8(a->L, 8, 512) || !dim8(a->R, 0, 64)) return KDA_E_UNSUPPORTED;
  if (a->Q > 1024 || a->H > 1024 || a->Q * a->H > 1024) return KDA_E_UNSUPPORTED;
  if (a->N > 65535) return KDA_E_UNSUPPORTED;  // sequences are a grid dimension
  if (!(a->scale > 0.f && a->scale <= kMostScale)) return KDA_E_UNSUPPORTED;
  const int64_t most = (int64_t)1 << 30, row = a->L + a->R;
  if (a->page_size > most || a->max_pages > most / a->page_size || a->num_pages > 0x7fffffff) return KDA_E_UNSUPPORTED;
  // (a workgroup's tiles are counted in 31 bits)
  if (a->N > 1 && a->max_pages * a->page_size > ((int64_t)1 << 40) / a->N) return KDA_E_UNSUPPORTED;
  if (a->N > 1 && a->table_stride < a->max_pages) return KDA_E_OVERLAP;
  if (a->page_stride < a->page_size * row) return KDA_E_OVERLAP;
  if (a->page_stride % 8 != 0) return KDA_E_LAYOUT;
  if (a->page_stride > kMaxSpan / a->num_pages || (a->N > 1 && a->table_stride > kMaxSpan / a->N)) return KDA_E_SHAPE;
  if (a->N == 0) return KDA_OK;
  if (!a->cache || !a->page_table || !a->lengths || !a->q || (a->R > 0 && !a->q_rope) || !a->out) return KDA_E_NULL;
  const int64_t nqh[3] = {a->N, a->Q, a->H};
  int64_t qn = 0, rn = 0;
  if (!outer_span(nqh, a->q_stride, 3, a->L, &qn) || (a->R > 0 && !outer_span(nqh, a->q_rope_stride, 3, a->R, &rn)))
    return KDA_E_LAYOUT;
  if (!aligned(a->cache, 16) || !aligned(a->q, 16) || (a->R > 0 && !aligned(a->q_rope, 16)) || !aligned(a->out, 16))
    return KDA_E_LAYOUT;
  const size_t need = kda::latent_decode_workspace_bytes(a->N, a->Q, a->H, a->L);
  if (!a->workspace || a->workspace_bytes < need) return KDA_E_WORKSPACE;
  if (!aligned(a->workspace, 16)) return KDA_E_LAYOUT;
  const int64_t rows = a->N * a->Q * a->H;
  const Span ins[5] = {{a->cache, ((a->num_pages - 1) * a->page_stride + a->page_size * row) * 2},
                       {a->page_table, ((a->N - 1) * a->table_stride + a->max_pages) * 4},
                       {a->lengths, a->N * 4},
                       {a->q, qn * 2},
                       {a->R > 0 ? a->q_rope : nullptr, rn * 2}};
  const Span outs[3] = {{a->out, rows * a->L * 2}, {a->lse, rows * 4}, {a->workspace, (int64_t)need}};
  const int same[3] = {-1, -1, -1};
  return alias_error(outs, same, 3, ins, 5) ? KDA_E_ALIAS : KDA_OK;
}

// The arrays of an 8-bit latent cache; spans: codes, scales, rope.
kda_status_t check_latent_store(const kda_latent_store_t* s, Span* spans) {
  if (!s) return KDA_E_NULL;
  if (s->num_pages <= 0 || s->page_size <= 0 || s->L <= 0 || s->R < 0) return KDA_E_SHAPE;
  if (s->L % 16 != 0 || s->L > 512 || !dim8(s->R, 0, 64)) return KDA_E_UNSUPPORTED;
  if (s->num_pages > 0x7fffffff / s->page_size) return KDA_E_UNSUPPORTED;
  const int64_t room = s->page_size;
  if (s->codes_page_stride < room * s->L || s->scales_page_stride < room ||
      (s->R > 0 && s->rope_page_stride < room * s->R))
    return KDA_E_OVERLAP;
  if (s->codes_page_stride % 16 != 0 || (s->R > 0 && s->rope_page_stride % 8 != 0)) return KDA_E_LAYOUT;
  const int64_t most = kMaxSpan / s->num_pages;
  if (s->codes_page_stride > most || s->scales_page_stride > most || (s->R > 0 && s->rope_page_stride > most))
    return KDA_E_SHAPE;
  if (!s->codes || !s->scales || (s->R > 0 && !s->rope)) return KDA_E_NULL;
  if (!aligned(s->codes, 16) || !aligned(s->scales, 4) || (s->R > 0 && !aligned(s->rope, 16))) return KDA_E_LAYOUT;
  spans[0] = {s->codes, (s->num_pages - 1) * s->codes_page_stride + room * s->L};
  spans[1] = {s->scales, ((s->num_pages - 1) * s->scales_page_stride + room) * 4};
  spans[2] = {s->R > 0 ? s->rope : nullptr, s->R > 0 ? ((s->num_pages - 1) * s->rope_page_stride + room * s->R) * 2 : 0};
  if (spans_overlap(spans[0], spans[1]) || spans_overlap(spans[0], spans[2]) || spans_overlap(spans[1], spans[2]))
    return KDA_E_ALIAS;
  return KDA_OK;
}

// Rows of a call on the 8-bit cache: the kernels count them in 31 bits to the end of the last workgroup.  (A call of
// more than a launch takes goes in several.)
constexpr int64_t kMostRows = ((int64_t)1 << 28) - 1;

kda_status_t check_latent_shared(const kda_latent_shared_args_t* a) {
  if (!a) return KDA_E_NULL;
  if (a->N < 0 || a->Q <= 0 || a->H <= 0 || a->L <= 0 || a->R < 0 || a->G < 0) return KDA_E_SHAPE;
  if (a->num_pages <= 0 || a->page_size <= 0 || a->max_pages <= 0) return KDA_E_SHAPE;
  if (a->cache_dtype != KDA_BF16 && a->cache_dtype != KDA_E4M3) return KDA_E_DTYPE;
  const bool f8 = a->cache_dtype == KDA_E4M3;
  if (!dim8(a->L, 8, 512) || !dim8(a->R, 0, 64) || (f8 && a->L % 16 != 0)) return KDA_E_UNSUPPORTED;
  if (a->Q > 1024 || a->H > 1024 || a->Q * a->H > 1024) return KDA_E_UNSUPPORTED;
  if (a->N > 65535 || a->G > 65535) return KDA_E_UNSUPPORTED;  // sequences are a grid dimension
  if (!(a->scale > 0.f && a->scale <= kMostScale)) return KDA_E_UNSUPPORTED;
  const int64_t most = (int64_t)1 << 30, row = a->L + a->R;
  if (a->page_size > most || a->max_pages > most / a->page_size || a->num_pages > 0x7fffffff) return KDA_E_UNSUPPORTED;
  // (a workgroup's tiles are counted in 31 bits)
  const int64_t room = a->max_pages * a->page_size;
  if (a->N > 1 && room > ((int64_t)1 << 40) / a->N) return KDA_E_UNSUPPORTED;
  if (a->N > 0 && room > ((int64_t)1 << 48) / (a->N * a->Q * a->H)) return KDA_E_UNSUPPORTED;
  if (a->N > 1 && a->table_stride < a->max_pages) return KDA_E_OVERLAP;
  if (a->N > 1 && a->table_stride > kMaxSpan / a->N) return KDA_E_SHAPE;
  Span store[3] = {{nullptr, 0}, {nullptr, 0}, {nullptr, 0}};
  if (f8) {
    const kda_latent_store_t s = {const_cast<void*>(a->cache), const_cast<float*>(a->scales), const_cast<void*>(a->rope),
                                  a->num_pages, a->page_size, a->L, a->R,
                                  a->page_stride, a->scales_page_stride, a->rope_page_stride};
    const kda_status_t st = check_latent_store(&s, store);
    if (st != KDA_OK) return st;
  } else {
    if (a->page_stride < a->page_size * row) return KDA_E_OVERLAP;
    if (a->page_stride % 8 != 0) return KDA_E_LAYOUT;
    if (a->page_stride > kMaxSpan / a->num_pages) return KDA_E_SHAPE;
    if (a->N > 0 && !a->cache) return KDA_E_NULL;
    if (!aligned(a->cache, 16)) return KDA_E_LAYOUT;
    store[0] = {a->cache, ((a->num_pages - 1) * a->page_stride + a->page_size * row) * 2};
  }
  // (the kernel's page strides are 32 bits of bytes)
  const int64_t far = (int64_t)1 << 32;
  if (a->num_pages > 1 && (a->page_stride * (f8 ? 1 : 2) >= far ||
                           (f8 && (a->scales_page_stride * 4 >= far || (a->R > 0 && a->rope_page_stride * 2 >= far)))))
    return KDA_E_UNSUPPORTED;
  if (a->N == 0) return KDA_OK;
  if (!a->page_table || !a->lengths || !a->q || (a->R > 0 && !a->q_rope) || !a->out) return KDA_E_NULL;
  if (a->G > 0 && (!a->cu_groups || !a->shared)) return KDA_E_NULL;
  const int64_t nqh[3] = {a->N, a->Q, a->H};
  int64_t qn = 0, rn = 0;
  if (!outer_span(nqh, a->q_stride, 3, a->L, &qn) || (a->R > 0 && !outer_span(nqh, a->q_rope_stride, 3, a->R, &rn)))
    return KDA_E_LAYOUT;
  if (!aligned(a->q, 16) || (a->R > 0 && !aligned(a->q_rope, 16)) || !aligned(a->out, 16)) return KDA_E_LAYOUT;
  const size_t need = kda::latent_shared_workspace_bytes(a->N, a->Q, a->H, a->L, a->G);
  if (!a->workspace || a->workspace_bytes < need) return KDA_E_WORKSPACE;
  if (!aligned(a->workspace, 16)) return KDA_E_LAYOUT;
  const int64_t rows = a->N * a->Q * a->H;
  const Span ins[9] = {store[0],
                       store[1],
                       store[2],
                       {a->page_table, ((a->N - 1) * a->table_stride + a->max_pages) * 4},
                       {a->lengths, a->N * 4},
                       {a->q, qn * 2},
                       {a->R > 0 ? a->q_rope : nullptr, rn * 2},
                       {a->G > 0 ? a->cu_groups : nullptr, (a->G + 1) * 4},
                       {a->G > 0 ? a->shared : nullptr, a->G * 4}};
  const Span outs[3] = {{a->out, rows * a->L * 2}, {a->lse, rows * 4}, {a->workspace, (int64_t)need}};
  const int same[3] = {-1, -1, -1};
  return alias_error(outs, same, 3, ins, 9) ? KDA_E_ALIAS : KDA_OK;
}

kda_status_t check_pool(const kda_page_pool_t* p, Span* spans) {
  if (!p) return KDA_E_NULL;
  if (p->num_seqs <= 0 || p->max_pages <= 0 || p->num_pages <= 0 || p->page_size <= 0) return KDA_E_SHAPE;
  if (p->num_seqs > ((int64_t)1 << 24) || p->max_pages > ((int64_t)1 << 20) || p->num_pages > ((int64_t)1 << 30) ||
      p->page_size > ((int64_t)1 << 30))
    return KDA_E_UNSUPPORTED;
  if (p->num_seqs > 1 && p->table_stride < p->max_pages) return KDA_E_OVERLAP;
  if (p->num_seqs > 1 && p->table_stride > kMaxSpan / p->num_seqs) return KDA_E_SHAPE;
  if (!p->table || !p->lengths || !p->refs) return KDA_E_NULL;
  spans[0] = {p->table, ((p->num_seqs - 1) * p->table_stride + p->max_pages) * 4};
  spans[1] = {p->lengths, p->num_seqs * 4};
  spans[2] = {p->refs, p->num_pages * 4};
  return KDA_OK;
}

kda_status_t check_stores(const kda_page_store_t* s, int64_t n, int64_t num_pages) {
  if (n < 0) return KDA_E_SHAPE;
  if (n > 4096) return KDA_E_UNSUPPORTED;
  if (n > 0 && !s) return KDA_E_NULL;
  for (int64_t i = 0; i < n; ++i) {
    if (s[i].page_bytes <= 0) return KDA_E_SHAPE;
    if (s[i].page_stride < s[i].page_bytes) return KDA_E_OVERLAP;
    if (s[i].page_stride > kMaxSpan / num_pages) return KDA_E_SHAPE;
    if (!s[i].data) return KDA_E_NULL;
  }
  return KDA_OK;
}

Span store_span(const kda_page_store_t& s, int64_t num_pages) {
  return {s.data, (num_pages - 1) * s.page_stride + s.page_bytes};
}

// Whether the stores overlap one another or one of ``spans``.
bool stores_alias(const kda_page_store_t* s, int64_t n, int64_t num_pages, const Span* spans, int num_spans) {
  for (int64_t i = 0; i < n; ++i) {
    const Span a = store_span(s[i], num_pages);
    for (int j = 0; j < num_spans; ++j)
      if (spans_overlap(a, spans[j])) return true;
    for (int64_t j = 0; j < i; ++j)
      if (spans_overlap(a, store_span(s[j], num_pages))) return true;
  }
  return false;
}

}  // namespace

extern "C" {

size_t kda_latent_prefill_workspace_size(int64_t T, int64_t S, int64_t N, int64_t H, int64_t E) {
  if (T <= 0 || S < 0 || N <= 0 || H <= 0 || E <= 0 || T > kMostTokens || S > kMostTokens || N > kMostTokens ||
      H > 65535 || E > 128)
    return 0;
  return kda::latent_prefill_workspace_bytes(T, S, N, H, E);
}

kda_status_t kda_latent_prefill(const kda_latent_prefill_args_t* a, void* stream) {
  const kda_status_t st = check_latent_prefill(a);
  if (st != KDA_OK || a->T == 0 || a->N == 0) return st;
  return hip_status("kda_latent_prefill launch", kda::launch_latent_prefill(*a, static_cast<hipStream_t>(stream)));
}

size_t kda_latent_decode_workspace_size(int64_t N, int64_t Q, int64_t H, int64_t L) {
  if (N <= 0 || Q <= 0 || H <= 0 || L <= 0 || Q > 1024 || H > 1024 || Q * H > 1024 || L > 512) return 0;
  return kda::latent_decode_workspace_bytes(N, Q, H, L);
}

kda_status_t kda_latent_decode(const kda_latent_decode_args_t* a, void* stream) {
  const kda_status_t st = check_latent_decode(a);
  if (st != KDA_OK || a->N == 0) return st;
  return hip_status("kda_latent_decode launch", kda::launch_latent_decode(*a, static_cast<hipStream_t>(stream)));
}

kda_status_t kda_latent_quantize_scatter(const kda_latent_store_t* store, const void* c, int64_t c_stride,
                                         const void* k_rope, int64_t k_rope_stride, kda_dtype_t dtype,
                                         const void* slots, kda_index_t it, int64_t num_rows, void* stream) {
  Span outs[3];
  const kda_status_t st = check_latent_store(store, outs);
  if (st != KDA_OK) return st;
  if (!valid_dtype(dtype) || (it != KDA_I32 && it != KDA_I64)) return KDA_E_DTYPE;
  if (num_rows < 0) return KDA_E_SHAPE;
  if (num_rows > kMostRows) return KDA_E_UNSUPPORTED;
  if (num_rows == 0) return KDA_OK;
  if (!c || !slots || (store->R > 0 && !k_rope)) return KDA_E_NULL;
  int64_t cn = 0, rn = 0;
  if (!outer_span(&num_rows, &c_stride, 1, store->L, &cn) ||
      (store->R > 0 && !outer_span(&num_rows, &k_rope_stride, 1, store->R, &rn)))
    return KDA_E_LAYOUT;
  if (!aligned(c, 16) || (store->R > 0 && !aligned(k_rope, 16))) return KDA_E_LAYOUT;
  const int64_t eb = dtype_bytes(dtype);
  const Span ins[3] = {{c, cn * eb},
                       {store->R > 0 ? k_rope : nullptr, rn * eb},
                       {slots, num_rows * (it == KDA_I64 ? 8 : 4)}};
  const int none[3] = {-1, -1, -1};
  if (alias_error(outs, none, 3, ins, 3)) return KDA_E_ALIAS;
  return hip_status("kda_latent_quantize_scatter launch",
                    kda::launch_latent_quantize_scatter(*store, c, c_stride, k_rope, k_rope_stride, dtype == KDA_BF16,
                                                        slots, it == KDA_I64, num_rows,
                                                        static_cast<hipStream_t>(stream)));
}

kda_status_t kda_latent_dequantize_gather(const kda_latent_store_t* store, const void* slots, kda_index_t it,
                                          int64_t num_rows, void* out, kda_dtype_t dtype, void* stream) {
  Span ins[4];
  const kda_status_t st = check_latent_store(store, ins);
  if (st != KDA_OK) return st;
  if (!valid_dtype(dtype) || (it != KDA_I32 && it != KDA_I64)) return KDA_E_DTYPE;
  if (num_rows < 0) return KDA_E_SHAPE;
  if (num_rows > kMostRows) return KDA_E_UNSUPPORTED;
  if (num_rows == 0) return KDA_OK;
  if (!out || !slots) return KDA_E_NULL;
  if (!aligned(out, 16)) return KDA_E_LAYOUT;
  ins[3] = {slots, num_rows * (it == KDA_I64 ? 8 : 4)};
  const Span outs[1] = {{out, num_rows * (store->L + store->R) * dtype_bytes(dtype)}};
  const int none[1] = {-1};
  if (alias_error(outs, none, 1, ins, 4)) return KDA_E_ALIAS;
  return hip_status("kda_latent_dequantize_gather launch",
                    kda::launch_latent_dequantize_gather(*store, slots, it == KDA_I64, num_rows, out,
                                                         dtype == KDA_BF16, static_cast<hipStream_t>(stream)));
}

size_t kda_latent_shared_workspace_size(int64_t N, int64_t Q, int64_t H, int64_t L, int64_t G) {
  if (N <= 0 || Q <= 0 || H <= 0 || L <= 0 || G < 0 || N > 65535 || Q > 1024 || H > 1024 || Q * H > 1024 || L > 512 ||
      G > 65535)
    return 0;
  return kda::latent_shared_workspace_bytes(N, Q, H, L, G);
}

kda_status_t kda_latent_decode_fp8(const kda_latent_shared_args_t* a, void* stream) {
  if (a && a->cache_dtype != KDA_E4M3) return KDA_E_DTYPE;
  if (a && a->G != 0) return KDA_E_SHAPE;
  const kda_status_t st = check_latent_shared(a);
  if (st != KDA_OK || a->N == 0) return st;
  return hip_status("kda_latent_decode_fp8 launch", kda::launch_latent_shared(*a, static_cast<hipStream_t>(stream)));
}

kda_status_t kda_latent_decode_shared(const kda_latent_shared_args_t* a, void* stream) {
  const kda_status_t st = check_latent_shared(a);
  if (st != KDA_OK || a->N == 0) return st;
  return hip_status("kda_latent_decode_shared launch", kda::launch_latent_shared(*a, static_cast<hipStream_t>(stream)));
}

size_t kda_page_fork_workspace_size(int64_t num_forks, int64_t max_pages, int64_t num_pages, int share) {
  if (num_forks <= 0 || max_pages <= 0 || num_pages <= 0) return 0;
  return kda::page_fork_workspace_bytes(num_forks, max_pages, num_pages, share != 0);
}

kda_status_t kda_page_fork(const kda_page_pool_t* pool, const kda_page_store_t* stores, int64_t num_stores,
                           const void* src, const void* dst, kda_index_t it, int64_t num_forks, int share,
                           int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  Span spans[7];
  kda_status_t st = check_pool(pool, spans);
  if (st != KDA_OK) return st;
  if ((st = check_stores(stores, num_stores, pool->num_pages)) != KDA_OK) return st;
  if (it != KDA_I32 && it != KDA_I64) return KDA_E_DTYPE;
  if (num_forks < 0) return KDA_E_SHAPE;
  if (num_forks > ((int64_t)1 << 16)) return KDA_E_UNSUPPORTED;  // (each entry's dst is compared with those before it)
  if (num_forks == 0) return KDA_OK;
  if (!src || !dst || !status) return KDA_E_NULL;
  const size_t need = kda::page_fork_workspace_bytes(num_forks, pool->max_pages, pool->num_pages, share != 0);
  if (!workspace || workspace_bytes < need) return KDA_E_WORKSPACE;
  if (!aligned(workspace, 4)) return KDA_E_LAYOUT;
  spans[3] = {status, num_forks * 4};
  spans[4] = {workspace, (int64_t)need};
  spans[5] = {src, num_forks * (it == KDA_I64 ? 8 : 4)};
  spans[6] = {dst, num_forks * (it == KDA_I64 ? 8 : 4)};
  const int none[5] = {-1, -1, -1, -1, -1};
  if (alias_error(spans, none, 5, spans + 5, 2) || stores_alias(stores, num_stores, pool->num_pages, spans, 7))
    return KDA_E_ALIAS;
  return hip_status("kda_page_fork launch",
                    kda::launch_page_fork(*pool, stores, num_stores, src, dst, it == KDA_I64, num_forks, share != 0,
                                          status, workspace, static_cast<hipStream_t>(stream)));
}

size_t kda_page_compact_workspace_size(int64_t num_pages) {
  return num_pages <= 0 ? 0 : kda::page_compact_workspace_bytes(num_pages);
}

kda_status_t kda_page_compact(const kda_page_pool_t* pool, const kda_page_store_t* stores, int64_t num_stores,
                              int32_t* live, void* workspace, size_t workspace_bytes, void* stream) {
  Span spans[5];
  kda_status_t st = check_pool(pool, spans);
  if (st != KDA_OK) return st;
  if ((st = check_stores(stores, num_stores, pool->num_pages)) != KDA_OK) return st;
  const size_t need = kda::page_compact_workspace_bytes(pool->num_pages);
  if (!workspace || workspace_bytes < need) return KDA_E_WORKSPACE;
  if (!aligned(workspace, 4)) return KDA_E_LAYOUT;
  spans[3] = {live, live ? 4 : 0};
  spans[4] = {workspace, (int64_t)need};
  const int none[5] = {-1, -1, -1, -1, -1};
  if (alias_error(spans, none, 5, spans, 0) || stores_alias(stores, num_stores, pool->num_pages, spans, 5))
    return KDA_E_ALIAS;
  return hip_status("kda_page_compact launch",
                    kda::launch_page_compact(*pool, stores, num_stores, live, workspace,
                                             static_cast<hipStream_t>(stream)));
}

kda_status_t kda_page_free(const kda_page_pool_t* pool, const uint8_t* release, void* stream) {
  Span spans[4];
  const kda_status_t st = check_pool(pool, spans);
  if (st != KDA_OK) return st;
  if (!release) return KDA_E_NULL;
  spans[3] = {release, pool->num_seqs};
  const int none[3] = {-1, -1, -1};
  if (alias_error(spans, none, 3, spans + 3, 1)) return KDA_E_ALIAS;
  return hip_status("kda_page_free launch", kda::launch_page_free(*pool, release, static_cast<hipStream_t>(stream)));
}

const char* kda_status_string(kda_status_t s) {
  switch (s) {
    case KDA_OK: return "KDA_OK";
    case KDA_E_NULL: return "KDA_E_NULL: a required pointer is NULL";
    case KDA_E_DTYPE: return "KDA_E_DTYPE: unsupported dtype or index type";
    case KDA_E_SHAPE: return "KDA_E_SHAPE: invalid size";
    case KDA_E_LAYOUT: return "KDA_E_LAYOUT: cache inner dims [H,V,K] are not dense";
    case KDA_E_OVERLAP: return "KDA_E_OVERLAP: cache row stride is smaller than the row payload";
    case KDA_E_UNSUPPORTED: return "KDA_E_UNSUPPORTED: no kernel for these sizes";
    case KDA_E_WORKSPACE: return "KDA_E_WORKSPACE: workspace missing or too small";
    case KDA_E_ALIAS: return "KDA_E_ALIAS: an output overlaps an input or another output";
    case KDA_E_HIP: return "KDA_E_HIP: HIP runtime error";
  }
  return "unknown kda_status_t";
}

const char* kda_last_error_detail(void) { return g_detail; }

}  // extern "C"
