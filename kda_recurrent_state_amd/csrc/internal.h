// Internal declarations shared by the host entry points and the kernel
// launchers of libkda.  Not part of the public ABI (see include/kda.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// Copies whole state rows between a cache view and a packed buffer.
// row_stride_bytes/payload_bytes are byte counts; indices are read in their
// own width.  gather: packed <- cache (zeros for invalid/flag-false rows);
// scatter: cache <- packed for valid rows only.
hipError_t launch_state_copy(bool gather, char* cache, int64_t row_stride_bytes, int64_t num_rows,
                             int64_t payload_bytes, const void* indices, bool index64, int64_t num_selected,
                             const uint8_t* flags, char* packed, hipStream_t stream);

// Enqueues the chunked gated-delta-rule prefill; arguments already validated.
hipError_t launch_chunk_prefill(const kda_prefill_args_t& a, hipStream_t stream);

// Enqueues one recurrent decode step on validated arguments (cache and args agree).
hipError_t launch_recurrent_decode(const kda_state_cache_t& cache, const kda_decode_args_t& a, hipStream_t stream);

// INT8 checkpoint codec: quantize-scatter (packed -> store slots) or
// dequantize-gather (store slots -> packed); arguments already validated.
hipError_t launch_int8_ckpt(bool quantize, const kda_int8_store_t& store, const void* indices, bool index64,
                            int64_t num_selected, const uint8_t* flags, void* packed, bool packed_bf16,
                            hipStream_t stream);

// Workspace bytes launch_chunk_prefill uses for these sizes.
size_t chunk_prefill_workspace_bytes(int64_t T, int64_t N, int64_t H, int64_t K, int64_t V);

// Device address of the current device's copy of the library's static
// scratch array (KDA_NOALLOC_SCRATCH_BYTES bytes), looked up once per device.
hipError_t noalloc_scratch(void** ptr);

// Latent attention; arguments already validated.
hipError_t launch_latent_prefill(const kda_latent_prefill_args_t& a, hipStream_t stream);
int64_t latent_prefill_workgroups(int64_t T, int64_t S, int64_t N, int64_t H);
size_t latent_prefill_workspace_bytes(int64_t T, int64_t S, int64_t N, int64_t H, int64_t E);
hipError_t launch_latent_decode(const kda_latent_decode_args_t& a, hipStream_t stream);
size_t latent_decode_workspace_bytes(int64_t N, int64_t Q, int64_t H, int64_t L);
hipError_t launch_latent_shared(const kda_latent_shared_args_t& a, hipStream_t stream);
size_t latent_shared_workspace_bytes(int64_t N, int64_t Q, int64_t H, int64_t L, int64_t G);

// Rows that one launch of the 8-bit cache's kernels takes, of ``rows`` a workgroup of 256 threads: HIP launches fewer
// than 2^32 threads a grid dimension.
constexpr int64_t cache_slice_rows(int rows) { return (((int64_t)1 << 24) - 1) * rows; }

// The 8-bit latent cache; arguments already validated.
hipError_t launch_latent_quantize_scatter(const kda_latent_store_t& s, const void* c, int64_t c_stride,
                                          const void* k_rope, int64_t k_rope_stride, bool bf16, const void* slots,
                                          bool index64, int64_t n, hipStream_t stream);
hipError_t launch_latent_dequantize_gather(const kda_latent_store_t& s, const void* slots, bool index64, int64_t n,
                                           void* out, bool bf16, hipStream_t stream);

// j / d = j mul >> shift for 0 <= j < 2^31: shift = 31 + s with 2^s >= d and mul
// = floor(2^shift / d) + 1; mul d passes 2^shift by at most d <= 2^s, too little
// to matter.
inline void page_divisor(int d, uint32_t* mul, int* shift) {
  int s = 0;
  while (((int64_t)1 << s) < d) ++s;
  *shift = 31 + s;
  *mul = (uint32_t)(((uint64_t)1 << (31 + s)) / (uint32_t)d + 1);
}

// Page pool operators; arguments already validated.
hipError_t launch_page_fork(const kda_page_pool_t& a, const kda_page_store_t* stores, int64_t num_stores,
                            const void* src, const void* dst, bool index64, int64_t num_forks, bool share,
                            int32_t* status, void* workspace, hipStream_t stream);
size_t page_fork_workspace_bytes(int64_t num_forks, int64_t max_pages, int64_t num_pages, bool share);
hipError_t launch_page_compact(const kda_page_pool_t& a, const kda_page_store_t* stores, int64_t num_stores,
                               int32_t* live, void* workspace, hipStream_t stream);
size_t page_compact_workspace_bytes(int64_t num_pages);
hipError_t launch_page_free(const kda_page_pool_t& a, const uint8_t* release, hipStream_t stream);

}  // namespace kda
