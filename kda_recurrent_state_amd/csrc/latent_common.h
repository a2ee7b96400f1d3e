// Device helpers shared by the latent-attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {
namespace latent {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

// 16 bytes from global memory straight to LDS.  ``lds`` is the wave's base:
// lane i's 16 bytes land at lds + 16 i; lanes that are switched off load and
// write nothing and leave their 16 bytes as they were.
__device__ __forceinline__ void load_lds16(const void* g, void* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// Waits for the wave's loads to LDS (a barrier then shows them to the others).
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0, the other counters free
  asm volatile("" ::: "memory");
}

// 8 bytes to LDS.  The compiler would wait for every load to LDS under way
// before a store that it cannot tell apart from them; lds_barrier() waits for
// the store itself.
__device__ __forceinline__ void store_lds8(void* lds, const bf16x4& x) {
  const unsigned at = (unsigned)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
  asm volatile("ds_write_b64 %0, %1" ::"v"(at), "v"(__builtin_bit_cast(uint64_t, x)) : "memory");
}

// Barrier of the workgroup for LDS: the wave's LDS accesses are done, its
// loads (to registers or to LDS) may still be under way.  (__syncthreads
// waits for those too, which would end every prefetch at the next barrier.)
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt 0, the other counters free
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Transposed 8-byte LDS read: in each group of 16 lanes, lane i reads the four
// bf16 of row i / 4, columns 4 (i % 4) .. + 3 of a 4 x 16 block (its address
// points at them), and receives column i of the four rows.
__device__ __forceinline__ s16x4 read_tr(const void* lds) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)lds);
}

// x, as a value the compiler cannot trace: what is computed from it inside a
// loop stays there and does not occupy registers around it.
__device__ __forceinline__ int keep_here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ bf16x8 join(const s16x4& lo, const s16x4& hi) {
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(bf16x8, (s16x8){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// The scheduler moves nothing across this.  By itself it puts each LDS read
// right before the product that needs it and waits for it, so the product
// loops read the next operands between two of these.
__device__ __forceinline__ void hold_order() { __builtin_amdgcn_sched_barrier(0); }

// x combined with the lane 32 (16) further on, the same bits in both
__device__ __forceinline__ float max_halves(float x) {
  const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x),
                                                  false, false);
  const unsigned a = s[0], b = s[1];
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

__device__ __forceinline__ float sum_halves(float x) {
  const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x),
                                                  false, false);
  const unsigned a = s[0], b = s[1];
  return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

__device__ __forceinline__ float max_quarters(float x) {
  const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x),
                                                  false, false);
  const unsigned a = s[0], b = s[1];
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

__device__ __forceinline__ float sum_quarters(float x) {
  const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x),
                                                  false, false);
  const unsigned a = s[0], b = s[1];
  return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

// inclusive prefix sum over the wave's lanes
__device__ __forceinline__ int wave_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}

}  // namespace latent
}  // namespace kda
