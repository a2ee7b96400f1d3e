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

// Loads from global memory straight to LDS: lane i's bytes land at lds + 16 i
// (4 i); lanes that are switched off load and write nothing.  ``lds`` is
// a uniform byte offset (lds_offset).  They have no destination register that could be taken for written,
// so nothing but LDS depends on their end, and that is waited for by hand:
// wait_loads() and a barrier before the bytes are read, and a barrier between
// the last read of a place and the next load to it.  (The compiler's own form
// of these loads makes it wait for all of them before any LDS access that it
// cannot tell apart, which ends the prefetch.)
__device__ __forceinline__ unsigned lds_offset(const void* lds) {
  return (unsigned)(uintptr_t)(const __attribute__((address_space(3))) void*)lds;
}
// base is uniform.  (A memory instruction may read a scalar register five wait
// states after a vector instruction, such as a read of one lane, has written it;
// the compiler does not count them for assembly.)
__device__ __forceinline__ void load_lds16(const char* base, unsigned offset, unsigned lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %0" ::"s"(base), "v"(offset), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void load_lds16(const char* lane_address, unsigned lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(lane_address), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void load_lds4(const void* lane_address, unsigned lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(lane_address), "s"(lds)
               : "memory");
}

// Waits until at most kLeft of the wave's loads are under way (a barrier then
// shows what loads to LDS have brought to the other waves).
template <int kLeft = 0>
__device__ __forceinline__ void wait_loads() {
  static_assert(kLeft < 64, "vmcnt has 6 bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (kLeft & 15) | (kLeft >> 4 << 14));  // the other counters free
  asm volatile("" ::: "memory");
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

// The softmax weights are 2^fma(s, scale2, -base): base is a rounded product
// (the maximum in use, s scale2 of some s), the fused operation's is not, and
// their difference is the same factor of all weights.  It is at most 2^16 up to
// |base| = kFar, but past the range of fp32 from 2^31 on, where the scores stand
// that were masked by the type's lowest value.  Rows out there (the maximum is
// finite) take their scores relative to the maximum, both products rounded, and
// the base 0, so that the maximum's own weight is 1.
constexpr float kFar = 268435456.f;  // 2^28: half a step is 16
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > kFar && m != -INFINITY; }
__device__ __forceinline__ float from_far(float s, float scale2, float m) {
#pragma clang fp contract(off)
  const float x = s * scale2;
  return (x - m) / scale2;
}

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

// The value of the first active lane, the same in all and known to be.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The value of lane ``src`` (uniform).
__device__ __forceinline__ int64_t lane64(int64_t x, int src) {
  const int lo = __builtin_amdgcn_readlane((int)x, src), hi = __builtin_amdgcn_readlane((int)(x >> 32), src);
  return ((int64_t)hi << 32) | (unsigned)lo;
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
