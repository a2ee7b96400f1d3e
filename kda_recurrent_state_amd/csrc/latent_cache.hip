// The 8-bit latent cache: token rows quantised as they are written into pages,
// and read back, for gfx950.
//
// A row is L latent values as e4m3 codes with one scale, and its rotary key in
// bf16 (its angles matter to the last bit of the score, and it is an eighth of the
// values).  The scale is a power of two: 2^e with the smallest e >= -126 for which the
// row's largest magnitude is at most 448 2^e.  A division by it is exact, so a
// code is the value itself rounded once (half a step: 2^-4 of the value down to
// 2^-6 of the scale), reading back is exact in fp32, and in bf16 too for rows written from
// bf16 and scales of 2^-124 and more (below, the smallest code, 2^-9 of the scale, lies under
// bf16's smallest subnormal, 2^-133, and is rounded), and writing again what was
// read exactly gives the same values.  One scale a row, not one a block: e4m3 is
// a floating format, and a value keeps its four bits down to 2^-13 of the row's
// largest, which is above 224 scales; and a scale per row leaves both products of decode as products of codes.
//
// Both kernels move each byte once and are bound by HBM.  A lane has 8
// values; 16, 32 or 64 lanes have a row.  98304 rows of 512 + 64 values (171 MB) are
// written in 29 us, 5.9 TB/s, and 120000 read in 34 us (215 MB, 6.4 TB/s), where
// a copy of 1 GiB runs at 5.1; 64 rows take 4 us and are one launch's latency.
#include "internal.h"
#include "latent_common.h"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

struct CacheParams {
  char* codes;
  char* scales;
  char* rope;
  int64_t codes_page, scales_page, rope_page;  // bytes
  int page_size, L, R;
  int64_t rows;       // num_pages page_size, below 2^31
  uint32_t page_mul;  // s / page_size = s page_mul >> page_shift
  int page_shift;
  const char* c;      // written from, with strides in bytes
  const char* k_rope;
  int64_t c_stride, k_rope_stride;
  char* out;          // read into
  const void* slots;
  int n;              // rows of the call
};

struct Place {
  int64_t page;
  int off;
};

template <typename Index>
__device__ __forceinline__ int64_t slot_of(const CacheParams& p, int t) {
  return t < p.n ? (int64_t) static_cast<const Index*>(p.slots)[t] : -1;
}

__device__ __forceinline__ bool in_cache(const CacheParams& p, int64_t slot) { return slot >= 0 && slot < p.rows; }

__device__ __forceinline__ Place place_of(const CacheParams& p, int64_t slot) {
  const unsigned page = (unsigned)(((uint64_t)(unsigned)slot * p.page_mul) >> p.page_shift);
  return {(int64_t)page, (int)((unsigned)slot - page * (unsigned)p.page_size)};
}

// ``kOnce``: for data that this call alone touches, so that it takes no other's place in
// the caches.
template <bool kOnce, typename V>
__device__ __forceinline__ V load_vec(const char* at) {
  const V* v = reinterpret_cast<const V*>(at);
  return kOnce ? __builtin_nontemporal_load(v) : *v;
}
template <bool kOnce, typename V>
__device__ __forceinline__ void store_vec(char* at, V x) {
  V* v = reinterpret_cast<V*>(at);
  if (kOnce)
    __builtin_nontemporal_store(x, v);
  else
    *v = x;
}

// 8 values as they are stored
template <typename T>
struct Eight;
template <>
struct Eight<__bf16> {
  u32x4 raw;
  template <bool kOnce>
  __device__ __forceinline__ void load(const char* at) { raw = load_vec<kOnce, u32x4>(at); }
  __device__ __forceinline__ void clear() { raw = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int i) const {
    const unsigned w = raw[i >> 1];
    return __builtin_bit_cast(float, i & 1 ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ u32x4 as_bf16() const { return raw; }
};
template <>
struct Eight<float> {
  f32x4 raw[2];
  template <bool kOnce>
  __device__ __forceinline__ void load(const char* at) {
    raw[0] = load_vec<kOnce, f32x4>(at);
    raw[1] = load_vec<kOnce, f32x4>(at + 16);
  }
  __device__ __forceinline__ void clear() { raw[0] = raw[1] = f32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int i) const { return raw[i >> 2][i & 3]; }
  __device__ __forceinline__ u32x4 as_bf16() const {
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (__bf16)raw[i >> 2][i & 3];
    return __builtin_bit_cast(u32x4, b);
  }
};

// The scale's exponent from the bits of the largest magnitude: 448 is 1.75 2^8.
__device__ __forceinline__ int scale_exponent(unsigned top) {
  const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}

// Many rows: two a lane group, their loads issued together, and read past the caches
template <typename T, typename Index, int LANES, bool kMany>
__global__ __launch_bounds__(kThreads) void quantize_scatter_kernel(CacheParams p) {
  constexpr int U = kMany ? 2 : 1, kRows = 64 / LANES;  // rows of a lane group, and of a wave at once
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane % LANES;
  const int first = (blockIdx.x * kWaves + wave) * kRows * U + lane / LANES;
  const bool has_c = 8 * i < p.L, has_r = 8 * i < p.R;
  Eight<T> x[U], r[U];
  int64_t slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = first + u * kRows;
    slot[u] = slot_of<Index>(p, t);
    x[u].clear();
    if (t < p.n && has_c) x[u].template load<kMany>(p.c + t * p.c_stride + i * (8 * (int)sizeof(T)));
    if (t < p.n && has_r)
      r[u].template load<kMany>(p.k_rope + t * p.k_rope_stride + i * (8 * (int)sizeof(T)));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    unsigned top = 0;  // of the magnitudes' bits: NaN and infinity are above all others
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const unsigned b = __builtin_bit_cast(unsigned, x[u].get(k)) & 0x7fffffffu;
      top = b > top ? b : top;
    }
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) {
      const unsigned o = (unsigned)__shfl_xor((int)top, d, 64);
      top = o > top ? o : top;
    }
    if (!in_cache(p, slot[u])) continue;
    const bool fine = top < 0x7f800000u;
    const int e = scale_exponent(top);
    const float inv = __builtin_bit_cast(float, (unsigned)(127 - e) << 23);
    const Place at = place_of(p, slot[u]);
    if (has_c) {
      u32x2 codes;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = fine ? x[u].get(4 * k + j) * inv : 0.f;
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        codes[k] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
      }
      *reinterpret_cast<u32x2*>(p.codes + at.page * p.codes_page + (int64_t)at.off * p.L + 8 * i) = codes;
    }
    if (has_r)
      *reinterpret_cast<u32x4*>(p.rope + at.page * p.rope_page + (int64_t)at.off * (2 * p.R) + 16 * i) = r[u].as_bf16();
    if (i == 0)
      *reinterpret_cast<float*>(p.scales + at.page * p.scales_page + (int64_t)at.off * 4) =
          fine ? __builtin_bit_cast(float, (unsigned)(127 + e) << 23) : __builtin_nanf("");
  }
}

template <typename T, bool kOnce>
__device__ __forceinline__ void store8(char* at, const float (&v)[8]) {
  if (sizeof(T) == 4) {
    store_vec<kOnce>(at, f32x4{v[0], v[1], v[2], v[3]});
    store_vec<kOnce>(at + 16, f32x4{v[4], v[5], v[6], v[7]});
  } else {
    bf16x8 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (__bf16)v[i];
    store_vec<kOnce>(at, b);
  }
}

// Many rows: two a lane group, written past the caches
template <typename T, typename Index, int LANES, bool kMany>
__global__ __launch_bounds__(kThreads) void dequantize_gather_kernel(CacheParams p) {
  constexpr int U = kMany ? 2 : 1, kRows = 64 / LANES;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane % LANES;
  const int first = (blockIdx.x * kWaves + wave) * kRows * U + lane / LANES;
  const bool has_c = 8 * i < p.L, has_r = 8 * i < p.R;
  int64_t slot[U];
  u32x2 codes[U];
  u32x4 r[U];
  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) slot[u] = slot_of<Index>(p, first + u * kRows);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    codes[u] = u32x2{0, 0};
    r[u] = u32x4{0, 0, 0, 0};
    scale[u] = 0.f;
    if (!in_cache(p, slot[u])) continue;
    const Place at = place_of(p, slot[u]);
    scale[u] = *reinterpret_cast<const float*>(p.scales + at.page * p.scales_page + (int64_t)at.off * 4);
    if (has_c)
      codes[u] = *reinterpret_cast<const u32x2*>(p.codes + at.page * p.codes_page + (int64_t)at.off * p.L + 8 * i);
    if (has_r)
      r[u] = *reinterpret_cast<const u32x4*>(p.rope + at.page * p.rope_page + (int64_t)at.off * (2 * p.R) + 16 * i);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = first + u * kRows;
    if (t >= p.n) continue;
    char* row = p.out + (int64_t)t * ((p.L + p.R) * (int)sizeof(T));
    if (has_c) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[u][k], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[u][k], true);
        v[4 * k] = lo[0] * scale[u];
        v[4 * k + 1] = lo[1] * scale[u];
        v[4 * k + 2] = hi[0] * scale[u];
        v[4 * k + 3] = hi[1] * scale[u];
      }
      store8<T, kMany>(row + i * (8 * (int)sizeof(T)), v);
    }
    if (has_r) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const unsigned w = r[u][k >> 1];
        v[k] = __builtin_bit_cast(float, k & 1 ? w & 0xffff0000u : w << 16);
      }
      store8<T, kMany>(row + (p.L + 8 * i) * (int)sizeof(T), v);
    }
  }
}

// Which calls have many rows: in bf16 alone.  Reading: those of more than 1024 workgroups (8192 rows of
// 512 + 64 values 9.4 us either way, 32768 10.7 against 12.2 with a row a lane group and
// plain stores, 120000 34 against 54).  Writing: inputs of more than 64 MiB, which the caches do
// not hold from whatever wrote them (32768 rows, 38 MB, read again and again: 13.1 against
// 12.2; 98304 rows, 113 MB: 29 against 34).  Four rows a lane group took 30 and 34 us, eight 33 and 35.
// In fp32 a lane has 32 bytes and an instruction moves 16 of each 32, which past the caches
// does not come together (32768 and 65536 rows read 26 and 51 us against 17 and 29, 131072 105
// against 95, of 128 + 64 values 33 against 22; 65536 and 98304 written 38 and 56 against 35 and 51).
template <bool kWrite, typename T, typename Index, int LANES>
hipError_t launch_lanes(const CacheParams& call, hipStream_t stream) {
  constexpr int kRows = 64 / LANES * kWaves;
  constexpr bool kBf16 = sizeof(T) == 2;
  const bool many = kBf16 && (kWrite ? (int64_t)call.n * (call.L + call.R) * 2 > (64 << 20) : call.n > 1024 * kRows);
  const int rows = kRows * (many ? 2 : 1);
  const int64_t most = cache_slice_rows(rows);
  for (int64_t done = 0; done < call.n; done += most) {
    CacheParams p = call;
    p.n = (int)(call.n - done < most ? call.n - done : most);
    p.slots = static_cast<const Index*>(call.slots) + done;
    if (kWrite) {
      p.c += done * call.c_stride;
      p.k_rope += done * call.k_rope_stride;  // (strides in bytes)
    } else {
      p.out += done * ((call.L + call.R) * (int)sizeof(T));
    }
    const dim3 grid((unsigned)(((int64_t)p.n + rows - 1) / rows)), block(kThreads);
    if (kWrite) {
      if (many)
        hipLaunchKernelGGL((quantize_scatter_kernel<T, Index, LANES, kBf16>), grid, block, 0, stream, p);
      else
        hipLaunchKernelGGL((quantize_scatter_kernel<T, Index, LANES, false>), grid, block, 0, stream, p);
    } else {
      if (many)
        hipLaunchKernelGGL((dequantize_gather_kernel<T, Index, LANES, kBf16>), grid, block, 0, stream, p);
      else
        hipLaunchKernelGGL((dequantize_gather_kernel<T, Index, LANES, false>), grid, block, 0, stream, p);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool kWrite, typename T, typename Index>
hipError_t launch_index(const CacheParams& p, hipStream_t stream) {
  if (p.L <= 128) return launch_lanes<kWrite, T, Index, 16>(p, stream);
  if (p.L <= 256) return launch_lanes<kWrite, T, Index, 32>(p, stream);
  return launch_lanes<kWrite, T, Index, 64>(p, stream);
}

template <bool kWrite>
hipError_t launch(const CacheParams& p, bool bf16, bool index64, hipStream_t stream) {
  if (index64) {
    return bf16 ? launch_index<kWrite, __bf16, int64_t>(p, stream) : launch_index<kWrite, float, int64_t>(p, stream);
  }
  return bf16 ? launch_index<kWrite, __bf16, int32_t>(p, stream) : launch_index<kWrite, float, int32_t>(p, stream);
}

CacheParams params(const kda_latent_store_t& s, const void* slots, int64_t n) {
  CacheParams p = {};
  p.codes = static_cast<char*>(s.codes);
  p.scales = reinterpret_cast<char*>(s.scales);
  p.rope = static_cast<char*>(s.rope);
  p.codes_page = s.codes_page_stride;
  p.scales_page = s.scales_page_stride * 4;
  p.rope_page = s.rope_page_stride * 2;
  p.page_size = (int)s.page_size;
  p.L = (int)s.L;
  p.R = (int)s.R;
  p.rows = s.num_pages * s.page_size;
  page_divisor(p.page_size, &p.page_mul, &p.page_shift);
  p.slots = slots;
  p.n = (int)n;
  return p;
}

}  // namespace

hipError_t launch_latent_quantize_scatter(const kda_latent_store_t& s, const void* c, int64_t c_stride,
                                          const void* k_rope, int64_t k_rope_stride, bool bf16, const void* slots,
                                          bool index64, int64_t n, hipStream_t stream) {
  CacheParams p = params(s, slots, n);
  const int eb = bf16 ? 2 : 4;
  p.c = static_cast<const char*>(c);
  p.k_rope = static_cast<const char*>(k_rope);
  p.c_stride = c_stride * eb;
  p.k_rope_stride = k_rope_stride * eb;
  return launch<true>(p, bf16, index64, stream);
}

hipError_t launch_latent_dequantize_gather(const kda_latent_store_t& s, const void* slots, bool index64, int64_t n,
                                           void* out, bool bf16, hipStream_t stream) {
  CacheParams p = params(s, slots, n);
  p.out = static_cast<char*>(out);
  return launch<false>(p, bf16, index64, stream);
}

}  // namespace kda
