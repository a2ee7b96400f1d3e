// Absorbed latent attention over a paged cache (one to a few new tokens a
// sequence) for gfx950.
//
// Every cache row is one token's latent c (L values) and rotary key kr (R
// values), shared by all heads.  With the key up-projection folded into the
// query, a query row (one head of one new token) computes
//   s_j = scale (q . c_j + q_rope . kr_j),  out = sum_j softmax(s)_j c_j
// over the rows its token sees, so the same row is key and value: it is read
// once from HBM, staged in LDS, and serves both products from there.
//
// Work split.  The batch's rows, cut into tiles of 64 tokens, form one long
// line of tiles (sequence after sequence); workgroup w of G takes an equal
// share of that line, whatever the lengths are.  A share may end one
// sequence, hold several and begin another.  A piece that is a whole sequence
// is written as output; the others go to the workspace as normalised fp32
// outputs with their log-sum, and the join kernel weighs them.  Both kernels
// derive the shares from the lengths on the device, so a captured call
// follows its lengths.
#include "internal.h"
#include "latent_common.h"

namespace kda {
namespace {

using namespace latent;

constexpr int kTile = 64;      // tokens a tile
constexpr int kThreads = 256;  // 4 waves

struct DecodeParams {
  const __bf16* cache;
  int64_t page_stride;  // elements
  int64_t num_pages;
  int page_size, L, R;
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
  const int32_t* lengths;
  const __bf16* q;
  int64_t qs[3];
  const __bf16* qr;
  int64_t qrs[3];
  __bf16* out;
  float* lse;
  int N, Q, H, rows, row_blocks, groups;
  float scale2;   // scale log2 e
  float* part;    // [row_blocks][2 groups][MB][L] normalised outputs
  float* plse;    // [row_blocks][2 groups][MB] log2 of the sums
};

__device__ __forceinline__ int seq_tokens(const DecodeParams& p, int n) {
  const int len = p.lengths[n];
  const int64_t room = (int64_t)p.max_pages * p.page_size;
  return len < 0 ? 0 : (len > room ? (int)room : len);
}
__device__ __forceinline__ int seq_tiles(const DecodeParams& p, int n) {
  return (int)(((int64_t)seq_tokens(p, n) + kTile - 1) / kTile);
}

// Sum of the sequences' tiles, the same in all threads.
__device__ int64_t total_tiles(const DecodeParams& p, int64_t* red) {
  int64_t mine = 0;
  for (int n = threadIdx.x; n < p.N; n += kThreads) mine += seq_tiles(p, n);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) mine += __shfl_xor(mine, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mine;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// The sequence that holds tile x of the line, and the line position of its
// first tile: each wave scans the lengths 64 at a time.
__device__ void find_tile(const DecodeParams& p, int64_t x, int lane, int* seq, int64_t* first) {
  int64_t base = 0;
  for (int n0 = 0; n0 < p.N; n0 += 64) {
    const int c = n0 + lane < p.N ? seq_tiles(p, n0 + lane) : 0;
    const int incl = wave_scan(c, lane);
    const unsigned long long past = __ballot(base + incl > x);
    if (past) {
      const int i = __ffsll(past) - 1;
      *seq = n0 + i;
      *first = base + __shfl(incl - c, i, 64);
      return;
    }
    base += __shfl(incl, 63, 64);
  }
  *seq = p.N;
  *first = base;
}

// LP, RP: L and R rounded up to what the kernel is built for; NB: blocks of 16
// query rows a workgroup.
template <int LP, int RP, int NB>
__global__ __launch_bounds__(kThreads, 2) void latent_decode_kernel(DecodeParams p) {
  constexpr int MB = 16 * NB;
  constexpr int DP = LP + RP;
  constexpr int KC = DP / 8;        // 16-byte chunks of a staged row
  constexpr int KS = DP / 32;       // contraction steps of the scores
  constexpr int MT = LP / 64;       // 16-column blocks of the output a wave
  constexpr int TB = NB;            // 16-token blocks a wave scores
  // staged row r: chunk c at position c ^ (r & 7), so that the 16 rows x 16 B
  // of a score operand and the 4 rows x 32 B of a transposed value read both
  // fall on distinct banks
  __shared__ __attribute__((aligned(16))) __bf16 tile[kTile * DP];
  __shared__ __attribute__((aligned(16))) __bf16 prob[MB * kTile];
  __shared__ float smax[4][16];
  __shared__ float ssum[4][16];
  __shared__ int64_t row_at[kTile];
  __shared__ int64_t red[4];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  // workgroups that share rows of the cache (the row blocks of one share) run
  // on one XCD, whose L2 then serves all but the first
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int rb = idx % p.row_blocks, w = (idx / p.row_blocks) * 8 + xcd;

  const int64_t total = total_tiles(p, red);
  const int64_t shares = total < p.groups ? total : p.groups;  // none is empty
  if (w >= shares) return;
  int64_t t0 = w * total / shares;
  const int64_t t1 = (w + 1) * total / shares;
  int n = 0;
  int64_t first = 0;
  find_tile(p, t0, lane, &n, &first);
  n = __builtin_amdgcn_readfirstlane(n);

  if (p.L < LP || p.R < RP) {  // padding columns are zero from here on
    for (int i = tid; i < kTile * KC; i += kThreads) reinterpret_cast<u32x4*>(tile)[i] = u32x4{0, 0, 0, 0};
    __syncthreads();
  }
  const int rblock = NB == 2 ? (wave & 1) : 0;          // query rows this wave scores
  const int tok0 = NB == 2 ? 32 * (wave >> 1) : 16 * wave;  // and tokens

  while (t0 < t1) {
    // ---- one piece: tiles [a, b) of sequence n
    int tiles = seq_tiles(p, n);
    while (first + tiles <= t0) {  // (empty sequences have no tiles)
      first += tiles;
      ++n;
      tiles = seq_tiles(p, n);
    }
    const int a = (int)(t0 - first);
    const int b = (int)((t1 - first) < tiles ? (t1 - first) : tiles);
    const int len = seq_tokens(p, n);
    const int32_t* table = p.table + n * p.table_stride;

    // query operand: row ln of the wave's row block, 8 values a step
    bf16x8 qf[KS];
    const int qrow = rb * MB + rblock * 16 + ln;
    {
      const bool have = qrow < p.rows;
      const int qi = have ? qrow / p.H : 0, qh = have ? qrow % p.H : 0;
      const __bf16* qp = p.q + n * p.qs[0] + qi * p.qs[1] + qh * p.qs[2];
      const __bf16* qrp = p.qr + n * p.qrs[0] + qi * p.qrs[1] + qh * p.qrs[2];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int c = 32 * s + 8 * lg;
        bf16x8 x = {};
        if (c < LP) {
          if (have && c < p.L) x = *reinterpret_cast<const bf16x8*>(qp + c);
        } else {
          if (have && c - LP < p.R) x = *reinterpret_cast<const bf16x8*>(qrp + (c - LP));
        }
        qf[s] = x;
      }
    }
    const int sees = len - (p.Q - 1 - (qrow < p.rows ? qrow / p.H : 0));  // tokens this lane's row sees
    const int all_see = len - (p.Q - 1);

    float m[NB], l = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i) m[i] = -INFINITY;
    f32x4 acc[MT][NB];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    for (int t = a; t < b; ++t) {
      // rows of this tile: lane i looks up token 64 t + i
      const int pos = t * kTile + lane;
      int64_t at = -1;
      if (pos < len) {
        const int pg = pos / p.page_size;
        const int page = table[pg];
        if (page >= 0 && page < p.num_pages)
          at = page * p.page_stride + (int64_t)(pos - pg * p.page_size) * (p.L + p.R);
      }
      const unsigned long long live = __ballot(at >= 0);
      __syncthreads();  // the last tile's readers are done
      if (wave == 0) row_at[lane] = at;
      __syncthreads();
#pragma unroll 6
      for (int i = 0; i < kTile * KC / kThreads; ++i) {
        const int c0 = (wave * (kTile * KC / kThreads) + i) * 64;
        const int c = c0 + lane;
        const int r = c / KC, src = (c - r * KC) ^ (r & 7);
        const int64_t ro = row_at[r];
        const int e = src < LP / 8 ? src * 8 : (src - LP / 8) * 8 + p.L;
        const bool have = src < LP / 8 ? src * 8 < p.L : (src - LP / 8) * 8 < p.R;
        if (have && ro >= 0) load_lds16(p.cache + ro + e, tile + c0 * 8);
        if (have && ro < 0) reinterpret_cast<u32x4*>(tile)[c] = u32x4{0, 0, 0, 0};
      }
      wait_loads();
      __syncthreads();

      // ---- scores, transposed: S^T[token][row]; lane holds tokens 4 lg + i
      f32x4 s[TB];
#pragma unroll
      for (int j = 0; j < TB; ++j) s[j] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
#pragma unroll
        for (int j = 0; j < TB; ++j) {
          const int r = tok0 + 16 * j + ln;
          const bf16x8 kf = *reinterpret_cast<const bf16x8*>(tile + (r * KC + ((4 * k + lg) ^ (r & 7))) * 8);
          s[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[k], s[j], 0, 0, 0);
        }
      }
      if (t * kTile + kTile > all_see || live != ~0ull) {
#pragma unroll
        for (int j = 0; j < TB; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tk = tok0 + 16 * j + 4 * lg + i;
            if (t * kTile + tk >= sees || !((live >> tk) & 1)) s[j][i] = -INFINITY;
          }
      }
      float mx = s[0][0];
#pragma unroll
      for (int j = 0; j < TB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[j][i]);
      mx = max_halves(max_quarters(mx));
      if (lg == 0) smax[wave][ln] = mx;
      __syncthreads();
      float alpha[NB], mb[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        float x;
        if (NB == 2) {
          x = fmaxf(smax[j][ln], smax[j + 2][ln]);
        } else {
          x = fmaxf(fmaxf(smax[0][ln], smax[1][ln]), fmaxf(smax[2][ln], smax[3][ln]));
        }
        const float mn = fmaxf(m[j], x * p.scale2);
        mb[j] = mn == -INFINITY ? 0.f : mn;
        alpha[j] = exp2_hw(m[j] - mb[j]);
        m[j] = mn;
      }
      const float base = NB == 2 && rblock ? mb[NB - 1] : mb[0];
      const float al = NB == 2 && rblock ? alpha[NB - 1] : alpha[0];
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        bf16x4 pb;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = exp2_hw(fmaf(s[j][i], p.scale2, -base));
          sum += e;
          // the weights go to the matrix unit in bf16, the values' own type;
          // their sum stays in fp32
          pb[i] = (__bf16)e;
        }
        const int r = rblock * 16 + ln, tk = tok0 + 16 * j + 4 * lg;
        *reinterpret_cast<bf16x4*>(prob + r * kTile + (((tk >> 3) ^ (r & 7)) << 3) + (tk & 7)) = pb;
      }
      l = l * al + sum;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] *= alpha[j];
      __syncthreads();

      // ---- out^T[column][row] += rows^T P^T; the wave's columns
#pragma unroll
      for (int k = 0; k < kTile / 32; ++k) {
        bf16x8 pf[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int r = j * 16 + ln;
          pf[j] = *reinterpret_cast<const bf16x8*>(prob + r * kTile + (((4 * k + lg) ^ (r & 7)) << 3));
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int col = wave * (LP / 4) + 16 * i + 4 * (ln & 3);
          const int r0 = 32 * k + 8 * lg + (ln >> 2), r1 = r0 + 4;
          const s16x4 lo = read_tr(tile + (r0 * KC + ((col >> 3) ^ (r0 & 7))) * 8 + (col & 7));
          const s16x4 hi = read_tr(tile + (r1 * KC + ((col >> 3) ^ (r1 & 7))) * 8 + (col & 7));
          const bf16x8 vf = join(lo, hi);
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[j], acc[i][j], 0, 0, 0);
        }
      }
    }

    // ---- the piece's sums over the lanes and waves that share a row
    l = sum_halves(sum_quarters(l));
    __syncthreads();
    if (lg == 0) ssum[wave][ln] = l;
    __syncthreads();
    const bool whole = a == 0 && b == tiles;
    const int slot = 2 * w + (a > 0 ? 0 : 1);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const float sum = NB == 2 ? ssum[j][ln] + ssum[j + 2][ln]
                                : (ssum[0][ln] + ssum[1][ln]) + (ssum[2][ln] + ssum[3][ln]);
      const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
      const int row = rb * MB + j * 16 + ln;
      if (row >= p.rows) continue;
      const float lse2 = sum == 0.f ? -INFINITY : m[j] + __log2f(sum);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int col = wave * (LP / 4) + 16 * i + 4 * lg;
        if (col >= p.L) continue;
        const f32x4 o = acc[i][j] * inv;
        if (whole) {
          const bf16x4 ob = {(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
          *reinterpret_cast<bf16x4*>(p.out + ((int64_t)n * p.rows + row) * p.L + col) = ob;
        } else {
          *reinterpret_cast<f32x4*>(p.part + (((int64_t)rb * 2 * p.groups + slot) * MB + j * 16 + ln) * p.L + col) = o;
        }
      }
      if (wave == 0 && lg == 0) {
        if (whole) {
          if (p.lse) p.lse[(int64_t)n * p.rows + row] = lse2 * kLn2;
        } else {
          p.plse[((int64_t)rb * 2 * p.groups + slot) * MB + j * 16 + ln] = lse2;
        }
      }
    }
    t0 = first + b;
  }
}

// Joins the pieces of sequences that several workgroups share, and writes the
// outputs of empty sequences.  Grid: (query row pairs, sequences); 128
// threads a row.
__global__ __launch_bounds__(kThreads) void latent_join_kernel(DecodeParams p, int MB) {
  __shared__ int64_t red[4];
  const int n = blockIdx.y, lane = threadIdx.x & 63;
  const int tiles = seq_tiles(p, n);
  const int row = blockIdx.x * 2 + (threadIdx.x >> 7), c = (threadIdx.x & 127) * 4;
  if (tiles == 0) {
    if (row < p.rows) {
      for (int k = c; k < p.L; k += 512)
        *reinterpret_cast<bf16x4*>(p.out + ((int64_t)n * p.rows + row) * p.L + k) = bf16x4{};
      if (p.lse && c == 0) p.lse[(int64_t)n * p.rows + row] = -INFINITY;
    }
    return;
  }
  const int64_t total = total_tiles(p, red);
  int64_t first = 0;  // line position of the sequence's first tile
  for (int n0 = 0; n0 < n; n0 += 64) {
    int x = n0 + lane < n ? seq_tiles(p, n0 + lane) : 0;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
    first += x;
  }
  // the shares that hold its first and its last tile
  const int64_t shares = total < p.groups ? total : p.groups;
  const int w0 = (int)(((first + 1) * shares - 1) / total), w1 = (int)(((first + tiles) * shares - 1) / total);
  if (w0 == w1 || row >= p.rows) return;
  const int rb = row / MB, rr = row % MB;
  // share w0 holds the sequence's beginning (slot 2 w0 + 1), the later ones
  // begin in mid-sequence (slot 2 w)
  const int64_t at = ((int64_t)rb * 2 * p.groups) * MB + rr;
  float top = -INFINITY;
  for (int w = w0; w <= w1; ++w) top = fmaxf(top, p.plse[at + (int64_t)(2 * w + (w == w0 ? 1 : 0)) * MB]);
  const float base = top == -INFINITY ? 0.f : top;
  f32x4 o = {0, 0, 0, 0};
  float sum = 0.f;
  for (int w = w0; w <= w1; ++w) {
    const int64_t s = at + (int64_t)(2 * w + (w == w0 ? 1 : 0)) * MB;
    const float f = exp2_hw(p.plse[s] - base);
    sum += f;
    if (c < p.L) o += f * *reinterpret_cast<const f32x4*>(p.part + s * p.L + c);
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  if (c < p.L) {
    const bf16x4 ob = {(__bf16)(o[0] * inv), (__bf16)(o[1] * inv), (__bf16)(o[2] * inv), (__bf16)(o[3] * inv)};
    *reinterpret_cast<bf16x4*>(p.out + ((int64_t)n * p.rows + row) * p.L + c) = ob;
  }
  if (p.lse && c == 0)
    p.lse[(int64_t)n * p.rows + row] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

struct Shape {
  int nb, row_blocks, groups;
};

// Query rows a workgroup and shares of the line.  Two workgroups fit a CU
// (LDS), so 512 in all; the shares are a multiple of 8, one set an XCD.
Shape decode_shape(int64_t Q, int64_t H) {
  Shape s;
  const int64_t rows = Q * H;
  s.nb = rows <= 16 ? 1 : 2;
  s.row_blocks = (int)((rows + 16 * s.nb - 1) / (16 * s.nb));
  int g = 512 / s.row_blocks;
  g = g / 8 * 8;
  s.groups = g < 8 ? 8 : g;
  return s;
}

template <int LP, int RP>
hipError_t launch_nb(const DecodeParams& p, int nb, hipStream_t stream) {
  const dim3 grid((unsigned)(p.groups * p.row_blocks));
  if (nb == 1)
    hipLaunchKernelGGL((latent_decode_kernel<LP, RP, 1>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((latent_decode_kernel<LP, RP, 2>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <int LP>
hipError_t launch_r(const DecodeParams& p, int nb, hipStream_t stream) {
  return p.R == 0 ? launch_nb<LP, 0>(p, nb, stream) : launch_nb<LP, 64>(p, nb, stream);
}

}  // namespace

size_t latent_decode_workspace_bytes(int64_t N, int64_t Q, int64_t H, int64_t L) {
  (void)N;
  const Shape s = decode_shape(Q, H);
  const int64_t slots = (int64_t)s.row_blocks * 2 * s.groups * 16 * s.nb;
  return (size_t)slots * (size_t)(L + 1) * 4;
}

hipError_t launch_latent_decode(const kda_latent_decode_args_t& a, hipStream_t stream) {
  const Shape s = decode_shape(a.Q, a.H);
  DecodeParams p;
  p.cache = static_cast<const __bf16*>(a.cache);
  p.page_stride = a.page_stride;
  p.num_pages = a.num_pages;
  p.page_size = (int)a.page_size;
  p.L = (int)a.L;
  p.R = (int)a.R;
  p.table = a.page_table;
  p.table_stride = a.table_stride;
  p.max_pages = (int)a.max_pages;
  p.lengths = a.lengths;
  p.q = static_cast<const __bf16*>(a.q);
  p.qr = a.R > 0 ? static_cast<const __bf16*>(a.q_rope) : p.q;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a.q_stride[i];
    p.qrs[i] = a.R > 0 ? a.q_rope_stride[i] : 0;
  }
  p.out = static_cast<__bf16*>(a.out);
  p.lse = a.lse;
  p.N = (int)a.N;
  p.Q = (int)a.Q;
  p.H = (int)a.H;
  p.rows = (int)(a.Q * a.H);
  p.row_blocks = s.row_blocks;
  p.groups = s.groups;
  p.scale2 = a.scale * kLog2e;
  const int64_t slots = (int64_t)s.row_blocks * 2 * s.groups * 16 * s.nb;
  p.part = static_cast<float*>(a.workspace);
  p.plse = p.part + slots * a.L;
  hipError_t e = a.L <= 128 ? launch_r<128>(p, s.nb, stream)
                            : (a.L <= 256 ? launch_r<256>(p, s.nb, stream) : launch_r<512>(p, s.nb, stream));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(latent_join_kernel, dim3((unsigned)((p.rows + 1) / 2), (unsigned)p.N), dim3(kThreads), 0, stream,
                     p, 16 * s.nb);
  return hipGetLastError();
}

}  // namespace kda
