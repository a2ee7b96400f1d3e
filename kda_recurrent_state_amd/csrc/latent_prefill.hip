// Expanded latent attention over a varlen batch for gfx950: keys and values
// per head, the rotary part of the key shared by the heads.
//   s_ij = scale (q_i[:D] . k_j + q_i[D:] . kr_j),  out_i = sum_j softmax(s_i)_j v_j
// One pass over the keys with a running maximum and sum.  A wave owns 32
// queries and computes S^T = K Q^T with 32x32x16 products: a lane then holds
// one query's scores of 16 of 32 tokens, so row maxima and sums are taken in
// the lane (and its partner 32 further on), and the packed weights are already
// the right-hand operand of out^T = V^T P^T -- with the contraction in the
// order the scores lie in, which the transposed reads of V follow.
//
// Bound.  2 (D + R + E) flop a visible pair and head: the matrix unit.  16384
// tokens, 16 heads, D = E = 128, R = 64: 1.16-1.26 ms, 1090-1180 TFLOP/s, where
// a large library product reaches 1350 and would take 1.02 ms; the clock falls
// to 1.4 GHz under it.  With the weights' arithmetic spread between the next
// tile's products the kernel was 2 % slower.  Few queries over many keys are
// bound by the bytes of K and V: 16 x 64 queries over 1088 keys, 32 heads, 285
// MB in 60 us.
//
// Tile.  4 waves of 32 queries share tiles of 64 keys in two stages (80 KB), two
// workgroups a CU, so that one's products run beside the other's weights.
// Operands are read from LDS a group of four products ahead of their use.
#include "internal.h"
#include "latent_common.h"

namespace kda {
namespace {

using namespace latent;

constexpr int kTile = 64;       // keys a tile
constexpr int kWaves = 4;       // 32 queries each
constexpr int kQueries = 32 * kWaves;
// Key tiles a piece has at least where a workgroup's keys are split: 8 take
// about 12 us, joining two pieces 8 (128 queries over 1024 keys, 16 heads: 22 us
// in two pieces, 27 in one; over 4096: 28 us in eight, 95 in one).
constexpr int kPiece = 8;
constexpr int kMostSplits = 32;

struct PrefillParams {
  const __bf16 *q, *k, *kr, *v;
  int64_t qs[2], ks[2], vs[2], krs;
  const int32_t *cu_q, *cu_k;
  __bf16* out;
  float* lse;
  int64_t T, S;
  int N, H, D, R, E, causal;
  int tiles;       // upper bound of the query tiles of a head
  int splits;      // pieces the keys of a query tile are cut into at most
  float scale2;    // scale log2 e
  float* part;     // [splits][T][H][E] normalised outputs of pieces
  float2* psum;    // [splits][T][H] their maxima and the sums against them
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : (x > hi ? hi : x); }

// A query tile: queries qfirst .. of a sequence with lq queries from q0 and lk
// keys from k0, and the keys that the tile's last query sees.
struct QueryTile {
  int64_t q0, k0;
  int qfirst, lq, lk, end;
};

// Query tile x of the batch; false if there are fewer.  Up to 64 sequences are
// taken in the order of their keys, most first (31 x 700 queries, the last ones
// over 8000 keys: 215 us, in the batch's order 335); of a sequence the last
// tile, which sees most keys, comes first.
__device__ __forceinline__ bool find_tile(const PrefillParams& p, int x, int lane, QueryTile* out) {
  int n = -1, t = 0;
  int64_t q0 = 0, q1 = 0;
  int64_t behind = 0;  // the largest offset before these sequences
  for (int n0 = 0; n0 < p.N; n0 += 64) {
    int64_t a = p.T, b = p.T;
    int mine = n0 + lane;
    if (mine < p.N) {
      a = clamp64(p.cu_q[mine], 0, p.T);
      b = clamp64(p.cu_q[mine + 1], 0, p.T);
    }
    // An offset below one before it is raised to that one, so that no two
    // sequences have a query in common: they would write the same rows.
    if (__any(b < a || a < behind)) {
      int top = (int)(a < behind ? behind : a);
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(top, d, 64);
        if (lane >= d && y > top) top = y;
      }
      a = top;
      if (b < a) b = a;
    }
    behind = lane64(b, 63);
    int c = (int)((b - a + kQueries - 1) / kQueries);
    if (p.N <= 64 && p.N > 1) {
      // c of the sequence of this rank, which is put in ``mine``
      const int keys = lane < p.N ? (int)((unsigned)p.cu_k[lane + 1] - (unsigned)p.cu_k[lane]) : 0;
      int rank = 0;
      for (int j = 0; j < p.N; ++j) {
        const int other = __builtin_amdgcn_readlane(keys, j);
        rank += other > keys || (other == keys && j < lane) ? 1 : 0;
      }
      rank = lane < p.N ? rank : lane;  // (a permutation of the lanes)
      mine = __builtin_amdgcn_ds_permute(rank * 4, lane);
      c = __shfl(c, mine, 64);
      a = __shfl(a, mine, 64);
      b = __shfl(b, mine, 64);
    }
    const int incl = wave_scan(c, lane);
    const unsigned long long past = __ballot(incl > x);
    if (past) {
      const int i = __ffsll(past) - 1;
      n = __builtin_amdgcn_readlane(mine, i);
      t = __builtin_amdgcn_readlane(incl, i) - 1 - x;
      q0 = lane64(a, i);
      q1 = lane64(b, i);
      break;
    }
    x -= __builtin_amdgcn_readlane(incl, 63);
  }
  if (n < 0) return false;
  out->q0 = q0;
  out->qfirst = t * kQueries;
  const int lq = (int)(q1 - q0);
  out->k0 = lane64(clamp64(p.cu_k[n], 0, p.S), 0);
  const int lk = uniform((int)(clamp64(p.cu_k[n + 1], out->k0, p.S) - out->k0));
  const int last = out->qfirst + kQueries < lq ? out->qfirst + kQueries : lq;
  const int end = p.causal ? lk - (lq - last) : lk;
  out->lq = lq;
  out->lk = lk;
  out->end = end < 0 ? 0 : end;
  return true;
}

// Key tiles of a piece of a query tile that sees ``ntiles`` of them.
__device__ __forceinline__ int piece_tiles(const PrefillParams& p, int ntiles) {
  const int per = (ntiles + p.splits - 1) / p.splits;
  return per < kPiece ? kPiece : per;
}

// DP, RP, EP: D, R and E rounded up to what the kernel is built for
template <int DP, int RP, int EP>
__global__ __launch_bounds__(kQueries * 2, 2) void latent_prefill_kernel(PrefillParams p) {
  constexpr int W = kWaves;
  constexpr int KC = DP / 8, RC = RP / 8, VC = EP / 8;  // 16-byte chunks of a staged row
  constexpr int KS = (DP + RP) / 16;
  constexpr int MT = EP / 32;
  constexpr int kKeyBytes = kTile * DP * 2, kRotBytes = kTile * RP * 2, kStage = kKeyBytes + kRotBytes + kTile * EP * 2;
  __shared__ __attribute__((aligned(16))) char lds[2 * kStage];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 31, lh = lane >> 5;

  // Work items, the longest first.  A head's items run on one XCD, whose L2
  // then holds its keys and values: heads are dealt to the XCDs where they come
  // out even, else the list of (head, tile) is cut into eight parts (prompts
  // over prefixes, 32 heads: 91 us dealt, 109 cut; the longest come first only
  // in the former).
  const int xcd = blockIdx.x & 7, idx = (blockIdx.x >> 3) / p.splits, piece = (blockIdx.x >> 3) % p.splits;
  int h, x;
  if ((p.H & 7) == 0) {
    const int heads = p.H >> 3;
    h = xcd * heads + idx % heads;
    x = idx / heads;
  } else {
    const int64_t items = (int64_t)p.tiles * p.H, per = (items + 7) / 8, item = xcd * per + idx;
    if (idx >= per || item >= items) return;
    h = (int)(item / p.tiles);
    x = (int)(item % p.tiles);
  }
  QueryTile tile;
  if (!find_tile(p, x, lane, &tile)) return;
  const int64_t q0 = tile.q0, k0 = tile.k0;
  const int lq = tile.lq, lk = tile.lk, qfirst = tile.qfirst;
  // key tiles [first, last) of this piece
  const int ntiles = (tile.end + kTile - 1) / kTile, per_piece = piece_tiles(p, ntiles);
  const int first = piece * per_piece, last = first + per_piece < ntiles ? first + per_piece : ntiles;
  if (piece > 0 && first >= ntiles) return;

  const int qi = qfirst + wave * 32 + ln;  // this lane's query
  const int64_t qrow = q0 + (qi < lq ? qi : lq - 1);
  bf16x8 qf[KS];
  {
    const __bf16* qp = p.q + qrow * p.qs[0] + h * p.qs[1];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int c = 16 * s + 8 * lh;
      bf16x8 v = {};
      if (s < DP / 16) {
        if (c < p.D) v = *reinterpret_cast<const bf16x8*>(qp + c);
      } else {
        if (c - DP < p.R) v = *reinterpret_cast<const bf16x8*>(qp + p.D + (c - DP));
      }
      qf[s] = v;
    }
  }
  // keys that this lane's query sees, and that the wave's last one sees (none:
  // a wave without queries)
  const int sees = p.causal ? lk - (lq - 1 - qi) : lk;
  const int wlast = qfirst + wave * 32 + 32 < lq ? qfirst + wave * 32 + 32 : lq;
  const int wend = qfirst + wave * 32 >= lq ? 0 : (p.causal ? lk - (lq - wlast) : lk);
  const int all_see = p.causal ? lk - (lq - 1 - (qfirst + wave * 32)) : lk;  // the wave's first query

  f32x16 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
  float m = -INFINITY, l = 0.f;  // in units of scale2 s
  bool far = false;              // whether a query of the wave is_far

  // Staged rows: chunk c of a key or rotary row r lies at c ^ (r / (rows in 256
  // B)), of a value row at c ^ 4 (r & 3) (of 8 chunks: c ^ 4 ((r >> 1) & 1)).
  // The 16 lanes of a cycle of a 16-byte operand read have 16 rows of the two
  // halves, the 32 of a transposed 8-byte read four rows of four chunks, and
  // these fall on distinct banks (two lanes on each: 1275 -> 1263 us for 16384
  // tokens, 16 heads).  Each region is filled by loads of whole rows; a lane's
  // rows in successive loads differ by a multiple of 16, so its chunk is the
  // same.  Padding columns (D < DP, R < RP) of keys stay 0 from the start, as
  // the queries are there: anything else times 0 could be NaN.  Those of values
  // get copies of a row's last chunk and end in outputs that are not written.
  struct Region {
    const char* base;  // key 0
    int64_t step;      // bytes from key to key
    unsigned col;      // the lane's chunk
    bool there;        // whether a row has it (else the lane is off)
    int row;           // and its row in the first load
  };
  auto kswz = [](int r, int chunks) { return r / (16 / chunks) % chunks; };
  auto vswz = [](int r, int chunks) { return chunks >= 16 ? (r & 3) << 2 : (r & 2) << 1; };
  auto region = [&](const __bf16* base, int64_t stride, int chunks, int have, bool values) {
    Region g;
    g.base = reinterpret_cast<const char*>(base);
    g.step = stride * 2;
    g.row = (wave * 64 + lane) / chunks;
    const int pos = lane % chunks, c = pos ^ (values ? vswz(g.row, chunks) : kswz(g.row, chunks));
    g.col = (unsigned)(c < have ? c : have - 1) * 16;
    g.there = values || c < have;
    return g;
  };
  const Region kreg = region(p.k + k0 * p.ks[0] + h * p.ks[1], p.ks[0], KC, p.D / 8, false);
  const Region rreg = region(p.kr + k0 * p.krs, p.krs, RC > 0 ? RC : 8, p.R / 8, false);
  const Region vreg = region(p.v + k0 * p.vs[0] + h * p.vs[1], p.vs[0], VC, p.E / 8, true);
  const unsigned lds_at = lds_offset(lds) + wave * 1024;
  // loads of region g for the tile at key j0, of whose rows ``rows`` are there
  // (the others get the last one's bytes: their weights are 0)
  auto fill = [&](const Region& g, int chunks, int j0, int rows, unsigned to) {
    const int per = W * 64 / chunks;  // rows of the workgroup's loads
    const char* base = g.base + j0 * g.step;
    if (!g.there) return;
    if (rows >= kTile) {
      const unsigned off = (unsigned)g.row * (unsigned)g.step + g.col;
#pragma unroll
      for (int i = 0; i < kTile / per; ++i) load_lds16(base + i * per * g.step, off, to + i * W * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < kTile / per; ++i) {
        const int r = g.row + i * per < rows ? g.row + i * per : rows - 1;
        load_lds16(base, (unsigned)r * (unsigned)g.step + g.col, to + i * W * 1024);
      }
    }
  };
  auto stage = [&](int j) {
    const unsigned to = lds_at + (j & 1) * kStage;
    const int rows = lk - j * kTile;
    fill(kreg, KC, j * kTile, rows, to);
    if (RP > 0) fill(rreg, RC > 0 ? RC : 8, j * kTile, rows, to + kKeyBytes);
    fill(vreg, VC, j * kTile, rows, to + kKeyBytes + kRotBytes);
  };

  // the lane's places in a stage: key operands (row ln of a 32-row block,
  // chunk 2 k + lh) and transposed value reads (4 rows x 16 columns a group)
  const int kat = ln * DP * 2 + ((lh ^ kswz(ln, KC)) << 4), rat = kKeyBytes + ln * RP * 2;
  const int rx = kswz(ln, RC > 0 ? RC : 8);
  const int vrow = 4 * lh + ((lane & 15) >> 2), vcol = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  const int vat = kKeyBytes + kRotBytes + vrow * EP * 2 + (lane & 1) * 8;

  if (p.D < DP || p.R < RP) {
    for (int i = tid * 16; i < kKeyBytes + kRotBytes; i += W * 64 * 16)
#pragma unroll
      for (int b = 0; b < 2; ++b) *reinterpret_cast<u32x4*>(lds + b * kStage + i) = u32x4{0, 0, 0, 0};
    __syncthreads();
  }
  if (first < last) stage(first);
  for (int j = first; j < last; ++j) {
    wait_loads<0>();
    lds_barrier();  // tile j is there, and the readers of tile j - 1 are done
    if (j + 1 < last) stage(j + 1);
    if (j * kTile >= wend) continue;
    const char* buf = lds + (j & 1) * kStage;

    // ---- scores, operands read a group ahead
    f32x16 s[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
    {
      constexpr int F = 2 * KS, G = 4;
      bf16x8 kf[2][G];
      auto read = [&](int g) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const int f = g * G + i, k = f / 2, b = f % 2;
          if (f >= F) continue;
          const char* at = k < DP / 16 ? buf + (kat ^ (k % 8 * 32)) + k / 8 * 256 + b * 32 * DP * 2
                                       : buf + rat + (((2 * (k - DP / 16) + lh) ^ rx) << 4) + b * 32 * RP * 2;
          kf[g & 1][i] = *reinterpret_cast<const bf16x8*>(at);
        }
      };
      read(0);
#pragma unroll
      for (int g = 0; g < F / G; ++g) {
        if (g + 1 < F / G) read(g + 1);
        hold_order();
#pragma unroll
        for (int i = 0; i < G; ++i)
          s[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[g & 1][i], qf[(g * G + i) / 2], s[i & 1], 0, 0, 0);
        hold_order();
      }
    }
    if (j * kTile + kTile > all_see || j * kTile + kTile > lk) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = j * kTile + 32 * b + 8 * (i >> 2) + 4 * lh + (i & 3);
          if (key >= sees) s[b][i] = -INFINITY;
        }
    }
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
    mx = max_halves(mx) * p.scale2;
    // The maximum in use follows the true one only when that has grown by more
    // than 8 (a factor of 256): the weights stay far inside the range and the
    // output is seldom rescaled.
    float base = m;
    if (__any(mx > m + 8.f) || far) {
      const float mn = mx > m + 8.f ? mx : m;
      const float alpha = exp2_hw(m - (mn == -INFINITY ? 0.f : mn));
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] *= alpha;
      l *= alpha;
      base = m = mn;
      far = __any(is_far(m));
      if (far && is_far(m)) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[b][i] = from_far(s[b][i], p.scale2, m);
        base = 0.f;
      }
    }
    base = base == -INFINITY ? 0.f : base;
    // weights: bf16 for the matrix unit (the values' own type), their sum fp32
    bf16x8 pf[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e = exp2_hw(fmaf(s[b][i], p.scale2, -base));
        l += e;
        pf[b][i >> 3][i & 7] = (__bf16)e;
      }
    // ---- step (b, u): keys 32 b + 16 u + {4 lh .. + 3, 8 + 4 lh .. + 3}
    {
      constexpr int F = 4 * MT, G = 2;
      bf16x8 vf[2][G];
      auto read = [&](int g) {
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const int f = g * G + q, bu = f / MT, i = f % MT;
          // rows vrow + 16 bu and 8 further on: the same chunk
          const char* at = buf + vat + (((4 * i + vcol) ^ vswz(vrow, VC)) << 4) + bu * 16 * EP * 2;
          vf[g & 1][q] = join(read_tr(at), read_tr(at + 8 * EP * 2));
        }
      };
      read(0);
#pragma unroll
      for (int g = 0; g < F / G; ++g) {
        if (g + 1 < F / G) read(g + 1);
        hold_order();
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const int f = g * G + q, bu = f / MT, i = f % MT;
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[g & 1][q], pf[bu >> 1][bu & 1], acc[i], 0, 0, 0);
        }
        hold_order();
      }
    }
  }

  l = sum_halves(l);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  if (qi >= lq) return;
  const int64_t row = (q0 + qi) * p.H + h;
  if (per_piece >= ntiles) {  // all of the keys
    __bf16* op = p.out + row * p.E;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int col = 32 * i + 8 * g + 4 * lh;
        if (col >= p.E) continue;
        const bf16x4 o = {(__bf16)(acc[i][4 * g] * inv), (__bf16)(acc[i][4 * g + 1] * inv),
                          (__bf16)(acc[i][4 * g + 2] * inv), (__bf16)(acc[i][4 * g + 3] * inv)};
        *reinterpret_cast<bf16x4*>(op + col) = o;
      }
    if (p.lse && lh == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  } else {
    const int64_t slot = piece * p.T * p.H + row;
    float* op = p.part + slot * p.E;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int col = 32 * i + 8 * g + 4 * lh;
        if (col >= p.E) continue;
        *reinterpret_cast<f32x4*>(op + col) = f32x4{acc[i][4 * g] * inv, acc[i][4 * g + 1] * inv,
                                                    acc[i][4 * g + 2] * inv, acc[i][4 * g + 3] * inv};
      }
    if (lh == 0) p.psum[slot] = make_float2(m, l);
  }
}

// Joins the pieces of a query tile: half a wave a row, 4 columns a lane, 8
// rows a workgroup (a workgroup a tile takes 30 us, one row after the other).
// Grid: (query tiles x their rows / 8, heads).
constexpr int kJoinRows = 8;
__global__ __launch_bounds__(256) void latent_pieces_kernel(PrefillParams p) {
  const int lane = threadIdx.x & 63, half = threadIdx.x >> 5, c = (threadIdx.x & 31) * 4, h = blockIdx.y;
  QueryTile tile;
  if (!find_tile(p, blockIdx.x / (kQueries / kJoinRows), lane, &tile)) return;
  const int ntiles = (tile.end + kTile - 1) / kTile, per = piece_tiles(p, ntiles);
  if (per >= ntiles) return;
  const int pieces = (ntiles + per - 1) / per;
  const int64_t step = p.T * p.H;
  const int i = tile.qfirst + blockIdx.x % (kQueries / kJoinRows) * kJoinRows + half;
  if (i >= tile.lq) return;
  const int64_t row = (tile.q0 + i) * p.H + h;
  float top = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (int s = 0; s < pieces; ++s) top = fmaxf(top, p.psum[s * step + row].x);
  const float base = top == -INFINITY ? 0.f : top;
  f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < pieces; ++s) {
    const float2 ml = p.psum[s * step + row];
    const float f = exp2_hw(ml.x - base) * ml.y;
    sum += f;
    if (c < p.E) o += f * *reinterpret_cast<const f32x4*>(p.part + (s * step + row) * p.E + c);
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  if (c < p.E) {
    const bf16x4 ob = {(__bf16)(o[0] * inv), (__bf16)(o[1] * inv), (__bf16)(o[2] * inv), (__bf16)(o[3] * inv)};
    *reinterpret_cast<bf16x4*>(p.out + row * p.E + c) = ob;
  }
  if (p.lse && c == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

// Query tiles of a head at most, and the pieces their keys are cut into.  With
// 512 workgroups (two a CU) or more, every workgroup takes all keys of its
// tile; with fewer, the keys are split so that there are about as many (64
// queries over 65536 keys, 8 heads: 1299 -> 75 us).  Splitting up to 2048
// workgroups made 4096 queries over as many keys, 32 heads, 221 us instead of
// 179, and prompts over prefixes (12 sequences, 32 heads) 153 instead of 90.
void prefill_shape(int64_t T, int64_t S, int64_t N, int64_t H, int64_t* tiles, int64_t* splits) {
  *tiles = (T + (kQueries - 1) * N) / kQueries;
  const int64_t items = *tiles * H, room = items > 0 ? 512 / items : 1;
  const int64_t longest = ((S + kTile - 1) / kTile + kPiece - 1) / kPiece;  // pieces of the longest sequence
  int64_t s = room < longest ? room : longest;
  s = s < kMostSplits ? s : kMostSplits;
  *splits = s < 1 ? 1 : s;
}

int64_t workgroups(int64_t tiles, int64_t splits, int64_t H) { return (tiles * H + 7) / 8 * 8 * splits; }

template <int DP, int RP, int EP>
hipError_t launch(const PrefillParams& p, hipStream_t stream) {
  const int64_t blocks = workgroups(p.tiles, p.splits, p.H);
  hipLaunchKernelGGL((latent_prefill_kernel<DP, RP, EP>), dim3((unsigned)blocks), dim3(kQueries * 2), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL(latent_pieces_kernel, dim3((unsigned)p.tiles * (kQueries / kJoinRows), (unsigned)p.H), dim3(256),
                     0, stream, p);
  return hipGetLastError();
}

template <int DP, int EP>
hipError_t launch_r(const PrefillParams& p, hipStream_t stream) {
  if (p.R == 0) return launch<DP, 0, EP>(p, stream);
  return p.R <= 32 ? launch<DP, 32, EP>(p, stream) : launch<DP, 64, EP>(p, stream);
}

}  // namespace

int64_t latent_prefill_workgroups(int64_t T, int64_t S, int64_t N, int64_t H) {
  int64_t tiles, splits;
  prefill_shape(T, S, N, H, &tiles, &splits);
  return workgroups(tiles, splits, H);
}

size_t latent_prefill_workspace_bytes(int64_t T, int64_t S, int64_t N, int64_t H, int64_t E) {
  int64_t tiles, splits;
  prefill_shape(T, S, N, H, &tiles, &splits);
  return splits == 1 ? 0 : (size_t)(splits * T * H * (E + 2)) * 4;
}

hipError_t launch_latent_prefill(const kda_latent_prefill_args_t& a, hipStream_t stream) {
  PrefillParams p;
  p.q = static_cast<const __bf16*>(a.q);
  p.k = static_cast<const __bf16*>(a.k);
  p.kr = a.R > 0 ? static_cast<const __bf16*>(a.k_rope) : p.k;
  p.v = static_cast<const __bf16*>(a.v);
  for (int i = 0; i < 2; ++i) {
    p.qs[i] = a.q_stride[i];
    p.ks[i] = a.k_stride[i];
    p.vs[i] = a.v_stride[i];
  }
  p.krs = a.R > 0 ? a.k_rope_stride : 0;
  p.cu_q = a.cu_seqlens_q;
  p.cu_k = a.cu_seqlens_k;
  p.out = static_cast<__bf16*>(a.out);
  p.lse = a.lse;
  p.T = a.T;
  p.S = a.S;
  p.N = (int)a.N;
  p.H = (int)a.H;
  p.D = (int)a.D;
  p.R = (int)a.R;
  p.E = (int)a.E;
  p.causal = a.causal != 0;
  p.scale2 = a.scale * kLog2e;
  int64_t tiles, splits;
  prefill_shape(a.T, a.S, a.N, a.H, &tiles, &splits);
  p.tiles = (int)tiles;
  p.splits = (int)splits;
  p.part = static_cast<float*>(a.workspace);
  p.psum = splits > 1 ? reinterpret_cast<float2*>(p.part + splits * a.T * a.H * a.E) : nullptr;
  // (8 x 2048 tokens, 16 heads of 64: 117 us, padded to 128 columns 167)
  return a.D <= 64 && a.E <= 64 ? launch_r<64, 64>(p, stream) : launch_r<128, 128>(p, stream);
}

}  // namespace kda
