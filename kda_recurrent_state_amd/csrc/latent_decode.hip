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
// Bound.  A row is 2 (L + R) bytes and 2 (2 L + R) flop a query row: with 64
// query rows about 120 flop a byte, below the 270 at which this chip's copies
// (5 TB/s) and matrix products (1350 TFLOP/s) balance.  64 query rows over 200
// ragged sequences (L = 512, R = 64, 414 MB): 127-145 us, join included, where a
// copy's rate gives 84; 128 rows over 64 x 16000 tokens: 366-384 us, 740
// TFLOP/s, where the bytes give 236 and the products 206.  What the kernel
// adds are the phases of a tile that do not overlap in a workgroup (scores,
// weights, output, two barriers) and, with 128 rows, the second row block's
// reads of the same rows from L2.
//
// Tile.  64 tokens in two stages of 72 KB fill the LDS, so a CU has one
// workgroup of 8 waves.  For the scores a wave takes a block of 16 query rows
// and a group of the tokens, for the output all rows and an eighth of the
// columns, so the weights go through LDS and the output stays in registers (64
// a lane at 64 rows).  Tiles of 32 tokens in four stages took 134 / 397 us
// where these then took 134 / 394; 4 waves of 512 registers 136 / 414 where 8
// took 143 / 400, and with 128 rows a workgroup 742 (the registers did not hold
// output, queries and scores).
//
// Work split.  The batch's rows, cut into tiles of 64 tokens, form one long
// line of tiles (sequence after sequence); workgroup w of G takes an equal
// share of that line, whatever the lengths are.  A share may end one
// sequence, hold several and begin another.  A piece that is a whole sequence
// is written as output; the others go to the workspace as normalised fp32
// outputs with their maximum and sum (one number for both would lose the sum of
// scores that are large), and the join kernel weighs them.  Both kernels
// derive the shares from the lengths on the device, so a captured call
// follows its lengths.
#include "internal.h"
#include "latent_tile.h"

namespace kda {
namespace {

using namespace latent;

struct DecodeParams {
  const __bf16* cache;
  int64_t page_stride;  // elements
  int num_pages, page_size, L, R;
  uint32_t page_mul;  // j / page_size = j page_mul >> page_shift, 0 <= j < 2^31
  int page_shift;
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
  float scale2;    // scale log2 e
  float* part;     // [row_blocks][2 groups][MB][L] normalised outputs
  float2* psum;    // [row_blocks][2 groups][MB] the maxima and the sums against them
  int32_t* shared; // [N][2] first and last share of a sequence
};

__device__ __forceinline__ int seq_tokens(const DecodeParams& p, int n) {
  const int len = p.lengths[n];
  const int64_t room = (int64_t)p.max_pages * p.page_size;
  return len < 0 ? 0 : (len > room ? (int)room : len);
}
__device__ __forceinline__ int tiles_of(int tokens) { return (int)(((int64_t)tokens + kTile - 1) / kTile); }

// Share w of the line: its tiles and where they begin.
struct Share {
  int left;  // tiles, 0: no such share
  int n, t;  // sequence and tile of the first one
  int len;   // and that sequence's tokens
};

// Shares are as equal as they can be and none is empty (there are fewer of
// them where there are fewer tiles).
__device__ __forceinline__ int64_t share_begin(const DecodeParams& p, int64_t total, int w, int* left) {
  const int64_t shares = total < p.groups ? total : p.groups;
  int64_t quot = 1, rem = 0;
  if (total >= p.groups) {
    quot = total <= 0xffffffffll ? (int64_t)((uint32_t)total / (uint32_t)p.groups) : total / p.groups;
    rem = total - quot * p.groups;
  }
  *left = w < shares ? (int)(quot + (w < rem ? 1 : 0)) : 0;
  return w * quot + (w < rem ? w : rem);
}

// Every wave scans the lengths by itself, 64 at a time, once for the sum and
// once for the place.
__device__ __forceinline__ Share find_share(const DecodeParams& p, int w, int lane) {
  Share s;
  int64_t total = 0;
  for (int n = lane; n < p.N; n += 64) total += tiles_of(seq_tokens(p, n));
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) total += __shfl_xor(total, d, 64);
  const int64_t t0 = share_begin(p, lane64(total, 0), w, &s.left);
  int64_t base = 0;
  for (int n0 = 0; s.left > 0 && n0 < p.N; n0 += 64) {
    const int tokens = n0 + lane < p.N ? seq_tokens(p, n0 + lane) : 0, c = tiles_of(tokens);
    const int incl = wave_scan(c, lane);
    const unsigned long long past = __ballot(base + incl > t0);
    if (past) {
      const int i = __ffsll(past) - 1;
      s.n = n0 + i;
      s.t = (int)(t0 - base) - __builtin_amdgcn_readlane(incl - c, i);
      s.len = __builtin_amdgcn_readlane(tokens, i);
      return s;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  s.left = 0;
  return s;
}

template <int LP, int RP, int NB, bool kPad>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void latent_decode_kernel(DecodeParams p) {
  using D = Bf16Tile<LP, RP, NB, kPad>;
  constexpr int MB = D::MB, KS = D::KS, MT = D::MT, TG = D::TG, TB = D::TB;
  __shared__ __attribute__((aligned(16))) __bf16 stage[2][D::kStage];
  __shared__ __attribute__((aligned(16))) __bf16 rotary[2][RP > 0 ? kTile * RP : 8];
  __shared__ __attribute__((aligned(16))) __bf16 prob[MB * kTile];
  __shared__ float smax[TG][MB];  // of a tile; at a piece's end the sums
  __shared__ float sfac[MB];      // factor of the older output; at a piece's end the maxima
  __shared__ int32_t pages[2][kWaves][64];  // page of token 64 t + lane of the tile located next
  __shared__ int grown[2];        // whether a row's maximum has grown much in this tile
  __shared__ int64_t qat[2][MB];           // of a query row: its q and q_rope in a sequence's
  __shared__ int32_t less[MB];             // and how many tokens less than the last one it sees

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  // workgroups that share rows of the cache (the row blocks of one share) run
  // on one XCD, whose L2 then serves all but the first
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int rb = idx % p.row_blocks, w = (idx / p.row_blocks) * 8 + xcd;

  if (tid < MB) {
    // (rows behind the last get the first one's queries; they are not written)
    const int row = rb * MB + tid < p.rows ? rb * MB + tid : 0, qi = row / p.H, qh = row - qi * p.H;
    qat[0][tid] = qi * p.qs[1] + qh * p.qs[2];
    qat[1][tid] = qi * p.qrs[1] + qh * p.qrs[2];
    less[tid] = p.Q - 1 - qi;
  }
  if (tid < 2) grown[tid] = 0;
  const Share share = find_share(p, w, lane);
  if (share.left == 0) return;
  if (kPad) {
    u32x4 *st = reinterpret_cast<u32x4*>(stage), *ro = reinterpret_cast<u32x4*>(rotary);
    for (unsigned i = tid; i < sizeof(stage) / 16; i += kThreads) st[i] = u32x4{0, 0, 0, 0};
    for (unsigned i = tid; i < sizeof(rotary) / 16; i += kThreads) ro[i] = u32x4{0, 0, 0, 0};
  }
  const bool scoring = wave < D::kScoring;
  const int rblock = wave % NB;                  // query rows this wave scores
  const int tg = (wave / NB) % TG;               // and tokens
  __syncthreads();
  const int sees_less = less[rblock * 16 + ln];
  auto tokens_of = [&](int n) { return uniform(seq_tokens(p, n)); };

  // where the page of token 64 t + lane of sequence s is, which has len tokens
  // (the last one's for lanes behind it), and that row's place; -1: no such row
  auto page_of = [&](int pos) { return (unsigned)(((uint64_t)(unsigned)pos * p.page_mul) >> p.page_shift); };
  auto lookup = [&](int s, int t, int len) {
    const int pos = t * kTile + lane;
    return p.table + s * p.table_stride + page_of(pos < len ? pos : len - 1);
  };
  auto place = [&](int page, int t, int len) {
    const int pos = t * kTile + lane;
    const bool there = pos < len && (unsigned)page < (unsigned)p.num_pages;
    return there ? (int64_t)page * p.page_stride + (int64_t)(pos - (int)page_of(pos) * p.page_size) * (p.L + p.R) : (int64_t)-1;
  };
  bf16x8 qf[KS];
  auto load_q = [&](int s) {
    const int row = keep_here(rblock * 16 + ln), lg = keep_here(lane >> 4);
    const __bf16* qp = p.q + s * p.qs[0] + qat[0][row] + 8 * lg;
    const __bf16* qrp = p.qr + s * p.qrs[0] + qat[1][row] + 8 * lg;
    if (!kPad) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
        qf[k] = *reinterpret_cast<const bf16x8*>(k < LP / 32 ? qp + 32 * k : qrp + (32 * k - LP));
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int c = 32 * k + 8 * lg;
        bf16x8 x = {};
        if (k < LP / 32 ? c < p.L : c - LP < p.R)
          x = *reinterpret_cast<const bf16x8*>(k < LP / 32 ? qp + 32 * k : qrp + (32 * k - LP));
        qf[k] = x;
      }
    }
  };

  // The tiles in hand: the one computed, the next one, and the one after it,
  // whose pages are being looked up.  ``left`` counts the share's tiles behind
  // the one computed.
  struct Tile {
    int n, t, len;            // tile t of sequence n, which has len tokens
    unsigned long long live;  // which rows are there
  };
  int left = uniform(share.left) - 1;
  Tile cur, next, ask;
  const char* at;      // rows of the last tile located (lane i: token i)
  // Rows that are not there are fetched from the first one that is (their
  // weights are 0); a tile without any is not fetched and not computed.
  auto locate = [&](int page, Tile& x) {
    int64_t row = place(page, x.t, x.len);
    x.live = __ballot(row >= 0);
    if (x.live != ~0ull) {
      const int64_t some = x.live != 0 ? lane64(row, __ffsll(x.live) - 1) : 0;
      row = row < 0 ? some : row;
    }
    at = reinterpret_cast<const char*>(p.cache + row);
  };
  auto follow = [&](Tile& x) {  // the tile behind x
    if (++x.t < tiles_of(x.len)) return;
    x.t = 0;
    do x.len = tokens_of(++x.n);
    while (x.len == 0);
  };
  const unsigned stage_at = lds_offset(stage), rotary_at = lds_offset(rotary), pages_at = lds_offset(pages[0][wave]);
  constexpr unsigned kStageBytes = D::kStage * 2, kRotaryBytes = sizeof(rotary[0]), kPagesBytes = sizeof(pages[0]);
  const typename D::Columns columns = D::columns(p.L, p.R, wave, lane);
  auto fetch = [&](int i, int to) { D::fetch(i, at, wave, lane, columns, stage_at + to * kStageBytes); };
  cur.n = uniform(share.n);
  cur.t = uniform(share.t);
  cur.len = uniform(share.len);
  locate(*lookup(cur.n, cur.t, cur.len), cur);
  D::fetch_rotary(at, wave, lane, columns, rotary_at);
#pragma unroll
  for (int i = 0; i < D::kLat; ++i) fetch(i, 0);
  next = ask = cur;
  if (left > 0) {
    follow(ask);
    load_lds4(lookup(ask.n, ask.t, ask.len), pages_at);
  }
  if (scoring) load_q(cur.n);
  int begin = cur.t;

  float m = -INFINITY, l = 0.f;  // of row ln of the wave's block, over its tokens; units of scale2 s
  bool far = false;              // whether one of the wave's rows is_far
  f32x4 acc[MT][NB];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  for (int par = 0;; par ^= 1) {
    wait_loads<0>();
    lds_barrier();  // this tile has landed, and the readers of the one before are done
    const bool more = left > 0;
    if (more) {
      next = ask;
      locate(pages[par][wave][lane], next);
      if (--left > 0) {
        follow(ask);
        load_lds4(lookup(ask.n, ask.t, ask.len), pages_at + (par ^ 1) * kPagesBytes);
      }
    }
    if (tid == 0) grown[par ^ 1] = 0;
    const bool fetches = more && next.live != 0;
    if (fetches) D::fetch_rotary(at, wave, lane, columns, rotary_at + (par ^ 1) * kRotaryBytes);
    if (fetches && !(scoring && cur.live)) {
#pragma unroll
      for (int i = 0; i < D::kLat; ++i) fetch(i, par ^ 1);
    }
    if (cur.live) {
      float sum = 0.f, fac = 1.f;
      f32x4 s[TB];
      // Weights of the scores against the maximum in use, for the matrix unit
      // in bf16, the values' own type; their sum stays in fp32.
      auto weigh = [&](float base) {
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < TB; ++j) {
          bf16x4 pb;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = exp2_hw(fmaf(s[j][i], p.scale2, -base));
            sum += e;
            pb[i] = (__bf16)e;
          }
          const int tk = 16 * (TB * tg + j) + 4 * lg;
          *reinterpret_cast<bf16x4*>(prob + (rblock * 16 + ln) * kTile + (((tk >> 3) ^ (ln & 7)) << 3) + (tk & 7)) = pb;
        }
      };
      if (scoring) {
        D::scores(stage[par] + (16 * TB * tg + ln) * LP, rotary[par] + (16 * TB * tg + ln) * RP, qf, ln, lg, s,
                  [&](int i) {
                    if (fetches) fetch(i, par ^ 1);
                  });
        if (cur.t * kTile + kTile > cur.len - (p.Q - 1) || cur.live != ~0ull) {
#pragma unroll
          for (int j = 0; j < TB; ++j) {
            // of the lane's four tokens: how many are seen, and which are there
            const int at4 = 16 * (TB * tg + j) + 4 * lg, sees = cur.len - sees_less - cur.t * kTile - at4;
            const unsigned there = (unsigned)(cur.live >> at4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i >= sees || !(there >> i & 1)) s[j][i] = -INFINITY;
          }
        }
        float mx = s[0][0];
#pragma unroll
        for (int j = 0; j < TB; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[j][i]);
        mx = max_halves(max_quarters(mx)) * p.scale2;
        if (lg == 0) smax[tg][rblock * 16 + ln] = mx;
        // The maximum in use follows the true one only when that is larger by
        // more than 8 (a factor of 256): the weights stay far inside the range,
        // and most tiles need neither an exchange of maxima between the waves
        // nor a rescaling of the output.  (Rows that are far go the same way.)
        if (__any(mx > m + 8.f) || far) {
          if (lane == 0) grown[par] = 1;
        }
        weigh(m == -INFINITY ? 0.f : m);
      }
      lds_barrier();
      if (grown[par]) {
        if (scoring) {
          float mx = smax[0][rblock * 16 + ln];
#pragma unroll
          for (int g = 1; g < TG; ++g) mx = fmaxf(mx, smax[g][rblock * 16 + ln]);
          const float mn = mx > m + 8.f ? mx : m;
          fac = exp2_hw(m - (mn == -INFINITY ? 0.f : mn));
          m = mn;
          if (tg == 0 && lg == 0) sfac[rblock * 16 + ln] = fac;
        }
        lds_barrier();  // (all have read the maxima; the weights are written again)
        if (scoring) {
          float base = m == -INFINITY ? 0.f : m;
          far = __any(is_far(m));
          if (far && is_far(m)) {
#pragma unroll
            for (int j = 0; j < TB; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[j][i] = from_far(s[j][i], p.scale2, m);
            base = 0.f;
          }
          weigh(base);
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const float f = sfac[j * 16 + ln];
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[i][j] *= f;
        }
        lds_barrier();
      }
      l = l * fac + sum;
      D::values(stage[par], prob, wave, ln, lg, acc);
    }

    if (!more || next.n != cur.n) {
      const int n = cur.n, t = cur.t, tiles = tiles_of(cur.len);
      // ---- the end of a piece: tiles [begin, t] of sequence n
      if (more && scoring) load_q(next.n);
      l = sum_halves(sum_quarters(l));
      lds_barrier();
      const int ln = keep_here(lane & 15), lg = keep_here(lane >> 4);
      if (scoring && lg == 0) {
        smax[tg][rblock * 16 + ln] = l;
        if (tg == 0) sfac[rblock * 16 + ln] = m;
      }
      lds_barrier();
      const bool whole = begin == 0 && t == tiles - 1;
      const int slot = rb * 2 * p.groups + 2 * w + (begin > 0 ? 0 : 1);
      if (tid == 0 && rb == 0) {
        if (begin == 0) p.shared[2 * n] = w;
        if (t == tiles - 1) p.shared[2 * n + 1] = w;
      }
      const int row0 = rb * MB + ln, col0 = wave * (MT * 16) + 4 * lg;
      __bf16* out = p.out + ((int64_t)n * p.rows + row0) * p.L + col0;
      float* part = p.part + ((int64_t)slot * MB + ln) * p.L + col0;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int row = row0 + j * 16;
        float sum = smax[0][j * 16 + ln];
#pragma unroll
        for (int g = 1; g < TG; ++g) sum += smax[g][j * 16 + ln];
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          if (row < p.rows && col0 + 16 * i < p.L) {
            const f32x4 o = acc[i][j] * inv;
            if (whole) {
              const bf16x4 ob = {(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
              *reinterpret_cast<bf16x4*>(out + 16 * i) = ob;
            } else {
              *reinterpret_cast<f32x4*>(part + 16 * i) = o;
            }
          }
          acc[i][j] = f32x4{0, 0, 0, 0};
        }
        out += 16 * p.L;
        part += 16 * p.L;
      }
      const int r = keep_here(tid);
      if (r < MB && rb * MB + r < p.rows) {
        float sum = smax[0][r];
#pragma unroll
        for (int g = 1; g < TG; ++g) sum += smax[g][r];
        if (!whole)
          p.psum[(int64_t)slot * MB + r] = make_float2(sfac[r], sum);
        else if (p.lse)
          p.lse[(int64_t)n * p.rows + rb * MB + r] = sum == 0.f ? -INFINITY : (sfac[r] + __log2f(sum)) * kLn2;
      }
      wait_loads<0>();  // the queries are there, and no load to LDS outlives the workgroup
      if (!more) return;
      m = -INFINITY;
      far = false;
      l = 0.f;
      begin = next.t;
    }
    cur = next;
  }
}

// Joins the pieces of a sequence that several workgroups share, and writes
// the outputs of empty sequences.  A wave takes one query row (8 columns a
// lane) and every ``parts``-th piece; grid: (groups of 8 / parts rows,
// sequences).  HBM-bound where there are many rows: 46 MB of pieces of 200
// sequences x 64 rows in 11.5 us, 51 MB in 13 us; a pass for the maxima before
// one for the outputs took 13 and 17.5.
__global__ __launch_bounds__(kThreads) void latent_join_kernel(DecodeParams p, int MB, int parts) {
  __shared__ f32x4 osum[kWaves][2][64];
  __shared__ float wtop[kWaves], wsum[kWaves];
  const int n = blockIdx.y, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int row = blockIdx.x * (kWaves / parts) + wave / parts, part = wave % parts, c = lane * 8;
  const bool have = row < p.rows;
  const int64_t at_out = ((int64_t)n * p.rows + row) * p.L + c;
  const int tokens = seq_tokens(p, n), w0 = p.shared[2 * n], w1 = p.shared[2 * n + 1];
  if (tokens == 0) {
    if (part != 0 || !have) return;
    if (c < p.L) *reinterpret_cast<u32x4*>(p.out + at_out) = u32x4{0, 0, 0, 0};
    if (p.lse && lane == 0) p.lse[(int64_t)n * p.rows + row] = -INFINITY;
    return;
  }
  if (w0 == w1) return;
  const int64_t at = ((int64_t)(row / MB) * 2 * p.groups) * MB + row % MB;
  // share w0 holds the sequence's beginning (slot 2 w0 + 1), the later ones
  // begin in mid-sequence (slot 2 w)
  auto slot = [&](int w) { return at + (int64_t)(2 * w + (w == w0 ? 1 : 0)) * MB; };
  // one pass with a running maximum, four pieces' loads at once
  float top = -INFINITY, sum = 0.f;
  f32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  if (have) {
    for (int first = w0 + part; first <= w1; first += 4 * parts) {
      float e[4], l[4];
      f32x4 x[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int w = first + u * parts;
        e[u] = -INFINITY;
        l[u] = 0.f;
        x[u][0] = x[u][1] = f32x4{0, 0, 0, 0};
        if (w > w1) continue;
        const int64_t s = slot(w);
        const float2 ml = p.psum[s];
        e[u] = ml.x;
        l[u] = ml.y;
        if (c < p.L) {
          x[u][0] = *reinterpret_cast<const f32x4*>(p.part + s * p.L + c);
          x[u][1] = *reinterpret_cast<const f32x4*>(p.part + s * p.L + c + 4);
        }
      }
      float mx = top;
#pragma unroll
      for (int u = 0; u < 4; ++u) mx = fmaxf(mx, e[u]);
      const float base = mx == -INFINITY ? 0.f : mx, old = exp2_hw(top - base);
      sum *= old;
      o[0] *= old;
      o[1] *= old;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = exp2_hw(e[u] - base) * l[u];
        sum += f;
        o[0] += f * x[u][0];
        o[1] += f * x[u][1];
      }
      top = mx;
    }
  }
  if (parts > 1) {  // (uniform over the workgroup)
    osum[wave][0][lane] = o[0];
    osum[wave][1][lane] = o[1];
    if (lane == 0) {
      wtop[wave] = top;
      wsum[wave] = sum;
    }
    __syncthreads();
    if (part == 0) {
      float mx = top;
      for (int i = 1; i < parts; ++i) mx = fmaxf(mx, wtop[wave + i]);
      const float base = mx == -INFINITY ? 0.f : mx, own = exp2_hw(top - base);
      sum *= own;
      o[0] *= own;
      o[1] *= own;
      for (int i = 1; i < parts; ++i) {
        const float f = exp2_hw(wtop[wave + i] - base);
        sum += f * wsum[wave + i];
        o[0] += f * osum[wave + i][0][lane];
        o[1] += f * osum[wave + i][1][lane];
      }
      top = mx;
    }
  }
  if (part != 0 || !have) return;
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  if (c < p.L) {
    bf16x8 ob;
#pragma unroll
    for (int i = 0; i < 8; ++i) ob[i] = (__bf16)(o[i >> 2][i & 3] * inv);
    *reinterpret_cast<bf16x8*>(p.out + at_out) = ob;
  }
  if (p.lse && lane == 0)
    p.lse[(int64_t)n * p.rows + row] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

struct Shape {
  int nb, row_blocks, groups;
};

// Query rows a workgroup (16, 32 or 64: 16 rows of 200 ragged sequences take 98
// us in workgroups of 16 and 112 of 64) and shares of the line: one workgroup a
// CU, 256 in all; the shares are a multiple of 8, one set an XCD.  (At L = 512
// the LDS holds no second one.  The builds for L <= 128, and for L <= 256
// without rotary columns, would leave room for it; that was not measured.)
Shape decode_shape(int64_t Q, int64_t H) {
  Shape s;
  const int64_t rows = Q * H;
  s.nb = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
  s.row_blocks = (int)((rows + 16 * s.nb - 1) / (16 * s.nb));
  const int g = 256 / s.row_blocks / 8 * 8;
  s.groups = g < 8 ? 8 : g;
  return s;
}

int64_t part_rows(const Shape& s) { return (int64_t)s.row_blocks * 2 * s.groups * 16 * s.nb; }

template <int LP, int RP, bool kPad>
hipError_t launch_nb(const DecodeParams& p, int nb, hipStream_t stream) {
  const dim3 grid((unsigned)(p.groups * p.row_blocks));
  switch (nb) {
    case 1:
      hipLaunchKernelGGL((latent_decode_kernel<LP, RP, 1, kPad>), grid, dim3(kThreads), 0, stream, p);
      break;
    case 2:
      hipLaunchKernelGGL((latent_decode_kernel<LP, RP, 2, kPad>), grid, dim3(kThreads), 0, stream, p);
      break;
    default:
      hipLaunchKernelGGL((latent_decode_kernel<LP, RP, 4, kPad>), grid, dim3(kThreads), 0, stream, p);
  }
  return hipGetLastError();
}

template <int LP>
hipError_t launch_r(const DecodeParams& p, int nb, hipStream_t stream) {
  if (p.R == 0) return p.L == LP ? launch_nb<LP, 0, false>(p, nb, stream) : launch_nb<LP, 0, true>(p, nb, stream);
  return p.L == LP && p.R == 64 ? launch_nb<LP, 64, false>(p, nb, stream) : launch_nb<LP, 64, true>(p, nb, stream);
}

}  // namespace

size_t latent_decode_workspace_bytes(int64_t N, int64_t Q, int64_t H, int64_t L) {
  return (size_t)(part_rows(decode_shape(Q, H)) * (L + 2) + 2 * N) * 4;
}

hipError_t launch_latent_decode(const kda_latent_decode_args_t& a, hipStream_t stream) {
  const Shape s = decode_shape(a.Q, a.H);
  DecodeParams p;
  p.cache = static_cast<const __bf16*>(a.cache);
  p.page_stride = a.page_stride;
  p.num_pages = (int)a.num_pages;
  p.page_size = (int)a.page_size;
  p.L = (int)a.L;
  p.R = (int)a.R;
  // j / d = j m >> (31 + s) with 2^s >= d and m = floor(2^(31+s) / d) + 1: m d
  // passes 2^(31+s) by at most d <= 2^s, too little to matter for j < 2^31
  int sh = 0;
  while ((1 << sh) < p.page_size) ++sh;
  p.page_shift = 31 + sh;
  p.page_mul = (uint32_t)(((uint64_t)1 << (31 + sh)) / (uint32_t)p.page_size + 1);
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
  p.part = static_cast<float*>(a.workspace);
  p.psum = reinterpret_cast<float2*>(p.part + part_rows(s) * a.L);
  p.shared = reinterpret_cast<int32_t*>(p.psum + part_rows(s));
  hipError_t e = a.L <= 128 ? launch_r<128>(p, s.nb, stream)
                            : (a.L <= 256 ? launch_r<256>(p, s.nb, stream) : launch_r<512>(p, s.nb, stream));
  if (e != hipSuccess) return e;
  // few rows: more waves share a row's pieces (one sequence of 4000 tokens, 32
  // rows: 19.5 us, a wave a row 31)
  int parts = kWaves;
  while (parts > 1 && (int64_t)p.rows * p.N * parts > 2048 * kWaves) parts >>= 1;
  const int per = kWaves / parts;
  hipLaunchKernelGGL(latent_join_kernel, dim3((unsigned)((p.rows + per - 1) / per), (unsigned)p.N), dim3(kThreads), 0,
                     stream, p, 16 * s.nb, parts);
  return hipGetLastError();
}

}  // namespace kda
