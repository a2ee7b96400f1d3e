// Absorbed latent attention over a paged cache, in 16 or in 8 bits, with the
// prefixes that sequences share computed once for all of them, for gfx950.
//
// The result is that of latent decode: query row (n, i, h) over the rows j <
// lengths[n] - (Q - 1 - i) of sequence n.  Softmax sums over disjoint sets of rows
// join exactly (each set's maximum, sum and output), so a sequence of a group is cut
// at the group's shared length: the query rows of all its sequences, which lie
// side by side in q, take the prefix together in blocks of MB rows, and each
// sequence's own go over its own rows.
//
// Work split.  The batch is a line of tiles of 64 tokens.  An entity is a group's prefix
// or a sequence's own tokens: T tiles for each of its row blocks.  It is cut into
// chunks of at least a workgroup's share, a chunk's tiles stand on the line for
// one row block after another, and workgroups get equal shares of the line, neighbours on one
// XCD: the row blocks of a chunk are computed at the same time behind one
// L2, which then serves all but the first.  What one workgroup computes of one
// chunk and row block, a piece, is written as output if it is all there is for
// its sequence, otherwise with its maximum and sum to the workspace, and
// the join kernel weighs the pieces of a row.  The plan is made on the device by one
// workgroup, so a captured call follows its lengths, groups and tables.
//
// Tile.  As in latent decode: 8 waves, 64 tokens, the scores of a row block and a
// group of tokens by a wave, the output's columns over the waves.  In 8 bits a
// tile is 40 KB and three stages fit.
#include <type_traits>

#include "internal.h"
#include "latent_tile.h"

namespace kda {
namespace {

using namespace latent;

constexpr int kShares = 256;       // workgroups, one a CU
constexpr int kPlanThreads = 1024;

struct Entity {
  int64_t base;            // place on the line
  int32_t tiles, row_blocks;
  int32_t chunks, chunk;   // and the tiles of one; the first ``longer`` ones have one more
  int32_t longer;
  int32_t row0, rows;      // query rows
  int32_t seq, t0, t1;     // tokens [t0, t1) of this sequence
  int32_t slot;            // of its first row block's pieces that no share cuts and that are not chunks
  int32_t group;           // of a sequence: the entity of its prefix, or -1

  __device__ __forceinline__ int chunk_begin(int k) const { return k * chunk + min(k, longer); }
  __device__ __forceinline__ int chunk_tiles(int k) const { return chunk + (k < longer ? 1 : 0); }
};

struct Start {  // where a workgroup begins: tile t of row block rb of chunk k of entity e
  int32_t left, w, e, k, rb, t;  // left: tiles of the share, 0: none
  Entity ent;
};

struct SharedParams {
  const char *lat, *rot, *scales;                // 16-bit cache: lat alone
  int64_t lat_page, rot_page, scales_page;       // bytes
  int lat_row;                                   // bytes from token to token
  int num_pages, page_size, L, R;
  uint32_t page_mul;
  int page_shift;
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
  const int32_t* lengths;
  const int32_t *cu, *shared;
  const __bf16* q;
  int64_t qs[3];
  const __bf16* qr;
  int64_t qrs[3];
  __bf16* out;
  float* lse;
  int N, Q, H, rows, G;                          // rows: Q H
  float scale2;                                  // scale log2 e
  float* part;                                   // [slots][MB][L] normalised outputs
  float2* psum;                                  // [slots][MB] the maxima and the sums against them
  Entity* ents;                                  // [G + N]
  Start* starts;                                 // [kShares], by workgroup
  int64_t* total;                                // tiles on the line
  int32_t *bounds, *prefix;                      // [G + 1] the groups' sequences, [G] their shared tokens
};

__device__ __forceinline__ int seq_tokens(const SharedParams& p, int n) {
  const int len = p.lengths[n];
  const int64_t room = (int64_t)p.max_pages * p.page_size;
  return len < 0 ? 0 : (len > room ? (int)room : len);
}

// The line in equal shares, none empty (fewer of them where there are fewer tiles).
struct Shares {
  int64_t quot, rem, count;
};
__device__ __forceinline__ Shares shares_of(int64_t total) {
  Shares s;
  s.count = total < kShares ? total : kShares;
  s.quot = total < kShares ? 1 : total / kShares;
  s.rem = total < kShares ? 0 : total % kShares;
  return s;
}
__device__ __forceinline__ int64_t share_begin(const Shares& s, int64_t w) { return w * s.quot + (w < s.rem ? w : s.rem); }
// the share that holds tile x
__device__ __forceinline__ int share_at(const Shares& s, int64_t x) {
  const int64_t longer = s.rem * (s.quot + 1);
  if ((uint64_t)(x | s.quot) < 0x7fffffffu) {
    const unsigned q = (unsigned)s.quot;
    return x < longer ? (int)((unsigned)x / (q + 1)) : (int)s.rem + (int)((unsigned)(x - longer) / q);
  }
  return x < longer ? (int)(x / (s.quot + 1)) : (int)(s.rem + (x - longer) / s.quot);
}

// Sums (inclusive) over the workgroup of the threads before and with this one;
// *all: over all.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* wsum, T* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  if (lane == 63) wsum[wave] = x;
  __syncthreads();
  T before = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 64; ++i) {
    const T v = wsum[i];
    before += i < wave ? v : 0;
    sum += v;
  }
  __syncthreads();
  *all = sum;
  return x + before;
}

__global__ __launch_bounds__(kPlanThreads) void shared_plan_kernel(SharedParams p, int MB) {
  __shared__ long long lsum[kPlanThreads / 64];
  __shared__ int isum[kPlanThreads / 64];
  const int own_blocks = (p.rows + MB - 1) / MB;
  const int tid = threadIdx.x, E = p.G + p.N;
  // the groups' bounds: inside the batch, and not before an earlier one
  if (p.G > 0) {
    int carry = 0;
    for (int i0 = 0; i0 <= p.G; i0 += kPlanThreads) {
      const int i = i0 + tid, lane = tid & 63, wave = tid >> 6;
      int v = 0;
      if (i <= p.G) {
        v = p.cu[i];
        v = v < 0 ? 0 : (v > p.N ? p.N : v);
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) v = max(v, __shfl_up(v, d, 64));
      if (lane == 63) isum[wave] = v;
      __syncthreads();
      int most = carry;
      for (int k = 0; k < kPlanThreads / 64; ++k) {
        if (k < wave) v = max(v, isum[k]);
        most = max(most, isum[k]);
      }
      v = max(v, carry);
      carry = most;
      __syncthreads();
      if (i <= p.G) p.bounds[i] = v;
    }
    __syncthreads();
    for (int g = tid; g < p.G; g += kPlanThreads) {
      const int n0 = p.bounds[g], n1 = p.bounds[g + 1];
      int pre = 0;
      if (n1 - n0 >= 2) {
        const int len = seq_tokens(p, n0), s = p.shared[g];
        pre = s < 0 ? 0 : (s > len ? len : s);
      }
      p.prefix[g] = pre;
    }
    __syncthreads();
  }
  // the entities, and the length of the line
  long long total = 0;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    const int e = e0 + tid;
    long long mine = 0;
    if (e < E) {
      Entity x;
      x.group = -1;
      if (e < p.G) {
        const int n0 = p.bounds[e], n1 = p.bounds[e + 1];
        x.row0 = n0 * p.rows;
        x.rows = (n1 - n0) * p.rows;
        x.seq = n0;
        x.t0 = 0;
        x.t1 = p.prefix[e];
        x.slot = 2 * kShares + p.N * own_blocks + x.row0 / MB + e;  // (an earlier group's are fewer)
      } else {
        const int n = e - p.G;
        x.row0 = n * p.rows;
        x.rows = p.rows;
        x.seq = n;
        x.t0 = 0;
        x.t1 = seq_tokens(p, n);
        x.slot = 2 * kShares + n * own_blocks;
        if (p.G > 0 && n >= p.bounds[0] && n < p.bounds[p.G]) {
          int lo = 0, hi = p.G;  // the last group that begins at n or before
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.bounds[mid] <= n) lo = mid; else hi = mid;
          }
          x.t0 = min(p.prefix[lo], x.t1);
          if (x.t0 > 0) x.group = lo;
        }
      }
      x.tiles = (int)(((int64_t)x.t1 - x.t0 + kTile - 1) / kTile);
      x.row_blocks = (x.rows + MB - 1) / MB;
      mine = (long long)x.tiles * x.row_blocks;
      p.ents[e] = x;
    }
    long long all;
    block_scan(mine, lsum, &all);
    total += all;
  }
  const Shares sh = shares_of(total);
  const int share = sh.quot > (1 << 30) ? 1 << 30 : (int)sh.quot;
  long long base = 0;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    const int e = e0 + tid;
    int tiles = 0, blocks = 0;
    if (e < E) {
      tiles = p.ents[e].tiles;
      blocks = p.ents[e].row_blocks;
    }
    const long long mine = (long long)tiles * blocks;
    long long all;
    const long long to = base + block_scan(mine, lsum, &all);
    if (e < E) {
      const int chunks = mine == 0 ? 0 : max(1, tiles / share);
      p.ents[e].base = to - mine;
      p.ents[e].chunks = chunks;
      p.ents[e].chunk = chunks > 0 ? tiles / chunks : 1;
      p.ents[e].longer = chunks > 0 ? tiles % chunks : 0;
    }
    base += all;
  }
  if (tid == 0) *p.total = total;
  __syncthreads();
  if (tid < kShares) {
    const int per = (int)((sh.count + 7) / 8), w = (tid & 7) * per + (tid >> 3);
    Start s = {};
    if ((tid >> 3) < per && w < sh.count) {
      const int64_t at = share_begin(sh, w);
      int lo = 0, hi = E;  // the last entity that begins there or before: it holds the tile, if empty ones at its
      while (hi - lo > 1) {  // place are before it
        const int mid = (lo + hi) >> 1;
        if (p.ents[mid].base <= at) lo = mid; else hi = mid;
      }
      s.ent = p.ents[lo];
      s.e = lo;
      s.w = w;
      s.left = (int)(share_begin(sh, w + 1) - at);
      const int64_t in = at - s.ent.base;
      const int y = (int)(in / s.ent.row_blocks), longer = s.ent.longer * (s.ent.chunk + 1);
      s.k = y < longer ? y / (s.ent.chunk + 1) : s.ent.longer + (y - longer) / s.ent.chunk;
      const int64_t rest = in - (int64_t)s.ent.chunk_begin(s.k) * s.ent.row_blocks;
      s.rb = (int)(rest / s.ent.chunk_tiles(s.k));
      s.t = (int)(rest - (int64_t)s.rb * s.ent.chunk_tiles(s.k));
    }
    p.starts[tid] = s;
  }
}

// Which tile, of which unit; the records are in scalar registers.
struct Tile {
  int seq, pos, end;        // tokens pos .. of this sequence, before end
  int row0, rows, slot;     // query rows, and the unit's own place in the workspace
  int flags;
  unsigned long long live;  // which rows are there
};
// tile of its unit; the unit is all there is of its entity for its rows; and of its sequence
constexpr int kFirst = 1, kLast = 2, kSingle = 4, kAlone = 8;

struct Walk {
  Entity x;
  int e, k, rb, t, tc;
};

template <typename T>
__device__ __forceinline__ T scalar_load(const T* at) {
  static_assert(sizeof(T) % 4 == 0, "");
  typedef const __attribute__((address_space(4))) int* Words;
  const Words w = (Words)(uintptr_t)at;
  int v[sizeof(T) / 4];
#pragma unroll
  for (unsigned i = 0; i < sizeof(T) / 4; ++i) v[i] = w[i];
  T r;
  __builtin_memcpy(&r, v, sizeof(T));
  return r;
}

template <bool F8, int LP, int RP, int NB, bool kPad>
struct Kind {
  typedef Bf16Tile<LP, RP, NB, kPad, true> D;
  static constexpr int kStages = 2, kStageBytes = D::kStage * 2;
};
template <int LP, int RP, int NB, bool kPad>
struct Kind<true, LP, RP, NB, kPad> {
  typedef Fp8Tile<LP, RP, NB, kPad> D;
  static constexpr int kStages = 3, kStageBytes = D::kStage;
};

template <bool F8, int LP, int RP, int NB, bool kPad>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void latent_shared_kernel(SharedParams p) {
  using K = Kind<F8, LP, RP, NB, kPad>;
  using D = typename K::D;
  constexpr int MB = D::MB, KS = D::KS, MT = D::MT, TG = D::TG, TB = D::TB, NS = K::kStages;
  constexpr unsigned kStageBytes = K::kStageBytes, kRotaryBytes = RP > 0 ? kTile * RP * 2 : 16;
  __shared__ __attribute__((aligned(16))) char stage[NS][kStageBytes];
  __shared__ __attribute__((aligned(16))) char rotary[NS][kRotaryBytes];
  __shared__ __attribute__((aligned(16))) float tscale[NS][F8 ? kTile : 4];
  __shared__ __attribute__((aligned(16))) __bf16 prob[MB * kTile];
  __shared__ float smax[TG][MB];  // of a tile; at a piece's end the sums
  __shared__ float sfac[MB];      // factor of the older output; at a piece's end the maxima
  __shared__ int32_t pages[2][kWaves][64];  // page of token lane of the tile located next
  __shared__ int grown[2];        // whether a row's maximum has grown much in this tile

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const Start start = scalar_load(p.starts + blockIdx.x);
  if (start.left == 0) return;
  if (tid < 2) grown[tid] = 0;
  if (kPad) {
    u32x4 *st = reinterpret_cast<u32x4*>(stage), *ro = reinterpret_cast<u32x4*>(rotary);
    for (unsigned i = tid; i < sizeof(stage) / 16; i += kThreads) st[i] = u32x4{0, 0, 0, 0};
    for (unsigned i = tid; i < sizeof(rotary) / 16; i += kThreads) ro[i] = u32x4{0, 0, 0, 0};
  }
  const bool scoring = wave < D::kScoring;
  const int rblock = wave % NB;     // query rows this wave scores
  const int tg = (wave / NB) % TG;  // and tokens
  __syncthreads();

  // ---- the tiles of the share, one after another
  Walk walk;
  walk.x = start.ent;
  walk.e = start.e;
  walk.k = start.k;
  walk.rb = start.rb;
  walk.t = start.t;
  walk.tc = walk.x.chunk_tiles(walk.k);
  auto here = [&]() {
    Tile x;
    x.seq = walk.x.seq;
    x.pos = walk.x.t0 + (walk.x.chunk_begin(walk.k) + walk.t) * kTile;
    x.end = walk.x.t1;
    x.row0 = walk.x.row0 + walk.rb * MB;
    x.rows = min(MB, walk.x.rows - walk.rb * MB);
    x.slot = walk.x.slot + walk.rb;
    x.flags = (walk.t == 0 ? kFirst : 0) | (walk.t == walk.tc - 1 ? kLast : 0) |
              (walk.x.chunks == 1 ? kSingle : 0) | (walk.x.chunks == 1 && walk.e >= p.G && walk.x.t0 == 0 ? kAlone : 0);
    x.live = 0;
    return x;
  };
  auto follow = [&]() {  // (there is a next tile)
    if (++walk.t < walk.tc) return;
    walk.t = 0;
    if (++walk.rb < walk.x.row_blocks) return;
    walk.rb = 0;
    if (++walk.k == walk.x.chunks) {
      walk.k = 0;
      do walk.x = scalar_load(p.ents + ++walk.e);
      while (walk.x.chunks == 0);
    }
    walk.tc = walk.x.chunk_tiles(walk.k);
  };

  // where the page of token pos + lane of a tile is (the last one's for lanes
  // behind the end), and that row's place; -1: no such row
  auto page_of = [&](int pos) { return (unsigned)(((uint64_t)(unsigned)pos * p.page_mul) >> p.page_shift); };
  auto lookup = [&](const Tile& x) {
    const int pos = x.pos + lane;
    return p.table + x.seq * p.table_stride + page_of(pos < x.end ? pos : x.end - 1);
  };
  const char *at, *rot_at, *scale_at;  // rows of the last tile located (lane i: token i)
  // Rows that are not there are fetched from the first one that is (their
  // weights are 0); a tile without any is not fetched and not computed.
  auto locate = [&](int page, Tile& x) {
    const int pos = x.pos + lane;
    const bool there = pos < x.end && (unsigned)page < (unsigned)p.num_pages;
    int off = pos - (int)page_of(pos) * p.page_size;
    x.live = __ballot(there);
    if (x.live != ~0ull) {
      const int some = x.live != 0 ? __ffsll(x.live) - 1 : 0;
      const int spage = x.live != 0 ? __builtin_amdgcn_readlane(page, some) : 0;
      const int soff = x.live != 0 ? __builtin_amdgcn_readlane(off, some) : 0;
      page = there ? page : spage;
      off = there ? off : soff;
    }
    at = p.lat + page * p.lat_page + (int64_t)off * p.lat_row;
    if (F8) {
      scale_at = p.scales + page * p.scales_page + (int64_t)off * 4;
      if (RP > 0) rot_at = p.rot + page * p.rot_page + (int64_t)off * (2 * p.R);
    }
  };
  const unsigned stage_at = lds_offset(stage), rotary_at = lds_offset(rotary), scale_lds = lds_offset(tscale);
  const unsigned pages_at = lds_offset(pages[0][wave]);
  constexpr unsigned kPagesBytes = sizeof(pages[0]), kScaleBytes = sizeof(tscale[0]);
  const typename D::Columns columns = D::columns(p.L, p.R, wave, lane);

  // ---- queries
  typedef bf16x8 Q16[F8 ? 1 : KS];
  Q16 qf;
  int sees = 0;  // tokens that row ln of the wave's block sees
  struct QueryAt {
    const __bf16 *q, *qr;
  };
  auto row_at = [&](const Tile& x) {
    // (rows behind the unit's last one get its first one's queries; they are not written)
    const int r = keep_here(rblock * 16 + ln);
    const unsigned row = x.row0 + (r < x.rows ? r : 0);
    const unsigned n = row / (unsigned)p.rows, in = row - n * p.rows, qi = in / (unsigned)p.H, h = in - qi * p.H;
    sees = seq_tokens(p, (int)n) - (p.Q - 1 - (int)qi);
    return QueryAt{p.q + n * p.qs[0] + qi * p.qs[1] + h * p.qs[2], p.qr + n * p.qrs[0] + qi * p.qrs[1] + h * p.qrs[2]};
  };
  auto load_q16 = [&](const Tile& x) {
    const QueryAt a = row_at(x);
    const int lg8 = 8 * keep_here(lane >> 4);
#pragma unroll
    for (int k = 0; k < (F8 ? 0 : KS); ++k) {
      const int c = 32 * k + lg8;
      bf16x8 y = {};
      if (!kPad || (k < LP / 32 ? c < p.L : c - LP < p.R))
        y = *reinterpret_cast<const bf16x8*>(k < LP / 32 ? a.q + c : a.qr + (c - LP));
      qf[k] = y;
    }
  };

  int left = start.left - 1;  // tiles behind the one computed
  int ahead = left;           // and behind the last one asked for
  Tile ring[NS];              // the one computed, and those under way
  Tile ask;
  auto ask_next = [&](int to) {
    follow();
    ask = here();
    load_lds4(lookup(ask), uniform(pages_at + to * kPagesBytes));
    --ahead;
  };
  [[maybe_unused]] auto fetch16 = [&](int i, int to) {
    if constexpr (!F8) D::fetch(i, at, wave, lane, columns, stage_at + to * kStageBytes);
  };
  auto fetch_all = [&](int to) {
    if constexpr (F8) {
      D::fetch(at, rot_at, scale_at, wave, lane, columns, stage_at + to * kStageBytes,
               rotary_at + to * kRotaryBytes, scale_lds + to * kScaleBytes);
    } else {
      D::fetch_rotary(at, wave, lane, columns, rotary_at + to * kRotaryBytes);
#pragma unroll
      for (int i = 0; i < D::kLat; ++i) D::fetch(i, at, wave, lane, columns, stage_at + to * kStageBytes);
    }
  };
  ring[0] = here();
  const int page0 = *lookup(ring[0]);
  int page1 = 0;
  if (NS == 3 && ahead > 0) {
    follow();
    ring[1] = here();
    --ahead;
    page1 = *lookup(ring[1]);
  }
  if (ahead > 0) ask_next(0);
  locate(page0, ring[0]);
  if (ring[0].live) fetch_all(0);
  if (NS == 3 && left > 0) {
    locate(page1, ring[1]);
    if (ring[1].live) fetch_all(1);
  }

  typedef typename std::conditional<F8, Fp8Tile<LP, RP, NB, kPad>, Fp8Tile<128, RP, NB, kPad>>::type F;
  typename F::Query q8;
  // (after the output has left its registers)
  [[maybe_unused]] auto load_q8 = [&](const Tile& x) {
    const QueryAt a = row_at(x);
    typename F::Raw raw;
    F::request(a.q, a.qr, p.L, p.R, keep_here(lane >> 4), raw);
    F::split(raw, q8);
  };
  if constexpr (F8)
    load_q8(ring[0]);
  else
    load_q16(ring[0]);
  bool begun = ring[0].flags & kFirst;  // whether the piece begins where its unit does
  int later = 0;                        // 1: behind the share's first piece

  float m, l;  // of row ln of the wave's block, over its tokens; units of scale2 s
  bool far;    // whether one of the wave's rows is_far
  f32x4 acc[MT][NB];
  auto clear = [&]() {
    m = -INFINITY;
    l = 0.f;
    far = false;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  };
  clear();

  int st = 0;  // the stage of the tile computed
  for (int par = 0;; par ^= 1) {
    // this tile has landed (in 8 bits the next one's loads may be under way, and
    // the lookup before them is done), and the readers of the one before are done
    if constexpr (F8) {
      if (left > 0 && ring[1].live)
        wait_loads<D::kLoads>();
      else
        wait_loads<0>();
    } else {
      wait_loads<0>();
    }
    lds_barrier();
    Tile& cur = ring[0];
    const bool more = left > 0;          // a tile behind this one
    const bool asked = left > NS - 2;    // and the one located now
    const int to = st == 0 ? NS - 1 : st - 1;  // its stage: the one before
    bool fetches = false;
    if (asked) {
      ring[NS - 1] = ask;
      locate(pages[par][wave][lane], ring[NS - 1]);
      if (ahead > 0) ask_next(par ^ 1);
      fetches = ring[NS - 1].live != 0;
    }
    if (tid == 0) grown[par ^ 1] = 0;
    if constexpr (F8) {
      if (fetches) fetch_all(to);
    } else {
      if (fetches) D::fetch_rotary(at, wave, lane, columns, rotary_at + to * kRotaryBytes);
      if (fetches && !(scoring && cur.live)) {
#pragma unroll
        for (int i = 0; i < D::kLat; ++i) fetch16(i, to);
      }
    }
    if (cur.live) {
      float sum = 0.f, fac = 1.f;
      f32x4 s[TB], sc[TB];
      // Weights of the scores against the maximum in use, for the matrix unit
      // in bf16; their sum stays in fp32.  In 8 bits the tokens' scales go into them
      // before they are rounded.
      auto weigh = [&](float base) {
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < TB; ++j) {
          bf16x4 pb;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = exp2_hw(fmaf(s[j][i], p.scale2, -base));
            sum += e;
            pb[i] = (__bf16)(F8 ? e * sc[j][i] : e);
          }
          const int tk = 16 * (TB * tg + j) + 4 * lg;
          *reinterpret_cast<bf16x4*>(prob + (rblock * 16 + ln) * kTile + (((tk >> 3) ^ (ln & 7)) << 3) + (tk & 7)) = pb;
        }
      };
      if (scoring) {
        const char* lat = stage[0] + st * kStageBytes;
        const __bf16* rot = reinterpret_cast<const __bf16*>(rotary[0] + st * kRotaryBytes);
        if constexpr (F8) {
          D::scores(lat + 16 * TB * tg * LP, rot + 16 * TB * tg * RP, tscale[st] + 16 * TB * tg, q8, ln, lg, s, sc);
        } else {
          D::scores(reinterpret_cast<const __bf16*>(lat) + (16 * TB * tg + ln) * LP, rot + (16 * TB * tg + ln) * RP, qf,
                    ln, lg, s, [&](int i) {
                      if (fetches) fetch16(i, to);
                    });
        }
        if (cur.live != ~0ull || __any(cur.pos + kTile > sees)) {
#pragma unroll
          for (int j = 0; j < TB; ++j) {
            // of the lane's four tokens: how many are seen, and which are there
            const int at4 = 16 * (TB * tg + j) + 4 * lg, n = sees - cur.pos - at4;
            const unsigned there = (unsigned)(cur.live >> at4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i >= n || !(there >> i & 1)) {
                s[j][i] = -INFINITY;
                if (F8) sc[j][i] = 0.f;  // (it may be NaN)
              }
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
        // more than 8 (a factor of 256), as in latent decode.
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
      if constexpr (F8)
        D::values(stage[0] + st * kStageBytes, prob, wave, ln, lg, acc);
      else
        D::values(reinterpret_cast<const __bf16*>(stage[0] + st * kStageBytes), prob, wave, ln, lg, acc);
    }

    if (!more || (cur.flags & kLast)) {
      // ---- the end of a piece
      if constexpr (!F8) {
        if (more) load_q16(ring[1]);
      }
      l = sum_halves(sum_quarters(l));
      lds_barrier();
      const int ln = keep_here(lane & 15), lg = keep_here(lane >> 4);
      if (scoring && lg == 0) {
        smax[tg][rblock * 16 + ln] = l;
        if (tg == 0) sfac[rblock * 16 + ln] = m;
      }
      lds_barrier();
      const bool whole = begun && (cur.flags & kLast), direct = whole && (cur.flags & kAlone);
      const int64_t slot = whole && (cur.flags & kSingle) ? cur.slot : 2 * start.w + later;
      const int col0 = wave * (MT * 16) + 4 * lg;
      __bf16* out = p.out + ((int64_t)cur.row0 + ln) * p.L + col0;
      float* part = p.part + (slot * MB + ln) * p.L + col0;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        float sum = smax[0][j * 16 + ln];
#pragma unroll
        for (int g = 1; g < TG; ++g) sum += smax[g][j * 16 + ln];
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          if (j * 16 + ln < cur.rows && col0 + 16 * i < p.L) {
            const f32x4 o = acc[i][j] * inv;
            if (direct) {
              const bf16x4 ob = {(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
              *reinterpret_cast<bf16x4*>(out + 16 * i) = ob;
            } else {
              *reinterpret_cast<f32x4*>(part + 16 * i) = o;
            }
          }
        }
        out += 16 * p.L;
        part += 16 * p.L;
      }
      const int r = keep_here(tid);
      if (r < cur.rows) {
        float sum = smax[0][r];
#pragma unroll
        for (int g = 1; g < TG; ++g) sum += smax[g][r];
        if (!direct)
          p.psum[slot * MB + r] = make_float2(sfac[r], sum);
        else if (p.lse)
          p.lse[(int64_t)cur.row0 + r] = sum == 0.f ? -INFINITY : (sfac[r] + __log2f(sum)) * kLn2;
      }
      if (!more) {
        wait_loads<0>();  // no load to LDS outlives the workgroup
        return;
      }
      if constexpr (F8) load_q8(ring[1]);
      clear();
      begun = true;
      later = 1;
    }
#pragma unroll
    for (int i = 0; i + 1 < NS; ++i) ring[i] = ring[i + 1];
    st = st == NS - 1 ? 0 : st + 1;
    --left;
  }
}

// Joins the pieces of a query row, its prefix's and its own, and writes the outputs of
// empty sequences.  A wave takes one query row (8 columns a lane) and every
// ``parts``-th chunk; grid: (groups of 8 / parts rows, sequences).
__global__ __launch_bounds__(kThreads) void shared_join_kernel(SharedParams p, int MB, int parts) {
  __shared__ f32x4 osum[kWaves][2][64];
  __shared__ float wtop[kWaves], wsum[kWaves];
  const int n = blockIdx.y, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int row = blockIdx.x * (kWaves / parts) + wave / parts, part = wave % parts, c = lane * 8;
  const bool have = row < p.rows;
  const int64_t grow = (int64_t)n * p.rows + row, at_out = grow * p.L + c;
  const Entity own = scalar_load(p.ents + p.G + n);
  if (own.t1 == 0) {
    if (part != 0 || !have) return;
    if (c < p.L) *reinterpret_cast<u32x4*>(p.out + at_out) = u32x4{0, 0, 0, 0};
    if (p.lse && lane == 0) p.lse[grow] = -INFINITY;
    return;
  }
  const Shares sh = shares_of(scalar_load(p.total));
  // a sequence that one piece holds whole has its output
  if (own.t0 == 0 && own.chunks == 1) {
    const int rb = (blockIdx.x * (kWaves / parts)) / MB;  // (that of all the workgroup's rows)
    const int64_t a = own.base + (int64_t)rb * own.tiles;
    if (share_at(sh, a) == share_at(sh, a + own.tiles - 1)) return;
  }
  float top = -INFINITY, sum = 0.f;
  f32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  auto join = [&](const Entity& x) {
    const int in = (int)(grow - x.row0), rb = in / MB, r = in - rb * MB;
    for (int k0 = 0; k0 < x.chunks; k0 += 64 * parts) {
      // lane i: the shares of the row block in chunk k0 + part + i parts
      const int mine = k0 + part + lane * parts;
      const bool there = mine < x.chunks;
      const int tc = x.chunk_tiles(mine);
      const int64_t a = x.base + (int64_t)x.chunk_begin(mine) * x.row_blocks + (int64_t)rb * tc;
      const int w0 = there ? share_at(sh, a) : 0, w1 = there ? share_at(sh, a + tc - 1) : 0;
      // the pieces' places: the whole unit's own, or 2 w (+ 1 where others are before it in share w)
      const int inside = there && a != share_begin(sh, w0) ? 1 : 0;
      const int one = w0 == w1 && x.chunks == 1 ? x.slot + rb : 2 * w0 + inside;
      const int here = min(64, (x.chunks - k0 - part + parts - 1) / parts);
      for (int i = 0; i < here; i += 2) {
        // two chunks at a time; one has at most three pieces, as it is at most two shares long
        float e[6], s[6];
        f32x4 v[6][2];
#pragma unroll
        for (int u = 0; u < 6; ++u) {
          const int j = i + u / 3;
          e[u] = -INFINITY;
          s[u] = 0.f;
          v[u][0] = v[u][1] = f32x4{0, 0, 0, 0};
          if (j >= here) continue;
          const int first = __builtin_amdgcn_readlane(w0, j), last = __builtin_amdgcn_readlane(w1, j);
          const int w = first + u % 3;
          if (w > last) continue;
          const int64_t slot = w == first ? __builtin_amdgcn_readlane(one, j) : 2 * w;
          const float2 ml = p.psum[slot * MB + r];
          e[u] = ml.x;
          s[u] = ml.y;
          if (c < p.L) {
            const float* at = p.part + (slot * MB + r) * p.L + c;
            v[u][0] = *reinterpret_cast<const f32x4*>(at);
            v[u][1] = *reinterpret_cast<const f32x4*>(at + 4);
          }
        }
        float mx = top;
#pragma unroll
        for (int u = 0; u < 6; ++u) mx = fmaxf(mx, e[u]);
        const float base = mx == -INFINITY ? 0.f : mx, old = exp2_hw(top - base);
        sum *= old;
        o[0] *= old;
        o[1] *= old;
#pragma unroll
        for (int u = 0; u < 6; ++u) {
          const float f = exp2_hw(e[u] - base) * s[u];
          sum += f;
          o[0] += f * v[u][0];
          o[1] += f * v[u][1];
        }
        top = mx;
      }
    }
  };
  if (have) {
    if (own.group >= 0) join(scalar_load(p.ents + own.group));
    if (own.chunks > 0) join(own);
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
      const float base = mx == -INFINITY ? 0.f : mx, first = exp2_hw(top - base);
      sum *= first;
      o[0] *= first;
      o[1] *= first;
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
  if (p.lse && lane == 0) p.lse[grow] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

// Blocks of 16 query rows a workgroup takes at once.
int blocks_of(int64_t N, int64_t Q, int64_t H, int64_t G) {
  const int64_t rows = G > 0 ? N * Q * H : Q * H;
  return rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
}

// Pieces in the workspace.  Two a share: of those that it begins with and of those
// behind, at most one is cut or a chunk (a chunk has a share's tiles at least, a share
// one more at most).  With groups, also one for each row block of each
// entity, for units that are whole.
int64_t slots_of(int64_t N, int64_t Q, int64_t H, int64_t G) {
  const int64_t mb = 16 * blocks_of(N, Q, H, G), rows = Q * H;
  return 2 * kShares + (G == 0 ? 0 : N * ((rows + mb - 1) / mb) + N * rows / mb + G + 1);
}

size_t round16(size_t x) { return (x + 15) & ~(size_t)15; }

template <bool F8, int LP, int RP, bool kPad>
hipError_t launch_nb(const SharedParams& p, int nb, hipStream_t stream) {
  const dim3 grid(kShares), block(kThreads);
  switch (nb) {
    case 1:
      hipLaunchKernelGGL((latent_shared_kernel<F8, LP, RP, 1, kPad>), grid, block, 0, stream, p);
      break;
    case 2:
      hipLaunchKernelGGL((latent_shared_kernel<F8, LP, RP, 2, kPad>), grid, block, 0, stream, p);
      break;
    default:
      hipLaunchKernelGGL((latent_shared_kernel<F8, LP, RP, 4, kPad>), grid, block, 0, stream, p);
  }
  return hipGetLastError();
}

template <bool F8, int LP>
hipError_t launch_r(const SharedParams& p, int nb, hipStream_t stream) {
  if (p.R == 0) return p.L == LP ? launch_nb<F8, LP, 0, false>(p, nb, stream) : launch_nb<F8, LP, 0, true>(p, nb, stream);
  return p.L == LP && p.R == 64 ? launch_nb<F8, LP, 64, false>(p, nb, stream) : launch_nb<F8, LP, 64, true>(p, nb, stream);
}

template <bool F8>
hipError_t launch_l(const SharedParams& p, int nb, hipStream_t stream) {
  if (p.L <= 128) return launch_r<F8, 128>(p, nb, stream);
  return p.L <= 256 ? launch_r<F8, 256>(p, nb, stream) : launch_r<F8, 512>(p, nb, stream);
}

}  // namespace

size_t latent_shared_workspace_bytes(int64_t N, int64_t Q, int64_t H, int64_t L, int64_t G) {
  const size_t rows = (size_t)slots_of(N, Q, H, G) * 16 * blocks_of(N, Q, H, G);
  return round16(rows * (size_t)L * 4) + round16(rows * 8) + (size_t)(G + N) * sizeof(Entity) + kShares * sizeof(Start) +
         16 + (size_t)(2 * G + 1) * 4;
}

hipError_t launch_latent_shared(const kda_latent_shared_args_t& a, hipStream_t stream) {
  const int nb = blocks_of(a.N, a.Q, a.H, a.G), MB = 16 * nb;
  const bool f8 = a.cache_dtype == KDA_E4M3;
  SharedParams p = {};
  p.lat = static_cast<const char*>(a.cache);
  p.lat_page = a.page_stride * (f8 ? 1 : 2);
  p.lat_row = (int)(f8 ? a.L : 2 * (a.L + a.R));
  if (f8) {
    p.scales = reinterpret_cast<const char*>(a.scales);
    p.scales_page = a.scales_page_stride * 4;
    p.rot = static_cast<const char*>(a.rope);
    p.rot_page = a.rope_page_stride * 2;
  }
  p.num_pages = (int)a.num_pages;
  p.page_size = (int)a.page_size;
  p.L = (int)a.L;
  p.R = (int)a.R;
  page_divisor(p.page_size, &p.page_mul, &p.page_shift);
  p.table = a.page_table;
  p.table_stride = a.table_stride;
  p.max_pages = (int)a.max_pages;
  p.lengths = a.lengths;
  p.cu = a.cu_groups;
  p.shared = a.shared;
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
  p.G = (int)a.G;
  p.scale2 = a.scale * kLog2e;
  const size_t rows = (size_t)slots_of(a.N, a.Q, a.H, a.G) * MB;
  char* ws = static_cast<char*>(a.workspace);
  p.part = reinterpret_cast<float*>(ws);
  ws += round16(rows * (size_t)a.L * 4);
  p.psum = reinterpret_cast<float2*>(ws);
  ws += round16(rows * 8);
  p.ents = reinterpret_cast<Entity*>(ws);
  ws += (size_t)(a.G + a.N) * sizeof(Entity);
  p.starts = reinterpret_cast<Start*>(ws);
  ws += kShares * sizeof(Start);
  p.total = reinterpret_cast<int64_t*>(ws);
  p.bounds = reinterpret_cast<int32_t*>(ws + 16);
  p.prefix = p.bounds + a.G + 1;
  hipLaunchKernelGGL(shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p, MB);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = f8 ? launch_l<true>(p, nb, stream) : launch_l<false>(p, nb, stream);
  if (e != hipSuccess) return e;
  // few rows: more waves share a row's pieces
  int parts = kWaves;
  while (parts > 1 && (int64_t)p.rows * p.N * parts > 2048 * kWaves) parts >>= 1;
  const int per = kWaves / parts;
  hipLaunchKernelGGL(shared_join_kernel, dim3((unsigned)((p.rows + per - 1) / per), (unsigned)p.N), dim3(kThreads), 0,
                     stream, p, MB, parts);
  return hipGetLastError();
}

}  // namespace kda
