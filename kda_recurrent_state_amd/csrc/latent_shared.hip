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
// or a sequence's own tokens: T tiles for each of its row blocks.  As many workgroups as a
// sequence has row blocks are a team, which goes over the line together, a row block each, so
// that a tile comes out of HBM once for all of them (64 x 16000 tokens, 128 rows: 650 MB are
// read, without teams 1230); a prefix has row blocks for many teams.  Teams get equal shares of the
// line, neighbours on one XCD.  An entity with row blocks for several teams is
// cut into chunks of at least a share, and a chunk's tiles stand on the line for
// one team's row blocks after another: these are then computed at about the same time, and the
// L2 serves some of the tiles.  A unit (a team's row blocks of a chunk) ends with
// queries to load and outputs to write, kEnd tiles' time; entities of one chunk, of which a
// share can hold many, have that much room on the line before each unit.  What one
// workgroup computes of one unit, a piece, is written as output if it is all there is for
// its sequence, otherwise with its maximum and sum to the workspace, and
// the join kernel weighs the pieces of a row.  The plan is made on the device by one
// workgroup, so a captured call follows its lengths, groups and tables.
//
// Tile.  As in latent decode: 8 waves, 64 tokens, the scores of a row block and a
// group of tokens by a wave, the output's columns over the waves.  In 8 bits a
// tile is 40 KB and three stages fit.
//
// What bounds it: the phases of a tile, which follow one another within the CU's
// one workgroup.  64 sequences of 12000 to 20000 tokens with 128 heads, 512 + 64
// components, take 385 us in 8 bits (660 MB, 131 us at a copy's rate; products 204 us at a large
// matrix product's); a tile of 64 rows takes 2.8 us, the matrix unit is busy for a third of
// it, and without its fetches, scores, softmax or output product the call is 75, 90, 40 or
// 72 us shorter.  40 sequences of 256 query rows behind 16384 shared tokens: 430 us in 16
// bits, 505 in 8 (products 273), where decode that reads the prefix for each sequence computes
// the same and reads 40 times as much, which at so many query rows takes no longer (426 and 493).  64
// sequences of 16 rows behind 32768 tokens take 130 us, and 221 without sharing.  The plan takes 5 to 9
// us, the join 6 to 18.
#include <type_traits>

#include "internal.h"
#include "latent_plan.h"
#include "latent_tile.h"

namespace kda {
namespace {

using namespace latent;

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kPlanThreads = 512;

struct Start {  // where a workgroup begins: tile t of a team's row block rb of chunk k of entity e
  int32_t left, w, e, k, rb, t;  // left: tiles of the share, 0: none; w: share * team + member
  Entity ent;
};

struct SharedParams {
  const char *lat, *rot, *scales;                // 16-bit cache: lat alone
  uint32_t lat_page, rot_page, scales_page;      // bytes
  int lat_row;                                   // bytes from token to token
  int num_pages, page_size, L, R;
  uint32_t page_mul;
  int page_shift;
  int eights;                                    // whether page_size is a multiple of 8
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
  int team;                                      // workgroups of a share
  float scale2;                                  // scale log2 e
  float* part;                                   // [slots][MB][L] normalised outputs
  float2* psum;                                  // [slots][MB] the maxima and the sums against them
  Entity* ents;                                  // [G + N]
  Start* starts;                                 // [kShares], by workgroup
  int64_t* total;                                // tiles on the line
  int32_t *bounds, *prefix;                      // [G + 1] the groups' sequences, [G] their shared tokens
};

__device__ __forceinline__ int tokens_of(const SharedParams& p, int len) {
  const int64_t room = (int64_t)p.max_pages * p.page_size;
  return len < 0 ? 0 : (len > room ? (int)room : len);
}
__device__ __forceinline__ int seq_tokens(const SharedParams& p, int n) { return tokens_of(p, p.lengths[n]); }

// Inclusive sums of two numbers over the workgroup's threads up to this one;
// *all_x, *all_y: over all of them.
__device__ __forceinline__ void block_scan(long long& x, long long& y, long long (&sums)[2][kPlanThreads / 64],
                                           long long* all_x, long long* all_y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long a = __shfl_up(x, d, 64), b = __shfl_up(y, d, 64);
    if (lane >= d) {
      x += a;
      y += b;
    }
  }
  if (lane == 63) {
    sums[0][wave] = x;
    sums[1][wave] = y;
  }
  __syncthreads();
  *all_x = *all_y = 0;
  long long px = 0, py = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / 64; ++i) {
    const long long a = sums[0][i], b = sums[1][i];
    px += i < wave ? a : 0;
    py += i < wave ? b : 0;
    *all_x += a;
    *all_y += b;
  }
  x += px;
  y += py;
  __syncthreads();
}

// One workgroup; what it reads is a few numbers a sequence, and what it takes is
// the latency of what depends on what: up to kPlanThreads entities stay in
// registers and LDS.
__global__ __launch_bounds__(kPlanThreads) void shared_plan_kernel(SharedParams p, int MB) {
  __shared__ long long sums[2][kPlanThreads / 64], number[kShares + 1];
  __shared__ int tops[kPlanThreads / 64];
  __shared__ Entity lents[kPlanThreads];
  __shared__ int lbounds[kPlanThreads + 1], lprefix[kPlanThreads];
  const int own_blocks = (p.rows + MB - 1) / MB, team_rows = MB * p.team;
  const int tid = threadIdx.x, E = p.G + p.N;
  const bool few = E <= kPlanThreads;
  int *bounds = few ? lbounds : p.bounds, *prefix = few ? lprefix : p.prefix;
  Entity* ents = few ? lents : p.ents;
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
      if (lane == 63) tops[wave] = v;
      __syncthreads();
      int most = carry;
      for (int k = 0; k < kPlanThreads / 64; ++k) {
        if (k < wave) v = max(v, tops[k]);
        most = max(most, tops[k]);
      }
      v = max(v, carry);
      carry = most;
      __syncthreads();
      if (i <= p.G) bounds[i] = v;
    }
    __syncthreads();
    for (int g = tid; g < p.G; g += kPlanThreads) {
      const int n0 = bounds[g], n1 = bounds[g + 1];
      int pre = 0;
      if (n1 - n0 >= 2) {
        const int len = seq_tokens(p, n0), s = p.shared[g];
        pre = s < 0 ? 0 : (s > len ? len : s);
      }
      prefix[g] = pre;
    }
    __syncthreads();
  }
  // entity e, but for its place and chunks
  auto entity = [&](int e) {
    Entity x;
    x.group = -1;
    x.t0 = 0;
    x.base = x.first = 0;
    x.chunks = 0;
    x.chunk = 1;
    x.longer = 0;
    if (e < p.G) {
      const int n0 = bounds[e], n1 = bounds[e + 1];
      x.row0 = n0 * p.rows;
      x.rows = (n1 - n0) * p.rows;
      x.seq = n0;
      x.t1 = prefix[e];
      x.slot = 2 * kShares + p.N * own_blocks + x.row0 / MB + e;  // (an earlier group's are fewer)
    } else {
      const int n = e - p.G;
      x.row0 = n * p.rows;
      x.rows = p.rows;
      x.seq = n;
      x.t1 = seq_tokens(p, n);
      x.slot = 2 * kShares + n * own_blocks;
      if (p.G > 0 && n >= bounds[0] && n < bounds[p.G]) {
        int lo = 0, hi = p.G;  // the last group that begins at n or before
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (bounds[mid] <= n) lo = mid; else hi = mid;
        }
        x.t0 = min(prefix[lo], x.t1);
        if (x.t0 > 0) x.group = lo;
      }
    }
    x.tiles = (int)((unsigned)(x.t1 - x.t0 + kTile - 1) / kTile);
    x.row_blocks = (unsigned)(x.rows + team_rows - 1) / (unsigned)team_rows;
    return x;
  };
  // the line's length with room for every entity, and from that the chunks; then the line
  long long total = 0, zero = 0;
  Entity mine;  // the last one of this thread: the only one, mostly
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    long long n = 0, all;
    if (e0 + tid < E) {
      mine = entity(e0 + tid);
      n = mine.tiles > 0 ? (long long)mine.row_blocks * (mine.tiles + kEnd) : 0;
    }
    block_scan(n, zero, sums, &all, &zero);
    total += all;
  }
  const long long quot = shares_of(p, total).quot;
  const unsigned share = quot > (1 << 30) ? 1u << 30 : (unsigned)quot;
  long long base = 0, first = 0;
  for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
    const int e = e0 + tid;
    long long n = 0, tiles = 0, all, all_tiles;
    if (e < E) {
      if (!few) mine = entity(e);
      if (mine.tiles > 0) {
        mine.cut(share);
        n = mine.line();
        tiles = (long long)mine.tiles * mine.row_blocks;
      }
    }
    long long upto = n, tiles_upto = tiles;
    block_scan(upto, tiles_upto, sums, &all, &all_tiles);
    if (e < E) {
      mine.base = base + upto - n;
      mine.first = first + tiles_upto - tiles;
      p.ents[e] = mine;
      if (few) lents[e] = mine;
    }
    base += all;
    first += all_tiles;
  }
  if (tid == 0) *p.total = base;
  if (tid < kShares) p.starts[tid].left = 0;
  __syncthreads();
  const Shares sh = shares_of(p, base);
  Start s;
  const int w = (unsigned)tid / (unsigned)p.team;  // thread: a member of this share's team
  if (w < sh.count) {
    const int64_t from = share_begin(sh, w);
    int lo = 0, hi = E;  // the last entity that begins there or before: it holds the place, if empty ones at its
    while (hi - lo > 1) {  // place are before it
      const int mid = (lo + hi) >> 1;
      if (ents[mid].base <= from) lo = mid; else hi = mid;
    }
    s.ent = ents[lo];
    const Entity& x = s.ent;
    const Spot at = x.at(from - x.base, sh.narrow);
    s.k = at.k;
    s.rb = at.rb;
    s.t = at.t;
    s.e = lo;
    s.w = tid;
    number[w] = x.first + (int64_t)x.chunk_begin(s.k) * x.row_blocks + (int64_t)s.rb * x.chunk_tiles(s.k) + s.t;
  }
  if (tid == 0) number[sh.count] = first;
  __syncthreads();
  if (w < sh.count) {
    s.left = (int)(number[w + 1] - number[w]);
    // neighbours to workgroups of one XCD, which are those of one number mod 8
    const unsigned per = (unsigned)(sh.count * p.team + 7) / 8;
    p.starts[(unsigned)tid % per * 8 + (unsigned)tid / per] = s;
  }
}

// A unit: the query rows that go over a chunk together.
struct Unit {
  int row0, rows;  // query rows
  int slot;        // its own place in the workspace
  int flags;
};
// The unit is all there is of its entity for its rows; and of its sequence.
constexpr int kSingle = 1, kAlone = 2;
constexpr int kUnits = 8;  // records kept: the tiles under way are of four units at most

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

// Global memory behind a pointer that came out of LDS.  (Without it the compiler takes flat
// instructions, and every barrier for LDS waits for those.)
template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* global(const void* at) {
  return (__attribute__((address_space(1))) T*)(uintptr_t)at;
}

// A cache's kind: its tile, and the stages that fit into the LDS.
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
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void latent_shared_kernel(
    SharedParams p) {
  using K = Kind<F8, LP, RP, NB, kPad>;
  using D = typename K::D;
  constexpr int MB = D::MB, KS = D::KS, MT = D::MT, TG = D::TG, TB = D::TB, NS = K::kStages;
  constexpr int kAhead = NS - 1;  // tiles fetched ahead of the one computed
  constexpr unsigned kStageBytes = K::kStageBytes, kRotaryBytes = RP > 0 ? kTile * RP * 2 : 16;
  __shared__ __attribute__((aligned(16))) char stage[NS][kStageBytes];
  __shared__ __attribute__((aligned(16))) char rotary[NS][kRotaryBytes];
  __shared__ __attribute__((aligned(16))) float tscale[NS][F8 ? kTile : 4];
  __shared__ __attribute__((aligned(16))) __bf16 prob[MB * kTile];
  __shared__ __attribute__((aligned(16))) int4 units[kUnits];
  __shared__ float smax[TG][MB];  // of a tile; at a piece's end the sums
  __shared__ float sfac[MB];      // factor of the older output; at a piece's end the maxima
  __shared__ int32_t pages[2][kWaves][64];  // of a batch's tokens, a copy a wave
  __shared__ int grown[2];        // whether a row's maximum has grown much in this tile
  // What is needed between units alone, so that it takes no scalar registers
  // within them (they do not hold everything, and what they do not hold is moved
  // to and from vector registers in every tile).
  __shared__ SharedParams cold;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const Start start = scalar_load(p.starts + blockIdx.x);
  if (start.left == 0) return;
  if (tid == 0) cold = p;
  if (tid < 2) grown[tid] = 0;
  if (kPad) {
    u32x4 *st = reinterpret_cast<u32x4*>(stage), *ro = reinterpret_cast<u32x4*>(rotary);
    for (unsigned i = tid; i < sizeof(stage) / 16; i += kThreads) st[i] = u32x4{0, 0, 0, 0};
    for (unsigned i = tid; i < sizeof(rotary) / 16; i += kThreads) ro[i] = u32x4{0, 0, 0, 0};
  }
  __syncthreads();
  const bool scoring = wave < D::kScoring;
  const int rblock = wave % NB;     // query rows this wave scores
  const int tg = (wave / NB) % TG;  // and tokens
  const int w = start.w;

  // ---- the tiles of the share, one after another.  Pages are looked up for a batch
  // of tiles of one unit at a time: 8 tiles and a lane for every 8 tokens of
  // them, where 8 tokens lie in one page (pages of a multiple of 8 tokens, an
  // entity that begins at one), otherwise one tile and a lane a token.  (A tile's
  // own lookup by each wave took a fifth of the time.)
  struct Batch {
    int pos, end, rem, group;  // its tokens pos .. before end; tiles to its unit's end; 2^group tokens a lane
  };
  Batch asked, now;            // the one being looked up, and the one in use
  int e = start.e, k = start.k, rb = start.rb;  // the unit of ``asked``
  const char* row_pages;                        // and its sequence's row of the table
  int asked_unit = 0;
  auto rows_of = [&](const Entity& x) {  // (a member without a row block computes the first row's and writes none)
    const unsigned team = cold.team, b = rb * team + (unsigned)w % team;
    const int n = min(MB, x.rows - (int)b * MB);
    return n > 0 ? Unit{x.row0 + (int)b * MB, n, x.slot + (int)b, 0} : Unit{x.row0, 0, 0, 0};
  };
  auto enter = [&](const Entity& x, int t) {
    asked.rem = x.chunk_tiles(k) - t;
    asked.pos = x.t0 + (x.chunk_begin(k) + t) * kTile;
    asked.end = x.t1;
    asked.group = p.eights && x.t0 % 8 == 0 ? 3 : 0;
    row_pages = uniform(reinterpret_cast<const char*>(cold.table + x.seq * cold.table_stride));
    if (tid == 0) {
      const int flags = x.chunks != 1 ? 0 : (e >= cold.G && x.t0 == 0 ? kSingle | kAlone : kSingle);
      const Unit u = rows_of(x);
      units[asked_unit % kUnits] = make_int4(u.row0, u.rows, u.slot, flags);
    }
  };
  auto follow = [&]() {  // (there is a next batch)
    const int n = min(asked.rem, 1 << asked.group);
    asked.rem -= n;
    asked.pos += n * kTile;
    if (asked.rem > 0) return;
    auto entity = [&]() {
      return scalar_load(reinterpret_cast<const Entity*>(uniform(reinterpret_cast<const char*>(cold.ents + e))));
    };
    Entity x = entity();
    if (++rb == x.row_blocks) {
      rb = 0;
      if (++k == x.chunks) {
        k = 0;
        do {
          ++e;
          x = entity();
        } while (x.chunks == 0);
      }
    }
    ++asked_unit;
    enter(x, 0);
  };
  auto unit_of = [&](int i) {
    const int4 v = units[i % kUnits];
    return Unit{uniform(v.x), uniform(v.y), uniform(v.z), uniform(v.w)};
  };

  // A tile under way.
  struct Tile {
    int pos, last;            // its first token; whether it is its unit's last tile
    unsigned long long live;  // which rows are there
  };
  auto page_of = [&](int at) { return (unsigned)(((uint64_t)(unsigned)at * p.page_mul) >> p.page_shift); };
  const unsigned pages_at = lds_offset(pages[0][wave]);
  int asked_to = 0;  // which copy of the pages ``asked`` goes to
  // (a lane behind the end looks up the last token's)
  auto ask = [&]() {
    const int at = min(asked.pos + (lane << asked.group), asked.end - 1);
    load_lds4(row_pages + (uint64_t)page_of(at) * 4, uniform(pages_at + asked_to * (unsigned)sizeof(pages[0])));
  };

  // Where rows lie: the wave's 8 of a tile, the same in all lanes, or one a lane.
  struct Rows {
    const char *lat, *rot, *scale;
  };
  auto place_at = [&](unsigned page, unsigned off) {
    Rows x;
    x.rot = x.scale = nullptr;
    x.lat = p.lat + (uint64_t)page * p.lat_page + (uint64_t)off * p.lat_row;
    if (F8) {
      x.scale = p.scales + (uint64_t)page * p.scales_page + (uint64_t)off * 4;
      if (RP > 0) x.rot = p.rot + (uint64_t)page * p.rot_page + (uint64_t)off * (unsigned)(2 * p.R);
    }
    return x;
  };
  const unsigned stage_at = lds_offset(stage), rotary_at = lds_offset(rotary), scale_at = lds_offset(tscale);
  constexpr unsigned kScaleBytes = sizeof(tscale[0]);
  // (anew for each tile: the loads' addresses then take no registers beside the products)
  auto columns_of = [&]() { return D::columns(p.L, p.R, wave, keep_here(tid & 63)); };
  typename D::Columns columns;
  // Load i, 0 <= i < kLoads, of a tile whose rows lie one behind the other, to stage ``to``.
  auto fetch = [&](const Rows& y, int i, int to) {
    const unsigned lat = stage_at + to * kStageBytes, rot = rotary_at + to * kRotaryBytes;
    if constexpr (F8)
      D::fetch_near(i, y.lat, y.rot, y.scale, kPad ? p.L : LP, kPad ? p.R : RP, wave, lane, columns, lat, rot,
                    scale_at + to * kScaleBytes);
    else
      D::fetch_near(i, y.lat, kPad ? p.lat_row : 2 * (LP + RP), wave, lane, columns, lat, rot);
  };

  int unlocated = start.left;     // tiles of the share behind the last one located
  int batch_left = 0, tile = 0;   // tiles of ``now`` not located, the next one's number in it
  unsigned long long sound = 0;   // from that one on: whether its tokens' pages are pages
  // The next tile, whose batch's pages have landed; the next batch's are asked for
  // with the last one.  True: it is near (all rows are there, and each wave's 8 lie one
  // behind the other) and its loads are the caller's to issue.  Otherwise they
  // are issued here: rows that are not there are fetched from the first one that
  // is (their weights are 0); a tile without any is not fetched and not computed.
  auto locate = [&](Tile& x, Rows& rows, int to) {
    if (batch_left == 0) {
      now = asked;
      batch_left = min(now.rem, 1 << now.group);
      tile = 0;
      const int page = pages[asked_to][wave][lane];
      sound = __ballot((unsigned)page < (unsigned)p.num_pages);
      asked_to ^= 1;
    }
    const int32_t* mine = pages[asked_to ^ 1][wave];
    const int pos = now.pos, number = tile;
    const bool near = now.group == 3 && (sound & 255) == 255 && pos + kTile <= now.end;
    const bool grouped = now.group == 3;
    const int end = now.end;
    x.pos = pos;
    x.last = now.rem == 1;
    x.live = ~0ull;
    now.pos += kTile;
    --now.rem;
    ++tile;
    sound >>= 8;
    --unlocated;
    if (--batch_left == 0 && unlocated > 0) {
      follow();
      ask();
    }
    columns = columns_of();
    if (near) {
      const int first = pos + 8 * wave;
      const unsigned page = uniform(mine[number * 8 + wave]);
      const Rows y = place_at(page, first - page_of(first) * p.page_size);
      rows.lat = uniform(y.lat);
      if (F8) {
        rows.scale = uniform(y.scale);
        if (RP > 0) rows.rot = uniform(y.rot);
      }
      return true;
    }
    int page = mine[grouped ? number * 8 + (lane >> 3) : lane];
    int off = pos + lane - (int)page_of(pos + lane) * p.page_size;
    x.live = __ballot(pos + lane < end && (unsigned)page < (unsigned)p.num_pages);
    if (x.live == 0) return false;
    const int some = __ffsll(x.live) - 1;
    const bool there = x.live >> lane & 1;
    const int spage = __builtin_amdgcn_readlane(page, some), soff = __builtin_amdgcn_readlane(off, some);
    const Rows y = place_at(there ? page : spage, there ? off : soff);
    const unsigned lat = stage_at + to * kStageBytes, rot = rotary_at + to * kRotaryBytes;
#pragma unroll
    for (int i = 0; i < D::kLoads; ++i) {
      if constexpr (F8)
        D::fetch_far(i, y.lat, y.rot, y.scale, wave, lane, columns, lat, rot, scale_at + to * kScaleBytes);
      else
        D::fetch_far(i, y.lat, wave, lane, columns, lat, rot);
    }
    return false;
  };
  auto fetch_all = [&](const Rows& y, int to) {
#pragma unroll
    for (int i = 0; i < D::kLoads; ++i) fetch(y, i, to);
  };

  // ---- queries
  bf16x8 qf[KS];
  int sees = 0;     // tokens that row ln of the wave's block sees
  int len = 0, behind = 0;  // its sequence's length, and the new tokens behind it
  auto load_q = [&](const Unit& u) {
    // (rows behind the unit's last one get its first one's queries; they are not written)
    const int r = keep_here(rblock * 16 + ln), lg = keep_here(lane >> 4);
    const unsigned row = u.row0 + (r < u.rows ? r : 0);
    const SharedParams& p = cold;
    const unsigned n = row / (unsigned)p.rows, in = row - n * p.rows, qi = in / (unsigned)p.H, h = in - qi * p.H;
    len = *global<const int>(p.lengths + n);
    const __bf16* q = p.q + n * p.qs[0] + qi * p.qs[1] + h * p.qs[2];
    const __bf16* qr = p.qr + n * p.qrs[0] + qi * p.qrs[1] + h * p.qrs[2];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      int c = 32 * i + 8 * lg;
      if constexpr (F8)
        c = D::component(i, lg);
      else if (i >= LP / 32)
        c -= LP;
      bf16x8 y = {};
      if (!kPad || c < (i < LP / 32 ? p.L : p.R)) y = *global<const bf16x8>((i < LP / 32 ? q : qr) + c);
      qf[i] = y;
    }
    behind = p.Q - 1 - (int)qi;
  };
  // They have landed, as has all that was asked for before.  (In every path of a piece's end: the
  // compiler would wait for them in every tile.)
  auto take_q = [&]() {
    wait_loads<0>();
#pragma unroll
    for (int i = 0; i < KS; ++i) asm volatile("" : "+v"(qf[i]));
    sees = tokens_of(cold, len) - behind;
  };
  int left = start.left - 1;  // tiles behind the one scored
  Tile ring[kAhead + 1];      // the one scored, and those fetched ahead
  {
    enter(start.ent, start.t);
    ask();
    load_q(rows_of(start.ent));
    take_q();
    Rows rows = {nullptr, nullptr, nullptr};
    if (locate(ring[0], rows, 0)) fetch_all(rows, 0);
    if (kAhead == 2 && left > 0) {
      if (batch_left == 0) wait_loads<0>();
      if (locate(ring[kAhead - 1], rows, 1)) fetch_all(rows, 1);
    }
    __syncthreads();  // (the units' records)
  }

  int unit = 0;               // of the tile computed
  bool begun = start.t == 0;  // whether the piece begins where its unit does
  int later = 0;              // 1: behind the share's first piece

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

  // ---- the scores of a tile and their weights
  float sum = 0.f, fac = 1.f;
  f32x4 s[TB], sc[TB];
  // Weights of the scores against the maximum in use, for the matrix unit in bf16;
  // their sum stays in fp32.  In 8 bits the tokens' scales go into them before
  // they are rounded.
  auto weigh = [&](float base) {
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      bf16x4 pb;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = exp2_hw(fmaf(s[j][i], p.scale2, -base));
        sum += w;
        pb[i] = (__bf16)(F8 ? w * sc[j][i] : w);
      }
      const int tk = 16 * (TB * tg + j) + 4 * lg;
      *reinterpret_cast<bf16x4*>(prob + (rblock * 16 + ln) * kTile + (((tk >> 3) ^ (ln & 7)) << 3) + (tk & 7)) = pb;
    }
  };
  // The scores of what a query row does not see, their maximum, and the weights.
  auto soften = [&](const Tile& x, int par) {
    if (x.live != ~0ull || __any(x.pos + kTile > sees)) {
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        // of the lane's four tokens: how many are seen, and which are there
        const int at4 = 16 * (TB * tg + j) + 4 * lg, n = sees - x.pos - at4;
        const unsigned there = (unsigned)(x.live >> at4);
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
  };
  // Behind a barrier, where ``grown`` is set: the new maxima, the weights again, and
  // the older output's factor.
  auto grow = [&]() {
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
  };
  // ---- the end of a piece, which is its unit's end too or not
  auto finish = [&](bool unit_ends) {
    const SharedParams& p = cold;
    const Unit u = unit_of(unit);
    const float lsum = sum_halves(sum_quarters(l));
    lds_barrier();
    const int ln = keep_here(lane & 15), lg = keep_here(lane >> 4);
    if (scoring && lg == 0) {
      smax[tg][rblock * 16 + ln] = lsum;
      if (tg == 0) sfac[rblock * 16 + ln] = m;
    }
    lds_barrier();
    const bool whole = begun && unit_ends, direct = whole && (u.flags & kAlone);
    const int64_t slot = whole && (u.flags & kSingle) ? u.slot : 2 * w + later;
    const int col0 = wave * (MT * 16) + 4 * lg;
    float inv[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float sum = smax[0][j * 16 + ln];
#pragma unroll
      for (int g = 1; g < TG; ++g) sum += smax[g][j * 16 + ln];
      inv[j] = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    }
    take_q();  // (before the stores, which nothing then waits for)
    if (direct) {
      __bf16* out = p.out + ((int64_t)u.row0 + ln) * p.L + col0;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (j * 16 + ln < u.rows) {
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const f32x4 o = acc[i][j] * inv[j];
            const bf16x4 ob = {(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
            if (!kPad || col0 + 16 * i < p.L) *global<bf16x4>(out + 16 * i) = ob;
          }
        }
        out += 16 * p.L;
      }
    } else {
      float* part = p.part + (slot * MB + ln) * p.L + col0;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (j * 16 + ln < u.rows) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
            if (!kPad || col0 + 16 * i < p.L) *global<f32x4>(part + 16 * i) = acc[i][j] * inv[j];
        }
        part += 16 * p.L;
      }
    }
    const int r = keep_here(tid);
    if (r < u.rows) {
      float sum = smax[0][r];
#pragma unroll
      for (int g = 1; g < TG; ++g) sum += smax[g][r];
      if (!direct)
        *global<f32x2>(p.psum + slot * MB + r) = f32x2{sfac[r], sum};
      else if (p.lse)
        *global<float>(p.lse + (int64_t)u.row0 + r) = sum == 0.f ? -INFINITY : (sfac[r] + __log2f(sum)) * kLn2;
    }
    ++unit;
    begun = true;
    later = 1;
  };
  int st = 0;           // the stage of the tile computed
  bool landed = false;  // whether it and the next one are known to be there
  for (int par = 0;; par ^= 1) {
    // this tile has landed (the next one's loads may be under way, and the lookup
    // before them is done), and the readers of the one before are done
    if (landed) {
      landed = false;  // (at the end of a piece)
    } else if constexpr (kAhead == 2) {
      if (left > 0 && ring[1].live)
        wait_loads<D::kLoads>();
      else
        wait_loads<0>();
    } else {
      wait_loads<0>();
    }
    lds_barrier();
    const Tile cur = ring[0];
    const bool more = left > 0;                // a tile behind this one
    const int to = st == 0 ? NS - 1 : st - 1;  // the stage fetched to: that of the tile before
    if (tid == 0) grown[par ^ 1] = 0;
    // A near tile's first load is issued here and the others along the scores, or all here by
    // waves that score nothing.
    Rows rows = {nullptr, nullptr, nullptr};
    const bool fetches = left > kAhead - 1 && locate(ring[kAhead], rows, to);
    const bool spread = fetches && scoring && cur.live;
    constexpr int kFirst = F8 ? 1 : D::kLoads - D::kLat;  // (a 16-bit tile's scores call for its latent loads alone)
    if (fetches && !spread) fetch_all(rows, to);
    if (kFirst > 0 && spread) fetch(rows, 0, to);
    if (cur.live) {
      if (scoring) {
        const char *lat = stage[0] + st * kStageBytes, *rot = rotary[0] + st * kRotaryBytes;
        auto load = [&](int i) {
          if (spread) fetch(rows, F8 ? i : i + kFirst, to);
        };
        if constexpr (F8)
          D::scores(lat + 16 * TB * tg * LP, rot + 16 * TB * tg * RP * 2, tscale[0] + st * kTile + 16 * TB * tg, qf,
                    ln, lg, s, sc, load);
        else
          D::scores(reinterpret_cast<const __bf16*>(lat) + (16 * TB * tg + ln) * LP,
                    reinterpret_cast<const __bf16*>(rot) + (16 * TB * tg + ln) * RP, qf, ln, lg, s, load);
        soften(cur, par);
      }
      lds_barrier();
      fac = 1.f;
      if (grown[par]) grow();
      l = l * fac + sum;
      if constexpr (F8)
        D::values(stage[0] + st * kStageBytes, prob, wave, ln, lg, acc);
      else
        D::values(reinterpret_cast<const __bf16*>(stage[0] + st * kStageBytes), prob, wave, ln, lg, acc);
    }
    if (!more || cur.last) {
      if (more) load_q(unit_of(unit + 1));
      finish(cur.last);
      if (!more) return;  // (no load to LDS outlives the workgroup)
      clear();
      landed = true;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ring[i] = ring[i + 1];
    st = st == NS - 1 ? 0 : st + 1;
    --left;
  }
}

// Joins the pieces of a query row, its prefix's and its own, and writes the outputs of
// empty sequences.  A wave takes one query row (8 columns a lane) and every
// ``parts``-th piece; grid: (groups of 8 / parts rows, sequences).
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
  const Shares sh = shares_of(p, scalar_load(p.total));
  // a sequence that one piece holds whole has its output
  if (own.t0 == 0 && own.chunks == 1) {
    const int rb = (blockIdx.x * (kWaves / parts)) / MB;  // (that of all the workgroup's rows)
    const int64_t a = own.base + own.unit_begin(0, rb / p.team) + own.room();
    if (share_at(sh, a) == share_at(sh, a + own.tiles - 1)) return;
  }
  float top = -INFINITY, sum = 0.f;
  f32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  for (int which = 0; have && which < 2; ++which) {  // the prefix's pieces, its own
    if (which == 0 && own.group < 0) continue;
    const Entity x = which == 1 ? own : scalar_load(p.ents + own.group);
    const int in = (int)(grow - x.row0), rb = in / MB, r = in - rb * MB;
    const int block = (unsigned)rb / (unsigned)p.team, member = rb - block * p.team;
    for (int k0 = 0; k0 < x.chunks; k0 += 64) {
      // lane i: the pieces of the row block's unit in chunk k0 + i, their number and where the first one is: the
      // whole unit's own place, or 2 w (+ 1 where others are before it in share w)
      const int k = k0 + lane;
      int first = 0, place = 0, count = 0;
      if (k < x.chunks) {
        const int64_t unit = x.base + x.unit_begin(k, block), a = unit + x.room();
        first = share_at(sh, a);
        count = share_at(sh, a + x.chunk_tiles(k) - 1) - first + 1;
        place = count == 1 && x.chunks == 1 ? x.slot + rb
                                            : 2 * (first * p.team + member) + (share_begin(sh, first) < unit ? 1 : 0);
      }
      const int upto = wave_scan(count, lane), pieces = __builtin_amdgcn_readlane(upto, 63);
      for (int q0 = part; q0 < pieces; q0 += 4 * parts) {
        // one pass with a running maximum, four pieces' loads at once
        float e[4], s[4];
        f32x4 v[4][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = q0 + u * parts;
          e[u] = -INFINITY;
          s[u] = 0.f;
          v[u][0] = v[u][1] = f32x4{0, 0, 0, 0};
          if (q >= pieces) continue;
          const int i = __ffsll(__ballot(upto > q)) - 1;
          const int in_unit = q - (__builtin_amdgcn_readlane(upto, i) - __builtin_amdgcn_readlane(count, i));
          const int64_t slot = in_unit == 0 ? __builtin_amdgcn_readlane(place, i)
                                            : 2 * ((__builtin_amdgcn_readlane(first, i) + in_unit) * p.team + member);
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
        for (int u = 0; u < 4; ++u) mx = fmaxf(mx, e[u]);
        const float base = mx == -INFINITY ? 0.f : mx, old = exp2_hw(top - base);
        sum *= old;
        o[0] *= old;
        o[1] *= old;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float f = exp2_hw(e[u] - base) * s[u];
          sum += f;
          o[0] += f * v[u][0];
          o[1] += f * v[u][1];
        }
        top = mx;
      }
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

// Blocks of 16 query rows a workgroup takes at once: as few as hold a sequence's rows (64 x 4000
// tokens in 8 bits, 16 heads: 57 us with one block, 63 with two, 76 with four; 32 heads: 64
// with two, 77 with four), with groups the whole batch's, whatever the sizes of the groups.  That suits prefixes
// of many rows (4096 tokens and 100 of each sequence's own in 8 bits: 8 groups of 12 sequences with 32 heads 114
// us with one block, 92 with two, 85 with four; one group of 64 with 16 heads 61, 57 and 60; in 16 bits 113, 86 and 78,
// and 58, 54 and 57) and costs groups of few (64 pairs with 8 heads 59, 65 and 79, 128 pairs with 4 heads 95, 106
// and 134; in 16 bits, which the bytes bound, 86, 86 and 87, and 144, 144 and 146).
int blocks_of(int64_t N, int64_t Q, int64_t H, int64_t G) {
  const int64_t rows = G > 0 ? N * Q * H : Q * H;
  return rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
}

// Pieces in the workspace.  Two a workgroup: of those that its share begins with and of those
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
  const bool whole = p.L == LP && (p.R == 0 || p.R == 64);  // no padding columns
  if (p.R == 0) return whole ? launch_nb<F8, LP, 0, false>(p, nb, stream) : launch_nb<F8, LP, 0, true>(p, nb, stream);
  return whole ? launch_nb<F8, LP, 64, false>(p, nb, stream) : launch_nb<F8, LP, 64, true>(p, nb, stream);
}

template <bool F8>
hipError_t launch_l(const SharedParams& p, int nb, hipStream_t stream) {
  if (p.L <= 128) return launch_r<F8, 128>(p, nb, stream);
  return p.L <= 256 ? launch_r<F8, 256>(p, nb, stream) : launch_r<F8, 512>(p, nb, stream);
}

}  // namespace

size_t latent_shared_workspace_bytes(int64_t N, int64_t Q, int64_t H, int64_t L, int64_t G) {
  const size_t rows = (size_t)slots_of(N, Q, H, G) * 16 * blocks_of(N, Q, H, G);
  return round16(rows * (size_t)L * 4) + round16(rows * 8) + (size_t)(G + N) * sizeof(Entity) +
         kShares * sizeof(Start) + 16 + (size_t)(2 * G + 1) * 4;
}

hipError_t launch_latent_shared(const kda_latent_shared_args_t& a, hipStream_t stream) {
  const int nb = blocks_of(a.N, a.Q, a.H, a.G), MB = 16 * nb;
  const bool f8 = a.cache_dtype == KDA_E4M3;
  SharedParams p = {};
  p.lat = static_cast<const char*>(a.cache);
  p.lat_page = (uint32_t)(a.page_stride * (f8 ? 1 : 2));
  p.lat_row = (int)(f8 ? a.L : 2 * (a.L + a.R));
  if (f8) {
    p.scales = reinterpret_cast<const char*>(a.scales);
    p.scales_page = (uint32_t)(a.scales_page_stride * 4);
    p.rot = static_cast<const char*>(a.rope);
    p.rot_page = (uint32_t)(a.rope_page_stride * 2);
  }
  p.num_pages = (int)a.num_pages;
  p.page_size = (int)a.page_size;
  p.L = (int)a.L;
  p.R = (int)a.R;
  page_divisor(p.page_size, &p.page_mul, &p.page_shift);
  p.eights = p.page_size % 8 == 0;
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
  p.team = (int)((a.Q * a.H + MB - 1) / MB);
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
  // Few rows: more waves share a row's pieces, 4096 waves in all (a call on 1 x 4000 tokens with 32
  // heads takes 27 us, with one wave a row 42; the join of 64 x 128 rows 14 us, with up to 16384
  // waves 20; of 64 x 16 rows of 30 pieces 15, with up to 8192 18).
  int parts = kWaves;
  while (parts > 1 && (int64_t)p.rows * p.N * parts > 512 * kWaves) parts >>= 1;
  const int per = kWaves / parts;
  hipLaunchKernelGGL(shared_join_kernel, dim3((unsigned)((p.rows + per - 1) / per), (unsigned)p.N), dim3(kThreads), 0,
                     stream, p, MB, parts);
  return hipGetLastError();
}

}  // namespace kda
