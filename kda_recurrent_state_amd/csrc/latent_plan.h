// Arithmetic of the plan of shared and 8-bit latent decode: entities on a line of
// tiles, the line in equal shares.  No HIP of its own, so that a host compiler takes it too.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define KDA_PLAN_FN __device__ __forceinline__
#else
#include <algorithm>
#define KDA_PLAN_FN inline
using std::max;
using std::min;
#endif

namespace kda {
namespace latent {

constexpr int kShares = 256;  // workgroups, one a CU
// Room before a unit of an entity of one chunk, in tiles: 40 sequences of 64 to 1024 tokens behind
// a prefix, 256 query rows each, take 436 us with 4, 476 with 3 and 525 with 2 (the shares with many
// units come last) and 433 with 6, where 200 ragged ones take 109, 110, 116 and 112.
constexpr int kEnd = 4;

// a / b of 0 <= a < 2^52, 0 < b, or with ``narrow`` (the same in all lanes) < 2^31.  (The quotient
// in fp64 is off by less than one; a division of 64-bit integers is four times the
// instructions, and the plan's and the join's time is much of their own code's way
// into the caches.)
KDA_PLAN_FN int64_t quotient(int64_t a, int64_t b, bool narrow) {
  if (narrow) return (unsigned)a / (unsigned)b;
  const int64_t q = (int64_t)((double)a / (double)b), r = a - q * b;
  return q + (r < 0 ? -1 : (r >= b ? 1 : 0));
}

struct Spot {  // tile t of a team's row block rb of chunk k
  int k, rb, t;
};

struct Entity {
  int64_t base, first;     // place on the line, and the number of its first tile
  int32_t tiles, row_blocks;  // row_blocks: a team's, of ``team`` blocks of MB rows each
  int32_t chunks, chunk;   // and the tiles of one; the first ``longer`` ones have one more
  int32_t longer;
  int32_t row0, rows;      // query rows
  int32_t seq, t0, t1;     // tokens [t0, t1) of this sequence
  int32_t slot;            // of its first row block's pieces that no share cuts and that are not chunks
  int32_t group;           // of a sequence: the entity of its prefix, or -1

  KDA_PLAN_FN int room() const { return chunks == 1 ? kEnd : 0; }
  // place on the line, from the entity's, of row block rb of chunk k (its room, then its tiles)
  KDA_PLAN_FN int64_t unit_begin(int k, int rb) const {
    return (int64_t)chunk_begin(k) * row_blocks + (int64_t)rb * (chunk_tiles(k) + room());
  }
  KDA_PLAN_FN int64_t line() const { return (int64_t)row_blocks * (tiles + room()); }
  KDA_PLAN_FN int chunk_begin(int k) const { return k * chunk + min(k, longer); }
  KDA_PLAN_FN int chunk_tiles(int k) const { return chunk + (k < longer ? 1 : 0); }
  // An entity with tiles, in chunks of at least a share where a team has several row blocks of it.
  KDA_PLAN_FN void cut(unsigned share) {
    chunks = row_blocks == 1 ? 1 : (int)max(1u, (unsigned)tiles / share);
    chunk = (int)((unsigned)tiles / (unsigned)chunks);
    longer = tiles - chunk * chunks;
  }
  // The unit and tile of place ``in`` of its line; a unit's room counts as its first tile.
  KDA_PLAN_FN Spot at(int64_t in, bool narrow) const {
    Spot s;
    if (chunks == 1) {
      s.k = 0;
      s.rb = (int)quotient(in, tiles + kEnd, narrow);
    } else {
      const unsigned y = (unsigned)quotient(in, row_blocks, narrow), ahead = longer * (chunk + 1);
      s.k = (int)(y < ahead ? y / (unsigned)(chunk + 1) : longer + (y - ahead) / (unsigned)chunk);
      s.rb = (int)quotient(in - unit_begin(s.k, 0), chunk_tiles(s.k), narrow);
    }
    const int64_t rest = in - unit_begin(s.k, s.rb) - room();
    s.t = rest > 0 ? (int)rest : 0;
    return s;
  }
};

// The line in equal shares, none empty (fewer of them where there are fewer tiles).
struct Shares {
  int64_t quot;
  int rem, count;
  bool narrow;  // whether the line has fewer than 2^31 places
};
// p.team: workgroups of a share.  (Given by itself, the compiler loads it another way, and a call of one
// sequence takes 0.7 us longer.)
template <typename Params>
KDA_PLAN_FN Shares shares_of(const Params& p, int64_t total) {
  const unsigned most = kShares / (unsigned)p.team;
  const bool few = total < most;
  return {few ? 1 : (int64_t)((uint64_t)total / most), few ? 0 : (int)((uint64_t)total % most),
          few ? (int)total : (int)most, total >> 31 == 0};
}
KDA_PLAN_FN int64_t share_begin(const Shares& s, int w) { return w * s.quot + min(w, s.rem); }
// the share that holds place x
KDA_PLAN_FN int share_at(const Shares& s, int64_t x) {
  const int64_t longer = s.rem * (s.quot + 1);
  const bool in = x < longer;
  return (in ? 0 : s.rem) + (int)quotient(in ? x : x - longer, in ? s.quot + 1 : s.quot, s.narrow);
}

}  // namespace latent
}  // namespace kda
