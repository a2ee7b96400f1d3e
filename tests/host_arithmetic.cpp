// The library's host and plan arithmetic as C functions, for tests on the CPU.
#include "internal.h"
#include "latent_plan.h"

using namespace kda::latent;

namespace {

struct Team {
  int team;
};

}  // namespace

extern "C" {

int64_t cache_slice_rows(int rows) { return kda::cache_slice_rows(rows); }

int64_t plan_quotient(int64_t a, int64_t b, int narrow) { return quotient(a, b, narrow != 0); }

// quot, rem, count, narrow
void plan_shares(int team, int64_t total, int64_t* out) {
  const Shares s = shares_of(Team{team}, total);
  out[0] = s.quot;
  out[1] = s.rem;
  out[2] = s.count;
  out[3] = s.narrow;
}
int64_t plan_share_begin(int team, int64_t total, int w) { return share_begin(shares_of(Team{team}, total), w); }
int plan_share_at(int team, int64_t total, int64_t x) { return share_at(shares_of(Team{team}, total), x); }

// An entity's chunks and line: chunks, chunk, longer, room, line
void plan_cut(int tiles, int row_blocks, unsigned share, int64_t* out) {
  Entity e = {};
  e.tiles = tiles;
  e.row_blocks = row_blocks;
  e.cut(share);
  out[0] = e.chunks;
  out[1] = e.chunk;
  out[2] = e.longer;
  out[3] = e.room();
  out[4] = e.line();
}
// Where unit (k, rb) begins and how many tiles it has; and what lies at a place: k, rb, t
void plan_unit(int tiles, int row_blocks, unsigned share, int k, int rb, int64_t* out) {
  Entity e = {};
  e.tiles = tiles;
  e.row_blocks = row_blocks;
  e.cut(share);
  out[0] = e.unit_begin(k, rb);
  out[1] = e.chunk_tiles(k);
}
void plan_at(int tiles, int row_blocks, unsigned share, int64_t in, int narrow, int* out) {
  Entity e = {};
  e.tiles = tiles;
  e.row_blocks = row_blocks;
  e.cut(share);
  const Spot s = e.at(in, narrow != 0);
  out[0] = s.k;
  out[1] = s.rb;
  out[2] = s.t;
}

}  // extern "C"
