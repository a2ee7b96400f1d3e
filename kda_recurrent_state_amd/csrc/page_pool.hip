// Pages of a cache shared by sequences: fork, compact and free, for gfx950.
//
// The bookkeeping is a page table [sequence slot][page], the slots' lengths in
// tokens and a reference count per page (free: not above zero).  All results
// are fixed by the inputs: free pages are taken in ascending order, in the
// order of the forks, and compaction moves the k-th live page behind the live
// count to the k-th free page before it.  The payload copies stream whole
// pages with the widest vector the alignment allows; a call's stores (one a
// layer) are copied by one launch, which finds each move's pages from what
// the planning kernel left in the workspace.
//
// Bound.  The copies by HBM: 256 state rows of 2 MiB in 191 us (1.07 GB, 5.6
// TB/s; a large library copy reaches 5.0), 280 MB of pages of 72 KB in 49 us
// (5.7).  The planning kernels are one workgroup, since each entry's place
// follows from all before it, and are bound by the latency of their few
// dependent loads (5 to 11 us); small calls are bound by their launches.
// Copies are cut into tiles of 16 KB: 256 threads with 4 vectors of 16 bytes in
// flight each.
#include "internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kMaxStores = 32;  // stores a copying launch takes
// Workgroups for the sequence slots of a launch: one each up to here, beyond it
// each takes several (HIP launches fewer than 2^32 threads a grid dimension).
constexpr int64_t kMostTables = 1 << 20;

struct Pool {
  int32_t* table;
  int64_t table_stride, num_seqs, max_pages;
  int32_t* lengths;
  int32_t* refs;
  int64_t num_pages, page_size;
};

struct Stores {
  char* data[kMaxStores];
  int64_t stride[kMaxStores];
  int64_t vecs[kMaxStores];   // vectors a page
  int64_t tiles[kMaxStores];  // tiles a page
  int64_t per_page;           // sum of tiles
  int n;
};

// (lengths are below 2^31 and page sizes at most 2^30: 32-bit arithmetic)
__device__ __forceinline__ int64_t used_pages(int64_t len, int64_t page) {
  return len <= 0 ? 0 : (int64_t)(((uint32_t)len + (uint32_t)page - 1) / (uint32_t)page);
}

// inclusive prefix sum over the workgroup; tmp holds one value a wave
__device__ __forceinline__ int block_scan(int x, int* tmp, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) tmp[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < waves; ++i) {
    before += i < wave ? tmp[i] : 0;
    all += tmp[i];
  }
  *total = all;
  return x + before;
}

__device__ __forceinline__ int pages_needed(int share, int64_t len, int64_t page, int64_t used) {
  return share ? ((uint32_t)len % (uint32_t)page != 0 ? 1 : 0) : (int)used;
}

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kUnroll = 4;  // vectors in flight a thread

// Copies tile ``tile`` of page ``from`` to page ``to`` of store c.
template <typename VecT>
__device__ __forceinline__ void copy_tile(const Stores& st, int c, int64_t tile, int64_t from, int64_t to) {
  const VecT* src = reinterpret_cast<const VecT*>(st.data[c] + from * st.stride[c]);
  VecT* dst = reinterpret_cast<VecT*>(st.data[c] + to * st.stride[c]);
  const int64_t begin = tile * kThreads * kUnroll;
  const int64_t end = begin + kThreads * kUnroll < st.vecs[c] ? begin + kThreads * kUnroll : st.vecs[c];
  if (end - begin == kThreads * kUnroll) {
    VecT buf[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) buf[u] = __builtin_nontemporal_load(src + begin + u * kThreads + threadIdx.x);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) __builtin_nontemporal_store(buf[u], dst + begin + u * kThreads + threadIdx.x);
  } else {
    for (int64_t i = begin + threadIdx.x; i < end; i += kThreads)
      __builtin_nontemporal_store(__builtin_nontemporal_load(src + i), dst + i);
  }
}

__device__ __forceinline__ int store_of(const Stores& st, int64_t* tile) {
  int c = 0;
  while (*tile >= st.tiles[c]) *tile -= st.tiles[c++];
  return c;
}

// ---------------------------------------------------------------------------
// fork

// Workspace of a fork call (int32 each).
struct ForkPlan {
  int32_t* need;   // [M] pages the entry takes, -1: bad entry
  int32_t* used;   // [M] pages the parent has
  int32_t* upto;   // [M] pages that the entries up to this one take; after the plan -1: not served
  int32_t* count;  // [1] pages taken by the served entries
  int32_t* free;   // the free pages taken, in order
};

// Many entries: a workgroup each.
template <typename IdxT>
__global__ __launch_bounds__(kThreads) void fork_check_kernel(Pool p, const IdxT* src, const IdxT* dst, int share,
                                                              ForkPlan w) {
  const int64_t i = blockIdx.x;
  const int64_t s = (int64_t)src[i], d = (int64_t)dst[i];
  bool ok = s >= 0 && s < p.num_seqs && d >= 0 && d < p.num_seqs && s != d;
  int64_t len = 0, used = 0;
  if (ok) {  // uniform
    len = p.lengths[s];
    used = used_pages(len, p.page_size);
    ok = len >= 0 && p.lengths[d] == 0 && used <= p.max_pages;
  }
  if (ok) {
    bool bad = false;
    for (int64_t j = threadIdx.x; j < i; j += kThreads) bad |= (int64_t)dst[j] == d;  // the slot is another entry's
    const int32_t* row = p.table + s * p.table_stride;
    for (int64_t j = threadIdx.x; j < used; j += kThreads) {
      const int64_t pg = row[j];
      bad |= pg < 0 || pg >= p.num_pages || p.refs[pg] <= 0;
    }
    ok = __syncthreads_or(bad) == 0;
  }
  if (threadIdx.x == 0) {
    w.need[i] = !ok ? -1 : pages_needed(share, len, p.page_size, used);
    w.used[i] = (int32_t)used;
  }
}

constexpr int kFew = 128;                         // entries the plan checks itself
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kEach = kFew / kPlanWaves;          // of which a wave takes up to so many

// The same checks for up to kFew entries by the planning workgroup (a launch
// less: 96 entries 21 us, in a kernel of their own 24): thread i fetches entry i, then a wave checks the pages of kEach
// entries at once, so that their loads overlap.
template <typename IdxT>
__device__ void fork_check_few(const Pool& p, const IdxT* src, const IdxT* dst, int M, int share, const ForkPlan& w,
                               int64_t (*entry)[kFew]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t *es = entry[0], *ed = entry[1], *eu = entry[2];  // slots, and pages of the parent (0 where the entry is bad)
  int need = -1;
  if (tid < M) {
    const int64_t s = (int64_t)src[tid], d = (int64_t)dst[tid];
    int64_t used = 0;
    if (s >= 0 && s < p.num_seqs && d >= 0 && d < p.num_seqs && s != d) {
      const int64_t len = p.lengths[s], pages = used_pages(len, p.page_size);
      if (len >= 0 && p.lengths[d] == 0 && pages <= p.max_pages) {
        used = pages;
        need = pages_needed(share, len, p.page_size, used);
      }
    }
    es[tid] = s;
    ed[tid] = d;
    eu[tid] = used;
    w.need[tid] = need;
    w.used[tid] = (int32_t)used;
  }
  __syncthreads();
  int32_t page[kEach];
  bool bad[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = wave + k * kPlanWaves;
    page[k] = -1;
    bad[k] = false;
    if (i < M && lane < eu[i]) page[k] = (p.table + es[i] * p.table_stride)[lane];
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = wave + k * kPlanWaves;
    if (i < M && lane < eu[i])
      bad[k] = page[k] < 0 || page[k] >= p.num_pages || p.refs[page[k]] <= 0;
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = wave + k * kPlanWaves;
    if (i >= M) continue;
    for (int64_t j = lane + 64; j < eu[i]; j += 64) {
      const int64_t pg = (p.table + es[i] * p.table_stride)[j];
      bad[k] |= pg < 0 || pg >= p.num_pages || p.refs[pg] <= 0;
    }
    for (int j = lane; j < i; j += 64) bad[k] |= ed[j] == ed[i];  // the slot is another entry's
    if (__ballot(bad[k]) != 0 && lane == 0) w.need[i] = -1;
  }
  __syncthreads();  // (the entries are read back by other threads)
}

template <typename IdxT>
__global__ __launch_bounds__(kPlanThreads) void fork_plan_kernel(Pool p, const IdxT* src, const IdxT* dst, int64_t M,
                                                                 int share, int32_t* status, ForkPlan w) {
  __shared__ int tmp[kPlanThreads / 64];
  __shared__ int64_t entry[3][kFew];
  if (M <= kFew) fork_check_few(p, src, dst, (int)M, share, w, entry);
  // pages the entries ask for, in order (64-bit totals: M max_pages may pass 32 bits)
  int64_t asked = 0;
  for (int64_t i0 = 0; i0 < M; i0 += kPlanThreads) {
    const int64_t i = i0 + threadIdx.x;
    const int x = i < M ? (w.need[i] > 0 ? w.need[i] : 0) : 0;
    int all = 0;
    const int incl = block_scan(x, tmp, &all);
    const int64_t upto = asked + incl;
    if (i < M) w.upto[i] = upto > 0x7fffffff ? 0x7fffffff : (int32_t)upto;
    asked += all;
  }
  if (asked > p.num_pages) asked = p.num_pages;
  // the first ``asked`` free pages
  int64_t found = 0;
  for (int64_t i0 = 0; i0 < p.num_pages && found < asked; i0 += kPlanThreads) {
    const int64_t i = i0 + threadIdx.x;
    const int x = i < p.num_pages && p.refs[i] <= 0 ? 1 : 0;
    int all = 0;
    const int64_t at = found + block_scan(x, tmp, &all) - 1;
    if (x && at < asked) w.free[at] = (int32_t)i;
    found += all;
  }
  // served: what the entries so far ask for is there
  int most = 0;
  for (int64_t i = threadIdx.x; i < M; i += kPlanThreads) {
    const bool ok = w.need[i] >= 0, served = ok && w.upto[i] <= found;
    status[i] = served ? 0 : (ok ? 1 : 2);
    if (served && w.upto[i] > most) most = w.upto[i];
    if (!served) w.need[i] = -1;
  }
  __syncthreads();
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const int y = __shfl_xor(most, d, 64);
    most = y > most ? y : most;
  }
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPlanThreads / 64; ++i) most = tmp[i] > most ? tmp[i] : most;
    *w.count = most;
  }
}

// Blocks [0, tables): the children's table rows, lengths and reference counts
// (``tables`` is M in a call's first launch, else 0); the others copy pages.
template <typename VecT, typename IdxT>
__global__ __launch_bounds__(kThreads) void fork_apply_kernel(Pool p, const IdxT* src, const IdxT* dst, int64_t M,
                                                              int64_t tables, ForkPlan w, Stores st) {
  if ((int64_t)blockIdx.x < tables) {
    const int64_t i = blockIdx.x;
    const int need = w.need[i];
    if (need < 0) return;
    const int64_t s = (int64_t)src[i], d = (int64_t)dst[i];
    const int used = w.used[i], fresh = used - need, at = w.upto[i] - need;
    const int32_t* from = p.table + s * p.table_stride;
    int32_t* to = p.table + d * p.table_stride;
    for (int64_t j = threadIdx.x; j < p.max_pages; j += kThreads) {
      int pg = -1;
      if (j < fresh) {
        pg = from[j];
        atomicAdd(p.refs + pg, 1);  // whole numbers: the order does not matter
      } else if (j < used) {
        pg = w.free[at + j - fresh];
        p.refs[pg] = 1;
      }
      to[j] = pg;
    }
    // (the slot of an empty parent may be another entry's child by now)
    if (threadIdx.x == 0) p.lengths[d] = used > 0 ? p.lengths[s] : 0;
    return;
  }
  const int64_t total = (int64_t)*w.count * st.per_page;
  for (int64_t it = blockIdx.x - tables; it < total; it += gridDim.x - tables) {
    const int64_t move = it / st.per_page;
    int64_t tile = it - move * st.per_page;
    // the entry that takes this page: the first whose pages reach past it (an
    // entry that takes none repeats the count before it and is never first)
    int64_t lo = 0, hi = M - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (w.upto[mid] > move) hi = mid;
      else lo = mid + 1;
    }
    const int64_t col = w.used[lo] - (w.upto[lo] - move);
    const int64_t from = p.table[(int64_t)src[lo] * p.table_stride + col];
    const int c = store_of(st, &tile);
    copy_tile<VecT>(st, c, tile, from, w.free[move]);
  }
}

// ---------------------------------------------------------------------------
// compact

struct CompactPlan {
  int32_t* rank;   // [num_pages] of a page behind the live count: its move, -1: none
  int32_t* from;   // [num_pages / 2] the moves
  int32_t* to;
  int32_t* count;  // [2] moves, live pages
};

// One workgroup.  A wave looks at 64 pages with one load and one ballot and
// holds the ballots of up to kChunks of them, chunk c's in lane c; up to
// kPlanThreads kChunks pages (32768) are loaded once, more of them in as many
// steps as it takes, three times over.  (8192 pages: 10 us; one page a thread
// and step took 14 us.)
constexpr int kChunks = 32;

__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(Pool p, CompactPlan w, int32_t* live_out) {
  __shared__ int tmp[kPlanThreads / 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // chunks a wave looks at in a step: few pages are spread over all waves
  const int64_t need = (p.num_pages + kPlanThreads - 1) / kPlanThreads;
  const int chunks = need < kChunks ? (int)need : kChunks;
  const int64_t step = (int64_t)kPlanThreads * chunks;
  const bool once = p.num_pages <= step;
  unsigned long long taken = 0;  // lane c: pages in use of the wave's chunk c in this step
  auto look = [&](int64_t i0) {
    const int64_t first = i0 + (int64_t)wave * chunks * 64 + lane;
    taken = 0;
    for (int c0 = 0; c0 < chunks; c0 += 8) {
      int32_t ref[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int64_t i = first + (c0 + c) * 64;
        ref[c] = c0 + c < chunks && i < p.num_pages ? p.refs[i] : 0;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const unsigned long long m = __ballot(ref[c] > 0);
        if (lane == c0 + c) taken = m;
      }
    }
  };
  int all = 0;
  int64_t live = 0, kept = 0;  // pages in use; those of them that stay
  for (int64_t i0 = 0; i0 < p.num_pages; i0 += step) {
    look(i0);
    block_scan(__popcll(taken), tmp, &all);
    live += all;
  }
  for (int64_t i0 = 0; i0 < live; i0 += step) {
    if (!once) look(i0);
    const int64_t below = live - (i0 + ((int64_t)wave * chunks + lane) * 64);  // of the lane's pages
    const unsigned long long in = below >= 64 ? ~0ull : (below > 0 ? (1ull << below) - 1 : 0);
    block_scan(__popcll(taken & in), tmp, &all);
    kept += all;
  }
  const int moves = (int)(live - kept);
  int before = 0;  // pages in use before this step
  for (int64_t i0 = 0; i0 < p.num_pages; i0 += step) {
    if (!once) look(i0);
    const int n = __popcll(taken);
    const int first = before + block_scan(n, tmp, &all) - n;  // and before the lane's pages
    before += all;
    for (int c = 0; c < chunks; ++c) {
      const int64_t i = i0 + ((int64_t)wave * chunks + c) * 64 + lane;
      if (i - lane >= p.num_pages) break;
      const unsigned lo = __builtin_amdgcn_readlane((unsigned)taken, c);
      const unsigned hi = __builtin_amdgcn_readlane((unsigned)(taken >> 32), c);
      // pages in use before page i
      const int rank = __builtin_amdgcn_readlane(first, c) + __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
      if (i >= p.num_pages) continue;
      const bool used = ((lane < 32 ? lo >> lane : hi >> (lane - 32)) & 1) != 0;
      if (i < live) {
        if (!used) w.to[i - rank] = (int32_t)i;
      } else {
        if (used) w.from[rank - kept] = (int32_t)i;
        w.rank[i] = used ? rank - (int)kept : -1;
      }
    }
  }
  if (threadIdx.x == 0) {
    w.count[0] = moves;
    w.count[1] = (int32_t)live;
    if (live_out) *live_out = (int32_t)live;
  }
}

// Blocks [0, tables): every tables-th sequence slot's table row and a part of
// the reference counts (``tables`` is 0 in a call's later launches); the others
// copy pages.
template <typename VecT>
__global__ __launch_bounds__(kThreads) void compact_apply_kernel(Pool p, int64_t tables, CompactPlan w, Stores st) {
  const int64_t moves = w.count[0], live = w.count[1];
  if ((int64_t)blockIdx.x < tables) {
    for (int64_t s = blockIdx.x; s < p.num_seqs; s += tables) {
      int64_t used = used_pages(p.lengths[s], p.page_size);
      if (used > p.max_pages) used = p.max_pages;
      int32_t* row = p.table + s * p.table_stride;
      for (int64_t j = threadIdx.x; j < used; j += kThreads) {
        const int64_t pg = row[j];
        if (pg < live || pg >= p.num_pages) continue;
        const int k = w.rank[pg];
        if (k >= 0) row[j] = w.to[k];
      }
    }
    for (int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x; k < moves; k += tables * kThreads) {
      p.refs[w.to[k]] = p.refs[w.from[k]];
      p.refs[w.from[k]] = 0;
    }
    return;
  }
  const int64_t total = moves * st.per_page;
  for (int64_t it = blockIdx.x - tables; it < total; it += gridDim.x - tables) {
    const int64_t move = it / st.per_page;
    int64_t tile = it - move * st.per_page;
    const int c = store_of(st, &tile);
    copy_tile<VecT>(st, c, tile, w.from[move], w.to[move]);
  }
}

// ---------------------------------------------------------------------------
// free

__global__ __launch_bounds__(kThreads) void free_kernel(Pool p, const uint8_t* release) {
  for (int64_t s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
    if (release[s] == 0) continue;
    int64_t used = used_pages(p.lengths[s], p.page_size);
    if (used > p.max_pages) used = p.max_pages;
    int32_t* row = p.table + s * p.table_stride;
    for (int64_t j = threadIdx.x; j < used; j += kThreads) {
      const int64_t pg = row[j];
      if (pg >= 0 && pg < p.num_pages) atomicAdd(p.refs + pg, -1);  // whole numbers: the order does not matter
      row[j] = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) p.lengths[s] = 0;
  }
}

// ---------------------------------------------------------------------------

Pool pool_of(const kda_page_pool_t& a) {
  return Pool{a.table, a.table_stride, a.num_seqs, a.max_pages, a.lengths, a.refs, a.num_pages, a.page_size};
}

// Up to kMaxStores stores from the ``at``-th, in vectors of ``width`` bytes.
Stores stores_of(const kda_page_store_t* s, int64_t num, int64_t at, int width) {
  Stores st;
  st.n = 0;
  st.per_page = 0;
  for (int64_t i = at; i < num && st.n < kMaxStores; ++i, ++st.n) {
    st.data[st.n] = static_cast<char*>(s[i].data);
    st.stride[st.n] = s[i].page_stride;
    st.vecs[st.n] = s[i].page_bytes / width;
    st.tiles[st.n] = (st.vecs[st.n] + kThreads * kUnroll - 1) / (kThreads * kUnroll);
    st.per_page += st.tiles[st.n];
  }
  return st;
}

// Widest vector (16, 4 or 1 bytes) all the stores' pages are aligned to.
int width_of(const kda_page_store_t* s, int64_t num) {
  uint64_t a = 0;
  for (int64_t i = 0; i < num; ++i)
    a |= (uint64_t)(uintptr_t)s[i].data | (uint64_t)s[i].page_stride | (uint64_t)s[i].page_bytes;
  return (a & 15) == 0 ? 16 : ((a & 3) == 0 ? 4 : 1);
}

int64_t copy_blocks(int64_t most_moves, int64_t per_page) {
  const int64_t most = 8192;
  if (per_page == 0 || most_moves == 0) return 0;
  return most_moves > most / per_page ? most : most_moves * per_page;
}

template <typename IdxT>
hipError_t fork_typed(const kda_page_pool_t& a, const kda_page_store_t* stores, int64_t num_stores, const void* src,
                      const void* dst, int64_t M, bool share, int32_t* status, const ForkPlan& w, int64_t most,
                      hipStream_t stream) {
  const Pool p = pool_of(a);
  const IdxT *s = static_cast<const IdxT*>(src), *d = static_cast<const IdxT*>(dst);
  hipError_t e = hipSuccess;
  if (M > kFew) {
    hipLaunchKernelGGL((fork_check_kernel<IdxT>), dim3((unsigned)M), dim3(kThreads), 0, stream, p, s, d, share ? 1 : 0,
                       w);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((fork_plan_kernel<IdxT>), dim3(1), dim3(kPlanThreads), 0, stream, p, s, d, M, share ? 1 : 0,
                     status, w);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int width = width_of(stores, num_stores);
  int64_t at = 0, tables = M;
  do {
    const Stores st = stores_of(stores, num_stores, at, width);
    const dim3 grid((unsigned)(tables + copy_blocks(most, st.per_page)));
    if (width == 16)
      hipLaunchKernelGGL((fork_apply_kernel<u32x4, IdxT>), grid, dim3(kThreads), 0, stream, p, s, d, M, tables, w, st);
    else if (width == 4)
      hipLaunchKernelGGL((fork_apply_kernel<unsigned, IdxT>), grid, dim3(kThreads), 0, stream, p, s, d, M, tables, w,
                         st);
    else
      hipLaunchKernelGGL((fork_apply_kernel<unsigned char, IdxT>), grid, dim3(kThreads), 0, stream, p, s, d, M, tables,
                         w, st);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    at += kMaxStores;
    tables = 0;
  } while (at < num_stores);
  return hipSuccess;
}

int64_t fork_most(int64_t M, int64_t max_pages, int64_t num_pages, bool share) {
  const int64_t asked = share ? M : (M > num_pages / max_pages ? num_pages : M * max_pages);
  return asked < num_pages ? asked : num_pages;
}

}  // namespace

size_t page_fork_workspace_bytes(int64_t M, int64_t max_pages, int64_t num_pages, bool share) {
  return (size_t)(3 * M + 1 + fork_most(M, max_pages, num_pages, share)) * 4;
}

hipError_t launch_page_fork(const kda_page_pool_t& a, const kda_page_store_t* stores, int64_t num_stores,
                            const void* src, const void* dst, bool index64, int64_t M, bool share, int32_t* status,
                            void* workspace, hipStream_t stream) {
  int32_t* ws = static_cast<int32_t*>(workspace);
  const ForkPlan w{ws, ws + M, ws + 2 * M, ws + 3 * M, ws + 3 * M + 1};
  const int64_t most = fork_most(M, a.max_pages, a.num_pages, share);
  if (index64)
    return fork_typed<int64_t>(a, stores, num_stores, src, dst, M, share, status, w, most, stream);
  return fork_typed<int32_t>(a, stores, num_stores, src, dst, M, share, status, w, most, stream);
}

size_t page_compact_workspace_bytes(int64_t num_pages) { return (size_t)(2 + num_pages + 2 * (num_pages / 2)) * 4; }

hipError_t launch_page_compact(const kda_page_pool_t& a, const kda_page_store_t* stores, int64_t num_stores,
                               int32_t* live, void* workspace, hipStream_t stream) {
  const Pool p = pool_of(a);
  int32_t* ws = static_cast<int32_t*>(workspace);
  const CompactPlan w{ws + 2, ws + 2 + a.num_pages, ws + 2 + a.num_pages + a.num_pages / 2, ws};
  hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p, w, live);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int width = width_of(stores, num_stores);
  int64_t at = 0, tables = a.num_seqs < kMostTables ? a.num_seqs : kMostTables;
  do {
    const Stores st = stores_of(stores, num_stores, at, width);
    const dim3 grid((unsigned)(tables + copy_blocks(a.num_pages / 2, st.per_page)));
    if (grid.x > 0) {
      if (width == 16)
        hipLaunchKernelGGL((compact_apply_kernel<u32x4>), grid, dim3(kThreads), 0, stream, p, tables, w, st);
      else if (width == 4)
        hipLaunchKernelGGL((compact_apply_kernel<unsigned>), grid, dim3(kThreads), 0, stream, p, tables, w, st);
      else
        hipLaunchKernelGGL((compact_apply_kernel<unsigned char>), grid, dim3(kThreads), 0, stream, p, tables, w, st);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    at += kMaxStores;
    tables = 0;
  } while (at < num_stores);
  return hipSuccess;
}

hipError_t launch_page_free(const kda_page_pool_t& a, const uint8_t* release, hipStream_t stream) {
  const int64_t blocks = a.num_seqs < kMostTables ? a.num_seqs : kMostTables;
  hipLaunchKernelGGL(free_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, pool_of(a), release);
  return hipGetLastError();
}

}  // namespace kda
