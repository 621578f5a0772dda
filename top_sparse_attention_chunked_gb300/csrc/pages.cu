// Page management for the paged caches: which row of the block table holds
// which block, how often, and moving the blocks' contents when they change
// hands.
//
// The state is a table [rows, W] of block indices and a reference count per
// block; free means count 0. There is no free list: the free blocks are found
// by scanning the counts, so the new state is a function of the old one alone
// (lowest index first), whatever the order in which the threads run.
//
// dsa_pages_update, four launches (steps 1 to 3 in one where one block does them):
//   1. the scratch (count changes, writers per block, a flag) is cleared;
//   2. pages_count_kernel, one thread per table entry: the entry's old block
//      loses a holder, the block it takes from its parent row gains one (an
//      entry that keeps its block touches nothing); the entry of a partly
//      filled last block that its row will write into registers as a writer
//      of that block. The sums are integer atomics: any order, same result.
//   3. pages_plan_kernel, one block of 1,024 threads: a row copies its last
//      block unless all holders are writers and it is the lowest of them;
//      prefix sums over the rows give every row its place in the list of free
//      blocks, and a walk over the counts (a slice of the blocks per warp,
//      ballots for the rank) writes that list and the new counts;
//   4. pages_commit_kernel: the new table, and the copies of the blocks.
// The new table goes through the workspace (rows trade places in it), so the
// call can work in place. Nothing of the old state is written before step 3
// knows that all of it can be done.
//
// dsa_pages_compact: a check of the entries, a plan (the holes below the live
// count and the live blocks above it, both ascending, are paired), a commit.
//
// Copies: the bytes are read once and written once, in 32 KB pieces of one
// block of one pool a thread block, eight 16-byte loads a thread in flight:
// 580 MB (290 read, 290 written) in 100 us, 5.8 TB/s of 6.8 measured.
//
// Without copies the time is launches and one block's walk: 16 x 32 entries of
// 1,024 blocks 6.0 us, 256 x 256 of 8,192 9.5 us; 65,536 blocks 25 us (the walk
// reads 1.3 MB through one SM; a plan by many blocks would need two launches
// more, which costs what it gains below some 40,000 blocks).
#include <algorithm>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kPgThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kCopyUnroll = 8;
// States that one block counts by itself, sums in shared memory: up to this many
// table entries and blocks (one block / many, of 1,024 blocks with 512 entries:
// 5.6 / 6.8 us; 8,192 blocks with 4,096 entries 10.2 / 10.2, 8,192 entries 12.5 /
// 10.0).
constexpr int kSmallEntries = 4096, kSmallBlocks = 8192;
// Times 32 blocks that a warp of a plan kernel looks at together: many keep loads
// in flight, few keep the code short, which is what a small state's time goes on
// (8 and 2 in a small state: 7.6 and 6.0 us; 65,536 blocks with 4 and 8, the loads
// before the first store: 25.8 and 25.0, one at a time 43.8).
constexpr int kWalkSmall = 2, kWalkLarge = 8;
constexpr long long kPiece = kPgThreads * 16LL * kCopyUnroll;   // bytes of one copy task

struct PageDims {
  int rows, W, nb, shift;
};

struct PoolList {
  uint8_t* base[DSA_MAX_POOLS];
  long long bytes[DSA_MAX_POOLS];
  int first[DSA_MAX_POOLS + 1];   // first task of each pool within one block's
  int n;
};

// Workspace: the status word (written by the plan kernels), then what is
// cleared (flag, delta, writers, low), then the rest.
struct PageWs {
  uint32_t* status;
  uint32_t* flag;        // an argument or entry out of range was seen
  int32_t* delta;        // change of each block's count
  int32_t* writers;      // rows that will write into the block (their last one)
  int32_t* low;          // rows - (lowest of those rows)
  int32_t* stage;        // [rows, W] blocks taken over from the parents
  int32_t* from;         // [rows] first entry that gets a fresh block
  int32_t* off;          // [rows] its place in the list of free blocks
  int32_t* copy_row;     // [rows] rows whose last block is copied
  int32_t* head;         // {copies, fresh blocks}
  int32_t* free_ids;     // [nb] free blocks, ascending (compact: the holes)
  int32_t* movers;       // [nb] compact: the blocks that move
  int32_t* remap;        // [nb] compact
  size_t zero_bytes, total;
};

PageWs page_ws(void* base, const PageDims& d) {
  PageWs w;
  size_t o = 256;
  const auto take = [&](size_t n) {
    int32_t* p = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(base) + o);
    o += (n * 4 + 255) & ~size_t(255);
    return p;
  };
  w.status = static_cast<uint32_t*>(base);
  w.flag = reinterpret_cast<uint32_t*>(take(1));
  w.delta = take(d.nb);
  w.writers = take(d.nb);
  w.low = take(d.nb);
  w.zero_bytes = o - 256;
  w.stage = take(static_cast<size_t>(d.rows) * d.W);
  w.from = take(d.rows);
  w.off = take(d.rows);
  w.copy_row = take(d.rows);
  w.head = take(2);
  w.free_ids = take(d.nb);
  w.movers = take(d.nb);
  w.remap = take(d.nb);
  w.total = o;
  return w;
}

__device__ __forceinline__ int ceil_shift(int n, int shift) {
  return static_cast<int>((static_cast<long long>(n) + (1LL << shift) - 1) >> shift);
}

// ------------------------------------------------------------------ update
// What the count step adds up, in the workspace or (small states) in shared
// memory.
struct Counts {
  uint32_t* flag;
  int32_t* delta;
  int32_t* writers;
  int32_t* low;
};

struct Rows {   // the caller's row arguments
  const int32_t* __restrict__ parent;
  const int32_t* __restrict__ keep_len;
  const int32_t* __restrict__ new_len;
  const int32_t* __restrict__ first_key;
};

// Table entry e.
__device__ __forceinline__ void count_entry(const PageDims& d, const Counts& c, int32_t* stage, const Rows& a,
                                            const int32_t* __restrict__ table, int e) {
  const int most = d.W << d.shift;   // (below 2^31, checked)
  const int r = e / d.W, j = e - r * d.W;
  const int old = table[e];
  const int p = a.parent[r], keep = a.keep_len[r], grown = a.new_len[r];
  const int drop = a.first_key ? a.first_key[r] : 0;
  bool bad = old >= d.nb || p < -1 || p >= d.rows || keep < 0 || grown < keep || grown > most ||
             (p < 0 && keep != 0) || drop < 0 || drop > keep;
  int got = -1;
  if (!bad) {
    const int kept = ceil_shift(keep, d.shift);
    if (j < kept && j >= (drop >> d.shift)) {
      got = p == r ? old : table[p * d.W + j];
      if (got < 0) got = -1;
      if (got >= d.nb) {
        bad = true;
        got = -1;
      }
    }
    if (j == kept - 1 && grown > keep && (keep & ((1 << d.shift) - 1)) != 0) {
      if (got < 0) {
        bad = true;            // nothing there to write into
      } else {
        atomicAdd(c.writers + got, 1);
        atomicMax(c.low + got, d.rows - r);
      }
    }
  }
  stage[e] = got;
  if (bad) *c.flag = 1u;
  if (old != got) {
    if (old >= 0 && old < d.nb) atomicAdd(c.delta + old, -1);
    if (got >= 0) atomicAdd(c.delta + got, 1);
  }
}

__global__ void __launch_bounds__(kPgThreads)
    pages_count_kernel(const PageDims d, const PageWs w, const Rows a, const int32_t* __restrict__ table) {
  pdl_wait();   // the cleared scratch
  const Counts c{w.flag, w.delta, w.writers, w.low};
  const int n = d.rows * d.W;
  for (int e = blockIdx.x * kPgThreads + threadIdx.x; e < n; e += gridDim.x * kPgThreads)
    count_entry(d, c, w.stage, a, table, e);
}

// The calling warp's slice of the blocks.
__device__ __forceinline__ void warp_slice(int nb, int* lo, int* hi) {
  const int warps = kPlanThreads / 32, wid = threadIdx.x >> 5;
  const int per = ((nb + warps - 1) / warps + 31) & ~31;
  *lo = min(nb, wid * per);
  *hi = min(nb, *lo + per);
}

// Exclusive prefix of one value per warp over the block's warps, and the sum.
// Every thread calls it with its warp's value.
__device__ __forceinline__ int warp_prefix(int v, int* tot, int* sum) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) tot[wid] = v;
  __syncthreads();
  int x = tot[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  *sum = __shfl_sync(0xffffffffu, x, 31);
  return __shfl_sync(0xffffffffu, x, wid) - v;
}

// One block: the rows' copies and fresh blocks, the list of free blocks, the
// new counts.
template <int WALK>
__device__ __forceinline__ void plan_update(const PageDims& d, const PageWs& w, const Counts& c, const Rows& a,
                                            const int32_t* refs, int32_t* refs_out, int32_t* counts) {
  __shared__ uint32_t scan_tot[32];
  __shared__ int warp_tot[32];
  const int lane = threadIdx.x & 31;
  const bool bad = *c.flag != 0;
  bool fail = bad;
  // rows: who copies, how many blocks each wants, where its share begins
  uint32_t wanted = 0, copies = 0;   // so far
  for (int r0 = 0; r0 < d.rows; r0 += kPlanThreads) {
    const int r = r0 + static_cast<int>(threadIdx.x);
    uint32_t want = 0, copy = 0;
    int from = 0;
    if (r < d.rows && !fail) {
      const int keep = a.keep_len[r], grown = a.new_len[r];
      const int kept = ceil_shift(keep, d.shift);
      if (grown > keep && (keep & ((1 << d.shift) - 1)) != 0) {
        const int t = w.stage[r * d.W + kept - 1];
        const int n = c.writers[t];
        copy = !(refs[t] + c.delta[t] == n && d.rows - c.low[t] == r);
      }
      from = kept - static_cast<int>(copy);
      want = static_cast<uint32_t>(ceil_shift(grown, d.shift) - from);
    }
    uint32_t sum_w, sum_c;
    const uint32_t off = block_exclusive_scan<kPlanThreads>(want, scan_tot, &sum_w);
    const uint32_t pos = block_exclusive_scan<kPlanThreads>(copy, scan_tot, &sum_c);
    if (r < d.rows) {
      w.from[r] = from;
      w.off[r] = static_cast<int>(wanted + off);
      if (copy) w.copy_row[copies + pos] = r;
    }
    wanted += sum_w;
    copies += sum_c;
  }
  // blocks: the free ones, in order
  int lo, hi;
  warp_slice(d.nb, &lo, &hi);
  int mine = 0, mine_before = 0;   // free after / before the releases
  for (int b = lo; b < hi; b += 32 * WALK) {
    int r[WALK], n[WALK];
#pragma unroll
    for (int i = 0; i < WALK; ++i) {
      const int id = b + 32 * i + lane;
      r[i] = id < hi ? refs[id] : 1;
      n[i] = id < hi ? r[i] + c.delta[id] : 1;
    }
#pragma unroll
    for (int i = 0; i < WALK; ++i) {
      mine += __popc(__ballot_sync(0xffffffffu, n[i] == 0));
      mine_before += __popc(__ballot_sync(0xffffffffu, r[i] == 0));
    }
  }
  int nfree, nbefore;
  int rank = warp_prefix(mine, warp_tot, &nfree);
  warp_prefix(mine_before, warp_tot, &nbefore);
  if (wanted > static_cast<uint32_t>(nfree)) fail = true;
  for (int b = lo; b < hi; b += 32 * WALK) {
    int old[WALK], n[WALK], wr[WALK];   // (all read first: refs_out may be refs)
#pragma unroll
    for (int i = 0; i < WALK; ++i) {
      const int id = b + 32 * i + lane;
      old[i] = id < hi ? refs[id] : 1;
      n[i] = id < hi ? old[i] + c.delta[id] : 1;
      wr[i] = id < hi ? c.writers[id] : 0;
    }
#pragma unroll
    for (int i = 0; i < WALK; ++i) {
      const int id = b + 32 * i + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, n[i] == 0);
      if (n[i] == 0) {
        const int k = rank + __popc(m & ((1u << lane) - 1u));
        w.free_ids[k] = id;
        if (k < static_cast<int>(wanted)) n[i] = 1;
      } else {
        // its writers that copy let go of it
        n[i] -= wr[i] - (wr[i] > 0 && n[i] == wr[i] ? 1 : 0);
      }
      rank += __popc(m);
      if (id < hi) refs_out[id] = fail ? old[i] : n[i];
    }
  }
  if (threadIdx.x == 0) {
    *w.status = bad ? kDevBadState : fail ? kDevNoPages : 0u;
    w.head[0] = fail ? -1 : static_cast<int>(copies);
    w.head[1] = static_cast<int>(wanted);
    if (counts) {
      counts[0] = fail ? -1 : static_cast<int>(copies);
      counts[1] = fail ? nbefore : nfree - static_cast<int>(wanted);
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads, 1)
    pages_plan_kernel(const PageDims d, const PageWs w, const Rows a, const int32_t* refs, int32_t* refs_out,
                      int32_t* counts) {
  pdl_wait();
  plan_update<kWalkLarge>(d, w, Counts{w.flag, w.delta, w.writers, w.low}, a, refs, refs_out, counts);
}

// Small states: the count and the plan in one block, the sums in shared memory
// (cleared here). One launch in place of three.
__global__ void __launch_bounds__(kPlanThreads, 1)
    pages_small_kernel(const PageDims d, const PageWs w, const Rows a, const int32_t* __restrict__ table,
                       const int32_t* refs, int32_t* refs_out, int32_t* counts) {
  extern __shared__ int32_t sums[];   // 3 * nb + 1
  const Counts c{reinterpret_cast<uint32_t*>(sums + 3 * d.nb), sums, sums + d.nb, sums + 2 * d.nb};
  pdl_trigger();
  for (int i = threadIdx.x; i <= 3 * d.nb; i += kPlanThreads) sums[i] = 0;
  __syncthreads();
  const int n = d.rows * d.W;
  for (int e = threadIdx.x; e < n; e += kPlanThreads) count_entry(d, c, w.stage, a, table, e);
  __syncthreads();
  plan_update<kWalkSmall>(d, w, c, a, refs, refs_out, counts);
}

// Copy task t of `src` -> `dst` in every pool: one piece of one pool's block.
__device__ __forceinline__ void copy_piece(const PoolList& pools, int t, int src, int dst) {
  int lo = 0, hi = pools.n;   // the pool whose tasks hold t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pools.first[mid] <= t) lo = mid;
    else hi = mid;
  }
  const long long bytes = pools.bytes[lo];
  const long long at = static_cast<long long>(t - pools.first[lo]) * kPiece;
  const uint8_t* s = pools.base[lo] + src * bytes + at;
  uint8_t* o = pools.base[lo] + dst * bytes + at;
  const long long left = bytes - at;
  uint4 u[kCopyUnroll];
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i) {
    const long long x = (static_cast<long long>(i) * kPgThreads + threadIdx.x) * 16;
    if (x < left) u[i] = *reinterpret_cast<const uint4*>(s + x);
  }
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i) {
    const long long x = (static_cast<long long>(i) * kPgThreads + threadIdx.x) * 16;
    if (x < left) *reinterpret_cast<uint4*>(o + x) = u[i];
  }
}

__global__ void __launch_bounds__(kPgThreads)
    pages_commit_kernel(const PageDims d, const PageWs w, const __grid_constant__ PoolList pools,
                        const int32_t* table, const int32_t* __restrict__ new_len, int32_t* table_out) {
  pdl_wait();
  const int copies = w.head[0];
  const int n = d.rows * d.W;
  if (copies < 0) {   // refused: the new table is the old one
    if (table_out != table)
      for (int e = blockIdx.x * kPgThreads + threadIdx.x; e < n; e += gridDim.x * kPgThreads) table_out[e] = table[e];
    return;
  }
  for (int e = blockIdx.x * kPgThreads + threadIdx.x; e < n; e += gridDim.x * kPgThreads) {
    const int r = e / d.W, j = e - r * d.W;
    const int from = w.from[r];
    int v = -1;
    if (j < from) v = w.stage[e];
    else if (j < ceil_shift(new_len[r], d.shift)) v = w.free_ids[w.off[r] + j - from];
    table_out[e] = v;
  }
  const int per = pools.first[pools.n];
  const long long tasks = static_cast<long long>(copies) * per;
  for (long long t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int c = static_cast<int>(t / per);
    const int r = w.copy_row[c];
    const int src = w.stage[r * d.W + w.from[r]];
    copy_piece(pools, static_cast<int>(t - static_cast<long long>(c) * per), src, w.free_ids[w.off[r]]);
  }
}

// ----------------------------------------------------------------- compact
__device__ __forceinline__ bool bad_entry(const PageDims& d, int x, const int32_t* __restrict__ refs) {
  return x >= 0 && (x >= d.nb || refs[x] <= 0);
}

__global__ void __launch_bounds__(kPgThreads)
    pages_check_kernel(const PageDims d, const PageWs w, const int32_t* __restrict__ table,
                       const int32_t* __restrict__ refs) {
  pdl_wait();   // the cleared flag
  const int n = d.rows * d.W;
  for (int e = blockIdx.x * kPgThreads + threadIdx.x; e < n; e += gridDim.x * kPgThreads)
    if (bad_entry(d, table[e], refs)) *w.flag = 1u;
}

// `table` is given where the block checks the entries itself (small states).
template <int WALK>
__global__ void __launch_bounds__(kPlanThreads, 1)
    compact_plan_kernel(const PageDims d, const PageWs w, const int32_t* table, const int32_t* refs,
                        int32_t* refs_out, int32_t* remap_out, int32_t* counts) {
  __shared__ int warp_tot[32];
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  bool fail = false;
  if (table) {
    for (int e = threadIdx.x; e < d.rows * d.W; e += kPlanThreads) fail = fail || bad_entry(d, table[e], refs);
    fail = __syncthreads_or(fail);
  } else {
    pdl_wait();
    fail = *w.flag != 0;
  }
  int lo, hi;
  warp_slice(d.nb, &lo, &hi);
  // live blocks of the warp's slice below `end`
  const auto count_live = [&](int end) {
    int n = 0;
    for (int b = lo; b < end; b += 32 * WALK) {
      bool used[WALK];
#pragma unroll
      for (int i = 0; i < WALK; ++i) {
        const int id = b + 32 * i + lane;
        used[i] = id < end && refs[id] > 0;
      }
#pragma unroll
      for (int i = 0; i < WALK; ++i) n += __popc(__ballot_sync(0xffffffffu, used[i]));
    }
    return n;
  };
  const int mine = count_live(hi);
  int live;
  const int before = warp_prefix(mine, warp_tot, &live);
  // k-th hole below `live`, k-th live block from `live` on: there are as many
  // of either. With x live blocks before block b, b - x free ones are.
  int x = before;
  const int high = count_live(min(hi, live));   // live blocks below `live`
  int below;
  warp_prefix(high, warp_tot, &below);
  for (int b = lo; b < hi; b += 32 * WALK) {
    bool used[WALK];
#pragma unroll
    for (int i = 0; i < WALK; ++i) {
      const int id = b + 32 * i + lane;
      used[i] = id < hi && refs[id] > 0;
    }
#pragma unroll
    for (int i = 0; i < WALK; ++i) {
      const int id = b + 32 * i + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, used[i]);
      const int rank = x + __popc(m & ((1u << lane) - 1u));   // live blocks before this one
      x += __popc(m);
      if (id >= hi) continue;
      const int to = used[i] ? id : -1;
      if (!fail) {
        if (!used[i] && id < live) w.free_ids[id - rank] = id;
        if (used[i] && id >= live) w.movers[rank - below] = id;
      }
      w.remap[id] = to;
      if (remap_out) remap_out[id] = to;
    }
  }
  const int moves = fail ? 0 : live - below;
  __syncthreads();   // the lists are complete (block-wide visibility of global writes)
  for (int k = threadIdx.x; k < moves; k += kPlanThreads) {
    const int from = w.movers[k], to = w.free_ids[k];
    w.remap[from] = to;
    if (remap_out) remap_out[from] = to;
  }
  // counts: the holes take their mover's, everything from `live` on is free
  for (int k = threadIdx.x; k < moves; k += kPlanThreads) refs_out[w.free_ids[k]] = refs[w.movers[k]];
  if (refs_out != refs)
    for (int b = threadIdx.x; b < d.nb; b += kPlanThreads) {
      const int r = refs[b];
      if (fail || (b < live && r > 0)) refs_out[b] = r;
    }
  __syncthreads();
  if (!fail)
    for (int b = live + static_cast<int>(threadIdx.x); b < d.nb; b += kPlanThreads) refs_out[b] = 0;
  if (threadIdx.x == 0) {
    *w.status = fail ? kDevBadState : 0u;
    w.head[0] = fail ? -1 : moves;
    if (counts) {
      counts[0] = fail ? -1 : moves;
      counts[1] = d.nb - live;
    }
  }
}

__global__ void __launch_bounds__(kPgThreads)
    compact_commit_kernel(const PageDims d, const PageWs w, const __grid_constant__ PoolList pools,
                          const int32_t* table, int32_t* table_out) {
  pdl_wait();
  const int moves = w.head[0];
  const int n = d.rows * d.W;
  if (moves >= 0 || table_out != table)
    for (int e = blockIdx.x * kPgThreads + threadIdx.x; e < n; e += gridDim.x * kPgThreads) {
      const int x = table[e];
      table_out[e] = moves < 0 || x < 0 ? x : w.remap[x];
    }
  if (moves <= 0) return;
  const int per = pools.first[pools.n];
  const long long tasks = static_cast<long long>(moves) * per;
  for (long long t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int c = static_cast<int>(t / per);
    copy_piece(pools, static_cast<int>(t - static_cast<long long>(c) * per), w.movers[c], w.free_ids[c]);
  }
}

// -------------------------------------------------------------------- host
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

int check_state(const dsa_page_state* st, PageDims* d) {
  if (!st) return report_error(DSA_ERR_INVALID_ARG, "page state is NULL");
  const int bs = st->block_size;
  if (bs < 128 || bs > (1 << 20) || (bs & (bs - 1)) != 0)
    return report_errorf(DSA_ERR_UNSUPPORTED, "block_size %d must be a power of two from 128 to 2^20", bs);
  if (st->num_blocks < 1 || st->num_blocks > (1 << 24))
    return report_errorf(DSA_ERR_INVALID_ARG, "num_blocks %d outside 1..2^24", st->num_blocks);
  if (st->rows < 1 || st->rows > 4096)
    return report_errorf(DSA_ERR_INVALID_ARG, "rows %d outside 1..4096", st->rows);
  if (st->blocks_per_seq < 1 || static_cast<long long>(st->rows) * st->blocks_per_seq > (1LL << 26) ||
      static_cast<long long>(st->blocks_per_seq) * bs > 0x7fffffffLL)
    return report_errorf(DSA_ERR_INVALID_ARG, "blocks_per_seq %d: rows * blocks_per_seq must be in 1..2^26 "
                         "and blocks_per_seq * block_size below 2^31", st->blocks_per_seq);
  d->rows = st->rows;
  d->W = st->blocks_per_seq;
  d->nb = st->num_blocks;
  d->shift = 0;
  while ((1 << d->shift) < bs) ++d->shift;
  return DSA_OK;
}

// What both calls check of the state's arrays, the pools and the workspace.
int check_common(const dsa_page_state* st, const PageDims& d, int num_pools, const dsa_page_pool* pools,
                 const int32_t* table_out, const int32_t* refs_out, const void* ws, size_t ws_bytes,
                 PoolList* list) {
  if (!st->block_table || !st->refs || !table_out || !refs_out)
    return report_error(DSA_ERR_INVALID_ARG, "a table or reference count pointer is NULL");
  if (!al4(st->block_table) || !al4(st->refs) || !al4(table_out) || !al4(refs_out))
    return report_error(DSA_ERR_MISALIGNED, "tables and reference counts must be 4-byte aligned");
  const long long tb = 4LL * d.rows * d.W, rb = 4LL * d.nb;
  if ((table_out != st->block_table && overlap(table_out, tb, st->block_table, tb)) ||
      (refs_out != st->refs && overlap(refs_out, rb, st->refs, rb)) ||
      overlap(table_out, tb, st->refs, rb) || overlap(refs_out, rb, st->block_table, tb) ||
      overlap(table_out, tb, refs_out, rb))
    return report_error(DSA_ERR_INVALID_ARG, "the new state must be the old one's arrays or overlap none of them");
  if (num_pools < 0 || num_pools > DSA_MAX_POOLS)
    return report_errorf(DSA_ERR_INVALID_ARG, "num_pools %d outside 0..%d", num_pools, DSA_MAX_POOLS);
  if (num_pools > 0 && !pools) return report_error(DSA_ERR_INVALID_ARG, "pools is NULL");
  long long first = 0;
  for (int i = 0; i < num_pools; ++i) {
    if (!pools[i].base) return report_errorf(DSA_ERR_INVALID_ARG, "pool %d has no base", i);
    if ((reinterpret_cast<uintptr_t>(pools[i].base) & 15) || pools[i].block_bytes % 16 != 0)
      return report_errorf(DSA_ERR_MISALIGNED, "pool %d: base and block_bytes must be multiples of 16", i);
    if (pools[i].block_bytes < 16 || pools[i].block_bytes > (1LL << 36))
      return report_errorf(DSA_ERR_INVALID_ARG, "pool %d: block_bytes outside 16..2^36", i);
    const long long bytes = pools[i].block_bytes * d.nb;
    if (overlap(pools[i].base, bytes, st->block_table, tb) || overlap(pools[i].base, bytes, st->refs, rb) ||
        overlap(pools[i].base, bytes, table_out, tb) || overlap(pools[i].base, bytes, refs_out, rb))
      return report_errorf(DSA_ERR_INVALID_ARG, "pool %d overlaps the page state", i);
    for (int k = 0; k < i; ++k)
      if (overlap(pools[i].base, bytes, pools[k].base, pools[k].block_bytes * d.nb))
        return report_errorf(DSA_ERR_INVALID_ARG, "pools %d and %d overlap", k, i);
    list->base[i] = static_cast<uint8_t*>(pools[i].base);
    list->bytes[i] = pools[i].block_bytes;
    list->first[i] = static_cast<int>(first);
    first += (pools[i].block_bytes + kPiece - 1) / kPiece;
    if (first > 0x7fffffffLL) return report_error(DSA_ERR_UNSUPPORTED, "a block holds too many bytes over all pools");
  }
  list->first[num_pools] = static_cast<int>(first);
  list->n = num_pools;
  return check_call_workspace(ws, ws_bytes, page_ws(nullptr, d).total);
}

// Whether a call's further array overlaps what the call writes: the new page
// state and the pools.
bool over_written(const void* x, long long bytes, const PageDims& d, const int32_t* table_out, const int32_t* refs_out,
                  const PoolList& pools) {
  if (!x) return false;
  bool over = overlap(x, bytes, table_out, 4LL * d.rows * d.W) || overlap(x, bytes, refs_out, 4LL * d.nb);
  for (int i = 0; i < pools.n; ++i) over = over || overlap(x, bytes, pools.base[i], pools.bytes[i] * d.nb);
  return over;
}
// The same for an array that the call writes: nor may it lie over the old state.
bool over_state(const void* x, long long bytes, const dsa_page_state* st, const PageDims& d, const int32_t* table_out,
                const int32_t* refs_out, const PoolList& pools) {
  return over_written(x, bytes, d, table_out, refs_out, pools) ||
         (x && (overlap(x, bytes, st->block_table, 4LL * d.rows * d.W) || overlap(x, bytes, st->refs, 4LL * d.nb)));
}

bool small_state(const PageDims& d) { return d.rows * d.W <= kSmallEntries && d.nb <= kSmallBlocks; }

unsigned entry_grid(const PageDims& d, int sms) {
  const long long n = (static_cast<long long>(d.rows) * d.W + kPgThreads - 1) / kPgThreads;
  return static_cast<unsigned>(std::min<long long>(n, 8LL * sms));
}

// The commit's grid: enough for the table, and for the copies that may come
// (how many is known on the device only).
unsigned commit_grid(const PageDims& d, int sms, const PoolList& pools, long long copies_bound) {
  const long long tasks = std::min<long long>(copies_bound * pools.first[pools.n], 8LL * sms);
  return static_cast<unsigned>(std::max<long long>(entry_grid(d, sms), tasks));
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return DSA_OK;
  return report_errorf(DSA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_pages_workspace_size(const dsa_page_state* st) {
  PageDims d;
  if (check_state(st, &d)) return 0;
  return page_ws(nullptr, d).total;
}

extern "C" int dsa_pages_update(const dsa_page_state* st, const int32_t* parent, const int32_t* keep_len,
                                const int32_t* new_len, const int32_t* first_key, int num_pools,
                                const dsa_page_pool* pools, int32_t* table_out, int32_t* refs_out,
                                int32_t* counts, void* ws, size_t ws_bytes, void* stream) {
  reset_launches();
  PageDims d;
  PoolList list;
  if (int rc = check_state(st, &d)) return rc;
  if (!parent || !keep_len || !new_len)
    return report_error(DSA_ERR_INVALID_ARG, "parent, keep_len and new_len are required");
  if (!al4(parent) || !al4(keep_len) || !al4(new_len) || !al4(first_key) || !al4(counts))
    return report_error(DSA_ERR_MISALIGNED, "parent, lengths and counts must be 4-byte aligned");
  if (int rc = check_common(st, d, num_pools, pools, table_out, refs_out, ws, ws_bytes, &list)) return rc;
  for (const int32_t* in : {parent, keep_len, new_len, first_key})
    if (over_written(in, 4LL * d.rows, d, table_out, refs_out, list) ||
        (in && counts && overlap(in, 4LL * d.rows, counts, 8)))
      return report_error(DSA_ERR_INVALID_ARG, "parent and lengths must not overlap the new page state, a pool or counts");
  if (over_state(counts, 8, st, d, table_out, refs_out, list))
    return report_error(DSA_ERR_INVALID_ARG, "counts must not overlap the page state or a pool");
  int sms = 0;
  if (int rc = current_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const PageWs w = page_ws(ws, d);
  const Rows rows{parent, keep_len, new_len, first_key};
  cudaError_t e;
  if (small_state(d)) {
    const int smem = (3 * d.nb + 1) * 4;
    e = set_max_smem(reinterpret_cast<const void*>(pages_small_kernel), (3 * kSmallBlocks + 1) * 4);
    if (e == cudaSuccess)
      e = launch_kernel("pages_small_kernel", pages_small_kernel, dim3(1), dim3(kPlanThreads), smem, s, false, d, w, rows,
                        st->block_table, st->refs, refs_out, counts);
  } else {
    e = launch_zero_scratch(w.flag, w.zero_bytes, s);
    if (e == cudaSuccess)
      e = launch_kernel("pages_count_kernel", pages_count_kernel, dim3(entry_grid(d, sms)), dim3(kPgThreads), 0, s, true,
                        d, w, rows, st->block_table);
    if (e == cudaSuccess)
      e = launch_kernel("pages_plan_kernel", pages_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, true, d, w, rows,
                        st->refs, refs_out, counts);
  }
  if (e == cudaSuccess)
    e = launch_kernel("pages_commit_kernel", pages_commit_kernel, dim3(commit_grid(d, sms, list, d.rows)),
                      dim3(kPgThreads), 0, s, true, d, w, list, st->block_table, new_len, table_out);
  return launched(e, "pages_update");
}

extern "C" int dsa_pages_compact(const dsa_page_state* st, int num_pools, const dsa_page_pool* pools,
                                 int32_t* table_out, int32_t* refs_out, int32_t* remap, int32_t* counts,
                                 void* ws, size_t ws_bytes, void* stream) {
  reset_launches();
  PageDims d;
  PoolList list;
  if (int rc = check_state(st, &d)) return rc;
  if (!al4(remap) || !al4(counts)) return report_error(DSA_ERR_MISALIGNED, "remap and counts must be 4-byte aligned");
  if (int rc = check_common(st, d, num_pools, pools, table_out, refs_out, ws, ws_bytes, &list)) return rc;
  if (over_state(remap, 4LL * d.nb, st, d, table_out, refs_out, list) || over_state(counts, 8, st, d, table_out, refs_out, list) ||
      (remap && counts && overlap(remap, 4LL * d.nb, counts, 8)))
    return report_error(DSA_ERR_INVALID_ARG, "remap and counts must not overlap each other, the page state or a pool");
  int sms = 0;
  if (int rc = current_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const PageWs w = page_ws(ws, d);
  cudaError_t e = cudaSuccess;
  const bool small = small_state(d);
  if (!small) {
    e = launch_zero_scratch(w.flag, 256, s);
    if (e == cudaSuccess)
      e = launch_kernel("pages_check_kernel", pages_check_kernel, dim3(entry_grid(d, sms)), dim3(kPgThreads), 0, s, true,
                        d, w, st->block_table, st->refs);
  }
  if (e == cudaSuccess)
    e = launch_kernel("compact_plan_kernel", small ? compact_plan_kernel<kWalkSmall> : compact_plan_kernel<kWalkLarge>,
                      dim3(1), dim3(kPlanThreads), 0, s, !small, d, w, small ? st->block_table : nullptr, st->refs, refs_out, remap, counts);
  if (e == cudaSuccess)
    e = launch_kernel("compact_commit_kernel", compact_commit_kernel,
                      dim3(commit_grid(d, sms, list, (d.nb + 1) / 2)), dim3(kPgThreads), 0, s, true, d, w, list,
                      st->block_table, table_out);
  return launched(e, "pages_compact");
}
