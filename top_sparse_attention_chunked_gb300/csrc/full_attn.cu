// Full GQA attention of every sequence's new tokens over its cached keys, on
// tcgen05 tensor cores (INT8 caches with few rows: see "few rows" below).
//
// With z_t = scale q.k_t (capped, biased), m any number and l = sum 2^(z_t log2 e
// - m): out = sum 2^(z_t log2 e - m) v_t / l, lse = (m + log2 l) ln 2. Sums over
// parts of the keys join by powers of two of the difference of their m.
//
// The query rows of one KV head -- all new tokens of a sequence times the G
// heads that share the KV head, row = token * G + head -- are cut into items of
// up to 256 rows; the keys an item sees are cut into tiles of 128. One thread
// block per SM walks a run of (item, tile) units of equal cost, whatever the
// mix of sequences: where a run begins or ends inside an item, the item's
// partial state (running maximum, sum, unnormalised output, fp32) goes to the
// workspace and full_attn_merge_kernel joins the parts. So one token over a
// long cache and thousands of tokens take the same path, and every SM gets the
// same share of tiles.
//
// Inside a block, two slots of 128 rows alternate on the tensor core:
//   rows mode (129 .. 256 rows): both slots take every key tile, each for its
//     own half of the rows (a tile of K or V is loaded once for 256 rows);
//   keys mode (up to 128 rows): the slots share the rows and take every other
//     key tile; their two states are joined at the item's end.
// Per slot and tile: S = Q K^T (128 x 128, fp32, in tensor memory), four warps
// read S (a row a thread, a part of it at a time), form P = exp2(S c - m) in 16
// bits and put it back over S, O += P V with P read from tensor memory. While one
// slot is in its softmax the other's two products run.
//
// What bounds it, BF16, 24 query and 2 KV heads where not said otherwise
// (measured rates: 6.80 TB/s, 1,884 TFLOP/s):
//   one token each on long caches: memory. 64 on 8,192: 87 us, 6.15 TB/s; 8 on
//     32,768 with 8/8 heads: 166 us, 6.48 TB/s;
//   few and short: two launches and the first tile's way through a cold block.
//     One token on 1,024: 9.6 us, on 16,384: 14.3 us (1.2 TB/s);
//   many tokens: the hand-over between tensor core and softmax. 4,096 on 16,384:
//     523 us, 1,381 TFLOP/s (the two products alone would take 460); 4,096 on
//     4,096: 110 us, 939 TFLOP/s (a block's share is 2.5 items in 3.2 segments, and
//     at each the output, the next queries and the first product follow one another);
//   capped scores: the multiply-adds of the cap. 4,096 on 4,096: 139 us, with
//     arguments beyond the polynomials (a cap of 3) 207.
//
// The running maximum m is raised (and O rescaled in tensor memory) only when
// a row's weights grow by more than 2^8 over it, and by a whole power of two, to
// just below the maximum. P = 2^kLift exp2(S c - m): the scale cancels in O / sum
// P, the largest weights stay below 2^15, inside either 16-bit type, and FP16's
// smallest step (2^-24) is at most 2^-31 of the weight at the maximum. A slot's S
// is only complete when its previous P V is (the products run in order), so the
// rescale needs no further synchronisation.
//
// K and V tiles arrive by TMA (128 consecutive cache rows of one head: a tile
// never straddles a block of a paged cache, whose blocks hold a multiple of 128
// tokens) in a ring of shared stages. INT8 tiles land as codes and four warps
// widen them to 16 bits (exact); the key's scale multiplies its column of S,
// the value's its column of P. Rows of V outside the item's keys are zeroed in
// shared memory (a masked weight is 0, but 0 times a NaN is not); masked
// columns of S are replaced before the maximum, whatever they hold.
//
// Types: the products take the cache's type (INT8: FP16 for S, which codes are
// widened to in the fewest instructions, and BF16 for P V, since a value's scale
// may lie outside FP16's range). A BF16 query for a product in FP16 is scaled by
// a power of two per row to at most 2^14 first, which is exact for all elements
// within 2^-28 of the row's largest. (An FP16 query on INT8: see split_p.)
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kTileKeys = 128;
constexpr int kSlotRows = 128;
constexpr int kItemRows = 2 * kSlotRows;
constexpr int kMaxCtas = 192;                          // thread blocks the schedule is laid out for
constexpr uint32_t kBlk = kTileKeys * 128;             // 64 columns of a 16-bit tile: 16 KB
constexpr uint32_t kTile16 = 2 * kBlk;                 // 32 KB
constexpr uint32_t kTile8 = kTileKeys * DSA_HEAD_DIM;  // 16 KB of codes
constexpr uint32_t kTmemCols = 512;                    // S 0-127, 128-255; O 256-383, 384-511
// Stages of the rings (a sixth 16-bit stage in place of the second query tile,
// which calls without an item of more than 128 rows do not need, gained nothing:
// 16 ragged decodes of up to 32K 52.0 us with it, 51.2 without).
constexpr int kRing16 = 5, kRing8 = 3, kRaw = 3;
constexpr int kScaleRing = 8;                          // see load_role
// Warps: 8 softmax (slot, quarter of the rows), 4 for the products and the
// loads, 4 that widen INT8 tiles.
constexpr int kSoftThreads = 256, kThreads16 = 384, kWidenThreads = 128, kThreads8 = kThreads16 + kWidenThreads;
// Columns of S that a softmax thread takes at once. INT8: fewer, for its code has
// to share the instruction cache with the widening (4,096 tokens on 4,096: 183 us
// with 64, 167 with 32).
template <bool INT8>
__host__ __device__ constexpr int part_cols() { return INT8 ? 32 : 64; }
// Registers: 16-bit blocks have enough as they are launched (168 a thread);
// with INT8 the softmax takes what the others give up. What the block needs in
// all must be within what it is launched with:
constexpr int kSoftRegs8 = 168, kMiscRegs8 = 72, kWidenRegs = 96;
constexpr int kRegs8 = kSoftThreads * kSoftRegs8 + 128 * kMiscRegs8 + kWidenThreads * kWidenRegs;
constexpr float kLift = 7.0f;                          // log2 of the weight at the running maximum
constexpr float kLeastUnit = 1.17549435e-38f;           // fp32's smallest normal number
constexpr float kRaise = 8.0f;                         // log2 growth that raises the running maximum

struct FullParams {
  const void* q;
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  const float* slopes;
  void* out;
  float* lse;
  uint32_t* status;
  uint32_t* errors;     // [blocks] status bits of each block, OR-ed into *status by the merge
  // [2 * blocks] parts: O as [32 groups of 4 dims][part_rows] (lanes that hold
  // consecutive rows write consecutive 16 bytes), then [part_rows] (m, l)
  float* partial;
  int part_rows;
  int B, Hq, Hkv, G, cap, window;
  int q_dtype, out_dtype;
  float scale_log2, softcap;
  float cap_log2, cap_inv;      // of softcap > 0: softcap * log2 e, and 1 over it
  float cap_pre, cap_ys;        // for FOLD: what z is scaled by first (1: nothing), the units of cap then
  Paging pg;
  // (what a block needs first lies together: every line of the parameters is a
  // miss to begin with)
  struct Seq {
    int q0, item0;                // its first query row, its first item
    int T, first;
  } seq[DSA_MAX_BATCH + 1];
  struct Run {
    int item, tile, b, pad;       // where a block's run begins, and the item's sequence
  } run[kMaxCtas + 1];
};

// One item: rows [row0, row0 + nrows) of (sequence b, KV head g) and the key
// tiles [tile0, tile0 + ntiles) that some row of it sees.
struct Item {
  int b, g, row0, nrows, tile0, ntiles;
  int q0, first;        // the sequence's first query row, its first key
  int past;             // position of the sequence's first new token
  int lo, hi;           // keys that some row sees
};

__host__ __device__ __forceinline__ int imax(int a, int b) { return a > b ? a : b; }
__host__ __device__ __forceinline__ int imin(int a, int b) { return a < b ? a : b; }

// (b: a sequence no later than the item's)
__host__ __device__ __forceinline__ Item make_item(const FullParams& p, int i, int b) {
  Item w;
  while (i >= p.seq[b + 1].item0) ++b;
  const FullParams::Seq q = p.seq[b];
  const int S = p.seq[b + 1].q0 - q.q0;
  const int rows = S * p.G;
  const int per_head = (rows + kItemRows - 1) / kItemRows;
  const int k = i - q.item0;
  w.b = b;
  w.g = k / per_head;
  w.row0 = (k - w.g * per_head) * kItemRows;
  w.nrows = imin(kItemRows, rows - w.row0);
  w.q0 = q.q0;
  w.first = q.first;
  w.past = q.T - S;
  w.hi = w.past + (w.row0 + w.nrows - 1) / p.G + 1;
  w.lo = q.first;
  if (p.window > 0) w.lo = imax(w.lo, w.past + w.row0 / p.G - p.window + 1);
  w.lo = imin(w.lo, w.hi);
  w.tile0 = w.lo / kTileKeys;
  w.ntiles = w.lo < w.hi ? (w.hi + kTileKeys - 1) / kTileKeys - w.tile0 : 0;
  return w;
}

// A block's run of units, one segment (a run of tiles of one item) at a time.
struct Segment {
  Item w;
  int t0, t1;           // tiles, within the item's
  bool rows_mode, whole;
  int part;             // where a partial state goes
};

struct Walk {
  int item, tile, b, end_item, end_tile;
  __device__ __forceinline__ explicit Walk(const FullParams& p) {
    const FullParams::Run at = p.run[blockIdx.x], end = p.run[blockIdx.x + 1];
    item = at.item;
    tile = at.tile;
    b = at.b;
    end_item = end.item;
    end_tile = end.tile;
  }
  __device__ __forceinline__ bool next(const FullParams& p, Segment* s) {
    if (item > end_item || (item == end_item && tile >= end_tile)) return false;
    s->w = make_item(p, item, b);
    b = s->w.b;
    s->t0 = tile;
    s->t1 = item == end_item ? end_tile : s->w.ntiles;
    s->rows_mode = s->w.nrows > kSlotRows;
    s->whole = s->t0 == 0 && s->t1 == s->w.ntiles;
    s->part = 2 * blockIdx.x + (s->t0 > 0 ? 0 : 1);
    ++item;
    tile = 0;
    return true;
  }
};

// What a slot does of a segment: its rows, its tiles (first, step, count).
struct SlotWork {
  int row0, nrows, first, step, n;
};
__device__ __forceinline__ SlotWork slot_work(const Segment& s, int slot) {
  SlotWork x;
  const int n = s.t1 - s.t0;
  if (s.rows_mode) {
    x.row0 = s.w.row0 + slot * kSlotRows;
    x.nrows = imin(kSlotRows, s.w.nrows - slot * kSlotRows);
    x.first = s.t0;
    x.step = 1;
    x.n = n;
  } else {
    x.row0 = s.w.row0;
    x.nrows = s.w.nrows;
    x.first = s.t0 + slot;
    x.step = 2;
    x.n = (n + 1 - slot) >> 1;
  }
  return x;
}

struct FullBars {
  uint64_t full[kRing16], empty[kRing16];       // 16-bit tiles ready / consumed
  uint64_t raw_full[kRaw], raw_empty[kRaw];     // INT8 codes landed / widened
  uint64_t scales[kScaleRing];                  // a tile's scales are in shared memory
  uint64_t q_ready[2], s_full[2], p_full[2], o_full[2];
  uint64_t fix;                                 // a tile whose rows are zeroed before use has landed
  uint64_t ml;                                  // keys mode: slot 1's statistics are in shared memory
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag, bad_page;
  // log2 units per unit of S of the slots' rows (keys mode: slot 0's). Not in m
  // and l: slot 1 goes on to the next segment before slot 0 has read those.
  float unit[2][kSlotRows];
  float m[kSlotRows], l[kSlotRows];             // a segment's end in keys mode: slot 1's statistics, for slot 0
};

template <bool INT8>
constexpr size_t full_smem() {
  return 2 * kTile16 + (INT8 ? kRing8 * kTile16 + kRaw * kTile8 + kScaleRing * 2 * kTileKeys * 4
                                    : kRing16 * kTile16) + sizeof(FullBars);
}
static_assert(full_smem<false>() <= 232448 && full_smem<true>() <= 232448, "shared memory of a block");

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Descriptor of a 128-byte-swizzled operand, 8-row groups 1,024 bytes apart.
// Low word: address / 16, and `lbo` / 16, the pitch of the 64-element column
// blocks of an MN-major operand; an offset adds to the address field alone.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

// kind::f16, fp32 accumulator, M = N = 128; B K-major or MN-major
__host__ __device__ constexpr uint32_t idesc128(bool f16, bool b_mn) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         (16u << 17) | (8u << 24);
}

// D[tmem] (+)= A * B with B, and A, in shared memory (ss), or A in tensor memory
// (ts). Descriptors by their low words: few scalar instructions per product, for
// the one thread that issues them is as busy as the tensor core.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(static_cast<int>(acc)), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(static_cast<int>(acc)), "r"(kDescHi)
      : "memory");
}

// 32 lanes x 32 columns of 32 bits, one lane a thread
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
      "%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  unsigned long long ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// Two signed codes, bytes 2i and 2i + 1 of `x`, as two exact 16-bit floats.
// BF16: 0x4300 | n is 128 + n for n < 128, and 0x4380 is 256, so
// (0x4300 | (c & 0x7f)) - (0x4300 | (c & 0x80)) is c. FP16: 0x6400 | u is
// 1,024 + u for any byte, and u = c + 128.
template <bool F16>
__device__ __forceinline__ uint32_t widen2(uint32_t x, int i) {
  if constexpr (F16) {
    const uint32_t u = __byte_perm(x ^ 0x80808080u, 0x64646464u, i ? 0x4342 : 0x4140);
    const uint32_t bias = 0x64806480u;   // 1,152
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&bias));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const uint32_t u = __byte_perm(x, 0u, i ? 0x4342 : 0x4140);
    const uint32_t a = (u & 0x007f007fu) | 0x43004300u, b = (u & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Byte e of x and of y, two signed codes, as two BF16 (see above).
__device__ __forceinline__ uint32_t widen_pair(uint32_t x, uint32_t y, int e) {
  const uint32_t u = __byte_perm(x, y, (4 + e) << 8 | e);
  const uint32_t a = (u & 0x007f007fu) | 0x43004300u, b = (u & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A wait of a whole warp: every lane gets the same answer, and the warp is
// converged afterwards.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag));
}

// Position in a ring.
struct RingPos {
  int stage = 0;
  uint32_t round = 0;       // parity: the round's `full`; of `empty`, the round before
  __device__ __forceinline__ void step(int stages) {
    if (++stage == stages) {
      stage = 0;
      ++round;
    }
  }
};

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {   // when this thread's copies so far have landed
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ---------------------------------------------------------------- loader
// Issues the tiles in the order the products consume them: rows mode K0 V0 K1
// V1 ..., keys mode K0 K1 V0 K2 V1 K3 ...
template <class F>
__device__ __forceinline__ bool for_tiles(const Segment& s, F&& f) {
  const int n = s.t1 - s.t0;
  if (s.rows_mode) {
    for (int j = 0; j < n; ++j)
      if (!f(s.t0 + j, false) || !f(s.t0 + j, true)) return false;
  } else {
    for (int i = 0; i < n + 2; ++i) {
      if (i >= 2 && !f(s.t0 + i - 2, true)) return false;
      if (i < n && !f(s.t0 + i, false)) return false;
      if (n == 1 && i == 0) {   // a single tile: K0 V0
        return f(s.t0, true);
      }
    }
  }
  return true;
}

//
// INT8: the scales of a K tile's keys, and of the same keys' values, are copied
// beside it, four bytes a key, into a ring of their own. A slot is written
// again eight tiles on. By then the softmax has read it: tile i + 8's K tile is
// issued when a raw stage is free, so V of tile i + 4 at least has been widened,
// so K of tile i + 3 has been consumed, and its product was issued after the
// weights of tile i + 1.
template <bool INT8>
__device__ __forceinline__ void load_role(const FullParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                          FullBars* bars, uint8_t* ring, float* scales,
                                          volatile int* abort_flag) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kBytes = INT8 ? kTile8 : kTile16;
  constexpr int stages = INT8 ? kRaw : kRing16;
  uint64_t* full = INT8 ? bars->raw_full : bars->full;
  uint64_t* empty = INT8 ? bars->raw_empty : bars->empty;
  if (lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  RingPos pos;
  uint32_t fixes = 0, tiles = 0;
  bool bad = false, begin = true;
  Walk walk(p);
  Segment s;
  while (walk.next(p, &s)) {
    if (s.t0 == s.t1) continue;
    // cache rows of 32 tiles, one a lane, looked up together and 32 tiles ahead
    const auto look_up = [&](int t) {
      return t < s.t1 ? cache_row(p.pg, s.w.b, p.cap, (s.w.tile0 + t) * kTileKeys, &bad) : 0;
    };
    int base = s.t0;
    long long rows = look_up(base + lane), rows_next = look_up(base + 32 + lane);
    // the item's queries, which the softmax warps load when they get there
    // (those of the first they load at the same time)
    for (int i = lane; !begin && i < s.w.nrows; i += 32) {
      const int r = s.w.row0 + i, tok = r / p.G;
      const uint16_t* q = static_cast<const uint16_t*>(p.q) +
                          ((static_cast<long long>(s.w.q0) + tok) * p.Hq + s.w.g * p.G + (r - tok * p.G)) * DSA_HEAD_DIM;
      prefetch_l2_line(q);
      prefetch_l2_line(q + 64);
    }
    begin = false;
    const bool ok = for_tiles(s, [&](int t, bool is_v) {
      const int st = pos.stage;
      if (pos.round > 0 && !warp_wait(&empty[st], (pos.round - 1) & 1, abort_flag)) return false;
      const int key = (s.w.tile0 + t) * kTileKeys;
      // (K runs up to two tiles ahead of V: the window moves when V has left it)
      if (is_v && t >= base + 32) {
        base += 32;
        rows = rows_next;
        rows_next = look_up(base + 32 + lane);
      }
      const long long first = __shfl_sync(0xffffffffu, t < base + 32 ? rows : rows_next, (t - base) & 31);
      const int row = static_cast<int>(first);
      uint8_t* dst = ring + st * kBytes;
      const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
      // rows of V that no query of the item sees
      const int lo = imax(0, s.w.lo - key), hi = imin(kTileKeys, s.w.hi - key);
      const bool fix = !INT8 && is_v && (lo > 0 || hi < kTileKeys);
      uint64_t* bar = fix ? &bars->fix : &full[st];
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, kBytes);
        tma_load_3d(dst, tm, bar, 0, s.w.g, row);
        if constexpr (!INT8) tma_load_3d(dst + kBlk, tm, bar, 64, s.w.g, row);
      }
      if constexpr (INT8) {
        if (!is_v) {
          float* sc = scales + (tiles % kScaleRing) * 2 * kTileKeys;
#pragma unroll
          for (int i = 0; i < kTileKeys / 32; ++i) {
            const int r = i * 32 + lane;
            const bool in = r >= lo && r < hi;
            const long long at = in ? (first + r) * p.Hkv + s.w.g : 0;
            cp_async4(sc + r, p.k_scale + at, in);
            cp_async4(sc + kTileKeys + r, p.v_scale + at, in);
          }
          cp_async_arrive(&bars->scales[tiles % kScaleRing]);
          ++tiles;
        }
      }
      __syncwarp();
      if (fix) {
        if (!warp_wait(&bars->fix, fixes++ & 1, abort_flag)) return false;
        for (int r = 0; r < kTileKeys; ++r) {
          if (r >= lo && r < hi) continue;
          if (lane < 16)
            *reinterpret_cast<uint4*>(dst + (lane >> 3) * kBlk + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      }
      pos.step(stages);
      return true;
    });
    if (!ok) break;
  }
  if (bad) bars->bad_page = 1;
  if constexpr (INT8) {
    cp_async_commit();
    cp_async_wait<0>();
  }
  if (lane == 0) {
    // a block must not end with copies in flight (the consumers may have given up)
    const auto drain = [](uint64_t* bar, uint32_t uses) {
      if (uses == 0) return;
      const long long t0 = clock64();
      while (!mbar_try_wait(bar, (uses - 1) & 1) && clock64() - t0 < kWaitBudgetCycles) {
      }
    };
    // (stage q's last use: this round if the position is past it, else the one before)
    for (int q = 0; q < stages; ++q) drain(&full[q], pos.round + (q < pos.stage ? 1 : 0));
    if constexpr (!INT8) drain(&bars->fix, fixes);
  }
}

// ------------------------------------------------------------ INT8 widening
// A tile of 128 x 128 codes (128-byte rows, swizzled) to a 16-bit tile, by
// kWidenThreads threads. Eight lanes take chunks 0-3 (16 codes each) of an even row and 4-7
// of the next, then the other halves: the reads, and the two 16-byte writes a
// chunk becomes, each touch eight different 16-byte columns.
struct WidenAt {   // this thread's places in a tile of codes and in a 16-bit tile
  int from, to;
  __device__ __forceinline__ explicit WidenAt(int tid) {
    const int half = (tid >> 2) & 1, row = (tid >> 3) * 2 + half;
    from = row * 128 + ((((tid & 3) + 4 * half) ^ (row & 7)) << 4);
    to = half * kBlk + row * 128 + ((((tid & 3) * 2) ^ (row & 7)) << 4);
  }
};
template <bool F16>
__device__ __forceinline__ void widen_tile(const uint8_t* src, uint8_t* dst, const WidenAt& at) {
  constexpr int kStep = kWidenThreads / 4 * 128;   // bytes of the rows taken at once, a multiple of eight rows
  static_assert(kWidenThreads % 32 == 0 && kTile8 % (2 * kStep) == 0, "rows a thread takes");
#pragma unroll 1
  for (int i = 0; i < static_cast<int>(kTile8); i += 2 * kStep) {
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[j] = *reinterpret_cast<const uint4*>(src + i + (j >> 1) * kStep + (at.from ^ ((j & 1) << 6)));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = widen2<F16>(w[e >> 1], e & 1);
      uint8_t* d = dst + i + (j >> 1) * kStep;
      const int to = at.to ^ ((j & 1) * kBlk);
      *reinterpret_cast<uint4*>(d + to) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(d + (to ^ 16)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

__device__ __forceinline__ void widen_role(const FullParams& p, FullBars* bars, uint8_t* ring, const uint8_t* raw,
                                           int tid, volatile int* abort_flag) {
  RingPos from, to;
  const WidenAt at(tid);
  Walk walk(p);
  Segment s;
  while (walk.next(p, &s)) {
    const bool ok = for_tiles(s, [&](int, bool is_v) {
      if (!warp_wait(&bars->raw_full[from.stage], from.round & 1, abort_flag)) return false;
      if (to.round > 0 && !warp_wait(&bars->empty[to.stage], (to.round - 1) & 1, abort_flag)) return false;
      const uint8_t* src = raw + from.stage * kTile8;
      uint8_t* dst = ring + to.stage * kTile16;
      if (is_v) widen_tile<false>(src, dst, at);
      else widen_tile<true>(src, dst, at);
      fence_async_smem();
      mbar_arrive(&bars->full[to.stage]);
      mbar_arrive(&bars->raw_empty[from.stage]);
      from.step(kRaw);
      to.step(kRing8);
      return true;
    });
    if (!ok) break;
  }
}

// ------------------------------------------------------------ tensor core
// An FP16 query on an INT8 cache: its output has three bits more than a BF16
// weight, so P goes as a BF16 pair, high and low part, and the second product is
// taken with both.
template <bool QK_F16, bool INT8>
__host__ __device__ constexpr bool split_p() { return QK_F16 && INT8; }

template <bool QK_F16, bool PV_F16, bool INT8>
__device__ __forceinline__ void mma_role(const FullParams& p, FullBars* bars, uint32_t tmem, uint32_t q_addr,
                                         uint32_t ring_addr, volatile int* abort_flag) {
  constexpr int stages = INT8 ? kRing8 : kRing16;
  constexpr uint32_t id_qk = idesc128(QK_F16 || INT8, false), id_pv = idesc128(PV_F16, true);
  const uint32_t qd = desc_lo(q_addr, 16), kd = desc_lo(ring_addr, 16), vd = desc_lo(ring_addr, kBlk);
  uint32_t nseg = 0, np[2] = {0, 0};
  RingPos pos;
  const auto wait_tile = [&](const RingPos& q) { return mbar_wait_bounded(&bars->full[q.stage], q.round & 1, abort_flag); };
  const auto qk = [&](int slot, uint32_t q_tile, const RingPos& q) {   // S[slot] = Q K^T
    const uint32_t a = qd + q_tile * (kTile16 / 16), b = kd + q.stage * (kTile16 / 16);
#pragma unroll
    for (int kk = 0; kk < DSA_HEAD_DIM / 16; ++kk) {
      constexpr uint32_t kStep = 32 / 16;
      const uint32_t off = (kk >> 2) * (kBlk / 16) + (kk & 3) * kStep;
      mma_ss(tmem + slot * 128, a + off, b + off, id_qk, kk > 0);
    }
    tc_commit(&bars->s_full[slot]);
  };
  const auto pv = [&](int slot, const RingPos& q, bool first) {        // O[slot] (+)= P V
    const uint32_t b = vd + q.stage * (kTile16 / 16);
    if (!mbar_wait_bounded(&bars->p_full[slot], np[slot] & 1, abort_flag)) return false;
    ++np[slot];
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < kTileKeys / 16; ++kk) {
      constexpr int kCols = part_cols<INT8>(), kSteps = kCols / 16;   // (a part's weights over its own columns)
      const uint32_t pa = tmem + slot * 128 + kk / kSteps * kCols + kk % kSteps * 8;
      mma_ts(tmem + 256 + slot * 128, pa, b + kk * (16 * 128 / 16), id_pv, !first || kk > 0);
      if constexpr (split_p<QK_F16, INT8>()) mma_ts(tmem + 256 + slot * 128, pa + kCols / 2, b + kk * (16 * 128 / 16), id_pv, true);
    }
    return true;
  };
  const auto release = [&](const RingPos& q) { tc_commit(&bars->empty[q.stage]); };
  Walk walk(p);
  Segment s;
  bool ok = true;
  while (ok && walk.next(p, &s)) {
    const int n = s.t1 - s.t0;
    if (n == 0) continue;   // (the softmax warps write its zeros)
    // both slots are done with the previous segment, the queries are in place
    if (!mbar_wait_bounded(&bars->q_ready[0], nseg & 1, abort_flag)) break;
    if (!mbar_wait_bounded(&bars->q_ready[1], nseg & 1, abort_flag)) break;
    ++nseg;
    tc_fence_after();
    if (s.rows_mode) {
      // round j: P V of tile j - 1 and S of tile j in slot 0, then in slot 1
      RingPos v = pos;
      for (int j = 0; j <= n && ok; ++j) {
        const RingPos k = pos;
        if (j > 0) ok = wait_tile(v);
        if (ok && j < n) ok = wait_tile(k);
        if (!ok) break;
        tc_fence_after();
        for (int slot = 0; slot < 2 && ok; ++slot) {
          if (j > 0) {
            ok = pv(slot, v, j == 1);
            if (!ok) break;
            if (slot == 1) release(v);
            if (j == n) tc_commit(&bars->o_full[slot]);
          }
          if (j < n) {
            qk(slot, slot, k);
            if (slot == 1) release(k);
          }
        }
        if (j < n) {
          pos.step(stages);
          v = pos;
          pos.step(stages);
        }
      }
    } else {
      // step i: P V of tile i - 2, then S of tile i, both in slot i & 1
      for (int i = 0; i < n + 2 && ok; ++i) {
        const int slot = i & 1;
        if (i >= 2 && i - 2 < n) {
          ok = wait_tile(pos);
          if (!ok) break;
          tc_fence_after();
          ok = pv(slot, pos, i < 4);
          if (!ok) break;
          release(pos);
          pos.step(stages);
          if (i >= n) tc_commit(&bars->o_full[slot]);
          // (slot 1 has no tile of a segment of one; it must not go on to the next one's
          // queries before this thread has seen that it was ready for this one)
          if (n == 1) tc_commit(&bars->o_full[1]);
        }
        if (i < n) {
          ok = wait_tile(pos);
          if (!ok) break;
          tc_fence_after();
          qk(slot, 0, pos);
          release(pos);
          pos.step(stages);
        }
      }
    }
  }
  tc_commit(&bars->done);
  const long long t0 = clock64();
  while (!mbar_try_wait(&bars->done, 0) && clock64() - t0 < kWaitBudgetCycles) {
  }
}

// ---------------------------------------------------------------- softmax
// cap y P(y^2) for N values, y = z * ys, P of K coefficients (highest first): K + 2
// cycles of the multiply-add pipe a value (paired arithmetic; eight pairs side
// by side, a chain of dependent operations each). FOLD: ys goes into the
// coefficients, K + 1 cycles; its powers are normal numbers.
template <int N, bool FOLD, int K>
__device__ __forceinline__ void odd_poly(float* z, float ys, float cap, const float (&k)[K]) {
  constexpr int kPairs = N < 16 ? N / 2 : 8;
  const auto both = [](float x) { return make_float2(x, x); };
  const float2 y2 = both(ys), zero = both(0.f);
  float c[K], f = FOLD ? cap * ys : cap;
#pragma unroll
  for (int d = K - 1; d >= 0; --d) {
    c[d] = k[d] * f;
    if constexpr (FOLD) f *= ys * ys;
  }
#pragma unroll
  for (int i = 0; i < N; i += 2 * kPairs) {
    float2 y[kPairs], t[kPairs], a[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      y[e] = make_float2(z[i + 2 * e], z[i + 2 * e + 1]);
      if constexpr (!FOLD) y[e] = fma_f32x2(y[e], y2, zero);
      t[e] = fma_f32x2(y[e], y[e], zero);
      a[e] = both(c[0]);
    }
#pragma unroll
    for (int d = 1; d < K; ++d)
#pragma unroll
      for (int e = 0; e < kPairs; ++e) a[e] = fma_f32x2(a[e], t[e], both(c[d]));
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      a[e] = fma_f32x2(a[e], y[e], zero);
      z[i + 2 * e] = a[e].x;
      z[i + 2 * e + 1] = a[e].y;
    }
  }
}

// z (units of S, c log2-units each) -> cap * tanh(z c ln2 / cap) in log2 units, to
// a relative error of 7e-7 of the result or 1.6e-5 of a logit, however far the cap
// lies above it (an error of some part of a wide cap would be one of the logits).
// Arguments y of up to 0.25, 0.4 and 0.7 take odd polynomials, fitted to tanh y / y
// for the least relative error (4e-7, 1e-7, 1e-8; the first is a multiply-add a
// value shorter). Parts with larger ones take tanh y = 1 - 2 / (1 + e^2y), whose two
// special-function calls a value would be the kernel's bound, and whose error is
// 2.5e-7 of the cap: with caps above 64, arguments of up to 0.4 take the second
// polynomial there too (4,096 tokens on 4,096 with a cap of 3: 207 us, 275 if small
// caps did that).
// FOLD (c is the problem's, not a row's): see odd_poly; the eleventh power of
// c / cap times cap has to be a normal number, else z is scaled first (cap_fold).
// N < 32: a shorter choice (the code of a few values, not their time, is what
// counts).
constexpr float kNearCap = 64.0f;
template <int N, bool FOLD>
__device__ __forceinline__ void cap_scores(float* z, float c, const FullParams& p) {
  const float cap = p.cap_log2, ys = FOLD ? p.cap_ys : fminf(c * p.cap_inv, 1e38f);
  if (FOLD && p.cap_pre != 1.0f) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] *= p.cap_pre;
  }
  float far[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) far[i & 3] = fmaxf(far[i & 3], fabsf(z[i]));
  const float y = fmaxf(fmaxf(far[0], far[1]), fmaxf(far[2], far[3])) * ys;
  const float k4[4] = {-0.0475536026f, 0.132709771f, -0.333313614f, 0.999999881f};
  if (N >= 32 && __all_sync(0xffffffffu, y <= 0.25f)) {
    const float k[3] = {0.128416136f, -0.333219081f, 0.999999583f};
    odd_poly<N, FOLD>(z, ys, cap, k);
  } else if (__all_sync(0xffffffffu, y <= 0.4f)) {
    odd_poly<N, FOLD>(z, ys, cap, k4);
  } else if (N >= 32 && __all_sync(0xffffffffu, y <= 0.7f)) {
    const float k[6] = {-0.0050883363f, 0.0200244579f, -0.0535260104f, 0.133284152f, -0.333331317f, 1.0f};
    odd_poly<N, FOLD>(z, ys, cap, k);
  } else if (p.softcap <= kNearCap) {
    const float two = ys * 2.8853900817779268f;
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = fmaf(-2.0f * cap, fast_rcp(1.0f + fast_exp2(z[i] * two)), cap);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = z[i] * ys, t = x * x;
      const float low = fmaf(fmaf(fmaf(k4[0], t, k4[1]), t, k4[2]), t, k4[3]) * cap * x;
      const float high = fmaf(-2.0f * cap, fast_rcp(1.0f + fast_exp2(x * 2.8853900817779268f)), cap);
      z[i] = fabsf(x) <= 0.4f ? low : high;
    }
  }
}

// N columns of P (2 N weights a row) at `addr` times f.
template <bool F16, int N>
__device__ __forceinline__ void rescale_p(uint32_t addr, float f) {
  tmem_st_wait();   // (this warp's own store of them)
#pragma unroll 1
  for (int i = 0; i < N; i += 16) {
    float v[16];
    uint32_t w[16];
    tmem_ld16(addr + i, v);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) asm volatile("" : "+f"(v[e]));
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t u = __float_as_uint(v[e]);
      const float2 x = F16 ? __half22float2(*reinterpret_cast<const __half2*>(&u))
                           : make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
      w[e] = pack2<F16>(x.x * f, x.y * f);
    }
    tmem_st16(addr + i, w);
  }
}

// A BF16 row whose largest element has the bits `top` (without sign) is taken as
// FP16 times 2^ex, the largest element's exponent 14; a row of zeros as it is.
__device__ __forceinline__ int row_exponent(uint32_t top) {
  return top == 0u ? 0 : imax(static_cast<int>(top >> 7), 1) - 127 - 14;
}
// Its log2 units per unit of S. Not 0: a masked column's -infinity times it
// would be a NaN (below fp32's normal numbers no such row's logits differ from 0).
__device__ __forceinline__ float row_unit(float scale_log2, int ex) { return fmaxf(ldexpf(scale_log2, ex), kLeastUnit); }

// The outputs of `n` rows (32 at the most) of an item from row0 on, none of which
// sees a key. One warp calls it; a lane finds a row's place.
__device__ __forceinline__ void write_no_key(const FullParams& p, const Item& w, int row0, int n) {
  if (n <= 0) return;
  const int lane = threadIdx.x & 31, r = row0 + imin(lane, n - 1), tok = r / p.G;
  const long long row = (static_cast<long long>(w.q0) + tok) * p.Hq + w.g * p.G + (r - tok * p.G);
  if (p.lse && lane < n) p.lse[row] = -INFINITY;
  const int vecs = p.out_dtype == DSA_FP32 ? 32 : 16;   // a row's, 16 bytes each
#pragma unroll 4
  for (int i = 0; i < n; i += 32 / vecs) {
    const int k = i + lane / vecs;
    const long long to = __shfl_sync(0xffffffffu, row, imin(k, n - 1));
    if (k < n) static_cast<uint4*>(p.out)[to * vecs + lane % vecs] = make_uint4(0, 0, 0, 0);
  }
}

// One slot's four warps, one row a thread. MOD: the scores are capped or get a
// bias.
//
// A row goes in parts of 64 or 32 columns (code and registers for one). The
// exponentials are formed with the running maximum as it was, next to the
// part's own maximum; only where that calls for raising the former are they
// formed again.
template <bool QK_F16, bool PV_F16, bool INT8, bool MOD>
__device__ __forceinline__ void softmax_role(const FullParams& p, FullBars* bars, uint32_t tmem, uint8_t* sQ,
                                             const float* scales, int slot, volatile int* abort_flag) {
  const int tid = threadIdx.x & 127, lane = tid & 31, warp_row = tid & ~31;
  constexpr bool kSplit = split_p<QK_F16, INT8>();
  constexpr int kCols = part_cols<INT8>();
  constexpr bool kMayScale = QK_F16 != INT8;   // a BF16 query for products in FP16
  const bool scaled = kMayScale && p.q_dtype == DSA_BF16;
  const uint32_t lane_addr = static_cast<uint32_t>(warp_row) << 16;
  const uint32_t tS = tmem + lane_addr + slot * 128, tO = tmem + lane_addr + 256 + slot * 128;
  uint32_t ns = 0, no = 0, nml = 0, nseg = 0, tile_seq = 0;
  Walk walk(p);
  Segment s;
  while (walk.next(p, &s)) {
    const SlotWork x = slot_work(s, slot);
    if (s.t0 == s.t1) {
      // No row sees a key. Such an item takes no part in the hand-over with the
      // tensor core: a slot that has nothing to wait for there would run ahead
      // of the other and of the barriers' phases.
      if (slot == 0 || s.rows_mode) write_no_key(p, s.w, x.row0 + warp_row, imin(32, x.nrows - warp_row));
      continue;
    }
    const int r = x.row0 + tid;
    const bool valid = tid < x.nrows;
    const bool warp_valid = (tid & ~31) < x.nrows;
    const int tok = r / p.G;
    const int pos = s.w.past + tok;
    const int head = s.w.g * p.G + (r - tok * p.G);
    const long long row = (static_cast<long long>(s.w.q0) + tok) * p.Hq + head;   // query row
    float c = p.scale_log2;   // logits in units of log2 e per unit of S
    if (slot == 0 || s.rows_mode) {
      // The warp's 32 rows, four at a time: eight lanes a row, lane k of them its
      // 16-byte chunks k and k + 8 (one in each block of 64 columns).
      volatile float* row_c = bars->unit[slot];
      const int sub = lane & 7;
      uint8_t* dst = sQ + slot * kTile16;
#pragma unroll 1
      for (int i0 = 0; i0 < 8; i0 += 4) {
        uint4 u[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = warp_row + (i0 + i) * 4 + (lane >> 3);
          const int rr = x.row0 + t, tk = rr / p.G;
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(p.q) +
              ((static_cast<long long>(s.w.q0) + tk) * p.Hq + s.w.g * p.G + (rr - tk * p.G)) * DSA_HEAD_DIM);
          const bool in = t < x.nrows;
          u[i][0] = in ? __ldg(src + sub) : make_uint4(0, 0, 0, 0);
          u[i][1] = in ? __ldg(src + sub + 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = warp_row + (i0 + i) * 4 + (lane >> 3);
          if constexpr (kMayScale) {
            if (scaled) {
              // the row's largest exponent to 14: scaled by 2^-ex
              uint32_t w[8] = {u[i][0].x, u[i][0].y, u[i][0].z, u[i][0].w, u[i][1].x, u[i][1].y, u[i][1].z, u[i][1].w};
              uint32_t top = 0;
#pragma unroll
              for (int e = 0; e < 8; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
              for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
              const int ex = row_exponent(top);
              // (two factors: 2^-ex may lie outside fp32's normal range)
              const float f0 = __int_as_float((127 - ex / 2) << 23), f1 = __int_as_float((127 - (ex - ex / 2)) << 23);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e] = pack2<true>(__uint_as_float(w[e] << 16) * f0 * f1, __uint_as_float(w[e] & 0xffff0000u) * f0 * f1);
              u[i][0] = make_uint4(w[0], w[1], w[2], w[3]);
              u[i][1] = make_uint4(w[4], w[5], w[6], w[7]);
              if (sub == 0) row_c[t] = row_unit(p.scale_log2, ex);
            }
          }
          uint8_t* d = dst + t * 128 + ((sub ^ (t & 7)) << 4);
          *reinterpret_cast<uint4*>(d) = u[i][0];
          *reinterpret_cast<uint4*>(d + kBlk) = u[i][1];
        }
      }
      __syncwarp();
      if (scaled) c = row_c[tid];
      fence_async_smem();
    }
    if (slot == 1 && !s.rows_mode) {
      // slot 0 loads the shared rows; what it scaled them by
      if (!warp_wait(&bars->q_ready[0], nseg & 1, abort_flag)) break;
      if (scaled) c = *const_cast<const volatile float*>(&bars->unit[0][tid]);
    }
    ++nseg;
    tc_fence_before();
    mbar_arrive(&bars->q_ready[slot]);
    const float slope = MOD && p.slopes && valid ? p.slopes[head] * 1.4426950408889634f : 0.f;
    const int pos0 = s.w.past + x.row0 / p.G, pos1 = s.w.past + (x.row0 + x.nrows - 1) / p.G;
    const int lo = imax(s.w.first, p.window > 0 ? pos - p.window + 1 : 0);
    const int lo1 = imax(s.w.first, p.window > 0 ? pos1 - p.window + 1 : 0);   // the last row's

    float m = -INFINITY, l = 0.f;   // running maximum (in S units, or log2 units where c = 1), sum
    const float cz = MOD ? 1.0f : c;
    bool ok = true;
    for (int j = 0; j < x.n; ++j) {
      const int t = x.first + j * x.step;
      const int key0 = (s.w.tile0 + t) * kTileKeys;
      if (!warp_wait(&bars->s_full[slot], ns & 1, abort_flag)) {
        ok = false;
        break;
      }
      ++ns;
      tc_fence_after();
      if constexpr (INT8) {
        const uint32_t q = tile_seq + (t - s.t0);
        if (!warp_wait(&bars->scales[q % kScaleRing], (q / kScaleRing) & 1, abort_flag)) {
          ok = false;
          break;
        }
      }
      const bool masked = key0 + kTileKeys - 1 > pos0 || key0 < lo1;
      const float* sc = scales + ((tile_seq + (t - s.t0)) % kScaleRing) * 2 * kTileKeys;
#pragma unroll 1
      for (int h = 0; h < kTileKeys / kCols; ++h) {
        if (warp_valid) {
          const int col = h * kCols, first = key0 + col;
          float z[kCols];
          tmem_ld32(tS + col, z);
          if constexpr (kCols > 32) tmem_ld32(tS + col + 32, z + 32);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kCols; ++i) asm volatile("" : "+f"(z[i]));   // no use before the wait
          if constexpr (INT8) {
#pragma unroll
            for (int i = 0; i < kCols; i += 4) {
              const float4 f = *reinterpret_cast<const float4*>(sc + col + i);
              z[i] *= f.x;
              z[i + 1] *= f.y;
              z[i + 2] *= f.z;
              z[i + 3] *= f.w;
            }
          }
          if constexpr (MOD) {
            if (p.softcap > 0.f) cap_scores<kCols, !kMayScale>(z, c, p);
            else
#pragma unroll
              for (int i = 0; i < kCols; ++i) z[i] *= c;
            if (p.slopes) {
              const float d = static_cast<float>(first - pos);
#pragma unroll
              for (int i = 0; i < kCols; ++i) z[i] = fmaf(slope, d + static_cast<float>(i), z[i]);
            }
          }
          if (masked) {
            const int a = lo - first, b = pos - first;   // columns a .. b are visible
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (i < a || i > b) z[i] = -INFINITY;
          }
          uint32_t w[kCols / 2], wl[kSplit ? kCols / 2 : 1];
          float2 sum[2];
#pragma unroll 1
          while (true) {
            const float mc = m == -INFINITY ? 0.f : kLift - m * cz;
            sum[0] = sum[1] = make_float2(0.f, 0.f);
            const float2 c2 = make_float2(cz, cz), m2 = make_float2(mc, mc);
            float mt[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
            for (int i = 0; i < kCols / 2; i += 8) {
              float2 pr[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) pr[e] = fma_f32x2(make_float2(z[2 * (i + e)], z[2 * (i + e) + 1]), c2, m2);
#pragma unroll
              for (int e = 0; e < 8; ++e) pr[e] = make_float2(fast_exp2(pr[e].x), fast_exp2(pr[e].y));
#pragma unroll
              for (int e = 0; e < 16; ++e) mt[e & 3] = fmaxf(mt[e & 3], z[2 * i + e]);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                sum[e & 1] = add_f32x2(pr[e], sum[e & 1]);
                if constexpr (INT8) {
                  const float2 vs = *reinterpret_cast<const float2*>(sc + kTileKeys + col + 2 * (i + e));
                  pr[e] = fma_f32x2(pr[e], vs, make_float2(0.f, 0.f));
                }
                w[i + e] = pack2<PV_F16>(pr[e].x, pr[e].y);
                if constexpr (kSplit)
                  wl[i + e] = pack2<false>(pr[e].x - __uint_as_float(w[i + e] << 16),
                                           pr[e].y - __uint_as_float(w[i + e] & 0xffff0000u));
              }
            }
            const float mn = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
            // (-inf stays as it is: nothing seen yet)
            const bool raise = mn > m && (m == -INFINITY || (mn - m) * cz > kRaise);
            if (!__any_sync(0xffffffffu, raise)) break;
            // by a power of two, not above it: nothing of P or O is rounded again (a second
            // rounding of a BF16 pair's high part would be lost to the low one)
            float f = 1.0f;
            if (mn > m) {
              const float up = m == -INFINITY ? 0.f : floorf((mn - m) * cz);
              f = m == -INFINITY ? 0.f : fast_exp2(-up);
              m = m == -INFINITY ? mn : m + up / cz;
            }
            l *= f;
#pragma unroll 1
            for (int e = 0; e < h; ++e) {   // the parts before, not yet in O
              rescale_p<PV_F16, kCols / 2>(tS + e * kCols, f);
              if constexpr (kSplit) rescale_p<PV_F16, kCols / 2>(tS + e * kCols + kCols / 2, f);
            }
            if (j > 0) {
#pragma unroll 1
              for (int i = 0; i < DSA_HEAD_DIM; i += 16) {
                float o[16];
                uint32_t v[16];
                tmem_ld16(tO + i, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) asm volatile("" : "+f"(o[e]));
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(o[e] * f);
                tmem_st16(tO + i, v);
              }
            }
          }
          // over columns of S that have been read
          if constexpr (kCols > 32) {
            tmem_st32(tS + col, w);
          } else {
            tmem_st16(tS + col, w);
            if constexpr (kSplit) tmem_st16(tS + col + kCols / 2, wl);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
      }
      if (warp_valid) tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->p_full[slot]);
    }
    if (!ok) break;
    tile_seq += s.t1 - s.t0;
    const float m_log2 = m == -INFINITY ? -INFINITY : m * cz;
    // in keys mode slot 0 joins the two states; it reads slot 1's O itself
    const auto leave = [&]() {
      bars->m[tid] = m_log2;
      bars->l[tid] = l;
      mbar_arrive(&bars->ml);
    };
    const bool left = !s.rows_mode && slot == 1;
    if (left && x.n == 0) leave();   // (slot 1 has no tile of a segment of one: slot 0 need not wait for it)
    if (!warp_wait(&bars->o_full[slot], no & 1, abort_flag)) break;
    ++no;
    tc_fence_after();
    if (left) {
      if (x.n > 0) leave();
      continue;
    }
    float f0 = 1.0f, f1 = 0.0f, mj = m_log2, lj = l;
    bool other = false;
    if (!s.rows_mode) {
      if (!warp_wait(&bars->ml, nml & 1, abort_flag)) break;
      ++nml;
      tc_fence_after();
      other = slot_work(s, 1).n > 0;
      if (other) {
        const volatile float* v = &bars->m[tid];
        const float m1 = v[0], l1 = v[kSlotRows];
        mj = fmaxf(m_log2, m1);
        f0 = m_log2 == -INFINITY ? 0.f : fast_exp2(m_log2 - mj);
        f1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - mj);
        lj = l * f0 + l1 * f1;
      }
    }
    if (!warp_valid) continue;
    float norm = 1.0f;
    float* part = nullptr;
    if (s.whole) {
      norm = lj > 0.f ? 1.0f / lj : 0.f;
      if (valid && p.lse) p.lse[row] = lj > 0.f ? (mj - kLift + log2f(lj)) * 0.6931471805599453f : -INFINITY;
    } else {
      part = p.partial + static_cast<long long>(s.part) * p.part_rows * (DSA_HEAD_DIM + 2);
      const int pr = r - s.w.row0;
      if (valid) *reinterpret_cast<float2*>(part + p.part_rows * DSA_HEAD_DIM + 2 * pr) = make_float2(mj, lj);
      part += pr * 4;
    }
    f0 *= norm;
    f1 *= norm;
#pragma unroll 1
    for (int i = 0; i < DSA_HEAD_DIM; i += 32) {
      float o[32];
      tmem_ld32(tO + i, o);
      if (other) {
        float b[32];
        tmem_ld32(tO + 128 + i, b);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) asm volatile("" : "+f"(o[e]), "+f"(b[e]));
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = f0 * o[e] + f1 * b[e];
      } else {
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) asm volatile("" : "+f"(o[e]));
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= f0;
      }
      // a row without a key: whatever the products hold, its output is 0
      if (s.whole && !(lj > 0.f)) {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
      }
      if (!valid) continue;
      if (part) {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(part + static_cast<long long>(i + e) * p.part_rows) =
              make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      } else if (p.out_dtype == DSA_FP32) {
        float* d = static_cast<float*>(p.out) + row * DSA_HEAD_DIM + i;
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(d + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      } else {
        uint16_t* d = static_cast<uint16_t*>(p.out) + row * DSA_HEAD_DIM + i;
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = p.out_dtype == DSA_FP16 ? pack2<true>(o[2 * e], o[2 * e + 1]) : pack2<false>(o[2 * e], o[2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(d + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
      }
    }
  }
}

template <bool QK_F16, bool PV_F16, bool INT8, bool MOD>
__global__ void __launch_bounds__(INT8 ? kThreads8 : kThreads16, 1)
    full_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ FullParams p) {
  // (the kernel has no static shared memory: the dynamic part begins on the
  // 1,024 bytes that the swizzled tiles need, of which there is none to spare)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw;
  if (smem_u32(base) & 1023u) {
    if (threadIdx.x == 0) p.errors[blockIdx.x] = kDevBounds;
    return;
  }
  // queries | (INT8: codes) | 16-bit tiles | (INT8: scales) | barriers
  uint8_t* sQ = base;
  uint8_t* raw = sQ + 2 * kTile16;
  uint8_t* ring = raw + (INT8 ? kRaw * kTile8 : 0);
  float* scales = reinterpret_cast<float*>(ring + (INT8 ? kRing8 : kRing16) * kTile16);
  FullBars* bars = reinterpret_cast<FullBars*>(reinterpret_cast<uint8_t*>(scales) + (INT8 ? kScaleRing * 2 * kTileKeys * 4 : 0));
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing16; ++i) {
      mbar_init(&bars->full[i], INT8 ? kWidenThreads : 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&bars->raw_full[i], 1);
      mbar_init(&bars->raw_empty[i], kWidenThreads);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_ready[i], 128);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 128);
      mbar_init(&bars->o_full[i], 1);
    }
    for (int i = 0; i < kScaleRing; ++i) mbar_init(&bars->scales[i], 32);
    mbar_init(&bars->fix, 1);
    mbar_init(&bars->ml, 128);
    mbar_init(&bars->done, 1);
    bars->abort_flag = 0;
    bars->bad_page = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(&bars->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  pdl_trigger();
  if (warp < 8) {
    if constexpr (INT8) regs_up<kSoftRegs8>();
    softmax_role<QK_F16, PV_F16, INT8, MOD>(p, bars, tmem, sQ, scales, warp >> 2, abort_flag);
  } else if (warp < 12) {
    if constexpr (INT8) regs_down<kMiscRegs8>();
    if (warp == 8) {
      if ((threadIdx.x & 31) == 0)
        mma_role<QK_F16, PV_F16, INT8>(p, bars, tmem, smem_u32(sQ), smem_u32(ring), abort_flag);
    } else if (warp == 9) {
      load_role<INT8>(p, tm_k, tm_v, bars, INT8 ? raw : ring, scales, abort_flag);
    }
  } else {
    if constexpr (INT8) {
      regs_down<kWidenRegs>();
      widen_role(p, bars, ring, raw, threadIdx.x - kThreads16, abort_flag);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, kTmemCols);
  if (threadIdx.x == 0)
    p.errors[blockIdx.x] = (bars->abort_flag ? kDevTimeout : 0u) | (bars->bad_page ? kDevBadPage : 0u);
}

// --------------------------------------------------------------- few rows
// INT8 caches, items of up to 16 rows (one token of up to 16 heads a KV head):
// the tensor core's tiles would be empty but for a few rows, and its operands
// have to pass through shared memory once more as 16-bit tiles. Here twelve
// warps take groups of 16 keys in turn, read the codes straight into the register
// layout of m16n8k16 products (rows of Q x 8 keys x 16 dims, rows x 8 dims x 16
// keys) and widen them there. The two contractions may take their indices in
// any order, and keys and output columns may be permuted, which is used so that
// every thread reads 16 consecutive codes at a time, without bank conflicts:
//   S: thread (g, c) = (lane / 4, lane % 4) holds, of key row 4 (g % 2) + g / 2
//      of eight, the dims 16 c .. and 64 + 16 c .. (16 each);
//   O: of keys c, c + 4, c + 8, c + 12 the dims 16 (4 (g % 2) + g / 2) .. (16).
// Each warp has its own running maximum, sum and output; they are joined at the
// segment's end. Schedule, parts and merge are as above.
//
// Bound by the integer pipe: widening a code takes 1.25 (K) and 2 (V) of its
// instructions, 530 of some 1,000 issue slots a tile and scheduler. 16 tokens on
// 16,384, 32/8 heads: 106 us, 5.2 TB/s, against 198 us through the tensor core's
// path; one on 65,536, 24/2 heads: 17.5 against 26.3; 64 on 2,048, 32/8: 70
// against 173. From 17 rows on every further 16 would widen all codes again.
// Twelve warps of 152 registers: eight of 168 took 155 us for the first of these.
constexpr int kFewRows = 16, kFewWarps = 12, kFewThreads = 32 * (kFewWarps + 4);   // (the loader's warpgroup last)
constexpr int kFewGroup = 16, kFewGroups = kTileKeys / kFewGroup;   // keys a warp takes at once; such groups of a tile
constexpr int kFewRing = 3;
constexpr int kFewRegs = 152, kFewLoadRegs = 56;
constexpr int kFewLaunchRegs = 32 * kFewWarps * kFewRegs + 128 * kFewLoadRegs;
constexpr uint32_t kFewStage = 2 * kTile8 + 2 * kTileKeys * 4;   // K, V, their scales (1 KB)
constexpr int kFewPitch = DSA_HEAD_DIM + 4;            // floats between rows of a warp's output

struct FewBars {
  uint64_t full[kFewRing], empty[kFewRing];
  int abort_flag, bad_page;
  float2 ml[kFewWarps][kFewRows];
};

constexpr size_t kFewJoin = sizeof(float) * kFewWarps * kFewRows * kFewPitch;
constexpr size_t few_smem() {
  return kFewRing * kFewStage + kFewJoin + sizeof(FewBars);
}

// One stage holds a tile's keys, values and scales.
__device__ __forceinline__ void few_load(const FullParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                         FewBars* bars, uint8_t* ring, volatile int* abort_flag) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  RingPos pos;
  bool bad = false, ok = true;
  Walk walk(p);
  Segment s;
  while (ok && walk.next(p, &s)) {
    long long rows = 0;
    for (int t = s.t0; t < s.t1; ++t) {
      // cache rows of 32 tiles, one a lane
      if (((t - s.t0) & 31) == 0)
        rows = t + lane < s.t1 ? cache_row(p.pg, s.w.b, p.cap, (s.w.tile0 + t + lane) * kTileKeys, &bad) : 0;
      const long long first = __shfl_sync(0xffffffffu, rows, (t - s.t0) & 31);
      if (pos.round > 0 && !warp_wait(&bars->empty[pos.stage], (pos.round - 1) & 1, abort_flag)) {
        ok = false;
        break;
      }
      uint8_t* dst = ring + pos.stage * kFewStage;
      uint64_t* bar = &bars->full[pos.stage];
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, 2 * kTile8);
        tma_load_3d(dst, &tm_k, bar, 0, s.w.g, static_cast<int>(first));
        tma_load_3d(dst + kTile8, &tm_v, bar, 0, s.w.g, static_cast<int>(first));
      }
      float* sc = reinterpret_cast<float*>(dst + 2 * kTile8);
      const int key = (s.w.tile0 + t) * kTileKeys;
#pragma unroll
      for (int i = 0; i < kTileKeys / 32; ++i) {
        const int r = i * 32 + lane;
        const bool in = key + r >= s.w.lo && key + r < s.w.hi;
        const long long at = in ? (first + r) * p.Hkv + s.w.g : 0;
        cp_async4(sc + r, p.k_scale + at, in);
        cp_async4(sc + kTileKeys + r, p.v_scale + at, in);
      }
      cp_async_arrive(bar);
      __syncwarp();
      pos.step(kFewRing);
    }
  }
  if (bad) bars->bad_page = 1;
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  if (lane == 0) {
    // (as load_role: no copy in flight at the end)
    for (int q = 0; q < kFewRing; ++q) {
      const uint32_t uses = pos.round + (q < pos.stage ? 1 : 0);
      if (uses == 0) continue;
      const long long t0 = clock64();
      while (!mbar_try_wait(&bars->full[q], (uses - 1) & 1) && clock64() - t0 < kWaitBudgetCycles) {
      }
    }
  }
}

// SPLIT: the weights go as BF16 pairs (an FP16 query, see split_p). MOD as above.
template <bool SPLIT, bool MOD>
__device__ __forceinline__ void few_role(const FullParams& p, FewBars* bars, const uint8_t* ring, float* join,
                                         volatile int* abort_flag) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int perm = 4 * (g & 1) + (g >> 1);             // key row, and 16-byte column, of g
  uint32_t before = 0;                                  // tiles of the segments before
  Walk walk(p);
  Segment s;
  while (walk.next(p, &s)) {
    // queries: rows g and g + 8, this thread's 32 dims
    uint32_t q[8][4];
    int at[2], lo[2];
    float slope[2], unit[2];                            // unit: log2 units per unit of S, without the key's scale
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = imin(g + 8 * i, s.w.nrows - 1), tok = r / p.G, head = s.w.g * p.G + (r - tok * p.G);
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(p.q) + ((static_cast<long long>(s.w.q0) + tok) * p.Hq + head) * DSA_HEAD_DIM);
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 u = __ldg(src + (j >> 1) * 8 + 2 * c + (j & 1));
        w[4 * j] = u.x;
        w[4 * j + 1] = u.y;
        w[4 * j + 2] = u.z;
        w[4 * j + 3] = u.w;
      }
      unit[i] = p.scale_log2;
      if constexpr (!SPLIT) {   // a BF16 row: to FP16, its largest exponent to 14 (see softmax_role)
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = row_exponent(top);
        const float f0 = __int_as_float((127 - ex / 2) << 23), f1 = __int_as_float((127 - (ex - ex / 2)) << 23);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack2<true>(__uint_as_float(w[e] << 16) * f0 * f1, __uint_as_float(w[e] & 0xffff0000u) * f0 * f1);
        unit[i] = row_unit(p.scale_log2, ex);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q[j][i] = w[2 * j];
        q[j][2 + i] = w[2 * j + 1];
      }
      at[i] = s.w.past + tok;
      lo[i] = imax(s.w.first, p.window > 0 ? at[i] - p.window + 1 : 0);
      slope[i] = MOD && p.slopes ? p.slopes[head] * 1.4426950408889634f : 0.f;
    }
    const int pos0 = s.w.past, lo1 = imax(s.w.first, p.window > 0 ? s.w.past + (s.w.nrows - 1) / p.G - p.window + 1 : 0);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // (m in log2 units)
    float o[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const int groups = (s.t1 - s.t0) * kFewGroups;
    for (int grp = warp; grp < groups; grp += kFewWarps) {
      const uint32_t tile = grp / kFewGroups, use = before + tile, stage = use % kFewRing;
      const int first = (grp % kFewGroups) * kFewGroup;   // within the tile
      if (!warp_wait(&bars->full[stage], (use / kFewRing) & 1, abort_flag)) break;
      const uint8_t* src = ring + stage * kFewStage + first * 128;
      // S of 2 x 8 keys
      uint4 u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = (j >> 1) * 8 + perm, chunk = (j & 1) * 4 + c;
        u[j] = *reinterpret_cast<const uint4*>(src + row * 128 + ((chunk ^ (row & 7)) << 4));
      }
      float z[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint4& x = u[2 * n + j];
            const uint32_t y = w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w;
            const uint32_t b[2] = {widen2<true>(y, 0), widen2<true>(y, 1)};
            mma_16816<true>(z[n], q[4 * j + w], b);
          }
      src += kTile8;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = 4 * j + c;
        u[j] = *reinterpret_cast<const uint4*>(src + row * 128 + ((perm ^ (row & 7)) << 4));
      }
      // logits: z[n][2 i + e] is row i's, key 8 n + 4 e + c
      const float* sc = reinterpret_cast<const float*>(ring + stage * kFewStage + 2 * kTile8) + first + c;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[n][e] *= sc[8 * n + 4 * (e & 1)];
      const int key0 = (s.w.tile0 + s.t0 + static_cast<int>(tile)) * kTileKeys;
      if constexpr (MOD) {   // to log2 units
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[n][e] *= unit[e >> 1];
        if (p.softcap > 0.f) cap_scores<8, false>(&z[0][0], 1.0f, p);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            z[n][e] = fmaf(slope[e >> 1], static_cast<float>(key0 + first + 8 * n + 4 * (e & 1) + c - at[e >> 1]), z[n][e]);
      }
      if (key0 + kTileKeys - 1 > pos0 || key0 < lo1) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + first + 8 * n + 4 * (e & 1) + c;
            if (key < lo[e >> 1] || key > at[e >> 1]) z[n][e] = -INFINITY;
          }
      }
      float top[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        top[i] = fmaxf(fmaxf(z[0][2 * i], z[0][2 * i + 1]), fmaxf(z[1][2 * i], z[1][2 * i + 1])) * (MOD ? 1.0f : unit[i]);
      if (__any_sync(0xffffffffu, top[0] > m[0] + kRaise || top[1] > m[1] + kRaise)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
          const float to = fmaxf(m[i], top[i]);
          const float f = m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - to);
          m[i] = to;
          l[i] *= f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j][2 * i] *= f;
            o[j][2 * i + 1] *= f;
          }
        }
      }
      uint32_t a[4], al[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mc = m[i] == -INFINITY ? 0.f : kLift - m[i], un = MOD ? 1.0f : unit[i];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float x = fast_exp2(fmaf(z[n][2 * i], un, mc)), y = fast_exp2(fmaf(z[n][2 * i + 1], un, mc));
          l[i] += x + y;
          x *= sc[kTileKeys + 8 * n];
          y *= sc[kTileKeys + 8 * n + 4];
          a[2 * n + i] = pack2<false>(x, y);
          if constexpr (SPLIT)
            al[2 * n + i] = pack2<false>(x - __uint_as_float(a[2 * n + i] << 16),
                                         y - __uint_as_float(a[2 * n + i] & 0xffff0000u));
        }
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const auto word = [&](const uint4& x) { return w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w; };
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // byte e of two keys, side by side
          const uint32_t b[2] = {widen_pair(word(u[0]), word(u[1]), e), widen_pair(word(u[2]), word(u[3]), e)};
          mma_16816<false>(o[4 * w + e], a, b);
          if constexpr (SPLIT) mma_16816<false>(o[4 * w + e], al, b);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->empty[stage]);
    }
    before += s.t1 - s.t0;
    // the warps' states, joined
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (c == 0) bars->ml[warp][g + 8 * i] = make_float2(m[i], l[i]);
      // columns 2 c and 2 c + 1 are dims 16 c .. and 64 + 16 c ..
      float* d = join + (warp * kFewRows + g + 8 * i) * kFewPitch + 16 * c;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(d + 64 * e + j) =
              make_float4(o[j][2 * i + e], o[j + 1][2 * i + e], o[j + 2][2 * i + e], o[j + 3][2 * i + e]);
    }
    named_bar_sync(1, 32 * kFewWarps);
    if (threadIdx.x < 16 * kFewRows) {   // 16 threads a row
      const int r = threadIdx.x >> 4, d = (threadIdx.x & 15) * 8;
      float mj = -INFINITY, lj = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) mj = fmaxf(mj, bars->ml[w][r].x);
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const float2 v = bars->ml[w][r];
        const float f = v.x == -INFINITY ? 0.f : fast_exp2(v.x - mj);
        lj = fmaf(v.y, f, lj);
        const float* y = join + (w * kFewRows + r) * kFewPitch + d;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(y[e], f, x[e]);
      }
      if (r < s.w.nrows) {
        const int tok = r / p.G, head = s.w.g * p.G + (r - tok * p.G);
        const long long row = (static_cast<long long>(s.w.q0) + tok) * p.Hq + head;
        if (s.whole) {
          const float norm = lj > 0.f ? 1.0f / lj : 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= norm;
          if (p.lse && d == 0) p.lse[row] = lj > 0.f ? (mj - kLift + log2f(lj)) * 0.6931471805599453f : -INFINITY;
          if (p.out_dtype == DSA_FP32) {
            float4* to = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * DSA_HEAD_DIM + d);
            to[0] = make_float4(x[0], x[1], x[2], x[3]);
            to[1] = make_float4(x[4], x[5], x[6], x[7]);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = p.out_dtype == DSA_FP16 ? pack2<true>(x[2 * e], x[2 * e + 1]) : pack2<false>(x[2 * e], x[2 * e + 1]);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * DSA_HEAD_DIM + d) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float* part = p.partial + static_cast<long long>(s.part) * p.part_rows * (DSA_HEAD_DIM + 2);
          if (d == 0) *reinterpret_cast<float2*>(part + p.part_rows * DSA_HEAD_DIM + 2 * r) = make_float2(mj, lj);
          part += d * p.part_rows + 4 * r;
          *reinterpret_cast<float4*>(part) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(part + 4 * p.part_rows) = make_float4(x[4], x[5], x[6], x[7]);
        }
      }
    }
    named_bar_sync(1, 32 * kFewWarps);
  }
}

template <bool SPLIT, bool MOD>
__global__ void __launch_bounds__(kFewThreads, 1)
    full_attn_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ FullParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) p.errors[blockIdx.x] = kDevBounds;
    return;
  }
  uint8_t* ring = smem_raw;
  float* join = reinterpret_cast<float*>(ring + kFewRing * kFewStage);
  FewBars* bars = reinterpret_cast<FewBars*>(reinterpret_cast<uint8_t*>(join) + kFewJoin);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFewRing; ++i) {
      mbar_init(&bars->full[i], 33);   // the copies' bytes, and 32 lanes' scales
      mbar_init(&bars->empty[i], kFewGroups);
    }
    bars->abort_flag = 0;
    bars->bad_page = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_trigger();
  if (threadIdx.x < 32 * kFewWarps) {
    regs_up<kFewRegs>();
    few_role<SPLIT, MOD>(p, bars, ring, join, &bars->abort_flag);
  } else {
    regs_down<kFewLoadRegs>();
    if (threadIdx.x < 32 * (kFewWarps + 1)) few_load(p, tm_k, tm_v, bars, ring, &bars->abort_flag);
  }
  __syncthreads();
  if (threadIdx.x == 0)
    p.errors[blockIdx.x] = (bars->abort_flag ? kDevTimeout : 0u) | (bars->bad_page ? kDevBadPage : 0u);
}

// ------------------------------------------------------------------ merge
// Joins the parts of the items that more than one block worked on. A thread
// block takes four query rows; 128 threads hold a row's four dims each, and
// `groups` such sets take every groups-th part.
struct MergeParams {
  const float* partial;
  void* out;
  float* lse;
  int part_rows, out_dtype, groups, splits, blocks;
  int first_cta[kMaxCtas], last_cta[kMaxCtas];   // blocks that hold split item i's parts
};
constexpr int kMergeRows = 4, kMergeSet = 32 * kMergeRows, kMaxGroups = 8;

__global__ void __launch_bounds__(kMergeSet * kMaxGroups)
    full_attn_merge_kernel(const __grid_constant__ FullParams p, const __grid_constant__ MergeParams mp) {
  __shared__ float4 s_o[kMergeSet * kMaxGroups];
  __shared__ float2 s_ml[kMergeRows * kMaxGroups];
  __shared__ uint32_t s_err;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (threadIdx.x == 0) s_err = 0u;
    __syncthreads();
    pdl_wait();
    uint32_t e = 0;
    for (int c = threadIdx.x; c < mp.blocks; c += blockDim.x) e |= __ldcg(p.errors + c);
    if (e) atomicOr(&s_err, e);
    __syncthreads();
    if (threadIdx.x == 0) *p.status = s_err;
  }
  if (mp.splits == 0) return;
  const int set = threadIdx.x / kMergeSet, t = threadIdx.x % kMergeSet;
  const int rr = t % kMergeRows, d4 = t / kMergeRows;   // (64 consecutive bytes of a part for four lanes)
  const int c0 = mp.first_cta[blockIdx.y], c1 = mp.last_cta[blockIdx.y];
  // the item is the one block c1's run begins in
  const FullParams::Run run = p.run[c1];
  const Item w = make_item(p, run.item, run.b);
  const int pr = blockIdx.x * kMergeRows + rr;
  pdl_wait();
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (pr < w.nrows) {
    const long long pitch = static_cast<long long>(mp.part_rows) * (DSA_HEAD_DIM + 2);
    const long long at_o = (static_cast<long long>(d4) * mp.part_rows + pr) * 4;
    const long long at_ml = static_cast<long long>(mp.part_rows) * DSA_HEAD_DIM + 2 * pr;
    // four parts at a time: all their loads in flight together
    for (int c = c0 + set; c <= c1; c += 4 * mp.groups) {
      float2 x[4];
      float4 y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int ck = c + k * mp.groups;
        x[k] = make_float2(-INFINITY, 0.f);
        if (ck > c1) continue;
        const float* q = mp.partial + (2 * ck + (ck == c0 ? 1 : 0)) * pitch;
        x[k] = __ldcg(reinterpret_cast<const float2*>(q + at_ml));
        y[k] = __ldcg(reinterpret_cast<const float4*>(q + at_o));
      }
      const float to = fmaxf(m, fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)));
      if (to == -INFINITY) continue;
      const float old = m == -INFINITY ? 0.f : fast_exp2(m - to);
      l *= old;
      o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
      m = to;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (x[k].x == -INFINITY) continue;
        const float f = fast_exp2(x[k].x - m);
        l = fmaf(x[k].y, f, l);
        o.x = fmaf(y[k].x, f, o.x);
        o.y = fmaf(y[k].y, f, o.y);
        o.z = fmaf(y[k].z, f, o.z);
        o.w = fmaf(y[k].w, f, o.w);
      }
    }
  }
  if (mp.groups > 1) {
    if (d4 == 0) s_ml[set * kMergeRows + rr] = make_float2(m, l);
    s_o[threadIdx.x] = o;
    __syncthreads();
    if (set != 0) return;
    float mm = -INFINITY;
    for (int k = 0; k < mp.groups; ++k) mm = fmaxf(mm, s_ml[k * kMergeRows + rr].x);
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < mp.groups; ++k) {
      const float2 x = s_ml[k * kMergeRows + rr];
      if (x.x == -INFINITY) continue;
      const float f = fast_exp2(x.x - mm);
      const float4 y = s_o[k * kMergeSet + t];
      l = fmaf(x.y, f, l);
      o.x = fmaf(y.x, f, o.x);
      o.y = fmaf(y.y, f, o.y);
      o.z = fmaf(y.z, f, o.z);
      o.w = fmaf(y.w, f, o.w);
    }
    m = mm;
  }
  if (pr >= w.nrows) return;
  const float norm = l > 0.f ? 1.0f / l : 0.f;
  const int r = w.row0 + pr, tok = r / p.G;
  const long long row = (static_cast<long long>(w.q0) + tok) * p.Hq + w.g * p.G + (r - tok * p.G);
  const float4 v = make_float4(o.x * norm, o.y * norm, o.z * norm, o.w * norm);
  if (mp.out_dtype == DSA_FP32)
    *(reinterpret_cast<float4*>(static_cast<float*>(mp.out) + row * DSA_HEAD_DIM) + d4) = v;
  else
    *(reinterpret_cast<uint2*>(static_cast<uint16_t*>(mp.out) + row * DSA_HEAD_DIM) + d4) =
        mp.out_dtype == DSA_FP16 ? make_uint2(pack2<true>(v.x, v.y), pack2<true>(v.z, v.w))
                                 : make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
  if (mp.lse && d4 == 0) mp.lse[row] = l > 0.f ? (m - kLift + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// -------------------------------------------------------------------- host
int check_full(const dsa_full_problem* p) {
  if (!p) return report_error(DSA_ERR_INVALID_ARG, "problem is NULL");
  if (p->batch < 1 || p->batch > DSA_MAX_BATCH)
    return report_errorf(DSA_ERR_INVALID_ARG, "batch %d outside 1..%d", p->batch, DSA_MAX_BATCH);
  if (p->head_dim != DSA_HEAD_DIM)
    return report_errorf(DSA_ERR_UNSUPPORTED, "head_dim must be %d (got %d)", DSA_HEAD_DIM, p->head_dim);
  if (p->num_q_heads < 1 || p->num_kv_heads < 1 || p->num_q_heads % p->num_kv_heads != 0 || p->num_q_heads > 65535)
    return report_errorf(DSA_ERR_INVALID_ARG, "num_q_heads %d must be a multiple of num_kv_heads %d, at most 65535",
                         p->num_q_heads, p->num_kv_heads);
  if (p->cache_capacity < 1 || p->cache_capacity > (1 << 30))
    return report_errorf(DSA_ERR_INVALID_ARG, "cache_capacity %d invalid", p->cache_capacity);
  if (p->window < 0) return report_errorf(DSA_ERR_INVALID_ARG, "window %d < 0", p->window);
  if (!(p->softmax_scale >= 0.0f) || std::isinf(p->softmax_scale))
    return report_error(DSA_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
  if (!(p->softcap >= 0.0f) || std::isinf(p->softcap))
    return report_error(DSA_ERR_INVALID_ARG, "softcap must be finite and >= 0");
  if (p->q_dtype != DSA_BF16 && p->q_dtype != DSA_FP16)
    return report_error(DSA_ERR_UNSUPPORTED, "q_dtype must be BF16 or FP16");
  if (p->kv_dtype != DSA_BF16 && p->kv_dtype != DSA_FP16 && p->kv_dtype != DSA_INT8)
    return report_error(DSA_ERR_UNSUPPORTED, "kv_dtype must be BF16, FP16 or INT8");
  if (p->q_dtype == DSA_FP16 && p->kv_dtype == DSA_BF16)
    return report_error(DSA_ERR_UNSUPPORTED, "FP16 query with a BF16 cache is not built");
  if (p->out_dtype != DSA_BF16 && p->out_dtype != DSA_FP16 && p->out_dtype != DSA_FP32)
    return report_error(DSA_ERR_UNSUPPORTED, "out_dtype must be BF16, FP16 or FP32");
  long long rows = 0;
  for (int b = 0; b < p->batch; ++b) {
    const int S = p->q_len[b], T = p->total_len[b], F = p->first_key[b];
    if (S < 0) return report_errorf(DSA_ERR_INVALID_ARG, "q_len[%d] = %d < 0", b, S);
    if (T < S || T > p->cache_capacity)
      return report_errorf(DSA_ERR_INVALID_ARG, "total_len[%d] = %d outside q_len..cache_capacity (%d..%d)", b, T, S,
                           p->cache_capacity);
    if (T > DSA_MAX_CONTEXT) return report_errorf(DSA_ERR_UNSUPPORTED, "total_len[%d] = %d above %d", b, T, DSA_MAX_CONTEXT);
    if (F < 0 || F > T) return report_errorf(DSA_ERR_INVALID_ARG, "first_key[%d] = %d outside 0..total_len (%d)", b, F, T);
    rows += S;
  }
  if (rows * p->num_q_heads > 0x7fffffffLL)
    return report_error(DSA_ERR_UNSUPPORTED, "new tokens * num_q_heads must be below 2^31");
  return DSA_OK;
}

// Costs of a unit, in quarters of a tile of 256 rows: a tile of up to 128 rows
// takes the same loads and half the products; an item, its queries and output
// (8 / 20 / 40: 2,048 tokens on 2,048 48.5 / 45.4 / 45.2 us, 32 single tokens on
// 300 .. 8,192 keys 94.4 / 93.8 / 96.4 us); an item without a key, its zeros
// (2 / 4 / 8: 4 prompts of 2,048, left-padded by 0 .. 2,000, 101 / 77 / 79 us, 8 of
// 1,000 65 / 61 / 65 us).
constexpr int kCostRows = 4, kCostKeys = 3, kCostItem = 20, kCostEmpty = 4;

// Lays the items out over at most min(sms, kMaxCtas, units) blocks (fp: the
// problem and the runs, mp: the items that are split) and returns their number.
// A unit is a tile, or an item without one: a left-padded prompt has hundreds of
// those, which would take longer than its tiles if they fell to one block.
// *bytes gets the workspace that holds two parts of as many blocks as any device
// may use. (More SMs may lead to fewer blocks: cuts that fall into the same tile
// are one.)
constexpr size_t kPartialAt = 256 + ((kMaxCtas * 4 + 255) / 256) * 256;

int schedule(const dsa_full_problem* p, int sms, FullParams* fp, MergeParams* mp, size_t* bytes) {
  fp->B = p->batch;
  fp->Hq = p->num_q_heads;
  fp->Hkv = p->num_kv_heads;
  fp->G = p->num_q_heads / p->num_kv_heads;
  fp->cap = p->cache_capacity;
  fp->window = p->window;
  fp->part_rows = 0;
  for (int b = 0; b < p->batch; ++b) {
    const long long rows = static_cast<long long>(p->q_len[b]) * fp->G;
    fp->seq[b + 1].q0 = fp->seq[b].q0 + p->q_len[b];
    fp->seq[b + 1].item0 = fp->seq[b].item0 + static_cast<int>((rows + kItemRows - 1) / kItemRows) * p->num_kv_heads;
    fp->seq[b].T = p->total_len[b];
    fp->seq[b].first = p->first_key[b];
    fp->part_rows = imax(fp->part_rows, static_cast<int>(rows < kItemRows ? rows : kItemRows));
  }
  fp->part_rows = (fp->part_rows + 3) & ~3;   // parts stay 16-byte aligned
  const int items = fp->seq[p->batch].item0;
  const auto item_cost = [](const Item& w) { return w.ntiles > 0 ? kCostItem : kCostEmpty; };
  long long cost = 0, units = 0;
  for (int i = 0, at = 0; i < items; ++i) {
    const Item w = make_item(*fp, i, at);
    at = w.b;
    cost += item_cost(w) + static_cast<long long>(w.ntiles) * (w.nrows > kSlotRows ? kCostRows : kCostKeys);
    units += imax(w.ntiles, 1);
  }
  const int most = static_cast<int>(std::min<long long>(kMaxCtas, std::max(units, 1LL)));
  const int want = imin(sms, most);
  *bytes = kPartialAt + static_cast<size_t>(2) * most * fp->part_rows * (DSA_HEAD_DIM + 2) * 4;
  int blocks = 0;
  if (units <= want) {
    // one each, for an item costs every block the same (16 tiles, 24/2 heads:
    // 9.5 us, against 10.1 with the cuts below, of which some fall into an item's
    // cost and leave other blocks two tiles; 4 x 600 keys 9.3 against 10.9)
    for (int i = 0, b = 0; i < items; ++i) {
      const Item w = make_item(*fp, i, b);
      b = w.b;
      for (int t = 0; t < imax(w.ntiles, 1); ++t) fp->run[blocks++] = FullParams::Run{i, t, b, 0};
    }
  } else {
    // run k begins where the costs reach k / want of their sum
    long long at = 0;
    for (int i = 0, b = 0, k = 0; i < items; ++i) {
      const Item w = make_item(*fp, i, b);
      b = w.b;
      const int unit = w.nrows > kSlotRows ? kCostRows : kCostKeys;
      const long long end = at + item_cost(w) + static_cast<long long>(w.ntiles) * unit;
      for (; k < want && cost * k < end * want; ++k) {
        const long long x = cost * k / want - at - item_cost(w);
        const int tile = x > 0 ? static_cast<int>(x / unit) : 0;
        if (blocks > 0 && fp->run[blocks - 1].item == i && fp->run[blocks - 1].tile >= tile) continue;
        fp->run[blocks++] = FullParams::Run{i, tile, b, 0};
      }
      at = end;
    }
  }
  fp->run[blocks] = FullParams::Run{items, 0, p->batch, 0};
  mp->splits = 0;
  int parts = 1;
  for (int c = 1; c < blocks; ++c) {
    if (fp->run[c].tile == 0) continue;
    const int n = mp->splits;
    if (n > 0 && mp->last_cta[n - 1] == c - 1 && fp->run[c].item == fp->run[c - 1].item) {
      mp->last_cta[n - 1] = c;
    } else {
      mp->first_cta[n] = c - 1;
      mp->last_cta[n] = c;
      ++mp->splits;
    }
    parts = imax(parts, c - mp->first_cta[mp->splits - 1] + 1);
  }
  mp->groups = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : kMaxGroups;   // four parts a thread at once
  return blocks;
}

// Launches one of two kernels of a family (with and without MOD). Where warps
// change their register counts, those must fit into what the block is launched
// with: a warp that asks for more would wait for ever.
template <typename K>
cudaError_t launch_one(const char* name, K* const (&kernels)[2], bool mod, std::atomic<int> (&regs)[2], int need, int blocks,
                       int threads, size_t smem, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const FullParams& fp,
                       cudaStream_t st) {
  K* const kern = kernels[mod];
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (need > 0 && regs[mod].load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes a;
    if ((e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(kern))) != cudaSuccess) return e;
    if (a.numRegs * threads < need) return cudaErrorInvalidConfiguration;
    regs[mod].store(a.numRegs, std::memory_order_relaxed);
  }
  return launch_kernel(name, kern, dim3(blocks), dim3(threads), smem, st, false, tm_k, tm_v, fp);
}

template <bool QK_F16, bool PV_F16, bool INT8>
cudaError_t launch_full(bool mod, int blocks, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const FullParams& fp,
                        cudaStream_t st) {
  static std::atomic<int> regs[2];
  using K = void(const CUtensorMap, const CUtensorMap, const FullParams);
  K* const kernels[2] = {full_attn_kernel<QK_F16, PV_F16, INT8, false>, full_attn_kernel<QK_F16, PV_F16, INT8, true>};
  return launch_one("full_attn_kernel", kernels, mod, regs, INT8 ? kRegs8 : 0, blocks, INT8 ? kThreads8 : kThreads16,
                    full_smem<INT8>(), tm_k, tm_v, fp, st);
}

template <bool SPLIT>
cudaError_t launch_few(bool mod, int blocks, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const FullParams& fp,
                       cudaStream_t st) {
  static std::atomic<int> regs[2];
  using K = void(const CUtensorMap, const CUtensorMap, const FullParams);
  K* const kernels[2] = {full_attn_few_kernel<SPLIT, false>, full_attn_few_kernel<SPLIT, true>};
  return launch_one("full_attn_few_kernel", kernels, mod, regs, kFewLaunchRegs, blocks, kFewThreads, few_smem(), tm_k, tm_v,
                    fp, st);
}

// What cap_scores takes of a cap. A cap beyond 1e30 leaves every logit as it is and
// is taken as that; 1 / cap stays below 1e38, a cap that small makes all logits 0.
void cap_fold(float softcap, FullParams* fp) {
  fp->softcap = std::min(softcap, 1e30f);
  if (!(softcap > 0.0f)) return;
  const float c = fp->scale_log2;
  fp->cap_log2 = fp->softcap * 1.4426950408889634f;
  fp->cap_inv = std::min(1.0f / fp->cap_log2, 1e38f);
  const float ys = std::min(c * fp->cap_inv, 1e38f);
  const bool fold = ys >= 0x1p-11f && ys <= 0x1p11f && c >= 0x1p-16f && c <= 0x1p16f;
  fp->cap_pre = fold ? 1.0f : ys;
  fp->cap_ys = fold ? ys : 1.0f;
}

int full_call(const dsa_full_problem* p, const dsa_kv_pages* pages, const void* q, const void* k, const void* v,
              const float* ks, const float* vs, const float* slopes, void* out, float* lse, void* ws,
              size_t ws_bytes, void* stream) {
  if (int rc = check_full(p)) return rc;
  Paging pg{};
  if (pages)
    if (int rc = check_full_pages(p, pages, &pg)) return rc;
  if (!q || !k || !v || !out) return report_error(DSA_ERR_INVALID_ARG, "a required tensor pointer is NULL");
  const auto off = [](const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) != 0; };
  if (p->kv_dtype == DSA_INT8) {
    if (!ks || !vs) return report_error(DSA_ERR_INVALID_ARG, "INT8 cache needs k_scale and v_scale");
  } else if (ks || vs) {
    return report_error(DSA_ERR_INVALID_ARG, "k_scale/v_scale must be NULL unless the cache is INT8");
  }
  if (off(q, 16) || off(k, 16) || off(v, 16) || off(out, 16))
    return report_error(DSA_ERR_MISALIGNED, "q, k, v and out must be 16-byte aligned");
  if (off(ks, 4) || off(vs, 4) || off(slopes, 4) || off(lse, 4))
    return report_error(DSA_ERR_MISALIGNED, "scales, slopes and lse must be 4-byte aligned");
  int sms = 0;
  const bool device = current_device(&sms) == DSA_OK;
  FullParams fp{};
  MergeParams mp;
  size_t need = 0;
  const int blocks = schedule(p, device ? sms : kMaxCtas, &fp, &mp, &need);
  if (int rc = check_call_workspace(ws, ws_bytes, need)) return rc;
  if (!device) return current_device(&sms);
  if (fp.seq[p->batch].q0 == 0) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, 4, static_cast<cudaStream_t>(stream));   // the status word
    return e == cudaSuccess ? DSA_OK : report_errorf(DSA_ERR_CUDA, "status clear: %s", cudaGetErrorString(e));
  }
  const long long rows = pages ? static_cast<long long>(pages->num_blocks) * pages->block_size
                               : static_cast<long long>(p->batch) * p->cache_capacity;
  if (rows >= (1LL << 31)) return report_error(DSA_ERR_UNSUPPORTED, "the caches must hold fewer than 2^31 tokens");
  const int elem = p->kv_dtype == DSA_INT8 ? 1 : 2;
  CUtensorMap tm_k, tm_v;
  if (int rc = kv_tile_map(&tm_k, k, rows, p->num_kv_heads, elem)) return rc;
  if (int rc = kv_tile_map(&tm_v, v, rows, p->num_kv_heads, elem)) return rc;
  fp.q = q;
  fp.k_scale = ks;
  fp.v_scale = vs;
  fp.slopes = slopes;
  fp.out = out;
  fp.lse = lse;
  fp.status = static_cast<uint32_t*>(ws);
  fp.errors = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + 256);
  fp.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kPartialAt);
  fp.q_dtype = p->q_dtype;
  fp.out_dtype = p->out_dtype;
  const float scale = p->softmax_scale > 0.0f ? p->softmax_scale : 1.0f / std::sqrt(static_cast<float>(p->head_dim));
  fp.scale_log2 = std::max(scale * 1.4426950408889634f, kLeastUnit);
  cap_fold(p->softcap, &fp);
  fp.pg = pg;
  mp.partial = fp.partial;
  mp.out = out;
  mp.lse = lse;
  mp.part_rows = fp.part_rows;
  mp.out_dtype = p->out_dtype;
  mp.blocks = blocks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool mod = p->softcap > 0.0f || slopes != nullptr;
  cudaError_t e;
  if (p->kv_dtype == DSA_INT8 && fp.part_rows <= kFewRows)
    e = p->q_dtype == DSA_FP16 ? launch_few<true>(mod, blocks, tm_k, tm_v, fp, st)
                               : launch_few<false>(mod, blocks, tm_k, tm_v, fp, st);
  else if (p->kv_dtype == DSA_BF16) e = launch_full<false, false, false>(mod, blocks, tm_k, tm_v, fp, st);
  else if (p->kv_dtype == DSA_FP16) e = launch_full<true, true, false>(mod, blocks, tm_k, tm_v, fp, st);
  else if (p->q_dtype == DSA_FP16) e = launch_full<true, false, true>(mod, blocks, tm_k, tm_v, fp, st);
  else e = launch_full<false, false, true>(mod, blocks, tm_k, tm_v, fp, st);
  if (e == cudaSuccess) {
    const dim3 grid = mp.splits ? dim3((fp.part_rows + kMergeRows - 1) / kMergeRows, mp.splits) : dim3(1);
    e = launch_kernel("full_attn_merge_kernel", full_attn_merge_kernel, grid, dim3(kMergeSet * mp.groups), 0, st, true, fp, mp);
  }
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "full attention launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_full_attn_workspace_size(const dsa_full_problem* p) {
  if (check_full(p)) return 0;
  FullParams fp{};
  MergeParams mp;
  size_t bytes = 0;
  schedule(p, kMaxCtas, &fp, &mp, &bytes);
  return bytes;
}

extern "C" int dsa_full_attn(const dsa_full_problem* p, const void* q, const void* k, const void* v,
                             const float* k_scale, const float* v_scale, const float* slopes, void* out,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  reset_launches();
  return full_call(p, nullptr, q, k, v, k_scale, v_scale, slopes, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int dsa_full_attn_paged(const dsa_full_problem* p, const dsa_kv_pages* pages, const void* q,
                                   const void* k, const void* v, const float* k_scale, const float* v_scale,
                                   const float* slopes, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  reset_launches();
  if (!pages) return report_error(DSA_ERR_INVALID_ARG, "pages is NULL");
  return full_call(p, pages, q, k, v, k_scale, v_scale, slopes, out, lse, workspace, workspace_bytes, stream);
}
