// Beam search's selection: the `select` best of score_i + log_softmax(logits_i)
// over beams x vocabulary, per batch entry.
//
// Two launches. beam_scan_kernel reads every logit once. Its blocks, as many as
// are resident at once, take equal runs of tiles (1,024 16-byte vectors of a
// row), a run spanning the end of one row and the start of the next where it
// must; a row's part in a block is a slice. Of each slice a block keeps, side
// by side, the sum of exponentials and the values that can be among the best.
// The latter through a lower bound: every thread holds the largest value it
// has seen, a warp's j-th largest of those (j = select / 8 warps) is reached by
// j values of the warp, so the smallest of the eight warps' is reached by
// `select` values of the slice. Values that reach it -- a few times `select`
// in all, one comparison per thread and tile for the rest -- are appended to a
// list, of which what the final bound leaves goes to the workspace as it is.
// Only a list that gets long (ties, rising rows) is cut to its best `select`.
// Within a row totals are ordered as the logits are, so that loses nothing.
//
// Sums: a thread's is sum 2^(x H + c) with H = log2(e) rounded to fp32 and c an
// integer (a large value's, negated; it moves when a term would pass 2^30): one
// paired multiply-add and one 2^ a value, and sums of different c join by exact
// powers of two. A tile's 16 or 32 values are added in fp32, the tiles' sums with
// what each addition rounds off kept beside (a thread may have thousands of terms,
// and of equal ones every addition rounds the same way). A slice's joins as 64-bit
// fixed point (2^-36 of a term at the maximum). H's rounding scales
// every exponent by 1 - 1.3e-8, which the merge undoes at the maximum; what is
// left is 1.3e-8 of a term's distance from it.
//
// beam_merge_kernel joins the slices' sums of each row, bounds the candidates'
// totals in the same way, forms the totals of those that reach the bound in 64
// bits (rows have different offsets: totals may lie closer together than fp32
// tells apart) and ranks them by counting.
//
// What bounds it: large batches the scan's latency (11 instructions of a warp for
// 32 bf16 values keep the scheduler 50% busy, the memory is 45% busy: one tile is
// in flight while one is worked on, with two barriers every second tile), 32 x 8
// beams of 128,000 27 us, 2.4 TB/s, as fp32 35 us, 3.7 TB/s, of 6.8 measured; small
// ones the two launches and the merge's chain of dependent steps, 4 beams of 32,000
// 9.3 us; many beams with a large `select` the merge of up to 512 lists by one
// block, 64 beams of 200,000 with 64 selected 78 us. Beams of equal scores, as of a
// first step, are compared besides (see the merge).
//
// The order of a list depends on the order of execution; its keys are distinct
// (value, then token), so what is picked out of it does not.
#include <algorithm>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kBmThreads = 256;
constexpr int kBmWarps = kBmThreads / 32;
constexpr int kVecs = 4;            // 16-byte vectors a thread takes per tile
constexpr int kTileVecs = kBmThreads * kVecs;
constexpr int kKeep = 128;          // candidates a slice may hand on
constexpr int kDrain = 256;         // list entries that are cut to the best at once
constexpr int kGroup = 2;           // tiles between two looks at the list's length
constexpr int kMergeThreads = 1024;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMaxLists = 512;      // slices of one batch entry
constexpr int kRound = kMergeWarps;               // lists that the merge takes at once
constexpr int kMergeList = 2 * kRound * kKeep;    // room for their candidates, and as many left from before
constexpr int kBounds = 4;                        // values of a warp that go into the merge's bound
constexpr int kShare = kKeep / kMergeWarps;
// Scan blocks per SM (70 KB of shared memory each for 16-bit logits). With two,
// 32 x 8 beams of 128,000 took 30.3 us and not 28.9, in fp32 41.5 and not 36.9.
constexpr int kResident = 3;

struct SliceSum {
  unsigned long long sum;   // of 2^(x H + c) with the c of `max`, times 2^36; kNaN: a NaN or +infinity
  float max;
  int count;                // candidates
};
constexpr unsigned long long kNaN = ~0ull;

struct BeamParams {
  uint32_t* status;   // device status word: nothing can go wrong on the device
  const void* logits;
  const float* scores;
  const uint8_t* finished;
  unsigned long long* cands;   // [rows, slices, kKeep] keys (cand_key)
  SliceSum* sums;     // [rows, slices], slice 0 the row's first
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
  long long stride;   // elements between rows
  unsigned per, extra;         // units of a block: per, one more in the first `extra`
  int row_tiles;
  int beams, vocab, select, slices, pad;
  int elem;           // bytes of a logit
};

// Block c takes the units (tiles of all rows) [run_begin(c), run_begin(c + 1)).
__device__ __forceinline__ unsigned run_begin(const BeamParams& p, unsigned c) { return c * p.per + min(c, p.extra); }
__device__ __forceinline__ unsigned run_of(const BeamParams& p, unsigned u) {
  const unsigned head = p.extra * (p.per + 1);
  return u < head ? u / (p.per + 1) : p.extra + (u - head) / p.per;
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269502e0f;           // H
constexpr float kLog2eRest = 1.925963033e-8f;     // log2(e) - H
// Up to this size of a maximum its c is an exact integer that cancels it to
// about 1; rows beyond (masked with the type's lowest value throughout) take
// the differences from it instead.
constexpr float kFar = 1e7f;
__device__ __forceinline__ float exp_neg(float x) { return ex2_ftz(x * kLog2e); }
__device__ __forceinline__ float offset_of(float m) { return -rintf(m * kLog2e); }   // c
// 2^n for an integer n <= 0 (0 from 2^-126 down)
__device__ __forceinline__ float pow2_int(float n) {
  return n > -126.f ? __int_as_float((static_cast<int>(n) + 127) << 23) : 0.f;
}
// What joins a sum at maximum m to one at maximum `to`.
__device__ __forceinline__ float join_factor(float m, float to) {
  if (!(m > -INFINITY)) return 0.f;
  if (m == to) return 1.f;
  if (fabsf(m) <= kFar && fabsf(to) <= kFar) return pow2_int(offset_of(to) - offset_of(m));
  // (a far sum's terms are relative to its maximum, a near one's to its c)
  float f = exp_neg(m - to);
  if (fabsf(m) <= kFar) f *= ex2_ftz(-fmaf(m, kLog2e, offset_of(m)));
  if (fabsf(to) <= kFar) f *= ex2_ftz(fmaf(to, kLog2e, offset_of(to)));
  return f;
}

// A row candidate as one key: larger value first, then the lower token.
__device__ __forceinline__ unsigned long long cand_key(float v, int token) {
  return (static_cast<unsigned long long>(float_key(v)) << 32) | static_cast<uint32_t>(~token);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// The next value above a finite one (the smallest positive one above either 0).
__device__ __forceinline__ float next_above(float x) {
  const uint32_t k = float_key(x);
  return key_value(static_cast<unsigned long long>(k == 0x7ffffffeu ? 0x80000000u : k + 1u) << 32);
}

// A total with its place: larger total first, then the lower place. hi = 0:
// none.
struct Total {
  unsigned long long hi;
  uint32_t lo;        // ~place
};
__device__ __forceinline__ bool above(const unsigned long long& a, const unsigned long long& b) { return a > b; }
__device__ __forceinline__ bool above(const Total& a, const Total& b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
// Puts the best `k` of list[0..n) into out[0..k), largest first, by counting
// for every key those above it; places that have no key get `none`. n is at
// most kBmThreads, the keys are distinct. A whole block of NT threads calls it
// after a barrier that completes the list; `rank` is kBmThreads ints, out is
// not list.
template <int NT, typename K>
__device__ void rank_best(K* out, const K* list, int n, int k, K none, int* rank) {
  const int t = threadIdx.x;
  int width = 32;                       // keys side by side; the rest of the block shares the counting
  while (width < n) width <<= 1;
  const int parts = NT / width, part = t / width, i = t & (width - 1);
  if (t < kBmThreads) rank[t] = 0;
  if (t < k) out[t] = none;
  __syncthreads();
  if (i < n) {
    const K key = list[i];
    int above_it = 0;
    const int step = (n + parts - 1) / parts, end = min(n, (part + 1) * step);
    for (int j = part * step; j < end; ++j) above_it += above(list[j], key) ? 1 : 0;
    if (above_it) atomicAdd(&rank[i], above_it);
  }
  __syncthreads();
  if (t < n && rank[t] < k) out[rank[t]] = list[t];
  __syncthreads();
}

// Puts the best `k` of the n keys get(0) .. get(n - 1) into best[0..k), in
// order, kBmThreads at a time through `buf`. Returns how many there are.
template <int NT, typename K, class F>
__device__ int cut_to_best(K* best, F&& get, int n, int k, K none, K* buf, int* rank) {
  const int t = threadIdx.x;
  int have = 0;
  for (int at = 0; at < n;) {
    const int here = min(n - at, kBmThreads - have);
    if (t < have) buf[t] = best[t];
    else if (t < have + here) buf[t] = get(at + t - have);
    __syncthreads();
    at += here;
    rank_best<NT>(best, buf, have + here, k, none, rank);
    have = min(k, have + here);
  }
  return have;
}

// The j-th largest of the warp's keys (0 if it has fewer than j that are not 0).
__device__ __forceinline__ uint32_t warp_jth(uint32_t key, int j) {
  uint32_t top = 0;
  for (int i = 0; i < j; ++i) {
    top = __reduce_max_sync(0xffffffffu, key);
    if (top == 0u) break;
    const uint32_t holders = __ballot_sync(0xffffffffu, key == top);
    if ((threadIdx.x & 31) == __ffs(holders) - 1) key = 0u;
  }
  return top;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}

// The four bytes of two 16-bit values, or one fp32 value, as floats.
template <typename T>
__device__ __forceinline__ float2 two_of(const uint32_t* w, int i);
template <>
__device__ __forceinline__ float2 two_of<__nv_bfloat16>(const uint32_t* w, int i) {
  return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 two_of<__half>(const uint32_t* w, int i) {
  return __half22float2(*reinterpret_cast<const __half2*>(w + i));
}
template <>
__device__ __forceinline__ float2 two_of<float>(const uint32_t* w, int i) {
  return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}

// The list (of tokens): a group's values and what it may hold before it.
template <typename T>
constexpr int kListLen = kGroup * kTileVecs * (16 / static_cast<int>(sizeof(T))) + kDrain;

// The largest of a thread's values (a NaN is passed over).
template <typename T>
__device__ __forceinline__ float top_of(const uint4* v) {
  if constexpr (sizeof(T) == 4) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      top = fmaxf(top, fmaxf(fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y)),
                             fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w))));
    return top;
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    T2 top = *reinterpret_cast<const T2*>(&v[0].x);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __hmax2(top, *reinterpret_cast<const T2*>(w + e));
    }
    const float2 f = two_of<T>(reinterpret_cast<const uint32_t*>(&top), 0);
    return fmaxf(fmaxf(f.x, f.y), -INFINITY);   // NaN: -infinity
  }
}

// A bit for each of a thread's values that is at least `lim`, and which value a
// bit stands for. 16-bit values are compared two at a time, bits p and 16 + p for
// the p-th pair, with the least value of their type that is not below `lim`.
template <typename T>
__device__ __forceinline__ uint32_t reached(const uint4* v, float lim) {
  uint32_t hits = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(T) == 4) {
        if (__uint_as_float(w[e]) >= lim) hits |= 1u << (4 * i + e);
      } else {
        uint32_t mask;
        if constexpr (std::is_same<T, __half>::value)
          mask = __hge2_mask(*reinterpret_cast<const __half2*>(w + e), __half2half2(__float2half_ru(lim)));
        else
          mask = __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(w + e), __bfloat162bfloat162(__float2bfloat16_ru(lim)));
        hits |= mask & (0x00010001u << (4 * i + e));
      }
    }
  }
  return hits;
}
template <typename T>
__device__ __forceinline__ int value_of(int bit) {
  return sizeof(T) == 4 ? bit : 2 * (bit & 15) + (bit >> 4);
}

template <typename T>
__global__ void __launch_bounds__(kBmThreads, kResident) beam_scan_kernel(const BeamParams p) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int kPairs = VE / 2;
  extern __shared__ int32_t s_list[];   // kListLen<T> tokens
  __shared__ unsigned long long s_buf[kBmThreads], s_best[DSA_MAX_SELECT];
  __shared__ int s_rank[kBmThreads];
  __shared__ volatile uint32_t s_bound[kBmWarps];
  __shared__ int s_count, s_kept;
  __shared__ unsigned long long s_sum[kBmWarps];
  __shared__ float s_max[kBmWarps];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int k = p.select, nth = (k + kBmWarps - 1) / kBmWarps;
  pdl_trigger();
  const unsigned u_end = run_begin(p, blockIdx.x + 1);
  for (unsigned u = run_begin(p, blockIdx.x); u < u_end;) {
    const int row = static_cast<int>(u / static_cast<unsigned>(p.row_tiles));
    const int t0 = static_cast<int>(u - static_cast<unsigned>(row) * p.row_tiles);
    const int t1 = static_cast<int>(min(static_cast<unsigned>(p.row_tiles), t0 + (u_end - u)));
    u += t1 - t0;
    if (p.finished && p.finished[row]) continue;   // the merge knows its one continuation
    const T* x0 = static_cast<const T*>(p.logits) + static_cast<long long>(row) * p.stride;
    // 16-byte vectors from the aligned address at or before the row's first element
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));

    const auto load = [&](int v) {
      const int e0 = v * VE - mis;
      uint4 r;
      if (e0 >= 0 && e0 + VE <= p.vocab) {
        r = __ldcs(reinterpret_cast<const uint4*>(x0 + e0));
      } else {
        alignas(16) T out[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) out[e] = e0 + e >= 0 && e0 + e < p.vocab ? x0[e0 + e] : T(-INFINITY);
        r = *reinterpret_cast<const uint4*>(out);
      }
      return r;
    };

    float m = -INFINITY;                 // this thread's maximum
    float ref = -INFINITY, c = 0.f;      // the maximum that its sum is relative to, and that one's offset
    float sum_hi = 0.f, sum_lo = 0.f;    // its sum, and what rounding left out of it
    float lim = key_value(1ull << 55);   // candidates are at least this (the smallest finite value to begin with)
    // a warp takes every eighth run of four vectors (64 bytes) of 256, so that a
    // tile that the row fills only in part still gives every warp its share and
    // the warps' bounds stay alike
    const int own_vec = (lane >> 2) * 32 + wid * 4 + (lane & 3);
    if (tid == 0) s_count = 0;
    if (lane == 0) s_bound[wid] = 0u;
    const auto fetch = [&](int t, uint4* v) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) v[i] = load(t * kTileVecs + i * kBmThreads + own_vec);
    };
    const auto tile = [&](int t, const uint4* cur) {
      const float top = top_of<T>(cur);
      m = fmaxf(m, top);
      // the reference moves when a term would pass 2^30 (most threads' largest
      // value rises a few times in a row)
      if (top > ref && !(fabsf(ref) <= kFar && fabsf(top) <= kFar && fmaf(top, kLog2e, c) <= 30.f)) {
        const float f = join_factor(ref, top);   // (0 * 0 keeps a NaN)
        sum_hi *= f;
        sum_lo *= f;
        ref = top;
        c = offset_of(ref);
      }
      float2 sum = make_float2(0.f, 0.f);   // this tile's: 16 additions at the most one after another
      if (fabsf(ref) <= kFar) {
        const float2 h2 = make_float2(kLog2e, kLog2e), c2 = make_float2(c, c);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const uint32_t w[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const float2 y = fma_f32x2(two_of<T>(w, e), h2, c2);
            sum = add2(sum, make_float2(ex2_ftz(y.x), ex2_ftz(y.y)));
          }
        }
      } else {
        // a far maximum, or nothing but -infinity (and NaN) so far
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const uint32_t w[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const float2 x = two_of<T>(w, e);
            if (ref > -INFINITY) sum = add2(sum, make_float2(exp_neg(x.x - ref), exp_neg(x.y - ref)));
            else if (x.x != x.x || x.y != x.y) sum.x = NAN;
          }
        }
      }
      const float part = sum.x + sum.y, next = sum_hi + part, got = next - sum_hi;
      sum_lo += (sum_hi - (next - got)) + (part - got);   // (an infinite sum leaves a NaN)
      sum_hi = next;
      // the bound so far; an older one of another warp is a bound as well, so
      // only the first tile's has to be waited for
      const int done = t - t0;
      if (done < 4 || (done & 3) == 0) {
        const uint32_t bound = warp_jth(float_key(m), nth);
        if (lane == 0) s_bound[wid] = bound;
        if (done == 0) __syncthreads();
        uint32_t b = s_bound[0];
#pragma unroll
        for (int i = 1; i < kBmWarps; ++i) b = min(b, s_bound[i]);
        if (b != 0u) lim = fmaxf(lim, key_value(static_cast<unsigned long long>(b) << 32));
      }
      // append the places that reach it
      if (top >= lim) {
        uint32_t hits = reached<T>(cur, lim);
        int at = atomicAdd(&s_count, __popc(hits));
        while (hits) {
          const int bit = __ffs(hits) - 1, i = value_of<T>(bit);
          hits &= hits - 1;
          s_list[at++] = (t * kTileVecs + (i / VE) * kBmThreads + own_vec) * VE - mis + (i % VE);
        }
      }
    };
    const auto key_at = [&](int i) {
      const int token = s_list[i];
      return cand_key(static_cast<float>(x0[token]), token);
    };
    uint4 va[kVecs], vb[kVecs];
    fetch(t0, va);
    __syncthreads();
    static_assert(kGroup == 2, "a group is what the two buffers hold");
    for (int t = t0; t < t1; t += kGroup) {
      if (t + 1 < t1) fetch(t + 1, vb);
      tile(t, va);
      if (t + 2 < t1) fetch(t + 2, va);
      if (t + 1 < t1) tile(t + 1, vb);
      __syncthreads();
      const int n = s_count;
      __syncthreads();
      if (n > kDrain) {
        const int have = cut_to_best<kBmThreads>(s_best, key_at, n, k, 0ull, s_buf, s_rank);
        if (tid < have) s_list[tid] = static_cast<int32_t>(~static_cast<uint32_t>(s_best[tid]));
        if (tid == 0) s_count = have;
        // what comes later in the row has higher tokens: equal is not enough
        if (have == k) lim = fmaxf(lim, next_above(key_value(s_best[k - 1])));
        __syncthreads();
      }
    }
    // hand on what the bound has not overtaken (n <= kDrain: one key a thread)
    const int n = s_count;
    const unsigned long long key = tid < n ? key_at(tid) : 0ull;
    float thr;
    {
      uint32_t b = s_bound[0];
#pragma unroll
      for (int i = 1; i < kBmWarps; ++i) b = min(b, s_bound[i]);
      // (not `lim`, which may lie above the last of a cut list)
      thr = b != 0u ? key_value(static_cast<unsigned long long>(b) << 32) : -INFINITY;
    }
    const bool keep = tid < n && key_value(key) >= thr;
    // the threads' sums join meanwhile
    float mm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    if (lane == 0) s_max[wid] = mm;
    if (tid == 0) s_kept = 0;
    __syncthreads();
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    int at = 0;
    if (lane == 0 && kept) at = atomicAdd(&s_kept, __popc(kept));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(kept & ((1u << lane) - 1u));
    mm = s_max[0];
#pragma unroll
    for (int i = 1; i < kBmWarps; ++i) mm = fmaxf(mm, s_max[i]);
    const float own = sum_hi + sum_lo;   // 0 (or a NaN) where nothing but -infinity was seen
    // (a thread's maximum may be +infinity, its sum is a NaN then)
    const bool bad = !(own < INFINITY);
    unsigned long long fixed =
        bad ? 0ull : static_cast<unsigned long long>(own * join_factor(ref, mm) * 0x1p36f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) fixed += __shfl_xor_sync(0xffffffffu, fixed, o);
    if (lane == 0) s_sum[wid] = fixed;
    const bool poison = __syncthreads_or(bad);
    const unsigned slice = blockIdx.x - run_of(p, static_cast<unsigned>(row) * p.row_tiles);
    const long long to = static_cast<long long>(row) * p.slices + slice;
    unsigned long long* out = p.cands + to * kKeep;
    int handed = s_kept;
    if (handed <= kKeep) {
      if (keep) out[at] = key;
    } else {
      if (keep) s_buf[at] = key;
      __syncthreads();
      rank_best<kBmThreads>(s_best, s_buf, handed, k, 0ull, s_rank);
      handed = k;
      if (tid < k) out[tid] = s_best[tid];
    }
    if (tid == 0) {
      fixed = 0ull;
      for (int i = 0; i < kBmWarps; ++i) fixed += s_sum[i];
      p.sums[to] = SliceSum{poison ? kNaN : fixed, mm, handed};
    }
    __syncthreads();   // (the next slice's lists)
  }
}

__device__ __forceinline__ unsigned long long double_key(double x) {
  if (x == 0.0) x = 0.0;   // -0 as +0
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_double(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// log(x / 2^36) of x > 0 is n log 2 + hi + lo with the n that is returned: with
// x = 2^e q, q in [1/sqrt 2, sqrt 2), and f = (q - 1) / (q + 1),
// log q = 2 f + 2 f (f^2 / 3 + f^4 / 5 + ...), |f| < 0.172. 2 f is taken to two
// fp32 numbers, the rest, below 4e-3, in fp32: together good to 2e-9. (64-bit
// arithmetic has a latency of some hundred cycles here, and this kernel's time
// is one dependent chain.)
__device__ __forceinline__ int log_fixed(unsigned long long x, float* hi, float* lo) {
  int e = 63 - __clzll(static_cast<long long>(x));
  // q - 1 in units of 2^-62, from the bits below the leading one
  long long d = static_cast<long long>((e < 62 ? x << (62 - e) : x >> (e - 62)) & 0x3fffffffffffffffull);
  if (d > 0x1A827999FCEF3243ll) {   // q > sqrt 2: halve it
    d = (d >> 1) - 0x2000000000000000ll;
    ++e;
  }
  const float dh = static_cast<float>(d) * 0x1p-62f;
  const float dl = static_cast<float>(d - static_cast<long long>(static_cast<float>(d))) * 0x1p-62f;
  // f = (dh + dl) / (2 + dh + dl)
  const float nh = 2.0f + dh, nl = (2.0f - nh) + dh + dl;
  const float r = __frcp_rn(nh);
  const float fh = dh * r;
  const float fl = (fmaf(-fh, nh, dh) + dl - fh * nl) * r;
  const float g = fh * fh;
  float s = 1.0f / 15;
  s = fmaf(s, g, 1.0f / 13);
  s = fmaf(s, g, 1.0f / 11);
  s = fmaf(s, g, 1.0f / 9);
  s = fmaf(s, g, 1.0f / 7);
  s = fmaf(s, g, 1.0f / 5);
  s = fmaf(s, g, 1.0f / 3);
  *hi = 2.0f * fh;
  *lo = 2.0f * fmaf(fh * g, s, fl);
  return e - 36;
}

// Whether the n logits at x and at y are the same (-0 as +0; a NaN's row has no
// candidate). The whole block calls it.
__device__ __forceinline__ bool same_logits(const uint8_t* x, const uint8_t* y, int n, int elem) {
  const uint32_t mag = elem == 4 ? 0x7fffffffu : 0x7fff7fffu;   // without the signs
  const auto differ = [&](uint32_t u, uint32_t v) {   // a value of 32 bits, or two of 16
    if (u == v) return false;
    if (elem == 4) return ((u | v) & mag) != 0u;
    const uint32_t d = u ^ v, w = (u | v) & mag;
    return ((d & 0xffffu) && (w & 0xffffu)) || ((d >> 16) && (w >> 16));
  };
  const auto one = [&](int e) {
    return elem == 4 ? differ(reinterpret_cast<const uint32_t*>(x)[e], reinterpret_cast<const uint32_t*>(y)[e])
                     : differ(reinterpret_cast<const uint16_t*>(x)[e], reinterpret_cast<const uint16_t*>(y)[e]);
  };
  // 16 bytes of x at a time, from its first such boundary; of y the five words
  // (within it) that hold the same values
  const int per = 16 / elem;
  const int head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / elem);
  const uint8_t* xv = x + head * elem;
  const uint8_t* yv = y + head * elem;
  const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(yv) & 3);   // 0, or 2 for 16-bit values
  const int vecs = max(0, (n - head - (odd ? 1 : 0)) / per), tail = head + vecs * per;
  const uint32_t* yw = reinterpret_cast<const uint32_t*>(yv - odd);
  bool diff = false;
  constexpr int kAhead = 4;
  for (int v0 = 0; v0 < vecs; v0 += kAhead * kMergeThreads) {
    uint4 u[kAhead];
    uint32_t w[kAhead][5];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = min(v0 + i * kMergeThreads + static_cast<int>(threadIdx.x), vecs - 1);
      u[i] = reinterpret_cast<const uint4*>(xv)[v];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[i][k] = yw[4 * v + k];
      w[i][4] = odd ? yw[4 * v + 4] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t c[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) diff = diff || differ(c[k], __funnelshift_r(w[i][k], w[i][k + 1], 8 * odd));
    }
    if (__syncthreads_or(diff)) return false;
  }
  // before the first vector and behind the last
  const int rest = head + n - tail;   // (fewer than 32)
  if (static_cast<int>(threadIdx.x) < rest) {
    const int e = threadIdx.x;
    diff = one(e < head ? e : tail + e - head) || diff;
  }
  return !__syncthreads_or(diff);
}

// One thread block per batch entry; its beams' slices are the lists
// b * slices + j.
__global__ void __launch_bounds__(kMergeThreads, 1) beam_merge_kernel(const BeamParams p) {
  extern __shared__ Total s_totals[];       // kMergeList + DSA_MAX_SELECT
  Total* s_list = s_totals;
  __shared__ Total s_buf[kBmThreads];
  __shared__ Total s_best[DSA_MAX_SELECT];
  __shared__ int s_rank[kBmThreads];
  __shared__ SliceSum s_sum[kMaxLists];
  __shared__ double s_off[DSA_MAX_BEAMS];   // score - log sum exp of each beam (a finished one: its score)
  __shared__ float s_score[DSA_MAX_BEAMS];
  __shared__ uint8_t s_over[DSA_MAX_BEAMS];
  __shared__ unsigned long long s_alike[DSA_MAX_BEAMS];   // lower beams of the same score
  __shared__ int s_first[DSA_MAX_BEAMS];    // the lowest beam of the same score and logits
  __shared__ uint32_t s_bound[kBounds * kMergeWarps];
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int row0 = blockIdx.x * p.beams;
  const int k = p.select;
  const Total none{0ull, 0u};
  const int lists = p.beams * p.slices;
  if (tid == 0) s_count = 0;
  // (scores and flags are the caller's, not the scan's)
  if (tid < p.beams) {
    s_score[tid] = p.scores[row0 + tid];
    s_over[tid] = p.finished && p.finished[row0 + tid];
    s_alike[tid] = 0ull;
    s_first[tid] = tid;
  }
  __syncthreads();
  // Beams of the same score and logits tie, but their rows are cut and aligned
  // differently, and so their sums rounded: rows of equal scores are compared, while
  // the scan runs, and a beam takes the sum of the lowest one that is the same. (Rows
  // that differ do so early as a rule. Four equal beams of 32,000 take 22 us and not
  // 9.3, 64 x 8 of 131,072 132 and not 41; compared by the scan's blocks these were
  // 13 and 204, but every call of 64 x 8 took 2.3 us more.)
  bool tied = false;
  for (int x = tid; x < p.beams * p.beams; x += kMergeThreads) {
    const int i = x / p.beams, j = x - i * p.beams;
    if (j < i && !s_over[i] && !s_over[j] && s_score[i] == s_score[j] && s_score[i] > -INFINITY) {
      atomicOr(&s_alike[i], 1ull << j);
      tied = true;
    }
  }
  if (__syncthreads_or(tied)) {
    const long long pitch = p.stride * p.elem;
    const uint8_t* rows = static_cast<const uint8_t*>(p.logits) + row0 * pitch;
    for (int i = 1; i < p.beams; ++i)
      for (unsigned long long left = s_alike[i]; left != 0ull; left &= left - 1) {
        const int j = __ffsll(static_cast<long long>(left)) - 1;
        if (s_first[j] != j || !same_logits(rows + i * pitch, rows + j * pitch, p.vocab, p.elem)) continue;
        if (tid == 0) s_first[i] = j;
        __syncthreads();
        break;
      }
  }
  int b = 0;
  bool there = false;
  if (tid < lists) {
    b = tid / p.slices;
    const unsigned u = static_cast<unsigned>(row0 + b) * p.row_tiles;
    there = !s_over[b] && tid - b * p.slices <= static_cast<int>(run_of(p, u + p.row_tiles - 1) - run_of(p, u));
  }
  pdl_wait();
  if (blockIdx.x == 0 && tid == 0) *p.status = 0u;
  if (tid < lists) {
    SliceSum s{0ull, -INFINITY, 0};
    if (there) s = p.sums[static_cast<long long>(row0) * p.slices + tid];
    else if (s_over[b] && tid == b * p.slices) s.count = 1;   // a finished beam's only candidate is pad_token
    s_sum[tid] = s;
  }
  __syncthreads();
  // A lane takes a list, a warp every 32nd of its candidates (beams may be far
  // apart: this way the warps' shares are alike). The first 64 lists' are read
  // while the sums are joined.
  const unsigned long long* cands = p.cands + static_cast<long long>(row0) * p.slices * kKeep;
  const auto fetch = [&](int i, uint32_t* key) {   // the warp's share of list i: the values' keys
    const int n = i < lists && !s_over[i / p.slices] ? s_sum[i].count : 0;
#pragma unroll
    for (int j = 0; j < kShare; ++j) {
      const int at = j * kMergeWarps + wid;
      key[j] = at < n ? reinterpret_cast<const uint32_t*>(cands + i * kKeep + at)[1] : 0u;
    }
  };
  uint32_t ahead[2][kShare];
  fetch(lane, ahead[0]);
  fetch(lane + 32, ahead[1]);
  if (tid < p.beams) {
    double off = s_score[tid];
    if (!s_over[tid]) {
      const SliceSum* s = s_sum + s_first[tid] * p.slices;
      float mm = -INFINITY;
      for (int j = 0; j < p.slices; ++j) mm = fmaxf(mm, s[j].max);
      unsigned long long sum = 0ull;
      bool bad = false;
      for (int j = 0; j < p.slices; ++j) {
        bad = bad || s[j].sum == kNaN;
        if (!(s[j].max > -INFINITY)) continue;
        if (fabsf(mm) <= kFar && fabsf(s[j].max) <= kFar) {
          const float d = offset_of(s[j].max) - offset_of(mm);   // >= 0
          sum += d < 64.f ? s[j].sum >> static_cast<int>(d) : 0ull;
        } else {
          sum += static_cast<unsigned long long>(static_cast<double>(s[j].sum) * join_factor(s[j].max, mm));
        }
      }
      if (bad || sum == 0ull) {
        off = NAN;   // nothing but -infinity: no candidate
      } else {
        // the logarithm, and H's part undone at the maximum
        float hi, lo;
        const int e = log_fixed(sum, &hi, &lo);
        const bool near = fabsf(mm) <= kFar;
        if (near) lo = fmaf(mm, kLog2eRest * 0.693147181f, lo);
        const float whole = static_cast<float>(e) - (near ? offset_of(mm) : 0.f);   // (below 2^24)
        double lse = fma(static_cast<double>(whole), 0.6931471805599453, static_cast<double>(hi)) + static_cast<double>(lo);
        if (!near) lse += static_cast<double>(mm);
        off -= lse;
      }
    }
    s_off[tid] = off;
  }
  __syncthreads();
  // A bound on the totals (fp32, rounded down): of the warps' four largest values
  // (one a lane) `select` reach the select-th largest.
  uint32_t best = 0u;
  const auto join_list = [&](int i, const uint32_t* key) {
    if (i >= lists) return;
    const int at = i / p.slices;
    uint32_t top = key[0];
#pragma unroll
    for (int j = 1; j < kShare; ++j) top = max(top, key[j]);
    const float off = __double2float_rd(s_off[at]);
    float t = -INFINITY;
    if (top != 0u) t = __fadd_rd(key_value(static_cast<unsigned long long>(top) << 32), off);
    else if (s_over[at] && wid == 0 && s_sum[i].count > 0) t = off;
    if (t > -INFINITY) best = max(best, float_key(t));   // (not for a NaN)
  };
  join_list(lane, ahead[0]);
  join_list(lane + 32, ahead[1]);
  for (int i = lane + 64; i < lists; i += 32) {
    uint32_t key[kShare];
    fetch(i, key);
    join_list(i, key);
  }
#pragma unroll
  for (int i = 0; i < kBounds; ++i) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t holders = __ballot_sync(0xffffffffu, best == top);
    if (lane == __ffs(holders) - 1) best = 0u;
    if (lane == 0) s_bound[i * kMergeWarps + wid] = top;
  }
  __syncthreads();
  if (wid == 0) {
    // the select-th largest of them (a lane's are in order)
    uint32_t cur[kBounds], bound = 0u;
#pragma unroll
    for (int i = 0; i < kBounds; ++i) cur[i] = s_bound[i * kMergeWarps + lane];
#pragma unroll 1
    for (int i = 0; i < k; ++i) {
      bound = __reduce_max_sync(0xffffffffu, cur[0]);
      if (bound == 0u) break;
      const uint32_t holders = __ballot_sync(0xffffffffu, cur[0] == bound);
      if (lane == __ffs(holders) - 1) {
#pragma unroll
        for (int j = 0; j + 1 < kBounds; ++j) cur[j] = cur[j + 1];
        cur[kBounds - 1] = 0u;
      }
    }
    __syncwarp();
    if (lane == 0) s_bound[0] = bound;
  }
  __syncthreads();
  best = s_bound[0];
  // the totals of those that may reach it, a round of lists at a time
  int have = 0;
  for (int r = 0; r < lists; r += kRound) {
    const int i = r + wid;
    if (i < lists) {
      const int at_b = i / p.slices, n = s_sum[i].count;
      const double off = s_off[at_b];
      const float off_up = __double2float_ru(off);
      const bool over = s_over[at_b];
#pragma unroll
      for (int j0 = 0; j0 < kKeep; j0 += 32) {
        const int j = j0 + lane;
        if (j >= n) continue;
        const unsigned long long key = over ? 0ull : cands[i * kKeep + j];
        const float up = over ? off_up : __fadd_ru(key_value(key), off_up);
        if (!(up > -INFINITY) || float_key(up) < best) continue;
        const double t = over ? off : static_cast<double>(key_value(key)) + off;
        if (!(t > -INFINITY)) continue;
        const int token = over ? p.pad : static_cast<int32_t>(~static_cast<uint32_t>(key));
        s_list[atomicAdd(&s_count, 1)] = Total{double_key(t), ~static_cast<uint32_t>(at_b * p.vocab + token)};
      }
    }
    __syncthreads();
    // join them with the best so far, when all are there or there may be no room for another round's
    const int n = s_count, old = have;
    if (r + kRound < lists && n <= kMergeList - kRound * kKeep) {
      __syncthreads();   // (the count has been read)
      continue;
    }
    if (old + n <= kBmThreads) {
      if (tid < old) s_buf[tid] = s_best[tid];
      else if (tid < old + n) s_buf[tid] = s_list[tid - old];
      __syncthreads();
      rank_best<kMergeThreads>(s_best, s_buf, old + n, k, none, s_rank);
      have = min(k, old + n);
    } else {
      // (ties, or far more candidates than the bound leaves in general)
      if (tid < old) s_list[n + tid] = s_best[tid];
      __syncthreads();
      have = cut_to_best<kMergeThreads>(s_best, [&](int x) { return s_list[x]; }, n + old, k, none, s_buf, s_rank);
    }
    if (tid == 0) s_count = 0;
    __syncthreads();
  }
  if (tid < k) {
    const Total t = s_best[tid];
    const long long o = static_cast<long long>(blockIdx.x) * k + tid;
    const uint32_t place = ~t.lo;
    const bool got = t.hi != 0ull;
    p.out_scores[o] = got ? static_cast<float>(key_double(t.hi)) : -INFINITY;
    p.out_tokens[o] = got ? static_cast<int32_t>(place % static_cast<uint32_t>(p.vocab)) : -1;
    p.out_parents[o] = got ? row0 + static_cast<int32_t>(place / static_cast<uint32_t>(p.vocab)) : -1;
  }
}

// -------------------------------------------------------------------- host
int check_beam(const dsa_beam_problem* p) {
  if (!p) return report_error(DSA_ERR_INVALID_ARG, "beam problem is NULL");
  if (p->batch < 1 || p->batch > 65535) return report_errorf(DSA_ERR_INVALID_ARG, "batch %d outside 1..65535", p->batch);
  if (p->beams < 1 || p->beams > DSA_MAX_BEAMS)
    return report_errorf(DSA_ERR_INVALID_ARG, "beams %d outside 1..%d", p->beams, DSA_MAX_BEAMS);
  if (static_cast<long long>(p->batch) * p->beams > 65535)
    return report_error(DSA_ERR_UNSUPPORTED, "batch * beams must be at most 65535");
  if (p->vocab < 1 || p->vocab > (1 << 24))
    return report_errorf(DSA_ERR_INVALID_ARG, "vocab %d outside 1..2^24", p->vocab);
  if (p->select < 1 || p->select > DSA_MAX_SELECT)
    return report_errorf(DSA_ERR_INVALID_ARG, "select %d outside 1..%d", p->select, DSA_MAX_SELECT);
  if (p->logits_dtype != DSA_BF16 && p->logits_dtype != DSA_FP16 && p->logits_dtype != DSA_FP32)
    return report_error(DSA_ERR_UNSUPPORTED, "logits must be BF16, FP16 or FP32");
  if (p->pad_token < 0 || p->pad_token >= p->vocab)
    return report_errorf(DSA_ERR_INVALID_ARG, "pad_token %d outside the vocabulary", p->pad_token);
  if (p->row_stride != 0 && p->row_stride < p->vocab)
    return report_error(DSA_ERR_INVALID_ARG, "row_stride must be 0 or at least vocab");
  return DSA_OK;
}

size_t up(size_t x) { return (x + 255) & ~size_t(255); }

// How the rows are cut: tiles per row, blocks (as many as are resident at
// once), slices a row may have.
int most_slices(const dsa_beam_problem* p) { return std::max(2, kMaxLists / p->beams); }
struct Cut {
  long long units;
  int row_tiles, blocks, slices;
};
Cut cut(const dsa_beam_problem* p, int sms, bool base_aligned) {
  Cut c;
  const int ve = p->logits_dtype == DSA_FP32 ? 4 : 8;
  // a row that does not begin on 16 bytes may take a vector more
  const bool even = base_aligned && p->row_stride % ve == 0 && (p->row_stride != 0 || p->vocab % ve == 0);
  const long long vecs = (p->vocab + ve - 1LL + (even ? 0 : ve - 1)) / ve;
  c.row_tiles = static_cast<int>((vecs + kTileVecs - 1) / kTileVecs);
  const long long rows = static_cast<long long>(p->batch) * p->beams;
  c.units = rows * c.row_tiles;
  // a run of `per` tiles cuts a row into at most (row_tiles - 2) / per + 2
  // slices; a batch entry has at most kMaxLists
  const auto slices = [&](long long n) {
    const long long per = c.units / n;
    return c.row_tiles == 1 ? 1LL : (c.row_tiles - 2) / per + 2;
  };
  long long blocks = std::min<long long>(c.units, static_cast<long long>(sms) * kResident);
  while (blocks > rows && slices(blocks) > most_slices(p)) blocks = std::max(rows, blocks * 7 / 8);
  c.blocks = static_cast<int>(blocks);
  c.slices = static_cast<int>(slices(blocks));
  return c;
}

size_t beam_bytes(const dsa_beam_problem* p, size_t* sums_at) {
  // the most slices any number of blocks leads to
  const int slices = std::min(cut(p, 1, false).row_tiles, most_slices(p));
  const size_t n = static_cast<size_t>(p->batch) * p->beams * slices;
  const size_t c = 256 + up(n * kKeep * sizeof(unsigned long long));
  if (sums_at) *sums_at = c;
  return c + up(n * sizeof(SliceSum));
}

template <typename T>
cudaError_t launch_scan(const BeamParams& p, int blocks, cudaStream_t s) {
  constexpr int smem = kListLen<T> * 4;
  const cudaError_t e = set_max_smem(reinterpret_cast<const void*>(beam_scan_kernel<T>), smem);
  if (e != cudaSuccess) return e;
  return launch_kernel("beam_scan_kernel", beam_scan_kernel<T>, dim3(blocks), dim3(kBmThreads), smem, s, false, p);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_beam_workspace_size(const dsa_beam_problem* p) {
  if (check_beam(p)) return 0;
  return beam_bytes(p, nullptr);
}

extern "C" int dsa_beam_select(const dsa_beam_problem* bp, const void* logits, const float* scores,
                               const uint8_t* finished, float* out_scores, int32_t* out_tokens,
                               int32_t* out_parents, void* ws, size_t ws_bytes, void* stream) {
  reset_launches();
  if (int rc = check_beam(bp)) return rc;
  if (!logits || !scores || !out_scores || !out_tokens || !out_parents)
    return report_error(DSA_ERR_INVALID_ARG, "a required tensor pointer is NULL");
  const uintptr_t la = bp->logits_dtype == DSA_FP32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(logits) & la) || (reinterpret_cast<uintptr_t>(scores) & 3) ||
      (reinterpret_cast<uintptr_t>(out_scores) & 3) || (reinterpret_cast<uintptr_t>(out_tokens) & 3) ||
      (reinterpret_cast<uintptr_t>(out_parents) & 3))
    return report_error(DSA_ERR_MISALIGNED, "tensors must be aligned to their elements");
  {
    // (a batch entry's scores are read before its results are written, no other's)
    const long long rows = static_cast<long long>(bp->batch) * bp->beams;
    const long long outs = static_cast<long long>(bp->batch) * bp->select * 4;
    const void* out[3] = {out_scores, out_tokens, out_parents};
    const bool in_place = out_scores == scores && bp->select == bp->beams;
    const long long elem = bp->logits_dtype == DSA_FP32 ? 4 : 2;
    const long long read = ((rows - 1) * (bp->row_stride ? bp->row_stride : bp->vocab) + bp->vocab) * elem;
    for (int i = 0; i < 3; ++i)
      if (overlap(out[i], outs, logits, read) || (overlap(out[i], outs, scores, rows * 4) && !(i == 0 && in_place)) ||
          (finished && overlap(out[i], outs, finished, rows)) || overlap(out[i], outs, out[(i + 1) % 3], outs))
        return report_error(DSA_ERR_INVALID_ARG, "the results must not overlap each other or an input (out_scores "
                            "may be `scores` itself where select == beams)");
  }
  size_t sums_at = 0;
  if (int rc = check_call_workspace(ws, ws_bytes, beam_bytes(bp, &sums_at))) return rc;
  int sms = 0;
  if (int rc = current_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  BeamParams p{};
  p.status = static_cast<uint32_t*>(ws);
  p.logits = logits;
  p.scores = scores;
  p.finished = finished;
  p.cands = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(ws) + 256);
  p.sums = reinterpret_cast<SliceSum*>(static_cast<uint8_t*>(ws) + sums_at);
  p.out_scores = out_scores;
  p.out_tokens = out_tokens;
  p.out_parents = out_parents;
  p.beams = bp->beams;
  p.vocab = bp->vocab;
  p.select = bp->select;
  p.pad = bp->pad_token;
  p.elem = bp->logits_dtype == DSA_FP32 ? 4 : 2;
  p.stride = bp->row_stride ? bp->row_stride : bp->vocab;
  const Cut c = cut(bp, sms, (reinterpret_cast<uintptr_t>(logits) & 15) == 0);
  p.per = static_cast<unsigned>(c.units / c.blocks);
  p.extra = static_cast<unsigned>(c.units % c.blocks);
  p.row_tiles = c.row_tiles;
  p.slices = c.slices;
  cudaError_t e = bp->logits_dtype == DSA_FP32   ? launch_scan<float>(p, c.blocks, s)
                  : bp->logits_dtype == DSA_FP16 ? launch_scan<__half>(p, c.blocks, s)
                                                 : launch_scan<__nv_bfloat16>(p, c.blocks, s);
  constexpr int merge_smem = (kMergeList + DSA_MAX_SELECT) * static_cast<int>(sizeof(Total));
  if (e == cudaSuccess) e = set_max_smem(reinterpret_cast<const void*>(beam_merge_kernel), merge_smem);
  if (e == cudaSuccess)
    e = launch_kernel("beam_merge_kernel", beam_merge_kernel, dim3(bp->batch), dim3(kMergeThreads), merge_smem, s, true, p);
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "beam_select launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}
