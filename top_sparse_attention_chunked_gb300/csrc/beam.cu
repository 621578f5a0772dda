// Beam search's selection: the `select` best of score_i + log_softmax(logits_i)
// over beams x vocabulary, per batch entry.
//
// Two launches. beam_scan_kernel reads every logit once. Its blocks, as many as
// are resident at once, take equal runs of tiles (512 16-byte vectors of a
// row), a run spanning the end of one row and the start of the next where it
// must; a row's part in a block is a slice. Of each slice a block keeps, side
// by side, the maximum and the sum of exponentials (one online state a thread,
// joined at the end) and the `select` largest logits. The latter through a
// lower bound: every thread holds the largest value it has seen, a warp's j-th
// largest of those (j = select / 8 warps) is reached by j values of the warp,
// so the smallest of the eight warps' is reached by `select` values of the
// slice. Values that reach it -- a few times `select` in all, one comparison
// per tile for the rest -- are appended to a list that the block sorts when
// it fills and at the end. Within a row totals are ordered as the logits are,
// so a row's candidates are its `select` largest logits, lower tokens first.
// beam_merge_kernel joins the slices' sums of each row in 64 bits, forms the
// candidates' totals in 64 bits (rows have different offsets: totals may lie
// closer together than fp32 tells apart), bounds them in the same way and
// sorts the few that are left.
//
// The order of a list depends on the order of execution; its keys are distinct
// (value, then token), so what is sorted out of it does not.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kBmThreads = 256;
constexpr int kBmWarps = kBmThreads / 32;
constexpr int kVecs = 2;            // 16-byte vectors a thread takes per tile
constexpr int kTileVecs = kBmThreads * kVecs;
constexpr int kDrain = 184;         // list entries that trigger a sort
constexpr int kMaxCands = 8192;     // candidates of one batch entry (all rows and slices)
constexpr int kMergeList = 1024;    // of which the merge sorts from a list
constexpr int kResident = 5;        // scan blocks per SM (37 KB of shared memory each)

struct Cand {
  float value;
  int32_t token;      // -1: none
};
struct SliceSum {
  double sum;         // of exp(x - max); NaN if the slice holds a NaN or +infinity
  float max;
};

struct BeamParams {
  uint32_t* status;   // device status word: nothing can go wrong on the device
  const void* logits;
  const float* scores;
  const uint8_t* finished;
  Cand* cands;        // [rows, slices, select]
  SliceSum* sums;     // [rows, slices], slice 0 the row's first
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
  long long stride;   // elements between rows
  long long units;    // tiles of all rows
  int row_tiles, blocks;
  int batch, beams, vocab, select, slices, pad;
};

// Block c takes the units [run_begin(c), run_begin(c + 1)).
__host__ __device__ __forceinline__ long long run_begin(long long units, int blocks, int c) {
  return units * c / blocks;
}
__device__ __forceinline__ int run_of(long long units, int blocks, long long u) {
  return static_cast<int>(((u + 1) * blocks - 1) / units);
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(x) for x <= 0: log2(e) in two parts, so that its own rounding does not
// bias the sum (one part: 1.3e-8 of x, the same sign for every term)
constexpr float kLog2eHi = 1.44269502e0f, kLog2eLo = 1.92596303e-8f;
__device__ __forceinline__ float exp_neg(float x) { return ex2_ftz(fmaf(x, kLog2eHi, x * kLog2eLo)); }

// A row candidate as one key: larger value first, then the lower token.
__device__ __forceinline__ unsigned long long cand_key(float v, int token) {
  return (static_cast<unsigned long long>(float_key(v)) << 32) | static_cast<uint32_t>(~token);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
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
__device__ __forceinline__ unsigned long long shfl_xor(unsigned long long k, int m) {
  return __shfl_xor_sync(0xffffffffu, k, m);
}
__device__ __forceinline__ Total shfl_xor(const Total& k, int m) {
  return Total{__shfl_xor_sync(0xffffffffu, k.hi, m), __shfl_xor_sync(0xffffffffu, k.lo, m)};
}

// Sorts keys of the block's first `size` threads (a power of two; what the
// others hold is not looked at), largest in thread 0. Bitonic; the exchanges
// beyond a warp go through `buf`. Up to 32 keys stay in the first warp.
template <typename K>
__device__ __forceinline__ K block_sort(K key, K* buf, int size) {
  const int t = threadIdx.x;
#pragma unroll 1
  for (int run = 2; run <= size; run <<= 1) {
    const bool down = (t & run) == 0;   // this run sorts largest first
#pragma unroll 1
    for (int m = run >> 1; m > 0; m >>= 1) {
      K other;
      if (m >= 32) {
        __syncthreads();
        buf[t] = key;
        __syncthreads();
        other = buf[t ^ m];
      } else {
        if (t >= size && size <= 32) break;
        other = shfl_xor(key, m);
      }
      const bool first = (t & m) == 0;
      const bool take_max = first == down;
      if (above(other, key) == take_max) key = other;
    }
  }
  return key;
}

// Sorts the best `k` of top[0..k) and list[0..n) into top, largest first.
// `none` fills places that have no key. The whole block calls it; `fresh`:
// top holds nothing yet.
template <typename K>
__device__ void drain(K* top, const K* list, int n, int k, K none, K* buf, bool fresh) {
  const int t = threadIdx.x;
  __syncthreads();
  for (int at = 0; at < n || fresh;) {
    const int have = fresh ? 0 : k;
    const int i = at + t - have;
    const int here = have + min(n - at, kBmThreads - have);
    int size = 32;
    while (size < here || size < k) size <<= 1;
    K key = t < have ? top[t] : (i < n && t < here ? list[i] : none);
    if (size > 32 || t < 32) key = block_sort(key, buf, size);
    __syncthreads();
    if (t < k) top[t] = t < size ? key : none;
    __syncthreads();
    at += kBmThreads - have;
    fresh = false;
  }
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

// Two exp(x) for x <= 0, as exp_neg.
__device__ __forceinline__ float2 exp_neg2(float2 x) {
  const float2 zero = make_float2(0.f, 0.f);
  const float2 lo = fma_f32x2(x, make_float2(kLog2eLo, kLog2eLo), zero);
  const float2 y = fma_f32x2(x, make_float2(kLog2eHi, kLog2eHi), lo);
  return make_float2(ex2_ftz(y.x), ex2_ftz(y.y));
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

template <typename T>
__global__ void __launch_bounds__(kBmThreads, kResident) beam_scan_kernel(const BeamParams p) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int kPairs = VE / 2;
  constexpr int kList = kTileVecs * VE + kDrain;
  __shared__ unsigned long long s_list[kList];
  __shared__ unsigned long long s_top[DSA_MAX_SELECT];
  __shared__ unsigned long long s_buf[kBmThreads];
  __shared__ uint32_t s_bound[2][kBmWarps];
  __shared__ int s_count;
  __shared__ double s_sum[kBmWarps];
  __shared__ float s_max[kBmWarps];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int k = p.select, nth = (k + kBmWarps - 1) / kBmWarps;
  pdl_trigger();
  const long long u_end = run_begin(p.units, p.blocks, blockIdx.x + 1);
  for (long long u = run_begin(p.units, p.blocks, blockIdx.x); u < u_end;) {
    const int row = static_cast<int>(u / p.row_tiles);
    const int t0 = static_cast<int>(u - static_cast<long long>(row) * p.row_tiles);
    const int t1 = static_cast<int>(min(static_cast<long long>(p.row_tiles), t0 + (u_end - u)));
    u += t1 - t0;
    if (p.finished && p.finished[row]) continue;   // the merge knows its one continuation
    const T* x0 = static_cast<const T*>(p.logits) + static_cast<long long>(row) * p.stride;
    // 16-byte vectors from the aligned address at or before the row's first element
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
    const int v_end = t1 * kTileVecs;              // (vectors past the row read as masked)

    const auto load = [&](int v) {
      const int e0 = v * VE - mis;
      uint4 r;
      if (v < v_end && e0 >= 0 && e0 + VE <= p.vocab) {
        r = __ldcs(reinterpret_cast<const uint4*>(x0 + e0));
      } else {
        alignas(16) T out[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const bool in = v < v_end && e0 + e >= 0 && e0 + e < p.vocab;
          out[e] = in ? x0[e0 + e] : T(-INFINITY);
        }
        r = *reinterpret_cast<const uint4*>(out);
      }
      return r;
    };

    float m = -INFINITY;                 // this thread's maximum
    float2 sum = make_float2(0.f, 0.f);  // and its sum of exp(x - m)
    float thr = -INFINITY, past = -INFINITY;   // candidates are >= thr and > past
    bool fresh = true;
    uint4 cur[kVecs], nxt[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) cur[i] = load(t0 * kTileVecs + i * kBmThreads + tid);
    if (tid == 0) s_count = 0;
    for (int t = t0; t < t1; ++t) {
      const int v0 = t * kTileVecs;
      if (t + 1 < t1) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) nxt[i] = load(v0 + kTileVecs + i * kBmThreads + tid);
      }
      float2 x[kVecs][kPairs];
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const uint32_t w[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          x[i][e] = two_of<T>(w, e);
          top = fmaxf(top, fmaxf(x[i][e].x, x[i][e].y));
        }
      }
      if (top > m) {
        const float f = exp_neg(m - top);   // the first time: 0 * exp(-inf)
        sum.x *= f;
        sum.y *= f;
        m = top;
      }
      if (m > -INFINITY) {
        const float2 neg = make_float2(-m, -m);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int e = 0; e < kPairs; ++e) sum = add2(sum, exp_neg2(add2(x[i][e], neg)));
      } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int e = 0; e < kPairs; ++e)
            if (x[i][e].x != x[i][e].x || x[i][e].y != x[i][e].y) sum.x = NAN;   // among masked tokens
      }
      // the bound so far; the first tile's is needed at once, later ones may lag
      const uint32_t bound = warp_jth(float_key(m), nth);
      if (lane == 0) s_bound[t & 1][wid] = bound;
      const auto join = [&] {
        uint32_t b = s_bound[t & 1][0];
#pragma unroll
        for (int i = 1; i < kBmWarps; ++i) b = min(b, s_bound[t & 1][i]);
        if (b != 0u) thr = key_value(static_cast<unsigned long long>(b) << 32);
      };
      if (t == t0) {
        __syncthreads();
        join();
      }
      // append what reaches it
      uint32_t hits = 0;
      if (top >= thr) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            if (x[i][e].x >= thr && x[i][e].x > past) hits |= 1u << (i * VE + 2 * e);
            if (x[i][e].y >= thr && x[i][e].y > past) hits |= 2u << (i * VE + 2 * e);
          }
      }
      bool full = false;
      if (__any_sync(0xffffffffu, hits != 0)) {
        const int n = __popc(hits);
        int before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        int at = 0;
        if (lane == 31) at = atomicAdd(&s_count, before);
        at = __shfl_sync(0xffffffffu, at, 31) + before - n;
        full = at + n > kDrain;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (hits & (1u << (i * VE + e)))
              s_list[at++] = cand_key((e & 1) ? x[i][e >> 1].y : x[i][e >> 1].x,
                                      (v0 + i * kBmThreads + tid) * VE - mis + e);
      }
      if (__syncthreads_or(full)) {
        const int n = s_count;
        drain(s_top, s_list, n, k, 0ull, s_buf, fresh);
        fresh = false;
        if (tid == 0) s_count = 0;
        // what comes later in the row has higher tokens: equal is not enough
        if (s_top[k - 1] != 0ull) past = key_value(s_top[k - 1]);
        __syncthreads();
      }
      join();
#pragma unroll
      for (int i = 0; i < kVecs; ++i) cur[i] = nxt[i];
    }
    drain(s_top, s_list, s_count, k, 0ull, s_buf, fresh);
    // join the threads' sums
    float mm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    if (lane == 0) s_max[wid] = mm;
    __syncthreads();
    mm = s_max[0];
#pragma unroll
    for (int i = 1; i < kBmWarps; ++i) mm = fmaxf(mm, s_max[i]);
    // (a thread that saw nothing but -infinity adds its 0, or its NaN)
    const float own = sum.x + sum.y;
    double d = static_cast<double>(m > -INFINITY ? own * exp_neg(m - mm) : own);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) s_sum[wid] = d;
    __syncthreads();
    const int slice = blockIdx.x - run_of(p.units, p.blocks, static_cast<long long>(row) * p.row_tiles);
    const long long at = static_cast<long long>(row) * p.slices + slice;
    if (tid == 0) {
      d = 0.0;
      for (int i = 0; i < kBmWarps; ++i) d += s_sum[i];
      p.sums[at] = SliceSum{d, mm};
    }
    if (tid < k) {
      const unsigned long long key = s_top[tid];
      p.cands[at * k + tid] = key ? Cand{key_value(key), static_cast<int32_t>(~static_cast<uint32_t>(key))} : Cand{0.0f, -1};
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

__global__ void __launch_bounds__(kBmThreads) beam_merge_kernel(const BeamParams p) {
  __shared__ Total s_list[kMergeList];
  __shared__ Total s_buf[kBmThreads];
  __shared__ Total s_top[DSA_MAX_SELECT];
  __shared__ double s_off[DSA_MAX_BEAMS];   // score - log sum exp of each beam
  __shared__ int s_slices[DSA_MAX_BEAMS];   // its slices (0: finished)
  __shared__ uint32_t s_bound[kBmWarps];
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int row0 = blockIdx.x * p.beams;
  const int k = p.select;
  const Total none{0ull, 0u};
  if (tid == 0) s_count = 0;
  pdl_wait();
  if (blockIdx.x == 0 && tid == 0) *p.status = 0u;
  for (int b = wid; b < p.beams; b += kBmThreads / 32) {
    const int row = row0 + b;
    const bool over = p.finished && p.finished[row];
    const long long u = static_cast<long long>(row) * p.row_tiles;
    const int slices = over ? 0 : run_of(p.units, p.blocks, u + p.row_tiles - 1) - run_of(p.units, p.blocks, u) + 1;
    if (lane == 0) s_slices[b] = slices;
    if (over) continue;
    const SliceSum* s = p.sums + static_cast<long long>(row) * p.slices;
    float mm = -INFINITY;
    for (int i = lane; i < slices; i += 32) mm = fmaxf(mm, s[i].max);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    double d = 0.0;
    for (int i = lane; i < slices; i += 32) {
      const double v = s[i].sum;
      // (0 from a slice of masked tokens only: its maximum has no exponential)
      if (v != 0.0) d += s[i].max > -INFINITY ? v * exp(static_cast<double>(s[i].max) - mm) : v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) s_off[b] = static_cast<double>(p.scores[row]) - (static_cast<double>(mm) + log(d));
  }
  __syncthreads();
  // candidate i of the entry's beams x slices x select (finished beams: one)
  const int per_row = p.slices * k, n = p.beams * per_row;
  const auto total = [&](int i) {
    const int b = i / per_row, j = i - b * per_row;
    const int row = row0 + b;
    double t;
    int token;
    if (s_slices[b] == 0) {
      if (j > 0) return none;
      t = p.scores[row];
      token = p.pad;
    } else {
      if (j >= s_slices[b] * k) return none;
      const Cand c = p.cands[static_cast<long long>(row) * per_row + j];
      if (c.token < 0) return none;
      t = static_cast<double>(c.value) + s_off[b];
      token = c.token;
    }
    if (!(t > -INFINITY)) return none;   // -infinity or NaN
    return Total{double_key(t), ~static_cast<uint32_t>(b * p.vocab + token)};
  };
  // a bound as in the scan, in fp32 rounded down (which keeps the order)
  const auto key32 = [&](const Total& t) { return t.hi ? float_key(__double2float_rd(key_double(t.hi))) : 0u; };
  uint32_t best = 0u;
  for (int i = tid; i < n; i += kBmThreads) best = max(best, key32(total(i)));
  best = warp_jth(best, (k + kBmWarps - 1) / kBmWarps);
  if (lane == 0) s_bound[wid] = best;
  __syncthreads();
  best = s_bound[0];
#pragma unroll
  for (int i = 1; i < kBmWarps; ++i) best = min(best, s_bound[i]);
  bool fresh = true;
  for (int i0 = 0; i0 < n; i0 += kBmThreads) {
    const int i = i0 + tid;
    const Total t = i < n ? total(i) : none;
    const bool hit = t.hi != 0ull && key32(t) >= best;
    const uint32_t hits = __ballot_sync(0xffffffffu, hit);
    int at = 0;
    if (lane == 0 && hits) at = atomicAdd(&s_count, __popc(hits));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(hits & ((1u << lane) - 1u));
    if (hit) s_list[at] = t;
    // room for the next round's?
    if (__syncthreads_or(hit && at >= kMergeList - kBmThreads)) {
      drain(s_top, s_list, s_count, k, none, s_buf, fresh);
      fresh = false;
      if (tid == 0) s_count = 0;
      __syncthreads();
    }
  }
  drain(s_top, s_list, s_count, k, none, s_buf, fresh);
  if (tid < k) {
    const Total t = s_top[tid];
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
struct Cut {
  long long units;
  int row_tiles, blocks, slices;
};
Cut cut(const dsa_beam_problem* p, int sms) {
  Cut c;
  const int ve = p->logits_dtype == DSA_FP32 ? 4 : 8;
  const long long vecs = (p->vocab + 2LL * ve - 2) / ve;   // whatever the row's alignment
  c.row_tiles = static_cast<int>((vecs + kTileVecs - 1) / kTileVecs);
  const long long rows = static_cast<long long>(p->batch) * p->beams;
  c.units = rows * c.row_tiles;
  // a run of `per` tiles cuts a row into at most (row_tiles - 2) / per + 2
  // slices; their candidates stay within kMaxCands per batch entry
  const long long most = std::max(2, kMaxCands / (p->beams * p->select));
  long long blocks = std::min<long long>(c.units, static_cast<long long>(sms) * kResident);
  const auto slices = [&](long long n) {
    const long long per = c.units / n;
    return c.row_tiles == 1 ? 1LL : (c.row_tiles - 2) / per + 2;
  };
  while (blocks > rows && slices(blocks) > most) blocks = std::max(rows, blocks * 7 / 8);
  c.blocks = static_cast<int>(blocks);
  c.slices = static_cast<int>(slices(blocks));
  return c;
}

size_t beam_bytes(const dsa_beam_problem* p, size_t* sums_at) {
  // the most slices any number of blocks leads to: one per tile of a row, no
  // more than the candidates allow, two where there is a block per row
  const int tiles = cut(p, 1).row_tiles;
  const int slices = std::min(tiles, std::max(2, kMaxCands / (p->beams * p->select)));
  const size_t n = static_cast<size_t>(p->batch) * p->beams * slices;
  const size_t c = 256 + up(n * p->select * sizeof(Cand));
  if (sums_at) *sums_at = c;
  return c + up(n * sizeof(SliceSum));
}

template <typename T>
cudaError_t launch_scan(const BeamParams& p, cudaStream_t s) {
  return launch_kernel("beam_scan_kernel", beam_scan_kernel<T>, dim3(p.blocks), dim3(kBmThreads),
                       0, s, false, p);
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
  p.cands = reinterpret_cast<Cand*>(static_cast<uint8_t*>(ws) + 256);
  p.sums = reinterpret_cast<SliceSum*>(static_cast<uint8_t*>(ws) + sums_at);
  p.out_scores = out_scores;
  p.out_tokens = out_tokens;
  p.out_parents = out_parents;
  p.batch = bp->batch;
  p.beams = bp->beams;
  p.vocab = bp->vocab;
  p.select = bp->select;
  p.pad = bp->pad_token;
  p.stride = bp->row_stride ? bp->row_stride : bp->vocab;
  const Cut c = cut(bp, sms);
  p.units = c.units;
  p.row_tiles = c.row_tiles;
  p.blocks = c.blocks;
  p.slices = c.slices;
  cudaError_t e = bp->logits_dtype == DSA_FP32   ? launch_scan<float>(p, s)
                  : bp->logits_dtype == DSA_FP16 ? launch_scan<__half>(p, s)
                                                 : launch_scan<__nv_bfloat16>(p, s);
  if (e == cudaSuccess)
    e = launch_kernel("beam_merge_kernel", beam_merge_kernel, dim3(bp->batch), dim3(kBmThreads), 0, s, true, p);
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "beam_select launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}
