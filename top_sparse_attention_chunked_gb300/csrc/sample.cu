// Sampling: temperature, top-k, top-p and min-p, and a draw from one given random
// number per row.
//
// With w_t = exp((x_t - max x) / T) and the tokens ranked by x (ties: the lower
// index first), top-k, top-p and min-p each keep a prefix of the ranking; the token
// is the first in index order at which the kept weights' running sum exceeds u times
// their sum. So all that is needed is the cut, the pair (x, index) of the last token
// kept, and two sums over the row.
//
// A draw between 100,000 tokens is next to a border nearly always, so weights and
// sums have to be the same whatever the order: a weight is a multiple of a fixed unit
// (2^-62 times the row's length, rounded up to a power of two, of the largest), formed
// in fp32 pairs to 2^-31 of itself, and all sums are of 64-bit integers.
//
// A cluster of blocks holds a row in shared memory (read once); everything else is
// passes over it and exchanges between the blocks. The cut is found by counts of the
// weights' logarithms in 1,024 bins, of which the one or few that can hold the cut are
// counted again (by the bits of x) until at most kSmList tokens are left; those are
// ranked against each other. Top-p takes bounds from the bins' edges, exact sums of
// what lies above them.
#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kSmThreads = 512, kSmWarps = kSmThreads / 32;
constexpr int kSmBins = 1024;
constexpr int kSmList = 512;                    // candidates that are ranked against each other
constexpr int kSmMaxVocab = 1 << 19;
constexpr int kSmMaxCluster = 16;
constexpr int kSmMaxData = 196608;              // bytes of a row that a block holds

// 2^(j / 512), j = 0 .. 511, times 2^30: as a float and rounded to an integer.
struct Pow2Table {
  uint32_t f[512], i[512];
};
constexpr double series_exp(double x) {         // |x| < 0.7: 1 + x (1 + x / 2 (1 + x / 3 (...)))
  double s = 1.0;
  for (int k = 24; k >= 1; --k) s = 1.0 + x * s / k;
  return s;
}
constexpr uint32_t bits_of_30(double v) {       // the fp32 nearest v in [2^30, 2^31)
  const uint32_t m = static_cast<uint32_t>(v / 128.0 + 0.5);      // 24 bits: v's last place is 2^7
  return m >= (1u << 24) ? (127u + 31u) << 23 : ((127u + 30u) << 23) | (m - (1u << 23));
}
constexpr Pow2Table make_table() {
  Pow2Table t{};
  for (int j = 0; j < 512; ++j) {
    const double v = series_exp(0.693147180559945309417 * j / 512.0) * 1073741824.0;
    t.f[j] = bits_of_30(v);
    t.i[j] = static_cast<uint32_t>(v + 0.5);
  }
  return t;
}
__device__ const Pow2Table g_pow2 = make_table();

struct SampleParams {
  const void* logits;
  const float* u;
  const float* heat;    // the per-row settings, or nullptr
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logprobs;      // or nullptr
  long long stride;
  int vocab, rows, slice;   // slice: tokens of a block
  int lg;                   // log2 of vocab, rounded up
};

struct SampleShared {
  uint2 tab[512];
  uint32_t hist[2][kSmBins];
  uint2 list[2][kSmList];     // this block's candidates: (bits of x, index)
  uint2 all[kSmList];         // the cluster's
  unsigned long long weight[kSmList];
  // what the blocks exchange (two sets: a block may be one exchange ahead)
  unsigned long long sum[2];
  uint32_t cnt[2], fill[2];
  float top[2];
  unsigned long long warp_sum[kSmWarps];
  uint32_t warp_cnt[kSmWarps];
  float2 warp_bound[kSmWarps];
  // found by one thread, read by all
  int lo_bin, hi_bin, at_index;
  float at_x;
  unsigned long long at_sum;
  double row_c, row_low;      // log2 e / T; T ln min_p
};

// --------------------------------------------------------------- clusters
template <typename T>
__device__ __forceinline__ T peer_load(const T* local, uint32_t rank) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "");
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  if constexpr (sizeof(T) == 4) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return *reinterpret_cast<T*>(&v);
  } else {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return *reinterpret_cast<T*>(&v);
  }
}
__device__ __forceinline__ void blocks_sync(uint32_t blocks) {
  if (blocks == 1) {
    __syncthreads();
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- weights
constexpr float kGrid = 24576.0f;               // 1.5 * 2^14: adding it rounds to multiples of 1 / 512
constexpr float kInt = 12582912.0f;             // 1.5 * 2^23: to whole numbers
constexpr int kGridSpan = 64;
constexpr int kZero = -44 * 512;                // weights from 2^-44 of the largest down are 0

// x -> log2 of the weight, in units of 1 / 512 and a rest. (x - b) log2 e / T is formed
// as a pair of floats; b is 0, or the largest x where that is too large to be a
// multiple of 1 / 512 in fp32 (then x - b is exact for all that have a weight).
struct Scale {
  float b, ch, cl, rest, floor, top;            // rest: what the largest x's exponent has beyond its grid point
  int base, lg;
};
__device__ __forceinline__ int grid_of(const Scale& s, float x, float* frac) {
  const float d = x - s.b, p = d * s.ch;
  const float c = fmaxf(p, s.floor);            // (NaN, -infinity: the floor)
  const float t = c + kGrid;
  const float lo = fmaf(d, s.cl, fmaf(d, s.ch, -p));
  *frac = (c - (t - kGrid)) + (lo - s.rest);
  return __float_as_int(t) - s.base;            // <= 0
}
__device__ __forceinline__ int bin_of(const Scale& s, float x) {   // 1 / 16 wide, 0 the largest weight's
  const float t = fmaxf((x - s.b) * s.ch, s.floor) + kGrid;
  return min((s.base - __float_as_int(t)) >> 5, kSmBins - 1);
}
// 2^r - 1 = r ln 2 + (r ln 2)^2 / 2 + (r ln 2)^3 / 6 (|r| <= 2^-9: off by 2^-38)
__device__ __forceinline__ unsigned long long weight_of(const Scale& s, const uint2* tab, float x) {
  float r;
  const int it = grid_of(s, x, &r);
  const uint2 t = tab[it & 511];
  const float q = r * fmaf(r, fmaf(r, 0.05550411f, 0.24022651f), 0.69314718f);
  const uint32_t w = t.y + (__float_as_uint(fmaf(q, __uint_as_float(t.x), kInt)) - __float_as_uint(kInt));
  // w 2^32 >> (lg - exponent), its last place set: the middle of what was cut off
  unsigned long long y;
  asm("shr.u64 %0, %1, %2;" : "=l"(y) : "l"(static_cast<unsigned long long>(w) << 32), "r"(s.lg - (it >> 9)));
  return it > kZero ? y | 1ull : 0ull;
}

// ------------------------------------------------------------------ row
// A block's tokens in shared memory as 16-byte vectors, aligned as in global
// memory; what is not the block's in the first and the last one is -infinity. A warp
// has consecutive vectors.
template <bool F32>
struct Slice {
  const uint4* img;
  int first, count;     // the warp's vectors
  int index0;           // index of element 0 of vector 0
  static constexpr int kVec = F32 ? 4 : 8;
  bool f16;
  __device__ __forceinline__ void unpack(const uint4& u, float (&x)[kVec]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
    } else if (f16) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __half2float(__ushort_as_half(static_cast<unsigned short>(w[e >> 1] >> (16 * (e & 1)))));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    }
  }
  // f(x[kVec], index of x[0]) for every vector of the warp; lanes beyond its end get
  // -infinity, and all lanes come along
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    const int lane = threadIdx.x & 31;
    for (int i = 0; i < count; i += 32) one(i, lane, f);
  }
  template <class F>
  __device__ __forceinline__ void one(int i, int lane, F&& f) const {
    float x[kVec];
    if (i + lane < count) {
      unpack(img[first + i + lane], x);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] = -INFINITY;
    }
    f(x, index0 + (first + i + lane) * kVec);
  }
};

__device__ __forceinline__ unsigned long long warp_add(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float key_float(uint32_t k) {      // float_key's inverse
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// Sums of a pass over the whole row.
struct Sums {
  unsigned long long sum, sum_before;   // before: of the cluster's blocks of lower rank
  uint32_t cnt, cnt_before;
};

template <bool F32>
struct Sampler {
  const SampleParams& p;
  SampleShared& sh;
  Slice<F32> row;
  Scale sc;
  uint32_t rank, blocks;
  uint32_t phase = 0;
  int warp, lane;

  __device__ __forceinline__ Sampler(const SampleParams& pp, SampleShared& s) : p(pp), sh(s) {}

  // Adds up every thread's sum and count over the cluster.
  __device__ __forceinline__ Sums exchange(unsigned long long sum, uint32_t cnt) {
    const uint32_t ph = phase++ & 1;
    sum = warp_add(sum);
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) {
      sh.warp_sum[warp] = sum;
      sh.warp_cnt[warp] = cnt;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long s = 0;
      uint32_t c = 0;
#pragma unroll
      for (int w = 0; w < kSmWarps; ++w) {
        s += sh.warp_sum[w];
        c += sh.warp_cnt[w];
      }
      sh.sum[ph] = s;
      sh.cnt[ph] = c;
    }
    blocks_sync(blocks);
    Sums r;
    const bool in = static_cast<uint32_t>(lane) < blocks;
    const unsigned long long s = in ? peer_load(&sh.sum[ph], lane) : 0ull;
    const uint32_t c = in ? peer_load(&sh.cnt[ph], lane) : 0u;
    r.sum = warp_add(s);
    r.cnt = __reduce_add_sync(0xffffffffu, c);
    const bool before = static_cast<uint32_t>(lane) < rank;
    r.sum_before = warp_add(before ? s : 0ull);
    r.cnt_before = __reduce_add_sync(0xffffffffu, before ? c : 0u);
    return r;
  }

  // Two bins a thread, the first thread's the top ones, with the cluster's counts.
  // (This block's are complete after a barrier that exchange() has.)
  __device__ __forceinline__ uint2 bins(const uint32_t* hist) {
    uint2 n = make_uint2(0, 0);
    for (uint32_t r = 0; r < blocks; ++r) {
      uint32_t a;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(hist + 2 * threadIdx.x)), "r"(r));
      uint2 v;
      asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
      n.x += v.x;
      n.y += v.y;
    }
    return n;
  }
  __device__ __forceinline__ uint32_t* clear_hist() {          // the set that the next exchange belongs to
    uint32_t* h = sh.hist[phase & 1];
    for (int i = threadIdx.x; i < kSmBins; i += kSmThreads) h[i] = 0;
    __syncthreads();
    return h;
  }
  __device__ __forceinline__ void count(uint32_t* hist, int bin, bool in) {
    // (rows of equal logits: one addition a warp)
    const uint32_t who = __ballot_sync(0xffffffffu, in);
    if (who == 0) return;
    const int lead = __ffs(who) - 1;
    const int first = __shfl_sync(0xffffffffu, bin, lead);
    const uint32_t same = __ballot_sync(0xffffffffu, in && bin == first);
    if (lane == lead) atomicAdd(hist + first, __popc(same));
    else if (in && bin != first) atomicAdd(hist + bin, 1u);
  }

  // Exclusive sum over the threads before this one.
  template <typename T>
  __device__ __forceinline__ T scan(T v, T* part) {
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    T before = 0;
    for (int w = 0; w < warp; ++w) before += part[w];
    __syncthreads();
    return before + x - v;
  }

  // The bin (of two a thread) in which a running count passes `need`.
  __device__ __forceinline__ void find_count(const uint2& n, uint32_t need) {
    const uint32_t a = scan<uint32_t>(n.x + n.y, sh.warp_cnt);
    if (a < need && need <= a + n.x + n.y) sh.lo_bin = sh.hi_bin = 2 * threadIdx.x + (a + n.x < need ? 1 : 0);
    __syncthreads();
  }
  // The bins in which a running sum may pass `need`: every token of bin i weighs
  // between lower and upper (two a thread each), all relative to the largest weight.
  __device__ __forceinline__ void find_bounds(const uint2& n, const float2& lower, const float2& upper, float need) {
    const float l0 = n.x * lower.x, l1 = n.y * lower.y, u0 = n.x * upper.x, u1 = n.y * upper.y;
    if (threadIdx.x == 0) {
      sh.lo_bin = kSmBins - 1;
      sh.hi_bin = kSmBins - 1;
    }
    __syncthreads();
    const float l = scan<float>(l0 + l1, reinterpret_cast<float*>(sh.warp_bound));
    const float u = scan<float>(u0 + u1, reinterpret_cast<float*>(sh.warp_bound));
    // (1e-4: far beyond what these sums of positive terms are off by)
    const float most = need * 1.0001f, least = need * 0.9999f;
    if (u + u0 >= least) atomicMin(&sh.lo_bin, 2 * static_cast<int>(threadIdx.x));
    else if (u + u0 + u1 >= least) atomicMin(&sh.lo_bin, 2 * static_cast<int>(threadIdx.x) + 1);
    if (l + l0 >= most) atomicMin(&sh.hi_bin, 2 * static_cast<int>(threadIdx.x));
    else if (l + l0 + l1 >= most) atomicMin(&sh.hi_bin, 2 * static_cast<int>(threadIdx.x) + 1);
    __syncthreads();
  }
  __device__ __forceinline__ void find_sum(const uint2& n, unsigned long long w0, unsigned long long w1, unsigned long long need) {
    const unsigned long long s0 = n.x * w0, s1 = n.y * w1;
    const unsigned long long a = scan<unsigned long long>(s0 + s1, sh.warp_sum);
    if (a < need && need <= a + s0 + s1) sh.lo_bin = sh.hi_bin = 2 * threadIdx.x + (a + s0 < need ? 1 : 0);
    __syncthreads();
  }

  // Where a running sum over the row in index order first reaches `need` (of counts of
  // tokens that are x, or exceeds it, of weights of kept tokens): f(x, index) gives the
  // terms, `mine` this warp's sum of them. The token is left in sh.at_index and at_x.
  template <class F>
  __device__ __forceinline__ void locate(unsigned long long mine, unsigned long long before, unsigned long long need, F&& f) {
    if (lane == 0) sh.warp_sum[warp] = mine;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
    if (before < need && need <= before + mine) {
      for (int i = 0; i < row.count; i += 32) {
        unsigned long long t[Slice<F32>::kVec], own = 0;
        float xs[Slice<F32>::kVec];
        int at = 0;
        row.one(i, lane, [&](const float (&x)[Slice<F32>::kVec], int idx) {
          at = idx;
#pragma unroll
          for (int e = 0; e < Slice<F32>::kVec; ++e) {
            xs[e] = x[e];
            t[e] = f(x[e], idx + e);
            own += t[e];
          }
        });
        unsigned long long s = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += y;
        }
        const unsigned long long total = __shfl_sync(0xffffffffu, s, 31);
        unsigned long long a = before + s - own;
        if (a < need && need <= a + own) {
#pragma unroll
          for (int e = 0; e < Slice<F32>::kVec; ++e) {
            if (a < need && need <= a + t[e]) {
              sh.at_index = at + e;
              sh.at_x = xs[e];
              sh.at_sum = t[e];
            }
            a += t[e];
          }
        }
        before += total;
        if (before >= need) break;
      }
    }
  }

  // The cut: the last of the first `need` tokens of the ranking, or the token with which
  // the weights' running sum reaches `need` (of the tokens up to the cut (cx, ci) that is
  // already there). Returns the sum of weights up to it.
  //
  // From [lo, hi], values that hold the cut (`few`: at most kSmList of them): exact counts
  // and sums of what lies above hi, and either the tokens themselves or counts of them in
  // bins. The bins are of the bits of x, or, for sums while the weights' logarithms are
  // kGridSpan grid points or more apart, of those: the bounds of the sums are as far apart
  // as the weights within a bin, so every round leaves that part of what the range weighs.
  template <bool SUM>
  __device__ __forceinline__ unsigned long long cut(unsigned long long need, float lo, float hi, bool few, float* cx, int* ci) {
    const float ox = *cx;
    const int oi = *ci;
    const auto kept = [&](float x, int idx) { return x > ox || (x == ox && idx <= oi); };
    // (four rounds from all values, seldom more. The bound is for what should not be.)
    for (int round = 0; round < 20; ++round) {
      const uint32_t klo = float_key(lo), khi = float_key(hi);
      const uint32_t ph = phase & 1;
      if (lo == hi && !few) break;
      float unused;
      const int ghi = grid_of(sc, hi, &unused), span = ghi - grid_of(sc, lo, &unused);
      const bool by_grid = SUM && span >= kGridSpan && round < 10;
      int shift = 0;
      while ((by_grid ? static_cast<uint32_t>(span) : khi - klo) >> shift >= kSmBins) ++shift;
      uint32_t* hist = nullptr;
      if (!few) hist = clear_hist();
      if (threadIdx.x == 0) sh.fill[ph] = 0;
      __syncthreads();
      unsigned long long above = 0;
      uint32_t n = 0;
      row.each([&](const float (&x)[Slice<F32>::kVec], int idx) {
#pragma unroll
        for (int e = 0; e < Slice<F32>::kVec; ++e) {
          if (x[e] > hi) {
            ++n;
            if (kept(x[e], idx + e)) above += weight_of(sc, sh.tab, x[e]);
          }
          const bool in = x[e] >= lo && x[e] <= hi && (!SUM || kept(x[e], idx + e));
          if (few) {
            if (in) {
              const uint32_t at = atomicAdd(&sh.fill[ph], 1u);
              if (at < kSmList) sh.list[ph][at] = make_uint2(__float_as_uint(x[e]), idx + e);
            }
          } else {
            int bin;
            if (by_grid) bin = in ? (ghi - grid_of(sc, x[e], &unused)) >> shift : 0;
            else bin = static_cast<int>((khi - float_key(x[e])) >> shift);
            count(hist, bin, in);
          }
        }
      });
      const Sums s = exchange(above, n);
      if (SUM ? s.sum >= need : s.cnt >= need) {   // (the range does not hold it: from all values)
        few = false;
        lo = -INFINITY;
        hi = sc.top;
        continue;
      }
      if (few) {
        // all candidates in every block; each is ranked against the others
        uint32_t at = 0;
        for (uint32_t r = 0; r < blocks; ++r) {
          const uint32_t m = min(peer_load(&sh.fill[ph], r), static_cast<uint32_t>(kSmList));
          for (uint32_t i = threadIdx.x; i < m && at + i < kSmList; i += kSmThreads) {
            const unsigned long long v = peer_load(reinterpret_cast<const unsigned long long*>(&sh.list[ph][i]), r);
            sh.all[at + i] = make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
          }
          at = min(at + m, static_cast<uint32_t>(kSmList));
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < at; i += kSmThreads) sh.weight[i] = weight_of(sc, sh.tab, __uint_as_float(sh.all[i].x));
        if (threadIdx.x == 0) sh.at_index = -1;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < at; i += kSmThreads) {
          const float x = __uint_as_float(sh.all[i].x);
          const uint32_t idx = sh.all[i].y;
          unsigned long long w = 0;
          uint32_t r = 0;
          for (uint32_t k = 0; k < at; ++k) {
            const uint2 o = sh.all[k];
            const float ox2 = __uint_as_float(o.x);
            if (ox2 > x || (ox2 == x && o.y < idx)) {
              ++r;
              w += sh.weight[k];
            }
          }
          const unsigned long long a = SUM ? s.sum + w : static_cast<unsigned long long>(s.cnt + r);
          if (a < need && need <= a + (SUM ? sh.weight[i] : 1ull)) {
            sh.at_index = static_cast<int>(idx);
            sh.at_x = x;
            sh.at_sum = s.sum + w + sh.weight[i];
          }
        }
        __syncthreads();
        const int found = sh.at_index;
        if (found >= 0) {
          *cx = sh.at_x;
          *ci = found;
          const unsigned long long sum = sh.at_sum;
          __syncthreads();
          return sum;
        }
        // (not among them: from all values, by counts alone)
        __syncthreads();
        few = false;
        lo = -INFINITY;
        hi = sc.top;
        continue;
      }
      const uint2 m = bins(hist);
      const uint32_t k0 = khi - ((2 * threadIdx.x) << shift), k1 = khi - ((2 * threadIdx.x + 1) << shift);   // the bins' top keys
      if constexpr (SUM) {
        const unsigned long long rest = need - s.sum;
        if (by_grid) {
          // (a grid point to spare on either side)
          const float unit = static_cast<float>(0x1p62 / static_cast<double>(1ull << sc.lg));
          const auto w = [&](int g) { return exp2f(static_cast<float>(min(g, 0)) * (1.0f / 512.0f)) * unit; };
          const int g = ghi - ((2 * static_cast<int>(threadIdx.x)) << shift), step = 1 << shift;
          find_bounds(m, make_float2(w(g - step), w(g - 2 * step)), make_float2(w(g + 1), w(g - step + 1)), static_cast<float>(rest));
        } else if (shift == 0) {
          const unsigned long long w0 = m.x ? weight_of(sc, sh.tab, key_float(k0)) : 0ull;
          const unsigned long long w1 = m.y ? weight_of(sc, sh.tab, key_float(k1)) : 0ull;
          find_sum(m, w0, w1, rest);
        } else {
          const uint32_t step = (1u << shift) - 1;
          const auto w = [&](uint32_t k) { return static_cast<float>(weight_of(sc, sh.tab, key_float(k))); };
          const float2 upper = make_float2(m.x ? w(k0) : 0.f, m.y ? w(k1) : 0.f);
          const float2 lower = make_float2(m.x ? w(max(klo, k0 - step)) : 0.f, m.y ? w(max(klo, k1 - step)) : 0.f);
          find_bounds(m, lower, upper, static_cast<float>(rest));
        }
      } else {
        find_count(m, static_cast<uint32_t>(need) - s.cnt);
      }
      const int b0 = sh.lo_bin, b1 = sh.hi_bin;
      // how many tokens those bins hold (and, of the grid's, those whose tokens the new range may hold)
      const int more = by_grid ? (3 >> shift) + 1 : 0, bin = 2 * static_cast<int>(threadIdx.x);
      const bool in0 = bin >= b0 - more && bin <= b1 + more, in1 = bin + 1 >= b0 - more && bin + 1 <= b1 + more;
      const uint32_t here = __reduce_add_sync(0xffffffffu, (in0 ? m.x : 0u) + (in1 ? m.y : 0u));
      if (lane == 0) sh.warp_cnt[warp] = here;
      __syncthreads();
      uint32_t left = 0;
      for (int w = 0; w < kSmWarps; ++w) left += sh.warp_cnt[w];
      __syncthreads();
      if (by_grid) {
        const float inv = 1.0f / (512.0f * sc.ch);
        const int g0 = ghi - (b0 << shift) + 2, g1 = ghi - ((b1 + 1) << shift) - 2;
        hi = fminf(hi, __fsub_ru(sc.top, __fmul_rd(static_cast<float>(-min(g0, 0)), inv)));
        lo = fmaxf(lo, __fsub_rd(sc.top, __fmul_ru(static_cast<float>(-g1), inv)));
      } else {
        const uint32_t down = ((static_cast<uint32_t>(b1) + 1) << shift) - 1;
        hi = key_float(khi - (static_cast<uint32_t>(b0) << shift));
        lo = key_float(down >= khi - klo ? klo : khi - down);
      }
      few = left <= kSmList;
    }
    // more tokens of one value than a list holds: the first of them, in index order
    const float v = lo;
    unsigned long long above = 0;
    uint32_t n = 0, ties = 0;
    row.each([&](const float (&x)[Slice<F32>::kVec], int idx) {
#pragma unroll
      for (int e = 0; e < Slice<F32>::kVec; ++e) {
        if (x[e] > v) {
          ++n;
          if (kept(x[e], idx + e)) above += weight_of(sc, sh.tab, x[e]);
        }
        ties += x[e] == v && (!SUM || kept(x[e], idx + e)) ? 1u : 0u;
      }
    });
    const Sums s = exchange(above, n);
    const Sums t = exchange(0, ties);
    const unsigned long long w = weight_of(sc, sh.tab, v);
    unsigned long long take = SUM ? (need - s.sum + w - 1) / max(w, 1ull) : need - s.cnt;
    take = min(max(take, 1ull), static_cast<unsigned long long>(t.cnt));
    if (threadIdx.x == 0) sh.at_index = -1;
    const unsigned long long mine = __reduce_add_sync(0xffffffffu, ties);
    __syncthreads();
    locate(mine, t.cnt_before, take, [&](float x, int idx) { return x == v && (!SUM || kept(x, idx)) ? 1ull : 0ull; });
    __syncthreads();
    const uint32_t found = share_index();
    *cx = v;
    *ci = static_cast<int>(found);
    return s.sum + take * w;
  }

  // The index that one block of the cluster has in sh.at_index (the others: -1), in all.
  __device__ __forceinline__ uint32_t share_index() {
    const int mine = sh.at_index;
    __syncthreads();
    const Sums s = exchange(0, threadIdx.x == 0 ? static_cast<uint32_t>(mine + 1) : 0u);
    return s.cnt - 1;
  }
};

template <bool F32>
__global__ void __launch_bounds__(kSmThreads) sample_kernel(const __grid_constant__ SampleParams p, int blocks, int f16) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(smem_raw);
  uint8_t* img = smem_raw + ((sizeof(SampleShared) + 15) & ~15);
  constexpr int kBytes = F32 ? 4 : 2, kVec = 16 / kBytes;
  Sampler<F32> s(p, sh);
  s.blocks = blocks;
  s.rank = blockIdx.x % blocks;
  s.warp = threadIdx.x >> 5;
  s.lane = threadIdx.x & 31;
  const int r = blockIdx.x / blocks;
  // the block's tokens
  const int t0 = s.rank * p.slice, len = max(0, min(p.slice, p.vocab - t0));
  const uint8_t* src = static_cast<const uint8_t*>(p.logits) + (r * p.stride + t0) * kBytes;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / kBytes;
  const int vecs = (off + len + kVec - 1) / kVec, per = (vecs + kSmWarps - 1) / kSmWarps;
  s.row.img = reinterpret_cast<const uint4*>(img);
  s.row.first = min(s.warp * per, vecs);
  s.row.count = min(per, vecs - s.row.first);
  s.row.index0 = t0 - off;
  s.row.f16 = f16 != 0;
  for (int i = s.lane; i < s.row.count; i += 32) {
    const int v = s.row.first + i, e0 = v * kVec - off;          // the vector's first token, of the block's
    uint8_t* d = img + v * 16;
    if (e0 >= 0 && e0 + kVec <= len) {
      cp_async16(d, src + e0 * kBytes, true);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const bool in = e0 + e >= 0 && e0 + e < len;
        if constexpr (F32)
          reinterpret_cast<float*>(d)[e] = in ? reinterpret_cast<const float*>(src)[e0 + e] : -INFINITY;
        else
          reinterpret_cast<uint16_t*>(d)[e] = in ? reinterpret_cast<const uint16_t*>(src)[e0 + e] : f16 ? 0xfc00u : 0xff80u;
      }
    }
  }
  cp_async_commit();
  for (int i = threadIdx.x; i < 512; i += kSmThreads) sh.tab[i] = make_uint2(g_pow2.f[i], g_pow2.i[i]);
  // the row's settings
  const float heat = p.heat ? __ldg(p.heat + r) : 1.0f;
  const int k = p.top_k ? __ldg(p.top_k + r) : 0;
  const float tp = p.top_p ? __ldg(p.top_p + r) : 1.0f;
  const float mp = p.min_p ? __ldg(p.min_p + r) : 0.0f;
  if (threadIdx.x == 0) sh.row_c = fmin(1.4426950408889634074 / static_cast<double>(heat), 0x1p100);
  if (threadIdx.x == 32) {
    // (x >= max + T ln min_p: added to the maximum in 64 bits below)
    sh.row_low = mp > 0.f ? static_cast<double>(heat) * log(static_cast<double>(fminf(mp, 1.0f))) : -INFINITY;
  }
  cp_async_wait<0>();
  // the largest logit
  float top = -INFINITY;
  s.row.each([&](const float (&x)[kVec], int) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) top = fmaxf(top, x[e]);        // (NaN: passed over)
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (s.lane == 0) sh.warp_bound[s.warp].x = top;
  __syncthreads();
  const uint32_t ph = s.phase++ & 1;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kSmWarps; ++w) top = fmaxf(top, sh.warp_bound[w].x);
    sh.top[ph] = top;
  }
  blocks_sync(blocks);
  top = s.lane < blocks ? peer_load(&sh.top[ph], s.lane) : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));

  if (!(top > -INFINITY)) {                                       // nothing to take
    if (s.rank == 0 && threadIdx.x == 0) {
      p.tokens[r] = -1;
      if (p.logprobs) p.logprobs[r] = -INFINITY;
    }
    blocks_sync(blocks);
    return;
  }
  const bool greedy = !(heat > 0.f) || top == INFINITY;
  Scale& sc = s.sc;
  const double c = sh.row_c;
  sc.top = top;
  sc.ch = static_cast<float>(c);
  sc.cl = static_cast<float>(c - static_cast<double>(sc.ch));
  sc.b = fabsf(top) * sc.ch < 4096.0f ? 0.f : top;
  const float t_top = (top - sc.b) * sc.ch + kGrid;
  sc.base = __float_as_int(t_top);
  sc.rest = static_cast<float>(static_cast<double>(top - sc.b) * c - static_cast<double>(t_top - kGrid));
  sc.floor = (t_top - kGrid) - 80.0f;
  sc.lg = p.lg;

  float cx = -INFINITY;                                           // the cut: nothing yet
  int ci = 0x7fffffff;
  unsigned long long total = 0;
  const bool by_k = !greedy && k > 0 && k < p.vocab, by_p = !greedy && tp < 1.0f;
  if (greedy) {
    cx = top;                                                     // (the lowest index of it, found below)
  } else if (by_k || by_p) {
    // counts by the weights' logarithm, and the sum of all weights where top-p is of all
    uint32_t* hist = s.clear_hist();
    unsigned long long all = 0;
    s.row.each([&](const float (&x)[kVec], int) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int b = bin_of(sc, x[e]);
        s.count(hist, b, b < kSmBins - 1);
        if (by_p && !by_k) all += weight_of(sc, sh.tab, x[e]);
      }
    });
    const Sums sums = s.exchange(all, 0);
    total = sums.sum;
    const uint2 n = s.bins(hist);
    const float inv_c = 1.0f / sc.ch;
    // values that surely hold all of bins b0 .. b1 (a bin more on either side), and
    // whether a list holds those bins' tokens
    const auto range = [&](int b0, int b1, float* lo, float* hi) {
      const int a0 = b0 - 1, a1 = b1 + 1, mine = 2 * static_cast<int>(threadIdx.x);
      const uint32_t here = __reduce_add_sync(0xffffffffu, (mine >= a0 && mine <= a1 ? n.x : 0u) + (mine + 1 >= a0 && mine + 1 <= a1 ? n.y : 0u));
      if (s.lane == 0) sh.warp_cnt[s.warp] = here;
      __syncthreads();
      uint32_t left = 0;
      for (int w = 0; w < kSmWarps; ++w) left += sh.warp_cnt[w];
      __syncthreads();
      *hi = b0 <= 1 ? top : fminf(top, __fsub_ru(top, __fmul_rd(static_cast<float>(b0) / 16.0f - 1.0f / 32.0f, inv_c)));
      *lo = __fsub_rd(top, __fmul_ru(static_cast<float>(b1 + 1) / 16.0f + 1.0f / 32.0f, inv_c));
      return left <= kSmList && a1 < kSmBins - 1;
    };
    float lo, hi;
    bool cut_k = false;
    if (by_k) {
      if (threadIdx.x == 0) sh.lo_bin = -1;
      __syncthreads();
      s.find_count(n, k);
      const int b = sh.lo_bin;
      __syncthreads();
      if (b >= 0) {                                               // (else: more tokens than have a weight)
        const bool few = range(b, b, &lo, &hi);
        total = s.template cut<false>(k, lo, hi, few, &cx, &ci);
        cut_k = true;
      } else if (by_p) {
        unsigned long long sum = 0;
        s.row.each([&](const float (&x)[kVec], int) {
#pragma unroll
          for (int e = 0; e < kVec; ++e) sum += weight_of(sc, sh.tab, x[e]);
        });
        total = s.exchange(sum, 0).sum;
      }
    }
    if (by_p) {
      // the least sum that is p of the total, rounded up
      const unsigned long long pf = tp > 0.f ? static_cast<unsigned long long>(static_cast<double>(tp) * 0x1p64) : 0ull;
      unsigned long long need = __umul64hi(pf, total) + (pf * total != 0 ? 1 : 0);
      need = max(need, 1ull);
      const float unit = static_cast<float>(0x1p62 / static_cast<double>(1ull << p.lg));   // the largest weight
      const auto edge = [&](int b) { return exp2f(-static_cast<float>(b) / 16.0f) * unit; };
      const int b = 2 * threadIdx.x;
      s.find_bounds(n, make_float2(edge(b + 1) * 0.997f, edge(b + 2) * 0.997f), make_float2(edge(b) * 1.003f, edge(b + 1) * 1.003f),
                    static_cast<float>(need));
      const int b0 = sh.lo_bin, b1 = sh.hi_bin;
      __syncthreads();
      const bool few = range(b0, b1, &lo, &hi);
      if (cut_k) {                                                // (the cut there is ends the range)
        lo = fmaxf(lo, cx);
        hi = fmaxf(hi, cx);
      }
      total = s.template cut<true>(need, lo, hi, few, &cx, &ci);
    }
  }
  if (!greedy && mp > 0.f) {
    const float f = __double2float_ru(static_cast<double>(top) + sh.row_low);
    if (f > cx) {
      cx = f;
      ci = 0x7fffffff;
    }
  }
  // the draw: the first token in index order at which the kept weights' sum exceeds u of all
  const auto term = [&](float x, int idx) -> unsigned long long {
    if (!(x > cx || (x == cx && idx <= ci))) return 0ull;
    return greedy ? 1ull : weight_of(sc, sh.tab, x);
  };
  unsigned long long sum = 0;
  s.row.each([&](const float (&x)[kVec], int idx) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum += term(x[e], idx + e);
  });
  const Sums all = s.exchange(sum, 0);
  unsigned long long need = 1;
  if (!greedy) {
    float u = __ldg(p.u + r);
    u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
    need = __umul64hi(static_cast<unsigned long long>(static_cast<double>(u) * 0x1p64), all.sum) + 1;
  }
  const unsigned long long mine = warp_add(sum);
  if (threadIdx.x == 0) sh.at_index = -1;
  __syncthreads();
  s.locate(mine, all.sum_before, need, term);
  __syncthreads();
  if (threadIdx.x == 0 && sh.at_index >= 0) {                     // one block has it
    p.tokens[r] = sh.at_index;
    if (p.logprobs) {
      float lp = 0.f;
      if (!greedy) {
        const unsigned long long rest = all.sum - sh.at_sum;
        if (rest < sh.at_sum) {
          lp = log1pf(-static_cast<float>(static_cast<double>(rest) / static_cast<double>(all.sum)));
        } else {
          const double unit = 0x1p62 / static_cast<double>(1ull << p.lg);
          lp = (sh.at_x - top) / heat - logf(static_cast<float>(static_cast<double>(all.sum) / unit));
        }
      }
      p.logprobs[r] = lp;
    }
  }
  blocks_sync(blocks);                                            // (nobody reads a block that has gone)
}


template <bool F32>
cudaError_t launch_sample(SampleParams p, int f16, int sms, cudaStream_t st) {
  constexpr int kBytes = F32 ? 4 : 2;
  // Blocks of a row: as few as hold it, and more where SMs would be idle and a block
  // would still have 4,096 tokens.
  int blocks = 1;
  const auto slice_of = [&](int n) { return ((p.vocab + n - 1) / n + 63) / 64 * 64; };
  while (blocks < kSmMaxCluster && slice_of(blocks) * kBytes > kSmMaxData) blocks *= 2;
  while (blocks < 8 && 2LL * p.rows * blocks <= sms && slice_of(2 * blocks) >= 4096) blocks *= 2;
  p.slice = slice_of(blocks);
  const size_t smem = ((sizeof(SampleShared) + 15) & ~size_t{15}) + static_cast<size_t>(p.slice) * kBytes + 32;
  const void* fn = reinterpret_cast<const void*>(&sample_kernel<F32>);
  cudaError_t e = set_max_smem(fn, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (blocks > 8 && (e = set_nonportable_cluster(fn)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * blocks);
  cfg.blockDim = dim3(kSmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, sample_kernel<F32>, p, blocks, f16);
  if (e == cudaSuccess) note_launch("sample_kernel");
  return e;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_sample(const dsa_sample_problem* sp, const void* logits, const float* uniform, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens, float* logprobs,
                          void* stream) {
  reset_launches();
  if (!sp) return report_error(DSA_ERR_INVALID_ARG, "problem is NULL");
  if (sp->rows < 1 || sp->rows > 65535) return report_errorf(DSA_ERR_INVALID_ARG, "rows %d outside 1..65535", sp->rows);
  if (sp->vocab < 1) return report_errorf(DSA_ERR_INVALID_ARG, "vocab %d < 1", sp->vocab);
  if (sp->vocab > kSmMaxVocab) return report_errorf(DSA_ERR_UNSUPPORTED, "vocab %d above %d", sp->vocab, kSmMaxVocab);
  if (sp->logits_dtype != DSA_BF16 && sp->logits_dtype != DSA_FP16 && sp->logits_dtype != DSA_FP32)
    return report_error(DSA_ERR_UNSUPPORTED, "logits_dtype must be BF16, FP16 or FP32");
  if (sp->row_stride != 0 && (sp->row_stride < sp->vocab || sp->row_stride > (1LL << 40)))
    return report_error(DSA_ERR_INVALID_ARG, "row_stride must be 0 or at least vocab");
  if (!logits || !uniform || !tokens) return report_error(DSA_ERR_INVALID_ARG, "logits, uniform and tokens are required");
  const int eb = sp->logits_dtype == DSA_FP32 ? 4 : 2;
  const auto off = [](const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) != 0; };
  if (off(logits, eb) || off(uniform, 4) || off(temperature, 4) || off(top_k, 4) || off(top_p, 4) || off(min_p, 4) ||
      off(tokens, 4) || off(logprobs, 4))
    return report_error(DSA_ERR_MISALIGNED, "arrays must be aligned to their elements");
  SampleParams p{};
  p.stride = sp->row_stride ? sp->row_stride : sp->vocab;
  const long long n = 4LL * sp->rows, all = ((sp->rows - 1) * p.stride + sp->vocab) * eb;
  for (const void* o : {static_cast<const void*>(tokens), static_cast<const void*>(logprobs)}) {
    if (!o) continue;
    bool over = overlap(o, n, logits, all);
    for (const void* i : {static_cast<const void*>(uniform), static_cast<const void*>(temperature), static_cast<const void*>(top_k),
                          static_cast<const void*>(top_p), static_cast<const void*>(min_p)})
      over = over || (i && overlap(o, n, i, n));
    if (over) return report_error(DSA_ERR_INVALID_ARG, "a result overlaps an input");
  }
  if (logprobs && overlap(tokens, n, logprobs, n)) return report_error(DSA_ERR_INVALID_ARG, "results overlap each other");
  int sms = 0;
  if (int rc = current_device(&sms)) return rc;
  p.logits = logits, p.u = uniform, p.heat = temperature, p.top_k = top_k, p.top_p = top_p, p.min_p = min_p;
  p.tokens = tokens, p.logprobs = logprobs, p.vocab = sp->vocab, p.rows = sp->rows;
  while ((1 << p.lg) < sp->vocab) ++p.lg;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = sp->logits_dtype == DSA_FP32 ? launch_sample<true>(p, 0, sms, st)
                                                     : launch_sample<false>(p, sp->logits_dtype == DSA_FP16, sms, st);
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "sample launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}
