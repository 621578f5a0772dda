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
// sums have to be the same whatever the order: a weight is a multiple of 2^-45 with the
// largest in [1/2, 1), formed in fp32 pairs to about 2^-33 of itself, and all sums are of
// 64-bit integers.
//
// A cluster of blocks holds a row in shared memory (read once); everything else is
// passes over it and exchanges between the blocks. A list of the tokens that reach a
// value, which enough of the threads' largest ones do, settles most rows: sorted, it
// has the cut of top-k, and of top-p where the list weighs enough. Otherwise the cut is
// looked for in counts of all tokens by the logarithm of the weight, 1,024 bins of 1/32 of
// its base-2 logarithm with the sum of what the tokens lie below their bin's edge: these
// bound the running sum to a part in 10,000, so that one or two bins hold the cut, and a
// pass that forms the exact sum of what lies before them and lists their tokens does the
// rest (if they are too many for a list, they are counted again, by smaller bins).
//
// What bounds it: not memory (64 rows of 131,072 in bf16 are 2.5 us of reads). About half is issue
// slots (top-p: 34 million warp instructions on 128 SMs, 32 us of 60 at 2.07 GHz; 30 a token in
// the passes that form weights), the rest waiting: one block of 1,024 threads an SM, whose
// barriers between passes nothing else runs under, atomics in shared memory, exchanges in the
// cluster, a microsecond each, and 24 of the 152 SMs idle with two blocks for each of 64 rows.
// Schedulers are busy 42 to 67% of the time, the half-rate integer pipe 23 to 37%. Measured
// (64 x 131,072 bf16, replayed, L2 flushed): temperature alone 22.5 us, min-p 23.3, top-k 26.2,
// top-p 63.5 (two passes that form weights and one that counts in shared memory), a mix of them
// 58; 256 x 32,000 mixed 48; 1 x 131,072 12.3 / 15.7 / 38 (temperature, top-k, top-p).
#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "kept_answers.h"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

constexpr int kSmThreads = 1024, kSmWarps = kSmThreads / 32;
constexpr int kSmBins = kSmThreads;             // one a thread
constexpr int kSmList = kSmThreads;             // candidates that are sorted, one a thread
constexpr int kSmFewK = 640, kSmFewP = 256;     // tokens that a list is expected to hold, of top-k and of top-p alone
constexpr int kSmMaxVocab = 1 << 19;
constexpr int kSmMaxCluster = 16;
constexpr int kSmMaxData = 172032;              // bytes of a row that a block holds

// 2^(j / 512), j = 0 .. 511, as pairs of floats.
struct Pow2Table {
  float2 v[512];
};
constexpr double series_exp(double x) {         // |x| < 0.7: 1 + x (1 + x / 2 (1 + x / 3 (...)))
  double s = 1.0;
  for (int k = 24; k >= 1; --k) s = 1.0 + x * s / k;
  return s;
}
constexpr Pow2Table make_table() {
  Pow2Table t{};
  for (int j = 0; j < 512; ++j) {
    const double v = series_exp(0.693147180559945309417 * j / 512.0);
    t.v[j].x = static_cast<float>(v);
    t.v[j].y = static_cast<float>(v - static_cast<double>(t.v[j].x));
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
};

struct SampleShared {
  float2 tab[512];
  unsigned long long sort[2][kSmList];            // (or two lists of candidates at once)
  // what the blocks exchange, in two sets: a block may be one exchange ahead
  uint32_t hist[2][kSmBins], below[2][kSmBins];   // tokens of a bin; the sum of what they lie below its edge
  unsigned long long list[2][kSmList];            // this block's candidates: (key of x, ~index)
  unsigned long long sum[2];
  uint32_t cnt[2], fill[2], fill_two[2];
  float top[2], low[2];
  // scratch of the block
  unsigned long long warp_sum[kSmWarps], cand_sum[kSmWarps];
  uint32_t warp_cnt[kSmWarps];
  float warp_bound[kSmWarps];
  // found by one thread, read by all
  int lo_bin, hi_bin, at_index;
  float at_x;
  unsigned long long at_sum;
  float2 row_c, row_low;      // log2 e / T and T ln min_p, as pairs of floats
};

// --------------------------------------------------------------- clusters
// The aligned barriers here and in sorted() want a warp's lanes together, and single lanes' work
// often comes just before them: __syncwarp says so to the compiler.
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
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A block must not end while another may read it: it arrives once it has read the
// others, and waits before it ends.
__device__ __forceinline__ void blocks_leave(uint32_t blocks) {
  __syncwarp();
  if (blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void blocks_left(uint32_t blocks) {
  __syncwarp();
  if (blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- weights
constexpr float kGrid = 24576.0f;               // 1.5 * 2^14: adding it rounds to multiples of 1 / 512
constexpr float kInt = 12582912.0f;             // 1.5 * 2^23: to whole numbers
constexpr float kHigh = 3.0f;                   // 1.5 * 2^1: to multiples of 2^-22
constexpr float kLow = 0x1.8p-22f;              // 1.5 * 2^-22: to multiples of 2^-45
constexpr int kGridSpan = 64;
constexpr int kBinShift = 4, kBinPoints = 1 << kBinShift;   // grid points of a bin
constexpr int kZero = 60 * 512;                 // weights from 2^-60 of the largest down are none at all
// What an exponent has beyond its grid point, in points: half of one by the rounding; an eighth that
// the product (x - b) ch is rounded by (of up to 4,096 + 80: half a unit in its last place is 2^-12);
// and another that cl adds (4,176 x 2^-24). In all 0.753.
constexpr float kRest = 0.76f;
// x -> log2 of the weight, in units of 1 / 512 and a rest: (x - b) (ch + cl), ch + cl =
// log2 e / T as a pair of floats. b is 0, or the largest x where that is too large to be a
// multiple of 1 / 512 in fp32 (x - b then is exact for all that have a weight).
struct Scale {
  float b, ch, cl, floor, top;                  // floor: exponents below it are taken as it
  int base, zero;                               // the largest x's grid point; the last one without a weight
  uint32_t power;                               // what turns a whole exponent's bits into its power of two's
  float rest;                                   // of the largest x, beside its grid point
};
__device__ __forceinline__ int point_of(const Scale& s, float x) {   // the grid point, as the bits of a float
  return __float_as_int(__fadd_rn(fmaxf(__fmul_rn(__fadd_rn(x, -s.b), s.ch), s.floor), kGrid));   // (NaN, -infinity: the floor's)
}
__device__ __forceinline__ int grid_of(const Scale& s, float x) { return point_of(s, x) - s.base; }   // <= 0

// A weight, the largest in [1/2, 1), as the bits of kHigh + h and kLow + l, h a multiple
// of 2^-22 and l the rest, of 2^-45 (rounded to the nearest). Nearly all in fp32 additions
// and multiply-adds with immediate operands: the integer pipe has half their rate, and
// pairs of fp32 operations need their constants in registers, which are not there.
struct Weight {
  uint32_t h, l;
  int point;                                    // the token's grid point,
  float r;                                      // and what its exponent has beyond it
  __device__ __forceinline__ unsigned long long value() const {   // in units of 2^-45
    return (static_cast<unsigned long long>(h - __float_as_uint(kHigh)) << 23) +
           static_cast<long long>(static_cast<int>(l - __float_as_uint(kLow)));
  }
};
// (in(point): whether it counts, else 0.) 2^r - 1 = r ln 2 + (r ln 2)^2 / 2 + (r ln 2)^3 / 6
// with |r| <= kRest / 512: off by 2^-44.
template <class F>
__device__ __forceinline__ Weight weight_if(const Scale& s, const float2* tab, float x, F&& in) {
  const float d = __fadd_rn(x, -s.b), n = __fmul_rn(d, s.ch), c = fmaxf(n, s.floor);
  const float t = __fadd_rn(c, kGrid), k = __fadd_rn(t, -kGrid);
  float r = __fadd_rn(__fadd_rn(c, -k), __fmaf_rn(d, s.cl, __fmaf_rn(d, s.ch, -n)));
  Weight y;
  y.point = __float_as_int(t);
  if (y.point <= s.zero) r = 0.f;               // (it may be infinite or NaN; the power leaves nothing)
  y.r = r;
  const float2 a = tab[y.point & 511];
  const float q = __fmul_rn(r, __fmaf_rn(r, __fmaf_rn(r, 0.05550411f, 0.24022651f), 0.69314718f));
  const float b = __fmaf_rn(a.x, q, a.y), w = __fadd_rn(a.x, b), e = __fadd_rn(__fadd_rn(a.x, -w), b);   // w + e = a (1 + q)
  float p = __uint_as_float(__float_as_uint(__fadd_rd(k, kInt)) * 0x800000u + s.power);
  if (!in(y.point)) p = 0.f;
  const float h = __fmaf_rn(w, p, kHigh);
  y.h = __float_as_uint(h);
  y.l = __float_as_uint(__fadd_rn(__fmaf_rn(e, p, __fmaf_rn(w, p, __fadd_rn(kHigh, -h))), kLow));
  return y;
}
__device__ __forceinline__ unsigned long long weight_of(const Scale& s, const float2* tab, float x) {
  return weight_if(s, tab, x, [](int) { return true; }).value();
}
// A thread's sum (of 512 weights at most: 32 bits each hold h and l).
struct WeightSum {
  uint32_t h = 0, l = 0, pairs = 0;             // of the bits: kHigh's and kLow's are taken off at the end
  __device__ __forceinline__ void add(const Weight& a, const Weight& b) {
    h += a.h + b.h;
    l += a.l + b.l;
    ++pairs;
  }
  __device__ __forceinline__ unsigned long long value() const {
    return (static_cast<unsigned long long>(h - pairs * (2 * __float_as_uint(kHigh))) << 23) +
           static_cast<long long>(static_cast<int>(l - pairs * (2 * __float_as_uint(kLow))));
  }
};

// ------------------------------------------------------------------ row
// A block's tokens in shared memory as 16-byte vectors, aligned as in global memory;
// what is not the block's in the first and the last one is -infinity, and so are the
// vectors up to a multiple of 32. A warp has consecutive ones.
template <int TYPE>
struct Slice {
  static constexpr bool kF32 = TYPE == DSA_FP32;
  static constexpr int kVec = kF32 ? 4 : 8;
  const uint4* img;
  int first, count;     // the warp's vectors: a multiple of 32
  int vecs, per;        // the block's, and a warp's
  int index0;           // index of element 0 of vector 0
  __device__ __forceinline__ static void unpack(const uint4& u, float (&x)[kVec]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if constexpr (kF32) x[e] = __uint_as_float(w[e]);
      else if constexpr (TYPE == DSA_FP16) x[e] = __half2float(__ushort_as_half(static_cast<unsigned short>(w[e >> 1] >> (16 * (e & 1)))));
      else x[e] = __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    }
  }
  // f(x[kVec], index of x[0]) for every vector of the warp; all lanes come along
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = 0; i < count; i += 32) one(first + i + lane, f);
  }
  template <class F>
  __device__ __forceinline__ void one(int v, F&& f) const {
    float x[kVec];
    unpack(img[v], x);
    f(x, index0 + v * kVec);
  }
  // f(x0, x1, index of x0) for every two tokens of n vectors from `from` on (a multiple of
  // 32): what passes that form weights take, for eight at once in each of them would be
  // more code than the instruction cache holds (top-p of 64 x 131,072: 83 and not 89 us).
  template <class F>
  __device__ __forceinline__ void pairs(int from, int n, F&& f) const {
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < n * (kVec / 2); i += 32) pair(from * (kVec / 2) + i, f);
  }
  // The same for every four, in the two passes of most nuclei (64 x 131,072 mixed: 58 and not 60 us).
  template <class F>
  __device__ __forceinline__ void quads(int from, int n, F&& f) const {
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < n * (kVec / 4); i += 32) {
      const int j = from * (kVec / 4) + i;
      float x[4];
      if constexpr (kF32) {
        const float4 v = reinterpret_cast<const float4*>(img)[j];
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
      } else {
        const uint2 w = reinterpret_cast<const uint2*>(img)[j];
        if constexpr (TYPE == DSA_FP16) {
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
          x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
        } else {
          x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xffff0000u);
          x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xffff0000u);
        }
      }
      f(x, index0 + 4 * j);
    }
  }
  template <class F>
  __device__ __forceinline__ void pair(int i, F&& f) const {
    if constexpr (kF32) {
      const float2 x = reinterpret_cast<const float2*>(img)[i];
      f(x.x, x.y, index0 + 2 * i);
    } else {
      const uint32_t w = reinterpret_cast<const uint32_t*>(img)[i];
      if constexpr (TYPE == DSA_FP16) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
        f(x.x, x.y, index0 + 2 * i);
      } else {
        f(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u), index0 + 2 * i);
      }
    }
  }
};

__device__ __forceinline__ unsigned long long warp_add(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
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

template <int TYPE>
struct Sampler {
  const SampleParams& p;
  SampleShared& sh;
  Slice<TYPE> row;
  Scale sc;
  uint32_t rank, blocks;
  uint32_t phase = 0;
  int warp, lane;
  // the list that the last cut was found in: this thread's candidate (0: none), its sum of
  // what lies above list_top, that of all threads
  bool listed = false;
  unsigned long long cand = 0, list_above = 0;
  Sums list_sums;
  float list_top;

  __device__ __forceinline__ Sampler(const SampleParams& pp, SampleShared& s) : p(pp), sh(s) {}

  // The weight of the largest x's grid point (its own is 2^rest times it).
  __device__ __forceinline__ float unit() const {
    return sh.tab[sc.base & 511].x * 0x1p44f;
  }

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
    if (warp == 0) {
      const unsigned long long s = warp_add(sh.warp_sum[lane]);
      const uint32_t c = __reduce_add_sync(0xffffffffu, sh.warp_cnt[lane]);
      if (lane == 0) {
        sh.sum[ph] = s;
        sh.cnt[ph] = c;
      }
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

  // The cluster's counts, a bin a thread. (This block's are complete after a barrier
  // that exchange() has.)
  __device__ __forceinline__ uint32_t bins(const uint32_t* hist) {
    uint32_t n = 0;
#pragma unroll
    for (uint32_t r = 0; r < kSmMaxCluster; ++r)
      if (r < blocks) n += peer_load(hist + threadIdx.x, r);
    return n;
  }
  __device__ __forceinline__ uint32_t* clear_hist() {          // the set that the next exchange belongs to
    uint32_t* h = sh.hist[phase & 1];
    for (int i = threadIdx.x; i < kSmBins; i += kSmThreads) h[i] = 0;
    __syncthreads();
    return h;
  }
  // Counts two tokens in their bins (-1: none), at once where it is the same: rows of equal
  // logits would otherwise meet in one place.
  __device__ __forceinline__ void count(uint32_t* hist, int b0, int b1) {
    if (b0 >= 0) atomicAdd(hist + b0, b0 == b1 ? 2u : 1u);
    if (b1 >= 0 && b0 != b1) atomicAdd(hist + b1, 1u);
  }
  // The same by the weights: bins of kBinPoints grid points, and how far below its bin's
  // edge a token lies, in 64ths of a point (and kBelow of them more, so that it is positive: a sum
  // of a bin that is not would wrap around, and its bounds with it).
  static constexpr int kBelow = 50;
  static_assert(kBelow >= 64 * kRest + 0.5f, "");
  __device__ __forceinline__ void count_weights(uint32_t* hist, uint32_t* below, const Weight& a, const Weight& b) {
    const int g0 = sc.base - a.point, g1 = sc.base - b.point, b0 = g0 >> kBinShift, b1 = g1 >> kBinShift;   // (both >= 0)
    const auto under = [](int g, float r) {
      return static_cast<uint32_t>((g & (kBinPoints - 1)) * 64 + kBelow + __float_as_int(fmaf(r, -32768.0f, kInt)) - __float_as_int(kInt));
    };
    uint32_t n = 1, s0 = under(g0, a.r);
    const uint32_t s1 = under(g1, b.r);
    if (b0 == b1) {
      n = 2;
      s0 += s1;
    }
    if (b0 < kSmBins - 1) {
      atomicAdd(hist + b0, n);
      atomicAdd(below + b0, s0);
    }
    if (b1 < kSmBins - 1 && b0 != b1) {
      atomicAdd(hist + b1, 1u);
      atomicAdd(below + b1, s1);
    }
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
    T before = lane < warp ? part[lane] : T(0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    __syncthreads();
    T own = __shfl_up_sync(0xffffffffu, x, 1);
    if (lane == 0) own = 0;
    return before + own;
  }

  // The bins in which a running count passes `need`, and `more`.
  __device__ __forceinline__ void find_count(uint32_t n, uint32_t need, uint32_t more) {
    const uint32_t a = scan<uint32_t>(n, sh.warp_cnt);
    if (a < need && need <= a + n) sh.lo_bin = threadIdx.x;
    if (a < more && more <= a + n) sh.hi_bin = threadIdx.x;
    __syncthreads();
  }
  __device__ __forceinline__ void find_count(uint32_t n, uint32_t need) { find_count(n, need, need); }
  // The bins in which a running sum may pass `need`: what the thread's bin holds weighs
  // between l0 and u0.
  __device__ __forceinline__ void find_bounds(float l0, float u0, float need) {
    if (threadIdx.x == 0) sh.lo_bin = sh.hi_bin = kSmBins - 1;
    const float l = scan<float>(l0, sh.warp_bound) + l0;
    const float u = scan<float>(u0, sh.warp_bound) + u0;
    // (2e-5: far beyond what these sums of positive terms are off by)
    if (u >= need * 0.99998f) atomicMin(&sh.lo_bin, static_cast<int>(threadIdx.x));
    if (l >= need * 1.00002f) atomicMin(&sh.hi_bin, static_cast<int>(threadIdx.x));
    __syncthreads();
  }
  __device__ __forceinline__ void find_sum(uint32_t n, unsigned long long w, unsigned long long need) {
    const unsigned long long s = n * w, a = scan<unsigned long long>(s, sh.warp_sum);
    if (a < need && need <= a + s) sh.lo_bin = sh.hi_bin = threadIdx.x;
    __syncthreads();
  }
  // Tokens in bins b0 .. b1.
  __device__ __forceinline__ uint32_t held(uint32_t n, int b0, int b1) {
    const int b = threadIdx.x;
    const uint32_t here = __reduce_add_sync(0xffffffffu, b >= b0 && b <= b1 ? n : 0u);
    if (lane == 0) sh.warp_cnt[warp] = here;
    __syncthreads();
    const uint32_t all = __reduce_add_sync(0xffffffffu, sh.warp_cnt[lane]);
    __syncthreads();
    return all;
  }
  // A sum over the block's threads.
  __device__ __forceinline__ unsigned long long block_add(unsigned long long v) {
    v = warp_add(v);
    if (lane == 0) sh.warp_sum[warp] = v;
    __syncthreads();
    v = warp_add(sh.warp_sum[lane]);
    __syncthreads();
    return v;
  }

  // Where a running sum over the row in index order first reaches `need` (of counts of
  // tokens that are x, or exceeds it, of weights of kept tokens): f(x, index) gives the
  // terms, `mine` this warp's sum of them. The token is left in sh.at_index and at_x.
  template <class F>
  __device__ __forceinline__ void locate(unsigned long long mine, unsigned long long before, unsigned long long need, F&& f) {
    if (lane == 0) sh.warp_sum[warp] = mine;
    __syncthreads();
    // the warp that has it, then its rounds of 32 vectors, one a warp (11 at most)
    unsigned long long x = sh.warp_sum[lane], own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t who = __ballot_sync(0xffffffffu, before + x - own < need && need <= before + x);
    __syncthreads();
    if (who == 0) return;
    const int w = __ffs(who) - 1;
    before += __shfl_sync(0xffffffffu, x - own, w);
    const int v0 = min(w * row.per, row.vecs), n = min(row.per, row.vecs - v0);
    constexpr int kPairs = Slice<TYPE>::kVec / 2;
    const int v = (v0 + warp * 32 + lane) * kPairs;               // the lane's first pair, of kPairs
    own = 0;
    if (warp * 32 < n) {
#pragma unroll 1
      for (int i = 0; i < kPairs; ++i) row.pair(v + i, [&](float x0, float x1, int idx) { own += f(x0, idx) + f(x1, idx + 1); });
    }
    const unsigned long long round = warp_add(own);
    if (lane == 0) sh.warp_sum[warp] = round;
    __syncthreads();
    before += warp_add(lane < warp ? sh.warp_sum[lane] : 0ull);
    if (before < need && need <= before + round) {
      unsigned long long s = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      unsigned long long a = before + s - own;
      if (a < need && need <= a + own) {
#pragma unroll 1
        for (int i = 0; i < kPairs; ++i)
          row.pair(v + i, [&](float x0, float x1, int idx) {
            const unsigned long long t0 = f(x0, idx), t1 = f(x1, idx + 1);
            const bool first = a < need && need <= a + t0, second = a + t0 < need && need <= a + t0 + t1;
            if (first || second) {
              sh.at_index = first ? idx : idx + 1;
              sh.at_x = first ? x0 : x1;
              sh.at_sum = first ? t0 : t1;
            }
            a += t0 + t1;
          });
      }
    }
  }

  // All blocks' candidates of a list: one a thread, 0 where there is none; returns how many
  // there are (more than kSmList: not all of them).
  __device__ __forceinline__ uint32_t collect(const unsigned long long* list, const uint32_t* fill, unsigned long long* mine) {
    const uint32_t m = static_cast<uint32_t>(lane) < blocks ? peer_load(fill, lane) : 0u;
    uint32_t end = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    const uint32_t n = __shfl_sync(0xffffffffu, end, 31);
    *mine = 0;
    if (n > kSmList) return n;
    // the block whose range the thread is in: as many ends as are at most its number
    uint32_t r = 0, first = 0;
    for (uint32_t k = 0; k + 1 < blocks; ++k) {
      const uint32_t e = __shfl_sync(0xffffffffu, end, k);
      if (threadIdx.x >= e) {
        r = k + 1;
        first = e;
      }
    }
    if (threadIdx.x < n) *mine = peer_load(list + (threadIdx.x - first), r);
    return n;
  }
  __device__ __forceinline__ static void offer(unsigned long long* list, uint32_t* fill, float x, int idx) {
    const uint32_t at = atomicAdd(fill, 1u);
    if (at < kSmList) list[at] = static_cast<unsigned long long>(float_key(x)) << 32 | static_cast<uint32_t>(~idx);
  }
  __device__ __forceinline__ void offer(uint32_t ph, float x, int idx) { offer(sh.list[ph], &sh.fill[ph], x, idx); }
  // Sorts the threads' first n candidates, the largest first: 32 by a bitonic sort within
  // a warp, then runs of 32, 64 .. merged: a candidate's place is its own in its run and
  // that of as many of the other's as are larger, by bisection. (Of 600 candidates: 5.4 us,
  // a bitonic sort across the block 8.5.) Only the warps that have some take part.
  __device__ __forceinline__ unsigned long long sorted(unsigned long long v, uint32_t n) {
    uint32_t size = 32;
    while (size < n) size <<= 1;
    if (threadIdx.x >= size) return 0;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
      for (int j = k >> 1; j > 0; j >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, v, j);
        const bool first = (lane & j) == 0, down = (lane & k) == 0 || k == 32;
        v = first == down ? max(v, o) : min(v, o);
      }
    const uint32_t t = threadIdx.x;
    unsigned long long *a = sh.sort[0], *b = sh.sort[1];
    for (uint32_t run = 32; run < size; run <<= 1) {
      a[t] = v;
      __syncwarp();
      named_bar_sync(1, size);
      // (empty places are zeros: of equal ones the first run's come first)
      const bool second = (t & run) != 0;
      const uint32_t other = (t & ~(2 * run - 1)) + (second ? 0 : run);
      uint32_t lo = 0, hi = run;
      while (lo < hi) {
        const uint32_t mid = (lo + hi) >> 1;
        const unsigned long long o = a[other + mid];
        if (o > v || (second && o == v)) lo = mid + 1;
        else hi = mid;
      }
      const uint32_t to = (t & ~(2 * run - 1)) + (t & (run - 1)) + lo;
      b[to] = v;
      __syncwarp();
      named_bar_sync(1, size);
      v = b[t];
    }
    return v;
  }
  // A candidate's value and index.
  __device__ __forceinline__ static float value_of(unsigned long long c) { return key_float(static_cast<uint32_t>(c >> 32)); }
  __device__ __forceinline__ static int index_of(unsigned long long c) { return static_cast<int>(~static_cast<uint32_t>(c)); }

  // The cut among the candidates of a list (`all` in number, this thread's in cand), which
  // `above` tokens of weight `sum` rank before: the need-th token of the ranking, or the one
  // with which the running sum reaches `need`. Whether it is there; *upto: the sum of
  // weights up to it.
  template <bool SUM>
  __device__ __forceinline__ bool settle(uint32_t all, unsigned long long sum, uint32_t above, unsigned long long need, float* cx,
                                         int* ci, unsigned long long* upto) {
    if (threadIdx.x == 0) sh.at_index = -1;
    cand = sorted(cand, min(all, static_cast<uint32_t>(kSmList)));
    const bool in = threadIdx.x < all && all <= kSmList;
    const unsigned long long own = in ? weight_of(sc, sh.tab, value_of(cand)) : 0ull;
    const unsigned long long before = sum + scan<unsigned long long>(own, sh.warp_sum);
    const unsigned long long a = SUM ? before : static_cast<unsigned long long>(above) + threadIdx.x;
    if (in && a < need && need <= a + (SUM ? own : 1ull)) {
      sh.at_index = index_of(cand);
      sh.at_x = value_of(cand);
      sh.at_sum = before + own;
    }
    __syncthreads();
    listed = sh.at_index >= 0;
    if (listed) {
      *cx = sh.at_x;
      *ci = sh.at_index;
      *upto = sh.at_sum;
    }
    if (!in) cand = 0;
    __syncthreads();
    return listed;
  }
  // The same of the tokens of bins b0 .. b1 (kSmList at most) of the counts by the weights,
  // `above` tokens in those before.
  template <bool SUM>
  __device__ __forceinline__ bool cut_bins(int b0, int b1, uint32_t above, unsigned long long need, float* cx, int* ci,
                                           unsigned long long* upto) {
    const uint32_t ph = phase & 1;
    const int p0 = sc.base - kBinPoints * b0, p1 = sc.base - kBinPoints * (b1 + 1) + 1;
    if (threadIdx.x == 0) sh.fill[ph] = 0;
    __syncthreads();
    WeightSum sum;
    const float low = below_bin(b1 + 1);          // (what lies in these bins does not lie below it)
    row.quads(row.first, row.count, [&](const float (&x)[4], int idx) {
      if (!__any_sync(0xffffffffu, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= low)) return;
      const auto over = [&](int point) { return point > p0; };
      const Weight a = weight_if(sc, sh.tab, x[0], over), b = weight_if(sc, sh.tab, x[1], over);
      const Weight c = weight_if(sc, sh.tab, x[2], over), d = weight_if(sc, sh.tab, x[3], over);
      sum.add(a, b);
      sum.add(c, d);
      const auto take = [&](const Weight& w, float x, int i) {
        if (static_cast<uint32_t>(w.point - p1) <= static_cast<uint32_t>(p0 - p1)) offer(ph, x, i);
      };
      take(a, x[0], idx);
      take(b, x[1], idx + 1);
      take(c, x[2], idx + 2);
      take(d, x[3], idx + 3);
    });
    const Sums s = exchange(sum.value(), 0);
    const uint32_t all = collect(sh.list[ph], &sh.fill[ph], &cand);
    if (!settle<SUM>(all, s.sum, above, need, cx, ci, upto)) return false;
    list_above = sum.value();
    list_sums = s;
    list_top = below_bin(b0);
    return true;
  }
  // The token with which the running sum reaches `need`, in bin b0 or in bins b0 + 1 .. b1
  // (kSmList tokens at most each): a list of either in one pass, and only the one that the
  // sums say is sorted.
  __device__ __forceinline__ bool cut_either(int b0, int b1, unsigned long long need, float* cx, int* ci, unsigned long long* upto) {
    const int p0 = sc.base - kBinPoints * b0, mid = p0 - kBinPoints, p1 = sc.base - kBinPoints * (b1 + 1) + 1;
    const float low = below_bin(b1 + 1);          // (what lies in these bins does not lie below it)
    if (threadIdx.x < 2) sh.fill_two[threadIdx.x] = 0;
    __syncthreads();
    WeightSum sum;
    unsigned long long first = 0;                 // what bin b0 weighs
    row.quads(row.first, row.count, [&](const float (&x)[4], int idx) {
      if (!__any_sync(0xffffffffu, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= low)) return;
      const auto over = [&](int point) { return point > mid; };
      const Weight a = weight_if(sc, sh.tab, x[0], over), b = weight_if(sc, sh.tab, x[1], over);
      const Weight c = weight_if(sc, sh.tab, x[2], over), d = weight_if(sc, sh.tab, x[3], over);
      sum.add(a, b);
      sum.add(c, d);
      const auto take = [&](const Weight& w, float x, int i) {
        if (static_cast<uint32_t>(w.point - p1) > static_cast<uint32_t>(p0 - p1)) return;
        const bool second = w.point <= mid;
        offer(sh.sort[second], &sh.fill_two[second], x, i);
        if (!second) first += w.value();
      };
      take(a, x[0], idx);
      take(b, x[1], idx + 1);
      take(c, x[2], idx + 2);
      take(d, x[3], idx + 3);
    });
    const Sums in = exchange(first, 0);
    Sums s = exchange(sum.value(), 0);            // of bin b0 and what lies before
    const bool second = need > s.sum;
    list_above = sum.value();
    if (!second) {
      list_above -= first;
      s.sum -= in.sum;
      s.sum_before -= in.sum_before;
    }
    const uint32_t all = collect(sh.sort[second], &sh.fill_two[second], &cand);
    blocks_sync(blocks);                          // (what is sorted overwrites the lists)
    if (!settle<true>(all, s.sum, 0, need, cx, ci, upto)) return false;
    list_sums = s;
    list_top = below_bin(b0 + second);
    return true;
  }
  // A value that all tokens before bin b exceed.
  __device__ __forceinline__ float below_bin(int b) const {
    return b > 0 ? __fsub_rd(sc.top, __fmul_ru(static_cast<float>(kBinPoints * b + 1), 1.0f / (512.0f * sc.ch))) : INFINITY;
  }

  // The bits of x in its own type, ordered as x is, and values from such: that value, and
  // bounds of it that no other value of the type lies within.
  static constexpr int kUnit = TYPE == DSA_FP32 ? 0 : TYPE == DSA_FP16 ? 13 : 16;
  __device__ __forceinline__ static uint32_t unit_key(float x) { return float_key(x) >> kUnit; }
  __device__ __forceinline__ static float unit_low(uint32_t k) { return key_float(k << kUnit); }
  __device__ __forceinline__ static float unit_high(uint32_t k) { return key_float((k << kUnit) | ((1u << kUnit) - 1)); }
  __device__ __forceinline__ static float unit_value(uint32_t k) { return (k << kUnit) & 0x80000000u ? unit_low(k) : unit_high(k); }

  // The cut: the last of the first `need` tokens of the ranking, or the token with which
  // the weights' running sum reaches `need`. Returns the sum of weights up to it.
  //
  // From [lo, hi], values that hold the cut (`few`: at most kSmList of them): exact counts
  // and sums of what lies above hi, and either the tokens themselves or counts of them in
  // bins. The bins are of the bits of x (of those that its type has: with a value a bin, the
  // sums are exact), or, for sums while the weights' logarithms are kGridSpan grid points or
  // more apart, of those: the bounds of the sums are as far apart as the weights within a
  // bin, so every round leaves that part of what the range weighs. Where the cut may still lie
  // at either end (two heavy values with nothing between), the next round's exact sum is
  // that of the upper half: every round leaves half of the bits' range or less.
  template <bool SUM>
  __device__ __forceinline__ unsigned long long cut(unsigned long long need, float lo, float hi, bool few, float* cx, int* ci) {
    listed = false;
    float next_lo = lo, next_hi = hi;             // of a probe: the range if its upper half holds the cut
    bool probe = false;
    // (four rounds from all values, seldom more: 32 halves of 32 bits, and a probe each, at most)
    for (int round = 0; round < 80; ++round) {
      const uint32_t klo = unit_key(lo), khi = unit_key(hi);
      const uint32_t ph = phase & 1;
      if (klo == khi && !few && !probe) break;
      const int ghi = grid_of(sc, hi), span = ghi - grid_of(sc, lo);
      const bool by_grid = SUM && span >= kGridSpan && round < 10;
      int shift = 0;
      while ((by_grid ? static_cast<uint32_t>(span) : khi - klo) >> shift >= kSmBins) ++shift;
      uint32_t* hist = nullptr;
      if (!few) hist = clear_hist();
      if (threadIdx.x == 0) sh.fill[ph] = 0;
      __syncthreads();
      WeightSum above;
      uint32_t n = 0;
      row.pairs(row.first, row.count, [&](float x0, float x1, int idx) {
        const float most = fmaxf(x0, x1);
        if (!__any_sync(0xffffffffu, most >= lo)) return;
        if (__any_sync(0xffffffffu, most > hi)) {
          n += (x0 > hi ? 1u : 0u) + (x1 > hi ? 1u : 0u);
          above.add(weight_if(sc, sh.tab, x0, [&](int) { return x0 > hi; }), weight_if(sc, sh.tab, x1, [&](int) { return x1 > hi; }));
        }
        const bool in0 = x0 >= lo && x0 <= hi, in1 = x1 >= lo && x1 <= hi;
        if (few) {
          if (in0) offer(ph, x0, idx);
          if (in1) offer(ph, x1, idx + 1);
        } else if (by_grid) {
          count(hist, in0 ? (ghi - grid_of(sc, x0)) >> shift : -1, in1 ? (ghi - grid_of(sc, x1)) >> shift : -1);
        } else {
          count(hist, in0 ? static_cast<int>((khi - unit_key(x0)) >> shift) : -1, in1 ? static_cast<int>((khi - unit_key(x1)) >> shift) : -1);
        }
      });
      const Sums s = exchange(above.value(), n);
      if (SUM ? s.sum >= need : s.cnt >= need) {   // (the range does not hold it: the upper half, or from all values)
        if (probe) {
          probe = false;
          lo = next_lo;
          hi = next_hi;
          continue;
        }
        few = false;
        lo = -INFINITY;
        hi = sc.top;
        continue;
      }
      if (few) {
        unsigned long long sum;
        const uint32_t all = collect(sh.list[ph], &sh.fill[ph], &cand);
        if (settle<SUM>(all, s.sum, s.cnt, need, cx, ci, &sum)) {
          list_above = above.value();
          list_sums = s;
          list_top = hi;
          return sum;
        }
        // (not among them: from all values, by counts alone)
        few = false;
        lo = -INFINITY;
        hi = sc.top;
        continue;
      }
      probe = false;
      const uint32_t m = bins(hist);
      const uint32_t top_key = khi - (threadIdx.x << shift);   // of the thread's bin
      if constexpr (SUM) {
        const unsigned long long rest = need - s.sum;
        if (by_grid) {
          // (a grid point to spare on either side)
          const auto w = [&](int g) { return exp2f(static_cast<float>(min(g, 1)) * (1.0f / 512.0f)) * unit(); };
          const int g = ghi - (static_cast<int>(threadIdx.x) << shift), step = 1 << shift;
          find_bounds(m * w(g - step), m * w(g + 1), static_cast<float>(rest));
        } else if (shift == 0) {
          find_sum(m, m ? weight_of(sc, sh.tab, unit_value(top_key)) : 0ull, rest);
        } else {
          const auto w = [&](uint32_t k) { return m ? static_cast<float>(weight_of(sc, sh.tab, unit_value(k))) : 0.f; };
          find_bounds(m * w(max(klo, top_key - ((1u << shift) - 1))), m * w(top_key), static_cast<float>(rest));
        }
      } else {
        find_count(m, static_cast<uint32_t>(need) - s.cnt);
      }
      const int b0 = sh.lo_bin, b1 = sh.hi_bin;
      // how many tokens those bins hold (and, of the grid's, those whose tokens the new range may hold)
      const int more = by_grid ? (3 >> shift) + 1 : 0;
      const uint32_t left = held(m, b0 - more, b1 + more);
      if (by_grid) {
        const float inv = 1.0f / (512.0f * sc.ch);
        const int g0 = ghi - (b0 << shift) + 2, g1 = ghi - ((b1 + 1) << shift) - 2;
        hi = fminf(hi, __fsub_ru(sc.top, __fmul_rd(static_cast<float>(-min(g0, 0)), inv)));
        lo = fmaxf(lo, __fsub_rd(sc.top, __fmul_ru(static_cast<float>(-g1), inv)));
      } else {
        const uint32_t down = ((static_cast<uint32_t>(b1) + 1) << shift) - 1;
        if (b0 > 0) hi = unit_high(khi - (static_cast<uint32_t>(b0) << shift));
        if (down < khi - klo) lo = unit_low(khi - down);
      }
      few = left <= kSmList;
      const uint32_t k0 = unit_key(lo), k1 = unit_key(hi);
      if (SUM && !few && k0 < k1 && k1 - k0 > (khi - klo) / 2) {
        const uint32_t mid = k0 + (k1 - k0) / 2;
        next_lo = unit_low(mid + 1);
        next_hi = hi;
        hi = unit_high(mid);
        probe = true;
      }
    }
    // more tokens of one value than a list holds: the first of them, in index order
    const float v = unit_value(unit_key(lo));
    unsigned long long above = 0;
    uint32_t n = 0, ties = 0;
    row.pairs(row.first, row.count, [&](float x0, float x1, int) {
      if (__any_sync(0xffffffffu, fmaxf(x0, x1) > v)) {
        n += (x0 > v ? 1u : 0u) + (x1 > v ? 1u : 0u);
        above += (x0 > v ? weight_of(sc, sh.tab, x0) : 0ull) + (x1 > v ? weight_of(sc, sh.tab, x1) : 0ull);
      }
      ties += (x0 == v ? 1u : 0u) + (x1 == v ? 1u : 0u);
    });
    const Sums s = exchange(above, n);
    const Sums t = exchange(0, ties);
    const unsigned long long w = weight_of(sc, sh.tab, v);
    unsigned long long take = SUM ? (need - s.sum + w - 1) / max(w, 1ull) : need - s.cnt;
    take = min(max(take, 1ull), static_cast<unsigned long long>(t.cnt));
    if (threadIdx.x == 0) sh.at_index = -1;
    const unsigned long long mine = __reduce_add_sync(0xffffffffu, ties);
    __syncthreads();
    locate(mine, t.cnt_before, take, [&](float x, int) { return x == v ? 1ull : 0ull; });
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

template <int TYPE>
__global__ void __launch_bounds__(kSmThreads) sample_kernel(const __grid_constant__ SampleParams p, int blocks) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(smem_raw);
  uint8_t* img = smem_raw + ((sizeof(SampleShared) + 15) & ~15);
  constexpr bool kF32 = TYPE == DSA_FP32;
  constexpr int kBytes = kF32 ? 4 : 2, kVec = 16 / kBytes;
  Sampler<TYPE> s(p, sh);
  s.blocks = blocks;
  s.rank = blockIdx.x % blocks;
  s.warp = threadIdx.x >> 5;
  s.lane = threadIdx.x & 31;
  const int r = blockIdx.x / blocks;
  // the block's tokens
  const int t0 = s.rank * p.slice, len = max(0, min(p.slice, p.vocab - t0));
  const uint8_t* src = static_cast<const uint8_t*>(p.logits) + (r * p.stride + t0) * kBytes;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / kBytes;
  const int vecs = ((off + len + kVec - 1) / kVec + 31) & ~31, per = (vecs + kSmThreads - 1) / kSmThreads * 32;
  s.row.img = reinterpret_cast<const uint4*>(img);
  s.row.vecs = vecs;
  s.row.per = per;
  s.row.first = min(s.warp * per, vecs);
  s.row.count = min(per, vecs - s.row.first);
  s.row.index0 = t0 - off;
  for (int i = s.lane; i < s.row.count; i += 32) {
    const int v = s.row.first + i, e0 = v * kVec - off;          // the vector's first token, of the block's
    uint8_t* d = img + v * 16;
    if (e0 >= 0 && e0 + kVec <= len) {
      cp_async16(d, src + e0 * kBytes, true);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const bool in = e0 + e >= 0 && e0 + e < len;
        if constexpr (kF32)
          reinterpret_cast<float*>(d)[e] = in ? reinterpret_cast<const float*>(src)[e0 + e] : -INFINITY;
        else
          reinterpret_cast<uint16_t*>(d)[e] = in ? reinterpret_cast<const uint16_t*>(src)[e0 + e] : TYPE == DSA_FP16 ? 0xfc00u : 0xff80u;
      }
    }
  }
  cp_async_commit();
  for (int i = threadIdx.x; i < 512; i += kSmThreads) sh.tab[i] = g_pow2.v[i];
  // the row's settings
  const float heat = p.heat ? __ldg(p.heat + r) : 1.0f;
  const int k = p.top_k ? __ldg(p.top_k + r) : 0;
  const float tp = p.top_p ? __ldg(p.top_p + r) : 1.0f;
  const float mp = p.min_p ? __ldg(p.min_p + r) : 0.0f;
  // (64-bit arithmetic is slow here: one thread's, beside the load)
  const auto pair = [](double v) {
    const float hi = static_cast<float>(v);
    return make_float2(hi, static_cast<float>(v - static_cast<double>(hi)));
  };
  if (threadIdx.x == 0) sh.row_c = pair(fmin(1.4426950408889634074 / static_cast<double>(heat), 0x1p100));
  if (threadIdx.x == 32 && mp > 0.f) sh.row_low = pair(static_cast<double>(heat) * log(static_cast<double>(fminf(mp, 1.0f))));
  const bool by_k = heat > 0.f && k > 0 && k < p.vocab, by_p = heat > 0.f && tp < 1.0f;
  const bool list_k = by_k && k <= kSmFewK, list_p = by_p && !by_k;
  sh.hist[0][threadIdx.x] = sh.hist[1][threadIdx.x] = sh.below[1][threadIdx.x] = 0;
  if (threadIdx.x == 64) sh.lo_bin = sh.hi_bin = -1;
  cp_async_wait<0>();
  // the largest logit
  float own = -INFINITY;
  s.row.each([&](const float (&x)[kVec], int) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) own = fmaxf(own, x[e]);        // (NaN: passed over)
  });
  float top = warp_max(own);
  if (s.lane == 0) sh.warp_bound[s.warp] = top;
  __syncthreads();
  top = warp_max(sh.warp_bound[s.lane]);
  // and a value that enough tokens reach for a list: the threads' largest ones, counted
  // in bins 1 / 16 of log2 of the weight wide below the block's. Enough is the block's share
  // (low; infinity: it is short of it, as where it is masked), or all, where others are short.
  const uint32_t enough = list_k ? k : kSmFewP;
  const auto edge = [&](float t, int bin) { return __fsub_rd(t, __fmul_ru(static_cast<float>(bin) + 1.01f, 1.0f / (16.0f * sh.row_c.x))); };
  float low = INFINITY;
  if (list_k || list_p) {
    const float ch = 16.0f * sh.row_c.x;
    const float b = fminf((top - own) * ch, static_cast<float>(kSmBins - 1));       // (NaN: no bin)
    if (b < kSmBins - 1) atomicAdd(&sh.hist[0][static_cast<int>(b)], 1u);
    __syncthreads();
    s.find_count(sh.hist[0][threadIdx.x], (enough + blocks - 1) / blocks, enough);
    if (sh.lo_bin >= 0) low = edge(top, sh.lo_bin);
  }
  const uint32_t ph = s.phase++ & 1;
  if (threadIdx.x == 0) {
    sh.top[ph] = top;
    sh.low[ph] = low;
    sh.cnt[ph] = sh.hi_bin;                                       // (a word that this exchange has no other use for)
  }
  if (threadIdx.x == 32) sh.fill[1] = 0;
  blocks_sync(blocks);
  const bool peer = static_cast<uint32_t>(s.lane) < s.blocks;
  const float top_there = peer ? peer_load(&sh.top[ph], s.lane) : -INFINITY;
  top = warp_max(top_there);
  if (list_k || list_p) {
    low = peer ? peer_load(&sh.low[ph], s.lane) : INFINITY;
    const uint32_t able = __popc(__ballot_sync(0xffffffffu, low < INFINITY));
    low = -warp_max(-low);
    // With blocks that are short of their share the others' are too few together: then what one of
    // them has enough of by itself, where the list holds as many of each. (64 x 131,072 with half of
    // every row masked, top-k 50 and top-p: 17 us, and 46 with all tokens offered to the list.)
    if (able < s.blocks) {
      const int bin = peer ? static_cast<int>(peer_load(&sh.cnt[ph], s.lane)) : -1;
      const float alone = warp_max(bin >= 0 ? edge(top_there, bin) : -INFINITY);
      low = able * enough <= kSmList && alone > -INFINITY ? alone : list_k ? INFINITY : low;
    }
    if (low == INFINITY) low = -INFINITY;                         // (no block has its share: all tokens)
  }

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
  sc.top = top;
  sc.ch = sh.row_c.x;
  sc.cl = sh.row_c.y;
  sc.b = fabsf(top) * sc.ch < 4096.0f ? 0.f : top;
  const float d_top = top - sc.b, p_top = __fmul_rn(d_top, sc.ch), t_top = __fadd_rn(p_top, kGrid);
  sc.base = __float_as_int(t_top);
  sc.rest = (p_top - (t_top - kGrid)) + fmaf(d_top, sc.cl, fmaf(d_top, sc.ch, -p_top));   // within kRest / 512 of 0
  sc.floor = (t_top - kGrid) - 80.0f;
  sc.zero = sc.base - kZero;
  // (the largest's power is 2^-1: sums of 2^19 weights below 2^45 stay below 2^64)
  sc.power = (126u << 23) - __float_as_uint(__fadd_rd(t_top - kGrid, kInt)) * 0x800000u;
  // a cutoff that does not depend on the others: the least x >= max + T ln min_p
  float least = -INFINITY;
  if (!greedy && mp > 0.f) {
    const float2 v = sh.row_low;
    const float a = __fadd_rn(top, v.x), b = __fsub_rn(a, top);
    const float e = __fadd_rn(__fadd_rn(__fsub_rn(top, __fsub_rn(a, b)), __fsub_rn(v.x, b)), v.y);   // what a is short of
    // (where max and T ln min_p nearly cancel, e is many steps of a. NaN: T ln min_p is infinite)
    least = e == e ? __fadd_ru(a, e) : a;
  }
  float u = __ldg(p.u + r);
  u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
  const auto fraction = [](float v) {                              // v 2^64, 0 <= v < 1
    const uint32_t bits = __float_as_uint(v);
    const int e = static_cast<int>(bits >> 23) - 86;               // v = mantissa 2^(e + 86 - 150)
    const unsigned long long m = (bits & 0x7fffffu) | 0x800000u;
    return e <= -24 ? 0ull : e < 0 ? m >> -e : m << e;
  };
  const auto drawn = [&](unsigned long long sum) { return __umul64hi(fraction(u), sum) + 1; };   // the running sum that the token reaches
  const auto answer = [&](int token, float x, unsigned long long w, unsigned long long sum) {
    p.tokens[r] = token;
    if (!p.logprobs) return;
    float lp = 0.f;
    if (!greedy) {
      const unsigned long long rest = sum - w;
      if (rest < w) {
        lp = log1pf(-(static_cast<float>(rest) / static_cast<float>(sum)));
      } else {
        lp = (x - top) / heat + sc.rest * 0.69314718f - logf(static_cast<float>(sum) / s.unit());
      }
    }
    p.logprobs[r] = lp;
  };
  // the least sum that is top-p's share of `sum`, rounded up
  const auto share = [&](unsigned long long sum) {
    const unsigned long long f = tp > 0.f ? fraction(tp) : 0ull;
    return max(__umul64hi(f, sum) + (f * sum != 0 ? 1 : 0), 1ull);
  };

  float cx = -INFINITY;                                           // the cut: nothing yet
  int ci = 0x7fffffff;
  unsigned long long total = 0;
  bool counted = false;
  if (greedy || list_k || list_p) {
    // what reaches `low` (greedy: the largest), in a list; with top-p alone, the sum of all
    // weights and the counts too
    if (greedy) low = top;
    const uint32_t lp = s.phase & 1;
    counted = list_p && !greedy;
    WeightSum sum;
    if (counted)
      s.row.quads(s.row.first, s.row.count, [&](const float (&x)[4], int) {
        const auto all = [](int) { return true; };
        const Weight a = weight_if(sc, sh.tab, x[0], all), b = weight_if(sc, sh.tab, x[1], all);
        const Weight c = weight_if(sc, sh.tab, x[2], all), d = weight_if(sc, sh.tab, x[3], all);
        sum.add(a, b);
        sum.add(c, d);
        s.count_weights(sh.hist[lp], sh.below[lp], a, b);
        s.count_weights(sh.hist[lp], sh.below[lp], c, d);
      });
    s.row.each([&](const float (&x)[kVec], int idx) {
      float most = x[0];
#pragma unroll
      for (int e = 1; e < kVec; ++e) most = fmaxf(most, x[e]);
      if (!(most >= low) || most == -INFINITY) return;
      // (all tokens: once they are too many for the list, no more of them queue up to be counted)
      if (low == -INFINITY && *reinterpret_cast<const volatile uint32_t*>(&sh.fill[lp]) > kSmList) return;
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (x[e] >= low && x[e] > -INFINITY) s.offer(lp, x[e], idx + e);
    });
    total = s.exchange(sum.value(), 0).sum;
    const uint32_t n = s.collect(sh.list[lp], &sh.fill[lp], &s.cand);
    bool fits = n <= kSmList;
    if (greedy && fits) {
      if (threadIdx.x == 0) sh.at_index = 0x7fffffff;
      __syncthreads();
      if (s.cand) atomicMin(&sh.at_index, s.index_of(s.cand));
      __syncthreads();
      if (s.rank == 0 && threadIdx.x == 0) answer(sh.at_index, top, 1, 1);
      blocks_sync(blocks);
      return;
    }
    fits = fits && !greedy && (!list_k || n >= k || low == -INFINITY);
    if (fits && list_p)                                           // (the list has to weigh enough)
      fits = s.block_add(s.cand ? weight_of(sc, sh.tab, s.value_of(s.cand)) : 0ull) >= share(total);
    if (fits) {
      s.cand = s.sorted(s.cand, n);
      const bool in = threadIdx.x < n;
      if (!in) s.cand = 0;
      const unsigned long long w = in ? weight_of(sc, sh.tab, s.value_of(s.cand)) : 0ull;
      const unsigned long long before = s.template scan<unsigned long long>(w, sh.warp_sum);
      // the last token that is kept: of the first k, the one that reaches top-p's share
      const uint32_t last = list_k ? min(static_cast<uint32_t>(k), n) - 1 : n - 1;
      if (threadIdx.x == last) sh.at_sum = before + w;
      if (threadIdx.x == 0) sh.at_index = -1;
      __syncthreads();
      const unsigned long long of = list_k ? sh.at_sum : total, need = by_p ? share(of) : of;
      if (by_p ? in && before < need && need <= before + w : threadIdx.x == last) {
        sh.at_index = s.index_of(s.cand);
        sh.at_x = s.value_of(s.cand);
      }
      __syncthreads();
      if (sh.at_index >= 0) {
        cx = sh.at_x;
        ci = sh.at_index;
        s.listed = true;
        s.list_above = 0;
        s.list_sums = Sums{0, 0, 0, 0};
        s.list_top = INFINITY;
      }
      __syncthreads();
    }
  }
  if (s.listed) {
  } else if (greedy) {
    s.template cut<false>(1, top, top, false, &cx, &ci);          // (more of the largest than a list holds)
  } else if (by_k || by_p) {
    // counts by the weights (and of all tokens that may be taken)
    uint32_t ph2 = 1, finite = 0;
    if (!counted) {
      ph2 = s.phase & 1;
      sh.below[ph2][threadIdx.x] = 0;
      uint32_t* hist = s.clear_hist();
      s.row.pairs(s.row.first, s.row.count, [&](float x0, float x1, int) {
        const auto all = [](int) { return true; };
        s.count_weights(hist, sh.below[ph2], weight_if(sc, sh.tab, x0, all), weight_if(sc, sh.tab, x1, all));
        finite += (x0 > -INFINITY ? 1u : 0u) + (x1 > -INFINITY ? 1u : 0u);
      });
      finite = s.exchange(0, finite).cnt;
    }
    const uint32_t n = s.bins(sh.hist[ph2]);
    const float inv_c = 1.0f / sc.ch;
    // values that surely hold all of bins b0 .. b1 (two grid points more on either side), and
    // whether a list holds these bins' tokens and their neighbours'. The last bin stands for all
    // that weighs less than the others' tokens, down to nothing: it has no lower end.
    const auto range = [&](int b0, int b1, float* lo, float* hi) {
      const uint32_t left = s.held(n, b0 - 1, b1 + 1);
      *hi = b0 <= 0 ? top : fminf(top, __fsub_ru(top, __fmul_rd(static_cast<float>(kBinPoints * b0 - 2) * (1.0f / 512.0f), inv_c)));
      *lo = b1 >= kSmBins - 1 ? -INFINITY : __fsub_rd(top, __fmul_ru(static_cast<float>(kBinPoints * (b1 + 1) + 2) * (1.0f / 512.0f), inv_c));
      return left <= kSmList && b1 + 1 < kSmBins - 1;
    };
    float lo, hi;
    bool cut_k = false;
    if (by_k && static_cast<uint32_t>(k) < finite) {
      if (threadIdx.x == 0) sh.lo_bin = -1;
      __syncthreads();
      s.find_count(n, k);
      const int b = sh.lo_bin;
      __syncthreads();
      if (b < 0) {                                                // (below the last bin)
        total = s.template cut<false>(k, -3.402823466e38f, top, false, &cx, &ci);
      } else if (s.held(n, b, b) > kSmList || !s.template cut_bins<false>(b, b, s.held(n, 0, b - 1), k, &cx, &ci, &total)) {
        const bool few = range(b, b, &lo, &hi);
        total = s.template cut<false>(k, lo, hi, few, &cx, &ci);
      }
      cut_k = true;
    } else if (by_k && by_p) {                                    // (k leaves everything)
      WeightSum sum;
      s.row.pairs(s.row.first, s.row.count, [&](float x0, float x1, int) {
        const auto all = [](int) { return true; };
        sum.add(weight_if(sc, sh.tab, x0, all), weight_if(sc, sh.tab, x1, all));
      });
      total = s.exchange(sum.value(), 0).sum;
    }
    if (by_p) {
      // A bin's n tokens lie m grid points below its edge on average, each between -kRest and
      // 15 + kRest (a sum's rounding is a 128th of a point a token). 2^-x is convex:
      // they weigh at least n times the weight at their mean, at most what the chord
      // between the ends gives.
      const unsigned long long need = share(total);
      const float m = n ? (static_cast<float>(s.bins(sh.below[ph2])) / static_cast<float>(n) - s.kBelow) * (1.0f / 64.0f) : 0.f;
      const float edge = -static_cast<float>(kBinPoints * static_cast<int>(threadIdx.x));
      const auto w = [&](float g) { return exp2f(g * (1.0f / 512.0f)) * s.unit(); };
      constexpr float kEnd = kBinPoints - 1 + kRest;
      const float w0 = w(edge + kRest), w1 = w(edge - kEnd);
      s.find_bounds(n * w(edge - m - 0.02f), n * (w0 + (m - 0.02f + kRest) * (1.0f / (kEnd + kRest)) * (w1 - w0)), static_cast<float>(need));
      const int b0 = sh.lo_bin, b1 = sh.hi_bin;
      __syncthreads();
      // one list of these bins, or (they are two, seldom more) one of the first and one of the rest
      bool found = false;
      if (b1 < kSmBins - 1) {
        const uint32_t all = s.held(n, b0, b1), one = s.held(n, b0, b0);
        if (all <= kSmList) found = s.template cut_bins<true>(b0, b1, 0, need, &cx, &ci, &total);
        else if (one <= kSmList && all - one <= kSmList) found = s.cut_either(b0, b1, need, &cx, &ci, &total);
      }
      if (!found) {
        const bool few = range(b0, b1, &lo, &hi);
        if (cut_k) {                                              // (the cut there is ends the range)
          lo = fmaxf(lo, cx);
          hi = fmaxf(hi, cx);
        }
        total = s.template cut<true>(need, lo, hi, few, &cx, &ci);
      }
    }
  }
  if (least > cx) {
    cx = least;
    ci = 0x7fffffff;
  }
  // the draw: the first token in index order at which the kept weights' sum exceeds u of all
  const auto kept = [&](float x, int idx) { return x > cx || (x == cx && idx <= ci); };
  const auto term = [&](float x, int idx) -> unsigned long long {
    return !kept(x, idx) ? 0ull : greedy ? 1ull : weight_of(sc, sh.tab, x);
  };
  unsigned long long mine, before, sum;
  if (s.listed && least <= s.list_top) {
    // all that is kept lies above the list, or in it
    const bool in = s.cand != 0;
    const float x = s.value_of(s.cand);
    const int idx = s.index_of(s.cand), owner = in ? idx / p.slice : 0;
    const unsigned long long w = in ? term(x, idx) : 0ull;
    if (threadIdx.x < kSmWarps) sh.cand_sum[threadIdx.x] = 0;
    __syncthreads();
    if (w && owner == static_cast<int>(s.rank)) atomicAdd(&sh.cand_sum[(idx - s.row.index0) / kVec / per], w);
    before = s.list_sums.sum_before + s.block_add(owner < static_cast<int>(s.rank) ? w : 0ull);
    sum = s.list_sums.sum + s.block_add(w);
    mine = warp_add(s.list_above) + sh.cand_sum[s.warp];
  } else {
    unsigned long long own_sum = 0;
    if (greedy) {
      s.row.pairs(s.row.first, s.row.count, [&](float x0, float x1, int idx) { own_sum += (kept(x0, idx) ? 1ull : 0ull) + (kept(x1, idx + 1) ? 1ull : 0ull); });
    } else if (cx == -INFINITY) {                                 // (a temperature alone: one pass)
      WeightSum w;
      s.row.each([&](const float (&x)[kVec], int) {
        const auto all = [](int) { return true; };
#pragma unroll
        for (int e = 0; e < kVec; e += 2) w.add(weight_if(sc, sh.tab, x[e], all), weight_if(sc, sh.tab, x[e + 1], all));
      });
      own_sum = w.value();
    } else {
      WeightSum w;
      const bool whole = ci == 0x7fffffff;                        // (no tie is cut)
      s.row.pairs(s.row.first, s.row.count, [&](float x0, float x1, int idx) {
        if (!__any_sync(0xffffffffu, fmaxf(x0, x1) >= cx)) return;
        bool in0 = x0 >= cx, in1 = x1 >= cx;
        if (!whole) {
          in0 = kept(x0, idx);
          in1 = kept(x1, idx + 1);
        }
        w.add(weight_if(sc, sh.tab, x0, [&](int) { return in0; }), weight_if(sc, sh.tab, x1, [&](int) { return in1; }));
      });
      own_sum = w.value();
    }
    const Sums all = s.exchange(own_sum, 0);
    mine = warp_add(own_sum);
    before = all.sum_before;
    sum = all.sum;
  }
  blocks_leave(blocks);
  if (threadIdx.x == 0) sh.at_index = -1;
  __syncthreads();
  s.locate(mine, before, greedy ? 1ull : drawn(sum), term);
  __syncthreads();
  if (threadIdx.x == 0 && sh.at_index >= 0) answer(sh.at_index, sh.at_x, sh.at_sum, sum);   // (one block has it)
  blocks_left(blocks);
}

constexpr size_t sample_smem(size_t data) { return ((sizeof(SampleShared) + 15) & ~size_t{15}) + data + 16 + 512; }
static_assert(sample_smem(kSmMaxData) <= 232448, "");

struct SampleConfig {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  SampleConfig(int rows, int blocks, size_t data, cudaStream_t st) {
    cfg.gridDim = dim3(static_cast<unsigned>(rows) * blocks);
    cfg.blockDim = dim3(kSmThreads);
    cfg.dynamicSmemBytes = sample_smem(data);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

// Clusters of `blocks` (8 at most) that the current device holds at once: not as many as
// its SMs would be enough for, since a cluster lies within one of their groups. (A block
// takes an SM, whatever the shared memory.)
template <int TYPE>
int sample_clusters(int blocks) {
  static KeptAnswers<64 * 9> kept;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  return kept.get(dev * 9 + blocks, [&](int* n) {
    const SampleConfig c(1, blocks, kSmMaxData, nullptr);
    if (cudaOccupancyMaxActiveClusters(n, sample_kernel<TYPE>, &c.cfg) == cudaSuccess) return true;
    cudaGetLastError();                           // (this query's own)
    return false;
  });
}

template <int TYPE>
cudaError_t launch_sample(SampleParams p, cudaStream_t st) {
  constexpr int kBytes = TYPE == DSA_FP32 ? 4 : 2;
  // (the largest size whatever the call's: another thread may be between this and its launch)
  const void* fn = reinterpret_cast<const void*>(&sample_kernel<TYPE>);
  cudaError_t e = set_max_smem(fn, static_cast<int>(sample_smem(kSmMaxData)));
  if (e != cudaSuccess) return e;
  // Blocks of a row: as few as hold it, and up to 8 while the rows' clusters all fit on the
  // chip at once and a block has 6,500 tokens. (Top-p: one row of 128,000 52 / 42 / 37 / 33 /
  // 32 us with 2, 3, 4, 6, 8; 32,000 in top-k 13.2 / 12.8 / 13.7 with 1, 4, 7; 37 of 50,257
  // 46 / 36 / 32 and, in turns, 40 / 66 with 1, 2, 3 and 4, 8; 20 of 131,072 57 / 41 / 38 and
  // 59 with 2, 4, 6 and 7.)
  int blocks = 1;
  const auto slice_of = [&](int n) { return ((p.vocab + n - 1) / n + 63) / 64 * 64; };
  while (blocks < kSmMaxCluster && slice_of(blocks) * kBytes > kSmMaxData) ++blocks;
  while (blocks < 8 && slice_of(blocks + 1) >= 6500 && p.rows <= sample_clusters<TYPE>(blocks + 1)) ++blocks;
  p.slice = slice_of(blocks);
  if (blocks > 8 && (e = set_nonportable_cluster(fn)) != cudaSuccess) return e;
  const SampleConfig c(p.rows, blocks, static_cast<size_t>(p.slice) * kBytes, st);
  e = cudaLaunchKernelEx(&c.cfg, sample_kernel<TYPE>, p, blocks);
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = sp->logits_dtype == DSA_FP32   ? launch_sample<DSA_FP32>(p, st)
                        : sp->logits_dtype == DSA_FP16 ? launch_sample<DSA_FP16>(p, st)
                                                       : launch_sample<DSA_BF16>(p, st);
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "sample launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}
