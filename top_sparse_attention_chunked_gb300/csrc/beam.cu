// Beam search's selection: the `select` best of score_i + log_softmax(logits_i)
// over beams x vocabulary, per batch entry.
//
// Two launches. beam_scan_kernel reads every logit once: a thread block takes
// a slice of one row and keeps, side by side, the slice's maximum and sum of
// exponentials (one online state per thread, joined at the end) and its
// `select` largest logits. Only values above the smallest of those so far are
// looked at: after the first tile that is one comparison per 16 bytes, and the
// few that pass are appended to a list that the block sorts into its best ones
// when it fills. Within a row totals are ordered as the logits are, so a row's
// candidates are its `select` largest logits, lower tokens first.
// beam_merge_kernel joins the slices' sums of each row in 64 bits, forms the
// candidates' totals in 64 bits (rows have different offsets: totals may lie
// closer together than fp32 tells apart) and sorts out the best.
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
constexpr int kVecs = 2;            // 16-byte vectors a thread takes per tile
constexpr int kDrain = 192;         // list entries that trigger a sort
constexpr int kMaxCands = 8192;     // candidates of one batch entry (all rows and slices)
constexpr int kMergeList = DSA_MAX_SELECT * (kMaxCands / kBmThreads);   // a thread's run, for each of `select` threads

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
  SliceSum* sums;     // [rows, slices]
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
  long long stride;   // elements between rows
  long long slice_vecs;
  int batch, beams, vocab, select, slices, pad;
};

__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(x) for x <= 0: log2(e) in two parts, so that its own rounding does not
// bias the sum (one part: 1.3e-8 of x, the same sign for every term)
__device__ __forceinline__ float exp_neg(float x) {
  return ex2_ftz(fmaf(x, 1.44269502e0f, x * 1.92596303e-8f));
}

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

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

// Sorts one key per thread over the block, largest in thread 0 (bitonic; the
// exchanges beyond a warp go through `buf`, kBmThreads keys).
template <typename K>
__device__ __forceinline__ K block_sort(K key, K* buf) {
  const int t = threadIdx.x;
#pragma unroll 1
  for (int size = 2; size <= kBmThreads; size <<= 1) {
    const bool down = (t & size) == 0;   // this run sorts largest first
#pragma unroll 1
    for (int m = size >> 1; m > 0; m >>= 1) {
      K other;
      if (m >= 32) {
        __syncthreads();
        buf[t] = key;
        __syncthreads();
        other = buf[t ^ m];
      } else {
        other = shfl_xor(key, m);
      }
      const bool first = (t & m) == 0;
      const bool take_max = first == down;
      if (above(other, key) == take_max) key = other;
    }
  }
  __syncthreads();
  return key;
}

// Sorts the best `k` of top[0..k) and list[0..n) into top, largest first.
// `none` fills places that have no key.
template <typename K>
__device__ void drain(K* top, const K* list, int n, int k, K none, K* buf) {
  const int t = threadIdx.x;
  for (int at = 0; at < n; at += kBmThreads - k) {
    const int i = at + t - k;
    K key = t < k ? top[t] : (i < n ? list[i] : none);
    key = block_sort(key, buf);
    if (t < k) top[t] = key;
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kBmThreads) beam_scan_kernel(const BeamParams p) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int kTileVecs = kBmThreads * kVecs;
  constexpr int kList = kTileVecs * VE + kDrain;
  __shared__ unsigned long long s_list[kList];
  __shared__ unsigned long long s_top[DSA_MAX_SELECT];
  __shared__ unsigned long long s_buf[kBmThreads];
  __shared__ int s_count;
  __shared__ double s_sum[kBmThreads / 32];
  __shared__ float s_max[kBmThreads / 32];
  const int row = blockIdx.y, slice = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  pdl_trigger();
  if (p.finished && p.finished[row]) return;   // the merge knows its one continuation
  const T* x0 = static_cast<const T*>(p.logits) + static_cast<long long>(row) * p.stride;
  // 16-byte vectors from the aligned address at or before the row's first element
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
  const long long nvec = (static_cast<long long>(p.vocab) + mis + VE - 1) / VE;
  const long long v_begin = slice * p.slice_vecs;
  const long long v_end = min(nvec, v_begin + p.slice_vecs);
  const int k = p.select;

  const auto load = [&](long long v, T* out) {
    const long long e0 = v * VE - mis;
    if (v < v_end && e0 >= 0 && e0 + VE <= p.vocab) {
      *reinterpret_cast<uint4*>(out) = __ldcs(reinterpret_cast<const uint4*>(x0 + e0));
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const bool in = v < v_end && e0 + e >= 0 && e0 + e < p.vocab;
        out[e] = in ? x0[e0 + e] : T(-INFINITY);
      }
    }
  };

  if (tid < DSA_MAX_SELECT) s_top[tid] = 0ull;
  if (tid == 0) s_count = 0;
  float m = -INFINITY, sum = 0.0f;   // this thread's maximum and sum of exp(x - m)
  float thr = -INFINITY;             // values at or below it cannot be among the best
  alignas(16) T cur[kVecs][VE];
  alignas(16) T nxt[kVecs][VE];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) load(v_begin + i * kBmThreads + tid, cur[i]);
  __syncthreads();
  for (long long v0 = v_begin; v0 < v_end; v0 += kTileVecs) {
    if (v0 + kTileVecs < v_end) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) load(v0 + kTileVecs + i * kBmThreads + tid, nxt[i]);
    }
    float x[kVecs][VE], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        x[i][e] = to_float(cur[i][e]);
        top = fmaxf(top, x[i][e]);
      }
    if (top > m) {
      sum *= exp_neg(m - top);   // the first time: 0 * exp(-inf)
      m = top;
    }
    if (m > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) sum += exp_neg(x[i][e] - m);
    } else {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (x[i][e] != x[i][e]) sum = x[i][e];   // NaN among masked tokens
    }
    if (v0 == v_begin && k < kBmThreads) {
      // the first threshold: `select` threads hold a value of at least the
      // select-th largest of the threads' maxima
      const unsigned long long key =
          block_sort(top > -INFINITY ? cand_key(top, 0) : 0ull, s_buf);
      if (tid == k - 1) s_buf[0] = key;
      __syncthreads();
      const uint32_t u = static_cast<uint32_t>(s_buf[0] >> 32);
      // the next smaller value (below +0 the keys go on at the largest negative
      // one: 0x7fffffff would be -0, which is not smaller)
      if (u != 0u) thr = key_value(static_cast<unsigned long long>(u == 0x80000000u ? u - 2u : u - 1u) << 32);
      __syncthreads();
    }
    // append what is above the threshold
    uint32_t hits = 0;
    if (top > thr) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (x[i][e] > thr) hits |= 1u << (i * VE + e);
    }
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
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (hits & (1u << (i * VE + e)))
            s_list[at++] = cand_key(x[i][e], static_cast<int>((v0 + i * kBmThreads + tid) * VE - mis + e));
    }
    __syncthreads();
    const int n = s_count;
    __syncthreads();
    if (n >= kDrain || v0 + kTileVecs >= v_end) {
      drain(s_top, s_list, n, k, 0ull, s_buf);
      if (tid == 0) s_count = 0;
      // what comes later in the row has higher tokens: equal is not enough
      if (s_top[k - 1] != 0ull) thr = key_value(s_top[k - 1]);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) *reinterpret_cast<uint4*>(cur[i]) = *reinterpret_cast<const uint4*>(nxt[i]);
  }
  // join the threads' sums
  float mm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  if (lane == 0) s_max[wid] = mm;
  __syncthreads();
  mm = s_max[0];
#pragma unroll
  for (int i = 1; i < kBmThreads / 32; ++i) mm = fmaxf(mm, s_max[i]);
  // (a thread that saw nothing but -infinity adds its 0, or its NaN)
  double d = static_cast<double>(m > -INFINITY ? sum * exp_neg(m - mm) : sum);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) s_sum[wid] = d;
  __syncthreads();
  const long long at = static_cast<long long>(row) * p.slices + slice;
  if (tid == 0) {
    d = 0.0;
    for (int i = 0; i < kBmThreads / 32; ++i) d += s_sum[i];
    p.sums[at] = SliceSum{d, mm};
  }
  if (tid < k) {
    const unsigned long long key = s_top[tid];
    p.cands[at * k + tid] = key ? Cand{key_value(key), static_cast<int32_t>(~static_cast<uint32_t>(key))} : Cand{0.0f, -1};
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
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int row0 = blockIdx.x * p.beams;
  const int k = p.select;
  const Total none{0ull, 0u};
  if (tid == 0) s_count = 0;
  if (tid < DSA_MAX_SELECT) s_top[tid] = none;
  pdl_wait();
  if (blockIdx.x == 0 && tid == 0) *p.status = 0u;
  for (int b = wid; b < p.beams; b += kBmThreads / 32) {
    const int row = row0 + b;
    if (p.finished && p.finished[row]) continue;
    const SliceSum* s = p.sums + static_cast<long long>(row) * p.slices;
    float mm = -INFINITY;
    for (int i = lane; i < p.slices; i += 32) mm = fmaxf(mm, s[i].max);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    double d = 0.0;
    for (int i = lane; i < p.slices; i += 32) {
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
    if (p.finished && p.finished[row]) {
      if (j > 0) return none;
      t = p.scores[row];
      token = p.pad;
    } else {
      const Cand c = p.cands[static_cast<long long>(row) * per_row + j];
      if (c.token < 0) return none;
      t = static_cast<double>(c.value) + s_off[b];
      token = c.token;
    }
    if (!(t > -INFINITY)) return none;   // -infinity or NaN
    return Total{double_key(t), ~static_cast<uint32_t>(b * p.vocab + token)};
  };
  Total best = none;
  for (int i = tid; i < n; i += kBmThreads) {
    const Total t = total(i);
    if (above(t, best)) best = t;
  }
  // `select` threads hold one at or above the select-th of the threads' best
  best = block_sort(best, s_buf);
  if (tid == k - 1) s_buf[0] = best;
  __syncthreads();
  const Total thr = s_buf[0];
  for (int i = tid; i < n; i += kBmThreads) {
    const Total t = total(i);
    if (t.hi != 0ull && !above(thr, t)) {
      const int at = atomicAdd(&s_count, 1);
      s_list[at] = t;
    }
  }
  __syncthreads();
  drain(s_top, s_list, s_count, k, none, s_buf);
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

// Slices a row may be cut into: its candidates stay within kMaxCands per batch
// entry, and a slice is worth a thread block from 1,024 vectors on.
int max_slices(const dsa_beam_problem* p) {
  const int ve = p->logits_dtype == DSA_FP32 ? 4 : 8;
  const long long vecs = (p->vocab + 2LL * ve - 2) / ve;
  const long long by_len = std::max<long long>(1, vecs / 1024);
  const long long by_cands = std::max(1, kMaxCands / (p->beams * p->select));
  return static_cast<int>(std::min<long long>({by_len, by_cands, 64}));
}

size_t beam_bytes(const dsa_beam_problem* p, size_t* sums_at) {
  const size_t n = static_cast<size_t>(p->batch) * p->beams * max_slices(p);
  const size_t c = 256 + up(n * p->select * sizeof(Cand));
  if (sums_at) *sums_at = c;
  return c + up(n * sizeof(SliceSum));
}

template <typename T>
cudaError_t launch_scan(const BeamParams& p, cudaStream_t s) {
  return launch_kernel("beam_scan_kernel", beam_scan_kernel<T>, dim3(p.slices, p.batch * p.beams), dim3(kBmThreads),
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
  const int ve = bp->logits_dtype == DSA_FP32 ? 4 : 8;
  const long long vecs = (bp->vocab + 2LL * ve - 2) / ve;   // whatever the row's alignment
  const long long rows = static_cast<long long>(bp->batch) * bp->beams;
  const long long want = std::max<long long>(1, (6LL * sms + rows - 1) / rows);
  p.slices = static_cast<int>(std::min<long long>(want, max_slices(bp)));
  p.slice_vecs = (vecs + p.slices - 1) / p.slices;
  cudaError_t e = bp->logits_dtype == DSA_FP32   ? launch_scan<float>(p, s)
                  : bp->logits_dtype == DSA_FP16 ? launch_scan<__half>(p, s)
                                                 : launch_scan<__nv_bfloat16>(p, s);
  if (e == cudaSuccess)
    e = launch_kernel("beam_merge_kernel", beam_merge_kernel, dim3(bp->batch), dim3(kBmThreads), 0, s, true, p);
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "beam_select launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}
