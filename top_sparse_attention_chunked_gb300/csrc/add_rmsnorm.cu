// The work between two layers in one pass: h = x + residual (rounded to the
// type of x, stored, and what is normalised), y = h * gamma / sqrt(mean(h^2) +
// eps) in fp32, stored in 16 bits or as 8-bit values with a scale per row or
// per 128 elements: scale = absmax(y) / top, code = y / scale rounded to nearest
// (e4m3: top 448; INT8: top 127).
//
// A row stays in registers from its load to its store, so every byte passes
// once; rows are spread over thread blocks, or over warps where they are short.
// The mean needs the whole row before the first element can leave: the loads of one
// block run under the arithmetic of the others on its SM.
//
// What bounds it: memory. 8,192 x 8,192 BF16, of the copy rate: BF16 out 83 us (96%), e4m3
// with a scale a row 79 us (88%), a scale per 128 elements 83 us (84%; the maxima's
// exchanges and the conversions keep the schedulers 72% busy); 4,096 x 4,096 25 us. Rows
// that cannot be moved as vectors (4,000 x 4,001): 56 us, issue-bound. Small calls: a
// launch and a row's way, 2.4 us for 8 x 5,120.
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kNormGroup = 128;                 // elements that share a scale
constexpr int kNormMaxWarps = 32;
constexpr int kNormMaxHidden = 32768;           // 32 elements a thread of a block of 1,024

struct NormParams {
  const void* x;
  const void* r;       // or nullptr
  const float* gamma;
  void* h;             // or nullptr
  void* y;
  float* scale;        // [rows, groups] (8 bits only)
  long long rows, xs, rs, hs, ys;               // elements from row to row
  int hidden, x_dtype, y_dtype, groups;         // groups: scales of a row
  float eps, inv_hidden;
};

__device__ __forceinline__ float from16(uint32_t u, bool f16) {   // low 16 bits
  return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(u))) : __uint_as_float(u << 16);
}
__device__ __forceinline__ uint32_t to16(float v, bool f16) {
  return f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// A step's elements as they lie in memory, all loads of a row before the first use (the
// stores of h may alias what is still to be read, as far as the compiler knows): eight
// consecutive ones (VEC), or four single ones.
template <bool F32, bool VEC>
struct Raw {
  uint32_t w[VEC ? (F32 ? 8 : 4) : (F32 ? 4 : 2)];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& x : w) x = 0;
  }
  __device__ __forceinline__ void load8(const void* base, long long i) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (F32 ? 4 : 2));
    const uint4 a = __ldcs(s);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    if constexpr (F32) {
      const uint4 b = __ldcs(s + 1);
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
  }
  __device__ __forceinline__ void load1(const void* base, long long i, int e) {
    if constexpr (F32) w[e] = static_cast<const uint32_t*>(base)[i];
    else w[e >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << (16 * (e & 1));
  }
  __device__ __forceinline__ float get(int e, bool f16) const {
    if constexpr (F32) return __uint_as_float(w[e]);
    return from16((w[e >> 1] >> (16 * (e & 1))) & 0xffffu, f16);
  }
};
__device__ __forceinline__ uint4 pack8(const float* v, bool f16) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = to16(v[2 * e], f16) | to16(v[2 * e + 1], f16) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint32_t code_pair(float a, float b, bool int8) {   // two codes, in 16 bits
  if (int8) {
    return (static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(a, -127.0f), 127.0f))) & 0xffu) |
           (static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(b, -127.0f), 127.0f))) & 0xffu) << 8;
  }
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Sum, or maximum, over the threads of a row: a warp's lanes, or a block's
// (slot: 0 or 1, so that one barrier an exchange is enough).
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int warps, float (*part)[kNormMaxWarps], int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[slot][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? part[slot][lane] : 0.f;    // (maxima are of absolute values)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  return v;
}

// Blocks an SM that the compiler is held to (0: it chooses). FP32 rows by single elements in blocks
// of 1,024 hold 32 elements of x, the residual and the sum each: left to itself it takes 32
// registers a thread, for two blocks an SM, and 1,360 bytes of the stack; with the 64 that one
// block may have 424 (4,000 x 32,767 1,061 -> 689 us, 4,000 x 20,001 636 -> 524).
constexpr int norm_blocks(bool f32, bool vec, int steps, int threads) { return f32 && !vec && steps == 8 && threads == 1024; }

// VEC: rows of aligned 8-element vectors; a thread's step is one of them. Else a
// warp's step is 128 elements, a lane's every 32nd of these.
template <bool F32, bool VEC, int STEPS, int THREADS>
__global__ void __launch_bounds__(THREADS, norm_blocks(F32, VEC, STEPS, THREADS)) add_rmsnorm_kernel(const __grid_constant__ NormParams p, int warps) {
  constexpr int E = VEC ? 8 : 4;
  __shared__ float s_part[2][kNormMaxWarps];
  const int lane = threadIdx.x & 31;
  const int warp = warps == 1 ? 0 : threadIdx.x >> 5;           // within the row
  const long long row = warps == 1 ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)
                                   : static_cast<long long>(blockIdx.x);
  if (row >= p.rows) return;                                    // (whole warps, and no barrier among them)
  const bool f16 = p.x_dtype == DSA_FP16;
  const auto at = [&](int s, int e) {
    return VEC ? ((s * warps + warp) * 32 + lane) * 8 + e : (s * warps + warp) * 128 + e * 32 + lane;
  };
  float v[STEPS][E];
  {
    Raw<F32, VEC> x[STEPS], r[STEPS];
    const auto load = [&](const void* base, long long first, Raw<F32, VEC> (&to)[STEPS]) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        if constexpr (VEC) {
          if (at(s, 0) < p.hidden) to[s].load8(base, first + at(s, 0));
          else to[s].zero();
        } else {
          to[s].zero();
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (at(s, e) < p.hidden) to[s].load1(base, first + at(s, e), e);
        }
      }
    };
    load(p.x, row * p.xs, x);
    if (p.r) load(p.r, row * p.rs, r);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[s][e] = x[s].get(e, f16);
      if (!p.r) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) v[s][e] += r[s].get(e, f16);
      if constexpr (VEC) {
        const long long i = row * p.hs + at(s, 0);
        const bool store = p.h && at(s, 0) < p.hidden;
        if constexpr (F32) {
          if (store) {
            float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.h) + i);
            d[0] = make_float4(v[s][0], v[s][1], v[s][2], v[s][3]);
            d[1] = make_float4(v[s][4], v[s][5], v[s][6], v[s][7]);
          }
        } else {
          const uint4 u = pack8(v[s], f16);
          if (store) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h) + i) = u;
          const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < E; ++e) v[s][e] = from16((w4[e >> 1] >> (16 * (e & 1))) & 0xffffu, f16);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool store = p.h && at(s, e) < p.hidden;
          if constexpr (F32) {
            if (store) static_cast<float*>(p.h)[row * p.hs + at(s, e)] = v[s][e];
          } else {
            const uint32_t u = to16(v[s][e], f16);
            if (store) static_cast<uint16_t*>(p.h)[row * p.hs + at(s, e)] = static_cast<uint16_t>(u);
            v[s][e] = from16(u, f16);
          }
        }
      }
    }
  }
  // 1 / sqrt(mean square + eps), all in fp32. Where the sum of squares leaves
  // [2^-100, 2^100] the row is scaled by 2^-+96 first: then it neither overflows
  // nor vanishes (32,768 values of up to 2^128, or one of 2^-149). The scale cancels
  // in y, and eps takes its square; a mean below 2^-24 of eps needs none.
  float ss = 0.f;
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
#pragma unroll
    for (int e = 0; e < E; ++e) ss = fmaf(v[s][e], v[s][e], ss);
  ss = row_reduce<false>(ss, warps, s_part, 0);
  float eps = p.eps;
  if (!(ss >= 0x1p-100f && ss <= 0x1p100f)) {                   // (the same for all threads of the row)
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(v[s][e]));
    top = row_reduce<true>(top, warps, s_part, 1);
    const float sc = top > 0x1p40f ? 0x1p-96f : top > 0.f && top < 0x1p-40f && eps < 0x1p-76f ? 0x1p96f : 1.0f;
    eps = eps * sc * sc;
    ss = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[s][e] *= sc;
        ss = fmaf(v[s][e], v[s][e], ss);
      }
    ss = row_reduce<false>(ss, warps, s_part, 0);
  }
  const float inv = rsqrtf(fmaf(ss, p.inv_hidden, eps));
  const bool q8 = p.y_dtype == DSA_FP8_E4M3 || p.y_dtype == DSA_INT8, int8 = p.y_dtype == DSA_INT8;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if constexpr (VEC) {
      if (at(s, 0) >= p.hidden) continue;
      const float4* g = reinterpret_cast<const float4*>(p.gamma + at(s, 0));
      const float4 a = __ldg(g), b = __ldg(g + 1);
      const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < E; ++e) v[s][e] = v[s][e] * inv * w[e];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (at(s, e) < p.hidden) v[s][e] = v[s][e] * inv * __ldg(p.gamma + at(s, e));
    }
  }
  const float most = int8 ? 127.0f : 448.0f;
  const bool per_row = q8 && p.groups == 1;
  float top = 0.f;
  if (per_row) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(v[s][e]));
    top = row_reduce<true>(top, warps, s_part, 1);
    if (warp == 0 && lane == 0) p.scale[row] = top / most;
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const long long i = at(s, 0);
    if (!q8) {
      const bool y16 = p.y_dtype == DSA_FP16;
      if constexpr (VEC) {
        if (i < p.hidden) __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + row * p.ys + i), pack8(v[s], y16));
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (at(s, e) < p.hidden) static_cast<uint16_t*>(p.y)[row * p.ys + at(s, e)] = static_cast<uint16_t>(to16(v[s][e], y16));
      }
      continue;
    }
    if (!per_row) {
      top = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(v[s][e]));
#pragma unroll
      for (int o = VEC ? 8 : 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int g = static_cast<int>(i) / kNormGroup;
      if ((VEC ? (lane & 15) : lane) == 0 && i < p.hidden) p.scale[row * p.groups + g] = top / most;
    }
    // y / scale as y times one quotient, of y lifted or lowered to where the fast division is
    // right to two units in the last place (83.5 -> 82.5 us; a code rounds to 2^-4 of itself)
    const float lift = top < 0x1p-100f ? 0x1p100f : top > 0x1p100f ? 0x1p-100f : 1.0f;
    const float by = top > 0.f ? __fdividef(most, top * lift) : 0.f;
    if constexpr (VEC) {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < E; e += 2) w[e >> 2] |= code_pair(v[s][e] * lift * by, v[s][e + 1] * lift * by, int8) << (8 * (e & 3));
      if (i < p.hidden) __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row * p.ys + i), make_uint2(w[0], w[1]));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (at(s, e) < p.hidden) static_cast<uint8_t*>(p.y)[row * p.ys + at(s, e)] = static_cast<uint8_t>(code_pair(v[s][e] * lift * by, 0.f, int8));
    }
  }
}

int dtype_bytes(int d) { return d == DSA_FP32 ? 4 : d == DSA_INT8 || d == DSA_FP8_E4M3 ? 1 : 2; }

template <bool F32, bool VEC>
cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t st) {
  const int per_warp = VEC ? 256 : 128;                         // elements of a warp's step
  const int units = (p.hidden + per_warp - 1) / per_warp;       // steps of a row, over all its warps
  // 8, 16 or 32 elements a thread: as few as it can be where the rows are few
  constexpr int S0 = VEC ? 1 : 2, S1 = 2 * S0, S2 = 4 * S0;
  int steps = S2;
  if (p.rows <= 2 * sms && units <= kNormMaxWarps * S0) steps = S0;
  else if (units <= S0) steps = S0;
  else if (units <= S1 || (p.rows <= 2 * sms && units <= kNormMaxWarps * S1)) steps = S1;
  const int warps = (units + steps - 1) / steps;
  const int threads = warps == 1 ? 256 : 32 * warps;
  const long long blocks = warps == 1 ? (p.rows + 7) / 8 : p.rows;
  const dim3 grid(static_cast<unsigned>(blocks));
  const char* name = "add_rmsnorm_kernel";
  if (steps == S0) return launch_kernel(name, add_rmsnorm_kernel<F32, VEC, S0, 1024>, grid, dim3(threads), 0, st, false, p, warps);
  if (steps == S1) return launch_kernel(name, add_rmsnorm_kernel<F32, VEC, S1, 1024>, grid, dim3(threads), 0, st, false, p, warps);
  // (32 elements a thread: up to 128 registers, which 512 threads may have; 1,024 have 64, which spill
  // 4 bytes of 16-bit rows of vectors, 68 of FP32, and 44 and 424 of rows by single elements)
  if (threads <= 512) return launch_kernel(name, add_rmsnorm_kernel<F32, VEC, S2, 512>, grid, dim3(threads), 0, st, false, p, warps);
  return launch_kernel(name, add_rmsnorm_kernel<F32, VEC, S2, 1024>, grid, dim3(threads), 0, st, false, p, warps);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_add_rmsnorm(const dsa_norm_problem* np, const void* x, const void* residual, const float* gamma,
                               void* h, void* y, float* scale, void* stream) {
  reset_launches();
  if (!np) return report_error(DSA_ERR_INVALID_ARG, "problem is NULL");
  if (np->rows < 0 || np->rows > 0x7fffffffLL) return report_error(DSA_ERR_INVALID_ARG, "rows must be 0 .. 2^31 - 1");
  if (np->hidden < 1 || np->hidden > kNormMaxHidden)
    return report_errorf(DSA_ERR_UNSUPPORTED, "hidden %d outside 1..%d", np->hidden, kNormMaxHidden);
  if (np->x_dtype != DSA_BF16 && np->x_dtype != DSA_FP16 && np->x_dtype != DSA_FP32)
    return report_error(DSA_ERR_UNSUPPORTED, "x_dtype must be BF16, FP16 or FP32");
  const bool q8 = np->y_dtype == DSA_INT8 || np->y_dtype == DSA_FP8_E4M3;
  if (!q8 && np->y_dtype != DSA_BF16 && np->y_dtype != DSA_FP16)
    return report_error(DSA_ERR_UNSUPPORTED, "y_dtype must be BF16, FP16, INT8 or FP8_E4M3");
  if (np->scale_group != 0 && (np->scale_group != kNormGroup || !q8))
    return report_errorf(DSA_ERR_UNSUPPORTED, "scale_group must be 0, or %d for an 8-bit y", kNormGroup);
  if (!(np->eps >= 0.0f) || std::isinf(np->eps)) return report_error(DSA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  const long long stride[4] = {np->x_stride, np->residual_stride, np->h_stride, np->y_stride};
  for (long long s : stride)
    if (s != 0 && (s < np->hidden || s > (1LL << 40))) return report_error(DSA_ERR_INVALID_ARG, "a row stride must be 0 or at least hidden");
  if (np->rows == 0) return DSA_OK;
  if (!x || !gamma || !y) return report_error(DSA_ERR_INVALID_ARG, "x, gamma and y are required");
  if (h && !residual) return report_error(DSA_ERR_INVALID_ARG, "h is the sum with a residual: there is none");
  if (q8 != (scale != nullptr)) return report_error(DSA_ERR_INVALID_ARG, "scale is required iff y is of 8 bits");
  NormParams p{};
  const auto pitch = [&](long long s) { return s ? s : static_cast<long long>(np->hidden); };
  p.x = x, p.r = residual, p.gamma = gamma, p.h = h, p.y = y, p.scale = scale;
  p.rows = np->rows, p.hidden = np->hidden, p.x_dtype = np->x_dtype, p.y_dtype = np->y_dtype;
  p.xs = pitch(np->x_stride), p.rs = pitch(np->residual_stride), p.hs = pitch(np->h_stride), p.ys = pitch(np->y_stride);
  p.groups = np->scale_group ? (np->hidden + kNormGroup - 1) / kNormGroup : 1;
  p.eps = np->eps;
  p.inv_hidden = 1.0f / static_cast<float>(np->hidden);
  const int xb = dtype_bytes(np->x_dtype), yb = dtype_bytes(np->y_dtype);
  const auto off = [](const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) != 0; };
  if (off(x, xb) || off(residual, xb) || off(h, xb) || off(y, yb) || off(gamma, 4) || off(scale, 4))
    return report_error(DSA_ERR_MISALIGNED, "tensors must be aligned to their elements");
  // A row is read before it is written, so h may be x or the residual, and y the one or the
  // other, in the same place; any other overlap is refused, y's with h too.
  struct Span {
    const void* at;
    long long pitch, bytes;
  };
  const auto span = [&](const void* q, long long pt, int b) {
    return Span{q, pt * b, q ? ((p.rows - 1) * pt + p.hidden) * b : 0};
  };
  const Span in[3] = {span(x, p.xs, xb), span(residual, p.rs, xb), {gamma, 0, 4LL * p.hidden}};
  const Span out[3] = {span(h, p.hs, xb), span(y, p.ys, yb), {scale, 0, scale ? 4 * p.rows * p.groups : 0}};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 3; ++i) {
      if (!out[o].bytes || !in[i].bytes || !overlap(out[o].at, out[o].bytes, in[i].at, in[i].bytes)) continue;
      const bool same = out[o].at == in[i].at && out[o].pitch == in[i].pitch && o < 2 && i < 2 && (o == 0 || xb == yb);
      if (!same) return report_error(DSA_ERR_INVALID_ARG, "a result overlaps an input other than row by row");
    }
    for (int k = 0; k < o; ++k)
      if (out[o].bytes && out[k].bytes && overlap(out[o].at, out[o].bytes, out[k].at, out[k].bytes))
        return report_error(DSA_ERR_INVALID_ARG, "results overlap each other");
  }
  int sms = 0;
  if (int rc = current_device(&sms)) return rc;
  const auto vec = [&](const void* q, long long pt, int b) { return !q || (!off(q, 8 * b > 16 ? 16 : 8 * b) && pt % 8 == 0); };
  const bool aligned = p.hidden % 8 == 0 && vec(x, p.xs, xb) && vec(residual, p.rs, xb) && vec(h, p.hs, xb) &&
                       vec(y, p.ys, yb) && !off(gamma, 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = np->x_dtype == DSA_FP32;
  const cudaError_t e = f32 ? (aligned ? launch_norm<true, true>(p, sms, st) : launch_norm<true, false>(p, sms, st))
                            : (aligned ? launch_norm<false, true>(p, sms, st) : launch_norm<false, false>(p, sms, st));
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "add_rmsnorm launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}
