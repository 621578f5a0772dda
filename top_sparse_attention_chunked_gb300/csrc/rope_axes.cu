// RMSNorm and rotary positions with several axes for a packed step's queries and
// keys, and its keys and values into the cache rows that a slot map names.
//
// A token has a position per axis (time, height, width of an image's patch; the
// same for text), and pair i of a head vector, elements i and i + r / 2, turns
// by the angle of its own axis's position:
//     y_i         = x_i cos - x_{i + r/2} sin
//     y_{i + r/2} = x_{i + r/2} cos + x_i sin.
// Eight lanes hold a head vector, a lane eight pairs of it (its elements
// 8 l .. and r / 2 + 8 l ..): both partners of a rotation are in one thread, the
// norm is a sum over eight lanes, and the angles, read once, serve all of the
// vectors that the lanes go through. They are kept multiplied by gamma: with c, s the
// angle's and g, h the partners' weights, y = (x g c - x' h s) / rms, y' = (x' h c + x g s) / rms.
//
// What bounds it: latency, short of the memory's rate. A batch of four vectors is loaded, computed
// and stored before the next one's loads begin, and the 16 warps that 128 registers leave an SM do
// not fill the gaps: schedulers are busy 40% of the time (INT8 47%), the ALU pipe 29%. 8,192 tokens of 32 / 8 heads, BF16: 37 us, 81% of the
// copy rate; 24 / 2 heads 24.2 us (74%); INT8 caches 41 us (68%). 16 tokens: 2.5 us, a
// launch and three dependent loads (position, angle, gamma beside the vector).
#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kRxPairs = DSA_HEAD_DIM / 2;
constexpr int kRxLanes = 8;                       // lanes of a head vector
constexpr int kRxThreads = 128;
constexpr int kRxBatch = 4;                       // vectors whose loads are in flight together

struct AxesParams {
  const void* q;
  const void* k;
  const void* v;
  const float* gq;      // [128] or nullptr (no norm)
  const float* gk;
  const void* cos;      // [max_pos, r / 2]
  const void* sin;
  const int32_t* pos;   // axis a of token n: pos[a * pos_stride + n]
  const int32_t* slots; // [N] cache rows, or negative
  void* out;
  void* kc;             // [cache rows, Hkv, 128]
  void* vc;
  float* ks;
  float* vs;
  long long tokens, qs, kst, vst, os, pos_stride, cache_rows;
  int hq, hkv, half, max_pos, q_dtype, kv_dtype;  // half: r / 2
  int per_unit, q_units, kv_units;                // vectors of a unit; units of a token's q, and of its k (and v)
  int q_blocks, kv_blocks;                        // thread blocks of the queries, of the keys (and values)
  int cos_f32, whole8, axes;   // whole8: a lane's eight pairs have one axis, and their angles may be read as vectors
  uint16_t axis[kRxLanes];     // the axes of a lane's pairs, two bits each
  float eps;
};

__device__ __forceinline__ float rx_from16(uint32_t u, bool f16) {
  return f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(u))) : __uint_as_float(u << 16);
}
// Two 16-bit values in a word, and the other way.
template <bool F16>
__device__ __forceinline__ uint32_t rx_pack(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool F16>
__device__ __forceinline__ float2 rx_unpack(uint32_t u) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Where the lane's eight first and eight second elements of a vector lie. Pairs
// from r / 2 on are not rotated: elements r + j and r + j + (128 - r) / 2.
struct LaneAt {
  int a, b;
  bool turns;
  __device__ __forceinline__ LaneAt(int l, int half) {
    const int p = 8 * l;
    turns = p < half;
    a = turns ? p : half + p;
    b = turns ? p + half : p + kRxPairs;
  }
};
// (r / 2 not a multiple of 8: element by element)
__device__ __forceinline__ int pair_a(int p, int half) { return p < half ? p : half + p; }
__device__ __forceinline__ int pair_b(int p, int half) { return p < half ? p + half : p + kRxPairs; }

template <bool VEC>
__device__ __forceinline__ void rx_load(const uint16_t* src, int l, int half, uint32_t (&u)[8]) {
  if constexpr (VEC) {
    const LaneAt at(l, half);
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(src + at.a)), y = __ldcs(reinterpret_cast<const uint4*>(src + at.b));
    u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
    u[4] = y.x; u[5] = y.y; u[6] = y.z; u[7] = y.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = 8 * l + 2 * e;
      u[e] = src[pair_a(p, half)] | static_cast<uint32_t>(src[pair_a(p + 1, half)]) << 16;
      u[4 + e] = src[pair_b(p, half)] | static_cast<uint32_t>(src[pair_b(p + 1, half)]) << 16;
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void rx_store(uint16_t* dst, int l, int half, const uint32_t (&u)[8]) {
  if constexpr (VEC) {
    const LaneAt at(l, half);
    *reinterpret_cast<uint4*>(dst + at.a) = make_uint4(u[0], u[1], u[2], u[3]);
    *reinterpret_cast<uint4*>(dst + at.b) = make_uint4(u[4], u[5], u[6], u[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = 8 * l + 2 * e;
      dst[pair_a(p, half)] = static_cast<uint16_t>(u[e]);
      dst[pair_a(p + 1, half)] = static_cast<uint16_t>(u[e] >> 16);
      dst[pair_b(p, half)] = static_cast<uint16_t>(u[4 + e]);
      dst[pair_b(p + 1, half)] = static_cast<uint16_t>(u[4 + e] >> 16);
    }
  }
}

__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// 1 over the root mean square of a vector (x[0..7]: the lane's first elements, x[8..15]:
// their partners); all lanes of the warp call it. Where a sum of squares lies outside
// [2^-100, 2^100] it is taken of the vector scaled by 2^-+96, which x becomes.
__device__ __forceinline__ float rx_rms(float (&x)[16], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
  ss = sum8(ss);
  if (__any_sync(0xffffffffu, !(ss >= 0x1p-100f && ss <= 0x1p100f))) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
    top = max8(top);
    const float sc = top > 0x1p40f ? 0x1p-96f : top > 0.f && top < 0x1p-40f && eps < 0x1p-76f ? 0x1p96f : 1.0f;
    eps = eps * sc * sc;
    ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] *= sc;
      ss = fmaf(x[e], x[e], ss);
    }
    ss = sum8(ss);
  }
  return rsqrtf(fmaf(ss, 1.0f / DSA_HEAD_DIM, eps));
}

// One 16-bit vector (the lane's packed elements u) into row `to` of a cache.
template <bool VEC, bool F16>
__device__ __forceinline__ void rx_append(const AxesParams& p, void* cache, float* scales, long long to, bool live, int l,
                                          uint32_t (&u)[8]) {
  if (p.kv_dtype == DSA_INT8) {
    float x[16], top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 v = rx_unpack<F16>(u[e]);
      x[2 * e] = v.x;
      x[2 * e + 1] = v.y;
      top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
    top = max8(top);
    if (!live) return;
    const float scale = __fdiv_rn(top, 127.0f);
    // x / scale, correctly rounded, from the scale's reciprocal (Markstein, 1990: if y is 1 / b
    // rounded to the nearest and q within a unit in the last place of a / b, then so is
    // q + (a - b q) y rounded once; x y is within two, the first step within one). What
    // 16-bit values hold is next to a half too often for a branch (one in 300: the largest
    // value's half is 63.5). Scales whose remainders would be subnormal are divided by.
    constexpr float kWhole = 12582912.0f;         // 1.5 * 2^23: adding it rounds, the low byte is the code
    const bool large = scale >= 0x1p-90f;
    const float by = large ? __fdiv_rn(1.0f, scale) : 0.f;
    uint32_t c[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float q = __fmul_rn(x[e], by);
      q = __fmaf_rn(__fmaf_rn(-q, scale, x[e]), by, q);
      q = __fmaf_rn(__fmaf_rn(-q, scale, x[e]), by, q);
      c[e] = __float_as_uint(__fadd_rn(q, kWhole));
    }
    if (!large && scale != 0.f) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        c[e] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fdiv_rn(x[e], scale), -127.0f), 127.0f), kWhole));
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
    uint8_t* d = static_cast<uint8_t*>(cache) + to * DSA_HEAD_DIM;
    if constexpr (VEC) {
      const LaneAt at(l, p.half);
      *reinterpret_cast<uint2*>(d + at.a) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(d + at.b) = make_uint2(w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[pair_a(8 * l + e, p.half)] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
        d[pair_b(8 * l + e, p.half)] = static_cast<uint8_t>(w[2 + (e >> 2)] >> (8 * (e & 3)));
      }
    }
    if (l == 0) scales[to] = scale;
    return;
  }
  if (!live) return;
  if constexpr (!F16) {
    if (p.kv_dtype == DSA_FP16) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 v = rx_unpack<false>(u[e]);
        u[e] = rx_pack<true>(v.x, v.y);
      }
    }
  }
  rx_store<VEC>(static_cast<uint16_t*>(cache) + to * DSA_HEAD_DIM, l, p.half, u);
}

// The angles of the lane's eight pairs (1 and 0 where they are not rotated).
template <bool VEC>
__device__ __forceinline__ void rx_angles(const AxesParams& p, int l, long long n, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }
  if (8 * l >= p.half) return;
  const uint32_t axes = p.axis[l];
  const auto row_of = [&](int a) {
    int at = __ldg(p.pos + a * p.pos_stride + n);
    at = at < 0 ? 0 : at >= p.max_pos ? p.max_pos - 1 : at;                    // clamped to the caches
    return static_cast<long long>(at) * p.half + 8 * l;
  };
  if (VEC && p.whole8) {
    const long long row = row_of(axes & 3u);
    if (p.cos_f32) {
      const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(p.cos) + row);
      const float4* y = reinterpret_cast<const float4*>(static_cast<const float*>(p.sin) + row);
      const float4 a0 = __ldg(x), a1 = __ldg(x + 1), b0 = __ldg(y), b1 = __ldg(y + 1);
      cs[0] = a0.x; cs[1] = a0.y; cs[2] = a0.z; cs[3] = a0.w; cs[4] = a1.x; cs[5] = a1.y; cs[6] = a1.z; cs[7] = a1.w;
      sn[0] = b0.x; sn[1] = b0.y; sn[2] = b0.z; sn[3] = b0.w; sn[4] = b1.x; sn[5] = b1.y; sn[6] = b1.z; sn[7] = b1.w;
    } else {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.cos) + row));
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.sin) + row));
      const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cs[e] = rx_from16((u[e >> 1] >> (16 * (e & 1))) & 0xffffu, false);
        sn[e] = rx_from16((v[e >> 1] >> (16 * (e & 1))) & 0xffffu, false);
      }
    }
    return;
  }
  // all positions, then all angles: two latencies, whatever the number of axes
  long long row[DSA_MAX_AXES];
#pragma unroll
  for (int a = 0; a < DSA_MAX_AXES; ++a) row[a] = a < p.axes ? row_of(a) : 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (8 * l + e >= p.half) continue;
    const uint32_t a = (axes >> (2 * e)) & 3u;
    const long long at = (a == 0 ? row[0] : a == 1 ? row[1] : a == 2 ? row[2] : row[3]) + e;
    cs[e] = p.cos_f32 ? __ldg(static_cast<const float*>(p.cos) + at) : rx_from16(__ldg(static_cast<const uint16_t*>(p.cos) + at), false);
    sn[e] = p.cos_f32 ? __ldg(static_cast<const float*>(p.sin) + at) : rx_from16(__ldg(static_cast<const uint16_t*>(p.sin) + at), false);
  }
}

// A unit is a run of up to per_unit vectors of one token: of its queries, keys or
// values. Eight lanes take one; a thread block's are all of the same kind.
template <bool VEC, bool F16>
__global__ void __launch_bounds__(kRxThreads, 4) rope_axes_append_kernel(const __grid_constant__ AxesParams p) {
  const int l = threadIdx.x & (kRxLanes - 1);
  const int block = blockIdx.x;
  const int kind = block < p.q_blocks ? 0 : block < p.q_blocks + p.kv_blocks ? 1 : 2;   // q, k, v
  const int per_token = kind == 0 ? p.q_units : p.kv_units, heads = kind == 0 ? p.hq : p.hkv;
  const long long all = p.tokens * per_token;
  const long long unit0 = static_cast<long long>(block - (kind == 0 ? 0 : kind == 1 ? p.q_blocks : p.q_blocks + p.kv_blocks)) *
                              (kRxThreads / kRxLanes) + threadIdx.x / kRxLanes;
  const bool in = unit0 < all;
  if (!__any_sync(0xffffffffu, in)) return;
  const long long unit = in ? unit0 : all - 1, n = unit / per_token;
  const int h0 = static_cast<int>(unit - n * per_token) * p.per_unit;
  const int nv = in ? min(p.per_unit, heads - h0) : 0;
  const uint16_t* src = static_cast<const uint16_t*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                        n * (kind == 0 ? p.qs : kind == 1 ? p.kst : p.vst) + h0 * DSA_HEAD_DIM;
  long long slot = -1;
  if (kind != 0) {
    slot = __ldg(p.slots + n);
    if (slot >= p.cache_rows) slot = -1;
  }
  int most = nv;                                                                // (the warp's lanes stay together)
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 8));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 16));
  const auto load = [&](int i, uint32_t (&u)[8]) {
    if (i < nv) {
      rx_load<VEC>(src + i * DSA_HEAD_DIM, l, p.half, u);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = 0;
    }
  };
  if (kind == 2) {
    for (int i0 = 0; i0 < most; i0 += kRxBatch) {
      uint32_t u[kRxBatch][8];
#pragma unroll
      for (int i = 0; i < kRxBatch; ++i) load(i0 + i, u[i]);
#pragma unroll
      for (int i = 0; i < kRxBatch; ++i)
        rx_append<VEC, F16>(p, p.vc, p.vs, slot * p.hkv + h0 + i0 + i, i0 + i < nv && slot >= 0, l, u[i]);
    }
    return;
  }
  uint32_t u[kRxBatch][8];
#pragma unroll
  for (int i = 0; i < kRxBatch; ++i) load(i, u[i]);                             // (in flight beside the angles)
  const float* gamma = kind == 0 ? p.gq : p.gk;
  // the factors of the lane's pairs: first elements gc, hs, partners hc, gs
  float gc[8], hs[8], hc[8], gs[8];
  {
    float cs[8], sn[8];
    rx_angles<VEC>(p, l, n, cs, sn);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = gamma ? __ldg(gamma + pair_a(8 * l + e, p.half)) : 1.f, h = gamma ? __ldg(gamma + pair_b(8 * l + e, p.half)) : 1.f;
      gc[e] = g * cs[e];
      gs[e] = g * sn[e];
      hc[e] = h * cs[e];
      hs[e] = h * sn[e];
    }
  }
  for (int i0 = 0; i0 < most; i0 += kRxBatch) {
    if (i0 > 0) {
#pragma unroll
      for (int i = 0; i < kRxBatch; ++i) load(i0 + i, u[i]);
    }
#pragma unroll
    for (int i = 0; i < kRxBatch; ++i) {
      if (i0 + i >= most) break;
      const bool live = i0 + i < nv;
      float x[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 v = rx_unpack<F16>(u[i][e]);
        x[2 * e] = v.x;
        x[2 * e + 1] = v.y;
      }
      const float inv = gamma ? rx_rms(x, p.eps) : 1.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = x[e], b = x[8 + e];
        x[e] = (a * gc[e] - b * hs[e]) * inv;
        x[8 + e] = (b * hc[e] + a * gs[e]) * inv;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] = rx_pack<F16>(x[2 * e], x[2 * e + 1]);
      if (kind == 0) {
        if (live) rx_store<VEC>(static_cast<uint16_t*>(p.out) + n * p.os + (h0 + i0 + i) * DSA_HEAD_DIM, l, p.half, u[i]);
      } else {
        rx_append<VEC, F16>(p, p.kc, p.ks, slot * p.hkv + h0 + i0 + i, live && slot >= 0, l, u[i]);
      }
    }
  }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_rope_axes_append(const dsa_axes_problem* ap, const void* q, const void* k, const void* v,
                                    const float* gamma_q, const float* gamma_k, const void* cos_cache, const void* sin_cache,
                                    const int32_t* positions, const int32_t* slots, void* q_out, void* k_cache, void* v_cache,
                                    float* k_scale, float* v_scale, void* stream) {
  reset_launches();
  if (!ap) return report_error(DSA_ERR_INVALID_ARG, "problem is NULL");
  if (ap->tokens < 0 || ap->tokens > 0x7fffffffLL) return report_error(DSA_ERR_INVALID_ARG, "tokens must be 0 .. 2^31 - 1");
  if (ap->head_dim != DSA_HEAD_DIM) return report_errorf(DSA_ERR_UNSUPPORTED, "head_dim must be %d (got %d)", DSA_HEAD_DIM, ap->head_dim);
  const int hq = ap->num_q_heads, hkv = ap->num_kv_heads;
  if (hq < 0 || hkv < 0 || hq + hkv < 1 || hq > 65535 || hkv > 65535)
    return report_error(DSA_ERR_INVALID_ARG, "head counts must be 0 .. 65535, one of them above 0");
  if (ap->axes < 1 || ap->axes > DSA_MAX_AXES) return report_errorf(DSA_ERR_INVALID_ARG, "axes %d outside 1..%d", ap->axes, DSA_MAX_AXES);
  int half = 0;
  for (int a = 0; a < ap->axes; ++a) {
    if (ap->sections[a] < 0 || ap->sections[a] > kRxPairs) return report_errorf(DSA_ERR_INVALID_ARG, "sections[%d] = %d", a, ap->sections[a]);
    half += ap->sections[a];
  }
  if (half < 1 || half > kRxPairs) return report_errorf(DSA_ERR_INVALID_ARG, "the sections hold %d pairs: 1..%d", half, kRxPairs);
  if (ap->max_pos < 1) return report_error(DSA_ERR_INVALID_ARG, "max_pos must be >= 1");
  if (ap->cos_dtype != DSA_FP32 && ap->cos_dtype != DSA_BF16) return report_error(DSA_ERR_UNSUPPORTED, "the cos / sin caches must be FP32 or BF16");
  if (!(ap->eps >= 0.0f) || std::isinf(ap->eps)) return report_error(DSA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (ap->q_dtype != DSA_BF16 && ap->q_dtype != DSA_FP16) return report_error(DSA_ERR_UNSUPPORTED, "q_dtype must be BF16 or FP16");
  const bool int8 = ap->kv_dtype == DSA_INT8;
  if (!int8 && ap->kv_dtype != DSA_BF16 && ap->kv_dtype != DSA_FP16)
    return report_error(DSA_ERR_UNSUPPORTED, "kv_dtype must be BF16, FP16 or INT8");
  if (ap->q_dtype == DSA_FP16 && ap->kv_dtype == DSA_BF16)
    return report_error(DSA_ERR_UNSUPPORTED, "FP16 vectors with a BF16 cache are not built");
  if (ap->cache_rows < 0 || ap->cache_rows >= (1LL << 31) || (hkv > 0 && ap->cache_rows < 1))
    return report_error(DSA_ERR_INVALID_ARG, "cache_rows must be below 2^31, and above 0 where there are KV heads");
  const long long wide[4] = {128LL * hq, 128LL * hkv, 128LL * hkv, 128LL * hq};
  const long long given[4] = {ap->q_stride, ap->k_stride, ap->v_stride, ap->out_stride};
  long long st4[4];
  for (int i = 0; i < 4; ++i) {
    if (given[i] != 0 && (given[i] < wide[i] || given[i] > (1LL << 40) || given[i] % 8 != 0))
      return report_error(DSA_ERR_INVALID_ARG, "a token stride must be 0, or a multiple of 8 that holds the token's heads");
    st4[i] = given[i] ? given[i] : wide[i];
  }
  const long long ps = ap->pos_stride;
  if (ps < 0 || ps > (1LL << 40)) return report_error(DSA_ERR_INVALID_ARG, "pos_stride must be >= 0");
  const long long N = ap->tokens;
  if (N == 0) return DSA_OK;
  if (!cos_cache || !sin_cache || !positions) return report_error(DSA_ERR_INVALID_ARG, "positions and the cos / sin caches are required");
  if ((hq > 0 && (!q || !q_out)) || (hkv > 0 && (!k || !v || !k_cache || !v_cache || !slots)))
    return report_error(DSA_ERR_INVALID_ARG, "a required tensor pointer is NULL");
  if ((int8 && hkv > 0) != (k_scale != nullptr) || (int8 && hkv > 0) != (v_scale != nullptr))
    return report_error(DSA_ERR_INVALID_ARG, "k_scale / v_scale are required iff the cache is INT8");
  const auto off = [](const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) & (a - 1)) != 0; };
  const int cb = ap->cos_dtype == DSA_FP32 ? 4 : 2;
  if (off(q, 16) || off(k, 16) || off(v, 16) || off(q_out, 16) || off(k_cache, 16) || off(v_cache, 16))
    return report_error(DSA_ERR_MISALIGNED, "q, k, v, q_out and the caches must be 16-byte aligned");
  if (off(gamma_q, 4) || off(gamma_k, 4) || off(positions, 4) || off(slots, 4) || off(k_scale, 4) || off(v_scale, 4) ||
      off(cos_cache, cb) || off(sin_cache, cb))
    return report_error(DSA_ERR_MISALIGNED, "gamma, positions, slots, scales, cos and sin must be aligned to their elements");
  // what is read and what is written: q_out may be q itself
  struct Span {
    const void* at;
    long long bytes;
  };
  const auto rows = [&](const void* x, int i) { return Span{x, wide[i] ? ((N - 1) * st4[i] + wide[i]) * 2 : 0}; };
  const long long cache_bytes = ap->cache_rows * hkv * 128LL * (int8 ? 1 : 2), scale_bytes = int8 ? ap->cache_rows * hkv * 4LL : 0;
  const Span in[9] = {rows(q, 0), rows(k, 1), rows(v, 2), {gamma_q, gamma_q ? 512 : 0}, {gamma_k, gamma_k ? 512 : 0},
                      {cos_cache, 1LL * ap->max_pos * half * cb}, {sin_cache, 1LL * ap->max_pos * half * cb},
                      {positions, ((ap->axes - 1) * ps + N) * 4}, {slots, hkv ? N * 4 : 0}};
  const Span out[5] = {rows(q_out, 3), {k_cache, cache_bytes}, {v_cache, cache_bytes}, {k_scale, scale_bytes}, {v_scale, scale_bytes}};
  for (int o = 0; o < 5; ++o) {
    if (!out[o].at || !out[o].bytes) continue;
    for (int i = 0; i < 9; ++i) {
      if (!in[i].at || !in[i].bytes || !overlap(out[o].at, out[o].bytes, in[i].at, in[i].bytes)) continue;
      if (o == 0 && i == 0 && q == q_out && st4[0] == st4[3]) continue;
      // (in place in a projection's rows, of which keys and values are columns too)
      if (o == 0 && (i == 1 || i == 2) && q == q_out && st4[0] == st4[3] && st4[i] == st4[0]) {
        const long long d = (static_cast<const uint8_t*>(in[i].at) - static_cast<const uint8_t*>(q)) / 2;
        const long long in_row = ((d % st4[0]) + st4[0]) % st4[0];
        if (in_row >= wide[0] && in_row + wide[i] <= st4[0]) continue;
      }
      return report_error(DSA_ERR_INVALID_ARG, "a result overlaps an input");
    }
    for (int j = 0; j < o; ++j)
      if (out[j].at && out[j].bytes && overlap(out[o].at, out[o].bytes, out[j].at, out[j].bytes))
        return report_error(DSA_ERR_INVALID_ARG, "results overlap each other");
  }
  int sms = 0;
  if (int rc = current_device(&sms)) return rc;
  AxesParams p{};
  p.q = q, p.k = k, p.v = v, p.gq = gamma_q, p.gk = gamma_k, p.cos = cos_cache, p.sin = sin_cache;
  p.pos = positions, p.slots = slots, p.out = q_out, p.kc = k_cache, p.vc = v_cache, p.ks = k_scale, p.vs = v_scale;
  p.tokens = N, p.qs = st4[0], p.kst = st4[1], p.vst = st4[2], p.os = st4[3], p.pos_stride = ps, p.cache_rows = ap->cache_rows;
  p.hq = hq, p.hkv = hkv, p.half = half, p.max_pos = ap->max_pos, p.q_dtype = ap->q_dtype, p.kv_dtype = ap->kv_dtype;
  p.cos_f32 = ap->cos_dtype == DSA_FP32, p.eps = ap->eps;
  p.axes = ap->axes;
  int axis[kRxPairs] = {};
  if (ap->in_turn) {
    int left[DSA_MAX_AXES], n = 0;
    for (int a = 0; a < ap->axes; ++a) left[a] = ap->sections[a];
    while (n < half)
      for (int a = 0; a < ap->axes; ++a)
        if (left[a] > 0) {
          --left[a];
          axis[n++] = a;
        }
  } else {
    for (int a = 0, n = 0; a < ap->axes; ++a)
      for (int i = 0; i < ap->sections[a]; ++i) axis[n++] = a;
  }
  bool whole8 = half % 8 == 0 && !off(cos_cache, 16) && !off(sin_cache, 16);
  for (int i = 0; i < half; ++i) {
    whole8 = whole8 && axis[i] == axis[i & ~7];
    p.axis[i / 8] |= static_cast<uint16_t>(axis[i] << (2 * (i % 8)));
  }
  p.whole8 = whole8;
  // A unit's vectors share their angles: as many (of 1, 2 .. 32) as leave every SM some 24
  // units, of the 64 that it takes at once. (8,192 tokens of 32 / 8 heads: units of 4, 8, 16,
  // 32 take 50, 41, 39, 37 us; 2,000: 16.6, 16.1, 14.3 with 4, 8, 16; 300 of 24 / 2 heads:
  // 5.0, 6.6, 11.3 with 1, 8, 16.)
  p.per_unit = 32;
  while (p.per_unit > 1 && N * ((std::max(hq, hkv) + p.per_unit - 1) / p.per_unit) < 24LL * sms) p.per_unit /= 2;
  p.q_units = (hq + p.per_unit - 1) / p.per_unit;
  p.kv_units = (hkv + p.per_unit - 1) / p.per_unit;
  constexpr int kUnits = kRxThreads / kRxLanes;
  const long long qb = (N * p.q_units + kUnits - 1) / kUnits, kb = (N * p.kv_units + kUnits - 1) / kUnits, blocks = qb + 2 * kb;
  if (blocks > 0x7fffffffLL) return report_error(DSA_ERR_UNSUPPORTED, "too many tokens and heads for one call");
  p.q_blocks = static_cast<int>(qb);
  p.kv_blocks = static_cast<int>(kb);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(blocks));
  const bool vec = half % 8 == 0, f16 = ap->q_dtype == DSA_FP16;
  using K = void(const AxesParams);
  K* const kernels[2][2] = {{rope_axes_append_kernel<false, false>, rope_axes_append_kernel<false, true>},
                            {rope_axes_append_kernel<true, false>, rope_axes_append_kernel<true, true>}};
  const cudaError_t e = launch_kernel("rope_axes_append_kernel", kernels[vec][f16], grid, dim3(kRxThreads), 0, st, false, p);
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "rope_axes_append launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}
