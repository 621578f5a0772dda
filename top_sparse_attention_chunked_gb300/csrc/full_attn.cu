// Full GQA attention of every sequence's new tokens over its cached keys.
//
// One warp per (query token, query head): four dims a lane, one key after the
// other, an online softmax in fp32.
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "sm100_ptx.cuh"

namespace dsa {
namespace {

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
  int B, Hq, Hkv, cap, window;
  int q_dtype, kv_dtype, out_dtype;
  float scale, softcap;
  Paging pg;
  int q0[DSA_MAX_BATCH + 1];     // first query row of each sequence
  int T[DSA_MAX_BATCH], first[DSA_MAX_BATCH];
};

__device__ __forceinline__ void load4(const void* p, int dtype, long long i, float* x) {
  if (dtype == DSA_INT8) {
    const char4 c = *reinterpret_cast<const char4*>(static_cast<const int8_t*>(p) + i);
    x[0] = c.x; x[1] = c.y; x[2] = c.z; x[3] = c.w;
    return;
  }
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  if (dtype == DSA_FP16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  } else {
    x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xffff0000u);
  }
}

__global__ void __launch_bounds__(32) full_attn_kernel(const __grid_constant__ FullParams p) {
  const int n = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  int b = 0;
  while (n >= p.q0[b + 1]) ++b;
  const int S = p.q0[b + 1] - p.q0[b];
  const int pos = p.T[b] - S + (n - p.q0[b]);
  int lo = p.first[b];
  if (p.window > 0) lo = max(lo, pos - p.window + 1);
  const int g = h / (p.Hq / p.Hkv);
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  const long long qi = (static_cast<long long>(n) * p.Hq + h) * DSA_HEAD_DIM + lane * 4;
  load4(p.q, p.q_dtype, qi, q);
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  bool bad = false;
  for (int t = lo; t <= pos; ++t) {
    const long long row = cache_row(p.pg, b, p.cap, t, &bad) * p.Hkv + g;
    float k[4], v[4];
    load4(p.k, p.kv_dtype, row * DSA_HEAD_DIM + lane * 4, k);
    load4(p.v, p.kv_dtype, row * DSA_HEAD_DIM + lane * 4, v);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) z = fmaf(q[i], k[i], z);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    z *= p.scale;
    float vs = 1.f;
    if (p.kv_dtype == DSA_INT8) {
      z *= p.k_scale[row];
      vs = p.v_scale[row];
    }
    if (p.softcap > 0.f) z = p.softcap * tanhf(z / p.softcap);
    z += slope * static_cast<float>(t - pos);
    const float mn = fmaxf(m, z);
    const float a = expf(m - mn), w = expf(z - mn);
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * a + w * vs * v[i];
    m = mn;
  }
  if (bad && lane == 0) atomicOr(p.status, kDevBadPage);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = l > 0.f ? o[i] / l : 0.f;
    if (p.out_dtype == DSA_BF16) static_cast<__nv_bfloat16*>(p.out)[qi + i] = __float2bfloat16_rn(x);
    else if (p.out_dtype == DSA_FP16) static_cast<__half*>(p.out)[qi + i] = __float2half_rn(x);
    else static_cast<float*>(p.out)[qi + i] = x;
  }
  if (p.lse && lane == 0) p.lse[static_cast<long long>(n) * p.Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
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
  if (int rc = check_call_workspace(ws, ws_bytes, dsa_full_attn_workspace_size(p))) return rc;
  int sms = 0;
  if (int rc = current_device(&sms)) return rc;
  FullParams fp{};
  fp.q = q;
  fp.k = k;
  fp.v = v;
  fp.k_scale = ks;
  fp.v_scale = vs;
  fp.slopes = slopes;
  fp.out = out;
  fp.lse = lse;
  fp.status = static_cast<uint32_t*>(ws);
  fp.B = p->batch;
  fp.Hq = p->num_q_heads;
  fp.Hkv = p->num_kv_heads;
  fp.cap = p->cache_capacity;
  fp.window = p->window;
  fp.q_dtype = p->q_dtype;
  fp.kv_dtype = p->kv_dtype;
  fp.out_dtype = p->out_dtype;
  fp.scale = p->softmax_scale > 0.0f ? p->softmax_scale : 1.0f / std::sqrt(static_cast<float>(p->head_dim));
  fp.softcap = p->softcap;
  fp.pg = pg;
  for (int b = 0; b < p->batch; ++b) {
    fp.q0[b + 1] = fp.q0[b] + p->q_len[b];
    fp.T[b] = p->total_len[b];
    fp.first[b] = p->first_key[b];
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  const int n = fp.q0[p->batch];
  if (e == cudaSuccess && n > 0)
    e = launch_kernel("full_attn_kernel", full_attn_kernel, dim3(n, p->num_q_heads), dim3(32), 0, st, false, fp);
  if (e != cudaSuccess) return report_errorf(DSA_ERR_CUDA, "full attention launch: %s", cudaGetErrorString(e));
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_full_attn_workspace_size(const dsa_full_problem* p) {
  if (check_full(p)) return 0;
  return 256;
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
