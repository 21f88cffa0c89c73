// Causal attention over a whole prompt batch (packed sequences) before anything
// is compressed.  One warp per (token, query head): lanes hold the query and
// the running value sum, keys go by one at a time, with the running maximum and
// sum of the softmax in float32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "sm100_common.cuh"
#include "tq_internal.h"

namespace tqi {
namespace {

struct PromptArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* cu;
  void* out;
  float* lse;
  int64_t total, q_stride, k_stride, v_stride;
  int nseq, Hq, Hkv, d;
  float scale_log2;
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(__half* p, float x) { *p = __float2half_rn(x); }

template <typename T>
__global__ void __launch_bounds__(128) prompt_rows_kernel(PromptArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t t = w / a.Hq;
  const int hq = (int)(w % a.Hq), hk = hq / (a.Hq / a.Hkv);
  if (t >= a.total) return;
  // the sequence of token t: bounds never decrease here, whatever the array holds
  int64_t lo = -1, prev = min((int64_t)max(a.cu[0], 0), a.total);
  for (int s = 0; s < a.nseq; ++s) {
    const int64_t end = max(prev, min((int64_t)a.cu[s + 1], a.total));
    if (t >= prev && t < end) {
      lo = prev;
      break;
    }
    prev = end;
  }
  if (lo < 0) return;
  const T* q = static_cast<const T*>(a.q) + t * a.q_stride + (int64_t)hq * a.d;
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) qv[i] = lane + 32 * i < a.d ? to_float(q[lane + 32 * i]) : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t j = lo; j <= t; ++j) {
    const T* k = static_cast<const T*>(a.k) + j * a.k_stride + (int64_t)hk * a.d;
    const T* v = static_cast<const T*>(a.v) + j * a.v_stride + (int64_t)hk * a.d;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.d) s = fmaf(qv[i], to_float(k[lane + 32 * i]), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= a.scale_log2;
    if (s > m || s != s) {
      const float alpha = exp2f(m - s);
      l *= alpha;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= alpha;
      m = s;
    }
    const float p = m == -INFINITY ? 0.f : exp2f(s - m);
    l += p;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 32 * i < a.d) acc[i] = fmaf(p, to_float(v[lane + 32 * i]), acc[i]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(a.out) + (t * a.Hq + hq) * a.d;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.d) from_float(out + lane + 32 * i, acc[i] * inv);
  if (a.lse && lane == 0) a.lse[t * a.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t prompt_workspace(const tq_ctx*, int, int64_t, int, int) { return 0; }

int launch_prompt(const tq_ctx* h, const void* q, const void* k, const void* v, int dtype, const int32_t* cu, int nseq,
                  int64_t total, int Hq, int Hkv, int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                  void* out, float* lse, void* workspace, void* stream) {
  (void)workspace;
  PromptArgs a{q, k, v, cu, out, lse, total, q_stride, k_stride, v_stride, nseq, Hq, Hkv, h->d, scale * 1.4426950408889634f};
  const unsigned grid = (unsigned)((total * Hq + 3) / 4);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == TQ_BF16)
    prompt_rows_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
  else
    prompt_rows_kernel<__half><<<grid, 128, 0, st>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace tqi

using namespace tqi;

extern "C" size_t tq_attn_prompt_workspace(tq_handle h, int nseq, int64_t total, int Hq, int Hkv) {
  if (!h || nseq < 0 || total < 0 || Hq < 0 || Hkv <= 0) return 0;
  return prompt_workspace(h, nseq, total, Hq, Hkv);
}

extern "C" int tq_attn_prompt(tq_handle h, const void* q, const void* k, const void* v, int dtype,
                              const int32_t* cu_seqlens, int nseq, int64_t total, int Hq, int Hkv, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, float scale, void* out, float* lse, void* workspace,
                              size_t ws_bytes, void* stream) {
  TQ_TRACE("tq_attn_prompt");
  const char* fn = "tq_attn_prompt";
  if (!h) return set_error(TQ_EINVAL, "%s: NULL handle", fn);
  if (h->d > 128) return set_error(TQ_EUNSUPPORTED, "%s: d = %d (need d <= 128)", fn, h->d);
  if (dtype != TQ_BF16 && dtype != TQ_F16) return set_error(TQ_EUNSUPPORTED, "%s: dtype %d (need TQ_BF16 or TQ_F16)", fn, dtype);
  if (nseq < 0 || total < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0)
    return set_error(TQ_EINVAL, "%s: bad shape (nseq=%d total=%lld Hq=%d Hkv=%d)", fn, nseq, (long long)total, Hq, Hkv);
  if (Hq / Hkv > 128) return set_error(TQ_EUNSUPPORTED, "%s: %d query heads per kv-head (at most 128)", fn, Hq / Hkv);
  if (nseq > TQ_MAX_SEQS) return set_error(TQ_EUNSUPPORTED, "%s: nseq = %d (at most %d)", fn, nseq, TQ_MAX_SEQS);
  if (total > INT32_MAX / 128 || total * Hkv > INT32_MAX / 2)
    return set_error(TQ_EUNSUPPORTED, "%s: total = %lld tokens of %d kv-heads", fn, (long long)total, Hkv);
  if (!std::isfinite(scale) || scale < 0.f) return set_error(TQ_EINVAL, "%s: scale is negative or not finite", fn);
  if (nseq == 0 || total == 0 || Hq == 0) return clear_error();
  const int64_t ld[3] = {q_stride, k_stride, v_stride};
  for (int i = 0; i < 3; ++i)
    if (total > 1 && (ld[i] < (int64_t)(i ? Hkv : Hq) * h->d || ld[i] % 8 != 0))
      return set_error(TQ_EINVAL, "%s: stride %lld (need >= heads * d and a multiple of 8)", fn, (long long)ld[i]);
  if (!q || !k || !v || !cu_seqlens || !out) return set_error(TQ_EINVAL, "%s: NULL pointer", fn);
  for (const void* p : {q, k, v, (const void*)cu_seqlens, (const void*)out, (const void*)lse, (const void*)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return set_error(TQ_EALIGN, "%s: a device pointer is not 16-byte aligned", fn);
  const size_t need = prompt_workspace(h, nseq, total, Hq, Hkv);
  if (need && (!workspace || ws_bytes < need))
    return set_error(TQ_EWORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  DeviceGuard guard(h->device);
  const int e = guard.error ? guard.error
                            : launch_prompt(h, q, k, v, dtype, cu_seqlens, nseq, total, Hq, Hkv, q_stride, k_stride,
                                            v_stride, scale, out, lse, workspace, stream);
  return e ? set_error(TQ_ECUDA, "%s: %s", fn, cudaGetErrorString((cudaError_t)e)) : clear_error();
}
