// Attention of a few drafted tokens per sequence (a tree; one token is the
// decode step) over the 8-bit paged cache.  One block per (sequence, token,
// query head): four warps take every fourth key, lanes hold the query and the
// running value sum, and the four partial softmaxes are merged at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "sm100_common.cuh"
#include "tq_internal.h"

namespace tqi {
namespace {

using namespace sm100;

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(__half* p, float x) { *p = __float2half_rn(x); }

template <typename T>
__global__ void __launch_bounds__(128) tree_rows_kernel(TreeArgs a) {
  __shared__ float sm[4][258];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hq = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq % a.n, b = blockIdx.x / a.Hq / a.n;
  const int hk = hq / (a.Hq / a.Hkv);
  const int drafts = a.draft_lens ? min(max(a.draft_lens[b], 0), a.n) : a.n;
  if (i >= drafts) return;
  const int64_t cap = (int64_t)a.max_pages * a.page;
  const int64_t ctx = max(a.ctx_lens[b], 0), end = min(ctx + drafts, cap);
  if (threadIdx.x == 0 && (a.ctx_lens[b] < 0 || ctx + drafts > cap || (a.draft_lens && a.draft_lens[b] != drafts)))
    atomicOr(a.status, kStatusRange);
  const int32_t* table = a.block_table + ((int64_t)b * a.Hkv + hk) * a.max_pages;
  const int64_t pages = a.rows / a.page;
  const int words = (a.n + 31) / 32;
  const T* q = static_cast<const T*>(a.q) + ((int64_t)b * a.n + i) * a.q_stride + (int64_t)hq * a.d;
  float qv[8], acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) qv[e] = lane + 32 * e < a.d ? to_float(q[lane + 32 * e]) : 0.f, acc[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t t = warp; t < end; t += 4) {
    if (t >= ctx) {
      const int j = (int)(t - ctx);
      const bool sees = a.mask ? (a.mask[((int64_t)b * a.n + i) * words + (j >> 5)] >> (j & 31)) & 1u : j <= i;
      if (!sees) continue;
    }
    const int page = table[t / a.page];
    if (page < 0 || page >= pages) {
      if (lane == 0) atomicOr(a.status, kStatusRange);
      continue;
    }
    const int64_t row = (int64_t)page * a.page + t % a.page;
    const int8_t* kc = a.kcodes + row * a.d;
    const int8_t* vc = a.vcodes + row * a.d;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (lane + 32 * e < a.d) s = fmaf(qv[e], (float)kc[lane + 32 * e], s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= a.scale_log2 * a.kscales[row];
    if (s > m || s != s) {
      const float alpha = exp2f(m - s);
      l *= alpha;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= alpha;
      m = s;
    }
    const float p = m == -INFINITY ? 0.f : exp2f(s - m);
    l += p;
    const float w = p * a.vscales[row];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (lane + 32 * e < a.d) acc[e] = fmaf(w, (float)vc[lane + 32 * e], acc[e]);
  }
  if (lane == 0) sm[warp][256] = m, sm[warp][257] = l;
#pragma unroll
  for (int e = 0; e < 8; ++e) sm[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  float M = -INFINITY;
  bool nan = false;
  for (int w = 0; w < 4; ++w) {
    nan |= sm[w][256] != sm[w][256];
    M = fmaxf(M, sm[w][256]);
  }
  float L = 0.f, f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w][256] == -INFINITY ? 0.f : exp2f(sm[w][256] - M);
    L += sm[w][257] * f[w];
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t row = ((int64_t)b * a.n + i) * a.Hq + hq;
  for (int e = threadIdx.x; e < a.d; e += 128) {
    float o = 0.f;
    for (int w = 0; w < 4; ++w)
      if (f[w] != 0.f) o = fmaf(sm[w][e], f[w], o);
    from_float(static_cast<T*>(a.out) + row * a.d + e, o * inv);
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace

size_t tree_workspace(const tq_ctx*, int, int, int, int) { return 0; }

int launch_tree(const tq_ctx*, const TreeArgs& a, int dtype, void* workspace, void* stream) {
  (void)workspace;
  const unsigned grid = (unsigned)(a.B * a.n * a.Hq);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == TQ_BF16)
    tree_rows_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
  else
    tree_rows_kernel<__half><<<grid, 128, 0, st>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace tqi

using namespace tqi;

extern "C" size_t tq_attn_tree_workspace(tq_handle h, int B, int n, int Hq, int Hkv) {
  if (!h || h->variant != TQ_KV8 || B < 0 || n < 0 || Hq < 0 || Hkv <= 0) return 0;
  return tree_workspace(h, B, n, Hq, Hkv);
}

extern "C" int tq_attn_tree(tq_handle h, const void* q, int dtype, int64_t q_stride, int B, int n, int Hq, int Hkv,
                            const int32_t* ctx_lens, const int32_t* draft_lens, const uint32_t* mask,
                            const int32_t* block_table, int max_pages, int page_size, const int8_t* kcodes,
                            const float* kscales, const int8_t* vcodes, const float* vscales, int64_t rows, float scale,
                            void* out, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  TQ_TRACE("tq_attn_tree");
  const char* fn = "tq_attn_tree";
  if (!h) return set_error(TQ_EINVAL, "%s: NULL handle", fn);
  if (h->variant != TQ_KV8) return set_error(TQ_EINVAL, "%s: need a TQ_KV8 handle", fn);
  if (dtype != TQ_BF16 && dtype != TQ_F16) return set_error(TQ_EUNSUPPORTED, "%s: dtype %d (need TQ_BF16 or TQ_F16)", fn, dtype);
  if (B < 0 || n < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv != 0)
    return set_error(TQ_EINVAL, "%s: bad shape (B=%d n=%d Hq=%d Hkv=%d)", fn, B, n, Hq, Hkv);
  if (n > TQ_MAX_DRAFT) return set_error(TQ_EUNSUPPORTED, "%s: n = %d drafted tokens (at most %d)", fn, n, TQ_MAX_DRAFT);
  if (B > TQ_MAX_SEQS) return set_error(TQ_EUNSUPPORTED, "%s: B = %d (at most %d)", fn, B, TQ_MAX_SEQS);
  if ((int64_t)B * n * Hq > INT32_MAX / 256 || (int64_t)B * Hkv > INT32_MAX / 256)
    return set_error(TQ_EUNSUPPORTED, "%s: B n Hq = %lld rows", fn, (long long)B * n * Hq);
  if (page_size < 8 || page_size % 8 != 0 || max_pages < 1 || (int64_t)max_pages * page_size > INT32_MAX - 4096)
    return set_error(TQ_EINVAL, "%s: page_size %d (need a multiple of 8), max_pages %d", fn, page_size, max_pages);
  if (rows < 0) return set_error(TQ_EINVAL, "%s: rows < 0", fn);
  if (rows > INT32_MAX - 4096) return set_error(TQ_EUNSUPPORTED, "%s: more than 2^31 - 4097 cache rows", fn);
  if (!std::isfinite(scale) || scale < 0.f) return set_error(TQ_EINVAL, "%s: scale is negative or not finite", fn);
  if (B == 0 || n == 0 || Hq == 0) return clear_error();
  if ((int64_t)B * n > 1 && (q_stride < (int64_t)Hq * h->d || q_stride % 8 != 0))
    return set_error(TQ_EINVAL, "%s: q_stride %lld (need >= Hq d and a multiple of 8)", fn, (long long)q_stride);
  if (!q || !ctx_lens || !block_table || !kcodes || !kscales || !vcodes || !vscales || !out)
    return set_error(TQ_EINVAL, "%s: NULL pointer", fn);
  for (const void* p : {q, (const void*)ctx_lens, (const void*)draft_lens, (const void*)mask, (const void*)block_table,
                        (const void*)kcodes, (const void*)kscales, (const void*)vcodes, (const void*)vscales,
                        (const void*)out, (const void*)lse, (const void*)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return set_error(TQ_EALIGN, "%s: a device pointer is not 16-byte aligned", fn);
  const size_t need = tree_workspace(h, B, n, Hq, Hkv);
  if (need && (!workspace || ws_bytes < need))
    return set_error(TQ_EWORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  TreeArgs a{};
  a.q = q, a.q_stride = q_stride, a.B = B, a.n = n, a.Hq = Hq, a.Hkv = Hkv, a.d = h->d;
  a.ctx_lens = ctx_lens, a.draft_lens = draft_lens, a.mask = mask, a.block_table = block_table;
  a.max_pages = max_pages, a.page = page_size;
  a.kcodes = kcodes, a.kscales = kscales, a.vcodes = vcodes, a.vscales = vscales, a.rows = rows;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = out, a.lse = lse, a.status = h->dev.status;
  DeviceGuard guard(h->device);
  const int e = guard.error ? guard.error : launch_tree(h, a, dtype, workspace, stream);
  return e ? set_error(TQ_ECUDA, "%s: %s", fn, cudaGetErrorString((cudaError_t)e)) : clear_error();
}
