// The 8-bit paged K/V cache: rows quantized as they are written, and read back.
//
// The cache of the newest and the drafted tokens, which come and go faster
// than a rotation and a codebook pay for (ttakun.com/news/45354,
// 新旧量化方案深度权衡矩阵: each token is compressed as it arrives; tmdm.cn, 实测数据:
// only the KV store and load change).  A row (one token of one kv-head) is
//   s = max_j |x_j| / 127 (float32),  c_j = x_j / s rounded to the nearest
//   integer (ties to even), kept in [-127, 127],
// and stands for c_j s.  Codes are exactly those of the quotient by the stored
// s: a first guess x (1/s) can only miss by one next to a tie, and the exact
// remainder x - c s (one fused multiply-add: x and c s are multiples of half
// an ulp of s, and their difference is at most about s / 2, so it has 24 bits)
// decides there.  A row that holds an infinity or a NaN has no such codes: it
// gets s = NaN and codes 0, so that what reads it gets NaN in that row alone.
//
// Reading is bound by HBM, writing by its instructions (16 an element, issue slots
// 70 % busy): d e + d + 4 bytes a row and tensor, plus 8 of the slot list (e: bytes of
// an element of x).  A thread takes two pieces of eight elements, `lanes` pieces
// apart, so that neighbouring lanes read and write neighbouring 16 (or 8) bytes, of
// each of two rows, whose loads are in flight together; what a row needs once (its
// maximum, its scale, 1 / s) is spread over sixteen elements.  65537 tokens of 8
// kv-heads, d = 128, bf16 (keys and values) are written in 87 us, 4730 GB/s of 6560
// (99 with the threads of a row and the heads not known to the compiler or divided
// beforehand; with one, four or eight rows a thread 1.1 to 1.8 times as long); 2^20
// rows are read in 143 us, 5750 GB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <initializer_list>
#include <new>

#include "sm100_common.cuh"
#include "tq_internal.h"

namespace tqi {
namespace {

using namespace sm100;

constexpr int kThreads = 128;
constexpr int kRowsPerThread = 2;

struct Kv8Args {
  const void* x[2];        // write: keys, values; read: unused
  void* out[2];            // read: keys, values
  int8_t* codes[2];
  float* scales[2];
  const int64_t* slots;
  int64_t x_stride[2];     // elements from one token to the next
  int64_t N;               // rows: tokens x heads
  int64_t rows;            // rows of the cache
  int Hkv, d;
  uint32_t hkv_mul;        // n / Hkv = n hkv_mul >> hkv_shift for n < 2^31
  int hkv_shift;
  int* status;
};

// eight elements as they lie in memory
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  return r;
}

template <typename T>
__device__ __forceinline__ Raw<T> zero_raw() {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = make_uint4(0u, 0u, 0u, 0u);
  return r;
}

__device__ __forceinline__ void floats_of(const Raw<float>& r, float (&v)[8]) {
  const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}

__device__ __forceinline__ void floats_of(const Raw<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void floats_of(const Raw<__half>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// the largest |x| seen, ordered by its bits (an infinity or a NaN comes out on
// top): of 32-bit elements in the whole word, of 16-bit ones in both halves
__device__ __forceinline__ uint32_t raw_max(const Raw<float>& r, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m = max(m, max(r.w[i].x & 0x7FFFFFFFu, r.w[i].y & 0x7FFFFFFFu));
    m = max(m, max(r.w[i].z & 0x7FFFFFFFu, r.w[i].w & 0x7FFFFFFFu));
  }
  return m;
}
template <typename T>
__device__ __forceinline__ uint32_t raw_max(const Raw<T>& r, uint32_t m) {
  m = __vmaxu2(m, __vmaxu2(r.w[0].x & 0x7FFF7FFFu, r.w[0].y & 0x7FFF7FFFu));
  return __vmaxu2(m, __vmaxu2(r.w[0].z & 0x7FFF7FFFu, r.w[0].w & 0x7FFF7FFFu));
}

// that maximum as a float32's bits
template <typename T>
__device__ __forceinline__ uint32_t max_bits(uint32_t m);
template <>
__device__ __forceinline__ uint32_t max_bits<float>(uint32_t m) { return m; }
template <>
__device__ __forceinline__ uint32_t max_bits<__nv_bfloat16>(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }
template <>
__device__ __forceinline__ uint32_t max_bits<__half>(uint32_t m) {
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)max(m & 0xFFFFu, m >> 16))));
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it leaves the nearest integer in the low bits

// m / 127, correctly rounded: the product by 1/127 and one correction by its
// remainder (Brisebarre, Muller and Raina's division by a known divisor, 2004;
// checked for every significand; subnormal results take the division)
__device__ __forceinline__ float scale_of(float m) {
  if (m < 0x1p-100f) return __fdiv_rn(m, 127.f);
  constexpr float c = 1.f / 127.f;
  const float q = m * c;
  return fmaf(fmaf(-q, 127.f, m), c, q);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// the code of x for scale s > 0: x / s to the nearest integer, ties to even
__device__ __forceinline__ int exact_code(float x, float s, float guess) {
  float q = fminf(fmaxf(guess, -127.f), 127.f);
  const float r = fmaf(-q, s, x);
  const float twice = fabsf(r) + fabsf(r);
  if (twice > s || (twice == s && ((int)q & 1))) q += r > 0.f ? 1.f : -1.f;
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// eight codes, one in the low byte of each word
__device__ __forceinline__ void codes_of(const float (&v)[8], float s, uint32_t (&c)[8]) {
  if (s >= 0x1p-80f) {
    const float inv = rcp_approx(s);
    float off = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = fmaf(v[e], inv, kMagic);
      c[e] = __float_as_uint(g);
      off = fmaxf(off, fabsf(fmaf(-(g - kMagic), s, v[e])));
    }
    // within just under half a step each: the guesses, off by 2^-15 of a step at
    // most, cannot have crossed a border
    if (off <= 0.4999f * s) return;
    // 16-bit inputs meet exact ties often (x / s = 127 x / max, a ratio of small
    // integers): one step towards the remainder r where |r| > s/2, or |r| = s/2
    // and the code is odd, that is |r| > the float before s/2
    const uint32_t half = __float_as_uint(0.5f * s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = fmaf(-(__uint_as_float(c[e]) - kMagic), s, v[e]);
      if (fabsf(r) > __uint_as_float(half - (c[e] & 1u))) c[e] += 1u | (uint32_t)(__float_as_int(r) >> 31);
    }
  } else {
    // 1/s would leave float32's range: the guess from both scaled up
    const float inv = rcp_approx(s * 0x1p100f);
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = (uint32_t)exact_code(v[e], s, rintf(v[e] * 0x1p100f * inv));
  }
}

// lanes: threads of a row (a power of two >= d / 16), so that a row never
// crosses a warp; pieces past d / 8 only take part in the shuffles
template <typename T, int lanes>
__global__ void __launch_bounds__(kThreads) kv8_write_kernel(Kv8Args a) {
  const int which = blockIdx.y;
  const int sub = threadIdx.x & (lanes - 1);
  const int groups = kThreads / lanes;
  const bool on[2] = {sub * 8 < a.d, (sub + lanes) * 8 < a.d};
  const T* x = static_cast<const T*>(which ? a.x[1] : a.x[0]);
  const int64_t x_stride = which ? a.x_stride[1] : a.x_stride[0];
  int8_t* codes = which ? a.codes[1] : a.codes[0];
  float* scales = which ? a.scales[1] : a.scales[0];
  const int64_t r0 = (int64_t)blockIdx.x * (groups * kRowsPerThread) + threadIdx.x / lanes;
  Raw<T> raw[kRowsPerThread][2];
  int64_t slot[kRowsPerThread];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int64_t n = r0 + (int64_t)i * groups;
    slot[i] = -1;
    raw[i][0] = raw[i][1] = zero_raw<T>();
    if (n < a.N) {
      slot[i] = __ldg(a.slots + n);
      const uint32_t t = (uint32_t)((uint64_t)(uint32_t)n * a.hkv_mul >> a.hkv_shift), h = (uint32_t)n - t * (uint32_t)a.Hkv;
      const T* row = x + (int64_t)t * x_stride + (int64_t)h * a.d;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (on[k]) raw[i][k] = load_raw(row + (sub + k * lanes) * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    uint32_t top = max_bits<T>(raw_max(raw[i][1], raw_max(raw[i][0], 0u)));
#pragma unroll
    for (int m = lanes >> 1; m; m >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    const bool finite = top < 0x7F800000u;
    const float s = finite ? scale_of(__uint_as_float(top)) : __uint_as_float(0x7FC00000u);
    const bool kept = slot[i] >= 0 && slot[i] < a.rows;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v[8];
      uint32_t c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      floats_of(raw[i][k], v);
      if (finite && s > 0.f) codes_of(v, s, c);
      if (kept && on[k]) {
        uint2 w;
        w.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        w.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
        *reinterpret_cast<uint2*>(codes + slot[i] * a.d + (sub + k * lanes) * 8) = w;
      }
    }
    if (sub == 0) {
      if (kept) scales[slot[i]] = s;
      else if (slot[i] >= a.rows) atomicOr(a.status, kStatusRange);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(Kv8Args a, int lanes) {
  const int which = blockIdx.y;
  const int sub = threadIdx.x & (lanes - 1);
  const int groups = kThreads / lanes;
  const bool on[2] = {sub * 8 < a.d, (sub + lanes) * 8 < a.d};
  T* out = static_cast<T*>(which ? a.out[1] : a.out[0]);
  const int8_t* codes = which ? a.codes[1] : a.codes[0];
  const float* scales = which ? a.scales[1] : a.scales[0];
  const int64_t r0 = (int64_t)blockIdx.x * (groups * kRowsPerThread) + threadIdx.x / lanes;
  int64_t slot[kRowsPerThread];
  uint2 w[kRowsPerThread][2];
  float s[kRowsPerThread];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int64_t n = r0 + (int64_t)i * groups;
    slot[i] = n < a.N ? __ldg(a.slots + n) : -1;
  }
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    w[i][0] = w[i][1] = make_uint2(0u, 0u);
    s[i] = 0.f;
    if (slot[i] >= 0 && slot[i] < a.rows) {
      const int8_t* row = codes + slot[i] * a.d;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (on[k]) w[i][k] = __ldg(reinterpret_cast<const uint2*>(row + (sub + k * lanes) * 8));
      s[i] = __ldg(scales + slot[i]);
    } else if (slot[i] >= a.rows && sub == 0) {
      atomicOr(a.status, kStatusRange);
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int64_t n = r0 + (int64_t)i * groups;
    if (n >= a.N) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!on[k]) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // a code + 128 in the low byte of 2^23: the conversion is one subtraction
        const uint32_t word = (e < 4 ? w[i][k].x : w[i][k].y) ^ 0x80808080u;
        v[e] = (__uint_as_float(__byte_perm(word, 0x4B000000u, 0x7650u + (e & 3))) - 8388736.f) * s[i];
      }
      store8(out + n * a.d + (sub + k * lanes) * 8, v);
    }
  }
}

int lanes_of(int d) {
  int l = 1;
  while (l * 16 < d) l *= 2;
  return l;
}

}  // namespace

int launch_kv8_write(const tq_ctx* h, const void* k, const void* v, int dtype, int64_t n, int Hkv, int64_t k_stride,
                     int64_t v_stride, const int64_t* slots, int8_t* kcodes, float* kscales, int8_t* vcodes,
                     float* vscales, int64_t rows, void* stream) {
  Kv8Args a{};
  a.x[0] = k, a.x[1] = v;
  a.codes[0] = kcodes, a.codes[1] = vcodes;
  a.scales[0] = kscales, a.scales[1] = vscales;
  a.slots = slots;
  a.x_stride[0] = k_stride, a.x_stride[1] = v_stride;
  a.N = n * Hkv, a.rows = rows, a.Hkv = Hkv, a.d = h->d, a.status = h->dev.status;
  // Granlund and Montgomery's division by an invariant integer: ceil(2^shift / Hkv), 2^(shift - 31) >= Hkv
  a.hkv_shift = 31;
  while ((1ll << (a.hkv_shift - 31)) < Hkv) ++a.hkv_shift;
  a.hkv_mul = (uint32_t)(((1ull << a.hkv_shift) + Hkv - 1) / (uint64_t)Hkv);
  const int lanes = lanes_of(h->d), per = kThreads / lanes * kRowsPerThread;
  const dim3 grid((unsigned)((a.N + per - 1) / per), v ? 2 : 1);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto launch = [&](auto type) {
    using T = decltype(type);
    switch (lanes) {
      case 1: kv8_write_kernel<T, 1><<<grid, kThreads, 0, st>>>(a); break;
      case 2: kv8_write_kernel<T, 2><<<grid, kThreads, 0, st>>>(a); break;
      case 4: kv8_write_kernel<T, 4><<<grid, kThreads, 0, st>>>(a); break;
      case 8: kv8_write_kernel<T, 8><<<grid, kThreads, 0, st>>>(a); break;
      default: kv8_write_kernel<T, 16><<<grid, kThreads, 0, st>>>(a);
    }
  };
  if (dtype == TQ_F32) launch(float());
  else if (dtype == TQ_BF16) launch(__nv_bfloat16());
  else launch(__half());
  return (int)cudaGetLastError();
}

int launch_kv8_read(const tq_ctx* h, int64_t N, const int64_t* slots, const int8_t* kcodes, const float* kscales,
                    const int8_t* vcodes, const float* vscales, int64_t rows, void* k, void* v, int dtype,
                    void* stream) {
  Kv8Args a{};
  a.out[0] = k, a.out[1] = v;
  a.codes[0] = const_cast<int8_t*>(kcodes), a.codes[1] = const_cast<int8_t*>(vcodes);
  a.scales[0] = const_cast<float*>(kscales), a.scales[1] = const_cast<float*>(vscales);
  a.slots = slots;
  a.N = N, a.rows = rows, a.Hkv = 1, a.d = h->d, a.status = h->dev.status;
  const int lanes = lanes_of(h->d), per = kThreads / lanes * kRowsPerThread;
  const dim3 grid((unsigned)((a.N + per - 1) / per), v ? 2 : 1);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == TQ_F32)
    kv8_read_kernel<float><<<grid, kThreads, 0, st>>>(a, lanes);
  else if (dtype == TQ_BF16)
    kv8_read_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, lanes);
  else
    kv8_read_kernel<__half><<<grid, kThreads, 0, st>>>(a, lanes);
  return (int)cudaGetLastError();
}

}  // namespace tqi

using namespace tqi;

namespace {

// the checks of the cache arrays that both directions share
int check_kv8(const char* fn, int64_t rows, const void* kcodes, const void* kscales, const void* vcodes,
              const void* vscales, bool values) {
  if (rows < 0) return set_error(TQ_EINVAL, "%s: rows < 0", fn);
  // arrays of no rows need no address: no slot lies in them
  if (rows > 0 && (!kcodes || !kscales || (values && (!vcodes || !vscales)))) return set_error(TQ_EINVAL, "%s: NULL pointer", fn);
  return TQ_OK;
}

int check_aligned(const char* fn, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15u)
      return set_error(TQ_EALIGN, "%s: a device pointer is not 16-byte aligned", fn);
  return TQ_OK;
}

}  // namespace

extern "C" int tq_create_kv8(tq_handle* out, int d) {
  TQ_TRACE("tq_create_kv8");
  if (!out) return set_error(TQ_EINVAL, "tq_create_kv8: NULL handle");
  *out = nullptr;
  if (d < 16 || d > 256 || d % 16 != 0)
    return set_error(TQ_EUNSUPPORTED, "tq_create_kv8: d = %d (need 16 <= d <= 256, d %% 16 == 0)", d);
  tq_ctx* h = new (std::nothrow) tq_ctx();
  if (!h) return set_error(TQ_ENOMEM, "tq_create_kv8: out of host memory");
  h->d = d, h->b = 8, h->bm = 8, h->variant = TQ_KV8;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) {
    h->block_bytes = 256;
    e = cudaMalloc(&h->block, h->block_bytes);
    if (e == cudaSuccess) e = cudaMemset(h->block, 0, h->block_bytes);
    // a memset does not wait, and other streams do not wait for it: without this it could
    // clear what the first call on one of them reports
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
    h->dev.status = static_cast<int*>(h->block);
  }
  if (e != cudaSuccess) {
    if (h->block) cudaFree(h->block);
    delete h;
    return set_error(e == cudaErrorMemoryAllocation ? TQ_ENOMEM : TQ_ECUDA, "tq_create_kv8: %s", cudaGetErrorString(e));
  }
  *out = h;
  return clear_error();
}

extern "C" int tq_quant_kv8(tq_handle h, const void* k, const void* v, int dtype, int64_t n, int Hkv,
                            int64_t k_stride, int64_t v_stride, const int64_t* slots, int8_t* kcodes, float* kscales,
                            int8_t* vcodes, float* vscales, int64_t rows, void* stream) {
  TQ_TRACE("tq_quant_kv8");
  const char* fn = "tq_quant_kv8";
  if (!h) return set_error(TQ_EINVAL, "%s: NULL handle", fn);
  if (h->variant != TQ_KV8) return set_error(TQ_EINVAL, "%s: need a TQ_KV8 handle", fn);
  if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return set_error(TQ_EUNSUPPORTED, "%s: dtype %d", fn, dtype);
  if (n < 0 || Hkv < 1) return set_error(TQ_EINVAL, "%s: n = %lld, Hkv = %d", fn, (long long)n, Hkv);
  if (n > INT32_MAX / Hkv) return set_error(TQ_EUNSUPPORTED, "%s: more than 2^31 - 1 rows", fn);
  const int unit = dtype == TQ_F32 ? 4 : 8;  // elements in 16 bytes
  for (const int64_t s : {k_stride, v ? v_stride : k_stride})
    if (n > 1 && (s < (int64_t)Hkv * h->d || s % unit != 0))
      return set_error(TQ_EINVAL, "%s: stride %lld (need >= Hkv d and a multiple of 16 bytes)", fn, (long long)s);
  if (n == 0) return clear_error();
  if (!k || !slots) return set_error(TQ_EINVAL, "%s: NULL pointer", fn);
  int rc = check_kv8(fn, rows, kcodes, kscales, vcodes, vscales, v != nullptr);
  if (!rc) rc = check_aligned(fn, {k, v, slots, kcodes, kscales, vcodes, vscales});
  if (rc) return rc;
  DeviceGuard guard(h->device);
  const int e = guard.error ? guard.error
                            : launch_kv8_write(h, k, v, dtype, n, Hkv, k_stride, v_stride, slots, kcodes, kscales,
                                               vcodes, vscales, rows, stream);
  return e ? set_error(TQ_ECUDA, "%s: %s", fn, cudaGetErrorString((cudaError_t)e)) : clear_error();
}

extern "C" int tq_dequant_kv8(tq_handle h, int64_t n, const int64_t* slots, const int8_t* kcodes,
                              const float* kscales, const int8_t* vcodes, const float* vscales, int64_t rows, void* k,
                              void* v, int out_dtype, void* stream) {
  TQ_TRACE("tq_dequant_kv8");
  const char* fn = "tq_dequant_kv8";
  if (!h) return set_error(TQ_EINVAL, "%s: NULL handle", fn);
  if (h->variant != TQ_KV8) return set_error(TQ_EINVAL, "%s: need a TQ_KV8 handle", fn);
  if (out_dtype != TQ_F32 && out_dtype != TQ_BF16 && out_dtype != TQ_F16)
    return set_error(TQ_EUNSUPPORTED, "%s: out_dtype %d", fn, out_dtype);
  if (n < 0) return set_error(TQ_EINVAL, "%s: n < 0", fn);
  if (n > INT32_MAX) return set_error(TQ_EUNSUPPORTED, "%s: more than 2^31 - 1 rows", fn);
  if (n == 0) return clear_error();
  if (!k || !slots) return set_error(TQ_EINVAL, "%s: NULL pointer", fn);
  int rc = check_kv8(fn, rows, kcodes, kscales, vcodes, vscales, v != nullptr);
  if (!rc) rc = check_aligned(fn, {k, v, slots, kcodes, kscales, vcodes, vscales});
  if (rc) return rc;
  DeviceGuard guard(h->device);
  const int e = guard.error ? guard.error
                            : launch_kv8_read(h, n, slots, kcodes, kscales, vcodes, vscales, rows, k, v, out_dtype,
                                              stream);
  return e ? set_error(TQ_ECUDA, "%s: %s", fn, cudaGetErrorString((cudaError_t)e)) : clear_error();
}
