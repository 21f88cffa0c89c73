// Attention of a few drafted tokens per sequence (a tree; one token is the
// decode step) over the 8-bit paged cache, on mma.sync (sm_100a).
//
// turboquant.net/zh, "实现步骤草图", 集成到 attention: decode attention reads the
// compressed cache; the 8-bit rows are c_t s_t (kv8.cu).  With the scales taken
// out of the products,
//   logit_t = scale s_t (q . c_t),  out = sum_t (p_t s'_t) c'_t / sum_t p_t,
// so both products run on the integer codes themselves: exact in 16 bits, the
// scales applied to the float32 logits and to the weights p_t.  Queries enter
// as fp16 (bf16 ones with a power of two per row: their 8 bits fit; what falls
// below fp16's range is under 2^-40 of the row's largest), the weights p s' as
// bf16, whose range holds whatever the scales are, in two terms: rounded once, few
// keys under a row cost 2^-8 beside the result's own rounding (measured on 1000
// keys: 0.0028 of the result, 0.0016 with the remainder's product, the plain
// formula in 64 bits rounded to bf16).  Up to 8 rows the remainders are the other
// half of the 16-row fragment and cost nothing; for 9 to 32 rows they are a second
// product (32 sequences of 4000 tokens, 16 rows: 109 us, 103 without).
//
// A kv-head's rows (drafted token, head of its group) form the M side of the
// products, 8, 16 or 32 rows of a block at a time; keys are the N side of the
// logits and the K side of the value product, so a logit fragment becomes a
// weight fragment in place.  Each of four warps takes 16 of the 64 keys of a
// tile with its own softmax (maximum, sum, value sum in registers), and the four
// are merged when a block is done with a work item.  The order of the d
// coordinates inside a product is free: a lane takes 16 or 32 neighbouring bytes
// of a key, and every 4-byte word is one K step's fragment.
//
// Work items are (sequence, kv-head, block of rows); their 64-key tiles, all
// items behind one another, are cut into equal ranges for a persistent grid,
// whatever the lengths are.  An item that a cut divides leaves softmax records
// in the workspace, at most two a block, which tree_merge_kernel joins.
//
// What bounds it: turning codes into 16-bit pairs and the softmax keep half of the
// issue slots busy; the rest is their latency, with 15 warps an SM.  One token for 8
// sequences of 131072, 8 kv-heads, 4 rows each, pages of 64: 0.529 ms, 4190 GB/s of
// 6560 (0.489 in a loop of nothing but this call over two caches).  At d > 128 blocks
// hold 16 rows at most, so 256 rows read and convert the context 16 times: 64 tokens for
// 4 sequences of 16384, d = 256: 0.97 ms (16 tokens, 64 rows: 0.28; one token for 8
// sequences of 131071: 0.854 ms, 5100 GB/s).
//
// A warp beside them keeps a ring of tiles filled: one TMA load per page piece for
// the codes (rows of 64 or 128 bytes, swizzled so that the lanes' 16-byte reads
// never share a bank), bulk copies for the scales, and a word of valid-key bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_tree.cuh"

namespace tqi {
namespace {

using namespace attn;
using namespace tree;

constexpr int kKeys = 64;            // keys of a tile
constexpr int kWarps = 4;            // consumer warps, 16 keys of a tile each
constexpr int kRegsConsumer = 216, kRegsProducer = 40;   // 216 + 40 = 2 x 128, the registers at launch

// what the shared window holds, by padded dimension and rows of a block
template <int D, int R>
struct Shape {
  static constexpr int rows = R;                           // 8, 16 or 32
  static constexpr int MT = R > 16 ? R / 16 : 1;           // fragments of 16 rows
  static constexpr int HF = R == 8 ? 1 : 2;                // halves of a fragment that hold rows
  static constexpr int slabs = D > 128 ? D / 128 : 1;      // a row's bytes come in slabs of at most 128
  static constexpr int slab_row = D > 128 ? 128 : D;
  static constexpr int codes = kKeys * D;
  static constexpr int stage = 2 * codes;                  // K and V codes (the swizzle repeats every 1024 bytes)
  static constexpr int scales = 2 * kKeys * 4;             // their scales
  static constexpr int ksteps = D / 16;
  // 16 rows of up to 128 (64) coordinates fit 128 (96) registers a thread (with the
  // query fragments in shared memory): three (four) blocks of five warps on an SM.
  // Wider ones take two blocks of two warpgroups, of which the consumers' takes
  // registers that the other, a single warp of which feeds the ring, gives back.
  // 16 sequences of 16000 tokens, 8 kv-heads, 4 rows each: d = 128 149 us (173 with two
  // wide blocks), d = 64 106 us (118 with three slim blocks, 114 with five, 155 wide).
  static constexpr bool slim = R <= 16 && D <= 128;
  static constexpr int blocks_per_sm = slim ? (D == 64 ? 4 : 3) : 2;
  static constexpr int threads = (slim ? kWarps + 1 : 2 * kWarps) * 32;
  static constexpr int stages = D == 256 ? 2 : D == 128 ? (slim ? 3 : 5) : (slim ? 5 : 8);
  static constexpr bool q_in_regs = !slim && MT * ksteps <= 8;
  static constexpr int off_scales = stages * stage;
  static constexpr int off_acc = off_scales + stages * scales;   // [rows][D + 4] merged value sums
  static constexpr int off_q = off_acc + rows * (D + 4) * 4;
  static constexpr int off_ml = off_q + (q_in_regs ? 0 : MT * ksteps * 256 * HF);   // [kWarps][rows] maxima, then sums
  static constexpr int off_bar = off_ml + 2 * kWarps * rows * 4;
  static constexpr int bytes = off_bar + 512 + 1024;
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// four int8 codes -> two fp16 pairs: a byte b + 128 under 0x64 is 1024 + 128 + b
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));
  uint32_t p = prmt(x, 0x64646464u, 0x4140u), q = prmt(x, 0x64646464u, 0x4342u);
  __half2 r = __hsub2(*reinterpret_cast<__half2*>(&p), bias), t = __hsub2(*reinterpret_cast<__half2*>(&q), bias);
  lo = *reinterpret_cast<uint32_t*>(&r);
  hi = *reinterpret_cast<uint32_t*>(&t);
}

// byte j of a and of b (two keys, the same coordinate) -> a bf16 pair: the low
// seven bits under 0x43 are 128 + them, the sign bit alone 128 or 256
__device__ __forceinline__ uint32_t codes_bf16(uint32_t a, uint32_t b, int j) {
  const uint32_t t = prmt(a, b, (uint32_t)(j * 0x0011 + (j + 4) * 0x1100));
  const uint32_t m = (t & 0x007F007Fu) | 0x43004300u, s = (t & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&s));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <typename T>
__device__ __forceinline__ void store_pair(T* p, float x, float y);
template <>
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}
template <>
__device__ __forceinline__ void store_pair(__half* p, float x, float y) {
  *reinterpret_cast<__half2*>(p) = __floats2half2_rn(x, y);
}

// 32 bits of q as an fp16 pair times f (a power of two)
template <typename T>
__device__ __forceinline__ uint32_t q_pair(uint32_t w, float f);
template <>
__device__ __forceinline__ uint32_t q_pair<__nv_bfloat16>(uint32_t w, float f) {
  const __half2 r = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t q_pair<__half>(uint32_t w, float) { return w; }

template <int D, int R, typename T>
__global__ void __launch_bounds__(Shape<D, R>::threads, Shape<D, R>::blocks_per_sm)
tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, TreeArgs a, int box,
            float* records, Cut* cuts) {
  using S = Shape<D, R>;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int MT = S::MT, HF = S::HF;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::off_bar);
  uint64_t* empty = full + S::stages;
  uint64_t* valid = empty + S::stages;                    // per stage: bit k = key k is there
  int64_t* found = reinterpret_cast<int64_t*>(valid + S::stages);   // scratch of range_of_block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.launch_dependents;");       // the merge may set itself up
  Walk<kKeys> walk;
  if (!range_of_block<kKeys, S::threads>(a, S::rows, found, walk)) {
    if (threadIdx.x == 0 && cuts) cuts[blockIdx.x].begin = -1;
    return;
  }
  Piece p;

  if (warp >= kWarps) {
    // ---------------- producer
    if constexpr (!S::slim) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsProducer));
    if (warp > kWarps) return;
    const int64_t pages = a.rows / a.page;
    const int boxes = kKeys / box;
    int it = 0;
    bool ok = true;
    while (ok && walk.next(a, S::rows, p)) {
      const int32_t* table = a.block_table + ((int64_t)p.b * a.Hkv + p.h) * a.max_pages;
      // lane i: piece i of a tile; its page id is read one tile ahead
      auto row_of = [&](int tile) -> int {
        const int t = tile * kKeys + lane * box;
        if (lane >= boxes || tile >= p.hi || t >= p.s.T) return -1;
        const int id = __ldg(table + t / a.page);
        if (id < 0 || id >= pages) {
          atomicOr(a.status, kStatusRange);
          return -1;
        }
        return id * a.page + t % a.page;
      };
      int row = row_of(p.lo);
      for (int tile = p.lo; tile < p.hi; ++tile, ++it) {
        const int s = it % S::stages;
        const int next = row_of(tile + 1);
        if (!wait_warp(&empty[s], (uint32_t)(((it / S::stages) & 1) ^ 1))) {
          ok = false;
          break;
        }
        const uint32_t live = __ballot_sync(kFull, row >= 0);
        if (lane == 0) {
          uint64_t bits = 0;
          const uint64_t piece = box == 64 ? ~0ull : (1ull << box) - 1;
          for (int i = 0; i < boxes; ++i)
            if (live >> i & 1) bits |= piece << (i * box);
          const int left = p.s.T - tile * kKeys;
          if (left < kKeys) bits &= (1ull << left) - 1;
          valid[s] = bits;
          mbar_arrive_expect_tx(&full[s], (uint32_t)(__popc(live) * box * 2 * (D + 4)));
        }
        __syncwarp();
        if (row >= 0) {
          uint8_t* st = smem + s * S::stage;
#pragma unroll
          for (int sl = 0; sl < S::slabs; ++sl) {
            const int at = sl * kKeys * S::slab_row + lane * box * S::slab_row;
            tma_load_2d(&kmap, &full[s], st + at, sl * 128, row);
            tma_load_2d(&vmap, &full[s], st + S::codes + at, sl * 128, row);
          }
          uint8_t* sc = smem + S::off_scales + s * S::scales + lane * box * 4;
          bulk_load(sc, a.kscales + row, box * 4, &full[s]);
          bulk_load(sc + kKeys * 4, a.vscales + row, box * 4, &full[s]);
        }
        row = next;
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.status, kStatusTimeout);
      // no copy may still be in flight when the block ends
      for (int i = it > S::stages ? it - S::stages : 0; i < it; ++i)
        wait(&full[i % S::stages], (uint32_t)((i / S::stages) & 1));
    }
    return;
  }

  // ---------------- consumers
  if constexpr (!S::slim) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsConsumer));
  const int g = lane >> 2, c = lane & 3;
  const int G = a.Hq / a.Hkv;
  const uint32_t ring = smem_u32(smem);
  float* acc_sm = reinterpret_cast<float*>(smem + S::off_acc);
  const uint32_t qbase = smem_u32(smem) + S::off_q;
  float* ml = reinterpret_cast<float*>(smem + S::off_ml);
  int it = 0, kept = 0;
  bool ok = true;
  while (walk.next(a, S::rows, p)) {
    const int live_rows = p.s.drafts * G - p.rb * S::rows;   // rows of the block that exist (may pass S::rows)
    // queries: fragments of rows (token, head) = divmod(row, G), scaled by a power of two each
    uint32_t qf[S::q_in_regs ? MT : 1][S::q_in_regs ? S::ksteps : 1][4];
    float rowf[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      constexpr int kChunks = D / 32;                        // 16-byte chunks of a lane's coordinates in a row
      uint4 raw[HF][kChunks];
      float f[HF];
#pragma unroll
      for (int hf = 0; hf < HF; ++hf) {
        const int r = mt * 16 + hf * 8 + g;
        const bool live = r < live_rows;
        const int x = p.rb * S::rows + r, tok = x / G, hd = x % G;
        const T* q = static_cast<const T*>(a.q) + ((int64_t)p.b * a.n + (live ? tok : 0)) * a.q_stride +
                     (int64_t)(p.h * G + (live ? hd : 0)) * a.d;
        uint32_t mx = 0;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          // lane c's bytes of a key: D <= 128: c * D/4 ..; above, c * 32 .. of every slab
          const int e = D <= 128 ? c * (D / 4) + 8 * k : (k >> 2) * 128 + c * 32 + 8 * (k & 3);
          raw[hf][k] = live && e < a.d ? __ldg(reinterpret_cast<const uint4*>(q + e)) : make_uint4(0u, 0u, 0u, 0u);
          if (!kHalf) {
            const uint32_t w[4] = {raw[hf][k].x, raw[hf][k].y, raw[hf][k].z, raw[hf][k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = max(mx, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
          }
        }
        f[hf] = 1.f;
        if (!kHalf) {
          mx = max(mx, __shfl_xor_sync(kFull, mx, 1));
          mx = max(mx, __shfl_xor_sync(kFull, mx, 2));
          // the largest of the row at 2^14 .. 2^15; 2^127 at most either way (rows of zeros or subnormals, infinities)
          const int ex = min(max((int)(mx >> 23) - 127, -112), 126);
          f[hf] = __uint_as_float((uint32_t)(127 + min(14 - ex, 126)) << 23);
        }
        rowf[mt][hf] = a.scale_log2 / f[hf];
      }
      if (!S::q_in_regs) {
        if (mt == 0) named_bar_sync(1, kWarps * 32);         // the piece before is done with its fragments
      }
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint32_t lo[4] = {raw[0][k].x, raw[0][k].y, raw[0][k].z, raw[0][k].w};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a0 = q_pair<T>(lo[2 * j], f[0]), a2 = q_pair<T>(lo[2 * j + 1], f[0]);
          const int at = (mt * S::ksteps + 2 * k + j) * 32 + lane;
          if constexpr (HF == 1) {
            if (warp == mt) reinterpret_cast<uint2*>(smem + S::off_q)[at] = make_uint2(a0, a2);
          } else {
            const uint32_t hi[4] = {raw[1][k].x, raw[1][k].y, raw[1][k].z, raw[1][k].w};
            const uint32_t a1 = q_pair<T>(hi[2 * j], f[1]), a3 = q_pair<T>(hi[2 * j + 1], f[1]);
            if constexpr (S::q_in_regs) {
              qf[mt][2 * k + j][0] = a0, qf[mt][2 * k + j][1] = a1, qf[mt][2 * k + j][2] = a2, qf[mt][2 * k + j][3] = a3;
            } else {
              if (warp == mt) reinterpret_cast<uint4*>(smem + S::off_q)[at] = make_uint4(a0, a1, a2, a3);
            }
          }
        }
      }
    }
    if (!S::q_in_regs) named_bar_sync(1, kWarps * 32);

    float o[MT][D / 8][4];
    float thr[MT][2], ref[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
#pragma unroll
      for (int hf = 0; hf < HF; ++hf) thr[mt][hf] = -INFINITY, ref[mt][hf] = 0.f, l[mt][hf] = 0.f;
    }

    for (int tile = p.lo; tile < p.hi; ++tile, ++it) {
      const int s = it % S::stages;
      if (ok) ok = wait_warp(&full[s], (uint32_t)((it / S::stages) & 1));
      if (!ok) continue;
      const uint32_t st = ring + s * S::stage;
      const uint32_t there = (uint32_t)(valid[s] >> (warp * 16)) & 0xFFFFu;
      const int t0 = tile * kKeys + warp * 16;
      if (there) {
        // S = Q C^T: 16 keys
        float sc[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
        constexpr int kLoads = S::slab_row / 64;             // 16-byte reads of a lane in a slab's row
#pragma unroll
        for (int sl = 0; sl < S::slabs; ++sl) {
          uint4 kw[2][kLoads];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int key = warp * 16 + nt * 8 + g;
            const uint32_t rowa = st + sl * kKeys * S::slab_row + key * S::slab_row;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
              const int u = kLoads * c + i;
              const int sw = S::slab_row == 128 ? u ^ (key & 7) : u ^ ((key >> 1) & 3);
              kw[nt][i] = lds128(rowa + sw * 16);
            }
          }
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int ks = (sl * kLoads + i) * 4 + w;
              uint32_t b[2][2];
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                const uint32_t word = w == 0 ? kw[nt][i].x : w == 1 ? kw[nt][i].y : w == 2 ? kw[nt][i].z : kw[nt][i].w;
                codes_f16(word, b[nt][0], b[nt][1]);
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                if constexpr (S::q_in_regs) {
                  mma_f16(sc[mt][0], qf[mt][ks], b[0][0], b[0][1]);
                  mma_f16(sc[mt][1], qf[mt][ks], b[1][0], b[1][1]);
                } else {
                  uint32_t qa[4] = {0u, 0u, 0u, 0u};
                  if constexpr (HF == 1) {
                    const uint2 qv = lds64(qbase + ((mt * S::ksteps + ks) * 32 + lane) * 8);
                    qa[0] = qv.x, qa[2] = qv.y;
                  } else {
                    const uint4 qv = lds128(qbase + ((mt * S::ksteps + ks) * 32 + lane) * 16);
                    qa[0] = qv.x, qa[1] = qv.y, qa[2] = qv.z, qa[3] = qv.w;
                  }
                  mma_f16(sc[mt][0], qa, b[0][0], b[0][1]);
                  mma_f16(sc[mt][1], qa, b[1][0], b[1][1]);
                }
              }
            }
        }
        // scales of this lane's keys: 2c, 2c + 1 of both groups of 8
        const uint32_t sca = ring + S::off_scales + s * S::scales + (warp * 16 + 2 * c) * 4;
        const float2 k0 = lds_f2(sca), k1 = lds_f2(sca + 32);
        float2 v0 = lds_f2(sca + kKeys * 4), v1 = lds_f2(sca + kKeys * 4 + 32);
        const float ksc[4] = {k0.x, k0.y, k1.x, k1.y};
        const bool masked = there != 0xFFFFu || t0 + 16 > p.s.ctx;
        uint32_t seen[MT][2];                                // bit nt * 2 + e: the row sees that key
        if (masked) {
          uint32_t any = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) any |= ((there >> ((x >> 1) * 8 + 2 * c + (x & 1))) & 1u) << x;
          const int words = (a.n + 31) / 32;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < HF; ++hf) {
              const int r = mt * 16 + hf * 8 + g;
              const int i = (p.rb * S::rows + r) / G;
              uint32_t bits = any;
              for (int x = 0; x < 4; ++x) {
                const int j = t0 + (x >> 1) * 8 + 2 * c + (x & 1) - p.s.ctx;
                if (j < 0 || !(any >> x & 1)) continue;
                const bool sees = r < live_rows &&
                                  (a.mask ? (__ldg(a.mask + ((int64_t)p.b * a.n + i) * words + (j >> 5)) >> (j & 31)) & 1u
                                          : j <= i);
                if (!sees) bits &= ~(1u << x);
              }
              seen[mt][hf] = bits;
            }
        }
        // base-2 logits, and whether one passes its row's reference by too much
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < HF; ++hf) {
            const uint64_t f2 = pair(rowf[mt][hf], rowf[mt][hf]);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              float* z = sc[mt][nt] + 2 * hf;
              unpair(mul2(pair(z[0], z[1]), mul2(pair(ksc[2 * nt], ksc[2 * nt + 1]), f2)), z[0], z[1]);
            }
          }
        if (masked) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int hf = 0; hf < HF; ++hf)
                if (!(seen[mt][hf] >> x & 1)) sc[mt][x >> 1][2 * hf + (x & 1)] = -INFINITY;
        }
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < HF; ++hf)
            grow |= fmaxf(fmaxf(sc[mt][0][2 * hf], sc[mt][0][2 * hf + 1]), fmaxf(sc[mt][1][2 * hf], sc[mt][1][2 * hf + 1])) > thr[mt][hf];
        if (__any_sync(kFull, grow)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < HF; ++hf) {
              float m = fmaxf(fmaxf(sc[mt][0][2 * hf], sc[mt][0][2 * hf + 1]), fmaxf(sc[mt][1][2 * hf], sc[mt][1][2 * hf + 1]));
              m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
              m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
              if (m > thr[mt][hf]) {
                const float f = thr[mt][hf] == -INFINITY ? 0.f : ex2(ref[mt][hf] - m);
                ref[mt][hf] = m;
                thr[mt][hf] = m + kLazy;
                l[mt][hf] *= f;
#pragma unroll
                for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
                  for (int e = 2 * hf; e < (HF == 1 ? 4 : 2 * hf + 2); ++e) o[mt][nt][e] *= f;
              }
            }
        }
        uint32_t pa[MT][4], pr[MT][4];                       // the weights, and what their rounding left
        const float vsc[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int hf = 0; hf < HF; ++hf) {
              float* z = sc[mt][nt] + 2 * hf;
              const float x = ex2(z[0] - ref[mt][hf]), y = ex2(z[1] - ref[mt][hf]);
              l[mt][hf] += x + y;
              z[0] = x * vsc[2 * nt], z[1] = y * vsc[2 * nt + 1];
            }
        if (masked) {                                        // 0 times whatever an unseen key's scale is
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int hf = 0; hf < HF; ++hf)
                if (!(seen[mt][hf] >> x & 1)) sc[mt][x >> 1][2 * hf + (x & 1)] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int hf = 0; hf < HF; ++hf) {
              const float* z = sc[mt][nt] + 2 * hf;
              const uint32_t w = pack_bf16(z[0], z[1]);
              pa[mt][2 * nt + hf] = w;
              if constexpr (HF == 1) pa[mt][2 * nt + 1] = pack_rest(z[0], z[1], w);
              else pr[mt][2 * nt + hf] = pack_rest(z[0], z[1], w);
            }
        // O += P C': lane's keys 2c, 2c + 1, 2c + 8, 2c + 9, coordinates g * D/8 ..
#pragma unroll
        for (int sl = 0; sl < S::slabs; ++sl) {
          constexpr int kTiles = S::slab_row / 8;            // 8-coordinate tiles of a slab = bytes of a lane in a row
          uint32_t vw[4][kTiles / 4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = warp * 16 + (x >> 1) * 8 + 2 * c + (x & 1);
            const uint32_t rowa = st + S::codes + sl * kKeys * S::slab_row + key * S::slab_row;
            if constexpr (kTiles == 16) {
              const uint4 v = lds128(rowa + ((g ^ (key & 7)) << 4));
              vw[x][0] = v.x, vw[x][1] = v.y, vw[x][2] = v.z, vw[x][3] = v.w;
            } else {
              const uint2 v = lds64(rowa + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
              vw[x][0] = v.x, vw[x][1] = v.y;
            }
          }
#pragma unroll
          for (int w = 0; w < kTiles / 4; ++w)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t b0 = codes_bf16(vw[0][w], vw[1][w], j), b1 = codes_bf16(vw[2][w], vw[3][w], j);
              const int nt = sl * kTiles + 4 * w + j;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_bf16(o[mt][nt], pa[mt], b0, b1);
                if constexpr (HF == 2) mma_bf16(o[mt][nt], pr[mt], b0, b1);
              }
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);

    // ---------------- the four warps' softmaxes become one
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < HF; ++hf) {
        l[mt][hf] += __shfl_xor_sync(kFull, l[mt][hf], 1);
        l[mt][hf] += __shfl_xor_sync(kFull, l[mt][hf], 2);
        if (c == 0) {
          const int r = mt * 16 + hf * 8 + g;
          ml[warp * S::rows + r] = thr[mt][hf] - kLazy;      // -infinity where nothing was seen
          ml[(kWarps + warp) * S::rows + r] = l[mt][hf];
        }
      }
    named_bar_sync(1, kWarps * 32);
    for (int w = 0; w < kWarps; ++w) {
      if (warp == w) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < HF; ++hf) {
            const int r = mt * 16 + hf * 8 + g;
            float m = ml[r];
#pragma unroll
            for (int x = 1; x < kWarps; ++x) m = fmaxf(m, ml[x * S::rows + r]);
            const float mine = thr[mt][hf] - kLazy;
            const float f = mine == -INFINITY ? 0.f : ex2(ref[mt][hf] - m);
            float* dst = acc_sm + r * (D + 4);
#pragma unroll
            for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // column 2c + e of the 8-column tile nt holds byte nt of lane group 2c + e
                constexpr int kTiles = S::slab_row / 8;
                const int col = (nt / kTiles) * 128 + (2 * c + e) * kTiles + nt % kTiles;
                const float v = f == 0.f ? 0.f : (HF == 1 ? o[mt][nt][e] + o[mt][nt][2 + e] : o[mt][nt][2 * hf + e]) * f;
                dst[col] = w ? dst[col] + v : v;
              }
          }
      }
      named_bar_sync(1, kWarps * 32);
    }
    const bool whole = p.lo == 0 && p.hi == p.s.tiles;
    float* rec = nullptr;
    if (!whole) {
      // the block's first record is of an item begun elsewhere, its second of one begun here
      rec = records + ((int64_t)blockIdx.x * 2 + (p.lo > 0 ? 0 : 1)) * S::rows * (D + 2);
      if (p.lo > 0 && threadIdx.x == 0) {
        cuts[blockIdx.x] = walk.cut_of(p);
        kept = 1;
      }
    }
    for (int r = warp; r < S::rows; r += kWarps) {
      if (r >= live_rows) continue;
      float m = ml[r], sum = 0.f;
#pragma unroll
      for (int x = 1; x < kWarps; ++x) m = fmaxf(m, ml[x * S::rows + r]);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float mx = ml[x * S::rows + r];
        if (mx != -INFINITY) sum += ml[(kWarps + x) * S::rows + r] * ex2(mx - m);
        else if (ml[(kWarps + x) * S::rows + r] != 0.f) sum = NAN;   // only unordered logits were seen
      }
      const float* src = acc_sm + r * (D + 4);
      if (whole) {
        const int x = p.rb * S::rows + r;
        const int64_t row = ((int64_t)p.b * a.n + x / G) * a.Hq + p.h * G + x % G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        T* out = static_cast<T*>(a.out) + row * a.d;
        for (int e = 2 * lane; e < a.d; e += 64) store_pair(out + e, src[e] * inv, src[e + 1] * inv);
        if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
      } else {
        float* dst = rec + r * (D + 2);
        for (int e = lane; e < D; e += 32) dst[e] = src[e];
        if (lane == 0) dst[D] = m, dst[D + 1] = sum;
      }
    }
    named_bar_sync(1, kWarps * 32);                          // acc_sm and ml are free again
  }
  if (threadIdx.x == 0 && cuts && !kept) cuts[blockIdx.x].begin = -1;
}

// Block i > 0: if block i of the main grid began inside an item, and i is the
// first cut of that item, the records of blocks i - 1 (its second), i, i + 1, ..
// (their first) become the item's rows.  A warp takes a row: first the records'
// maxima and sums, a lane each, then their value sums one by one.
template <int D, int R, typename T>
__global__ void __launch_bounds__(128) tree_merge_kernel(TreeArgs a, const float* records, const Cut* cuts) {
  using S = Shape<D, R>;
  asm volatile("griddepcontrol.wait;" ::: "memory");         // the main grid is done
  const int i = blockIdx.x + 1;
  const Cut cut = cuts[i];
  if (cut.begin != i - 1) return;
  const int n = cut.end - cut.begin + 1;
  const int G = a.Hq / a.Hkv;
  const int drafts = a.draft_lens ? min(max(__ldg(a.draft_lens + cut.b), 0), a.n) : a.n;
  const int rows = min(S::rows, drafts * G - cut.rb * S::rows);
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < rows; r += 4) {
    auto rec = [&](int x) { return records + ((int64_t)(i - 1 + x) * 2 + (x == 0 ? 1 : 0)) * S::rows * (D + 2) + r * (D + 2); };
    float m = -INFINITY, l = 0.f;
    for (int x = lane; x < n; x += 32) m = fmaxf(m, __ldcg(rec(x) + D));
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    for (int x = lane; x < n; x += 32) {
      const float mx = __ldcg(rec(x) + D), lx = __ldcg(rec(x) + D + 1);
      l += mx == -INFINITY ? lx : lx * ex2(mx - m);          // nothing seen: 0, or NaN
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
    float v[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) v[e] = 0.f;
#pragma unroll 8
    for (int x = 0; x < n; ++x) {
      const float* p = rec(x);
      const float mx = __ldcg(p + D), f = mx == -INFINITY ? 0.f : ex2(mx - m);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(p + 64 * e + 2 * lane));
        v[2 * e] = f == 0.f ? v[2 * e] : fmaf(y.x, f, v[2 * e]);
        v[2 * e + 1] = f == 0.f ? v[2 * e + 1] : fmaf(y.y, f, v[2 * e + 1]);
      }
    }
    const int x = cut.rb * S::rows + r;
    const int64_t row = ((int64_t)cut.b * a.n + x / G) * a.Hq + cut.h * G + x % G;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* out = static_cast<T*>(a.out) + row * a.d;
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
      if (64 * e + 2 * lane < a.d) store_pair(out + 64 * e + 2 * lane, v[2 * e] * inv, v[2 * e + 1] * inv);
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

int padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// rows of a block: 8 or 16 where a kv-head's rows fit in them (or d > 128, for the
// registers), else 32.  4 rows of 16 x 16000 keys: 149 us in blocks of 8, 164 of 16;
// 32 rows of 32 x 4000 keys: 166 us in one block of 32, 181 in two of 16
int block_rows(int d, int64_t rows) { return rows <= 8 ? 8 : rows <= 16 || d > 128 ? 16 : 32; }

bool code_map(CUtensorMap* m, const int8_t* base, int d, int64_t rows, int box) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const int D = padded(d);
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)std::max<int64_t>(rows, 1)};
  cuuint64_t strides[1] = {(cuuint64_t)d};
  cuuint32_t boxd[2] = {(cuuint32_t)(D > 128 ? 128 : D), (cuuint32_t)box};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, boxd, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int R, typename T>
int launch_shape(const TreeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, int box, int grid, bool merge,
                 void* workspace, cudaStream_t st) {
  using S = Shape<D, R>;
  static_assert(S::bytes + 1024 <= 228 * 1024 / S::blocks_per_sm, "the blocks of an SM must fit");
  int e = ensure_dyn_smem(reinterpret_cast<const void*>(tree_kernel<D, R, T>), S::bytes);
  if (e) return e;
  Cut* cuts = static_cast<Cut*>(workspace);
  float* records = reinterpret_cast<float*>(static_cast<char*>(workspace) + ((size_t)grid * sizeof(Cut) + 255) / 256 * 256);
  tree_kernel<D, R, T><<<grid, S::threads, S::bytes, st>>>(km, vm, a, box, merge ? records : nullptr, merge ? cuts : nullptr);
  e = (int)cudaGetLastError();
  if (e || !merge) return e;
  return launch_beside(tree_merge_kernel<D, R, T>, dim3(grid - 1), 128, st, a, (const float*)records, (const Cut*)cuts);
}

int blocks_per_sm(int d, int rows) { return rows <= 16 && d <= 128 ? (d <= 64 ? 4 : 3) : 2; }

int tree_grid(const tq_ctx* h, int blocks_sm, int B, int Hkv, int64_t row_blocks, int64_t tiles) {
  const int64_t most = (int64_t)h->sm_count * blocks_sm;
  const int64_t items = (int64_t)B * Hkv * row_blocks;
  // compare without the product's overflow
  return (int)(items >= most || tiles >= most ? most : std::min(most, items * tiles));
}

}  // namespace

size_t tree_workspace(const tq_ctx* h, int B, int n, int Hq, int Hkv) {
  if (B == 0 || n == 0 || Hq == 0) return 0;
  if (tree_tc_supported(h, n, Hq, Hkv)) return tree_tc_workspace(h, n, Hq, Hkv);
  const int64_t rows = (int64_t)n * (Hq / Hkv);
  const int R = block_rows(h->d, rows), grid = h->sm_count * blocks_per_sm(h->d, R);
  return ((size_t)grid * sizeof(Cut) + 255) / 256 * 256 + (size_t)grid * 2 * R * (padded(h->d) + 2) * 4;
}

int launch_tree(const tq_ctx* h, const TreeArgs& a, int dtype, void* workspace, void* stream) {
  if (tree_tc_supported(h, a.n, a.Hq, a.Hkv)) return launch_tree_tc(h, a, dtype, workspace, stream);
  int box = kKeys;
  while (a.page % box) box /= 2;  // page pieces that a tile never splits: 8, 16, 32 or 64 keys
  CUtensorMap km, vm;
  if (!code_map(&km, a.kcodes, h->d, a.rows, box) || !code_map(&vm, a.vcodes, h->d, a.rows, box))
    return (int)cudaErrorInvalidValue;
  const int64_t rows = (int64_t)a.n * (a.Hq / a.Hkv);
  const int R = block_rows(h->d, rows);
  const int64_t blocks = (rows + R - 1) / R, tiles = ((int64_t)a.max_pages * a.page + kKeys - 1) / kKeys;
  const int64_t items = a.B * (int64_t)a.Hkv * blocks;
  const bool merge = tiles > 1;
  const int per_sm = blocks_per_sm(h->d, R);
  int grid = tree_grid(h, per_sm, a.B, a.Hkv, blocks, tiles);
  if (!merge) grid = (int)std::min<int64_t>(items, (int64_t)h->sm_count * per_sm);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == TQ_BF16;
#define TQ_TREE(D, R)                                                                                       \
  return bf ? launch_shape<D, R, __nv_bfloat16>(a, km, vm, box, grid, merge && grid > 1, workspace, st)    \
            : launch_shape<D, R, __half>(a, km, vm, box, grid, merge && grid > 1, workspace, st)
  switch (padded(h->d) + R) {
    case 64 + 8: TQ_TREE(64, 8);
    case 64 + 16: TQ_TREE(64, 16);
    case 64 + 32: TQ_TREE(64, 32);
    case 128 + 8: TQ_TREE(128, 8);
    case 128 + 16: TQ_TREE(128, 16);
    case 128 + 32: TQ_TREE(128, 32);
    case 256 + 8: TQ_TREE(256, 8);
    default: TQ_TREE(256, 16);
  }
#undef TQ_TREE
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
  if (!q || !ctx_lens || !block_table || !out || (rows > 0 && (!kcodes || !kscales || !vcodes || !vscales)))
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
  if (rows == 0) {
    // no page id lies in it and nothing is loaded, but the tensor maps need an address and a row
    a.kcodes = a.vcodes = static_cast<const int8_t*>(q);
  }
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = out, a.lse = lse, a.status = h->dev.status;
  DeviceGuard guard(h->device);
  const int e = guard.error ? guard.error : launch_tree(h, a, dtype, workspace, stream);
  return e ? set_error(TQ_ECUDA, "%s: %s", fn, cudaGetErrorString((cudaError_t)e)) : clear_error();
}
