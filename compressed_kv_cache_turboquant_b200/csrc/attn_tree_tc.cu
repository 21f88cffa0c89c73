// Attention of many drafted tokens per sequence over the 8-bit paged cache, on
// the tensor cores' own path (tcgen05, sm_100a).
//
// The arithmetic is that of attn_tree.cu: both products run on the integer
// codes, exact in 16 bits, with the scales on the float32 logits and on the
// weights (rounded once to bf16; for fp16 results the remainder of that rounding
// takes a second product; attn_tree.cu has it for both, so that a bf16 result of up to
// 32 rows is off by 0.0016 of itself where this one is off by 0.0024).  A row is a (token, head of a kv-head's group) pair,
// 128 / G tokens of a group of G heads in a tile of 128 rows, one or two tiles a
// block; queries enter as they are.  Against attn_tree.cu's blocks of 32 rows
// the codes of a key tile are converted once for up to 256 rows.
//
// What bounds it: the softmax, which reads two scales a key (16 bytes at a time, the
// same for all lanes) beside its 2^x, and packs the weights once, or twice with the
// remainders.  64 tokens for 4 sequences of 16384, 8 kv-heads of 4 heads, d = 128:
// 0.140 ms, 490 TFLOP/s; 61 tokens for 4 of 64000, 4 kv-heads, d = 64: 0.191 ms for
// bf16 (335 TFLOP/s), 0.230 for fp16.  A second term for bf16 weights would cost a
// third (0.179 ms in the first case).
//
// With one row tile its key tiles go to two streams in turn, each with its own
// logits, weights, value sums and softmax, joined at the end of a piece: one's
// softmax runs beside the other's products.  With two row tiles they are the two
// streams.
//
// Warps (512 threads, one block per SM, persistent over equal ranges of 128-key
// tiles; what a cut divides is joined by tree_tc_merge_kernel):
//   0-3, 4-7  softmax of stream 0, 1: thread = row (TMEM lane)
//   8         TMA of the item's queries and of raw code tiles, a page piece at a
//             time, K and V alternating in a ring
//   9         the MMA issuer
//   12-15     converters: raw codes -> swizzled 16-bit operand tiles (one K tile,
//             two V tiles), scales and the bits of the keys that are there
// Tensor memory: S/P of streams 0, 1 at 0, 128; O at 256, 384.  The weights of the
// first 64 keys take 32 columns from the start of their tile's S, those of the
// other 64 from its middle, and remainders follow each.
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

constexpr int kTile = 128;                    // rows of a row tile, keys of a tile
constexpr int kThreads = 512;
constexpr int kConverters = 4;
constexpr int kRegsSoftmax = 192, kRegsOther = 64;   // 2 x 192 + 2 x 64 = 4 x 128, the registers at launch
constexpr uint32_t kColS = 0, kColO = 256;
constexpr int kBarBytes = 640;   // barriers, valid bits, scratch, the tensor-memory address

template <int D, int NT>
struct Shape {
  static constexpr int slabs = D / 64;
  static constexpr int tile = kTile * D * 2;  // bytes of a 16-bit operand tile
  static constexpr int raw = kTile * D;       // bytes of a raw tile
  static constexpr int scales = 2 * kTile * 4;   // a tile's K and V scales
  static constexpr int stages = D == 128 ? (NT == 2 ? 3 : 5) : 8;
  static constexpr int off_k = NT * tile;
  static constexpr int off_v = off_k + tile;
  static constexpr int off_raw = off_v + 2 * tile;
  static constexpr int off_rows = off_raw + stages * raw;        // [stages][16] cache rows of a K tile's page pieces
  static constexpr int off_sc = off_rows + stages * 64;          // [4 tiles in turn][K scales x logit scale, V scales][128]
  static constexpr int off_valid = off_sc + 4 * scales;          // [4][bits of the keys, whether a value scale is not finite][4] words
  static constexpr int off_swap = off_valid + 4 * 32;            // [2][128] maxima and sums of the second stream
  static constexpr int off_bar = off_swap + 2 * kTile * 4;
  static constexpr int bytes = off_bar + kBarBytes + 1024;
  static constexpr int rows = NT * kTile;
};

// four int8 codes -> two 16-bit pairs.  bf16: the low seven bits under 0x43 are
// 128 + them, the sign bit alone 128 or 256; fp16: a byte + 128 under 0x64 is
// 1024 + 128 + the code
__device__ __forceinline__ uint2 codes4(uint32_t w, __nv_bfloat16) {
  uint2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = prmt(w, 0x43434343u, i ? 0x4342u : 0x4140u);
    const uint32_t m = t & 0xFF7FFF7Fu, s = t & 0xFF80FF80u;
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&s));
    (i ? r.y : r.x) = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}
__device__ __forceinline__ uint2 codes4(uint32_t w, __half) {
  const uint32_t x = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));
  uint2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = prmt(x, 0x64646464u, i ? 0x4342u : 0x4140u);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&t), bias);
    (i ? r.y : r.x) = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}

struct TcArgs {
  TreeArgs t;
  int G, tq;       // tq = 128 / G tokens of a row tile
  int box;         // keys of a page piece
  float* records;  // [blocks][2][D + 2][rows]: value sums, maximum, sum
  Cut* cuts;
};

template <int D, int NT, typename T>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap, const TcArgs ta) {
  using S = Shape<D, NT>;
  constexpr bool kTwoTerms = std::is_same<T, __half>::value;
  const TreeArgs& a = ta.t;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + S::off_bar);   // [stages] tx
  uint64_t* raw_empty = raw_full + S::stages;   // [stages] converters
  uint64_t* valid = raw_empty + S::stages;      // [stages][2] bits of the keys that a K tile holds
  uint64_t* k_ready = valid + 2 * S::stages;    // converters
  uint64_t* k_free = k_ready + 1;               // MMA commit
  uint64_t* v_ready = k_free + 1;               // [2] converters
  uint64_t* v_free = v_ready + 2;               // [2] MMA commit
  uint64_t* q_full = v_free + 2;                // tx
  uint64_t* q_free = q_full + 1;                // MMA commit
  uint64_t* s_full = q_free + 1;                // [2] MMA commit
  uint64_t* p_ready = s_full + 2;               // [2][2] 4 softmax warps: weights of the first, second 64 keys
  uint64_t* pv_done = p_ready + 4;              // [2] MMA commit
  uint64_t* x_ready = pv_done + 2;              // 4 warps of stream 1: its maxima and sums written, its values done
  uint64_t* x_free = x_ready + 1;               // 4 warps of stream 0: they and its O read
  uint64_t* done = x_free + 1;
  int64_t* scratch = reinterpret_cast<int64_t*>(done + 1);                // [2 + 16]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scratch + 18);
  static_assert((4 * S::stages + 19 + 18) * 8 + 4 <= kBarBytes && S::bytes <= 232448, "shared memory");
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kConverters);
    }
    mbar_init(k_ready, kConverters);
    mbar_init(k_free, 1);
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(x_ready, 4);
    mbar_init(x_free, 4);
    mbar_init(done, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&v_ready[x], kConverters);
      mbar_init(&v_free[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_ready[2 * x], 4);
      mbar_init(&p_ready[2 * x + 1], 4);
      mbar_init(&pv_done[x], 1);
    }
    fence_mbar_init();
  }
  // rows of a block in whole tokens: what seq_of counts blocks by
  const int block_rows = NT * ta.tq * ta.G;
  asm volatile("griddepcontrol.launch_dependents;");       // the merge may set itself up
  Walk<kTile> walk;
  if (!range_of_block<kTile, kThreads>(a, block_rows, scratch, walk)) {
    if (threadIdx.x == 0 && ta.cuts) ta.cuts[blockIdx.x].begin = -1;
    return;
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Piece p;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
      // ---------------- TMA
      const int64_t pages = a.rows / a.page;
      const int boxes = kTile / ta.box;
      int x = 0, i = 0;
      bool ok = true;
      while (ok && walk.next(a, block_rows, p)) {
        if (i > 0 && !wait_warp(q_free, (uint32_t)((i - 1) & 1))) {
          ok = false;
          break;
        }
        ++i;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, (uint32_t)(NT * S::slabs * ta.tq * ta.G * 128));
          for (int t = 0; t < NT; ++t)
            for (int sl = 0; sl < S::slabs; ++sl)
              tma_load_3d(&qmap, q_full, smem + t * S::tile + sl * kTile * 128, sl * 64, p.h * ta.G,
                          p.b * a.n + (p.rb * NT + t) * ta.tq);
        }
        const int32_t* table = a.block_table + ((int64_t)p.b * a.Hkv + p.h) * a.max_pages;
        // lane i: piece i of a tile; its page id is read one tile ahead
        auto row_of = [&](int tile) -> int {
          const int t = tile * kTile + lane * ta.box;
          if (lane >= boxes || tile >= p.hi || t >= p.s.T) return -1;
          const int id = __ldg(table + t / a.page);
          if (id < 0 || id >= pages) {
            atomicOr(a.status, kStatusRange);
            return -1;
          }
          return id * a.page + t % a.page;
        };
        int row = row_of(p.lo);
        for (int tile = p.lo; ok && tile < p.hi; ++tile) {
          const int next = row_of(tile + 1);
          const uint32_t live = __ballot_sync(kFull, row >= 0);
          for (int kv = 0; kv < 2; ++kv, ++x) {
            const int s = x % S::stages;
            if (!wait_warp(&raw_empty[s], (uint32_t)(((x / S::stages) & 1) ^ 1))) {
              ok = false;
              break;
            }
            if (kv == 0 && lane < 16) reinterpret_cast<int*>(smem + S::off_rows)[s * 16 + lane] = row;
            __syncwarp();
            if (lane == 0) {
              if (kv == 0) {
                const int left = p.s.T - tile * kTile;
                for (int half = 0; half < 2; ++half) {
                  uint64_t bits = 0;
                  for (int b = 0; b < boxes; ++b) {
                    const int at = b * ta.box - half * 64;
                    if ((live >> b & 1) && at >= 0 && at < 64) bits |= (ta.box == 64 ? ~0ull : (1ull << ta.box) - 1) << at;
                  }
                  const int here = left - half * 64;
                  if (here < 64) bits &= here <= 0 ? 0ull : (1ull << here) - 1;
                  valid[2 * s + half] = bits;
                }
              }
              mbar_arrive_expect_tx(&raw_full[s], (uint32_t)(__popc(live) * ta.box * D));
            }
            __syncwarp();
            if (row >= 0) {
              tma_load_2d(kv ? &vmap : &kmap, &raw_full[s], smem + S::off_raw + s * S::raw + lane * ta.box * D, 0, row);
            }
          }
          row = next;
        }
      }
      if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
      // no copy may still be in flight when the block ends
      if (lane == 0) {
        for (int y = x > S::stages ? x - S::stages : 0; y < x; ++y)
          if (!wait(&raw_full[y % S::stages], (uint32_t)((y / S::stages) & 1))) atomicOr(a.status, kStatusTimeout);
        if (i > 0 && !wait(q_full, (uint32_t)((i - 1) & 1))) atomicOr(a.status, kStatusTimeout);
      }
    } else if (warp == 9) {
      // ---------------- MMA
      constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
      constexpr uint32_t idesc_s = idesc_f16(kTile, kTile, bf), idesc_o = idesc_f16(kTile, D, true) | (1u << 16);
      const uint32_t lead = elect_one();
      const uint64_t qd = sw128_kmajor_desc(smem_u32(smem)), kd = sw128_kmajor_desc(smem_u32(smem + S::off_k));
      const uint64_t vd = sw128_mnmajor_desc(smem_u32(smem + S::off_v), kTile * 128);
      int kt = 0, i = 0, pv[2] = {0, 0};                    // tiles, items, value products of the streams so far
      bool ok = true;
      // stream t, queries of row tile qt; the buffer's last weights must have been consumed
      auto logits = [&](int t, int qt, int n) -> bool {
        if (n > 0 && !wait_warp(&pv_done[t], (uint32_t)((n - 1) & 1))) return false;
        tc_fence_after();
        const uint64_t q = qd + qt * (S::tile >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (uint32_t)((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4;
          mma_ss(tmem + kColS + t * 128, q + off, kd + off, idesc_s, ks ? 1u : 0u, lead);
        }
        commit(&s_full[t], lead);
        return true;
      };
      auto values = [&](int t, int n, int buf, bool first) -> bool {
        const uint64_t v = vd + buf * (S::tile >> 4);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!wait_warp(&p_ready[2 * t + hf], (uint32_t)(n & 1))) return false;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t pc = tmem + kColS + t * 128 + 64 * hf + 8 * ks;
            const uint64_t vk = v + (4 * hf + ks) * (2048 >> 4);
            mma_ts(tmem + kColO + t * 128, pc, vk, idesc_o, (first && hf == 0 && ks == 0) ? 0u : 1u, lead);
            if constexpr (kTwoTerms) mma_ts(tmem + kColO + t * 128, pc + 32, vk, idesc_o, 1u, lead);
          }
        }
        commit(&pv_done[t], lead);
        return true;
      };
      while (ok && walk.next(a, block_rows, p)) {
        const bool two = NT == 2 && (p.rb * NT + 1) * ta.tq < p.s.drafts;
        ok = wait_warp(q_full, (uint32_t)(i++ & 1)) && wait_warp(k_ready, (uint32_t)(kt & 1)) && logits(0, 0, pv[0]) &&
             (!two || logits(1, 1, pv[1]));
        if (!ok) break;
        commit(k_free, lead);
        if (p.hi - p.lo == 1) commit(q_free, lead);
        for (int tile = p.lo; tile < p.hi; ++tile, ++kt) {
          const int buf = kt & 1;
          const bool more = tile + 1 < p.hi;
          if constexpr (NT == 1) {
            // the next tile's logits go to the other stream, ahead of this one's values
            const int t = (tile - p.lo) & 1;
            if (more) {
              if (!(ok = wait_warp(k_ready, (uint32_t)((kt + 1) & 1)) && logits(t ^ 1, 0, t ? pv[0] : pv[1]))) break;
              commit(k_free, lead);
              if (tile + 2 == p.hi) commit(q_free, lead);
            }
            if (!(ok = wait_warp(&v_ready[buf], (uint32_t)((kt >> 1) & 1)))) break;
            if (!(ok = values(t, t ? pv[1] : pv[0], buf, tile - p.lo < 2))) break;
            ++(t ? pv[1] : pv[0]);
            commit(&v_free[buf], lead);
          } else {
            if (!(ok = wait_warp(&v_ready[buf], (uint32_t)((kt >> 1) & 1)))) break;
            if (!(ok = values(0, pv[0]++, buf, tile == p.lo))) break;
            if (more && !(ok = wait_warp(k_ready, (uint32_t)((kt + 1) & 1)) && logits(0, 0, pv[0]))) break;
            if (two && !(ok = values(1, pv[1]++, buf, tile == p.lo))) break;
            commit(&v_free[buf], lead);
            if (more && two && !(ok = logits(1, 1, pv[1]))) break;
            if (more) commit(k_free, lead);
            if (tile + 2 == p.hi) commit(q_free, lead);
          }
        }
      }
      if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
      // nothing may still run when tensor memory is given back
      commit(done, lead);
      if (!wait_warp(done, 0) && lane == 0) atomicOr(a.status, kStatusTimeout);
    } else if (warp >= 12) {
      // ---------------- converters
      const int w = warp - 12;
      constexpr int kPer = D / 16;                          // 16-byte pieces of a key's codes
      const int key8 = lane & 7, u = lane >> 3;             // eight neighbouring keys, one of four pieces
      // a piece in the raw row's swizzle (128 or 64 bytes), its two halves in the operand's
      const uint32_t raw_at = (uint32_t)(key8 * D + ((D == 128 ? u ^ key8 : u ^ (key8 >> 1)) << 4));
      int x = 0, kt = 0;
      bool ok = true;
      auto convert = [&](const uint8_t* raw, uint8_t* dst, auto type) {
        // 16 keys of a warp at a time: their D / 16 pieces in steps of four (lanes / 8) pieces of 8 keys
#pragma unroll 1
        for (int k0 = w * 16; k0 < kTile; k0 += kConverters * 16) {
          uint4 c[2 * kPer / 4];
#pragma unroll
          for (int i = 0; i < 2 * kPer / 4; ++i)
            c[i] = *reinterpret_cast<const uint4*>(raw + (k0 + (i & 1) * 8) * D + (raw_at ^ ((i >> 1) << 6)));
#pragma unroll
          for (int i = 0; i < 2 * kPer / 4; ++i) {
            const int group = k0 + (i & 1) * 8, q = i >> 1;   // eight keys; the four pieces 4 q ..
            const uint2 e0 = codes4(c[i].x, type), e1 = codes4(c[i].y, type), e2 = codes4(c[i].z, type), e3 = codes4(c[i].w, type);
            // 64 coordinates a slab: pieces 4 q .. 4 q + 3 are slab q
            uint8_t* rowp = dst + q * kTile * 128 + (group + key8) * 128;
            *reinterpret_cast<uint4*>(rowp + (((2 * u) ^ key8) << 4)) = make_uint4(e0.x, e0.y, e1.x, e1.y);
            *reinterpret_cast<uint4*>(rowp + (((2 * u + 1) ^ key8) << 4)) = make_uint4(e2.x, e2.y, e3.x, e3.y);
          }
        }
      };
      while (ok && walk.next(a, block_rows, p)) {
        for (int tile = p.lo; ok && tile < p.hi; ++tile, ++kt) {
          for (int kv = 0; kv < 2; ++kv, ++x) {
            const int s = x % S::stages, buf = kt & 1;
            const uint8_t* raw = smem + S::off_raw + s * S::raw;
            ok = wait_warp(&raw_full[s], (uint32_t)((x / S::stages) & 1)) &&
                 (kv ? kt < 2 || wait_warp(&v_free[buf], (uint32_t)(((kt >> 1) - 1) & 1))
                     : kt < 1 || wait_warp(k_free, (uint32_t)((kt - 1) & 1)));
            if (!ok) break;
            // the scales of this warp's keys, on their way while the codes are converted
            const int key = w * 32 + lane;
            const bool there = !kv && (valid[2 * s + (key >> 6)] >> (key & 63) & 1);
            float ksc = 0.f, vsc = 0.f;
            if (there) {
              const int64_t at = reinterpret_cast<const int*>(smem + S::off_rows)[s * 16 + key / ta.box] + key % ta.box;
              ksc = __ldg(a.kscales + at);
              vsc = __ldg(a.vscales + at);
            }
            uint8_t* dst = smem + (kv ? S::off_v + buf * S::tile : S::off_k);
            if constexpr (kTwoTerms) {
              if (kv) convert(raw, dst, __nv_bfloat16());
              else convert(raw, dst, T());
            } else {
              convert(raw, dst, T());
            }
            if (kv == 0) {
              float* sc = reinterpret_cast<float*>(smem + S::off_sc + (kt & 3) * S::scales);
              sc[key] = ksc * a.scale_log2;
              sc[kTile + key] = vsc;
              const uint32_t bits = __ballot_sync(kFull, there);
              const bool odd = __any_sync(kFull, !(fabsf(vsc) < INFINITY));
              if (lane == 0) {
                uint32_t* to = reinterpret_cast<uint32_t*>(smem + S::off_valid) + (kt & 3) * 8 + w;
                to[0] = bits;
                to[4] = odd;
              }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(kv ? &v_ready[buf] : k_ready);
              mbar_arrive(&raw_empty[s]);
            }
          }
        }
      }
      if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
    }
  } else {
    // ---------------- softmax of stream t: thread = row of its row tile
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, rt = NT == 2 ? t : 0, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sc = tmem + lanes + kColS + t * 128, oc = tmem + lanes + kColO + t * 128;
    const int row_tok = r / ta.G, row_head = r % ta.G;
    const int words = (a.n + 31) / 32;
    float* swap = reinterpret_cast<float*>(smem + S::off_swap) + r;
    int kt0 = 0, steps = 0, kept = 0, joined = 0;           // tiles before this piece; steps of the stream; pieces of two streams
    bool ok = true;
    while (ok && walk.next(a, block_rows, p)) {
      const int first = NT == 1 ? p.lo + t : p.lo, by = NT == 1 ? 2 : 1, base = kt0 - p.lo;
      kt0 += p.hi - p.lo;
      if (first >= p.hi || (p.rb * NT + rt) * ta.tq >= p.s.drafts) continue;   // no tiles, or no rows
      const bool join = NT == 1 && p.hi - p.lo > 1;
      // stream 0 has taken the last piece's sums
      if (join && t == 1 && joined > 0 && !(ok = wait_warp(x_free, (uint32_t)((joined - 1) & 1)))) break;
      const int tok = (p.rb * NT + rt) * ta.tq + row_tok;
      const bool live = row_tok < ta.tq && tok < p.s.drafts;
      float m = -INFINITY, l = 0.f;
      for (int tile = first; tile < p.hi; tile += by, ++steps) {
        if (!(ok = wait_warp(&s_full[t], (uint32_t)(steps & 1)))) break;
        tc_fence_after();
        float x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(sc + 32 * c, x[c]);
        const int slot = (base + tile) & 3;
        const ulonglong2* kscale = reinterpret_cast<const ulonglong2*>(smem + S::off_sc + slot * S::scales);
        const ulonglong2* vscale = kscale + kTile / 4;
        const int t0 = tile * kTile;
        // which keys the row sees: those that are there, and of the drafted ones its own
        const uint4 there = *reinterpret_cast<const uint4*>(smem + S::off_valid + slot * 32);
        uint32_t sees[4] = {there.x, there.y, there.z, there.w};
        const bool whole = t0 + kTile <= p.s.ctx && (there.x & there.y & there.z & there.w) == kFull;
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = t0 + 32 * c - p.s.ctx;            // the group's first key among the drafted ones
            if (j + 31 < 0) continue;
            uint32_t bits = 0;
            if (live) {
              if (a.mask) {
                const uint32_t* mk = a.mask + ((int64_t)p.b * a.n + tok) * words;
                const int w0 = j < 0 ? 0 : j >> 5;
                const uint32_t lo = w0 < words ? __ldg(mk + w0) : 0u, hi = w0 + 1 < words ? __ldg(mk + w0 + 1) : 0u;
                bits = j < 0 ? lo << -j : __funnelshift_r(lo, hi, j & 31);
              } else {
                const int upto = tok - j;                   // the last drafted key it sees, from the group's first
                bits = upto < 0 ? 0u : upto >= 31 ? kFull : (2u << upto) - 1;
              }
            }
            if (j < 0) bits |= (1u << -j) - 1;              // context
            sees[c] &= bits;
          }
        }
        tmem_wait_ld();
        // base-2 logits, and the row's largest
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          regs_after_wait(x[c]);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const ulonglong2 k = kscale[8 * c + e / 4];
            unpair(mul2(pair(x[c][e], x[c][e + 1]), k.x), x[c][e], x[c][e + 1]);
            unpair(mul2(pair(x[c][e + 2], x[c][e + 3]), k.y), x[c][e + 2], x[c][e + 3]);
          }
        }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) x[c][e] = sees[c] >> e & 1 ? x[c][e] : -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = max3(x[c][0], x[c][1], x[c][2]);
#pragma unroll
          for (int e = 3; e + 1 < 32; e += 2) mx[c] = max3(mx[c], x[c][e], x[c][e + 1]);
          mx[c] = max3(mx[c], x[c][31], x[c][31]);
        }
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]);
        if (!(top < INFINITY)) l = NAN;                     // a seen logit is NaN or infinite: so is the row
        const bool grow = top > m + kLazy || (m == -INFINITY && top > m);
        if (__any_sync(kFull, grow)) {
          float f = 1.f;
          if (grow) {
            f = m == -INFINITY ? 0.f : ex2(m - top);
            l *= f;
            m = top;
          }
          if (tile > first) {
            // the stream's value product before was done before these logits began
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(oc + c, o);
              tmem_wait_ld();
              uint32_t y[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                asm volatile("" : "+f"(o[e])::"memory");
                y[e] = __float_as_uint(f == 0.f ? 0.f : o[e] * f);
              }
              tmem_st16(oc + c, y);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t ref2 = pair(-ref, -ref);
        uint64_t sum[2] = {0, 0};
        // 0 times a scale that is not finite is NaN; such keys are drafted ones that
        // someone else sees, or nobody
        const uint4 odd = *reinterpret_cast<const uint4*>(smem + S::off_valid + slot * 32 + 16);
        const bool clean = whole || !(odd.x | odd.y | odd.z | odd.w);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = 2 * hf + h;
            uint32_t y[16], z[kTwoTerms ? 16 : 1];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const ulonglong2 v = vscale[8 * c + e / 4];
              float* q = x[c] + e;
              unpair(add2(pair(q[0], q[1]), ref2), q[0], q[1]);
              unpair(add2(pair(q[2], q[3]), ref2), q[2], q[3]);
              const uint64_t p0 = pair(ex2(q[0]), ex2(q[1])), p1 = pair(ex2(q[2]), ex2(q[3]));
              sum[0] = add2(sum[0], p0);
              sum[1] = add2(sum[1], p1);
              unpair(mul2(p0, v.x), q[0], q[1]);
              unpair(mul2(p1, v.y), q[2], q[3]);
            }
            if (!clean) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[c][e] = sees[c] >> e & 1 ? x[c][e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              y[e / 2] = pack_bf16(x[c][e], x[c][e + 1]);
              if constexpr (kTwoTerms) z[e / 2] = pack_rest(x[c][e], x[c][e + 1], y[e / 2]);
            }
            tmem_st16(sc + 64 * hf + 16 * h, y);
            if constexpr (kTwoTerms) tmem_st16(sc + 64 * hf + 32 + 16 * h, z);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[2 * t + hf]);
        }
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      if (!(ok = wait_warp(&pv_done[t], (uint32_t)((steps - 1) & 1)))) break;
      tc_fence_after();
      float f = 1.f, f1 = 0.f;                              // of this stream's sums, of the other's
      if (join) {
        if (t == 1) {
          swap[0] = m;
          swap[kTile] = l;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(x_ready);
          ++joined;
          continue;
        }
        if (!(ok = wait_warp(x_ready, (uint32_t)(joined++ & 1)))) break;
        tc_fence_after();
        const float m1 = swap[0], l1 = swap[kTile], both = fmaxf(m, m1);
        f = m == -INFINITY ? 0.f : ex2(m - both);
        f1 = m1 == -INFINITY ? 0.f : ex2(m1 - both);
        // a stream that saw nothing has l = 0, or NaN
        l = (m == -INFINITY ? l : l * f) + (m1 == -INFINITY ? l1 : l1 * f1);
        m = both;
      }
      const bool all = p.lo == 0 && p.hi == p.s.tiles;
      if (!all && p.lo > 0 && threadIdx.x == 0) {
        ta.cuts[blockIdx.x] = walk.cut_of(p);
        kept = 1;
      }
      float* rec = all ? nullptr
                       : ta.records + ((int64_t)blockIdx.x * 2 + (p.lo > 0 ? 0 : 1)) * (D + 2) * S::rows + rt * kTile + r;
      const int64_t row = ((int64_t)p.b * a.n + tok) * a.Hq + p.h * ta.G + row_head;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(oc + c, o);
        if (join) {
          float o1[32];
          tmem_ld32(oc + 128 + c, o1);
          tmem_wait_ld();
          regs_after_wait(o);
          regs_after_wait(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = (f == 0.f ? 0.f : o[e] * f) + (f1 == 0.f ? 0.f : o1[e] * f1);
        } else {
          tmem_wait_ld();
          regs_after_wait(o);
        }
        if (all) {
          if (live) {
            T* out = static_cast<T*>(a.out) + row * a.d + c;
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              if (c + e < a.d)
                *reinterpret_cast<uint4*>(out + e) =
                    make_uint4(pack(o[e] * inv, o[e + 1] * inv, T()), pack(o[e + 2] * inv, o[e + 3] * inv, T()),
                               pack(o[e + 4] * inv, o[e + 5] * inv, T()), pack(o[e + 6] * inv, o[e + 7] * inv, T()));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) rec[(int64_t)(c + e) * S::rows] = o[e];   // a column of rows at a time
        }
      }
      if (all) {
        if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        rec[(int64_t)D * S::rows] = m;
        rec[(int64_t)(D + 1) * S::rows] = l;
      }
      tc_fence_before();
      if (join) {
        __syncwarp();
        if (lane == 0) mbar_arrive(x_free);
      }
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
    if (threadIdx.x == 0 && ta.cuts && !kept) ta.cuts[blockIdx.x].begin = -1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the parts of an item that a cut divides: blocks begin .. end of the main grid
// hold them, the first in its second record, the others in their first.  A block takes
// some rows (z) and coordinates (y) of one.  Where there are many items, thread = row,
// and blockIdx.x + 1 is the main grid's block whose cut it looks at (most are not an
// item's first).  Few items have many records each: blockIdx.x counts the items, and
// four slices of threads take every fourth record (8000 tokens of two heads in 63
// records: 32 us, 40 with one slice; 64 sequences of 1000 tokens: 203 us, 185 with one).
template <int kSlices, int NT>
struct Merge {
  static constexpr int rows = kSlices == 1 ? NT * kTile : 64, cols = kSlices == 1 ? 4 : 8;
};

template <int D, int NT, int kSlices, typename T>
__global__ void __launch_bounds__(kSlices * Merge<kSlices, NT>::rows) tree_tc_merge_kernel(const TcArgs ta, int blocks) {
  using S = Shape<D, NT>;
  constexpr int kRows = Merge<kSlices, NT>::rows, kCols = Merge<kSlices, NT>::cols, kWarps = kSlices * kRows / 32;
  const TreeArgs& a = ta.t;
  __shared__ uint32_t first[kWarps];                         // bit: block i is the first cut of its item
  __shared__ float part[kSlices > 1 ? kSlices : 1][kCols + 2][kSlices > 1 ? kRows : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");         // the main grid is done
  const int tid = threadIdx.x, lane = tid & 31;
  int at = blockIdx.x + 1;
  if constexpr (kSlices > 1) {
    int left = blockIdx.x;
    at = -1;
    for (int b0 = 1; b0 < blocks && at < 0; b0 += 32 * kWarps) {
      const int i = b0 + tid;
      const uint32_t m = __ballot_sync(kFull, i < blocks && __ldcg(&ta.cuts[i].begin) == i - 1);
      if (b0 > 1) __syncthreads();
      if (lane == 0) first[tid >> 5] = m;
      __syncthreads();
      for (int w = 0; w < kWarps && at < 0; ++w) {
        uint32_t bits = first[w];
        const int n = __popc(bits);
        if (left >= n) {
          left -= n;
          continue;
        }
        while (left--) bits &= bits - 1;
        at = b0 + 32 * w + __ffs(bits) - 1;
      }
    }
    if (at < 0) return;                                      // fewer items are divided
  }
  const Cut cut = ta.cuts[at];
  if (cut.begin != at - 1) return;
  const int r = blockIdx.z * kRows + tid % kRows, slice = tid / kRows, c0 = blockIdx.y * kCols;
  const int t = r / kTile, row_tok = r % kTile / ta.G, row_head = r % kTile % ta.G;
  const int tok = (cut.rb * NT + t) * ta.tq + row_tok;
  const int drafts = a.draft_lens ? min(max(__ldg(a.draft_lens + cut.b), 0), a.n) : a.n;
  const bool live = row_tok < ta.tq && tok < drafts;
  float m = -INFINITY, l = 0.f, v[kCols];
#pragma unroll
  for (int e = 0; e < kCols; ++e) v[e] = 0.f;
  if (live) {
    auto rec = [&](int x) { return ta.records + ((int64_t)x * 2 + (x == cut.begin ? 1 : 0)) * (D + 2) * S::rows + r; };
#pragma unroll 8
    for (int x = cut.begin + slice; x <= cut.end; x += kSlices) m = fmaxf(m, __ldcg(rec(x) + (int64_t)D * S::rows));
#pragma unroll 8
    for (int x = cut.begin + slice; x <= cut.end; x += kSlices) {
      const float* p = rec(x);
      const float mx = __ldcg(p + (int64_t)D * S::rows), lx = __ldcg(p + (int64_t)(D + 1) * S::rows);
      const float f = mx == -INFINITY ? 0.f : ex2(mx - m);
      l += mx == -INFINITY ? lx : lx * f;                    // nothing seen: 0, or NaN
#pragma unroll
      for (int e = 0; e < kCols; ++e) {
        const float y = __ldcg(p + (int64_t)(c0 + e) * S::rows);
        v[e] = f == 0.f ? v[e] : fmaf(y, f, v[e]);
      }
    }
  }
  if constexpr (kSlices > 1) {
    float (*mine)[kRows] = part[slice];
    const int k = tid % kRows;
    mine[0][k] = m;
    mine[1][k] = l;
#pragma unroll
    for (int e = 0; e < kCols; ++e) mine[2 + e][k] = v[e];
    __syncthreads();
    if (slice) return;
#pragma unroll
    for (int x = 1; x < kSlices; ++x) m = fmaxf(m, part[x][0][k]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kCols; ++e) v[e] = 0.f;
#pragma unroll
    for (int x = 0; x < kSlices; ++x) {
      const float mx = part[x][0][k], lx = part[x][1][k], f = mx == -INFINITY ? 0.f : ex2(mx - m);
      l += mx == -INFINITY ? lx : lx * f;
#pragma unroll
      for (int e = 0; e < kCols; ++e) v[e] = f == 0.f ? v[e] : fmaf(part[x][2 + e][k], f, v[e]);
    }
  }
  if (!live) return;
  const int64_t row = ((int64_t)cut.b * a.n + tok) * a.Hq + cut.h * ta.G + row_head;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (c0 < a.d) {
    T* out = static_cast<T*>(a.out) + row * a.d + c0;
#pragma unroll
    for (int e = 0; e < kCols; e += 4)
      *reinterpret_cast<uint2*>(out + e) = make_uint2(pack(v[e] * inv, v[e + 1] * inv, T()), pack(v[e + 2] * inv, v[e + 3] * inv, T()));
  }
  if (a.lse && blockIdx.y == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// raw rows of one page piece, swizzled so that eight keys' same 16 bytes lie in different banks
bool raw_map(CUtensorMap* m, const int8_t* base, int d, int64_t rows, int box) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)std::max<int64_t>(rows, 1)};
  cuuint64_t strides[1] = {(cuuint64_t)d};
  cuuint32_t boxd[2] = {(cuuint32_t)(d <= 64 ? 64 : 128), (cuuint32_t)box};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, boxd, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d <= 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, typename T>
int launch_shape(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, TcArgs ta, int grid, int merge,
                 void* workspace, cudaStream_t st) {
  using S = Shape<D, NT>;
  const int e = ensure_dyn_smem(reinterpret_cast<const void*>(tree_tc_kernel<D, NT, T>), S::bytes);
  if (e) return e;
  if (merge) {
    ta.cuts = static_cast<Cut*>(workspace);
    ta.records = reinterpret_cast<float*>(static_cast<char*>(workspace) + ((size_t)grid * sizeof(Cut) + 255) / 256 * 256);
  }
  tree_tc_kernel<D, NT, T><<<grid, kThreads, S::bytes, st>>>(qm, km, vm, ta);
  const int e2 = (int)cudaGetLastError();
  if (e2 || !merge) return e2;
  constexpr int kSlices = 4;
  if (merge * 4 < grid)                                      // more than four records an item
    return launch_beside(tree_tc_merge_kernel<D, NT, kSlices, T>,
                         dim3(merge, D / Merge<kSlices, NT>::cols, NT * kTile / Merge<kSlices, NT>::rows),
                         kSlices * Merge<kSlices, NT>::rows, st, ta, grid);
  return launch_beside(tree_tc_merge_kernel<D, NT, 1, T>, dim3(grid - 1, D / Merge<1, NT>::cols), NT * kTile, st, ta, grid);
}

int row_tiles(int64_t rows) { return rows <= kTile ? 1 : 2; }

}  // namespace

bool tree_tc_supported(const tq_ctx* h, int n, int Hq, int Hkv) {
  const int64_t G = Hq / Hkv;
  return h->d <= 128 && G <= kTile && n * G > kTreeTcRows;
}

size_t tree_tc_workspace(const tq_ctx* h, int n, int Hq, int Hkv) {
  const size_t grid = h->sm_count, rows = (size_t)row_tiles((int64_t)n * (Hq / Hkv)) * kTile;
  return (grid * sizeof(Cut) + 255) / 256 * 256 + grid * 2 * ((h->d <= 64 ? 64 : 128) + 2) * rows * 4;
}

int launch_tree_tc(const tq_ctx* h, const TreeArgs& a, int dtype, void* workspace, void* stream) {
  TcArgs ta{};
  ta.t = a;
  ta.G = a.Hq / a.Hkv, ta.tq = kTile / ta.G;
  ta.box = 64;
  while (a.page % ta.box) ta.box /= 2;   // page pieces that a tile never splits
  const bool bf = dtype == TQ_BF16;
  CUtensorMap qm, km, vm;
  const int64_t tokens = (int64_t)a.B * a.n;
  if (!token_map(&qm, a.q, bf, h->d, a.Hq, tokens, tokens > 1 ? a.q_stride : (int64_t)a.Hq * h->d, ta.G, ta.tq) ||
      !raw_map(&km, a.kcodes, h->d, a.rows, ta.box) || !raw_map(&vm, a.vcodes, h->d, a.rows, ta.box))
    return (int)cudaErrorInvalidValue;
  const int nt = row_tiles((int64_t)a.n * ta.G);
  const int64_t blocks = (a.n + nt * ta.tq - 1) / (nt * ta.tq), tiles = ((int64_t)a.max_pages * a.page + kTile - 1) / kTile;
  const int64_t items = (int64_t)a.B * a.Hkv * blocks;
  const int grid = (int)(items >= h->sm_count || tiles >= h->sm_count ? h->sm_count : std::min<int64_t>(h->sm_count, items * tiles));
  // items that may be divided
  const int merge = tiles > 1 ? (int)std::min<int64_t>(items, grid - 1) : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define TQ_TREE(D, NT)                                                                       \
  return bf ? launch_shape<D, NT, __nv_bfloat16>(qm, km, vm, ta, grid, merge, workspace, st) \
            : launch_shape<D, NT, __half>(qm, km, vm, ta, grid, merge, workspace, st)
  if (h->d <= 64) {
    if (nt == 1) TQ_TREE(64, 1);
    TQ_TREE(64, 2);
  }
  if (nt == 1) TQ_TREE(128, 1);
  TQ_TREE(128, 2);
#undef TQ_TREE
}

}  // namespace tqi
