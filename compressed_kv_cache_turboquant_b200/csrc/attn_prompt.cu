// Causal attention over packed prompts on the tensor cores (sm_100a).
//
// turboquant.net/zh, "实现步骤草图", 集成到 attention: the cache is compressed for the
// steps after the prompt; the prompt's own attention runs on the exact keys and
// values.  With a softmax in base 2 (c = scale log2 e, m_i a running reference
// of row i's largest logit),
//   S = Q K^T,  P = 2^(c S - m),  O += P V,  l += sum P,
//   out = O / l,  lse = (m + log2 l) ln 2.
// A row is a (token, head of a kv-head's group) pair: 128 / G tokens of a group
// of G heads fill the 128 rows of a tile, so every key tile serves all heads of
// its group.  A work item is two such row tiles of one sequence and kv-head, and
// the key tiles of 128 up to its last token.
//
// Q and K tiles are shared-memory operands, S and O accumulate in tensor memory,
// and P overwrites the first half of its S as the tensor-memory operand of the
// value product.  The two row tiles take turns: while one's softmax runs on the
// CUDA cores, the tensor cores work for the other.  At d <= 64, where O is half as
// wide, P has columns of its own, and a tile's next logits are computed beside its
// softmax (8192 tokens, 32 heads: 385 us; 427 with P in the place of S).  P is the inputs' type: one
// rounding of 2^-8 or 2^-11 relative (l sums the unrounded weights).  float16's range is
// short, so its weights are 2^7 larger (m lies 7 below the largest logit; O, l and lse
// follow): they reach 2^15 of 65504, and only below 2^-21 of the reference become
// subnormal, off by up to 2^-32 of it.  Without the 2^7 it was 2^-25: behind one
// dominant key, a tail of 131071 keys of 2^-25.2 each (2^-8.2 of the row together) was lost.
//
// Warps (384 threads, one block per SM, persistent over the items):
//   0-3, 4-7  softmax of row tile 0, 1: thread = row (TMEM lane); the reference
//             moves, and O is rescaled, only when a logit passes it by 2^8
//   8         TMA: the item's Q tiles, then K and V tiles through a ring
//   9         the MMA issuer
//   10, 11    look through the V tiles that some row does not see whole: an
//             infinity or NaN there, times a weight of 0, would spoil rows that
//             must not see it.  Such elements become 0 in shared memory, and the
//             rows that do see them add them at the end (a bit per key)
//
// What bounds it: a pair of row tiles passes a tile of 128 keys every 3460 cycles,
// 1870 of softmax (2^x: 16384 a tile at 16 a cycle for both tiles of the SM) and the
// row tile's own half value product (256), logits (512) and two hand-offs between
// the warps (330 each), which its softmax cannot overlap while P takes the place of
// S.  8192 tokens, 32 heads, d = 128: 0.478 ms, 1150 TFLOP/s of 1654 that the
// library's matrix product reaches; 32768 tokens 8.28 ms, 1062.
//
// Items are sorted by length of their key range, longest first, by a one-block
// kernel (prompt_plan_kernel: 6 us for 144 items; 0.14 ms of 2.39 for 65536 of them, 128
// heads of one kv-head, where an item is two tokens), and a block takes the next one when it has loaded
// its last tile (nine prompts, 8191 tokens in all, 16 heads of d = 64: 75 us; 86 with
// the list dealt out beforehand).  A grid with no more items than blocks finds
// them itself (six prompts, 331 tokens in all: 14.2 us, 17.2 with the list).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_common.cuh"
#include "tq_internal.h"

namespace tqi {
namespace {

using namespace attn;

constexpr int kTile = 128;                 // rows of a row tile, keys of a key tile
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 208, kRegsOther = 88;   // 2 x 208 + 88 = 3 x 168, the registers at launch
constexpr int kBadSlots = 8;               // items whose bad-key bits are kept (more than the ring can run ahead)
constexpr int kBadTiles = 4;               // key tiles of an item that some row does not see whole: 3 at most
constexpr int kBadWords = 4 + 4 * kBadTiles;   // what each scanning warp found in all (two words, two spare), then a bit per key
constexpr int kBuckets = 1024;
constexpr int kItemSlots = 4;              // items on their way to the warps
constexpr int kBarBytes = 448;             // room for the barriers and the tensor-memory address

template <int D>
struct Shape {
  static constexpr int slabs = D / 64;
  static constexpr int tile = kTile * D * 2;           // bytes of a Q, K or V tile
  // tensor memory: S of the two row tiles; O; and for D = 64, where that leaves room, P
  // apart from S, so that the next logits are under way while the softmax works
  static constexpr bool apart = D == 64;
  static constexpr uint32_t col_s = 0, col_p = apart ? 256 : 0, step_p = apart ? 64 : 128;
  static constexpr uint32_t col_o = apart ? 384 : 256, step_o = apart ? 64 : 128;
  static constexpr int stages = D == 128 ? 4 : 8;
  static constexpr int off_ring = 2 * tile;
  static constexpr int off_out = off_ring + stages * tile;   // [8 warps][32 rows][128 bytes] results
  static constexpr int off_bad = off_out + 8 * 32 * 128;     // [kBadSlots][kBadWords]
  static constexpr int off_bar = off_bad + kBadSlots * kBadWords * 4;
  static constexpr int bytes = off_bar + kBarBytes + 16 * (1 + kItemSlots) + 1024;
};

struct PromptArgs {
  const void* v;
  void* out;
  float* lse;
  const int32_t* cu;
  const int4* items;      // (first token, tokens, item of the sequence, 0), by key range
  int32_t* count;         // items, then the next of all their heads that no block has taken
  int64_t v_stride;
  int total, nseq, Hq, Hkv, d, G, tq;   // tq = 128 / G tokens of a row tile
  int direct;             // no plan: block i finds item i / Hkv
  int out_box;            // tokens in 32 rows, where they are whole (0: they are not)
  float scale_log2;
  int* status;
};

template <typename T>
struct Bits;   // exponent bits of a 16-bit element, and what lifts them into the sign when all are set
template <>
struct Bits<__nv_bfloat16> {
  static constexpr uint32_t exponent = 0x7F807F80u, one = 0x00800080u;
  static constexpr float raise = 0.f;   // weights are 2^raise times 2^(logit - the reference's)
};
template <>
struct Bits<__half> {
  static constexpr uint32_t exponent = 0x7C007C00u, one = 0x04000400u;
  static constexpr float raise = 7.f;
};

// two weights in the operand's type.  float16: the largest finite number for what would
// pass it, which logits of 2^24 and more can, whose own float32 rounding is 1 and more
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi, __nv_bfloat16) { return pack_bf16(lo, hi); }
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi, __half) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// sign bits of the halves that are infinite or NaN
template <typename T>
__device__ __forceinline__ uint32_t bad_halves(uint32_t w) {
  return ((w & Bits<T>::exponent) + Bits<T>::one) & 0x80008000u;
}

struct Item {
  int start, len;   // the sequence's first token and tokens
  int h;
  int tok[2];       // first token of each row tile, in the sequence
  int n[2];         // key tiles of each (0: no rows)
  int tiles;        // key tiles to load
};

// Lists the items of all sequences (one every 2 tq tokens), the longest key
// ranges first.  Bounds that fall below an earlier one or leave 0..total count
// as the nearest that do not, so the sequences never overlap and the list never
// holds more than total / (2 tq) + nseq items.
__global__ void __launch_bounds__(1024) prompt_plan_kernel(const int32_t* cu, int nseq, int total, int per_item,
                                                           int4* items, int32_t* count, int grid) {
  __shared__ int bound[4097];
  __shared__ int before[4097];              // items of the sequences before
  __shared__ int bucket[kBuckets];
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");   // the main grid sets itself up meanwhile
  // running maximum of the clamped bounds, then running sums of the items: 1024 at a time
  int carry = 0;
  for (int b0 = 0; b0 <= nseq; b0 += 1024) {
    const int i = b0 + tid;
    int v = i <= nseq ? min(max(cu[i], 0), total) : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v = max(v, x);
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    int m = carry;
    for (int w = 0; w < warp; ++w) m = max(m, warp_sum[w]);
    v = max(v, m);
    if (i <= nseq) bound[i] = v;
    for (int w = 0; w < 32; ++w) carry = max(carry, warp_sum[w]);
    __syncthreads();
  }
  carry = 0;
  for (int b0 = 0; b0 < nseq; b0 += 1024) {
    const int i = b0 + tid;
    const int own = i < nseq ? (bound[i + 1] - bound[i] + per_item - 1) / per_item : 0;
    int v = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    int m = carry;
    for (int w = 0; w < warp; ++w) m += warp_sum[w];
    if (i < nseq) before[i] = m + v - own;
    for (int w = 0; w < 32; ++w) carry += warp_sum[w];
    __syncthreads();
  }
  const int n = carry;
  if (tid == 0) before[nseq] = n, count[0] = n, count[1] = grid;
  bucket[tid] = 0;
  __syncthreads();
  // a bucket per key-range length (or so many of them alike that 1024 do)
  const int span = (total + per_item - 1) / per_item / kBuckets + 1;
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = tid; i < n; i += 1024) {
      int lo = 0, hi = nseq;                 // the last sequence with before <= i that has items
      while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= i) lo = mid; else hi = mid;
      }
      const int at = i - before[lo];
      int* b = &bucket[min(at / span, kBuckets - 1)];
      const int place = atomicAdd(b, 1);
      if (pass) items[place] = make_int4(bound[lo], bound[lo + 1] - bound[lo], at, 0);
    }
    __syncthreads();
    if (pass == 0) {
      // the longest first: a bucket begins behind all longer ones
      const int r = kBuckets - 1 - tid, own = bucket[r];
      int v = own;
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += x;
      }
      if (lane == 31) warp_sum[warp] = v;
      __syncthreads();
      for (int w = 0; w < warp; ++w) v += warp_sum[w];
      bucket[r] = v - own;
      __syncthreads();
    }
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap, PromptArgs a) {
  using S = Shape<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + S::off_ring;
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + S::off_bad);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::off_bar);   // [stages] tx
  uint64_t* empty = full + S::stages;    // [stages] MMA commit and both scanning warps
  uint64_t* q_full = empty + S::stages;  // tx
  uint64_t* q_free = q_full + 1;         // MMA commit: the item's logit products are done
  uint64_t* clean = q_free + 1;          // [stages] both scanning warps: looked through, where it needs that
  uint64_t* s_full = clean + S::stages;       // [2] MMA commit: logits of a tile
  uint64_t* p_ready = s_full + 2;        // [2][2] 4 softmax warps: weights of a tile's first, second 64 keys written
  uint64_t* pv_done = p_ready + 4;       // [2] MMA commit: value product done
  uint64_t* s_taken = pv_done + 2;       // [2] 4 softmax warps: logits of a tile read
  uint64_t* item_full = s_taken + 2;     // [kItemSlots] the TMA warp
  uint64_t* item_free = item_full + kItemSlots;   // [kItemSlots] every other warp at work
  uint64_t* done = item_free + kItemSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  int4* direct_item = reinterpret_cast<int4*>(smem + S::off_bar + kBarBytes);
  int4* slots = direct_item + 1;         // [kItemSlots] (first token, tokens, item of the sequence or -1, kv-head)
  static_assert((3 * S::stages + 13 + 2 * kItemSlots) * 8 + 4 <= kBarBytes && S::bytes <= 232448, "shared memory");

  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 3);
      mbar_init(&clean[s], 2);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_ready[2 * t], 4);
      mbar_init(&p_ready[2 * t + 1], 4);
      mbar_init(&pv_done[t], 1);
      mbar_init(&s_taken[t], 4);
    }
    for (int x = 0; x < kItemSlots; ++x) {
      mbar_init(&item_full[x], 1);
      mbar_init(&item_free[x], 8 + 1 + 2);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  if (a.direct && warp == 0) {
    // the sequence of item blockIdx.x / Hkv, with the plan's reading of the bounds
    int left = blockIdx.x / a.Hkv, prev = min(max(__ldg(a.cu), 0), a.total);
    int4 found = make_int4(0, 0, -1, 0);
    const int per_item = 2 * a.tq;
    for (int s0 = 0; s0 < a.nseq && found.z < 0; s0 += 32) {
      int v = s0 + lane < a.nseq ? min(max(__ldg(a.cu + s0 + lane + 1), 0), a.total) : 0;
      v = max(v, prev);
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v = max(v, x);
      }
      int first = __shfl_up_sync(kFull, v, 1);
      if (lane == 0) first = prev;
      const int own = (v - first + per_item - 1) / per_item;
      int upto = own;
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t past = __ballot_sync(kFull, upto > left);
      if (past) {
        const int who = __ffs(past) - 1;
        found = make_int4(__shfl_sync(kFull, first, who), __shfl_sync(kFull, v - first, who),
                          left - __shfl_sync(kFull, upto - own, who), 0);
      } else {
        left -= __shfl_sync(kFull, upto, 31);
        prev = __shfl_sync(kFull, v, 31);
      }
    }
    if (lane == 0) *direct_item = found;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (!a.direct) asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan is written
  // The block's items: the TMA warp takes the next one of the list whenever it is
  // about to run out, and tells the other warps
  const int all = a.direct ? 0 : __ldcg(a.count) * a.Hkv;
  auto entry = [&](int x) -> int4 {
    if (x >= all) return make_int4(0, 0, -1, 0);
    int4 e = __ldcg(a.items + x / a.Hkv);    // ld.cg: the plan may still be writing when this grid starts
    e.w = x % a.Hkv;
    return e;
  };
  auto unpack = [&](const int4& e, Item& it) {
    it.h = e.w;
    it.start = e.x;
    it.len = e.y;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      it.tok[t] = (e.z * 2 + t) * a.tq;
      it.n[t] = it.tok[t] < it.len ? (min(it.tok[t] + a.tq, it.len) - 1) / kTile + 1 : 0;
    }
    it.tiles = max(it.n[0], it.n[1]);
  };
  auto item = [&](int i, Item& it, bool& ok) -> bool {
    if (!ok || !(ok = mbar_wait_warp(&item_full[i % kItemSlots], (uint32_t)((i / kItemSlots) & 1)))) return false;
    const int4 e = slots[i % kItemSlots];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_free[i % kItemSlots]);
    if (e.z < 0) return false;
    unpack(e, it);
    return true;
  };
  // the first key tile that some row of the item does not see whole
  auto first_cut = [&](const Item& it) { return (it.tok[0] + 1) / kTile; };
  Item it;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
      // ---------------- TMA
      if (lane == 0) {
        int st = 0, queries = 0;
        bool ok = true;
        int4 e = a.direct ? make_int4(direct_item->x, direct_item->y, direct_item->z, blockIdx.x % a.Hkv) : entry(blockIdx.x);
        for (int i = 0;; ++i) {
          ok = mbar_wait(&item_free[i % kItemSlots], (uint32_t)(((i / kItemSlots) & 1) ^ 1));
          if (!ok) break;
          slots[i % kItemSlots] = e;
          mbar_arrive(&item_full[i % kItemSlots]);
          if (e.z < 0) break;
          unpack(e, it);
          auto load = [&](const CUtensorMap* map, int j) -> bool {
            const int s = st % S::stages;
            if (!mbar_wait(&empty[s], (uint32_t)(((st / S::stages) & 1) ^ 1))) return false;
            mbar_arrive_expect_tx(&full[s], S::tile);
            for (int sl = 0; sl < S::slabs; ++sl)
              tma_load_3d(map, &full[s], ring + s * S::tile + sl * kTile * 128, sl * 64, it.h, it.start + j * kTile);
            ++st;
            return true;
          };
          if (i > 0 && !mbar_wait(q_free, (uint32_t)((i - 1) & 1))) ok = false;
          if (ok) {
            const int rows = a.G * a.tq;
            ++queries;
            mbar_arrive_expect_tx(q_full, (uint32_t)((it.n[1] ? 2 : 1) * S::slabs * rows * 128));
            for (int t = 0; t < (it.n[1] ? 2 : 1); ++t)
              for (int sl = 0; sl < S::slabs; ++sl)
                tma_load_3d(&qmap, q_full, smem + t * S::tile + sl * kTile * 128, sl * 64, it.h * a.G,
                            it.start + it.tok[t]);
          }
          for (int j = 0; ok && j < it.tiles; ++j) ok = load(&kmap, j) && load(&vmap, j);
          if (!ok) break;
          e = a.direct ? make_int4(0, 0, -1, 0) : entry(atomicAdd(a.count + 1, 1));
          // the next item's queries cannot be loaded before this one's last logits:
          // have them on their way to L2 until then
          if (e.z >= 0)
            for (int t = 0; t < 2; ++t)
              for (int sl = 0; sl < S::slabs; ++sl)
                tma_prefetch_3d(&qmap, sl * 64, e.w * a.G, min(e.x + (e.z * 2 + t) * a.tq, a.total - 1));
        }
        if (!ok) atomicOr(a.status, kStatusTimeout);
        // no copy may still be in flight when the block ends
        for (int x = st > S::stages ? st - S::stages : 0; x < st; ++x)
          if (!mbar_wait(&full[x % S::stages], (uint32_t)((x / S::stages) & 1))) atomicOr(a.status, kStatusTimeout);
        if (queries && !mbar_wait(q_full, (uint32_t)((queries - 1) & 1))) atomicOr(a.status, kStatusTimeout);
      }
    } else if (warp == 9) {
      // ---------------- MMA
      constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
      constexpr uint32_t kColS = S::col_s, kColP = S::col_p, kColO = S::col_o;
      constexpr uint32_t idesc_s = idesc_f16(kTile, kTile, bf), idesc_o = idesc_f16(kTile, D, bf) | (1u << 16);
      const uint32_t lead = elect_one();
      const uint64_t qd = sw128_kmajor_desc(smem_u32(smem)), kd = sw128_kmajor_desc(smem_u32(ring));
      const uint64_t vd = sw128_mnmajor_desc(smem_u32(ring), kTile * 128);
      int st = 0, pv0 = 0, pv1 = 0;                         // ring steps; value products of tiles 0, 1 so far
      int qk[2] = {0, 0};                                   // logit products of tiles 0, 1
      bool ok = true;
      auto wait_full = [&](int x) { return mbar_wait_warp(&full[x % S::stages], (uint32_t)((x / S::stages) & 1)); };
      // S of tile t from the K tile of ring step x; the buffer's last S must have been
      // read, or the P that took its place consumed
      auto logits = [&](int t, int pv, int x) -> bool {
        if (S::apart) {
          if (qk[t] > 0 && !mbar_wait_warp(&s_taken[t], (uint32_t)((qk[t] - 1) & 1))) return false;
          ++qk[t];
        } else {
          if (pv > 0 && !mbar_wait_warp(&pv_done[t], (uint32_t)((pv - 1) & 1))) return false;
        }
        tc_fence_after();
        const uint64_t q = qd + t * (S::tile >> 4), k = kd + (uint32_t)(x % S::stages) * (S::tile >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (uint32_t)((ks >> 2) * kTile * 128 + (ks & 3) * 32) >> 4;
          mma_ss(tmem + kColS + t * 128, q + off, k + off, idesc_s, ks ? 1u : 0u, lead);
        }
        commit(&s_full[t], lead);
        return true;
      };
      auto values = [&](int t, int pv, int x, bool first) -> bool {
        const uint64_t v = vd + (uint32_t)(x % S::stages) * (S::tile >> 4);
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks) {
          // the weights come in two halves
          if (ks % (kTile / 32) == 0) {
            if (!mbar_wait_warp(&p_ready[2 * t + ks / (kTile / 32)], (uint32_t)(pv & 1))) return false;
            tc_fence_after();
          }
          mma_ts(tmem + kColO + t * S::step_o, tmem + kColP + t * S::step_p + 8 * ks, v + ks * (2048 >> 4), idesc_o,
                 (first && ks == 0) ? 0u : 1u, lead);
        }
        commit(&pv_done[t], lead);
        return true;
      };
      for (int i = 0; item(i, it, ok); ++i) {
        ok = mbar_wait_warp(q_full, (uint32_t)(i & 1)) && wait_full(st) && (!it.n[0] || logits(0, pv0, st)) &&
             (!it.n[1] || logits(1, pv1, st));
        if (!ok) break;
        commit(&empty[st % S::stages], lead);
        if (it.tiles == 1) commit(q_free, lead);
        const int cut = first_cut(it);
        for (int j = 0; j < it.tiles; ++j) {
          const int xv = st + 2 * j + 1, xk = xv + 1;
          // a tile that some row does not see whole has to be looked through first
          ok = wait_full(xv) && (j < cut || mbar_wait_warp(&clean[xv % S::stages], (uint32_t)((xv / S::stages) & 1)));
          if (!ok) break;
          const bool more = j + 1 < it.tiles;
          if constexpr (S::apart) {
            if (more && !(ok = wait_full(xk))) break;
            if (j + 1 < it.n[0] && !(ok = logits(0, 0, xk))) break;
            if (j < it.n[0] && !(ok = values(0, pv0++, xv, j == 0))) break;
            if (j + 1 < it.n[1] && !(ok = logits(1, 0, xk))) break;
            if (more) commit(&empty[xk % S::stages], lead);
            if (j + 2 == it.tiles) commit(q_free, lead);
            if (j < it.n[1] && !(ok = values(1, pv1++, xv, j == 0))) break;
            commit(&empty[xv % S::stages], lead);
          } else {
            if (j < it.n[0] && !(ok = values(0, pv0++, xv, j == 0))) break;
            if (more && !(ok = wait_full(xk))) break;
            if (j + 1 < it.n[0] && !(ok = logits(0, pv0, xk))) break;
            if (j < it.n[1] && !(ok = values(1, pv1++, xv, j == 0))) break;
            commit(&empty[xv % S::stages], lead);
            if (j + 1 < it.n[1] && !(ok = logits(1, pv1, xk))) break;
            if (more) commit(&empty[xk % S::stages], lead);
            if (j + 2 == it.tiles) commit(q_free, lead);
          }
        }
        st += 2 * it.tiles;
      }
      if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
      // nothing may still run when tensor memory is given back
      commit(done, lead);
      if (!mbar_wait_warp(done, 0) && lane == 0) atomicOr(a.status, kStatusTimeout);
    } else {
      // ---------------- V tiles that some row does not see whole
      const int w = warp - 10;
      int st = 0;
      bool ok = true;
      for (int i = 0; item(i, it, ok); ++i) {
        uint32_t* bits = bad + (i % kBadSlots) * kBadWords;
        uint32_t found = 0;
        const int cut = first_cut(it);
        for (int j = 0; j < it.tiles; ++j) {
          for (int kv = 0; kv < 2; ++kv, ++st) {
            const int s = st % S::stages;
            if (!(ok = mbar_wait_warp(&full[s], (uint32_t)((st / S::stages) & 1)))) break;
            if (kv && j >= cut) {
              // lane = key of a 32-key group: two groups a warp
              uint8_t* vt = ring + s * S::tile;
              for (int gr = 0; gr < 2; ++gr) {
                const int key = w * 64 + gr * 32 + lane;
                bool any = false;
                // keys up to the item's first token are seen by all its rows
                const int chunks = j * kTile + w * 64 + gr * 32 + 31 <= it.tok[0] ? 0 : D / 8;
#pragma unroll 4
                for (int u = 0; u < chunks; ++u) {
                  uint4* p = reinterpret_cast<uint4*>(vt + (u >> 3) * kTile * 128 + key * 128 + (((u & 7) ^ (key & 7)) << 4));
                  uint4 x = *p;
                  const uint32_t b0 = bad_halves<T>(x.x), b1 = bad_halves<T>(x.y), b2 = bad_halves<T>(x.z), b3 = bad_halves<T>(x.w);
                  if (b0 | b1 | b2 | b3) {
                    any = true;
                    // a set sign bit -> a half of zeros
                    x.x &= ~((b0 >> 15) * 0xFFFFu), x.y &= ~((b1 >> 15) * 0xFFFFu);
                    x.z &= ~((b2 >> 15) * 0xFFFFu), x.w &= ~((b3 >> 15) * 0xFFFFu);
                    *p = x;
                  }
                }
                const uint32_t m = __ballot_sync(kFull, any);
                found |= m;
                if (lane == 0) bits[4 + (j - cut) * 4 + w * 2 + gr] = m;
              }
              if (lane == 0) bits[w] = found;
              fence_async_smem();
              __syncwarp();
            }
            // every step of the ring, so that neither side ever runs two uses of a stage ahead
            if (lane == 0) {
              mbar_arrive(&clean[s]);
              mbar_arrive(&empty[s]);
            }
          }
          if (!ok) break;
        }
      }
      if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
    }
  } else {
    // ---------------- softmax: thread = row of tile t
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sc = tmem + lanes + S::col_s + t * 128, pc = tmem + lanes + S::col_p + t * S::step_p;
    const uint32_t oc = tmem + lanes + S::col_o + t * S::step_o;
    const int row_tok = r / a.G, row_head = r % a.G;
    const int warp_tok = __shfl_sync(kFull, row_tok, 0);    // of the warp's first row
    const float cl = a.scale_log2;
    uint8_t* stage = smem + S::off_out + warp * 32 * 128;
    int steps = 0;
    bool ok = true;
    for (int i = 0; item(i, it, ok); ++i) {
      const int n = it.n[t];
      if (n == 0) continue;
      const int pos = it.tok[t] + row_tok;                  // the row's token in its sequence
      const bool live = row_tok < a.tq && pos < it.len;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++steps) {
        if (!(ok = mbar_wait_warp(&s_full[t], (uint32_t)(steps & 1)))) break;
        tc_fence_after();
        float x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(sc + 32 * c, x[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) regs_after_wait(x[c]);
        if (S::apart) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_taken[t]);
        }
        // keys past the row's own take no part; a group of 32 that the warp's
        // first row sees whole needs no look
        const int lim = pos - j * kTile, low = it.tok[t] + warp_tok - j * kTile;
        if (low < kTile - 1) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (low < 32 * c + 31) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[c][e] = 32 * c + e <= lim ? x[c][e] : -INFINITY;
            }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = max3(x[c][0], x[c][1], x[c][2]);
#pragma unroll
          for (int e = 3; e + 1 < 32; e += 2) mx[c] = max3(mx[c], x[c][e], x[c][e + 1]);
          mx[c] = max3(mx[c], x[c][31], x[c][31]);
        }
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]) * cl;
        if (!(top < INFINITY)) l = NAN;                     // a seen logit is NaN or infinite: so is the row
        const bool grow = top > m + (kLazy + Bits<T>::raise) || (m == -INFINITY && top > m);
        // O and the weights' buffer are free once the value product of tile j - 1 is done
        // (where these logits took the weights' place, it was done before them)
        if (S::apart && j > 0) {
          if (!(ok = mbar_wait_warp(&pv_done[t], (uint32_t)((steps - 1) & 1)))) break;
          tc_fence_after();
        }
        if (__any_sync(kFull, grow)) {
          float f = 1.f;
          if (grow) {
            const float next = top - Bits<T>::raise;
            f = m == -INFINITY ? 0.f : ex2(m - next);
            l *= f;
            m = next;
          }
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(oc + c, o);
              tmem_wait_ld();
              uint32_t u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                asm volatile("" : "+f"(o[e])::"memory");
                u[e] = __float_as_uint(f == 0.f ? 0.f : o[e] * f);
              }
              tmem_st16(oc + c, u);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t cl2 = pair(cl, cl), ref2 = pair(-ref, -ref);
        uint64_t sum[2] = {0, 0};
        // half the keys at a time: the value product of the first half runs during the second
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              uint64_t z = fma2(pair(x[c][2 * e], x[c][2 * e + 1]), cl2, ref2);
              float p0, p1;
              unpair(z, p0, p1);
              p0 = ex2(p0), p1 = ex2(p1);
              sum[e & 1] = add2(sum[e & 1], pair(p0, p1));
              u[e] = pack_weights(p0, p1, T());
            }
            tmem_st16(pc + 16 * c, u);
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
      if (!(ok = mbar_wait_warp(&pv_done[t], (uint32_t)((steps - 1) & 1)))) break;
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t row = (int64_t)(it.start + pos) * a.Hq + it.h * a.G + row_head;
      const int cut = first_cut(it);
      const uint32_t* bits = bad + (i % kBadSlots) * kBadWords;
      const uint32_t some = it.tiles > cut ? bits[0] | bits[1] : 0u;
      bits += 4;
      // whole tokens of the group in the warp's rows, all of the sequence: one TMA
      // store per 64 coordinates, which nothing waits for but the next use of the
      // buffer (stores by the lanes hold the warps for as long as memory takes)
      const int first = it.tok[t] + warp_tok, tokens = a.out_box;
      const bool whole = tokens > 0 && first + tokens <= it.len;
#pragma unroll 1
      for (int sl = 0; sl < S::slabs; ++sl) {
        float o[2][32];
        tmem_ld32(oc + 64 * sl, o[0]);
        tmem_ld32(oc + 64 * sl + 32, o[1]);
        tmem_wait_ld();
        if (lane == 0) bulk_wait_read<0>();                 // the buffer's last store has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          regs_after_wait(o[c]);
          if (some) {
            // infinities and NaN that the row does see, taken out of the V tiles above
            for (int x = 0; x < (it.tiles - cut) * 4; ++x)
              for (uint32_t b = bits[x]; b; b &= b - 1) {
                const int key = cut * kTile + x * 32 + __ffs(b) - 1;
                if (!live || key > pos) continue;
                const T* v = static_cast<const T*>(a.v) + (int64_t)(it.start + key) * a.v_stride + (int64_t)it.h * a.d;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const float y = 64 * sl + 32 * c + e < a.d ? (float)v[64 * sl + 32 * c + e] : 0.f;
                  if (!(fabsf(y) < INFINITY)) o[c][e] += y;
                }
              }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float* y = o[c] + 8 * u;
            uint4 w;
            w.x = pack(y[0] * inv, y[1] * inv, T());
            w.y = pack(y[2] * inv, y[3] * inv, T());
            w.z = pack(y[4] * inv, y[5] * inv, T());
            w.w = pack(y[6] * inv, y[7] * inv, T());
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c + u) ^ (lane & 7)) << 4)) = w;
          }
        }
        if (whole) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&omap, stage, sl * 64, it.h * a.G, it.start + first);
            bulk_commit();
          }
        } else {
          __syncwarp();
#pragma unroll 1
          for (int k = 0; k < 32; k += 4) {                 // eight lanes a row
            const int x = k + (lane >> 3), y = (warp & 3) * 32 + x, tok = y / a.G, col = sl * 64 + (lane & 7) * 8;
            if (tok < a.tq && it.tok[t] + tok < it.len && col < a.d)
              *reinterpret_cast<uint4*>(static_cast<T*>(a.out) +
                                        ((int64_t)(it.start + it.tok[t] + tok) * a.Hq + it.h * a.G + y % a.G) * a.d + col) =
                  *reinterpret_cast<const uint4*>(stage + x * 128 + (((lane & 7) ^ (x & 7)) << 4));
          }
          __syncwarp();
        }
      }
      if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      tc_fence_before();
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
    if (lane == 0) bulk_wait_all();                         // the buffer is read until then
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// more items than this never come out of `total` tokens in `nseq` sequences
int64_t most_items(int nseq, int64_t total, int tq) { return total / (2 * tq) + nseq; }

template <int D, typename T>
int launch_main(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& om, const PromptArgs& a, int grid,
                cudaStream_t st) {
  const int e = ensure_dyn_smem(reinterpret_cast<const void*>(prompt_kernel<D, T>), Shape<D>::bytes);
  if (e) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<D>::bytes;
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = a.direct ? 0 : 1;   // beside the plan's kernel
  return (int)cudaLaunchKernelEx(&cfg, prompt_kernel<D, T>, qm, km, vm, om, a);
}

}  // namespace

size_t prompt_workspace(const tq_ctx* h, int nseq, int64_t total, int Hq, int Hkv) {
  if (nseq == 0 || total == 0 || Hq < Hkv || Hq / Hkv > kTile) return 0;
  const int64_t items = most_items(nseq, total, kTile / (Hq / Hkv));
  return items * Hkv <= h->sm_count ? 0 : 256 + (size_t)items * sizeof(int4);
}

int launch_prompt(const tq_ctx* h, const void* q, const void* k, const void* v, int dtype, const int32_t* cu, int nseq,
                  int64_t total, int Hq, int Hkv, int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                  void* out, float* lse, void* workspace, void* stream) {
  PromptArgs a{};
  const bool bf = dtype == TQ_BF16;
  a.v = v, a.out = out, a.lse = lse, a.cu = cu;
  a.G = Hq / Hkv, a.tq = kTile / a.G;
  // one token has no stride of its own
  const int64_t vs = total > 1 ? v_stride : (int64_t)Hkv * h->d;
  a.v_stride = vs, a.total = (int)total, a.nseq = nseq, a.Hq = Hq, a.Hkv = Hkv, a.d = h->d;
  // never 0: masked logits are -infinity before they are scaled, and 0 times that is NaN
  a.scale_log2 = std::max(scale * 1.4426950408889634f, 1e-37f);
  a.status = h->dev.status;
  a.out_box = 32 % a.G ? 0 : 32 / a.G;
  CUtensorMap qm, km, vm, om;
  if (!token_map(&qm, q, bf, h->d, Hq, total, total > 1 ? q_stride : (int64_t)Hq * h->d, a.G, a.tq) ||
      !token_map(&km, k, bf, h->d, Hkv, total, total > 1 ? k_stride : (int64_t)Hkv * h->d, 1, kTile) ||
      !token_map(&vm, v, bf, h->d, Hkv, total, vs, 1, kTile) ||
      !token_map(&om, out, bf, h->d, Hq, total, (int64_t)Hq * h->d, a.G, std::max(a.out_box, 1)))
    return (int)cudaErrorInvalidValue;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t work = most_items(nseq, total, a.tq) * Hkv;
  a.direct = work <= h->sm_count;
  if (!a.direct) {
    a.count = static_cast<int32_t*>(workspace);
    a.items = reinterpret_cast<const int4*>(static_cast<char*>(workspace) + 256);
    prompt_plan_kernel<<<1, 1024, 0, st>>>(cu, nseq, (int)total, 2 * a.tq, const_cast<int4*>(a.items),
                                           a.count, (int)std::min<int64_t>(work, h->sm_count));
    const int e = (int)cudaGetLastError();
    if (e) return e;
  }
  const int grid = (int)std::min<int64_t>(work, h->sm_count);
  if (h->d <= 64)
    return bf ? launch_main<64, __nv_bfloat16>(qm, km, vm, om, a, grid, st) : launch_main<64, __half>(qm, km, vm, om, a, grid, st);
  return bf ? launch_main<128, __nv_bfloat16>(qm, km, vm, om, a, grid, st) : launch_main<128, __half>(qm, km, vm, om, a, grid, st);
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
  if (Hq > INT32_MAX / (128 * h->d)) return set_error(TQ_EUNSUPPORTED, "%s: Hq = %d", fn, Hq);
  if (Hq / Hkv > 128) return set_error(TQ_EUNSUPPORTED, "%s: %d query heads per kv-head (at most 128)", fn, Hq / Hkv);
  if (nseq > TQ_MAX_SEQS) return set_error(TQ_EUNSUPPORTED, "%s: nseq = %d (at most %d)", fn, nseq, TQ_MAX_SEQS);
  if (total > INT32_MAX / 128 || (total + nseq) * Hkv > INT32_MAX / 2)
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
