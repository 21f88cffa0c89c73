// What the two kernels of tq_attn_tree share: how the work of ragged sequences
// is cut into equal ranges, and where the parts of a divided item go.
#pragma once

#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "tq_internal.h"

namespace tqi {
namespace tree {

using attn::kFull;

// A block owns two records of the workspace (value sums, maximum and sum of every
// row): the first for an item that began in an earlier block, the second for one
// that goes on in a later one.  This says which item the first belongs to.
struct Cut {
  int b, h, rb;
  int begin, end;  // the blocks that hold the item's first and last unit; begin < 0: no such item
};

struct Seq {
  int ctx, T, drafts, tiles, blocks;  // blocks of rows
};

template <int kKeys>
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b, int rows_per_block) {
  Seq s;
  const int cap = a.max_pages * a.page;
  s.drafts = a.draft_lens ? min(max(__ldg(a.draft_lens + b), 0), a.n) : a.n;
  s.ctx = max(__ldg(a.ctx_lens + b), 0);
  s.T = (int)min((int64_t)s.ctx + s.drafts, (int64_t)cap);
  s.tiles = (s.T + kKeys - 1) / kKeys;
  s.blocks = (s.drafts * (a.Hq / a.Hkv) + rows_per_block - 1) / rows_per_block;
  return s;
}

__device__ __forceinline__ int64_t units_of(const TreeArgs& a, const Seq& s) {
  return (int64_t)a.Hkv * s.blocks * s.tiles;
}

// one work item's share of a block: tiles lo .. hi - 1 of kv-head h, rows block rb
struct Piece {
  Seq s;
  int b, h, rb, lo, hi;
  int64_t begin;  // first unit of the item
};

// walks the pieces of units u .. end - 1; b, base: a sequence at or before u's and its first unit
template <int kKeys>
struct Walk {
  int64_t u, end, base;
  int64_t total;
  int b, blocks;
  // the block that unit x belongs to: the last whose range begins at or before it
  __device__ __forceinline__ int block_of(int64_t x) const { return (int)(((x + 1) * blocks - 1) / total); }
  __device__ __forceinline__ Cut cut_of(const Piece& p) const {
    return Cut{p.b, p.h, p.rb, block_of(p.begin), block_of(p.begin + p.s.tiles - 1)};
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, int rows_per_block, Piece& p) {
    if (u >= end) return false;
    p.s = seq_of<kKeys>(a, b, rows_per_block);
    int64_t n = units_of(a, p.s);
    while (u - base >= n) {
      base += n;
      ++b;
      p.s = seq_of<kKeys>(a, b, rows_per_block);
      n = units_of(a, p.s);
    }
    const int64_t item = (u - base) / p.s.tiles;
    p.b = b;
    p.h = (int)(item / p.s.blocks);
    p.rb = (int)(item % p.s.blocks);
    p.begin = base + item * p.s.tiles;
    p.lo = (int)(u - p.begin);
    p.hi = (int)min((int64_t)p.s.tiles, p.lo + (end - u));
    u += p.hi - p.lo;
    return true;
  }
};

// The units [u0, u1) of this block: the tiles of all items, cut into as many equal
// ranges as there are blocks (no more than units, so that none between two others
// is idle), and the sequence that u0 lies in.  Called by the whole block; scratch
// holds 2 + warps words.  False: nothing to do.
template <int kKeys, int kThreads>
__device__ __forceinline__ bool range_of_block(const TreeArgs& a, int rows, int64_t* scratch, Walk<kKeys>& walk) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t* part = scratch + 2;
  int64_t sum = 0;
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    const Seq s = seq_of<kKeys>(a, b, rows);
    sum += units_of(a, s);
    const int cl = __ldg(a.ctx_lens + b);
    if (blockIdx.x == 0 && (cl < 0 || (int64_t)s.ctx + s.drafts > s.T || (a.draft_lens && __ldg(a.draft_lens + b) != s.drafts)))
      atomicOr(a.status, sm100::kStatusRange);
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) total += part[w];
  const int64_t blocks = min((int64_t)gridDim.x, total);
  if (blockIdx.x >= blocks) return false;
  walk.total = total;
  walk.blocks = (int)blocks;
  walk.u = total * blockIdx.x / blocks;
  walk.end = total * (blockIdx.x + 1) / blocks;
  if (warp == 0) {
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int64_t mine = b0 + lane < a.B ? units_of(a, seq_of<kKeys>(a, b0 + lane, rows)) : 0;
      int64_t upto = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t past = __ballot_sync(kFull, base + upto > walk.u);
      if (past) {
        if (lane == __ffs(past) - 1) scratch[0] = b0 + lane, scratch[1] = base + upto - mine;
        break;
      }
      base += __shfl_sync(kFull, upto, 31);
    }
  }
  __syncthreads();
  walk.b = (int)scratch[0];
  walk.base = scratch[1];
  return true;
}

// Launches a kernel that may start beside the grid before it (and waits for it by
// griddepcontrol.wait).
template <typename... P, typename... A>
int launch_beside(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace tree
}  // namespace tqi
