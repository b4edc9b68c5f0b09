// Checkpoint-slot planning shared by the one-CTA planner kernels of branching
// layers (misc.cu, prefill.cu, rows.cu).
#pragma once

#include "rssm_device.cuh"

namespace rssm {
namespace {

// Exclusive prefix sum of one int per thread over the block (blockDim.x a
// multiple of 32, at most 1024); `total` is the block's sum.
__device__ __forceinline__ void block_scan(int v, int &excl, int &total) {
  __shared__ int warp_tot[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += t;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = lane < nw ? warp_tot[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(kFull, w, d);
      if (lane >= d) w += t;
    }
    if (lane < nw) warp_tot[lane] = w;   // inclusive over warps
  }
  __syncthreads();
  excl = inc - v + (warp > 0 ? warp_tot[warp - 1] : 0);
  total = warp_tot[nw - 1];
  __syncthreads();   // warp_tot is reused by the next call
}

// A fold of the previous launch wrote row b's new checkpoint to dst[b] and
// counted itself in flushes[b]: make that slot the row's own.
__device__ __forceinline__ void adopt_folds(int B, int32_t *slot, const int32_t *dst, int32_t *seen,
                                            const int32_t *flushes) {
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const int f = flushes[b];
    if (f != seen[b]) {
      slot[b] = dst[b];
      seen[b] = f;
    }
  }
}

// The ids of the slots (0 .. 2B-1) that no row reads, packed at the front of
// freelist; returns their number (at least B: rows read at most B slots).
// Called by the whole block.
__device__ __forceinline__ int free_slots(int B, const int32_t *slot, int32_t *freelist) {
  const int S = 2 * B, nt = blockDim.x;
  for (int s = threadIdx.x; s < S; s += nt) freelist[s] = 1;
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += nt) {
    const int sl = slot[b];
    if (sl >= 0 && sl < S) freelist[sl] = 0;
  }
  __syncthreads();
  // compact the free slot ids to the front, tile by tile (a tile's flags are
  // read before any id is written, and ids land at or before their slot)
  int nfree = 0;
  for (int s0 = 0; s0 < S; s0 += nt) {
    const int s = s0 + threadIdx.x;
    const int flag = s < S ? freelist[s] : 0;
    __syncthreads();
    int excl, tot;
    block_scan(flag, excl, tot);
    if (flag) freelist[nfree + excl] = s;
    nfree += tot;
    __syncthreads();
  }
  return nfree;
}

}  // namespace
}  // namespace rssm
