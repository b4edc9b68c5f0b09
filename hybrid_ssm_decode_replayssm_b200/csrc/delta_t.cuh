// T = (I + A)^-1 of a chunk of 64 tokens of the delta rules (gdn_prefill.cu, kda_prefill.cu).
#pragma once

#include "chunk.cuh"

namespace rssm {
namespace chunk {

constexpr int kPart = 8192;                 // 64 x 64 bf16
constexpr int kALd = 68, kTLd = 36, kXLd = 20;   // floats per row of A^T, of 32-wide and of 16-wide blocks
constexpr int kFloatsTab = 32 * kTLd, kFloatsX = 4 * 16 * kXLd;   // of sTa or sTb, of sX
static_assert(32 * kTLd <= kFloatsX, "the blocks on the way");

// Pairs of parts whose product matters in fp32.  Sums run from the small parts to the
// large: the tensor core truncates each addition, and only those of the last, large
// parts then count (1.1e-6 of the result's norm in the other order, 8192 tokens).
// (1,1) (0,2) (2,0) (0,1) (1,0) (0,0), four bits each, for loops that stay rolled: code in a
// straight line waits for its instructions (GDN, 8192 tokens on 32 heads: 701 us against 686).
__device__ __forceinline__ uint32_t part_a(int c) { return 0x010201u >> (4 * c) & 3u; }
__device__ __forceinline__ uint32_t part_b(int c) { return 0x001021u >> (4 * c) & 3u; }

// (4 x NC outputs) sum_k L[k][r..r+3] R[k][c..c+NC-1], k < n: the left operand is stored
// by columns, the right by rows.
template <int NC>
__device__ __forceinline__ void block_product(float (&o)[4][NC], const float *L, int ll, const float *Rr, int lr, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float4 x = *reinterpret_cast<const float4 *>(L + k * ll);
    float y[NC];
    if constexpr (NC == 2) {
      const float2 v = *reinterpret_cast<const float2 *>(Rr + k * lr);
      y[0] = v.x; y[1] = v.y;
    } else {
      y[0] = Rr[k * lr];
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      o[0][c] = fmaf(x.x, y[c], o[0][c]);
      o[1][c] = fmaf(x.y, y[c], o[1][c]);
      o[2][c] = fmaf(x.z, y[c], o[2][c]);
      o[3][c] = fmaf(x.w, y[c], o[3][c]);
    }
  }
}

// From A^T, [s][t], in sA (only s < t is read) to the three parts of T at `to`, [t][s] in the
// 128-byte swizzle; 128 threads.  In fp32 by blocks: sixteen-wide diagonal blocks by
// substitution, one per warp, a column per lane; then T_10 = -T_11 (A_10 T_00) for pairs of
// blocks, and again for pairs of those.  sTa, T's first 32 rows and columns [row][column],
// and sTb, its last 32, [column][row], are zero above the diagonal; sX: blocks on the way.
__device__ __forceinline__ void invert_store(const float *sA, float *sTa, float *sTb, float *sX, uint8_t *to, int t) {
  const int lane = t & 31, w = t >> 5;
  {
    const int c = lane & 15;
    float acc[16], val[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      val[k] = k == c ? 1.f : -acc[k];
#pragma unroll
      for (int j = (k + 1) / 4 * 4; j < 16; j += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(sA + (w * 16 + k) * kALd + w * 16 + j);
        const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e > k) acc[j + e] = fmaf(xs[e], val[k], acc[j + e]);
      }
    }
    if (lane < 16) {
      const int o = (w & 1) * 16;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        if (w < 2) sTa[(o + k) * kTLd + o + c] = val[k];
        if (w == 1) sX[c * kXLd + k] = val[k];                    // T_11 by columns
        if (w == 2) sX[(16 + k) * kXLd + c] = val[k];             // T_22 by rows
      }
      if (w >= 2) {
#pragma unroll
        for (int k = 0; k < 16; k += 4)
          *reinterpret_cast<float4 *>(sTb + (o + c) * kTLd + o + k) = make_float4(val[k], val[k + 1], val[k + 2], val[k + 3]);
      }
    }
  }
  __syncthreads();
  {
    const int pr = w >> 1, id2 = t & 63, c = id2 & 15, r4 = (id2 >> 4) * 4;
    float x[4][1];
    float *sXp = sX + (32 + pr * 16) * kXLd;
    block_product<1>(x, sA + (pr * 32) * kALd + pr * 32 + 16 + r4, kALd, pr ? sX + 16 * kXLd + c : sTa + c,
                     pr ? kXLd : kTLd, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) sXp[(r4 + e) * kXLd + c] = x[e][0];
    __syncthreads();
    block_product<1>(x, pr ? sTb + 16 * kTLd + 16 + r4 : sX + r4, pr ? kTLd : kXLd, sXp + c, kXLd, 16);
    if (pr) {
      *reinterpret_cast<float4 *>(sTb + c * kTLd + 16 + r4) = make_float4(-x[0][0], -x[1][0], -x[2][0], -x[3][0]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) sTa[(16 + r4 + e) * kTLd + c] = -x[e][0];
    }
  }
  __syncthreads();
  {
    const int c = (t & 15) * 2, r4 = (t >> 4) * 4;
    auto put = [&](int row, int col, float v0, float v1) {
      uint32_t hi, mid, lo;
      split3(v0, v1, hi, mid, lo);
      uint8_t *at = to + sw128(row, col >> 3) + (col & 7) * 2;
      *reinterpret_cast<uint32_t *>(at) = hi;
      *reinterpret_cast<uint32_t *>(at + kPart) = mid;
      *reinterpret_cast<uint32_t *>(at + 2 * kPart) = lo;
    };
    float x[4][2];
    block_product<2>(x, sA + 32 + r4, kALd, sTa + c, kTLd, 32);
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<float2 *>(sX + (r4 + e) * kTLd + c) = make_float2(x[e][0], x[e][1]);
    __syncthreads();
    block_product<2>(x, sTb + r4, kTLd, sX + c, kTLd, 32);
    const float4 b0 = *reinterpret_cast<const float4 *>(sTb + c * kTLd + r4);
    const float4 b1 = *reinterpret_cast<const float4 *>(sTb + (c + 1) * kTLd + r4);
    const float y0[4] = {b0.x, b0.y, b0.z, b0.w}, y1[4] = {b1.x, b1.y, b1.z, b1.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = *reinterpret_cast<const float2 *>(sTa + (r4 + e) * kTLd + c);
      put(r4 + e, c, v.x, v.y);
      put(r4 + e, 32 + c, 0.f, 0.f);
      put(32 + r4 + e, c, -x[e][0], -x[e][1]);
      put(32 + r4 + e, 32 + c, y0[e], y1[e]);
    }
  }
}

}  // namespace chunk
}  // namespace rssm
