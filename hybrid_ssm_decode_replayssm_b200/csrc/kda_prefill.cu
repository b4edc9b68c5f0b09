// Chunked delta rule with a gate per key channel (KDA, bf16 inputs, headdim = dstate = 128)
// on the 5th-generation tensor cores: one CTA per (sequence, head), chunks of 64 tokens.
//
// With p_t the running product of the gates inside the chunk (a value per channel), d_ts that
// of the gates s+1 .. t, f_s that of the gates behind s, and S [dv, dk] the state before it:
//   A_ts = b_t sum_c d_ts k_t k_s (s < t)      T = (I + A)^-1
//   M_ts = scale sum_c d_ts q_t k_s (s <= t)
//   W = T R,  R_t = b_t (v_t - S (p_t k_t))
//   O_t = scale S (p_t q_t) + sum_{s<=t} M_ts w_s
//   S' = S diag(p_last) + sum_s w_s (f_s k_s)^T
// Every gate product is a product, never a ratio, so none overflows and gates of 0 hold.
// As in the kernel of scalar gates everything that depends on the state is computed transposed,
// one value row per tensor-memory lane; here both operands of every product are fp32 in three
// bf16 parts, six products each:
//   U^T = S K^T, Z^T = S Q^T (K, Q: p_t k_t, p_t q_t), W^T = R^T T^T, S' += W^T F
//   (F: f_s k_s), O^T = W^T M^T
// T and M come from a kernel before (kda_pre_kernel), which has no chain to wait for.
//
// Bound by the chain S -> U -> R -> W -> S' of one chunk after the other, 12800 cycles a chunk
// (of them 6200 the tensor core's, by its counter), and before it by the instructions of
// kda_pre_kernel, 12 us per SM for a chunk and head.  8192 tokens on 32 heads: 1265 us, of them
// 350 in kda_pre_kernel (0.45 GB of inputs, outputs and states); four tokens at a time on the
// CUDA cores 1800; 8 sequences of 1024 tokens 602 against 1440.  The products unrolled take 10%
// more cycles a chunk: their instructions are waited for.
#include "delta_t.cuh"
#include "rssm_prefill.h"

namespace rssm {
namespace {

using namespace chunk;

constexpr int kT = 64;                      // tokens per chunk
constexpr int kD = 128;
constexpr int kBlk = 16384;                 // 128 rows x 64 bf16
constexpr int kRecord = 6 * kPart;          // a chunk and head in the workspace: the parts of T, of M

// ------------------------------------------------------------------ T and M
// One CTA of four warps per (chunk, head), four of them per SM, 32 channels at a time.  By
// blocks of sixteen tokens: between blocks d_ts = (gates of t's block up to t) x (those of
// whole blocks between) x (those behind s in its block), so that A and M are plain products of
// scaled keys and queries; inside a block each lane takes a column s and runs the product along t.
// In fp32 on the CUDA cores.
constexpr int kPreThreads = 128;
constexpr int kCh = 32, kLd = 36;           // channels at a time, floats per row of them
constexpr int kArr = kT * kLd;
constexpr int kMLd = 68;
// floats: k, q, g as they are; k, q by the gates before, k by those behind; products of whole blocks
constexpr int kFE = 6 * kArr, kFB = kFE + 4 * kCh, kFAll = kFB + kT;
// in their place afterwards: A^T, T's tables, M
constexpr int kFTa = kT * kALd, kFTb = kFTa + kFloatsTab, kFX = kFTb + kFloatsTab, kFM = kFX + kFloatsX;
static_assert(kFM + kT * kMLd <= kFE, "in the place of the operands");
constexpr int kSmemPre = kFAll * 4;

__device__ __forceinline__ float dot4(const float4 &a, const float4 &b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ float4 mul4(const float4 &a, const float4 &b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

__global__ void __launch_bounds__(kPreThreads, 4) kda_pre_kernel(const PrefillArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  float *sm = reinterpret_cast<float *>(smem);
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  float *rk = sm, *rq = sm + kArr, *rg = sm + 2 * kArr, *hk = sm + 3 * kArr, *hq = sm + 4 * kArr, *fk = sm + 5 * kArr;
  float *sE = sm + kFE;            // the gates of whole blocks
  float *sB = sm + kFB;
  float *sA = sm, *sTa = sm + kFTa, *sTb = sm + kFTb, *sX = sm + kFX, *sM = sm + kFM;
  grid_wait();
  grid_launch_next();
  const int total = a.queue[kChunkTotal], longs = a.queue[kLongCount];
  if (longs == 0) return;
  for (size_t id = blockIdx.x; id < (size_t)total * a.H; id += gridDim.x) {
    const int h = (int)(id % a.H), chunk = (int)(id / a.H);
    int lo = 0, hi = longs - 1;   // the last sequence that begins at or before this chunk (and is not empty)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.seqs[mid].first <= chunk) lo = mid;
      else hi = mid - 1;
    }
    const PrefillSeq q = a.seqs[lo];
    const int t0 = (chunk - q.first) * kT, left = q.n - t0;
    const __nv_bfloat16 *pq = static_cast<const __nv_bfloat16 *>(a.in[0]) + (size_t)h * kD + lane;
    const __nv_bfloat16 *pk = static_cast<const __nv_bfloat16 *>(a.in[1]) + (size_t)h * kD + lane;
    const float *pg = static_cast<const float *>(a.in[3]) + (size_t)h * kD + lane;
    if (t < kT) sB[t] = t < left ? static_cast<const float *>(a.in[4])[(int64_t)(q.tok + t0 + t) * a.stride[4] + h] : 0.f;
    // products between blocks: unit w + 4 j is A (j, then w, below 6) or M of one pair of blocks;
    // a lane has four rows (rg + 4 i) and two columns (cg + 8 j)
    float off[3][4][2];
#pragma unroll
    for (int u = 0; u < 3; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) off[u][i][0] = off[u][i][1] = 0.f;
    const int rgp = lane >> 3, cgp = lane & 7;
    float da[16], dm[16];          // inside block w: column s, rows 0 .. 15
#pragma unroll
    for (int j = 0; j < 16; ++j) da[j] = dm[j] = 0.f;
    const int ds = lane & 15, dh = (lane >> 4) * 16;
    auto blocks = [](int pr, int &I, int &J) {   // (1,0) (2,1) (3,2) (2,0) (3,1) (3,0)
      I = pr < 3 ? pr + 1 : pr == 3 ? 2 : 3;
      J = pr < 3 ? pr : pr == 4 ? 1 : 0;
    };
    for (int c0 = 0; c0 < kD; c0 += kCh) {
      __syncthreads();   // the last channels, or the last item, are read
      {   // sixteen tokens of one channel
        float g[16];
        __nv_bfloat16 k[16], x[16];
        const int64_t first = q.tok + t0 + w * 16;
        const int mine = left - w * 16;   // zeros and gates of 1 behind the end
        const float *at_g = pg + first * a.stride[3] + c0;
        const __nv_bfloat16 *at_k = pk + first * a.stride[1] + c0, *at_q = pq + first * a.stride[0] + c0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          g[j] = 1.f;
          k[j] = x[j] = __nv_bfloat16(0.f);
          if (j < mine) {
            g[j] = __ldg(at_g);
            k[j] = __ldg(at_k);
            x[j] = __ldg(at_q);
          }
          at_g += a.stride[3];
          at_k += a.stride[1];
          at_q += a.stride[0];
        }
        float p = 1.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int s = (w * 16 + j) * kLd + lane;
          const float kj = __bfloat162float(k[j]), xj = __bfloat162float(x[j]);
          p *= g[j];
          rk[s] = kj;
          rq[s] = xj;
          rg[s] = g[j];
          hk[s] = kj * p;
          hq[s] = xj * p;
        }
        float f = 1.f;
#pragma unroll
        for (int j = 15; j >= 0; --j) {
          fk[(w * 16 + j) * kLd + lane] = __bfloat162float(k[j]) * f;
          f *= g[j];
        }
        sE[w * kCh + lane] = p;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        const int unit = w + 4 * u, pr = unit >= 6 ? unit - 6 : unit;
        int I, J;
        blocks(pr, I, J);
        const float *X = (unit >= 6 ? hq : hk) + (I * 16 + rgp) * kLd, *Y = fk + (J * 16 + cgp) * kLd;
        const float *e1 = sE + (J + 1) * kCh, *e2 = sE + 2 * kCh;
#pragma unroll 2
        for (int c = 0; c < kCh; c += 4) {
          float4 y[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) y[j] = *reinterpret_cast<const float4 *>(Y + j * 8 * kLd + c);
          if (pr >= 3) {
            float4 e = *reinterpret_cast<const float4 *>(e1 + c);
            if (pr == 5) e = mul4(e, *reinterpret_cast<const float4 *>(e2 + c));
            y[0] = mul4(y[0], e);
            y[1] = mul4(y[1], e);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(X + i * 4 * kLd + c);
            off[u][i][0] = dot4(x, y[0], off[u][i][0]);
            off[u][i][1] = dot4(x, y[1], off[u][i][1]);
          }
        }
      }
#pragma unroll 1
      for (int c = dh; c < dh + 16; c += 4) {
        const int at = w * 16 * kLd + c;
        float4 x = *reinterpret_cast<const float4 *>(rk + at + ds * kLd);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float4 g = *reinterpret_cast<const float4 *>(rg + at + j * kLd);
          if (j > ds) x = mul4(x, g);
          da[j] = dot4(*reinterpret_cast<const float4 *>(rk + at + j * kLd), x, da[j]);
          dm[j] = dot4(*reinterpret_cast<const float4 *>(rq + at + j * kLd), x, dm[j]);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const int unit = w + 4 * u, pr = unit >= 6 ? unit - 6 : unit;
      int I, J;
      blocks(pr, I, J);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = I * 16 + rgp + 4 * i, col = J * 16 + cgp + 8 * j;
          if (unit >= 6) sM[row * kMLd + col] = a.out_scale * off[u][i][j];
          else sA[col * kALd + row] = sB[row] * off[u][i][j];
        }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = da[j] + __shfl_xor_sync(0xffffffffu, da[j], 16), y = dm[j] + __shfl_xor_sync(0xffffffffu, dm[j], 16);
      const int row = w * 16 + j, col = w * 16 + ds;
      if (lane < 16) {
        sA[col * kALd + row] = j > ds ? sB[row] * x : 0.f;
        sM[row * kMLd + col] = j >= ds ? a.out_scale * y : 0.f;
      }
    }
    for (int i = t; i < 2 * kFloatsTab + kFloatsX; i += kPreThreads) sTa[i] = 0.f;
    __syncthreads();
    uint8_t *to = a.parts + id * kRecord;
    for (int i = t; i < kT * 8; i += kPreThreads) {   // M, eight columns at a time, zero above the diagonal blocks
      const int row = i >> 3, c = i & 7;
      uint4 o[3];
      uint32_t *u = reinterpret_cast<uint32_t *>(o);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (c >> 1) <= (row >> 4) ? sM[row * kMLd + c * 8 + j] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) split3(v[2 * j], v[2 * j + 1], u[j], u[4 + j], u[8 + j]);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4 *>(to + (3 + p) * kPart + sw128(row, c)) = o[p];
    }
    invert_store(sA, sTa, sTb, sX, to, t);
  }
}

// ------------------------------------------------------------------ the chain
// Roles: warps 0-7 the chain (one value row per lane, two halves of the columns); warps 8-15
// scale and split K, Q and F and take the outputs away; warp 16 issues the products; warps
// 18-19 load V, T and M.  Every barrier completes once per chunk, and none can complete again
// before its waiters have passed.
constexpr int kThreadsK = 640;
// registers per thread: 256 x 128 + 256 x 88 + 128 x 48 = 640 x 96
constexpr int kRegsLaunch = 96, kRegsChain = 128, kRegsOut = 88, kRegsRest = 48;
static_assert(256 * kRegsChain + 256 * kRegsOut + 128 * kRegsRest <= kThreadsK * kRegsLaunch, "registers of the CTA");
constexpr int kOffKQ = 0;                   // three parts of 128 rows (0-63 K, 64-127 Q), two column blocks each
constexpr int kOffF = kOffKQ + 6 * kBlk;    // three parts of 64 rows, two column blocks each
constexpr int kOffT = kOffF + 6 * kPart;    // three parts, [t][s]
constexpr int kOffM = kOffT + 3 * kPart;
constexpr int kOffV = kOffM + 3 * kPart;    // [t][dv]
constexpr int kOffSc = kOffV + kBlk;        // b [64], p_last [2][128], gates of every eight tokens [2][8][128]
constexpr int kOffBar = kOffSc + (kT + 18 * kD) * 4;
enum { kKQ = 0, kSp0, kSp1, kVf, kTf, kMf, kF, kU, kQ, kRp, kW, kWp, kUpd, kO, kOfree, kTot, kDrain, kBars };
constexpr int kSmemK = kOffBar + kBars * 8 + 32;
static_assert(kSmemK <= 232448, "shared memory of one CTA");
// tensor memory columns: U^T, then W^T; Z^T; the parts of S; of W, in the second half of every 32
// columns of S's (which are read by then, and written last); the state's update, before it
// the parts of R; O^T
constexpr int kTmU = 0, kTmZ = 64, kTmS = 128, kTmW = kTmS + 16, kTmD = 320, kTmR = 320, kTmO = 448;

__global__ void __launch_bounds__(kThreadsK, 1) kda_chunk_kernel(const PrefillArgs a) {
  grid_wait();
  grid_launch_next();
  if (a.queue[kLongCount] == 0) return;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kOffBar);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffBar + kBars * 8);
  uint32_t *tm_slot = reinterpret_cast<uint32_t *>(smem + kOffBar + kBars * 8 + 8);
  float *s_be = reinterpret_cast<float *>(smem + kOffSc), *s_dec = s_be + kT, *s_tot = s_dec + 2 * kD;
  const uint32_t base = smem_u32(smem);
  constexpr int count[kBars] = {8, 8, 8, 64, 1, 1, 8, 1, 1, 8, 1, 8, 1, 1, 8, 8, 1};
  if (t == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bar + i, count[i]);
    abort[0] = abort[1] = 0;   // the second is never set
    mbar_fence_init();
  }
  if (warp == 16) {
    umma::alloc(tm_slot, 512);
    umma::relinquish();
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tm = *tm_slot;
  const long long lim = a.wait_limit;
  PrefillSeq q;
  int h, *s_item = reinterpret_cast<int *>(smem + kOffBar + kBars * 8 + 12);
  auto next = [&]() { return next_item<kThreadsK, kBars>(a, bar, count, s_item, abort, q, h); };

  if (warp < 8) {
    // -------------------------------------------------------- the chain
    more_registers<kRegsChain>();
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    float S[64];
    if (q.src < 0) {
#pragma unroll
      for (int c = 0; c < 64; ++c) S[c] = 0.f;
    } else {
      const float *src = a.hc + (((size_t)q.src * a.H + h) * kD + row) * kD + wg * 64;
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 v = ld_stream(src + c);
        S[c] = v.x; S[c + 1] = v.y; S[c + 2] = v.z; S[c + 3] = v.w;
      }
    }
    bool good = true;
    if (a.stall_test && blockIdx.x == 0) stall_on_unset_flag(const_cast<int *>(abort) + 1, abort, lim);
    for (int i = 0;; ++i) {
      const uint32_t ph = i & 1;
      const bool more = i < chunks;
      const float *dec = s_dec + (ph ^ 1) * kD + wg * 64;
#pragma unroll
      for (int c = 0; c < 64; c += 16) {   // the state before chunk i, and its parts
        if (c == 32 && more && i > 0) {   // the parts of W, where these go, are read
          good = warp_wait(bar + kO, ph ^ 1, abort, lim);
          umma::fence_after_sync();
        }
        if (i > 0) {
          float d[16];
          umma::ld_32x32b_x16(lanes + kTmD + wg * 64 + c, d);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 e = *reinterpret_cast<const float4 *>(dec + c + j);
            S[c + j] = fmaf(e.x, S[c + j], d[j]);
            S[c + j + 1] = fmaf(e.y, S[c + j + 1], d[j + 1]);
            S[c + j + 2] = fmaf(e.z, S[c + j + 2], d[j + 2]);
            S[c + j + 3] = fmaf(e.w, S[c + j + 3], d[j + 3]);
          }
        }
        if (more) {
          split_store(lanes + kTmS + wg * 32 + c / 2, 64, S + c);
          if (c & 16) {
            wait_st();
            umma::fence_before_sync();
            warp_arrive(bar + kSp0 + (c >> 5));
          }
        }
      }
      umma::fence_before_sync();
      if (!more || !good) break;
      good = warp_wait(bar + kVf, ph, abort, lim);
      if (!good) break;
      float v[32];   // v of this half's 32 tokens
      {
        const __nv_bfloat16 *pv = reinterpret_cast<const __nv_bfloat16 *>(smem + kOffV) + wg * 32 * kD + row;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __bfloat162float(pv[j * kD]);
      }
      good = warp_wait(bar + kU, ph, abort, lim);
      if (!good) break;
      umma::fence_after_sync();
#pragma unroll
      for (int c = 0; c < 32; c += 16) {   // R
        float u[16];
        umma::ld_32x32b_x16(lanes + kTmU + wg * 32 + c, u);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 b = *reinterpret_cast<const float4 *>(s_be + wg * 32 + c + j);
          v[c + j] = b.x * (v[c + j] - u[j]);
          v[c + j + 1] = b.y * (v[c + j + 1] - u[j + 1]);
          v[c + j + 2] = b.z * (v[c + j + 2] - u[j + 2]);
          v[c + j + 3] = b.w * (v[c + j + 3] - u[j + 3]);
        }
        split_store(lanes + kTmR + wg * 16 + c / 2, 32, v + c);
      }
      wait_st();
      umma::fence_before_sync();
      warp_arrive(bar + kRp);
      good = warp_wait(bar + kW, ph, abort, lim);
      if (!good) break;
      umma::fence_after_sync();
      umma::ld_32x32b_x32(lanes + kTmU + wg * 32, v);
#pragma unroll
      for (int c = 0; c < 32; c += 16) split_store(lanes + kTmW + wg * 32 + c / 2, 64, v + c);
      wait_st();
      umma::fence_before_sync();
      good = warp_wait(bar + kF, ph, abort, lim);   // p_last is there; before the arrival that lets F's barrier go on
      warp_arrive(bar + kWp);
      if (!good) break;
      good = warp_wait(bar + kUpd, ph, abort, lim);
      if (!good) break;
      umma::fence_after_sync();
    }
    if (good) {
      float *dst = a.hc + (((size_t)q.dst * a.H + h) * kD + row) * kD + wg * 64;
#pragma unroll
      for (int c = 0; c < 64; c += 8) st_sector(dst + c, S + c);
    }
    }
  } else if (warp < 16) {
    // ------------------------------------- K, Q and F, and the outputs of the chunk before
    fewer_registers<kRegsOut>();
    // four tokens of eight channels per thread: half a warp has whole rows, a warp eight tokens
    const int w8 = warp - 8, tg = w8 * 2 + (lane >> 4), ch = (lane & 15) * 8;
    const int wg = (warp - 8) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    const __nv_bfloat16 *pq = static_cast<const __nv_bfloat16 *>(a.in[0]) + (size_t)h * kD + ch;
    const __nv_bfloat16 *pk = static_cast<const __nv_bfloat16 *>(a.in[1]) + (size_t)h * kD + ch;
    const float *pg = static_cast<const float *>(a.in[3]) + (size_t)h * kD + ch;
    // what a token gives: zeros and gates of 1 behind the end
    auto load_gates = [&](float4 (&g)[2], int s) {
      const float4 *p = reinterpret_cast<const float4 *>(pg + (int64_t)(q.tok + s) * a.stride[3]);
      g[0] = g[1] = make_float4(1.f, 1.f, 1.f, 1.f);
      if (s < q.n) g[0] = __ldg(p), g[1] = __ldg(p + 1);
    };
    auto load_row = [&](uint4 &x, const __nv_bfloat16 *p, int64_t stride, int s) {
      x = make_uint4(0, 0, 0, 0);
      if (s < q.n) x = __ldg(reinterpret_cast<const uint4 *>(p + (int64_t)(q.tok + s) * stride));
    };
    auto times = [](float (&p)[8], const float4 (&g)[2]) {
      p[0] *= g[0].x; p[1] *= g[0].y; p[2] *= g[0].z; p[3] *= g[0].w;
      p[4] *= g[1].x; p[5] *= g[1].y; p[6] *= g[1].z; p[7] *= g[1].w;
    };
    // eight scaled values of a row to their three parts
    auto put = [&](uint8_t *to, int step, const float (&p)[8], const uint4 &raw) {
      const uint32_t y[4] = {raw.x, raw.y, raw.z, raw.w};
      uint4 o[3];
      uint32_t *d = reinterpret_cast<uint32_t *>(o);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        split3(p[2 * c] * __uint_as_float(y[c] << 16), p[2 * c + 1] * __uint_as_float(y[c] & 0xFFFF0000u), d[c], d[4 + c],
               d[8 + c]);
#pragma unroll
      for (int c = 0; c < 3; ++c) *reinterpret_cast<uint4 *>(to + c * step) = o[c];
    };
    // the tokens' arrays move down by one as they are used: the loops stay rolled
    float4 g[4][2];
    uint4 k[4];
    auto down_by_one = [&]() {
#pragma unroll
      for (int j = 0; j < 3; ++j) g[j][0] = g[j + 1][0], g[j][1] = g[j + 1][1], k[j] = k[j + 1];
    };
    for (int i = 0; i <= chunks; ++i) {
      const uint32_t ph = i & 1;
      const int s0 = i * kT + tg * 4;
      float *tot = s_tot + ph * 8 * kD;   // the products of every warp's eight tokens
      if (i < chunks) {
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) load_gates(g[j], s0 + j);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_row(k[j], pk, a.stride[1], s0 + j);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_row(x[j], pq, a.stride[0], s0 + j);
        float p[8];   // the gates of the tokens before the four
        {
          float all[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) all[c] = 1.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) times(all, g[j]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float y = __shfl_xor_sync(0xffffffffu, all[c], 16);
            p[c] = lane < 16 ? 1.f : y;
            all[c] *= y;
          }
          if (lane < 16) {
            float4 *d = reinterpret_cast<float4 *>(tot + w8 * kD + ch);
            d[0] = make_float4(all[0], all[1], all[2], all[3]);
            d[1] = make_float4(all[4], all[5], all[6], all[7]);
          }
        }
        warp_arrive(bar + kTot);
        if (!warp_wait(bar + kTot, ph, abort, lim)) break;
#pragma unroll 1
        for (int v = 0; v < w8; ++v) {
          const float4 *d = reinterpret_cast<const float4 *>(tot + v * kD + ch);
          const float4 e[2] = {d[0], d[1]};
          times(p, e);
        }
        if (i > 0 && !warp_wait(bar + kQ, ph ^ 1, abort, lim)) break;
        uint8_t *to = smem + kOffKQ + (ch >> 6) * kBlk;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          times(p, g[0]);
          uint8_t *at = to + sw128(tg * 4 + j, (ch >> 3) & 7);
          put(at, 2 * kBlk, p, k[0]);
          put(at + kPart, 2 * kBlk, p, x[0]);
          down_by_one();
          x[0] = x[1];
          x[1] = x[2];
          x[2] = x[3];
        }
        fence_proxy_async();
        warp_arrive(bar + kKQ);
      }
      if (i > 0) {   // a value row per lane, half of the tokens
        if (!warp_wait(bar + kO, ph ^ 1, abort, lim)) break;
        umma::fence_after_sync();
        const int left = q.n - (i - 1) * kT - wg * 32;
        const size_t step = (size_t)a.H * kD;
        float *o = a.out + ((size_t)(q.tok + (i - 1) * kT + wg * 32) * a.H + h) * kD + r;
#pragma unroll 1
        for (int c = 0; c < 32; c += 16) {
          float z[16], m[16];
          umma::ld_32x32b_x16(lanes + kTmZ + wg * 32 + c, z);
          umma::ld_32x32b_x16(lanes + kTmO + wg * 32 + c, m);
          if (c == 16) {
            umma::fence_before_sync();
            warp_arrive(bar + kOfree);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j, o += step)
            if (c + j < left) __stcs(o, fmaf(a.out_scale, z[j], m[j]));
        }
      }
      if (i < chunks) {
#pragma unroll
        for (int j = 0; j < 4; ++j) load_gates(g[3 - j], s0 + j);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_row(k[3 - j], pk, a.stride[1], s0 + j);
        float p[8];   // the gates behind these four
        {
          float all[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) all[c] = 1.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) times(all, g[j]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float y = __shfl_xor_sync(0xffffffffu, all[c], 16);
            p[c] = lane < 16 ? y : 1.f;
          }
        }
#pragma unroll 1
        for (int v = w8 + 1; v < 8; ++v) {
          const float4 *d = reinterpret_cast<const float4 *>(tot + v * kD + ch);
          const float4 e[2] = {d[0], d[1]};
          times(p, e);
        }
        if (i > 0 && !warp_wait(bar + kUpd, ph ^ 1, abort, lim)) break;
        uint8_t *to = smem + kOffF + (ch >> 6) * kPart;
#pragma unroll 1
        for (int j = 3; j >= 0; --j) {
          put(to + sw128(tg * 4 + j, (ch >> 3) & 7), 2 * kPart, p, k[0]);
          times(p, g[0]);
          down_by_one();
        }
        if (tg == 0) {   // p_last; read by the chain before the next chunk but one, whose update comes later
          float4 *d = reinterpret_cast<float4 *>(s_dec + ph * kD + ch);
          d[0] = make_float4(p[0], p[1], p[2], p[3]);
          d[1] = make_float4(p[4], p[5], p[6], p[7]);
        }
        fence_proxy_async();
        warp_arrive(bar + kF);
      }
    }
    }
  } else if (warp == 16) {
    // -------------------------------------------------------- the products
    fewer_registers<kRegsRest>();
    // descriptors: the address, in units of 16 bytes, is in the low bits
    const uint64_t dK = desc_sw128(base + kOffKQ, 16), dQ = desc_sw128(base + kOffKQ + kPart, 16);
    const uint64_t dT = desc_sw128(base + kOffT, 16), dM = desc_sw128(base + kOffM, 16), dF = desc_sw128(base + kOffF, kPart);
    auto done = [&](int b) {
      if (elect_one()) umma::commit(bar + b);
      __syncwarp();
    };
    // S (over half of the columns: 32 from either half of the chain) with K or Q
    auto state_product = [&](uint32_t d, uint64_t tile, int half) {
      if (elect_one()) {
#pragma unroll 1
        for (int c = 0; c < 6; ++c) {
          const uint32_t at = tm + kTmS + part_a(c) * 64;
          const uint64_t b = tile + part_b(c) * (2 * kBlk / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int kk = (k & 1) + 4 * (k >> 1) + 2 * half;
            mma_ts(tm + d, at + kk * 8, b + ((kk / 4) * kBlk + (kk % 4) * 32) / 16, idesc(128, kT, false, false),
                   half > 0 || c > 0 || k > 0);
          }
        }
      }
      __syncwarp();
    };
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    bool good = true;
    for (int i = 0; i < chunks; ++i) {
      const uint32_t ph = i & 1;
      good = false;
      if (!warp_wait(bar + kKQ, ph, abort, lim)) break;
      if (!warp_wait(bar + kSp0, ph, abort, lim)) break;
      umma::fence_after_sync();
      state_product(kTmU, dK, 0);
      if (!warp_wait(bar + kSp1, ph, abort, lim)) break;
      umma::fence_after_sync();
      state_product(kTmU, dK, 1);
      done(kU);
      if (i > 0 && !warp_wait(bar + kOfree, ph ^ 1, abort, lim)) break;
      umma::fence_after_sync();
      state_product(kTmZ, dQ, 0);   // while the chain makes R
      state_product(kTmZ, dQ, 1);
      done(kQ);
      if (!warp_wait(bar + kRp, ph, abort, lim) || !warp_wait(bar + kTf, ph, abort, lim)) break;
      umma::fence_after_sync();
      if (elect_one()) {
#pragma unroll 1
        for (int c = 0; c < 6; ++c) {
          const uint32_t at = tm + kTmR + part_a(c) * 32;
          const uint64_t b = dT + part_b(c) * (kPart / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ts(tm + kTmU, at + k * 8, b + k * 2, idesc(128, kT, false, false), c + k > 0);
        }
        umma::commit(bar + kW);
      }
      __syncwarp();
      if (!warp_wait(bar + kWp, ph, abort, lim) || !warp_wait(bar + kF, ph, abort, lim)) break;
      umma::fence_after_sync();
      if (elect_one()) {
#pragma unroll 1
        for (int c = 0; c < 6; ++c) {
          const uint32_t at = tm + kTmW + part_a(c) * 64;
          const uint64_t b = dF + part_b(c) * (2 * kPart / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tm + kTmD, at + (k >> 1) * 32 + (k & 1) * 8, b + k * 128, idesc(128, kD, false, true), c + k > 0);
        }
        umma::commit(bar + kUpd);
      }
      __syncwarp();
      if (!warp_wait(bar + kMf, ph, abort, lim)) break;
      umma::fence_after_sync();
      if (elect_one()) {   // the outputs, while the chain splits the next state
#pragma unroll 1
        for (int c = 0; c < 6; ++c) {
          const uint32_t at = tm + kTmW + part_a(c) * 64;
          const uint64_t b = dM + part_b(c) * (kPart / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tm + kTmO, at + (k >> 1) * 32 + (k & 1) * 8, b + k * 2, idesc(128, kT, false, false), c + k > 0);
        }
        umma::commit(bar + kO);
      }
      __syncwarp();
      good = true;
    }
    // the arrivals that nobody else waits for, before the barriers start anew
    if (good && chunks > 0) warp_wait(bar + kQ, (chunks - 1) & 1, abort, lim);
    }
  } else if (warp == 17) {
    fewer_registers<kRegsRest>();
    while (next()) {
    }
  } else {
    // -------------------------------------------------------- tiles
    fewer_registers<kRegsRest>();
    const int l = t - 576;   // 0..63
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    const __nv_bfloat16 *pv = static_cast<const __nv_bfloat16 *>(a.in[2]) + (size_t)h * kD;
    const float *pb = static_cast<const float *>(a.in[4]) + h;
    int t_issued = 0, m_issued = 0;
    for (int i = 0; i < chunks; ++i) {
      const uint32_t before = (i & 1) ^ 1;
      const uint8_t *rec = a.parts + ((size_t)(q.first + i) * a.H + h) * kRecord;
      if (i > 0 && !warp_wait(bar + kRp, before, abort, lim)) break;
      const int left = q.n - i * kT;
      const int64_t first = q.tok + i * kT;
      const int c = l & 15;
#pragma unroll
      for (int k = 0; k < kT / 4; ++k) {
        const int s = k * 4 + (l >> 4);
        cp_async16_zfill(base + kOffV + s * 256 + c * 16, s < left ? pv + (first + s) * a.stride[2] + c * 8 : pv, s < left);
      }
      s_be[l] = l < left ? __ldg(pb + (first + l) * a.stride[4]) : 0.f;
      cp_commit();
      cp_wait<0>();
      mbar_arrive(bar + kVf);
      if (i > 0 && !warp_wait(bar + kW, before, abort, lim)) break;
      if (l == 0) {
        mbar_arrive_expect_tx(bar + kTf, 3 * kPart);
        bulk_g2s(smem + kOffT, rec, 3 * kPart, bar + kTf);
      }
      t_issued = i + 1;
      if (i > 0 && !warp_wait(bar + kO, before, abort, lim)) break;
      if (l == 0) {
        mbar_arrive_expect_tx(bar + kMf, 3 * kPart);
        bulk_g2s(smem + kOffM, rec + 3 * kPart, 3 * kPart, bar + kMf);
      }
      m_issued = i + 1;
    }
    cp_async_wait_all();
    // the bulk copies have landed before this CTA goes on, or ends, whatever came
    if (l == 0) {
      if (t_issued > 0) mbar_wait_bounded(bar + kTf, (t_issued - 1) & 1, nullptr, lim);
      if (m_issued > 0) mbar_wait_bounded(bar + kMf, (m_issued - 1) & 1, nullptr, lim);
    }
    __syncwarp();
    }
  }
  // -------------------------------------------------------- end
  __syncwarp();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  if (warp == 16) {
    if (*abort) {   // products may still be in flight: wait for them before their memory goes
      if (lane == 0) {
        umma::commit(bar + kDrain);
        mbar_wait_bounded(bar + kDrain, 0, nullptr, lim);
      }
      __syncwarp();
    }
    umma::dealloc(tm, 512);
  }
  if (t == 0 && *abort) atomicOr(a.status, (unsigned)RSSM_STATUS_TIMEOUT);
}

}  // namespace

bool kda_chunk_path(const PrefillArgs &a, int in_dtype) {
  return a.kind == RSSM_KDA && in_dtype == RSSM_BF16 && a.R == kD && a.C == kD;
}

size_t kda_chunk_work(size_t chunks, int H) { return chunks * H * kRecord; }

cudaError_t kda_chunk_prefill(const PrefillArgs &a, cudaStream_t s) {
  cudaError_t e = allow_smem(kda_pre_kernel, kSmemPre);
  if (e == cudaSuccess) e = allow_smem(kda_chunk_kernel, kSmemK);
  if (e != cudaSuccess) return e;
  const size_t chunks = most_chunks(a.n_seq, a.n_tokens, a.scan_most) * a.H, items = (size_t)a.n_seq * a.H;
  e = launch_early(kda_pre_kernel, (unsigned)(chunks < 4 * kPrefillSms ? chunks : 4 * kPrefillSms), kPreThreads, kSmemPre,
                   s, a);
  if (e != cudaSuccess) return e;
  return launch_early(kda_chunk_kernel, (unsigned)(items < kPrefillSms ? items : kPrefillSms), kThreadsK, kSmemK, s, a);
}

}  // namespace rssm
