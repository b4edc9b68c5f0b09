// Chunked gated delta rule prefill on the 5th-generation tensor cores (GDN, bf16
// inputs, headdim = dstate = 128): one CTA per (sequence, head), chunks of 64 tokens.
//
// With G_t the running log decay inside the chunk, S [dv, dk] the state before it
// (rows t, s of K, Q, V, W are tokens):
//   A_ts = b_t e^{G_t - G_s} k_t.k_s (s < t)       T = (I + A)^-1
//   W = T R,  R_t = b_t (v_t - e^{G_t} S k_t)
//   O_t = scale (e^{G_t} S q_t + sum_{s<=t} e^{G_t - G_s} (q_t.k_s) w_s)
//   S' = e^{G_last} S + sum_s (e^{G_last - G_s} w_s) k_s^T
// Everything that depends on the state is computed transposed, one value row per
// tensor-memory lane (M = 128), with the fp32 operand in three bf16 parts in tensor
// memory and the other operand in shared memory:
//   U^T, Z^T = S [K; Q]^T   three products (K, Q exact in bf16)
//   W^T = R^T T^T           six (both sides split; the parts below 2^-24 left out)
//   O^T = W^T M^T           six
//   S' += (fw W)^T K        three
// so states and outputs keep fp32 accuracy.  [K; Q] K^T gives A and M; T comes
// from a kernel of its own before (gdn_pre_kernel), which has no chain to wait for.
// Far decays are differences of double prefix sums kept as two floats.
//
// Bound by the chain S -> U -> R -> W -> S' of one chunk after the other, 4.6 us or 8800 cycles
// a chunk (the tensor cores busy for 47% of them, the issue slots for 46%) on one SM per head,
// so one sequence of 32 heads has 32 of the SMs: 8192 tokens take 690 us (0.34 GB of inputs,
// outputs and states), of them 72 in gdn_pre_kernel; a ragged batch of 11 sequences and 20011
// tokens 840 us.
//
// Roles: warps 0-7 the chain (one value row per lane, two halves of the columns),
// warps 8-11 and 12-15 M and the outputs of every second chunk, warp 16 issues
// the products, warps 18-19 load the tiles with zeros behind the sequence's end; warp 17
// only fills its warpgroup.
#include "delta_t.cuh"
#include "rssm_prefill.h"

namespace rssm {
namespace {

using namespace chunk;

constexpr int kT = 64;                      // tokens per chunk
constexpr int kD = 128;
constexpr int kBlk = 16384;                 // 128 rows x 64 bf16
constexpr int kThreadsG = 640;
// registers per thread: 256 x 128 + 256 x 80 + 128 x 64 = 640 x 96
constexpr int kRegsLaunch = 96, kRegsChain = 128, kRegsOut = 80, kRegsRest = 64;
static_assert(256 * kRegsChain + 256 * kRegsOut + 128 * kRegsRest <= kThreadsG * kRegsLaunch, "registers of the CTA");
// shared memory
constexpr int kOffKQ = 0;                   // two stages: rows 0-63 K, 64-127 Q, two column blocks
constexpr int kOffV = 4 * kBlk;             // two stages [t][dv]
constexpr int kOffT = kOffV + 2 * kBlk;     // two buffers of three parts, [t][s]
constexpr int kOffM = kOffT + 6 * kPart;
constexpr int kOffSc = kOffM + 6 * kPart;
struct Scalars {        // of a chunk, made with its T
  float2 g[kT];        // G as two floats, in powers of two
  float be[kT];        // b_t
  float bg[kT];        // b_t e^{G_t}
  float zg[kT];        // scale e^{G_t}
  float fw[kT];        // e^{G_last - G_t}
  float last, pad[3];  // e^{G_last}
};
constexpr int kRecord = 3 * kPart + 2048;   // a chunk and head in the workspace: T's parts, the scalars
static_assert(sizeof(Scalars) % 16 == 0 && sizeof(Scalars) <= 2048, "record");
// four places for scalars: those of chunk i are read by its outputs, and chunk i + 4 comes
// after the update of chunk i + 2, which the same warps' outputs precede
constexpr int kOffBar = kOffSc + 4 * (int)sizeof(Scalars);
enum { kFull0 = 0, kFull1, kStage0, kStage1, kA0, kA1, kM0, kM1, kO0, kO1,
       kSp0, kSp1, kU, kRp, kW, kWp, kFwp, kUpd, kOfree, kAfree, kDrain, kBars };
constexpr int kSmemG = kOffBar + kBars * 8 + 32;
static_assert(kSmemG <= 232448, "shared memory of one CTA");
// tensor memory columns.  U^T, then W^T, then the masked product; Z^T; the parts of S, then
// of fw W and of W; the state's update, before it the parts of R; [K; Q] K^T.  Products in
// flight together (the outputs' and the update) share no column that either writes: two of
// unequal shape are ordered by a completed commit only.
constexpr int kTmU = 0, kTmZ = 64, kTmS = 128, kTmFw = 128, kTmW = 224, kTmD = 320, kTmR = 320, kTmA = 448;
static_assert(kTmFw + 96 <= kTmW && kTmW + 96 <= kTmD, "parts of W and of fw W outside the update's columns");

// T = (I + A)^-1 of every chunk and head of the long sequences, in the three parts and the
// place of each that the chain's kernel reads: everything that does not wait for a state.
// One CTA of four warps at a time per (chunk, head), four of them per SM.  K K^T on
// mma.sync (64 x 64 outputs of exact products; the 5th-generation cores take 128 rows at
// least, half of them wasted here); T in fp32 from A (invert_store).
constexpr int kPreThreads = 128;
constexpr int kPreOffA = 2 * kPart;                      // K: two blocks of 64 columns; A^T, [s][t]
constexpr int kPreOffTa = kPreOffA + kT * kALd * 4;      // T's first 32 rows and columns, [row][column]
constexpr int kPreOffTb = kPreOffTa + 32 * kTLd * 4;     // its last 32, [column][row]
constexpr int kPreOffX = kPreOffTb + 32 * kTLd * 4;      // blocks on the way
constexpr int kPreOffG = kPreOffX + 4 * 16 * kXLd * 4;   // G as two floats, b
constexpr int kSmemPre = kPreOffG + kT * 12 + 16;

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The running sum of the log gates (base 2) of a chunk, two tokens per lane, and its total.
__device__ __forceinline__ double gate_sums(const float (&al)[2], int lane, double (&G)[2]) {
  // a gate of 0 forgets all: any power of two this far down does
  G[0] = fmax(log2((double)al[0]), -16384.0);
  G[1] = G[0] + fmax(log2((double)al[1]), -16384.0);
  double inc = G[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  const double before = inc - G[1];
  G[0] += before;
  G[1] += before;
  return __shfl_sync(0xffffffffu, inc, 31);
}

__global__ void __launch_bounds__(kPreThreads, 4) gdn_pre_kernel(const PrefillArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const uint32_t base = smem_u32(smem);
  float *sA = reinterpret_cast<float *>(smem + kPreOffA), *sTa = reinterpret_cast<float *>(smem + kPreOffTa);
  float *sTb = reinterpret_cast<float *>(smem + kPreOffTb), *sX = reinterpret_cast<float *>(smem + kPreOffX);
  float2 *sG = reinterpret_cast<float2 *>(smem + kPreOffG);
  float *sBe = reinterpret_cast<float *>(smem + kPreOffG + kT * 8);
  grid_wait();
  grid_launch_next();
  const int total = a.queue[kChunkTotal], longs = a.queue[kLongCount];
  if (longs == 0) return;
  for (int i = t; i < (kPreOffG - kPreOffTa) / 4; i += kPreThreads) sTa[i] = 0.f;   // zero above the diagonal
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
    __syncthreads();   // the last item's blocks are read
    {
      const __nv_bfloat16 *pk = static_cast<const __nv_bfloat16 *>(a.in[1]) + (size_t)h * kD;
      const int c = t & 15;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int s = k * 8 + (t >> 4);
        const bool take = s < left;
        cp_async16_zfill(base + (c >> 3) * kPart + sw128(s, c & 7),
                         pk + (int64_t)(q.tok + t0 + (take ? s : 0)) * a.stride[1] + c * 8, take);
      }
      cp_commit();
    }
    if (w == 0) {
      const float *pa = static_cast<const float *>(a.in[3]) + h, *pb = static_cast<const float *>(a.in[4]) + h;
      float al[2], be[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int s = lane * 2 + k;
        al[k] = s < left ? pa[(int64_t)(q.tok + t0 + s) * a.stride[3]] : 1.f;
        be[k] = s < left ? pb[(int64_t)(q.tok + t0 + s) * a.stride[4]] : 0.f;
      }
      double G[2];
      const double last = gate_sums(al, lane, G);
      Scalars &sc = *reinterpret_cast<Scalars *>(a.parts + id * kRecord + 3 * kPart);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int s = lane * 2 + k;
        const float hi = (float)G[k], e = ex2((float)G[k]);
        sc.g[s] = sG[s] = make_float2(hi, (float)(G[k] - (double)hi));
        sc.be[s] = sBe[s] = be[k];
        sc.bg[s] = be[k] * e;
        sc.zg[s] = a.out_scale * e;
        sc.fw[s] = ex2((float)(last - G[k]));
      }
      if (lane == 0) sc.last = ex2((float)last);
    }
    cp_wait<0>();
    __syncthreads();
    {   // rows 16 w .. of K K^T up to the diagonal, then A
      float acc[4][2][4];
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[p][n][j] = 0.f;
      const int ra = w * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, ca = lane >> 4;
      const int rb = (lane & 7) + ((lane >> 4) & 1) * 8, cb = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t fa[4];
        ldmatrix4(fa, base + (k >> 2) * kPart + sw128(ra, (k & 3) * 2 + ca));
#pragma unroll
        for (int p = 0; p < 4; ++p)
          if (p <= w) {
            uint32_t fb[4];
            ldmatrix4(fb, base + (k >> 2) * kPart + sw128(p * 16 + rb, (k & 3) * 2 + cb));
            mma_16816(acc[p][0], fa, fb[0], fb[1]);
            mma_16816(acc[p][1], fa, fb[2], fb[3]);
          }
      }
      const int row = w * 16 + (lane >> 2);
      const float2 g0 = sG[row], g1 = sG[row + 8];
      const float b0 = sBe[row], b1 = sBe[row + 8];
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (p <= w)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int s = p * 16 + n * 8 + (lane & 3) * 2 + j;
              const float2 o = sG[s];
              sA[s * kALd + row] = s < row ? b0 * (ex2((g0.x - o.x) + (g0.y - o.y)) * acc[p][n][j]) : 0.f;
              sA[s * kALd + row + 8] = s < row + 8 ? b1 * (ex2((g1.x - o.x) + (g1.y - o.y)) * acc[p][n][2 + j]) : 0.f;
            }
    }
    __syncthreads();
    invert_store(sA, sTa, sTb, sX, a.parts + id * kRecord, t);
  }
}

__global__ void __launch_bounds__(kThreadsG, 1) gdn_chunk_kernel(const PrefillArgs a) {
  grid_wait();
  grid_launch_next();
  if (a.queue[kLongCount] == 0) return;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kOffBar);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffBar + kBars * 8);
  uint32_t *tm_slot = reinterpret_cast<uint32_t *>(smem + kOffBar + kBars * 8 + 8);
  Scalars *scs = reinterpret_cast<Scalars *>(smem + kOffSc);
  const uint32_t base = smem_u32(smem);
  constexpr int count[kBars] = {64, 64, 1, 1, 1, 1, 4, 4, 1, 1, 8, 8, 1, 8, 1, 8, 8, 1, 4, 2, 1};
  if (t == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bar + i, count[i]);
    abort[0] = abort[1] = 0;   // the second is never set
    mbar_fence_init();
  }
  if (warp == 16) {
    umma::alloc(tm_slot, 512);
    umma::relinquish();
  }
  for (int i = t; i < (kOffSc - kOffM) / 16; i += kThreadsG)   // M stays zero above the diagonal
    reinterpret_cast<uint4 *>(smem + kOffM)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tm = *tm_slot;
  const long long lim = a.wait_limit;
  PrefillSeq q;
  int h, *s_item = reinterpret_cast<int *>(smem + kOffBar + kBars * 8 + 12);
  auto next = [&]() { return next_item<kThreadsG, kBars>(a, bar, count, s_item, abort, q, h); };

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
    auto put_state = [&](int c) { split_store(lanes + kTmS + wg * 32 + c / 2, 64, S + c); };
    auto state_ready = [&](int half) {
      wait_st();
      umma::fence_before_sync();
      warp_arrive(bar + kSp0 + half);
    };
    bool good = true;
    float dec = 0.f;
    if (a.stall_test && blockIdx.x == 0) stall_on_unset_flag(const_cast<int *>(abort) + 1, abort, lim);
    for (int i = 0;; ++i) {
      const uint32_t ph = i & 1, sp = (i >> 1) & 1;
      const bool more = i < chunks;
#pragma unroll
      for (int c = 0; c < 64; c += 16) {   // the state before chunk i, and its parts
        if (i > 0) {
          float d[16];
          umma::ld_32x32b_x16(lanes + kTmD + wg * 64 + c, d);
#pragma unroll
          for (int j = 0; j < 16; ++j) S[c + j] = fmaf(dec, S[c + j], d[j]);
        }
        if (more) {
          put_state(c);
          if (c & 16) state_ready(c >> 5);
        }
      }
      umma::fence_before_sync();
      if (!more) break;
      const Scalars &sc = scs[i & 3];
      good = warp_wait(bar + kFull0 + (i & 1), sp, abort, lim);
      if (!good) break;
      float v[32];   // b v of this half's 32 tokens
      {
        const __nv_bfloat16 *pv =
            reinterpret_cast<const __nv_bfloat16 *>(smem + kOffV + (i & 1) * kBlk) + wg * 32 * kD + row;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 b = *reinterpret_cast<const float4 *>(&sc.be[wg * 32 + j]);
          v[j] = b.x * __bfloat162float(pv[j * kD]);
          v[j + 1] = b.y * __bfloat162float(pv[(j + 1) * kD]);
          v[j + 2] = b.z * __bfloat162float(pv[(j + 2) * kD]);
          v[j + 3] = b.w * __bfloat162float(pv[(j + 3) * kD]);
        }
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
          const float4 b = *reinterpret_cast<const float4 *>(&sc.bg[wg * 32 + c + j]);
          v[c + j] = fmaf(-b.x, u[j], v[c + j]);
          v[c + j + 1] = fmaf(-b.y, u[j + 1], v[c + j + 1]);
          v[c + j + 2] = fmaf(-b.z, u[j + 2], v[c + j + 2]);
          v[c + j + 3] = fmaf(-b.w, u[j + 3], v[c + j + 3]);
        }
        split_store(lanes + kTmR + wg * 16 + c / 2, 32, v + c);
      }
      wait_st();
      umma::fence_before_sync();
      warp_arrive(bar + kRp);
      good = warp_wait(bar + kW, ph, abort, lim);
      if (!good) break;
      umma::fence_after_sync();
      {   // W: first its parts, for the outputs; then those of fw W, for the state; both where the
          // parts of S were, which the products before W's have read
        umma::ld_32x32b_x32(lanes + kTmU + wg * 32, v);
#pragma unroll
        for (int c = 0; c < 32; c += 16) split_store(lanes + kTmW + wg * 16 + c / 2, 32, v + c);
        wait_st();
        umma::fence_before_sync();
        warp_arrive(bar + kWp);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(&sc.fw[wg * 32 + j]);
          v[j] *= f.x; v[j + 1] *= f.y; v[j + 2] *= f.z; v[j + 3] *= f.w;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 16) split_store(lanes + kTmFw + wg * 16 + c / 2, 32, v + c);
      }
      wait_st();
      umma::fence_before_sync();
      warp_arrive(bar + kFwp);
      dec = sc.last;
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
    // ------------------------------------- M and the outputs of every second chunk
    fewer_registers<kRegsOut>();
    const int me4 = (warp - 8) >> 2, w = warp & 3, r = w * 32 + lane;
    const uint32_t lanes = tm + ((uint32_t)(w * 32) << 16);
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    for (int i = me4; i < chunks; i += 2) {
      const int buf = me4;
      const Scalars &sc = scs[i & 3];
      if (!warp_wait(bar + kFull0 + buf, (i >> 1) & 1, abort, lim)) break;
      if (w >= 2) {   // a row of M per lane
        if (!warp_wait(bar + kA0 + buf, (i >> 1) & 1, abort, lim) ||
            (i > 1 && !warp_wait(bar + kStage0 + buf, ((i >> 1) - 1) & 1, abort, lim)))   // the last M is read
          break;
        umma::fence_after_sync();
        const int tt = r - 64;
        const float2 me = sc.g[tt];
#pragma unroll 1
        for (int cb = 0; cb < (w == 2 ? 2 : 4); ++cb) {     // up to the diagonal
          float v[16];
          umma::ld_32x32b_x16(lanes + kTmA + cb * 16, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 o = sc.g[cb * 16 + j];
            v[j] = cb * 16 + j <= tt ? a.out_scale * (ex2((me.x - o.x) + (me.y - o.y)) * v[j]) : 0.f;
          }
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            uint4 o[3];
            uint32_t *u = reinterpret_cast<uint32_t *>(o);
#pragma unroll
            for (int k = 0; k < 4; ++k) split3(v[j + 2 * k], v[j + 2 * k + 1], u[k], u[4 + k], u[8 + k]);
#pragma unroll
            for (int p = 0; p < 3; ++p)
              *reinterpret_cast<uint4 *>(smem + kOffM + (buf * 3 + p) * kPart + sw128(tt, cb * 2 + j / 8)) = o[p];
          }
        }
        umma::fence_before_sync();
        fence_proxy_async();
        warp_arrive(bar + kAfree);
      }
      warp_arrive(bar + kM0 + buf);   // of all four warps: none may miss a phase of kFull
      // the chunk's outputs, a value row per lane
      if (!warp_wait(bar + kO0 + buf, (i >> 1) & 1, abort, lim)) break;
      umma::fence_after_sync();
      const int left = q.n - i * kT;
      const size_t step = (size_t)a.H * kD;
      float *o = a.out + ((size_t)(q.tok + i * kT) * a.H + h) * kD + r;
#pragma unroll 1
      for (int c = 0; c < kT; c += 16) {
        float u[16], z[16];
        umma::ld_32x32b_x16(lanes + kTmU + c, u);
        umma::ld_32x32b_x16(lanes + kTmZ + c, z);
        if (c + 16 == kT) {
          umma::fence_before_sync();
          warp_arrive(bar + kOfree);
        }
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 g = *reinterpret_cast<const float4 *>(&sc.zg[c + j]);
          u[j] = fmaf(g.x, z[j], u[j]);
          u[j + 1] = fmaf(g.y, z[j + 1], u[j + 1]);
          u[j + 2] = fmaf(g.z, z[j + 2], u[j + 2]);
          u[j + 3] = fmaf(g.w, z[j + 3], u[j + 3]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j, o += step)
          if (c + j < left) __stcs(o, u[j]);
      }
    }
    }
  } else if (warp == 16) {
    // -------------------------------------------------------- the products
    fewer_registers<kRegsRest>();
    auto kmaj = [](uint32_t tile, int k) { return desc_sw128(tile + (k / 4) * kBlk + (k % 4) * 32, 16); };
    auto gram = [&](int i) {   // [K; Q] K^T
      const uint32_t kq = base + kOffKQ + (i & 1) * 2 * kBlk;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma::mma_bf16(tm + kTmA, kmaj(kq, k), kmaj(kq, k), idesc(128, kT, false, false), k > 0);
        umma::commit(bar + kA0 + (i & 1));
      }
      __syncwarp();
    };
    // S (rows of tile)^T over half of the columns: 32 from either half of the chain
    auto state_product = [&](uint32_t d, uint32_t tile, int half) {
      if (elect_one()) {
        const uint64_t b = desc_sw128(tile, 16);
#pragma unroll 1
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int kk = (k & 1) + 4 * (k >> 1) + 2 * half;
            mma_ts(tm + d, tm + kTmS + p * 64 + kk * 8, b + ((kk / 4) * kBlk + (kk % 4) * 32) / 16,
                   idesc(128, kT, false, false), half > 0 || p < 2 || k > 0);
          }
      }
      __syncwarp();
    };
    auto done = [&](uint64_t *b) {
      if (elect_one()) umma::commit(b);
      __syncwarp();
    };
    auto pair_product = [&](uint32_t parts, uint32_t tile, uint64_t *b) {   // into U's place
      if (elect_one()) {
        const uint64_t d = desc_sw128(tile, 16);
#pragma unroll 1
        for (int c = 0; c < 6; ++c) {
          const uint32_t at = tm + parts + part_a(c) * 32;
          const uint64_t b = d + part_b(c) * (kPart / 16);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ts(tm + kTmU, at + k * 8, b + k * 2, idesc(128, kT, false, false), c + k > 0);
        }
        umma::commit(b);
      }
      __syncwarp();
    };
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    bool good = warp_wait(bar + kFull0, 0, abort, lim);
    umma::fence_after_sync();
    if (good) gram(0);
    for (int i = 0; good && i < chunks; ++i) {
      const uint32_t ph = i & 1;
      const uint32_t kq = base + kOffKQ + (i & 1) * 2 * kBlk;
      if (!warp_wait(bar + kSp0, ph, abort, lim)) break;
      if (i > 0 && !warp_wait(bar + kOfree, ph ^ 1, abort, lim)) break;
      umma::fence_after_sync();
      state_product(kTmU, kq, 0);
      if (!warp_wait(bar + kSp1, ph, abort, lim)) break;
      umma::fence_after_sync();
      state_product(kTmU, kq, 1);
      done(bar + kU);
      state_product(kTmZ, kq + kPart, 0);   // while the chain makes R
      state_product(kTmZ, kq + kPart, 1);
      if (!warp_wait(bar + kRp, ph, abort, lim)) break;
      umma::fence_after_sync();
      pair_product(kTmR, base + kOffT + (i & 1) * 3 * kPart, bar + kW);
      if (i + 1 < chunks) {   // while the chain splits W
        if (!warp_wait(bar + kAfree, ph, abort, lim)) break;
        if (!warp_wait(bar + kFull0 + ((i + 1) & 1), ((i + 1) >> 1) & 1, abort, lim)) break;
        umma::fence_after_sync();
        gram(i + 1);
      }
      if (!warp_wait(bar + kWp, ph, abort, lim) || !warp_wait(bar + kM0 + (i & 1), (i >> 1) & 1, abort, lim)) break;
      umma::fence_after_sync();
      pair_product(kTmW, base + kOffM + (i & 1) * 3 * kPart, bar + kO0 + (i & 1));
      if (!warp_wait(bar + kFwp, ph, abort, lim)) break;
      umma::fence_after_sync();
      if (elect_one()) {
        const uint64_t b = desc_sw128(kq, kBlk);
#pragma unroll 1
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tm + kTmD, tm + kTmFw + p * 32 + k * 8, b + k * 128, idesc(128, kD, false, true), p < 2 || k > 0);
        umma::commit(bar + kUpd);
        umma::commit(bar + kStage0 + (i & 1));
      }
      __syncwarp();
    }
    // the arrivals that nobody else waits for, before the barriers start anew
    for (int i = chunks > 1 ? chunks - 2 : 0; good && i < chunks; ++i)
      warp_wait(bar + kStage0 + (i & 1), (i >> 1) & 1, abort, lim);
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
    const __nv_bfloat16 *in[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) in[k] = static_cast<const __nv_bfloat16 *>(a.in[k]) + (size_t)h * kD;
    int issued = 0;
    for (int i = 0; i < chunks; ++i) {
      const int st = i & 1;
      if (i > 1 && !warp_wait(bar + kStage0 + st, ((i >> 1) - 1) & 1, abort, lim)) break;
      const uint32_t kq = base + kOffKQ + st * 2 * kBlk, v = base + kOffV + st * kBlk;
      if (l == 0) {
        const uint8_t *rec = a.parts + ((size_t)(q.first + i) * a.H + h) * kRecord;
        mbar_expect_tx(bar + kFull0 + st, 3 * kPart + (uint32_t)sizeof(Scalars));
        bulk_g2s(smem + kOffT + st * 3 * kPart, rec, 3 * kPart, bar + kFull0 + st);
        bulk_g2s(scs + (i & 3), rec + 3 * kPart, sizeof(Scalars), bar + kFull0 + st);
      }
      // a thread keeps its 16-byte column and takes every fourth row; the swizzle of the rows
      // changes between two patterns
      const int s0 = l >> 4, c = l & 15, left = q.n - i * kT - s0;
      const int64_t first = q.tok + i * kT + s0;
      const __nv_bfloat16 *at[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) at[k] = in[k] + first * a.stride[k] + c * 8;
      const uint32_t to = kq + (c >> 3) * kBlk, even = to + sw128(s0, c & 7), odd = to + sw128(s0 + 4, c & 7);
#pragma unroll
      for (int k = 0; k < kT / 4; ++k) {
        const bool take = left > k * 4;
        const uint32_t row = (k & 1 ? odd : even) + (k >> 1) * 1024;
        cp_async16_zfill(row, take ? at[1] : in[1], take);
        cp_async16_zfill(row + 64 * 128, take ? at[0] : in[0], take);
        cp_async16_zfill(v + (s0 + k * 4) * 256 + c * 16, take ? at[2] : in[2], take);
#pragma unroll
        for (int j = 0; j < 3; ++j) at[j] += 4 * a.stride[j];
      }
      cp_commit();
      cp_wait<0>();
      fence_proxy_async();
      mbar_arrive(bar + kFull0 + st);
      issued = i + 1;
    }
    cp_async_wait_all();
    // the bulk copies have landed before this CTA goes on, or ends, whatever came
    for (int i = issued > 1 ? issued - 2 : 0; i < issued; ++i)
      mbar_wait_bounded(bar + kFull0 + (i & 1), (i >> 1) & 1, nullptr, lim);
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

bool gdn_chunk_path(const PrefillArgs &a, int in_dtype) {
  return a.kind == RSSM_GDN && in_dtype == RSSM_BF16 && a.R == kD && a.C == kD;
}

size_t gdn_chunk_work(size_t chunks, int H) { return chunks * H * kRecord; }

cudaError_t gdn_chunk_prefill(const PrefillArgs &a, cudaStream_t s) {
  cudaError_t e = allow_smem(gdn_pre_kernel, kSmemPre);
  if (e == cudaSuccess) e = allow_smem(gdn_chunk_kernel, kSmemG);
  if (e != cudaSuccess) return e;
  const size_t chunks = most_chunks(a.n_seq, a.n_tokens, a.scan_most) * a.H, items = (size_t)a.n_seq * a.H;
  e = launch_early(gdn_pre_kernel, (unsigned)(chunks < 4 * kPrefillSms ? chunks : 4 * kPrefillSms), kPreThreads, kSmemPre,
                   s, a);
  if (e != cudaSuccess) return e;
  return launch_early(gdn_chunk_kernel, (unsigned)(items < kPrefillSms ? items : kPrefillSms), kThreadsG, kSmemG, s, a);
}

}  // namespace rssm
