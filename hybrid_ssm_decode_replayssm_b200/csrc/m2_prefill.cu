// Chunked Mamba-2 prefill on the 5th-generation tensor cores (bf16 inputs,
// headdim 64): one CTA per (sequence, head), chunks of 128 tokens.
//
// With a_s = dt_s A, G_t = a_1 + .. + a_t inside the chunk and h the state before
// it ([P, N]; rows t, s are tokens, every sum over one operand's columns):
//   y  = e^{G_t} (C h^T) + L x + D x,   L_ts = e^{G_t - G_s} dt_s (C B^T)_ts, s <= t
//   h' = e^{G_last} h + (e^{G_last - G_s} dt_s x_s)^T B
// as four products per chunk, each with M = 128:
//   CB    = C B^T            [t, s]  both operands bf16 inputs: exact products
//   inter = C h^T            [t, p]  h in three bf16 parts
//   upd   = B^T (fw x)       [n, p]  fw x in three parts: the state's update, transposed
//   intra = L x              [t, p]  L in three parts; adds to e^{G_t} inter
// A three-part split carries fp32 to 2^-24, so outputs and states keep fp32 accuracy.
// C and L are operands in tensor memory: reading all of them from shared memory costs
// more than the tensor core's own time.  The state lives in registers, one column n per
// thread; it is never scaled in tensor memory.  G is a double prefix sum kept as two
// floats, so differences of far decays lose nothing.
//
// Every barrier completes once per chunk (the stage barriers once per two), and no
// barrier can complete again before all its waiters have passed: full -> stage freed
// by y, CB -> L, inter -> y, upd -> the next fw x, decays -> both users.
//
// Roles: warps 0-7 (one token per lane, two halves of the columns) make L from CB and
// write y; warps 8-15 (one n per lane, two halves of p) make fw x, update the state and
// split it; warp 16 issues the products; warp 17 computes the decays; warps 18-21 load the
// tiles with zeros behind the sequence's end, so that nothing past it is ever read.
//
// Bound by the hand-overs from role to role in a chunk's 8200 cycles: shared memory is busy for
// 65% of them (the kernel's loads and stores 3160, the products' operand reads 2180), the issue
// slots for 45%, the tensor cores for 35% (counters, 3000 tokens).  8192 tokens on 128 heads
// (N = 128) take 280 us, 440 MB of inputs, outputs and states at 1.6 TB/s; L on 16 warps of
// eight columns 299, L and C in shared memory and y stored a token per lane slower still.
#include "chunk.cuh"
#include "rssm_prefill.h"

namespace rssm {
namespace {

using namespace chunk;

constexpr int kT = 128;                // tokens per chunk
constexpr int kP = 64;
constexpr int kBlk = 16384;            // 128 rows x 64 bf16
constexpr int kWarpsM = 22;
constexpr int kThreadsM = kWarpsM * 32;
// shared memory
constexpr int kOffB = 0;               // two stages of B, two 64-column blocks each
constexpr int kOffC = 4 * kBlk;
constexpr int kOffX = 6 * kBlk;        // two stages
constexpr int kOffH = 8 * kBlk;        // three parts of the state, [n][p]
constexpr int kOffXp = 11 * kBlk;      // three parts of fw x, [s][p]
constexpr int kOffSc = 14 * kBlk;      // float4 (G hi, G lo, dt, fw) per token
constexpr int kOffOd = kOffSc + kT * 16;   // e^{G_32w - G_s} dt_s for the rows of block w = 1, 2, 3
constexpr int kOffBar = kOffOd + 192 * 4;
enum { kFull0 = 0, kFull1, kCt, kCb, kInter, kYs, kUpd, kIntra, kL0, kL1, kHp, kXp, kXfree, kYfree, kScFull, kScFree, kStage0, kStage1,
       kDrain, kBars };
constexpr int kYRow = 272;             // bytes per token of the outputs on their way out, in the place of fw x
constexpr int kSmemM = kOffBar + kBars * 8 + 32;
static_assert(kSmemM <= 232448, "shared memory of one CTA");
// tensor memory columns (kTmC: C as an operand)
constexpr int kTmCb = 0, kTmY = 128, kTmC = 192, kTmU = 256, kTmL = 320;

template <int N> struct Cols {
  static constexpr int value = N;
};

template <int N>
__global__ void __launch_bounds__(kThreadsM, 1) m2_chunk_kernel(const PrefillArgs a) {
  grid_wait();
  grid_launch_next();
  if (a.queue[kLongCount] == 0) return;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kOffBar);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffBar + kBars * 8);
  uint32_t *tm_slot = reinterpret_cast<uint32_t *>(smem + kOffBar + kBars * 8 + 8);
  float *s_last = reinterpret_cast<float *>(smem + kOffBar + kBars * 8 + 16);   // e^{G_last}
  float4 *sc = reinterpret_cast<float4 *>(smem + kOffSc);
  const uint32_t base = smem_u32(smem);
  constexpr int count[kBars] = {128, 128, 8, 1, 1, 8, 1, 1, 8, 8, 8, 8, 8, 8, 1, 16, 8, 8, 1};
  if (t == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bar + i, count[i]);
    abort[0] = abort[1] = 0;   // the second is never set
    mbar_fence_init();
  }
  if (warp == 16) {
    umma::alloc(tm_slot, 512);
    umma::relinquish();
  }
  if constexpr (N == 64) {   // the second column block of B and C stays zero
    for (int i = t; i < kBlk / 16; i += kThreadsM) {
      const uint4 z = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4 *>(smem + kOffB + kBlk)[i] = z;
      reinterpret_cast<uint4 *>(smem + kOffB + 3 * kBlk)[i] = z;
      reinterpret_cast<uint4 *>(smem + kOffC + kBlk)[i] = z;
    }
    fence_proxy_async();
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tm = *tm_slot;
  const long long lim = a.wait_limit;
  PrefillSeq q;
  int h, *s_item = reinterpret_cast<int *>(smem + kOffBar + kBars * 8 + 12);
  auto next = [&]() { return next_item<kThreadsM, kBars>(a, bar, count, s_item, abort, q, h); };

  if (warp < 8) {
    // ------------------------------------------------ L, and the outputs
    // two warps per 32 tokens: each takes sixteen of every 32 columns of L, and half of y
    const int wg = warp >> 2, w = warp & 3, row = w * 32 + lane;
    const uint32_t lanes = tm + ((uint32_t)(w * 32) << 16);
    {
      const uint32_t z[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      for (int cb = w + 1; cb < 4; ++cb)   // above the diagonal L stays zero
        for (int p = 0; p < 3; ++p) st_x8(lanes + kTmL + p * 64 + cb * 16 + wg * 8, z);
    }
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    const float Dh = __ldg(a.D + h);
    for (int i = 0; i < chunks; ++i) {
      const uint32_t ph = i & 1;
      if (!warp_wait(bar + kScFull, ph, abort, lim)) break;
      const float4 me = sc[row];
      // below the diagonal blocks e^{G_t - G_s} splits at the block's start, and one
      // factor per column is left; the diagonal block's are made while C B^T is
      const float4 ref = sc[w > 0 ? w * 32 - 1 : 0];
      const float at = ex2((me.x - ref.x) + (me.y - ref.y));
      const float *od = reinterpret_cast<const float *>(smem + kOffOd) + (w == 3 ? 96 : w == 2 ? 32 : 0);
      float e[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 s = sc[w * 32 + wg * 16 + j];
        e[j] = wg * 16 + j <= lane ? ex2((me.x - s.x) + (me.y - s.y)) * s.z : 0.f;
      }
      if (!warp_wait(bar + kCb, ph, abort, lim)) break;
      umma::fence_after_sync();
      bool ok = true;
      for (int cb = 0; cb < 4; ++cb) {
        if (cb <= w) {
          const int c0 = cb * 32 + wg * 16;
          float v[16];
          umma::ld_32x32b_x16(lanes + kTmCb + c0, v);
          if (cb < w) {
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(od + c0 + j);
              v[j] *= at * f.x; v[j + 1] *= at * f.y; v[j + 2] *= at * f.z; v[j + 3] *= at * f.w;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = wg * 16 + j <= lane ? e[j] * v[j] : 0.f;
          }
          split_store(lanes + kTmL + cb * 16 + wg * 8, 64, v);
        }
        if (cb & 1) {   // the product can start on half of the columns
          wait_st();
          umma::fence_before_sync();
          warp_arrive(bar + kL0 + (cb >> 1));
        }
        if (cb == 1) {   // e^{G_t} C h^T, in its place; the masked product adds to it
          ok = warp_wait(bar + kInter, ph, abort, lim);
          if (!ok) break;
          umma::fence_after_sync();
          const float g = ex2(me.x + me.y);
#pragma unroll
          for (int c = 0; c < 32; c += 16) {
            float v[16];
            uint32_t o[16];
            umma::ld_32x32b_x16(lanes + kTmY + wg * 32 + c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(g * v[j]);
            st_x16(lanes + kTmY + wg * 32 + c, o);
          }
          wait_st();
          umma::fence_before_sync();
          warp_arrive(bar + kYs);
        }
      }
      if (!ok) break;
      warp_arrive(bar + kScFree);
      if (!warp_wait(bar + kFull0 + (i & 1), (i >> 1) & 1, abort, lim) || !warp_wait(bar + kIntra, ph, abort, lim)) break;
      umma::fence_after_sync();
      const uint8_t *xrow = smem + kOffX + (i & 1) * kBlk;
      float y[32];
      umma::ld_32x32b_x32(lanes + kTmY + wg * 32, y);
      umma::fence_before_sync();
      warp_arrive(bar + kYfree);
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        const uint4 raw = *reinterpret_cast<const uint4 *>(xrow + sw128(row, wg * 4 + j / 8));
        const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[j + 2 * k] = fmaf(Dh, __uint_as_float(x[k] << 16), y[j + 2 * k]);
          y[j + 2 * k + 1] = fmaf(Dh, __uint_as_float(x[k] & 0xFFFF0000u), y[j + 2 * k + 1]);
        }
      }
      warp_arrive(bar + kStage0 + (i & 1));
      // y leaves through the place of fw x (read by now), four rows per store: a token per
      // lane would touch 32 lines per store and hold up all of shared memory
      uint8_t *stage = smem + kOffXp + w * 32 * kYRow + wg * 128;
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4 *>(stage + lane * kYRow + j * 4) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
      __syncwarp();
      const int first = i * kT + w * 32 + (lane >> 3);
      float *o = a.out + ((size_t)(q.tok + first) * a.H + h) * kP + wg * 32 + (lane & 7) * 4;
      const size_t step = (size_t)4 * a.H * kP;
      float4 z[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        z[k] = *reinterpret_cast<const float4 *>(stage + (k * 4 + (lane >> 3)) * kYRow + (lane & 7) * 16);
#pragma unroll
      for (int k = 0; k < 8; ++k, o += step)
        if (first + k * 4 < q.n) st_stream(o, z[k]);
      warp_arrive(bar + kXfree);
    }
    }
  } else if (warp < 16) {
    // ------------------------------------------------ the state
    const int u = t - 256, wg = (warp - 8) >> 2, n = (warp & 3) * 32 + lane, p0 = wg * 32;
    const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    const float *src = a.hc + ((size_t)(q.src < 0 ? 0 : q.src) * a.H + h) * kP * N;
    float *dst = a.hc + ((size_t)q.dst * a.H + h) * kP * N;
    float S[32];
#pragma unroll
    for (int p = 0; p < 32; ++p) S[p] = q.src < 0 || n >= N ? 0.f : __ldcs(src + (size_t)(p0 + p) * N + n);
    auto put = [&](int part_off, int row, const float *v8, int c16) {   // 8 values -> three parts
      uint4 w[3];
      uint32_t *x = reinterpret_cast<uint32_t *>(w);
#pragma unroll
      for (int k = 0; k < 4; ++k) split3(v8[2 * k], v8[2 * k + 1], x[k], x[4 + k], x[8 + k]);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4 *>(smem + part_off + p * kBlk + sw128(row, c16)) = w[p];
    };
    auto put_state = [&](int c) {
      put(kOffH, n, S + c, (p0 + c) / 8);
      put(kOffH, n, S + c + 8, (p0 + c) / 8 + 1);
    };
    auto state_ready = [&]() {
      fence_proxy_async();
      warp_arrive(bar + kHp);
    };
    bool good = true;
    if (a.stall_test && blockIdx.x == 0) stall_on_unset_flag(const_cast<int *>(abort) + 1, abort, lim);
    if (chunks > 0) {
      put_state(0);
      put_state(16);
      state_ready();
    }
    for (int i = 0; i < chunks; ++i) {
      const uint32_t ph = i & 1;
      good = warp_wait(bar + kFull0 + (i & 1), (i >> 1) & 1, abort, lim);
      if (!good) break;
      {   // C to tensor memory, where two products take it from without reading shared memory
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4 *>(smem + kOffC + wg * kBlk + sw128(n, c));
        st_x16(lanes + kTmC + wg * 32, *reinterpret_cast<const uint32_t (*)[16]>(&v[0]));
        st_x16(lanes + kTmC + wg * 32 + 16, *reinterpret_cast<const uint32_t (*)[16]>(&v[4]));
        wait_st();
        umma::fence_before_sync();
        warp_arrive(bar + kCt);
      }
      good = warp_wait(bar + kScFull, ph, abort, lim) && (i == 0 || warp_wait(bar + kXfree, ph ^ 1, abort, lim));
      if (!good) break;
      const float dec = *s_last;
      const uint8_t *x = smem + kOffX + (i & 1) * kBlk;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int s = k * 32 + u / 8, c16 = u % 8;
        const float fw = sc[s].w;
        const uint4 raw = *reinterpret_cast<const uint4 *>(x + sw128(s, c16));
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = fw * __uint_as_float(w[j] << 16);
          v[2 * j + 1] = fw * __uint_as_float(w[j] & 0xFFFF0000u);
        }
        put(kOffXp, s, v, c16);
      }
      fence_proxy_async();
      warp_arrive(bar + kXp);
      warp_arrive(bar + kScFree);
      good = warp_wait(bar + kUpd, ph, abort, lim);
      if (!good) break;
      umma::fence_after_sync();
      const bool more = i + 1 < chunks;
#pragma unroll
      for (int c = 0; c < 32; c += 16) {
        float v[16];
        umma::ld_32x32b_x16(lanes + kTmU + p0 + c, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) S[c + j] = fmaf(dec, S[c + j], v[j]);
        if (more) put_state(c);
      }
      umma::fence_before_sync();
      if (more) state_ready();
    }
    if (good && n < N)
#pragma unroll
      for (int p = 0; p < 32; ++p) dst[(size_t)(p0 + p) * N + n] = S[p];
    }
  } else if (warp == 16) {
    // ------------------------------------------------ the products
    constexpr int KN = N / 16;   // K steps along n
    // sums run from the small parts of a split to the large: the tensor core truncates
    // each addition, and only those of the last, large part then count
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    for (int i = 0; i < chunks; ++i) {
      const uint32_t ph = i & 1;
      const uint32_t Bt = base + kOffB + (i & 1) * 2 * kBlk, Xt = base + kOffX + (i & 1) * kBlk;
      auto kmaj = [](uint32_t tile, int k) { return desc_sw128(tile + (k / 4) * kBlk + (k % 4) * 32, 16); };
      auto mnmaj = [](uint32_t tile, int k) { return desc_sw128(tile + k * 2048, kBlk); };
      if (!warp_wait(bar + kFull0 + (i & 1), (i >> 1) & 1, abort, lim) || !warp_wait(bar + kCt, ph, abort, lim)) break;
      umma::fence_after_sync();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < KN; ++k)
          mma_ts(tm + kTmCb, tm + kTmC + k * 8, kmaj(Bt, k), idesc(128, 128, false, false), k > 0);
        umma::commit(bar + kCb);
      }
      __syncwarp();
      if (!warp_wait(bar + kHp, ph, abort, lim)) break;
      if (i > 0 && !warp_wait(bar + kYfree, ph ^ 1, abort, lim)) break;
      umma::fence_after_sync();
      if (elect_one()) {
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int k = 0; k < KN; ++k)
            mma_ts(tm + kTmY, tm + kTmC + k * 8, mnmaj(base + kOffH + p * kBlk, k), idesc(128, kP, false, true),
                   p < 2 || k > 0);
        umma::commit(bar + kInter);
      }
      __syncwarp();
      if (!warp_wait(bar + kXp, ph, abort, lim)) break;
      umma::fence_after_sync();
      if (elect_one()) {
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int k = 0; k < kT / 16; ++k)
            umma::mma_bf16(tm + kTmU, mnmaj(Bt, k), mnmaj(base + kOffXp + p * kBlk, k), idesc(128, kP, true, true),
                           p < 2 || k > 0);
        umma::commit(bar + kUpd);
      }
      __syncwarp();
      bool ok = true;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        ok = ok && warp_wait(bar + kL0 + half, ph, abort, lim) && (half > 0 || warp_wait(bar + kYs, ph, abort, lim));
        if (!ok) break;
        umma::fence_after_sync();
        if (elect_one()) {
#pragma unroll
          for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int k = half * 4; k < half * 4 + 4; ++k)
              mma_ts(tm + kTmY, tm + kTmL + p * 64 + k * 8, mnmaj(Xt, k), idesc(128, kP, false, true), true);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) umma::commit(bar + kIntra);
      __syncwarp();
    }
    }
  } else if (warp == 17) {
    // ------------------------------------------------ decays
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    const double Ah = (double)__ldg(a.A + h) * 1.4426950408889634;   // in powers of two
    // a step that forgets all: any power of two this far down does, and the sums behind it keep
    // their precision (unbounded, a dt of 1e12 cost the decays of its chunk 1%)
    const float most = (float)(16384.0 / fabs(Ah));
    const __nv_bfloat16 *pdt = static_cast<const __nv_bfloat16 *>(a.in[3]) + h;
    auto load = [&](int i, float (&v)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int s = i * kT + lane * 4 + k;
        v[k] = s < q.n ? __bfloat162float(pdt[(int64_t)(q.tok + s) * a.stride[3]]) : 0.f;
      }
    };
    float dt[4];
    if (chunks > 0) load(0, dt);
    for (int i = 0; i < chunks; ++i) {
      float next[4] = {0.f, 0.f, 0.f, 0.f};
      if (i + 1 < chunks) load(i + 1, next);
      double G[4], sum = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum += (double)fminf(dt[k], most) * Ah;
        G[k] = sum;
      }
      double inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      const double before = inc - sum, last = __shfl_sync(0xffffffffu, inc, 31);
      const double at[3] = {__shfl_sync(0xffffffffu, inc, 7), __shfl_sync(0xffffffffu, inc, 15),
                            __shfl_sync(0xffffffffu, inc, 23)};   // G at the ends of 32, 64, 96 tokens
      if (i > 0 && !warp_wait(bar + kScFree, (i - 1) & 1, abort, lim)) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const double g = G[k] + before;
        const float hi = (float)g;
        sc[lane * 4 + k] = make_float4(hi, (float)(g - (double)hi), dt[k], dt[k] * ex2((float)(last - g)));
        const int s = lane * 4 + k;
        float *od = reinterpret_cast<float *>(smem + kOffOd);
#pragma unroll
        for (int w = 1; w < 4; ++w)
          if (s < 32 * w) od[(w == 3 ? 96 : w == 2 ? 32 : 0) + s] = dt[k] * ex2((float)(at[w - 1] - g));
        dt[k] = next[k];
      }
      if (lane == 0) *s_last = ex2((float)last);
      warp_arrive(bar + kScFull);
    }
    }
  } else {
    // ------------------------------------------------ tiles
    const int l = t - 576;   // 0..127
    while (next()) {
    const int chunks = (q.n + kT - 1) / kT;
    const int g = h / a.hpg;
    const __nv_bfloat16 *px = static_cast<const __nv_bfloat16 *>(a.in[0]) + (size_t)h * kP;
    const __nv_bfloat16 *pB = static_cast<const __nv_bfloat16 *>(a.in[1]) + (size_t)g * N;
    const __nv_bfloat16 *pC = static_cast<const __nv_bfloat16 *>(a.in[2]) + (size_t)g * N;
    // a thread keeps its 16-byte column and takes every eighth (or sixteenth) row: the
    // swizzle of its rows is the same
    auto tile = [&](uint32_t to, const __nv_bfloat16 *p, int64_t stride, int i, auto cols) {
      constexpr int per = decltype(cols)::value / 8, rows = 128 / per;
      const int s0 = l / per, c = l % per, left = q.n - i * kT - s0;
      const __nv_bfloat16 *at = p + (int64_t)(q.tok + i * kT + s0) * stride + c * 8;
      uint32_t dst = to + (c / 8) * kBlk + sw128(s0, c % 8);
#pragma unroll
      for (int k = 0; k < kT / rows; ++k) {
        cp_async16_zfill(dst, left > k * rows ? at : p, left > k * rows);
        at += rows * stride;
        dst += rows * 128;
      }
    };
    for (int i = 0; i < chunks; ++i) {
      const int st = i & 1;
      if (i > 1 && !warp_wait(bar + kStage0 + st, ((i >> 1) - 1) & 1, abort, lim)) break;
      tile(base + kOffB + st * 2 * kBlk, pB, a.stride[1], i, Cols<N>());
      tile(base + kOffX + st * kBlk, px, a.stride[0], i, Cols<kP>());
      if (i > 0 && !warp_wait(bar + kCt, (i - 1) & 1, abort, lim)) break;
      tile(base + kOffC, pC, a.stride[2], i, Cols<N>());
      cp_commit();
      cp_wait<0>();
      fence_proxy_async();
      mbar_arrive(bar + kFull0 + st);
    }
    cp_async_wait_all();
    }
  }
  // ------------------------------------------------ end
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

bool m2_chunk_path(const PrefillArgs &a, int in_dtype) {
  return a.kind == RSSM_MAMBA2 && in_dtype == RSSM_BF16 && a.R == kP && (a.C == 64 || a.C == 128);
}

cudaError_t m2_chunk_prefill(const PrefillArgs &a, cudaStream_t s) {
  auto kernel = a.C == 64 ? m2_chunk_kernel<64> : m2_chunk_kernel<128>;
  const cudaError_t e = allow_smem(kernel, kSmemM);
  if (e != cudaSuccess) return e;
  const size_t items = (size_t)a.n_seq * a.H;
  return launch_early(kernel, (unsigned)(items < kPrefillSms ? items : kPrefillSms), kThreadsM, kSmemM, s, a);
}

}  // namespace rssm
