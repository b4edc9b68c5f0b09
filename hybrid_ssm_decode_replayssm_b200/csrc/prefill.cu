// Prefill: a ragged batch of prompts run through a layer's recurrence, from the
// rows' checkpoints (or zero) to their new checkpoints, with every output.
//
//   plan_prefill_kernel   decides each sequence from the pointers (one CTA)
//   m2_chunk_kernel, or   long sequences of bf16 tokens in chunks on the tensor cores
//   gdn_/kda_pre_kernel   (m2_prefill.cu, gdn_prefill.cu, kda_prefill.cu)
//   and .._chunk_kernel
//   scan_kernel           the others, and fp32 inputs: four tokens at a time, the state in
//                         registers, beside the chunked kernel
//   requantize_kernel     the read copies of the rows written
//
// The planner waits for all work before it, the read copies for all of the call; the kernels
// between are launched programmatically, each resident before the one ahead of it ends.  Of a
// short call's 18 us (Mamba-2, 7 turns) the GPU works 12, the host needs 17 to send it.
#include "rssm_prefill.h"
#include "chunk.cuh"
#include "slots.cuh"

namespace rssm {
namespace {

// ------------------------------------------------------------------ planner
// One CTA.  A sequence is refused (STATE) when the offsets are not a
// non-decreasing list inside [0, n_tokens] (then all are), its row is out of
// range or named by another sequence too, or it continues a row whose window is
// not empty.  An accepted sequence counts as one fold of its row; on branching
// layers it gets a free slot, adopted by the next launch like any fold's.
// Accepted sequences are listed longest first, so that the longest start first.
constexpr int kPlanThreads = 1024;

// The token scan takes sequences of more tokens than this by 32 rows per item, the others by 64,
// as long as each of those items has an SM of its own: a shorter chain per token (fp32 inputs, 32
// heads, one sequence of 1024 tokens beside 11 of 64: GDN 247 us against 309, KDA 319 against
// 338), but half as many rows per reading of the tokens.  Where they are too many for that, all go
// by 64 (4 sequences of 1024: GDN 452 us against 694 by 32, KDA 510 against 861, Mamba-2 on 128
// heads 681 against 921); at 512 tokens beside short ones both cost the same (KDA 196, 198).
constexpr int kFineTokens = 512;
constexpr int kBins = 66;
__device__ __forceinline__ int length_bin(int n, int scan_most) { return (n > scan_most ? 33 : 0) + 32 - __clz(n); }

__global__ void __launch_bounds__(kPlanThreads) plan_prefill_kernel(const PrefillArgs a) {
  const int nt = blockDim.x, t = threadIdx.x;
  chunk::grid_launch_next();   // the kernels behind wait for this grid themselves
  if (a.slot) adopt_folds(a.B, a.slot, a.dst, a.seen, a.flushes);
  for (int b = t; b < a.B; b += nt) a.named[b] = 0;
  static_assert(kCounters + kSmCounters <= 256, "the smallest planner");
  if (t < kCounters + kSmCounters) a.queue[t] = 0;
  bool bad = false;
  for (int i = t; i < a.n_seq; i += nt) {
    const int o0 = a.offsets[i], o1 = a.offsets[i + 1];
    bad |= o0 < 0 || o1 < o0 || o1 > a.n_tokens;
  }
  bad = __syncthreads_or(bad);
  for (int i = t; i < a.n_seq; i += nt) {
    const int r = a.rows ? a.rows[i] : i;
    if (r >= 0 && r < a.B) atomicAdd(a.named + r, 1);
  }
  int nfree = 0;
  if (a.slot) nfree = free_slots(a.B, a.slot, a.freelist);
  // Up to 1024 sequences are sorted by comparing all pairs; more of them by powers of two of
  // their lengths, those of the chunked kernels first (the order decides when a sequence
  // runs, nothing in it).
  const bool many = a.n_seq > kPlanThreads;
  __shared__ int bins[kBins];
  if (many) {
    if (t < kBins) bins[t] = 0;
    __syncthreads();
    for (int i = t; i < a.n_seq; i += nt) {
      const int n = bad ? 0 : a.offsets[i + 1] - a.offsets[i];
      atomicAdd(bins + length_bin(n, a.scan_most), 1);
    }
    __syncthreads();
    if (t == 0)
      for (int b = kBins - 1, sum = 0; b >= 0; --b) {
        const int c = bins[b];
        bins[b] = sum;
        sum += c;
      }
  }
  __syncthreads();
  int rank = 0;
  for (int i0 = 0; i0 < a.n_seq; i0 += nt) {
    const int i = i0 + t;
    int take = 0, r = 0, o0 = 0, n = 0, src = -1;
    if (i < a.n_seq) {
      r = a.rows ? a.rows[i] : i;
      const bool fresh = a.fresh && a.fresh[i] != 0;
      bool refuse = bad || r < 0 || r >= a.B || a.named[r] != 1;
      if (!refuse && !fresh) refuse = a.len[r] != 0 || a.pending[r] != 0;
      if (refuse) atomicOr(a.status, (unsigned)RSSM_STATUS_STATE);
      o0 = refuse ? 0 : a.offsets[i];
      n = refuse ? 0 : a.offsets[i + 1] - o0;
      take = !refuse && (n > 0 || fresh);
      if (take) {
        src = fresh ? -1 : a.slot ? a.slot[r] : r;
        a.len[r] = 0;
        a.pending[r] = 0;
        a.flushes[r] += 1;
      }
    }
    int excl = 0, tot = 0;
    if (a.slot) block_scan(take, excl, tot);
    if (i < a.n_seq) {
      int to = -1;
      if (take) {
        to = r;
        if (a.slot) a.dst[r] = to = rank + excl < nfree ? a.freelist[rank + excl] : a.slot[r];   // nfree >= B
      }
      int place;
      if (many) {
        place = atomicAdd(bins + length_bin(bad ? 0 : a.offsets[i + 1] - a.offsets[i], a.scan_most), 1);
      } else if (bad) {
        place = i;
      } else {   // how many sequences are longer, or as long and before it
        const int full = a.offsets[i + 1] - a.offsets[i];
        place = 0;
        for (int j = 0; j < a.n_seq; ++j) {
          const int m = a.offsets[j + 1] - a.offsets[j];
          place += m > full || (m == full && j < i);
        }
      }
      PrefillSeq q = {};
      q.tok = o0;
      q.n = n;
      q.src = src;
      q.dst = to;
      a.seqs[place] = q;
      if (n > a.scan_most) atomicMax(a.queue + kLongCount, place + 1);
      else if (n > kFineTokens) atomicMax(a.queue + kFineCount, place + 1);
    }
    rank += tot;
  }
  if (a.parts) {   // the long sequences' chunks, in the order of the list
    __syncthreads();
    int total = 0;
    for (int i0 = 0; i0 < a.n_seq; i0 += nt) {
      const int i = i0 + t;
      const int n = i < a.n_seq ? a.seqs[i].n : 0;
      int excl, tot;
      block_scan(n > a.scan_most ? (n + 63) / 64 : 0, excl, tot);
      if (i < a.n_seq) a.seqs[i].first = total + excl;
      total += tot;
    }
    if (t == 0) a.queue[kChunkTotal] = total;
  }
  if (a.chunks) {   // for the scan; the armed self-test keeps it waiting
    __syncthreads();
    if (t == 0 && !a.stall_test) chunk::word_release(a.queue + kPlanned, kPlanWritten);
  }
}

// -------------------------------------------------------- four tokens at a time
// One CTA of 256 threads per (sequence, head, 32 or 64 state rows): four warps run the
// recurrence, the state in registers (16 columns of one to four rows per thread, as
// packed pairs); four warps bring the tokens, eight at a time, as fp32 into two buffers of
// shared memory, with what depends on the tokens alone, and take the outputs away.
// Four tokens i = 0..3 go together: with p_i the product of their gates up to i and
// d_ij that of the gates j+1..i (products, never ratios),
//   u_i = S k_i,  z_i = S q_i                              (S before the four)
//   w_i = b_i v_i - b_i p_i u_i - sum_{j<i} b_i d_ij (k_i.k_j) w_j
//   o_i = scale (p_i z_i + sum_{j<=i} d_ij (q_i.k_j) w_j)
//   S  <- p_3 S + sum_j d_3j w_j k_j^T
// so the sums of a row cross the lanes in two rounds instead of eight, and an element
// costs 3.25 multiply-adds per token instead of 4.  Mamba-2: k, q, v = B, C, x,
// no u, w = dt x.  KDA: one gate per channel, so p and d go into the vectors (p_i k_i,
// p_i q_i, d_3j k_j).  Bound by the CUDA cores' issue and the latency of those rounds: 0.18 us per
// token of a Mamba-2 or GDN sequence, 0.22 of a KDA one, while its items have SMs of their own.
constexpr int kScanThreads = 256;
constexpr int kScanTok = 8;    // tokens per buffer: two blocks of four
// registers per thread: 128 x 184 + 128 x 72 = 256 x 128, so that two CTAs fit
constexpr int kScanRegs = 184, kBringRegs = 72;

typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float x, float y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
  return x + y;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Eight consecutive elements (16-byte aligned), as they come and as fp32.
template <typename T> struct Raw8 {
  uint4 x[sizeof(T) / 2];
};
template <typename T> __device__ __forceinline__ void ld8(Raw8<T> &o, const T *p) {
#pragma unroll
  for (int c = 0; c < (int)sizeof(T) / 2; ++c) o.x[c] = __ldg(reinterpret_cast<const uint4 *>(p) + c);
}
template <typename T> __device__ __forceinline__ void widen(float (&o)[8], const Raw8<T> &r) {
  const T *e = reinterpret_cast<const T *>(r.x);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = to_f32<T>(e[j]);
}
__device__ __forceinline__ void named_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// What the tokens of a block give: b (Mamba-2: dt), b p, scale p, d_3j, p_3, and by rows the
// two triangles b_i d_ij (k_i.k_j) and scale d_ij (q_i.k_j).
struct __align__(16) ScanBlock {
  float be[4], bg[4], p[4], f[4];
  float A[4][4], M[4][4];
  float pc, pad[3];
};

template <int N> struct Const {
  static constexpr int value = N;
};

template <int KIND, typename Tin, int C>
__global__ void __launch_bounds__(kScanThreads, 2) scan_kernel(const PrefillArgs a, int fine_all) {
  constexpr bool M2 = KIND == RSSM_MAMBA2, KDA = KIND == RSSM_KDA;
  constexpr int LPR = C / 16;                       // lanes per row
  constexpr int GROUPS = 128 / LPR;                 // rows per pass: 16 or 32
  struct Buf {
    float k[kScanTok][C], q[kScanTok][C];           // KDA: p_i k_i, p_i q_i
    float kt[KDA ? kScanTok : 1][C], pc[KDA ? 2 : 1][C];   // KDA: d_3j k_j, p_3
    float v[kScanTok][64], o[kScanTok][64];
    ScanBlock blk[2];
  };
  __shared__ __align__(16) Buf buf[2];
  __shared__ __align__(16) float raw_k[KDA ? kScanTok : 1][C], raw_g[KDA ? kScanTok : 1][C];
  __shared__ __align__(16) float s_gate[kScanTok], s_beta[kScanTok];
  __shared__ int s_item;
  // Alone, this grid waits for the planner's.  Beside a chunked kernel, whose CTAs have all
  // waited for the planner before this grid began, its own wait would be for the chunked
  // kernel's end, so that comes last; what the planner wrote is taken behind a word that it
  // releases.  The last CTA to end takes the word back, for the next call in this workspace.
  if (!a.chunks) {
    chunk::grid_wait();
  } else {
    if (threadIdx.x == 0) s_item = chunk::word_acquire(a.queue + kPlanned, kPlanWritten, a.wait_limit);
    __syncthreads();
    if (!s_item) {
      if (threadIdx.x == 0) atomicOr(a.status, (unsigned)RSSM_STATUS_TIMEOUT);
      return chunk::grid_wait();
    }
    __syncthreads();
  }
  // the items: the long sequences of this kernel (or all) by 32 rows, then the others by 64
  const int from = a.queue[kLongCount], to_long = max(from, a.queue[kFineCount]);
  const int per32 = a.H * (a.R / 32), per64 = a.H * (a.R / 64);
  const int to_fine = fine_all ? a.n_seq : to_long - from <= kPrefillSms / per32 ? to_long : from;
  const int fine_items = (to_fine - from) * per32, items = fine_items + (a.n_seq - to_fine) * per64;
  const int t = threadIdx.x, lane = t & 31;
  const size_t tile = (size_t)a.R * C;
  // barriers: 1, 2 a buffer is full; 3, 4 it is empty; 5 the bringing warps among themselves;
  // 6, 7 the begin and the end of an item
  if (t < 128) {
    // -------------------------------------------------- the recurrence
    chunk::more_registers<kScanRegs>();
    // items in turn: an SM's first CTA takes the longest one left, its second the shortest,
    // so that long sequences do not share an SM (which CTA runs an item changes nothing in it)
    uint32_t sm;
    asm volatile("mov.u32 %0, %smid;" : "=r"(sm));
    const bool front = t != 0 || sm >= kSmCounters || atomicAdd(a.queue + kCounters + sm, 1) == 0;
    for (;;) {
      if (t == 0) {
        const bool any = atomicAdd(a.queue + kScanTaken, 1) < items;
        s_item = !any ? items
                      : front ? atomicAdd(a.queue + kScanFront, 1)
                              : items - 1 - atomicAdd(a.queue + kScanBack, 1);
      }
      named_sync(6, kScanThreads);
      const int item = s_item;
      if (item >= items) break;
      const bool fine = item < fine_items;
      const int id = fine ? item : item - fine_items, each = fine ? per32 : per64;
      const int h = id % a.H, sl = id % each / a.H;
      const PrefillSeq q = a.seqs[(fine ? from : to_fine) + id / each];
      if (q.dst < 0 || q.n > a.scan_most) {
        named_sync(7, kScanThreads);
        continue;
      }
      const int tiles = (q.n + kScanTok - 1) / kScanTok;
      auto recur = [&](auto rows) {
      constexpr int ROWS = decltype(rows)::value;
      constexpr int RPT = ROWS / GROUPS;                // rows per thread
      constexpr int NV = RPT * 4;                       // a thread's sums for four tokens
      constexpr int PL = NV / LPR, LR = 4 / PL;         // the sums it keeps; lanes that hold a row's four
      static_assert(PL == 1 || PL == 2, "sums per lane");
      const int sub = t % LPR, grp = t / LPR, lane0 = lane - sub;
      const int mine = grp + sub / LR * GROUPS, i0 = sub % LR * PL;   // the row and tokens whose sums this lane keeps
      f32x2 S[RPT][8];
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const int row = sl * ROWS + grp + r * GROUPS;
        const float *src = a.hc + ((size_t)(q.src < 0 ? 0 : q.src) * a.H + h) * tile + (size_t)row * C;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 v = q.src < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : ld_stream(src + c * (C / 4) + sub * 4);
          S[r][2 * c] = pack2(v.x, v.y);
          S[r][2 * c + 1] = pack2(v.z, v.w);
        }
      }
      const float Dh = M2 ? __ldg(a.D + h) : 0.f;
      for (int n = 0; n < tiles; ++n) {
        Buf &B = buf[n & 1];
        const int blocks = q.n - n * kScanTok > 4 ? 2 : 1;
        named_sync(1 + (n & 1), kScanThreads);
#pragma unroll 1
        for (int b = 0; b < blocks; ++b) {
          const ScanBlock &K = B.blk[b];
          const float4 be = *reinterpret_cast<const float4 *>(K.be);
          float w[4] = {be.x * B.v[b * 4][mine], be.y * B.v[b * 4 + 1][mine], be.z * B.v[b * 4 + 2][mine],
                        be.w * B.v[b * 4 + 3][mine]};
          [[maybe_unused]] float u[M2 ? 1 : NV];
          float z[NV];   // S k_i and S q_i
          {
            [[maybe_unused]] f32x2 au[M2 ? 1 : NV];
            f32x2 az[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              az[j] = 0;
              if constexpr (!M2) au[j] = 0;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if constexpr (!M2) {
                  const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&B.k[b * 4 + i][c * (C / 4) + sub * 4]);
#pragma unroll
                  for (int r = 0; r < RPT; ++r)
                    au[r * 4 + i] = fma2(S[r][2 * c + 1], x.y, fma2(S[r][2 * c], x.x, au[r * 4 + i]));
                }
                const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(&B.q[b * 4 + i][c * (C / 4) + sub * 4]);
#pragma unroll
                for (int r = 0; r < RPT; ++r)
                  az[r * 4 + i] = fma2(S[r][2 * c + 1], y.y, fma2(S[r][2 * c], y.x, az[r * 4 + i]));
              }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
              z[j] = sum2(az[j]);
              if constexpr (!M2) u[j] = sum2(au[j]);
            }
          }
          if constexpr (!M2) tr_sum<NV, LPR / 2>(u, lane);
          tr_sum<NV, LPR / 2>(z, lane);
          if constexpr (!M2) {
            float u4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u4[i] = __shfl_sync(kFull, u[i % PL], lane - sub % LR + i / PL);
            const float4 bg = *reinterpret_cast<const float4 *>(K.bg);
            const float4 a1 = *reinterpret_cast<const float4 *>(K.A[1]), a2 = *reinterpret_cast<const float4 *>(K.A[2]);
            const float4 a3 = *reinterpret_cast<const float4 *>(K.A[3]);
            w[0] = fmaf(-bg.x, u4[0], w[0]);
            w[1] = fmaf(-a1.x, w[0], fmaf(-bg.y, u4[1], w[1]));
            w[2] = fmaf(-a2.y, w[1], fmaf(-a2.x, w[0], fmaf(-bg.z, u4[2], w[2])));
            w[3] = fmaf(-a3.z, w[2], fmaf(-a3.y, w[1], fmaf(-a3.x, w[0], fmaf(-bg.w, u4[3], w[3]))));
          }
          const float4 f4 = *reinterpret_cast<const float4 *>(K.f);
          const float fs[4] = {f4.x, f4.y, f4.z, f4.w};
          f32x2 fw[RPT][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float own = KDA ? w[j] : fs[j] * w[j];
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
              const float x = __shfl_sync(kFull, own, lane0 + LR * r);
              fw[r][j] = pack2(x, x);
            }
          }
#pragma unroll
          for (int s = 0; s < PL; ++s) {   // the outputs of this lane's row and tokens
            const int i = i0 + s;
            const float4 m = *reinterpret_cast<const float4 *>(K.M[i]);
            const float o = fmaf(m.x, w[0], fmaf(m.y, w[1], fmaf(m.z, w[2], fmaf(m.w, w[3], K.p[i] * z[s]))));
            B.o[b * 4 + i][mine] = M2 ? fmaf(Dh, B.v[b * 4 + i][mine], o) : o;
          }
          asm volatile("" ::: "memory");   // k is read again: there are no registers to keep it
          const f32x2 pc = pack2(K.pc, K.pc);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            ulonglong2 g = make_ulonglong2(pc, pc);
            if constexpr (KDA) g = *reinterpret_cast<const ulonglong2 *>(&B.pc[b][c * (C / 4) + sub * 4]);
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
              S[r][2 * c] = mul2(S[r][2 * c], g.x);
              S[r][2 * c + 1] = mul2(S[r][2 * c + 1], g.y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float *kv = KDA ? &B.kt[b * 4 + j][c * (C / 4) + sub * 4] : &B.k[b * 4 + j][c * (C / 4) + sub * 4];
              const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(kv);
#pragma unroll
              for (int r = 0; r < RPT; ++r) {
                S[r][2 * c] = fma2(fw[r][j], x.x, S[r][2 * c]);
                S[r][2 * c + 1] = fma2(fw[r][j], x.y, S[r][2 * c + 1]);
              }
            }
          }
        }
        named_arrive(3 + (n & 1), kScanThreads);
      }
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const int row = sl * ROWS + grp + r * GROUPS;
        float *dst = a.hc + ((size_t)q.dst * a.H + h) * tile + (size_t)row * C;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<ulonglong2 *>(dst + c * (C / 4) + sub * 4) = make_ulonglong2(S[r][2 * c], S[r][2 * c + 1]);
      }
      };
      if (fine) recur(Const<32>());
      else recur(Const<64>());
      named_sync(7, kScanThreads);   // the buffers and barriers start anew
    }
  } else {
    // -------------------------------------------------- tokens in, outputs out
    chunk::fewer_registers<kBringRegs>();
    for (;;) {
      named_sync(6, kScanThreads);
      const int item = s_item;
      if (item >= items) break;
      const bool fine = item < fine_items;
      const int id = fine ? item : item - fine_items, each = fine ? per32 : per64;
      const int h = id % a.H, sl = id % each / a.H;
      const PrefillSeq q = a.seqs[(fine ? from : to_fine) + id / each];
      if (q.dst < 0 || q.n > a.scan_most) {
        named_sync(7, kScanThreads);
        continue;
      }
      const int tiles = (q.n + kScanTok - 1) / kScanTok;
      const int l = t - 128, rows = fine ? 32 : 64;
      const int hk = M2 ? h / a.hpg : h;                 // head (or group) of k and q
      const Tin *pk = static_cast<const Tin *>(a.in[1]) + (size_t)hk * C;
      const Tin *pq = static_cast<const Tin *>(a.in[M2 ? 2 : 0]) + (size_t)hk * C;
      const Tin *pv = static_cast<const Tin *>(a.in[M2 ? 0 : 2]) + (size_t)h * a.R + sl * rows;
      const int64_t dk = a.stride[1], dq = a.stride[M2 ? 2 : 0], dv = a.stride[M2 ? 0 : 2];
      const float Ah = M2 ? __ldg(a.A + h) : 0.f;
      const float scale = M2 ? 1.f : a.out_scale;
      constexpr int per = C / 8;                         // threads per token: 16 or 8
      const int e = l / per, c8 = l % per * 8;           // this thread's token and columns
      const int bi = e & 3, bb = e & ~3;                 // its place in its block, and the block's first
      const int ve = fine ? l >> 3 : l >> 4, vc = (fine ? l & 7 : l & 15) * 4;   // and its four values of v
      float k8[8], q8[8], g8[8];
      // the next tile's values as they come: widened only when they are used, so that
      // nothing waits for them before
      Raw8<Tin> rk, rq;
      Raw8<float> rg;
      uint4 rv = make_uint4(0, 0, 0, 0);
      Tin rdt = Tin(0.f);
      float ra = 1.f, rb = 0.f;
      auto load = [&](int n) {   // zeros behind the end: k = q = v = b = 0, gate 1
        const int64_t tok = (int64_t)q.tok + n * kScanTok;
        const int m = q.n - n * kScanTok;
        if (m < kScanTok) {
          const uint4 zero = make_uint4(0, 0, 0, 0), one = make_uint4(0x3F800000u, 0x3F800000u, 0x3F800000u, 0x3F800000u);
#pragma unroll
          for (int c = 0; c < (int)sizeof(Tin) / 2; ++c) rk.x[c] = rq.x[c] = zero;
          rg.x[0] = rg.x[1] = one;
          rv = zero;
          rdt = Tin(0.f);
          ra = 1.f;
          rb = 0.f;
        }
        if (e < m && e < kScanTok) {
          ld8<Tin>(rk, pk + (tok + e) * dk + c8);
          ld8<Tin>(rq, pq + (tok + e) * dq + c8);
          if constexpr (KDA)
            ld8<float>(rg, static_cast<const float *>(a.in[3]) + (tok + e) * a.stride[3] + (size_t)h * C + c8);
          if (c8 == 0) {
            if constexpr (M2) {
              rdt = __ldg(static_cast<const Tin *>(a.in[3]) + (tok + e) * a.stride[3] + h);
            } else {
              if constexpr (!KDA) ra = __ldg(static_cast<const float *>(a.in[3]) + (tok + e) * a.stride[3] + h);
              rb = __ldg(static_cast<const float *>(a.in[4]) + (tok + e) * a.stride[4] + h);
            }
          }
        }
        if (ve < m && ve < kScanTok) {
          const Tin *p = pv + (tok + ve) * dv + vc;
          if constexpr (sizeof(Tin) == 4) {
            rv = __ldg(reinterpret_cast<const uint4 *>(p));
          } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
            rv.x = x.x;
            rv.y = x.y;
          }
        }
      };
      auto put8 = [&](float *p, const float *x) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
      };
      auto flush = [&](int n) {   // the outputs of tile n
        const int64_t tok = (int64_t)q.tok + n * kScanTok;
        if (ve < kScanTok && ve < q.n - n * kScanTok)
          st_stream(a.out + ((tok + ve) * a.H + h) * a.R + sl * rows + vc,
                    *reinterpret_cast<const float4 *>(&buf[n & 1].o[ve][vc]));
      };
      if (tiles > 0) load(0);
      for (int n = 0; n < tiles; ++n) {
        Buf &B = buf[n & 1];
        if (n > 1) {
          named_sync(3 + (n & 1), kScanThreads);
          flush(n - 2);
        }
        if (n > 0) named_sync(5, 128);   // the last tile's gates and keys are read
        if (e < kScanTok) {
          widen<Tin>(k8, rk);
          widen<Tin>(q8, rq);
          if constexpr (KDA) {
            widen<float>(g8, rg);
            put8(&raw_k[e][c8], k8);
            put8(&raw_g[e][c8], g8);
          } else {
            put8(&B.k[e][c8], k8);
            put8(&B.q[e][c8], q8);
          }
          if (c8 == 0) {
            if constexpr (M2) {
              const float dt = to_f32<Tin>(rdt);
              s_gate[e] = expf(dt * Ah);
              s_beta[e] = dt;
            } else {
              s_gate[e] = ra;
              s_beta[e] = rb;
            }
          }
        }
        {
          float4 x;
          if constexpr (sizeof(Tin) == 4)
            x = *reinterpret_cast<const float4 *>(&rv);
          else
            x = make_float4(__uint_as_float(rv.x << 16), __uint_as_float(rv.x & 0xFFFF0000u), __uint_as_float(rv.y << 16),
                            __uint_as_float(rv.y & 0xFFFF0000u));
          if (ve < kScanTok) *reinterpret_cast<float4 *>(&B.v[ve][vc]) = x;
        }
        if (n + 1 < tiles) load(n + 1);
        named_sync(5, 128);
        if (e < kScanTok) {
          float pair[8];   // k_i.k_j and q_i.k_j, j = 0..3, over this thread's columns
          float D[8];      // KDA: d_ij of this thread's channels
#pragma unroll
          for (int j = 0; j < 8; ++j) pair[j] = 0.f, D[j] = 1.f;
#pragma unroll
          for (int j = 3; j >= 0; --j)
            if (j <= bi) {
              float x[8];
              const float *kj = KDA ? &raw_k[bb + j][c8] : &B.k[bb + j][c8];
              *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(kj);
              *reinterpret_cast<float4 *>(x + 4) = *reinterpret_cast<const float4 *>(kj + 4);
              if constexpr (KDA) {
#pragma unroll
                for (int c = 0; c < 8; ++c) x[c] *= D[c];
                if (bi == 3) put8(&B.kt[bb + j][c8], x);
              }
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                pair[j] = fmaf(k8[c], x[c], pair[j]);
                pair[4 + j] = fmaf(q8[c], x[c], pair[4 + j]);
              }
              if constexpr (KDA) {
#pragma unroll
                for (int c = 0; c < 8; ++c) D[c] *= raw_g[bb + j][c8 + c];
              }
            }
          if constexpr (KDA) {   // D is p_i now
            if (bi == 3) put8(&B.pc[bb >> 2][c8], D);
#pragma unroll
            for (int c = 0; c < 8; ++c) k8[c] *= D[c], q8[c] *= D[c];
            put8(&B.k[e][c8], k8);
            put8(&B.q[e][c8], q8);
          }
          tr_sum<8, per / 2>(pair, lane);
          const int val = tr_base<8, per / 2>(lane), j = val & 3;
          ScanBlock &K = B.blk[bb >> 2];
          float d = 1.f, p = 1.f, f = 1.f;   // d_ij, p_i and d_3i of scalar gates
          if constexpr (!KDA) {
            const float4 g4 = *reinterpret_cast<const float4 *>(&s_gate[bb]);
            const float g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (r <= bi) p *= g[r];
              if (r > j && r <= bi) d *= g[r];
              if (r > bi) f *= g[r];
            }
          }
          const float be = s_beta[e];
          if (val < 4) K.A[bi][j] = j < bi ? be * d * pair[0] : 0.f;
          else K.M[bi][j] = j <= bi ? scale * d * pair[0] : 0.f;
          if (c8 == 0) {
            K.be[bi] = be;
            K.bg[bi] = be * p;
            K.p[bi] = scale * p;
            if (bi == 3) K.pc = p;
            K.f[bi] = f;
          }
        }
        named_arrive(1 + (n & 1), kScanThreads);
      }
      for (int n = max(0, tiles - 2); n < tiles; ++n) {
        named_sync(3 + (n & 1), kScanThreads);
        flush(n);
      }
      named_sync(7, kScanThreads);
    }
  }
  if (a.chunks) {
    chunk::grid_wait();
    if (threadIdx.x == 0 && atomicAdd(a.queue + kScanEnded, 1) == (int)gridDim.x - 1) a.queue[kPlanned] = 0;
  }
}

// ------------------------------------------------------------- read copies
// The read copy of every row written, as rssm_quantize_read_copy makes it.
template <int C, int RF>
__global__ void __launch_bounds__(256) requantize_kernel(const PrefillArgs a) {
  constexpr int LPR = C / 4, RPI = 32 / LPR;
  constexpr int RB = RF == RSSM_READ_NVFP4 ? C / 2 : C;
  const int lane = threadIdx.x & 31, c0 = (lane % LPR) * 4;
  const PrefillSeq q = a.seqs[blockIdx.x / a.H];
  if (q.dst < 0) return;
  const size_t base = ((size_t)q.dst * a.H + blockIdx.x % a.H) * a.R;
  for (int r = (threadIdx.x >> 5) * RPI + lane / LPR; r < a.R; r += 8 * RPI) {
    const size_t row = base + r;
    const float4 v = *reinterpret_cast<const float4 *>(a.hc + row * C + c0);
    quantize4<RF, LPR>(v, a.rc_codes + row * RB, a.rc_scales, row, C, c0, lane);
  }
}

template <int KIND, typename Tin>
cudaError_t launch_scan(const PrefillArgs &a, cudaStream_t s) {
  // 32 rows per item for all while every item then has an SM of its own (GDN, 32 heads, fp32: 40
  // tokens 20.5 us against 24, 1000 tokens 201 against 256; Mamba-2, 64 heads: 200 tokens 45
  // against 51), else for a few sequences of more than kFineTokens; 64 for the others
  const bool fine = (long long)a.n_seq * a.H * a.R <= (long long)kPrefillSms * 32;
  const size_t items = (size_t)a.n_seq * a.H * (a.R / (fine || a.scan_most > kFineTokens ? 32 : 64));
  const unsigned grid = (unsigned)(items < 2 * kPrefillSms ? items : 2 * kPrefillSms);
  if constexpr (KIND == RSSM_MAMBA2)
    if (a.C == 64)
      return launch_early(scan_kernel<KIND, Tin, 64>, grid, kScanThreads, 0, s, a, (int)fine);
  return launch_early(scan_kernel<KIND, Tin, 128>, grid, kScanThreads, 0, s, a, (int)fine);
}

// Sequences of up to this many tokens run four tokens at a time even where a chunked kernel
// serves the layer, whose first chunk costs as much as a full one (32 sequences on 32 GDN
// heads: at 32 tokens 117 us against 147, at 64 tokens 217 against 163; Mamba-2 on 128
// heads 180 against 240 and 309 against 246).  A GDN call of few tokens in all does without
// the chunked kernels' two launches (192 tokens in one sequence: 38 us either way; KDA 51
// against 60).  KDA's chunks cost more (32 sequences on 32 heads: at 96 tokens 333 us
// against 364, at 128 tokens 436 against 371).
constexpr int kScanMost = 40, kScanMostKda = 96, kDeltaFew = 192;

int scan_most(int kind) { return kind == RSSM_KDA ? kScanMostKda : kScanMost; }
bool chunked(int kind, int n_tokens) { return n_tokens > (kind == RSSM_MAMBA2 ? kScanMost : kDeltaFew); }

size_t seq_bytes(int n_seq) { return ((size_t)n_seq * sizeof(PrefillSeq) + 255) & ~(size_t)255; }

size_t fixed_bytes(int n_seq, int batch) {
  return (seq_bytes(n_seq) + (kCounters + kSmCounters + (size_t)batch) * sizeof(int32_t) + 255) & ~(size_t)255;
}

}  // namespace

size_t prefill_work_bytes(const rssm_layer_desc &d, int n_seq, int n_tokens) {
  size_t parts = 0;
  if (d.kind != RSSM_MAMBA2 && d.in_dtype == RSSM_BF16 && chunked(d.kind, n_tokens)) {
    const size_t chunks = most_chunks(n_seq, n_tokens, scan_most(d.kind));
    parts = d.kind == RSSM_GDN ? gdn_chunk_work(chunks, d.nheads) : kda_chunk_work(chunks, d.nheads);
  }
  return fixed_bytes(n_seq, d.batch) + parts;
}

cudaError_t prefill(PrefillArgs a, void *work, int in_dtype, int read_fmt, int *launches, cudaStream_t s) {
  a.seqs = static_cast<PrefillSeq *>(work);
  a.queue = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(work) + seq_bytes(a.n_seq));
  a.named = a.queue + kCounters + kSmCounters;
  *launches = 0;
  const bool m2_chunks = m2_chunk_path(a, in_dtype), delta_chunks = gdn_chunk_path(a, in_dtype) || kda_chunk_path(a, in_dtype);
  const bool chunks = (m2_chunks || delta_chunks) && chunked(a.kind, a.n_tokens);
  a.chunks = chunks;
  a.scan_most = chunks ? scan_most(a.kind) : a.n_tokens;
  a.parts = chunks && delta_chunks ? static_cast<uint8_t *>(work) + fixed_bytes(a.n_seq, a.B) : nullptr;
  plan_prefill_kernel<<<1, a.n_seq > 256 || a.B > 2048 ? kPlanThreads : 256, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  ++*launches;
  if (e != cudaSuccess) return e;
  if (chunks) {
    e = m2_chunks ? m2_chunk_prefill(a, s) : a.kind == RSSM_GDN ? gdn_chunk_prefill(a, s) : kda_chunk_prefill(a, s);
    *launches += m2_chunks ? 1 : 2;
    if (e != cudaSuccess) return e;
  }
  const bool bf16 = in_dtype == RSSM_BF16;
  switch (a.kind) {
    case RSSM_MAMBA2:
      e = bf16 ? launch_scan<RSSM_MAMBA2, __nv_bfloat16>(a, s) : launch_scan<RSSM_MAMBA2, float>(a, s);
      break;
    case RSSM_GDN:
      e = bf16 ? launch_scan<RSSM_GDN, __nv_bfloat16>(a, s) : launch_scan<RSSM_GDN, float>(a, s);
      break;
    default:
      e = bf16 ? launch_scan<RSSM_KDA, __nv_bfloat16>(a, s) : launch_scan<RSSM_KDA, float>(a, s);
  }
  ++*launches;
  if (e != cudaSuccess || read_fmt == RSSM_READ_FP32) return e;
  const dim3 grid((unsigned)((size_t)a.n_seq * a.H));
  if (a.C == 64)
    read_fmt == RSSM_READ_NVFP4 ? requantize_kernel<64, RSSM_READ_NVFP4><<<grid, 256, 0, s>>>(a)
                                : requantize_kernel<64, RSSM_READ_FP8_E4M3_ROW><<<grid, 256, 0, s>>>(a);
  else
    read_fmt == RSSM_READ_NVFP4 ? requantize_kernel<128, RSSM_READ_NVFP4><<<grid, 256, 0, s>>>(a)
                                : requantize_kernel<128, RSSM_READ_FP8_E4M3_ROW><<<grid, 256, 0, s>>>(a);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace rssm
