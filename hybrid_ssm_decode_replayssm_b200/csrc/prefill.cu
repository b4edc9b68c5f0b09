// Prefill: a ragged batch of prompts run through a layer's recurrence, from the
// rows' checkpoints (or zero) to their new checkpoints, with every output.
//
//   plan_prefill_kernel   decides each sequence from the pointers (one CTA)
//   scan_kernel           token by token, the state in registers
//   requantize_kernel     the read copies of the rows written
#include "rssm_prefill.h"
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

__global__ void __launch_bounds__(kPlanThreads) plan_prefill_kernel(const PrefillArgs a) {
  const int nt = blockDim.x, t = threadIdx.x;
  if (a.slot) adopt_folds(a.B, a.slot, a.dst, a.seen, a.flushes);
  for (int b = t; b < a.B; b += nt) a.named[b] = 0;
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
    int excl, tot;
    block_scan(take, excl, tot);
    if (i < a.n_seq) {
      int to = -1;
      if (take) {
        to = r;
        if (a.slot) a.dst[r] = to = rank + excl < nfree ? a.freelist[rank + excl] : a.slot[r];   // nfree >= B
      }
      // the place of i: how many sequences are longer, or as long and before it
      int place = 0;
      if (bad) {
        place = i;
      } else {
        const int full = a.offsets[i + 1] - a.offsets[i];
        for (int j = 0; j < a.n_seq; ++j) {
          const int m = a.offsets[j + 1] - a.offsets[j];
          place += m > full || (m == full && j < i);
        }
      }
      PrefillSeq q;
      q.tok = o0;
      q.n = n;
      q.src = src;
      q.dst = to;
      a.seqs[place] = q;
    }
    rank += tot;
  }
}

// ----------------------------------------------------------- token by token
// One CTA of 128 threads per (sequence, head, 32 state rows); a thread holds 16
// columns of two rows.  All three recurrences read the state before the token,
//   z = S (g q),  u = S (g k),  w = beta (v - u)   (Mamba-2: w = dt x, no u)
//   out = z + w (k.q),  S <- S g + w k^T
// with g the gate (a scalar, or one per channel for KDA) and k, q, w = B, C, dt x
// for Mamba-2, so both reductions over a row go together and one token costs one
// round of shuffles.  Bound by that chain of latencies, and with many sequences
// by the CUDA cores (4 operations per state element and token).
constexpr int kScanThreads = 128;
constexpr int kScanRows = 32;
constexpr int kScanTok = 16;   // tokens staged in shared memory at a time

template <typename T> __device__ __forceinline__ float ld_in(const void *p, int64_t i) {
  return to_f32<T>(__ldg(static_cast<const T *>(p) + i));
}

template <int KIND, typename Tin, int C>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const PrefillArgs a) {
  constexpr bool M2 = KIND == RSSM_MAMBA2, KDA = KIND == RSSM_KDA;
  constexpr int LPR = C / 16;                       // lanes per row
  constexpr int GROUPS = kScanThreads / LPR;        // row pairs per pass: 16 or 32
  constexpr int RPT = kScanRows / GROUPS;           // rows per thread: 2 or 1
  constexpr int kPer = 16 / sizeof(Tin);
  const int slices = a.R / kScanRows;
  const int h = (int)(blockIdx.x % a.H), sl = (int)(blockIdx.x / a.H % slices);
  const PrefillSeq q = a.seqs[blockIdx.x / a.H / slices];
  if (q.dst < 0) return;
  __shared__ __align__(16) float s_k[kScanTok][C], s_q[kScanTok][C];
  __shared__ __align__(16) float s_g[KDA ? kScanTok : 1][C];
  __shared__ float s_v[kScanTok][kScanRows], s_o[kScanTok][kScanRows];
  __shared__ float s_a[kScanTok], s_b[kScanTok], s_kq[kScanTok];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int sub = t % LPR, grp = t / LPR;
  const size_t tile = (size_t)a.R * C;
  float S[RPT][16];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = sl * kScanRows + grp + r * GROUPS;
    const float *src = a.hc + ((size_t)q.src * a.H + h) * tile + (size_t)row * C;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 v = q.src < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : ld_stream(src + c * (C / 4) + sub * 4);
      S[r][4 * c] = v.x; S[r][4 * c + 1] = v.y; S[r][4 * c + 2] = v.z; S[r][4 * c + 3] = v.w;
    }
  }
  const float Ah = M2 ? __ldg(a.A + h) : 0.f, Dh = M2 ? __ldg(a.D + h) : 0.f;
  const int hk = M2 ? h / a.hpg : h;                 // head (or group) of k and q
  const Tin *pk = static_cast<const Tin *>(a.in[1]) + (size_t)hk * C;
  const Tin *pq = static_cast<const Tin *>(a.in[M2 ? 2 : 0]) + (size_t)hk * C;
  const Tin *pv = static_cast<const Tin *>(a.in[M2 ? 0 : 2]) + (size_t)h * a.R + sl * kScanRows;
  const int64_t dk = a.stride[1], dq = a.stride[M2 ? 2 : 0], dv = a.stride[M2 ? 0 : 2];
  for (int t0 = 0; t0 < q.n; t0 += kScanTok) {
    const int m = min(kScanTok, q.n - t0);
    const int64_t tok = q.tok + t0;
    __syncthreads();
    for (int i = t; i < m * (C / kPer); i += kScanThreads) {
      const int e = i / (C / kPer), c = i % (C / kPer) * kPer;
      stage_row<Tin>(&s_k[e][c], pk + (tok + e) * dk + c, kPer, 0, 1);
      stage_row<Tin>(&s_q[e][c], pq + (tok + e) * dq + c, kPer, 0, 1);
    }
    for (int i = t; i < m * (kScanRows / kPer); i += kScanThreads) {
      const int e = i / (kScanRows / kPer), c = i % (kScanRows / kPer) * kPer;
      stage_row<Tin>(&s_v[e][c], pv + (tok + e) * dv + c, kPer, 0, 1);
    }
    if constexpr (KDA)
      for (int i = t; i < m * (C / 4); i += kScanThreads) {
        const int e = i / (C / 4), c = i % (C / 4) * 4;
        *reinterpret_cast<float4 *>(&s_g[e][c]) = __ldg(reinterpret_cast<const float4 *>(
            static_cast<const float *>(a.in[3]) + (tok + e) * a.stride[3] + (size_t)h * C + c));
      }
    if (t < m) {
      if constexpr (M2) {
        const float dt = ld_in<Tin>(a.in[3], (tok + t) * a.stride[3] + h);
        s_a[t] = expf(dt * Ah);
        s_b[t] = dt;
      } else {
        if constexpr (!KDA) s_a[t] = ld_in<float>(a.in[3], (tok + t) * a.stride[3] + h);
        s_b[t] = ld_in<float>(a.in[4], (tok + t) * a.stride[4] + h);
      }
    }
    __syncthreads();
    for (int e = warp; e < m; e += kScanThreads / 32) {
      float d = 0.f;
#pragma unroll
      for (int c = 0; c < C; c += 32) d = fmaf(s_k[e][c + lane], s_q[e][c + lane], d);
      d = warp_sum(d);
      if (lane == 0) s_kq[e] = d;
    }
    __syncthreads();
    for (int e = 0; e < m; ++e) {
      float k[16], qv[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        *reinterpret_cast<float4 *>(k + 4 * c) = *reinterpret_cast<const float4 *>(&s_k[e][c * (C / 4) + sub * 4]);
        *reinterpret_cast<float4 *>(qv + 4 * c) = *reinterpret_cast<const float4 *>(&s_q[e][c * (C / 4) + sub * 4]);
      }
      const float al = KDA ? 1.f : s_a[e], be = s_b[e], kq = s_kq[e];
      float u[RPT], z[RPT];
      if constexpr (KDA) {   // decay the state first: one product per element serves both dots
        float g[16];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<float4 *>(g + 4 * c) = *reinterpret_cast<const float4 *>(&s_g[e][c * (C / 4) + sub * 4]);
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
          for (int c = 0; c < 16; ++c) S[r][c] *= g[c];
      }
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        float u0 = 0.f, u1 = 0.f, z0 = 0.f, z1 = 0.f;
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          z0 = fmaf(S[r][c], qv[c], z0);
          z1 = fmaf(S[r][c + 1], qv[c + 1], z1);
          if constexpr (!M2) {
            u0 = fmaf(S[r][c], k[c], u0);
            u1 = fmaf(S[r][c + 1], k[c + 1], u1);
          }
        }
        u[r] = u0 + u1;
        z[r] = z0 + z1;
      }
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1)
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
          z[r] += __shfl_xor_sync(kFull, z[r], o);
          if constexpr (!M2) u[r] += __shfl_xor_sync(kFull, u[r], o);
        }
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const float v = s_v[e][grp + r * GROUPS];
        const float w = M2 ? be * v : be * fmaf(-al, u[r], v);
        const float o = fmaf(al, z[r], w * kq);
        if (sub == 0) s_o[e][grp + r * GROUPS] = M2 ? fmaf(Dh, v, o) : a.out_scale * o;
#pragma unroll
        for (int c = 0; c < 16; ++c) S[r][c] = KDA ? fmaf(w, k[c], S[r][c]) : fmaf(al, S[r][c], w * k[c]);
      }
    }
    __syncthreads();
    for (int i = t; i < m * (kScanRows / 4); i += kScanThreads) {
      const int e = i / (kScanRows / 4), c = i % (kScanRows / 4) * 4;
      st_stream(a.out + ((tok + e) * a.H + h) * a.R + sl * kScanRows + c, *reinterpret_cast<const float4 *>(&s_o[e][c]));
    }
  }
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = sl * kScanRows + grp + r * GROUPS;
    float *dst = a.hc + ((size_t)q.dst * a.H + h) * tile + (size_t)row * C;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<float4 *>(dst + c * (C / 4) + sub * 4) =
          make_float4(S[r][4 * c], S[r][4 * c + 1], S[r][4 * c + 2], S[r][4 * c + 3]);
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
void launch_scan(const PrefillArgs &a, cudaStream_t s) {
  const dim3 grid((unsigned)((size_t)a.n_seq * a.H * (a.R / kScanRows)));
  if constexpr (KIND == RSSM_MAMBA2)
    if (a.C == 64) {
      scan_kernel<KIND, Tin, 64><<<grid, kScanThreads, 0, s>>>(a);
      return;
    }
  scan_kernel<KIND, Tin, 128><<<grid, kScanThreads, 0, s>>>(a);
}

size_t seq_bytes(int n_seq) { return ((size_t)n_seq * sizeof(PrefillSeq) + 255) & ~(size_t)255; }

}  // namespace

size_t prefill_work_bytes(const rssm_layer_desc &d, int n_seq, int n_tokens) {
  return seq_bytes(n_seq) + (size_t)d.batch * sizeof(int32_t);
}

cudaError_t prefill(PrefillArgs a, void *work, int in_dtype, int read_fmt, int *launches, cudaStream_t s) {
  a.seqs = static_cast<PrefillSeq *>(work);
  a.named = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(work) + seq_bytes(a.n_seq));
  *launches = 0;
  plan_prefill_kernel<<<1, kPlanThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  ++*launches;
  if (e != cudaSuccess) return e;
  const bool bf16 = in_dtype == RSSM_BF16;
  if (m2_chunk_path(a, in_dtype))
    e = m2_chunk_prefill(a, s);
  else if (gdn_chunk_path(a, in_dtype))
    e = gdn_chunk_prefill(a, s);
  else switch (a.kind) {
    case RSSM_MAMBA2:
      bf16 ? launch_scan<RSSM_MAMBA2, __nv_bfloat16>(a, s) : launch_scan<RSSM_MAMBA2, float>(a, s);
      break;
    case RSSM_GDN:
      bf16 ? launch_scan<RSSM_GDN, __nv_bfloat16>(a, s) : launch_scan<RSSM_GDN, float>(a, s);
      break;
    default:
      bf16 ? launch_scan<RSSM_KDA, __nv_bfloat16>(a, s) : launch_scan<RSSM_KDA, float>(a, s);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
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
