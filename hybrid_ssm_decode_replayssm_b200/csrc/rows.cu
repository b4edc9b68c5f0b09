// Row moves: sequences' states copied between rows of one or two layers, rows
// emptied, and the live rows of a batch packed together.
//
// A row is its checkpoint (and read copy), the entries of its rings that are in
// use, and its pointers.  Bound by HBM: each byte is read and written once.  A row is cut
// into parts so that the copies fill the GPU: 96 Mamba-2 rows with FP8 read copies
// (1.04 GB) take 179 us, 5.8 TB/s, 89% of a plain copy's rate; 3 GDN rows (14 MB) 8.4 us, most
// of it the launch and the host's call.
#include "rssm_prefill.h"
#include "chunk.cuh"
#include "slots.cuh"

namespace rssm {
namespace {

constexpr int kMoveThreads = 512;
constexpr int kPlanThreads = 1024;

// What a call does with pair i, from the row lists and pointers alone.
struct Pair {
  int d, s;        // rows; s = -1: empty d
  bool move;       // do it
  bool refuse;     // STATE
};

__device__ __forceinline__ int slot_of(const RowsSide &x, int b) {
  return !x.slot ? b : x.flushes[b] != x.seen[b] ? x.dst[b] : x.slot[b];
}

// Pair i of rssm_copy_rows, its conflicts with the other pairs looked up by the
// calling threads [t, t + nt) together: returns this thread's part of "some
// other pair writes the same row, or (one layer) reads it".
__device__ __forceinline__ bool conflicts(const RowsArgs &a, int i, int d, int s, int t, int nt) {
  const bool reads = a.same && d != s;   // a row copied to itself is not written
  bool hit = false;
  for (int j = t; j < a.n; j += nt)
    if (j != i) hit |= a.dst_rows[j] == d || (reads && a.src_rows[j] == d);
  return hit;
}
__device__ __forceinline__ Pair classify(const RowsArgs &a, int d, int s, bool hit) {
  Pair p;
  p.d = d;
  p.s = s;
  p.refuse = hit || d < 0 || d >= a.d.B || s < -1 || s >= a.s.B || (s >= 0 && a.s.pending[s] != 0);
  p.move = !p.refuse && !(a.same && d == s);
  return p;
}

// Branching destinations (one CTA): a row copied inside the layer shares its
// source's slot; one copied from another layer, or emptied, gets a free slot.
__global__ void __launch_bounds__(kPlanThreads) plan_copy_kernel(const RowsArgs a) {
  const int nt = blockDim.x;
  adopt_folds(a.d.B, a.d.slot, a.d.dst, a.d.seen, a.d.flushes);
  __syncthreads();
  const int nfree = free_slots(a.d.B, a.d.slot, a.d.freelist);
  __syncthreads();
  // how often each row is written, and read
  int32_t *writes = a.d.freelist + 2 * (size_t)a.d.B, *reads = writes + a.d.B;
  for (int b = threadIdx.x; b < a.d.B; b += nt) writes[b] = reads[b] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += nt) {
    const int d = a.dst_rows[i], s = a.src_rows[i];
    if (d >= 0 && d < a.d.B) atomicAdd(writes + d, 1);
    if (a.same && s >= 0 && s < a.d.B) atomicAdd(reads + s, 1);
  }
  __syncthreads();
  int rank = 0;
  for (int i0 = 0; i0 < a.n; i0 += nt) {
    const int i = i0 + threadIdx.x;
    Pair p;
    p.move = false;
    if (i < a.n) {
      const int d = a.dst_rows[i], s = a.src_rows[i];
      // as conflicts(): another pair writes d, or (unless d is only copied to itself) reads it
      const bool hit = d >= 0 && d < a.d.B && (writes[d] > 1 || (a.same && d != s && reads[d] > 0));
      p = classify(a, d, s, hit);
    }
    const bool share = p.move && a.same && p.s >= 0;
    const int need = p.move && !share;
    int excl, tot;
    block_scan(need, excl, tot);
    if (share) a.d.slot[p.d] = a.d.slot[p.s];   // no pair writes the row of a source
    if (need) a.d.slot[p.d] = rank + excl < nfree ? a.d.freelist[rank + excl] : a.d.slot[p.d];   // nfree >= B
    rank += tot;
  }
}

// n 16-byte words from src to dst (src NULL: zeros), part x of nx; eight loads
// in flight per thread before their stores.
__device__ __forceinline__ void move_words(uint4 *dst, const uint4 *src, size_t n, int x, int nx) {
  constexpr int U = 8;
  const size_t step = (size_t)nx * kMoveThreads;
  size_t i = (size_t)x * kMoveThreads + threadIdx.x;
  if (!src) {
    for (; i < n; i += step) __stcs(dst + i, make_uint4(0, 0, 0, 0));
    return;
  }
  for (; i + (U - 1) * step < n; i += U * step) {
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = __ldcs(src + i + k * step);
#pragma unroll
    for (int k = 0; k < U; ++k) __stcs(dst + i + k * step, v[k]);
  }
  for (; i < n; i += step) __stcs(dst + i, __ldcs(src + i));
}

// The ring entries (st + e) % cap, e < n, of one row's region, part x of nx.
template <typename W>
__device__ __forceinline__ void move_entries(uint8_t *dst, const uint8_t *src, int outer, int cap, int ew, int n,
                                             int st, int x, int nx) {
  const W *s = reinterpret_cast<const W *>(src);
  W *d = reinterpret_cast<W *>(dst);
  const int per = n * ew, total = outer * per;
  for (int w = x * kMoveThreads + threadIdx.x; w < total; w += nx * kMoveThreads) {
    const int o = w / per, rem = w - o * per, e = rem / ew;
    int idx = st + e;
    if (idx >= cap) idx -= cap;
    const size_t off = ((size_t)o * cap + idx) * ew + (rem - e * ew);
    d[off] = s[off];
  }
}

// Row s of a.s (-1: nothing) into row d of a.d, by part x of nx of the CTAs.
__device__ __forceinline__ void move_row(const RowsArgs &a, int d, int s, int x, int nx) {
  const bool share = a.same && a.d.slot && s >= 0;   // the slot itself was handed over
  if (!share) {
    const size_t to = a.d.slot ? a.d.slot[d] : d, from = s < 0 ? 0 : slot_of(a.s, s);
    move_words(reinterpret_cast<uint4 *>(a.d.hc) + to * a.hc_words,
               s < 0 ? nullptr : reinterpret_cast<const uint4 *>(a.s.hc) + from * a.hc_words, a.hc_words, x, nx);
    if (a.d.codes) {
      move_words(reinterpret_cast<uint4 *>(a.d.codes) + to * a.code_words,
                 s < 0 ? nullptr : reinterpret_cast<const uint4 *>(a.s.codes) + from * a.code_words, a.code_words, x,
                 nx);
      const size_t nw = a.scale_bytes / 4;
      uint32_t *ds = reinterpret_cast<uint32_t *>(a.d.scales + to * a.scale_bytes);
      const uint32_t *ss = reinterpret_cast<const uint32_t *>(a.s.scales + from * a.scale_bytes);
      for (size_t i = (size_t)x * kMoveThreads + threadIdx.x; i < nw; i += (size_t)nx * kMoveThreads)
        ds[i] = s < 0 ? 0u : ss[i];
    }
  }
  const int st = s < 0 ? 0 : a.s.start[s], len = s < 0 ? 0 : a.s.len[s], pend = s < 0 ? 0 : a.s.pending[s];
  const int n = len + pend;
  if (n > 0 && n <= a.cap)
    for (int r = 0; r < a.nreg; ++r) {
      const int eb = a.entry_bytes[r];
      const size_t rb = (size_t)a.outer[r] * a.cap * eb;
      if (eb % 16 == 0)
        move_entries<uint4>(a.d.ring[r] + d * rb, a.s.ring[r] + s * rb, a.outer[r], a.cap, eb / 16, n, st, x, nx);
      else
        move_entries<uint32_t>(a.d.ring[r] + d * rb, a.s.ring[r] + s * rb, a.outer[r], a.cap, eb / 4, n, st, x, nx);
    }
  if (x == 0 && threadIdx.x == 0) {
    const int f = s < 0 ? 0 : a.s.flushes[s];
    a.d.start[d] = st;
    a.d.len[d] = len;
    a.d.pending[d] = pend;
    a.d.flushes[d] = f;
    if (a.d.slot) a.d.seen[d] = f;
  }
}

__global__ void __launch_bounds__(kMoveThreads) copy_rows_kernel(const RowsArgs a, int nx) {
  const int i = (int)(blockIdx.x / nx), x = (int)(blockIdx.x % nx);
  const int d = a.dst_rows[i], s = a.src_rows[i];
  const bool hit = __syncthreads_or(conflicts(a, i, d, s, threadIdx.x, kMoveThreads));
  const Pair p = classify(a, d, s, hit);
  if (p.refuse && x == 0 && threadIdx.x == 0) atomicOr(a.status, (unsigned)RSSM_STATUS_STATE);
  if (p.move) move_row(a, p.d, p.s, x, nx);
}

// One CTA.  n_live rows are live; a dead row among the first n_live is a hole
// that takes the next live row from behind.  The list of holes is kept in the
// front of new_row until every mover behind has read its own.
__global__ void __launch_bounds__(kPlanThreads) plan_compact_kernel(const RowsArgs a) {
  const int B = a.d.B, nt = blockDim.x;
  chunk::grid_launch_next();   // the moves wait for this grid themselves
  if (a.d.slot) adopt_folds(B, a.d.slot, a.d.dst, a.d.seen, a.d.flushes);
  int n_live = 0;
  for (int b0 = 0; b0 < B; b0 += nt) {
    const int b = b0 + threadIdx.x;
    int excl, tot;
    block_scan(b < B && a.live[b] != 0, excl, tot);
    n_live += tot;
  }
  int holes = 0;
  for (int b0 = 0; b0 < n_live; b0 += nt) {
    const int b = b0 + threadIdx.x;
    const int hole = b < n_live && a.live[b] == 0;
    int excl, tot;
    block_scan(hole, excl, tot);
    if (hole) a.new_row[holes + excl] = b;
    holes += tot;
  }
  __syncthreads();
  int movers = 0;
  for (int b0 = n_live; b0 < B; b0 += nt) {
    const int b = b0 + threadIdx.x;
    const int mover = b < B && a.live[b] != 0;
    int excl, tot;
    block_scan(mover, excl, tot);
    const int to = mover ? a.new_row[movers + excl] : -1;   // as many movers as holes
    if (b < B) a.new_row[b] = to;
    if (mover && a.d.slot) a.d.slot[to] = a.d.slot[b];
    movers += tot;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < n_live; b += nt) a.new_row[b] = a.live[b] != 0 ? b : -1;
  if (threadIdx.x == 0) *a.n_live = n_live;
}

// Sources lie behind the first n_live rows and destinations among them, so no
// row is read after it is written.
__global__ void __launch_bounds__(kMoveThreads) compact_rows_kernel(const RowsArgs a, int nx) {
  chunk::grid_wait();
  const int b = (int)(blockIdx.x / nx), x = (int)(blockIdx.x % nx);
  const int to = a.new_row[b];
  if (to >= 0 && to != b) move_row(a, to, b, x, nx);
}

// CTAs per row: enough that `rows` rows give every SM its four, and no part
// shorter than a thread's eight loads.
int parts(const RowsArgs &a, int rows) {
  const size_t most = (a.hc_words + 8 * kMoveThreads - 1) / (8 * kMoveThreads);
  size_t nx = (148 * 4 + (size_t)rows - 1) / (size_t)rows;
  nx = nx > most ? most : nx;
  return nx < 1 ? 1 : (int)nx;
}

}  // namespace

cudaError_t copy_rows(const RowsArgs &a, int *launches, cudaStream_t s) {
  *launches = 0;
  if (a.d.slot) {
    plan_copy_kernel<<<1, kPlanThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    ++*launches;
    if (e != cudaSuccess) return e;
  }
  const int nx = parts(a, a.n);
  copy_rows_kernel<<<(unsigned)((size_t)a.n * nx), kMoveThreads, 0, s>>>(a, nx);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t compact_rows(const RowsArgs &a, int *launches, cudaStream_t s) {
  plan_compact_kernel<<<1, a.d.B > 256 ? kPlanThreads : 256, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  *launches = 1;
  if (e != cudaSuccess) return e;
  const int nx = parts(a, (a.d.B + 3) / 4);
  ++*launches;
  return launch_early(compact_rows_kernel, (unsigned)((size_t)a.d.B * nx), kMoveThreads, 0, s, a, nx);
}

}  // namespace rssm
