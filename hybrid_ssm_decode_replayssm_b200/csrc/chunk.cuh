// Helpers of the chunked prefill kernels: operand tiles in the 128-byte swizzle
// for tcgen05, operands in tensor memory, the three-part bf16 split of fp32
// values, and bounded waits that stop the whole CTA.
#pragma once

#include "rssm_device.cuh"
#include "rssm_prefill.h"
#include "umma.cuh"

namespace rssm {
namespace chunk {

// A tile of 64 bf16 columns is stored as rows of 128 bytes, the 16-byte chunk c
// of row r at chunk position c ^ (r % 8); wider tiles are several such blocks
// of columns.  The same bytes serve as an operand whose K runs along a row (K-major:
// 8-row groups `1024` bytes apart, K = 16 step 32 bytes inside a block) and as one
// whose K runs over the rows (MN-major: 64-column blocks `lbo` bytes apart, 8-row
// groups 1024 bytes apart, K = 16 step 2048 bytes).  Blocks start on 1024 bytes.
__device__ __forceinline__ uint32_t sw128(int row, int c16) {
  return (uint32_t)(row * 128 + ((c16 ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint64_t desc_sw128(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;   // version
  d |= (uint64_t)2 << 61;   // 128-byte swizzle
  return d;
}
// kind::f16, D fp32, A and B bf16; a_mn / b_mn: the operand is MN-major.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem]: A is K-major in tensor memory, lane = row, two
// consecutive K elements per 32-bit column (K = 16: 8 columns).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t id, bool acc) {
  const uint32_t z = 0u;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(id), "r"((uint32_t)acc), "r"(z)
      : "memory");
}
// Store 16 32-bit columns of this warp's lanes.
__device__ __forceinline__ void st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Store 8 32-bit columns of this warp's lanes.
__device__ __forceinline__ void st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 values to three bf16 pairs, x = hi + mid + lo to 2^-24 |x| (element 0
// in the low half); see umma::split3_bf16.
__device__ __forceinline__ uint32_t pack_bf16(float x0, float x1) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x0, x1);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// (x0, x1) - (h0, h1), one packed instruction (exact here: h is x rounded).
__device__ __forceinline__ void sub2(float &x0, float &x1, float h0, float h1) {
  asm("{\n\t.reg .b64 x, h, m;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 h, {%2, %3};\n\tmov.b64 m, {%4, %4};\n\t"
      "fma.rn.f32x2 x, h, m, x;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(h0), "f"(h1), "f"(-1.0f));
}
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  hi = pack_bf16(x0, x1);
  sub2(x0, x1, __uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u));
  mid = pack_bf16(x0, x1);
  sub2(x0, x1, __uint_as_float(mid << 16), __uint_as_float(mid & 0xFFFF0000u));
  lo = pack_bf16(x0, x1);
}

// Sixteen values to three parts of eight 32-bit columns, `step` columns apart.
__device__ __forceinline__ void split_store(uint32_t taddr, int step, const float *v) {
  uint32_t hi[8], mid[8], lo[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) split3(v[2 * j], v[2 * j + 1], hi[j], mid[j], lo[j]);
  st_x8(taddr, hi);
  st_x8(taddr + step, mid);
  st_x8(taddr + 2 * step, lo);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes global -> shared, zeros where `take` is false (the source is not read).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Eight consecutive floats, a whole 32-byte sector, to global memory.
__device__ __forceinline__ void st_sector(float *p, const float *v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// One lane of a converged warp.  (A product issued under `lane == 0` costs 50 cycles of
// issue, under this predicate 32 at N = 64, the tensor core's own time.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Registers per thread of the calling warpgroup (all of its warps call).
template <int N> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Every lane of the warp arrives through lane 0, its writes before it.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// All lanes wait; false (for all) once the CTA gives up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, long long limit) {
  return warp_all(mbar_wait_bounded(bar, parity, abort, limit));
}

// Programmatic launches: wait for the grids before (complete, their writes visible), and
// let the next one begin.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// One thread tells another grid's that what its CTA wrote (before a barrier) is there.
__device__ __forceinline__ void word_release(int32_t *p, int32_t v) {
  asm volatile("st.release.gpu.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ bool word_acquire(const int32_t *p, int32_t want, long long limit) {
  const long long t0 = clock64();
  for (;;) {
    int32_t v;
    asm volatile("ld.acquire.gpu.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v == want) return true;
    if (clock64() - t0 > limit) return false;
    __nanosleep(64);
  }
}

// The next (sequence, head) of a persistent chunk kernel, longest sequences first: every
// thread of the CTA calls, having finished the one before.  False: none is left, or a
// wait gave up.
template <int THREADS, int BARS>
__device__ __forceinline__ bool next_item(const PrefillArgs &a, uint64_t *bar, const int (&count)[BARS], int *s_item,
                                          volatile int *abort, PrefillSeq &q, int &h) {
  for (;;) {
    umma::fence_before_sync();
    named_sync(0, THREADS);
    umma::fence_after_sync();
    if (*abort) return false;
    if (threadIdx.x == 0) {
      *s_item = atomicAdd(a.queue + kChunkQueue, 1);
#pragma unroll
      for (int i = 0; i < BARS; ++i) {
        asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar + i)) : "memory");
        mbar_init(bar + i, count[i]);
      }
      mbar_fence_init();
    }
    named_sync(0, THREADS);
    const int item = *s_item;
    if (item >= a.queue[kLongCount] * a.H) return false;
    q = a.seqs[item / a.H];
    h = item % a.H;
    if (q.dst >= 0 && q.n > a.scan_most) return true;
  }
}

}  // namespace chunk
}  // namespace rssm
