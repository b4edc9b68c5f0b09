// Launchers of the prefill scans (prefill.cu) and the row moves (rows.cu) for
// the C-ABI host code.
#pragma once

#include <atomic>

#include "rssm_internal.h"

namespace rssm {

// One sequence of a prefill call as its planner decided it: tokens
// [tok, tok + n) of the packed inputs, the checkpoint slots it reads (src, -1 =
// zero state) and writes (dst).  dst = -1: refused, or nothing to do.
// first: its first chunk in the list of the long sequences' chunks.
struct PrefillSeq {
  int32_t tok, n, src, dst, first, pad[3];
};

// Counters in the workspace: three of the token scan's items, one of the chunked
// kernels', the number of sequences up to the last long one, the long ones' chunks of 64
// tokens, the number up to the last that the token scan takes by 32 rows; the word that says
// the plan is written, and the scan's CTAs that have ended (see scan_kernel); then CTAs begun
// per SM.
enum { kScanTaken = 0, kScanFront, kScanBack, kChunkQueue, kLongCount, kChunkTotal, kFineCount, kPlanned, kScanEnded,
       kCounters };
constexpr int kPlanWritten = 0x5EA7ED01;   // in kPlanned; anything else: not yet
constexpr int kSmCounters = 256 - kCounters;
constexpr int kPrefillSms = 148;   // CTAs of the persistent kernels, one per SM

struct PrefillArgs {
  int kind;
  int B, H, G, hpg, R, C;
  int n_seq, n_tokens;
  int scan_most;              // longest sequence of the token-by-token kernel
  int chunks;                 // a chunked kernel runs in the call, the token scan beside it
  float out_scale;
  const float *A, *D;
  float *hc;
  const void *in[5];
  int64_t stride[5];          // elements between consecutive tokens
  float *out;
  const int32_t *offsets, *rows, *fresh;
  // workspace: the planned sequences, longest first, work counters, and a counter per row
  PrefillSeq *seqs;
  int32_t *queue;
  uint8_t *parts;             // GDN, KDA: what the kernel before the chunks makes of each chunk and head
  int32_t *named;
  // bookkeeping
  int32_t *len, *pending, *flushes;
  int32_t *slot, *dst, *seen, *freelist;   // branching layers only (else NULL)
  uint32_t *status;
  // read copy (NULL: none)
  uint8_t *rc_codes;
  void *rc_scales;
  long long wait_limit;
  int stall_test;             // the first CTA of a chunked kernel, and the scan beside it, take the timeout path
};

// Bytes of the caller's workspace of one call.
size_t prefill_work_bytes(const rssm_layer_desc &d, int n_seq, int n_tokens);
// Binds the workspace in `a` and enqueues the call; *launches counts its kernels.
cudaError_t prefill(PrefillArgs a, void *work, int in_dtype, int read_fmt, int *launches, cudaStream_t s);

// The chunked Mamba-2 scan (m2_prefill.cu): bf16 inputs, headdim 64.
bool m2_chunk_path(const PrefillArgs &a, int in_dtype);
cudaError_t m2_chunk_prefill(const PrefillArgs &a, cudaStream_t s);   // sequences longer than a.scan_most

// The chunked gated delta rule (gdn_prefill.cu): GDN, bf16 inputs.
bool gdn_chunk_path(const PrefillArgs &a, int in_dtype);
size_t gdn_chunk_work(size_t chunks, int H);   // bytes for that many chunks of 64 tokens
cudaError_t gdn_chunk_prefill(const PrefillArgs &a, cudaStream_t s);   // two kernels

// The same with a gate per key channel (kda_prefill.cu): KDA, bf16 inputs.
bool kda_chunk_path(const PrefillArgs &a, int in_dtype);
size_t kda_chunk_work(size_t chunks, int H);
cudaError_t kda_chunk_prefill(const PrefillArgs &a, cudaStream_t s);   // two kernels

// Chunks of 64 tokens that the sequences of more than scan_most tokens can have in a call: they are
// no more than those tokens allow, however many sequences there are.
inline size_t most_chunks(int n_seq, int n_tokens, int scan_most) {
  const size_t fit = (size_t)n_tokens / ((size_t)scan_most + 1);
  return (size_t)n_tokens / 64 + (fit < (size_t)n_seq ? fit : (size_t)n_seq);
}

// Dynamic shared memory beyond the default, asked for once per kernel and device.
inline cudaError_t allow_smem(void (*kernel)(PrefillArgs), int bytes) {
  struct Seen {
    std::atomic<void (*)(PrefillArgs)> kernel[8];
    std::atomic<int> n;
  };
  static Seen seen[64];   // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  Seen *s = dev >= 0 && dev < 64 ? &seen[dev] : nullptr;
  if (s)
    for (int i = 0, n = s->n.load(std::memory_order_acquire); i < n && i < 8; ++i)
      if (s->kernel[i].load(std::memory_order_acquire) == kernel) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && s) {
    const int i = s->n.fetch_add(1, std::memory_order_acq_rel);
    if (i < 8) s->kernel[i].store(kernel, std::memory_order_release);
  }
  return e;
}

// Launch with programmatic stream serialisation: the kernel may begin before the grid
// ahead of it ends, and waits for it itself.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// One side of a row move: the buffers of a layer.
struct RowsSide {
  int B;
  float *hc;
  uint8_t *codes, *scales;
  uint8_t *ring[5];
  int32_t *start, *len, *pending, *flushes;
  int32_t *slot, *dst, *seen, *freelist;   // branching layers only (else NULL)
};
struct RowsArgs {
  RowsSide d, s;              // destination and source layer (equal: one layer)
  int same;                   // one layer is both
  size_t hc_words, code_words, scale_bytes;   // per row: 16-byte words, and bytes of the scales
  int nreg, cap;
  int outer[5], entry_bytes[5];
  uint32_t *status;           // of the destination
  int n;                      // pairs
  const int32_t *dst_rows, *src_rows;
  // rssm_compact_rows
  const int32_t *live;
  int32_t *new_row, *n_live;
};
cudaError_t copy_rows(const RowsArgs &a, int *launches, cudaStream_t s);
cudaError_t compact_rows(const RowsArgs &a, int *launches, cudaStream_t s);

}  // namespace rssm
