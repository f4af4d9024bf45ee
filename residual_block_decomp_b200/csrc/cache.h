// Internal declarations of the packed key/value cache: the handle, the layout of a
// chunk, and the step's description as the kernels take it.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace bs {

constexpr int kChunkTokens = 16;     // tokens of a chunk: one matrix tile's rows
constexpr int kCacheMaxSeqs = 4096;  // sequences of a step (their tile counts are prefix-summed in shared memory)

constexpr int kCacheMaxPos = 0x7fffffff - 511;   // positions are below it: the end of a tile stays an int

constexpr uint32_t kErrRange = 2u;   // device error word bit: a step left its bounds

__host__ __device__ constexpr int chunk_bytes(int dim) { return 20 * dim; }

// A step as the kernels take it (pointers to device memory).  The kernels start while the one before them in
// the stream may still run (launch_chained) and wait for it before they load anything: with ordinary loads, as what
// an earlier kernel of the chain wrote is not constant over the life of a kernel that waits for it.
struct StepParams {
  uint8_t* pages;
  unsigned long long page_bytes;
  uint32_t* err;
  const int* cu;
  const int* start;
  const int* table;
  int n_seqs, n_tokens, max_new, width, stride;   // width, stride: entries of a table row, and between rows
  int n_pages, heads;
  int page_shift;                    // log2 of the tokens of a page
};

// What a step says of one sequence, after its checks: `rows` new tokens from row `row0`
// at positions start ..; `live` false where nothing is stored or attended.  Of rows that leave the dense tensors
// those inside them remain.
struct SeqSpan {
  int row0, rows, start;
  bool live, bad;
};
__device__ __forceinline__ SeqSpan seq_span(const StepParams& p, int i) {
  SeqSpan s;
  long long lo, hi;
  if (p.cu != nullptr) {
    lo = p.cu[i];
    hi = p.cu[i + 1];
  } else {
    lo = i;
    hi = i + 1;
  }
  const int start = p.start[i];
  s.bad = lo < 0 || hi < lo || hi > p.n_tokens;
  if (s.bad) {
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.n_tokens ? p.n_tokens : hi;
    if (hi < lo) hi = lo;                        // none
  }
  s.row0 = static_cast<int>(lo);
  s.rows = static_cast<int>(hi - lo);
  s.start = start;
  s.live = !s.bad && start >= 0 && s.rows > 0;
  const long long end = static_cast<long long>(start) + s.rows;
  if (s.live && (s.rows > p.max_new || end > (static_cast<long long>(p.width) << p.page_shift) || end > kCacheMaxPos)) {
    s.live = false;
    s.bad = true;
  }
  return s;
}

// Device bytes of the chunk that holds `pos` of sequence i, head h; nullptr for a page
// outside the pool.
__device__ __forceinline__ uint8_t* chunk_at(const StepParams& p, int page, int pos, int h, int dim) {
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) return nullptr;
  const int cpp = (1 << p.page_shift) / kChunkTokens;
  const int c = (pos & ((1 << p.page_shift) - 1)) / kChunkTokens;
  return p.pages + static_cast<unsigned long long>(page) * p.page_bytes +
         static_cast<unsigned long long>(h * cpp + c) * chunk_bytes(dim);
}

// Attention over the cache: arguments and workspace carve-up.
struct CacheAttnParams {
  StepParams st;
  const void* q;
  long long q_tok, q_head;           // strides in elements
  int q_heads, group;
  int bf16, window;                  // window: 2^31 - 1 when unlimited
  float scale_log2;                  // scale * log2(e): scores are kept in the log2 domain
  void* out;
  float* lse;
  uint32_t* cnt;                     // [grid] arrivals of the item that begins in CTA i's range and leaves it
  float* part;                       // [grid][2] partial results that other CTAs join
  float* frag;                       // [grid][warps] partial results that the CTA itself joins
  int grid;
  unsigned long long timeout_ns;     // bound on every wait of the kernel for many rows
  int inject_unreachable;            // its first CTA leaves out its first copy: those waits run out
};
struct CacheAttnWs {
  size_t cnt, part, frag, total;
};
CacheAttnWs cache_attn_ws(int dim, int rows, int sms);
// Whether `rows` query rows a key/value head (at most) run on the kernel for many rows.
bool cache_attn_many(int dim, int rows, int n_seqs, int heads, int sms);
cudaError_t launch_cache_attention(const CacheAttnParams& p, int dim, int rows, cudaStream_t stream);
// The kernel for many rows (cache_prefill.cu).
size_t cache_prefill_smem(int dim, int n_seqs);
size_t cache_prefill_part_floats(int dim);             // of one partial result
cudaError_t launch_cache_prefill(const CacheAttnParams& p, int dim, cudaStream_t stream);

struct CacheCopyParams {
  StepParams st;
  const void* in[2];                 // keys, values (append)
  void* out[2];                      // keys, values (read)
  long long tok[2], head[2];         // strides of `in` in elements
  int sms;
};
cudaError_t launch_cache_append(const CacheCopyParams& p, int dim, int dtype, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheCopyParams& p, int dim, int dtype, cudaStream_t stream);

// Launches the cache's kernels with programmatic dependent launch: a kernel's blocks may be set up while the kernel ahead
// on the stream ends; each waits for it (griddepcontrol.wait) before it touches device memory.
template <typename P>
cudaError_t launch_chained(void (*kernel)(P), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const P& p) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace bs

// The handle.  Host memory only.
struct bs_cache_s {
  int heads, dim, page_tokens, n_pages;
  uint8_t* pages;
  size_t page_bytes;
  uint32_t* err;
  int device, sm_count;
  unsigned long long timeout_ns;
  int inject_unreachable;
};
