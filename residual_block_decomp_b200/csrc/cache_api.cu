// Host side of the packed key/value cache: sizes, the pool's handle, argument checks and
// kernel dispatch (include/bitstack.h, "packed key/value cache").  No device memory is
// allocated here; what the step's arrays hold is checked by the kernels that read them.
#include <cmath>
#include <new>

#include "cache.h"
#include "internal.h"

using namespace bs;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bs_status cuda_status(cudaError_t e) { return e == cudaSuccess ? BS_OK : BS_ERR_CUDA; }

int page_shift(int page_tokens) {
  for (int s = 4; s <= 8; ++s)
    if (page_tokens == 1 << s) return s;
  return -1;
}
bool shape_ok(int heads, int dim, int page_tokens) {
  return heads >= 1 && heads <= 1024 && (dim == 64 || dim == 128 || dim == 256) && page_shift(page_tokens) >= 0;
}
size_t elem_bytes(bs_dtype dt) { return dt == BS_F32 ? 4 : 2; }

// The checks every step call makes; n_tokens == 0 leaves nothing to do.
bs_status check_step(bs_cache_t cache, const bs_cache_step* st) {
  if (cache == nullptr || st == nullptr) return BS_ERR_INVALID_ARG;
  if (st->n_seqs < 1 || st->n_seqs > kCacheMaxSeqs || st->n_tokens < 0 || st->max_new < 0 || st->table_width < 0 ||
      (st->n_seqs > 1 && st->table_stride < st->table_width))
    return BS_ERR_INVALID_ARG;
  if (st->cu_new == nullptr && st->n_tokens < st->n_seqs) return BS_ERR_INVALID_ARG;
  if (st->start == nullptr || (st->page_table == nullptr && st->table_width > 0)) return BS_ERR_INVALID_ARG;
  if (!aligned(st->cu_new, 4) || !aligned(st->start, 4) || !aligned(st->page_table, 4)) return BS_ERR_ALIGNMENT;
  // rows x heads x words of a row are counted in 32 bits by the kernels
  if (static_cast<long long>(st->n_tokens) * cache->heads * 2 * (cache->dim / 8) > 0x7fffffffll) return BS_ERR_RANGE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BS_ERR_NO_DEVICE;
  return dev == cache->device ? BS_OK : BS_ERR_INVALID_ARG;
}

StepParams step_params(bs_cache_t cache, const bs_cache_step* st) {
  StepParams p{};
  p.pages = cache->pages;
  p.page_bytes = cache->page_bytes;
  p.err = cache->err;
  p.cu = st->cu_new;
  p.start = st->start;
  p.table = st->page_table;
  p.n_seqs = st->n_seqs;
  p.n_tokens = st->n_tokens;
  p.max_new = st->max_new;
  p.width = st->table_width;
  p.stride = st->table_stride;
  p.n_pages = cache->n_pages;
  p.heads = cache->heads;
  p.page_shift = page_shift(cache->page_tokens);
  return p;
}

bool strides_ok(long long tok, long long head, bs_dtype dt) {
  const long long unit = static_cast<long long>(16 / elem_bytes(dt));
  return tok >= 0 && head >= 0 && tok % unit == 0 && head % unit == 0;
}

}  // namespace

extern "C" {

size_t bs_cache_page_bytes(int heads, int dim, int page_tokens) {
  if (!shape_ok(heads, dim, page_tokens)) return 0;
  return static_cast<size_t>(heads) * (page_tokens / kChunkTokens) * chunk_bytes(dim);
}

size_t bs_cache_device_bytes(int heads, int dim, int page_tokens, int n_pages) {
  const size_t page = bs_cache_page_bytes(heads, dim, page_tokens);
  if (page == 0 || n_pages <= 0) return 0;
  return align_up(page * static_cast<size_t>(n_pages), 256) + 256;
}

bs_status bs_cache_create(int heads, int dim, int page_tokens, int n_pages, void* dev_pages, size_t dev_bytes,
                          bs_stream_t stream, bs_cache_t* out) {
  if (out == nullptr || dev_pages == nullptr || n_pages <= 0) return BS_ERR_INVALID_ARG;
  *out = nullptr;
  if (!shape_ok(heads, dim, page_tokens)) return BS_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(dev_pages, 256)) return BS_ERR_ALIGNMENT;
  const size_t need = bs_cache_device_bytes(heads, dim, page_tokens, n_pages);
  if (dev_bytes < need) return BS_ERR_CAPACITY;
  int dev = -1, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || major != 10 || minor != 0)
    return BS_ERR_NO_DEVICE;
  bs_cache_s* c = new (std::nothrow) bs_cache_s();
  if (c == nullptr) return BS_ERR_INVALID_ARG;
  c->heads = heads;
  c->dim = dim;
  c->page_tokens = page_tokens;
  c->n_pages = n_pages;
  c->pages = static_cast<uint8_t*>(dev_pages);
  c->page_bytes = bs_cache_page_bytes(heads, dim, page_tokens);
  c->err = reinterpret_cast<uint32_t*>(c->pages + need - 256);
  c->device = dev;
  c->sm_count = sms;
  c->timeout_ns = 500000000ull;
  c->inject_unreachable = 0;
  if (cudaMemsetAsync(c->err, 0, 256, stream) != cudaSuccess) {
    delete c;
    return BS_ERR_CUDA;
  }
  *out = c;
  return BS_OK;
}

bs_status bs_cache_destroy(bs_cache_t cache) {
  if (cache == nullptr) return BS_ERR_INVALID_ARG;
  delete cache;
  return BS_OK;
}

bs_status bs_cache_append(bs_cache_t cache, const bs_cache_step* step, const void* k, long long k_token_stride,
                          long long k_head_stride, const void* v, long long v_token_stride, long long v_head_stride,
                          bs_dtype dt, bs_stream_t stream) {
  const bs_status s = check_step(cache, step);
  if (s != BS_OK) return s;
  if (dt != BS_F16 && dt != BS_BF16 && dt != BS_F32) return BS_ERR_INVALID_ARG;
  if (step->n_tokens == 0) return BS_OK;
  if (k == nullptr || v == nullptr || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 ||
      v_head_stride < 0)
    return BS_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !strides_ok(k_token_stride, k_head_stride, dt) ||
      !strides_ok(v_token_stride, v_head_stride, dt))
    return BS_ERR_ALIGNMENT;
  CacheCopyParams p{};
  p.st = step_params(cache, step);
  p.in[0] = k;
  p.in[1] = v;
  p.tok[0] = k_token_stride;
  p.tok[1] = v_token_stride;
  p.head[0] = k_head_stride;
  p.head[1] = v_head_stride;
  p.sms = cache->sm_count;
  return cuda_status(launch_cache_append(p, cache->dim, dt, stream));
}

bs_status bs_cache_read(bs_cache_t cache, const bs_cache_step* step, void* k_out, void* v_out, bs_dtype dt,
                        bs_stream_t stream) {
  const bs_status s = check_step(cache, step);
  if (s != BS_OK) return s;
  if (dt != BS_F16 && dt != BS_BF16 && dt != BS_F32) return BS_ERR_INVALID_ARG;
  if (step->n_tokens == 0) return BS_OK;
  if (k_out == nullptr && v_out == nullptr) return BS_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return BS_ERR_ALIGNMENT;
  CacheCopyParams p{};
  p.st = step_params(cache, step);
  p.out[0] = k_out;
  p.out[1] = v_out;
  return cuda_status(launch_cache_read(p, cache->dim, dt, stream));
}

size_t bs_cache_attention_workspace_bytes(bs_cache_t cache, const bs_cache_step* step, int q_heads) {
  if (cache == nullptr || step == nullptr || q_heads <= 0 || q_heads % cache->heads != 0 || step->max_new < 0) return 0;
  const long long rows = static_cast<long long>(step->max_new) * (q_heads / cache->heads);
  return cache_attn_ws(cache->dim, rows > 0x7fffffffll ? 0x7fffffff : static_cast<int>(rows), cache->sm_count).total;
}

bs_status bs_cache_attention(bs_cache_t cache, const bs_cache_step* step, const void* q, long long q_token_stride,
                             long long q_head_stride, int q_heads, bs_dtype dt, float scale, int window, void* out,
                             float* lse, void* workspace, size_t workspace_bytes, bs_stream_t stream) {
  const bs_status s = check_step(cache, step);
  if (s != BS_OK) return s;
  if ((dt != BS_F16 && dt != BS_BF16) || q_heads <= 0 || q_heads % cache->heads != 0 || window < 0 ||
      !std::isfinite(scale * 1.4426950408889634f))
    return BS_ERR_INVALID_ARG;
  if (step->n_tokens == 0) return BS_OK;
  if (q == nullptr || out == nullptr || q_token_stride < 0 || q_head_stride < 0) return BS_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !strides_ok(q_token_stride, q_head_stride, dt))
    return BS_ERR_ALIGNMENT;
  const long long most = static_cast<long long>(step->max_new < step->n_tokens ? step->max_new : step->n_tokens) *
                         (q_heads / cache->heads);
  if (static_cast<long long>(step->n_tokens) * q_heads > 0x7fffffffll) return BS_ERR_RANGE;
  const CacheAttnWs W = cache_attn_ws(cache->dim, static_cast<int>(most), cache->sm_count);
  if (workspace == nullptr || workspace_bytes < W.total) return BS_ERR_CAPACITY;
  if (!aligned(workspace, 256)) return BS_ERR_ALIGNMENT;
  CacheAttnParams p{};
  p.st = step_params(cache, step);
  p.q = q;
  p.q_tok = q_token_stride;
  p.q_head = q_head_stride;
  p.q_heads = q_heads;
  p.group = q_heads / cache->heads;
  p.bf16 = dt == BS_BF16 ? 1 : 0;
  p.window = window == 0 ? 0x7fffffff : window;   // positions are below it
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  p.lse = lse;
  p.cnt = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + W.cnt);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + W.part);
  p.frag = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + W.frag);
  p.grid = cache->sm_count;
  p.timeout_ns = cache->timeout_ns;
  p.inject_unreachable = cache->inject_unreachable;
  return cuda_status(launch_cache_attention(p, cache->dim, static_cast<int>(most), stream));
}

bs_status bs_cache_debug_set_wait(bs_cache_t cache, long long timeout_ns, int unreachable_flag) {
  if (cache == nullptr || timeout_ns <= 0) return BS_ERR_INVALID_ARG;
  cache->timeout_ns = static_cast<unsigned long long>(timeout_ns < 1000 ? 1000 : timeout_ns);
  cache->inject_unreachable = unreachable_flag ? 1 : 0;
  return BS_OK;
}

bs_status bs_cache_get_device_error(bs_cache_t cache) {
  if (cache == nullptr) return BS_ERR_INVALID_ARG;
  // the whole device: the calls may have run on streams that a copy does not wait for
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || (dev != cache->device && cudaSetDevice(cache->device) != cudaSuccess))
    return BS_ERR_CUDA;
  uint32_t v = 0;
  bool ok = cudaDeviceSynchronize() == cudaSuccess && cudaMemcpy(&v, cache->err, sizeof(v), cudaMemcpyDeviceToHost) == cudaSuccess;
  if (ok && v != 0) ok = cudaMemset(cache->err, 0, sizeof(v)) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess;
  if (dev != cache->device) cudaSetDevice(dev);
  if (!ok) return BS_ERR_CUDA;
  if (v == 0) return BS_OK;
  return (v & kErrTimeout) ? BS_ERR_TIMEOUT : (v & kErrRange) ? BS_ERR_RANGE : BS_ERR_CUDA;
}

}  // extern "C"
