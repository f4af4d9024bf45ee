// The packed key/value cache: quantising new tokens into their pages, and reading them
// back.  The layout of a page and the arithmetic of a group are stated in
// include/bitstack.h.
//
// A thread takes 8 dense numbers at a time (16 bytes, 32 for fp32) or 16 bytes of codes; dense accesses are
// contiguous over a row's lanes and packed ones stay within its 32 to 128 bytes.
//
// A group is s = fp16((max - min) / 15), b = fp16(min + 8 (max - min) / 15),
// c = rint((x - b) / s + 8) in fp32.  A true division for every number made the writing kernel
// slower still; the reciprocal decides all codes but those
// next to a rounding border, which are divided, so the codes are the definition's for every input.
//
// Bytes a (token, head): 4 D dense and 1.25 D packed.  Measured (8 heads of 128, bf16): writing prompts of 8417
// tokens in all and reading them back 29 us together, 0.48 of the copy rate (writing takes 19 of them, fp32 numbers 24, bound
// by its instructions, 28.7 a number at 62 % of the issue slots: half for the codes, the rest for ranges, pairs and
// addresses); reading contexts of 88 thousand tokens 162 to 172 us, 0.84 to 0.89 of it (fp32 377, twice the bytes written); one
// token written and read back 4 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.h"
#include "ptx.cuh"

namespace bs {
namespace {

constexpr int kThreads = 256;
constexpr float kCacheClamp = 65000.0f;   // b + s (c - 8) then stays below fp16's 65504 with both roundings

// Where word w and pair g of a row stand, and token t's row (keys in order, values as
// the attention kernel's fragments want them).
template <int D>
__device__ __forceinline__ int word_place(bool value, int w) {
  return value ? (w & 7) * (D / 64) + (w >> 3) : (w & 3) * (D / 32) + (w >> 2);
}
template <int D>
__device__ __forceinline__ int pair_place(bool value, int g) {
  return value ? (g & 1) * (D / 64) + (g >> 1) : g;
}
__device__ __forceinline__ int token_row(bool value, int t) { return value ? (t >> 1) + 8 * (t & 1) : t; }

template <typename T>
struct Eight;   // 8 dense numbers
template <>
struct Eight<__half> {
  uint4 a;
  // Smallest and largest, NaN if there is one.
  __device__ void range(float& lo, float& hi) const {
    const __half2* h = reinterpret_cast<const __half2*>(&a);
    const __half2 n = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
    const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    lo = __half2float(__hmin_nan(__low2half(n), __high2half(n)));
    hi = __half2float(__hmax_nan(__low2half(m), __high2half(m)));
  }
  __device__ void load(const void* p) { a = *static_cast<const uint4*>(p); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
  __device__ static void store(void* p, const float (&x)[8]) {
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
      r[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *static_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ void range(float& lo, float& hi) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&a);
    const __nv_bfloat162 n = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    lo = __bfloat162float(__hmin_nan(__low2bfloat16(n), __high2bfloat16(n)));
    hi = __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
  }
  __device__ void load(const void* p) { a = *static_cast<const uint4*>(p); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(r[e] << 16);
      x[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
    }
  }
  __device__ static void store(void* p, const float (&x)[8]) {
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      r[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *static_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ void range(float& lo, float& hi) const {
    lo = fminf(fminf(fminf(a.x, a.y), fminf(a.z, a.w)), fminf(fminf(b.x, b.y), fminf(b.z, b.w)));
    hi = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
    const float sum = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));   // NaN if one is, or of infinities
    if (sum != sum) hi = sum;
  }
  __device__ void load(const void* p) {
    a = *static_cast<const float4*>(p);
    b = static_cast<const float4*>(p)[1];
  }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ static void store(void* p, const float (&x)[8]) {
    static_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    static_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// A warp quantises the keys and values of one token for HB heads, 8 numbers a lane and step, all loads first.
// The token's page is looked up once.  grid: (blocks of tokens and head blocks of a sequence, sequences).
template <int D, typename T, int STEPS>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ CacheCopyParams p) {
  constexpr int LR = D / 8;                      // lanes of a row
  constexpr int HB = STEPS * 16 / LR;            // heads of a warp's step run
  griddep_launch_dependents();
  griddep_wait();
  const int seq = blockIdx.y, lane = threadIdx.x & 31;
  const SeqSpan s = seq_span(p.st, seq);
  if (s.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.st.err, kErrRange);
  if (!s.live) return;
  const int heads = p.st.heads;
  const unsigned blocks = (heads + HB - 1) / HB, jobs = static_cast<unsigned>(s.rows) * blocks;
  const unsigned warps = gridDim.x * (kThreads / 32);
  for (unsigned v = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); v < jobs; v += warps) {
    const int i = static_cast<int>(v / blocks), h0 = static_cast<int>(v % blocks) * HB;
    const int pos = s.start + i;
    Eight<T> in[STEPS];
#pragma unroll
    for (int e = 0; e < STEPS; ++e) {
      const int u = e * 32 + lane, h = h0 + u / (2 * LR), kv = u / LR % 2;
      in[e] = Eight<T>{};
      if (h < heads)
        in[e].load(static_cast<const T*>(p.in[kv]) + (s.row0 + i) * p.tok[kv] + h * p.head[kv] + u % LR * 8);
    }
    const int page = p.st.table[static_cast<size_t>(seq) * p.st.stride + (pos >> p.st.page_shift)];
    uint8_t* ch = chunk_at(p.st, page, pos, h0, D);
    if (ch == nullptr) {
      if (lane == 0) atomicOr(p.st.err, kErrRange);
      continue;
    }
    const int head_bytes = (1 << p.st.page_shift) / kChunkTokens * chunk_bytes(D);
#pragma unroll
    for (int e = 0; e < STEPS; ++e) {
      const int u = e * 32 + lane, hd = u / (2 * LR), kv = u / LR % 2, word = u % LR;
      float x[8];
      in[e].get(x);
      float lo, hi;
      in[e].range(lo, hi);
      if (!(lo >= -kCacheClamp && hi <= kCacheClamp)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = x[k] != x[k] ? 0.0f : fminf(fmaxf(x[k], -kCacheClamp), kCacheClamp);
        lo = fminf(fminf(fminf(x[0], x[1]), fminf(x[2], x[3])), fminf(fminf(x[4], x[5]), fminf(x[6], x[7])));
        hi = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      }
#pragma unroll
      for (int o = 1; o < 4; o *= 2) {           // a group is four lanes
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      const float step = __fdiv_rn(hi - lo, 15.0f);
      const __half sh = __float2half_rn(step), bh = __float2half_rn(fmaf(8.0f, step, lo));
      const float sf = __half2float(sh), bf = __half2float(bh);
      // c = rint((x - b) / s + 8) of the definition, by the reciprocal where that decides it: t = ((x - b) / s + 8) / 15
      // clamped to [0, 1] is within 2^-22.5 of its value (the quotient's 2 ulp, the fma's half), and 15 t, like
      // the definition's own sum, within 2^-18.  Codes are put together as fp32 integers below 2^16.
      const float inv = __fdividef(1.0f, 15.0f * sf);
      constexpr float kInt = 12582912.0f;        // 1.5 2^23: adding it rounds to an integer
      float far[8], code[8], most = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float t = __saturatef(fmaf(x[k] - bf, inv, 8.0f / 15.0f));
        code[k] = fmaf(t, 15.0f, kInt) - kInt;
        far[k] = fabsf(fmaf(t, 15.0f, -code[k]));
        most = fmaxf(most, far[k]);
      }
      uint32_t half[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        half[k] = __float_as_uint(fmaf(fmaf(fmaf(code[4 * k + 3], 16.0f, code[4 * k + 2]), 16.0f, code[4 * k + 1]), 16.0f, code[4 * k]) + 8388608.0f);
      uint32_t w = __byte_perm(half[0], half[1], 0x5410);
      constexpr float kBorder = 0.5f - 0x1p-16f;
      if (!(sf > 0.0f)) {
        w = 0x88888888u;
      } else if (most > kBorder) {               // next to a half (numbers on a coarse grid often are): divide
        uint32_t which = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) which |= far[k] > kBorder ? 1u << k : 0u;
#pragma unroll 1
        for (; which != 0; which &= which - 1) {
          const int k = __ffs(which) - 1;
          float xk = x[0];
#pragma unroll
          for (int q = 1; q < 8; ++q) xk = k == q ? x[q] : xk;
          const float c = fminf(fmaxf(rintf(__fadd_rn(__fdiv_rn(xk - bf, sf), 8.0f)), 0.0f), 15.0f);
          w = (w & ~(15u << (4 * k))) | static_cast<uint32_t>(c) << (4 * k);
        }
      }
      if (h0 + hd < heads) {
        uint8_t* at = ch + hd * head_bytes + kv * 10 * D;
        const int row = token_row(kv != 0, pos & (kChunkTokens - 1));
        reinterpret_cast<uint32_t*>(at + row * (D / 2))[word_place<D>(kv != 0, word)] = w;
        if ((lane & 3) == 0)
          reinterpret_cast<uint32_t*>(at + 8 * D + row * (D / 8))[pair_place<D>(kv != 0, word >> 2)] =
              static_cast<uint32_t>(__half_as_ushort(sh)) | static_cast<uint32_t>(__half_as_ushort(bh)) << 16;
      }
    }
  }
}

// 8 codes of a word as numbers b + s (c - 8).
__device__ __forceinline__ void numbers(uint32_t w, uint32_t pair, float (&x)[8]) {
  const float2 sb = __half22float2(*reinterpret_cast<const __half2*>(&pair));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // nibbles k and k + 4: 64 + c (k odd) or 1024 + c in fp16, exact
    uint32_t v = k & 2 ? w >> 8 : w;
    v = k & 1 ? (v & 0x00f000f0u) | 0x54005400u : (v & 0x000f000fu) | 0x64006400u;
    const uint32_t off = k & 1 ? 0xd480d480u : 0xe408e408u;   // - 72, - 1032
    const float2 c = __half22float2(__hadd2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&off)));
    x[k] = fmaf(sb.x, c.x, sb.y);
    x[k + 4] = fmaf(sb.x, c.y, sb.y);
  }
}

// A warp reads one chunk of one head: 16 bytes of codes a lane and access, a quarter to a whole row's worth of
// consecutive lanes, with the pairs they need; a store writes 8 numbers.  grid: (blocks of chunks and heads of a
// sequence, sequences).  Rows of an empty slot, and of pages outside the pool, are zeros.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheCopyParams p) {
  constexpr int UR = D / 32;                     // 16-byte units of a row of codes
  constexpr int N = 16 * UR / 32;                // units of a lane: keys, and as many of values
  constexpr int GR = D / 32, J = D / 64;
  griddep_launch_dependents();
  griddep_wait();
  const int seq = blockIdx.y, lane = threadIdx.x & 31;
  const SeqSpan s = seq_span(p.st, seq);
  if (s.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.st.err, kErrRange);
  if (s.rows == 0) return;
  const int heads = p.st.heads;
  const int start = s.live ? s.start : 0;        // an empty slot's rows go by as if they stood at 0
  const int first = start / kChunkTokens;
  const unsigned chunks = static_cast<unsigned>((start + s.rows - 1) / kChunkTokens - first + 1);
  const unsigned warps = gridDim.x * (kThreads / 32);
  for (unsigned v = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); v < chunks * heads; v += warps) {
    const int h = static_cast<int>(v % heads), pos0 = (first + static_cast<int>(v / heads)) * kChunkTokens;
    const uint8_t* ch = nullptr;
    if (s.live) {
      const int page = p.st.table[static_cast<size_t>(seq) * p.st.stride + (pos0 >> p.st.page_shift)];
      ch = chunk_at(p.st, page, pos0, h, D);
      if (ch == nullptr && lane == 0) atomicOr(p.st.err, kErrRange);
    }
    uint4 code[2][N], pair[2][N];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = i * 32 + lane, row = u / UR, c = u % UR;
        const int r = pos0 + (kv ? (row & 7) * 2 + (row >> 3) : row) - start;
        code[kv][i] = pair[kv][i] = make_uint4(0, 0, 0, 0);
        if (ch == nullptr || r < 0 || r >= s.rows || p.out[kv] == nullptr) continue;
        const uint8_t* base = ch + kv * 10 * D;
        code[kv][i] = *reinterpret_cast<const uint4*>(base + u * 16);
        const uint8_t* pr = base + 8 * D + row * (D / 8);
        if (kv ? J == 4 : GR >= 4) {             // four consecutive pairs
          pair[kv][i] = *reinterpret_cast<const uint4*>(pr + (kv ? c / 4 : c % (GR < 4 ? 1 : GR / 4)) * 16);
        } else if (kv ? J == 2 : true) {         // two, for words 0, 1 and 2, 3
          const uint2 two = *reinterpret_cast<const uint2*>(pr + (kv ? c / 2 * 8 : 0));
          pair[kv][i] = make_uint4(two.x, two.y, two.x, two.y);
        } else {
          const uint32_t one = *reinterpret_cast<const uint32_t*>(pr + c * 4);
          pair[kv][i] = make_uint4(one, one, one, one);
        }
      }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = i * 32 + lane, row = u / UR, c = u % UR;
        const int r = pos0 + (kv ? (row & 7) * 2 + (row >> 3) : row) - start;
        if (r < 0 || r >= s.rows || p.out[kv] == nullptr) continue;
        T* out = static_cast<T*>(p.out[kv]) + (static_cast<size_t>(s.row0 + r) * heads + h) * D;
        const uint32_t cw[4] = {code[kv][i].x, code[kv][i].y, code[kv][i].z, code[kv][i].w};
        const uint32_t pw[4] = {pair[kv][i].x, pair[kv][i].y, pair[kv][i].z, pair[kv][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int place = 4 * c + e;
          const int w = kv ? place / J + 8 * (place % J) : 4 * (place % GR) + place / GR;
          float x[8];
          numbers(cw[e], pw[e], x);
          Eight<T>::store(out + w * 8, x);
        }
      }
  }
}

// Blocks for the longest sequence the step may hold; sequences loop over theirs.
dim3 copy_grid(const StepParams& s, long long warps_of_longest) {
  const long long blocks = (warps_of_longest + kThreads / 32 - 1) / (kThreads / 32);
  return dim3(static_cast<unsigned>(blocks < 1 ? 1 : (blocks > 65535 ? 65535 : blocks)), static_cast<unsigned>(s.n_seqs));
}
long long longest(const StepParams& s) { return s.max_new < s.n_tokens ? s.max_new : s.n_tokens; }

template <int D, typename T, int STEPS>
cudaError_t append_steps(const CacheCopyParams& p, cudaStream_t stream) {
  constexpr int HB = STEPS * 16 / (D / 8);
  return launch_chained(cache_append_kernel<D, T, STEPS>, copy_grid(p.st, longest(p.st) * ((p.st.heads + HB - 1) / HB)),
                        kThreads, 0, stream, p);
}
// Four steps of loads in flight a lane where there is work for all SMs' warps, the fewest otherwise.
template <int D, typename T>
cudaError_t append_as(const CacheCopyParams& p, cudaStream_t stream) {
  const long long units = static_cast<long long>(p.st.n_tokens) * p.st.heads * 2 * (D / 8);
  return units >= p.sms * 64ll * 32 * 4 ? append_steps<D, T, 4>(p, stream) : append_steps<D, T, D == 256 ? 2 : 1>(p, stream);
}
template <int D, typename T>
cudaError_t read_as(const CacheCopyParams& p, cudaStream_t stream) {
  // a sequence of n positions touches at most n / 16 + 2 chunks
  return launch_chained(cache_read_kernel<D, T>, copy_grid(p.st, (longest(p.st) / kChunkTokens + 2) * p.st.heads), kThreads,
                        0, stream, p);
}
template <int D>
cudaError_t append_dim(const CacheCopyParams& p, int dtype, cudaStream_t stream) {
  return dtype == BS_F16 ? append_as<D, __half>(p, stream)
         : dtype == BS_BF16 ? append_as<D, __nv_bfloat16>(p, stream) : append_as<D, float>(p, stream);
}
template <int D>
cudaError_t read_dim(const CacheCopyParams& p, int dtype, cudaStream_t stream) {
  return dtype == BS_F16 ? read_as<D, __half>(p, stream)
         : dtype == BS_BF16 ? read_as<D, __nv_bfloat16>(p, stream) : read_as<D, float>(p, stream);
}

}  // namespace

cudaError_t launch_cache_append(const CacheCopyParams& p, int dim, int dtype, cudaStream_t stream) {
  return dim == 64 ? append_dim<64>(p, dtype, stream)
         : dim == 128 ? append_dim<128>(p, dtype, stream) : append_dim<256>(p, dtype, stream);
}
cudaError_t launch_cache_read(const CacheCopyParams& p, int dim, int dtype, cudaStream_t stream) {
  return dim == 64 ? read_dim<64>(p, dtype, stream)
         : dim == 128 ? read_dim<128>(p, dtype, stream) : read_dim<256>(p, dtype, stream);
}

}  // namespace bs
