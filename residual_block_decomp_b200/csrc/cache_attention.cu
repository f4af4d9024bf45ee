// Attention over the packed key/value cache, for few query rows per key/value head (the
// tokens a model generates; include/bitstack.h, bs_cache_attention).
//
//     o_r = sum_t p_rt v_t / sum_t p_rt,   p_rt = 2^(x_rt - m_r),   x_rt = scale log2(e) q_r . k_t
//
// in one pass over the packed pages with a running maximum m and sum: every packed byte
// is read once, 1.25 D bytes a (token, head), and nothing dense is written.
//
// Work.  An item is one (sequence, head, tile of R = 8 NT query rows); its context is cut
// into tiles of 5120 packed bytes (64, 32 or 16 tokens for D = 64, 128, 256).  The tiles of all
// items form one list, split evenly over the CTAs and, inside a CTA, over its warps, so that one long
// context and many short ones keep all SMs equally busy whatever the lengths (which only the device
// knows).  A warp streams its run of tiles through its own ring of shared-memory stages with
// 16-byte asynchronous copies and never waits for another warp.  What is left of items that several
// warps share is joined in shared memory, of items that several CTAs share in the workspace by the CTA
// that arrives last; both add in the order of the tiles, so results do not depend on timing.
//
// Products.  Tokens are the M side of mma.sync and query rows its N side (8 rows: the heads that share a
// key/value head), so few rows waste little.  tcgen05 would need 128 rows of queries or would take the
// keys through shared memory as dense operands; here the codes go from their packed words to fragments in
// registers.
//  * Keys: (word >> s) & 0x00f000f0 | 0x5400 is a pair of codes as the exact fp16 numbers 64 + c. Per group of
//    32, acc = sum (64 + c) q, and a token's score is the sum over groups of s acc + (b - 72 s) sum q; the
//    second part is one product of the (s, b) pairs as they are stored with (-72 sum, sum), each in two fp16
//    parts (22 bits).  So the scales of keys cost one fp32 fma a group and score, none a number.
//    A query row enters as fp16, scaled by a power of two to have its largest entry in [1, 2) (undone in
//    the fp32 scores): exact down to 2^-14 of that entry (bf16: 2^-17), and within 2^-25 of it below.
//  * Softmax: the accumulator layout holds rows = tokens, columns = query rows.  The reference m of the weights
//    2^(x - m) is taken 7 below the running maximum, and again only when a score passes it by more than 15 (weights
//    stay at or below 2^15, inside fp16): most tiles then need no shuffles and no rescaling, only a vote.  The 7
//    puts fp16's smallest half step, 2^-25, at 2^-32 of the largest weight: with the reference at the maximum the
//    weights of a long flat tail behind one large score, 2^-25 of it each, were all lost to the product, though not to
//    the sum (0.3 % of the row for 128K of them).
//    movmatrix turns the fp16 weights into the next product's B fragment.  Rows that are fp16 themselves take the
//    weights in two fp16 parts: one rounding of the weights and that of the values together moved an fp16 result by
//    1.5 times what its own rounding does, the values' alone move it by 1.3 to 1.4 times (4 sequences of 128K took 8 %
//    longer).  A bf16 result is rounded by 8 times as much, and one part is enough.
//  * Values: bytes of two neighbouring tokens are paired by prmt, made exact fp16 c - 8, then one fma
//    with the tokens' (s, b) pairs rounds the value to fp16 (half a step of fp16, 2^-11 of its size).
//    Scales cannot stay outside the product here as for keys: the token is what is summed over.
//
// What bounds it.  A tile (5120 bytes) takes 702 warp instructions for bf16 rows, 727 for fp16 (keys 190, values 300, softmax
// 70, copies and the loop 150), 0.52 to 0.53 of the issue slots with three warps a scheduler; the arithmetic pipes are 30 to
// 44 % busy.  Measured on the device: 64 sequences of up to 8K (8 heads of 128, 4 queries a head) 104 to 109 us, 0.62 to 0.66
// of the copy rate; 4 of 128K in fp16 160 to 171 us, 0.60 to 0.64; one of 32K 24 us; 777 tokens 12 us, 2 of them for tiles: the list, the
// first copy, the queries and the joins are the rest.  Taken back, each 1 to 3 % slower: three stages a warp instead of two,
// 8, 10, 14 or 16 warps instead of 12, and the keys of the next tile between the values of this one in one stretch of code:
// neither the copies' latency nor the products' is what is waited for.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "cache.h"
#include "ptx.cuh"

namespace bs {
namespace {

constexpr int kTileBytes5k = 5120;
constexpr int kWarps = 12;
constexpr float kNegInf = -INFINITY;
constexpr float kNothing = -3.0e38f;   // the reference before any score
constexpr float kHead = 7.0f;          // how far below the largest score it is taken
constexpr float kLag = 15.0f;          // how far scores may pass it

template <int D, int NT>
struct Cfg {
  static constexpr int TILE = 4096 / D;                       // tokens of a tile: 5120 packed bytes
  static constexpr int TM = TILE / kChunkTokens;              // chunks of a tile
  static constexpr int GR = D / 32;                           // groups of a row
  static constexpr int J = D / 64;                            // value words of a lane and token
  static constexpr int R = 8 * NT;                            // query rows of an item
  static constexpr int OREG = NT * J * 16;                    // accumulators of a lane
  static constexpr int FREG = OREG + 4 * NT;                  // and its maxima and sums
  static constexpr int NW = (NT == 1 && D <= 128) ? kWarps : 8;   // warps
  static constexpr int ST = 2;                                // stages of a warp
  // Tiles (4096 tokens) after which a warp's output is added to a sum in shared memory and begins anew.  A product cuts its
  // terms off at the accumulator's last place instead of rounding them, so that sums of many tokens come out too
  // small, by 2^-30 to 2^-28 of them a token: 0.05 % for a run of 128K, 0.4 % for 1M (an fp16 result's half step is 0.05 %).
  static constexpr int FOLD = 4096 / TILE;
};

// Partial results are laid out [register][lane].
struct FragMeta {
  long long id;          // number of the item's first tile in the list; -1: no partial result here
  int tiles, row0, rows, h, rt;
};
// A warp keeps the partial result of its run's last item in its stages, which are free by then, and that of its
// first item, if others follow, in the workspace (its own CTA reads it back).

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_zfill(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// Nibbles 1 and 5 of a word as the fp16 pair 64 + c; nibbles 0 and 4 as 1024 + c.
__device__ __forceinline__ uint32_t pair64(uint32_t w) { return and_or(w, 0x00f000f0u, 0x54005400u); }
__device__ __forceinline__ uint32_t pair1024(uint32_t w) { return and_or(w, 0x000f000fu, 0x64006400u); }

template <int N>
__device__ __forceinline__ void lds(uint32_t (&r)[N], const uint8_t* p) {
  if constexpr (N == 1) {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x; r[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r[4 * i] = v.x; r[4 * i + 1] = v.y; r[4 * i + 2] = v.z; r[4 * i + 3] = v.w;
    }
  }
}

// A place in the list of tiles: item (seq, h, rt) and tile t of its `tiles`.
struct Cursor {
  int seq, h, rt, t, tiles, rts, first;   // first: the position the item's tiles begin at (a multiple of 16)
  int row0, rows, start, end;             // the sequence's rows and positions; end: positions seen
};
// Where the copies of a warp's run stand: the next chunk's address inside its page, and the table's entries
// for the pages 32 k .. 32 k + 31 of a sequence, one a lane.
struct Feed {
  const uint8_t* next;   // this lane's 16 bytes of the next chunk
  bool good;             // its page is in the pool
  int seq, block, page;
};

template <int D, int NT>
struct Shared {
  using C = Cfg<D, NT>;
  uint8_t stage[C::NW][C::ST][kTileBytes5k];
  float4 sum[C::NW][C::OREG / 4][32];   // State::fold of the lanes
  FragMeta meta[2 * C::NW];
  long long wsum[32];
  int last[2];            // slot of a shared item whose parts this CTA adds up; -1: none
  long long scan_total;
  // then long long prefix[n_seqs + 1]
};

template <int D, int NT>
struct Worker {
  using C = Cfg<D, NT>;
  const CacheAttnParams& p;
  const long long* prefix;
  int lane;

  // Rows, positions and tile count of sequence i (tiles 0 where nothing is attended).
  __device__ void seq(Cursor& c, int i) const {
    const SeqSpan s = seq_span(p.st, i);
    c.seq = i;
    c.row0 = s.row0;
    c.rows = s.rows;
    c.start = s.start;
    c.end = s.start + s.rows;
    c.first = 0;
    c.tiles = 0;
    c.rts = 0;
    if (!s.live) return;
    if (s.start >= p.window) c.first = (s.start - p.window + 1) / kChunkTokens * kChunkTokens;
    c.tiles = (c.end - c.first + C::TILE - 1) / C::TILE;
    c.rts = (s.rows * p.group + C::R - 1) / C::R;
  }
  __device__ void seek(Cursor& c, long long tile) const {
    int lo = 0, hi = p.st.n_seqs - 1;      // the last sequence whose tiles begin at or before `tile`
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (prefix[mid] <= tile) lo = mid;
      else hi = mid - 1;
    }
    seq(c, lo);
    const unsigned long long off = static_cast<unsigned long long>(tile - prefix[lo]);
    unsigned item;                         // fewer than 2^31 of a sequence
    if (off >> 32 == 0) {                  // (divisions in 32 bits where they can be)
      item = static_cast<unsigned>(off) / c.tiles;
      c.t = static_cast<unsigned>(off) % c.tiles;
    } else {
      item = static_cast<unsigned>(off / c.tiles);
      c.t = static_cast<int>(off % c.tiles);
    }
    c.h = item / c.rts;
    c.rt = item % c.rts;
  }
  __device__ void next_item(Cursor& c) const {
    c.t = 0;
    if (++c.rt < c.rts) return;
    c.rt = 0;
    if (++c.h < p.st.heads) return;
    c.h = 0;
    int i = c.seq + 1;
    while (i < p.st.n_seqs - 1 && prefix[i + 1] == prefix[i]) ++i;
    if (i < p.st.n_seqs) seq(c, i);
  }

  // 5120 bytes from the tile's chunks; chunks that are not there (ALL false) become zeros.
  template <bool ALL>
  __device__ __forceinline__ void copy(const uint8_t* const (&src)[C::TM], uint32_t ok, uint32_t stage) const {
    auto one = [&](uint32_t dst, const uint8_t* from, int m) {
      if (ALL) {
        cp16(dst, from);
      } else {
        const bool there = (ok >> m) & 1;
        cp16_zfill(dst, there ? from : p.st.pages, there ? 16 : 0);
      }
    };
    const uint32_t dst = stage + lane * 16;
    if constexpr (D == 64) {
      // two chunks are 160 units: 5 copies a lane, the third astride
#pragma unroll
      for (int m = 0; m < C::TM; m += 2) {
        const bool second = lane >= 16;
        one(dst + m * chunk_bytes(D), src[m], m);
        one(dst + m * chunk_bytes(D) + 512, src[m] + 512, m);
        one(dst + m * chunk_bytes(D) + 1024, second ? src[m + 1] + (1024 - chunk_bytes(D)) : src[m] + 1024, second ? m + 1 : m);
        one(dst + m * chunk_bytes(D) + 1536, src[m + 1] + (1536 - chunk_bytes(D)), m + 1);
        one(dst + m * chunk_bytes(D) + 2048, src[m + 1] + (2048 - chunk_bytes(D)), m + 1);
      }
    } else if constexpr (D == 128) {
#pragma unroll
      for (int m = 0; m < C::TM; ++m)
#pragma unroll
        for (int k = 0; k < 5; ++k) one(dst + m * chunk_bytes(D) + k * 512, src[m] + k * 512, m);
    } else {
      // rows of 128 bytes: the lanes' units are spread over the banks
      const uint32_t dk = stage + (lane ^ ((lane >> 3) & 1)) * 16, dv = stage + (lane ^ ((lane >> 3) << 1)) * 16;
#pragma unroll
      for (int k = 0; k < 10; ++k) one((k < 4 ? dk : (k > 4 && k < 9) ? dv : dst) + k * 512, src[0] + k * 512, 0);
    }
  }

  // Requests tile c.t of the item into `stage`; returns which of its chunks are in the pool.
  __device__ uint32_t request(const Cursor& c, Feed& fd, uint32_t stage) const {
    const uint8_t* src[C::TM];
    uint32_t ok = 0;
    const int pos0 = c.first + c.t * C::TILE, shift = p.st.page_shift;
#pragma unroll
    for (int m = 0; m < C::TM; ++m) {
      const int pos = pos0 + m * kChunkTokens;
      if ((pos & ((1 << shift) - 1)) == 0 || (m == 0 && (c.t == 0 || fd.seq < 0))) {   // a new page, item or run
        const int idx = pos >> shift;
        if (fd.seq != c.seq || fd.block != idx >> 5) {
          fd.seq = c.seq;
          fd.block = idx >> 5;
          const int mine = (fd.block << 5) + lane;
          fd.page = mine <= (c.end - 1) >> shift ? p.st.table[static_cast<size_t>(c.seq) * p.st.stride + mine] : 0;
        }
        const uint32_t page = __shfl_sync(0xffffffffu, fd.page, idx & 31);
        const int in_page = (1 << shift) / kChunkTokens;
        const uint32_t chunk = c.h * in_page + ((pos / kChunkTokens) & (in_page - 1));
        fd.good = page < static_cast<uint32_t>(p.st.n_pages);
        fd.next = p.st.pages + lane * 16 + chunk * chunk_bytes(D);
        if (fd.good) fd.next += static_cast<unsigned long long>(page) * static_cast<uint32_t>(p.st.page_bytes);
        else if (pos < c.end && lane == 0) atomicOr(p.st.err, kErrRange);
      }
      src[m] = fd.next;
      fd.next += chunk_bytes(D);
      if (fd.good && pos < c.end) ok |= 1u << m;
    }
    if (ok == (1u << C::TM) - 1) copy<true>(src, ok, stage);
    else copy<false>(src, ok, stage);
    return ok;
  }
};

// The rows of an item as a lane needs them: query fragments (its row's numbers), the sums over groups as the
// operand of the pairs' product, and for the accumulator columns 2 (lane % 4) + {0, 1} score factors and
// positions.
template <int D, int NT>
struct Rows {
  using C = Cfg<D, NT>;
  uint32_t q[NT][C::GR][4];
  uint32_t sums[NT][C::GR > 4 ? 2 : 1][2];
  float factor[NT][2];
  int pos[NT][2];        // position of the row's token; -1: no such row
  int lowest, highest;   // positions of the item's first and last row

  __device__ void load(const CacheAttnParams& p, const Cursor& c, int lane) {
    const int n = lane >> 2, cc = lane & 3;
    const int total = c.rows * p.group;
    lowest = c.start + c.rt * C::R / p.group;
    highest = c.start + (min((c.rt + 1) * C::R, total) - 1) / p.group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = c.rt * C::R + nt * 8 + n;
      const int i = row / p.group, g = row % p.group;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + (c.row0 + i) * p.q_tok +
                            static_cast<long long>(c.h * p.group + g) * p.q_head + cc * 8;
      uint4 raw[C::GR];
#pragma unroll
      for (int gr = 0; gr < C::GR; ++gr)
        raw[gr] = row < total ? *reinterpret_cast<const uint4*>(src + gr * 32) : make_uint4(0, 0, 0, 0);
      auto two = [&](uint32_t r) {   // two numbers in fp32
        return p.bf16 ? make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u)) : __half22float2(u2h(r));
      };
      uint32_t top = 0;              // exponent bits of the row's largest entry
#pragma unroll
      for (int gr = 0; gr < C::GR; ++gr) {
        const uint32_t r[4] = {raw[gr].x, raw[gr].y, raw[gr].z, raw[gr].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = two(r[e]);
          top = max(top, max(__float_as_uint(v.x) & 0x7f800000u, __float_as_uint(v.y) & 0x7f800000u));
        }
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = static_cast<int>(top >> 23);
      // 2^(127 - ex) as far as that is a normal float; the scale's sign goes with it, so that factors are positive
      const int up = min(max(254 - ex, 1), 254);
      float scale = __uint_as_float(static_cast<uint32_t>(up) << 23);
      float f = ldexpf(fabsf(p.scale_log2), 127 - up);
      f = fmaxf(f, 0x1p-120f);                           // 0 times a hidden score of -inf would be NaN
      if (ex == 255) {                                   // a row with inf or NaN is NaN
        f = __int_as_float(0x7fffffff);
        scale = 0.0f;
      }
      if (p.scale_log2 < 0.0f) scale = -scale;
      if (p.scale_log2 == 0.0f) scale = 0.0f;
      float sum[C::GR];
#pragma unroll
      for (int gr = 0; gr < C::GR; ++gr) {
        uint32_t r[4] = {raw[gr].x, raw[gr].y, raw[gr].z, raw[gr].w};
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = two(r[e]);
          const __half2 h = ex == 255 ? __floats2half2_rn(0.0f, 0.0f) : __floats2half2_rn(v.x * scale, v.y * scale);
          const float2 back = __half22float2(h);
          s += back.x + back.y;
          r[e] = h2u(h);
        }
        // numbers (d, d + 4) pair up as the codes of a word do
        q[nt][gr][0] = __byte_perm(r[0], r[2], 0x5410);
        q[nt][gr][1] = __byte_perm(r[0], r[2], 0x7632);
        q[nt][gr][2] = __byte_perm(r[1], r[3], 0x5410);
        q[nt][gr][3] = __byte_perm(r[1], r[3], 0x7632);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        sum[gr] = s;
      }
      // the pairs' operand: k = 2 cc, 2 cc + 1 meet (s, b) of group cc, the second k half holds what fp16
      // leaves of the sums (D = 64: lanes cc >= 2 of the first half do)
#pragma unroll
      for (int k = 0; k < (C::GR > 4 ? 2 : 1); ++k) {
        float v = sum[k * 4];
#pragma unroll
        for (int gr = 1; gr < (C::GR < 4 ? C::GR : 4); ++gr)
          if ((C::GR < 4 ? cc & 1 : cc) == gr) v = sum[k * 4 + gr];
        const float w = -72.0f * v;
        const __half2 hi = __floats2half2_rn(w, v);
        const float2 hf = __half22float2(hi);
        const __half2 lo = __floats2half2_rn(w - hf.x, v - hf.y);
        sums[nt][k][0] = h2u(C::GR < 4 && cc >= 2 ? lo : hi);
        sums[nt][k][1] = C::GR < 4 ? 0 : h2u(lo);
      }
      const int at = row < total ? c.start + i : -1;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        factor[nt][k] = __shfl_sync(0xffffffffu, f, 8 * cc + 4 * k);
        pos[nt][k] = __shfl_sync(0xffffffffu, at, 8 * cc + 4 * k);
      }
    }
  }
};

// Running softmax state and output of a warp for its item.
template <int D, int NT>
struct State {
  using C = Cfg<D, NT>;
  float o[NT][C::J][4][4];
  float m[NT][2], l[NT][2];   // m: the weights' reference; l: this lane's tokens only until reduce()
  bool folded;                // part of the output is in `sum`, with the same reference

  __device__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < C::J; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[nt][j][e / 4][e % 4] = 0.0f;
      m[nt][0] = m[nt][1] = kNothing;
      l[nt][0] = l[nt][1] = 0.0f;
    }
    folded = false;
  }
  // The output so far goes to the sum (END: the sum comes back to the output).
  template <bool END>
  __device__ void fold(float4 (*sum)[32], int lane) {
#pragma unroll
    for (int i = 0; i < C::OREG / 4; ++i) {
      float(&x)[4] = o[i / (4 * C::J)][i / 4 % C::J][i % 4];
      const float4 s = END || folded ? sum[i][lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (END) {
        x[0] += s.x; x[1] += s.y; x[2] += s.z; x[3] += s.w;
      } else {
        sum[i][lane] = make_float4(x[0] + s.x, x[1] + s.y, x[2] + s.z, x[3] + s.w);
        x[0] = x[1] = x[2] = x[3] = 0.0f;
      }
    }
    folded = !END;
  }
  __device__ void reduce() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int o2 = 4; o2 < 32; o2 *= 2) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], o2);
  }

  // One tile: positions pos0 .., of which `ok` chunks hold tokens; the sequence's rows see begin .. end - 1; `masked`: some
  // (row, token) is hidden.  FINE: weights in two fp16 parts.
  template <bool FINE>
  __device__ void tile(const Rows<D, NT>& q, uint8_t* st, int pos0, int begin, int end, uint32_t ok, bool masked, int window,
                       float4 (*sum)[32], int lane) {
    const int t = lane >> 2, cc = lane & 3;
    if (pos0 + C::TILE > end || pos0 < begin) {
      // tokens behind the context, or in its first chunk before the window, may hold anything: their values become
      // 0 + 0 (c - 8), as 0 times them has to be 0
      for (int i = lane; i < C::TILE; i += 32) {
        if (pos0 + i >= begin && pos0 + i < end) continue;
        uint32_t* pr = reinterpret_cast<uint32_t*>(st + (i >> 4) * chunk_bytes(D) + 18 * D + (((i & 15) >> 1) + 8 * (i & 1)) * (D / 8));
#pragma unroll
        for (int g = 0; g < C::GR; ++g) pr[g] = 0;
      }
      __syncwarp();
    }
    float s[C::TM][NT][4];
#pragma unroll
    for (int mt = 0; mt < C::TM; ++mt) {
      const uint8_t* ch = st + mt * chunk_bytes(D);
      uint32_t wa[C::GR], wb[C::GR], pa[C::GR], pb[C::GR];
      if constexpr (D == 256) {
        const int x = t & 1;   // units are swapped in odd rows
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t r[4];
          lds<4>(r, ch + t * 128 + ((cc * 2 + i) ^ x) * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) wa[4 * i + e] = r[e];
          lds<4>(r, ch + (t + 8) * 128 + ((cc * 2 + i) ^ x) * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) wb[4 * i + e] = r[e];
        }
      } else {
        lds<C::GR>(wa, ch + t * (D / 2) + cc * (D / 8));
        lds<C::GR>(wb, ch + (t + 8) * (D / 2) + cc * (D / 8));
      }
      lds<C::GR>(pa, ch + 8 * D + t * (D / 8));
      lds<C::GR>(pb, ch + 8 * D + (t + 8) * (D / 8));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < (C::GR > 4 ? 2 : 1); ++k) {
        uint32_t ra[1], rb[1];
        const int at = 16 * k + (C::GR < 4 ? cc & 1 : cc) * 4;
        lds<1>(ra, ch + 8 * D + t * (D / 8) + at);
        lds<1>(rb, ch + 8 * D + (t + 8) * (D / 8) + at);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(s[mt][nt], ra[0], rb[0], ra[0], rb[0], q.sums[nt][k][0], q.sums[nt][k][1]);
      }
#pragma unroll
      for (int g = 0; g < C::GR; ++g) {
        const float fa = __low2float(u2h(pa[g])), fb = __low2float(u2h(pb[g]));
        const uint32_t a0 = pair64(wa[g] << 4), a1 = pair64(wb[g] << 4), a2 = pair64(wa[g]), a3 = pair64(wb[g]);
        const uint32_t a4 = pair64(wa[g] >> 4), a5 = pair64(wb[g] >> 4), a6 = pair64(wa[g] >> 8), a7 = pair64(wb[g] >> 8);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma16816(acc, a0, a1, a2, a3, q.q[nt][g][0], q.q[nt][g][1]);
          mma16816(acc, a4, a5, a6, a7, q.q[nt][g][2], q.q[nt][g][3]);
          s[mt][nt][0] = fmaf(fa, acc[0], s[mt][nt][0]);
          s[mt][nt][1] = fmaf(fa, acc[1], s[mt][nt][1]);
          s[mt][nt][2] = fmaf(fb, acc[2], s[mt][nt][2]);
          s[mt][nt][3] = fmaf(fb, acc[3], s[mt][nt][3]);
        }
      }
    }
    if (masked) {
#pragma unroll
      for (int mt = 0; mt < C::TM; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tp = pos0 + mt * 16 + t + (e >> 1) * 8, rp = q.pos[nt][e & 1];
            if (tp > rp || tp <= rp - window || !((ok >> mt) & 1)) s[mt][nt][e] = kNegInf;
          }
    }
    float mx[NT][2];
    bool passed = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mx[nt][k] = fmaxf(s[0][nt][k], s[0][nt][2 + k]);
#pragma unroll
        for (int mt = 1; mt < C::TM; ++mt) mx[nt][k] = fmaxf(mx[nt][k], fmaxf(s[mt][nt][k], s[mt][nt][2 + k]));
        mx[nt][k] *= q.factor[nt][k];
        passed |= mx[nt][k] > __fadd_rd(m[nt][k], kLag);
      }
    if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float corr[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 *= 2) mx[nt][k] = fmaxf(mx[nt][k], __shfl_xor_sync(0xffffffffu, mx[nt][k], o2));
          const float mn = fmaxf(m[nt][k], mx[nt][k] - kHead);
          corr[k] = ex2(m[nt][k] - mn);
          m[nt][k] = mn;
          l[nt][k] *= corr[k];
        }
#pragma unroll
        for (int j = 0; j < C::J; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[nt][j][e / 4][e % 4] *= corr[e & 1];
        if (folded)
#pragma unroll
          for (int i = nt * 4 * C::J; i < (nt + 1) * 4 * C::J; ++i) {
            const float4 x = sum[i][lane];
            sum[i][lane] = make_float4(x.x * corr[0], x.y * corr[1], x.z * corr[0], x.w * corr[1]);
          }
      }
    }
#pragma unroll
    for (int mt = 0; mt < C::TM; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          // From rounded products, as m is one: with a fused one the difference is off by half a step of m, and scores
          // from 2^26 on, whose steps are 8 and more, gave weights of 2^16 and more (infinities) or 0.
          mul_sub2(s[mt][nt][e], s[mt][nt][e + 1], q.factor[nt][0], q.factor[nt][1], m[nt][0], m[nt][1]);
          s[mt][nt][e] = ex2(s[mt][nt][e]);
          s[mt][nt][e + 1] = ex2(s[mt][nt][e + 1]);
        }
#pragma unroll
    for (int mt = 0; mt < C::TM; ++mt) {
      uint32_t b[NT][2], lo[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        l[nt][0] += s[mt][nt][0] + s[mt][nt][2];
        l[nt][1] += s[mt][nt][1] + s[mt][nt][3];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const __half2 hi = __floats2half2_rn(s[mt][nt][2 * k], s[mt][nt][2 * k + 1]);
          b[nt][k] = movmatrix(h2u(hi));
          if (FINE) {
            const float2 f = __half22float2(hi);
            lo[nt][k] = movmatrix(h2u(__floats2half2_rn(s[mt][nt][2 * k] - f.x, s[mt][nt][2 * k + 1] - f.y)));
          }
        }
      }
      // the lane's tokens 2 cc, 2 cc + 1, 2 cc + 8, 2 cc + 9: rows cc, cc + 8, cc + 4, cc + 12
      const uint8_t* ch = st + mt * chunk_bytes(D) + 10 * D;
      uint32_t w[4][C::J], pr[4][C::J];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = cc + (i & 1) * 8 + (i >> 1) * 4;
        if constexpr (D == 256) lds<C::J>(w[i], ch + row * 128 + ((t ^ ((row & 3) << 1)) * 16));
        else lds<C::J>(w[i], ch + row * (D / 2) + t * (D / 16));
        lds<C::J>(pr[i], ch + 8 * D + row * (D / 8) + (t >> 2) * (D / 16));
      }
#pragma unroll
      for (int j = 0; j < C::J; ++j) {
        const uint32_t xl = __byte_perm(w[0][j], w[1][j], 0x5410), xh = __byte_perm(w[0][j], w[1][j], 0x7632);
        const uint32_t yl = __byte_perm(w[2][j], w[3][j], 0x5410), yh = __byte_perm(w[2][j], w[3][j], 0x7632);
        const __half2 sx = u2h(__byte_perm(pr[0][j], pr[1][j], 0x5410)), bx = u2h(__byte_perm(pr[0][j], pr[1][j], 0x7632));
        const __half2 sy = u2h(__byte_perm(pr[2][j], pr[3][j], 0x5410)), by = u2h(__byte_perm(pr[2][j], pr[3][j], 0x7632));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // nibble e of both halves: 1024 + c in place 0, 64 + c in place 1
          auto code = [&](uint32_t w) {
            if (e & 2) w >>= 8;
            return e & 1 ? __hadd2(u2h(pair64(w)), u2h(0xd480d480u))       // - 72
                         : __hadd2(u2h(pair1024(w)), u2h(0xe408e408u));    // - 1032
          };
          const __half2 c0 = code(xl), c1 = code(xh), c2 = code(yl), c3 = code(yh);
          const uint32_t a0 = h2u(__hfma2(c0, sx, bx)), a1 = h2u(__hfma2(c1, sx, bx));
          const uint32_t a2 = h2u(__hfma2(c2, sy, by)), a3 = h2u(__hfma2(c3, sy, by));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[nt][j][e], a0, a1, a2, a3, b[nt][0], b[nt][1]);
            if (FINE) mma16816(o[nt][j][e], a0, a1, a2, a3, lo[nt][0], lo[nt][1]);
          }
        }
      }
    }
  }

  // [four registers][lane] float4: the accumulators, then (m, m, l, l) of the row blocks' columns
  __device__ void store(float* f, int lane) const {
    float4* to = reinterpret_cast<float4*>(f) + lane;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < C::J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          to[((nt * C::J + j) * 4 + e) * 32] = make_float4(o[nt][j][e][0], o[nt][j][e][1], o[nt][j][e][2], o[nt][j][e][3]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) to[(C::OREG / 4 + nt) * 32] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
  }
};

// Writes 8 numbers (dims 8 w ..) of column k of row block nt, and with w == 0 the row's lse.
template <int D, int NT, typename Item>
__device__ __forceinline__ void write_row(const CacheAttnParams& p, const Item& c, int nt, int k, int w, const float (&x)[8],
                                          float m, float l, int lane) {
  const int row = c.rt * Cfg<D, NT>::R + nt * 8 + (lane & 3) * 2 + k;
  if (row >= c.rows * p.group) return;
  const size_t at = static_cast<size_t>(c.row0 + row / p.group) * p.q_heads + c.h * p.group + row % p.group;
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // nothing seen: 0; NaN stays
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = x[2 * e] * inv, b = x[2 * e + 1] * inv;
    if (p.bf16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      r[e] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      r[e] = h2u(__floats2half2_rn(a, b));
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + 8 * w) = make_uint4(r[0], r[1], r[2], r[3]);
  if (p.lse != nullptr && w == 0) p.lse[at] = l == 0.0f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
}

// Joins partial results first, first + step, ... < n of an item (addresses from `at(i)`), in that order, for
// one block of registers, row block nt and word j: 8 numbers each of two rows (columns) a lane.  Two are loaded at a
// time.
struct Joined {
  float4 x[4], ml;   // x[e]: dim e of both columns, dim 4 + e of both; m, m, l, l
};
template <int D, int NT, typename At>
__device__ __forceinline__ Joined join(int first, int step, int n, const At& at, int nt, int j, int lane) {
  using C = Cfg<D, NT>;
  constexpr int B = 2;
  const int r0 = (nt * C::J + j) * 128 + lane, mr = (C::OREG / 4 + nt) * 32 + lane;
  Joined r;
  r.ml = make_float4(kNothing, kNothing, 0.0f, 0.0f);
#pragma unroll
  for (int e = 0; e < 4; ++e) r.x[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int i = first; i < n; i += B * step) {
    float4 ml[B], x[B][4];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      ml[b] = make_float4(kNothing, kNothing, 0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[b][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i + b * step < n) {
        const float4* f = reinterpret_cast<const float4*>(at(i + b * step));
        ml[b] = f[mr];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[b][e] = f[r0 + e * 32];
      }
    }
    const float m0 = fmaxf(r.ml.x, fmaxf(ml[0].x, ml[1].x)), m1 = fmaxf(r.ml.y, fmaxf(ml[0].y, ml[1].y));
    const float k0 = ex2(r.ml.x - m0), k1 = ex2(r.ml.y - m1);
    r.ml = make_float4(m0, m1, r.ml.z * k0, r.ml.w * k1);
#pragma unroll
    for (int e = 0; e < 4; ++e) r.x[e] = make_float4(r.x[e].x * k0, r.x[e].y * k1, r.x[e].z * k0, r.x[e].w * k1);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const float w0 = ex2(ml[b].x - m0), w1 = ex2(ml[b].y - m1);
      r.ml.z = fmaf(w0, ml[b].z, r.ml.z);
      r.ml.w = fmaf(w1, ml[b].w, r.ml.w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r.x[e].x = fmaf(w0, x[b][e].x, r.x[e].x);
        r.x[e].y = fmaf(w1, x[b][e].y, r.x[e].y);
        r.x[e].z = fmaf(w0, x[b][e].z, r.x[e].z);
        r.x[e].w = fmaf(w1, x[b][e].w, r.x[e].w);
      }
    }
  }
  return r;
}
// Both rows of a joined block to the output.
template <int D, int NT>
__device__ __forceinline__ void write_joined(const CacheAttnParams& p, const FragMeta& fm, int nt, int j, const Joined& r, int lane) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = r.x[e].x;
    y[4 + e] = r.x[e].z;
  }
  write_row<D, NT>(p, fm, nt, 0, (lane >> 2) + 8 * j, y, r.ml.x, r.ml.z, lane);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = r.x[e].y;
    y[4 + e] = r.x[e].w;
  }
  write_row<D, NT>(p, fm, nt, 1, (lane >> 2) + 8 * j, y, r.ml.y, r.ml.w, lane);
}
template <int D, int NT>
__device__ __forceinline__ void store_joined(float* f, int nt, int j, const Joined& r, int lane) {
  using C = Cfg<D, NT>;
  float4* to = reinterpret_cast<float4*>(f) + lane;
#pragma unroll
  for (int e = 0; e < 4; ++e) to[((nt * C::J + j) * 4 + e) * 32] = r.x[e];
  if (j == 0) to[(C::OREG / 4 + nt) * 32] = r.ml;
}

template <int D, int NT, bool FINE>
__global__ void __launch_bounds__(Cfg<D, NT>::NW * 32, 1) cache_attention_kernel(const __grid_constant__ CacheAttnParams p) {
  using C = Cfg<D, NT>;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared<D, NT>& sh = *reinterpret_cast<Shared<D, NT>*>(raw);
  long long* prefix = reinterpret_cast<long long*>(raw + sizeof(Shared<D, NT>));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Worker<D, NT> wk{p, prefix, lane};

  griddep_launch_dependents();
  griddep_wait();
  // Tile counts of all sequences, prefix-summed: by every warp for itself up to 32 sequences (the values they write are
  // the same), by the CTA beyond.
  if (lane < 2) sh.meta[2 * warp + lane].id = -1;
  long long T = 0;
  auto tiles_of = [&](int i) -> long long {
    if (i >= p.st.n_seqs) return 0;
    Cursor c;
    wk.seq(c, i);
    return static_cast<long long>(c.tiles) * c.rts * p.st.heads;
  };
  auto scan = [&](long long v) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  if (p.st.n_seqs <= 32) {
    const long long n = tiles_of(lane), upto = scan(n);
    T = __shfl_sync(0xffffffffu, upto, 31);
    if (lane < p.st.n_seqs) prefix[lane] = upto - n;
    if (lane == 0) prefix[p.st.n_seqs] = T;
    __syncwarp();
  } else {
    if (tid == 0) sh.scan_total = 0;
    for (int base = 0; base < p.st.n_seqs; base += C::NW * 32) {
      const int i = base + tid;
      const long long n = tiles_of(i), upto = scan(n);
      if (lane == 31) sh.wsum[warp] = upto;
      __syncthreads();
      long long before = sh.scan_total;
      for (int w = 0; w < warp; ++w) before += sh.wsum[w];
      if (i < p.st.n_seqs) prefix[i] = before + upto - n;
      __syncthreads();
      if (tid == C::NW * 32 - 1) sh.scan_total = before + upto;
      __syncthreads();
    }
    T = sh.scan_total;
    if (tid == 0) prefix[p.st.n_seqs] = T;
    __syncthreads();
  }

  // Tiles of a CTA: a tile for every warp before another CTA takes part, as fewer CTAs have less to join.
  const bool small = T >> 31 == 0;               // divisions in 32 bits where they can be
  const long long per = max(small ? static_cast<long long>((static_cast<uint32_t>(T) + gridDim.x - 1) / gridDim.x)
                                  : (T + gridDim.x - 1) / gridDim.x,
                            static_cast<long long>(C::NW));
  const long long c0 = per * blockIdx.x, c1 = max(min(c0 + per, T), c0);
  const long long share = c1 - c0;
  const long long w0 = c0 + (small ? static_cast<uint32_t>(share) * static_cast<uint32_t>(warp) / C::NW : share * warp / C::NW),
                  w1 = c0 + (small ? static_cast<uint32_t>(share) * static_cast<uint32_t>(warp + 1) / C::NW : share * (warp + 1) / C::NW);
  // Rows that see nothing, and the step's errors: the last CTAs, which have the least to do.
  for (int i = gridDim.x - 1 - blockIdx.x; i < p.st.n_seqs; i += gridDim.x) {
    const SeqSpan s = seq_span(p.st, i);
    if (s.bad && tid == 0) atomicOr(p.st.err, kErrRange);
    if (s.live || s.rows == 0) continue;
    const size_t n = static_cast<size_t>(s.rows) * p.q_heads, at = static_cast<size_t>(s.row0) * p.q_heads;
    for (size_t e = tid; e < n * (D / 8); e += C::NW * 32)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + e * 8) = make_uint4(0, 0, 0, 0);
    if (p.lse != nullptr)
      for (size_t e = tid; e < n; e += C::NW * 32) p.lse[at + e] = kNegInf;
  }
  if (share == 0) return;

  if (w0 < w1) {
    Cursor c, ahead;
    wk.seek(c, w0);
    ahead = c;
    Feed feed{nullptr, false, -1, 0, 0};
    int todo = static_cast<int>(w1 - w0), unasked = todo;
    uint32_t have = 0;                // bits of the requested tiles' chunks, the oldest lowest
    const uint32_t stage0 = smem_u32(sh.stage[warp][0]);
    auto ask = [&](int slot) {
      uint32_t r = 0;
      if (unasked > 0) {
        r = wk.request(ahead, feed, stage0 + slot * kTileBytes5k);
        --unasked;
        if (++ahead.t == ahead.tiles && unasked > 0) wk.next_item(ahead);
      }
      cp_async_commit();
      have = have >> C::TM | r << ((C::ST - 1) * C::TM);
    };
    for (int s = 0; s < C::ST; ++s) ask(s);
    Rows<D, NT> q;
    State<D, NT> st;
    long long item = w0 - c.t;       // number of the item's first tile
    bool fresh = true;
    int seg0 = c.t;
    int slot = 0, stop = 0;          // stop: the tile in front of which the item's run ends or its output is folded
    while (todo > 0) {
      if (fresh) {
        q.load(p, c, lane);
        st.clear();
        fresh = false;
        stop = min(c.tiles, c.t + min(todo, C::FOLD));
      }
      cp_async_wait<C::ST - 1>();
      __syncwarp();
      const int pos0 = c.first + c.t * C::TILE;
      const uint32_t ok = have & ((1u << C::TM) - 1);
      const bool masked = ok != (1u << C::TM) - 1 || pos0 + C::TILE - 1 > q.lowest || pos0 <= q.highest - p.window;
      st.template tile<FINE>(q, sh.stage[warp][slot], pos0, c.start - p.window + 1, c.end, ok, masked, p.window,
                             sh.sum[warp], lane);
      __syncwarp();
      ask(slot);
      slot = slot + 1 == C::ST ? 0 : slot + 1;
      --todo;
      ++c.t;
      if (c.t < stop) continue;
      if (c.t < c.tiles && todo > 0) {
        st.template fold<false>(sh.sum[warp], lane);
        stop = min(c.tiles, c.t + min(todo, C::FOLD));
      } else {
        if (st.folded) st.template fold<true>(sh.sum[warp], lane);
        st.reduce();
        if (seg0 == 0 && c.t == c.tiles) {   // the whole item was this warp's
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < C::J; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  x[e] = st.o[nt][j][e][k];
                  x[4 + e] = st.o[nt][j][e][2 + k];
                }
                write_row<D, NT>(p, c, nt, k, (lane >> 2) + 8 * j, x, st.m[nt][k], st.l[nt][k], lane);
              }
        } else {
          float* f = todo > 0 ? p.frag + static_cast<size_t>(blockIdx.x * C::NW + warp) * (C::FREG * 32)
                              : reinterpret_cast<float*>(sh.stage[warp][0]);
          st.store(f, lane);
          if (lane == 0) sh.meta[2 * warp + (todo > 0 ? 0 : 1)] = FragMeta{item, c.tiles, c.row0, c.rows, c.h, c.rt};
        }
        if (todo > 0) {
          wk.next_item(c);
          item = w1 - todo;
          seg0 = 0;
          fresh = true;
        }
      }
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  // Join what warps share; of what CTAs share write this CTA's part.  Slots are in the order of the list, so an
  // item's are neighbours: every warp finds the items' first slots by vote.
  constexpr int kUnits = NT * C::J;              // blocks of registers: 8 numbers of two rows a lane
  static_assert(2 * C::NW <= 32, "a lane a slot");
  const long long my_id = lane < 2 * C::NW ? sh.meta[lane].id : -1;
  const uint32_t present = __ballot_sync(0xffffffffu, my_id >= 0);
  const uint32_t below = present & ((1u << lane) - 1);
  const long long prev_id = __shfl_sync(0xffffffffu, my_id, below ? 31 - __clz(below) : lane);
  const uint32_t heads = __ballot_sync(0xffffffffu, my_id >= 0 && (below == 0 || prev_id != my_id));
  auto slot_at = [&](int s) -> const float* {
    return s & 1 ? reinterpret_cast<const float*>(sh.stage[s >> 1][0])
                 : static_cast<const float*>(p.frag + static_cast<size_t>(blockIdx.x * C::NW + (s >> 1)) * (C::FREG * 32));
  };
  auto cta_of = [&](long long tile) {
    return small ? static_cast<int>(static_cast<uint32_t>(tile) / static_cast<uint32_t>(per)) : static_cast<int>(tile / per);
  };
  const int n_items = __popc(heads);
#pragma unroll 1
  for (int v = warp; v < n_items * kUnits; v += C::NW) {
    uint32_t hm = heads;
    for (int i = v / kUnits; i > 0; --i) hm &= hm - 1;
    const int head = __ffs(hm) - 1;
    hm &= hm - 1;
    uint32_t slots = present >> head << head;
    if (hm != 0) slots &= (hm & -hm) - 1;
    const FragMeta& fm = sh.meta[head];
    const int u = v % kUnits, j = u % C::J, nt = u / C::J;
    const Joined r = join<D, NT>(0, 1, __popc(slots),
                                 [&](int) {    // asked for in order
                                   const int s = __ffs(slots) - 1;
                                   slots &= slots - 1;
                                   return slot_at(s);
                                 },
                                 nt, j, lane);
    if (fm.id >= c0 && fm.id + fm.tiles <= c1)
      write_joined<D, NT>(p, fm, nt, j, r, lane);
    else
      store_joined<D, NT>(p.part + static_cast<size_t>(blockIdx.x * 2 + (fm.id >= c0 ? 1 : 0)) * (C::FREG * 32), nt, j, r, lane);
  }
  if (tid < 2) sh.last[tid] = -1;
  __syncthreads();

  // Count this CTA's parts (of the item that began before it, and of the one that goes on behind it); the CTA that
  // counts an item's last one adds them up.  The barrier and the count's release order the parts before it.
  if (warp == 0) {
    const bool mine = (heads >> lane) & 1;
    if (mine) {
      const FragMeta& fm = sh.meta[lane];
      if (fm.id < c0 || fm.id + fm.tiles > c1) {
        const int f0 = cta_of(fm.id), f1 = cta_of(fm.id + fm.tiles - 1);
        if (atom_add_acq_rel_gpu(p.cnt + f0, 1u) == static_cast<uint32_t>(f1 - f0)) {
          sh.last[fm.id >= c0 ? 1 : 0] = lane;
          p.cnt[f0] = 0;          // as the next call needs it; nobody else touches it any more
        }
      }
    }
  }
  __syncthreads();
  constexpr int kGroups = C::NW / kUnits;      // warps of a block of registers share the parts
  float4* scratch = reinterpret_cast<float4*>(sh.stage);
  static_assert(2 * C::NW * 2560 <= sizeof(sh.stage), "the groups' results");
#pragma unroll 1
  for (int it = 0; it < 2; ++it) {
    const int slot = sh.last[it];
    if (slot < 0) continue;
    const FragMeta& fm = sh.meta[slot];
    const int f0 = cta_of(fm.id), parts = cta_of(fm.id + fm.tiles - 1) - f0 + 1;
    const int u = warp % kUnits, grp = warp / kUnits, j = u % C::J, nt = u / C::J;
    const float* base = p.part + static_cast<size_t>(f0) * 2 * (C::FREG * 32);
    Joined r;
    if (grp < kGroups)
      r = join<D, NT>(grp, kGroups, parts, [&](int i) { return base + static_cast<size_t>(2 * i + (i == 0 ? 1 : 0)) * (C::FREG * 32); },
                      nt, j, lane);
    if (kGroups > 1) {
      float4* mine = scratch + (it * C::NW + warp) * 160 + lane;
      if (grp > 0 && grp < kGroups) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[e * 32] = r.x[e];
        mine[128] = r.ml;
      }
      __syncthreads();
      if (grp == 0) {
#pragma unroll 1
        for (int g = 1; g < kGroups; ++g) {
          const float4* f = scratch + (it * C::NW + g * kUnits + u) * 160 + lane;
          const float4 ml = f[128];
          const float m0 = fmaxf(r.ml.x, ml.x), m1 = fmaxf(r.ml.y, ml.y);
          const float k0 = ex2(r.ml.x - m0), k1 = ex2(r.ml.y - m1), w0 = ex2(ml.x - m0), w1 = ex2(ml.y - m1);
          r.ml = make_float4(m0, m1, r.ml.z * k0 + w0 * ml.z, r.ml.w * k1 + w1 * ml.w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 x = f[e * 32];
            r.x[e] = make_float4(r.x[e].x * k0 + w0 * x.x, r.x[e].y * k1 + w1 * x.y, r.x[e].z * k0 + w0 * x.z, r.x[e].w * k1 + w1 * x.w);
          }
        }
      }
    }
    if (grp == 0) write_joined<D, NT>(p, fm, nt, j, r, lane);
  }
}

template <int D, int NT, bool FINE>
cudaError_t launch_as(const CacheAttnParams& p, cudaStream_t stream) {
  constexpr int kMost = static_cast<int>(sizeof(Shared<D, NT>) + (kCacheMaxSeqs + 1) * 8);
  // the attribute is the device's: set it once for each (up to 64 devices; every call beyond)
  static std::atomic<unsigned long long> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (bit == 0 || !(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(cache_attention_kernel<D, NT, FINE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  const size_t smem = sizeof(Shared<D, NT>) + (static_cast<size_t>(p.st.n_seqs) + 1) * 8;
  return launch_chained(cache_attention_kernel<D, NT, FINE>, dim3(p.grid), Cfg<D, NT>::NW * 32, smem, stream, p);
}
template <int D, int NT>
cudaError_t launch_type(const CacheAttnParams& p, cudaStream_t stream) {
  return p.bf16 ? launch_as<D, NT, false>(p, stream) : launch_as<D, NT, true>(p, stream);
}
}  // namespace

// The kernel for few rows unpacks a context once for 16 rows (8 at D = 256), the one for many once for 128, but with a
// tile's dozen hand-overs and larger parts to join where an item is split.  So the border is lower where there are
// items for half the SMs and few are split.  The contexts' lengths, which only the device knows, matter as much: the longer
// they are, the fewer rows pay for the kernel for many.  Measured, us (few / many) by rows a head, 4 queries a head, bf16:
//   border 48:  D = 64, 32 sequences of 4000, 4 heads: 48: 53 / 61, 64: 66 / 62, 96: 91 / 62;
//               64 of 1000, 8 heads: 64: 85 / 83, 96: 106 / 84;  of 300: 64: 35 / 56, 96: 63 / 57
//               D = 128, the same: 32 of 4000 48: 85 / 81, 64: 110 / 81;  64 of 1000 48: 99 / 108, 64: 126 / 109;  of 300 64: 70 / 69
//               D = 256: 32 of 4000 32: 151 / 149, 48: 220 / 150;  64 of 300 32: 74 / 106, 48: 93 / 109, 64: 133 / 111
//   border 96:  D = 64, 8 of 4096, 4 heads: 96: 33 / 36, 128: 40 / 37;  1 of 30000: 96: 32 / 39, 128: 37 / 39;
//               1 of 120000, 8 heads: 64: 109 / 108, 96: 158 / 109
//               D = 128: 8 of 4096 96: 49 / 48, 128: 61 / 50;  1 of 30000 96: 47 / 66, 192: 79 / 87, 256: 99 / 85;
//               1 of 4000, 8 heads 128: 26 / 36, 256: 37 / 48;  1 of 120000 64: 187 / 153, 96: 273 / 154
//   border 64:  D = 256: 8 of 4096 48: 65 / 78, 64: 81 / 79, 96: 118 / 82;  1 of 30000 64: 76 / 115, 96: 108 / 118;
//               1 of 120000 48: 394 / 296, 64: 510 / 298
// So the borders fit contexts of some thousand tokens; over 120000 they come up to 1.8 times too late, and over one short
// context, or one of 30000 with few heads, up to 1.4 times too early.
bool cache_attn_many(int dim, int rows, int n_seqs, int heads, int sms) {
  const bool spread = static_cast<long long>(n_seqs) * heads * 2 >= sms;
  return rows > (spread ? 48 : dim == 256 ? 64 : 96) && cache_prefill_smem(dim, n_seqs) <= 227 * 1024;
}

CacheAttnWs cache_attn_ws(int dim, int rows, int sms) {
  CacheAttnWs w{};
  const int nt = rows > 8 && dim <= 128 ? 2 : 1;
  const size_t result = (static_cast<size_t>(nt) * (dim / 64) * 16 + 4 * nt) * 128;
  const size_t warps = nt == 1 && dim <= 128 ? kWarps : 8;
  w.cnt = 0;
  w.part = (static_cast<size_t>(sms) * 4 + 255) / 256 * 256;
  w.frag = w.part + static_cast<size_t>(sms) * 2 * result;
  w.total = w.frag + sms * warps * result;
  // the kernel for many rows has larger parts, and a sum of the same size a CTA
  if (rows > 48) {
    const size_t many = w.part + static_cast<size_t>(sms) * 3 * cache_prefill_part_floats(dim) * 4;
    if (many > w.total) w.total = many;
  }
  return w;
}

// Rows of an item: 8, or 16 where a head has more than 8 (the packed bytes are then
// unpacked half as often); D = 256 keeps 8, whose accumulators are 64 registers already.
cudaError_t launch_cache_attention(const CacheAttnParams& p, int dim, int rows, cudaStream_t stream) {
  if (cache_attn_many(dim, rows, p.st.n_seqs, p.st.heads, p.grid)) return launch_cache_prefill(p, dim, stream);
  if (dim == 64) return rows > 8 ? launch_type<64, 2>(p, stream) : launch_type<64, 1>(p, stream);
  if (dim == 128) return rows > 8 ? launch_type<128, 2>(p, stream) : launch_type<128, 1>(p, stream);
  return launch_type<256, 1>(p, stream);
}

}  // namespace bs
