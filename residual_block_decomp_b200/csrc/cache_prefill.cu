// Attention over the packed key/value cache for many query rows per key/value head: a prompt's pieces, or many
// drafted tokens (include/bitstack.h, bs_cache_attention; few rows: cache_attention.cu, whose comments state the
// list of tiles and how it is split).
//
// With many query rows the products bound the time, so they run on tcgen05: an item is one (sequence, head, tile of
// 128 query rows), its context is taken in tiles of 128 tokens (D = 256: 64), and a tile's packed bytes are expanded
// once in shared memory for all rows.  Per tile
//     S = Q K^T             (Q and S in tensor memory, K in shared memory, fp32 sums)
//     P = 2^(S f - m)       as fp16 (two parts for fp16 rows, as in the kernel for few), over S in tensor memory
//     O += P V              (P and O in tensor memory, V in shared memory with the dims contiguous)
// with the reference and sum of a row in registers.  As in the kernel for few rows the reference m lies 7 below the
// maximum and follows it only when a score passes it by 15 (weights up to 2^15), so O is hardly ever rescaled.
//
// Scores stay exact to fp32: a key is b + s (c - 8); s (c - 8) / 2 has 15 bits, so fp16 parts hi = round(s (c - 8) / 2)
// and lo = the fma's remainder hold it exactly (halved, as s (c - 8) alone may pass fp16's range), and the b of a group
// meets the sum of its query numbers in 16 more columns (b in fp16 as stored, the sums in two fp16 parts).  So S costs
// 17 products of K = 16 instead of 8 (D = 128): one fp16 rounding of the keys would have moved the weights by as much
// as the rounding of P does, and the lse, which is fp32, by more than fp32 allows.  Values are rounded to fp16 by
// one fma.
//
// Roles: 8 warps own 16 rows each (softmax, output): they take S and O in the shape in which four neighbouring lanes hold a
// row, so that a row's maximum is two shuffles and no warp waits for another; one warp walks the list
// and has the packed tiles copied ahead (one bulk copy a chunk); 8 warps expand them, the keys of tile t + 1 before the
// values of tile t, whose stage waits for tile t - 1's products; one thread issues all products, S of tile t before O of
// tile t - 1, so that the tensor pipe works on the next tile while the rows are at this one's softmax.
// What was measured on the way (2 sequences of 512 new tokens over 4K, 4 heads a key head): two groups of 128 rows with
// Q in shared memory, 64-token products 141 us, 128-token products 128 us: an operand in shared memory is read at 128
// bytes a clock, and Q and K together take the products' whole time (or more, at 64 tokens) for it.  Q in tensor memory
// halves that, and leaves room for two buffers of S with one group: 111 us; rows held by four neighbouring lanes instead
// of two warps that meet 101; parts of split items joined by 16 warps 97; a tile's own sums and O added up apart 98 (fp16
// rows 108).  A prompt of 4096 over 4096 tokens takes 708 us, from an empty cache 830: tiles are split evenly, and the first
// CTA's are 70 items of one or two, each with 10 us of its own.  The tensor pipe is 27 % busy, the issue slots 41 %.  What bounds it now: a tile of 128 x 128 takes
// 2.9 thousand cycles, of which the expanding warps need 2.6, the rows' warps 2.6 and the products 2.0, each waiting for the
// others a little; about 232 KB go through shared memory (expanded keys 64, values 32, written once and read once,
// packed bytes 20 twice), 1.8 thousand cycles' worth.  Pairs of SMs (cta_group::2) that expand half a tile each
// for 256 rows took 97 to 102 us: the products and the rows' warps then bound a tile.
//
// 8 numbers of a word are kept in the order (0, 4, 1, 5, 2, 6, 3, 7) that unpacking gives, in Q and K alike (a sum
// does not mind), and in V as the order of O's columns, undone where rows are written.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "cache.h"
#include "ptx.cuh"

namespace bs {
namespace {

constexpr float kNothing = -3.0e38f;    // the reference before any score
constexpr float kHead = 7.0f;           // how far below the largest score it is taken
constexpr float kLag = 15.0f;           // how far scores may pass it

// A run of tiles of one item: tiles t0 .. t1 - 1 of `tiles`.
struct Segment {
  long long id;                         // number of the item's first tile
  int seq, row0, rows, start;           // the sequence
  int rt, h, first, tiles;              // the item: its row tile, head, first position and tiles
  int t0, t1;
  int end;                              // positions its last row sees
};

template <int D>
struct PCfg {
  static constexpr int R = 128;                            // query rows of an item
  static constexpr int BT = D == 256 ? 64 : 128;           // tokens of a tile
  static constexpr int KST = 2, VST = D == 64 ? 2 : 1;     // stages of K and V
  static constexpr int H = D / 64;                         // 128-byte column blocks of a row
  static constexpr int GR = D / 32;
  static constexpr int CHUNKS = BT / kChunkTokens;
  static constexpr int TILE_BYTES = CHUNKS * chunk_bytes(D);
  static constexpr int RT = 256, XT = 256;                 // threads of the rows, of the expansion
  static constexpr int HALF_BYTES = TILE_BYTES / 2;        // its keys or its values
  static constexpr int THREADS = RT + XT + 64;
  static constexpr int O_COL = 2 * BT, Q_COL = O_COL + D;  // tensor memory columns: S twice, O, Q
  static constexpr uint32_t TMEM = 512;
  // Tiles (8192 tokens) of a segment after which O is added to a sum in the workspace and begins anew: see the kernel for
  // few rows.  (Half as many tokens would halve what is cut off and double the time that this takes, some 2 us of 100.)
  static constexpr int FOLD = 8192 / BT;
  static_assert(Q_COL + D / 2 <= 512, "tensor memory");
};

template <int D>
struct alignas(1024) PShared {
  using C = PCfg<D>;
  uint8_t khi[C::KST][C::H][C::BT * 128];   // 128-byte swizzled rows
  uint8_t klo[C::KST][C::H][C::BT * 128];
  uint8_t v[C::VST][C::H][C::BT * 128];
  uint8_t qx[128 * 32];                     // the 16 columns of sums and of b: core matrices of 8 rows x 16 bytes
  uint8_t kx[C::KST][C::BT * 32];
  uint8_t staging[2][2][C::HALF_BYTES];     // packed keys, packed values: of the tile in use and of the next
  uint32_t top[2][128];                     // loading Q: the largest entries of a row's halves
  float factor[128];                        // a row's score factor
  uint64_t kfull[C::KST], kempty[C::KST], vfull[C::VST], vempty[C::VST];
  uint64_t qfull, sfull[2], pfull[2], pvdone[2], drained;
  uint64_t cfull[2][2], cempty[2][2];       // staging: [keys, values][slot]
  uint64_t pair[4];                         // the two warps of the same rows meet
  int say[2][8];                            // and what they have to say then
  Segment ends[2];                          // the first and the last one of this CTA
  long long scan_total, wsum[32];
  uint32_t tmem;
  int abort, last[2];
  int good[8], from[8], live[8];            // of tile i % 8: the chunks that are in the pool, the tokens from .. live - 1
                                            // that some row of the item sees
  // then long long prefix[n_seqs + 1]
};

template <int D>
struct List {
  using C = PCfg<D>;
  const CacheAttnParams& p;
  const long long* prefix;

  __device__ int row_tiles(const SeqSpan& s) const { return (s.rows * p.group + C::R - 1) / C::R; }
  // First position, positions seen and tiles of row tile rt of a sequence.
  __device__ void item(const SeqSpan& s, int rt, int& first, int& end, int& tiles) const {
    const int total = s.rows * p.group;
    const int lowest = s.start + rt * C::R / p.group;
    end = s.start + (min((rt + 1) * C::R, total) - 1) / p.group + 1;
    first = lowest >= p.window ? (lowest - p.window + 1) / kChunkTokens * kChunkTokens : 0;
    tiles = (end - first + C::BT - 1) / C::BT;
  }
  // Tiles of row tiles rt0, rt0 + step, ... of sequence i, for all heads.
  __device__ long long count(int i, int rt0, int step) const {
    const SeqSpan s = seq_span(p.st, i);
    if (!s.live) return 0;
    const int rts = row_tiles(s);
    long long n = 0;
    for (int rt = rt0; rt < rts; rt += step) {
      int first, end, tiles;
      item(s, rt, first, end, tiles);
      n += tiles;
    }
    return n * p.st.heads;
  }
  __device__ void cut(Segment& g, long long stop) const {
    g.t1 = static_cast<int>(min(static_cast<long long>(g.tiles), stop - g.id));
  }
  // The segment that begins at `tile` and goes no further than `stop`.  For whole warps: 32 row tiles at a time.
  __device__ Segment at(long long tile, long long stop, int lane) const {
    int lo = 0, hi = p.st.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (prefix[mid] <= tile) lo = mid;
      else hi = mid - 1;
    }
    const SeqSpan s = seq_span(p.st, lo);
    const int rts = row_tiles(s);
    Segment g;
    g.seq = lo;
    g.row0 = s.row0;
    g.rows = s.rows;
    g.start = s.start;
    long long off = tile - prefix[lo];
    for (int base = 0;; base += 32) {
      int first = 0, end = 0, tiles = 0;
      if (base + lane < rts) item(s, base + lane, first, end, tiles);
      long long upto = static_cast<long long>(tiles) * p.st.heads;   // tiles up to and with this lane's row tile
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned behind = __ballot_sync(0xffffffffu, upto > off);
      if (behind == 0 && base + 32 < rts) {
        off -= __shfl_sync(0xffffffffu, upto, 31);
        continue;
      }
      const int at = __ffs(behind) - 1;
      g.rt = base + at;
      g.first = __shfl_sync(0xffffffffu, first, at);
      g.end = __shfl_sync(0xffffffffu, end, at);
      g.tiles = __shfl_sync(0xffffffffu, tiles, at);
      off -= __shfl_sync(0xffffffffu, upto, at) - static_cast<long long>(g.tiles) * p.st.heads;
      break;
    }
    g.h = static_cast<int>(off / g.tiles);
    g.t0 = static_cast<int>(off % g.tiles);
    g.id = tile - g.t0;
    cut(g, stop);
    return g;
  }
  // The one behind it, which begins an item.
  __device__ void next(Segment& g, long long stop, int lane) const {
    const long long tile = g.id + g.tiles;
    if (tile >= stop) return;
    if (g.h + 1 < p.st.heads) {
      ++g.h;
      g.id = tile;
      g.t0 = 0;
      cut(g, stop);
    } else {
      g = at(tile, stop, lane);
    }
  }
};

// Products of one tile are issued by one thread at a rate that counts, so descriptors are taken as their low words
// (address and leading offset); the high words are constants.
template <uint32_t HI>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(HI)
      : "memory");
}
template <uint32_t HI>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(HI)
      : "memory");
}
// 128-byte swizzle: rows of 128 bytes, 16-byte units permuted by the row, groups of 8 rows 1024 bytes apart (high
// word); `lbo` (operands with M or N contiguous only) is the distance of 64-number blocks along M or N.
constexpr uint32_t kSw128 = 1024 >> 4 | 1u << 14 | 2u << 29;
// No swizzle: core matrices of 8 rows x 16 bytes, along M or N 128 bytes apart (high word), along K `lbo`.
constexpr uint32_t kPlain = 128 >> 4 | 1u << 14;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFFu) | (lbo >> 4) << 16;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 64 columns: register 4 n + e of lane 4 r + c holds row r + 8 (e / 2), column 8 n + 2 c + e % 2.
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 lanes x 32 columns: register 2 n + e of lane 4 r + c holds row r + 8 e, column 4 n + c: pairs of the above, packed.
__device__ __forceinline__ void tmem_st_pairs(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void sts16(uint8_t* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}
// Unit (16 bytes) w of row r in a block of 128-byte rows.
__device__ __forceinline__ int swz(int r, int w) { return r * 128 + ((w ^ (r & 7)) << 4); }

// A word of a row from the four lanes that hold it: lane c has columns 2 c, 2 c + 1, which are dims c and c + 4; it
// writes dims 2 c and 2 c + 1.
__device__ __forceinline__ void write_word(uint16_t* row, int w, float a, float b, int bf16, bool there, int lane) {
  uint32_t mine;
  if (bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    mine = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    mine = h2u(__floats2half2_rn(a, b));
  }
  const int from = (lane & ~3) + 2 * (lane & 1);
  const uint32_t u = __shfl_sync(0xffffffffu, mine, from), v = __shfl_sync(0xffffffffu, mine, from + 1);
  if (there) reinterpret_cast<uint32_t*>(row + 8 * w)[lane & 3] = __byte_perm(u, v, lane & 2 ? 0x7632 : 0x5410);
}

template <int D>
__global__ void __launch_bounds__(PCfg<D>::THREADS, 1) cache_prefill_kernel(const __grid_constant__ CacheAttnParams p) {
  using C = PCfg<D>;
  extern __shared__ uint8_t raw[];
  PShared<D>& sh = *reinterpret_cast<PShared<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  long long* prefix = reinterpret_cast<long long*>(&sh + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kRowWarps = C::RT / 32, kCopyWarp = kRowWarps + C::XT / 32, kMmaWarp = kCopyWarp + 1, BT = C::BT;
  const List<D> list{p, prefix};

  if (warp == kMmaWarp) tmem_alloc(&sh.tmem, C::TMEM);
  if (tid == 0) {
    for (int i = 0; i < C::KST; ++i) {
      mbar_init(&sh.kfull[i], C::XT / 32);
      mbar_init(&sh.kempty[i], 1);
    }
    for (int i = 0; i < C::VST; ++i) {
      mbar_init(&sh.vfull[i], C::XT / 32);
      mbar_init(&sh.vempty[i], 1);
    }
    mbar_init(&sh.qfull, kRowWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pfull[i], kRowWarps);
      mbar_init(&sh.pvdone[i], 1);
      for (int kv = 0; kv < 2; ++kv) {
        mbar_init(&sh.cfull[kv][i], 1);
        mbar_init(&sh.cempty[kv][i], C::XT / 32);
      }
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.pair[i], 2);
    mbar_init(&sh.drained, 1);
    fence_barrier_init();
    sh.abort = 0;
    sh.scan_total = 0;
  }
  // extra columns that hold no sum are zero
  for (int i = tid; i < 256; i += C::THREADS) sts16(sh.qx + i * 16, 0, 0, 0, 0);
  for (int i = tid; i < C::KST * BT * 2; i += C::THREADS) sts16(sh.kx[0] + i * 16, 0, 0, 0, 0);
  fence_proxy_async_smem();
  griddep_launch_dependents();
  griddep_wait();
  // Tiles of every sequence: a thread counts a sequence's, or a warp where a sequence may have many row tiles; then
  // their prefix sums.
  if (static_cast<long long>(p.st.max_new) * p.group > 4 * C::R) {
    for (int i = warp; i < p.st.n_seqs; i += C::THREADS / 32) {
      long long n = list.count(i, lane, 32);
#pragma unroll
      for (int o = 16; o > 0; o /= 2) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (lane == 0) prefix[i] = n;
    }
  } else {
    for (int i = tid; i < p.st.n_seqs; i += C::THREADS) prefix[i] = list.count(i, 0, 1);
  }
  __syncthreads();
  for (int base = 0; base < p.st.n_seqs; base += C::THREADS) {
    const int i = base + tid;
    const long long n = i < p.st.n_seqs ? prefix[i] : 0;
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sh.wsum[warp] = inc;
    __syncthreads();
    long long before = sh.scan_total;
    for (int w = 0; w < warp; ++w) before += sh.wsum[w];
    if (i < p.st.n_seqs) prefix[i] = before + inc - n;
    __syncthreads();
    if (tid == C::THREADS - 1) sh.scan_total = before + inc;
    __syncthreads();
  }
  const long long T = sh.scan_total;
  if (tid == 0) prefix[p.st.n_seqs] = T;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  // rows that see nothing, and the step's errors
  for (int i = blockIdx.x; i < p.st.n_seqs; i += gridDim.x) {
    const SeqSpan s = seq_span(p.st, i);
    if (s.bad && tid == 0) atomicOr(p.st.err, kErrRange);
    if (s.live || s.rows == 0) continue;
    const size_t n = static_cast<size_t>(s.rows) * p.q_heads, at = static_cast<size_t>(s.row0) * p.q_heads;
    for (size_t e = tid; e < n * (D / 8); e += C::THREADS)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + e * 8) = make_uint4(0, 0, 0, 0);
    if (p.lse != nullptr)
      for (size_t e = tid; e < n; e += C::THREADS) p.lse[at + e] = -INFINITY;
  }

  // CTAs with work: at least two tiles each, as what is split has to be joined
  const long long n = min(static_cast<long long>(gridDim.x), (T + 1) / 2);
  const bool works = blockIdx.x < n;
  const long long c0 = works ? T * blockIdx.x / n : 0, c1 = works ? T * (blockIdx.x + 1) / n : 0;
  volatile int* abort = &sh.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {   // whole warps; false once something gave up
    if (__all_sync(0xffffffffu, mbar_test(bar, parity & 1))) return true;
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity & 1, globaltimer_ns() + p.timeout_ns, abort));
    if (!ok && lane == 0) {
      *abort = 1;
      atomicOr(p.st.err, kErrTimeout);
    }
    return ok;
  };

  if (warp < kRowWarps) {
    // ------------------------------------------------------------ rows: softmax and output
    // Warp (quadrant, hf): rows 32 quadrant + 16 hf .. of the item, two a lane; for Q the quadrant's 32 rows, a lane a row,
    // and half hf of its numbers.
    const int quadrant = warp & 3, hf = warp >> 2;
    const uint32_t quad_at = tmem + (static_cast<uint32_t>(quadrant * 32) << 16);
    const uint32_t lanes = quad_at + (static_cast<uint32_t>(hf * 16) << 16);
    uint32_t i = 0;                                             // tiles so far: phases of all barriers
    bool ok = true;
    // The two warps of a quadrant meet: what either wrote to shared memory before is there for the other, and both know
    // whether one gave up.
    uint32_t met = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) {
        *reinterpret_cast<volatile int*>(&sh.say[met & 1][warp]) = ok ? 0 : 1;
        mbar_arrive(&sh.pair[quadrant]);
      }
      __syncwarp();
      ok = wait(&sh.pair[quadrant], met) && ok;
      if (*reinterpret_cast<volatile int*>(&sh.say[met & 1][warp ^ 4]) != 0) ok = false;
      ++met;
    };
    Segment sg{};
    if (works) sg = list.at(c0, c1, lane);
    for (long long tile = c0; tile < c1 && ok; list.next(sg, c1, lane)) {
      tile = sg.id + sg.t1;
      const int total = sg.rows * p.group;
      const int lowest = sg.start + sg.rt * C::R / p.group, highest = sg.end - 1;
      {
        // a row as fp16, its largest entry in [1, 2), into tensor memory; sums over groups, halved, into qx.  (Loops are
        // kept as loops: this runs once an item, and instructions that run once are fetched at memory's pace.)
        const int r = quadrant * 32 + lane, row = sg.rt * C::R + r;
        const bool there = row < total;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (sg.row0 + row / p.group) * p.q_tok +
                                                          static_cast<long long>(sg.h * p.group + row % p.group) * p.q_head) + hf * (D / 16);
        uint32_t top = 0;
#pragma unroll 4
        for (int w = 0; w < D / 16; ++w) {
          const uint4 a = there ? src[w] : make_uint4(0, 0, 0, 0);
          top = __vmaxu2(__vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu)), top);
        }
        top = max(top & 0xffffu, top >> 16);
        sh.top[hf][r] = top;
        uint4 raw[4];                                           // a group's numbers, loaded one group ahead
#pragma unroll
        for (int k = 0; k < 4; ++k) raw[k] = there ? src[k] : make_uint4(0, 0, 0, 0);
        meet();
        if (!ok) break;
        top = max(top, sh.top[hf ^ 1][r]);
        const uint32_t bits = p.bf16 ? top << 16 : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
        const int ex = static_cast<int>(bits >> 23);
        const int up = min(max(254 - ex, 1), 254);
        float scale = __uint_as_float(static_cast<uint32_t>(up) << 23);
        float f = fmaxf(ldexpf(fabsf(p.scale_log2), 128 - up), 0x1p-120f);   // 2 for the halved keys
        if (ex == 255) f = __int_as_float(0x7fffffff);          // a row with inf or NaN is NaN
        if (p.scale_log2 < 0.0f) scale = -scale;
        if (p.scale_log2 == 0.0f) scale = 0.0f;
        if (hf == 0) sh.factor[r] = f;
#pragma unroll 1
        for (int g = 0; g < C::GR / 2; ++g) {
          const int gr = hf * (C::GR / 2) + g;
          float sum = 0.0f;
          uint32_t cols[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool finite = ex != 255;
            const uint32_t x[4] = {finite ? raw[k].x : 0, finite ? raw[k].y : 0, finite ? raw[k].z : 0, finite ? raw[k].w : 0};
            if (there && g + 1 < C::GR / 2) raw[k] = src[4 * (g + 1) + k];
            uint32_t h[4];                                      // dims 2 e, 2 e + 1
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = p.bf16 ? make_float2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u)) : __half22float2(u2h(x[e]));
              const __half2 y = __floats2half2_rn(v.x * scale, v.y * scale);
              const float2 b = __half22float2(y);
              sum += b.x + b.y;
              h[e] = h2u(y);
            }
            cols[4 * k] = __byte_perm(h[0], h[2], 0x5410);
            cols[4 * k + 1] = __byte_perm(h[0], h[2], 0x7632);
            cols[4 * k + 2] = __byte_perm(h[1], h[3], 0x5410);
            cols[4 * k + 3] = __byte_perm(h[1], h[3], 0x7632);
          }
          __syncwarp();
          tmem_st16(quad_at + C::Q_COL + gr * 16, cols);
          sum *= 0.5f;
          const __half hi = __float2half_rn(sum), lo = __float2half_rn(sum - __half2float(hi));
          auto put = [&](int col, __half x) {
            *reinterpret_cast<__half*>(sh.qx + (col >> 3) * (128 * 16) + r * 16 + (col & 7) * 2) = x;
          };
          put(gr, hi);
          put(C::GR + gr, lo);
        }
        tc_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.qfull);
        meet();                                                 // the rows' factors
        if (!ok) break;
      }
      // the lane's two rows
      float f[2], m[2], l[2];
      int pos[2];                                               // -1: no such row
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = quadrant * 32 + hf * 16 + (lane >> 2) + 8 * k, row = sg.rt * C::R + r;
        pos[k] = row < total ? sg.start + row / p.group : -1;
        f[k] = sh.factor[r];
        m[k] = kNothing;
        l[k] = 0.0f;
      }
      for (int t = sg.t0; t < sg.t1; ++t, ++i) {
        const int buf = i & 1;
        const uint32_t s_at = lanes + buf * BT;
        const int pos0 = sg.first + t * BT;
        ok = wait(&sh.sfull[buf], i >> 1);
        if (!ok) break;
        tc_fence_after();
        const int good = *reinterpret_cast<volatile int*>(&sh.good[i & 7]);
        const bool masked = pos0 + BT - 1 > lowest || pos0 <= highest - p.window || good != (1 << C::CHUNKS) - 1;
        // 64 tokens at a time, twice: for the maximum, and for the weights.  Hidden scores become -inf: tokens behind the
        // row's own, those the window leaves out, chunks outside the pool.
        uint32_t x[32];
        auto load = [&](int c) {
          tmem_ld_rows(s_at + c, x);
          tc_wait_ld();
          if (masked) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int col = c + (j >> 2) * 8 + 2 * (lane & 3) + (j & 1), k = (j >> 1) & 1;
              if (pos0 + col > pos[k] || pos0 + col <= pos[k] - p.window || !((good >> (col >> 4)) & 1)) x[j] = 0xff800000u;
            }
          }
        };
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < BT; c += 64) {
          load(c);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            top[0] = fmaxf(top[0], fmaxf(__uint_as_float(x[j]), __uint_as_float(x[j + 1])));
            top[1] = fmaxf(top[1], fmaxf(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])));
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 1));
          top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 2)) * f[k];
        }
        const bool fold = t > sg.t0 && ((t - sg.t0) & (C::FOLD - 1)) == 0;   // O of the tiles so far goes to the sum
        if (__any_sync(0xffffffffu, fold || top[0] > __fadd_rd(m[0], kLag) || top[1] > __fadd_rd(m[1], kLag))) {
          float keep[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float mn = top[k] > __fadd_rd(m[k], kLag) ? top[k] - kHead : m[k];
            keep[k] = ex2(m[k] - mn);
            l[k] *= keep[k];
            m[k] = mn;
          }
          if (t > sg.t0) {                                      // O of this item exists once the tile before is added
            ok = wait(&sh.pvdone[(i - 1) & 1], (i - 1) >> 1);
            if (!ok) break;
            tc_fence_after();
            float* sum_at = p.part + static_cast<size_t>(gridDim.x * 2 + blockIdx.x) * ((D + 2) * C::R);
            float* ref_at = sum_at + D * C::R + quadrant * 32 + hf * 16 + (lane >> 2);
            const bool more = t - sg.t0 > C::FOLD;
            const float was[2] = {fold && more ? ex2(ref_at[0] - m[0]) : 0.0f, fold && more ? ex2(ref_at[8] - m[1]) : 0.0f};
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
              tmem_ld_rows(lanes + C::O_COL + c, x);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * keep[(j >> 1) & 1]);
              if (!fold) {
                tmem_st_rows(lanes + C::O_COL + c, x);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  float* to = sum_at + (c / 2 + j) * C::RT + tid;
                  *to = __uint_as_float(x[j]) + (more ? *to * was[(j >> 1) & 1] : 0.0f);
                }
              }
            }
            if (fold) {
              __syncwarp();
              if ((lane & 3) == 0) {
                ref_at[0] = m[0];
                ref_at[8] = m[1];
              }
              __syncwarp();
            }
          }
        }
        // a tile's weights are summed by themselves: one by one, those below 2^-25 of a long context's sum would be lost
        float sum[2] = {0.0f, 0.0f};
#pragma unroll 1
        for (int c = 0; c < BT; c += 64) {
          load(c);
          uint32_t pr[16];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float a = __uint_as_float(x[j]), b = __uint_as_float(x[j + 1]);
            float d = __uint_as_float(x[j + 2]), e = __uint_as_float(x[j + 3]);
            mul_sub2(a, b, f[0], f[0], m[0], m[0]);             // rounded products, as the reference is one (see the kernel
            mul_sub2(d, e, f[1], f[1], m[1], m[1]);             // for few rows)
            a = ex2(a), b = ex2(b), d = ex2(d), e = ex2(e);
            sum[0] += a + b;
            sum[1] += d + e;
            pr[j / 2] = h2u(__floats2half2_rn(a, b));
            pr[j / 2 + 1] = h2u(__floats2half2_rn(d, e));
            x[j] = __float_as_uint(a);
            x[j + 1] = __float_as_uint(b);
            x[j + 2] = __float_as_uint(d);
            x[j + 3] = __float_as_uint(e);
          }
          tmem_st_pairs(s_at + c, pr);                          // over scores of these rows that have been read
          if (!p.bf16) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 h = __half22float2(u2h(pr[j / 2]));   // registers (j, j + 1) of both arrays are the same pair
              pr[j / 2] = h2u(__floats2half2_rn(__uint_as_float(x[j]) - h.x, __uint_as_float(x[j + 1]) - h.y));
            }
            tmem_st_pairs(s_at + c + 32, pr);
          }
        }
        l[0] += sum[0];
        l[1] += sum[1];
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pfull[buf]);
      }
      if (!ok) break;
      // The segment's O: all of the item, or this CTA's part of it.  (Two barriers for the tiles' ends, as that of tile
      // i - 1 may or may not have been waited for: the one two tiles before it is over for sure when S of
      // tile i is there, so a parity never stands for an older phase.)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
      }
      ok = wait(&sh.pvdone[(i - 1) & 1], (i - 1) >> 1);
      if (!ok) break;
      tc_fence_after();
      size_t at[2];
      bool there[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = sg.rt * C::R + quadrant * 32 + hf * 16 + (lane >> 2) + 8 * k;
        there[k] = row < total;
        at[k] = static_cast<size_t>(sg.row0 + row / p.group) * p.q_heads + sg.h * p.group + row % p.group;
      }
      const bool whole = sg.t0 == 0 && sg.t1 == sg.tiles;
      float* part = p.part + static_cast<size_t>(blockIdx.x * 2 + (sg.t0 == 0 ? 1 : 0)) * ((D + 2) * C::R);
      uint16_t* out = static_cast<uint16_t*>(p.out);
      float inv[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) inv[k] = l[k] > 0.0f ? 1.0f / l[k] : (l[k] == 0.0f ? 0.0f : l[k]);
#pragma unroll 1
      for (int c = 0; c < D; c += 64) {
        uint32_t o[32];
        tmem_ld_rows(lanes + C::O_COL + c, o);
        tc_wait_ld();
        if (sg.t1 - sg.t0 > C::FOLD) {
          const float* sum_at = p.part + static_cast<size_t>(gridDim.x * 2 + blockIdx.x) * ((D + 2) * C::R);
          const float* ref_at = sum_at + D * C::R + quadrant * 32 + hf * 16 + (lane >> 2);
          const float was[2] = {ex2(ref_at[0] - m[0]), ex2(ref_at[8] - m[1])};
#pragma unroll
          for (int j = 0; j < 32; ++j)
            o[j] = __float_as_uint(fmaf(sum_at[(c / 2 + j) * C::RT + tid], was[(j >> 1) & 1], __uint_as_float(o[j])));
        }
        if (whole) {
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const int k = (j >> 1) & 1;
            write_word(out + at[k] * D, (c >> 3) + (j >> 2), __uint_as_float(o[j]) * inv[k], __uint_as_float(o[j + 1]) * inv[k], p.bf16,
                       there[k], lane);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) part[(c / 2 + j) * C::RT + tid] = __uint_as_float(o[j]);
        }
      }
      tc_fence_before();
      if ((lane & 3) == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = quadrant * 32 + hf * 16 + (lane >> 2) + 8 * k;
          if (!whole) {
            part[D * C::R + r] = m[k];
            part[(D + 1) * C::R + r] = l[k];
          } else if (there[k] && p.lse != nullptr) {
            p.lse[at[k]] = l[k] == 0.0f ? -INFINITY : (m[k] + log2f(l[k])) * 0.6931471805599453f;
          }
        }
      }
      __syncwarp();
    }
  } else if (warp < kCopyWarp) {
    // ------------------------------------------------------------ packed tiles to operands
    const int d = tid - C::RT;                                  // 0 .. XT - 1
    const uint32_t tiles = static_cast<uint32_t>(c1 - c0);
    bool ok = true;
    // K of tile i, then V of tile i - 1
    for (uint32_t i = 0; i <= tiles && tiles > 0; ++i) {
      if (i < tiles) {
        const int st = i % C::KST;
        ok = wait(&sh.cfull[0][i & 1], i >> 1) && (i < C::KST || wait(&sh.kempty[st], i / C::KST - 1));
        if (!ok) break;
        const uint8_t* tb = sh.staging[0][i & 1];
        // K: 16 bytes of codes at a time; rows r and r + 4 in neighbouring quarter warps fill all banks
#pragma unroll
        for (int k = 0; k < BT * (D / 32) / C::XT; ++k) {
          constexpr int UR = D / 32;                            // units of a row
          const int u = k * C::XT + d, q = u / UR, c = u % UR;
          const int row = UR == 4 ? (q & ~7) | ((q & 1) << 2) | ((q >> 1) & 3) : q;
          const uint8_t* ch = tb + (row >> 4) * (10 * D);
          const uint4 cw = *reinterpret_cast<const uint4*>(ch + (row & 15) * (D / 2) + c * 16);
          const uint32_t w4[4] = {cw.x, cw.y, cw.z, cw.w};
          const uint32_t* prs = reinterpret_cast<const uint32_t*>(ch + 8 * D + (row & 15) * (D / 8));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int place = 4 * c + e, gr = place % C::GR, w = 4 * gr + place / C::GR;
            const __half2 s2 = __low2half2(u2h(prs[gr]));
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int n4 = 0; n4 < 4; ++n4) {
              // (c - 8) / 2, exact: 512 + c / 2 in place 0, 32 + c / 2 in place 1
              const uint32_t x = n4 & 2 ? w4[e] >> 8 : w4[e];
              const __half2 c2 = n4 & 1 ? __hadd2(u2h(and_or(x, 0x00f000f0u, 0x50005000u)), u2h(0xd080d080u))     // - 36
                                        : __hadd2(u2h(and_or(x, 0x000f000fu, 0x60006000u)), u2h(0xe008e008u));    // - 516
              const __half2 h = __hmul2(c2, s2);
              hi[n4] = h2u(h);
              lo[n4] = h2u(__hfma2(c2, s2, __hneg2(h)));
            }
            sts16(sh.khi[st][w >> 3] + swz(row, w & 7), hi[0], hi[1], hi[2], hi[3]);
            sts16(sh.klo[st][w >> 3] + swz(row, w & 7), lo[0], lo[1], lo[2], lo[3]);
          }
        }
        if (d < BT) {                                           // the b of a token's groups, twice
          const uint32_t* prs = reinterpret_cast<const uint32_t*>(tb + (d >> 4) * (10 * D) + 8 * D + (d & 15) * (D / 8));
          uint32_t b[4];
          if constexpr (D == 64) {
            b[0] = __byte_perm(prs[0], prs[1], 0x7632);
            b[1] = b[0];
            b[2] = b[3] = 0;
          } else if constexpr (D == 128) {
            b[0] = b[2] = __byte_perm(prs[0], prs[1], 0x7632);
            b[1] = b[3] = __byte_perm(prs[2], prs[3], 0x7632);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = __byte_perm(prs[2 * e], prs[2 * e + 1], 0x7632);
            sts16(sh.kx[st] + BT * 16 + d * 16, b[0], b[1], b[2], b[3]);
          }
          sts16(sh.kx[st] + d * 16, b[0], b[1], b[2], b[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.kfull[st]);
        if (lane == 0) mbar_arrive(&sh.cempty[0][i & 1]);
      }
      if (i > 0) {
        const uint32_t j = i - 1;
        const int vs = j % C::VST;
        ok = wait(&sh.cfull[1][j & 1], j >> 1) && (j < C::VST || wait(&sh.vempty[vs], j / C::VST - 1));
        if (!ok) break;
        const uint8_t* tb = sh.staging[1][j & 1];
        const int good = sh.good[j & 7], from = sh.from[j & 7], live = sh.live[j & 7];
        // V: rows of tokens as they are; tokens behind the item's context, and in its first chunk before the window, become
        // zeros: they may hold anything
#pragma unroll
        for (int k = 0; k < BT * (D / 32) / C::XT; ++k) {
          constexpr int UR = D / 32;
          const int u = k * C::XT + d, q = u / UR, c = u % UR;
          const int pr = UR == 4 ? (q & ~15) | ((q & 1) << 3) | ((q >> 1) & 7) : q;   // rows p and p + 8: tokens 2 p, 2 p + 1
          const int row = (pr & ~15) | ((pr & 7) * 2 + ((pr >> 3) & 1));              // the token
          const uint8_t* ch = tb + (pr >> 4) * (10 * D);
          const uint4 cw = *reinterpret_cast<const uint4*>(ch + (pr & 15) * (D / 2) + c * 16);
          const uint32_t w4[4] = {cw.x, cw.y, cw.z, cw.w};
          const uint32_t* prs = reinterpret_cast<const uint32_t*>(ch + 8 * D + (pr & 15) * (D / 8));
          const bool there = row >= from && row < live && ((good >> (row >> 4)) & 1);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int place = 4 * c + e, w = place / C::H + 8 * (place % C::H);       // C::H = D / 64
            const int gr = w >> 2, pp = (gr & 1) * C::H + (gr >> 1);
            const uint32_t sb = there ? prs[pp] : 0;
            const __half2 s2 = __low2half2(u2h(sb)), b2 = __high2half2(u2h(sb));
            uint32_t x4[4];
#pragma unroll
            for (int n4 = 0; n4 < 4; ++n4) {
              const uint32_t x = n4 & 2 ? w4[e] >> 8 : w4[e];
              const __half2 c2 = n4 & 1 ? __hadd2(u2h(and_or(x, 0x00f000f0u, 0x54005400u)), u2h(0xd480d480u))     // - 72
                                        : __hadd2(u2h(and_or(x, 0x000f000fu, 0x64006400u)), u2h(0xe408e408u));    // - 1032
              x4[n4] = h2u(__hfma2(c2, s2, b2));
            }
            sts16(sh.v[vs][w >> 3] + swz(row, w & 7), x4[0], x4[1], x4[2], x4[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.vfull[vs]);
          mbar_arrive(&sh.cempty[1][j & 1]);
        }
      }
    }
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------ packed tiles, ahead of their use
    uint32_t i = 0, asked[2] = {0, 0};                          // tiles, and those whose keys and values were asked for
    bool ok = true;
    const bool skip_first = p.inject_unreachable && blockIdx.x == 0;   // timeout test: the first keys are left out
    int entry = 0;                                              // lane m: the table's entry of the next tile's chunk m
    Segment sg{};
    if (works) sg = list.at(c0, c1, lane);
    if (lane == 0) sh.ends[0] = sg;
    for (long long tile = c0; tile < c1 && ok; list.next(sg, c1, lane)) {
      tile = sg.id + sg.t1;
      if (lane == 0) sh.ends[1] = sg;
      auto look = [&](int t) {
        const int pos = sg.first + t * BT + lane * kChunkTokens;
        entry = lane < C::CHUNKS && pos < sg.end
                    ? p.st.table[static_cast<size_t>(sg.seq) * p.st.stride + (pos >> p.st.page_shift)] : -1;
      };
      look(sg.t0);
      for (int t = sg.t0; t < sg.t1 && ok; ++t, ++i) {
        const int pos0 = sg.first + t * BT, pos = pos0 + lane * kChunkTokens;
        const bool wanted = lane < C::CHUNKS && pos < sg.end;
        const uint8_t* src = wanted ? chunk_at(p.st, entry, pos, sg.h, D) : nullptr;
        if (t + 1 < sg.t1) look(t + 1);
        if (wanted && src == nullptr) atomicOr(p.st.err, kErrRange);
        const unsigned there = __ballot_sync(0xffffffffu, src != nullptr);
        if (lane == 0) {
          sh.good[i & 7] = static_cast<int>(there);
          sh.from[i & 7] = max(sg.start + sg.rt * C::R / p.group - p.window + 1, 0) - pos0;
          sh.live[i & 7] = sg.end - pos0;
        }
#pragma unroll
        for (int kv = 0; kv < 2 && ok; ++kv) {
          if (i >= 2) ok = wait(&sh.cempty[kv][i & 1], (i >> 1) - 1);
          if (!ok) break;
          ++asked[kv];
          if (skip_first && i == 0 && kv == 0) continue;
          if (lane == 0) mbar_arrive_expect_tx(&sh.cfull[kv][i & 1], __popc(there) * 10 * D);
          __syncwarp();
          if (src != nullptr)
            bulk_g2s(sh.staging[kv][i & 1] + lane * 10 * D, src + kv * 10 * D, 10 * D, &sh.cfull[kv][i & 1]);
          __syncwarp();
        }
      }
    }
    // What either slot was asked for last may still be on its way if another role gave up: no copy may land in shared memory
    // that the CTA has left.
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      for (uint32_t back = 1; back <= 2 && back <= asked[kv]; ++back) {
        const uint32_t x = asked[kv] - back;
        if (skip_first && x == 0 && kv == 0) continue;
        mbar_wait(&sh.cfull[kv][x & 1], (x >> 1) & 1, globaltimer_ns() + 100000000ull, nullptr);
      }
  } else {
    // ------------------------------------------------------------ products
    constexpr uint32_t kIdS = make_idesc(1u, 0u, 0u, 128u, BT);
    constexpr uint32_t kIdO = make_idesc(1u, 0u, 0u, 128u, D) | 1u << 16;   // B with N contiguous
    uint32_t i = 0, segs = 0;
    bool ok = true;
    auto add_values = [&](uint32_t j, bool begin) {             // O += P V of tile j (O = P V: O was read, or is none)
      const int st = j % C::VST, buf = j & 1;
      ok = wait(&sh.vfull[st], j / C::VST) && wait(&sh.pfull[buf], j >> 1);
      if (!ok) return;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t a = tmem + buf * BT, o = tmem + C::O_COL, vb = desc_lo(smem_u32(sh.v[st][0]), BT * 128);
#pragma unroll
        for (int k = 0; k < BT / 16; ++k)
          mma_ts<kSw128>(o, a + (k >> 2) * 64 + (k & 3) * 8, vb + k * (2048 >> 4), kIdO, begin && k == 0 ? 0u : 1u);
        if (!p.bf16) {
#pragma unroll
          for (int k = 0; k < BT / 16; ++k) mma_ts<kSw128>(o, a + (k >> 2) * 64 + 32 + (k & 3) * 8, vb + k * (2048 >> 4), kIdO, 1u);
        }
        tc_commit(&sh.pvdone[buf]);
        tc_commit(&sh.vempty[st]);
      }
      __syncwarp();
    };
    Segment sg{};
    if (works) sg = list.at(c0, c1, lane);
    for (long long tile = c0; tile < c1 && ok; ++segs, list.next(sg, c1, lane)) {
      tile = sg.id + sg.t1;
      ok = wait(&sh.qfull, segs);
#pragma unroll 1
      for (int t = sg.t0; t < sg.t1 && ok; ++t, ++i) {
        const int st = i % C::KST, buf = i & 1;
        ok = wait(&sh.kfull[st], i / C::KST);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t hb = desc_lo(smem_u32(sh.khi[st][0]), 16), lb = desc_lo(smem_u32(sh.klo[st][0]), 16);
          const uint32_t s = tmem + buf * BT, q = tmem + C::Q_COL;
          // smallest parts first: b sum q, then the remainders, then the rest
          mma_ss<kPlain>(s, desc_lo(smem_u32(sh.qx), 128 * 16), desc_lo(smem_u32(sh.kx[st]), BT * 16), kIdS, 0u);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) mma_ts<kSw128>(s, q + k * 8, lb + (((k >> 2) * BT * 128 + (k & 3) * 32) >> 4), kIdS, 1u);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) mma_ts<kSw128>(s, q + k * 8, hb + (((k >> 2) * BT * 128 + (k & 3) * 32) >> 4), kIdS, 1u);
          tc_commit(&sh.sfull[buf]);
          tc_commit(&sh.kempty[st]);
        }
        __syncwarp();
        if (t > sg.t0) add_values(i - 1, ((t - 1 - sg.t0) & (C::FOLD - 1)) == 0);
      }
      if (ok) add_values(i - 1, ((sg.t1 - 1 - sg.t0) & (C::FOLD - 1)) == 0);
    }
    if (lane == 0) tc_commit(&sh.drained);
    __syncwarp();
    mbar_wait(&sh.drained, 0, globaltimer_ns() + p.timeout_ns, nullptr);   // no product in flight below
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, C::TMEM);
  if (!works || sh.abort) return;

  // Count this CTA's parts (of the item that began before it, of the one that goes on behind it); the CTA that counts
  // an item's last one adds them up in their order.
  auto cta_of = [&](long long x) { return static_cast<int>(((x + 1) * n - 1) / T); };
  if (tid < 2) {
    sh.last[tid] = 0;
    const Segment sg = sh.ends[tid];
    // tid 0: the item at the range's begin, if it began before; tid 1: the one at its end, if it began here and goes on
    const bool mine = tid == 0 ? sg.id < c0 : sg.id >= c0 && sg.id + sg.tiles > c1;
    if (mine) {
      const int f0 = cta_of(sg.id), f1 = cta_of(sg.id + sg.tiles - 1);
      if (atom_add_acq_rel_gpu(p.cnt + f0, 1u) == static_cast<uint32_t>(f1 - f0)) {
        sh.last[tid] = 1;
        p.cnt[f0] = 0;
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int it = 0; it < 2; ++it) {
    if (!sh.last[it]) continue;
    const Segment sg = sh.ends[it];
    const int f0 = cta_of(sg.id), parts = cta_of(sg.id + sg.tiles - 1) - f0 + 1;
    if (tid >= 512) continue;
    // As the rows' warps hold them, two threads a place: `half` of its columns each.  Loads of two parts are in flight
    // together, with the weights they need.
    const int place = tid & 255, half = tid >> 8;
    const float* base = p.part + static_cast<size_t>(f0) * 2 * ((D + 2) * C::R);
    auto part_of = [&](int x) { return base + static_cast<size_t>(2 * x + (x == 0 ? 1 : 0)) * ((D + 2) * C::R); };
    const int r0 = ((place >> 5) & 3) * 32 + (place >> 7) * 16 + (lane >> 2);
    float m[2] = {kNothing, kNothing}, l[2] = {0.0f, 0.0f}, inv[2];
#pragma unroll 1
    for (int x = 0; x < parts; x += 2) {
      float pm[2][2], pl[2][2];
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool in = x + y < parts;
          pm[y][k] = in ? part_of(x + y)[D * C::R + r0 + 8 * k] : kNothing;
          pl[y][k] = in ? part_of(x + y)[(D + 1) * C::R + r0 + 8 * k] : 0.0f;
        }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float mn = fmaxf(m[k], fmaxf(pm[0][k], pm[1][k]));
        l[k] = l[k] * ex2(m[k] - mn) + ex2(pm[0][k] - mn) * pl[0][k] + ex2(pm[1][k] - mn) * pl[1][k];
        m[k] = mn;
      }
    }
    size_t at[2];
    bool there[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = sg.rt * C::R + r0 + 8 * k;
      there[k] = row < sg.rows * p.group;
      at[k] = static_cast<size_t>(sg.row0 + row / p.group) * p.q_heads + sg.h * p.group + row % p.group;
      inv[k] = l[k] > 0.0f ? 1.0f / l[k] : (l[k] == 0.0f ? 0.0f : l[k]);
    }
#pragma unroll 1
    for (int c = half * (D / 4); c < (half + 1) * (D / 4); c += 16) {   // of the place's D / 2 numbers
      float o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = 0.0f;
#pragma unroll 1
      for (int x = 0; x < parts; x += 2) {
        const float *fa = part_of(x), *fb = part_of(x + 1 < parts ? x + 1 : x);
        float va[16], vb[16], wa[2], wb[2];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          va[j] = fa[(c + j) * C::RT + place];
          vb[j] = fb[(c + j) * C::RT + place];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          wa[k] = ex2(fa[D * C::R + r0 + 8 * k] - m[k]);
          wb[k] = x + 1 < parts ? ex2(fb[D * C::R + r0 + 8 * k] - m[k]) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = fmaf(wb[(j >> 1) & 1], vb[j], fmaf(wa[(j >> 1) & 1], va[j], o[j]));
      }
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const int k = (j >> 1) & 1;
        write_word(static_cast<uint16_t*>(p.out) + at[k] * D, (c + j) >> 2, o[j] * inv[k], o[j + 1] * inv[k], p.bf16, there[k], lane);
      }
    }
    if (p.lse != nullptr && (lane & 3) == 0 && half == 0)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (there[k]) p.lse[at[k]] = l[k] == 0.0f ? -INFINITY : (m[k] + log2f(l[k])) * 0.6931471805599453f;
  }
}

template <int D>
cudaError_t launch_as(const CacheAttnParams& p, cudaStream_t stream) {
  constexpr int kMost = static_cast<int>(sizeof(PShared<D>) + 1024 + (kCacheMaxSeqs + 1) * 8);
  static_assert(sizeof(PShared<D>) + 1024 + 8 <= 227 * 1024, "shared memory");
  constexpr int kCap = kMost < 227 * 1024 ? kMost : 227 * 1024;
  static std::atomic<unsigned long long> set{0};   // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (bit == 0 || !(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(cache_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCap);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_chained(cache_prefill_kernel<D>, dim3(p.grid), PCfg<D>::THREADS, cache_prefill_smem(D, p.st.n_seqs), stream, p);
}

}  // namespace

size_t cache_prefill_smem(int dim, int n_seqs) {
  const size_t fixed = dim == 64 ? sizeof(PShared<64>) : dim == 128 ? sizeof(PShared<128>) : sizeof(PShared<256>);
  return fixed + 1024 + (static_cast<size_t>(n_seqs) + 1) * 8;
}
size_t cache_prefill_part_floats(int dim) { return static_cast<size_t>(dim + 2) * PCfg<128>::R; }
cudaError_t launch_cache_prefill(const CacheAttnParams& p, int dim, cudaStream_t stream) {
  return dim == 64 ? launch_as<64>(p, stream) : dim == 128 ? launch_as<128>(p, stream) : launch_as<256>(p, stream);
}

}  // namespace bs
