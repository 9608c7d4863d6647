// Attention of many queries on one cached prefix (the prefix pass of
// kvq_decode_attention_shared), on the tensor cores.
//
// All query heads of a group's sequences that read one kv head are rows of one matrix: with
// rotated queries q~ (rows) and the decoded rotated keys and values K, V of a chunk of the
// prefix,
//   S = q~ K^T,  P = 2^(S - m),  O = P V,  l = rowsum P
// with an m that follows the row's running maximum.  The cache is read and decoded once for up to 128 rows,
// instead of once for every sequence.
//
// A block takes one work item: (chunk of the prefix, kv head, 128 rows).  Roles:
//   8 softmax warps (two groups of 128 threads, a thread per row): S from TMEM, P back to TMEM
//   4 + 4 decoding warps: K and V tiles of 128 tokens; rows travel by asynchronous copies into slots of
//     the decoding thread, and are decoded to fp16 into shared memory (128-byte swizzle)
//   1 warp: issues the products and allocates TMEM
//   2 warps: look up page numbers, rows, norms and scales, up to four tiles ahead.
// All products are tcgen05.mma of 128 x 128 x 16 steps: S = q~ K^T from shared memory, O += P V
// with P read from TMEM (it overwrites S) and V as it lies (tokens x coordinates, the
// MN-major form).  The two softmax groups hold the same rows and take alternate tiles, so that one's
// products run while the other works on its scores; that leaves two partial results.  TMEM: two S
// and two O of 128 columns, all 512.
//
// m lies 2 (a factor of 4) below the largest score of the half tile that last raised it, so that
// fp16 rounds a weight by at most 2^-27 of the largest: a tail of 2^17 such tokens is off by
// 2^-10 of it at most.  An accumulator is rescaled only when half a tile's weights sum to more than
// 2^15 in some row of a warp, which after the first tile is rare: until then weights stay inside
// fp16.
//
// Scores, maxima, sums and accumulators are float32.  What the tensor cores multiply is fp16, and each
// rounding to it (2^-11 of a number at most, 2e-4 in the mean) is weighed against the output's own
// (2.1e-4 of it, 2-norm):
//   queries   two fp16 numbers, the nearest one and the rest (2^-22): one alone would add 2.5e-4 on
//             fp16 keys and up to 6.5e-4 on codes with x30 outlier channels
//   weights   one fp16 number (of codebooks the weight times the value's norm), 1e-4 over a long context;
//             where a few tokens have most of the weight the sum is taken of the rounded numbers (not of
//             codebooks, where that costs a tenth of the time and gains nothing measurable)
//   values    INT4 levels times their scale one number (1.9e-4); of codebooks the centroid alone (norms in
//             the values, rounded once more, would be 2.9e-4)
//   centroids one number, scaled so that their roundings matter least (scale_table, 1.3e-4); a key's norm
//             multiplies its scores in float32.
// Together 2.3e-4 to 3.3e-4 of the output on caches with outlier channels.  (With queries, and values times
// norms, as single numbers, it was 5e-4 to 9e-4, with twice the rows in a block and 150 instead of
// 202 us for the largest case below; the others took 0 to 10% less.)
//
// Every wait has a limit: a block whose wait runs out sets KVQ_DEVERR_COPY_TIMEOUT and ends.
#pragma once
#include <type_traits>

#include "chunk.cuh"
#include "shared.cuh"
#include "table_scale.cuh"
#include "tc.cuh"

namespace kvq {
namespace {

constexpr int kDim = 128;
constexpr int kThreads = 640;
// registers per thread after the split: launched with 96 x 640 = 61440 = 256 x 128 + 256 x 80 + 128 x 64
constexpr int kSoftmaxRegs = 128, kDecodeRegs = 80, kIssueRegs = 64;
constexpr int kTileBytes = kTileTokens * kDim * 2;  // 32 KB: two halves of 128 rows x 128 bytes
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kStages = 2;
// Beside the operand tiles: codebook tables, then of kAhead tiles the rows and per side the
// norms or scales.
constexpr int kOffQ = 0, kOffK = 2 * kTileBytes, kOffV = kOffK + kStages * kTileBytes;
constexpr int kOffLut = kOffV + kStages * kTileBytes, kLutBytes = 24 << 10;
constexpr int kAhead = 4;
constexpr int kOffRow = kOffLut + kLutBytes, kRowBytes = kTileTokens * 4;                       // a tile
// (keys: a float32 norm a token; values: the same, or four fp16 scales, in 8 bytes)
constexpr int kOffKAux = kOffRow + kAhead * kRowBytes, kOffVAux = kOffKAux + kAhead * kTileTokens * 4;
constexpr int kOffCtl = kOffVAux + kAhead * kTileTokens * 8;
constexpr int kSmem = kOffCtl + 512 + 1024;  // 1024: the base is aligned by hand
static_assert(kSmem <= 227 * 1024, "shared memory of a block");

// barriers, in units of 8 bytes from kOffCtl
enum { B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_QFULL = 8, B_SFULL = 10, B_PREADY = 12, B_OFULL = 14, B_QROT = 16, B_ROWS = 18, B_ROWS_READ = 22, B_AUX = 26, B_COUNT = 30 };

struct Ctl {
  unsigned long long bars[B_COUNT];
  uint32_t tmem;
  int abort;
  int bad_page;        // a token of the item lies in a page outside the pool
  float best[2][4];    // per side and warp: a table scale's error, and
  int best_at[2][4];   // which it is
  float best_slope[2][4];  // and the slope of its roundings
  float unscale[2];    // what a side's table values are to be multiplied by
  float norm_unit;     // what the values' norms are divided by: a power of two
  float norm_top[kAhead];  // of a tile, above all of its values' norms (so divided): a power of two
  uint32_t not_finite[kAhead][4];  // a chunk's items: tokens of a tile whose values were not finite and are zero
};
static_assert(sizeof(Ctl) <= 512, "control block");

// f16 inputs, f32 accumulator, 128 x 128; bit 16: B is MN-major
constexpr uint32_t kIdescQK = (1u << 4) | ((kTileTokens >> 3) << 17) | ((kTileRows >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((kDim >> 3) << 17) | ((kTileRows >> 4) << 24);

// ------------------------------------------------------------------------ decoding a tile
// Formats as the decoding warps see them.
enum { D_F16, D_F8, D_I4, D_CB4, D_CB3, D_CB2 };

// A thread's piece of a row ("unit"), the passes of 128 threads that cover a tile, and how many
// passes' units are on their way at a time.
__host__ __device__ constexpr int unit_bytes(int f) { return f == D_CB3 ? 12 : (f == D_CB2 ? 8 : 16); }
__host__ __device__ constexpr int unit_passes(int f) { return f == D_F16 ? 16 : (f == D_F8 ? 8 : 4); }

// What one side (K or V) of an item reads, and where its pieces of shared memory lie.
struct Source {
  const uint8_t* rows;
  int row_bytes;
  uint32_t raw;               // shared addresses: the threads' slots;
  uint32_t rowbuf, auxbuf;    // kAhead tiles of rows; of the values' scales
  uint32_t lut, lut_stride;   // the lane's copy of entry 0, bytes between entries (codebooks)
};
// What the look-ups read.
struct Pages {
  const int32_t* table;  // the group's block-table row
  int num_pages, page_size, page_shift, hkv, hk;
  int end;               // tokens of the prefix
  int hide, hidden;      // a chunk's items (MASKED): no row sees tokens hide .. hide + hidden - 1
};
struct Ring {
  uint32_t tiles, full, empty;  // shared addresses
  uint32_t rows, aux, rows_read;  // the look-ups' barriers
  uint32_t first_use;             // what the second stage waits for before its first tile, or 0
};

// Half a tile's weights may sum to this before m is raised (the largest fp16 is 2^16), and m is then
// this far below the largest score (64 weights of 2^2 are 2^8).
constexpr float kMostWeight = 32768.0f, kHeadroom = 2.0f;

// A token that is not there reads as zero.  Past the end of the prefix its score is -inf, where no row of a chunk sees
// it its weights are hidden; in a page outside the pool it has a score like any other, and the whole item is left out
// (Ctl::bad_page).
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

// Whether token t is looked up.  Of a chunk's tiles only what some row sees: the block table's other entries may be
// of pages that the sequence has given back.
template <bool MASKED>
__device__ __forceinline__ bool there(const Pages& s, int t) {
  return t < s.end && (!MASKED || (unsigned)(t - s.hide) >= (unsigned)s.hidden);
}
// Page of token t (-1 where it is not there).
template <bool MASKED>
__device__ __forceinline__ int page_of(const Pages& s, int t) {
  if (!there<MASKED>(s, t)) return -1;
  return __ldg(s.table + (s.page_shift >= 0 ? t >> s.page_shift : t / s.page_size));
}
// Its row in the pool: kNoRow where it is not there, and for a page outside the pool (reported in bits).
template <bool MASKED>
__device__ __forceinline__ uint32_t row_of(const Pages& s, int t, int page, int* bits) {
  if (!there<MASKED>(s, t) || !page_in_pool(page, s.num_pages, bits)) return kNoRow;
  const uint32_t off = s.page_shift >= 0 ? t & (s.page_size - 1) : t % s.page_size;
  return ((uint32_t)page * s.hkv + s.hk) * s.page_size + off;  // below 2^32: the plan checks
}
// Token (row of the tile) and unit of a thread in pass p.  A quarter-warp holds eight tokens
// and one unit, so that its 16-byte stores meet eight different banks of the swizzled tile; a
// warp reads 64 neighbouring bytes of each row.
template <int F>
__device__ __forceinline__ void place(int p, int tid, int& t, int& u) {
  if constexpr (F == D_F16) {
    t = p * 8 + (tid >> 4);
    u = tid & 15;
  } else if constexpr (F == D_F8) {
    t = (p >> 1) * 32 + (tid >> 5) * 8 + (tid & 7);
    u = (p & 1) * 4 + ((tid >> 3) & 3);
  } else {
    t = p * 32 + (tid >> 5) * 8 + (tid & 7);
    u = (tid >> 3) & 3;
  }
}

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src, bool there) {
  const int n = there ? N : 0;  // no bytes read, N zeros written
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Look-up warp `first` of kLookUps, which take tiles in turn (a look-up is a chain of three
// loads, longer than a tile's products): rows of a tile's tokens, then their norms (codebooks) or
// group scales (INT4 values).  Page numbers are read a turn ahead.  kLookUps divides kAhead, so
// that a stage belongs to one warp, which waits for every one of its releases: the softmax groups
// release stages out of order, and a warp that waited only for some of them could take one
// phase of the barrier for the one before the last.
constexpr int kLookUps = 2;
static_assert(kAhead % kLookUps == 0, "a stage's releases are waited for by one warp");
template <bool MASKED, class TileOf>
__device__ __forceinline__ void first_pages(const Pages& s, const TileOf& tile_of, int n, int first, int (&page)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    page[j] = first < n ? page_of<MASKED>(s, tile_of(first) * kTileTokens + (threadIdx.x & 31) + 32 * j) : -1;
}
// The power of two above the finite norms of a tile's values, from the largest of each lane's four as
// fp16 bits (2^-13 where all are zero).  Norms are divided by that of the item's first tile, so that a weight
// times a norm is an fp16 number like a weight.
__device__ __forceinline__ float power_above(uint32_t most) {
  return __uint_as_float(((__reduce_max_sync(0xFFFFFFFFu, max(most, 0x0400u)) >> 10) + 113u) << 23);
}
__device__ __forceinline__ uint32_t finite_bits(uint32_t norm) {
  norm &= 0x7FFFu;
  return norm < 0x7C00u ? norm : 0u;
}

// The exponent of the power of two above a value's norm: at least -40 (an fp16 number over another's power), so that
// the weight of a token whose norm is zero stays finite, and at most 20, for a norm that is not.
__device__ __forceinline__ float power_of(float norm) {
  return (float)(min(max((int)(__float_as_uint(norm) >> 23 & 255u) - 126, -40), 20));
}

// MASKED (a chunk's items): where some row sees not all of a tile (`edge`), an INT4 scale that is not finite becomes
// zero and its token is noted: a weight of zero must meet no NaN.
template <bool MASKED, class TileOf, class Edge>
__device__ __forceinline__ void look_up(const Pages& s, int (&page)[4], const __half* k_norm, const __half* v_norm,
                                        const __half* v_scale, Ctl* ctl, uint32_t smem, uint32_t bars, const TileOf& tile_of,
                                        const Edge& edge, int n, int first, volatile int* abort, int* err) {
  const int lane = threadIdx.x & 31;
  int bits = 0;
  const float key_unit = k_norm ? *reinterpret_cast<volatile float*>(&ctl->unscale[0]) : 0.f;  // of the keys' table
  float value_unit = 0.f;  // 1 / the norms' power, once it is known
#pragma unroll 1
  for (int i = first; i < n; i += kLookUps) {
    const int at = i % kAhead;
    if (i >= kAhead && !bar_wait(bars + 8 * (B_ROWS_READ + at), ((i / kAhead) & 1) ^ 1, abort, err)) break;
    const int t0 = tile_of(i) * kTileTokens + lane;
    uint32_t row[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      row[j] = row_of<MASKED>(s, t0 + 32 * j, page[j], &bits);
      sts32(smem + kOffRow + at * kRowBytes + 4 * (lane + 32 * j), row[j]);
    }
    if (bits & KVQ_DEVERR_PAGE_INDEX) *reinterpret_cast<volatile int*>(&ctl->bad_page) = 1;
    if constexpr (MASKED) {
      if (lane < 4) *reinterpret_cast<volatile uint32_t*>(&ctl->not_finite[at][lane]) = 0u;
    }
    bar_arrive(bars + 8 * (B_ROWS + at));
    uint2 aux[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      aux[j] = make_uint2(0u, 0u);
      if (row[j] != kNoRow && k_norm) {
        aux[j].x = __half_as_ushort(__ldg(k_norm + row[j]));
        aux[j].y = __half_as_ushort(__ldg(v_norm + row[j]));
      } else if (row[j] != kNoRow && v_scale) {
        aux[j] = __ldg(reinterpret_cast<const uint2*>(v_scale) + row[j]);
        // a finite scale above 9352: seven times it is no fp16 number
        const uint32_t w[4] = {aux[j].x, aux[j].x >> 16, aux[j].y, aux[j].y >> 16};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if ((w[k] & 0x7FFFu) - 0x7092u < 0x7C00u - 0x7092u) bits |= KVQ_DEVERR_VALUE_RANGE;
      }
    }
    if constexpr (MASKED) {
      if (v_scale && edge(i)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w[2] = {aux[j].x, aux[j].y};
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 2; ++k) bad = bad || (w[k] & 0x7C00u) == 0x7C00u || (w[k] & 0x7C000000u) == 0x7C000000u;
          const uint32_t which = __ballot_sync(0xFFFFFFFFu, bad);
          if (bad) aux[j] = make_uint2(0u, 0u);
          if (which && lane == 0) *reinterpret_cast<volatile uint32_t*>(&ctl->not_finite[at][j]) = which;
        }
      }
    }
    if (i + kLookUps < n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) page[j] = page_of<MASKED>(s, tile_of(i + kLookUps) * kTileTokens + lane + 32 * j);
    }
    if (k_norm) {
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) most = max(most, finite_bits(aux[j].y));  // (0 where the token is not there)
      const float top = power_above(most);
      if (i == first) {
        float power = top;  // of the item's first tile, which another warp may look after
        if (first) {
          most = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            int ignored = 0;
            const int t = tile_of(0) * kTileTokens + lane + 32 * j;
            const uint32_t head = row_of<MASKED>(s, t, page_of<MASKED>(s, t), &ignored);
            if (head != kNoRow) most = max(most, finite_bits(__half_as_ushort(__ldg(v_norm + head))));
          }
          power = power_above(most);
        }
        value_unit = 1.0f / power;
        if (!first && lane == 0) *reinterpret_cast<volatile float*>(&ctl->norm_unit) = power;
      }
      if (lane == 0) *reinterpret_cast<volatile float*>(&ctl->norm_top[at]) = top * value_unit;
    }
    const uint32_t ka = smem + kOffKAux + at * kTileTokens * 4 + 4 * lane;
    const uint32_t va = smem + kOffVAux + at * kTileTokens * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (k_norm) {
        // (1 for a token that is not there: past the end its score, -inf, stays that, and its weight 0)
        const float kn = __half2float(__ushort_as_half((uint16_t)aux[j].x)) * key_unit;
        const float vn = __half2float(__ushort_as_half((uint16_t)aux[j].y)) * value_unit;
        sts32(ka + 128 * j, __float_as_uint(row[j] != kNoRow ? kn : 1.0f));
        sts32(va + 4 * lane + 128 * j, __float_as_uint(row[j] != kNoRow ? vn : 1.0f));
        if constexpr (MASKED) sts32(va + 4 * (kTileTokens + lane) + 128 * j, __float_as_uint(power_of(vn) - kHeadroom));
      } else if (v_scale) {
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(va + 8 * lane + 256 * j), "r"(aux[j].x), "r"(aux[j].y) : "memory");
      }
    }
    bar_arrive(bars + 8 * (B_AUX + at));
  }
  if (bits) atomicOr(err, bits);
}

// A unit of the row, on its way to the thread's slot.
template <int F>
__device__ __forceinline__ void request(const Source& s, uint32_t row, int u, uint32_t slot) {
  const bool there = row != kNoRow;
  const uint8_t* src = s.rows + (size_t)(there ? row : 0) * s.row_bytes + u * unit_bytes(F);
  if constexpr (unit_bytes(F) == 12) {
#pragma unroll
    for (int k = 0; k < 3; ++k) copy_async<4>(slot + 4 * k, src + 4 * k, there);
  } else {
    copy_async<unit_bytes(F)>(slot, src, there);
  }
}
template <int F>
__device__ __forceinline__ void take(uint32_t slot, uint32_t (&w)[4]) {
  if constexpr (unit_bytes(F) == 16) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(slot) : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < unit_bytes(F) / 4; ++k) w[k] = lds32(slot + 4 * k);
  }
}

// A table entry (not volatile: the table does not change, so look-ups may move).
__device__ __forceinline__ uint32_t look_pair(uint32_t addr) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// A unit decoded to fp16, into row t of the tile.
template <int F>
__device__ __forceinline__ void decode_unit(const Source& s, uint32_t tile, int t, int u, uint32_t half_scale,
                                            const uint32_t (&w)[4]) {
  const uint32_t row = tile + t * 128;
  const int x = t & 7;
  if constexpr (F == D_F8) {  // 16 values: two chunks
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[k]) : "h"((uint16_t)(w[k / 2] >> (16 * (k & 1)))));
    const uint32_t at = row + (u >> 2) * kHalfBytes;
    const int c = (2 * u) & 7;
    sts16(at + ((c ^ x) << 4), h[0], h[1], h[2], h[3]);
    sts16(at + (((c + 1) ^ x) << 4), h[4], h[5], h[6], h[7]);
  } else {  // 32 values: four chunks of 8
    constexpr int B = F == D_I4 || F == D_CB4 ? 4 : (F == D_CB3 ? 3 : 2);
    uint32_t c[4], h[16];
    if constexpr (B == 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = w[k];
    } else if constexpr (B == 3) {
      c[0] = w[0];
      c[1] = __funnelshift_r(w[0], w[1], 24);
      c[2] = __funnelshift_r(w[1], w[2], 16);
      c[3] = w[2] >> 8;
    } else {
      c[0] = w[0];
      c[1] = w[0] >> 16;
      c[2] = w[1];
      c[3] = w[1] >> 16;
    }
    if constexpr (F == D_I4) {
      // Levels n - 8 of nibbles (k, k + 4), exact in fp16: 1024 + n less 1032, or (from the
      // upper nibble of a byte) (1024 + 16 n) / 16 less 72; times the scale, rounded once.  The
      // pairs leave a chunk's coordinates in the order 0 4 1 5 2 6 3 7, and so the accumulator's
      // columns (undone where it is stored).
      const __half2 a = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));  // 1032
      const __half2 b = __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00));  // 1 / 16
      const __half2 d = __halves2half2(__ushort_as_half(0xD480), __ushort_as_half(0xD480));  // -72
      const uint32_t scale = half_scale * 0x10001u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v = i & 1 ? c[i / 2] >> 8 : c[i / 2];
        const uint32_t lo = (v & 0x000F000Fu) | 0x64006400u, hi = (v & 0x00F000F0u) | 0x64006400u;
        const __half2 nl = __hsub2(*reinterpret_cast<const __half2*>(&lo), a);
        const __half2 nh = __hfma2(*reinterpret_cast<const __half2*>(&hi), b, d);
        h[2 * i] = hmul2(*reinterpret_cast<const uint32_t*>(&nl), scale);
        h[2 * i + 1] = hmul2(*reinterpret_cast<const uint32_t*>(&nh), scale);
      }
    } else {
      // pairs of codes through the block's table of scaled centroid pairs
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t e = (c[i / 4] >> (2 * B * (i % 4))) & ((1u << (2 * B)) - 1u);
        h[i] = look_pair(s.lut + e * s.lut_stride);
      }
    }
    const uint32_t at = row + (u >> 1) * kHalfBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sts16(at + (((4 * (u & 1) + i) ^ x) << 4), h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
  }
}

// The side's four warps look for the scale of its table (table_candidates).
__device__ __forceinline__ float scale_table(Ctl* ctl, float c, int bits, int side, int tid) {
  const int lane = tid & 31, warp = tid >> 5;
  float least, slope;
  int at;
  table_candidates(c, bits, tid, least, slope, at);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(0xFFFFFFFFu, least, o), its = __shfl_xor_sync(0xFFFFFFFFu, slope, o);
    const int k = __shfl_xor_sync(0xFFFFFFFFu, at, o);
    if (other < least || (other == least && k < at)) {
      least = other;
      slope = its;
      at = k;
    }
  }
  if (lane == 0) {
    ctl->best[side][warp] = least;
    ctl->best_slope[side][warp] = slope;
    ctl->best_at[side][warp] = at;
  }
  if (side == 0) asm volatile("bar.sync 1, 128;" ::: "memory");
  else asm volatile("bar.sync 2, 128;" ::: "memory");
  for (int i = 0; i < 4; ++i) {
    const float other = ctl->best[side][i];
    const int k = ctl->best_at[side][i];
    if (other < least || (other == least && k < at)) {
      least = other;
      slope = ctl->best_slope[side][i];
      at = k;
    }
  }
  const float beta = exp2f((float)at * (1.0f / kTableSteps)) *
                     table_unit(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(c))));
  if (tid == 0) ctl->unscale[side] = inv_sqrt_dim(kDim) * (1.0f - slope) / beta;
  return beta;
}

// Pairs of scaled centroids in fp16: entry e = codes (e mod 2^b, e / 2^b), in copies, one per
// lane where there is room (a warp's look-ups then never meet in a bank), else 16 or 8 of them
// (two or three bank rounds a look-up).  tid: 128 threads; c as above, times the scale.
__device__ __forceinline__ void build_lut(uint32_t lut, int copies, float c, int bits, int tid) {
  for (int e = tid; e < max(128, 1 << (2 * bits)); e += 128) {  // (whole warps: the shuffles need them)
    const float lo = __shfl_sync(0xFFFFFFFFu, c, e & ((1 << bits) - 1)), hi = __shfl_sync(0xFFFFFFFFu, c, (e >> bits) & 31);
    if (e >= (1 << (2 * bits))) break;
    const uint32_t v = half2_bits(lo, hi);
    // (each lane begins at another copy: side by side they would meet in one bank)
    for (int i = 0; i < copies; i += 4) sts16(lut + 4u * (e * copies + ((i + 4 * e) & (copies - 1))), v, v, v, v);
  }
}

// Where the two tables lie, and the slots, in 24 KB: fp8 keys and INT4 values use them for slots
// alone (16 and 8 KB); codebooks have 16 KB of tables (16 copies of one where keys and values have
// the same, else 8 of each) and 4 KB of slots a side.
struct Tables {
  uint32_t at[2], raw[2];
  int copies[2];
};
__device__ __forceinline__ Tables place_tables(uint32_t smem, int k_bits, int v_bits, bool same) {
  const uint32_t lut = smem + kOffLut;
  Tables t;
  const int of_1kb = same ? 16 : 8;
  t.copies[0] = k_bits == 4 ? of_1kb : 32;  // (smaller tables: 8 KB at most)
  t.copies[1] = v_bits == 4 ? of_1kb : 32;
  t.at[0] = lut;
  t.at[1] = t.at[0] + (same ? 0 : 8 << 10);
  t.raw[0] = lut + (16 << 10);
  t.raw[1] = t.raw[0] + (4 << 10);
  return t;
}

// The side's n tiles, into the ring.  A thread's units travel by asynchronous copies into slots
// of its own (nobody else waits for them), `slots` passes ahead, a slot being requested anew as
// soon as it is taken.  The loop stays rolled, a pass of 32 values or two of 16 a turn: warps of
// several kinds share a scheduler's instruction cache, and with all passes unrolled (217 KB of
// text) they spent more time fetching instructions than running them.
template <int F, int SLOTS>
__device__ __forceinline__ void produce(const Source& s, const Ring& ring, int n, int tid, volatile int* abort,
                                        int* err) {
  constexpr int kPasses = unit_passes(F), kTurn = F == D_F8 ? 2 : 1;  // passes a turn
  constexpr uint32_t kSlotStep = 128 * unit_bytes(F);
  static_assert(SLOTS % kTurn == 0 && SLOTS <= kPasses && kPasses % SLOTS == 0, "slots");
  const uint32_t slot0 = s.raw + tid * unit_bytes(F);
  if (!bar_wait(ring.rows, 0, abort, err)) return;
#pragma unroll 1
  for (int p = 0; p < SLOTS; p += kTurn) {
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      int t, u;
      place<F>(p + j, tid, t, u);
      request<F>(s, lds32(s.rowbuf + 4u * t), u, slot0 + (p + j) * kSlotStep);
    }
    copy_commit();
  }
  for (int i = 0; i < n; ++i) {
    const int st = i & 1, at = i % kAhead, after = (i + 1) % kAhead;
    const bool more = i + 1 < n;
    if (more && !bar_wait(ring.rows + 8 * after, ((i + 1) / kAhead) & 1, abort, err)) break;
    if (F == D_I4 && !bar_wait(ring.aux + 8 * at, (i / kAhead) & 1, abort, err)) break;
    if (i >= kStages && !bar_wait(ring.empty + 8 * st, ((i >> 1) & 1) ^ 1, abort, err)) break;
    if (i == 1 && ring.first_use && !bar_wait(ring.first_use, 0, abort, err)) break;
    const uint32_t tile = ring.tiles + st * kTileBytes, aux = s.auxbuf + (uint32_t)(at * kTileTokens * 8);
    uint32_t slot = slot0;
#pragma unroll 1
    for (int p = 0; p < kPasses; p += kTurn) {
      const bool here = p + SLOTS < kPasses;  // the slots' next units are of this tile
      const int q = here ? p + SLOTS : p + SLOTS - kPasses;
      const uint32_t rows = s.rowbuf + (here ? at : after) * kRowBytes;
      copy_wait<SLOTS / kTurn - 1>();
      uint32_t w[kTurn][4], row[kTurn];
      uint32_t scale = 0;
#pragma unroll
      for (int j = 0; j < kTurn; ++j) {
        int t, u;
        take<F>(slot + j * kSlotStep, w[j]);
        place<F>(q + j, tid, t, u);
        row[j] = lds32(rows + 4u * t);
        if constexpr (F == D_I4) {
          uint16_t v;
          place<F>(p, tid, t, u);
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(aux + 8u * t + 2u * u));
          scale = v;
        }
      }
#pragma unroll
      for (int j = 0; j < kTurn; ++j) {
        int t, u;
        place<F>(p + j, tid, t, u);
        decode_unit<F>(s, tile, t, u, scale, w[j]);
        place<F>(q + j, tid, t, u);
        if (here || more) request<F>(s, row[j], u, slot + j * kSlotStep);
      }
      copy_commit();
      slot = p + kTurn == SLOTS || p + kTurn == 2 * SLOTS ? slot0 : slot + kTurn * kSlotStep;
    }
    fence_async_smem();
    bar_arrive(ring.full + 8 * st);
    bar_arrive(ring.rows_read + 8 * at);
  }
  copy_wait<0>();
}

// fp16 rows need no decoding: copies straight into the tile, a tile signalled once the next
// one's copies are under way.  Checked (values of a chunk's items): where `edge` says so, pieces that are not finite
// become zeros and their tokens are noted.
struct NoCheck {
  __device__ __forceinline__ void operator()(int, uint32_t) const {}
};
template <class Check>
__device__ __forceinline__ void produce_fp16(const Source& s, const Ring& ring, int n, int tid, volatile int* abort, int* err,
                                             const Check& check) {
  bool ok = true;
  for (int i = 0; i < n; ++i) {
    const int st = i & 1, at = i % kAhead;
    if (!(ok = bar_wait(ring.rows + 8 * at, (i / kAhead) & 1, abort, err))) break;
    if (i >= kStages && !(ok = bar_wait(ring.empty + 8 * st, ((i >> 1) & 1) ^ 1, abort, err))) break;
    if (i == 1 && ring.first_use && !(ok = bar_wait(ring.first_use, 0, abort, err))) break;
#pragma unroll 2
    for (int p = 0; p < unit_passes(D_F16); ++p) {
      int r, u;
      place<D_F16>(p, tid, r, u);
      const uint32_t row = lds32(s.rowbuf + at * kRowBytes + 4u * r);
      const bool there = row != kNoRow;
      copy_async<16>(ring.tiles + st * kTileBytes + (u >> 3) * kHalfBytes + r * 128 + (((u & 7) ^ (r & 7)) << 4),
                     s.rows + (size_t)(there ? row : 0) * s.row_bytes + u * 16, there);
    }
    copy_commit();
    bar_arrive(ring.rows_read + 8 * at);
    if (i > 0) {
      copy_wait<1>();
      check(i - 1, ring.tiles + (st ^ 1) * kTileBytes);
      fence_async_smem();
      bar_arrive(ring.full + 8 * (st ^ 1));
    }
  }
  copy_wait<0>();
  if (ok) {
    check(n - 1, ring.tiles + ((n - 1) & 1) * kTileBytes);
    fence_async_smem();
    bar_arrive(ring.full + 8 * ((n - 1) & 1));
  }
}

template <bool CODES, class Check>
__device__ __forceinline__ void produce_any(int f, const Source& s, const Ring& ring, int n, int tid, volatile int* abort,
                                            int* err, const Check& check) {
  if constexpr (!CODES) {
    if (f == D_F16) produce_fp16(s, ring, n, tid, abort, err, check);
    else if (f == D_F8) produce<D_F8, 8>(s, ring, n, tid, abort, err);
    else produce<D_I4, 4>(s, ring, n, tid, abort, err);
  } else {
    if (f == D_CB4) produce<D_CB4, 2>(s, ring, n, tid, abort, err);
    else if (f == D_CB3) produce<D_CB3, 2>(s, ring, n, tid, abort, err);
    else produce<D_CB2, 2>(s, ring, n, tid, abort, err);
  }
}

__device__ __forceinline__ int decode_kind(int fmt, int bits) {
  switch (fmt) {
    case KVQ_FMT_FP16: return D_F16;
    case KVQ_FMT_FP8_E4M3: return D_F8;
    case KVQ_FMT_INT4_G32: return D_I4;
    default: return bits == 4 ? D_CB4 : (bits == 3 ? D_CB3 : D_CB2);
  }
}

// ------------------------------------------------------------------------ softmax
// m of a chunk's row before it has seen a token: finite, so that hidden scores weigh nothing.
constexpr float kNothing = -1e30f;
// A weight where columns are hidden (not in `see`: none) or their values were not finite (`bad`: NaN).
__device__ __forceinline__ float weight_of(float w, uint32_t see, uint32_t bad, int e) {
  w = bad >> e & 1u ? __uint_as_float(0x7FC00000u) : w;
  return see >> e & 1u ? w : 0.f;
}

// A row's m has grown, f = 2^(old - new): the accumulator (if any product has gone into it)
// and the tile's first `done` weight columns are scaled.  Both may have been stored for this
// same tile (the weights of its first half, the accumulator by a rescaling for that half), and a load
// is not ordered behind a store that has not been waited for.
__device__ __forceinline__ void rescale(uint32_t o_at, bool acc, uint32_t p_at, int done, float f) {
  tc_wait_st();
  uint32_t v[16];
#pragma unroll 1
  for (int c = 0; acc && c < kDim; c += 16) {
    tc_ld16(o_at + c, v);
    tc_wait_ld(v);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
    tc_st16(o_at + c, v);
  }
#pragma unroll 1
  for (int c = 0; c < done; c += 16) {
    tc_ld16(p_at + c, v);
    tc_wait_ld(v);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 x = unpack_half2(v[e]);
      v[e] = half2_bits(x.x * f, x.y * f);
    }
    tc_st16(p_at + c, v);
  }
}

// ------------------------------------------------------------------------ the kernel
// CODES: tiers of codebook formats, else of the others (a branch on the format in the softmax loop
// made it a third slower for both).
// Measured (GB300): 256 sequences x 64 / 8 heads on 16384 tokens of fp8 keys and INT4 values, 202 us,
// 1.5 us a tile of 128 rows on 128 of 152 SMs: a softmax group's chain of scores, weights and products
// (issue slots 59% busy; the sum of rounded weights is 12 us of it, and without the queries' second
// part it takes the same time).  8 sequences x 32 heads on 8192 tokens of 4-bit codes, 47 us: 1.4 us a
// tile whatever the rows (table look-ups, tiles written and read), and about 10 us of set-up, first
// tile and drain.
//
// With ChunkParams the items are those of a chunk call's plan: the rows of one sequence's tokens, each of which sees
// its own part of the tiles (chunk.cuh).  Tiles that all rows of the block see whole run as above; in the others
// hidden columns weigh nothing, whatever they hold.
template <bool CODES, class P = SharedParams>
__global__ void __launch_bounds__(kThreads, 1) shared_prefix_kernel(const __grid_constant__ P p) {
  constexpr bool MASKED = std::is_same<P, ChunkParams>::value;
  if constexpr (MASKED) {
    // (behind another pass over the cache, whose blocks all have waited for the plan, there is nothing to wait for)
    if (p.wait_first) grid_wait();
    grid_release();
  } else {
    // the pass over the sequences' own tiers may start on SMs that this grid leaves idle
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw + (smem - smem_u32(smem_raw)) + kOffCtl);
  volatile int* abort = &ctl->abort;
  const uint32_t bars = smem + kOffCtl;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);

  int hk, g, rows, n, len, tile0 = 0, lb = 0, split = 0, ti = 0;
  ChunkItem job;
  if constexpr (MASKED) {
    const int at = (int)blockIdx.x / p.hkv;
    if (at >= p.head->items[CODES ? 2 : 1]) {
      if (!p.wait_first) grid_wait();
      return;
    }
    hk = (int)blockIdx.x % p.hkv;
    job = p.item[CODES ? 2 : 1][at];
    g = job.seq;
    ti = job.tier;
    n = job.count;
    const ChunkSeq& sq = p.seq[g];
    rows = min((sq.tokens << p.group_shift) - job.row0, kTileRows);
    len = (ti + 1 < p.num_tiers ? sq.base[ti + 1] : sq.len) - sq.base[ti];  // of the tier
  } else {
    // ---- the item: split, kv head, row block (blocks of one split and head side by side, so
    // that they meet the same cache bytes in L2)
    int item = blockIdx.x;
    const int blk = item % p.num_blocks;
    item /= p.num_blocks;
    hk = item % p.hkv;
    split = item / p.hkv;
    int lo = 0, hi = p.num_groups;  // the group whose row blocks hold blk
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.block[mid] <= blk) lo = mid;
      else hi = mid;
    }
    g = lo;
    lb = blk - p.block[g];
    rows = min((p.offset[g + 1] - p.offset[g]) * p.group - lb * kTileRows, kTileRows);  // > 0
    while (ti + 1 < p.num_tiers && split >= p.tier[ti + 1].first) ++ti;
    const SharedTier& T = p.tier[ti];
    split -= T.first;  // of the tier's
    int bits = 0;
    len = checked_len(__ldg(T.lens + g), T.max_pages, p.page_size, &bits);
    if (bits && threadIdx.x == 0) atomicOr(p.err, bits);
    const int all = (len + kTileTokens - 1) / kTileTokens;
    const int per = (all + T.num_splits - 1) / T.num_splits;
    tile0 = min(split * per, all);
    const int tile1 = min(tile0 + per, all);
    n = tile1 - tile0;
  }
  const auto& T = p.tier[ti];
  int* const err = [&] {
    if constexpr (MASKED) return &p.head->err;
    else return p.err;
  }();
  // Tile i of the item.
  auto tile_of = [&](int i) {
    if constexpr (MASKED) {
      const int x = job.first + i;
      return x < job.sinks ? x : job.begin + x - job.sinks;
    } else {
      return tile0 + i;
    }
  };
  // Where the block's first row stands, of the tier's tokens; and whether a row of the block sees not all of tile i.
  int stands = 0;
  if constexpr (MASKED) {
    const ChunkSeq& sq = p.seq[g];
    stands = sq.len - sq.tokens + (job.row0 >> p.group_shift) - sq.base[ti];
  }
  auto edge = [&](int i) {
    if constexpr (MASKED) {
      const int start = tile_of(i) * kTileTokens, end = start + kTileTokens;
      const int last = stands + ((rows - 1) >> p.group_shift);  // (row blocks begin with a token's first row)
      const bool inside = !p.window || start > last - p.window || end <= p.sinks - (p.seq[g].base[ti]);
      return !(end <= len && end <= stands + 1 && inside);
    } else {
      return false;
    }
  };
  const int w = warp >> 2;  // softmax group of the first eight warps
  const int r = threadIdx.x & 127;
  // Row of this softmax thread, as an output row (sequence, query head), or -1; and where the group's
  // partials lie (tiles w, w + 2, ...).  Worked out where they are used: registers are short in between.
  auto output_row = [&]() -> long long {
    if (warp >= 8 || r >= rows) return -1;
    if constexpr (MASKED) return r;
    else {
      const int gr = lb * kTileRows + r, i = gr / p.group;
      return (long long)(p.offset[g] + i) * p.hq + hk * p.group + (gr - i * p.group);
    }
  };
  auto partials = [&]() -> size_t {
    if constexpr (MASKED) return ((size_t)(job.part + w) * p.hkv + hk) * kTileRows;
    else return (2 * (size_t)(T.split_begin + split) + w) * ((size_t)p.batch * p.hq);
  };
  float* const all_ml = reinterpret_cast<float*>(p.ml);

  if (n == 0) {  // no tokens: partials of weight zero
    const long long out_row = output_row();
    if (out_row >= 0) *reinterpret_cast<float2*>(all_ml + 2 * (partials() + out_row)) = make_float2(-INFINITY, 0.f);
    if constexpr (MASKED) {
      if (!p.wait_first) grid_wait();
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(bars + 8 * (B_KFULL + i), 128);
      bar_init(bars + 8 * (B_KEMPTY + i), 1);
      bar_init(bars + 8 * (B_VFULL + i), 128);
      bar_init(bars + 8 * (B_VEMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bars + 8 * (B_SFULL + i), 1);
      bar_init(bars + 8 * (B_PREADY + i), (rows + 31) / 32 * 32);  // the warps that hold rows
      bar_init(bars + 8 * (B_OFULL + i), 1);
    }
    bar_init(bars + 8 * B_QFULL, 128);
    bar_init(bars + 8 * B_QROT, 1);
    for (int i = 0; i < kAhead; ++i) {
      bar_init(bars + 8 * (B_ROWS + i), 32);
      bar_init(bars + 8 * (B_AUX + i), 32);
      // the decoding threads, and (norms of keys) the softmax warps that read the tile's scores
      bar_init(bars + 8 * (B_ROWS_READ + i), 256 + (CODES || MASKED ? (rows + 31) / 32 : 0));
    }
    ctl->abort = 0;
    ctl->bad_page = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  Tables tables;
  int page[4];
  Pages pages;
  if constexpr (MASKED) pages.table = T.block_table + (size_t)g * T.table_pages;
  else pages.table = T.block_table + (size_t)g * T.max_pages;
  pages.num_pages = T.num_pages;
  pages.page_size = p.page_size;
  pages.page_shift = p.page_shift;
  pages.hkv = p.hkv;
  pages.hk = hk;
  pages.end = len;
  if constexpr (MASKED) {
    pages.hide = max(0, p.sinks - p.seq[g].base[ti]);
    pages.hidden = p.window ? max(0, stands - p.window + 1 - pages.hide) : 0;
  }
  // ---- before the block meets: everything that needs no barrier
  if (warp < 8) {
    // The block's queries are rotated as one more product, of the queries as they come (fp16,
    // exact) and the matrix of elements s_k (-1)^popc(n & k) (exact too), in float32: here both
    // are laid out.  (Butterflies by shuffles took 15 us for 256 rows.)
    const int tid = threadIdx.x & 255;
    const int shift = __ffs(p.group) - 1;
    {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = i * 16 + (tid >> 4);
        v[i] = make_uint4(0, 0, 0, 0);
        if (row < rows) {
          const int gr = lb * kTileRows + row, sq = gr >> shift;
          if constexpr (MASKED) {
            const int qr = job.row0 + row;
            const uint16_t* src = p.q + (p.seq[g].q0 + (qr >> shift)) * p.q_token + ((hk << shift) + (qr & (p.group - 1))) * p.q_head;
            v[i] = __ldg(reinterpret_cast<const uint4*>(src) + (tid & 15));
          } else {
            const size_t orow = (size_t)(p.offset[g] + sq) * p.hq + hk * p.group + (gr - (sq << shift));
            v[i] = __ldg(reinterpret_cast<const uint4*>(p.q + orow * kDim) + (tid & 15));
          }
        }
      }
      const uint32_t to = smem + kOffQ + ((tid & 15) >> 3) * kHalfBytes;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * 16 + (tid >> 4);
        sts16(to + r * 128 + (((tid & 7) ^ (r & 7)) << 4), v[i].x, v[i].y, v[i].z, v[i].w);
      }
    }
    const int c = tid & 15;  // elements 8c .. 8c + 7 of rows n
    const uint2 sg = __ldg(reinterpret_cast<const uint2*>(p.k_signs + (size_t)hk * kDim) + c);
    const uint32_t to = smem + kOffV + kTileBytes + (c >> 3) * kHalfBytes;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n7 = (tid >> 4) & 7, nr = i * 16 + (tid >> 4);
      const bool flip = __popc((nr >> 3) & c) & 1;  // the chunk's part of the parity
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t s0 = (k < 2 ? sg.x >> (16 * k) : sg.y >> (16 * (k - 2)));  // sign bytes 2k, 2k + 1
        const uint32_t lo = ((s0 >> 7) ^ __popc(n7 & (2 * k)) ^ (uint32_t)flip) & 1u;
        const uint32_t hi = ((s0 >> 15) ^ __popc(n7 & (2 * k + 1)) ^ (uint32_t)flip) & 1u;
        h[k] = 0x3C003C00u | (lo << 15) | (hi << 31);
      }
      sts16(to + nr * 128 + (((c & 7) ^ (nr & 7)) << 4), h[0], h[1], h[2], h[3]);
    }
    fence_async_smem();
  } else if (warp < 16) {
    if constexpr (CODES) {
      const bool keys = warp < 12;
      const int side = keys ? 0 : 1, tid = threadIdx.x & 127, lane = threadIdx.x & 31;
      const float kc = lane < (1 << T.k_bits) ? __ldg(T.k_cent + lane) : 0.f;
      const float vc = lane < (1 << T.v_bits) ? __ldg(T.v_cent + lane) : 0.f;
      const bool same = T.k_bits == T.v_bits && __all_sync(0xFFFFFFFFu, kc == vc);  // one table (often so)
      tables = place_tables(smem, T.k_bits, T.v_bits, same);
      const int bits = keys ? T.k_bits : T.v_bits;
      const float beta = scale_table(ctl, keys ? kc : vc, bits, side, tid);
      if (keys || !same) build_lut(tables.at[side], tables.copies[side], (keys ? kc : vc) * beta, bits, tid);
    }
  } else if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctl->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp < 17 + kLookUps) {
    first_pages<MASKED>(pages, tile_of, n, warp - 17, page);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp < 8) {
    // ---- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // The rotated queries, from TMEM: times log2(e) / D (1 / sqrt(D) of the rotation and of the
    // scores, which are then in base-2 units), as two fp16 numbers into the query tiles.
    bool ok = true;
    if (w == 0) {
      ok = __all_sync(0xFFFFFFFFu, bar_wait(bars + 8 * B_QROT, 0, abort, err));
      tc_fence_after();
      const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t to = smem + kOffQ + r * 128, rest = kTileBytes;
      constexpr float scale = 1.4426950408889634f / kDim;
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        uint32_t v[32];
        tc_ld32(from + 32 * part, v);
        tc_wait_ld(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t h[4], l[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = __uint_as_float(v[8 * i + 2 * k]) * scale, b = __uint_as_float(v[8 * i + 2 * k + 1]) * scale;
            h[k] = half2_bits(a, b);
            const float2 near = unpack_half2(h[k]);
            l[k] = half2_bits(a - near.x, b - near.y);
          }
          const int at = 4 * part + i;
          const uint32_t chunk = to + (at >> 3) * kHalfBytes + (((at & 7) ^ (r & 7)) << 4);
          sts16(chunk, h[0], h[1], h[2], h[3]);
          sts16(chunk + rest, l[0], l[1], l[2], l[3]);
        }
      }
      tc_fence_before();
      fence_async_smem();
      bar_arrive(bars + 8 * B_QFULL);
    }
    const int my_tiles = n > w ? (n - w + 1) / 2 : 0;
    const bool live = (warp & 3) * 32 < rows;  // the warp holds rows
    if (live && my_tiles > 0) {
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_at = lane_base + w * 128, o_at = lane_base + 256 + w * 128;
      float m = MASKED ? kNothing : -INFINITY;
      unsigned long long l2 = 0;  // the row's sum, even and odd columns
      for (int k = 0; k < my_tiles && ok; ++k) {
        const int i = 2 * k + w, at = i % kAhead;
        const int valid = MASKED ? kTileTokens : min(kTileTokens, len - tile_of(i) * kTileTokens);
        // a chunk's row sees columns below `until`, and of those the ones from `from` on or below `sinks`
        const bool hides = edge(i);
        int until = 0, from = 0, sinks = 0;
        if constexpr (MASKED) {
          const int start = tile_of(i) * kTileTokens, stand = stands + (min(r, rows - 1) >> p.group_shift);
          until = min(stand + 1, len) - start;
          from = p.window ? stand - p.window + 1 - start : 0;
          sinks = p.sinks - p.seq[g].base[ti] - start;
        }
        auto sees = [&](int c) { return below(until, c) & (~below(from, c) | below(sinks, c)); };
        const uint8_t* base = reinterpret_cast<const uint8_t*>(ctl) - kOffCtl;
        const float* norm = reinterpret_cast<const float*>(base + kOffKAux) + at * kTileTokens;
        const float* v_norm = reinterpret_cast<const float*>(base + kOffVAux) + at * kTileTokens * 2;
        ok = bar_wait(bars + 8 * (B_SFULL + w), k & 1, abort, err);
        if (CODES) ok = ok && bar_wait(bars + 8 * (B_AUX + at), (i / kAhead) & 1, abort, err);
        if constexpr (MASKED && !CODES) {  // what was found in the values that is not finite
          if (hides) {
            ok = ok && bar_wait(bars + 8 * (B_AUX + at), (i / kAhead) & 1, abort, err);
            ok = ok && bar_wait(bars + 8 * (B_VFULL + w), k & 1, abort, err);
          }
        }
        if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
        tc_fence_after();
        // Half a tile's weights at a time, against m as it is, in registers: no maximum is taken.
        // All weights are positive, so a sum of at most kMostWeight says that none is too large for
        // fp16 either; only where it is exceeded (always at first, where m is -inf) m is raised
        // and the half, still in TMEM, weighed again.  Of codebooks P holds weights times values'
        // norms: both steps allow for the tile's largest.  (A chunk's items raise m above the largest product of a
        // weight and its own norm instead: behind a large value with next to no weight, small ones that have it all
        // would be fp16 subnormals, 8e-3 of the output for norms 2^19 apart.)
        const float top = CODES ? *reinterpret_cast<volatile float*>(&ctl->norm_top[at]) : 1.f;
#pragma unroll 1
        for (int c0 = 0; c0 < kTileTokens; c0 += 64) {
          uint32_t h[32];
          unsigned long long sum;
#pragma unroll 1
          for (int again = 0;; ++again) {
            const unsigned long long neg = pack2(-m, -m);
            unsigned long long s0 = 0, s1 = 0;
            auto weigh = [&](int c, uint32_t (&v)[32]) {
              uint32_t see = 0, bad = 0;
              if constexpr (MASKED) {
                if (hides) {
                  see = sees(c0 + c);
                  if (!CODES) bad = *reinterpret_cast<volatile uint32_t*>(&ctl->not_finite[at][(c0 + c) / 32]);
                }
              }
              if (!MASKED && valid < kTileTokens) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (c0 + c + e >= valid) v[e] = 0xFF800000u;  // -inf: weight 0
              }
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                unsigned long long t0 = pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                unsigned long long t1 = pack2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                if constexpr (CODES) {  // scores are multiplied by the keys' norms
                  const float4 n = *reinterpret_cast<const float4*>(norm + c0 + c + e);
                  t0 = fma2(t0, pack2(n.x, n.y), neg);
                  t1 = fma2(t1, pack2(n.z, n.w), neg);
                } else {
                  t0 = add2(t0, neg);
                  t1 = add2(t1, neg);
                }
                const float2 x = unpack2(t0), y = unpack2(t1);
                float w0 = ex2(x.x), w1 = ex2(x.y), w2 = ex2(y.x), w3 = ex2(y.y);
                if constexpr (MASKED) {
                  if (hides) {
                    w0 = weight_of(w0, see, bad, e);
                    w1 = weight_of(w1, see, bad, e + 1);
                    w2 = weight_of(w2, see, bad, e + 2);
                    w3 = weight_of(w3, see, bad, e + 3);
                  }
                }
                unsigned long long a = pack2(w0, w1), b = pack2(w2, w3);
                if constexpr (CODES) {
                  s0 = add2(s0, a);
                  s1 = add2(s1, b);
                  const float4 n = *reinterpret_cast<const float4*>(v_norm + c0 + c + e);
                  a = mul2(a, pack2(n.x, n.y));
                  b = mul2(b, pack2(n.z, n.w));
                  if constexpr (MASKED) {  // (a norm may be infinite)
                    if (hides) {
                      const float2 u = unpack2(a), v = unpack2(b);
                      a = pack2(weight_of(u.x, see, 0u, e), weight_of(u.y, see, 0u, e + 1));
                      b = pack2(weight_of(v.x, see, 0u, e + 2), weight_of(v.y, see, 0u, e + 3));
                    }
                  }
                }
                const float2 u = unpack2(a), w = unpack2(b);
                h[(c + e) / 2] = half2_bits(u.x, u.y);
                h[(c + e) / 2 + 1] = half2_bits(w.x, w.y);
                if constexpr (!CODES) {  // the sum of what is multiplied: a token that outweighs all others keeps its value
                  const float2 ru = unpack_half2(h[(c + e) / 2]), rw = unpack_half2(h[(c + e) / 2 + 1]);
                  s0 = add2(s0, pack2(ru.x, ru.y));
                  s1 = add2(s1, pack2(rw.x, rw.y));
                }
              }
            };
            uint32_t va[32], vb[32];
            tc_ld32(s_at + c0, va);
            tc_wait_ld(va);
            tc_ld32(s_at + c0 + 32, vb);
            weigh(0, va);
            tc_wait_ld(vb);
            weigh(32, vb);
            sum = add2(s0, s1);
            const float2 t = unpack2(sum);
            // (a chunk's items: also behind the sinks, where the maximum of a few tokens would be exceeded row by row; a sum
            // of NaN stays that)
            const bool raise = MASKED && ((k > 0 && job.first + i >= job.sinks && job.first + i - 2 < job.sinks && c0 == 0) ||
                                          (t.x + t.y) * top > kMostWeight);
            if (again || __all_sync(0xFFFFFFFFu, MASKED ? !raise : (t.x + t.y) * top <= kMostWeight)) break;
            const float head = kHeadroom - (float)((int)(__float_as_uint(top) >> 23) - 127);
            float mx = m;
#pragma unroll 1
            for (int c = c0; c < c0 + 64; c += 16) {
              uint32_t x[16];
              tc_ld16(s_at + c, x);
              tc_wait_ld(x);
              const uint32_t see = MASKED ? sees(c) : 0u;
              if constexpr (MASKED && CODES) {
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float4 n = *reinterpret_cast<const float4*>(norm + c + e);
                  const float4 w = *reinterpret_cast<const float4*>(v_norm + kTileTokens + c + e);
                  const float y[4] = {fmaf(__uint_as_float(x[e]), n.x, w.x), fmaf(__uint_as_float(x[e + 1]), n.y, w.y),
                                      fmaf(__uint_as_float(x[e + 2]), n.z, w.z), fmaf(__uint_as_float(x[e + 3]), n.w, w.w)};
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    if (!hides || (see >> (e + k) & 1u)) mx = fmaxf(mx, y[k]);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (MASKED ? !hides || (see >> e & 1u) : c + e < valid)
                    mx = fmaxf(mx, __uint_as_float(x[e]) * (CODES ? norm[c + e] : 1.f) - head);
              }
            }
            // (of codebooks the sum of the weights says only that a product may be too large)
            if (MASKED && CODES && __all_sync(0xFFFFFFFFu, mx <= m)) break;
            const float f = ex2(m - mx);
            m = mx;
            const float2 ll = unpack2(l2);
            l2 = pack2(ll.x * f, ll.y * f);
            // (the products of earlier tiles are complete: they precede these scores)
            rescale(o_at, k > 0, s_at, c0 / 2, f);
          }
          l2 = add2(l2, sum);
#pragma unroll
          for (int c = 0; c < 32; c += 16) {  // over the scores
            uint32_t part[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) part[e] = h[c + e];
            tc_st16(s_at + c0 / 2 + c, part);
          }
        }
        if constexpr (CODES || MASKED) {
          __syncwarp();
          if ((threadIdx.x & 31) == 0) bar_arrive(bars + 8 * (B_ROWS_READ + at));
        }
        tc_wait_st();
        tc_fence_before();
        bar_arrive(bars + 8 * (B_PREADY + w));
      }
      if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait(bars + 8 * (B_OFULL + w), (my_tiles - 1) & 1, abort, err));
      tc_fence_after();
      const long long out_row = output_row();
      const size_t part = partials();
      // The accumulator leaves through shared memory, 16 KB a warp, so that rows are written
      // whole: the tiles are free (the group that ends first has the key stages, whose products
      // precede its last one, the other the value stages).
      if (ok) {
        const bool last = ((n - 1) & 1) == w;
        const int lane = threadIdx.x & 31;
        const uint32_t stage = smem + (last ? kOffV : kOffK) + (warp & 3) * (32 * kDim * 4);
        const float value_unit = CODES ? *reinterpret_cast<volatile float*>(&ctl->unscale[1]) *
                                             *reinterpret_cast<volatile float*>(&ctl->norm_unit) : 1.f;
        const bool int4 = T.v_fmt == KVQ_FMT_INT4_G32;  // columns 0 4 1 5 2 6 3 7 of every eight
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tc_ld32(o_at + 32 * c, v);
          tc_wait_ld(v);
          if constexpr (CODES) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * value_unit);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            const uint32_t o1 = int4 ? v[e + 2] : v[e + 1], o2 = int4 ? v[e + 4] : v[e + 2];
            const uint32_t o3 = int4 ? v[e + 6] : v[e + 3], o4 = int4 ? v[e + 1] : v[e + 4];
            const uint32_t o5 = int4 ? v[e + 3] : v[e + 5], o6 = int4 ? v[e + 5] : v[e + 6];
            const int at = 8 * c + e / 4;  // 16-byte chunk of the lane's row
            sts16(stage + lane * (kDim * 4) + ((at ^ (lane & 7)) << 4), v[e], o1, o2, o3);
            sts16(stage + lane * (kDim * 4) + (((at + 1) ^ (lane & 7)) << 4), o4, o5, o6, v[e + 7]);
          }
        }
        __syncwarp();
        float* base = p.acc + part * kDim;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
          const long long to = __shfl_sync(0xFFFFFFFFu, out_row, i);
          float4 x;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                       : "r"(stage + i * (kDim * 4) + ((lane ^ (i & 7)) << 4)));
          if (to >= 0) reinterpret_cast<float4*>(base + to * kDim)[lane] = x;
        }
      }
      // A page outside the pool anywhere in the item leaves it out of the result.  (The other group's
      // last tile may be one behind: its look-ups too have to be over.)
      if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait(bars + 8 * (B_ROWS + (n - 1) % kAhead), ((n - 1) / kAhead) & 1, abort, err));
      ok = ok && !*reinterpret_cast<volatile int*>(&ctl->bad_page);
      if (out_row >= 0) {
        // (a row of NaN has no maximum: its partial must not pass for one without tokens)
        const float l = unpack2(l2).x + unpack2(l2).y;
        *reinterpret_cast<float2*>(all_ml + 2 * (part + out_row)) =
            ok && !(MASKED && l == 0.f) ? make_float2(l == l ? m : l, l) : make_float2(-INFINITY, 0.f);
      }
    } else if (const long long out_row = output_row(); out_row >= 0) {  // a second group without a tile of its own
      *reinterpret_cast<float2*>(all_ml + 2 * (partials() + out_row)) = make_float2(-INFINITY, 0.f);
    }
  } else if (warp < 16) {
    // ---- decoding
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDecodeRegs));
    const bool keys = warp < 12;
    Source s;
    s.rows = keys ? T.k_rows : T.v_rows;
    s.row_bytes = keys ? T.k_row_bytes : T.v_row_bytes;
    if constexpr (CODES) {
      const int side = keys ? 0 : 1;
      s.lut = tables.at[side] + 4u * (threadIdx.x & (tables.copies[side] - 1));
      s.lut_stride = 4u * tables.copies[side];
      s.raw = tables.raw[side];
    } else {
      s.raw = smem + kOffLut + (keys ? 0 : 16 << 10);
    }
    s.rowbuf = smem + kOffRow;
    s.auxbuf = smem + kOffVAux;
    Ring ring;
    ring.tiles = smem + (keys ? kOffK : kOffV);
    ring.full = bars + 8 * (keys ? B_KFULL : B_VFULL);
    ring.empty = bars + 8 * (keys ? B_KEMPTY : B_VEMPTY);
    ring.rows = bars + 8 * B_ROWS;
    ring.aux = bars + 8 * B_AUX;
    ring.rows_read = bars + 8 * B_ROWS_READ;
    ring.first_use = keys ? 0 : bars + 8 * B_QROT;  // the second value stage first holds the rotation
    const int kind = keys ? decode_kind(T.k_fmt, T.k_bits) : decode_kind(T.v_fmt, T.v_bits);
    if constexpr (MASKED && !CODES) {
      auto check = [&](int i, uint32_t tile) {
        if (keys || !edge(i)) return;
#pragma unroll 1
        for (int pass = 0; pass < unit_passes(D_F16); ++pass) {
          int t, u;
          place<D_F16>(pass, threadIdx.x & 127, t, u);
          const uint32_t piece = tile + (u >> 3) * kHalfBytes + t * 128 + (((u & 7) ^ (t & 7)) << 4);
          uint32_t x[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(piece) : "memory");
          bool fine = true;
#pragma unroll
          for (int k = 0; k < 4; ++k) fine = fine && (x[k] & 0x7C00u) != 0x7C00u && (x[k] & 0x7C000000u) != 0x7C000000u;
          if (!fine) {
            sts16(piece, 0u, 0u, 0u, 0u);
            atomicOr(&ctl->not_finite[i % kAhead][t / 32], 1u << (t % 32));
          }
        }
      };
      produce_any<CODES>(kind, s, ring, n, threadIdx.x & 127, abort, err, check);
    } else {
      produce_any<CODES>(kind, s, ring, n, threadIdx.x & 127, abort, err, NoCheck{});
    }
  } else {
    // ---- products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    // The whole warp walks the jobs and one lane issues: with all of it uniform, descriptors are
    // formed in uniform registers (issued from one lane's branch, each product cost about 110
    // cycles of register moves, twice what it takes to run).
    if (warp == 16) {
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint64_t qd = desc_at(desc_base(16, 1024), smem + kOffQ), kd = desc_at(desc_base(16, 1024), smem + kOffK);
      const uint64_t vd = desc_at(desc_base(kHalfBytes, 1024), smem + kOffV);
      auto well = [&](uint32_t bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, abort, err));
      };
      auto scores = [&](int i) -> bool {  // S of tile i, for softmax group i & 1
        const int st = i & 1;
        if (!well(bars + 8 * (B_KFULL + st), (i >> 1) & 1)) return false;
        tc_fence_after();
        const uint64_t b = kd + st * (kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {  // the queries' first parts, then the second (unrolled, descriptors spill)
            const uint64_t a = qd + half * (kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < kDim / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
              mma_ss(tm + st * 128, a + off, b + off, kIdescQK, half + kk > 0);
            }
          }
          tc_commit(bars + 8 * (B_SFULL + st));
          tc_commit(bars + 8 * (B_KEMPTY + st));
        }
        __syncwarp();
        return true;
      };
      {  // the rotated queries, into the score columns
        const uint64_t rd = desc_at(desc_base(16, 1024), smem + kOffV + kTileBytes);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kDim / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
            mma_ss(tm, qd + off, rd + off, kIdescQK, kk > 0);
          }
          tc_commit(bars + 8 * B_QROT);
        }
        __syncwarp();
      }
      bool ok = well(bars + 8 * B_QFULL, 0);
      for (int i = 0; i < 2 && i < n && ok; ++i) ok = scores(i);
      for (int i = 0; i < n && ok; ++i) {
        const int st = i & 1;
        ok = well(bars + 8 * (B_VFULL + st), (i >> 1) & 1) && well(bars + 8 * (B_PREADY + st), (i >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t b = vd + st * (kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTileTokens / 16; ++kk)
            mma_ts(tm + 256 + st * 128, tm + st * 128 + kk * 8, b + ((kk * 2048) >> 4), kIdescPV, i > 1 || kk > 0);
          tc_commit(bars + 8 * (B_OFULL + st));
          tc_commit(bars + 8 * (B_VEMPTY + st));
        }
        __syncwarp();
        if (i + 2 < n) ok = scores(i + 2);
      }
    } else if (warp < 17 + kLookUps) {
      // ---- look-ups
      look_up<MASKED>(pages, page, CODES ? T.k_aux : nullptr, CODES ? T.v_aux : nullptr, T.v_fmt == KVQ_FMT_INT4_G32 ? T.v_aux : nullptr,
              ctl, smem, bars, tile_of, edge, n, warp - 17, abort, err);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if constexpr (MASKED) {  // complete only behind the pass before, for what waits for this grid
    if (!p.wait_first) grid_wait();
  }
}

}  // namespace
}  // namespace kvq
