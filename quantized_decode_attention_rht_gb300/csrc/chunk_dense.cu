// Attention of long chunks (kvq_chunk_attention): what a chunk sees is unpacked once into tiles of
// fp16 numbers, and each unit of up to 256 query rows runs over them on the tensor cores.
//
//   S = q~ K^T,  P = 2^(S - m),  O += P V,  l += rowsum P,
// with rotated queries q~ (times log2 e / sqrt(D)) and the rotated keys and values as the cache holds them; the
// value rotation is undone where results are stored or joined.
//
// prepare_kernel writes every operand as the products read it (rows of 128 bytes, 16-byte pieces swizzled), so that
// attention loads whole tiles by one bulk copy each:
//   queries   two fp16 numbers, the nearest one and the rest: rounded once they would be off by 2^-12 of their size,
//             which keys with outlier channels turn into 6e-4 of the output
//   keys      fp16 and fp8 keys as they are; of codebooks the centroid under its table's scale, and the key's norm as
//             a factor of its scores; keys with a sketch or outliers as two fp16 numbers, as queries (one
//             alone: 1.7e-3 of the output where channels thirty times the others make keys large)
//   values    fp16 as they are, INT4 levels times their scale (one rounding); of codebooks the centroid times the
//             norm's power of two, and the norm's mantissa as a factor of the weights.
// Why unpack: a unit's products over 128 tokens take about 2 us on an SM, decoding the tokens 1.4 us; a chunk of 2048
// tokens with four query heads a kv head would decode each token 32 times.
// Bounded by memory: a token's row is read once, 4 head_dim bytes a kv head are written, and written back where they
// pass the L2.  75 us for 32768 tokens x 8 heads of fp8 keys and INT4 values (286 MB, 3.8 TB/s), 155 us for 2 x 16896
// tokens x 16 heads x 256 of 4-bit codes.  (Rows of the next tile loaded ahead, or a key's and a value's together, took
// the same time.)
//
// attend_kernel: one item (tiles of a unit) a block of 10 warps: 2 x 4 softmax warps, a thread a row of two blocks of
// 128 rows; one warp that loads, one that issues products.  While one row block's scores become weights, the other's
// products run.  TMEM: two blocks of scores, over which the weights are written, and two accumulators, all 512
// columns at head_dim 128.  (head_dim 256: one row block, tiles of 64 tokens, two score blocks in turn.)
// Bounded by the products and by waves: 4096 tokens x 32/8 heads on 28672 of fp8 keys and INT4 values take 1960 us,
// unpacking among them: 1.05 PFLOP/s, 1.57 with the queries' second part.  Its 512 items of one length are 3.37 waves of
// 152 SMs, 966 tiles one after the other where equal shares would be 820.  A pair of row blocks over 128 tokens takes 3770 cycles, 3070
// of them products: a row block's scores (1024), weights (about 2000) and values (512) follow one another, as
// the weights lie over the scores and TMEM has no room for more.  Where products are shorter or weights longer the softmax
// warps' latency alone counts, two warps a scheduler (tensor pipe 31%, issue slots 29%): 270 us for a prompt of 4096
// tokens x 32 heads of 4-bit codes, whose factors make weights 2200 to 3000 cycles, 150 us for 3 x 777 tokens x 16/4
// heads x 64 on 5001.  (Two threads a row took the same time; scores two tiles ahead, at head_dim 64, which TMEM holds
// for tiles of 64 tokens, 171 instead of 148 us; a quarter to a third of the powers as polynomials, beside the
// special-function unit, up to a fifth longer.)
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "chunk.cuh"
#include "tc.cuh"

namespace kvq {
namespace {

constexpr int kPrepareThreads = 256;

// ------------------------------------------------------------------------ unpacking
constexpr uint32_t kNone = 0xFFFFFFFFu;

// Formats as unpacking sees them.
enum { U_F16, U_F8, U_I4, U_C4, U_C3, U_C2 };
__device__ __forceinline__ int unpack_kind(int fmt, int bits) {
  switch (fmt) {
    case KVQ_FMT_FP16: return U_F16;
    case KVQ_FMT_FP8_E4M3: return U_F8;
    case KVQ_FMT_INT4_G32: return U_I4;
    default: return bits == 4 ? U_C4 : (bits == 3 ? U_C3 : U_C2);
  }
}

// 16 stored coordinates, from 16 c on, of a row.
template <int F>
struct Raw {
  uint32_t w[F == U_F16 ? 8 : (F == U_F8 ? 4 : 2)];
  uint16_t scale;
};
template <int F>
__device__ __forceinline__ void load_raw(const uint8_t* row, const __half* scales, int c, Raw<F>& x) {
  if constexpr (F == U_F16) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(row) + 2 * c), b = __ldg(reinterpret_cast<const uint4*>(row) + 2 * c + 1);
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w, x.w[4] = b.x, x.w[5] = b.y, x.w[6] = b.z, x.w[7] = b.w;
  } else if constexpr (F == U_F8) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(row) + c);
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
  } else if constexpr (F == U_I4 || F == U_C4) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(row) + c);
    x.w[0] = a.x, x.w[1] = a.y;
    if constexpr (F == U_I4) x.scale = __half_as_ushort(__ldg(scales + c / 2));
  } else if constexpr (F == U_C3) {  // (rows of head_dim 64 are of 24 bytes)
    const uint16_t* a = reinterpret_cast<const uint16_t*>(row) + 3 * c;
    x.w[0] = (uint32_t)__ldg(a) | (uint32_t)__ldg(a + 1) << 16;
    x.w[1] = __ldg(a + 2);
  } else {
    x.w[0] = __ldg(reinterpret_cast<const uint32_t*>(row) + c);
    x.w[1] = 0;
  }
}
// As fp16 pairs: values of the plain formats, table entries of codebooks.
template <int F>
__device__ __forceinline__ void decode_raw(const Raw<F>& x, const uint16_t* table, uint32_t (&h)[8], int* over) {
  if constexpr (F == U_F16) {
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = x.w[k];
  } else if constexpr (F == U_F8) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[k]) : "h"((uint16_t)(x.w[k / 2] >> (16 * (k & 1)))));
  } else if constexpr (F == U_I4) {
    const uint16_t size = x.scale & 0x7FFFu;
    if (size >= 0x7092u && size < 0x7C00u) *over = 1;  // a finite scale above 9352: seven times it is no fp16 number
    const uint32_t s2 = x.scale * 0x10001u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // levels n - 8, exact in fp16: 1024 + n less 1032
      const uint32_t v = x.w[k / 4] >> (8 * (k & 3));
      const uint32_t up = (v & 15u) | (v & 0xF0u) << 12 | 0x64006400u;
      const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&up), __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408)));
      h[k] = hmul2(*reinterpret_cast<const uint32_t*>(&n), s2);
    }
  } else {
    constexpr int B = F == U_C4 ? 4 : (F == U_C3 ? 3 : 2);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t e[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = (2 * k + i) * B;
        const uint32_t f = at % 32 + B <= 32 ? x.w[at / 32] >> (at % 32) : __funnelshift_r(x.w[0], x.w[1], at % 32);
        e[i] = table[f & ((1u << B) - 1u)];  // (16 entries lie in eight banks: no two lanes wait for one another)
      }
      h[k] = e[0] | e[1] << 16;
    }
  }
}
// Any format, one row.
__device__ __forceinline__ void unpack16(int fmt, int bits, const uint8_t* row, const __half* scales, int c,
                                         const uint16_t* table, uint32_t (&h)[8], int* over) {
  auto one = [&](auto f) {
    Raw<decltype(f)::value> x;
    load_raw(row, scales, c, x);
    decode_raw(x, table, h, over);
  };
  switch (unpack_kind(fmt, bits)) {
    case U_F16: one(std::integral_constant<int, U_F16>{}); break;
    case U_F8: one(std::integral_constant<int, U_F8>{}); break;
    case U_I4: one(std::integral_constant<int, U_I4>{}); break;
    case U_C4: one(std::integral_constant<int, U_C4>{}); break;
    case U_C3: one(std::integral_constant<int, U_C3>{}); break;
    default: one(std::integral_constant<int, U_C2>{});
  }
}

__device__ __forceinline__ bool half2_finite(uint32_t h) {
  return (h & 0x7C00u) != 0x7C00u && (h & 0x7C000000u) != 0x7C000000u;
}
// A power of two above a finite x >= 0.
__device__ __forceinline__ float two_above(float x) {
  return __uint_as_float((min(max(__float_as_uint(x) >> 23, 64u), 190u) + 1u) << 23);
}
__device__ __forceinline__ float finite_or_zero(float x) { return x < INFINITY ? x : 0.f; }  // (NaN: zero)

// Offset of coordinate c (a multiple of 8) of row r in an operand tile of `rows` rows.
__device__ __forceinline__ uint32_t tile_at(int rows, int r, int c) {
  return (uint32_t)(c / 64) * rows * 128 + r * 128 + ((((c / 8) & 7) ^ (r & 7)) << 4);
}

// 16 coordinates from 16 c on, which are neighbouring pieces whatever the row's swizzle: one store.
__device__ __forceinline__ void store16(uint8_t* tile, int rows, int r, int c, const uint32_t (&x)[8]) {
  const bool turn = r & 1;
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(tile + (tile_at(rows, r, 16 * c) & ~16u)),
               "r"(turn ? x[4] : x[0]), "r"(turn ? x[5] : x[1]), "r"(turn ? x[6] : x[2]), "r"(turn ? x[7] : x[3]),
               "r"(turn ? x[0] : x[4]), "r"(turn ? x[1] : x[5]), "r"(turn ? x[2] : x[6]), "r"(turn ? x[3] : x[7])
               : "memory");
}

// The norm of a codebook token's key (side 0) or value.
__device__ __forceinline__ float norm_of(const ChunkTier& t, int side, uint32_t row) {
  if (side) return __half2float(t.v_aux[row]);
  if (t.k_fmt == KVQ_FMT_CODEBOOK_QJL) return __half2float(t.k_aux[2 * (size_t)row]);
  if (t.k_fmt == KVQ_FMT_CODEBOOK_OUTLIER)
    return __half2float(*reinterpret_cast<const __half*>(reinterpret_cast<const uint8_t*>(t.k_aux) + (size_t)row * (4 + KVQ_OUTLIER_CHANNELS)));
  return __half2float(t.k_aux[row]);
}

// Tier and row in its pool of a sequence's position (row kNone: no token there, none that a query sees, whose
// block-table entry may be of a page that the sequence has given back, or its page outside the pool).
__device__ __forceinline__ uint32_t find_row(const ChunkParams& p, const ChunkSeq& s, int seq, int h, int pos, int& tier, int* bits) {
  tier = 0;
  if (pos < 0 || pos >= s.len || (p.window && pos <= s.len - s.tokens - p.window && pos >= p.sinks)) return kNone;
#pragma unroll
  for (int k = 1; k < KVQ_MAX_TIERS; ++k)
    if (k < p.num_tiers && pos >= s.base[k]) tier = k;
  const ChunkTier& t = p.tier[tier];
  pos -= s.base[tier];
  const int page = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
  const int phys = __ldg(t.block_table + (size_t)seq * t.table_pages + page);
  if (!page_in_pool(phys, t.num_pages, bits)) return kNone;
  return ((uint32_t)phys * p.hkv + h) * p.page_size + (pos - page * p.page_size);  // below 2^32: the host checks
}

// A side of a tile whose tokens all lie in one tier, all of a thread's rows on their way at once.  VALUES: a row that
// is not finite becomes zeros and is noted in s_bad; keys of such rows become NaN.
template <int D, int F, bool VALUES>
__device__ __forceinline__ void unpack_side(const ChunkTier& t, uint8_t* to, const uint16_t* table, const uint32_t* s_row,
                                            const uint32_t* s_power, int* s_bad, int* over) {
  constexpr int TT = dense_tile(D), C = D / 16, kEach = TT * C / kPrepareThreads;
  const uint8_t* rows = VALUES ? t.v_rows : t.k_rows;
  const int row_bytes = VALUES ? t.v_row_bytes : t.k_row_bytes, c = threadIdx.x % C, r0 = threadIdx.x / C;
  Raw<F> raw[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t row = s_row[r0 + i * (kPrepareThreads / C)];
    load_raw(rows + (size_t)(row != kNone ? row : 0) * row_bytes, VALUES ? t.v_aux + (size_t)(row != kNone ? row : 0) * (D / kGroup) : nullptr,
             c, raw[i]);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = r0 + i * (kPrepareThreads / C);
    uint32_t x[8];
    int wide = 0;
    decode_raw(raw[i], table, x, &wide);
    bool zero = s_row[r] == kNone;  // (its raw coordinates are another token's)
    if (!zero) *over |= wide;
    if constexpr (VALUES && (F == U_F16 || F == U_F8 || F == U_I4)) {
      bool fine = true;
#pragma unroll
      for (int k = 0; k < 8; ++k) fine = fine && half2_finite(x[k]);
      if (!fine && !zero) s_bad[r] = 1;
      zero = zero || !fine;
    } else if constexpr (VALUES) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = hmul2(x[k], s_power[r]);
    } else {
      if (s_bad[r]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0x7E007E00u;
      }
    }
    if (zero) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = 0;
    }
    store16(to, TT, r, c, x);
  }
}
template <int D, bool VALUES>
__device__ __forceinline__ void unpack_any(const ChunkTier& t, uint8_t* to, const uint16_t* table, const uint32_t* s_row,
                                           const uint32_t* s_power, int* s_bad, int* over) {
  switch (VALUES ? unpack_kind(t.v_fmt, t.v_bits) : unpack_kind(t.k_fmt, t.k_bits)) {
    case U_F16: unpack_side<D, U_F16, VALUES>(t, to, table, s_row, s_power, s_bad, over); break;
    case U_F8:
      if constexpr (!VALUES) unpack_side<D, U_F8, VALUES>(t, to, table, s_row, s_power, s_bad, over);
      break;
    case U_I4:
      if constexpr (VALUES) unpack_side<D, U_I4, VALUES>(t, to, table, s_row, s_power, s_bad, over);
      break;
    case U_C4: unpack_side<D, U_C4, VALUES>(t, to, table, s_row, s_power, s_bad, over); break;
    case U_C3: unpack_side<D, U_C3, VALUES>(t, to, table, s_row, s_power, s_bad, over); break;
    default: unpack_side<D, U_C2, VALUES>(t, to, table, s_row, s_power, s_bad, over);
  }
}

template <int D>
__device__ __forceinline__ void unpack_tile(const ChunkParams& p, int tile, int h, const uint16_t (*tables)[2][16],
                                            uint32_t* s_row, uint32_t* s_power, int* s_tier, int* s_bad, float* s_max,
                                            int* s_tiers) {
  constexpr int TT = dense_tile(D), C = D / 16;
  const int tid = threadIdx.x, lane = tid & 31;
  // the sequence: the last whose tiles begin at or before this one (unpacked ones alone have any)
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.seq[mid].tile0 <= tile) lo = mid;
    else hi = mid;
  }
  const ChunkSeq s = p.seq[lo];
  const int i = tile - s.tile0, j = i < s.sink_tiles ? i : s.window_tile + i - s.sink_tiles;
  int bits = 0;
  __syncthreads();  // (the item before is done with the shared arrays)
  if (tid < TT) {
    int tier;
    s_row[tid] = find_row(p, s, lo, h, j * TT + tid, tier, &bits);
    s_tier[tid] = tier;
    s_bad[tid] = 0;
    const int tiers = __reduce_or_sync(0xFFFFFFFFu, s_row[tid] != kNone ? 1 << tier : 0);
    if (lane == 0) s_tiers[tid >> 5] = tiers;
  }
  // A codebook value's norm is split in two: a mantissa in [1, 2), which multiplies weights, and a power of two, which
  // goes into its row, where the table's entries take it without a rounding: weights then keep their precision however
  // small the value, and the sum can be taken of what is multiplied (a token that outweighs all others keeps its
  // value).  Rows hold 2^-6 to 2^15, so that no entry leaves fp16's normal numbers (the largest is 2^-3 to 2^-1); the mantissa of
  // norms below 2^-6 is smaller instead, by up to 2^-8, and below 2^-14, where the output is an fp16 subnormal, rows too.
  // Nothing is scaled by other tokens' norms, which the queries may not see, nor by other tiers' values.
  float mantissa = 1.0f;
  if (p.codes && tid < TT) {
    float power = 1.0f;
    const uint32_t row = s_row[tid];
    if (row != kNone && p.tier[s_tier[tid]].v_fmt == KVQ_FMT_CODEBOOK) {
      float norm = norm_of(p.tier[s_tier[tid]], 1, row);
      // (one tier's table scale comes behind the products; of several tiers it goes in here, rounded once)
      if (p.codes > 1) norm *= p.head->unscale[s_tier[tid]][1];
      if (norm == 0.f) {
        power = 0.f;
      } else if (finite_or_zero(norm) != 0.f) {
        const float two = __uint_as_float(__float_as_uint(norm) & 0x7F800000u);
        power = two >= 0x1p-14f ? fminf(fmaxf(two, 0x1p-6f), 0x1p15f) : (two >= 0x1p-24f ? two * 0x1p8f : 0.f);
        mantissa = power > 0.f ? norm / power : 1.0f;
        if (p.codes > 1) mantissa = __half2float(__float2half_rn(mantissa));
      } else {
        mantissa = norm;
      }
    }
    s_power[tid] = half2_bits(power, power);
  }
  __syncthreads();
  const size_t at = ((size_t)tile * p.hkv + h) * (TT * D * 2);
  int over = 0;
  // One tier's tokens alone, but for those that are not there, and keys without a sketch or an outlier stream?
  int tiers = 0;
#pragma unroll
  for (int k = 0; k < TT / 32; ++k) tiers |= s_tiers[k];
  const int first = max(0, __ffs(tiers) - 1), fmt = p.tier[first].k_fmt;
  const bool simple = __popc(tiers) == 1 && fmt != KVQ_FMT_CODEBOOK_QJL && fmt != KVQ_FMT_CODEBOOK_OUTLIER;
  if (simple) {
    const ChunkTier& t = p.tier[first];
    unpack_any<D, true>(t, p.vt + at, tables[first][1], s_row, s_power, s_bad, &over);
    __syncthreads();
    unpack_any<D, false>(t, p.kt + p.key_parts * at, tables[first][0], s_row, s_power, s_bad, &over);
    if (p.key_parts == 2) {  // (another tier's keys have a second part)
      const uint32_t none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int u = tid; u < TT * C; u += kPrepareThreads) store16(p.kt + 2 * at + TT * D * 2, TT, u / C, u % C, none);
    }
  }
  // values
  for (int u = tid; !simple && u < TT * C; u += kPrepareThreads) {
    const int r = u / C, c = u % C;
    uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const uint32_t row = s_row[r];
    if (row != kNone) {
      const ChunkTier& t = p.tier[s_tier[r]];
      unpack16(t.v_fmt, t.v_bits, t.v_rows + (size_t)row * t.v_row_bytes, t.v_aux + (size_t)row * (D / kGroup), c,
               tables[s_tier[r]][1], x, &over);
      bool fine = true;
#pragma unroll
      for (int k = 0; k < 8; ++k) fine = fine && half2_finite(x[k]);
      if (!fine) {  // a weight of zero must meet no infinity: the token's scores say it instead (its key is NaN)
        s_bad[r] = 1;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0;
      }
      if (t.v_fmt == KVQ_FMT_CODEBOOK) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = hmul2(x[k], s_power[r]);
      }
    }
    store16(p.vt + at, TT, r, c, x);
  }
  if (!simple) __syncthreads();
  // keys
  for (int u = tid; !simple && u < TT * C; u += kPrepareThreads) {
    const int r = u / C, c = u % C;
    uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, rest[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const uint32_t row = s_row[r];
    if (row != kNone) {
      const int tier = s_tier[r];
      const ChunkTier& t = p.tier[tier];
      unpack16(t.k_fmt, t.k_bits, t.k_rows + (size_t)row * t.k_row_bytes, nullptr, c, tables[tier][0], x, &over);
      if (t.k_fmt == KVQ_FMT_CODEBOOK_QJL || t.k_fmt == KVQ_FMT_CODEBOOK_OUTLIER) {
        const float kn = norm_of(t, 0, row) * p.head->unscale[tier][0];
        float y[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 f = unpack_half2(x[k]);
          y[2 * k] = f.x * kn;
          y[2 * k + 1] = f.y * kn;
        }
        if (t.k_fmt == KVQ_FMT_CODEBOOK_QJL) {
          // + ||r|| sqrt(pi / 2) / m * sum_j z_j S_j
          const float f = __half2float(t.k_aux[2 * (size_t)row + 1]) * (1.2533141373155003f / KVQ_QJL_DIM);
          const uint32_t* z = reinterpret_cast<const uint32_t*>(t.k_rows + (size_t)row * t.k_row_bytes + D * t.k_bits / 8);
          float sum[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[k] = 0.f;
#pragma unroll 1
          for (int m = 0; m < KVQ_QJL_DIM; ++m) {
            const uint32_t flip = ((__ldg(z + m / 32) >> (m % 32)) & 1u) ? 0u : 0x80000000u;
            const float4* sj = reinterpret_cast<const float4*>(t.k_qjl + (size_t)m * D + 16 * c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 v = __ldg(sj + k);
              sum[4 * k] += __uint_as_float(__float_as_uint(v.x) ^ flip);
              sum[4 * k + 1] += __uint_as_float(__float_as_uint(v.y) ^ flip);
              sum[4 * k + 2] += __uint_as_float(__float_as_uint(v.z) ^ flip);
              sum[4 * k + 3] += __uint_as_float(__float_as_uint(v.w) ^ flip);
            }
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = fmaf(f, sum[k], y[k]);
        } else {
          // + the rotated outliers: q_j s times column c_j of H diag(s) / sqrt(D)
          const uint8_t* rec = reinterpret_cast<const uint8_t*>(t.k_aux) + (size_t)row * (4 + KVQ_OUTLIER_CHANNELS);
          const float f = __half2float(*reinterpret_cast<const __half*>(rec + 2)) * inv_sqrt_dim(D);
#pragma unroll 1
          for (int m = 0; m < KVQ_OUTLIER_CHANNELS; ++m) {
            const int ch = __ldg(t.k_outl + h * KVQ_OUTLIER_CHANNELS + m);
            float v = f * (float)reinterpret_cast<const int8_t*>(rec)[4 + m];
            if (__ldg(p.k_signs + (size_t)h * D + ch) < 0) v = -v;
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] += __popc((16 * c + k) & ch) & 1 ? -v : v;
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = half2_bits(y[2 * k], y[2 * k + 1]);
          const float2 near = unpack_half2(x[k]);
          rest[k] = half2_bits(y[2 * k] - near.x, y[2 * k + 1] - near.y);
        }
      }
      if (s_bad[r]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0x7E007E00u;
      }
    }
    store16(p.kt + p.key_parts * at, TT, r, c, x);
    if (p.key_parts == 2) store16(p.kt + 2 * at + TT * D * 2, TT, r, c, rest);
  }
  if (p.codes) {
    if (tid < TT) {
      float kn = 1.0f;
      const uint32_t row = s_row[tid];
      if (row != kNone && p.tier[s_tier[tid]].k_fmt == KVQ_FMT_CODEBOOK)
        kn = norm_of(p.tier[s_tier[tid]], 0, row) * p.head->unscale[s_tier[tid]][0];
      const size_t n = ((size_t)tile * p.hkv + h) * TT + tid;
      p.kn[n] = kn;
      p.fn[n] = p.summed ? 1.0f / mantissa : mantissa;
      if (p.summed) p.hn[n] = __float2half_rn(mantissa);  // (exact: eleven bits)
      const float most = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(finite_or_zero(mantissa))));
      if (lane == 0) s_max[tid >> 5] = most;
    }
    __syncthreads();
    if (tid == 0) {
      float most = s_max[0];
      for (int k = 1; k < TT / 32; ++k) most = fmaxf(most, s_max[k]);
      p.top[(size_t)tile * p.hkv + h] = two_above(most);
    }
  }
  if (over) bits |= KVQ_DEVERR_VALUE_RANGE;
  if (bits) atomicOr(&p.head->err, bits);
}

// The rows of a unit's queries of one kv head: rotated, times log2(e) / D (1 / sqrt(D) of the rotation and of the
// scores, which are then in base-2 units), as two fp16 numbers.  D / 32 neighbouring lanes share a row, 32 coordinates
// each: five stages of the transform run in a lane's registers, the others between them (a third of the instructions of
// a warp a row).
template <int D>
__device__ __forceinline__ void rotate_queries(const ChunkParams& p, int unit, int h) {
  constexpr int L = D / 32, kRows = kChunkRows * dense_blocks(D), kAtOnce = kPrepareThreads / L;
  constexpr float scale = 1.4426950408889634f / D;
  const int sub = threadIdx.x % L;
  const ChunkUnit& x = p.unit[0][unit];
  const ChunkSeq& s = p.seq[x.seq];
  const int rows = s.tokens << p.group_shift;
  uint32_t sg[8];
  {
    const uint4* from = reinterpret_cast<const uint4*>(p.k_signs + (size_t)h * D + 32 * sub);
    const uint4 a = __ldg(from), b = __ldg(from + 1);
    sg[0] = a.x, sg[1] = a.y, sg[2] = a.z, sg[3] = a.w, sg[4] = b.x, sg[5] = b.y, sg[6] = b.z, sg[7] = b.w;
  }
#pragma unroll 1
  for (int r = threadIdx.x / L; r < kRows; r += kAtOnce) {
    const int row = x.row0 + r;
    if (r >= kChunkRows && x.row0 + kChunkRows >= rows) break;  // no second block (the warps agree: rows of a pass do)
    unsigned long long y[16];
    {
      const int safe = min(row, rows - 1), token = s.q0 + (safe >> p.group_shift);
      const int head = (h << p.group_shift) + (safe & (p.group - 1));
      const uint4* from = reinterpret_cast<const uint4*>(p.q + token * p.q_token + head * p.q_head + 32 * sub);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 v = __ldg(from + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * k + j;  // coordinates 2 e, 2 e + 1: sign bytes to the sign bits of the pair
          const uint32_t flip = __byte_perm(sg[e / 2], 0, (e & 1) ? 0x3424 : 0x1404) & 0x80008000u;
          const float2 f = unpack_half2(w[j] ^ flip);
          y[e] = pack2(f.x + f.y, f.x - f.y);
        }
      }
    }
#pragma unroll
    for (int step = 1; step < 16; step <<= 1) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e & step) continue;
        const unsigned long long a = y[e], c = y[e + step];
        y[e] = add2(a, c);
        y[e + step] = fma2(c, pack2(-1.f, -1.f), a);
      }
    }
#pragma unroll
    for (int step = 1; step < L; step <<= 1) {
      const float sign = sub & step ? -1.0f : 1.0f;  // the upper lane keeps the other's less its own
      const unsigned long long sign2 = pack2(sign, sign);
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = fma2(y[e], sign2, __shfl_xor_sync(0xFFFFFFFFu, y[e], step));
    }
    uint8_t* to = p.qt + (((size_t)unit * p.hkv + h) * dense_blocks(D) + r / kChunkRows) * (2 * kChunkRows * D * 2);
    const float by = row < rows ? scale : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2(mul2(y[4 * k + j], pack2(by, by)));
        hi[j] = half2_bits(f.x, f.y);
        const float2 near = unpack_half2(hi[j]);
        lo[j] = half2_bits(f.x - near.x, f.y - near.y);
      }
      const uint32_t at = tile_at(kChunkRows, r % kChunkRows, 32 * sub + 8 * k);
      *reinterpret_cast<uint4*>(to + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(to + kChunkRows * D * 2 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kPrepareThreads, 4) prepare_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int TT = dense_tile(D);
  __shared__ uint32_t s_row[TT], s_power[TT];
  __shared__ int s_tier[TT], s_bad[TT], s_tiers[TT / 32];
  __shared__ float s_max[TT / 32];
  __shared__ uint16_t tables[KVQ_MAX_TIERS][2][16];
  grid_wait();
  grid_release();
  if (threadIdx.x < KVQ_MAX_TIERS * 2 * 16) {
    const int tier = threadIdx.x / 32, side = threadIdx.x / 16 % 2, code = threadIdx.x % 16;
    float c = 0.f;
    if (tier < p.num_tiers && p.tier[tier].v_fmt == KVQ_FMT_CODEBOOK) {
      const ChunkTier& t = p.tier[tier];
      if (code < 1 << (side ? t.v_bits : t.k_bits)) c = __ldg((side ? t.v_cent : t.k_cent) + code) * p.head->beta[tier][side];
    }
    tables[tier][side][code] = __half_as_ushort(__float2half_rn(c));
  }
  __syncthreads();
  const int tiles = p.head->num_tiles * p.hkv, items = tiles + p.head->units[0] * p.hkv;
  for (int x = blockIdx.x; x < items; x += gridDim.x) {
    if (x < tiles) unpack_tile<D>(p, x / p.hkv, x % p.hkv, tables, s_row, s_power, s_tier, s_bad, s_max, s_tiers);
    else rotate_queries<D>(p, (x - tiles) / p.hkv, (x - tiles) % p.hkv);
  }
}

// ------------------------------------------------------------------------ attention
// Half a tile's weights may sum to this before m is raised (the largest fp16 is 2^16), and m is then this far
// below the largest score.
constexpr float kMostWeight = 32768.0f, kHeadroom = 2.0f;
constexpr float kNothing = -1e30f;  // m before any token is seen: finite, so that hidden scores (-inf) weigh 0

// The order of loads, the keys' KP parts one behind the other.  With two row blocks keys and values take turns; with one,
// scores run a tile further ahead, and the keys with them: K0 K1 V0 K2 V1 ...
template <int RT, int KP>
__device__ __forceinline__ constexpr int key_load(int i) { return RT == 2 ? (KP + 1) * i : (i ? KP + (KP + 1) * (i - 1) : 0); }
template <int RT, int KP>
__device__ __forceinline__ constexpr int value_load(int i, int n) {
  return RT == 2 ? (KP + 1) * i + KP : (i + 1 < n ? KP + (KP + 1) * i + KP : (KP + 1) * n - 1);
}

template <int D>
struct Shape {
  static constexpr int TT = dense_tile(D), RT = dense_blocks(D);
  static constexpr int kQBytes = 2 * kChunkRows * D * 2;  // a row block's queries, both parts
  static constexpr int kTileBytes = TT * D * 2;
  static constexpr int kBuffers = D == 64 ? 6 : 3;
  static constexpr int kNormStages = RT == 1 ? 3 : (kBuffers + 2) / 2;  // a stage is free before the keys that need it are loaded
  static constexpr int kOffRing = RT * kQBytes, kOffNorm = kOffRing + kBuffers * kTileBytes;
  static constexpr int kNormBytes = 10 * TT;  // factors of a tile's scores and of its weights (weigh)
  static constexpr int kOffCtl = kOffNorm + kNormStages * kNormBytes;
  static constexpr int kSmem = kOffCtl + 512;
  static constexpr int kThreads = RT * 128 + 64;
  // TMEM: two blocks of scores, then the accumulators
  static constexpr int kAccAt = 2 * TT, kColumns = 512;
  static_assert(kAccAt + RT * D <= kColumns, "tensor memory");
  static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};

enum { A_FULL = 0, A_EMPTY = 6, A_Q = 12, A_S = 13, A_P = 15, A_O = 17, A_DONE = 18, A_N = 19, A_COUNT = 23 };
struct AttendCtl {
  unsigned long long bars[A_COUNT];
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// An accumulator row times f.
template <int D>
__device__ __forceinline__ void scale_row(uint32_t at, float f) {
  uint32_t v[32];
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    tc_ld32(at + c, v);
    tc_wait_ld_only(v);
    uint32_t x[16], y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] = __float_as_uint(__uint_as_float(v[e]) * f);
      y[e] = __float_as_uint(__uint_as_float(v[16 + e]) * f);
    }
    tc_st16(at + c, x);
    tc_st16(at + c + 16, y);
  }
}

// A pair of fp16 numbers added to two float32 sums, without conversions between.
__device__ __forceinline__ unsigned long long add_halves(unsigned long long sum, uint32_t h) {
  float2 s = unpack2(sum);
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\nadd.rn.f32.f16 %0, lo, %0;\nadd.rn.f32.f16 %1, hi, %1;\n}"
      : "+f"(s.x), "+f"(s.y)
      : "r"(h));
  return pack2(s.x, s.y);
}

// What an item's tiles hold: values as they are; or codebooks, whose norms are factors of scores and weights, with the sum
// of the weights as they are (kCodes) or of the weights that the rounded products stand for (kCodesSummed).  Values of four
// bits take the last: a token that outweighs all others then keeps its value, 2.8e-4 of the output instead of 3.4e-4, for
// 268 instead of 250 us of a 4096-token prompt x 32 heads; those of two and three bits, whose fewer centroids lose less,
// stay below 2.9e-4 without, of one tier (337 instead of 360 us for 16 ragged chunks on 8000 tokens).
enum { kValues, kCodes, kCodesSummed };

// 32 scores -> 16 weight pairs (codebooks: times the values' factors) and their sum.  HIDE: columns that are not in `see`
// weigh nothing, whatever they hold.  fn: the factors (kCodes) or their inverses; hn: the factors as fp16, exact.
template <int KIND, bool HIDE>
__device__ __forceinline__ void weigh(const uint32_t (&v)[32], uint32_t see, float m, const float* kn, const float* fn,
                                      const uint2* hn, uint32_t* h, unsigned long long& s0, unsigned long long& s1) {
  const unsigned long long neg = pack2(-m, -m);
  auto hide = [&](unsigned long long x, int e) {
    const float2 y = unpack2(x);
    return pack2(see >> e & 1u ? y.x : 0.f, see >> (e + 1) & 1u ? y.y : 0.f);
  };
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    unsigned long long t0 = pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
    unsigned long long t1 = pack2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
    if constexpr (KIND != kValues) {  // scores are multiplied by the keys' norms
      const float4 n = *reinterpret_cast<const float4*>(kn + e);
      t0 = fma2(t0, pack2(n.x, n.y), neg);
      t1 = fma2(t1, pack2(n.z, n.w), neg);
    } else {
      t0 = add2(t0, neg);
      t1 = add2(t1, neg);
    }
    const float2 x = unpack2(t0), y = unpack2(t1);
    unsigned long long a = pack2(ex2(x.x), ex2(x.y)), b = pack2(ex2(y.x), ex2(y.y));
    if constexpr (HIDE) {
      a = hide(a, e);
      b = hide(b, e + 2);
    }
    if constexpr (KIND == kCodes) {
      s0 = add2(s0, a);
      s1 = add2(s1, b);
      const float4 n = *reinterpret_cast<const float4*>(fn + e);
      a = mul2(a, pack2(n.x, n.y));
      b = mul2(b, pack2(n.z, n.w));
    }
    if constexpr (KIND == kCodesSummed) {
      const uint2 n = hn[e / 4];
      const float2 n0 = unpack_half2(n.x), n1 = unpack_half2(n.y);
      a = mul2(a, pack2(n0.x, n0.y));
      b = mul2(b, pack2(n1.x, n1.y));
    }
    if constexpr (HIDE && KIND != kValues) {  // (a factor may be infinite)
      a = hide(a, e);
      b = hide(b, e + 2);
    }
    const float2 p = unpack2(a), q = unpack2(b);
    h[e / 2] = half2_bits(p.x, p.y);
    h[e / 2 + 1] = half2_bits(q.x, q.y);
    if constexpr (KIND != kCodes) {
      const float2 u = unpack_half2(h[e / 2]), w = unpack_half2(h[e / 2 + 1]);
      if constexpr (KIND == kCodesSummed) {
        const float4 n = *reinterpret_cast<const float4*>(fn + e);
        unsigned long long n0 = pack2(n.x, n.y), n1 = pack2(n.z, n.w);
        if constexpr (HIDE) {
          n0 = hide(n0, e);
          n1 = hide(n1, e + 2);
        }
        s0 = fma2(pack2(u.x, u.y), n0, s0);
        s1 = fma2(pack2(w.x, w.y), n1, s1);
      } else {
        s0 = add_halves(s0, h[e / 2]);
        s1 = add_halves(s1, h[e / 2 + 1]);
      }
    }
  }
}

// An accumulator row times f with the value rotation undone, as fp16: y = s H (f o).  The thread's coordinates are its
// registers: one stage of the transform after the other (head_dim 256: its last stage first, of which each half of the
// row is one result).  Lanes without an address only take part.
template <int D>
__device__ __forceinline__ void store_turned(uint32_t o_at, int part, float f, const uint4* signs, uint16_t* to) {
  constexpr int N = D == 256 ? 128 : D;
  unsigned long long y[N / 2];
  const unsigned long long f2 = pack2(f, f), g2 = pack2(part ? -f : f, part ? -f : f);
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    uint32_t v[32];
    tc_ld32(o_at + c, v);
    tc_wait_ld(v);
#pragma unroll
    for (int e = 0; e < 16; ++e) y[c / 2 + e] = mul2(pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), f2);
    if constexpr (D == 256) {
      tc_ld32(o_at + 128 + c, v);
      tc_wait_ld(v);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        y[c / 2 + e] = fma2(pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), g2, y[c / 2 + e]);
    }
  }
#pragma unroll
  for (int step = 1; step < N / 2; step <<= 1) {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      if (e & step) continue;
      const unsigned long long a = y[e], c = y[e + step];
      y[e] = add2(a, c);
      y[e + step] = fma2(c, pack2(-1.f, -1.f), a);
    }
  }
  if (!to) return;
#pragma unroll
  for (int k = 0; k < N / 16; ++k) {  // 16 coordinates
    const uint4 sg = __ldg(signs + part * (N / 16) + k);
    const uint32_t sw[4] = {sg.x, sg.y, sg.z, sg.w};
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 x = unpack2(y[8 * k + j]);
      w[j] = half2_bits(x.x + x.y, x.x - x.y) ^ (__byte_perm(sw[j / 2], 0, (j & 1) ? 0x3424 : 0x1404) & 0x80008000u);
    }
    uint4* dst = reinterpret_cast<uint4*>(to + part * N) + 2 * k;
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int D, int KIND, int KP>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) attend_kernel(const __grid_constant__ ChunkParams p) {
  using X = Shape<D>;
  constexpr bool CODES = KIND != kValues;
  constexpr int TT = X::TT, RT = X::RT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_u32(smem_raw);
  AttendCtl* ctl = reinterpret_cast<AttendCtl*>(smem_raw + X::kOffCtl);
  volatile int* abort = &ctl->abort;
  const uint32_t bars = smem + X::kOffCtl;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  grid_wait();
  grid_release();
  const int num = p.head->items[0];
  // longer items first; all heads of one unit, or (keys and values beyond L2) all units of one head side by side
  const bool by_head = (size_t)p.head->num_tiles * p.hkv * ((KP + 1) * X::kTileBytes) > ((size_t)64 << 20);
  const int at = by_head ? (int)blockIdx.x % max(1, num) : (int)blockIdx.x / p.hkv;
  const int h = by_head ? (int)blockIdx.x / max(1, num) : (int)blockIdx.x % p.hkv;
  if (at >= num || h >= p.hkv) return;
  const ChunkItem item = p.item[0][num - 1 - at];
  const ChunkSeq& s = p.seq[item.seq];
  const int n = item.count;
  int* err = &p.head->err;
  const int rows = s.tokens << p.group_shift;
  const int blocks = RT == 2 && item.row0 + kChunkRows < rows ? 2 : 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < X::kBuffers; ++i) {
      bar_init(bars + 8 * (A_FULL + i), 1);
      bar_init(bars + 8 * (A_EMPTY + i), 1);
    }
    bar_init(bars + 8 * A_Q, 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(bars + 8 * (A_S + i), 1);
      bar_init(bars + 8 * (A_P + i), 128);
    }
    for (int i = 0; i < X::kNormStages; ++i) bar_init(bars + 8 * (A_N + i), 1);
    bar_init(bars + 8 * A_O, 1);
    bar_init(bars + 8 * A_DONE, 1);
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == RT * 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem)), "n"(X::kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp < RT * 4) {
    // ---- softmax: a thread a row
    const int w = warp >> 2, r = threadIdx.x & 127;
    if (w < blocks) {
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t o_at = lane_base + X::kAccAt + w * D;
      const int row = min(item.row0 + w * kChunkRows + r, rows - 1);
      const int pos = s.len - s.tokens + (row >> p.group_shift);
      const int from = p.window ? pos - p.window + 1 : 0;
      float m = kNothing;
      unsigned long long l2 = 0;
      bool ok = true;
      const float* tops = CODES ? p.top + h : nullptr;
      auto tile_of = [&](int i) {  // of the sequence's unpacked tiles
        const int x = item.first + i;
        return x < item.sinks ? x : item.begin + x - item.sinks;
      };
      float top = 1.f, next_top = 1.f;
      if (CODES) next_top = __ldg(tops + (size_t)(s.tile0 + tile_of(0)) * p.hkv);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int x = tile_of(i), start = (x < s.sink_tiles ? x : s.window_tile + x - s.sink_tiles) * TT;
        const int b = RT == 2 ? w : i & 1;
        const uint32_t s_at = lane_base + b * TT;
        const float* kn = reinterpret_cast<const float*>(smem_raw + X::kOffNorm + i % X::kNormStages * X::kNormBytes);
        const float* fn = kn + TT;
        const uint2* hn = reinterpret_cast<const uint2*>(fn + TT);
        top = next_top;
        if (CODES && i + 1 < n) next_top = __ldg(tops + (size_t)(s.tile0 + tile_of(i + 1)) * p.hkv);
        // columns below `end`, and from `begin` on or below `first`
        const int end = pos + 1 - start, begin = from - start, first = p.sinks - start;
        const bool all = __all_sync(0xFFFFFFFFu, end >= TT && (begin <= 0 || first >= TT));
        ok = bar_wait(bars + 8 * (A_S + b), (RT == 2 ? i : i >> 1) & 1, abort, err);
        if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
        tc_fence_after();
        if (CODES) {
          ok = bar_wait(bars + 8 * (A_N + i % X::kNormStages), (i / X::kNormStages) & 1, abort, err);
          if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
        }
        auto see = [&](int c) { return below(end, c) & (~below(begin, c) | below(first, c)); };
        uint32_t g[TT / 2];
        unsigned long long sum;
        // All weights are positive: a sum of at most kMostWeight says that none is too large for fp16 either.  Only
        // where it is exceeded m is raised and the tile, still in TMEM, weighed again: of all rows of the warp.  (A sum of
        // NaN stays that.)  The first tile raises m anyway, and so does the first behind the sinks, where the maximum
        // of a few tokens would be exceeded row by row.
        bool raise = i == 0 || item.first + i == item.sinks;
#pragma unroll 1
        for (bool again = raise;; again = true) {
          uint32_t va[32], vb[32];
          if (raise) {
            const float head = kHeadroom - (float)((int)(__float_as_uint(top) >> 23) - 127);
            float mx = m;
#pragma unroll 1
            for (int c = 0; c < TT; c += 32) {
              tc_ld32(s_at + c, va);
              tc_wait_ld_only(va);
              const uint32_t sees = see(c);
              float best = -INFINITY;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float y = __uint_as_float(va[e]) * (CODES ? kn[c + e] : 1.f);
                best = fmaxf(best, all || sees >> e & 1u ? y : -INFINITY);
              }
              mx = fmaxf(mx, best - head);
            }
            const float f = ex2(m - mx);
            m = mx;
            const float2 ll = unpack2(l2);
            l2 = pack2(ll.x * f, ll.y * f);
            if (i > 0) {
              // (with two row blocks the products of earlier tiles precede these scores; with one they may still run)
              if (RT == 1 && !__all_sync(0xFFFFFFFFu, bar_wait(bars + 8 * A_O, (i - 1) & 1, abort, err))) {
                ok = false;
                break;
              }
              tc_fence_after();
              scale_row<D>(o_at, f);
            }
          }
          unsigned long long s0 = 0, s1 = 0;
          tc_ld32(s_at, va);
#pragma unroll
          for (int c = 0; c < TT; c += 64) {
            tc_wait_ld_only(va);
            tc_ld32(s_at + c + 32, vb);
            if (all) weigh<KIND, false>(va, 0, m, kn + c, fn + c, hn + c / 4, g + c / 2, s0, s1);
            else weigh<KIND, true>(va, see(c), m, kn + c, fn + c, hn + c / 4, g + c / 2, s0, s1);
            tc_wait_ld_only(vb);
            if (c + 64 < TT) tc_ld32(s_at + c + 64, va);
            if (all) weigh<KIND, false>(vb, 0, m, kn + c + 32, fn + c + 32, hn + c / 4 + 8, g + c / 2 + 16, s0, s1);
            else weigh<KIND, true>(vb, see(c + 32), m, kn + c + 32, fn + c + 32, hn + c / 4 + 8, g + c / 2 + 16, s0, s1);
          }
          sum = add2(s0, s1);
          const float2 t = unpack2(sum);
          if (again || __all_sync(0xFFFFFFFFu, !((t.x + t.y) * top > kMostWeight))) break;
          raise = true;
        }
        if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
        l2 = add2(l2, sum);
#pragma unroll
        for (int c = 0; c < TT / 2; c += 16) {  // over the scores
          uint32_t part[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) part[e] = g[c + e];
          tc_st16(s_at + c, part);
        }
        tc_wait_st();
        tc_fence_before();
        bar_arrive(bars + 8 * (A_P + b));
      }
      // all products are complete
      if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait(bars + 8 * A_DONE, 0, abort, err));
      tc_fence_after();
      const bool there = item.row0 + w * kChunkRows + r < rows;
      const float l = unpack2(l2).x + unpack2(l2).y;
      const float unscale = CODES && ok && p.codes == 1 ? p.head->unscale[0][1] : 1.f;
      if (item.part < 0) {
        // all of the row's tiles were here: the value rotation is undone in the thread's registers
        if (ok) {
          const float inv = l == 0.f ? 0.f : unscale * inv_sqrt_dim(D) / l;
          const int token = s.q0 + (row >> p.group_shift), head = (h << p.group_shift) + (row & (p.group - 1));
          uint16_t* to = p.out + token * p.out_token + head * p.out_head;
          const uint4* signs = reinterpret_cast<const uint4*>(p.v_signs + (size_t)h * D);
#pragma unroll 1
          for (int part = 0; part < (D == 256 ? 2 : 1); ++part) store_turned<D>(o_at, part, inv, signs, there ? to : nullptr);
        }
      } else {
        const size_t part = ((size_t)(item.part + w) * p.hkv + h) * kChunkRows + r;
        if (ok) {
          float* to = p.acc + part * D;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            tc_ld32(o_at + c, v);
            tc_wait_ld(v);
            if (there) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(v[e + k]) * unscale;
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + c + e),
                             "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
                             : "memory");
              }
            }
          }
        }
        // (a row of NaN has no maximum: its partial must not pass for one without tokens)
        if (there) p.ml[part] = ok && l != 0.f ? make_float2(l == l ? m : l, l) : make_float2(-INFINITY, 0.f);
      }
    }
  } else if (warp == RT * 4) {
    // ---- products: the whole warp walks, one lane issues
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    constexpr uint32_t kIdescS = (1u << 4) | ((TT >> 3) << 17) | ((kChunkRows >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((D >> 3) << 17) | ((kChunkRows >> 4) << 24);
    const uint64_t qd = desc_at(desc_base(16, 1024), smem), kd = desc_at(desc_base(16, 1024), smem + X::kOffRing);
    const uint64_t vd = desc_at(desc_base(TT * 128, 1024), smem + X::kOffRing);
    auto well = [&](uint32_t bar, uint32_t parity) -> bool {
      return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, abort, err));
    };
    auto full = [&](int load) { return well(bars + 8 * (A_FULL + load % X::kBuffers), (load / X::kBuffers) & 1); };
    auto keys_full = [&](int i) {
      bool ok = full(key_load<RT, KP>(i));
      if (KP == 2) ok = ok && full(key_load<RT, KP>(i) + 1);
      return ok;
    };
    auto scores = [&](int block, int i, int buffer) {  // of row block `block` and tile i
      // the queries' two parts with the keys, and of keys of two parts the first with the second
#pragma unroll 1
      for (int part = 0; part < KP + 1; ++part) {
        const uint64_t a = qd + ((block * X::kQBytes + (part & 1) * (X::kQBytes / 2)) >> 4);
        const uint64_t b = kd + ((key_load<RT, KP>(i) + (part >> 1)) % X::kBuffers) * (X::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tm + buffer * TT, a + (((kk >> 2) * (kChunkRows * 128) + (kk & 3) * 32) >> 4),
                 b + (((kk >> 2) * (TT * 128) + (kk & 3) * 32) >> 4), kIdescS, part + kk > 0);
      }
      tc_commit(bars + 8 * (A_S + buffer));
    };
    auto values = [&](int block, int i, int buffer) {
      const uint64_t b = vd + (value_load<RT, KP>(i, n) % X::kBuffers) * (X::kTileBytes >> 4);
#pragma unroll
      for (int kk = 0; kk < TT / 16; ++kk)
        mma_ts(tm + X::kAccAt + block * D, tm + buffer * TT + kk * 8, b + ((kk * 2048) >> 4), kIdescO, i > 0 || kk > 0);
    };
    auto free_buffer = [&](int load) { tc_commit(bars + 8 * (A_EMPTY + load % X::kBuffers)); };
    auto free_keys = [&](int i) {
      for (int part = 0; part < KP; ++part) free_buffer(key_load<RT, KP>(i) + part);
    };
    bool ok = well(bars + 8 * A_Q, 0) && keys_full(0);
    if (ok) {
      tc_fence_after();
      if (elect_one()) {
        for (int b = 0; b < blocks; ++b) scores(b, 0, b);
        free_keys(0);
      }
      __syncwarp();
    }
    if (RT == 1 && ok && n > 1 && (ok = keys_full(1))) {
      tc_fence_after();
      if (elect_one()) {
        scores(0, 1, 1);
        free_keys(1);
      }
      __syncwarp();
    }
    for (int i = 0; i < n && ok; ++i) {
      const bool more = i + 1 < n;
      if constexpr (RT == 2) {
        for (int b = 0; b < blocks && ok; ++b) {
          if (b == 0) ok = full(value_load<RT, KP>(i, n));
          ok = ok && well(bars + 8 * (A_P + b), i & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            values(b, i, b);
            if (b + 1 == blocks) free_buffer(value_load<RT, KP>(i, n));
          }
          __syncwarp();
          if (!more) continue;
          if (b == 0 && !(ok = keys_full(i + 1))) break;
          tc_fence_after();
          if (elect_one()) {
            scores(b, i + 1, b);
            if (b + 1 == blocks) free_keys(i + 1);
          }
          __syncwarp();
        }
      } else {
        ok = full(value_load<RT, KP>(i, n)) && well(bars + 8 * (A_P + (i & 1)), (i >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          values(0, i, i & 1);
          free_buffer(value_load<RT, KP>(i, n));
          tc_commit(bars + 8 * A_O);
        }
        __syncwarp();
        if (i + 2 < n) {
          if (!(ok = keys_full(i + 2))) break;
          tc_fence_after();
          if (elect_one()) {
            scores(0, i + 2, i & 1);
            free_keys(i + 2);
          }
          __syncwarp();
        }
      }
    }
    // everything issued is over before tensor memory and the operands go
    if (elect_one()) tc_commit(bars + 8 * A_DONE);
    __syncwarp();
    for (int i = 0; i < 1 << 22 && !bar_try(bars + 8 * A_DONE, 0); ++i) {
    }
  } else {
    // ---- loads, one lane
    int issued = 0, norms = 0;
    if ((threadIdx.x & 31) == 0) {
      const uint32_t q_bytes = blocks * X::kQBytes;
      const uint8_t* q = p.qt + ((size_t)(s.unit0 + item.row0 / (kChunkRows * RT)) * p.hkv + h) * (RT * X::kQBytes);
      bar_expect(bars + 8 * A_Q, q_bytes);
      bulk_load(smem, q, q_bytes, bars + 8 * A_Q);
      bool ok = true;
      for (int load = 0; load < (KP + 1) * n && ok; ++load) {
        // tile and part of this load: the keys' parts, then the values (key_load, value_load)
        const int turns = RT == 2 ? load : load - KP, step = turns >= 0 ? turns / (KP + 1) : -1;
        int part = turns - step * (KP + 1), i = RT == 2 ? step : step + 1;
        if (RT == 1 && load < KP) part = load;
        if (RT == 1 && load >= KP) i -= part == KP;  // values of the tile before
        if (RT == 1 && load == (KP + 1) * n - 1) part = KP, i = n - 1;
        const bool value = part == KP;
        const int x = item.first + i, slot = load % X::kBuffers, turn = load / X::kBuffers;
        const size_t tile = (size_t)(s.tile0 + (x < item.sinks ? x : item.begin + x - item.sinks)) * p.hkv + h;
        if (turn > 0 && !(ok = bar_wait(bars + 8 * (A_EMPTY + slot), (turn - 1) & 1, abort, err))) break;
        const uint32_t bar = bars + 8 * (A_FULL + slot);
        bar_expect(bar, X::kTileBytes);
        bulk_load(smem + X::kOffRing + slot * X::kTileBytes, value ? p.vt + tile * X::kTileBytes : p.kt + (tile * KP + part) * X::kTileBytes,
                  X::kTileBytes, bar);
        if (CODES && part == 0) {  // (a stage's norms have been read: the keys' buffer waits for later products)
          const uint32_t to = smem + X::kOffNorm + i % X::kNormStages * X::kNormBytes, nbar = bars + 8 * (A_N + i % X::kNormStages);
          bar_expect(nbar, (KIND == kCodesSummed ? 10 : 8) * TT);
          bulk_load(to, p.kn + tile * TT, TT * 4, nbar);
          bulk_load(to + TT * 4, p.fn + tile * TT, TT * 4, nbar);
          if (KIND == kCodesSummed) bulk_load(to + TT * 8, p.hn + tile * TT, TT * 2, nbar);
          norms = i + 1;
        }
        issued = load + 1;
      }
      // no copy is under way when the block ends
      for (int i = 0; i < 1 << 22 && !bar_try(bars + 8 * A_Q, 0); ++i) {
      }
      for (int i = max(0, norms - X::kNormStages); i < norms; ++i)
        for (int k = 0; k < 1 << 22 && !bar_try(bars + 8 * (A_N + i % X::kNormStages), (i / X::kNormStages) & 1); ++k) {
        }
      for (int load = max(0, issued - X::kBuffers); load < issued; ++load)
        for (int i = 0; i < 1 << 22 && !bar_try(bars + 8 * (A_FULL + load % X::kBuffers), (load / X::kBuffers) & 1); ++i) {
        }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == RT * 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(X::kColumns));
}

template <int D, int KIND, int KP = 1>
cudaError_t launch_attend(const ChunkParams& p, cudaStream_t stream) {
  auto kern = attend_kernel<D, KIND, KP>;
  static std::atomic<bool> configured[64];  // shared-memory limit raised on this device (a racing second raise is
                                            // harmless)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  const long long grid = (long long)p.max_items[0] * p.hkv;
  return launch_dependent(reinterpret_cast<const void*>(kern), (unsigned)grid, Shape<D>::kThreads, Shape<D>::kSmem, p, stream);
}

}  // namespace

cudaError_t launch_chunk_prepare(const ChunkParams& p, cudaStream_t stream) {
  const long long items = ((long long)p.max_tiles + p.max_units[0]) * p.hkv;
  const unsigned grid = (unsigned)std::max(1LL, std::min(items, p.sms * 8LL));
  const void* k = p.head_dim == 64    ? reinterpret_cast<const void*>(prepare_kernel<64>)
                  : p.head_dim == 128 ? reinterpret_cast<const void*>(prepare_kernel<128>)
                                      : reinterpret_cast<const void*>(prepare_kernel<256>);
  return launch_dependent(k, grid, kPrepareThreads, 0, p, stream);
}

cudaError_t launch_chunk_dense(const ChunkParams& p, cudaStream_t stream) {
  auto kind = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (!p.codes) return launch_attend<D, kValues>(p, stream);
    if constexpr (D != 64) {  // (such keys are of 128 or 256 coordinates, with codebook values)
      if (p.key_parts == 2) return p.summed ? launch_attend<D, kCodesSummed, 2>(p, stream) : launch_attend<D, kCodes, 2>(p, stream);
    }
    return p.summed ? launch_attend<D, kCodesSummed>(p, stream) : launch_attend<D, kCodes>(p, stream);
  };
  if (p.head_dim == 64) return kind(std::integral_constant<int, 64>{});
  if (p.head_dim == 128) return kind(std::integral_constant<int, 128>{});
  return kind(std::integral_constant<int, 256>{});
}

}  // namespace kvq
