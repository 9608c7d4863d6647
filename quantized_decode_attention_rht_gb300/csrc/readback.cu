// Cached tokens read back as fp16 vectors (kvq_dequantize).
//
// With the stored rotated vector x~ = H s x / sqrt(D), x = s H x~ / sqrt(D).  H is a product of
// one butterfly stage per bit of the coordinate's index, in any order: four of them (the two
// that a lane number selects and two inside a lane) are one product with the 16 x 16 matrix
// (-1)^popc(m & k) on the tensor cores, the others run on the product's float32 results in
// registers.  A warp takes eight vectors (head_dim 256: four, their halves being columns of
// their own) of one head and neighbouring tokens; the product's operand and result layouts
// make every lane read 2 x 2T neighbouring coordinates (T = 8 result tiles; 4 for head_dim 64) of
// one vector and end with 2T neighbouring ones of two, so nothing passes through shared memory.
//
// The product multiplies fp16 and adds in float32.  Nothing is lost: fp16 and fp8 rows are fp16
// values; an INT4 level times its scale and a centroid are the sum of two fp16 numbers, the
// first the nearest one (levels exactly, centroids to 2^-22), and go in as two products.
// Norms and 1 / sqrt(D) are applied in float32 behind it.
//
// What bounds it is memory: the next vectors' rows are on their way while these are worked on.
// 65536 tokens x 8 heads of fp8 keys and INT4 values (373 MB): 67.8 us, 81% of the measured copy rate,
// with six blocks of 128 threads an SM (80 registers; five 71.5, eight, which spill, 91.4).  With the
// transposes in shared memory it took 93.5.
#include <algorithm>

#include "api_checks.cuh"
#include "quantize.cuh"

namespace kvq {
namespace {

struct ReadSide {
  const uint8_t* rows;
  const __half* aux;
  const float* cent;
  const int8_t* signs;
  const float* qjl;
  const int32_t* outl;
  uint16_t* out;  // null: the side is not wanted
  int fmt, bits, row_bytes;
};
struct ReadParams {
  ReadSide side[2];
  const int32_t* slots;
  int num_tokens, hkv, page_size, page_shift, num_slots;
  int kind_first;
};

// y = centroids of the thread's 32 codes.
template <int BITS>
__device__ __forceinline__ void decode_codes(const uint8_t* row, const float* cent, float (&y)[32]) {
  uint32_t w[BITS + 1];
  if constexpr (BITS == 4) {
    *reinterpret_cast<uint4*>(w) = __ldcs(reinterpret_cast<const uint4*>(row));
  } else if constexpr (BITS == 2) {
    *reinterpret_cast<uint2*>(w) = __ldcs(reinterpret_cast<const uint2*>(row));
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k) w[k] = __ldcs(reinterpret_cast<const uint32_t*>(row) + k);
  }
  w[BITS] = 0u;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const int at = e * BITS;
    const uint32_t f = at % 32 + BITS <= 32 ? w[at / 32] >> (at % 32)
                                            : __funnelshift_r(w[at / 32], w[at / 32 + 1], at % 32);
    y[e] = cent[f & ((1u << BITS) - 1u)];
  }
}

// The thread's coordinates [32 sub, 32 sub + 32) of the rotated vector.
template <int TPV>
__device__ __forceinline__ void decode_row(const ReadSide& s, size_t prow, int sub, const float* cent,
                                           float (&y)[32]) {
  constexpr int D = 32 * TPV;
  const uint8_t* row = s.rows + prow * s.row_bytes;
  float scale;
  switch (s.fmt) {
    case KVQ_FMT_FP16: {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + 64 * sub) + k);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          y[8 * k + 2 * j] = f.x;
          y[8 * k + 2 * j + 1] = f.y;
        }
      }
      return;
    }
    case KVQ_FMT_FP8_E4M3: {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + 32 * sub) + k);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t h2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[j / 2] >> (16 * (j & 1)))));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          y[16 * k + 2 * j] = f.x;
          y[16 * k + 2 * j + 1] = f.y;
        }
      }
      return;
    }
    case KVQ_FMT_INT4_G32: {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + 16 * sub));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      scale = __half2float(s.aux[prow * (D / kGroup) + sub]);
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] = scale * (float)((int)((w[e / 8] >> (4 * (e % 8))) & 15u) - 8);
      return;
    }
    default: break;
  }
  if (s.bits == 4) decode_codes<4>(row + 16 * sub, cent, y);
  else if (s.bits == 3) decode_codes<3>(row + 12 * sub, cent, y);
  else decode_codes<2>(row + 8 * sub, cent, y);
  if (s.fmt == KVQ_FMT_CODEBOOK) scale = __half2float(s.aux[prow]);
  else if (s.fmt == KVQ_FMT_CODEBOOK_QJL) scale = __half2float(s.aux[2 * prow]);
  else scale = __half2float(*reinterpret_cast<const __half*>(reinterpret_cast<const uint8_t*>(s.aux) +
                                                             prow * (4 + KVQ_OUTLIER_CHANNELS)));
  scale *= inv_sqrt_dim(D);
#pragma unroll
  for (int e = 0; e < 32; ++e) y[e] *= scale;
  if (s.fmt == KVQ_FMT_CODEBOOK_QJL) {
    // + ||r|| sqrt(pi / 2) / m * sum_j z_j S_j: the projection rows stay in L1 / L2
    const float c = __half2float(s.aux[2 * prow + 1]) * (1.2533141373155003f / KVQ_QJL_DIM);
    const uint32_t* z = reinterpret_cast<const uint32_t*>(row + D * s.bits / 8);
    float r[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) r[e] = 0.f;
    for (int j = 0; j < KVQ_QJL_DIM; ++j) {
      const float4* sj = reinterpret_cast<const float4*>(s.qjl + (size_t)j * D + 32 * sub);
      const uint32_t flip = ((__ldg(z + j / 32) >> (j % 32)) & 1u) ? 0u : 0x80000000u;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 v = __ldg(sj + k);
        r[4 * k] += __uint_as_float(__float_as_uint(v.x) ^ flip);
        r[4 * k + 1] += __uint_as_float(__float_as_uint(v.y) ^ flip);
        r[4 * k + 2] += __uint_as_float(__float_as_uint(v.z) ^ flip);
        r[4 * k + 3] += __uint_as_float(__float_as_uint(v.w) ^ flip);
      }
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) y[e] = fmaf(c, r[e], y[e]);
  }
}

// Caches whose keys carry a residual sketch or an outlier stream: D / 32 neighbouring lanes share a
// vector, each decoding 32 neighbouring coordinates (and adding the sketch's estimate to them);
// five stages run in its registers, one transpose through shared memory hands it the runs for the
// others.  Bounded by the sketch's arithmetic (128 projection rows a vector).
template <int TPV>
__global__ void __launch_bounds__(kThreads, 2) read_extra_kernel(const ReadParams p) {
  constexpr int D = 32 * TPV, R = 32 / TPV, VPB = kThreads / TPV;
  extern __shared__ __align__(16) float area_all[];  // D floats per vector of the block
  __shared__ float cent[16];
  const ReadSide side = (p.kind_first + blockIdx.y) ? p.side[1] : p.side[0];
  if (side.cent && threadIdx.x < 16) cent[threadIdx.x] = (int)threadIdx.x < (1 << side.bits) ? side.cent[threadIdx.x] : 0.f;
  __syncthreads();
  const int lane = threadIdx.x & 31, sub = lane % TPV, vw = lane / TPV;
  const unsigned gmask = ((1u << TPV) - 1u) << (lane - sub);
  const uint32_t area =
      static_cast<uint32_t>(__cvta_generic_to_shared(area_all)) + (uint32_t)(threadIdx.x / TPV) * (D * 4);
  const long long nvec = (long long)p.num_tokens * p.hkv, stride = (long long)gridDim.x * VPB;
  for (long long v = (long long)blockIdx.x * VPB + threadIdx.x / TPV; v < nvec; v += stride) {
    const int token = (int)(v / p.hkv), h = (int)(v - (long long)token * p.hkv);
    const int slot = __ldg(p.slots + token);
    if (slot < 0 || slot >= p.num_slots) continue;  // the vector's lanes agree
    const int page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size;
    const size_t prow = ((size_t)page * p.hkv + h) * p.page_size + (slot - page * p.page_size);
    float y[32];
    decode_row<TPV>(side, prow, sub, cent, y);
    // index bits 0 .. 4
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float a = y[e], c = y[e + 1];
      y[e] = a + c;
      y[e + 1] = a - c;
    }
#pragma unroll
    for (int hs = 2; hs < 32; hs <<= 1) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        if ((e & hs) == 0) {
          const u64 a = pk(y[e], y[e + 1]), c = pk(y[e + hs], y[e + hs + 1]);
          upk(add2(a, c), y[e], y[e + 1]);
          upk(sub2(a, c), y[e + hs], y[e + hs + 1]);
        }
      }
    }
    __syncwarp(gmask);  // the group's reads of the previous vector are done
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t col = (uint32_t)j ^ swz<TPV>(sub, vw);
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(area + 16u * (8u * sub + col)), "f"(y[4 * j]),
                   "f"(y[4 * j + 1]), "f"(y[4 * j + 2]), "f"(y[4 * j + 3])
                   : "memory");
    }
    __syncwarp(gmask);
#pragma unroll
    for (int k = 0; k < TPV; ++k) {
#pragma unroll
      for (int q = 0; q < R / 4; ++q) {
        const uint32_t col = ((uint32_t)((R / 4) * sub + q)) ^ swz<TPV>(k, vw);
        const int e = k * R + 4 * q;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(y[e]), "=f"(y[e + 1]), "=f"(y[e + 2]), "=f"(y[e + 3])
                     : "r"(area + 16u * (8u * k + col))
                     : "memory");
      }
    }
    // index bits 5 ..: runs k of the vector
#pragma unroll
    for (int hs = R; hs < 32; hs <<= 1) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        if ((e & hs) == 0) {
          const u64 a = pk(y[e], y[e + 1]), c = pk(y[e + hs], y[e + hs + 1]);
          upk(add2(a, c), y[e], y[e + 1]);
          upk(sub2(a, c), y[e + hs], y[e + hs + 1]);
        }
      }
    }
    uint32_t sw[8];
    load_signs<TPV>(side.signs + (size_t)h * D, sub, sw);
    constexpr float inv = inv_sqrt_dim(D);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint32_t neg = (sw[e / 4] << (24 - 8 * (e % 4))) & 0x80000000u;
      y[e] = __uint_as_float(__float_as_uint(y[e] * inv) ^ neg);
    }
    if (side.fmt == KVQ_FMT_CODEBOOK_OUTLIER) {  // + q_j s at channel c_j
      const uint8_t* rec = reinterpret_cast<const uint8_t*>(side.aux) + prow * (4 + KVQ_OUTLIER_CHANNELS);
      const float s = __half2float(*reinterpret_cast<const __half*>(rec + 2));
      for (int j = 0; j < KVQ_OUTLIER_CHANNELS; ++j) {
        const int c = __ldg(side.outl + h * KVQ_OUTLIER_CHANNELS + j);
        const float add = s * (float)reinterpret_cast<const int8_t*>(rec)[4 + j];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (c == 32 * (e / R) + R * sub + e % R) y[e] += add;
      }
    }
    uint16_t* dst = side.out + (size_t)v * D;
#pragma unroll
    for (int k = 0; k < TPV; ++k) {
      uint32_t w[R / 2];
#pragma unroll
      for (int i = 0; i < R / 2; ++i) {
        const __half2 h2 = __floats2half2_rn(y[k * R + 2 * i], y[k * R + 2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      uint16_t* run = dst + 32 * k + R * sub;
      if constexpr (R == 4) {
        *reinterpret_cast<uint2*>(run) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int i = 0; i < R / 8; ++i)
          reinterpret_cast<uint4*>(run)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      }
    }
  }
}

// ------------------------------------------------------------------------ plain formats
enum { R_F16, R_F8, R_I4, R_C4, R_C3, R_C2 };
constexpr int kReadThreads = 128, kReadBlocks = 6;  // blocks an SM

__host__ __device__ constexpr int code_bits(int kind) { return kind == R_C4 ? 4 : (kind == R_C3 ? 3 : 2); }
// Bytes of a lane's coordinates in a row, and the registers that hold them.
__host__ __device__ constexpr int lane_bytes(int kind, int n) {
  return kind == R_F16 ? 2 * n : (kind == R_F8 ? n : (kind == R_I4 || kind == R_C4 ? n / 2 : n * code_bits(kind) / 8));
}
__host__ __device__ constexpr int lane_words(int kind, int n) { return (lane_bytes(kind, n) + 3) / 4; }

template <int BYTES>
__device__ __forceinline__ void load_bytes(const uint8_t* src, uint32_t* w) {
  if constexpr (BYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(src) + i);
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
  } else if constexpr (BYTES == 8) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(src));
    w[0] = u.x;
    w[1] = u.y;
  } else if constexpr (BYTES % 4 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) w[i] = __ldcs(reinterpret_cast<const uint32_t*>(src) + i);
  } else {  // 6 bytes: 3-bit codes of head_dim 64
    const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
    w[0] = (uint32_t)__ldcs(h) | ((uint32_t)__ldcs(h + 1) << 16);
    w[1] = __ldcs(h + 2);
  }
}

__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }

// The operand words of coordinates (c, c + 2T) of the lane: their fp16 value, or the nearest one
// (hi) and the rest (lo).  w: the lane's packed coordinates; scale: INT4's, twice.
template <int KIND, int T>
__device__ __forceinline__ void operand(const uint32_t* w, int c, __half2 scale, const uint32_t* table, uint32_t& hi,
                                        uint32_t& lo) {
  if constexpr (KIND == R_F16) {
    hi = __byte_perm(w[c / 2], w[c / 2 + T], c % 2 ? 0x7632 : 0x5410);
  } else if constexpr (KIND == R_F8) {
    const uint32_t two = __byte_perm(w[c / 4], w[c / 4 + T / 2], (uint32_t)(c % 4) | ((uint32_t)(c % 4 + 4) << 4));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)two));
  } else if constexpr (KIND == R_I4) {
    constexpr int kFar = T == 8 ? 2 : 1;  // words from c's to (c + 2T)'s
    const uint32_t both = __byte_perm(w[c / 8], w[c / 8 + kFar], c % 8 < 4 ? 0x5410 : 0x7632);
    const __half2 level = __hsub2(half2_of(((both >> (4 * (c % 4))) & 0x000F000Fu) | 0x64006400u),
                                  __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408)));
    const __half2 x = __hmul2(level, scale);
    hi = bits_of(x);
    lo = bits_of(__hfma2(level, scale, __hneg2(x)));  // exact: 15 bits of product, 11 taken
  } else {
    constexpr int B = code_bits(KIND);
    uint32_t e[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (c + 2 * T * i) * B;
      const uint32_t f = at % 32 + B <= 32 ? w[at / 32] >> (at % 32) : __funnelshift_r(w[at / 32], w[at / 32 + 1], at % 32);
      e[i] = table[f & ((1u << B) - 1u)];
    }
    hi = __byte_perm(e[0], e[1], 0x5410);
    lo = __byte_perm(e[0], e[1], 0x7632);
  }
}

__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2 x 16 bytes, in one store where the address allows it.
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&w)[8], bool aligned32) {
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Lane (g, q) = (lane / 4, lane % 4).  With k the bits of a row of the operand and m those of a
// result row, k bit 0 (the two halves of a word) is coordinate bit log2(2T), k bits 1, 2 (q) the
// two bits above it, k bit 3 (the two words) coordinate bit log2(T), the tile the bits below:
// lane q reads coordinates [4T q, 4T q + 4T) of column g's vector, and result rows g and g + 8 of
// all tiles are coordinates [2T g, 2T g + 2T) of columns 2q and 2q + 1.
template <int D, int KIND>
__device__ __forceinline__ void read_side(const ReadParams& p, const ReadSide& side, uint32_t* table) {
  constexpr int T = D == 64 ? 4 : 8, kRun = 4 * T, kWords = lane_words(KIND, kRun);
  constexpr int kHalves = D == 256 ? 2 : 1, kTokens = 8 / kHalves;  // columns a token takes, tokens of a warp
  constexpr bool kCodes = KIND >= R_C4;
  constexpr float inv = inv_sqrt_dim(D);
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  float unit = inv;
  if constexpr (kCodes) {
    // centroids times a power of two that takes the largest to [2^9, 2^10): neither part leaves
    // fp16's normal range, unless it is below 2^-10 of the largest centroid's rounding
    constexpr int n = 1 << code_bits(KIND);
    float most = 0.f;
    for (int i = 0; i < n; ++i) most = fmaxf(most, fabsf(__ldg(side.cent + i)));
    int e = 0;
    if (most > 0.f && most < INFINITY) frexpf(most, &e);
    const int up = max(-100, min(100, 10 - e));
    if (threadIdx.x < n) {
      const float c = ldexpf(__ldg(side.cent + threadIdx.x), up);
      const __half hi = __float2half_rn(c);
      table[threadIdx.x] = bits_of(__halves2half2(hi, __float2half_rn(c - __half2float(hi))));
    }
    unit = inv * inv * ldexpf(1.0f, -up);
    __syncthreads();
  }
  // rows g and g + 8, columns (2q, 2q + 1) and those + 8 of (-1)^popc(m & k)
  uint32_t a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = g + (i & 1) * 8, k = 2 * q + (i >> 1) * 8;
    a[i] = 0x3C003C00u | ((uint32_t)(__popc(m & k) & 1) << 15) | ((uint32_t)(__popc(m & (k + 1)) & 1) << 31);
  }
  const int my_token = g / kHalves, my_half = kHalves == 2 ? g & 1 : 0;
  const bool wide = (reinterpret_cast<uintptr_t>(side.out) & 31) == 0;
  // Items: kTokens tokens of a head; neighbouring warps take neighbouring heads of the same tokens.
  // (below 2^32, as the host checks; the step in tokens and heads is divided out once)
  const uint32_t hkv = p.hkv, stride = gridDim.x * (kReadThreads / 32);
  const uint32_t step_tokens = stride / hkv * kTokens, step_heads = stride % hkv;
  struct At {
    long long token;  // the first
    uint32_t head;
  };
  auto advance = [&](At& at) {
    at.token += step_tokens;
    if ((at.head += step_heads) >= hkv) {
      at.head -= hkv;
      at.token += kTokens;
    }
  };
  auto slot_of = [&](const At& at) -> int {
    const long long t = at.token + my_token;
    const int slot = t < p.num_tokens ? __ldg(p.slots + t) : -1;
    return slot < p.num_slots ? slot : -1;
  };
  struct Fetched {
    uint32_t w[kWords + (KIND == R_C3 ? 1 : 0)];
    __half aux;
  };
  auto fetch = [&](const At& at, int slot, Fetched& f) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(f.w) / 4); ++i) f.w[i] = 0u;
    f.aux = __ushort_as_half(0);
    if (slot < 0) return;
    const int page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size;
    const size_t prow = ((size_t)page * p.hkv + at.head) * p.page_size + (slot - page * p.page_size);
    const int part = 4 * my_half + q;  // of the row, in runs
    load_bytes<lane_bytes(KIND, kRun)>(side.rows + prow * side.row_bytes + part * lane_bytes(KIND, kRun), f.w);
    if constexpr (KIND == R_I4) f.aux = side.aux[prow * (D / kGroup) + part * kRun / kGroup];
    if constexpr (kCodes) f.aux = side.aux[prow];
  };

  const uint32_t first = blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5);
  At here = {(long long)(first / hkv) * kTokens, first % hkv}, then = here, later;
  advance(then);
  int slot = slot_of(here), next_slot = slot_of(then);
  Fetched cur, next;
  fetch(here, slot, cur);
  while (here.token < p.num_tokens) {
    fetch(then, next_slot, next);
    later = then;
    advance(later);
    const int after = slot_of(later);
    const uint32_t there = __ballot_sync(0xFFFFFFFFu, slot >= 0);
    __half2 scale = __half2half2(cur.aux);
    uint32_t big = 0;  // lanes of vectors with a scale whose products could leave fp16: an eighth of it
    if constexpr (KIND == R_I4) {
      big = __ballot_sync(0xFFFFFFFFu, __half2float(cur.aux) > 8000.0f);
      constexpr uint32_t kOwn = kHalves == 2 ? 0xFFu : 0xFu;
      if (big & (kOwn << (4 * (g / kHalves * kHalves)))) scale = __hmul2(scale, __float2half2_rn(0.125f));
    }
    float c[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      uint32_t h0, h1, l0, l1;
      operand<KIND, T>(cur.w, t, scale, table, h0, l0);
      operand<KIND, T>(cur.w, t + T, scale, table, h1, l1);
      c[t][0] = c[t][1] = c[t][2] = c[t][3] = 0.f;
      mma16(c[t], a, h0, h1);
      if constexpr (KIND >= R_I4) mma16(c[t], a, l0, l1);
    }
    u64 y[2][T];  // result rows g, g + 8: columns (2q, 2q + 1)
#pragma unroll
    for (int t = 0; t < T; ++t) {
      y[0][t] = pk(c[t][0], c[t][1]);
      y[1][t] = pk(c[t][2], c[t][3]);
    }
#pragma unroll
    for (int hs = 1; hs < T; hs <<= 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
          if ((t & hs) == 0) {
            const u64 u = y[i][t], v = y[i][t + hs];
            y[i][t] = add2(u, v);
            y[i][t + hs] = sub2(u, v);
          }
        }
      }
    }
    // what the columns are multiplied by
    float s0 = unit, s1 = unit;
    if constexpr (kCodes) {
      s0 *= __shfl_sync(0xFFFFFFFFu, __half2float(cur.aux), 8 * q);
      s1 *= __shfl_sync(0xFFFFFFFFu, __half2float(cur.aux), 8 * q + 4);
    }
    if constexpr (KIND == R_I4) {
      if (kHalves == 2) {
        if (big & (0xFFu << (8 * q))) s0 = s1 = 8.0f * unit;
      } else {
        if (big & (0xFu << (8 * q))) s0 = 8.0f * unit;
        if (big & (0xFu << (8 * q + 4))) s1 = 8.0f * unit;
      }
    }
    const u64 s2 = pk(s0, s1);
    const uint32_t h = here.head;
    float z[2][2 * T];  // the columns' runs
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float u, v;
        upk(mul2(y[i][t], s2), u, v);
        z[0][i * T + t] = kHalves == 2 ? u + v : u;  // the stage of coordinate bit 7
        z[1][i * T + t] = kHalves == 2 ? u - v : v;
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int token = kHalves == 2 ? q : 2 * q + k, at = (kHalves == 2 ? k * 128 : 0) + 2 * T * g;
      uint32_t sw[T / 2];  // sign bytes of the run
      const int8_t* signs = side.signs + (size_t)h * D + at;
      if constexpr (T == 8) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(signs));
        sw[0] = u.x;
        sw[1] = u.y;
        sw[2] = u.z;
        sw[3] = u.w;
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(signs));
        sw[0] = u.x;
        sw[1] = u.y;
      }
      uint32_t w[T];
#pragma unroll
      for (int j = 0; j < T; ++j) {
        const __half2 h2 = __floats2half2_rn(z[k][2 * j], z[k][2 * j + 1]);
        w[j] = bits_of(h2) ^ (__byte_perm(sw[j >> 1], 0, (j & 1) ? 0x3424 : 0x1404) & 0x80008000u);
      }
      if (!((there >> (4 * kHalves * token)) & 1u)) continue;
      uint16_t* dst = side.out + ((size_t)(here.token + token) * hkv + h) * D + at;
      if constexpr (T == 8) store32(dst, w, wide);
      else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    here = then;
    then = later;
    cur = next;
    slot = next_slot;
    next_slot = after;
  }
}

// Grid row blockIdx.y: side kind_first + y.
template <int D>
__global__ void __launch_bounds__(kReadThreads, kReadBlocks) read_kernel(const ReadParams p) {
  __shared__ uint32_t table[16];
  const ReadSide& side = p.side[p.kind_first + blockIdx.y];
  switch (side.fmt) {
    case KVQ_FMT_FP16: read_side<D, R_F16>(p, side, table); break;
    case KVQ_FMT_FP8_E4M3: read_side<D, R_F8>(p, side, table); break;
    case KVQ_FMT_INT4_G32: read_side<D, R_I4>(p, side, table); break;
    default:
      if (side.bits == 4) read_side<D, R_C4>(p, side, table);
      else if (side.bits == 3) read_side<D, R_C3>(p, side, table);
      else read_side<D, R_C2>(p, side, table);
  }
}

template <int D>
cudaError_t launch_read(const ReadParams& p, int sides, int sms, cudaStream_t stream) {
  const int kf = p.kind_first == 0 ? p.side[0].fmt : KVQ_FMT_CODEBOOK;
  if (kf == KVQ_FMT_CODEBOOK_QJL || kf == KVQ_FMT_CODEBOOK_OUTLIER) {
    if constexpr (D != 64) {  // (such keys have head_dim 128 or 256)
      constexpr int VPB = kThreads / (D / 32);
      const long long nvec = (long long)p.num_tokens * p.hkv;
      const long long blocks = std::max<long long>(1, std::min<long long>((nvec + VPB - 1) / VPB, sms * 2LL / sides));
      read_extra_kernel<D / 32><<<dim3((unsigned)blocks, sides), kThreads, kXposeBytes, stream>>>(p);
    }
  } else {
    constexpr int kTokens = D == 256 ? 4 : 8, kWarps = kReadThreads / 32;
    const long long items = ((long long)p.num_tokens + kTokens - 1) / kTokens * p.hkv;
    const long long blocks =
        std::max<long long>(1, std::min<long long>((items + kWarps - 1) / kWarps, (long long)sms * kReadBlocks / sides));
    read_kernel<D><<<dim3((unsigned)blocks, sides), kReadThreads, 0, stream>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace
}  // namespace kvq

extern "C" KVQ_API kvq_status kvq_dequantize(const kvq_cache* cache, const int32_t* slots, int32_t num_tokens,
                                             uint16_t* k_out, uint16_t* v_out, void* stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (num_tokens < 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return KVQ_OK;
  if (!k_out && !v_out) return KVQ_ERR_INVALID_ARGUMENT;
  if (!slots || !aligned(slots, 4) || (k_out && !aligned(k_out, 16)) || (v_out && !aligned(v_out, 16)))
    return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_cache* c = cache;
  if (k_out && (st = check_side(c, c->k_format, c->k_bits, c->k_rows, c->k_aux, c->k_centroids, c->k_bounds,
                                c->k_signs, false, true)) != KVQ_OK)
    return st;
  if (v_out && (st = check_side(c, c->v_format, c->v_bits, c->v_rows, c->v_aux, c->v_centroids, c->v_bounds,
                                c->v_signs, false, false)) != KVQ_OK)
    return st;
  // sign runs are read in pieces of up to 16 bytes
  if ((k_out && !aligned(c->k_signs, 16)) || (v_out && !aligned(c->v_signs, 16))) return KVQ_ERR_INVALID_ARGUMENT;
  ReadParams p;
  memset(&p, 0, sizeof(p));
  const int fmts[2] = {c->k_format, c->v_format}, bits[2] = {c->k_bits, c->v_bits};
  const void* rows[2] = {c->k_rows, c->v_rows};
  const void* aux[2] = {c->k_aux, c->v_aux};
  const float* cent[2] = {c->k_centroids, c->v_centroids};
  const int8_t* signs[2] = {c->k_signs, c->v_signs};
  uint16_t* out[2] = {k_out, v_out};
  for (int i = 0; i < 2; ++i)
    p.side[i] = {static_cast<const uint8_t*>(rows[i]), static_cast<const __half*>(aux[i]),
                 is_codebook(fmts[i]) ? cent[i] : nullptr, signs[i], i ? nullptr : c->k_qjl,
                 i ? nullptr : c->k_outliers, out[i], fmts[i], bits[i],
                 side_row_bytes(fmts[i], bits[i], c->head_dim)};
  p.slots = slots;
  p.num_tokens = num_tokens;
  p.hkv = c->num_kv_heads;
  p.page_size = c->page_size;
  p.page_shift = page_shift_of(c->page_size);
  p.num_slots = c->num_pages * c->page_size;
  p.kind_first = k_out ? 0 : 1;
  const int sides = (k_out && v_out) ? 2 : 1, sms = device_sms();
  if (p.num_slots == 0) return KVQ_OK;
  if ((long long)num_tokens * c->num_kv_heads > (1LL << 32)) return KVQ_ERR_INVALID_ARGUMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c->head_dim == 64) e = launch_read<64>(p, sides, sms, s);
  else if (c->head_dim == 128) e = launch_read<128>(p, sides, sms, s);
  else e = launch_read<256>(p, sides, sms, s);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
