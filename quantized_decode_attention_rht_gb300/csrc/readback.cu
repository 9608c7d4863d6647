// Cached tokens read back as fp16 vectors (kvq_dequantize).
//
// The mirror image of the append's per-thread kernel: D / 32 neighbouring lanes share a
// vector, each decoding 32 neighbouring coordinates of the stored row; five Walsh-Hadamard
// stages run in its registers, one transpose through shared memory hands it runs of
// R = 32 / (lanes per vector) coordinates at every multiple of 32, the remaining stages run
// on those, and each run is stored with the signs and 1 / sqrt(D) applied.  Stage order does
// not matter (the stages commute), so no exchange between lanes is needed beyond the one
// transpose.  Codebook centroids come from a 16-entry shared table: 16 words in 16 banks, so
// a warp's lookups never conflict whatever the codes.  Four blocks of 256 threads an SM (64
// registers; three, at 80, took 98.7 us instead of 93.9 for 65536 tokens x 8 heads of fp8 keys and
// INT4 values, 59% of the measured copy rate).  What bounds it is the shared-memory pipe: per
// vector of 128 coordinates, 8 wavefronts of transpose, 4 of table look-ups and 2 to 3 of rows
// in and out, against 14 cycles of an SM's share of the memory rate.  (Prefetching the next
// vector's row into L2 cost more than it hid: 102 us.)
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
// EXTRA: keys with a residual sketch or an outlier stream, which need more registers.
template <int TPV, bool EXTRA>
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
  if (!EXTRA || s.fmt == KVQ_FMT_CODEBOOK) scale = __half2float(s.aux[prow]);
  else if (s.fmt == KVQ_FMT_CODEBOOK_QJL) scale = __half2float(s.aux[2 * prow]);
  else scale = __half2float(*reinterpret_cast<const __half*>(reinterpret_cast<const uint8_t*>(s.aux) +
                                                             prow * (4 + KVQ_OUTLIER_CHANNELS)));
  scale *= inv_sqrt_dim(D);
#pragma unroll
  for (int e = 0; e < 32; ++e) y[e] *= scale;
  if (EXTRA && s.fmt == KVQ_FMT_CODEBOOK_QJL) {
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

template <int TPV, bool EXTRA>
__global__ void __launch_bounds__(kThreads, EXTRA ? 2 : 4) read_kernel(const ReadParams p) {
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
    decode_row<TPV, EXTRA>(side, prow, sub, cent, y);
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
    if (EXTRA && side.fmt == KVQ_FMT_CODEBOOK_OUTLIER) {  // + q_j s at channel c_j
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

template <int TPV>
cudaError_t launch_read(const ReadParams& p, int sides, int sms, cudaStream_t stream) {
  constexpr int VPB = kThreads / TPV;
  const long long nvec = (long long)p.num_tokens * p.hkv;
  const long long blocks = std::max<long long>(1, std::min<long long>((nvec + VPB - 1) / VPB, sms * 4LL / sides));
  const dim3 grid((unsigned)blocks, sides);
  const int kf = p.kind_first == 0 ? p.side[0].fmt : KVQ_FMT_CODEBOOK;
  if (kf == KVQ_FMT_CODEBOOK_QJL || kf == KVQ_FMT_CODEBOOK_OUTLIER)
    read_kernel<TPV, true><<<grid, kThreads, kXposeBytes, stream>>>(p);
  else
    read_kernel<TPV, false><<<grid, kThreads, kXposeBytes, stream>>>(p);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c->head_dim == 64) e = launch_read<2>(p, sides, sms, s);
  else if (c->head_dim == 128) e = launch_read<4>(p, sides, sms, s);
  else e = launch_read<8>(p, sides, sms, s);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
