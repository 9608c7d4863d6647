// Large rotary appends: the per-thread kernel of quantize.cuh on strided inputs, its keys
// turned by their positions between the load and the rotation.
//
// The angles of a token are the same for all its heads.  Where the vectors of a warp belong
// to one token (the usual case: the warp holds 32 / TPV neighbouring heads), its lanes work
// the token's cos and sin out once, rot / 64 pairs a lane, into the shared area that the
// first vector's transpose uses afterwards; otherwise each vector's lanes fill the vector's
// own area.  rot / 2 pairs of 8 bytes fit the D floats of an area exactly.
//
// Bounded by instruction issue and shared memory (60% and 60 to 70% busy): 262144 vectors of 256 to
// 4-bit codes, keys 102 us, values 73 us, 24% and 34% of the measured copy rate.  (The butterflies
// as a product on the tensor cores, as in the read-back, took 103 and 63 us there but 136
// instead of 88 for both sides at head_dim 128: a turned key is float32, two fp16 operands.)
#pragma once
#include "quantize.cuh"
#include "rope.cuh"

namespace kvq {

struct LargeParams : QuantParams {
  RopeParams rope;
  long long xt, xh;  // token and head strides of the side's input
};

// The per-thread kernel for one side (p.kind_first): keys turned, values as they are.
cudaError_t launch_append_keys(const LargeParams& p, int head_dim, int sms, cudaStream_t stream);
cudaError_t launch_append_values(const LargeParams& p, int head_dim, int sms, cudaStream_t stream);

namespace {

__device__ __forceinline__ float2 lds_cs(uint32_t table, int pair) {
  float2 f;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f.x), "=f"(f.y) : "r"(table + 8u * pair) : "memory");
  return f;
}

// y (run order: run k, offset r at k R + r, coordinate 32k + R sub + r) turned by the (cos,
// sin) pairs at `table`; xv: the vector, for partners that other lanes hold.
template <int TPV>
__device__ __forceinline__ void turn_runs(const uint16_t* xv, const RopeParams& rope, uint32_t table, int sub,
                                          float (&y)[32]) {
  constexpr int R = 32 / TPV, D = 32 * TPV;
  const int half = rope.rot / 2;
  if (rope.layout == KVQ_ROPE_INTERLEAVED) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const int c = 32 * (e / R) + R * sub + e % R;
      if (c < rope.rot) {
        const float2 f = lds_cs(table, c / 2);
        const float a = y[e], b = y[e + 1];
        y[e] = fmaf(a, f.x, -(b * f.y));
        y[e + 1] = fmaf(b, f.x, a * f.y);
      }
    }
  } else if (rope.rot == D) {  // the partner is the same place of run k + TPV / 2
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int c = 32 * (e / R) + R * sub + e % R;
      const float2 f = lds_cs(table, c);
      const float a = y[e], b = y[e + 16];
      y[e] = fmaf(a, f.x, -(b * f.y));
      y[e + 16] = fmaf(b, f.x, a * f.y);
    }
  } else {  // partners by a second read of the vector (L1), four at a time where they allow it
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const int c0 = 32 * (e / R) + R * sub + e % R;
      if (c0 < rope.rot) {
        float o[4];
        if (half % 4 == 0) {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(xv + (c0 < half ? c0 + half : c0 - half)));
          const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
          const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
          o[0] = lo.x;
          o[1] = lo.y;
          o[2] = hi.x;
          o[3] = hi.y;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = c0 + i;
            o[i] = c < rope.rot ? __half2float(__ushort_as_half(__ldg(xv + (c < half ? c + half : c - half)))) : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + i;
          if (c < rope.rot) {
            const bool low = c < half;
            const float2 f = lds_cs(table, low ? c : c - half);
            y[e + i] = low ? fmaf(y[e + i], f.x, -(o[i] * f.y)) : fmaf(y[e + i], f.x, o[i] * f.y);
          }
        }
      }
    }
  }
}

template <int TPV, int FMT, int BITS, bool TURN>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(FMT, FMT) - (TURN ? 1 : 0)) append_large_kernel(const LargeParams p) {
  constexpr int kE = kCoords, D = kE * TPV, VPB = kThreads / TPV;
  __shared__ Table table;
  extern __shared__ __align__(16) float2 cells[];
  const QuantSide& side = p.side[p.kind_first];
  if constexpr (FMT == F_CB) build_table(table, cells, side.bounds, side.centroids, (1 << BITS) - 1, D);
  const uint32_t xpose =
      static_cast<uint32_t>(__cvta_generic_to_shared(cells)) + (uint32_t)(quant_smem<FMT, FMT>() - kXposeBytes);
  const int lane = threadIdx.x & 31, sub = lane % TPV, vw = lane / TPV;
  const unsigned gmask = ((1u << TPV) - 1u) << (lane - sub);
  const uint32_t warp_area = xpose + (uint32_t)((threadIdx.x & ~31u) / TPV) * (D * 4);
  const uint32_t area = warp_area + (uint32_t)vw * (D * 4);
  const long long nvec = (long long)p.num_tokens * p.hkv, stride = (long long)gridDim.x * VPB;
  const uint16_t* x = p.x[p.kind_first];
  // the loop's bound is the warp's (a warp past the end in part works its last vectors on
  // the last one, again), so that the warp may share a table
  for (long long v0 = (long long)blockIdx.x * VPB + (threadIdx.x & ~31u) / TPV; v0 < nvec; v0 += stride) {
    const long long v = min(v0 + vw, nvec - 1);
    const int token = (int)(v / p.hkv), h = (int)(v - (long long)token * p.hkv);
    const uint16_t* xv = x + token * p.xt + h * p.xh;
    float y[kE];
    if constexpr (TURN) {
      uint32_t xw[16];
      load_runs<TPV>(xv, sub, xw);
      const int pos = __ldg(p.rope.positions + token), pairs = p.rope.rot / 2;
      const bool one = __all_sync(0xFFFFFFFFu, token == __shfl_sync(0xFFFFFFFFu, token, 0));
      __syncwarp();  // the areas' reads of the previous vectors are done
      const uint32_t cs = one ? warp_area : area;
      for (int i = one ? lane : sub; i < pairs; i += one ? 32 : TPV) {
        const float2 f = rope_cos_sin(p.rope, i, pos);
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(cs + 8u * i), "f"(f.x), "f"(f.y) : "memory");
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&xw[j]));
        y[2 * j] = f.x;
        y[2 * j + 1] = f.y;
      }
      turn_runs<TPV>(xv, p.rope, cs, sub, y);
      __syncwarp();  // the table has been read; the transposes may write
      uint32_t sw[8];
      load_signs<TPV>(side.signs + (size_t)h * D, sub, sw);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const uint32_t w = sw[e / 4];
        const float a = __uint_as_float(__float_as_uint(y[e]) ^ ((w << (24 - 8 * (e % 4))) & 0x80000000u));
        const float c = __uint_as_float(__float_as_uint(y[e + 1]) ^ ((w << (16 - 8 * (e % 4))) & 0x80000000u));
        y[e] = a + c;
        y[e + 1] = a - c;
      }
      rotate_runs<TPV>(area, sub, vw, gmask, y);
    } else {
      uint32_t sw[8];
      load_signs<TPV>(side.signs + (size_t)h * D, sub, sw);
      load_rotate<TPV>(xv, sw, area, sub, vw, gmask, y);
    }
    if (v0 + stride < nvec) {
      const long long vn = min(v0 + stride + vw, nvec - 1);
      const int tn = (int)(vn / p.hkv), hn = (int)(vn - (long long)tn * p.hkv);
      prefetch_l2(x + tn * p.xt + hn * p.xh + sub * kE);
    }
    quantize_vector<TPV, kE, FMT, BITS>(p, side, table, y, token, h, sub, gmask);
  }
}

template <int TPV, int FMT, int BITS, bool TURN>
cudaError_t launch_large(const LargeParams& p, int sms, cudaStream_t stream) {
  constexpr int VPB = kThreads / TPV, smem = quant_smem<FMT, FMT>();
  auto kern = append_large_kernel<TPV, FMT, BITS, TURN>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  const long long nvec = (long long)p.num_tokens * p.hkv;
  const long long blocks = std::max<long long>(
      1, std::min<long long>((nvec + VPB - 1) / VPB, (long long)sms * (blocks_per_sm(FMT, FMT) - (TURN ? 1 : 0))));
  kern<<<(unsigned)blocks, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

template <int TPV, bool TURN>
cudaError_t launch_large_fmt(const LargeParams& p, int sms, cudaStream_t stream) {
  const QuantSide& s = p.side[p.kind_first];
  switch (s.fmt) {
    case KVQ_FMT_CODEBOOK:
      return s.bits == 4 ? launch_large<TPV, F_CB, 4, TURN>(p, sms, stream)
                         : (s.bits == 3 ? launch_large<TPV, F_CB, 3, TURN>(p, sms, stream)
                                        : launch_large<TPV, F_CB, 2, TURN>(p, sms, stream));
    case KVQ_FMT_FP16: return launch_large<TPV, F_F16, 0, TURN>(p, sms, stream);
    case KVQ_FMT_FP8_E4M3: return launch_large<TPV, F_F8, 0, TURN>(p, sms, stream);
    case KVQ_FMT_INT4_G32: return launch_large<TPV, F_I4, 0, TURN>(p, sms, stream);
    default: return cudaErrorNotSupported;  // sketched and outlier keys take the warp kernel
  }
}

template <bool TURN>
cudaError_t launch_large_dim(const LargeParams& p, int head_dim, int sms, cudaStream_t stream) {
  if (head_dim == 64) return launch_large_fmt<2, TURN>(p, sms, stream);
  if (head_dim == 128) return launch_large_fmt<4, TURN>(p, sms, stream);
  return launch_large_fmt<8, TURN>(p, sms, stream);
}

}  // namespace
}  // namespace kvq
