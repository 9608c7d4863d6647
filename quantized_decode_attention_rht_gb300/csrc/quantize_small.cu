// Quantise-and-append for small appends: the warp-per-vector kernel's instances and launches
// (the kernel's parts are in quantize_small.cuh).
#include "quantize_small.cuh"

namespace kvq {
namespace {

// Grid row blockIdx.y = side kind_first + y; the format is a warp-uniform branch (only the
// taken path's instructions are fetched).
template <int D, bool FROM_ROWS>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const QuantParams p) {
  constexpr int kSrc = FROM_ROWS ? SRC_ROWS : SRC_NEW;
  __shared__ __align__(16) uint32_t words[kWarps][32];
  const int kind = p.kind_first + blockIdx.y;  // 0 or 1
  const QuantSide side = kind ? p.side[1] : p.side[0];
  const uint16_t* x = kind ? p.x[1] : p.x[0];
  const uint8_t* src = kind ? p.src_rows[1] : p.src_rows[0];
  uint32_t* buf = words[threadIdx.x >> 5];
  switch (side.fmt) {
    case KVQ_FMT_CODEBOOK: append_bits<D, F_CB, kSrc>(p, side, x, src, buf); break;
    case KVQ_FMT_CODEBOOK_QJL: append_bits<D, F_CBQ, kSrc>(p, side, x, src, buf); break;
    case KVQ_FMT_CODEBOOK_OUTLIER:  // new vectors only (the host refuses a re-encode into it)
      if constexpr (!FROM_ROWS) append_bits<D, F_CBO, SRC_NEW>(p, side, x, src, buf);
      break;
    case KVQ_FMT_FP16: append_side<D, F_F16, 0, kSrc>(p, side, x, src, buf); break;
    case KVQ_FMT_FP8_E4M3: append_side<D, F_F8, 0, kSrc>(p, side, x, src, buf); break;
    default: append_side<D, F_I4, 0, kSrc>(p, side, x, src, buf); break;
  }
}

template <bool FROM_ROWS>
cudaError_t launch_warp_kernel(const QuantParams& p, int head_dim, int sms, cudaStream_t stream) {
  const bool sketch = p.side[0].fmt == KVQ_FMT_CODEBOOK_QJL && p.kind_first == 0;
  const long long nvec = (long long)p.num_tokens * p.hkv * (sketch ? KVQ_QJL_DIM / 32 : 1);  // work units
  const unsigned blocks =
      (unsigned)std::max<long long>(1, std::min<long long>((nvec + kWarps - 1) / kWarps, (long long)sms * 8));
  const dim3 grid(blocks, p.num_kinds);
  if (head_dim == 64) append_kernel<64, FROM_ROWS><<<grid, kWarps * 32, 0, stream>>>(p);
  else if (head_dim == 128) append_kernel<128, FROM_ROWS><<<grid, kWarps * 32, 0, stream>>>(p);
  else append_kernel<256, FROM_ROWS><<<grid, kWarps * 32, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t launch_quantize_small(const QuantParams& p, int head_dim, int sms, cudaStream_t stream) {
  return launch_warp_kernel<false>(p, head_dim, sms, stream);
}

cudaError_t launch_requantize(const QuantParams& p, int head_dim, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  if ((long long)p.num_tokens * p.hkv > (1LL << 28)) return cudaErrorInvalidValue;  // four units per sketched key fit an int
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return launch_warp_kernel<true>(p, head_dim, sms, stream);
}

}  // namespace kvq
