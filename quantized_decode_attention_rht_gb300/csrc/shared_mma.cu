// The prefix pass's launches (the kernel: shared_mma.cuh).
#include <atomic>

#include "shared_mma.cuh"

namespace kvq {

bool shared_tier_supported(int head_dim, int k_fmt, int v_fmt) {
  if (head_dim != kDim) return false;
  if (k_fmt == KVQ_FMT_FP16) return v_fmt == KVQ_FMT_FP16;
  if (k_fmt == KVQ_FMT_FP8_E4M3) return v_fmt == KVQ_FMT_INT4_G32 || v_fmt == KVQ_FMT_FP16;
  return k_fmt == KVQ_FMT_CODEBOOK && v_fmt == KVQ_FMT_CODEBOOK;
}

namespace {

template <bool CODES>
cudaError_t launch_kind(const SharedParams& all, cudaStream_t stream) {
  SharedParams p = all;
  p.num_tiers = 0;
  int splits = 0;
  for (int i = 0; i < all.num_tiers; ++i) {
    if ((all.tier[i].k_fmt == KVQ_FMT_CODEBOOK) != CODES) continue;
    SharedTier& t = p.tier[p.num_tiers++];
    t = all.tier[i];
    t.first = splits;
    splits += t.num_splits;
  }
  const long long items = (long long)p.num_blocks * p.hkv * splits;
  if (items == 0) return cudaSuccess;
  auto kern = shared_prefix_kernel<CODES>;
  static std::atomic<bool> configured[64];  // shared-memory limit raised on this device (a racing second
                                           // raise is harmless)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  kern<<<(unsigned)items, kThreads, kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

// One launch per kind of tier.
cudaError_t launch_shared_prefix(const SharedParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_kind<false>(p, stream);
  return e == cudaSuccess ? launch_kind<true>(p, stream) : e;
}

}  // namespace kvq
