// Chunks with few rows, on the packed cache: the prefix kernel over a plan's items (shared_mma.cuh), with a mask where a
// row block's tokens do not all see a tile.  Bounded as there, by 1.4 to 1.5 us a tile whatever the rows, and, where
// there are few tiles, by the plan before it and the item's start: 4 x 5 tokens x 32/8 heads on 2000 of fp8 keys and INT4
// values 33 us, 8 chunks of up to 64 tokens on up to 8192, the newest 256 in fp16, 81 to 97 us by the
// lengths drawn (the newest are items of their own, two tiles long behind the same start).
#include <atomic>

#include "shared_mma.cuh"

namespace kvq {
namespace {

template <bool CODES>
cudaError_t launch_kind(const ChunkParams& p, cudaStream_t stream) {
  auto kern = shared_prefix_kernel<CODES, ChunkParams>;
  static std::atomic<bool> configured[64];  // shared-memory limit raised on this device (a racing second raise is
                                            // harmless)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  return launch_dependent(reinterpret_cast<const void*>(kern), (unsigned)((long long)p.max_items[1] * p.hkv), kThreads, kSmem, p, stream);
}

}  // namespace

cudaError_t launch_chunk_packed(const ChunkParams& all, bool behind, cudaStream_t stream) {
  ChunkParams p = all;
  p.wait_first = !behind;
  bool kinds[2] = {false, false};
  for (int i = 0; i < p.num_tiers; ++i)
    if (p.tier[i].max_pages) kinds[p.tier[i].v_fmt == KVQ_FMT_CODEBOOK] = true;
  cudaError_t e = cudaSuccess;
  if (kinds[0]) {
    e = launch_kind<false>(p, stream);
    p.wait_first = 0;
  }
  if (e == cudaSuccess && kinds[1]) e = launch_kind<true>(p, stream);
  return e;
}

}  // namespace kvq
