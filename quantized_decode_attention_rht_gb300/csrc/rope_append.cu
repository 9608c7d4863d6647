// New tokens in one call (kvq_rope_append): queries turned by their positions, keys turned,
// rotated, encoded and stored, values rotated, encoded and stored.
//
// Small appends (a decode step) take one launch: grid rows for the keys, the values and the
// queries, one warp per vector (quantize_small.cuh).  Large ones take the per-thread kernel
// of quantize.cuh, one launch per side (rope_append_large.cuh), and the rotary kernel for the
// queries.  32 tokens x (32 + 8 + 8) heads x 128: 4 us, a launch and one chain of load, turn,
// exchange and store.  The bound between the two is the plain append's (kSmallMaxVectors).
#include "api_checks.cuh"
#include "quantize_small.cuh"
#include "rope_append_large.cuh"

namespace kvq {
namespace {

struct SmallParams : TurnParams {
  const uint16_t* q;
  uint16_t* q_out;
  long long qt, qh, ot, oh;  // strides of q and its output
  int hq;
};

// One warp per query head: its D / 32 neighbouring elements per lane, turned and stored.
template <int D>
__device__ __forceinline__ void turn_queries(const SmallParams& p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long n = (long long)p.num_tokens * p.hq;
  for (long long v = blockIdx.x * kWarps + (threadIdx.x >> 5); v < n; v += (long long)gridDim.x * kWarps) {
    const int token = (int)(v / p.hq), h = (int)(v - (long long)token * p.hq);
    float y[E];
    load_heads<D, E, true, true>(p.q + token * p.qt + h * p.qh, p.rope, token, lane, y);
    uint32_t w[E / 2];
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
      const __half2 h2 = __floats2half2_rn(y[2 * k], y[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h2);
    }
    __syncwarp();  // in place: every lane has read its partner's elements
    uint16_t* dst = p.q_out + token * p.ot + h * p.oh + lane * E;
    if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
    else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int D, int SRC>
__device__ __forceinline__ void append_any(const SmallParams& p, const QuantSide& side, const uint16_t* x,
                                           uint32_t* buf) {
  switch (side.fmt) {
    case KVQ_FMT_CODEBOOK: append_bits<D, F_CB, SRC>(p, side, x, nullptr, buf); break;
    case KVQ_FMT_CODEBOOK_QJL:  // keys only, as the host checks
      if constexpr (SRC == SRC_TURNED) append_bits<D, F_CBQ, SRC>(p, side, x, nullptr, buf);
      break;
    case KVQ_FMT_CODEBOOK_OUTLIER:
      if constexpr (SRC == SRC_TURNED) append_bits<D, F_CBO, SRC>(p, side, x, nullptr, buf);
      break;
    case KVQ_FMT_FP16: append_side<D, F_F16, 0, SRC>(p, side, x, nullptr, buf); break;
    case KVQ_FMT_FP8_E4M3: append_side<D, F_F8, 0, SRC>(p, side, x, nullptr, buf); break;
    default: append_side<D, F_I4, 0, SRC>(p, side, x, nullptr, buf); break;
  }
}

// Grid row blockIdx.y: side kind_first + y, or the queries in the row after the sides.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) rope_append_kernel(const SmallParams p) {
  __shared__ __align__(16) uint32_t words[kWarps][32];
  uint32_t* buf = words[threadIdx.x >> 5];
  if ((int)blockIdx.y == p.num_kinds) turn_queries<D>(p);
  else if (p.kind_first + blockIdx.y == 0) append_any<D, SRC_TURNED>(p, p.side[0], p.x[0], buf);
  else append_any<D, SRC_STRIDED>(p, p.side[1], p.x[1], buf);
}

cudaError_t launch_small(const SmallParams& p, int dim, int sms, bool queries, cudaStream_t stream) {
  const bool sketch = p.kind_first == 0 && p.side[0].fmt == KVQ_FMT_CODEBOOK_QJL;
  long long n = (long long)p.num_tokens * p.hkv * (sketch ? KVQ_QJL_DIM / 32 : 1);
  if (queries) n = std::max(n, (long long)p.num_tokens * p.hq);
  const unsigned blocks = (unsigned)std::max<long long>(1, std::min<long long>((n + kWarps - 1) / kWarps, sms * 8LL));
  const dim3 grid(blocks, p.num_kinds + (queries ? 1 : 0));
  if (dim == 64) rope_append_kernel<64><<<grid, kWarps * 32, 0, stream>>>(p);
  else if (dim == 128) rope_append_kernel<128><<<grid, kWarps * 32, 0, stream>>>(p);
  else rope_append_kernel<256><<<grid, kWarps * 32, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

bool wide_heads(const kvq_heads* h) { return aligned(h->x, 16) && (h->x_token_stride | h->x_head_stride) % 8 == 0; }

}  // namespace
}  // namespace kvq

extern "C" KVQ_API kvq_status kvq_rope_append(const kvq_cache* cache, const kvq_rope* rope, const int32_t* positions,
                                              const kvq_heads* k, const kvq_heads* v, const kvq_heads* q,
                                              int32_t num_tokens, const int32_t* slot_mapping, void* stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK || (st = check_rope(rope, cache->head_dim)) != KVQ_OK) return st;
  if (num_tokens < 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return KVQ_OK;
  if (!k && !v) return KVQ_ERR_INVALID_ARGUMENT;
  if (!positions || !aligned(positions, 4) || !slot_mapping || !aligned(slot_mapping, 4))
    return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_cache* c = cache;
  const int d = c->head_dim;
  for (const kvq_heads* h : {k, v}) {
    if (!h) continue;
    if ((st = check_heads(h, num_tokens, d, false)) != KVQ_OK) return st;
    if (h->num_heads != c->num_kv_heads || !wide_heads(h)) return KVQ_ERR_INVALID_ARGUMENT;
  }
  if (q && (st = check_heads(q, num_tokens, d, true)) != KVQ_OK) return st;
  if (k && (st = check_side(c, c->k_format, c->k_bits, c->k_rows, c->k_aux, c->k_centroids, c->k_bounds, c->k_signs,
                            true, true)) != KVQ_OK)
    return st;
  if (v && (st = check_side(c, c->v_format, c->v_bits, c->v_rows, c->v_aux, c->v_centroids, c->v_bounds, c->v_signs,
                            true, false)) != KVQ_OK)
    return st;
  if ((long long)num_tokens * c->num_kv_heads > (1LL << 28)) return KVQ_ERR_INVALID_ARGUMENT;
  // the large kernel reads sign runs in pieces of up to 16 bytes
  if ((k && !aligned(c->k_signs, 16)) || (v && !aligned(c->v_signs, 16))) return KVQ_ERR_INVALID_ARGUMENT;
  SmallParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  fill_sides(c, &p);
  p.x[0] = k ? k->x : nullptr;
  p.x[1] = v ? v->x : nullptr;
  for (int i = 0; i < 2; ++i) {
    const kvq_heads* h = i ? v : k;
    p.xt[i] = h ? h->x_token_stride : 0;
    p.xh[i] = h ? h->x_head_stride : 0;
  }
  p.rope = rope_params(rope, positions, 0);
  p.slots = slot_mapping;
  p.num_tokens = num_tokens;
  p.hkv = c->num_kv_heads;
  p.page_size = c->page_size;
  p.page_shift = page_shift_of(c->page_size);
  p.num_slots = c->num_pages * c->page_size;
  p.kind_first = k ? 0 : 1;
  p.num_kinds = (k && v) ? 2 : 1;
  p.num_vectors = (long long)p.num_kinds * num_tokens * c->num_kv_heads;
  const int sms = device_sms();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  // keys with a sketch or an outlier stream are built for the warp kernel only
  const bool warp_keys = k && (c->k_format == KVQ_FMT_CODEBOOK_QJL || c->k_format == KVQ_FMT_CODEBOOK_OUTLIER);
  if ((long long)num_tokens * c->num_kv_heads > kSmallMaxVectors) {
    for (int side = p.kind_first; side < p.kind_first + p.num_kinds && e == cudaSuccess; ++side) {
      if (side == 0 && warp_keys) {
        SmallParams keys = p;
        keys.num_kinds = 1;
        e = launch_small(keys, d, sms, false, s);
        continue;
      }
      LargeParams l;
      memset(static_cast<void*>(&l), 0, sizeof(l));
      static_cast<QuantParams&>(l) = p;
      l.kind_first = side;
      l.num_kinds = 1;
      l.rope = p.rope;
      l.xt = p.xt[side];
      l.xh = p.xh[side];
      e = side == 0 ? launch_append_keys(l, d, sms, s) : launch_append_values(l, d, sms, s);
    }
    if (e == cudaSuccess && q) e = launch_rope(p.rope, q, nullptr, num_tokens, d, sms, s);
  } else {
    // one launch, queries too where their rows are of 16-byte units
    const bool q_wide = q && wide_heads(q) && aligned(q->out, 16) && (q->out_token_stride | q->out_head_stride) % 8 == 0;
    if (q_wide) {
      p.q = q->x;
      p.q_out = q->out;
      p.qt = q->x_token_stride;
      p.qh = q->x_head_stride;
      p.ot = q->out_token_stride;
      p.oh = q->out_head_stride;
      p.hq = q->num_heads;
    }
    e = launch_small(p, d, sms, q_wide, s);
    if (e == cudaSuccess && q && !q_wide) e = launch_rope(p.rope, q, nullptr, num_tokens, d, sms, s);
  }
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
