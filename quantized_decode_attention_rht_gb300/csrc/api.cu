// C ABI of libkvq.so: argument checks, split-K planning and kernel launches.
#include "api_checks.cuh"

namespace kvq {
static std::atomic<uint64_t> g_launches{0};
void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }
}

extern "C" {

KVQ_API const char* kvq_status_string(kvq_status s) {
  switch (s) {
    case KVQ_OK: return "KVQ_OK";
    case KVQ_ERR_INVALID_ARGUMENT: return "KVQ_ERR_INVALID_ARGUMENT";
    case KVQ_ERR_UNSUPPORTED: return "KVQ_ERR_UNSUPPORTED";
    case KVQ_ERR_WORKSPACE_TOO_SMALL: return "KVQ_ERR_WORKSPACE_TOO_SMALL";
    case KVQ_ERR_CUDA: return "KVQ_ERR_CUDA";
  }
  return "KVQ_ERR_UNKNOWN";
}

KVQ_API uint64_t kvq_kernel_launches(void) { return kvq::g_launches.load(std::memory_order_relaxed); }

KVQ_API kvq_status kvq_row_bytes(int32_t format, int32_t bits, int32_t head_dim, size_t* row_bytes,
                                 size_t* aux_bytes) {
  if (!row_bytes || !aux_bytes) return KVQ_ERR_INVALID_ARGUMENT;
  return side_bytes(format, bits, head_dim, row_bytes, aux_bytes);
}

KVQ_API kvq_status kvq_outlier_calibrate(const uint16_t* k, int32_t num_tokens, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t* out_idx, void* stream) {
  if (!k || !out_idx || !aligned(k, 4) || !aligned(out_idx, 4) || num_tokens < 1 || num_kv_heads < 1)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (head_dim != 128 && head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  cudaError_t e = launch_outlier_calibrate(k, num_tokens, num_kv_heads, head_dim, out_idx,
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

KVQ_API kvq_status kvq_requantize(const kvq_cache* src, const int32_t* src_slots, const kvq_cache* dst,
                                  const int32_t* dst_slots, int32_t num_tokens, void* stream) {
  kvq_status st = check_cache(src);
  if (st != KVQ_OK || (st = check_cache(dst)) != KVQ_OK) return st;
  if (num_tokens < 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (src->k_format != KVQ_FMT_FP16 || src->v_format != KVQ_FMT_FP16) return KVQ_ERR_UNSUPPORTED;
  if (dst->k_format == KVQ_FMT_CODEBOOK_OUTLIER) return KVQ_ERR_UNSUPPORTED;
  if (src->head_dim != dst->head_dim || src->num_kv_heads != dst->num_kv_heads ||
      src->page_size != dst->page_size || src->k_signs != dst->k_signs || src->v_signs != dst->v_signs)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (!src->k_rows || !src->v_rows || !aligned(src->k_rows, 16) || !aligned(src->v_rows, 16))
    return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_cache* c = dst;
  if ((st = check_side(c, c->k_format, c->k_bits, c->k_rows, c->k_aux, c->k_centroids, c->k_bounds, c->k_signs,
                       true, true)) != KVQ_OK ||
      (st = check_side(c, c->v_format, c->v_bits, c->v_rows, c->v_aux, c->v_centroids, c->v_bounds, c->v_signs,
                       true, false)) != KVQ_OK)
    return st;
  if (num_tokens == 0) return KVQ_OK;
  if (!src_slots || !dst_slots || !aligned(src_slots, 4) || !aligned(dst_slots, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  QuantParams p;
  memset(&p, 0, sizeof(p));
  fill_sides(dst, &p);
  p.src_rows[0] = static_cast<const uint8_t*>(src->k_rows);
  p.src_rows[1] = static_cast<const uint8_t*>(src->v_rows);
  p.src_slots = src_slots;
  p.src_num_slots = src->num_pages * src->page_size;
  p.slots = dst_slots;
  p.num_tokens = num_tokens;
  p.hkv = dst->num_kv_heads;
  p.page_size = dst->page_size;
  p.page_shift = page_shift_of(dst->page_size);
  p.num_slots = dst->num_pages * dst->page_size;
  p.kind_first = 0;
  p.num_kinds = 2;
  p.num_vectors = 2LL * num_tokens * dst->num_kv_heads;
  if (p.num_slots == 0 || p.src_num_slots == 0) return KVQ_OK;
  if ((long long)num_tokens * dst->num_kv_heads > (1LL << 28)) return KVQ_ERR_INVALID_ARGUMENT;
  cudaError_t e = launch_requantize(p, dst->head_dim, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

KVQ_API kvq_status kvq_quantize_append(const kvq_cache* cache, const uint16_t* k, const uint16_t* v,
                                       int32_t num_tokens, const int32_t* slot_mapping, void* stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (num_tokens < 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return KVQ_OK;  // nothing to append (an empty tensor may have no address)
  if (!k && !v) return KVQ_ERR_INVALID_ARGUMENT;
  if (!slot_mapping || !aligned(slot_mapping, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if ((k && !aligned(k, 16)) || (v && !aligned(v, 16))) return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_cache* c = cache;
  if (k && (st = check_side(c, c->k_format, c->k_bits, c->k_rows, c->k_aux, c->k_centroids, c->k_bounds,
                            c->k_signs, true, true)) != KVQ_OK)
    return st;
  if (v && (st = check_side(c, c->v_format, c->v_bits, c->v_rows, c->v_aux, c->v_centroids, c->v_bounds,
                            c->v_signs, true, false)) != KVQ_OK)
    return st;
  // a lane reads the signs of its head_dim / 32 coordinates in one piece
  const int run = c->head_dim / 32;
  if ((k && !aligned(c->k_signs, run)) || (v && !aligned(c->v_signs, run))) return KVQ_ERR_INVALID_ARGUMENT;
  QuantParams p;
  memset(&p, 0, sizeof(p));
  p.x[0] = k;
  p.x[1] = v;
  fill_sides(c, &p);
  p.slots = slot_mapping;
  p.num_tokens = num_tokens;
  p.hkv = c->num_kv_heads;
  p.page_size = c->page_size;
  p.page_shift = page_shift_of(c->page_size);
  p.num_slots = c->num_pages * c->page_size;
  p.kind_first = k ? 0 : 1;
  p.num_kinds = (k && v) ? 2 : 1;
  p.num_vectors = (long long)p.num_kinds * num_tokens * c->num_kv_heads;
  if (p.num_slots == 0) return KVQ_OK;
  cudaError_t e = launch_quantize(p, c->head_dim, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

KVQ_API kvq_status kvq_decode_workspace_size(const kvq_tier_view* tiers, int32_t num_tiers, int32_t batch,
                                             int32_t num_q_heads, int32_t split_tokens, size_t* bytes) {
  if (!bytes) return KVQ_ERR_INVALID_ARGUMENT;
  kvq_status st = check_tiers(tiers, num_tiers, batch, num_q_heads);
  if (st != KVQ_OK) return st;
  // the plan depends on whether q is 16-byte aligned (the fused fp16 / fp8 kernel loads it in
  // 16-byte pieces): size for the larger of the two, so any valid q fits
  size_t most = 0;
  for (const bool q16 : {true, false}) {
    Plan plan;
    if ((st = make_plan(tiers, num_tiers, batch, num_q_heads, split_tokens, q16, &plan)) != KVQ_OK) return st;
    most = std::max(most, workspace_bytes(batch, num_q_heads, tiers[0].cache->head_dim, plan.total,
                                          has_sketch(tiers, num_tiers)));
  }
  *bytes = most;
  return KVQ_OK;
}

KVQ_API kvq_status kvq_decode_attention(const kvq_tier_view* tiers, int32_t num_tiers, const uint16_t* q,
                                        int32_t batch, int32_t num_q_heads, int32_t split_tokens, float* out,
                                        void* workspace, size_t ws_bytes, void* stream) {
  return kvq_decode_attention_ex(tiers, num_tiers, q, batch, num_q_heads, split_tokens, out, workspace, ws_bytes,
                                 nullptr, stream);
}

KVQ_API kvq_status kvq_decode_attention_ex(const kvq_tier_view* tiers, int32_t num_tiers, const uint16_t* q,
                                           int32_t batch, int32_t num_q_heads, int32_t split_tokens, float* out,
                                           void* workspace, size_t ws_bytes, const kvq_decode_options* options,
                                           void* stream) {
  kvq_status st = check_tiers(tiers, num_tiers, batch, num_q_heads);
  if (st != KVQ_OK) return st;
  if (options && options->spike_flags && !aligned(options->spike_flags, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (options && options->status && !aligned(options->status, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (batch == 0) return KVQ_OK;
  if (!q || !out || !aligned(q, 4) || !aligned(out, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  const int d = tiers[0].cache->head_dim, hkv = tiers[0].cache->num_kv_heads;
  Plan plan;
  if ((st = make_plan(tiers, num_tiers, batch, num_q_heads, split_tokens, aligned(q, 16), &plan)) != KVQ_OK)
    return st;
  const bool sketch = has_sketch(tiers, num_tiers);
  const size_t need = workspace_bytes(batch, num_q_heads, d, plan.total, sketch);
  if (need > 0 && (!workspace || !aligned(workspace, 256))) return KVQ_ERR_INVALID_ARGUMENT;
  if (ws_bytes < need) return KVQ_ERR_WORKSPACE_TOO_SMALL;

  DecParams p;
  fill_decode(tiers, num_tiers, plan, q, batch, num_q_heads, workspace, sketch, &p);
  p.out = out;
  p.spike = options ? options->spike_flags : nullptr;
  p.status = options ? options->status : nullptr;
  p.gate = options && options->score_gate ? 1 : 0;
  // one split-K launch per kernel family present (the fused fp16 / fp8 + INT4 kernel takes
  // all its tiers at once, the codebook and generic kernels one launch per tier), all
  // writing partials into the one workspace, then the combine pass over every tier
  int* counters = reinterpret_cast<int*>(static_cast<char*>(workspace) + need - 256);
  p.err = counters + kErrorWord;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool fam[3] = {false, false, false};
  for (int i = 0; i < num_tiers; ++i) fam[plan.kind[i]] = true;
  cudaError_t e = cudaMemsetAsync(counters, 0, 256, s);  // work counters and the error word
  if (e == cudaSuccess && fam[TIER_GQA]) e = launch_decode_gqa(p, counters + kGqaCounter, s, fam[TIER_CB]);
  if (e == cudaSuccess && fam[TIER_CB]) e = launch_decode_cb(p, d, counters, s, fam[TIER_GQA]);
  if (e == cudaSuccess && fam[TIER_GENERIC]) e = launch_decode(p, d, num_q_heads / hkv, s);
  if (e == cudaSuccess) e = launch_combine(p, d, s);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
