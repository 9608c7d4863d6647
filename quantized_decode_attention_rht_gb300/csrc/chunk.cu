// kvq_chunk_attention and kvq_decode_attention_window: argument checks, workspace and launches.
//
// A call is the plan (chunk_plan.cu), the passes over the cache that some of its sequences may need (chunk_dense.cu
// for those with many rows, chunk_packed.cu for the others), and the joining of partial results.
#include "api_checks.cuh"
#include "chunk.cuh"
#include "rope.cuh"
#include "shared.cuh"
#include "window.cuh"

namespace kvq {
namespace {

// Query rows a kv head above which a sequence is unpacked.  A row block costs 1.45 us a tile of packed tokens, a pair of
// them 2 us a tile of unpacked ones, and the unpacking as much once more.  Measured (GB300, 32/8 heads, fp8 keys and
// INT4 values), packed and unpacked: 64 tokens (256 rows) on 8000 54 and 63 us, 128 tokens (512 rows) on 8000 72 and 72,
// 8 x 256 tokens (1024 rows) on 4000 323 and 267, 512 tokens (2048 rows) on 30000 449 and 333.
constexpr int kDenseRows = 512;

// Tokens of a sequence at most: positions, and their distances over windows, then stay in 32 bits.
constexpr long long kMostTokens = 1LL << 30;

struct ChunkCall {
  const kvq_tier_view* tiers;
  int num_tiers, batch, num_tokens, hq;
  bool offsets;  // chunks of any length; else one token a sequence
  const kvq_visible* visible;
};

// Checks, and everything of the parameters that does not depend on the workspace.
kvq_status chunk_plan(const ChunkCall& c, ChunkParams* p) {
  memset(static_cast<void*>(p), 0, sizeof(*p));
  if (c.num_tokens < 0 || c.batch < 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (!c.offsets && c.num_tokens != c.batch) return KVQ_ERR_INVALID_ARGUMENT;
  kvq_status st = check_tiers(c.tiers, c.num_tiers, c.batch, c.hq);
  if (st != KVQ_OK) return st;
  for (int i = 0; i < c.num_tiers; ++i)
    if (!aligned(c.tiers[i].block_table, 4) || !aligned(c.tiers[i].seq_lens, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (c.visible && (c.visible->window < 0 || c.visible->sinks < 0 || (c.visible->window == 0 && c.visible->sinks)))
    return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_cache* c0 = c.tiers[0].cache;
  if (!aligned(c0->k_signs, 16) || !aligned(c0->v_signs, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  if ((long long)c.num_tokens * c.hq > (1LL << 26) || c.batch > 65536) return KVQ_ERR_UNSUPPORTED;
  const int d = c0->head_dim, hkv = c0->num_kv_heads;
  long long room = 0;
  p->key_parts = 1;
  for (int i = 0; i < c.num_tiers; ++i) {
    const kvq_cache* k = c.tiers[i].cache;
    room += (long long)usable_pages(c.tiers[i]) * k->page_size;
    if ((long long)k->num_pages * k->page_size * hkv >= 0xFFFFFFFFLL) return KVQ_ERR_UNSUPPORTED;
    ChunkTier& t = p->tier[i];
    t.k_rows = static_cast<const uint8_t*>(k->k_rows);
    t.v_rows = static_cast<const uint8_t*>(k->v_rows);
    t.k_aux = static_cast<const __half*>(k->k_aux);
    t.v_aux = static_cast<const __half*>(k->v_aux);
    t.k_cent = k->k_centroids;
    t.v_cent = k->v_centroids;
    t.k_qjl = k->k_qjl;
    t.k_outl = k->k_outliers;
    t.block_table = c.tiers[i].block_table;
    t.lens = c.tiers[i].seq_lens;
    t.k_fmt = k->k_format;
    t.v_fmt = k->v_format;
    t.k_bits = k->k_bits;
    t.v_bits = k->v_bits;
    t.k_row_bytes = side_row_bytes(k->k_format, k->k_bits, d);
    t.v_row_bytes = side_row_bytes(k->v_format, k->v_bits, d);
    t.num_pages = k->num_pages;
    t.max_pages = usable_pages(c.tiers[i]);
    t.table_pages = c.tiers[i].max_pages;
    if (is_codebook(k->v_format)) {
      p->codes = c.num_tiers > 1 ? 2 : 1;
      p->summed |= k->v_bits == 4;
    }
    if (k->k_format == KVQ_FMT_CODEBOOK_QJL || k->k_format == KVQ_FMT_CODEBOOK_OUTLIER) p->key_parts = 2;
  }
  if (room > kMostTokens) return KVQ_ERR_UNSUPPORTED;
  p->num_tiers = c.num_tiers;
  p->k_signs = c0->k_signs;
  p->v_signs = c0->v_signs;
  p->batch = c.batch;
  p->num_tokens = c.num_tokens;
  p->hq = c.hq;
  p->hkv = hkv;
  p->group = c.hq / hkv;
  while ((1 << p->group_shift) < p->group) ++p->group_shift;
  p->page_size = c0->page_size;
  p->page_shift = page_shift_of(c0->page_size);
  p->window = c.visible ? (int)std::min<long long>(c.visible->window, kMostTokens) : 0;  // (all there can be)
  p->sinks = c.visible ? (int)std::min<long long>(c.visible->sinks, kMostTokens) : 0;
  p->head_dim = d;
  p->sms = device_sms();
  // Sequences of few rows stay packed where the prefix kernel takes all formats.  (A batch that is long in the mean could
  // be unpacked as a whole, which saves a launch whose blocks find nothing to do, but not where single tokens stand
  // beside a long chunk.  Measured (GB300, 32/8 heads, fp8 keys and INT4 values), by sequence and as a whole: 4 x 2048
  // tokens 278 and 275 us, 16 x 600 on 1000 393 and 389; 8192 and 15 x 1 on 4000 1054 and 1102, 2048 and 3 x 1 on 8000 370
  // and 380, 4096 and 7 x 1 on 30000 2173 and 2188.)
  const long long rows = (long long)c.num_tokens * p->group, seqs = std::min(c.batch, c.num_tokens);
  p->dense_rows = seqs == 1 && rows > kDenseRows ? -1 : kDenseRows;
  for (int i = 0; i < c.num_tiers; ++i) {
    const kvq_cache* k = c.tiers[i].cache;
    if (!shared_tier_supported(d, k->k_format, k->v_format) || (k->v_format == KVQ_FMT_INT4_G32 && !aligned(k->v_aux, 8)))
      p->dense_rows = -1;
  }
  // capacities
  const long long dense_seqs = p->dense_rows < 0 ? seqs : std::min(seqs, rows / (p->dense_rows + 1LL));
  const long long blocks = c.offsets ? rows / kChunkRows + seqs : seqs;
  const long long tile = dense_tile(d), unit_rows = kChunkRows * dense_blocks(d);
  const long long most = p->window ? std::min(room, (long long)p->window) + std::min(room, (long long)p->sinks) : room;
  const long long tiles = dense_seqs ? dense_seqs * (most / tile + 4) + c.num_tokens / tile : 0;
  const long long units = dense_seqs ? rows / unit_rows + dense_seqs : 0;
  const long long extra = (2LL * p->sms + hkv - 1) / hkv, packed = p->dense_rows < 0 ? 0 : std::min(blocks, seqs * (p->dense_rows / kChunkRows));
  const long long items[2] = {units ? units + extra : 0, packed ? packed * c.num_tiers + extra : 0};
  const long long parts = items[0] * dense_blocks(d) + items[1] * 2;
  if (tiles * hkv > 0x7FFFFFFFLL || parts * hkv * kChunkRows > 0x7FFFFFFFLL) return KVQ_ERR_UNSUPPORTED;
  p->max_blocks = (int)blocks;
  p->max_tiles = (int)tiles;
  p->max_parts = (int)parts;
  p->max_units[0] = (int)units;
  p->max_units[1] = (int)packed;
  p->max_items[0] = (int)items[0];
  p->max_items[1] = (int)items[1];
  p->extra_items = (int)extra;
  return KVQ_OK;
}

// Lays the workspace out from `base` on; returns its bytes.
size_t chunk_layout(ChunkParams* p, uint8_t* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* x = base + at;
    at += align_up(bytes, 256);
    return x;
  };
  const size_t d = p->head_dim, hkv = p->hkv, tile = dense_tile(p->head_dim), tiles = p->max_tiles;
  p->head = reinterpret_cast<ChunkHead*>(take(sizeof(ChunkHead)));
  p->seq = reinterpret_cast<ChunkSeq*>(take(p->batch * sizeof(ChunkSeq)));
  p->block = reinterpret_cast<ChunkBlock*>(take(p->max_blocks * sizeof(ChunkBlock)));
  for (int i = 0; i < 2; ++i) p->unit[i] = reinterpret_cast<ChunkUnit*>(take(p->max_units[i] * sizeof(ChunkUnit)));
  for (int i = 0; i < 3; ++i) {
    p->unit_items[i] = reinterpret_cast<int*>(take(p->max_units[i > 0] * sizeof(int)));
    p->item[i] = reinterpret_cast<ChunkItem*>(take(p->max_items[i > 0] * sizeof(ChunkItem)));
  }
  p->ml = reinterpret_cast<float2*>(take(p->max_parts * hkv * kChunkRows * sizeof(float2)));
  p->acc = reinterpret_cast<float*>(take(p->max_parts * hkv * kChunkRows * d * sizeof(float)));
  p->qt = take(p->max_units[0] * hkv * dense_blocks(p->head_dim) * 2 * kChunkRows * d * 2);
  p->kt = take(p->key_parts * tiles * hkv * tile * d * 2);
  p->vt = take(tiles * hkv * tile * d * 2);
  if (p->codes) {
    p->kn = reinterpret_cast<float*>(take(tiles * hkv * tile * sizeof(float)));
    p->fn = reinterpret_cast<float*>(take(tiles * hkv * tile * sizeof(float)));
    p->hn = reinterpret_cast<__half*>(take(p->summed * tiles * hkv * tile * sizeof(__half)));
    p->top = reinterpret_cast<float*>(take(tiles * hkv * sizeof(float)));
  }
  return at;
}

kvq_status chunk_size(const ChunkCall& c, size_t* bytes) {
  if (!bytes) return KVQ_ERR_INVALID_ARGUMENT;
  ChunkParams p;
  const kvq_status st = chunk_plan(c, &p);
  if (st == KVQ_OK) *bytes = chunk_layout(&p, nullptr);
  return st;
}

kvq_status chunk_run(const ChunkCall& c, const kvq_heads& q, const int32_t* offsets, void* workspace, size_t ws_bytes,
                     int32_t* status, cudaStream_t stream) {
  ChunkParams p;
  kvq_status st = chunk_plan(c, &p);
  if (st != KVQ_OK) return st;
  if (status && !aligned(status, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (c.batch == 0 || c.num_tokens == 0) return KVQ_OK;
  if ((st = check_heads(&q, c.num_tokens, p.head_dim, true)) != KVQ_OK) return st;
  if (!aligned(q.x, 16) || !aligned(q.out, 16) ||
      (q.x_token_stride | q.x_head_stride | q.out_token_stride | q.out_head_stride) % 8)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (c.offsets && !aligned(offsets, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (!workspace || !aligned(workspace, 256)) return KVQ_ERR_INVALID_ARGUMENT;
  if (chunk_layout(&p, static_cast<uint8_t*>(workspace)) > ws_bytes) return KVQ_ERR_WORKSPACE_TOO_SMALL;
  p.q = q.x;
  p.out = q.out;
  p.q_token = q.x_token_stride;
  p.q_head = q.x_head_stride;
  p.out_token = q.out_token_stride;
  p.out_head = q.out_head_stride;
  p.offsets = c.offsets ? offsets : nullptr;
  p.status = status;
  cudaError_t e = launch_chunk_plan(p, stream);
  if (e == cudaSuccess && p.max_units[0]) e = launch_chunk_prepare(p, stream);
  if (e == cudaSuccess && p.max_units[0]) e = launch_chunk_dense(p, stream);
  if (e == cudaSuccess && p.max_units[1]) e = launch_chunk_packed(p, p.max_units[0] > 0, stream);
  if (e == cudaSuccess) e = launch_chunk_join(p, stream);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace
}  // namespace kvq

extern "C" {

KVQ_API kvq_status kvq_chunk_workspace_size(const kvq_tier_view* tiers, int32_t num_tiers, int32_t batch,
                                            int32_t num_tokens, int32_t num_q_heads, const kvq_visible* visible,
                                            size_t* bytes) {
  return chunk_size({tiers, num_tiers, batch, num_tokens, num_q_heads, true, visible}, bytes);
}

KVQ_API kvq_status kvq_chunk_attention(const kvq_tier_view* tiers, int32_t num_tiers, const kvq_heads* q,
                                       const int32_t* q_offsets, int32_t batch, int32_t num_tokens,
                                       const kvq_visible* visible, void* workspace, size_t workspace_bytes,
                                       int32_t* status, void* stream) {
  if (!q) return KVQ_ERR_INVALID_ARGUMENT;
  return chunk_run({tiers, num_tiers, batch, num_tokens, q->num_heads, q_offsets != nullptr, visible}, *q, q_offsets,
                   workspace, workspace_bytes, status, static_cast<cudaStream_t>(stream));
}

// One token a sequence runs on the decode kernels where their plan allows it, else as a chunk call.
KVQ_API kvq_status kvq_decode_window_workspace_size(const kvq_tier_view* tiers, int32_t num_tiers, int32_t batch,
                                                    int32_t num_q_heads, const kvq_visible* visible, size_t* bytes) {
  const ChunkCall c = {tiers, num_tiers, batch, batch, num_q_heads, false, visible};
  if (!bytes) return KVQ_ERR_INVALID_ARGUMENT;
  ChunkParams p;
  const kvq_status st = chunk_plan(c, &p);
  if (st != KVQ_OK) return st;
  if (!window_plan(tiers, num_tiers, batch, num_q_heads, p.window, p.sinks, bytes)) *bytes = chunk_layout(&p, nullptr);
  return KVQ_OK;
}

KVQ_API kvq_status kvq_decode_attention_window(const kvq_tier_view* tiers, int32_t num_tiers, const uint16_t* q,
                                               int32_t batch, int32_t num_q_heads, const kvq_visible* visible,
                                               uint16_t* out, void* workspace, size_t workspace_bytes,
                                               int32_t* status, void* stream) {
  const ChunkCall c = {tiers, num_tiers, batch, batch, num_q_heads, false, visible};
  const int64_t d = tiers && num_tiers > 0 && tiers[0].cache ? tiers[0].cache->head_dim : 0;
  const kvq_heads h = {q, out, num_q_heads, num_q_heads * d, d, num_q_heads * d, d};
  ChunkParams p;
  const kvq_status st = chunk_plan(c, &p);
  if (st != KVQ_OK) return st;
  size_t need;
  if (!window_plan(tiers, num_tiers, batch, num_q_heads, p.window, p.sinks, &need))
    return chunk_run(c, h, nullptr, workspace, workspace_bytes, status, static_cast<cudaStream_t>(stream));
  if (status && !aligned(status, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (batch == 0) return KVQ_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  if (!workspace || !aligned(workspace, 256)) return KVQ_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < need) return KVQ_ERR_WORKSPACE_TOO_SMALL;
  const cudaError_t e = window_run(tiers, num_tiers, q, batch, num_q_heads, p.window, p.sinks, out, workspace, status,
                                   static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
