// Internal declarations of attention over chunks of new tokens (kvq_chunk_attention) and of the
// windowed decode (kvq_decode_attention_window).
//
// Sequence b holds len tokens, its tiers' one after the other; its chunk is the last `tokens` of
// them, and query i of the chunk stands at position p = len - tokens + i.  It sees position t where
//   t <= p  and  (window == 0  or  t > p - window  or  t < sinks).
// Query heads that share a kv head are rows of one matrix: row r of a sequence is head r % group of
// token r / group.  128 neighbouring rows make a row block.
#pragma once
#include "kvq_internal.cuh"

namespace kvq {

constexpr int kChunkRows = 128;
constexpr int kMaskedTile = 128;  // tokens of a tile of the packed path

// Tokens of a tile, row blocks of a work item and buffers of keys or values of the unpacked path.
__host__ __device__ constexpr int dense_tile(int d) { return d == 256 ? 64 : 128; }
__host__ __device__ constexpr int dense_blocks(int d) { return d == 256 ? 1 : 2; }

struct ChunkTier {
  const uint8_t* k_rows;
  const uint8_t* v_rows;
  const __half* k_aux;
  const __half* v_aux;
  const float* k_cent;
  const float* v_cent;
  const float* k_qjl;
  const int32_t* k_outl;
  const int32_t* block_table;  // [batch][table_pages]
  const int32_t* lens;         // [batch]
  int k_fmt, v_fmt, k_bits, v_bits, k_row_bytes, v_row_bytes;
  int num_pages, max_pages, table_pages;
};

// What the plan says of a sequence.
struct ChunkSeq {
  int q0, tokens, len;        // first token in q, tokens of the chunk, cached tokens
  int first_block;            // its first row block
  int base[KVQ_MAX_TIERS];    // position of each tier's first token
  int dense;                  // takes the unpacked path
  int tile0, sink_tiles, window_tile, tiles;  // its unpacked tiles: those of the sinks, then all from window_tile on
  int unit0;                  // its first unit of work (row block, or dense_blocks of them)
};

// A row block: where its partial results lie (in partials of kChunkRows rows and one kv head, all heads of a
// partial side by side); parts -1: nowhere, its one item stores its rows.
struct ChunkBlock {
  int seq, row0;  // of the sequence's rows
  int part0, parts, step;
  int pad[3];
};

// A unit of work: a sequence's rows from row0 on and the tiles they see, in one tier: `sinks` tiles from 0 on, the
// others from `begin` on; n in all.
struct ChunkUnit {
  int seq, row0;
  int n[KVQ_MAX_TIERS], sinks[KVQ_MAX_TIERS], begin[KVQ_MAX_TIERS];
  int pad[2];
};

// A work item (of every kv head): tiles first .. first + count - 1 of a unit's.  part -1: it stores its rows.
struct ChunkItem {
  int seq, row0, tier, part;
  int first, count, sinks, begin;
};

struct ChunkHead {
  int err;            // KVQ_DEVERR_* bits
  int num_blocks;     // row blocks
  int num_tiles;      // unpacked tiles
  int num_dense;      // unpacked sequences' units
  int items[3];       // of the unpacked path; of the packed path on plain formats, on codebooks
  int units[2];       // unpacked, packed
  int pad[7];
  float unscale[KVQ_MAX_TIERS][2];  // what a tier's table values (keys, values) are to be multiplied by
  float beta[KVQ_MAX_TIERS][2];     // scale of the tables
};

struct ChunkParams {
  ChunkTier tier[KVQ_MAX_TIERS];
  int num_tiers;
  const uint16_t* q;
  uint16_t* out;
  long long q_token, q_head, out_token, out_head;  // strides in elements
  const int32_t* offsets;  // null: one token a sequence
  const int8_t* k_signs;
  const int8_t* v_signs;
  int* status;
  int batch, num_tokens, hq, hkv, group, group_shift, page_size, page_shift, window, sinks, head_dim;
  int codes;       // norms beside the unpacked tiles: 1: the one tier is of codebooks, 2: one of several is
  int summed;      // codebook values of four bits: weights are summed as they are rounded
  int key_parts;   // fp16 numbers of an unpacked key's coordinate: 2 where a tier's keys have a sketch or an outlier stream
  int dense_rows;  // sequences of more rows a kv head are unpacked (-1: all)
  // capacities that the workspace was laid out for
  int max_blocks, max_tiles, max_parts;
  int max_units[2], max_items[2];  // unpacked, packed
  int extra_items;  // that splitting may add to one a unit and tier
  int sms;
  int wait_first;  // a pass on packed tiles directly behind the plan: it waits for it (else for the pass before, at its end)
  // in the workspace
  ChunkHead* head;
  ChunkSeq* seq;        // [batch]
  ChunkBlock* block;    // [max_blocks]
  ChunkUnit* unit[2];   // [max_units]: unpacked, packed
  int* unit_items[3];   // [max_units] the first of a unit's items in each list
  ChunkItem* item[3];   // [max_items]
  float* acc;           // [max_parts][hkv][kChunkRows][D]
  float2* ml;           // [max_parts][hkv][kChunkRows]: (m, l)
  uint8_t* qt;          // rotated queries of units [max_units][hkv][dense_blocks][2 parts][128 * D * 2]
  uint8_t* kt;          // unpacked keys [max_tiles][hkv][key_parts][tile * D * 2] and
  uint8_t* vt;          // values [max_tiles][hkv][tile * D * 2]
  float* kn;            // [max_tiles][hkv][tile] factors of the scores,
  float* fn;            // of the weights (the mantissas of the values' norms) or, where `summed`, their inverses
  __half* hn;           // where `summed`, those factors
  float* top;           // [max_tiles][hkv] a power of two above a tile's weights' factors
};

cudaError_t launch_dependent(const void* kernel, unsigned grid, unsigned block, size_t smem, const ChunkParams& p,
                             cudaStream_t stream);
cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_join(const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_prepare(const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_dense(const ChunkParams& p, cudaStream_t stream);
// Items on the packed cache (shared_mma.cuh); behind: whether the unpacked path precedes.
cudaError_t launch_chunk_packed(const ChunkParams& p, bool behind, cudaStream_t stream);

// Programmatic dependents: a grid that may start while the one before it drains, and waits for it first of all.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace kvq
