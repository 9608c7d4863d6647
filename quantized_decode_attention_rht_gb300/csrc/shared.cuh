// Internal declarations of the shared-prefix decode (kvq_decode_attention_shared).
#pragma once
#include "kvq_internal.cuh"

namespace kvq {

// Tokens of a tile, query rows of a work item.
constexpr int kTileTokens = 128, kTileRows = 128;

struct SharedTier {
  const uint8_t* k_rows;
  const uint8_t* v_rows;
  const __half* k_aux;
  const __half* v_aux;
  const float* k_cent;
  const float* v_cent;
  const int32_t* block_table;  // [groups][max_pages]
  const int32_t* lens;         // [groups]
  int k_fmt, v_fmt, k_bits, v_bits, k_row_bytes, v_row_bytes;
  int num_pages, max_pages;
  int split_begin, num_splits;
  int first;  // first split of the tier in its launch
};

struct SharedParams {
  SharedTier tier[KVQ_MAX_TIERS];
  int num_tiers, num_groups;
  const __half* q;        // queries [batch * hq][128]
  const int8_t* k_signs;  // [hkv][128]
  float* acc;        // partials [2 * splits][batch * hq][128]: of each split's even and odd tiles
  float* ml;         // (max, sum) [2 * splits][batch * hq][2]
  int* err;
  int batch, hq, hkv, group, page_size, page_shift;
  int total_splits, num_blocks;           // num_blocks: row blocks of all groups
  int offset[KVQ_MAX_PREFIX_GROUPS + 1];    // first sequence of each group
  int block[KVQ_MAX_PREFIX_GROUPS + 1];     // first row block of each group
};

bool shared_tier_supported(int head_dim, int k_fmt, int v_fmt);
cudaError_t launch_shared_prefix(const SharedParams& p, cudaStream_t stream);

}  // namespace kvq
