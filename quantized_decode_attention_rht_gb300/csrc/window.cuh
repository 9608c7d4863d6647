// Internal declarations of the windowed decode (kvq_decode_attention_window).
#pragma once
#include "kvq_internal.cuh"

namespace kvq {

// Whether the decode kernels run a call with these sizes, and the workspace that it then needs.
bool window_plan(const kvq_tier_view* tiers, int num_tiers, int batch, int hq, int window, int sinks, size_t* bytes);
cudaError_t window_run(const kvq_tier_view* tiers, int num_tiers, const uint16_t* q, int batch, int hq, int window, int sinks,
                       uint16_t* out, void* workspace, int* status, cudaStream_t stream);

}  // namespace kvq
