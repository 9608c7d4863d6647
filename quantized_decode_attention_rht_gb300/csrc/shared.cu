// Decode attention for groups of sequences that share a cached prefix
// (kvq_decode_attention_shared): host side and the pass that
// joins the partial results.
//
// With O_i = sum_t 2^(s_t - m_i) V_t, l_i = sum_t 2^(s_t - m_i) over the tokens of part i of a
// row's context and m_i the part's largest score, the row's output is
//   (sum_i 2^(m_i - m) O_i) / (sum_i 2^(m_i - m) l_i),   m = max_i m_i,
// whatever the parts are: chunks of the prefix (shared_mma.cu) and split-K chunks of the
// sequence's own tiers (the decode kernels).  The value rotation is undone once, at the end.
//
// Where the prefix kernel is not built for a prefix's formats or head_dim, the prefix is
// attended as one more tier of every sequence: block tables and lengths of the groups are
// copied to their sequences, and the ordinary decode runs over all tiers.
#include "api_checks.cuh"
#include "quantize_small.cuh"
#include "shared.cuh"

namespace kvq {
namespace {

// ------------------------------------------------------------------------ joining
struct JoinTier {  // of the sequences' own
  const int32_t* seq_lens;
  int max_pages, chunk, num_splits, split_begin;
};
struct JoinParams {  // small: a launch's parameters are read through a cold cache
  const float* acc;  // the prefix's partials [2 * splits][rows][128], (max, sum) beside them
  const float2* ml;
  const float* own_acc;  // [rows][own splits][128]
  const float2* own_ml;
  const int8_t* v_signs;
  __half* out;
  int* status;
  int* err;
  int batch, hq, group_shift, page_size;
  int splits, own_splits, num_tiers, num_groups;
  JoinTier tier[KVQ_MAX_TIERS];
  const int32_t* idle_lens[KVQ_MAX_TIERS];  // per group, of prefix tiers without pages: 0, or out of range
  int num_idle;
  int offset[KVQ_MAX_PREFIX_GROUPS + 1];
};

// Where row (b, h)'s partials lie: the prefix's first, then those of the sequence's tiers.
struct Parts {
  int pre;                       // prefix partials, two a split
  int own[KVQ_MAX_TIERS];        // split-K chunks of each tier that hold tokens
  int total;
};

__device__ __forceinline__ void find_prefix_parts(const JoinParams& p, int b, Parts& n) {
  int lo = 0, hi = p.num_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.offset[mid] <= b) lo = mid;
    else hi = mid;
  }
  const int first = p.offset[lo], end = p.offset[lo + 1];
  n.pre = b >= first && b < end ? 2 * p.splits : 0;
}
__device__ __forceinline__ void find_own_parts(const JoinParams& p, const int (&lens)[KVQ_MAX_TIERS], Parts& n) {
  n.total = n.pre;
#pragma unroll
  for (int i = 0; i < KVQ_MAX_TIERS; ++i) {
    n.own[i] = 0;
    if (i < p.num_tiers) {
      int bits = 0;
      n.own[i] = splits_holding_tokens(checked_len(lens[i], p.tier[i].max_pages, p.page_size, &bits), p.tier[i].chunk,
                                       p.tier[i].num_splits);
      n.total += n.own[i];
    }
  }
}

// Partial j of the row: its (max, sum) and accumulator.
__device__ __forceinline__ size_t prefix_part(const JoinParams& p, size_t row, int j) {
  return (size_t)j * p.batch * p.hq + row;
}
__device__ __forceinline__ size_t own_part(const JoinParams& p, const Parts& n, size_t row, int j) {
  int split = 0;
  j -= n.pre;
#pragma unroll
  for (int i = 0; i < KVQ_MAX_TIERS; ++i) {
    if (j >= 0 && j < n.own[i]) split = p.tier[i].split_begin + j;
    j -= n.own[i];
  }
  return row * p.own_splits + split;
}

// kRowWarps warps per row: one where rows have few partials, eight where they have many (more than 24:
// one warp would wait for its accumulators in turn).  Bounded by the latency of two dependent
// loads, (max, sum) and accumulator: 3 to 4.5 us behind the passes.
template <int kRowWarps>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinParams p) {
  constexpr int kRows = 8 / kRowWarps;
  __shared__ float s_acc[kRowWarps > 1 ? kRowWarps : 1][128];
  __shared__ float s_l[kRowWarps], s_m[kRowWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kRows + warp / kRowWarps;
  const int part = warp % kRowWarps, j0 = lane * kRowWarps + part;
  const bool there = row < (long long)p.batch * p.hq;  // whole warps; with eight warps a row, whole blocks
  const int b = there ? (int)(row / p.hq) : 0, h = there ? (int)(row - (long long)b * p.hq) : 0;
  Parts n;
  find_prefix_parts(p, b, n);
  const uint32_t sg =
      __ldg(reinterpret_cast<const uint32_t*>(p.v_signs + (size_t)(h >> p.group_shift) * 128) + lane);
  int lens[KVQ_MAX_TIERS];
#pragma unroll
  for (int i = 0; i < KVQ_MAX_TIERS; ++i) lens[i] = i < p.num_tiers ? __ldg(p.tier[i].seq_lens + b) : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // every partial is complete
  if (p.status && blockIdx.x == gridDim.x - 1) {  // a block of its own
    int bits = 0;  // lengths out of range, of sequences; the prefix pass reports its own
    for (int i = threadIdx.x; i < p.batch * p.num_tiers; i += 256) {
      const JoinTier& T = p.tier[i % p.num_tiers];
      checked_len(T.seq_lens[i / p.num_tiers], T.max_pages, p.page_size, &bits);
    }
    for (int i = threadIdx.x; i < p.num_groups * p.num_idle; i += 256)
      if (p.offset[i / p.num_idle] < p.offset[i / p.num_idle + 1])
        checked_len(p.idle_lens[i % p.num_idle][i / p.num_idle], 0, p.page_size, &bits);
    if (bits) atomicOr(p.err, bits);
    __syncthreads();
    if (threadIdx.x == 0) *p.status = *reinterpret_cast<volatile int*>(p.err);
    return;
  }
  if (!there) return;
  // a lane looks after one partial at a time: its (max, sum) and where its accumulator lies
  float2 x0 = make_float2(-INFINITY, 0.f), x;
  const float* acc0 = nullptr;
  if (j0 < n.pre) {
    const size_t at = prefix_part(p, row, j0);
    x0 = p.ml[at];
    acc0 = p.acc + at * 128;
  }
  find_own_parts(p, lens, n);
  if (j0 >= n.pre && j0 < n.total) {
    const size_t at = own_part(p, n, row, j0);
    x0 = p.own_ml[at];
    acc0 = p.own_acc + at * 128;
  }
  auto look = [&](int j, float2& y) -> const float* {
    y = make_float2(-INFINITY, 0.f);
    if (j >= n.total) return nullptr;
    const size_t at = j < n.pre ? prefix_part(p, row, j) : own_part(p, n, row, j);
    y = j < n.pre ? p.ml[at] : p.own_ml[at];
    return (j < n.pre ? p.acc : p.own_acc) + at * 128;
  };
  float mx = x0.x;
  for (int j = j0 + 32 * kRowWarps; j < n.total; j += 32 * kRowWarps) {
    look(j, x);
    mx = fmaxf(mx, x.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if constexpr (kRowWarps > 1) {
    if (lane == 0) s_m[part] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) mx = fmaxf(mx, s_m[i]);
  }
  float y[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  for (int first = 0; first < n.total; first += 32 * kRowWarps) {  // once, but for very many partials
    const float* acc = acc0;
    x = x0;
    if (first) acc = look(first + j0, x);
    float f = 0.f;  // a part without tokens leaves its accumulator unwritten: weight 0, not read
    if (x.x != -INFINITY) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(x.x - mx));
    l = fmaf(x.y, f, l);
    const int live = min(32, (n.total - first - part + kRowWarps - 1) / kRowWarps);
#pragma unroll 8
    for (int i = 0; i < live; ++i) {
      const float fi = __shfl_sync(0xFFFFFFFFu, f, i);
      const float* ai = reinterpret_cast<const float*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(acc), i));
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (fi != 0.f) a = reinterpret_cast<const float4*>(ai)[lane];
      y[0] = fmaf(a.x, fi, y[0]);
      y[1] = fmaf(a.y, fi, y[1]);
      y[2] = fmaf(a.z, fi, y[2]);
      y[3] = fmaf(a.w, fi, y[3]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  if constexpr (kRowWarps > 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) s_acc[part][4 * lane + k] = y[k];
    if (lane == 0) s_l[part] = l;
    __syncthreads();
    if (part) return;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = 0.f;
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) {
      l += s_l[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] += s_acc[i][4 * lane + k];
    }
  }
  // No token at all: zeros.  (A query that is not finite has no maximum and a sum of NaN: NaN.)
  const float inv = l == 0.f ? 0.f : inv_sqrt_dim(128) / l;
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] *= inv;
  sign_free_rotate<4>(lane, y);
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = (sg >> (8 * k)) & 0x80u ? -y[k] : y[k];
  const __half2 a = __floats2half2_rn(y[0], y[1]), c = __floats2half2_rn(y[2], y[3]);
  reinterpret_cast<uint2*>(p.out + row * 128)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
}

// ------------------------------------------------------------------------ prefix as a tier of every sequence
// (Two small kernels around the ordinary decode, which they add a launch each to.)
struct SpreadParams {
  const int32_t* table;
  const int32_t* lens;
  int32_t* seq_table;  // [batch][max_pages]
  int32_t* seq_lens;   // [batch]
  int max_pages, batch, num_groups;
  int offset[KVQ_MAX_PREFIX_GROUPS + 1];
};

__global__ void __launch_bounds__(256) spread_kernel(const __grid_constant__ SpreadParams p) {
  const long long n = (long long)p.batch * max(1, p.max_pages);
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const int b = (int)(i / max(1, p.max_pages)), page = (int)(i - (long long)b * max(1, p.max_pages));
    int lo = 0, hi = p.num_groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.offset[mid] <= b) lo = mid;
      else hi = mid;
    }
    const bool in = b >= p.offset[lo] && b < p.offset[lo + 1];
    if (page < p.max_pages) p.seq_table[(size_t)b * p.max_pages + page] = in ? p.table[(size_t)lo * p.max_pages + page] : 0;
    if (page == 0) p.seq_lens[b] = in ? p.lens[lo] : 0;
  }
}

__global__ void __launch_bounds__(256) round_kernel(const float4* x, uint2* out, long long n) {
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const float4 v = x[i];
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    out[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// ------------------------------------------------------------------------ plan
struct SharedPlan {
  bool fast;
  // prefix pass
  int splits[KVQ_MAX_TIERS], total_splits, num_blocks;
  int block[KVQ_MAX_PREFIX_GROUPS + 1];
  // the sequences' own tiers (fast), or all tiers (otherwise)
  Plan dec;
  bool sketch;
  // workspace: byte offsets
  size_t dec_bytes, acc, ml, tables, lens, out32, total;
};

struct Call {
  const kvq_tier_view* prefix;
  const kvq_tier_view* tiers;
  const int32_t* offsets;
  int num_prefix, num_tiers, num_groups, batch, hq;
};

kvq_status check_call(const Call& c, kvq_tier_view* all) {
  if (!c.prefix || c.num_prefix < 1 || c.num_tiers < 0 || c.num_prefix + c.num_tiers > KVQ_MAX_TIERS ||
      (c.num_tiers > 0 && !c.tiers) || !c.offsets || c.batch < 0 || c.hq < 1)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (c.num_groups < 1 || c.num_groups > KVQ_MAX_PREFIX_GROUPS) return KVQ_ERR_INVALID_ARGUMENT;
  if (c.offsets[0] < 0 || c.offsets[c.num_groups] > c.batch) return KVQ_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < c.num_groups; ++i)
    if (c.offsets[i + 1] < c.offsets[i]) return KVQ_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < c.num_prefix; ++i) all[i] = c.prefix[i];
  for (int i = 0; i < c.num_tiers; ++i) all[c.num_prefix + i] = c.tiers[i];
  for (int i = 0; i < c.num_prefix + c.num_tiers; ++i)
    if (!aligned(all[i].block_table, 4) || !aligned(all[i].seq_lens, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  const kvq_status st = check_tiers(all, c.num_prefix + c.num_tiers, c.batch, c.hq);
  if (st != KVQ_OK) return st;
  if ((long long)c.batch * c.hq > (1LL << 24)) return KVQ_ERR_UNSUPPORTED;
  // the prefix pass counts the tokens of a tile, the last one's end among them, in 32 bits
  for (int i = 0; i < c.num_prefix; ++i)
    if ((long long)usable_pages(all[i]) * all[i].cache->page_size > 0x7FFFFFFFLL - 2 * kTileTokens) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

// Chunks of the prefix: enough items to fill the GPU in whole waves, few enough that writing
// and joining partial results does not cost more than the idle SMs would.  In units of one
// tile's time: an item is its tiles plus a fixed start and end, a split's
// partials are a pass over them at memory speed.
int choose_splits(long long row_blocks, long long rows, int max_tiles, int sms, int own_blocks) {
  const double start = 5.0;                                   // tiles' worth of set-up, fill and drain
  const double partial = (double)rows * 2080.0 / 3.5e12 / 1.5e-6;  // write + read of one split's two partials
  int best = 1;
  double least = 1e300;
  // (beyond two waves more splits only add partials)
  const int most = (int)std::min<long long>(std::min(max_tiles, 256), 2LL * sms / std::max<long long>(1, row_blocks) + 1);
  for (int s = 1; s <= most; ++s) {
    const int per = (max_tiles + s - 1) / s;
    if ((max_tiles + per - 1) / per != s) continue;  // the same chunks with fewer splits
    // one wave leaves the sequences' own pass SMs to run on beside it; more make room as they end
    const long long items = row_blocks * s;
    const int room = items <= sms ? std::max(1, sms - own_blocks) : sms;
    const double waves = (double)((items + room - 1) / room);
    const double t = waves * (per + start) + s * partial;
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

kvq_status make_shared_plan(const Call& c, const kvq_tier_view* all, bool q16, SharedPlan* plan) {
  memset(static_cast<void*>(plan), 0, sizeof(*plan));
  const kvq_cache* c0 = all[0].cache;
  const int d = c0->head_dim, ps = c0->page_size, group = c.hq / c0->num_kv_heads;
  plan->fast = q16;
  for (int i = 0; i < c.num_prefix; ++i)
    plan->fast = plan->fast && shared_tier_supported(d, all[i].cache->k_format, all[i].cache->v_format);
  plan->fast = plan->fast && aligned(c0->k_signs, 16) && aligned(c0->v_signs, 16);
  for (int i = 0; i < c.num_prefix; ++i) {
    // the prefix kernel reads INT4 scales four at a time and counts rows in 32 bits
    const kvq_cache* k = all[i].cache;
    plan->fast = plan->fast && (k->v_format != KVQ_FMT_INT4_G32 || aligned(k->v_aux, 8)) &&
                 (long long)k->num_pages * k->page_size * k->num_kv_heads < 0xFFFFFFFFLL;
  }
  kvq_status st;
  size_t at = 0;
  const size_t rows = (size_t)c.batch * c.hq;
  if (!plan->fast) {
    plan->sketch = has_sketch(all, c.num_prefix + c.num_tiers);
    if ((st = make_plan(all, c.num_prefix + c.num_tiers, c.batch, c.hq, 0, q16, &plan->dec)) != KVQ_OK) return st;
    plan->dec_bytes = workspace_bytes(c.batch, c.hq, d, plan->dec.total, plan->sketch);
    at = align_up(plan->dec_bytes, 256);
    plan->tables = at;
    for (int i = 0; i < c.num_prefix; ++i)
      at += align_up((size_t)c.batch * std::max(1, all[i].max_pages) * 4, 256);
    plan->lens = at;
    at += c.num_prefix * align_up((size_t)c.batch * 4, 256);
    plan->out32 = at;
    at += align_up(rows * d * 4, 256);
    plan->total = at;
    return KVQ_OK;
  }
  if (c.num_tiers > 0) {
    const kvq_tier_view* own = all + c.num_prefix;
    plan->sketch = has_sketch(own, c.num_tiers);
    if ((st = make_plan(own, c.num_tiers, c.batch, c.hq, 0, q16, &plan->dec)) != KVQ_OK) return st;
  }
  plan->dec_bytes = workspace_bytes(c.batch, c.hq, d, plan->dec.total, plan->sketch);
  at = align_up(plan->dec_bytes, 256);
  for (int g = 0; g < c.num_groups; ++g) {
    const long long r = (long long)(c.offsets[g + 1] - c.offsets[g]) * group;
    plan->block[g + 1] = plan->block[g] + (int)((r + kTileRows - 1) / kTileRows);
  }
  plan->num_blocks = plan->block[c.num_groups];
  long long tiles[KVQ_MAX_TIERS], sum = 0;
  for (int i = 0; i < c.num_prefix; ++i) {
    tiles[i] = ((long long)usable_pages(all[i]) * ps + kTileTokens - 1) / kTileTokens;
    sum += tiles[i];
  }
  const long long prefix_rows = (long long)(c.offsets[c.num_groups] - c.offsets[0]) * c.hq;
  // A seventh of the SMs is left to the sequences' own pass where one wave holds the prefix: 32 sequences on 32768 +
  // 512 tokens take 50.6 us with it, 60.4 with none and 54.8 with a quarter, 8 x 32 heads on 8192 + 256 take
  // 46.9, 46.8 and 63.3; a fourteenth is as good.  Own lengths of thousands make no difference.
  const int want = sum ? choose_splits((long long)plan->num_blocks * c0->num_kv_heads, prefix_rows,
                                       (int)std::min<long long>(sum, 1 << 30), device_sms(),
                                       c.num_tiers > 0 ? device_sms() / 7 : 0)
                       : 0;
  const long long per = want ? (sum + want - 1) / want : 1;
  for (int i = 0; i < c.num_prefix; ++i) {
    plan->splits[i] = (int)((tiles[i] + per - 1) / per);
    plan->total_splits += plan->splits[i];
  }
  if (plan->num_blocks == 0) plan->total_splits = 0;
  if ((long long)plan->num_blocks * c0->num_kv_heads * plan->total_splits > 0x7FFFFFFFLL) return KVQ_ERR_UNSUPPORTED;
  plan->ml = at;
  at += align_up(2 * (size_t)plan->total_splits * rows * 8, 256);
  plan->acc = at;
  at += align_up(2 * (size_t)plan->total_splits * rows * d * 4, 256);
  plan->total = at;
  return KVQ_OK;
}

cudaError_t launched() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

// The split-K passes over the sequences' own tiers.  after: the prefix pass precedes; the
// fused kernels then start on SMs it leaves idle and complete only after it.
cudaError_t launch_own(const DecParams& p, const Plan& plan, int d, int group, int* counters, bool after, cudaStream_t s) {
  bool fam[3] = {false, false, false};
  for (int i = 0; i < p.num_tiers; ++i) fam[plan.kind[i]] = true;
  cudaError_t e = cudaSuccess;
  if (fam[TIER_GQA]) e = launch_decode_gqa(p, counters + kGqaCounter, s, fam[TIER_CB], after);
  if (e == cudaSuccess && fam[TIER_CB]) e = launch_decode_cb(p, d, counters, s, fam[TIER_GQA] || after);
  if (e == cudaSuccess && fam[TIER_GENERIC]) e = launch_decode(p, d, group, s);
  return e;
}

}  // namespace
}  // namespace kvq

extern "C" {

KVQ_API kvq_status kvq_decode_shared_workspace_size(const kvq_tier_view* prefix_tiers, int32_t num_prefix_tiers,
                                                    const int32_t* group_offsets, int32_t num_groups,
                                                    const kvq_tier_view* tiers, int32_t num_tiers, int32_t batch,
                                                    int32_t num_q_heads, size_t* bytes) {
  if (!bytes) return KVQ_ERR_INVALID_ARGUMENT;
  const Call c = {prefix_tiers, tiers, group_offsets, num_prefix_tiers, num_tiers, num_groups, batch, num_q_heads};
  kvq_tier_view all[KVQ_MAX_TIERS];
  kvq_status st = check_call(c, all);
  if (st != KVQ_OK) return st;
  SharedPlan plan;
  if ((st = make_shared_plan(c, all, true, &plan)) != KVQ_OK) return st;
  *bytes = plan.total;
  return KVQ_OK;
}

KVQ_API kvq_status kvq_decode_attention_shared(const kvq_tier_view* prefix_tiers, int32_t num_prefix_tiers,
                                               const int32_t* group_offsets, int32_t num_groups,
                                               const kvq_tier_view* tiers, int32_t num_tiers, const uint16_t* q,
                                               int32_t batch, int32_t num_q_heads, uint16_t* out, void* workspace,
                                               size_t ws_bytes, int32_t* status, void* stream) {
  const Call c = {prefix_tiers, tiers, group_offsets, num_prefix_tiers, num_tiers, num_groups, batch, num_q_heads};
  kvq_tier_view all[KVQ_MAX_TIERS];
  kvq_status st = check_call(c, all);
  if (st != KVQ_OK) return st;
  if (status && !aligned(status, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (batch == 0) return KVQ_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  SharedPlan plan;
  if ((st = make_shared_plan(c, all, true, &plan)) != KVQ_OK) return st;
  if (!workspace || !aligned(workspace, 256)) return KVQ_ERR_INVALID_ARGUMENT;
  if (ws_bytes < plan.total) return KVQ_ERR_WORKSPACE_TOO_SMALL;
  const kvq_cache* c0 = all[0].cache;
  const int d = c0->head_dim, hkv = c0->num_kv_heads, group = num_q_heads / hkv, sms = device_sms();
  const long long rows = (long long)batch * num_q_heads;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!plan.fast) {
    SpreadParams sp;
    memset(&sp, 0, sizeof(sp));
    for (int g = 0; g <= num_groups; ++g) sp.offset[g] = group_offsets[g];
    sp.num_groups = num_groups;
    sp.batch = batch;
    uint8_t* table = ws + plan.tables;
    e = cudaSuccess;
    for (int i = 0; i < num_prefix_tiers && e == cudaSuccess; ++i) {
      sp.table = all[i].block_table;
      sp.lens = all[i].seq_lens;
      sp.max_pages = all[i].max_pages;
      sp.seq_table = reinterpret_cast<int32_t*>(table);
      sp.seq_lens = reinterpret_cast<int32_t*>(ws + plan.lens + i * align_up((size_t)batch * 4, 256));
      all[i].block_table = sp.seq_table;
      all[i].seq_lens = sp.seq_lens;
      const long long n = (long long)batch * std::max(1, sp.max_pages);
      spread_kernel<<<(unsigned)std::min<long long>((n + 255) / 256, sms * 8LL), 256, 0, s>>>(sp);
      e = launched();
      table += align_up((size_t)n * 4, 256);
    }
    if (e != cudaSuccess) return KVQ_ERR_CUDA;
    float* out32 = reinterpret_cast<float*>(ws + plan.out32);
    kvq_decode_options opts;
    memset(&opts, 0, sizeof(opts));
    opts.status = status;
    if ((st = kvq_decode_attention_ex(all, num_prefix_tiers + num_tiers, q, batch, num_q_heads, 0, out32, ws,
                                      plan.dec_bytes, &opts, stream)) != KVQ_OK)
      return st;
    const long long n = rows * d / 4;
    round_kernel<<<(unsigned)std::min<long long>((n + 255) / 256, sms * 8LL), 256, 0, s>>>(
        reinterpret_cast<const float4*>(out32), reinterpret_cast<uint2*>(out), n);
    return launched() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
  }

  DecParams own;
  memset(&own, 0, sizeof(own));
  if (num_tiers > 0)
    fill_decode(all + num_prefix_tiers, num_tiers, plan.dec, q, batch, num_q_heads, ws, plan.sketch, &own);
  int* counters = reinterpret_cast<int*>(ws + plan.dec_bytes - 256);
  own.err = counters + kErrorWord;
  SharedParams p;
  memset(&p, 0, sizeof(p));
  int at = 0;
  for (int i = 0; i < num_prefix_tiers; ++i) {
    const kvq_cache* k = all[i].cache;
    if (plan.splits[i] == 0) continue;  // a tier without pages
    SharedTier& t = p.tier[p.num_tiers++];
    t.k_rows = static_cast<const uint8_t*>(k->k_rows);
    t.v_rows = static_cast<const uint8_t*>(k->v_rows);
    t.k_aux = static_cast<const __half*>(k->k_aux);
    t.v_aux = static_cast<const __half*>(k->v_aux);
    t.k_cent = k->k_centroids;
    t.v_cent = k->v_centroids;
    t.block_table = all[i].block_table;
    t.lens = all[i].seq_lens;
    t.k_fmt = k->k_format;
    t.v_fmt = k->v_format;
    t.k_bits = k->k_bits;
    t.v_bits = k->v_bits;
    t.k_row_bytes = side_row_bytes(k->k_format, k->k_bits, d);
    t.v_row_bytes = side_row_bytes(k->v_format, k->v_bits, d);
    t.num_pages = k->num_pages;
    t.max_pages = usable_pages(all[i]);
    t.split_begin = at;
    t.num_splits = plan.splits[i];
    at += plan.splits[i];
  }
  p.q = reinterpret_cast<const __half*>(q);
  p.k_signs = c0->k_signs;
  p.acc = reinterpret_cast<float*>(ws + plan.acc);
  p.ml = reinterpret_cast<float*>(ws + plan.ml);
  p.err = own.err;
  p.batch = batch;
  p.hq = num_q_heads;
  p.hkv = hkv;
  p.group = group;
  p.page_size = c0->page_size;
  p.page_shift = page_shift_of(c0->page_size);
  p.num_groups = num_groups;
  p.num_blocks = plan.num_blocks;
  p.total_splits = plan.total_splits;
  for (int g = 0; g <= num_groups; ++g) {
    p.offset[g] = group_offsets[g];
    p.block[g] = plan.block[g];
  }
  JoinParams j;
  memset(&j, 0, sizeof(j));
  j.acc = p.acc;
  j.ml = reinterpret_cast<const float2*>(p.ml);
  j.own_acc = own.ws_acc;
  j.own_ml = reinterpret_cast<const float2*>(own.ws_ml);
  j.v_signs = c0->v_signs;
  j.out = reinterpret_cast<__half*>(out);
  j.status = status;
  j.err = p.err;
  j.batch = batch;
  j.hq = num_q_heads;
  while ((1 << j.group_shift) < group) ++j.group_shift;
  j.page_size = c0->page_size;
  j.splits = p.total_splits;
  j.own_splits = plan.dec.total;
  j.num_tiers = num_tiers;
  j.num_groups = num_groups;
  for (int i = 0; i < num_tiers; ++i)
    j.tier[i] = {own.tier[i].seq_lens, own.tier[i].max_pages, own.tier[i].chunk, own.tier[i].num_splits,
                 own.tier[i].split_begin};
  for (int i = 0; i < num_prefix_tiers; ++i)
    if (plan.splits[i] == 0) j.idle_lens[j.num_idle++] = all[i].seq_lens;
  for (int g = 0; g <= num_groups; ++g) j.offset[g] = group_offsets[g];
  e = cudaMemsetAsync(counters, 0, 256, s);  // work counters and the error word
  const bool prefix = plan.num_blocks > 0 && plan.total_splits > 0;
  if (e == cudaSuccess && prefix) e = launch_shared_prefix(p, s);
  if (e == cudaSuccess && num_tiers > 0) e = launch_own(own, plan.dec, d, group, counters, prefix, s);
  if (e == cudaSuccess) {
    // eight warps a row where a row has many partials (one warp would wait for them in turn)
    const bool many = 2 * plan.total_splits + plan.dec.total > 24;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((many ? rows : (rows + 7) / 8) + (status ? 1 : 0)));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = many ? cudaLaunchKernelEx(&cfg, join_kernel<8>, j) : cudaLaunchKernelEx(&cfg, join_kernel<1>, j);
    if (e == cudaSuccess) e = launched();
  }
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
