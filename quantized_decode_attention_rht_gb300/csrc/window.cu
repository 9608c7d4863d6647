// The windowed decode on the decode kernels (kvq_decode_attention_window).
//
// The newest token of a sequence of L sees [0, sinks) and [L - window, L).  Of a tier's tokens these are two
// runs, [0, first) and [from, len).  A narrower block table holds their pages, one run behind the other, and
// the tokens between the runs on the pages where the first ends and the second begins are hidden: one
// interval of the narrower sequence, which the decode kernels leave out (DecTier::hidden).  So a call reads what
// is seen, in whole pages, once.
//
// narrow_kernel writes tables, lengths and intervals, a block a sequence and tier; bounded by its launch and a
// chain of two loads, 3.5 us.  The calls are bounded as their decode kernels are: 64 x 32/8 heads on 4100 tokens of fp8
// keys and INT4 values 99 to 104 us (54 to 57% of the copy rate), 16 x 32 heads on 2064 of 4-bit codes 68 us, 32 x 16/8 heads x 256 on
// up to 1037 of 3/2-bit codes 53 us; 1 x 8 heads on 516 of 4-bit codes 18.5 us, three launches and the loads' latency.
#include "window.cuh"

#include "api_checks.cuh"

namespace kvq {
namespace {

struct NarrowTier {
  const int32_t* table;
  const int32_t* lens;
  int32_t* to_table;  // [batch][to_pages]
  int32_t* to_lens;   // [batch]
  int2* hidden;       // [batch]
  int max_pages, table_pages, to_pages;
};
struct NarrowParams {
  NarrowTier tier[KVQ_MAX_TIERS];
  int num_tiers, batch, page_size, window, sinks;
  int* counters;  // 64, cleared for the kernels behind
  int* bits;      // [batch][num_tiers] KVQ_DEVERR_* bits
};

__global__ void __launch_bounds__(128) narrow_kernel(const __grid_constant__ NarrowParams p) {
  const int b = blockIdx.x, ti = blockIdx.y, ps = p.page_size;
  const NarrowTier& t = p.tier[ti];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the decode kernels wait where they need this)
  if (b == 0 && ti == 0 && threadIdx.x < 64) p.counters[threadIdx.x] = 0;
  int bits = 0, base = 0, all = 0, len = 0;
#pragma unroll
  for (int k = 0; k < KVQ_MAX_TIERS; ++k) {
    if (k >= p.num_tiers) continue;
    const int n = checked_len(__ldg(p.tier[k].lens + b), p.tier[k].max_pages, ps, &bits);
    if (k == ti) {
      base = all;
      len = n;
    }
    all += n;
  }
  const int from = min(len, max(0, max(0, all - p.window) - base)), first = min(from, max(0, p.sinks - base));
  // A tier that ends before the window has no second run: its last page, full or not, goes with the tokens on it.
  const int end = from < len ? len : first, last = (end + ps - 1) / ps;
  const int page1 = from < len ? from / ps : last, pages0 = min((first + ps - 1) / ps, page1);  // the second run's first page, the first run's pages
  const int pages = pages0 + last - page1, moved = (page1 - pages0) * ps;
  const int32_t* row = t.table + (size_t)b * t.table_pages;
  for (int i = threadIdx.x; i < pages; i += 128)
    t.to_table[(size_t)b * t.to_pages + i] = __ldg(row + (i < pages0 ? i : page1 + i - pages0));
  if (threadIdx.x == 0) {
    t.to_lens[b] = end - moved;
    t.hidden[b] = make_int2(first, from < len ? from - moved - first : 0);
    p.bits[b * p.num_tiers + ti] = bits;
  }
}

// A window is a small cache, whose chunks the decode's plan makes too long for a full GPU: codebook tiers get 24 items
// an SM (54 with one query head a kv head; of 32 x 8 heads on 66 pages that is four pages an item), others on the
// generic kernel four.  Measured (GB300), with the plan's chunks and with these: 32 x 16/8 heads x 256 on 1037 tokens of 3/2-bit codes 85 and 56 us, 1 x 8 heads on 516 of
// 4-bit 38 and 24, 8 x 32/8 heads on 1024 of 4-bit 42 and 32, 16 x 16/4 heads x 64 on 1024 42 and 30; 16 x 32 heads on
// 2064 71 and 71.  (fp16 and fp8 tiers: no change, 64 x 32/8 heads on 4100 tokens 112 us.)
void shorten_chunks(const kvq_tier_view* tiers, int n, int batch, int hq, Plan* plan) {
  Plan x = *plan;
  const int sms = device_sms(), hkv = tiers[0].cache->num_kv_heads, ps = tiers[0].cache->page_size;
  x.total = 0;
  for (int i = 0; i < n; ++i) {
    const long long pages = (long long)batch * hkv * usable_pages(tiers[i]), room = (long long)usable_pages(tiers[i]) * ps;
    long long chunk = x.chunk[i];
    if (x.kind[i] == TIER_CB) chunk = std::min(chunk, std::max(1LL, pages / (sms * (hq == hkv ? 54LL : 24LL))) * ps);
    if (x.kind[i] == TIER_GENERIC) chunk = std::min(chunk, std::max((64LL + ps - 1) / ps, pages / (sms * 4LL)) * ps);
    x.chunk[i] = (int)chunk;
    x.splits[i] = room ? (int)((room + chunk - 1) / chunk) : 0;
    x.total += x.splits[i];
  }
  if (x.total <= KVQ_MAX_SPLITS) *plan = x;
}

// Tiers as the decode kernels see them, in the workspace from `base` on.
struct Narrowed {
  kvq_tier_view view[KVQ_MAX_TIERS];
  NarrowParams narrow;
  Plan plan;
  size_t decode_bytes, total;
  bool sketch;
};

bool narrowed(const kvq_tier_view* tiers, int n, int batch, int hq, int window, int sinks, uint8_t* base, Narrowed* x) {
  memset(static_cast<void*>(x), 0, sizeof(*x));
  const kvq_cache* c0 = tiers[0].cache;
  const int ps = c0->page_size;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* y = base + at;
    at += align_up(bytes, 256);
    return y;
  };
  for (int i = 0; i < n; ++i) x->view[i] = tiers[i];
  if (window) {
    NarrowParams& p = x->narrow;
    p.num_tiers = n;
    p.batch = batch;
    p.page_size = ps;
    p.window = window;
    p.sinks = sinks;
    for (int i = 0; i < n; ++i) {
      NarrowTier& t = p.tier[i];
      t.table = tiers[i].block_table;
      t.lens = tiers[i].seq_lens;
      t.max_pages = usable_pages(tiers[i]);
      t.table_pages = tiers[i].max_pages;
      // (a run of m tokens touches at most (m - 1) / ps + 2 pages)
      t.to_pages = (int)std::min<long long>(t.max_pages, (sinks + (ps - 1LL)) / ps + (window + (ps - 1LL)) / ps + 1);
      t.to_table = reinterpret_cast<int32_t*>(take((size_t)batch * t.to_pages * 4));
      t.to_lens = reinterpret_cast<int32_t*>(take((size_t)batch * 4));
      t.hidden = reinterpret_cast<int2*>(take((size_t)batch * 8));
      x->view[i].block_table = t.to_table;
      x->view[i].seq_lens = t.to_lens;
      x->view[i].max_pages = t.to_pages;
    }
    p.bits = reinterpret_cast<int*>(take((size_t)batch * n * 4));
  }
  if (make_plan(x->view, n, batch, hq, 0, true, &x->plan) != KVQ_OK) return false;
  if (window) shorten_chunks(x->view, n, batch, hq, &x->plan);
  x->sketch = has_sketch(x->view, n);
  x->decode_bytes = workspace_bytes(batch, hq, c0->head_dim, x->plan.total, x->sketch);
  x->total = at + x->decode_bytes;
  return true;
}

}  // namespace

bool window_plan(const kvq_tier_view* tiers, int num_tiers, int batch, int hq, int window, int sinks, size_t* bytes) {
  Narrowed x;
  if (!narrowed(tiers, num_tiers, batch, hq, window, sinks, nullptr, &x)) return false;
  *bytes = x.total;
  return true;
}

cudaError_t window_run(const kvq_tier_view* tiers, int num_tiers, const uint16_t* q, int batch, int hq, int window, int sinks,
                       uint16_t* out, void* workspace, int* status, cudaStream_t stream) {
  Narrowed x;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (!narrowed(tiers, num_tiers, batch, hq, window, sinks, ws, &x)) return cudaErrorInvalidValue;
  const kvq_cache* c0 = tiers[0].cache;
  DecParams p;
  fill_decode(x.view, num_tiers, x.plan, q, batch, hq, ws + (x.total - x.decode_bytes), x.sketch, &p);
  p.out16 = out;
  p.status = status;
  int* counters = reinterpret_cast<int*>(ws + x.total - 256);  // work counters and the error word
  p.err = counters + kErrorWord;
  cudaError_t e;
  if (window) {
    const int ps = c0->page_size;
    for (int i = 0; i < num_tiers; ++i) {
      p.tier[i].hidden = x.narrow.tier[i].hidden;
      p.tier[i].hide_end = (int)std::min<long long>(((sinks + (ps - 1LL)) / ps + 1) * ps, 0x7FFFFFFF);
    }
    p.more_bits = x.narrow.bits;
    x.narrow.counters = counters;
    narrow_kernel<<<dim3((unsigned)batch, (unsigned)num_tiers), 128, 0, stream>>>(x.narrow);
    if ((e = cudaGetLastError()) == cudaSuccess) note_launch();
  } else {
    e = cudaMemsetAsync(counters, 0, 256, stream);
  }
  bool fam[3] = {false, false, false};
  for (int i = 0; i < num_tiers; ++i) fam[x.plan.kind[i]] = true;
  if (e == cudaSuccess && fam[TIER_GQA]) e = launch_decode_gqa(p, counters + kGqaCounter, stream, fam[TIER_CB], window != 0);
  if (e == cudaSuccess && fam[TIER_CB])
    e = (window ? launch_decode_cb_hiding : launch_decode_cb)(p, c0->head_dim, counters, stream, fam[TIER_GQA] || window);
  if (e == cudaSuccess && fam[TIER_GENERIC]) e = launch_decode(p, c0->head_dim, hq / c0->num_kv_heads, stream);
  if (e == cudaSuccess) e = launch_combine(p, c0->head_dim, stream);
  return e;
}

}  // namespace kvq
