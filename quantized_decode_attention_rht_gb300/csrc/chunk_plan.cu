// The plan of a chunk call, on the device: lengths and chunk offsets lie there, and a captured call
// reads them when it runs.  One block works out, from them,
//   which positions each row block sees (tiles of the sinks, and from the window's begin to the block's
//   last token),
//   which sequences are unpacked (many rows: chunk_dense.cu) and where their unpacked tiles lie,
//   how the tiles are split where there are too few row blocks to fill the GPU.
// Bounded by latency: 7 to 13 us of dependent loads, scans and barriers, with one sequence or 64; most for codebooks,
// whose tables' scales are chosen here too.  Everything of the call waits for it.
#include "chunk.cuh"
#include "rotate.cuh"
#include "table_scale.cuh"

namespace kvq {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
// A small plan is made in shared memory (a phase then costs a fifth of what it does through L2), and copied out.
constexpr int kNearSeqs = 256, kNearUnits = 384;

struct Sums {
  int a, b, c, d;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) { return {x.a + y.a, x.b + y.b, x.c + y.c, x.d + y.d}; }

// Sums of the threads before this one, on top of `carry`, which grows by the block's.
__device__ __forceinline__ Sums scan(const Sums& mine, Sums& carry, Sums (&warps)[kPlanWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto shift = [&](int x, int o) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    return lane >= o ? y : 0;
  };
  auto sweep = [&](Sums x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) x = x + Sums{shift(x.a, o), shift(x.b, o), shift(x.c, o), shift(x.d, o)};
    return x;
  };
  const Sums in = sweep(mine);
  if (lane == 31) warps[warp] = in;
  __syncthreads();
  if (warp == 0) {
    const Sums w = sweep(warps[lane]);
    warps[lane] = w;
  }
  __syncthreads();
  const Sums before = warp ? warps[warp - 1] : Sums{0, 0, 0, 0};
  const Sums out = {carry.a + before.a + in.a - mine.a, carry.b + before.b + in.b - mine.b,
                    carry.c + before.c + in.c - mine.c, carry.d + before.d + in.d - mine.d};
  carry = carry + warps[kPlanWarps - 1];
  __syncthreads();
  return out;
}

// The largest offset up to this thread's, `carry` among them.
__device__ __forceinline__ int scan_max(int x, int& carry, int (&warps)[kPlanWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x = max(x, y);
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w = max(w, y);
    }
    warps[lane] = w;
  }
  __syncthreads();
  const int before = warp ? max(carry, warps[warp - 1]) : carry;
  carry = max(carry, warps[kPlanWarps - 1]);
  __syncthreads();
  return max(x, before);
}

// The scales of a codebook tier's tables: keys by the first half of the block, values by the second, a candidate a thread.
struct TablePick {
  float least, slope;
  int at;
};
__device__ __forceinline__ void plan_tables(const ChunkParams& p, int tier, TablePick (&picks)[kPlanWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, side = warp / (kPlanWarps / 2);
  const ChunkTier& t = p.tier[tier];
  const int bits = side ? t.v_bits : t.k_bits;
  const float c = lane < (1 << bits) ? __ldg((side ? t.v_cent : t.k_cent) + lane) : 0.f;
  TablePick x;
  table_candidates<1>(c, bits, (int)threadIdx.x % kTableSteps, x.least, x.slope, x.at);
  auto better = [](const TablePick& a, const TablePick& b) { return a.least < b.least || (a.least == b.least && a.at < b.at); };
  auto other = [&](const TablePick& a, int o) {
    return TablePick{__shfl_xor_sync(0xFFFFFFFFu, a.least, o), __shfl_xor_sync(0xFFFFFFFFu, a.slope, o),
                     __shfl_xor_sync(0xFFFFFFFFu, a.at, o)};
  };
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    const TablePick y = other(x, o);
    if (better(y, x)) x = y;
  }
  if (lane == 0) picks[warp] = x;
  __syncthreads();
  if (warp % (kPlanWarps / 2) == 0) {
    x = picks[warp + lane % (kPlanWarps / 2)];
#pragma unroll 1
    for (int o = kPlanWarps / 4; o > 0; o >>= 1) {
      const TablePick y = other(x, o);
      if (better(y, x)) x = y;
    }
    const float beta = exp2f((float)x.at * (1.0f / kTableSteps)) * table_unit(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(c))));
    if (lane == 0) {
      p.head->beta[tier][side] = beta;
      p.head->unscale[tier][side] = inv_sqrt_dim(p.head_dim) * (1.0f - x.slope) / beta;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }
// ceil(a / b) of 0 <= a < 2^24 (tiles), inverse = 1 / b rounded.
__device__ __forceinline__ int ceil_times(int a, int b, float inverse) {
  int q = (int)((float)a * inverse);
  q -= q * b > a;
  q += (q + 1) * b <= a;
  return q + (q * b < a);
}

// Positions that rows [row0, row1) of a sequence see: [0, sinks) and [lo, hi); the first ends where the second begins
// at the latest.
struct Seen {
  int sinks, lo, hi;
};
__device__ __forceinline__ Seen seen_by(const ChunkParams& p, const ChunkSeq& s, int row0, int row1) {
  const int first = s.len - s.tokens + (row0 >> p.group_shift), last = s.len - s.tokens + ((row1 - 1) >> p.group_shift);
  Seen x;
  x.hi = max(0, last + 1);
  x.lo = p.window ? max(0, first - p.window + 1) : 0;
  x.lo = min(x.lo, x.hi);
  x.sinks = min(p.sinks, x.lo);
  return x;
}

// Tokens per split, in tiles, of class c (0: unpacked, 1: packed): the cheapest of the longest unit's
// tiles over 1, 2, ... 160.  Time in tiles (of 2 and 1.45 us): an item is its tiles and a fixed start and end, about 6
// and 7 us; partial results cost their pass through memory.
__device__ __forceinline__ int choose_per(const ChunkParams& p, int c, const ChunkUnit* unit, int units, int longest,
                                          unsigned long long* best) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float start = c ? 5.0f : 3.0f;
  // (more row blocks than fill the GPU several times over need no search)
  const bool search = (long long)units * p.hkv <= 4LL * p.sms;
  if (threadIdx.x == 0) *best = ~0ull;
  __syncthreads();
  for (int s = warp + 1; search && s <= min(160, longest); s += kPlanWarps) {
    const int per = ceil_div(longest, s);
    if (s > 1 && ceil_div(longest, per) != s) continue;  // the same split as with fewer
    int items = 0, sum = 0;
    const float inverse = 1.0f / per;
    for (int u = lane; u < units; u += 32) {
#pragma unroll 1
      for (int k = 0; k < p.num_tiers; ++k) {
        const int n = unit[u].n[k];
        items += ceil_times(n, per, inverse);
        sum += n;
      }
    }
    items = __reduce_add_sync(0xFFFFFFFFu, items);
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    const float all = (float)items * p.hkv, load = ((float)sum * p.hkv + all * start) / p.sms, each = per + start;
    // items of one length run in waves; of different lengths, the longest first, until the last ends
    const float waves = ceilf(all / p.sms), last = (float)sum > 0.9f * items * per ? waves * each : load + 0.12f * each;
    const float cost = fmaxf(last, each) + (s > 1 ? 0.08f * all / p.sms : 0.f);
    if (lane == 0 && items <= units * (c ? p.num_tiers : 1) + p.extra_items && cost < 1e9f)
      atomicMin(best, (unsigned long long)__float_as_uint(cost) << 32 | (unsigned)s);
  }
  __syncthreads();
  const int s = *best == ~0ull ? 1 : (int)(*best & 0xFFFFFFFFu);
  __syncthreads();
  return max(1, ceil_div(longest, s));
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ ChunkParams p) {
  __shared__ Sums warps[kPlanWarps];
  __shared__ int imax[kPlanWarps];
  __shared__ TablePick picks[kPlanWarps];
  __shared__ int err, longest[2];
  __shared__ unsigned long long best;
  __shared__ ChunkSeq near_seq[kNearSeqs];
  __shared__ ChunkUnit near_unit[kNearUnits];
  ChunkSeq* const seq = p.batch <= kNearSeqs ? near_seq : p.seq;
  const bool near_units = p.max_units[0] + p.max_units[1] <= kNearUnits;
  ChunkUnit* const unit[2] = {near_units ? near_unit : p.unit[0], near_units ? near_unit + p.max_units[0] : p.unit[1]};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_release();
  if (tid == 0) {
    err = 0;
    longest[0] = longest[1] = 0;
  }
  __syncthreads();
  int bits = 0;
  const int tile = dense_tile(p.head_dim), per_unit = dense_blocks(p.head_dim);
  // ---- sequences
  Sums total = {0, 0, 0, 0};  // row blocks, unpacked units, packed units, unpacked tiles
  int most = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    ChunkSeq s;
    memset(&s, 0, sizeof(s));
    int own = 0, next = 0;
    if (p.offsets) {
      own = b < p.batch ? __ldg(p.offsets + b) : 0;
      next = b < p.batch ? __ldg(p.offsets + b + 1) : 0;
    }
    if (b < p.batch) {
#pragma unroll 1
      for (int k = 0; k < p.num_tiers; ++k) {
        s.base[k] = s.len;
        s.len += checked_len(__ldg(p.tier[k].lens + b), p.tier[k].max_pages, p.page_size, &bits);
      }
    }
    if (p.offsets) {
      // offsets that fall or leave [0, num_tokens] are brought into order and reported
      const int clipped = min(max(own, 0), p.num_tokens);
      const int start = scan_max(clipped, most, imax), end = max(start, min(max(next, 0), p.num_tokens));
      if (b < p.batch && (start != own || end != next)) bits |= KVQ_DEVERR_OFFSETS;
      s.q0 = start;
      s.tokens = end - start;
    } else {
      s.q0 = b;
      s.tokens = 1;
    }
    if (b >= p.batch) s.tokens = 0;
    const int rows = s.tokens << p.group_shift, blocks = ceil_div(rows, kChunkRows);
    s.dense = rows > p.dense_rows;
    if (s.dense && s.tokens > 0) {
      const Seen x = seen_by(p, s, 0, rows);
      s.window_tile = x.lo / tile;
      s.sink_tiles = min(ceil_div(x.sinks, tile), s.window_tile);
      s.tiles = s.sink_tiles + max(0, ceil_div(x.hi, tile) - s.window_tile);
    }
    const int units = s.dense ? ceil_div(blocks, per_unit) : blocks;
    Sums mine = {blocks, s.dense ? units : 0, s.dense ? 0 : units, s.tiles};
    Sums carry = total;
    Sums at = scan(mine, carry, warps);
    total = carry;
    s.first_block = at.a;
    s.tile0 = at.d;
    s.unit0 = s.dense ? at.b : at.c;
    if (b < p.batch) {
      seq[b] = s;
      if (seq != p.seq) p.seq[b] = s;
    }
  }
  if (bits) atomicOr(&err, bits);
  __syncthreads();
  if (p.codes)
#pragma unroll 1
    for (int k = 0; k < p.num_tiers; ++k)
      if (p.tier[k].v_fmt == KVQ_FMT_CODEBOOK) plan_tables(p, k, picks);
  // ---- units of work, a warp a sequence
  for (int b = warp; b < p.batch; b += kPlanWarps) {
    const ChunkSeq& s = seq[b];
    const int rows = s.tokens << p.group_shift, step = kChunkRows * (s.dense ? per_unit : 1);
    int n_most = 0;
    for (int r = lane * step; r < rows; r += 32 * step) {
      const Seen x = seen_by(p, s, r, min(rows, r + step));
      ChunkUnit u;
      memset(&u, 0, sizeof(u));
      u.seq = b;
      u.row0 = r;
      if (s.dense) {
        const int lo = max(s.window_tile, x.lo / tile);
        // (where the sinks reach the sequence's window, its unpacked tiles are all from 0 on)
        u.sinks[0] = min(ceil_div(x.sinks, tile), lo);
        u.begin[0] = s.sink_tiles + lo - s.window_tile;
        u.n[0] = u.sinks[0] + max(0, ceil_div(x.hi, tile) - lo);
        n_most = max(n_most, u.n[0]);
      } else {
#pragma unroll 1
        for (int k = 0; k < p.num_tiers; ++k) {
          const int end = k + 1 < p.num_tiers ? s.base[k + 1] : s.len;
          const int lo = max(0, x.lo - s.base[k]), hi = min(x.hi, end) - s.base[k];
          // (of a tier that ends before the window, the sinks alone)
          u.begin[k] = hi > lo ? lo / kMaskedTile : ceil_div(max(0, hi), kMaskedTile);
          u.sinks[k] = min(max(0, ceil_div(min(x.sinks, end) - s.base[k], kMaskedTile)), u.begin[k]);
          u.n[k] = u.sinks[k] + max(0, ceil_div(max(0, hi), kMaskedTile) - u.begin[k]);
          n_most = max(n_most, u.n[k]);
        }
      }
      unit[s.dense ? 0 : 1][s.unit0 + r / step] = u;
      if (near_units && s.dense) p.unit[0][s.unit0 + r / step] = u;  // (read again where queries are rotated)
    }
    n_most = __reduce_max_sync(0xFFFFFFFFu, n_most);
    if (lane == 0) atomicMax(&longest[s.dense ? 0 : 1], n_most);
  }
  __syncthreads();
  // ---- splits, items, and where their partial results go
  int parts = 0, items[3] = {0, 0, 0};
  for (int c = 0; c < 2; ++c) {
    const int units = c ? total.c : total.b;
    if (units == 0) continue;
    const int per = choose_per(p, c, unit[c], units, longest[c], &best);
    const int a_part = c ? 2 : per_unit;  // partials of kChunkRows rows an item leaves
    Sums all = {0, 0, 0, 0};
    for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
      const int u = u0 + tid;
      Sums mine = {0, 0, 0, 0};
      if (u < units) {
#pragma unroll 1
        for (int k = 0; k < p.num_tiers; ++k) {
          const int n = ceil_times(unit[c][u].n[k], per, 1.0f / per);
          if (c && p.tier[k].v_fmt == KVQ_FMT_CODEBOOK) mine.b += n;
          else mine.a += n;
        }
      }
      const Sums at = scan(mine, all, warps);
      if (u < units) {
        const ChunkUnit& x = unit[c][u];
        const ChunkSeq& s = seq[x.seq];
        const int rows = s.tokens << p.group_shift, n = mine.a + mine.b, part0 = parts + a_part * (at.a + at.b);
        if (c) {
          p.unit_items[1][u] = at.a;
          p.unit_items[2][u] = at.b;
        } else {
          p.unit_items[0][u] = at.a;
        }
        for (int i = 0; i < (c ? 1 : per_unit); ++i) {
          const int r = x.row0 + i * kChunkRows;
          if (r >= rows) break;
          ChunkBlock y;
          memset(&y, 0, sizeof(y));
          y.seq = x.seq;
          y.row0 = r;
          y.part0 = part0 + i;
          y.parts = c ? 2 * n : (n == 1 ? -1 : n);  // (one unpacked item writes its rows itself)
          y.step = c ? 1 : per_unit;
          p.block[s.first_block + r / kChunkRows] = y;
        }
      }
    }
    __syncthreads();
    for (int u = warp; u < units; u += kPlanWarps) {
      const ChunkUnit& x = unit[c][u];
      int before = 0;
      const int part0 = parts + a_part * (c ? p.unit_items[1][u] + p.unit_items[2][u] : p.unit_items[0][u]);
      int at[2] = {p.unit_items[c ? 1 : 0][u], c ? p.unit_items[2][u] : 0};
#pragma unroll 1
      for (int k = 0; k < p.num_tiers; ++k) {
        const int n = ceil_times(x.n[k], per, 1.0f / per), kind = c && p.tier[k].v_fmt == KVQ_FMT_CODEBOOK ? 1 : 0;
        // the tiles of a tier in equal shares
        const int share = n ? ceil_div(x.n[k], n) : 0;
        for (int i = lane; i < n; i += 32) {
          ChunkItem y;
          y.seq = x.seq;
          y.row0 = x.row0;
          y.tier = k;
          y.part = !c && n == 1 ? -1 : part0 + a_part * (before + i);
          y.first = min(x.n[k], i * share);
          y.count = min(x.n[k], (i + 1) * share) - y.first;
          y.sinks = x.sinks[k];
          y.begin = x.begin[k];
          p.item[c + kind][at[kind] + i] = y;
        }
        before += n;
        at[kind] += n;
      }
    }
    items[c] = all.a;
    if (c) items[2] = all.b;
    parts += a_part * (all.a + all.b);
  }
  __syncthreads();
  if (tid == 0) {
    ChunkHead* h = p.head;
    h->err = err;
    h->num_blocks = total.a;
    h->num_tiles = total.d;
    h->units[0] = total.b;
    h->units[1] = total.c;
    for (int i = 0; i < 3; ++i) h->items[i] = items[i];
  }
}

// ------------------------------------------------------------------------ joining
// Row r of a row block: its partial results O_i, l_i under m_i become
//   (sum 2^(m_i - m) O_i) / (sum 2^(m_i - m) l_i),  m = max m_i,
// the value rotation is undone and the result rounded to fp16.  A warp a row.
template <int E>
__device__ __forceinline__ void store_row(uint16_t* dst, int lane, const float (&y)[E]) {
  uint32_t w[E / 2];
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    const __half2 h = __floats2half2_rn(y[2 * k], y[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if constexpr (E == 2) reinterpret_cast<uint32_t*>(dst)[lane] = w[0];
  else if constexpr (E == 4) reinterpret_cast<uint2*>(dst)[lane] = make_uint2(w[0], w[1]);
  else reinterpret_cast<uint4*>(dst)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  grid_wait();
  if (p.status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = p.head->err;
  const long long rows = (long long)p.head->num_blocks * p.hkv * kChunkRows;
  for (long long x = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); x < rows; x += (long long)gridDim.x * 8) {
    // (blocks of rows of one kv head side by side)
    const int r = (int)(x % kChunkRows), hk = (int)(x / kChunkRows % p.hkv), b = (int)(x / kChunkRows / p.hkv);
    const ChunkBlock y = p.block[b];
    if (y.parts < 0) continue;
    const ChunkSeq& s = p.seq[y.seq];
    const int row = y.row0 + r;
    if (row >= s.tokens << p.group_shift) continue;
    const size_t at = (size_t)hk * kChunkRows + r, step = (size_t)p.hkv * kChunkRows;
    float m = -INFINITY;
    for (int i = lane; i < y.parts; i += 32) m = fmaxf(m, p.ml[(y.part0 + (size_t)i * y.step) * step + at].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int i = 0; i < y.parts; ++i) {
      const size_t part = (y.part0 + (size_t)i * y.step) * step + at;
      const float2 ml = p.ml[part];
      if (ml.x == -INFINITY) continue;  // no token: its accumulator was not written
      const float f = exp2f(ml.x - m);
      l = fmaf(ml.y, f, l);
      const float* a = p.acc + part * D + lane * E;
      if constexpr (E == 2) {
        const float2 v = *reinterpret_cast<const float2*>(a);
        o[0] = fmaf(v.x, f, o[0]);
        o[1] = fmaf(v.y, f, o[1]);
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 v = *reinterpret_cast<const float4*>(a + e);
          o[e] = fmaf(v.x, f, o[e]);
          o[e + 1] = fmaf(v.y, f, o[e + 1]);
          o[e + 2] = fmaf(v.z, f, o[e + 2]);
          o[e + 3] = fmaf(v.w, f, o[e + 3]);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : inv_sqrt_dim(D) / l;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= inv;
    sign_free_rotate<E>(lane, o);
    const int8_t* sg = p.v_signs + (size_t)hk * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = __ldg(sg + e) < 0 ? -o[e] : o[e];
    const int token = s.q0 + (row >> p.group_shift), h = (hk << p.group_shift) + (row & (p.group - 1));
    store_row<E>(p.out + token * p.out_token + h * p.out_head, lane, o);
  }
}

}  // namespace

cudaError_t launch_dependent(const void* kernel, unsigned grid, unsigned block, size_t smem, const ChunkParams& p,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<ChunkParams*>(&p)};
  cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t stream) {
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_chunk_join(const ChunkParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.max_blocks * p.hkv * kChunkRows;
  const unsigned grid = (unsigned)min((rows + 7) / 8, (long long)p.sms * 16);
  const void* k = p.head_dim == 64    ? reinterpret_cast<const void*>(chunk_join_kernel<64>)
                  : p.head_dim == 128 ? reinterpret_cast<const void*>(chunk_join_kernel<128>)
                                      : reinterpret_cast<const void*>(chunk_join_kernel<256>);
  return launch_dependent(k, grid ? grid : 1, 256, 0, p, stream);
}

}  // namespace kvq
