// Rotary positions of query and key heads (kvq_rope_apply).
//
// For each pair (a, b) of the rotated part, a' = s (a cos - b sin), b' = s (b cos + a sin);
// the rest of the head is copied.  The transpose (the gradient) turns the other way.  A
// token's cos and sin do not depend on the head, so a block takes all heads (or a share of
// them) of a few tokens, works the coefficients out once into shared memory, and turns every
// head with them.  Each thread has its first 32 bytes in flight before the coefficients are
// computed, and keeps the coefficients in registers while its next heads need the same.
// Bounded by memory: 16384 tokens x 32 heads x 256 (537 MB), 94 us, 84% of the measured copy rate;
// 64 tokens x 40 heads x 128, 4.1 us, a launch and one chain of loads.
#include <algorithm>

#include "api_checks.cuh"
#include "rope.cuh"

namespace kvq {
namespace {

struct RopeSide {
  const uint16_t* x;
  uint16_t* out;
  long long xt, xh, ot, oh;  // strides in elements: token, head
};

struct RopeApply {
  RopeParams rope;
  RopeSide side[2];
  int heads0, heads;      // heads of side 0, of both
  int tokens, per_block;  // tokens a block takes
  int head_units, rot_units;  // units of 2 V elements in a head, and in its rotated part
  int units, share;       // units of one token; units a block of the grid's y extent takes
  int in_place[2];        // the rest of the head is already where it belongs
};

// V pairs of a unit: 8 where every address and stride is a multiple of 16 bytes and the
// rotated part of 16 elements, else 1 (two-byte accesses: any even size, any stride).
template <int V>
struct Unit {
  uint16_t a[V], b[V];
};

template <int V>
__device__ __forceinline__ void load_run(const uint16_t* src, uint16_t (&v)[V]) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(src));
  else v[0] = *src;
}
template <int V>
__device__ __forceinline__ void store_run(uint16_t* dst, const uint16_t (&v)[V]) {
  if constexpr (V == 8) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(v);
  else *dst = v[0];
}

template <int V, bool HALF>
__global__ void __launch_bounds__(512) rope_kernel(const RopeApply p) {
  extern __shared__ __align__(16) float2 cs[];  // [per_block][rot / 2]
  const int t0 = blockIdx.x * p.per_block;
  const int nt = min(p.per_block, p.tokens - t0);
  const int u0 = blockIdx.y * p.share, nu = min(p.share, p.units - u0);
  const int total = nt * nu, pairs = p.rope.rot / 2;

  // unit i of the block: token, head, and the two runs of V elements it covers
  auto locate = [&](int i, const uint16_t*& src, uint16_t*& dst, int& tl, int& c, int& off_a, int& off_b) -> bool {
    tl = i / nu;
    const int u = u0 + i - tl * nu;
    const int head = u / p.head_units;
    c = u - head * p.head_units;
    const int s = head >= p.heads0;
    const RopeSide& side = p.side[s];
    const int h = s ? head - p.heads0 : head;
    src = side.x + (long long)(t0 + tl) * side.xt + h * side.xh;
    dst = side.out + (long long)(t0 + tl) * side.ot + h * side.oh;
    const bool turned = c < p.rot_units;
    off_a = HALF && turned ? c * V : 2 * V * c;
    off_b = HALF && turned ? off_a + pairs : off_a + V;
    return turned || !p.in_place[s];
  };

  const uint16_t* src;
  uint16_t* dst;
  int tl, c, oa, ob;
  Unit<V> w;
  bool live = false;
  if ((int)threadIdx.x < total) {
    live = locate(threadIdx.x, src, dst, tl, c, oa, ob);
    if (live) {
      load_run<V>(src + oa, w.a);
      load_run<V>(src + ob, w.b);
    }
  }
  for (int i = threadIdx.x; i < nt * pairs; i += blockDim.x) {
    const int t = i / pairs, j = i - t * pairs;
    cs[t * pairs + (j % V) * p.rot_units + j / V] = rope_cos_sin(p.rope, j, __ldg(p.rope.positions + t0 + t));
  }
  __syncthreads();
  float2 k[V];
  int held = -1;  // the unit (of which token) whose coefficients k holds
  for (int i = threadIdx.x; i < total;) {
    if (live) {
      if (c < p.rot_units) {
        if (const int unit = tl * pairs + c; unit != held) {
          held = unit;
#pragma unroll
          for (int e = 0; e < V; ++e) k[e] = cs[tl * pairs + e * p.rot_units + c];
        }
        if constexpr (HALF) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float a = __half2float(__ushort_as_half(w.a[e])), b = __half2float(__ushort_as_half(w.b[e]));
            const float2 f = k[e];
            w.a[e] = __half_as_ushort(__float2half_rn(fmaf(a, f.x, -(b * f.y))));
            w.b[e] = __half_as_ushort(__float2half_rn(fmaf(b, f.x, a * f.y)));
          }
        } else {
          auto turn = [&](uint16_t& lo, uint16_t& hi, const float2 f) {
            const float a = __half2float(__ushort_as_half(lo)), b = __half2float(__ushort_as_half(hi));
            lo = __half_as_ushort(__float2half_rn(fmaf(a, f.x, -(b * f.y))));
            hi = __half_as_ushort(__float2half_rn(fmaf(b, f.x, a * f.y)));
          };
          if constexpr (V == 1) {
            turn(w.a[0], w.b[0], k[0]);
          } else {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              turn(w.a[2 * e], w.a[2 * e + 1], k[e]);
              turn(w.b[2 * e], w.b[2 * e + 1], k[V / 2 + e]);
            }
          }
        }
      }
      store_run<V>(dst + oa, w.a);
      store_run<V>(dst + ob, w.b);
    }
    i += blockDim.x;
    if (i < total) {
      live = locate(i, src, dst, tl, c, oa, ob);
      if (live) {
        load_run<V>(src + oa, w.a);
        load_run<V>(src + ob, w.b);
      }
    }
  }
}

template <int V>
cudaError_t launch_rope_v(const RopeApply& p, dim3 grid, int threads, size_t smem, cudaStream_t s) {
  if (p.rope.layout == KVQ_ROPE_HALF) rope_kernel<V, true><<<grid, threads, smem, s>>>(p);
  else rope_kernel<V, false><<<grid, threads, smem, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

cudaError_t launch_rope(const RopeParams& rope, const kvq_heads* a, const kvq_heads* b, int tokens, int dim, int sms,
                        cudaStream_t stream) {
  RopeApply p;
  memset(&p, 0, sizeof(p));
  p.rope = rope;
  bool wide = rope.rot % 16 == 0 && dim % 16 == 0;
  const kvq_heads* both[2] = {a, b};
  for (int i = 0; i < 2; ++i) {
    const kvq_heads* h = both[i];
    if (!h) continue;
    p.side[i] = {h->x, h->out, h->x_token_stride, h->x_head_stride, h->out_token_stride, h->out_head_stride};
    p.in_place[i] = h->x == h->out;
    wide = wide && aligned(h->x, 16) && aligned(h->out, 16) &&
           (h->x_token_stride | h->x_head_stride | h->out_token_stride | h->out_head_stride) % 8 == 0;
  }
  p.heads0 = a->num_heads;
  p.heads = a->num_heads + (b ? b->num_heads : 0);
  p.tokens = tokens;
  const int v = wide ? 8 : 1;
  p.head_units = dim / (2 * v);
  p.rot_units = rope.rot / (2 * v);
  const long long units = (long long)p.heads * p.head_units;
  if (units > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  p.units = (int)units;
  // a block takes whole tokens while they are small, up to 256 units; where there are fewer
  // tokens than would fill the GPU, its share of one token's heads
  p.per_block = (int)std::max<long long>(1, std::min<long long>(256 / std::max<long long>(1, units), tokens));
  long long blocks = (tokens + p.per_block - 1) / p.per_block;
  long long parts = 1;
  if (p.per_block == 1 && blocks < 2LL * sms) parts = std::min((2LL * sms + blocks - 1) / blocks, (units + 63) / 64);
  parts = std::max(parts, (units + 4095) / 4096);
  if (parts > 65535) return cudaErrorInvalidValue;
  p.share = (int)((units + parts - 1) / parts);
  parts = (units + p.share - 1) / p.share;
  const long long work = (long long)p.per_block * p.share;
  // about four units a thread where there is work for all SMs, else one
  const long long each = blocks * parts >= 4LL * sms ? 4 : 1;
  long long threads = std::min<long long>(512, std::max<long long>(64, (work + each - 1) / each));
  threads = (threads + 31) / 32 * 32;
  while (threads + 32 <= 512 && threads % p.head_units != 0 && p.head_units <= 64) threads += 32;
  const size_t smem = (size_t)p.per_block * (rope.rot / 2) * sizeof(float2);
  const dim3 grid((unsigned)blocks, (unsigned)parts);
  return wide ? launch_rope_v<8>(p, grid, (int)threads, smem, stream) : launch_rope_v<1>(p, grid, (int)threads, smem, stream);
}

kvq_status check_rope(const kvq_rope* rope, int head_dim) {
  if (!rope) return KVQ_ERR_INVALID_ARGUMENT;
  if (rope->layout != KVQ_ROPE_HALF && rope->layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_INVALID_ARGUMENT;
  if (rope->rot_dim < 2 || rope->rot_dim > head_dim || rope->rot_dim % 2) return KVQ_ERR_INVALID_ARGUMENT;
  if (!rope->turns || !aligned(rope->turns, 8)) return KVQ_ERR_INVALID_ARGUMENT;
  return KVQ_OK;
}

// A set of heads: addresses, and rows of `dim` elements that neither overlap one another in
// the output nor leave 64-bit index arithmetic.
kvq_status check_heads(const kvq_heads* h, int tokens, int dim, bool need_out) {
  if (!h || h->num_heads < 1 || !h->x || !aligned(h->x, 2)) return KVQ_ERR_INVALID_ARGUMENT;
  const long long far = 1LL << 31;  // elements
  if (h->x_token_stride < 0 || h->x_head_stride < 0 || h->x_token_stride > far || h->x_head_stride > far)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (!need_out) return KVQ_OK;
  if (!h->out || !aligned(h->out, 2)) return KVQ_ERR_INVALID_ARGUMENT;
  const long long ot = h->out_token_stride, oh = h->out_head_stride, nh = h->num_heads;
  if (ot < 0 || oh < 0 || ot > far || oh > far) return KVQ_ERR_INVALID_ARGUMENT;
  // token-major or head-major, with room for every row
  const bool heads_inside = (nh == 1 || oh >= dim) && (tokens <= 1 || ot >= (nh - 1) * oh + dim);
  const bool tokens_inside = (tokens <= 1 || ot >= dim) && (nh == 1 || oh >= (tokens - 1) * ot + dim);
  if (!heads_inside && !tokens_inside) return KVQ_ERR_INVALID_ARGUMENT;
  // in place means exactly that: the same rows
  if (h->out == h->x && ((tokens > 1 && ot != h->x_token_stride) || (nh > 1 && oh != h->x_head_stride)))
    return KVQ_ERR_INVALID_ARGUMENT;
  return KVQ_OK;
}

RopeParams rope_params(const kvq_rope* rope, const int32_t* positions, int neg) {
  RopeParams r;
  r.turns = reinterpret_cast<const unsigned long long*>(rope->turns);
  r.positions = positions;
  r.scale = rope->scale;
  r.rot = rope->rot_dim;
  r.layout = rope->layout;
  r.neg = neg;
  return r;
}

}  // namespace kvq

extern "C" KVQ_API kvq_status kvq_rope_apply(const kvq_rope* rope, const int32_t* positions, const kvq_heads* a,
                                             const kvq_heads* b, int32_t num_tokens, int32_t head_dim,
                                             int32_t transpose, void* stream) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  kvq_status st = check_rope(rope, head_dim);
  if (st != KVQ_OK) return st;
  if (num_tokens < 0 || (transpose != 0 && transpose != 1)) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return KVQ_OK;
  if (!positions || !aligned(positions, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if ((st = check_heads(a, num_tokens, head_dim, true)) != KVQ_OK) return st;
  if (b && (st = check_heads(b, num_tokens, head_dim, true)) != KVQ_OK) return st;
  const cudaError_t e = launch_rope(rope_params(rope, positions, transpose), a, b, num_tokens, head_dim, device_sms(),
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
