// Attention of many queries on one cached prefix (the prefix pass of
// kvq_decode_attention_shared), on the tensor cores.
//
// All query heads of a group's sequences that read one kv head are rows of one matrix: with
// rotated queries q~ (rows) and the decoded rotated keys and values K, V of a chunk of the
// prefix,
//   S = q~ K^T,  P = 2^(S - m),  O = P V,  l = rowsum P
// with a running row maximum m.  The cache is read and decoded once for up to 256 rows,
// instead of once for every sequence.
//
// A block takes one work item: (chunk of the prefix, kv head, 256 rows).  Roles:
//   8 softmax warps (two groups of 128 threads, a thread per row): S from TMEM, P back to TMEM
//   4 + 4 decoding warps: K and V tiles of 128 tokens, read from the packed cache into
//     registers two tiles ahead, decoded to fp16 into shared memory (128-byte swizzle)
//   1 warp: issues the products and allocates TMEM.
// Both products are tcgen05.mma of 128 x 128 x 16 steps: S = q~ K^T from shared memory, O += P V
// with P read from TMEM (it overwrites S) and V as it lies (tokens x coordinates, the
// MN-major form).  The two softmax groups alternate, so that one's products run while the
// other works on its scores: with more than 128 rows each has its own rows and both use every
// tile; with up to 128 rows both have the same rows and take alternate tiles, which leaves two
// partial results.  TMEM: two S and two O of 128 columns, all 512.
//
// An accumulator is rescaled only when its row's maximum grows by more than 2^8 (weights
// then stay below 256, far inside fp16, and the sums are float32), which after the first tiles
// is rare.
//
// Rounded to fp16 on the way, each a half-ulp of 2^-11: the rotated queries, the decoded keys
// and values where their format is not exact in fp16 (fp16 and fp8 are; INT4 levels times
// their scale and centroids times their norm are not), the weights.  fp16 is what the tensor
// cores multiply at full rate; the output is fp16, and none of these errors is larger than
// its own rounding.  Scores, maxima, sums and accumulators are float32.
//
// Every wait has a limit: a block whose wait runs out sets KVQ_DEVERR_COPY_TIMEOUT and ends.
#include <atomic>

#include "shared.cuh"

namespace kvq {
namespace {

constexpr int kDim = 128;
constexpr int kThreads = 640;
// registers per thread after the split: launched with 96 x 640 = 61440 = 256 x 136 + 256 x 88 + 128 x 32
constexpr int kSoftmaxRegs = 136, kDecodeRegs = 88, kIssueRegs = 32;
constexpr int kTileBytes = kTileTokens * kDim * 2;  // 32 KB: two halves of 128 rows x 128 bytes
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kStages = 2;
constexpr int kLutBytes = 16 << 10;  // per side
constexpr int kOffQ = 0, kOffK = 2 * kTileBytes, kOffV = kOffK + kStages * kTileBytes;
constexpr int kOffLut = kOffV + kStages * kTileBytes, kOffCtl = kOffLut + 2 * kLutBytes;
constexpr int kSmem = kOffCtl + 256 + 1024;  // 1024: the base is aligned by hand

// barriers, in units of 8 bytes from kOffCtl
enum { B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_QFULL = 8, B_SFULL = 10, B_PREADY = 12, B_OFULL = 14, B_COUNT = 16 };

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

struct Ctl {
  unsigned long long bars[B_COUNT];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Ctl) <= 256, "control block");

// Waits for a phase; false once the block has given up (two seconds for any one wait).
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, int* err) {
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  for (;;) {
    if (bar_try(bar, parity)) return true;
    if (*abort) return false;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (t - t0 > 2000000000ull) {
      *abort = 1;
      atomicOr(err, KVQ_DEVERR_COPY_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort, int* err) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (bar_try(bar, parity)) return true;
  return bar_wait_slow(bar, parity, abort, err);
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// (the loaded registers pass through, so that nothing reads them before the wait)
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                 "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15])::"memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Shared-memory descriptors of the 128-byte swizzle.  A tile is two halves (64 elements of the
// 128) of 128 rows x 128 bytes, 16-byte chunk c of row r at chunk c ^ (r & 7).
//   K-major (queries, keys): rows of 8 are 1024 bytes apart (stride offset)
//   MN-major (values): 8-token groups 1024 bytes apart (stride), the halves kHalfBytes (leading)
__device__ __forceinline__ uint64_t desc_base(uint32_t leading, uint32_t stride) {
  return ((uint64_t)(leading >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t addr) { return base | ((addr >> 4) & 0x3FFFu); }

// f16 inputs, f32 accumulator, 128 x 128; bit 16: B is MN-major
constexpr uint32_t kIdescQK = (1u << 4) | ((kTileTokens >> 3) << 17) | ((kTileRows >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((kDim >> 3) << 17) | ((kTileRows >> 4) << 24);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// ------------------------------------------------------------------------ decoding a tile
// What one side (K or V) of an item reads.
struct Source {
  const uint8_t* rows;
  const __half* aux;
  const int32_t* table;  // the group's block-table row
  int row_bytes, num_pages, page_size, page_shift, hkv, hk;
  int end;               // tokens of the prefix
  uint32_t lut;          // shared address of the pair table (codebooks)
};

// Formats as the decoding warps see them.
enum { D_F16, D_F8, D_I4, D_CB4, D_CB3, D_CB2 };
__host__ __device__ constexpr int lanes_per_row(int f) { return f == D_F16 ? 16 : (f == D_F8 ? 8 : 4); }
__host__ __device__ constexpr int unit_words(int f) { return f == D_CB3 ? 3 : (f == D_CB2 ? 2 : 4); }

// A unit of one pass in a thread's registers, with its norm or group scale in both halves.
template <int F>
struct Unit {
  uint32_t w[unit_words(F)], scale;
};

// Page of the token that the thread reads in pass P of the tile at t0 (-1 past the end).
template <int F>
__device__ __forceinline__ int page_of(const Source& s, int t0, int pass, int tid) {
  const int t = t0 + pass * (128 / lanes_per_row(F)) + tid / lanes_per_row(F);
  if (t >= s.end) return -1;
  return __ldg(s.table + (s.page_shift >= 0 ? t >> s.page_shift : t / s.page_size));
}

// Where that token's unit lies, if it is there: false past the end and for a page outside the
// pool (reported in bits).
template <int F>
__device__ __forceinline__ bool find_unit(const Source& s, int t0, int pass, int tid, int page, int* bits, size_t* row) {
  const int t = t0 + pass * (128 / lanes_per_row(F)) + tid / lanes_per_row(F);
  if (t >= s.end || !page_in_pool(page, s.num_pages, bits)) return false;
  const int off = s.page_shift >= 0 ? t & (s.page_size - 1) : t % s.page_size;
  *row = ((size_t)page * s.hkv + s.hk) * s.page_size + off;
  return true;
}

template <int F>
__device__ __forceinline__ void load_unit(const Source& s, int t0, int pass, int tid, int page, Unit<F>& x, int* bits) {
  constexpr int L = lanes_per_row(F), W = unit_words(F);
  const int u = tid % L;
  size_t row;
#pragma unroll
  for (int k = 0; k < W; ++k) x.w[k] = 0u;  // a token that is not there reads as zero
  x.scale = 0u;
  if (!find_unit<F>(s, t0, pass, tid, page, bits, &row)) return;
  const uint8_t* src = s.rows + row * s.row_bytes + u * (4 * W);
  if constexpr (W == 4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
    x.w[0] = v.x;
    x.w[1] = v.y;
    x.w[2] = v.z;
    x.w[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
    x.w[0] = v.x;
    x.w[1] = v.y;
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k) x.w[k] = __ldg(reinterpret_cast<const uint32_t*>(src) + k);
  }
  if constexpr (F == D_I4) x.scale = __half_as_ushort(__ldg(s.aux + row * 4 + u));
  else if constexpr (F >= D_CB4) x.scale = __half_as_ushort(__ldg(s.aux + row));
}

// The unit decoded to fp16, into its row of the tile.
template <int F>
__device__ __forceinline__ void store_unit(const Source& s, uint32_t tile, int pass, int tid, const Unit<F>& z) {
  constexpr int L = lanes_per_row(F);
  const int u = tid % L, t = pass * (128 / L) + tid / L;  // t: row of the tile
  const uint32_t row = tile + t * 128;
  const int x = t & 7;
  if constexpr (F == D_F8) {
    // 16 values, two chunks; the upper half's lanes store theirs in the other order, so that
    // the eight lanes of a row meet eight different 16-byte banks
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[k]) : "h"((uint16_t)(z.w[k / 2] >> (16 * (k & 1)))));
    const uint32_t at = row + (u >> 2) * kHalfBytes;
    const int c = (2 * u) & 7, odd = u >> 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool second = (i ^ odd) != 0;
      sts16(at + (((c + second) ^ x) << 4), second ? h[4] : h[0], second ? h[5] : h[1], second ? h[6] : h[2],
            second ? h[7] : h[3]);
    }
  } else {
    // 32 values, four chunks of 8 (b bytes each); lanes of a row pair store them in four
    // different orders, so that eight lanes meet eight different 16-byte banks
    constexpr int B = F == D_I4 || F == D_CB4 ? 4 : (F == D_CB3 ? 3 : 2);
    const uint32_t scale = z.scale * 0x10001u;
    uint32_t c[4];
    if constexpr (B == 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = z.w[k];
    } else if constexpr (B == 3) {
      c[0] = z.w[0];
      c[1] = __funnelshift_r(z.w[0], z.w[1], 24);
      c[2] = __funnelshift_r(z.w[1], z.w[2], 16);
      c[3] = z.w[2] >> 8;
    } else {
      c[0] = z.w[0];
      c[1] = z.w[0] >> 16;
      c[2] = z.w[1];
      c[3] = z.w[1] >> 16;
    }
    const int flip = (u >> 1) ^ ((t & 1) << 1);
    if (flip & 1) {
      uint32_t y = c[0];
      c[0] = c[1];
      c[1] = y;
      y = c[2];
      c[2] = c[3];
      c[3] = y;
    }
    if (flip & 2) {
      uint32_t y = c[0];
      c[0] = c[2];
      c[2] = y;
      y = c[1];
      c[1] = c[3];
      c[3] = y;
    }
    const uint32_t at = row + (u >> 1) * kHalfBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[4];
      if constexpr (F == D_I4) {
        // nibbles as 1024 + n in fp16, minus 1032: exact; times the scale, rounded once
        const uint32_t even = c[i] & 0x0F0F0F0Fu, odd = (c[i] >> 4) & 0x0F0F0F0Fu;
        const __half2 off = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t v = (__byte_perm(even, odd, k | (k << 4) | ((4 + k) << 8) | (k << 12)) & 0x00FF00FFu) | 0x64006400u;
          const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&v), off);
          h[k] = hmul2(*reinterpret_cast<const uint32_t*>(&n), scale);
        }
      } else {
        // pairs of codes through the block's table of centroid pairs / sqrt(D)
        constexpr int C = F == D_CB4 ? 16 : 32;  // copies: one per lane (4 bits: per half-warp lane)
        const uint32_t base = s.lut + 4u * (tid & (C - 1));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t e = (c[i] >> (2 * B * k)) & ((1u << (2 * B)) - 1u);
          h[k] = hmul2(lds32(base + e * (4u * C)), scale);
        }
      }
      sts16(at + (((4 * (u & 1) + (i ^ flip)) ^ x) << 4), h[0], h[1], h[2], h[3]);
    }
  }
}

// Tiles [tile0, tile1) of one side, into the ring.
struct Ring {
  uint32_t tiles, full, empty;  // shared addresses
};

// A pass's registers are loaded with the next tile's unit as soon as its unit of this tile is
// decoded, and its page number a tile before that: every load has a tile's time to arrive.
template <int F>
__device__ __forceinline__ void produce(const Source& s, const Ring& ring, int tile0, int tile1, int tid,
                                        volatile int* abort, int* err) {
  constexpr int kPasses = lanes_per_row(F);  // 128 threads, 128 rows
  int bits = 0;
  Unit<F> x[kPasses];
  int page[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) page[p] = page_of<F>(s, tile0 * kTileTokens, p, tid);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) load_unit<F>(s, tile0 * kTileTokens, p, tid, page[p], x[p], &bits);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) page[p] = page_of<F>(s, (tile0 + 1) * kTileTokens, p, tid);
  for (int t = tile0, i = 0; t < tile1; ++t, ++i) {
    const int st = i & 1;
    if (i >= kStages && !bar_wait(ring.empty + 8 * st, ((i >> 1) & 1) ^ 1, abort, err)) break;
    const bool more = t + 1 < tile1;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      store_unit<F>(s, ring.tiles + st * kTileBytes, p, tid, x[p]);
      if (more) {
        load_unit<F>(s, (t + 1) * kTileTokens, p, tid, page[p], x[p], &bits);
        page[p] = page_of<F>(s, (t + 2) * kTileTokens, p, tid);
      }
    }
    fence_async_smem();
    bar_arrive(ring.full + 8 * st);
  }
  if (bits) atomicOr(err, bits);
}

// fp16 rows need no decoding: asynchronous copies, a tile signalled once the next one's copies
// are under way.
template <>
__device__ __forceinline__ void produce<D_F16>(const Source& s, const Ring& ring, int tile0, int tile1, int tid,
                                               volatile int* abort, int* err) {
  constexpr int kPasses = lanes_per_row(D_F16);
  int bits = 0;
  int page[kPasses];
  const int u = tid % 16;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) page[p] = page_of<D_F16>(s, tile0 * kTileTokens, p, tid);
  bool ok = true;
  for (int t = tile0, i = 0; t < tile1; ++t, ++i) {
    const int st = i & 1;
    if (i >= kStages && !(ok = bar_wait(ring.empty + 8 * st, ((i >> 1) & 1) ^ 1, abort, err))) break;
    const uint32_t tile = ring.tiles + st * kTileBytes + (u >> 3) * kHalfBytes;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      size_t row = 0;
      const bool there = find_unit<D_F16>(s, t * kTileTokens, p, tid, page[p], &bits, &row);
      const int r = p * 8 + tid / 16;
      // (a row that is not there: no bytes read, 16 zeros written)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile + r * 128 + (((u & 7) ^ (r & 7)) << 4)),
                   "l"(s.rows + row * s.row_bytes + u * 16), "r"(there ? 16 : 0)
                   : "memory");
      page[p] = page_of<D_F16>(s, (t + 1) * kTileTokens, p, tid);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (i > 0) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      fence_async_smem();
      bar_arrive(ring.full + 8 * (st ^ 1));
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (ok) {
    fence_async_smem();
    bar_arrive(ring.full + 8 * ((tile1 - tile0 - 1) & 1));
  }
  if (bits) atomicOr(err, bits);
}

__device__ __forceinline__ void produce_any(int f, const Source& s, const Ring& ring, int tile0, int tile1, int tid,
                                            volatile int* abort, int* err) {
  switch (f) {
    case D_F16: produce<D_F16>(s, ring, tile0, tile1, tid, abort, err); break;
    case D_F8: produce<D_F8>(s, ring, tile0, tile1, tid, abort, err); break;
    case D_I4: produce<D_I4>(s, ring, tile0, tile1, tid, abort, err); break;
    case D_CB4: produce<D_CB4>(s, ring, tile0, tile1, tid, abort, err); break;
    case D_CB3: produce<D_CB3>(s, ring, tile0, tile1, tid, abort, err); break;
    default: produce<D_CB2>(s, ring, tile0, tile1, tid, abort, err); break;
  }
}

__device__ __forceinline__ int decode_kind(int fmt, int bits) {
  switch (fmt) {
    case KVQ_FMT_FP16: return D_F16;
    case KVQ_FMT_FP8_E4M3: return D_F8;
    case KVQ_FMT_INT4_G32: return D_I4;
    default: return bits == 4 ? D_CB4 : (bits == 3 ? D_CB3 : D_CB2);
  }
}

// Pairs of centroids / sqrt(D) in fp16: entry e = codes (e mod 2^b, e / 2^b), a copy per lane of
// a warp (16 copies of 4-bit pairs).  tid: 256 threads.
__device__ __forceinline__ void build_lut(uint32_t lut, const float* cent, int bits, int tid) {
  const int copies = bits == 4 ? 16 : 32;
  if (tid >= (1 << (2 * bits))) return;
  const float inv = inv_sqrt_dim(kDim);
  const uint32_t v = half2_bits(__ldg(cent + (tid & ((1 << bits) - 1))) * inv, __ldg(cent + (tid >> bits)) * inv);
  for (int i = 0; i < copies; i += 4) sts16(lut + 4u * (tid * copies + i), v, v, v, v);
}

// ------------------------------------------------------------------------ softmax
// A row's maximum has grown: from f on (2^(old - new)), scale what the old one is in: the
// accumulator (if any product has gone into it) and the tile's first `done` weight columns.
__device__ __forceinline__ void rescale(uint32_t o_at, bool acc, uint32_t p_at, int done, float f) {
  uint32_t v[16];
  if (acc) {
#pragma unroll 1
    for (int c = 0; c < kDim; c += 16) {
      tc_ld16(o_at + c, v);
      tc_wait_ld(v);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
      tc_st16(o_at + c, v);
    }
  }
  for (int c = 0; c < done; c += 16) {
    tc_ld16(p_at + c, v);
    tc_wait_ld(v);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
      v[e] = half2_bits(x.x * f, x.y * f);
    }
    tc_st16(p_at + c, v);
  }
  tc_wait_st();
}

__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long r) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
  return f;
}

// ------------------------------------------------------------------------ the kernel
__global__ void __launch_bounds__(kThreads, 1) shared_prefix_kernel(const __grid_constant__ SharedParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw + (smem - smem_u32(smem_raw)) + kOffCtl);
  volatile int* abort = &ctl->abort;
  const uint32_t bars = smem + kOffCtl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- the item: split, kv head, row block (blocks of one split and head side by side, so
  // that they meet the same cache bytes in L2)
  int item = blockIdx.x;
  const int blk = item % p.num_blocks;
  item /= p.num_blocks;
  const int hk = item % p.hkv, split = item / p.hkv;
  int lo = 0, hi = p.num_groups;  // the group whose row blocks hold blk
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.block[mid] <= blk) lo = mid;
    else hi = mid;
  }
  const int g = lo, lb = blk - p.block[g];
  const int rows = (p.offset[g + 1] - p.offset[g]) * p.group - lb * kItemRows;  // > 0
  const bool both = rows <= kTileRows;  // both softmax groups on the same rows
  int ti = 0;
  while (ti + 1 < p.num_tiers && split >= p.tier[ti + 1].split_begin) ++ti;
  const SharedTier& T = p.tier[ti];
  int bits = 0;
  const int len = checked_len(__ldg(T.lens + g), T.max_pages, p.page_size, &bits);
  if (bits && threadIdx.x == 0) atomicOr(p.err, bits);
  const int all = (len + kTileTokens - 1) / kTileTokens;
  const int per = (all + T.num_splits - 1) / T.num_splits;
  const int tile0 = min((split - T.split_begin) * per, all), tile1 = min(tile0 + per, all);
  const int n = tile1 - tile0;
  const int jobs = both ? n : 2 * n;  // job i: softmax group i & 1, tile both ? i : i / 2

  // row of this softmax thread, as an output row (sequence, query head), or -1
  const int w = warp >> 2;  // softmax group of the first eight warps
  const int r = (both ? 0 : w * kTileRows) + (threadIdx.x & 127);
  long long out_row = -1;
  if (warp < 8 && r < rows) {
    const int gr = lb * kItemRows + r, i = gr / p.group;
    out_row = (long long)(p.offset[g] + i) * p.hq + hk * p.group + (gr - i * p.group);
  }
  const size_t out_rows = (size_t)p.batch * p.hq;
  const size_t part = (2 * (size_t)split + (both ? w : 0)) * out_rows;

  if (n == 0) {  // no tokens: partials of weight zero
    if (out_row >= 0) *reinterpret_cast<float2*>(p.ml + 2 * (part + out_row)) = make_float2(-INFINITY, 0.f);
    return;
  }

  const int rows_of_group = both ? min(rows, kTileRows) : min(rows - w * kTileRows, kTileRows);  // w of a softmax warp
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(bars + 8 * (B_KFULL + i), 128);
      bar_init(bars + 8 * (B_KEMPTY + i), 1);
      bar_init(bars + 8 * (B_VFULL + i), 128);
      bar_init(bars + 8 * (B_VEMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      const int live = both ? rows : min(max(rows - i * kTileRows, 0), kTileRows);
      bar_init(bars + 8 * (B_QFULL + i), 128);
      bar_init(bars + 8 * (B_SFULL + i), 1);
      bar_init(bars + 8 * (B_PREADY + i), max(1, (live + 31) / 32 * 32));  // the warps that hold rows
      bar_init(bars + 8 * (B_OFULL + i), 1);
    }
    ctl->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctl->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (T.k_fmt == KVQ_FMT_CODEBOOK && warp < 8) build_lut(smem + kOffLut, T.k_cent, T.k_bits, threadIdx.x);
  if (T.v_fmt == KVQ_FMT_CODEBOOK && warp >= 8 && warp < 16)
    build_lut(smem + kOffLut + kLutBytes, T.v_cent, T.v_bits, threadIdx.x - 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  // chunks of the sequences' own tiers may start on SMs that this grid leaves idle
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp < 8) {
    // ---- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const uint32_t q_tile = smem + kOffQ + w * kTileBytes;
    {
      // the group's queries into shared memory, 16 lanes a row
      const int tid = threadIdx.x & 127;
      for (int i = tid; i < kTileRows * 16; i += 128) {
        const int row = i >> 4, c = i & 15;
        uint4 x = make_uint4(0, 0, 0, 0);
        const int rr = (both ? 0 : w * kTileRows) + row;
        if (rr < rows) {
          const int gr = lb * kItemRows + rr, sq = gr / p.group;
          const size_t orow = (size_t)(p.offset[g] + sq) * p.hq + hk * p.group + (gr - sq * p.group);
          x = __ldg(reinterpret_cast<const uint4*>(p.q + orow * kDim) + c);
        }
        sts16(q_tile + (c >> 3) * kHalfBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4), x.x, x.y, x.z, x.w);
      }
      fence_async_smem();
      bar_arrive(bars + 8 * (B_QFULL + w));
    }
    const int my_jobs = jobs > w ? (jobs - w + 1) / 2 : 0;
    const bool live = (warp & 3) * 32 < rows_of_group;  // the warp holds rows
    if (live && my_jobs > 0) {
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_at = lane_base + w * 128, o_at = lane_base + 256 + w * 128;
      float m = -INFINITY;
      unsigned long long l2 = 0;  // the row's sum, even and odd columns
      bool ok = true;
      for (int k = 0; k < my_jobs; ++k) {
        const int i = 2 * k + w, tile = tile0 + (both ? i : i >> 1);
        const int valid = min(kTileTokens, len - tile * kTileTokens);
        if (!(ok = __all_sync(0xFFFFFFFFu, bar_wait(bars + 8 * (B_SFULL + w), k & 1, abort, p.err)))) break;
        tc_fence_after();
        uint32_t va[32], vb[32];
        tc_ld32(s_at, va);
        // 32 scores: the row's maximum (a rise of more than 2^8 rescales), weights, their sum
        auto weigh = [&](int c, uint32_t (&v)[32], uint32_t (&next)[32]) {
          if (valid < kTileTokens) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= valid) v[e] = 0xFF800000u;  // -inf: weight 0
          }
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            m0 = fmaxf(fmaxf(m0, __uint_as_float(v[e])), __uint_as_float(v[e + 1]));
            m1 = fmaxf(fmaxf(m1, __uint_as_float(v[e + 2])), __uint_as_float(v[e + 3]));
          }
          const float mx = fmaxf(m0, m1);
          if (__any_sync(0xFFFFFFFFu, mx > m + 8.0f)) {
            const float mn = fmaxf(m, mx), f = ex2(m - mn);
            m = mn;
            const float2 ll = unpack2(l2);
            l2 = pack2(ll.x * f, ll.y * f);
            // (the products of earlier tiles are complete: they precede these scores)
            tc_wait_ld(next);  // nothing in flight across the call
            if (k > 0 || c > 0) rescale(o_at, k > 0, s_at, 16 * c, f);
          }
          const unsigned long long neg = pack2(-m, -m);
          uint32_t h[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = unpack2(add2(pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), neg));
            const float a = ex2(x.x), b = ex2(x.y);
            l2 = add2(l2, pack2(a, b));
            h[e] = half2_bits(a, b);
          }
          tc_st16(s_at + 16 * c, h);  // over scores that this warp has read
        };
        tc_wait_ld(va);
        tc_ld32(s_at + 32, vb);
        weigh(0, va, vb);
        tc_wait_ld(vb);
        tc_ld32(s_at + 64, va);
        weigh(1, vb, va);
        tc_wait_ld(va);
        tc_ld32(s_at + 96, vb);
        weigh(2, va, vb);
        tc_wait_ld(vb);
        weigh(3, vb, va);
        tc_wait_st();
        tc_fence_before();
        bar_arrive(bars + 8 * (B_PREADY + w));
      }
      if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait(bars + 8 * (B_OFULL + w), (my_jobs - 1) & 1, abort, p.err));
      tc_fence_after();
      if (ok) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tc_ld32(o_at + 32 * c, v);
          tc_wait_ld(v);
          if (out_row >= 0) {
            float* dst = p.acc + (part + out_row) * kDim + 32 * c;
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + e), "r"(v[e]),
                           "r"(v[e + 1]), "r"(v[e + 2]), "r"(v[e + 3]), "r"(v[e + 4]), "r"(v[e + 5]), "r"(v[e + 6]),
                           "r"(v[e + 7])
                           : "memory");
          }
        }
      }
      if (out_row >= 0) *reinterpret_cast<float2*>(p.ml + 2 * (part + out_row)) =
            ok ? make_float2(m, unpack2(l2).x + unpack2(l2).y) : make_float2(-INFINITY, 0.f);
    } else if (out_row >= 0) {  // a second group without a tile of its own
      *reinterpret_cast<float2*>(p.ml + 2 * (part + out_row)) = make_float2(-INFINITY, 0.f);
    }
  } else if (warp < 16) {
    // ---- decoding
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDecodeRegs));
    const bool keys = warp < 12;
    Source s;
    s.rows = keys ? T.k_rows : T.v_rows;
    s.aux = keys ? T.k_aux : T.v_aux;
    s.table = T.block_table + (size_t)g * T.max_pages;
    s.row_bytes = keys ? T.k_row_bytes : T.v_row_bytes;
    s.num_pages = T.num_pages;
    s.page_size = p.page_size;
    s.page_shift = p.page_shift;
    s.hkv = p.hkv;
    s.hk = hk;
    s.end = len;
    s.lut = smem + kOffLut + (keys ? 0 : kLutBytes);
    Ring ring;
    ring.tiles = smem + (keys ? kOffK : kOffV);
    ring.full = bars + 8 * (keys ? B_KFULL : B_VFULL);
    ring.empty = bars + 8 * (keys ? B_KEMPTY : B_VEMPTY);
    produce_any(keys ? decode_kind(T.k_fmt, T.k_bits) : decode_kind(T.v_fmt, T.v_bits), s, ring, tile0, tile1,
                threadIdx.x & 127, abort, p.err);
  } else {
    // ---- products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 16 && lane == 0) {
    const uint64_t kmajor = desc_base(16, 1024), mnmajor = desc_base(kHalfBytes, 1024);
    auto scores = [&](int i) -> bool {  // S of job i
      const int tile = both ? i : i >> 1, st = tile & 1, ws = i & 1;
      if (!bar_wait(bars + 8 * (B_KFULL + st), (tile >> 1) & 1, abort, p.err)) return false;
      tc_fence_after();
      const uint32_t a = smem + kOffQ + ws * kTileBytes, b = smem + kOffK + st * kTileBytes;
#pragma unroll
      for (int kk = 0; kk < kDim / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
        mma_ss(tmem + ws * 128, desc_at(kmajor, a + off), desc_at(kmajor, b + off), kIdescQK, kk > 0);
      }
      tc_commit(bars + 8 * (B_SFULL + ws));
      if (both || ws) tc_commit(bars + 8 * (B_KEMPTY + st));
      return true;
    };
    bool ok = true;
    for (int i = 0; i < 2 && i < jobs && ok; ++i)
      ok = bar_wait(bars + 8 * (B_QFULL + i), 0, abort, p.err) && scores(i);
    for (int i = 0; i < jobs && ok; ++i) {
      const int tile = both ? i : i >> 1, st = tile & 1, ws = i & 1;
      ok = bar_wait(bars + 8 * (B_VFULL + st), (tile >> 1) & 1, abort, p.err) &&
           bar_wait(bars + 8 * (B_PREADY + ws), (i >> 1) & 1, abort, p.err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t b = smem + kOffV + st * kTileBytes;
#pragma unroll
      for (int kk = 0; kk < kTileTokens / 16; ++kk)
        mma_ts(tmem + 256 + ws * 128, tmem + ws * 128 + kk * 8, desc_at(mnmajor, b + kk * 2048), kIdescPV,
               i > 1 || kk > 0);
      tc_commit(bars + 8 * (B_OFULL + ws));
      if (both || ws) tc_commit(bars + 8 * (B_VEMPTY + st));
      if (i + 2 < jobs) ok = scores(i + 2);
    }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace

bool shared_tier_supported(int head_dim, int k_fmt, int v_fmt) {
  if (head_dim != kDim) return false;
  if (k_fmt == KVQ_FMT_FP16) return v_fmt == KVQ_FMT_FP16;
  if (k_fmt == KVQ_FMT_FP8_E4M3) return v_fmt == KVQ_FMT_INT4_G32 || v_fmt == KVQ_FMT_FP16;
  return k_fmt == KVQ_FMT_CODEBOOK && v_fmt == KVQ_FMT_CODEBOOK;
}

cudaError_t launch_shared_prefix(const SharedParams& p, cudaStream_t stream) {
  if (p.num_items == 0) return cudaSuccess;
  static std::atomic<bool> configured[64];  // shared-memory limit raised on this device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(shared_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  shared_prefix_kernel<<<p.num_items, kThreads, kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace kvq
