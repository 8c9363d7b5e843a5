// attn_few.cu -- attention of few rows over the paged 8-bit cache (bf16 io): one
// new token of a sequence, or a handful, times the query heads of a key head.
//
// Bound by the cache's bytes, which the rows of a key head share.  The products
// run transposed, so that the cache is the operand with 16 rows and the queries
// the one with 8 columns:  S^T = K q^T  and  O^T = V^T P^T  by
// mma.m16n8k16 in fp16, whose e4m3 operands are exact; q enters with a power of
// two per row, p with one that keeps it normal down to 2^-29 (11 bits of p
// where bf16 would keep 8).
//
// A slab is 16 tokens: its k and v are two contiguous blocks of a page, and its
// scales two numbers.  Each warp copies its own slabs ahead into its own ring
// (bulk copies; no warp waits for another) and keeps its own running maximum,
// sum and output; they meet when a piece of work ends.  Of a slab of 16 tokens
// mma row g and g + 8 are tokens  4 ((t + 2 b + half) & 3) + 2 b + half  with
// t = g / 2, b = g % 2: with 32 bytes between the slab's groups of 4 tokens
// neither the rows of k nor the columns of v that a quarter warp loads share a
// bank.
//
// Work is cut evenly: the slabs of all sequences, key heads and row tiles in a
// row, an equal range of them to each block.  A unit (sequence, key head, row
// tile) that lies in several ranges leaves partial results, which a second
// launch joins.
#include "cache_device.cuh"
#include "tma_host.h"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kSlab = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPScale = 32768.f;  // on p, in fp16: p <= 1 stays finite, p >= 2^-29 normal

template <int D>
struct Geo {
  static constexpr int kGroup = 4 * D + 32;       // bytes of 4 tokens, and the distance that spreads the banks
  static constexpr int kHalfSlab = 4 * kGroup;    // k, then v
  static constexpr int kSlabBytes = 2 * kHalfSlab;
  static constexpr int kDepth = D == 256 ? 3 : 6;
  static constexpr int kRing = kWarps * kDepth * kSlabBytes;
};
template <int D, int NT>
struct Smem {
  static constexpr int kRows = 8 * NT;
  static constexpr int kMerge = kWarps * kRows * D * 4;  // takes the ring's place when a piece ends
  static constexpr int kBig = Geo<D>::kRing > kMerge ? Geo<D>::kRing : kMerge;
  static constexpr int kQ = (D / 16) * NT * 256;
  static constexpr int kBytes = kBig + kQ;
};

// Positions of a call's work: slabs of all units in a row.
struct Place {
  Seq s;
  int hk, tile, slabs;  // of every unit of the sequence
  int slab;             // in the unit
};

struct SeqLen {
  Seq s;
  int slabs, tiles;
  long long len;  // of the sequence's units together
};
__device__ __forceinline__ SeqLen seq_len(const AttnArgs &a, int b, int rows_tile) {
  SeqLen x{};
  const int lo = a.seq.cu ? a.seq.cu[b] : b * a.seq.T, n = a.seq.cu ? a.seq.cu[b + 1] - lo : a.seq.T;
  x.s = Seq{-1, lo, n, 0};
  if (lo < 0 || n < 0 || (a.seq.cu && (long long)lo + n > a.seq.T)) return x;  // recorded by the scan
  x.s = load_seq(a.seq, b, lo, n);
  if (x.s.b < 0 || n == 0) return x;
  x.slabs = max(1, (x.s.kv + kSlab - 1) / kSlab);
  x.tiles = (n * a.r + rows_tile - 1) / rows_tile;
  x.len = (long long)x.slabs * x.tiles * a.cache.Hk;
  return x;
}

__device__ __forceinline__ long long warp_sum_incl(long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += up;
  }
  return v;
}

// The length of all the work, and where position pos = index * share lies;
// for the whole block.  share: an equal part for each of `parts`, `least` at
// least; whole != 0: a unit counts as one slab.
struct Located {
  long long total, share;
  int b;              // sequence at pos, -1: none
  long long in_seq;   // position there
};
__device__ Located locate(const AttnArgs &a, int rows_tile, int index, int parts, int least, bool whole) {
  __shared__ long long sums[kWarps], base;
  __shared__ int bad, at_b;
  __shared__ long long at_in;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    bad = 0;
    at_b = -1;
    at_in = 0;
  }
  auto len_of = [&](int b) -> long long {
    if (b >= a.seq.B) return 0;
    if (a.seq.cu) {
      const int lo = a.seq.cu[b], hi = a.seq.cu[b + 1];
      if (lo < 0 || hi < lo || hi > a.seq.T) {
        atomicOr(a.seq.err, kErrSeqlens);
        bad = 1;
        return 0;
      }
    }
    const SeqLen x = seq_len(a, b, rows_tile);
    return whole ? (long long)x.tiles * a.cache.Hk : x.len;
  };
  Located r{};
  __syncthreads();
  long long own = 0;
  for (int b = tid; b < a.seq.B; b += kThreads) own += len_of(b);
  const bool one = a.seq.B <= kThreads;
  const long long mine = own;
  const long long incl = warp_sum_incl(own, lane);
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  long long before = incl - own;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sums[w];
    r.total += sums[w];
  }
  r.b = -1;
  if (bad) {
    r.total = 0;
    return r;
  }
  r.share = max((r.total + parts - 1) / parts, (long long)least);
  const long long pos = r.share * index;
  if (pos >= r.total) return r;
  if (one) {
    if (pos >= before && pos < before + mine) {
      at_b = tid;
      at_in = pos - before;
    }
  } else {
    if (tid == 0) base = 0;
    for (int b0 = 0; b0 < a.seq.B; b0 += kThreads) {
      __syncthreads();
      const long long len = len_of(b0 + tid), in = warp_sum_incl(len, lane);
      if (lane == 31) sums[warp] = in;
      const long long start = base;
      __syncthreads();
      long long p = start + in - len, all = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) p += sums[w];
        all += sums[w];
      }
      if (pos >= p && pos < p + len) {
        at_b = b0 + tid;
        at_in = pos - p;
      }
      if (tid == 0) base = start + all;
      if (pos < start + all) break;
    }
  }
  __syncthreads();
  r.b = at_b;
  r.in_seq = at_in;
  return r;
}

// Partial results: [2 parts][rows of a tile][D] values, then [2 parts][rows] (maximum, sum).  A block's range
// may end in a unit that it starts (slot 1) and start in one that another block started (slot 0).
__device__ __forceinline__ float *part_o(void *ws, int slot, int rows, int D) {
  return static_cast<float *>(ws) + (long long)slot * rows * D;
}
__device__ __forceinline__ float2 *part_ml(void *ws, int slots, int slot, int rows, int D) {
  return reinterpret_cast<float2 *>(static_cast<float *>(ws) + (long long)slots * rows * D) + (long long)slot * rows;
}

__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w, int high) {
  uint32_t o;
  if (high)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(o) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(o) : "r"(w));
  return o;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit values over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Bytes 4w .. 4w+3 of a 16-byte word.
__device__ __forceinline__ uint32_t word(const uint4 &v, int w) { return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w; }

// q of a row tile as mma operands: element (row n, dim 64 c + 16 t + 4 s + e) is in k step 4 c + s, lane 4 (n % 8) + t,
// times a power of two that brings the row's largest into [2^14, 2^15).
template <int D, int NT>
__device__ __forceinline__ void load_q(const AttnArgs &a, const Seq &s, int hk, int first, uint8_t *sq, float *qscale) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = s.n * a.r;
  for (int n = warp; n < 8 * NT; n += kWarps) {
    const int rr = first + n;
    const bool real = rr < rows;
    const __nv_bfloat16 *const src = static_cast<const __nv_bfloat16 *>(a.q) + (long long)(s.row0 + (real ? rr / a.r : 0)) * a.ldq +
                                     (long long)(hk * a.r + (real ? rr % a.r : 0)) * D;
    constexpr int G = D / 4;  // groups of 4 elements
    float2 x[(G + 31) / 32][2];
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < (G + 31) / 32; ++i) {
      const int gr = lane + 32 * i;
      uint2 w = make_uint2(0, 0);
      if (real && gr < G) w = *reinterpret_cast<const uint2 *>(src + 4 * gr);
      x[i][0] = unpack_bf16(w.x);
      x[i][1] = unpack_bf16(w.y);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        top = fmaxf(top, fmaxf(fabsf(x[i][u].x), fabsf(x[i][u].y)));
        bad |= !(fabsf(x[i][u].x) < INFINITY) || !(fabsf(x[i][u].y) < INFINITY);
      }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    bad = __any_sync(0xffffffffu, bad);
    const int e = top > 0.f && !bad ? min(14 - ((int)(__float_as_uint(top) >> 23) - 127), 120) : 0;
    const float up = bad ? __int_as_float(0x7fc00000) : __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
    for (int i = 0; i < (G + 31) / 32; ++i) {
      const int gr = lane + 32 * i;
      if (gr >= G) break;
      const int kstep = (gr >> 4) * 4 + (gr & 3), t = (gr >> 2) & 3;
      const uint32_t at = ((kstep * NT + (n >> 3)) * 32 + (n & 7) * 4 + t) * 8;
      *reinterpret_cast<uint2 *>(sq + at) =
          make_uint2(pack2_sat(x[i][0].x * up, x[i][0].y * up), pack2_sat(x[i][1].x * up, x[i][1].y * up));
    }
    if (lane == 0) qscale[n] = __uint_as_float((uint32_t)(127 - e) << 23) * (a.scale * kLog2e);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) attn_few_kernel(const AttnArgs a, int least) {
  using G = Geo<D>;
  using S = Smem<D, NT>;
  constexpr int RT = 8 * NT, MT = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *const sq = smem + S::kBig;
  __shared__ __align__(8) uint64_t bars[kWarps][G::kDepth];
  __shared__ float qscale[RT], wm[kWarps][RT], wl[kWarps][RT], wref[kWarps], row_m[RT], row_l[RT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const CacheArgs &c = a.cache;
  if (tid < kWarps * G::kDepth) bar_init(&bars[tid / G::kDepth][tid % G::kDepth], 1);
  const bool whole = a.ws == nullptr;
  const Located loc = locate(a, RT, blockIdx.x, gridDim.x, whole ? 1 : least, whole);
  if (loc.b < 0) return;
  long long left = min(loc.share, loc.total - loc.share * blockIdx.x);
  SeqLen q = seq_len(a, loc.b, RT);
  int unit = (int)(whole ? loc.in_seq : loc.in_seq / q.slabs), slab0 = (int)(whole ? 0 : loc.in_seq % q.slabs);
  uint8_t *const ring = smem + warp * (G::kDepth * G::kSlabBytes);
  uint64_t *const bar = bars[warp];
  uint32_t uses = 0;  // of the ring so far: slot uses % depth, phase (uses / depth) & 1
  bool dead = false;
  const int page = 1 << c.page_shift;

  while (left > 0) {
    if (unit >= q.tiles * c.Hk) {  // the next sequence that has rows
      for (int nb = q.s.b + 1;; ++nb) {
        if (nb >= a.seq.B) return;
        q = seq_len(a, nb, RT);
        if (q.len > 0) break;
      }
      unit = 0;
      slab0 = 0;
    }
    const int hk = unit / q.tiles, tile = unit % q.tiles, first = tile * RT;
    const int count = min(RT, q.s.n * a.r - first);
    const int slab1 = whole ? q.slabs : (int)min((long long)q.slabs, slab0 + left);
    const bool starts = slab0 == 0, ends = slab1 == q.slabs;
    const int seen = a.causal ? min(q.s.kv, max(0, q.s.kv - q.s.n + (first + count - 1) / a.r + 1)) : q.s.kv;
    const int slab_hi = min(slab1, (seen + kSlab - 1) / kSlab);
    load_q<D, NT>(a, q.s, hk, first, sq, qscale);
    __syncthreads();  // q is in place; the merge of the piece before is done with the ring

    float acc[MT][NT][4], m[NT][2], l[NT][2], qs[NT][2];
    int last[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 8 * j + 2 * t + u;
        m[j][u] = -INFINITY;
        l[j][u] = 0.f;
        qs[j][u] = qscale[row];
        last[j][u] = row >= count ? -1 : a.causal ? q.s.kv - q.s.n + (first + row) / a.r : q.s.kv - 1;
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i][j][u] = acc[i][j][2 + u] = 0.f;
      }
    float ref = 0.f;
    // this warp's slabs: slab0 + warp + 8 i, i < mine; pages and scales of 32 of them at a time, one per lane
    const int mine = slab_hi - slab0 > warp ? (slab_hi - slab0 - warp + kWarps - 1) / kWarps : 0;
    const int *const table = c.table + (long long)q.s.b * c.table_ld;
    auto slab_of = [&](int i) { return slab0 + warp + kWarps * i; };
    auto load_page = [&](int i) -> int {
      if (i >= mine) return -1;
      const int p = table[(slab_of(i) * kSlab) >> c.page_shift];
      if (p >= 0 && p < c.n_pages) return p;
      atomicOr(a.seq.err, kErrSeqlens);
      return -1;
    };
    auto load_scales = [&](int p) -> float2 {
      if (p < 0) return make_float2(0.f, 0.f);
      const long long at = (long long)p * c.Hk + hk;
      return make_float2(c.ks[at], c.vs[at]);
    };
    int pg[2];
    float2 sc[2];
    pg[0] = load_page(lane);
    pg[1] = load_page(lane + 32);
    sc[0] = load_scales(pg[0]);
    sc[1] = load_scales(pg[1]);
    auto issue = [&](int i, int p) {  // the copies of slab i, whose page is p, into the ring
      const uint32_t use = uses + i, slot = use % G::kDepth;
      uint64_t *const b = bar + slot;
      const uint32_t dst = smem_u32(ring + slot * G::kSlabBytes);
      if (p < 0) {
        if (lane == 0) bar_arrive(b);
      } else {
        if (lane == 0) bar_expect_tx(b, 8 * 4 * D);
        __syncwarp();
        if (lane < 8) {
          const int tok = (slab_of(i) * kSlab) & (page - 1);
          const uint8_t *const src = (lane < 4 ? c.k : c.v) + (((long long)p * c.Hk + hk) * page + tok + 4 * (lane & 3)) * D;
          bulk_load(dst + lane * G::kGroup, src, 4 * D, b);
        }
      }
      __syncwarp();
    };
#pragma unroll 1
    for (int i = 0; i < min(mine, G::kDepth); ++i) issue(i, __shfl_sync(0xffffffffu, pg[0], i));

#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      const int in = i & 31;
      if (in == 0 && i > 0) {
        pg[0] = pg[1];
        sc[0] = sc[1];
        pg[1] = load_page(i + 32 + lane);
      }
      if (in == 16 && i > 16) sc[1] = load_scales(pg[1]);
      const int p = __shfl_sync(0xffffffffu, pg[0], in);
      const float ks = __shfl_sync(0xffffffffu, sc[0].x, in), vs = __shfl_sync(0xffffffffu, sc[0].y, in);
      const uint32_t use = uses + i, slot = use % G::kDepth, phase = (use / G::kDepth) & 1;
      if (!dead && !bar_wait(bar + slot, phase)) {
        dead = true;
        atomicOr(a.seq.err, kErrTimeout);
      }
      dead = __any_sync(0xffffffffu, dead);
      const uint8_t *const sk = ring + slot * G::kSlabBytes, *const sv = sk + G::kHalfSlab;
      const int tok0 = slab_of(i) * kSlab;
      if (p >= 0 && !dead) {
        // S^T: rows g and g + 8 are the tokens of half 0 and 1
        float st[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) st[j][0] = st[j][1] = st[j][2] = st[j][3] = 0.f;
        const int tg = g >> 1, bg = g & 1;
        const int m0 = 2 * bg, gr0 = (tg + 2 * bg) & 3, gr1 = (tg + 2 * bg + 1) & 3;
        const uint8_t *const k0 = sk + gr0 * G::kGroup + m0 * D + 16 * t, *const k1 = sk + gr1 * G::kGroup + (m0 + 1) * D + 16 * t;
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch) {
          const uint4 w0 = *reinterpret_cast<const uint4 *>(k0 + 64 * ch), w1 = *reinterpret_cast<const uint4 *>(k1 + 64 * ch);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t x0 = word(w0, s), x1 = word(w1, s);
            const uint32_t a0 = e4m3x2_to_h2(x0, 0), a1 = e4m3x2_to_h2(x1, 0), a2 = e4m3x2_to_h2(x0, 1), a3 = e4m3x2_to_h2(x1, 1);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const uint2 bq = *reinterpret_cast<const uint2 *>(sq + (((4 * ch + s) * NT + j) * 32 + lane) * 8);
              mma16816(st[j], a0, a1, a2, a3, bq.x, bq.y);
            }
          }
        }
        const int t0 = tok0 + 4 * gr0 + m0, t1 = tok0 + 4 * gr1 + m0 + 1;
        float x[NT][4];
        bool rescale = false;
        float mn[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float f = qs[j][u] * ks;
            x[j][u] = t0 <= last[j][u] ? st[j][u] * f : -INFINITY;
            x[j][2 + u] = t1 <= last[j][u] ? st[j][2 + u] * f : -INFINITY;
            float top = fmaxf(x[j][u], x[j][2 + u]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            mn[j][u] = fmaxf(m[j][u], top);
            rescale |= mn[j][u] != m[j][u];
          }
        float shrink = 1.f;  // on the values so far, where a larger value scale sets in
        if (vs > ref) {
          shrink = ref / vs;
          ref = vs;
          rescale = true;
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float al[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              al[u] = mn[j][u] == -INFINITY ? 1.f : exp2f(m[j][u] - mn[j][u]);
              l[j][u] *= al[u];
              m[j][u] = mn[j][u];
              al[u] *= shrink;
            }
#pragma unroll
            for (int i2 = 0; i2 < MT; ++i2) {
              acc[i2][j][0] *= al[0];
              acc[i2][j][1] *= al[1];
              acc[i2][j][2] *= al[0];
              acc[i2][j][3] *= al[1];
            }
          }
        }
        const float pv = ref > 0.f ? vs / ref * kPScale : vs * 0.f;  // 0 or NaN where no scale is above 0
        uint32_t pb[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float pp[4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float base = m[j][u] == -INFINITY ? 0.f : m[j][u];
            const float p0 = t0 <= last[j][u] ? exp2f(x[j][u] - base) : 0.f, p1 = t1 <= last[j][u] ? exp2f(x[j][2 + u] - base) : 0.f;
            l[j][u] += p0 + p1;
            pp[u] = t0 <= last[j][u] ? p0 * pv : 0.f;
            pp[2 + u] = t1 <= last[j][u] ? p1 * pv : 0.f;
          }
          pb[j][0] = transpose8(pack2_sat(pp[0], pp[1]));
          pb[j][1] = transpose8(pack2_sat(pp[2], pp[3]));
        }
        // O^T: this lane's tokens are k = 2 t, 2 t + 1 (half 0) and 2 t + 8, 2 t + 9 (half 1)
        const int ga = t, gb = (t + 2) & 3, gc = (t + 1) & 3, gd = (t + 3) & 3;
        constexpr int W = D >= 128 ? 16 : 8;  // bytes of a lane per token and load
        const bool tail = tok0 + kSlab > q.s.kv;
#pragma unroll
        for (int ch = 0; ch < (D >= 128 ? D / 128 : 1); ++ch) {
          uint32_t w[4][W / 4];
          const uint8_t *const src[4] = {sv + ga * G::kGroup, sv + gb * G::kGroup + 2 * D, sv + gc * G::kGroup + D,
                                         sv + gd * G::kGroup + 3 * D};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (W == 16) {
              const uint4 v = *reinterpret_cast<const uint4 *>(src[k] + 128 * ch + 16 * g);
              w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2 *>(src[k] + 8 * g);
              w[k][0] = v.x, w[k][1] = v.y;
            }
          }
          if (tail) {  // bytes behind the end may be anything, NaN too
            const int tk[4] = {4 * ga, 4 * gb + 2, 4 * gc + 1, 4 * gd + 3};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (tok0 + tk[k] >= q.s.kv)
#pragma unroll
                for (int e = 0; e < W / 4; ++e) w[k][e] = 0;
          }
#pragma unroll
          for (int e = 0; e < W / 4; ++e) {
            const uint32_t lo01 = __byte_perm(w[0][e], w[1][e], 0x5140), hi01 = __byte_perm(w[0][e], w[1][e], 0x7362);
            const uint32_t lo23 = __byte_perm(w[2][e], w[3][e], 0x5140), hi23 = __byte_perm(w[2][e], w[3][e], 0x7362);
            const int i2 = ch * 8 + 2 * e;
            const uint32_t a00 = e4m3x2_to_h2(lo01, 0), a01 = e4m3x2_to_h2(lo01, 1), a02 = e4m3x2_to_h2(lo23, 0), a03 = e4m3x2_to_h2(lo23, 1);
            const uint32_t a10 = e4m3x2_to_h2(hi01, 0), a11 = e4m3x2_to_h2(hi01, 1), a12 = e4m3x2_to_h2(hi23, 0), a13 = e4m3x2_to_h2(hi23, 1);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma16816(acc[i2][j], a00, a01, a02, a03, pb[j][0], pb[j][1]);
              mma16816(acc[i2 + 1][j], a10, a11, a12, a13, pb[j][0], pb[j][1]);
            }
          }
        }
      }
      __syncwarp();
      if (i + G::kDepth < mine) {
        const int nx = i + G::kDepth, pn = __shfl_sync(0xffffffffu, (nx >> 5) == (i >> 5) ? pg[0] : pg[1], nx & 31);
        issue(nx, pn);
      }
    }
    uses += mine;

    // ---- the warps' results together
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float s = l[j][u];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (g == 0) {
          wm[warp][8 * j + 2 * t + u] = m[j][u];
          wl[warp][8 * j + 2 * t + u] = s;
        }
      }
    if (lane == 0) wref[warp] = ref;
    __syncthreads();  // every warp is through with its ring
    float *const merge = reinterpret_cast<float *>(smem) + warp * RT * D;
    if (tid < RT) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, wm[w][tid]);
      float sum = 0.f;
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += exp2f(wm[w][tid] - base) * wl[w][tid];
      row_m[tid] = top;
      row_l[tid] = sum;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 8 * j + 2 * t + u;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, wm[w][row]);
        const float f = exp2f(m[j][u] - (top == -INFINITY ? 0.f : top)) * (ref * (1.f / kPScale));
#pragma unroll
        for (int i2 = 0; i2 < MT; ++i2) {
          const int dim = D >= 128 ? 128 * (i2 >> 3) + 16 * g + 2 * (i2 & 7) : 8 * g + 2 * i2;
          *reinterpret_cast<float2 *>(merge + row * D + dim) = make_float2(acc[i2][j][u] * f, acc[i2][j][2 + u] * f);
        }
      }
    __syncthreads();
    const int slot = 2 * blockIdx.x + (starts ? 1 : 0);
    for (int x = tid * 4; x < count * D; x += kThreads * 4) {
      const int row = x / D, dim = x % D, rr = first + row;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem) + w * RT * D + x);
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      }
      if (starts && ends) {
        const float ls = row_l[row], inv = ls == 0.f ? 0.f : 1.f / ls;
        __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(a.o) + (long long)(q.s.row0 + rr / a.r) * a.ldo +
                                   (long long)(hk * a.r + rr % a.r) * D + dim;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
      } else {
        *reinterpret_cast<float4 *>(part_o(a.ws, slot, RT, D) + x) = o;
        if (dim == 0) part_ml(a.ws, 2 * gridDim.x, slot, RT, D)[row] = make_float2(row_m[row], row_l[row]);
      }
    }
    fence_smem_to_async();  // before the next copies into what was written here
    __syncthreads();
    left -= whole ? 1 : slab1 - slab0;
    slab0 = 0;
    ++unit;
  }
}

// Joins the parts of the unit in which boundary blockIdx.x + 1 between the blocks' ranges is the first:
// o = sum 2^(m_p - m) o_p / sum 2^(m_p - m) l_p.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) attn_few_join(const AttnArgs a, int least, int parts) {
  constexpr int RT = 8 * NT;
  const int i = blockIdx.x + 1;
  const Located loc = locate(a, RT, i, parts, least, false);
  if (loc.b < 0) return;
  const SeqLen q = seq_len(a, loc.b, RT);
  const int unit = (int)(loc.in_seq / q.slabs), slab = (int)(loc.in_seq % q.slabs);
  if (slab == 0 || slab > loc.share) return;  // between two units, or not the first boundary inside
  const int c1 = (int)((loc.share * i - slab + q.slabs - 1) / loc.share);
  const int hk = unit / q.tiles, first = unit % q.tiles * RT, count = min(RT, q.s.n * a.r - first);
  for (int x = threadIdx.x * 4; x < count * D; x += kThreads * 4) {
    const int row = x / D, dim = x % D, rr = first + row;
    float m = -INFINITY;
    for (int c = i - 1; c <= c1; ++c) m = fmaxf(m, part_ml(a.ws, 2 * parts, 2 * c + (c == i - 1 ? 1 : 0), RT, D)[row].x);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = i - 1; c <= c1; ++c) {
      const int slot = 2 * c + (c == i - 1 ? 1 : 0);
      const float2 ml = part_ml(a.ws, 2 * parts, slot, RT, D)[row];
      const float4 v = *reinterpret_cast<const float4 *>(part_o(a.ws, slot, RT, D) + x);
      const float w = exp2f(ml.x - base);
      l += w * ml.y;
      o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(a.o) + (long long)(q.s.row0 + rr / a.r) * a.ldo +
                               (long long)(hk * a.r + rr % a.r) * D + dim;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  }
}

template <int D, int NT>
struct FewTag {};

constexpr int kLeast = 8;  // slabs of a block's range: one per warp

template <int D, int NT>
cudaError_t launch(const AttnArgs &a, int num_sms, cudaStream_t s) {
  cudaError_t e = allow_smem<FewTag<D, NT>>(attn_few_kernel<D, NT>, Smem<D, NT>::kBytes);
  if (e != cudaSuccess) return e;
  attn_few_kernel<D, NT><<<num_sms, kThreads, Smem<D, NT>::kBytes, s>>>(a, kLeast);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.ws || num_sms < 2) return e;
  attn_few_join<D, NT><<<num_sms - 1, kThreads, 0, s>>>(a, kLeast, num_sms);
  return cudaGetLastError();
}

}  // namespace

int attn_few_rows(int D, long long rows) {
  const int most = 4096 / D;
  for (int t = 8; t <= most; t *= 2)
    if (rows <= t) return t;
  return 0;
}

size_t attn_few_ws_bytes(int D, int rows_tile, int num_sms) { return (size_t)2 * num_sms * rows_tile * (D + 2) * sizeof(float); }

cudaError_t launch_attn_few(const AttnArgs &a, int rows_tile, int num_sms, cudaStream_t s) {
  const int nt = rows_tile / 8;
  switch (a.cache.D) {
    case 256: return nt == 1 ? launch<256, 1>(a, num_sms, s) : launch<256, 2>(a, num_sms, s);
    case 128: return nt == 1 ? launch<128, 1>(a, num_sms, s) : nt == 2 ? launch<128, 2>(a, num_sms, s) : launch<128, 4>(a, num_sms, s);
    default:
      return nt == 1 ? launch<64, 1>(a, num_sms, s) : nt == 2 ? launch<64, 2>(a, num_sms, s)
             : nt == 4 ? launch<64, 4>(a, num_sms, s) : launch<64, 8>(a, num_sms, s);
  }
}

}  // namespace gdn
