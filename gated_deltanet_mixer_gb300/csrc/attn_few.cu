// attn_few.cu -- attention of few rows over the paged 8-bit cache (bf16 io): one
// new token of a sequence, or a handful, times the query heads of a key head.
//
// Bound by the cache's bytes, which the rows of a key head share (64 x 1 token over
// 8192, 24/4 heads of 256: 170 us, 6.3 TB/s; 16 x 4 tokens, ragged, 32/8 heads of 128,
// 87 MB: 33 us, of which some 10 are a block's start, end and the join).  The products
// run transposed, so that the cache is the operand with 16 rows and the queries
// the one with 8 columns:  S^T = K q^T  and  O^T = V^T P^T  by
// mma.m16n8k16 in fp16, whose e4m3 operands are exact; q enters with a power of
// two per row, p with its page's value scale and one that keeps the product normal
// down to 2^-25 of the row's largest (11 bits of p where bf16 would keep 8).  What O
// is relative to is the running maximum of these products, apart from that of p
// alone, which the sum of the weights is relative to: a page of large values and
// hardly any weight costs the others no bits.
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
// row, an equal range of them to each block (a unit - sequence, key head, row
// tile - counts as some slabs more than it has).  A unit that lies in several
// ranges leaves partial results, which a second launch joins.
#include <algorithm>

#include "cache_device.cuh"
#include "tma_host.h"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kBlocksSM = 2;
constexpr float kNone = -1.7e38f;  // the running maximum of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f;
// The references of a row's exponents are its running maxima, less kLift and moved only
// when a score passes them by kSlack (in powers of 2).  Weights stay below 2^(kSlack + kLift),
// and what is far below the largest, but has larger values, does not vanish before it
// gets its scale (2^-120 to 2^7; the exponential ends at 2^-126); their products with the
// scales stay below 2^(kSlack + kPExp) in fp16, finite, and normal from 2^-25 on.
constexpr float kSlack = 4.f;
constexpr float kLift = 30.f;
constexpr float kPExp = 11.f;

// A slab's copies: kSub times 16 tokens, of a page each, in a ring of kDepth slabs per warp.  More tokens at a
// time spread what a slab costs whatever its width (waits, votes, copies; some 250 instructions of a warp with
// 16 tokens); wide heads have no room for them.
template <int D, int NT>
struct Geo {
  static constexpr int kRows = 8 * NT;
  static constexpr int kSub = D == 256 ? 1 : D == 128 ? 2 : NT == 1 ? 4 : 2;
  static constexpr int kSlab = 16 * kSub;
  static constexpr int kGroup = 4 * D + 32;         // bytes of 4 tokens, and the distance that spreads the banks
  static constexpr int kK = 4 * kGroup;             // of 16 tokens' keys; their values follow
  static constexpr int kSlabBytes = 2 * kK * kSub;
  static constexpr int kDepth = D == 64 && kSub == 2 ? 5 : 3;
  static constexpr int kRing = kWarps * kDepth * kSlabBytes;
  static constexpr int kPitch = D + 4;  // of a row of the merge, in floats
  // A warp's results at the end of a piece take the first slots of its ring.
  static constexpr int kMergeSlots = (kRows * kPitch * 4 + kSlabBytes - 1) / kSlabBytes;
  static_assert(kMergeSlots < kDepth, "no slot is left for the next piece");
  static constexpr int kQ = (D / 16) * NT * 256;
  static constexpr int kBytes = kRing + kQ;
  // What going on to another unit costs a block, in slabs (some 7 us): counted with the unit's own where the work is
  // cut.  32 x 1 token over 200 to 15,000, 4 heads of 256: 47 us, with half of it 51, without 67; heads of 64 25, with
  // twice as much 26.3, without 37; 300 x 1 over 500 the same but for heads of 128, which lose: 49.5, without 47.
  static constexpr int kStart = D == 64 ? 32 / kSub : 16;
};

struct SeqLen {
  Seq s;
  int slabs, tiles;
  int each;       // of a unit: what its start costs, and its slabs
  long long len;  // of the sequence's units together
};
// What the kernels of a tile have in common: its rows, a slab's tokens, a unit's start in slabs.
struct Cut {
  int rows_tile, slab, start;
};
__device__ __forceinline__ SeqLen seq_len(const AttnArgs &a, int b, const Cut &cut) {
  SeqLen x{};
  const int lo = a.seq.cu ? a.seq.cu[b] : b * a.seq.T, n = a.seq.cu ? a.seq.cu[b + 1] - lo : a.seq.T;
  x.s = Seq{-1, lo, n, 0};
  if (lo < 0 || n < 0 || (a.seq.cu && (long long)lo + n > a.seq.T)) return x;  // recorded by the scan
  x.s = load_seq(a.seq, b, lo, n);
  if (x.s.b < 0 || n == 0) return x;
  x.slabs = max(1, (x.s.kv + cut.slab - 1) / cut.slab);
  x.each = x.slabs + cut.start;
  x.tiles = (n * a.r + cut.rows_tile - 1) / cut.rows_tile;
  x.len = (long long)x.each * x.tiles * a.cache.Hk;
  return x;
}

// a / b rounded up; a 64-bit division takes some hundred instructions
__device__ __forceinline__ long long div_up(long long a, int b) {
  return a < 0x40000000 ? ((int)a + b - 1) / b : (a + b - 1) / b;
}
__device__ __forceinline__ int quotient(long long a, int b) { return a < 0x7fffffff ? (int)a / b : (int)(a / b); }
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
// least; whole != 0: a unit counts as one slab.  of >= 0: in_seq is where sequence `of` starts instead.
struct Located {
  long long total, share;
  int b;              // sequence at pos, -1: none
  long long in_seq;   // position there
};
template <int kThreads>
__device__ Located locate(const AttnArgs &a, const Cut &cut, int index, int parts, int least, bool whole, int of = -1) {
  constexpr int kWarps = kThreads / 32;
  __shared__ long long sums[kWarps], base;
  __shared__ int bad, at_b;
  __shared__ long long at_in;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (a.seq.B <= 32) {  // each warp for itself, without a barrier (1 token over 4096: 13.2 us, with them 13.7)
    bool wrong = false;
    long long len = 0;
    if (lane < a.seq.B) {
      if (a.seq.cu) {
        const int lo = a.seq.cu[lane], hi = a.seq.cu[lane + 1];
        wrong = lo < 0 || hi < lo || hi > a.seq.T;
      }
      const SeqLen x = seq_len(a, lane, cut);
      len = whole ? (long long)x.tiles * a.cache.Hk : x.len;
    }
    Located r{};
    r.b = -1;
    if (__any_sync(0xffffffffu, wrong)) {
      if (tid == 0) atomicOr(a.seq.err, kErrSeqlens);
      return r;
    }
    const long long incl = warp_sum_incl(len, lane);
    r.total = __shfl_sync(0xffffffffu, incl, 31);
    r.share = max(div_up(r.total, parts), (long long)least);
    const long long pos = r.share * index;
    const uint32_t at = __ballot_sync(0xffffffffu, pos >= incl - len && pos < incl);
    const int from = of >= 0 ? of : at ? __ffs(at) - 1 : 0;
    const long long before = __shfl_sync(0xffffffffu, incl - len, from);
    if (of >= 0 || at) {
      r.b = from;
      r.in_seq = of >= 0 ? before : pos - before;
    }
    return r;
  }
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
    const SeqLen x = seq_len(a, b, cut);
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
  r.share = max(div_up(r.total, parts), (long long)least);
  const long long pos = r.share * index;
  if (of >= 0) {
    long long lower = 0;  // before sequence `of`
    if (one && tid == of) at_in = before;
    if (!one) {
      for (int b = tid; b < of; b += kThreads) lower += len_of(b);
      lower = warp_sum_incl(lower, lane);
      __syncthreads();
      if (lane == 31) sums[warp] = lower;
    }
    __syncthreads();
    r.b = of;
    if (one) {
      r.in_seq = at_in;
    } else {
      for (int w = 0; w < kWarps; ++w) r.in_seq += sums[w];
    }
    return r;
  }
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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit values over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// Bytes 4w .. 4w+3 of a 16-byte word.
__device__ __forceinline__ uint32_t word(const uint4 &v, int w) { return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w; }

// Where a row of the merge has the two dimensions of product row i of lane group g: dimension 16 g + 2 i (and 128 on
// from i = 8; D = 64: 8 g + 2 i), the pairs of 16 in an order that spreads the groups over the banks.
template <int D>
__device__ __forceinline__ int merge_at(int g, int i) {
  return D >= 128 ? 128 * (i >> 3) + 16 * g + 2 * ((i & 7) ^ (g >> 1)) : 8 * g + 2 * i;
}
// Token row and query head of a row of the tile.
struct RowAt {
  long long token;
  int head;
};

// A warp's rows of q, n = warp + kWarps i: 4 elements to a lane, 128 apart.
template <int D, int NT>
struct QRows {
  static constexpr int kOf = 8 * NT / kWarps, kParts = D == 256 ? 2 : 1;
  uint2 w[kOf][kParts];
};
template <int D, int NT>
__device__ __forceinline__ void fetch_q(const AttnArgs &a, const Seq &s, int hk, int first, int count, QRows<D, NT> &q) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < QRows<D, NT>::kOf; ++i) {
    const int n = warp + kWarps * i, rr = first + n, tok = rr / a.r;
    const __nv_bfloat16 *const src =
        static_cast<const __nv_bfloat16 *>(a.q) + (s.row0 + (long long)tok) * a.ldq + (hk * a.r + rr - tok * a.r) * D + 4 * lane;
#pragma unroll
    for (int u = 0; u < QRows<D, NT>::kParts; ++u)
      q.w[i][u] = n < count && 4 * lane < D ? *reinterpret_cast<const uint2 *>(src + 128 * u) : make_uint2(0, 0);
  }
}
// q as mma operands: element (row n, dim 64 c + 16 t + 4 s + e) is in k step 4 c + s, lane 4 (n % 8) + t,
// times a power of two that brings the row's largest into [2^14, 2^15).
template <int D, int NT>
__device__ __forceinline__ void store_q(const AttnArgs &a, const QRows<D, NT> &q, uint8_t *sq, float *qscale) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kOf = QRows<D, NT>::kOf, kParts = QRows<D, NT>::kParts;
  uint32_t top[kOf];  // bits of the largest size: those of NaN are above infinity's
#pragma unroll
  for (int i = 0; i < kOf; ++i) {
    top[i] = 0;
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
      const uint32_t x = q.w[i][u].x & 0x7fff7fffu, y = q.w[i][u].y & 0x7fff7fffu;
      top[i] = max(top[i], max(max(x & 0xffffu, x >> 16), max(y & 0xffffu, y >> 16)));
    }
  }
#pragma unroll
  for (int i = 0; i < kOf; ++i) top[i] = __reduce_max_sync(0xffffffffu, top[i]);
#pragma unroll
  for (int i = 0; i < kOf; ++i) {
    const int n = warp + kWarps * i;
    const bool bad = top[i] >= 0x7f80u;
    const int e = top[i] > 0 && !bad ? min(14 - ((int)(top[i] >> 7) - 127), 120) : 0;
    const float up = bad ? __int_as_float(0x7fc00000) : __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
      const int gr = lane + 32 * u;  // group of 4 elements
      if (4 * lane >= D) break;
      const int kstep = (gr >> 4) * 4 + (gr & 3), t = (gr >> 2) & 3;
      const uint32_t at = ((kstep * NT + (n >> 3)) * 32 + (n & 7) * 4 + t) * 8;
      const float2 x = unpack_bf16(q.w[i][u].x), y = unpack_bf16(q.w[i][u].y);
      *reinterpret_cast<uint2 *>(sq + at) = make_uint2(pack2_sat(x.x * up, x.y * up), pack2_sat(y.x * up, y.y * up));
    }
    if (lane == 0) qscale[n] = __uint_as_float((uint32_t)(127 - e) << 23) * (a.scale * kLog2e);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, kBlocksSM) attn_few_kernel(const AttnArgs a, int least) {
  using G = Geo<D, NT>;
  constexpr int RT = 8 * NT, MT = D / 16, SUB = G::kSub;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *const sq = smem + G::kRing;
  __shared__ __align__(8) uint64_t bars[kWarps][G::kDepth];
  __shared__ RowAt at_row[2][RT];  // of the piece at hand, and of the one whose results go out
  __shared__ float qscale[RT], wm[kWarps][RT], wl[kWarps][RT], row_m[RT], row_l[RT];
  __shared__ volatile int gave_up;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const CacheArgs &c = a.cache;
  if (tid < kWarps * G::kDepth) bar_init(&bars[tid / G::kDepth][tid % G::kDepth], 1);
  if (tid == 0) gave_up = 0;
  __syncthreads();
  const bool whole = a.ws == nullptr;
  constexpr Cut cut{RT, G::kSlab, G::kStart};
  const Located loc = locate<kThreads>(a, cut, blockIdx.x, gridDim.x, whole ? 1 : least, whole);
  if (loc.b < 0) return;
  long long left = min(loc.share, loc.total - loc.share * blockIdx.x);  // of the range, from the next slab on
  SeqLen q = seq_len(a, loc.b, cut);
  int unit = whole ? (int)loc.in_seq : quotient(loc.in_seq, q.each);
  int slab0 = 0;
  if (!whole) {
    slab0 = (int)(loc.in_seq - (long long)unit * q.each) - cut.start;
    if (slab0 < 0) {  // the range starts with a unit's start
      left += slab0;
      slab0 = 0;
      if (left <= 0) return;
    }
  }
  uint8_t *const ring = smem + warp * (G::kDepth * G::kSlabBytes);
  uint64_t *const bar = bars[warp];
  uint32_t parity = 0;  // bit i: of slot i's next phase
  const int page = 1 << c.page_shift;
  const long long page_bytes = (long long)c.Hk * page * D;
  constexpr int kStep = kWarps * G::kSlab;  // tokens from one of a warp's slabs to the next

  // The piece of work at hand: rows first .. first + count - 1 of a key head, slabs slab0 .. slab1 - 1 of their tokens.
  // A warp's are slab0 + warp + kWarps i, i < mine; the pages and scales of 32 of their 16 tokens at a time, one per lane.
  int hk, first, count, seen, mine, tok_first, slab1, turn = 0;
  bool starts, ends;
  const int *table;
  const uint8_t *copy_src;
  int pg[2];
  float2 sc[2];
  QRows<D, NT> rows;
  auto load_page = [&](int x) -> int {  // x: 16 tokens, SUB to a slab
    const int i = x / SUB, tok = tok_first + i * kStep + (x % SUB) * 16;
    if (i >= mine || tok >= seen) return -1;
    const int p = table[tok >> c.page_shift];
    if (p >= 0 && p < c.n_pages) return p;
    atomicOr(a.seq.err, kErrSeqlens);
    return -1;
  };
  auto load_scales = [&](int p) -> float2 {
    if (p < 0) return make_float2(0.f, 0.f);
    const long long at = (long long)p * c.Hk + hk;
    return make_float2(c.ks[at], c.vs[at]);
  };
  // Makes the piece at (q, unit, slab0) the one at hand and asks for its pages, queries (ahead of the copies, which
  // would hold them up) and scales.
  auto open = [&] {
    const int tile = unit % q.tiles;
    hk = unit / q.tiles;
    first = tile * RT;
    count = min(RT, q.s.n * a.r - first);
    slab1 = whole ? q.slabs : (int)min((long long)q.slabs, slab0 + left);
    starts = slab0 == 0;
    ends = slab1 == q.slabs;
    seen = a.causal ? min(q.s.kv, max(0, q.s.kv - q.s.n + (first + count - 1) / a.r + 1)) : q.s.kv;
    const int slab_hi = min(slab1, (seen + G::kSlab - 1) / G::kSlab);
    mine = slab_hi - slab0 > warp ? (slab_hi - slab0 - warp + kWarps - 1) / kWarps : 0;
    table = c.table + (long long)q.s.b * c.table_ld;
    tok_first = (slab0 + warp) * G::kSlab;
    // Lane 8 sub + 0 .. 3 copies 4 tokens each of 16 tokens' k, 4 .. 7 of their v.  What has no page is copied
    // from page 0 and not looked at.
    copy_src = (lane & 4 ? c.v : c.k) + ((long long)hk * page + 4 * (lane & 3)) * D;
    turn ^= 1;
    pg[0] = load_page(lane);
    pg[1] = load_page(lane + 32);
    fetch_q<D, NT>(a, q.s, hk, first, count, rows);
    if (tid < RT) {
      const int rr = first + tid, tok = rr / a.r;
      at_row[turn][tid] = RowAt{(long long)q.s.row0 + tok, hk * a.r + rr - tok * a.r};
    }
    sc[0] = load_scales(pg[0]);
    sc[1] = load_scales(pg[1]);
  };
  const uint32_t copy_dst = (lane >> 3) * 2 * G::kK + (lane & 7) * G::kGroup;
  auto issue = [&](int i, int p, uint32_t slot) {  // the copies of slab i into the ring; p: the lane's page
    uint64_t *const b = bar + slot;
    if (lane == 0) bar_expect_tx(b, SUB * 8 * 4 * D);
    __syncwarp();
    if (lane < 8 * SUB) {
      const int tok = (tok_first + i * kStep + (lane >> 3) * 16) & (page - 1);
      bulk_load(smem_u32(ring + slot * G::kSlabBytes) + copy_dst, copy_src + max(p, 0) * page_bytes + tok * D, 4 * D, b);
    }
    __syncwarp();
  };
  // A piece's slabs go round the ring from behind the slots that the last piece's results are merged in.
  auto issue_first = [&](int i0, int i1) {
#pragma unroll 1
    for (int i = i0; i < min(mine, i1); ++i)
      issue(i, __shfl_sync(0xffffffffu, pg[0], (i * SUB + (lane >> 3)) & 31), (uint32_t)(i + G::kMergeSlots) % G::kDepth);
  };

  open();
  issue_first(0, G::kDepth);
  while (true) {
    store_q<D, NT>(a, rows, sq, qscale);
    __syncthreads();

    constexpr bool kQRegs = D * NT <= 256;
    uint2 qr[kQRegs ? MT : 1][kQRegs ? NT : 1];
    if constexpr (kQRegs) {
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int j = 0; j < NT; ++j) qr[k][j] = *reinterpret_cast<const uint2 *>(sq + ((k * NT + j) * 32 + lane) * 8);
    }
    // m, l: what the weights are relative to, their sum; mv: what acc is, in weight times value scale; up: 2^(m - mv) as fp16 has it
    float acc[MT][NT][4], m[NT][2], l[NT][2], mv[NT][2], up[NT][2], qs[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        m[j][u] = mv[j][u] = kNone;
        l[j][u] = up[j][u] = 0.f;
        qs[j][u] = qscale[8 * j + 2 * t + u];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i][j][u] = acc[i][j][2 + u] = 0.f;
      }
    auto last_of = [&](int j, int u) {  // the last token that a row sees
      const int row = 8 * j + 2 * t + u;
      return row >= count ? -1 : a.causal ? q.s.kv - q.s.n + (int)(at_row[turn][row].token - q.s.row0) : q.s.kv - 1;
    };
    // Tokens up to this one are seen by every row (rows that are none may see them too: nothing reads those).
    const int all_see = a.causal ? q.s.kv - q.s.n + first / a.r : q.s.kv - 1;
    // Rows g and g + 8 of S^T are these tokens of 16.
    const int tg = g >> 1, bg = g & 1, gr0 = (tg + 2 * bg) & 3, gr1 = (tg + 2 * bg + 1) & 3;
    const int in0 = 4 * gr0 + 2 * bg, in1 = 4 * gr1 + 2 * bg + 1;
    const uint32_t k_at0 = gr0 * G::kGroup + 2 * bg * D + 16 * t, k_at1 = gr1 * G::kGroup + (2 * bg + 1) * D + 16 * t;

    auto wait = [&](uint32_t slot) {
      const uint32_t phase = parity >> slot & 1;
      parity ^= 1u << slot;
      if (!bar_try_wait(bar + slot, phase)) {
        const uint64_t t0 = global_ns();
        while (!gave_up && !bar_try_wait(bar + slot, phase))
          if (global_ns() - t0 > 1000000000ull) {
            gave_up = 1;  // what follows is not right, and stays in its bounds
            atomicOr(a.seq.err, kErrTimeout);
          }
      }
      __syncwarp();
    };
    // S^T of a slab; 16 tokens alone in two chains of products
    auto scores = [&](uint32_t slot, float (&st)[SUB][NT][4]) {
      constexpr int kChains = SUB == 1 ? 2 : 1;
      float sb[kChains][NT][4];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int j = 0; j < NT; ++j) st[u][j][0] = st[u][j][1] = st[u][j][2] = st[u][j][3] = 0.f;
      if constexpr (kChains == 2)
#pragma unroll
        for (int j = 0; j < NT; ++j) sb[1][j][0] = sb[1][j][1] = sb[1][j][2] = sb[1][j][3] = 0.f;
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch)
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const uint8_t *const sk = ring + slot * G::kSlabBytes + u * 2 * G::kK;
          const uint4 w0 = *reinterpret_cast<const uint4 *>(sk + k_at0 + 64 * ch), w1 = *reinterpret_cast<const uint4 *>(sk + k_at1 + 64 * ch);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t x0 = word(w0, s), x1 = word(w1, s);
            const uint32_t a0 = e4m3x2_to_h2(x0, 0), a1 = e4m3x2_to_h2(x1, 0), a2 = e4m3x2_to_h2(x0, 1), a3 = e4m3x2_to_h2(x1, 1);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              uint2 bq;
              if constexpr (kQRegs)
                bq = qr[4 * ch + s][j];
              else
                bq = *reinterpret_cast<const uint2 *>(sq + (((4 * ch + s) * NT + j) * 32 + lane) * 8);
              if (kChains == 2 && (s & 1))
                mma16816(sb[kChains - 1][j], a0, a1, a2, a3, bq.x, bq.y);
              else
                mma16816(st[u][j], a0, a1, a2, a3, bq.x, bq.y);
            }
          }
        }
      if constexpr (kChains == 2)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) st[0][j][e] += sb[1][j][e];
    };

    float st[SUB][NT][4];
    uint32_t slot = G::kMergeSlots % G::kDepth;
    if (mine > 0) {
      wait(slot);
      scores(slot, st);
    }
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      constexpr int kBatch = 32 / SUB;  // slabs
      const int in = i & (kBatch - 1);
      if (in == 0 && i > 0) {
        pg[0] = pg[1];
        sc[0] = sc[1];
        pg[1] = load_page((i + kBatch) * SUB + lane);
      }
      if (in == kBatch / 2 && i > kBatch) sc[1] = load_scales(pg[1]);
      float ks[SUB], vs[SUB], lv[SUB];
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        ks[u] = __shfl_sync(0xffffffffu, sc[0].x, in * SUB + u);
        vs[u] = __shfl_sync(0xffffffffu, sc[0].y, in * SUB + u);
        lv[u] = __log2f(vs[u]);  // of 0: below all; of NaN: passed over by the maxima
      }
      const uint32_t next = slot + 1 == G::kDepth ? 0 : slot + 1;
      const int tok0 = tok_first + i * kStep;
      float y[SUB][NT][4];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[u][j][e] = st[u][j][e] * (qs[j][e & 1] * ks[u]);
      // The next slab's scores are on their way while this one's weights are formed.
      if (i + 1 < mine) {
        wait(next);
        scores(next, st);
      }
      // Tokens that some row does not see, or that have no page.
      const uint32_t gone = (__ballot_sync(0xffffffffu, pg[0] < 0) >> (in * SUB)) & ((1u << SUB) - 1);  // bit u: no page
      const bool masked = gone != 0 || tok0 + G::kSlab - 1 > all_see;
      if (masked) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int last = gone >> u & 1 ? -1 : last_of(j, e);
              y[u][j][e] = tok0 + 16 * u + in0 > last ? -INFINITY : y[u][j][e];
              y[u][j][2 + e] = tok0 + 16 * u + in1 > last ? -INFINITY : y[u][j][2 + e];
            }
        __syncwarp();
      }
      float top[NT][2], topv[NT][2], high = -INFINITY;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[j][e] = fmaxf(y[0][j][e], y[0][j][2 + e]);
          topv[j][e] = top[j][e] + lv[0];
#pragma unroll
          for (int u = 1; u < SUB; ++u) {
            const float x = fmaxf(y[u][j][e], y[u][j][2 + e]);
            top[j][e] = fmaxf(top[j][e], x);
            topv[j][e] = fmaxf(topv[j][e], x + lv[u]);
          }
          high = fmaxf(high, fmaxf(top[j][e] - m[j][e], topv[j][e] - mv[j][e]));
        }
      if (__any_sync(0xffffffffu, high > kSlack + kLift)) {
        auto over_lanes = [](float x) {
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        };
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = fmaxf(over_lanes(top[j][e]) - kLift, m[j][e]), z = fmaxf(over_lanes(topv[j][e]) - kLift, mv[j][e]);
            l[j][e] *= ex2(m[j][e] - x);
            al[e] = ex2(mv[j][e] - z);
            m[j][e] = x;
            mv[j][e] = z;
            up[j][e] = ex2(fminf(x - z + (kPExp - kLift), 120.f));  // at most 2^105 where a value scale is above 0
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
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float pv[2] = {vs[u] * up[j][0], vs[u] * up[j][1]};  // NaN where the scale is
          float pp[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = ex2(y[u][j][e] - m[j][e & 1]);
            l[j][e & 1] += w;
            pp[e] = masked && y[u][j][e] == -INFINITY ? 0.f : w * pv[e & 1];  // 0 whatever the scale is
          }
          pb[j][0] = transpose8(pack2_sat(pp[0], pp[1]));
          pb[j][1] = transpose8(pack2_sat(pp[2], pp[3]));
        }
        // O^T: this lane's tokens are k = 2 t, 2 t + 1 (half 0) and 2 t + 8, 2 t + 9 (half 1)
        const uint8_t *const sv = ring + slot * G::kSlabBytes + u * 2 * G::kK + G::kK;
        const int ga = t, gb = (t + 2) & 3, gc = (t + 1) & 3, gd = (t + 3) & 3;
        constexpr int W = D >= 128 ? 16 : 8;  // bytes of a lane per token and load
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
          if (masked) {  // bytes behind the end, or of no page, may be anything, NaN too
            const int tk[4] = {4 * ga, 4 * gb + 2, 4 * gc + 1, 4 * gd + 3};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const bool none = tok0 + 16 * u + tk[k] >= q.s.kv || (gone >> u & 1);
#pragma unroll
              for (int e = 0; e < W / 4; ++e) w[k][e] = none ? 0 : w[k][e];
            }
            __syncwarp();  // the lanes' tests are behind: what follows takes the warp
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
        const int x = (i + G::kDepth) * SUB + (lane >> 3), src = x & 31;
        const int p0 = __shfl_sync(0xffffffffu, pg[0], src), p1 = __shfl_sync(0xffffffffu, pg[1], src);
        issue(i + G::kDepth, x / 32 == i / kBatch ? p0 : p1, slot);
      }
      slot = next;
    }

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
    asm volatile("griddepcontrol.launch_dependents;");  // the join may come up
    __syncthreads();  // every warp is through with its ring
    float *const merge = reinterpret_cast<float *>(ring);
    if (tid < RT) {
      float top = kNone, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, wm[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += ex2(wm[w][tid] - top) * wl[w][tid];
      row_m[tid] = top;
      row_l[tid] = sum;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 8 * j + 2 * t + u;
        float top = kNone;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, wm[w][row]);
        const float f = ex2(mv[j][u] - top + (kLift - kPExp));  // never below 2^-110: a value scale is above 2^-121, or all are 0
#pragma unroll
        for (int i2 = 0; i2 < MT; ++i2)
          *reinterpret_cast<float2 *>(merge + row * G::kPitch + merge_at<D>(g, i2)) = make_float2(acc[i2][j][u] * f, acc[i2][j][2 + u] * f);
      }
    // The next piece is asked for while this one's results go out.
    const bool whole_unit = starts && ends;
    const int part = 2 * blockIdx.x + (starts ? 1 : 0), out_rows = count;
    const RowAt *const out_at = at_row[turn];
    left -= whole ? 1 : slab1 - slab0 + cut.start;
    slab0 = 0;
    ++unit;
    bool more = left > 0;
    if (more && unit >= q.tiles * c.Hk) {  // the next sequence that has rows
      unit = 0;
      for (int nb = q.s.b + 1;; ++nb) {
        more = nb < a.seq.B;
        if (!more) break;
        q = seq_len(a, nb, cut);
        if (q.len > 0) break;
      }
    }
    if (more) {
      open();
      issue_first(0, G::kDepth - G::kMergeSlots);
    }
    __syncthreads();
#pragma unroll 4
    for (int x = tid; x < out_rows * (D / 2); x += kThreads) {
      const int row = x / (D / 2), dim = x % (D / 2) * 2;
      const int at = D >= 128 ? merge_at<D>((dim >> 4) & 7, (dim >> 7) * 8 + ((dim >> 1) & 7)) : dim;
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = *reinterpret_cast<const float2 *>(smem + w * (G::kDepth * G::kSlabBytes) + (row * G::kPitch + at) * 4);
        o.x += v.x, o.y += v.y;
      }
      if (whole_unit) {
        const float ls = row_l[row], inv = ls == 0.f ? 0.f : 1.f / ls;
        __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(a.o) + out_at[row].token * a.ldo + out_at[row].head * D + dim;
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16(o.x * inv, o.y * inv);
      } else {
        *reinterpret_cast<float2 *>(part_o(a.ws, part, RT, D) + row * D + dim) = o;
        if (dim == 0) part_ml(a.ws, 2 * gridDim.x, part, RT, D)[row] = make_float2(row_m[row], row_l[row]);
      }
    }
    if (!more) break;
    fence_smem_to_async();  // before the next copies into what was written here
    __syncthreads();
    issue_first(G::kDepth - G::kMergeSlots, G::kDepth);
  }
  if (gave_up) settle();
}

// Joins a unit's parts:  o = sum 2^(m_p - m) o_p / sum 2^(m_p - m) l_p.  by_unit: block x takes unit x (of
// tiles_max Hk to a sequence); else the unit in which boundary x + 1 between the blocks' ranges is the first.
// Rows of its tile over blockIdx.y; the threads stand side by side over 4 columns each and over the parts.
template <int D, int NT, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads) attn_few_join(const AttnArgs a, int least, int parts, int tiles_max, int by_unit) {
  using G = Geo<D, NT>;
  constexpr int RT = 8 * NT, kCols = D / 4, kSide = kJoinThreads / kCols;
  constexpr Cut cut{RT, G::kSlab, G::kStart};
  __shared__ float4 sums[kSide][kCols];
  __shared__ float side_l[kSide], side_m[kSide];
  const int col = threadIdx.x % kCols, side = threadIdx.x / kCols;
  SeqLen q{};
  long long start = 0, share = 0;  // of the unit's first slab; a block's range
  int unit = 0;
  if (by_unit) {
    const int per = tiles_max * a.cache.Hk, b = blockIdx.x / per, x = blockIdx.x % per;
    const Located loc = locate<kJoinThreads>(a, cut, 0, parts, least, false, b);
    q = seq_len(a, b, cut);
    const int hk = x / tiles_max, tile = x % tiles_max;
    unit = hk * q.tiles + tile;
    share = loc.share;
    start = loc.in_seq + (long long)unit * q.each + cut.start;
    if (loc.total == 0 || q.len == 0 || tile >= q.tiles) share = 0;
  } else {
    const Located loc = locate<kJoinThreads>(a, cut, blockIdx.x + 1, parts, least, false);
    if (loc.b >= 0) {
      q = seq_len(a, loc.b, cut);
      unit = quotient(loc.in_seq, q.each);
      const int slab = (int)(loc.in_seq - (long long)unit * q.each) - cut.start;
      if (slab > 0 && slab <= loc.share) share = loc.share;  // else before the slabs, or not the first boundary inside
      start = loc.share * (blockIdx.x + 1) - slab;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial results are written (no block ends before that)
  if (share == 0) return;
  const int c0 = quotient(start, (int)share), c1 = quotient(start + q.slabs - 1, (int)share);
  if (c0 == c1) return;  // in one range: written already
  const int hk = unit / q.tiles, first = unit % q.tiles * RT, rows = min(RT, q.s.n * a.r - first);
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const int rr = first + row;
    const auto slot_of = [&](int c) { return 2 * c + (c == c0 ? 1 : 0); };  // its first part starts it
    float m = kNone, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // Each side with a maximum of its own; 4 parts' loads in flight.
#pragma unroll 1
    for (int c = c0 + side; c <= c1; c += 4 * kSide) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int cu = c + u * kSide;
        ml[u] = make_float2(kNone, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cu <= c1) {
          ml[u] = part_ml(a.ws, 2 * parts, slot_of(cu), RT, D)[row];
          v[u] = *reinterpret_cast<const float4 *>(part_o(a.ws, slot_of(cu), RT, D) + row * D + 4 * col);
        }
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < 4; ++u) mn = fmaxf(mn, ml[u].x);
      const float w0 = ex2(m - mn);
      l *= w0;
      o.x *= w0, o.y *= w0, o.z *= w0, o.w *= w0;
      m = mn;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float w = ex2(ml[u].x - mn);
        l += w * ml[u].y;
        o.x += w * v[u].x, o.y += w * v[u].y, o.z += w * v[u].z, o.w += w * v[u].w;
      }
    }
    if (col == 0) side_m[side] = m;
    __syncthreads();
    float top = kNone;
#pragma unroll
    for (int u = 0; u < kSide; ++u) top = fmaxf(top, side_m[u]);
    const float w = ex2(m - top);
    sums[side][col] = make_float4(o.x * w, o.y * w, o.z * w, o.w * w);
    if (col == 0) side_l[side] = l * w;
    __syncthreads();
    if (side == 0) {
      float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
      float ls = 0.f;
#pragma unroll
      for (int u = 0; u < kSide; ++u) {
        const float4 v = sums[u][col];
        all.x += v.x, all.y += v.y, all.z += v.z, all.w += v.w;
        ls += side_l[u];
      }
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(a.o) + (long long)(q.s.row0 + rr / a.r) * a.ldo +
                                 (long long)(hk * a.r + rr % a.r) * D + 4 * col;
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(all.x * inv, all.y * inv), pack_bf16(all.z * inv, all.w * inv));
    }
    __syncthreads();
  }
}

template <int D, int NT>
struct FewTag {};

// Slabs of a block's range at least: one per warp, and 128 tokens (1 token over 4096, 4 heads of 256, 12 us:
// 64 tokens take 2.1 more, 256 0.2 and 512 3.4; heads of 64 and 128 lose with every slab beyond one per warp).
template <int D, int NT>
constexpr int kLeast = Geo<D, NT>::kSlab * kWarps >= 128 ? kWarps : 128 / Geo<D, NT>::kSlab;

template <int D, int NT>
cudaError_t launch(const AttnArgs &a, int num_sms, cudaStream_t s) {
  cudaError_t e = allow_smem<FewTag<D, NT>>(attn_few_kernel<D, NT>, Geo<D, NT>::kBytes);
  if (e != cudaSuccess) return e;
  const int blocks = kBlocksSM * num_sms;
  attn_few_kernel<D, NT><<<blocks, kThreads, Geo<D, NT>::kBytes, s>>>(a, kLeast<D, NT>);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.ws) return e;
  // The join comes up while the last pieces end, and waits for them.
  cudaLaunchConfig_t cfg{};
  const int tiles_max = (int)(((long long)a.seq.max_new * a.r + 8 * NT - 1) / (8 * NT));
  const long long units = (long long)a.seq.B * tiles_max * a.cache.Hk;
  const int by_unit = units < blocks;
  // rows of a tile side by side, as many as are all up at once
  cfg.gridDim = dim3(by_unit ? (unsigned)units : blocks - 1);
  cfg.gridDim.y = std::max(1u, std::min(8u * NT, 8u * num_sms / cfg.gridDim.x));
  // Few units have many parts each: 8 side by side (1 token over 16384, heads of 256, in a graph: 20.0 us with 2, 17.2
  // with 8; 16 x 4 tokens, whose parts are few, 34.9 and 47).
  const bool wide = units * 8 * NT <= num_sms;
  cfg.blockDim = dim3(wide ? 2 * D : kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, wide ? attn_few_join<D, NT, 2 * D> : attn_few_join<D, NT, kThreads>, a, kLeast<D, NT>, blocks, tiles_max, by_unit);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

// From where on tiles of 128 rows are faster: with heads of 128 and 32 rows (16 x 4 tokens over 16000, 4 key heads) they
// take 91 us where this kernel takes 115, one sequence 21 and 32; with 16 rows (8 key heads) 164 and 113, with heads of
// 64 and 32 rows 81 and 76; with heads of 256 and 32 rows 80 and 104, 16 rows 113 and 103.
int attn_few_rows(int D, long long rows) {
  const int most = D == 64 ? 32 : 16;
  for (int t = 8; t <= most; t *= 2)
    if (rows <= t) return t;
  return 0;
}

size_t attn_few_ws_bytes(int D, int rows_tile, int num_sms) { return (size_t)2 * kBlocksSM * num_sms * rows_tile * (D + 2) * sizeof(float); }

cudaError_t launch_attn_few(const AttnArgs &a, int rows_tile, int num_sms, cudaStream_t s) {
  const int nt = rows_tile / 8;
  switch (a.cache.D) {
    case 256: return nt == 1 ? launch<256, 1>(a, num_sms, s) : launch<256, 2>(a, num_sms, s);
    case 128: return nt == 1 ? launch<128, 1>(a, num_sms, s) : launch<128, 2>(a, num_sms, s);
    default: return nt == 1 ? launch<64, 1>(a, num_sms, s) : nt == 2 ? launch<64, 2>(a, num_sms, s) : launch<64, 4>(a, num_sms, s);
  }
}

}  // namespace gdn
