// attn_tile.cu -- attention of many rows over the paged 8-bit cache (bf16 io): prompts.
//
// A CTA takes 128 rows (query tokens x the query heads of one key head) and goes
// over the tokens in tiles of 64 on the tensor cores, one pass with the running
// maximum and sum of each row:
//   S = Q K^T   e4m3 products straight on the cache's bytes, which TMA brings from
//               the pages.  Q stands in TMEM (or shared memory) as two e4m3 values
//               per element, hi + lo of q times a power of two per row: all 8 bits of
//               a bf16 that is not below 2^-9 of its row's largest, and never off by
//               more than 2^-17 of that largest.
//   O += P V    fp16 products: P, rounded to fp16, in TMEM where S was; V's bytes
//               become fp16 (exact) on the way through a group of four warps.
// A page's key scale multiplies its scores.  Its value scale enters p as a term of the
// exponent, and leaves the row's sum again as a factor on the page's part of it: no
// product per element.  What O is relative to is the running maximum of weight times
// value scale, apart from that of the weights alone: in fp16 p has 11 bits down to 2^-25
// of the row's largest product, and is within 2^-36 of it below that.
//
// Bound by the products for heads of 256 (8192 tokens over 24576, 24/4 heads: 3.3 to
// 3.6 ms as the power cap leaves it, 1.6 to 1.75 PFLOP/s of bf16's 1.7 sustained; the products of
// q's two parts are twice those of one, at twice the rate), by the softmax's instructions for
// narrower ones (2048 over 8192, 32/4 heads of 128: 260 us, 1.19 PFLOP/s; of 64: 235 us, 0.66).
//
// Warps: 4 for the softmax (thread = row), 4 for the values, one for the keys
// (TMA) and one for the products.  For a tile of 64 tokens and D = 256 the products
// take 1024 cycles; a tile's way through the softmax is longer than that: two groups
// of warps, which take tiles in turns.  Narrower heads have two blocks to an SM for
// that.  The running maximum goes from one group to the other as soon as it is known,
// ahead of the exponentials; each keeps a sum of its own.
#include <algorithm>

#include "cache_device.cuh"
#include "tma_host.h"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int kRows = 128;    // of a CTA
constexpr int kTile = 64;     // tokens
constexpr int kSubs = kTile / 16;
constexpr int kRing = 8;      // tiles whose scales are kept
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -1.7e38f;
constexpr float kSlack = 4.f;   // p may reach 2^kSlack before the running maximum moves
constexpr float kPExp = 11.f;   // p stands times 2^11 in fp16
constexpr float kMinRatio = -60.f;
constexpr float kNoScale = -200.f;  // the logarithm of a value scale of 0

template <int D>
struct Geo {
  // Blocks of an SM, groups of softmax warps of a block, which take tiles in turns, and buffers of S.  Where TMEM holds
  // two blocks (Q is in shared memory then) they take turns by themselves, and one works while the other starts or ends.
  static constexpr int kBlocks = D == 256 ? 1 : 2, kGroups = D == 256 ? 2 : 1, kBufs = 2;
  static constexpr bool kQSmem = D < 256;
  static constexpr int kValueWarp = 4 * kGroups, kKeyWarp = kValueWarp + 4, kProductWarp = kKeyWarp + 1;
  static constexpr int kThreads = 32 * (kProductWarp + 1);
  // A softmax warp that waits for the products of tile j - 1 knows those of tile j - 1 - kBufs to be done, from the
  // scores that followed them: a slot of V, whose phases it tells apart by their parity, comes round no sooner.
  static constexpr int kKStages = 4, kVStages = 2;
  static_assert(kVStages >= kBufs, "phases of V");
  static constexpr int kKBytes = kTile * D, kVBytes = kTile * D * 2, kQBytes = kQSmem ? 2 * kRows * D : 0;
  // The rows of q, then of o, between global memory and the threads that have a row each: where V is before and after.
  static constexpr int kRowPitch = 2 * D;
  static_assert(kRows * kRowPitch <= kVStages * kVBytes, "rows");
  static constexpr int kSmem = kKStages * kKBytes + kVStages * kVBytes + kQBytes + 1024;
  // TMEM columns
  [[maybe_unused]] static constexpr int kQ = 0;
  static constexpr int kO = kQSmem ? 0 : D / 2, kS = kO + D;
  static constexpr int kCols = 512 / kBlocks;
  static_assert(kS + kBufs * kTile <= kCols, "TMEM");
  // K-major rows of 128 bytes (D = 64: 64) with the swizzle of that width
  static constexpr int kRowBytes = D >= 128 ? 128 : 64;
};

// One lane of a converged warp.  Instructions that a warp issues once (products, commits) stand in a branch on it: the
// compiler then knows that a single lane is there and keeps their operands uniform (a predicate per product on the
// lane's number takes twice the issue time, which bounds a tile: 8192 over 24576 4.4 ms, so 3.5).
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}\n" : "=r"(p));
  return p != 0;
}
// tcgen05.mma with A in TMEM: e4m3 operands (4 bytes along K to a column: a K step of 32 advances 8), or fp16 ones.
template <bool kF8, bool kAccumulate>
__device__ __forceinline__ void mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t id) {
  if constexpr (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(id), "n"(kAccumulate ? 1 : 0));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(id), "n"(kAccumulate ? 1 : 0));
}
// The same of e4m3 operands, both in shared memory with the same strides.
template <bool kAccumulate>
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(id), "n"(kAccumulate ? 1 : 0));
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 t = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&t);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z, w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(w) : "l"(x), "l"(y), "l"(z));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(w));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t x, y, w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(w) : "l"(x), "l"(y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(w));
  return r;
}

// 16-byte chunk `ch` of a row of q or o in shared memory, turned so that neither rows nor chunks side by side share banks.
template <int D>
__device__ __forceinline__ uint32_t row_at(int row, int ch) {
  return (uint32_t)(row * Geo<D>::kRowPitch + ((ch ^ (row & 7)) << 4));
}
// 16 e4m3 values of a row as an operand with K contiguous: rows of 128 bytes (64 for D = 64) with the swizzle of that width.
template <int D>
__device__ __forceinline__ uint32_t f8_at(int row, int ch) {
  return D >= 128 ? (uint32_t)(row * 128 + ((ch ^ (row & 7)) << 4)) : (uint32_t)(row * 64 + ((ch ^ ((row >> 1) & 3)) << 4));
}
// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

struct Bars {
  uint64_t q_read, k_full[4], k_empty[4], v_full[2], v_empty[2], s_full[2], p_full[2], scales[kRing];
  uint64_t moved[2][4];  // the running maximum after a tile, per warp
};

// Entries of the table for the 16 tokens `sub` of a tile.  ask() loads one (kUnseen: its tokens are not looked
// at); a tile or two later page() says what it is worth, so that nothing waits for the load.
constexpr int kUnseen = -0x40000000;
struct TilePages {
  const CacheArgs &c;
  const int *table;
  int base, seen;  // tile 0, the tokens looked at
  unsigned int *err;
  __device__ __forceinline__ int ask(int tile, int sub) const {
    const int tok = (base + tile) * kTile + sub * 16;
    return tok < seen ? table[tok >> c.page_shift] : kUnseen;
  }
  __device__ __forceinline__ int page(int entry) const {
    if ((unsigned)entry < (unsigned)c.n_pages) return entry;
    if (entry != kUnseen) atomicOr(err, kErrSeqlens);
    return -1;
  }
};

// The last blocks' tokens may be cut into a.splits parts (all blocks' where they do not fill the GPU): a part is a
// block from number a.whole on, and leaves 128 rows of D values; behind those of all parts their (maximum, sum).
__device__ __forceinline__ long long part_row(long long part) { return part * kRows; }
__device__ __forceinline__ float *part_ml(const AttnArgs &a, long long parts, int D) { return static_cast<float *>(a.ws) + parts * kRows * D; }

// Blocks start with the tiles that see the most, whatever sequence and head they are of, so that what runs last is
// short (12 prompts: 73.6 us, in the sequences' order 76.5).  Tile t of a sequence counts as P + t, P the 128s of rows
// that its cached tokens would have been; of all tiles this finds number `rank` from the largest down (equal ones in the
// sequences' order), for the whole block: how many are above a size is a sum over the sequences, which one warp forms,
// and the range of sizes is quartered until one is left.  More sequences than 4 to a lane are taken in order, the
// last first.
constexpr int kSeqsLane = 4;
__device__ __forceinline__ Seq find_largest(const AttnArgs &a, int rank, int ranks, int *local) {
  const SeqArgs &g = a.seq;
  if (g.B == 1) {  // nothing to search
    const int lo = g.cu ? g.cu[0] : 0, hi = g.cu ? g.cu[1] : g.T, kv = g.kv_lens[0];
    if (lo < 0 || hi < lo || hi > g.T) {
      if (threadIdx.x == 0) atomicOr(g.err, kErrSeqlens);
      return Seq{-1, 0, 0, 0};
    }
    *local = (int)(((long long)(hi - lo) * a.r + kRows - 1) / kRows) - 1 - rank;
    Seq s = checked_seq(g, 0, lo, hi - lo, kv);
    if (*local < 0) s.b = -1;
    return s;
  }
  if (g.B > 32 * kSeqsLane) return find_seq(g, ranks - 1 - rank, a.r, kRows, 1, local);
  __shared__ Seq found;
  __shared__ int at;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int row0[kSeqsLane], n[kSeqsLane], kv[kSeqsLane], from[kSeqsLane], tiles[kSeqsLane];
    bool bad = false, out = false;
#pragma unroll
    for (int k = 0; k < kSeqsLane; ++k) {
      const int b = lane + 32 * k;
      row0[k] = n[k] = kv[k] = 0;
      if (b < g.B) {
        row0[k] = g.cu ? g.cu[b] : b * g.T;
        n[k] = g.cu ? g.cu[b + 1] : g.T;
        kv[k] = g.kv_lens[b];
      }
    }
    int end = 0;
#pragma unroll
    for (int k = 0; k < kSeqsLane; ++k) {
      if (g.cu) {
        bad |= row0[k] < 0 || n[k] < row0[k] || n[k] > g.T;
        n[k] -= row0[k];
      }
      const bool use = n[k] <= g.max_new && kv[k] >= 0 && kv[k] <= g.max_kv;
      out |= !use;
      tiles[k] = use && lane + 32 * k < g.B ? (int)(((long long)n[k] * a.r + kRows - 1) / kRows) : 0;
      from[k] = (int)((long long)max(0, kv[k] - n[k]) * a.r / kRows);
      end = max(end, tiles[k] > 0 ? from[k] + tiles[k] : 0);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (__any_sync(0xffffffffu, out || bad) && lane == 0) atomicOr(g.err, kErrSeqlens);
    const bool one = g.B <= 32;
    auto above = [&](int x) {  // tiles of size x or more
      int c = min(max(from[0] + tiles[0] - x, 0), tiles[0]);
      if (!one)
#pragma unroll
        for (int k = 1; k < kSeqsLane; ++k) c += min(max(from[k] + tiles[k] - x, 0), tiles[k]);
      return __reduce_add_sync(0xffffffffu, c);
    };
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, end);
    if (lane == 0) found.b = -1;
    __syncwarp();
    if (!bad && rank < above(0)) {
      while (hi - lo > 1) {
        const int q = (hi - lo + 3) >> 2, x1 = lo + q, x2 = min(x1 + q, hi), x3 = min(x2 + q, hi);
        const int c1 = above(x1), c2 = above(x2), c3 = above(x3);
        if (c3 > rank) {
          lo = x3;
        } else if (c2 > rank) {
          lo = x2;
          hi = x3;
        } else if (c1 > rank) {
          lo = x1;
          hi = x2;
        } else {
          hi = x1;
        }
      }
      int rest = rank - above(hi);  // among those of size lo
#pragma unroll
      for (int k = 0; k < kSeqsLane; ++k) {
        const bool here = from[k] <= lo && lo < from[k] + tiles[k];
        const uint32_t all = __ballot_sync(0xffffffffu, here);
        if (here && __popc(all & ((1u << lane) - 1)) == rest) {
          found = Seq{lane + 32 * k, row0[k], n[k], kv[k]};
          at = lo - from[k];
        }
        rest -= __popc(all);
      }
    }
  }
  __syncthreads();
  *local = at;
  return found;
}

// Block `n` of a call: a tile of a key head.  The heads of a tile start side by side; but those of one sequence whose
// keys and values would not all stay in a die's half of the L2 one after the other (8192 tokens over 24576, 67 MB:
// 3.66 ms, side by side 3.71).
__device__ __forceinline__ Seq find_block(const AttnArgs &a, int n, int *hk, int *local) {
  const int Hk = a.cache.Hk, ranks = a.blocks / Hk;
  const bool apart = a.seq.B == 1 && 2ll * a.seq.kv_lens[0] * Hk * a.cache.D > (48 << 20);
  *hk = apart ? n / ranks : n % Hk;
  return find_largest(a, apart ? n % ranks : n / Hk, ranks, local);
}

// What the softmax needs of a tile's 4 pages: key scales and logarithms of value scales.
struct Scales {
  float4 ks, lvs;
  uint32_t flags;  // a byte per page: 1 none, 2 a NaN value scale
};

template <int D>
__global__ void __launch_bounds__(Geo<D>::kThreads, Geo<D>::kBlocks) attn_tile_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap) {
  using G = Geo<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int gave_up;
  __shared__ float2 moved[G::kGroups][kRows];  // running maxima, of scores and with value scales, after a group's tile
  __shared__ Scales ring[kRing];
  __shared__ long long row_q[kRows], row_o[kRows];  // elements before a row
  __shared__ float other[G::kGroups][kRows];  // sum of each group at the end
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const CacheArgs &c = a.cache;
  int local = 0;
  const int split = (int)blockIdx.x < a.whole ? 1 : a.splits, part_no = (int)blockIdx.x - a.whole;
  const int z = split > 1 ? part_no % split : 0;
  int hk = 0;
  const Seq s = find_block(a, split > 1 ? a.whole + part_no / split : (int)blockIdx.x, &hk, &local);
  if (s.b < 0) return;
  const int first = local * kRows, count = (int)min((long long)kRows, (long long)s.n * a.r - first);
  if (count <= 0) return;
  const int seen = a.causal ? min(s.kv, max(0, s.kv - s.n + (first + count - 1) / a.r + 1)) : s.kv;
  // this block's tiles: base .. base + ntiles - 1 of the rows'
  const int all = (seen + kTile - 1) / kTile, part = (all + split - 1) / split, base = part * z;
  const int ntiles = max(0, min(part, all - base));

  uint8_t *const smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *const sk = smem, *const sv = smem + G::kKStages * G::kKBytes, *const sq = sv + G::kVStages * G::kVBytes;
  uint8_t *const stage = sv;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      bar_init(&bars.k_full[i], 1);
      bar_init(&bars.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&bars.s_full[i], 1);
      bar_init(&bars.p_full[i], 128);
      for (int w = 0; w < 4; ++w) bar_init(&bars.moved[i][w], 32);
      bar_init(&bars.v_full[i], 128);
      bar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < kRing; ++i) bar_init(&bars.scales[i], 4);
    bar_init(&bars.q_read, 128 * G::kGroups);
    gave_up = 0;
  }
  if (tid < kRows) {
    const int rr = first + tid, tok = rr / a.r;
    row_q[tid] = (s.row0 + (long long)tok) * a.ldq + (long long)(hk * a.r + rr - tok * a.r) * D;
    row_o[tid] = (s.row0 + (long long)tok) * a.ldo + (long long)(hk * a.r + rr - tok * a.r) * D;
  }
  __syncwarp();
  if (warp == G::kProductWarp) tmem_alloc(&tmem_slot, G::kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;

  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (bar_try_wait(bar, parity)) return;
    const uint64_t t0 = global_ns();
    while (!gave_up && !bar_try_wait(bar, parity))
      if (global_ns() - t0 > 1000000000ull) {
        gave_up = 1;  // what follows is not right, and stays in its bounds
        atomicOr(a.seq.err, kErrTimeout);
      }
  };
  const TilePages pages{c, c.table + (long long)s.b * c.table_ld, base, min(seen, (base + ntiles) * kTile), a.seq.err};
  const int page = 1 << c.page_shift;

  auto sync_softmax = [] {
    __syncwarp();
    asm volatile("bar.sync 2, %0;" ::"n"(128 * G::kGroups) : "memory");
  };
  auto sync_products = [] {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(128 * G::kGroups + 32) : "memory");
  };
  if (warp < G::kValueWarp) {
    // ---------------------------------------------------------------- softmax
    const int group = warp >> 2, quarter = warp & 3, row = tid & (kRows - 1), rr = first + row, tok = rr / a.r;
    const bool real = row < count;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    constexpr int kChunks = D / 8;  // 16 bytes each, of a row
#pragma unroll
    for (int x = tid; x < kRows * kChunks; x += 128 * G::kGroups) {  // rows that are none become 0
      const int rw = x / kChunks, ch = x % kChunks;
      copy16(stage + row_at<D>(rw, ch), static_cast<const __nv_bfloat16 *>(a.q) + (rw < count ? row_q[rw] + ch * 8 : 0), rw < count);
    }
    copies_done();
    sync_softmax();
    // q as hi + lo, times a power of two that brings the row's largest into [2^7, 2^8); a share of the columns to each group
    constexpr int kShare = D / G::kGroups;
    float f;  // on a score, without its page's scale
    {
      uint32_t top = 0;
#pragma unroll 8
      for (int d = 0; d < D; d += 8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(stage + row_at<D>(row, d / 8));
        const uint32_t x[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0xffffu, x[i] >> 16));
      }
      const bool bad = top >= 0x7f80u;
      const int e = top > 0 && !bad ? min(7 - ((int)(top >> 7) - 127), 120) : 0;
      const float up = (a.scale < 0.f ? -1.f : 1.f) * __uint_as_float((uint32_t)(e + 127) << 23);
      f = bad ? __int_as_float(0x7fc00000) : __uint_as_float((uint32_t)(127 - e) << 23) * (fabsf(a.scale) * kLog2e);
#pragma unroll 2
      for (int d = group * kShare; d < (group + 1) * kShare; d += 32) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = bad ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(stage + row_at<D>(row, d / 8 + i));
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 x = unpack_bf16(u[2 * k]), y = unpack_bf16(u[2 * k + 1]);
            const float v[4] = {x.x * up, x.y * up, y.x * up, y.y * up};
            const uint32_t h0 = float2_to_e4m3(v[0], v[1]), h1 = float2_to_e4m3(v[2], v[3]);
            const float2 b0 = e4m3_to_float2(h0), b1 = e4m3_to_float2(h1);
            hi[2 * i + k] = h0 | h1 << 16;
            lo[2 * i + k] = float2_to_e4m3(v[0] - b0.x, v[1] - b0.y) | float2_to_e4m3(v[2] - b1.x, v[3] - b1.y) << 16;
          }
        }
        if constexpr (G::kQSmem) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = f8_at<D>(row, d / 16 + i);
            *reinterpret_cast<uint4 *>(sq + at) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
            *reinterpret_cast<uint4 *>(sq + kRows * D + at) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
          }
        } else {
          __syncwarp();
          tmem_st8w_nw(lanes + G::kQ + d / 4, hi);
          tmem_st8w_nw(lanes + G::kQ + D / 4 + d / 4, lo);
        }
      }
      if constexpr (G::kQSmem) {
        fence_smem_to_async();
      } else {
        __syncwarp();
        tmem_wait_st();
      }
    }
    fence_before();
    bar_arrive(&bars.q_read);  // V may come
    __syncwarp();
    sync_products();  // with the products' warp: Q is in place
    const int last = !real ? -1 : a.causal ? s.kv - s.n + tok : s.kv - 1;
    const int all_see = a.causal ? s.kv - s.n + first / a.r : s.kv - 1;
    float m = kNone, l = 0.f, mv = kNone;  // what the weights' sum l is relative to, and O: the largest weight times value scale
#pragma unroll 1
    for (int j = group; j < ntiles; j += G::kGroups) {
      const int buf = j % G::kBufs;
      wait(&bars.scales[j % kRing], (j / kRing) & 1);
      const Scales &sc = ring[j % kRing];
      const float4 ks4 = sc.ks, lvs = sc.lvs;
      const uint32_t flags = sc.flags;
      const float fs[kSubs] = {f * ks4.x, f * ks4.y, f * ks4.z, f * ks4.w}, lv[kSubs] = {lvs.x, lvs.y, lvs.z, lvs.w};
      wait(&bars.s_full[buf], (j / G::kBufs) & 1);
      __syncwarp();
      fence_after();
      const uint32_t scores = lanes + G::kS + buf * kTile;
      const int tok0 = (base + j) * kTile;
      // Some row does not see all, or some value scale is NaN: then scores get their scales first, so that a scale
      // (NaN, 0) does not bring back what is not seen, and a NaN value scale reaches what is.
      const bool odd = flags != 0 || tok0 + kTile - 1 > all_see;
      auto one_by_one = [&](uint32_t (&x)[32], int h) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int u = 2 * h + i / 16;
          const float y = flags >> (8 * u + 1) & 1 ? __int_as_float(0x7fc00000) : __uint_as_float(x[i]) * fs[u];
          x[i] = __float_as_uint(tok0 + 32 * h + i <= last && !(flags >> (8 * u) & 1) ? y : -INFINITY);
        }
      };
      float top = -INFINITY, topv = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[32];
        tmem_ld32_nw(scores + 32 * h, x);
        tmem_wait_ld();
        if (odd) one_by_one(x, h);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t *const y = x + 16 * v;
          float t0 = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1])), t1 = fmaxf(__uint_as_float(y[2]), __uint_as_float(y[3]));
#pragma unroll
          for (int i = 4; i < 16; i += 4) {
            t0 = fmaxf(fmaxf(t0, __uint_as_float(y[i])), __uint_as_float(y[i + 1]));
            t1 = fmaxf(fmaxf(t1, __uint_as_float(y[i + 2])), __uint_as_float(y[i + 3]));
          }
          const float t = odd ? fmaxf(t0, t1) : fmaxf(t0, t1) * fs[2 * h + v];
          top = fmaxf(top, t);
          topv = fmaxf(topv, t + lv[2 * h + v]);
        }
        __syncwarp();
      }
      float mc = m;
      if constexpr (G::kGroups > 1) {
        if (j > 0) {  // the other group's word on the tile before
          wait(&bars.moved[group ^ 1][quarter], ((j - 1) / G::kGroups) & 1);
          const float2 x = moved[group ^ 1][row];
          mc = x.x;
          mv = x.y;
        }
      }
      if (__any_sync(0xffffffffu, top > mc + kSlack || topv > mv + kSlack)) {
        const float mvn = fmaxf(mv, topv), shrink = ex2(mv - mvn);
        mc = fmaxf(mc, top);
        mv = mvn;
        if (j > 0) {
          wait(&bars.v_empty[(j - 1) % G::kVStages], ((j - 1) / G::kVStages) & 1);  // the products so far are in O
          __syncwarp();
          fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t w[32];
            tmem_ld32_nw(lanes + G::kO + d, w);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * shrink);
            tmem_st32w_nw(lanes + G::kO + d, w);
          }
        }
      }
      if constexpr (G::kGroups > 1) {
        moved[group][row] = make_float2(mc, mv);
        bar_arrive(&bars.moved[group][quarter]);
      }
      l *= ex2(m - mc);
      m = mc;
      // the value scales, over what brings the largest product to 1, in the exponent: at least so much that weights which
      // count in the sum do not vanish (as products they do, in fp16)
      const float up2 = kPExp - m, ratio = mv - m;
      const float lr[kSubs] = {fmaxf(lv[0] - ratio, kMinRatio), fmaxf(lv[1] - ratio, kMinRatio), fmaxf(lv[2] - ratio, kMinRatio),
                               fmaxf(lv[3] - ratio, kMinRatio)};
      // the scores once more, half a tile at a time: fewer registers, and more of them for what runs side by side
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[32], p[16];
        __syncwarp();
        tmem_ld32_nw(scores + 32 * h, x);
        tmem_wait_ld();
        if (odd) one_by_one(x, h);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int u = 2 * h + v;
          const float shift = lr[u] + up2, fu = odd ? 1.f : fs[u];
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float2 e = fma2(make_float2(__uint_as_float(x[16 * v + i]), __uint_as_float(x[16 * v + i + 1])), make_float2(fu, fu),
                            make_float2(shift, shift));
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum = add2(sum, e);
            p[8 * v + i / 2] = pack2(e.x, e.y);
          }
          l = fmaf(sum.x + sum.y, ex2(-lr[u] - kPExp), l);
        }
        __syncwarp();
        tmem_st16w_nw(scores + 16 * h, p);  // in the place of scores that have been read
      }
      tmem_wait_st();
      fence_before();
      bar_arrive(&bars.p_full[buf]);
    }
    // ---- out: the groups' sums together, a share of the columns to each
    if constexpr (G::kGroups > 1) {
      if (ntiles > 0) {
        const int g_last = (ntiles - 1) % G::kGroups;
        wait(&bars.moved[g_last][quarter], ((ntiles - 1) / G::kGroups) & 1);
        const float2 x = moved[g_last][row];
        l *= ex2(m - x.x);
        m = x.x;
        mv = x.y;
      }
      other[group][row] = l;
      sync_softmax();
      l += other[group ^ 1][row];
    }
    if (ntiles > 0) wait(&bars.v_empty[(ntiles - 1) % G::kVStages], ((ntiles - 1) / G::kVStages) & 1);
    __syncwarp();
    fence_after();
    if (split > 1) {  // a part: fp32, relative to m
      const long long at = part_row(part_no) + row;
      if (group == 0) reinterpret_cast<float2 *>(part_ml(a, (int)gridDim.x - a.whole, D))[at] = make_float2(ntiles > 0 ? m : -INFINITY, l);
      const float un = ex2(-kPExp), scale = ex2(mv - m);
      constexpr int kRounds = 2, kCols = kShare / kRounds;  // of a group in a round
#pragma unroll 1
      for (int h = 0; ntiles > 0 && h < kRounds; ++h) {
#pragma unroll 1
        for (int d = 0; d < kCols; d += 32) {
          uint32_t w[32];
          __syncwarp();
          tmem_ld32_nw(lanes + G::kO + group * kShare + h * kCols + d, w);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4 *>(stage + row_at<D>(row, (group * kCols + d + i) / 4)) =
                make_float4(__uint_as_float(w[i]) * un * scale, __uint_as_float(w[i + 1]) * un * scale,
                            __uint_as_float(w[i + 2]) * un * scale, __uint_as_float(w[i + 3]) * un * scale);
        }
        sync_softmax();
        float *const dst = static_cast<float *>(a.ws) + (at - row) * D + h * kCols;
#pragma unroll 4
        for (int x = tid; x < count * (D / 8); x += 128 * G::kGroups) {
          const int rw = x / (D / 8), ch = x % (D / 8), g = ch / (kCols / 4), col = ch % (kCols / 4) * 4;
          *reinterpret_cast<float4 *>(dst + (long long)rw * D + g * kShare + col) =
              *reinterpret_cast<const float4 *>(stage + row_at<D>(rw, ch));
        }
        sync_softmax();
      }
    } else {
      const float inv = l == 0.f ? 0.f : ex2(-kPExp) / l, scale = ex2(mv - m);  // the smallest scales first would be lost
#pragma unroll 1
      for (int d = group * kShare; d < (group + 1) * kShare; d += 32) {
        uint32_t w[32];
        __syncwarp();
        tmem_ld32_nw(lanes + G::kO + d, w);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = ntiles > 0 ? pack_bf16(__uint_as_float(w[i + 2 * k]) * inv * scale, __uint_as_float(w[i + 2 * k + 1]) * inv * scale) : 0u;
          *reinterpret_cast<uint4 *>(stage + row_at<D>(row, (d + i) / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      sync_softmax();
#pragma unroll 8
      for (int x = tid; x < count * kChunks; x += 128 * G::kGroups) {
        const int rw = x / kChunks, ch = x % kChunks;
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + row_o[rw] + ch * 8) =
            *reinterpret_cast<const uint4 *>(stage + row_at<D>(rw, ch));
      }
    }
    fence_before();
  } else if (warp < G::kKeyWarp) {
    // ----------------------------------------------------------------- values
    // 16 tokens to a warp: lane / 4 (and 8 more), 16 dimensions at lane % 4 of every 64.
    const int w = warp - G::kValueWarp, t8 = lane >> 2, d16 = lane & 3;
    constexpr int kLoads = 2 * (D / 64);
    uint4 x[2][kLoads];  // of the next two tiles
    auto load = [&](int j, int p, uint4 (&r)[kLoads]) {
      const int tok = (base + j) * kTile + 16 * w;
      const uint8_t *const src = c.v + (((long long)max(p, 0) * c.Hk + hk) * page + (tok & (page - 1)) + t8) * D + d16 * 16;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        r[i] = make_uint4(0, 0, 0, 0);
        if (p >= 0 && tok + t8 + 8 * (i & 1) < s.kv) r[i] = *reinterpret_cast<const uint4 *>(src + 8 * (i & 1) * D + (i >> 1) * 64);
      }
    };
    // where a lane's 16 dimensions go, as an operand with the dimensions contiguous; what follows is a fixed way on
    uint8_t *const put_lo = sv + mnmaj(d16 * 16, 16 * w + t8, kTile), *const put_hi = sv + mnmaj(d16 * 16 + 8, 16 * w + t8, kTile);
    auto put = [&](int j, const uint4 (&r)[kLoads]) {
      const int slot = j % G::kVStages;
      if (j >= G::kVStages) wait(&bars.v_empty[slot], (j / G::kVStages - 1) & 1);
      uint8_t *const lo = put_lo + slot * G::kVBytes, *const hi = put_hi + slot * G::kVBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t u[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[2 * e] = e4m3x2_to_h2(u[e], 0);
          h[2 * e + 1] = e4m3x2_to_h2(u[e], 1);
        }
        constexpr int kBlock = kTile * 128;  // 64 dimensions of a tile
        *reinterpret_cast<uint4 *>(lo + (i >> 1) * kBlock + (i & 1) * 1024) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(hi + (i >> 1) * kBlock + (i & 1) * 1024) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      fence_smem_to_async();
      bar_arrive(&bars.v_full[slot]);
    };
    // A tile's loads are asked for two tiles ahead, behind the fence, which would wait for them; the pages and scales of
    // 32 tiles at a time, one per lane, 32 ahead.  The scales go to the softmax warps two tiles ahead as well: the place
    // of tile j + 2 in the ring was tile j - 6's, which they have done when the products of tile j - 3 are.
    auto scales = [&](int p) {
      if (p < 0) return make_float2(0.f, 0.f);
      const long long at = (long long)p * c.Hk + hk;
      return make_float2(c.ks[at], c.vs[at]);
    };
    int pg = pages.page(pages.ask(lane, w)), pg_next = -1, entry = pages.ask(32 + lane, w);
    float2 sc = scales(pg), sc_next = make_float2(0.f, 0.f);
    auto prepare = [&](int j, uint4 (&r)[kLoads]) {  // of the batch of 32 at hand
      const int p = __shfl_sync(0xffffffffu, pg, j & 31);
      const float ks = __shfl_sync(0xffffffffu, sc.x, j & 31), vs = __shfl_sync(0xffffffffu, sc.y, j & 31);
      load(j, p, r);
      if (lane == 0 && j < ntiles) {
        Scales &out = ring[j % kRing];
        reinterpret_cast<float *>(&out.ks)[w] = ks;
        reinterpret_cast<float *>(&out.lvs)[w] = fmaxf(__log2f(vs), kNoScale);  // fmaxf: of 0, and of a NaN, which the flag tells of
        reinterpret_cast<uint8_t *>(&out.flags)[w] = (p < 0 ? 1 : 0) | (vs != vs ? 2 : 0);
        bar_arrive(&bars.scales[j % kRing]);
      }
      __syncwarp();
    };
    prepare(0, x[0]);
    prepare(1, x[1]);
    wait(&bars.q_read, 0);
#pragma unroll 1
    for (int j = 0; j < ntiles; j += 2) {
      if ((j & 31) == 16) {
        pg_next = pages.page(entry);
        sc_next = scales(pg_next);
      }
      if ((j & 31) == 30) {  // what follows is of the next batch
        pg = pg_next;
        sc = sc_next;
        entry = pages.ask(j + 34 + lane, w);
      }
      put(j, x[0]);
      prepare(j + 2, x[0]);
      if (j + 1 < ntiles) put(j + 1, x[1]);
      prepare(j + 3, x[1]);
    }
  } else if (warp == G::kKeyWarp) {
    // ------------------------------------------------------------------- keys
    // Lane 4 i + u has page u of tile i of a batch of 8; those of the next are asked for when one begins.
    int pg = pages.page(pages.ask(lane >> 2, lane & 3)), entry = pages.ask(8 + (lane >> 2), lane & 3);
#pragma unroll 1
    for (int j = 0; j < ntiles; ++j) {
      const int i = j & 7, slot = j % G::kKStages;
      if (i == 0 && j > 0) {
        pg = pages.page(entry);
        entry = pages.ask(j + 8 + (lane >> 2), lane & 3);
      }
      const int p = __shfl_sync(0xffffffffu, pg, 4 * i + (lane & 3));
      const uint32_t there = __ballot_sync(0xffffffffu, p >= 0) & ((1u << kSubs) - 1);
      if (j >= G::kKStages) wait(&bars.k_empty[slot], (j / G::kKStages - 1) & 1);
      __syncwarp();
      if (lane == 0) bar_expect_tx(&bars.k_full[slot], __popc(there) * 16 * D);
      __syncwarp();
      if (lane < kSubs && p >= 0 && !gave_up) {
        const uint32_t dst = smem_u32(sk + slot * G::kKBytes) + lane * 16 * G::kRowBytes;
        const int tok = ((base + j) * kTile + lane * 16) & (page - 1);
#pragma unroll
        for (int b = 0; b < (D + 127) / 128; ++b)
          tma_load_3d(dst + b * kTile * 128, &kmap, b * 128, hk * page + tok, p, &bars.k_full[slot]);
      }
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------------- products
    constexpr uint32_t id_s = idesc(kRows, kTile, 0, 0), id_o = idesc(kRows, D, 0, 1);
    // Descriptors' halves: address and leading stride, group stride, version and swizzle (keys of 64 bytes a row: the
    // swizzle of that width, 8 rows in 512 bytes).
    constexpr uint32_t k_hi = D >= 128 ? 1024 >> 4 | 1 << 14 | 2u << 29 : 512 >> 4 | 1 << 14 | 4u << 29;
    constexpr uint32_t v_hi = 1024 >> 4 | 1 << 14 | 2u << 29;
    const uint32_t q_lo = smem_u32(sq) >> 4 | 1 << 16, k_lo = smem_u32(sk) >> 4 | 1 << 16, v_lo = smem_u32(sv) >> 4 | (uint32_t)(kTile / 8 * 1024 >> 4) << 16;
    __syncwarp();
    sync_products();
    fence_after();
    auto scores = [&](int j) {
      const int slot = j % G::kKStages;
      wait(&bars.k_full[slot], (j / G::kKStages) & 1);
      __syncwarp();
      fence_after();
      if (elect()) {
        const uint32_t lo = k_lo + slot * (G::kKBytes >> 4), d = tmem + G::kS + (j % G::kBufs) * kTile;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < D / 32; ++ks) {
            const uint32_t at = lo + (((ks >> 2) * (kTile * 128) + (ks & 3) * 32) >> 4);
            if constexpr (G::kQSmem) {
              const uint32_t q = q_lo + ((part * kRows * D + ks * 32) >> 4);
              if (part + ks == 0)
                mma_f8_ss<false>(d, q, at, k_hi, id_s);
              else
                mma_f8_ss<true>(d, q, at, k_hi, id_s);
            } else {
              const uint32_t q = tmem + G::kQ + part * (D / 4) + ks * 8;
              if (part + ks == 0)
                mma_ta<true, false>(d, q, at, k_hi, id_s);
              else
                mma_ta<true, true>(d, q, at, k_hi, id_s);
            }
          }
        commit(&bars.s_full[j % G::kBufs]);
        commit(&bars.k_empty[slot]);
      }
      __syncwarp();
    };
#pragma unroll 1
    for (int j = 0; j < min(ntiles, G::kBufs); ++j) scores(j);
#pragma unroll 1
    for (int j = 0; j < ntiles; ++j) {
      const int slot = j % G::kVStages;
      wait(&bars.v_full[slot], (j / G::kVStages) & 1);
      wait(&bars.p_full[j % G::kBufs], (j / G::kBufs) & 1);
      __syncwarp();
      fence_after();
      if (elect()) {
        const uint32_t lo = v_lo + slot * (G::kVBytes >> 4), p = tmem + G::kS + (j % G::kBufs) * kTile;
        if (j == 0)
          mma_ta<false, false>(tmem + G::kO, p, lo, v_hi, id_o);
        else
          mma_ta<false, true>(tmem + G::kO, p, lo, v_hi, id_o);
#pragma unroll
        for (int ks = 1; ks < kTile / 16; ++ks) mma_ta<false, true>(tmem + G::kO, p + ks * 8, lo + ks * (2048 >> 4), v_hi, id_o);
        commit(&bars.v_empty[slot]);
      }
      __syncwarp();
      if (j + G::kBufs < ntiles) scores(j + G::kBufs);  // where P was: products follow each other
    }
  }
  if (gave_up) settle();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == G::kProductWarp) tmem_dealloc(tmem, G::kCols);
}

// Joins the parts of an item's rows: o = sum 2^(m_p - m) o_p / sum 2^(m_p - m) l_p.  A thread has 4 columns of a row.
constexpr int kJoinRows = 16;
template <int D>
__global__ void __launch_bounds__(256) attn_tile_join(const AttnArgs a) {
  const int parts = a.splits;
  int local = 0, hk = 0;
  const Seq s = find_block(a, a.whole + blockIdx.x, &hk, &local);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written (no block ends before that)
  if (s.b < 0) return;
  const int row0 = blockIdx.y * kJoinRows, first = local * kRows + row0;
  const int count = (int)min((long long)kJoinRows, (long long)s.n * a.r - first);
  const float *const o = static_cast<const float *>(a.ws);
  const float2 *const ml = reinterpret_cast<const float2 *>(part_ml(a, (long long)gridDim.x * parts, D));
  const long long base = part_row((long long)blockIdx.x * parts) + row0;
  for (int x = threadIdx.x; x < count * (D / 4); x += 256) {
    const int row = x / (D / 4), d = x % (D / 4) * 4, rr = first + row, tok = rr / a.r;
    float m = kNone, l = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < parts; p += 8) {  // 8 parts' loads in flight
      float2 z[8];
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        z[u] = make_float2(-INFINITY, 0.f);
        if (p + u < parts) {
          z[u] = ml[base + (p + u) * kRows + row];
          v[u] = *reinterpret_cast<const float4 *>(o + (base + (p + u) * kRows + row) * D + d);
        }
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < 8; ++u) mn = fmaxf(mn, z[u].x);
      const float old = ex2(m - mn);
      m = mn;
      l *= old;
      sum.x *= old, sum.y *= old, sum.z *= old, sum.w *= old;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (z[u].x != -INFINITY) {  // else a part without tokens, which left no values
          const float w = ex2(z[u].x - m);
          l += w * z[u].y;
          sum.x += w * v[u].x, sum.y += w * v[u].y, sum.z += w * v[u].z, sum.w += w * v[u].w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(a.o) + (s.row0 + (long long)tok) * a.ldo +
                               (long long)(hk * a.r + rr - tok * a.r) * D + d;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
  }
}

template <int D>
struct TileTag {};

template <int D>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
  using G = Geo<D>;
  cudaError_t e = allow_smem<TileTag<D>>(attn_tile_kernel<D>, G::kSmem);
  if (e != cudaSuccess) return e;
  const EncodeTiled encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const CacheArgs &c = a.cache;
  CUtensorMap map;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)c.Hk << c.page_shift, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)D, ((cuuint64_t)c.Hk << c.page_shift) * D};
  const cuuint32_t box[3] = {(cuuint32_t)G::kRowBytes, 16, 1}, steps[3] = {1, 1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.k, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int cut = a.blocks - a.whole;
  attn_tile_kernel<D><<<a.whole + cut * a.splits, G::kThreads, G::kSmem, s>>>(a, map);
  e = cudaGetLastError();
  if (e != cudaSuccess || cut == 0) return e;
  // The join comes up while the last blocks end, and waits for them.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cut, kRows / kJoinRows);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_tile_join<D>, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

// Tiles of a call and key heads, at most (packed: of any lengths).
static long long tile_blocks(const SeqArgs &q, int r, int Hk) {
  const long long each = ((long long)q.T * r + kRows - 1) / kRows;
  return (q.B > 32 * kSeqsLane ? item_count(q, r, kRows, 1) : !q.cu || q.B == 1 ? each * q.B : (long long)q.T * r / kRows + q.B) * Hk;
}
// Parts at most: of the blocks that are left for the last time where blocks fill the GPU, of all where they do not.  None
// has less than 8 tiles.
static int slots_of(int D, int num_sms) { return num_sms * (D == 256 ? Geo<256>::kBlocks : Geo<128>::kBlocks); }
static int most_parts_last(long long blocks, int tiles, int slots) {
  const int left = (int)(blocks % slots);
  return blocks > slots && left ? std::min({slots / left, tiles / 8, 32}) : 1;
}
static int most_parts_all(long long blocks, int max_kv, int num_sms) {
  return (int)std::max(1LL, std::min({32LL, (long long)max_kv / (8 * kTile), (num_sms + blocks - 1) / blocks + 1}));
}
// Where blocks do not fill the GPU all are cut: a block takes a tile's time per tile and about that of kEnds to start
// and end, one block to an SM at a time; a part's values cost kPart more, a join kJoin: the number of parts with
// the least time.  Where they fill it some times over, and all have about the same length (one sequence, or fixed
// lengths; others' blocks get shorter to the end), those that are left for the last time are cut into as many parts
// as fill it once more, if the time saved is more than those cost (8192 tokens over 24576, 10.1 times: 3.65 to
// 3.49 ms; 1.03 times, 2048 tokens, heads of 256: 62 to 53 us).
TileCut attn_tile_cut(const SeqArgs &q, int r, int Hk, int D, int max_kv, int num_sms) {
  constexpr int kEnds = 10, kPart = 8, kJoin = 6;
  const long long blocks = tile_blocks(q, r, Hk);
  const int tiles = (int)(((long long)max_kv + kTile - 1) / kTile), slots = slots_of(D, num_sms);
  TileCut c{(int)blocks, (int)blocks, 1};
  if (blocks >= num_sms) {
    const int parts = most_parts_last(blocks, tiles, slots);
    const bool even = !q.cu || q.B == 1;
    if (even && parts > 1 && tiles + kEnds > (tiles + parts - 1) / parts + kEnds + kPart + kJoin + parts / 4) {
      c.whole = (int)(blocks - blocks % slots);
      c.parts = parts;
    }
    return c;
  }
  const int up_to = most_parts_all(blocks, max_kv, num_sms);
  long long least = 0;
  for (int p = 1; p <= up_to; ++p) {
    const long long time =
        (blocks * p + num_sms - 1) / num_sms * ((tiles + p - 1) / p + kEnds + (p > 1 ? kPart : 0)) + (p > 1 ? kJoin + p / 4 : 0);
    if (p == 1 || time < least) {
      least = time;
      c.parts = p;
    }
  }
  if (c.parts > 1) c.whole = 0;
  return c;
}

size_t attn_tile_ws_bytes(const TileCut &c, int D) {
  return (size_t)(c.blocks - c.whole) * c.parts * kRows * (D + 2) * sizeof(float);
}

// Of so many blocks or fewer; from twice the slots on what is left for the last time comes round again.
size_t attn_tile_room(const SeqArgs &q, int r, int Hk, int D, int max_kv, int num_sms) {
  const int tiles = (int)(((long long)max_kv + kTile - 1) / kTile), slots = slots_of(D, num_sms);
  const long long blocks = std::min(tile_blocks(q, r, Hk), 2LL * slots);
  size_t most = 0;
  for (long long b = 1; b <= blocks; ++b) {
    const int parts = b < num_sms ? most_parts_all(b, max_kv, num_sms) : most_parts_last(b, tiles, slots);
    const long long cut = b < num_sms ? b : b % slots;
    if (parts > 1) most = std::max(most, attn_tile_ws_bytes(TileCut{(int)cut, 0, parts}, D));
  }
  return most;
}

cudaError_t launch_attn_tile(const AttnArgs &a, cudaStream_t s) {
  return a.cache.D == 64 ? launch<64>(a, s) : a.cache.D == 128 ? launch<128>(a, s) : launch<256>(a, s);
}

}  // namespace gdn
