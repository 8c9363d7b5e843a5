// attn_tile.cu -- attention of many rows over the paged 8-bit cache (bf16 io): prompts.
//
// A CTA takes 128 rows (query tokens x the query heads of one key head) and goes
// over the tokens in tiles of 64 on the tensor cores, one pass with the running
// maximum and sum of each row:
//   S = Q K^T   e4m3 products straight on the cache's bytes, which TMA brings from
//               the pages.  Q stands in TMEM as two e4m3 values per element, hi +
//               lo of q times a power of two per row (8 bits of a bf16 where it is
//               within 2^10 of its row's largest; 2^-19 of that largest at worst).
//   O += P V    fp16 products: P, rounded to fp16, in TMEM where S was; V's bytes
//               become fp16 (exact) on the way through a group of four warps.
// A page's key scale multiplies its scores.  Its value scale, over the largest
// so far, enters p as a term of the exponent, and leaves the row's sum again as a
// factor on the page's part of it: no product per element.
//
// Warps: 0-3 and 4-7 softmax (thread = row; even and odd tiles), 8-11 values, 12
// keys (TMA), 13 products.  For a tile of 64 tokens and D = 256 the products take
// 1024 cycles; a tile's way through one group of softmax warps is longer than
// that, so that two take turns.  The running maximum goes from one to the other
// as soon as it is known, ahead of the exponentials; each keeps a sum of its own.
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
constexpr int kThreads = 448;
constexpr int kValueWarp = 8, kKeyWarp = 12, kProductWarp = 13;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -1.7e38f;
constexpr float kSlack = 4.f;   // p may reach 2^kSlack before the running maximum moves
constexpr float kPExp = 11.f;   // p stands times 2^11 in fp16
constexpr float kMinRatio = -60.f;
constexpr float kNoRef = -200.f;  // the logarithm of the value scales where there is none above 0

template <int D>
struct Geo {
  static constexpr int kKStages = 4, kVStages = 2;
  static constexpr int kKBytes = kTile * D, kVBytes = kTile * D * 2;
  static constexpr int kSmem = kKStages * kKBytes + kVStages * kVBytes + 1024;
  // TMEM columns
  static constexpr int kQ = 0, kO = D / 2, kS = kO + D;
  static constexpr int kCols = kS + 2 * kTile <= 256 ? 256 : 512;
  // K-major rows of 128 bytes (D = 64: 64) with the swizzle of that width
  static constexpr int kRowBytes = D >= 128 ? 128 : 64;
};

// tcgen05.mma of e4m3 operands, A in TMEM (4 bytes along K to a column: a K step of 32 advances 8), by lane 0 of a converged warp.
__device__ __forceinline__ void mma_f8_ta_w(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .u32 l;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(id), "r"(accumulate));
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w, int high) {
  uint32_t o;
  if (high)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(o) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(o) : "r"(w));
  return o;
}

struct Bars {
  uint64_t k_full[4], k_empty[4], v_full[2], v_empty[2], s_full[2], p_full[2];
  uint64_t moved[2][4];  // the running maximum after a tile, per warp
};

// Entries of the table for the 16 tokens `sub` of a tile.  ask() loads one (kUnseen: its tokens are not looked
// at); a tile or two later page() says what it is worth, so that nothing waits for the load.
constexpr int kUnseen = -0x40000000;
struct TilePages {
  const CacheArgs &c;
  const int *table;
  int seen;
  unsigned int *err;
  __device__ __forceinline__ int ask(int tile, int sub) const {
    const int tok = tile * kTile + sub * 16;
    return tok < seen ? table[tok >> c.page_shift] : kUnseen;
  }
  __device__ __forceinline__ int page(int entry) const {
    if ((unsigned)entry < (unsigned)c.n_pages) return entry;
    if (entry != kUnseen) atomicOr(err, kErrSeqlens);
    return -1;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tile_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap) {
  using G = Geo<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int gave_up;
  __shared__ float2 moved[2][kRows];  // running maximum and largest value scale after a tile, even and odd
  __shared__ float2 other[2][kRows];  // maximum and sum of each group at the end
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const CacheArgs &c = a.cache;
  int local = 0;
  const long long item = (long long)gridDim.x - 1 - blockIdx.x;  // the later rows of a prompt, which see more, first
  const Seq s = find_seq(a.seq, item, a.r, kRows, 1, &local);
  if (s.b < 0) return;
  const int first = local * kRows, count = (int)min((long long)kRows, (long long)s.n * a.r - first);
  if (count <= 0) return;
  const int hk = blockIdx.y;
  const int seen = a.causal ? min(s.kv, max(0, s.kv - s.n + (first + count - 1) / a.r + 1)) : s.kv;
  const int ntiles = (seen + kTile - 1) / kTile;

  uint8_t *const smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *const sk = smem, *const sv = smem + G::kKStages * G::kKBytes;
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      bar_init(&bars.k_full[i], 1);
      bar_init(&bars.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&bars.v_full[i], 128);
      bar_init(&bars.v_empty[i], 1);
      bar_init(&bars.s_full[i], 1);
      bar_init(&bars.p_full[i], 128);
      for (int w = 0; w < 4; ++w) bar_init(&bars.moved[i][w], 32);
    }
    gave_up = 0;
  }
  if (warp == kProductWarp) tmem_alloc(&tmem_slot, G::kCols);
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
  const TilePages pages{c, c.table + (long long)s.b * c.table_ld, seen, a.seq.err};
  const int page = 1 << c.page_shift;

  if (warp < kValueWarp) {
    // ---------------------------------------------------------------- softmax
    const int group = warp >> 2, quarter = warp & 3, row = tid & (kRows - 1), rr = first + row, tok = rr / a.r;
    const bool real = row < count;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    // q as hi + lo, times a power of two that brings the row's largest into [2^7, 2^8); half the columns to a group
    const __nv_bfloat16 *const src = static_cast<const __nv_bfloat16 *>(a.q) + (s.row0 + (long long)tok) * a.ldq +
                                     (long long)(hk * a.r + rr - tok * a.r) * D;
    float f;  // on a score, without its page's scale
    {
      uint32_t top = 0;
#pragma unroll 8
      for (int d = 0; d < D; d += 8) {
        const uint4 w = real ? *reinterpret_cast<const uint4 *>(src + d) : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0xffffu, x[i] >> 16));
      }
      const bool bad = top >= 0x7f80u;
      const int e = top > 0 && !bad ? min(7 - ((int)(top >> 7) - 127), 120) : 0;
      const float up = (a.scale < 0.f ? -1.f : 1.f) * __uint_as_float((uint32_t)(e + 127) << 23);
      f = bad ? __int_as_float(0x7fc00000) : __uint_as_float((uint32_t)(127 - e) << 23) * (fabsf(a.scale) * kLog2e);
#pragma unroll 1
      for (int d = group * (D / 2); d < (group + 1) * (D / 2); d += 32) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = real && !bad ? *reinterpret_cast<const uint4 *>(src + d + 8 * i) : make_uint4(0, 0, 0, 0);
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
        __syncwarp();
        tmem_st8w_nw(lanes + G::kQ + d / 4, hi);
        tmem_st8w_nw(lanes + G::kQ + D / 4 + d / 4, lo);
      }
      tmem_wait_st();
    }
    fence_before();
    __syncwarp();
    asm volatile("bar.sync 1, 288;" ::: "memory");  // with the products' warp: Q is in place
    const int last = !real ? -1 : a.causal ? s.kv - s.n + tok : s.kv - 1;
    const int all_see = a.causal ? s.kv - s.n + first / a.r : s.kv - 1;
    float m = kNone, l = 0.f, lref = kNoRef;  // m: what l is relative to; the largest value scale's logarithm
    // Lane u of four has page u of a tile: its key scale, and its value scale's logarithm.
    auto scales = [&](int p) {
      if (p < 0) return make_float2(0.f, 0.f);
      const long long at = (long long)p * c.Hk + hk;
      return make_float2(c.ks[at], c.vs[at]);
    };
    int pg = pages.page(pages.ask(group, lane & 3)), entry = pages.ask(group + 2, lane & 3);
    float2 sc = scales(pg);
#pragma unroll 1
    for (int j = group; j < ntiles; j += 2) {
      const float ks = sc.x, lvs = fmaxf(__log2f(sc.y), kNoRef);  // fmaxf: of 0, and of a NaN, which `odd` looks after
      const uint32_t gone = __ballot_sync(0xffffffffu, pg < 0) & ((1u << kSubs) - 1);
      const uint32_t no_v = __ballot_sync(0xffffffffu, sc.y != sc.y) & ((1u << kSubs) - 1);
      pg = pages.page(entry);
      entry = pages.ask(j + 4, lane & 3);
      sc = scales(pg);
      float fs[kSubs], ltop = lvs;
#pragma unroll
      for (int u = 0; u < kSubs; ++u) fs[u] = f * __shfl_sync(0xffffffffu, ks, u);
      ltop = fmaxf(ltop, __shfl_xor_sync(0xffffffffu, ltop, 1));
      ltop = fmaxf(ltop, __shfl_xor_sync(0xffffffffu, ltop, 2));
      wait(&bars.s_full[group], (j >> 1) & 1);
      __syncwarp();
      fence_after();
      uint32_t x0[32], x1[32];
      tmem_ld32_nw(lanes + G::kS + group * kTile, x0);
      tmem_ld32_nw(lanes + G::kS + group * kTile + 32, x1);
      tmem_wait_ld();
      float y[kTile];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        y[i] = __uint_as_float(x0[i]);
        y[32 + i] = __uint_as_float(x1[i]);
      }
      const int tok0 = j * kTile;
      if ((gone | no_v) != 0 || tok0 + kTile - 1 > all_see) {
        // Some row does not see all, or some value scale is NaN: here the scores get their scales, so that a scale
        // (NaN, 0) does not bring back what is not seen, and a NaN value scale reaches what is.
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
          const float x = (no_v >> (i / 16)) & 1 ? __int_as_float(0x7fc00000) : y[i] * fs[i / 16];
          y[i] = tok0 + i <= last && !(gone >> (i / 16) & 1) ? x : -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < kSubs; ++u) fs[u] = 1.f;
      }
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < kSubs; ++u) {
        float t0 = fmaxf(y[16 * u], y[16 * u + 1]), t1 = fmaxf(y[16 * u + 2], y[16 * u + 3]);
#pragma unroll
        for (int i = 4; i < 16; i += 4) {
          t0 = fmaxf(fmaxf(t0, y[16 * u + i]), y[16 * u + i + 1]);
          t1 = fmaxf(fmaxf(t1, y[16 * u + i + 2]), y[16 * u + i + 3]);
        }
        top = fmaxf(top, fmaxf(t0, t1) * fs[u]);
      }
      // the other group's word on the tile before
      float mc = kNone;
      if (j > 0) {
        wait(&bars.moved[group ^ 1][quarter], ((j - 1) >> 1) & 1);
        const float2 x = moved[group ^ 1][row];
        mc = x.x;
        lref = x.y;
      }
      if (__any_sync(0xffffffffu, top > mc + kSlack || ltop > lref)) {
        const float mn = fmaxf(mc, top), ln = fmaxf(lref, ltop), shrink = ex2(mc - mn + (lref - ln));
        mc = mn;
        lref = ln;
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
      moved[group][row] = make_float2(mc, lref);
      bar_arrive(&bars.moved[group][quarter]);
      l *= ex2(m - mc);
      m = mc;
      // the value scale over the largest, in the exponent
      const float lr = fmaxf(lvs - lref, kMinRatio), back = ex2(-lr - kPExp), base = kPExp - m;
      uint32_t p[kTile / 2];
#pragma unroll
      for (int u = 0; u < kSubs; ++u) {
        const float shift = __shfl_sync(0xffffffffu, lr, u) + base, undo = __shfl_sync(0xffffffffu, back, u);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float2 e = fma2(make_float2(y[16 * u + i], y[16 * u + i + 1]), make_float2(fs[u], fs[u]), make_float2(shift, shift));
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          sum = add2(sum, e);
          p[8 * u + i / 2] = pack2(e.x, e.y);
        }
        l = fmaf(sum.x + sum.y, undo, l);
      }
      __syncwarp();
      tmem_st32w_nw(lanes + G::kS + group * kTile, p);
      tmem_wait_st();
      fence_before();
      bar_arrive(&bars.p_full[group]);
    }
    // ---- out: the groups' sums together, half the columns to each
    if (ntiles > 0) {
      const int g_last = (ntiles - 1) & 1;
      wait(&bars.moved[g_last][quarter], ((ntiles - 1) >> 1) & 1);
      const float2 x = moved[g_last][row];
      l *= ex2(m - x.x);
      m = x.x;
      lref = x.y;
    }
    other[group][row] = make_float2(m, l);
    asm volatile("bar.sync 2, 256;" ::: "memory");
    l += other[group ^ 1][row].y;
    if (ntiles > 0) wait(&bars.v_empty[(ntiles - 1) % G::kVStages], ((ntiles - 1) / G::kVStages) & 1);
    __syncwarp();
    fence_after();
    const float inv = l == 0.f ? 0.f : ex2(lref - kPExp) / l;
    __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(a.o) + (s.row0 + (long long)tok) * a.ldo +
                               (long long)(hk * a.r + rr - tok * a.r) * D;
#pragma unroll 1
    for (int d = group * (D / 2); d < (group + 1) * (D / 2); d += 32) {
      uint32_t w[32];
      __syncwarp();
      tmem_ld32_nw(lanes + G::kO + d, w);
      tmem_wait_ld();
      if (real) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = ntiles > 0 ? pack_bf16(__uint_as_float(w[i + 2 * k]) * inv, __uint_as_float(w[i + 2 * k + 1]) * inv) : 0u;
          *reinterpret_cast<uint4 *>(dst + d + i) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    fence_before();
  } else if (warp < kKeyWarp) {
    // ----------------------------------------------------------------- values
    // 16 tokens to a warp: lane / 4 (and 8 more), 16 dimensions at lane % 4 of every 64.
    const int w = warp - kValueWarp, t8 = lane >> 2, d16 = lane & 3;
    constexpr int kLoads = 2 * (D / 64);
    uint4 x[kLoads];
    auto load = [&](int j, int p) {
      const int tok = j * kTile + 16 * w;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int t = t8 + 8 * (i & 1);
        x[i] = make_uint4(0, 0, 0, 0);
        if (p >= 0 && tok + t < s.kv)
          x[i] = *reinterpret_cast<const uint4 *>(c.v + (((long long)p * c.Hk + hk) * page + (tok & (page - 1)) + t) * D + (i >> 1) * 64 + d16 * 16);
      }
    };
    int entry = pages.ask(1, w);
    load(0, pages.page(pages.ask(0, w)));
#pragma unroll 1
    for (int j = 0; j < ntiles; ++j) {
      const int slot = j % G::kVStages;
      if (j >= G::kVStages) wait(&bars.v_empty[slot], (j / G::kVStages - 1) & 1);
      uint8_t *const tile = sv + slot * G::kVBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int k = 16 * w + t8 + 8 * (i & 1), dim = (i >> 1) * 64 + d16 * 16;
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[2 * e] = e4m3x2_to_h2(u[e], 0);
          h[2 * e + 1] = e4m3x2_to_h2(u[e], 1);
        }
        *reinterpret_cast<uint4 *>(tile + mnmaj(dim, k, kTile)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(tile + mnmaj(dim + 8, k, kTile)) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      load(j + 1, pages.page(entry));
      entry = pages.ask(j + 2, w);
      fence_smem_to_async();
      bar_arrive(&bars.v_full[slot]);
    }
  } else if (warp == kKeyWarp) {
    // ------------------------------------------------------------------- keys
    int entry = pages.ask(0, lane & 3), entry_next = pages.ask(1, lane & 3);
#pragma unroll 1
    for (int j = 0; j < ntiles; ++j) {
      const int slot = j % G::kKStages, now = lane < kSubs ? pages.page(entry) : -1;
      entry = entry_next;
      entry_next = pages.ask(j + 2, lane & 3);
      if (j >= G::kKStages) wait(&bars.k_empty[slot], (j / G::kKStages - 1) & 1);
      __syncwarp();
      const uint32_t there = __ballot_sync(0xffffffffu, now >= 0);
      if (lane == 0) bar_expect_tx(&bars.k_full[slot], __popc(there) * 16 * D);
      __syncwarp();
      if (now >= 0) {
        const uint32_t dst = smem_u32(sk + slot * G::kKBytes) + lane * 16 * G::kRowBytes;
        const int tok = (j * kTile + lane * 16) & (page - 1);
#pragma unroll
        for (int b = 0; b < (D + 127) / 128; ++b)
          tma_load_3d(dst + b * kTile * 128, &kmap, b * 128, hk * page + tok, now, &bars.k_full[slot]);
      }
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------------- products
    constexpr uint32_t id_s = idesc(kRows, kTile, 0, 0), id_o = idesc(kRows, D, 0, 1);
    __syncwarp();
    asm volatile("bar.sync 1, 288;" ::: "memory");
    fence_after();
    auto scores = [&](int j) {
      const int slot = j % G::kKStages;
      wait(&bars.k_full[slot], (j / G::kKStages) & 1);
      __syncwarp();
      fence_after();
      const uint32_t kb = smem_u32(sk + slot * G::kKBytes), d = tmem + G::kS + (j & 1) * kTile;
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
          uint64_t b;
          if constexpr (D >= 128)
            b = desc_k(kb, ks, kTile);
          else  // rows of 64 bytes: 64-byte swizzle, 8 rows in 512 bytes
            b = (uint64_t)(((kb + ks * 32) >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(512 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)4 << 61);
          mma_f8_ta_w(d, tmem + G::kQ + part * (D / 4) + ks * 8, b, id_s, part + ks > 0);
        }
      commit_w(&bars.s_full[j & 1]);
      commit_w(&bars.k_empty[slot]);
    };
    if (ntiles > 0) scores(0);
    if (ntiles > 1) scores(1);
#pragma unroll 1
    for (int j = 0; j < ntiles; ++j) {
      const int slot = j % G::kVStages;
      wait(&bars.v_full[slot], (j / G::kVStages) & 1);
      wait(&bars.p_full[j & 1], (j >> 1) & 1);
      __syncwarp();
      fence_after();
      const uint32_t vb = smem_u32(sv + slot * G::kVBytes), p = tmem + G::kS + (j & 1) * kTile;
#pragma unroll
      for (int ks = 0; ks < kTile / 16; ++ks)
        mma_ta_w(tmem + G::kO, p + ks * 8, desc_mn(vb, ks, kTile), id_o, j + ks > 0);
      commit_w(&bars.v_empty[slot]);
      if (j + 2 < ntiles) scores(j + 2);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kProductWarp) tmem_dealloc(tmem, G::kCols);
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
  const dim3 grid((unsigned)item_count(a.seq, a.r, kRows, 1), c.Hk);
  attn_tile_kernel<D><<<grid, kThreads, G::kSmem, s>>>(a, map);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tile(const AttnArgs &a, cudaStream_t s) {
  return a.cache.D == 64 ? launch<64>(a, s) : a.cache.D == 128 ? launch<128>(a, s) : launch<256>(a, s);
}

}  // namespace gdn
