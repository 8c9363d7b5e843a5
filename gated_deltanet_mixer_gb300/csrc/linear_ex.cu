// linear_ex.cu -- projections with their epilogue:
//   p[t, n] = sum_k x[t, k] w[n, k] + bias[n]
//   y[t, n] = act(p[t, n]) + residual[t, n]                     (plain)
//   y[t, n] = act(p[t, n]) p[t, N + n] + residual[t, n]         (gated, w [2N][K])
// bf16 in and out, fp32 accumulation on the tcgen05 tensor cores, everything
// behind the sum in fp32 and rounded once.
//
// Three kernels:
//   lin_pair_kernel   256 x 256 tiles by pairs of CTAs: bound by the tensor pipe,
//                     92 % active (calls of 8192 tokens 5120 -> 16480 in three
//                     ranges: 840 to 870 us by the power there is, 1.6 PFLOP/s;
//                     the tile kernel below: 1.1 times as long).  Persistent,
//                     the epilogue of a tile under the next tile's MMAs.
//   lin_tile_kernel   128 x 64 .. 256 tiles of one CTA, where pairs' tiles are too
//                     few for the SMs (1024 x 2048 x 2048: 12 us).
//   lin_skinny_kernel fewer tiles (few tokens, or few columns): bound by
//                     reading w once.  128 rows of w on the M side, the tokens
//                     on the N side (16 .. 256), and the contraction split over
//                     a cluster of CTAs, which hand each other their partial
//                     sums through distributed shared memory and add them in a
//                     fixed order: no workspace, no second launch, the same
//                     result every time (64 tokens 6144 -> 5120 with a residual:
//                     18.7 us, 3.4 TB/s).
// Figures below are of launches in a graph; calls in a row take 2 us more each.
#include <atomic>
#include <cmath>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>

#include "gdn.h"
#include "gdn_device.cuh"
#include "launch.h"
#include "tma_host.h"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;
using bf16 = __nv_bfloat16;

constexpr int BK = 64;

// Instruction descriptor, kind::f16 with bf16 A and B (format 1), fp32 D.
constexpr uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// x Phi(x), Phi of a negative argument from its tail: 1 + erf(x / sqrt 2) cancels
// there, is 4 % off at -5 and 0 from -6 on.  With a = |x| and t = 1 / (1 + 0.33 a),
//   Phi(-a) = t 2^(poly(t) - a^2 log2(e) / 2):
// poly is a fit of log2(Phi(-a) / t) + a^2 log2(e) / 2 over 0 <= a <= 14, off by
// 2^-21; with the roundings Phi(-a) is good to 2^-19 up to a = 3 and to 2^-16 at 12,
// where a^2 has lost bits.  erfcf would do, but 32 of them side by side are more
// code than the instruction cache takes beside the epilogue's loop, whichever
// activation runs (calls of 4096 x 6552 x 144 with none: 34 us so, 41 with erff, 72
// with erfcf).
__device__ __forceinline__ float gelu(float x) {
  const float a = fabsf(x), t = __fdividef(1.0f, fmaf(0.33f, a, 1.0f));
  float p = -0.27709153f;
  p = fmaf(p, t, 1.2414080f);
  p = fmaf(p, t, -1.9668245f);
  p = fmaf(p, t, 1.1140870f);
  p = fmaf(p, t, -0.28061262f);
  p = fmaf(p, t, 0.66262490f);
  p = fmaf(p, t, 1.4310480f);
  p = fmaf(p, t, -2.9246387f);
  float tail;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(tail) : "f"(fmaf(a * a, -0.72134752f, p)));
  tail *= t;
  return x * (x < 0.f ? tail : 1.0f - tail);
}
// The fast exponential's error grows with its argument (2^-21 near 0, 2^-19 at 20,
// 2^-17 at 80), the fast division's is 2^-22: far below the bf16 rounding of the
// result.  A SiLU or sigmoid below about 1e-36 in size comes out as 0.
__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case GDN_ACT_SILU: return __fdividef(x, 1.0f + __expf(-x));
    case GDN_ACT_GELU: return gelu(x);
    case GDN_ACT_SIGMOID: return __fdividef(1.0f, 1.0f + __expf(-x));
    default: return x;
  }
}

__device__ __forceinline__ void arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// =============================================================================
// lin_tile_kernel
// =============================================================================
constexpr int BM = 128;
constexpr int kEpiWarps = 8;  // two per TMEM quarter, a half of the columns each
constexpr int kTileThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxStages = 8;

// Tiles 256 columns wide carry the most arithmetic per byte; narrower ones give
// small problems more CTAs and shorter epilogues.
template <int BN>
struct Tile {
  static constexpr uint32_t kA = BM * BK * 2, kB = BN * BK * 2, kStage = kA + kB;
  static constexpr int kStages = 192 * 1024 / kStage < kMaxStages ? (int)(192 * 1024 / kStage) : kMaxStages;
  static constexpr uint32_t kBars = kStages * kStage;
  static constexpr uint32_t kRun = kBars + 256;  // per epilogue warp: a 32 x 32 run of the tile, rows 33 apart
  static constexpr uint32_t kSmem = kRun + kEpiWarps * 32 * 33 * 4 + 1024;
  static_assert(kSmem <= 232448, "shared memory per CTA");
};
struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t end;
  uint32_t tmem;
};
static_assert(sizeof(Bars) <= 256, "barriers");

// Tile t of the persistent schedule: bands of 8 m tiles walk across n, so the
// CTAs that run at once share their w tiles in L2.
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int &mt, int &nt) {
  constexpr int G = 8;
  const int band = t / (G * tiles_n), r = t % (G * tiles_n);
  const int rows = min(G, tiles_m - band * G);
  mt = band * G + r % rows;
  nt = r / rows;
}

// bias[at .. at + 31] added to v; columns from `limit` on are left alone.
__device__ __forceinline__ void add_bias(float (&v)[32], const bf16 *bias, long long at, int limit) {
  if (limit >= 32 && ((reinterpret_cast<uintptr_t>(bias + at) & 15u) == 0)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 u = *reinterpret_cast<const uint4 *>(bias + at + 8 * q);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[8 * q + 2 * e] += __uint_as_float(w[e] << 16);
        v[8 * q + 2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 32; ++q)
      if (q < limit) v[q] += __bfloat162float(bias[at + q]);
  }
}

template <int R>
__device__ __forceinline__ void activate_run(float (&v)[R], int act) {
  switch (act) {  // outside the loop
    case GDN_ACT_SILU:
#pragma unroll
      for (int e = 0; e < R; ++e) v[e] = activate(v[e], GDN_ACT_SILU);
      break;
    case GDN_ACT_GELU:
#pragma unroll
      for (int e = 0; e < R; ++e) v[e] = activate(v[e], GDN_ACT_GELU);
      break;
    case GDN_ACT_SIGMOID:
#pragma unroll
      for (int e = 0; e < R; ++e) v[e] = activate(v[e], GDN_ACT_SIGMOID);
      break;
    default: break;
  }
}

__device__ __forceinline__ bool whole_run(const LinOut &out, int col0, int N) {
  return col0 >= out.col_begin && col0 + 32 <= min(out.col_end, N) && out.vec_ok;
}
// The residual of range `out` under columns col0 .. col0 + 31 of rows row0 ..
// row0 + 31: 32 bf16 of this lane's row (whole runs) or of its column.
__device__ __forceinline__ void load_residual(const LinArgs &g, const LinOut &out, long long row0, int lane, int col0,
                                              uint32_t (&x)[16]) {
  const int rows = (int)min(32LL, g.M - row0), col = col0 + lane;
  const bf16 *res = static_cast<const bf16 *>(out.res) - out.col_begin;
  if (whole_run(out, col0, g.N)) {
    const uint4 *src = reinterpret_cast<const uint4 *>(res + (row0 + min(lane, rows - 1)) * out.ldres + col0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 r = src[q];
      x[4 * q] = r.x, x[4 * q + 1] = r.y, x[4 * q + 2] = r.z, x[4 * q + 3] = r.w;
    }
  } else if (col >= out.col_begin && col < min(out.col_end, g.N)) {
    const uint16_t *src = reinterpret_cast<const uint16_t *>(res + row0 * out.ldres + col);
    const long long ld = out.ldres;
    if (rows == 32) {
#pragma unroll
      for (int e = 0; e < 16; ++e, src += 2 * ld) x[e] = (uint32_t)src[0] | (uint32_t)src[ld] << 16;
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e, src += 2 * ld)
        x[e] = (2 * e < rows ? src[0] : 0u) | (2 * e + 1 < rows ? (uint32_t)src[ld] << 16 : 0u);
    }
  }
}
// The first range with a residual under these columns, loaded ahead into x; -1: none.
__device__ __forceinline__ int prefetch_residual(const LinArgs &g, long long row0, int lane, int col0, uint32_t (&x)[16]) {
  if (row0 >= g.M) return -1;
  for (int o = 0; o < g.n_out; ++o) {
    const LinOut out = g.out[o];  // in registers: the parameters are indexed once
    if (!out.res || max(col0, out.col_begin) >= min(min(col0 + 32, out.col_end), g.N)) continue;
    load_residual(g, out, row0, lane, col0, x);
    return o;
  }
  return -1;
}

// Columns col0 .. col0 + 31 of the warp's rows row0 .. row0 + 31, lane = row:
// v = p (bias added), u = the up half (gated), x = the residual of range
// `loaded`.  Whole aligned runs are stored 16 bytes per lane.  Others go through
// shared memory, so that a warp stores 32 neighbouring columns of one row at a
// time: a lane storing its own row would touch 32 rows with every 2-byte store
// (4069 x 6549 x 144 with a residual: ten times as long so; 53 us this way).  What
// bounds these loops is instructions: with the fields of a range read from the
// parameters at each use, and every row tested against the last one, it took 1.8
// times as long.
template <bool kGated>
__device__ __forceinline__ void store_run(const LinArgs &g, long long row0, int lane, int col0, const float (&v)[32],
                                          const float (&u)[32], float *run, int loaded, uint32_t (&x)[16]) {
  for (int o = 0; o < g.n_out; ++o) {
    const LinOut out = g.out[o];
    const int lo = max(col0, out.col_begin), hi = min(min(col0 + 32, out.col_end), g.N);
    if (lo >= hi) continue;
    const int rows = (int)min(32LL, g.M - row0), col = col0 + lane;
    const bool whole = whole_run(out, col0, g.N), inside = col >= lo && col < hi;
    if (out.res && o != loaded) load_residual(g, out, row0, lane, col0, x);
    float y[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) y[e] = v[e];
    activate_run(y, out.act);
    if (kGated) {
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] *= u[e];
    }
    bf16 *dst = static_cast<bf16 *>(out.ptr) - out.col_begin;
    const long long ld = out.ld;
    const bool add = out.res != nullptr;
    if (whole) {
      if (lane >= rows) continue;
      uint4 *to = reinterpret_cast<uint4 *>(dst + (row0 + lane) * ld + col0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a = y[8 * q + 2 * e], b = y[8 * q + 2 * e + 1];
          if (add) a += __uint_as_float(x[4 * q + e] << 16), b += __uint_as_float(x[4 * q + e] & 0xffff0000u);
          __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
          w[e] = *reinterpret_cast<uint32_t *>(&t);
        }
        to[q] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      continue;
    }
    __syncwarp();  // the run before this one has been read
#pragma unroll
    for (int e = 0; e < 32; ++e) run[lane * 33 + e] = y[e];
    __syncwarp();
    if (inside) {
      bf16 *to = dst + row0 * ld + col;
      auto column = [&](auto full) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (full || e < rows) {
            float z = run[e * 33 + lane];
            if (add) z += __uint_as_float(e & 1 ? x[e / 2] & 0xffff0000u : x[e / 2] << 16);
            *to = __float2bfloat16_rn(z);
            to += ld;
          }
      };
      if (rows == 32)
        column(std::true_type{});
      else
        column(std::false_type{});
    }
  }
}

// One epilogue warp's share of a tile: rows row0 .. row0 + 31 (the TMEM lanes at
// taddr), kCols / 2 output columns from tile0 + first.  `wait` waits for the
// accumulator; the residual is loaded one run ahead, the first one before it.
template <int kCols, bool kGated, typename Wait>
__device__ __forceinline__ bool tile_epilogue(const LinArgs &g, float *run, int lane, long long row0, int tile0, int first,
                                              uint32_t taddr, Wait wait) {
  const bf16 *bias = static_cast<const bf16 *>(g.bias);
  uint32_t ahead[16];
  int loaded = prefetch_residual(g, row0, lane, tile0 + first, ahead);
  if (!wait()) {
    if (lane == 0) atomicOr(g.err, kErrTimeout);
    return false;
  }
  fence_after();
#pragma unroll 1
  for (int c = first; c < first + kCols / 2; c += 32) {
    uint32_t x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = ahead[e];
    const int now = loaded;
    const int col0 = tile0 + c;
    if (c + 32 < first + kCols / 2) loaded = prefetch_residual(g, row0, lane, col0 + 32, ahead);
    float v[32], u[32];
    __syncwarp();  // lanes parted on their rows and columns: the TMEM loads take the whole warp together
    tmem_ld32(taddr + c, v);
    if (kGated) tmem_ld32(taddr + kCols + c, u);
    if (row0 >= g.M || col0 >= g.N) continue;
    if (bias) {
      add_bias(v, bias, col0, g.N - col0);
      if (kGated) add_bias(u, bias, (long long)g.N + col0, g.N - col0);
    }
    store_run<kGated>(g, row0, lane, col0, v, u, run, now, x);
  }
  fence_before();
  __syncwarp();
  return true;
}

template <int BN, bool kGated>
__global__ void __launch_bounds__(kTileThreads, 1)
    lin_tile_kernel(const LinArgs g, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w) {
  using L = Tile<BN>;
  constexpr int kStages = L::kStages;
  constexpr int kCols = kGated ? BN / 2 : BN;  // output columns of a tile (gated: the gate rows of w, then the up rows)
  static_assert(kCols >= 64, "two runs of 32 columns at least");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Bars &B = *reinterpret_cast<Bars *>(sm + L::kBars);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + kCols - 1) / kCols;
  const int ntiles = tiles_m * tiles_n;
  const int nk = (g.K + BK - 1) / BK;
  const uint32_t sbase = smem_u32(sm);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(&B.full[s], 1);
      bar_init(&B.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      bar_init(&B.tfull[a], 1);
      bar_init(&B.tempty[a], kEpiWarps);
    }
    bar_init(&B.end, 1);
  }
  if (warp == 1) tmem_alloc(&B.tmem, 2 * BN);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = B.tmem;
  bool ok = true;

  // The loads' and the MMAs' warps stay converged, lane 0 issuing: their operands
  // then live in uniform registers (a lone thread issues at about half the rate).
  if (warp == 0) {
    // ---- TMA producer
    uint32_t it = 0;
    for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
      int mt, nt;
      tile_of(t, tiles_m, tiles_n, mt, nt);
      for (int kb = 0; kb < nk && ok; ++kb, ++it) {
        const int s = it % kStages;
        ok = __all_sync(0xffffffffu, bar_wait(&B.empty[s], ((it / kStages) & 1) ^ 1));
        if (!ok) break;
        const uint32_t dst = sbase + s * L::kStage;
        bar_expect_tx_w(&B.full[s], L::kStage);
        tma_load_3d_w(dst, &tm_x, kb * BK, mt * BM, 0, &B.full[s]);
        tma_load_3d_w(dst + L::kA, &tm_w, kb * BK, nt * kCols, 0, &B.full[s]);
        if (kGated) tma_load_3d_w(dst + L::kA + L::kB / 2, &tm_w, kb * BK, g.N + nt * kCols, 0, &B.full[s]);
      }
    }
    // Leave only when every stage issued has been consumed (bounded).
    for (uint32_t j = (it > kStages ? it - kStages : 0); ok && j < it; ++j)
      ok = __all_sync(0xffffffffu, bar_wait(&B.empty[j % kStages], (j / kStages) & 1));
    if (!ok && lane == 0) atomicOr(g.err, kErrTimeout);
  } else if (warp == 1) {
    // ---- MMA issuer
    const uint32_t id = idesc_bf16(BM, BN), td = __shfl_sync(0xffffffffu, tmem, 0);
    uint32_t it = 0;
    int local = 0;
    for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x, ++local) {
      const int acc = local & 1;
      ok = __all_sync(0xffffffffu, bar_wait(&B.tempty[acc], ((local >> 1) & 1) ^ 1));
      if (!ok) break;
      fence_after();
      const uint32_t d = td + (uint32_t)(acc * BN);
      for (int kb = 0; kb < nk; ++kb, ++it) {
        const int s = it % kStages;
        ok = __all_sync(0xffffffffu, bar_wait(&B.full[s], (it / kStages) & 1));
        if (!ok) break;
        fence_after();
        const uint32_t a0 = sbase + s * L::kStage, b0 = a0 + L::kA;
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks)
          mma_w(d, desc_k(a0, ks, BM), desc_k(b0, ks, BN), id, (kb > 0 || ks > 0) ? 1u : 0u);
        commit_w(&B.empty[s]);
      }
      if (!ok) break;
      commit_w(&B.tfull[acc]);
    }
    commit_w(&B.end);  // every MMA issued is complete before TMEM is freed
    if (!__all_sync(0xffffffffu, bar_wait(&B.end, 0))) ok = false;
    if (!ok && lane == 0) atomicOr(g.err, kErrTimeout);
  } else {
    // ---- epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 = tile rows
    const int quad = warp & 3, half = (warp - 2) >> 2;
    float *run = reinterpret_cast<float *>(sm + L::kRun) + (warp - 2) * 32 * 33;
    int local = 0;
    for (int t = blockIdx.x; t < ntiles; t += gridDim.x, ++local) {
      int mt, nt;
      tile_of(t, tiles_m, tiles_n, mt, nt);
      const int acc = local & 1;
      const auto wait = [&]() { return __all_sync(0xffffffffu, bar_wait(&B.tfull[acc], (local >> 1) & 1)); };
      const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(acc * BN);
      if (!tile_epilogue<kCols, kGated>(g, run, lane, (long long)mt * BM + 32 * quad, nt * kCols, half * (kCols / 2), taddr, wait))
        break;
      if (lane == 0) arrive(&B.tempty[acc]);  // this warp has read its lanes: the accumulator may be refilled
    }
  }

  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_dealloc(tmem, 2 * BN);
  }
}

// =============================================================================
// lin_pair_kernel: 256 x 256 tiles by pairs of CTAs (cta_group::2).  Each CTA
// loads half of x's rows and half of w's; one MMA of the pair reads both, so that
// a CTA moves a third fewer bytes per flop than with a 128 x 256 tile of its own.
// Each CTA's TMEM holds its 128 rows of the result.  Gated: CTA 0's rows of w are
// the gate's, CTA 1's the up half's.
// =============================================================================
constexpr int kPairStages = 6;
constexpr uint32_t kPairHalf = 128 * BK * 2;          // 16 KB: this CTA's rows of x, or of w
constexpr uint32_t kPairStage = 2 * kPairHalf;
constexpr uint32_t kPairBars = kPairStages * kPairStage;
constexpr uint32_t kPairRun = kPairBars + 256;
constexpr uint32_t kPairSmem = kPairRun + kEpiWarps * 32 * 33 * 4 + 1024;
static_assert(kPairSmem <= 232448, "shared memory per CTA");

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's `saddr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// Lane 0 of a converged warp: a 3-d box into this CTA, completing on the mbarrier
// at the cluster address `bar`, which may be the pair's other CTA's.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void *map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .u32 l;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(0), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .u32 l;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate));
}
// Arrive on `bar` in both CTAs once every MMA issued before is complete.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .u32 l;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

template <bool kGated>
__global__ void __launch_bounds__(kTileThreads, 1)
    lin_pair_kernel(const LinArgs g, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w) {
  constexpr int kCols = kGated ? 128 : 256;  // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  // The same offset in both CTAs: the descriptors of one serve the other's tiles.
  uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Bars &B = *reinterpret_cast<Bars *>(sm + kPairBars);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles_m = (g.M + 255) / 256, tiles_n = (g.N + kCols - 1) / kCols;
  const int ntiles = tiles_m * tiles_n;
  const int nk = (g.K + BK - 1) / BK;
  const uint32_t sbase = smem_u32(sm);

  if (tid == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      bar_init(&B.full[s], 1);
      bar_init(&B.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      bar_init(&B.tfull[a], 1);
      bar_init(&B.tempty[a], 2 * kEpiWarps);  // both CTAs' (used in CTA 0)
    }
    bar_init(&B.end, 1);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are ready too
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, B.tmem, 0);
  bool ok = true;

  if (warp == 0) {
    // ---- TMA producer: both CTAs' tiles complete on CTA 0's barriers
    uint32_t it = 0;
    for (int t = pair; t < ntiles && ok; t += pairs) {
      int mt, nt;
      tile_of(t, tiles_m, tiles_n, mt, nt);
      const int xrow = mt * 256 + 128 * rank;
      const int wrow = kGated ? rank * g.N + nt * kCols : nt * kCols + 128 * rank;
      for (int kb = 0; kb < nk && ok; ++kb, ++it) {
        const int s = it % kPairStages;
        ok = __all_sync(0xffffffffu, bar_wait(&B.empty[s], ((it / kPairStages) & 1) ^ 1));
        if (!ok) break;
        const uint32_t dst = sbase + s * kPairStage, bar = map_rank(smem_u32(&B.full[s]), 0);
        if (rank == 0) bar_expect_tx_w(&B.full[s], 2 * kPairStage);
        tma_load_3d_pair(dst, &tm_x, kb * BK, xrow, bar);
        tma_load_3d_pair(dst + kPairHalf, &tm_w, kb * BK, wrow, bar);
      }
    }
    // Leave only when every stage issued has been consumed (bounded).
    for (uint32_t j = (it > kPairStages ? it - kPairStages : 0); ok && j < it; ++j)
      ok = __all_sync(0xffffffffu, bar_wait(&B.empty[j % kPairStages], (j / kPairStages) & 1));
    if (!ok && lane == 0) atomicOr(g.err, kErrTimeout);
  } else if (warp == 1 && rank == 0) {
    // ---- MMA issuer of the pair
    const uint32_t id = idesc_bf16(256, 256);
    uint32_t it = 0;
    int local = 0;
    for (int t = pair; t < ntiles && ok; t += pairs, ++local) {
      const int acc = local & 1;
      ok = __all_sync(0xffffffffu, bar_wait(&B.tempty[acc], ((local >> 1) & 1) ^ 1));
      if (!ok) break;
      fence_after();
      const uint32_t d = tmem + (uint32_t)(acc * 256);
      for (int kb = 0; kb < nk; ++kb, ++it) {
        const int s = it % kPairStages;
        ok = __all_sync(0xffffffffu, bar_wait(&B.full[s], (it / kPairStages) & 1));
        if (!ok) break;
        fence_after();
        const uint32_t a0 = sbase + s * kPairStage, b0 = a0 + kPairHalf;
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks)
          mma_pair(d, desc_k(a0, ks, 128), desc_k(b0, ks, 128), id, (kb > 0 || ks > 0) ? 1u : 0u);
        commit_pair(&B.empty[s]);
      }
      if (!ok) break;
      commit_pair(&B.tfull[acc]);
    }
    commit_pair(&B.end);  // every MMA issued is complete before TMEM is freed
    if (!__all_sync(0xffffffffu, bar_wait(&B.end, 0))) ok = false;
    if (!ok && lane == 0) atomicOr(g.err, kErrTimeout);
  } else if (warp >= 2) {
    // ---- epilogue of this CTA's 128 rows
    const int quad = warp & 3, half = (warp - 2) >> 2;
    float *run = reinterpret_cast<float *>(sm + kPairRun) + (warp - 2) * 32 * 33;
    int local = 0;
    for (int t = pair; t < ntiles; t += pairs, ++local) {
      int mt, nt;
      tile_of(t, tiles_m, tiles_n, mt, nt);
      const int acc = local & 1;
      const auto wait = [&]() { return __all_sync(0xffffffffu, bar_wait(&B.tfull[acc], (local >> 1) & 1)); };
      const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(acc * 256);
      if (!tile_epilogue<kCols, kGated>(g, run, lane, (long long)mt * 256 + 128 * rank + 32 * quad, nt * kCols,
                                        half * (kCols / 2), taddr, wait))
        break;
      if (lane == 0)  // this warp has read its lanes: the accumulator may be refilled
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         map_rank(smem_u32(&B.tempty[acc]), 0))
                     : "memory");
    }
  }
  __syncwarp();

  fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other reads its tiles or arrives on its barriers
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// =============================================================================
// lin_skinny_kernel
// =============================================================================
constexpr int kRowsW = 128;  // rows of w per tile at most (gated: half of them gate rows, half up rows)
constexpr int kSkinnyThreads = 192;

template <int NT>
struct Skinny {
  // 64-wide k blocks per stage: two for the smallest, whose blocks are short
  // against a wait (16 tokens, 6144 -> 5120: 15.0 us, 4 % more with one).
  static constexpr int kSteps = NT <= 16 ? 2 : 1;
  static constexpr uint32_t kA = kRowsW * BK * 2, kB = NT * BK * 2;
  static constexpr uint32_t kBlock = kA + kB;
  static constexpr uint32_t kStage = kSteps * kBlock;
  static constexpr int kRing = (int)(200u * 1024 / kStage);
  static constexpr uint32_t kBars = kRing * kStage;
  static constexpr uint32_t kSmem = kBars + 512 + 1024;
  static constexpr uint32_t kCols = NT < 32 ? 32 : NT;  // TMEM columns
  static_assert(kRowsW * NT * 4 <= kBars, "the partial sums take the ring's place");
  static_assert(kSmem <= 232448, "shared memory per CTA");
};
struct SkinnyBars {
  uint64_t full[12], empty[12];
  uint64_t done;
  uint32_t tmem;
};

// A store to an address of the cluster (map_rank).
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// 8 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Where output column `col` goes: its range's activation and its pointers, row 0.
struct LinCol {
  bf16 *y;
  const bf16 *res;
  long long ld, ldres;
  int act;
};
__device__ __forceinline__ LinCol column(const LinArgs &g, int col) {
  LinCol c{nullptr, nullptr, 0, 0, 0};
  if (col >= g.N) return c;
  for (int o = 0; o < g.n_out; ++o) {
    const LinOut &out = g.out[o];
    if (col < out.col_begin || col >= out.col_end) continue;
    c.y = static_cast<bf16 *>(out.ptr) + (col - out.col_begin);
    c.res = out.res ? static_cast<const bf16 *>(out.res) + (col - out.col_begin) : nullptr;
    c.ld = out.ld;
    c.ldres = out.ldres;
    c.act = out.act;
  }
  return c;
}
// The residual of R rows, row0, row0 + step, .. of which the first `count` exist.
template <int R>
__device__ __forceinline__ void load_rows(const LinCol &c, long long row0, int step, int count, bf16 (&r)[R]) {
  if (!c.res) return;
  const bf16 *res = c.res + row0 * c.ldres;
  const long long d = step * c.ldres;
#pragma unroll
  for (int e = 0; e < R; ++e)
    if (e < count) r[e] = res[e * d];
}
// p (and u, and the residual r) of those rows: independent work, so nothing
// branches on one of them alone.
template <bool kGated, int R>
__device__ __forceinline__ void finish(const LinCol &c, long long row0, int step, int count, float (&p)[R],
                                       const float (&u)[R], const bf16 (&r)[R]) {
  activate_run(p, c.act);
  if (kGated) {
#pragma unroll
    for (int e = 0; e < R; ++e) p[e] *= u[e];
  }
  if (c.res) {
#pragma unroll
    for (int e = 0; e < R; ++e)
      if (e < count) p[e] += __bfloat162float(r[e]);
  }
  bf16 *y = c.y + row0 * c.ld;
  const long long d = step * c.ld;
#pragma unroll
  for (int e = 0; e < R; ++e)
    if (e < count) y[e * d] = __float2bfloat16_rn(p[e]);
}

template <int NT, bool kGated>
__global__ void __launch_bounds__(kSkinnyThreads, 1)
    lin_skinny_kernel(const LinArgs g, int split, int rows_w, const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ CUtensorMap tm_w) {
  using L = Skinny<NT>;
  static_assert(L::kRing <= 12, "barriers");
  constexpr int kOut = kGated ? kRowsW / 2 : kRowsW;  // output columns of a tile at most
  const int out = kGated ? rows_w / 2 : rows_w;       // and of this call's
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  SkinnyBars &B = *reinterpret_cast<SkinnyBars *>(sm + L::kBars);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x % split, tile = blockIdx.x / split;
  const int tiles_n = (g.N + out - 1) / out;
  const int n0 = (tile % tiles_n) * out, m0 = (tile / tiles_n) * NT;
  const int nk = (g.K + BK - 1) / BK;
  const int kb0 = (int)((long long)nk * rank / split), kb1 = (int)((long long)nk * (rank + 1) / split);
  const uint32_t sbase = smem_u32(sm);

  if (tid == 0) {
    for (int s = 0; s < L::kRing; ++s) {
      bar_init(&B.full[s], 1);
      bar_init(&B.empty[s], 1);
    }
    bar_init(&B.done, 1);
  }
  if (warp == 1) tmem_alloc(&B.tmem, L::kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = B.tmem;

  // The loads' and the MMAs' warps stay converged, lane 0 issuing: their operands
  // then live in uniform registers (a lone thread issues at about half the rate).
  bool ok = true;
  const int nst = (kb1 - kb0 + L::kSteps - 1) / L::kSteps;
  if (warp == 0) {
    for (int it = 0; it < nst && ok; ++it) {
      const int s = it % L::kRing;
      ok = __all_sync(0xffffffffu, bar_wait(&B.empty[s], ((it / L::kRing) & 1) ^ 1));
      if (!ok) break;
      const int n = min(L::kSteps, kb1 - kb0 - it * L::kSteps);
      bar_expect_tx_w(&B.full[s], n * (rows_w * BK * 2 + L::kB));
      for (int i = 0; i < n; ++i) {
        const uint32_t dst = sbase + s * L::kStage + i * L::kBlock;
        const int k = (kb0 + it * L::kSteps + i) * BK;
        // One copy for all rows of w, gate and up: the rows past rows_w, if any, stay
        // what they are and so does what the MMAs make of them, which nothing reads.
        tma_load_3d_w(dst, &tm_w, k, n0, 0, &B.full[s]);
        tma_load_3d_w(dst + L::kA, &tm_x, k, m0, 0, &B.full[s]);
      }
    }
  } else if (warp == 1) {
    const uint32_t id = idesc_bf16(kRowsW, NT), d = __shfl_sync(0xffffffffu, tmem, 0);
    for (int it = 0; it < nst && ok; ++it) {
      const int s = it % L::kRing;
      ok = __all_sync(0xffffffffu, bar_wait(&B.full[s], (it / L::kRing) & 1));
      if (!ok) break;
      fence_after();
      const int n = min(L::kSteps, kb1 - kb0 - it * L::kSteps);
#pragma unroll
      for (int i = 0; i < L::kSteps; ++i) {
        if (i >= n) break;
        const uint32_t a0 = sbase + s * L::kStage + i * L::kBlock, b0 = a0 + L::kA;
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks)
          mma_w(d, desc_k(a0, ks, kRowsW), desc_k(b0, ks, NT), id, (it > 0 || i > 0 || ks > 0) ? 1u : 0u);
      }
      commit_w(&B.empty[s]);
    }
    commit_w(&B.done);
  }
  __syncwarp();
  // Every load has landed and every MMA is complete (bounded): the ring is free.
  if (!bar_wait(&B.done, 0)) ok = false;
  if (!__all_sync(0xffffffffu, ok) && lane == 0) atomicOr(g.err, kErrTimeout);
  __syncwarp();
  fence_after();
  const int rows = min(NT, g.M - m0);
  const bf16 *bias = static_cast<const bf16 *>(g.bias);
  if (split > 1) cluster_sync();  // every CTA's ring is free: its first part takes the partial sums
  // Token t is finished by CTA t % split of the cluster, in place t / split.
  const int per = (rows + split - 1) / split;
  float *part = reinterpret_cast<float *>(sm);  // [source CTA][place][128]
  if (warp >= 2) {
    const int n = 32 * (warp & 3) + lane;
    const uint32_t taddr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const bool direct = split == 1 && !kGated;  // this lane already holds its column's sums
    LinCol c{};
    float b = 0.f;
    if (direct) {
      if (n < out) c = column(g, n0 + n);
      if (bias && c.y) b = __bfloat162float(bias[n0 + n]);
    }
    uint32_t to = 0, at = sbase + (uint32_t)(rank * per * kRowsW + n) * 4;
#pragma unroll 1
    for (int t0 = 0; t0 < rows; t0 += 8) {
      float v[8];
      __syncwarp();  // lanes without a column skipped the stores
      tmem_ld8(taddr + t0, v);
      if (direct) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += b;
        if (c.y) {
          bf16 r[8];
          load_rows(c, (long long)m0 + t0, 1, rows - t0, r);
          finish<false>(c, (long long)m0 + t0, 1, rows - t0, v, v, r);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (t0 + e < rows) st_cluster(map_rank(at, to), v[e]);
          const bool wrap = ++to == (uint32_t)split;
          to = wrap ? 0u : to;
          at += wrap ? kRowsW * 4 : 0;
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
  if (split == 1 && !kGated) return;
  // This CTA's tokens, every column of the tile: a thread keeps to one column.
  // The residual is loaded one run of tokens ahead.
  const int mine = (rows - rank + split - 1) / split;
  const int n = tid % kOut;
  constexpr int kShare = kSkinnyThreads / kOut;  // 1 or 3 threads per column
  constexpr int kRun = NT <= 32 ? 4 : 8;         // tokens finished side by side
  const LinCol c = tid < kShare * kOut && n < out ? column(g, n0 + n) : LinCol{};
  const long long row0 = (long long)m0 + rank;
  bf16 ahead[kRun];
  int t = kRun * (tid / kOut);
  if (c.y) load_rows(c, row0 + (long long)t * split, split, mine - t, ahead);
  __syncwarp();  // the barrier takes whole warps
  if (split > 1) cluster_sync();
  if (!c.y) return;
  float b = 0.f, bu = 0.f;
  if (bias) {
    b = __bfloat162float(bias[n0 + n]);
    if (kGated) bu = __bfloat162float(bias[(long long)g.N + n0 + n]);
  }
  for (; t < mine; t += kRun * kShare) {
    bf16 res[kRun];
#pragma unroll
    for (int e = 0; e < kRun; ++e) res[e] = ahead[e];
    const int next = t + kRun * kShare;
    load_rows(c, row0 + (long long)next * split, split, mine - next, ahead);
    float p[kRun], u[kRun];
#pragma unroll
    for (int e = 0; e < kRun; ++e) p[e] = b, u[e] = bu;
    for (int r = 0; r < split; ++r) {
      const float *src = part + (r * per + t) * kRowsW + n;
#pragma unroll
      for (int e = 0; e < kRun; ++e)
        if (t + e < mine) {
          p[e] += src[e * kRowsW];
          if (kGated) u[e] += src[e * kRowsW + out];
        }
    }
    finish<kGated>(c, row0 + (long long)t * split, split, mine - t, p, u, res);
  }
}

// A row-major [rows][K] bf16 matrix, or `parts` of them one after the other, as a
// 3-d map with 128-byte-swizzled boxes of 64 columns x box_rows rows of each part.
bool encode_kmajor(CUtensorMap *m, const void *base, long long rows, long long K, long long ld, int box_rows,
                   int parts = 1) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)rows, (cuuint64_t)parts};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * (cuuint64_t)rows};
  const cuuint32_t box[3] = {(cuuint32_t)BK, (cuuint32_t)box_rows, (cuuint32_t)parts};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool kGated>
struct TileTag {};
template <int NT, bool kGated>
struct SkinnyTag {};

template <bool kGated>
struct PairTag {};

template <bool kGated>
cudaError_t launch_pair(const LinArgs &a, int num_sms, cudaStream_t s) {
  CUtensorMap tm_x, tm_w;
  if (!encode_kmajor(&tm_x, a.x, a.M, a.K, a.ldx, 128) ||
      !encode_kmajor(&tm_w, a.w, (long long)a.N * (kGated ? 2 : 1), a.K, a.ldw, 128))
    return cudaErrorInvalidValue;
  auto *kernel = lin_pair_kernel<kGated>;
  cudaError_t e = allow_smem<PairTag<kGated>>(kernel, kPairSmem);
  if (e != cudaSuccess) return e;
  constexpr int kCols = kGated ? 128 : 256;
  const long long ntiles = (long long)((a.M + 255) / 256) * ((a.N + kCols - 1) / kCols);
  const long long pairs = ntiles < num_sms / 2 ? ntiles : num_sms / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, tm_x, tm_w);
}

template <int BN, bool kGated>
cudaError_t launch_tile(const LinArgs &a, int num_sms, cudaStream_t s) {
  CUtensorMap tm_x, tm_w;
  if (!encode_kmajor(&tm_x, a.x, a.M, a.K, a.ldx, BM) ||
      !encode_kmajor(&tm_w, a.w, (long long)a.N * (kGated ? 2 : 1), a.K, a.ldw, kGated ? BN / 2 : BN))
    return cudaErrorInvalidValue;
  constexpr size_t kSmem = Tile<BN>::kSmem;
  cudaError_t e = allow_smem<TileTag<BN, kGated>>(lin_tile_kernel<BN, kGated>, kSmem);
  if (e != cudaSuccess) return e;
  constexpr int kCols = kGated ? BN / 2 : BN;
  const long long ntiles = (long long)((a.M + BM - 1) / BM) * ((a.N + kCols - 1) / kCols);
  lin_tile_kernel<BN, kGated><<<(int)(ntiles < num_sms ? ntiles : num_sms), kTileThreads, kSmem, s>>>(a, tm_x, tm_w);
  return cudaGetLastError();
}

// How many clusters of `size` CTAs of the skinny kernel run at once: fewer than
// the SMs would take, since a cluster stays within one group of SMs (152 SMs: 46
// of 3, 36 of 4, 28 of 5, 23 of 6, 15 of 7 or 8).  Asked once per device.
template <int NT, bool kGated>
cudaError_t cluster_caps(int num_sms, int (&cap)[9]) {
  using L = Skinny<NT>;
  static std::atomic<uint64_t> known[64];  // a byte per size
  auto *kernel = lin_skinny_kernel<NT, kGated>;
  cudaError_t e = allow_smem<SkinnyTag<NT, kGated>>(kernel, L::kSmem);
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  uint64_t bytes = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (bytes == 0) {
    for (int size = 2; size <= 8; ++size) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3((unsigned)(size * num_sms));
      cfg.blockDim = dim3(kSkinnyThreads);
      cfg.dynamicSmemBytes = L::kSmem;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = (unsigned)size;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) return e;
      bytes |= (uint64_t)(n < 255 ? n : 255) << (8 * (size - 1));
    }
    bytes |= 1;  // asked
    if (dev < 64) known[dev].store(bytes, std::memory_order_relaxed);
  }
  cap[0] = 0, cap[1] = num_sms;
  for (int size = 2; size <= 8; ++size) cap[size] = (int)(bytes >> (8 * (size - 1)) & 255);
  return cudaSuccess;
}

// The widest split of `tiles` whose CTAs all run at once, each with some k steps
// and (the partial sums' space) whole tokens; 1 where they do not.  A wider one
// costs a second wave (16 tokens, 4096 -> 2560, w in L2: 6.6 us with 6 CTAs per
// cluster, 11.8 with 7, whose 20 clusters do not fit).
template <int NT>
int skinny_split(long long tiles, int nk, const int (&cap)[9]) {
  int split = nk / 2 < 8 ? nk / 2 : 8;
  while (split > 1 && (tiles > cap[split] || split * ((NT + split - 1) / split) * kRowsW * 4 > (int)Skinny<NT>::kBars)) --split;
  return split < 1 ? 1 : split;
}

// The skinny kernel's tiles: NT tokens by rows_w rows of w, over clusters of
// `split`.  Microseconds, measured: a wave's loads (w and x) at 11.5 TB/s from
// L2, w at 6.5 from memory, or a CTA's k steps at 0.15; per wave a start, the
// partial sums' exchange by the tokens, and the finishing by a CTA's share of them.
struct SkinnyPlan {
  int rows_w, split;
  long long tiles;
  float cost;
};
template <int NT, bool kGated>
cudaError_t skinny_plan(const LinArgs &a, int num_sms, bool residual, SkinnyPlan &plan) {
  int cap[9];
  const cudaError_t e = cluster_caps<NT, kGated>(num_sms, cap);
  if (e != cudaSuccess) return e;
  const int nk = (a.K + BK - 1) / BK;
  const long long tiles_m = (a.M + NT - 1) / NT;
  const float tokens = (float)(a.M < NT ? a.M : NT);
  // All 128 rows of w, or fewer where the tiles come in several waves and smaller
  // ones fill the last better (8 tokens, 5120 -> 24576: 43.9 us with 112 rows, 45.7
  // with 128).  From 128 tokens on the loads of x count as much.
  for (int rows = kRowsW; rows >= (NT <= 64 ? 80 : kRowsW); rows -= 16) {
    const int out = kGated ? rows / 2 : rows;
    const long long n = (a.N + out - 1) / out * tiles_m;
    const int split = skinny_split<NT>(n, nk, cap);
    const float steps = (float)nk / split;
    const float cta = steps * BK * 2e-6f;  // MB per row
    const float load = cta * (rows + NT) / 11.5f, mem = cta * rows / 6.5f / tiles_m;
    const bool direct = split == 1 && !kGated;
    const float rest = 4.3f + (direct ? 0.03f : 0.016f + 0.06f / split) * tokens +
                       (!residual ? 0.f : direct ? 0.03f * tokens : 0.5f + 0.01f * tokens);
    auto wave = [&](long long clusters) {
      const float all = (load > mem ? load : mem) * (clusters * split), one = 0.15f * steps;
      return (all > one ? all : one) + rest;
    };
    const long long waves = n / cap[split], left = n % cap[split];
    // Part of a start runs beside the wave before it.
    const float cost = waves * wave(cap[split]) + (left ? wave(left) : 0.f) - 2.3f * (waves - (left ? 0 : 1));
    if (rows == kRowsW || cost < 0.97f * plan.cost) plan = SkinnyPlan{rows, split, n, cost};
  }
  return cudaSuccess;
}

template <int NT, bool kGated>
cudaError_t launch_skinny(const LinArgs &a, const LinForm &plan, cudaStream_t s) {
  CUtensorMap tm_x, tm_w;
  if (!encode_kmajor(&tm_x, a.x, a.M, a.K, a.ldx, NT) ||
      !encode_kmajor(&tm_w, a.w, a.N, a.K, a.ldw, kGated ? plan.rows_w / 2 : plan.rows_w, kGated ? 2 : 1))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(plan.tiles * plan.split));
  cfg.blockDim = dim3(kSkinnyThreads);
  cfg.dynamicSmemBytes = Skinny<NT>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)plan.split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lin_skinny_kernel<NT, kGated>, a, plan.split, plan.rows_w, tm_x, tm_w);
}

// Microseconds of the tile kernel with tiles of BN w rows: a wave's k steps or
// its epilogue, whichever is longer, and the last epilogue.  Measured: 0.40 us per
// 64-wide k step at 256, which falls less than the tile does; 1.5 us per 64
// columns of epilogue.
template <bool kGated>
float tile_cost(const LinArgs &a, int BN, int num_sms) {
  const int cols = kGated ? BN / 2 : BN, nk = (a.K + BK - 1) / BK;
  const long long tiles = (long long)((a.M + BM - 1) / BM) * ((a.N + cols - 1) / cols);
  const float loop = (BN == 256 ? 0.40f : BN == 128 ? 0.24f : 0.19f) * nk, epi = 1.5f * cols / 64;
  return (float)((tiles + num_sms - 1) / num_sms) * (loop > epi ? loop : epi) + epi;
}

// The form with the least cost.
template <bool kGated>
cudaError_t choose(const LinArgs &a, int num_sms, LinForm *form) {
  const int nk = (a.K + BK - 1) / BK;
  bool residual = false;
  for (int o = 0; o < a.n_out; ++o) residual |= a.out[o].res != nullptr;
  // Few tokens or few columns: tiles of 16 to 256 tokens, fewer than there are
  // where that fills the SMs (219 tokens, 3640 -> 421: 7.8 us in tiles of 32, 15.3
  // in one of 256, 19.5 by the tile kernel; 128 tokens, 6144 -> 5120: 21 in one of
  // 128, 38.7 in tiles of 32).
  constexpr int kMostTokens = 2048;  // beyond, other forms have the tiles
  SkinnyPlan best{0, 0, 0, 1e30f};
  int nt = 0;
  cudaError_t e = cudaSuccess;
  auto consider = [&](auto tokens) {
    constexpr int NT = decltype(tokens)::value;
    if (e != cudaSuccess || (NT > 16 && a.M <= NT / 2)) return;
    SkinnyPlan p{0, 0, 0, 1e30f};
    e = skinny_plan<NT, kGated>(a, num_sms, residual, p);
    if (p.cost < best.cost) best = p, nt = NT;
  };
  if (a.M <= kMostTokens) {
    consider(std::integral_constant<int, 16>());
    consider(std::integral_constant<int, 32>());
    consider(std::integral_constant<int, 64>());
    consider(std::integral_constant<int, 128>());
    consider(std::integral_constant<int, 256>());
    if (e != cudaSuccess) return e;
  }
  // Against the tile kernel and the pairs, whose costs are without the launch.
  const float t256 = tile_cost<kGated>(a, 256, num_sms), t128 = tile_cost<kGated>(a, 128, num_sms);
  const float t64 = kGated ? 1e30f : tile_cost<kGated>(a, 64, num_sms);
  // Pairs: 0.37 us per k step of a wave of their 256 x 256 tiles.
  const int cols = kGated ? 128 : 256;
  const long long tiles = (long long)((a.M + 255) / 256) * ((a.N + cols - 1) / cols);
  const float loop = 0.37f * nk, epi = 1.5f * cols / 64;
  const float pair = (float)((tiles + num_sms / 2 - 1) / (num_sms / 2)) * (loop > epi ? loop : epi) + epi;
  const float mem = (kGated ? 4e-6f : 2e-6f) * a.N / 6.5f * a.K;  // w, once
  const float least = fmaxf(fminf(fminf(t256, t128), fminf(t64, pair)), mem) + (residual ? 6.f : 4.5f);
  // Up to 128 tokens they read w once as well, but in fewer pieces: a clear gain only
  // (107 tokens, 920 -> 6856 with a residual: 9.6 us by tiles, 11.9 so).
  if (best.cost < least * (a.M <= 128 ? 1.1f : 0.9f)) {
    *form = LinForm{GDN_LINEAR_EX_FEW, nt, best.tiles, best.rows_w, best.split};
    return cudaSuccess;
  }
  if (pair <= t256 && pair <= t128 && pair <= t64) {
    *form = LinForm{GDN_LINEAR_EX_PAIR, cols, tiles, 0, 0};
    return cudaSuccess;
  }
  const int BN = t256 <= t128 && t256 <= t64 ? 256 : t128 <= t64 ? 128 : 64, out = kGated ? BN / 2 : BN;
  *form = LinForm{GDN_LINEAR_EX_TILE, out, (long long)((a.M + BM - 1) / BM) * ((a.N + out - 1) / out), 0, 0};
  return cudaSuccess;
}

template <bool kGated>
cudaError_t launch(const LinArgs &a, int num_sms, cudaStream_t s) {
  LinForm form;
  const cudaError_t e = choose<kGated>(a, num_sms, &form);
  if (e != cudaSuccess) return e;
  if (form.kernel == GDN_LINEAR_EX_PAIR) return launch_pair<kGated>(a, num_sms, s);
  if (form.kernel == GDN_LINEAR_EX_TILE) {
    if (form.tile == (kGated ? 128 : 256)) return launch_tile<256, kGated>(a, num_sms, s);
    if (form.tile == (kGated ? 64 : 128)) return launch_tile<128, kGated>(a, num_sms, s);
    return launch_tile<kGated ? 128 : 64, kGated>(a, num_sms, s);
  }
  switch (form.tile) {
    case 16: return launch_skinny<16, kGated>(a, form, s);
    case 32: return launch_skinny<32, kGated>(a, form, s);
    case 64: return launch_skinny<64, kGated>(a, form, s);
    case 128: return launch_skinny<128, kGated>(a, form, s);
    default: return launch_skinny<256, kGated>(a, form, s);
  }
}

}  // namespace

cudaError_t launch_linear_ex(const LinArgs &a, int num_sms, cudaStream_t s) {
  return a.gated ? launch<true>(a, num_sms, s) : launch<false>(a, num_sms, s);
}
cudaError_t linear_ex_form(const LinArgs &a, int num_sms, LinForm *form) {
  return a.gated ? choose<true>(a, num_sms, form) : choose<false>(a, num_sms, form);
}

}  // namespace gdn
