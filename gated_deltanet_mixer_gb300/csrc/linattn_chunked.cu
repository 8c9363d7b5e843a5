// linattn_chunked.cu -- linear attention with a decay for each head over
// prompts (bf16 io), in chunks of 64 tokens on the tcgen05 tensor cores.
//
// With G_i the sum of the log decays of the chunk's tokens up to i, the
// recurrence S_t = e^{g_t} S_{t-1} + v_t k_t^T, o_t = S_t q_t becomes, kept
// value-major (S[v][k]) and with tokens along the columns,
//   O^T = e^{G_i} (S Q^T) + V^T P^T,  P_ij = e^{G_i - G_j} q_i . k_j (j <= i),
//   S'  = e^{G_last} S + V^T (Gamma K),  Gamma_j = e^{G_last - G_j}.
// Every exponent is <= 0.  Only S Q^T and the sum of S' carry the state: the
// products P, V^T P^T and V^T (Gamma K) of a chunk do not wait for it.
//
// One CTA walks the chunks of one (sequence, value head, segment):
//   warp 16      TMA: q, k, v tiles into a 3-stage ring; the chunk's decays
//   warp 17      issues the MMAs
//   warps 8-11   Gamma K into shared memory; P from TMEM into shared memory
//   warps 0-7    the state, fp32 in registers: copies it to TMEM as the MMA
//                operand, then adds the chunk's update
//   warps 12-15  the output
// Precision: bf16 holds 8 significant bits, so what is not bf16 already goes
// to the MMA as a sum of bf16 pieces.  Gamma K, which feeds the carried fp32
// state, takes three (24 bits); P and S, which feed the bf16 output only, two
// (16 bits).  Every product starts from a zero accumulator and the state is
// summed in fp32 registers, because an MMA truncates what it adds to.
//
// Few units (sequences x value heads) leave SMs idle, so a sequence can be cut
// into segments: a first launch (kStateOnly) forms each segment's state from
// zero, a second starts every segment from the decayed sum of those before it.
// Cost: k and v are read twice.
#include <cuda.h>
#include <cuda_bf16.h>

#include "gdn_device.cuh"
#include "launch.h"
#include "tma_host.h"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace umma;

constexpr int kC = 64;  // tokens per chunk
constexpr int kStages = 3;
constexpr int kVecs = 8;  // chunk vectors in flight (the output warps lag the loads by less)
constexpr float kMinLogDecay = -80.f;  // a decay below e^-80 acts as e^-80: sums of it stay finite

constexpr uint32_t kTile = kC * kD * 2;             // 16 KB: 64 tokens x 128
constexpr uint32_t kStageBytes = 3 * kTile;         // q, k, v
constexpr uint32_t kGk = kStages * kStageBytes;     // Gamma K, three pieces
constexpr uint32_t kP = kGk + 3 * kTile;            // P, two pieces of 8 KB
constexpr uint32_t kPTile = kC * kC * 2;
constexpr uint32_t kShared = kP + 2 * kPTile;

struct ChunkVec {
  float G[kC];    // sums of the log decays from the chunk's first token
  float eG[kC];   // e^G
  float gam[kC];  // e^{G_last - G}, 0 past the sequence's end
  float d;        // e^{G_last}
  float pad[3];
};
struct Shared {
  ChunkVec vec[kVecs];
  uint64_t full[kStages], empty[kStages];
  uint64_t qk_done, p_ready, gk_ready, su_done, ds_free, s_ready, o_done, o_free, end;
  uint32_t tmem;
};
constexpr uint32_t kSmem = kShared + ((sizeof(Shared) + 127) / 128) * 128 + 1024;
static_assert(kSmem <= 232448, "shared memory per CTA");

constexpr int kThreads = 18 * 32;
// TMEM columns (fp32, or bf16 pairs for the state operand).
constexpr uint32_t kTDs = 0, kTSh = 128, kTSl = 192, kTO1 = 256, kTO2 = 320, kTP = 384;

// Instruction descriptor, kind::f16 with bf16 A and B (format 1), fp32 D.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
  return idesc(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);
}

__device__ __forceinline__ void arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&t);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 64 columns of 16 lanes: register 4 b + (0, 1) holds columns 8 b + 2 (lane % 4)
// + (0, 1) of row lane / 4, registers 4 b + (2, 3) the same of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld16x64(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  tmem_wait_ld();
}

// Warp-wide bounded wait: every lane looks at the barrier.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity));
}

// The decays of a chunk, by one warp: lane L holds tokens L and L + 32.
__device__ __forceinline__ void chunk_vec(ChunkVec &cv, float g0, float g1, int len, int lane) {
  float p0 = g0, p1 = g1;  // inclusive sums from the front
  float s0 = g0, s1 = g1;  // and from the back: no cancellation in e^{G_last - G_j}
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float a = __shfl_up_sync(0xffffffffu, p0, off), b = __shfl_up_sync(0xffffffffu, p1, off);
    const float c = __shfl_down_sync(0xffffffffu, s0, off), d = __shfl_down_sync(0xffffffffu, s1, off);
    if (lane >= off) p0 += a, p1 += b;
    if (lane + off < 32) s0 += c, s1 += d;
  }
  p1 += __shfl_sync(0xffffffffu, p0, 31);
  s0 += __shfl_sync(0xffffffffu, s1, 0);
  // sums over the tokens behind: shift the inclusive sums by one token
  float e0 = __shfl_down_sync(0xffffffffu, s0, 1), e1 = __shfl_down_sync(0xffffffffu, s1, 1);
  const float first1 = __shfl_sync(0xffffffffu, s1, 0);
  if (lane == 31) e0 = first1, e1 = 0.f;
  cv.G[lane] = p0;
  cv.G[lane + 32] = p1;
  cv.eG[lane] = expf(p0);
  cv.eG[lane + 32] = expf(p1);
  cv.gam[lane] = lane < len ? expf(e0) : 0.f;
  cv.gam[lane + 32] = lane + 32 < len ? expf(e1) : 0.f;
  if (lane == 0) cv.d = expf(s0);
}

template <bool kStateOnly>
__global__ void __launch_bounds__(kThreads, 1)
    linattn_chunked_kernel(const LinAttnArgs a, const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Shared &B = *reinterpret_cast<Shared *>(sm + kShared);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- the work of this CTA; consecutive CTAs are the heads of one segment
  const int launched_seg = kStateOnly ? a.nseg - 1 : a.nseg;
  const int h = blockIdx.x % a.Hv, kh = h / (a.Hv / a.Hk);
  const int seg = (blockIdx.x / a.Hv) % launched_seg;
  int b = blockIdx.x / (a.Hv * launched_seg);
  long long row0;
  int T;
  if (a.cu_seqlens) {
    if (a.B <= kLongestFirstMax) b = longest_first(a.cu_seqlens, a.B, b, reinterpret_cast<int *>(sm));
    const int s0 = a.cu_seqlens[b], s1 = a.cu_seqlens[b + 1];
    if (s0 < 0 || s1 < s0 || s1 > a.T) {
      if (tid == 0) atomicOr(a.err, kErrSeqlens);
      return;
    }
    row0 = s0;
    T = s1 - s0;
  } else {
    row0 = (long long)b * a.T;
    T = a.T;
  }
  const int unit = b * a.Hv + h;
  const long long units = (long long)a.B * a.Hv;
  const int nch = (T + kC - 1) / kC, per = (nch + a.nseg - 1) / a.nseg;
  const int c0 = min(nch, seg * per), c1 = min(nch, c0 + per);
  const int n_chunks = c1 - c0;
  constexpr long long kState = kD * kD;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(&B.full[s], 2);
      bar_init(&B.empty[s], 1);
    }
    bar_init(&B.qk_done, 1);
    bar_init(&B.p_ready, 128);
    bar_init(&B.gk_ready, 128);
    bar_init(&B.su_done, 1);
    bar_init(&B.ds_free, 256);
    bar_init(&B.s_ready, 256);
    bar_init(&B.o_done, 1);
    bar_init(&B.o_free, 128);
    bar_init(&B.end, 1);
  }
  if (warp == 17) tmem_alloc(&B.tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = B.tmem;
  bool ok = true;

  if (warp == 16) {
    // ---- TMA producer and the chunk vectors
    auto load_g = [&](int c, float &g0, float &g1) {
      g0 = g1 = 0.f;
      const int t = c * kC + lane;
      if (a.g) {
        if (t < T) g0 = a.g[(row0 + t) * a.Hv + h];
        if (t + 32 < T) g1 = a.g[(row0 + t + 32) * a.Hv + h];
      } else {
        const float gh = a.log_decay[h];
        if (t < T) g0 = gh;
        if (t + 32 < T) g1 = gh;
      }
      g0 = fmaxf(g0, kMinLogDecay);
      g1 = fmaxf(g1, kMinLogDecay);
    };
    float g0 = 0.f, g1 = 0.f;
    if (n_chunks > 0) load_g(c0, g0, g1);
    int n = 0;
    for (; n < n_chunks; ++n) {
      const int s = n % kStages;
      if (!warp_wait(&B.empty[s], ((n / kStages) & 1) ^ 1)) {
        ok = false;
        break;
      }
      const int c = c0 + n;
      if (lane == 0) {
        const uint32_t dst = sbase + s * kStageBytes;
        const int row = (int)(row0 + (long long)c * kC);
        bar_expect_tx(&B.full[s], kStateOnly ? 2 * kTile : 3 * kTile);
        for (int x = 0; x < 2; ++x) {
          if (!kStateOnly) tma_load_3d(dst + x * (kTile / 2), &tm_q, kh * kD + 64 * x, row, 0, &B.full[s]);
          tma_load_3d(dst + kTile + x * (kTile / 2), &tm_k, kh * kD + 64 * x, row, 0, &B.full[s]);
          tma_load_3d(dst + 2 * kTile + x * (kTile / 2), &tm_v, h * kD + 64 * x, row, 0, &B.full[s]);
        }
      }
      chunk_vec(B.vec[n % kVecs], g0, g1, T - c * kC, lane);
      __syncwarp();
      if (lane == 0) arrive(&B.full[s]);
      if (n + 1 < n_chunks) load_g(c + 1, g0, g1);
    }
    // Leave only when every tile issued has been consumed (bounded).
    for (int j = max(0, n - kStages); ok && j < n; ++j)
      if (!warp_wait(&B.empty[j % kStages], (j / kStages) & 1)) ok = false;
  } else if (warp == 17) {
    // ---- MMA issuer (the whole warp; lane 0 issues)
    const uint32_t id_p = idesc_bf16(64, 64, 0, 0);     // Q K^T
    const uint32_t id_o1 = idesc_bf16(128, 64, 0, 0);   // S Q^T
    const uint32_t id_o2 = idesc_bf16(128, 64, 1, 0);   // V^T P^T
    const uint32_t id_su = idesc_bf16(128, 128, 1, 1);  // V^T (Gamma K)
    auto issue_qk = [&](int s) {
      const uint32_t q = sbase + s * kStageBytes, k = q + kTile;
#pragma unroll
      for (int ks = 0; ks < kD / 16; ++ks) mma_w(tmem + kTP, desc_k(q, ks, kC), desc_k(k, ks, kC), id_p, ks > 0);
      commit_w(&B.qk_done);
    };
    auto issue_su = [&](int s) {
      const uint32_t v = sbase + s * kStageBytes + 2 * kTile;
#pragma unroll
      for (int p = 2; p >= 0; --p)  // small pieces first
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          mma_w(tmem + kTDs, desc_mn(v, ks, kC), desc_mn(sbase + kGk + p * kTile, ks, kC), id_su, p < 2 || ks > 0);
      commit_w(&B.su_done);
    };
    if (n_chunks > 0) {
      ok = warp_wait(&B.full[0], 0);
      if (ok && !kStateOnly) issue_qk(0);
      if (ok) ok = warp_wait(&B.gk_ready, 0);
      fence_after();
      if (ok) issue_su(0);
    }
    for (int n = 0; n < n_chunks && ok; ++n) {
      const int s = n % kStages, s1 = (n + 1) % kStages;
      const uint32_t par = n & 1;
      const bool more = n + 1 < n_chunks;
      if (!kStateOnly) {
        ok = warp_wait(&B.p_ready, par);  // P(n) is in shared memory, its TMEM columns are free
        if (ok && more) {
          ok = warp_wait(&B.full[s1], ((n + 1) / kStages) & 1);
          fence_after();
          if (ok) issue_qk(s1);
        }
        if (ok) ok = warp_wait(&B.o_free, par ^ 1);
        if (!ok) break;
        fence_after();
        const uint32_t q = sbase + s * kStageBytes, v = q + 2 * kTile;
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_w(tmem + kTO2, desc_mn(v, ks, kC), desc_k(sbase + kP + p * kPTile, ks, kC), id_o2, p < 1 || ks > 0);
        ok = warp_wait(&B.s_ready, par);
        if (!ok) break;
        fence_after();
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks)
            mma_ta_w(tmem + kTO1, tmem + (p ? kTSl : kTSh) + ks * 8, desc_k(q, ks, kC), id_o1, p < 1 || ks > 0);
        commit_w(&B.o_done);
      }
      commit_w(&B.empty[s]);  // the update of chunk n was issued before
      if (more) {
        if (kStateOnly) ok = warp_wait(&B.full[s1], ((n + 1) / kStages) & 1);
        ok = ok && warp_wait(&B.gk_ready, par ^ 1) && warp_wait(&B.ds_free, par);
        fence_after();
        if (ok) issue_su(s1);
      }
    }
    commit_w(&B.end);  // every MMA issued is complete before TMEM is freed
    if (!warp_wait(&B.end, 0)) ok = false;
  } else if (warp >= 8 && warp < 12) {
    // ---- Gamma K and P
    const int t = tid - 256, j = t & 63, half = t >> 6;
    const uint32_t krow = (uint32_t)(half * (kTile / 2) + (j >> 3) * 1024 + (j & 7) * 128);
    const int w = warp - 8;  // TMEM quarter: rows 16 w .. 16 w + 15 of P
    const int i0 = 16 * w + (lane >> 2), cc = 2 * (lane & 3);
    if (!kStateOnly) {  // P above the diagonal block stays zero
      for (int blk = 2 * w + 2; blk < 8; ++blk)
        for (int p = 0; p < 2; ++p)
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<uint32_t *>(sm + kP + p * kPTile + kmaj(i0 + 8 * r, 8 * blk + cc, kC)) = 0;
    }
    for (int n = 0; n < n_chunks; ++n) {
      const int s = n % kStages;
      const uint32_t par = n & 1;
      const ChunkVec &cv = B.vec[n % kVecs];
      ok = warp_wait(&B.full[s], (n / kStages) & 1);
      if (ok && n > 0) ok = warp_wait(&B.su_done, par ^ 1);  // the last update has read its Gamma K
      if (!ok) break;
      {
        const uint8_t *src = sm + s * kStageBytes + kTile + krow;
        uint8_t *dst = sm + kGk + krow;
        const float gam = cv.gam[j];
        const bool inside = (c0 + n) * kC + j < T;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t at = (uint32_t)((c ^ (j & 7)) << 4);
          const uint4 u = *reinterpret_cast<const uint4 *>(src + at);
          const uint32_t in[4] = {u.x, u.y, u.z, u.w};
          uint32_t p0[4], p1[4], p2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = inside ? lo_f(in[e]) * gam : 0.f, y = inside ? hi_f(in[e]) * gam : 0.f;
            p0[e] = pack_bf16(x, y);
            const float x1 = x - lo_f(p0[e]), y1 = y - hi_f(p0[e]);
            p1[e] = pack_bf16(x1, y1);
            p2[e] = pack_bf16(x1 - lo_f(p1[e]), y1 - hi_f(p1[e]));
          }
          *reinterpret_cast<uint4 *>(dst + at) = make_uint4(p0[0], p0[1], p0[2], p0[3]);
          *reinterpret_cast<uint4 *>(dst + kTile + at) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
          *reinterpret_cast<uint4 *>(dst + 2 * kTile + at) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
        }
        if (!inside) {  // rows past the end (another sequence's, or none): 0 x value must be 0
          uint8_t *v = sm + s * kStageBytes + 2 * kTile + krow;
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(v + 16 * c) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_smem_to_async();
      arrive(&B.gk_ready);
      if (kStateOnly) continue;
      ok = warp_wait(&B.qk_done, par);
      if (ok && n > 0) ok = warp_wait(&B.o_done, par ^ 1);  // the last output has read its P
      if (!ok) break;
      fence_after();
      uint32_t r[32];
      tmem_ld16x64(tmem + ((uint32_t)(32 * w) << 16) + kTP, r);
      const float ga = cv.G[i0], gb = cv.G[i0 + 8];
#pragma unroll
      for (int blk = 0; blk < 8; ++blk) {
        if (blk > 2 * w + 1) break;
        const int jc = 8 * blk + cc;
        const float2 gj = *reinterpret_cast<const float2 *>(&cv.G[jc]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = i0 + 8 * q;
          const float gi = q ? gb : ga;
          const float x = jc <= i ? __uint_as_float(r[4 * blk + 2 * q]) * __expf(gi - gj.x) : 0.f;
          const float y = jc + 1 <= i ? __uint_as_float(r[4 * blk + 2 * q + 1]) * __expf(gi - gj.y) : 0.f;
          const uint32_t p0 = pack_bf16(x, y);
          uint8_t *dst = sm + kP + kmaj(i, jc, kC);
          *reinterpret_cast<uint32_t *>(dst) = p0;
          *reinterpret_cast<uint32_t *>(dst + kPTile) = pack_bf16(x - lo_f(p0), y - hi_f(p0));
        }
      }
      fence_before();
      fence_smem_to_async();
      arrive(&B.p_ready);
    }
  } else if (warp < 8) {
    // ---- the state: row v, columns 64 half .. 64 half + 63
    const int v = 32 * (warp & 3) + lane, half = warp >> 2;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const long long at = (long long)unit * kState + v * kD + 64 * half;
    float *dec = a.ws + a.nseg * units * kState;  // [nseg][units]
    float S[64];
    auto read = [&](const float *src, float mul, bool add) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(src + 4 * i);
        S[4 * i] = add ? fmaf(mul, S[4 * i], x.x) : x.x;
        S[4 * i + 1] = add ? fmaf(mul, S[4 * i + 1], x.y) : x.y;
        S[4 * i + 2] = add ? fmaf(mul, S[4 * i + 2], x.z) : x.z;
        S[4 * i + 3] = add ? fmaf(mul, S[4 * i + 3], x.w) : x.w;
      }
    };
    auto write = [&](float *dst) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float4 *>(dst + 4 * i) = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    };
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
    if (kStateOnly) {
      // The call's S_T may be S0 itself: the second launch reads S0 from slot 0.
      if (seg == 0 && a.S0) {
        read(a.S0 + at, 0.f, false);
        write(a.ws + at);
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = 0.f;
      }
    } else if (a.nseg > 1) {
      if (a.S0) read(a.ws + at, 0.f, false);
      for (int m = 1; m <= seg; ++m) read(a.ws + m * units * kState + at, dec[m * units + unit], true);
    } else if (a.S0) {
      read(a.S0 + at, 0.f, false);
    }
    float dtot = 1.f;
    for (int n = 0; n < n_chunks; ++n) {
      const uint32_t par = n & 1;
      if (!kStateOnly) {
        if (n > 0) ok = warp_wait(&B.o_done, par ^ 1);  // the last output has read its state
        if (!ok) break;
        uint32_t hi[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) hi[i] = pack_bf16(S[2 * i], S[2 * i + 1]);
        tmem_st32w_nw(tl + kTSh + 32 * half, hi);
#pragma unroll
        for (int i = 0; i < 32; ++i) hi[i] = pack_bf16(S[2 * i] - lo_f(hi[i]), S[2 * i + 1] - hi_f(hi[i]));
        tmem_st32w_nw(tl + kTSl + 32 * half, hi);
        tmem_wait_st();
        fence_before();
        arrive(&B.s_ready);
      }
      ok = warp_wait(&B.su_done, par);
      if (!ok) break;
      fence_after();
      const float d = B.vec[n % kVecs].d;
      if (kStateOnly) dtot *= d;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t r[32];
        tmem_ld32_nw(tl + kTDs + 64 * half + 32 * i, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) S[32 * i + e] = fmaf(d, S[32 * i + e], __uint_as_float(r[e]));
      }
      fence_before();
      arrive(&B.ds_free);
    }
    if (kStateOnly) {
      write(a.ws + (seg + 1) * units * kState + at);
      if (tid == 0) dec[(seg + 1) * units + unit] = dtot;
    } else if (seg == a.nseg - 1) {
      if (in_bounds(at + 64, units * kState, a.err)) write(a.S_T + at);
    }
  } else if (!kStateOnly) {
    // ---- the output: lane = value index, one column per token
    const int v = 32 * (warp & 3) + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + (row0 + (long long)c0 * kC) * a.ldo + h * kD + v;
    const long long o_at = (row0 + (long long)c0 * kC) * a.ldo + h * kD + v;
    const long long o_size = ((a.cu_seqlens ? a.T : (long long)a.B * a.T) - 1) * a.ldo + (long long)a.Hv * kD;
    for (int n = 0; n < n_chunks; ++n) {
      ok = warp_wait(&B.o_done, n & 1);
      if (!ok) break;
      fence_after();
      const ChunkVec &cv = B.vec[n % kVecs];
      const int len = min(kC, T - (c0 + n) * kC);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t r1[32], r2[32];
        tmem_ld32_nw(tl + kTO1 + 32 * i, r1);
        tmem_ld32_nw(tl + kTO2 + 32 * i, r2);
        tmem_wait_ld();
        if (i == 1) {
          fence_before();
          arrive(&B.o_free);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int tk = 32 * i + e;
          const float y = a.scale * fmaf(cv.eG[tk], __uint_as_float(r1[e]), __uint_as_float(r2[e]));
          const long long off = (long long)(n * kC + tk) * a.ldo;
          if (tk < len && in_bounds(o_at + off + 1, o_size, a.err)) o[off] = __float2bfloat16_rn(y);
        }
      }
    }
  }
  if (!ok && lane == 0) atomicOr(a.err, kErrTimeout);

  fence_before();
  __syncthreads();
  if (warp == 17) {
    fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Token rows of a [rows][cols] bf16 tensor, ld elements apart: boxes of 64
// columns x 64 rows, 128-byte swizzle (third extent 1).
bool encode_rows(CUtensorMap *m, const void *base, long long rows, long long cols, long long ld) {
  EncodeTiled enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 1};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * (cuuint64_t)rows};
  const cuuint32_t box[3] = {64, (cuuint32_t)kC, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int linattn_segments(int B, int Hv, long long tokens, bool packed, int sms) {
  const long long units = (long long)B * Hv;
  // The chunks of a sequence (packed: of the average one).
  const long long nch = packed ? (tokens / B + kC - 1) / kC : (tokens / B + kC - 1) / kC;
  long long n = sms / units;  // one CTA per SM
  if (n > nch / 4) n = nch / 4;
  if (n > kLinAttnMaxSeg) n = kLinAttnMaxSeg;
  return n < 2 ? 1 : (int)n;
}

cudaError_t launch_linattn_chunked(const LinAttnArgs &a, cudaStream_t s) {
  const long long rows = a.cu_seqlens ? a.T : (long long)a.B * a.T;
  CUtensorMap tm_q, tm_k, tm_v;
  if (!encode_rows(&tm_q, a.q, rows, (long long)a.Hk * kD, a.ldq) ||
      !encode_rows(&tm_k, a.k, rows, (long long)a.Hk * kD, a.ldk) ||
      !encode_rows(&tm_v, a.v, rows, (long long)a.Hv * kD, a.ldv))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(linattn_chunked_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e == cudaSuccess && a.nseg > 1) {
    e = cudaFuncSetAttribute(linattn_chunked_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    linattn_chunked_kernel<true><<<(unsigned)((long long)a.B * a.Hv * (a.nseg - 1)), kThreads, kSmem, s>>>(a, tm_q, tm_k, tm_v);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  linattn_chunked_kernel<false><<<(unsigned)((long long)a.B * a.Hv * a.nseg), kThreads, kSmem, s>>>(a, tm_q, tm_k, tm_v);
  return cudaGetLastError();
}

}  // namespace gdn
