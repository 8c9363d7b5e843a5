// linattn_chunked.cu -- linear attention with a decay for each head over
// prompts (bf16 io), in chunks of 64 tokens on the tcgen05 tensor cores.
//
// With G_i the sum of the log decays of the chunk's tokens up to i, the
// recurrence S_t = e^{g_t} S_{t-1} + v_t k_t^T, o_t = S_t q_t becomes, kept
// value-major (S[v][k]) and with tokens along the columns,
//   O^T = e^{F_i} (S Q^T + V^T P^T),  P_ij = e^{G_i - F_i - G_j} q_i . k_j (j <= i),
//   S'  = e^{G_last} S + (Gamma V)^T K,  Gamma_j = e^{G_last - G_j},
// with F_i = max(G_i, -58 ln 2), so that one accumulator takes both products of an
// output: P grows to 2^58 at most, and an output of a token further below the chunk's
// start sees 2^-58 of the state where it should see less.  Only S Q^T
// and the sum of S' carry the state: the products P, V^T P^T and (Gamma V)^T K of a
// chunk do not wait for it.
//
// One CTA walks the chunks of one (sequence, value head, segment):
//   warp 20      TMA: q, k, v tiles into a 4-stage ring
//   warp 21      issues the MMAs
//   warp 22      the chunk's decays
//   warps 16-19  (Gamma V)^T from shared memory into TMEM (a transposing load
//                hands each thread the words that its TMEM lanes hold)
//   warps 8-11   P from TMEM into shared memory
//   warps 0-7    the state, fp32 in registers: copies it to TMEM as the MMA
//                operand, then adds the chunk's update
//   warps 12-15  the output
// Precision: bf16 holds 8 significant bits, so what is not bf16 already goes
// to the MMA as a sum of bf16 pieces.  P and S, which feed the bf16 output
// only, take two (16 bits).  Gamma V feeds the carried fp32 state and takes
// four, which packed bf16 arithmetic forms without a conversion: with
// Gamma = c0 + c1 + c2 in bf16, v c0 = fl(v c0) + fma(v, c0, -fl(v c0)) exactly,
// v c1 likewise, and the last rest takes v c2 along (24 bits in all).  Every
// product starts from a zero accumulator and the state is summed in fp32
// registers, because an MMA truncates what it adds to.
//
// Few units (sequences x value heads) leave SMs idle, so a sequence can be cut
// into segments: a first launch (kStateOnly) forms the state of each segment's
// parts from zero, a small one turns those into the state before every segment,
// and a third starts every segment from its own.  Cost: k and v are read twice.
//
// Bound: a chunk of 64 tokens takes about 3,400 cycles of its SM, of which the
// tensor pipe works 51 % and instruction issue 54 %; what paces it is the chain
// update -> P and Gamma V -> next update and the MMAs in their order, not memory
// (calls of 4 x 8192 tokens, 16/32 heads: 256 us, 3.2 TB/s of the 0.82 GB that they
// cannot do without, where a copy runs at 6.8; of 65536 tokens, 16/48 heads: 940).
// The state-only form is paced by Gamma V and by adding the update (tensor pipe
// 32 %, issue 30 %).  Measured and not taken, against 240 us of an earlier form: two
// issuing warps (256 us), all of an iteration's waits before its first MMA (251),
// Q K^T after the output's products (271) or between them (246).  The loops of the
// roles share one instruction cache: a form with 82 KB of code instead of 58 (61
// now) waited for instructions in a third of its samples and took 1.4 times as long.
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
constexpr int kStages = 4;
constexpr int kVecs = 8;  // chunk vectors in flight (the output warps lag the loads by less)
constexpr int kFloor = -58;  // of the sum of a chunk's log2 decays in front of an output (above)
constexpr float kMinLogDecay = -80.f;  // a decay below e^-80 acts as e^-80: sums of it stay finite

constexpr uint32_t kTile = kC * kD * 2;             // 16 KB: 64 tokens x 128
constexpr uint32_t kStageBytes = 3 * kTile;         // q, k, v
constexpr uint32_t kP = kStages * kStageBytes;      // P, two pieces of 8 KB
constexpr uint32_t kPTile = kC * kC * 2;
constexpr uint32_t kShared = kP + 2 * kPTile;

struct ChunkVec {
  // Sums of the log2 decays from the chunk's first token, G = n + f with n whole
  // and 0 <= f <= 1: (-n, -n, -f, -f) of the tokens 2 i, 2 i + 1.  The ratio of two
  // decays is 2 to a difference of sums that may be thousands: in one fp32 number
  // each, 40 decays of e^-80 would leave the ratio of those behind them 10 bits.
  float4 G[kC / 2];
  float eF[kC];  // scale 2^F, F = max(G, kFloor)
  // e^{G_last - G} of the tokens 2 i, 2 i + 1 as bf16 pairs (c0, 0) and (c1, c2)
  // with c0 + c1 + c2 = it to 24 bits; 0 past the sequence's end
  uint2 gam[2][kC / 2];
  Decay d;       // e^{G_last}
  float total;   // G_last (natural)
  float pad;
};
struct Shared {
  ChunkVec vec[kVecs];
  uint64_t full[kStages], empty[kStages];
  uint64_t qk_done, p_loaded, p_ready, gv_ready[2], su_half[2], su_done[2], ds_free[2], s_ready, o_done, o_free, end;
  uint32_t tmem;
  int unit, seg;  // for the state's warps, whose registers are full
};
constexpr uint32_t kSmem = kShared + ((sizeof(Shared) + 127) / 128) * 128 + 1024;
static_assert(kSmem <= 232448, "shared memory per CTA");

// Six warpgroups; warp 23 only takes part in barriers.
// Registers per thread: launched with 80, then split by what a group holds
// (256 x 136 + 128 x (64 + 56 + 56 + 32) = 768 x 80; P with 56 and the last
// group with 40: 4 x 8192 tokens take 258 us, so 256).
constexpr int kThreads = 24 * 32;
constexpr int kRegsState = 136, kRegsP = 64, kRegsOut = 56, kRegsGv = 56, kRegsIssue = 32;
static_assert(256 * kRegsState + 128 * (kRegsP + kRegsOut + kRegsGv + kRegsIssue) <= kThreads * 80, "register split");
// TMEM columns (fp32, or bf16 pairs for the operands): all 512 are used.  The
// state-only form double-buffers both the update and Gamma V.
constexpr uint32_t kTDs = 0, kTSh = 128, kTSl = 192, kTO = 256, kTP = 320, kTG = 384;
constexpr int kPieces = 4;
template <bool kStateOnly>
__device__ __forceinline__ uint32_t ds_col(int n) { return kStateOnly && (n & 1) ? 128u : kTDs; }
template <bool kStateOnly>
__device__ __forceinline__ uint32_t gv_col(int n) { return kStateOnly && (n & 1) ? 256u : kTG; }

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
template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
__device__ __forceinline__ float ex2(float x) {  // 2^x to about 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The bf16 pair nearest to x; x keeps the rest.
__device__ __forceinline__ uint32_t take_bf16(float2 &x) {
  const uint32_t w = pack_bf16(x.x, x.y);
  x = __ffma2_rn(make_float2(lo_f(w), hi_f(w)), make_float2(-1.f, -1.f), x);
  return w;
}
// Packed bf16 products: rounded once, exact where the result fits.
__device__ __forceinline__ uint32_t bf16_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// 16 consecutive 32-bit columns of this warp's 32 lanes, without the wait.
__device__ __forceinline__ void tmem_ld16_nw(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

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

// Four 8 x 8 bf16 matrices of shared memory, transposed: lane L gives the
// address of row L % 8 of matrix L / 8 and gets, of each, the word
// (rows 2 (L % 4), + 1) of column L / 4 (a: matrix 0, .. d: matrix 3).
__device__ __forceinline__ void ldsm4t(uint32_t saddr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(saddr));
}
// 16 columns of 16 lanes: register 2 b + r holds column 4 b + lane % 4 of row lane / 4 + 8 r.
__device__ __forceinline__ void tmem_st16x16(uint32_t taddr, const uint32_t (&w)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]));
}

// Warp-wide wait, bounded to a second; short, because it is inlined often and
// the roles' loops together have to stay within the instruction cache.
__device__ __forceinline__ uint32_t global_ns_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
  bool ok = bar_try_wait(bar, parity);
  if (!ok) {
    const uint32_t t0 = global_ns_lo();
#pragma unroll 1
    do ok = bar_try_wait(bar, parity);
    while (!ok && global_ns_lo() - t0 < 1000000000u);
  }
  return __all_sync(0xffffffffu, ok);
}
// Two barriers: both are looked at before either answer is needed.
__device__ __forceinline__ bool warp_wait2(uint64_t *bar0, uint32_t parity0, uint64_t *bar1, uint32_t parity1) {
  bool ok0 = bar_try_wait(bar0, parity0), ok1 = bar_try_wait(bar1, parity1);
  if (!(ok0 && ok1)) {
    const uint32_t t0 = global_ns_lo();
#pragma unroll 1
    do {
      ok0 = ok0 || bar_try_wait(bar0, parity0);
      ok1 = ok1 || bar_try_wait(bar1, parity1);
    } while (!(ok0 && ok1) && global_ns_lo() - t0 < 1000000000u);
  }
  return __all_sync(0xffffffffu, ok0 && ok1);
}
// One arrival per warp, behind all of its lanes.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar);
}

// The decays of a chunk, by one warp: lane L holds tokens L and L + 32.
__device__ __forceinline__ void chunk_vec(ChunkVec &cv, float g0, float g1, float scale, int len, int lane) {
  // Sums from the front, of log2 decays in units of 2^-48 (64 of them take 62 bits):
  // exact, so that those to the chunk's end, their differences, are as well.
  constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
  using Fixed = unsigned long long;
  Fixed p0 = (Fixed)__float2ll_rn(g0 * kLog2e * 0x1p48f), p1 = (Fixed)__float2ll_rn(g1 * kLog2e * 0x1p48f);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Fixed a = __shfl_up_sync(0xffffffffu, p0, off), b = __shfl_up_sync(0xffffffffu, p1, off);
    if (lane >= off) p0 += a, p1 += b;
  }
  p1 += __shfl_sync(0xffffffffu, p0, 31);
  const Fixed last = __shfl_sync(0xffffffffu, p1, 31);
  // A NaN, which whole numbers do not hold, gets into the outputs from its token on by eF, into the state by d.
  const unsigned nan0 = __ballot_sync(0xffffffffu, g0 != g0), nan1 = __ballot_sync(0xffffffffu, g1 != g1);
  const unsigned upto = 0xffffffffu >> (31 - lane);
  const float nan = __int_as_float(0x7fc00000);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    const Fixed p = i ? p1 : p0;
    const int n = (int)((long long)p >> 48);
    const float f = (float)(unsigned)(p >> 16) * 0x1p-32f;
    float *G = reinterpret_cast<float *>(&cv.G[t >> 1]) + (t & 1);
    G[0] = (float)-n;
    G[2] = -f;
    const bool bad = i ? nan0 || (nan1 & upto) : nan0 & upto;
    const float eF = n < kFloor ? scale * 0x1p-58f : scale * ex2(f) * __int_as_float((min(n, 128) + 127) << 23);
    cv.eF[t] = bad ? nan : eF;
    const float x = t < len ? expf((float)(long long)(last - p) * (kLn2 * 0x1p-48f)) : 0.f;
    const __nv_bfloat16 g0 = __float2bfloat16_rn(x);
    const __nv_bfloat16 g1 = __float2bfloat16_rn(x - __bfloat162float(g0));
    const __nv_bfloat16 g2 = __float2bfloat16_rn(x - __bfloat162float(g0) - __bfloat162float(g1));
    __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(&cv.gam[0][t >> 1]) + (t & 1);
    to[0] = g0;
    to[2] = __float2bfloat16_rn(0.f);
    to[4 * (kC / 2)] = g1;
    to[4 * (kC / 2) + 2] = g2;
  }
  if (lane == 0) {
    cv.total = nan0 | nan1 ? nan : (float)(long long)last * (kLn2 * 0x1p-48f);
    cv.d = Decay::of(cv.total);
  }
}

template <bool kStateOnly>
__global__ void __launch_bounds__(kThreads, 1)
    linattn_chunked_kernel(const LinAttnArgs a, const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  Shared &B = *reinterpret_cast<Shared *>(sm + kShared);
  const uint32_t sbase = smem_u32(sm);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  // ---- the work of this CTA; consecutive CTAs are the heads of one segment
  // A segment is a.sub parts of `per` chunks; the state-only launch has a CTA
  // for each part of all segments but the last.
  const int launched_seg = kStateOnly ? (a.nseg - 1) * a.sub : a.nseg;
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
  const int nch = (T + kC - 1) / kC, per = (nch + a.nseg * a.sub - 1) / (a.nseg * a.sub);
  const int len_seg = kStateOnly ? per : per * a.sub;
  const int c0 = min(nch, seg * len_seg), c1 = min(nch, c0 + len_seg);
  const int n_chunks = c1 - c0;
  constexpr long long kState = kD * kD;

  // The log decays of chunk c, tokens lane and lane + 32; the first chunk's are
  // asked for before anything else.
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
    if (g0 < kMinLogDecay) g0 = kMinLogDecay;  // a NaN stays one
    if (g1 < kMinLogDecay) g1 = kMinLogDecay;
  };
  float g0 = 0.f, g1 = 0.f;
  if (warp == 22 && n_chunks > 0) load_g(c0, g0, g1);

  if (tid == 0) {
    auto bar_init = [](uint64_t *bar, uint32_t count) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
    };
    for (int s = 0; s < kStages; ++s) {
      bar_init(&B.full[s], 2);
      bar_init(&B.empty[s], 1);
    }
    bar_init(&B.qk_done, 1);
    bar_init(&B.p_loaded, 4);
    bar_init(&B.p_ready, 4);
    for (int i = 0; i < 2; ++i) {
      bar_init(&B.gv_ready[i], 4);
      bar_init(&B.su_half[i], 1);
      bar_init(&B.su_done[i], 1);
      bar_init(&B.ds_free[i], 8);
    }
    bar_init(&B.s_ready, 8);
    bar_init(&B.o_done, 1);
    bar_init(&B.o_free, 4);
    bar_init(&B.end, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");  // one for all of them
    B.unit = unit;
    B.seg = seg;
  }
  if (warp == 20 && lane < 3) {
    const CUtensorMap *map = lane == 0 ? &tm_k : lane == 1 ? &tm_v : &tm_q;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  if (warp == 21) tmem_alloc(&B.tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, B.tmem, 0);  // known to be the same in every lane
  bool ok = true;

  // ---- Gamma V of the chunks first, first + step, ..: 32 tokens x 16 value indices of a warp's 32 at a time
  auto gamma_v = [&](int first, int step) {
    const int j = tid & 63, half = (tid >> 6) & 1;
    const uint32_t jrow = (uint32_t)(half * (kTile / 2) + (j >> 3) * 1024 + (j & 7) * 128);
    const int w = warp & 3;  // TMEM quarter: value indices 32 w .. 32 w + 31
    const uint32_t tw = tmem + ((uint32_t)(32 * w) << 16);
    // This lane's row of the transposing loads: token lane % 8 (+ 8), value indices 8 (4 w + lane / 8 % 2) ..
    const uint32_t vrow = (uint32_t)((lane >> 4) * 1024 + (lane & 7) * 128);
    const int vchunk = 4 * w + ((lane >> 3) & 1), cc = 2 * (lane & 3);
    for (int n = first; n < n_chunks; n += step) {
      const int s = n % kStages;
      const ChunkVec &cv = B.vec[n % kVecs];
      const int len = T - (c0 + n) * kC;
      ok = warp_wait(&B.full[s], (n / kStages) & 1);
      // the update that read these columns
      if (kStateOnly) {
        if (n > 1) ok = ok && warp_wait(&B.su_done[n & 1], ((n >> 1) & 1) ^ 1);
      } else {
        if (n > 0) ok = ok && warp_wait(&B.su_half[(n - 1) & 1], ((n - 1) >> 1) & 1);
      }
      if (!ok) break;
      fence_after();
      if (j >= len) {  // rows past the end (another sequence's, or none) must count as 0, whatever they hold
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          *reinterpret_cast<uint4 *>(sm + s * kStageBytes + kTile + jrow + 16 * c) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(sm + s * kStageBytes + 2 * kTile + jrow + 16 * c) = make_uint4(0, 0, 0, 0);
        }
      }
      __syncwarp();  // the transposing loads and TMEM stores take the whole warp together
      const uint32_t vbase = sbase + s * kStageBytes + 2 * kTile + vrow;
      // Two pieces at a time, the small ones first: the last update has read those.
#pragma unroll 1
      for (int pass = 1; pass >= 0; --pass) {
        if (pass == 0 && !kStateOnly && n > 0) {
          ok = warp_wait(&B.su_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
          if (!ok) break;
          fence_after();
        }
#pragma unroll 1
        for (int jh = 0; jh < 2; ++jh) {
          uint32_t v[2][8];
#pragma unroll
          for (int vh = 0; vh < 2; ++vh) {
            const int ch = vchunk + 2 * vh;
            const uint32_t at = vbase + (uint32_t)((ch >> 3) * (kTile / 2) + (((ch & 7) ^ (lane & 7)) << 4) + jh * 4096);
            ldsm4t(at, v[vh][0], v[vh][1], v[vh][2], v[vh][3]);
            ldsm4t(at + 2048, v[vh][4], v[vh][5], v[vh][6], v[vh][7]);
          }
          if (len < kC) {  // rows past the end are being zeroed by other threads
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int token = 32 * jh + 8 * ((i & 7) >> 1) + cc;
              uint32_t &x = v[i >> 3][i & 7];
              x = token + 1 < len ? x : token < len ? x & 0xffffu : 0u;
            }
          }
          uint2 g[4];  // the factors of this pass: (c0, 0) or (c1, c2)
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = cv.gam[pass][16 * jh + 4 * e + (lane & 3)];
          const uint32_t to = tw + gv_col<kStateOnly>(n) + (1 - pass) * kC + 16 * jh;
#pragma unroll
          for (int vh = 0; vh < 2; ++vh) {
            uint32_t a0[8], a1[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t x = v[vh][i];
              a1[i] = bf16_mul(x, g[i >> 1].x);
              a0[i] = bf16_fma(x, g[i >> 1].y, bf16_fma(x, g[i >> 1].x, a1[i] ^ 0x80008000u));
            }
            tmem_st16x16(to + ((uint32_t)(16 * vh) << 16), a0);
            tmem_st16x16(to + ((uint32_t)(16 * vh) << 16) + kC / 2, a1);
          }
        }
      }
      if (!ok) break;
      tmem_wait_st();
      fence_before();
      fence_smem_to_async();
      warp_arrive(&B.gv_ready[n & 1]);
    }
  };

  if (warp >= 20) {
    regs_dec<kRegsIssue>();
    if (warp == 20) {
      // ---- TMA producer
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
      }
      // Leave only when every tile issued has been consumed (bounded).
      for (int j = max(0, n - kStages); ok && j < n; ++j)
        if (!warp_wait(&B.empty[j % kStages], (j / kStages) & 1)) ok = false;
    } else if (warp == 21) {
      // ---- MMA issuer (the whole warp; lane 0 issues)
      const uint32_t id_p = idesc_bf16(64, 64, 0, 0);     // Q K^T
      const uint32_t id_o1 = idesc_bf16(128, 64, 0, 0);   // S Q^T
      const uint32_t id_o2 = idesc_bf16(128, 64, 1, 0);   // V^T P^T
      const uint32_t id_su = idesc_bf16(128, 128, 0, 1);  // (Gamma V)^T K
      auto issue_qk = [&](int s) {
        const uint32_t q = sbase + s * kStageBytes, k = q + kTile;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)  // 64 of the 128 columns at a time
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_w(tmem + kTP, desc_k(q + kb * (kTile / 2), ks, kC), desc_k(k + kb * (kTile / 2), ks, kC), id_p, kb > 0 || ks > 0);
        commit_w(&B.qk_done);
      };
      auto issue_su = [&](int n) {
        const uint32_t k = sbase + (n % kStages) * kStageBytes + kTile;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {  // small pieces first
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_ta_w(tmem + ds_col<kStateOnly>(n), tmem + gv_col<kStateOnly>(n) + p * (kC / 2) + ks * 8, desc_mn(k, ks, kC),
                     id_su, p > 0 || ks > 0);
          if (p == 1 && !kStateOnly) commit_w(&B.su_half[n & 1]);  // the next chunk's may take their place
        }
        commit_w(&B.su_done[n & 1]);
      };
      if (n_chunks > 0) {
        ok = warp_wait(&B.full[0], 0);
        fence_after();
        if (ok && !kStateOnly) issue_qk(0);
        if (ok) ok = warp_wait(&B.gv_ready[0], 0);
        fence_after();
        if (ok) issue_su(0);
      }
      for (int n = 0; n < n_chunks && ok; ++n) {
        const int s = n % kStages, s1 = (n + 1) % kStages;
        const uint32_t par = n & 1;
        const bool more = n + 1 < n_chunks;
        if (!kStateOnly) {
          if (more) {  // the next P
            ok = warp_wait2(&B.full[s1], ((n + 1) / kStages) & 1, &B.p_loaded, par);
            fence_after();
            if (ok) issue_qk(s1);
          }
          ok = ok && warp_wait2(&B.p_ready, par, &B.o_free, par ^ 1);
          if (!ok) break;
          fence_after();
          const uint32_t q = sbase + s * kStageBytes, v = q + 2 * kTile;
#pragma unroll
          for (int p = 1; p >= 0; --p)
#pragma unroll
            for (int ks = 0; ks < kC / 16; ++ks)
              mma_w(tmem + kTO, desc_mn(v, ks, kC), desc_k(sbase + kP + p * kPTile, ks, kC), id_o2, p < 1 || ks > 0);
          ok = ok && warp_wait(&B.s_ready, par);
          if (!ok) break;
          fence_after();
#pragma unroll
          for (int p = 3; p >= 0; --p) {  // the second piece's two halves, then the first's
            const uint32_t qh = q + (p & 1) * (kTile / 2);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ta_w(tmem + kTO, tmem + kTSh + p * 32 + ks * 8, desc_k(qh, ks, kC), id_o1, 1);
          }
          commit_w(&B.o_done);
        }
        commit_w(&B.empty[s]);  // the update of chunk n was issued before
        if (more) {
          if (kStateOnly) ok = warp_wait(&B.full[s1], ((n + 1) / kStages) & 1);
          // Gamma V is there, and the columns that the update goes to have been read
          const int before = kStateOnly ? n - 1 : n;
          if (before >= 0)
            ok = ok && warp_wait2(&B.gv_ready[(n + 1) & 1], ((n + 1) >> 1) & 1, &B.ds_free[before & 1], (before >> 1) & 1);
          else
            ok = ok && warp_wait(&B.gv_ready[(n + 1) & 1], ((n + 1) >> 1) & 1);
          fence_after();
          if (ok) issue_su(n + 1);
        }
      }
      commit_w(&B.end);  // every MMA issued is complete before TMEM is freed
      if (!warp_wait(&B.end, 0)) ok = false;
    } else if (warp == 22) {
      // ---- the chunk vectors, each with its stage (a warp of their own on another
      // scheduler: with the TMA's warp 4 x 8192 tokens take 4 us more)
      for (int n = 0; n < n_chunks; ++n) {
        const int s = n % kStages, c = c0 + n;
        ok = warp_wait(&B.empty[s], ((n / kStages) & 1) ^ 1);
        if (!ok) break;
        chunk_vec(B.vec[n % kVecs], g0, g1, a.scale, T - c * kC, lane);
        warp_arrive(&B.full[s]);
        if (n + 1 < n_chunks) load_g(c + 1, g0, g1);
      }
    }
  } else if (warp >= 16) {
    regs_dec<kRegsGv>();
    gamma_v(0, kStateOnly ? 2 : 1);
  } else if (warp >= 8 && warp < 12) {
    regs_dec<kRegsP>();
    if (kStateOnly) {
      gamma_v(1, 2);
    } else {
      // ---- P, rows 16 w .. 16 w + 15 in TMEM quarter w
      const int w = warp - 8, i0 = 16 * w + (lane >> 2), cc = 2 * (lane & 3);
      uint8_t *prow = sm + kP + (i0 >> 3) * 1024 + (i0 & 7) * 128 + cc * 2;
      for (int n = 0; n < n_chunks; ++n) {
        const uint32_t par = n & 1;
        const ChunkVec &cv = B.vec[n % kVecs];
        ok = warp_wait(&B.full[n % kStages], (n / kStages) & 1) && warp_wait(&B.qk_done, par);
        if (!ok) break;
        fence_after();
        uint32_t r[32];
        tmem_ld16x64(tmem + ((uint32_t)(32 * w) << 16) + kTP, r);
        fence_before();
        warp_arrive(&B.p_loaded);
        // G - F of this thread's rows: 0 down to the floor, below it what is missing.
        float2 over[2];  // (whole part, fraction)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float *G = reinterpret_cast<const float *>(&cv.G[(i0 + 8 * q) >> 1]) + (i0 & 1);
          const bool below = -G[0] < (float)kFloor;
          over[q] = below ? make_float2(-G[0] - (float)kFloor, -G[2]) : make_float2(0.f, 0.f);
        }
        // r becomes the pieces: register 4 b + 2 q the first of row i0 + 8 q, the next one the second.
#pragma unroll
        for (int blk = 0; blk < 8; ++blk) {
          const int jc = 8 * blk + cc;
          const float4 gj = cv.G[jc >> 1];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = i0 + 8 * q;
            const float2 e = __fadd2_rn(__fadd2_rn(make_float2(over[q].x, over[q].x), make_float2(gj.x, gj.y)),
                                        __fadd2_rn(make_float2(over[q].y, over[q].y), make_float2(gj.z, gj.w)));
            float2 x = __fmul2_rn(make_float2(__uint_as_float(r[4 * blk + 2 * q]), __uint_as_float(r[4 * blk + 2 * q + 1])),
                                  make_float2(ex2(e.x), ex2(e.y)));
            if (jc > i) x.x = 0.f;
            if (jc + 1 > i) x.y = 0.f;
            r[4 * blk + 2 * q] = take_bf16(x);
            r[4 * blk + 2 * q + 1] = pack_bf16(x.x, x.y);
          }
        }
        if (n > 0) ok = warp_wait(&B.o_done, par ^ 1);  // the last output has read its P
        if (!ok) break;
#pragma unroll
        for (int blk = 0; blk < 8; ++blk) {
          uint8_t *dst = prow + ((blk ^ (i0 & 7)) << 4);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int p = 0; p < 2; ++p) *reinterpret_cast<uint32_t *>(dst + q * 1024 + p * kPTile) = r[4 * blk + 2 * q + p];
        }
        fence_smem_to_async();
        warp_arrive(&B.p_ready);
      }
    }
  } else if (warp < 8) {
    regs_inc<kRegsState>();
    // ---- the state: row v, columns 64 half .. 64 half + 63
    const int v = 32 * (warp & 3) + lane, half = warp >> 2;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const long long at = (long long)unit * kState + v * kD + 64 * half;
    const auto dec_at = [&](int slot, int u) -> float & {  // [slot][units]: the parts' log decays
      return a.ws[linattn_slots(a.nseg, a.sub) * units * kState + slot * units + u];
    };
    float S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
    if (kStateOnly) {
      // The call's S_T may be S0 itself: the second launch reads S0 from slot 0.
      if (seg == 0 && a.S0)
        for (int i = 0; i < 64; i += 4)
          *reinterpret_cast<float4 *>(a.ws + at + i) = *reinterpret_cast<const float4 *>(a.S0 + at + i);
    } else {
      const float *src = a.nseg == 1 ? a.S0 : seg > 0 || a.S0 ? a.ws + (long long)seg * a.sub * units * kState : nullptr;
      if (src) {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float4 x = *reinterpret_cast<const float4 *>(src + at + i);
          S[i] = x.x;
          S[i + 1] = x.y;
          S[i + 2] = x.z;
          S[i + 3] = x.w;
        }
      }
    }
    float total = 0.f;  // the log decay over the part
    uint32_t hi[32], lo[32];  // the state as two bf16 pieces
    auto pieces = [&]() {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float2 x = make_float2(S[2 * i], S[2 * i + 1]);
        hi[i] = take_bf16(x);
        lo[i] = pack_bf16(x.x, x.y);
      }
    };
    if (!kStateOnly) pieces();
    for (int n = 0; n < n_chunks; ++n) {
      const uint32_t par = n & 1;
      if (!kStateOnly) {
        if (n > 0) ok = warp_wait(&B.o_done, par ^ 1);  // the last output has read its state
        if (!ok) break;
        __syncwarp();
        tmem_st32w_nw(tl + kTSh + 32 * half, hi);
        tmem_st32w_nw(tl + kTSl + 32 * half, lo);
        tmem_wait_st();
        fence_before();
        warp_arrive(&B.s_ready);
      }
      ok = warp_wait(&B.su_done[n & 1], (n >> 1) & 1);
      if (!ok) break;
      fence_after();
      const Decay d = B.vec[n % kVecs].d;
      if (kStateOnly) total += B.vec[n % kVecs].total;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t r[16];
        tmem_ld16_nw(tl + ds_col<kStateOnly>(n) + 64 * half + 16 * i, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int x = 16 * i + 2 * e;
          const float2 y = d.apply(make_float2(S[x], S[x + 1]),
                                   make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])));
          S[x] = y.x;
          S[x + 1] = y.y;
        }
      }
      fence_before();
      warp_arrive(&B.ds_free[n & 1]);
      if (!kStateOnly) pieces();
    }
    // From here on with values read anew, so that none is held through the loop.
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    const int seg_ = *const_cast<volatile int *>(&B.seg), unit_ = *const_cast<volatile int *>(&B.unit);
    if (kStateOnly && t == 0) dec_at(seg_ + 1, unit_) = total;
    if (kStateOnly || seg_ == a.nseg - 1) {
      // Through shared memory, so that a warp stores whole rows: 16-byte piece c of
      // row v lies at piece c ^ (v % 32) there, and neither side has a bank
      // conflict.  The stages that the last chunk does not use are free.
      float4 *buf = reinterpret_cast<float4 *>(sm + (n_chunks > 0 && (n_chunks - 1) % kStages < 2 ? 2 * kStageBytes : 0));
      const int l = t & 31, row_ = t & 127, piece = t >> 7 << 4;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        buf[row_ * 32 + ((piece + i) ^ l)] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
      __syncwarp();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      float *dst = kStateOnly ? a.ws + (seg_ + 1) * units * kState : a.S_T;
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const int row = 16 * (t >> 5) + i;
        const long long to = (long long)unit_ * kState + row * kD + 4 * l;
        if (in_bounds(to + 4, units * kState, a.err))
          *reinterpret_cast<float4 *>(dst + to) = buf[row * 32 + (l ^ (row & 31))];
      }
    }
  } else {
    regs_dec<kRegsOut>();
    if (!kStateOnly) {
      // ---- the output: lane = value index, one column per token.  Neighbouring
      // lanes swap halves of a token pair, so that a lane stores two values of one
      // token: even lanes of the pair's first token, odd lanes of its second.
      const int v = 32 * (warp & 3) + lane;
      const bool odd = lane & 1;
      const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
      const long long o_size = ((a.cu_seqlens ? a.T : (long long)a.B * a.T) - 1) * a.ldo + (long long)a.Hv * kD;
      long long at = (row0 + (long long)c0 * kC + odd) * a.ldo + h * kD + (v & ~1);
      __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o);
      const uint32_t take = odd ? 0x3276 : 0x5410;  // (other's, own) high halves, or (own, other's) low halves
      for (int n = 0; n < n_chunks; ++n) {
        ok = warp_wait(&B.o_done, n & 1);
        if (!ok) break;
        fence_after();
        const ChunkVec &cv = B.vec[n % kVecs];
        const int len = T - (c0 + n) * kC - odd;  // this lane's tokens are those below it
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          uint32_t r[16];
          __syncwarp();  // lanes past the sequence's end skipped the stores
          tmem_ld16_nw(tl + kTO + 16 * i, r);
          tmem_wait_ld();
          if (i == 3) {
            fence_before();
            warp_arrive(&B.o_free);
          }
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 y = __fmul2_rn(*reinterpret_cast<const float2 *>(&cv.eF[16 * i + e]),
                                        make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])));
            const uint32_t own = pack_bf16(y.x, y.y), other = __shfl_xor_sync(0xffffffffu, own, 1);
            const uint32_t w = __byte_perm(own, other, take);
            if (16 * i + e < len && in_bounds(at + 2, o_size, a.err)) *reinterpret_cast<uint32_t *>(o + at) = w;
            at += 2 * a.ldo;
          }
        }
      }
    }
    }
  if (!ok && lane == 0) atomicOr(a.err, kErrTimeout);

  fence_before();
  __syncthreads();
  if (warp == 21) {
    fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The state before every segment but the first, in place of that of the part
// before it: S <- decay of the part S + its state from zero, from S0 on.
constexpr int kCombineThreads = 256;
__global__ void __launch_bounds__(kCombineThreads) linattn_combine_kernel(LinAttnArgs a) {
  const long long units = (long long)a.B * a.Hv, unit = blockIdx.y;
  const long long at = unit * kD * kD + 4 * (blockIdx.x * kCombineThreads + threadIdx.x), step = units * kD * kD;
  const int parts = (a.nseg - 1) * a.sub;
  const float *dec = a.ws + linattn_slots(a.nseg, a.sub) * step;  // log decays
  float4 S = a.S0 ? *reinterpret_cast<const float4 *>(a.ws + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAhead = 8;
  for (int m0 = 1; m0 <= parts; m0 += kAhead) {
    float4 x[kAhead];
    float d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (m0 + i <= parts) {
        x[i] = *reinterpret_cast<const float4 *>(a.ws + (m0 + i) * step + at);
        d[i] = dec[(m0 + i) * units + unit];
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (m0 + i <= parts) {
        const Decay e = Decay::of(d[i]);
        const float2 lo = e.apply(make_float2(S.x, S.y), make_float2(x[i].x, x[i].y));
        const float2 hi = e.apply(make_float2(S.z, S.w), make_float2(x[i].z, x[i].w));
        S = make_float4(lo.x, lo.y, hi.x, hi.y);
        if ((m0 + i) % a.sub == 0) *reinterpret_cast<float4 *>(a.ws + (m0 + i) * step + at) = S;
      }
  }
}

template <bool kStateOnly>
struct ChunkTag {};

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

// Microseconds, measured: a CTA's start and end, a chunk with its output, a
// chunk's state alone, a token of the recurrent kernel (one CTA per SM; above
// that by the unit).
namespace {
constexpr float kStart = 9.f, kChunkOut = 2.1f, kChunkState = 1.2f, kToken = 0.11f, kTokenUnit = 0.0033f;
}

LinAttnCut linattn_cut(int B, int Hv, long long tokens, bool packed, int sms) {
  const long long units = (long long)B * Hv;
  // The chunks of a sequence; of a packed batch, whose lengths the host does not
  // know, those of one three times the average.
  const long long len = packed ? (tokens < 3 * (tokens / B + 1) ? tokens : 3 * (tokens / B + 1)) : tokens / B;
  const long long nch = (len + kC - 1) / kC;
  LinAttnCut best{1, 1};
  float least = (float)((units + sms - 1) / sms) * (kStart + kChunkOut * nch);
  for (int n = 2; n <= kLinAttnMaxSeg && n <= nch && units * n <= 2LL * sms; ++n)
    for (int k = 1; k <= 3 && n * k <= nch; ++k) {
      const long long per = (nch + n * k - 1) / (n * k);
      const float out = (float)((units * n + sms - 1) / sms) * (kStart + kChunkOut * per * k);
      const float state = (float)((units * (n - 1) * k + sms - 1) / sms) * (kStart + kChunkState * per);
      if (out + state + 4.f < least) {  // 4: the launch between them
        least = out + state + 4.f;
        best = {n, k};
      }
    }
  return best;
}

bool linattn_recurrent_pays(int B, int Hv, long long longest, int sms) {
  const float units = (float)B * Hv, nch = (float)((longest + kC - 1) / kC);
  const float token = kToken > kTokenUnit * units ? kToken : kTokenUnit * units;
  const float waves = (float)(((long long)B * Hv + sms - 1) / sms);
  return 3.f + token * longest < waves * (kStart + kChunkOut * nch);
}

cudaError_t launch_linattn_chunked(const LinAttnArgs &a, cudaStream_t s) {
  const long long rows = a.cu_seqlens ? a.T : (long long)a.B * a.T;
  CUtensorMap tm_q, tm_k, tm_v;
  if (!encode_rows(&tm_q, a.q, rows, (long long)a.Hk * kD, a.ldq) ||
      !encode_rows(&tm_k, a.k, rows, (long long)a.Hk * kD, a.ldk) ||
      !encode_rows(&tm_v, a.v, rows, (long long)a.Hv * kD, a.ldv))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<ChunkTag<false>>(linattn_chunked_kernel<false>, kSmem);
  if (e == cudaSuccess && a.nseg > 1) {
    e = allow_smem<ChunkTag<true>>(linattn_chunked_kernel<true>, kSmem);
    if (e != cudaSuccess) return e;
    linattn_chunked_kernel<true><<<(unsigned)((long long)a.B * a.Hv * (a.nseg - 1) * a.sub), kThreads, kSmem, s>>>(a, tm_q, tm_k, tm_v);
    linattn_combine_kernel<<<dim3(kD * kD / (4 * kCombineThreads), (unsigned)(a.B * a.Hv)), kCombineThreads, 0, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  linattn_chunked_kernel<false><<<(unsigned)((long long)a.B * a.Hv * a.nseg), kThreads, kSmem, s>>>(a, tm_q, tm_k, tm_v);
  return cudaGetLastError();
}

}  // namespace gdn
