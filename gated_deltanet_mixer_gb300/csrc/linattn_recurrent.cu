// linattn_recurrent.cu -- linear attention with a decay for each head, token
// by token from the state (decode, and the prefill with fp32 io):
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t.
//
// Row i of S (value index i) needs only v_t[i], so the 128 rows are
// independent: a warp owns kRows of them in fp32 registers, lane L holding
// columns 4L .. 4L+3, and a CTA covers kWarps kRows rows of one
// (sequence, value head).  The state is read once and written once per call,
// whatever the number of tokens.  Tokens are copied kTB at a time into a ring in
// shared memory, three blocks ahead of the one worked on.
//
// One token is bound by the state's traffic, 128 KB per unit against 128 x 128
// fused multiply-adds (calls of 256 sequences x 48 heads on states in turn: 243 us,
// 6.65 TB/s, a copy's rate; 1 x 16 heads: 2.3 us on the device, 7.2 a call); a few
// tokens by that and by instruction issue (64 x 48 heads, 4 tokens: 76 us, 5.4
// TB/s); long runs of few units by a token's loads from shared memory, its
// arithmetic and its sums in turn: one warp per scheduler, which issues in 24 % of
// its cycles (2 x 1001 tokens, 8 heads, fp32: 111 us, 0.11 us per token).
//
// Figures with two forms below: launches in a graph, both on one box.
#include <type_traits>

#include "gdn_device.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kTB = 8;    // tokens per block
constexpr int kRing = 4;  // blocks in the ring

// Sums part[0 .. R) over the warp; lane L returns the total of part[L / (32 / R)].
template <int R>
__device__ __forceinline__ float reduce_rows(float (&part)[R], int lane) {
#pragma unroll
  for (int n = R, off = 16; off >= 1; off >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < R / 2; ++i)
        if (i < n) {
          const float send = upper ? part[i] : part[i + n];
          const float keep = upper ? part[i + n] : part[i];
          part[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    } else {
      part[0] += __shfl_xor_sync(0xffffffffu, part[0], off);
    }
  }
  return part[0];
}

__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// e^g s + v k
__device__ __forceinline__ float4 decayed(float4 s, Decay a, float v, float4 k) {
  const float2 v2 = make_float2(v, v);
  const float2 x = a.apply(make_float2(s.x, s.y), __fmul2_rn(v2, make_float2(k.x, k.y)));
  const float2 y = a.apply(make_float2(s.z, s.w), __fmul2_rn(v2, make_float2(k.z, k.w)));
  return make_float4(x.x, x.y, y.x, y.y);
}

// kGroup: tokens whose sums are reduced together.
template <typename IO, int kRows, int kGroup, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) linattn_recurrent_kernel(LinAttnArgs a) {
  constexpr int kThreads = kWarps * 32;
  constexpr int kSplit = kD / (kWarps * kRows);  // CTAs per unit
  constexpr int kCtaRows = kWarps * kRows;
  __shared__ __align__(16) IO s_q[kRing][kTB][kD], s_k[kRing][kTB][kD], s_v[kRing][kTB][kCtaRows];
  __shared__ Decay s_a[kRing][kTB];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / kSplit, part = blockIdx.x % kSplit;
  const int b = unit / a.Hv, h = unit % a.Hv, kh = h / (a.Hv / a.Hk);
  long long row0;
  int T;
  if (a.cu_seqlens) {
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
  const long long total_rows = a.cu_seqlens ? a.T : (long long)a.B * a.T;
  const int r0 = part * kCtaRows + warp * kRows;  // this warp's first state row

  constexpr int kPiece = 16 / sizeof(IO);  // values per 16-byte copy
  const IO *q = static_cast<const IO *>(a.q) + row0 * a.ldq + kh * kD;
  const IO *k = static_cast<const IO *>(a.k) + row0 * a.ldk + kh * kD;
  const IO *v = static_cast<const IO *>(a.v) + row0 * a.ldv + h * kD + part * kCtaRows;
  auto fetch = [&](int block) {  // copies block `block` into its place in the ring
    const int t0 = block * kTB, slot = block % kRing;
    constexpr int kWide = kD / kPiece, kNarrow = kCtaRows / kPiece;  // copies per row of q, k; of v
#pragma unroll
    for (int i = 0; i < kTB * kWide; i += kThreads) {
      const int t = (tid + i) / kWide, c = tid % kWide * kPiece;
      if (t < kTB && t0 + t < T) {
        copy16(&s_q[slot][t][c], q + (t0 + t) * a.ldq + c);
        copy16(&s_k[slot][t][c], k + (t0 + t) * a.ldk + c);
      }
    }
    const int tv = tid / kNarrow, cv = tid % kNarrow * kPiece;
    if (tv < kTB && t0 + tv < T) copy16(&s_v[slot][tv][cv], v + (t0 + tv) * a.ldv + cv);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  static_assert(kThreads % (kD / kPiece) == 0 && kTB * kCtaRows / kPiece <= kThreads, "copies");
  auto decay = [&](int t) { return a.g ? a.g[(row0 + t) * a.Hv + h] : a.log_decay[h]; };
  for (int b = 0; b < kRing - 1; ++b) fetch(b);
  if (tid < kTB * (kRing - 1) && tid < T) s_a[tid / kTB][tid % kTB] = Decay::of(decay(tid));
  const long long s_at = ((long long)unit * kD + r0) * kD + 4 * lane;
  float4 S[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    S[r] = a.S0 ? ld_stream(a.S0 + s_at + r * kD) : make_float4(0.f, 0.f, 0.f, 0.f);
  IO *o = static_cast<IO *>(a.o) + row0 * a.ldo + h * kD + r0;
  const long long o_size = (total_rows - 1) * a.ldo + (long long)a.Hv * kD;
  // N tokens from `t` on: their sums over the columns are reduced together, so
  // that the shuffles of one do not hold up the next one's update.
  auto tokens = [&](auto count, int buf, int t0, int t) {
    constexpr int N = decltype(count)::value;
    float p[N * kRows];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Decay al = s_a[buf][t + i];
      const float4 kv = ld_io4(&s_k[buf][t + i][4 * lane]);
      const float4 qv = ld_io4(&s_q[buf][t + i][4 * lane]);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        S[r] = decayed(S[r], al, ld_io(&s_v[buf][t + i][warp * kRows + r]), kv);
        // Groups of bf16 tokens: in packed pairs (64 x 48 heads, 4 tokens, CTAs of 8
        // warps of 4 rows: 74 us, 80 without; groups of fp32 tokens and single ones are slower with them).
        if (kGroup > 1 && sizeof(IO) == 2) {
          const float2 pq = __ffma2_rn(make_float2(S[r].x, S[r].y), make_float2(qv.x, qv.y),
                                       __fmul2_rn(make_float2(S[r].z, S[r].w), make_float2(qv.z, qv.w)));
          p[i * kRows + r] = pq.x + pq.y;
        } else {
          p[i * kRows + r] = dot4(S[r], qv);
        }
      }
    }
    const float sum = reduce_rows<N * kRows>(p, lane);
    constexpr int kPer = 32 / (N * kRows);  // lanes per sum
    const int i = lane / kPer / kRows, r = lane / kPer % kRows;
    const long long at = (long long)(t0 + t + i) * a.ldo + r;
    if (lane % kPer == 0 && in_bounds(row0 * a.ldo + h * kD + r0 + at + 1, o_size, a.err)) st_io(o + at, sum * a.scale);
  };
  for (int t0 = 0, block = 0; t0 < T; t0 += kTB, ++block) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");  // this block has landed
    __syncthreads();  // for every thread; and the block before this one is done with
    fetch(block + kRing - 1);
    const int next = t0 + (kRing - 1) * kTB + tid;
    float na = 0.f;
    if (tid < kTB && next < T) na = decay(next);  // used after this block's work
    const int n = min(kTB, T - t0), buf = block % kRing;
    int t = 0;
    if (kGroup > 1)
      for (; t + kGroup <= n; t += kGroup) tokens(std::integral_constant<int, kGroup>(), buf, t0, t);
    if (kGroup > 4)
      for (; t + 4 <= n; t += 4) tokens(std::integral_constant<int, 4>(), buf, t0, t);
    for (; t < n; ++t) tokens(std::integral_constant<int, 1>(), buf, t0, t);
    if (tid < kTB && next < T) s_a[(block + kRing - 1) % kRing][tid] = Decay::of(na);
  }
  const long long s_size = (long long)a.B * a.Hv * kD * kD;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (in_bounds(s_at + r * kD + 4, s_size, a.err)) st_stream(a.S_T + s_at + r * kD, S[r]);
}

template <typename IO, int kRows, int kGroup, int kWarps>
void launch(const LinAttnArgs &a, cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * a.Hv * (kD / (kWarps * kRows)));
  linattn_recurrent_kernel<IO, kRows, kGroup, kWarps><<<grid, kWarps * 32, 0, s>>>(a);
}

template <typename IO>
void launch_form(const LinAttnArgs &a, int num_sms, cudaStream_t s) {
  const long long units = (long long)a.B * a.Hv;
  const long long tokens = a.cu_seqlens ? a.T / a.B : a.T;  // of a sequence (packed: on average)
  // From four tokens on: CTAs of 4 warps, which drift apart, so that one's loads
  // from shared memory run beside another's arithmetic and sums; 8 rows per warp
  // where the units fill the SMs, else 4 rows and the sums of 8 tokens together.
  // (fp32, 2 x 1001 tokens, 8 heads: 102 us, with CTAs of 8 warps of 2 rows and
  // groups of 4 121; 4 x 1001, 12 heads: 186, with 8 warps of 4 rows 257, 4 warps of
  // 8 236; 16 x 256, 32 heads: 360 with 8 rows in groups of 4, 377 with 4 rows in
  // groups of 8, 407 with 8 warps of 4 rows; 64 x 48 heads, 4 tokens: 71, 74 with 8
  // warps of 4 rows.)
  if (tokens >= 4) {
    if (units < num_sms)
      launch<IO, 4, 8, 4>(a, s);
    else
      launch<IO, 8, 4, 4>(a, s);
    return;
  }
  // Up to three tokens are bound by the state's traffic: no groups, and the
  // registers of more CTAs per SM instead (64 x 48 heads, 3 tokens: 72 us, in
  // groups 75).  Few units: the rows of a unit over more CTAs (1 x 16 heads, one
  // token: 2.5 us with 2 rows per warp, 2.8 with 4, 3.0 with 8; 64 x 48 heads: 71,
  // 60, 61 us.)
  if (units * 4 <= num_sms)
    launch<IO, 2, 1, 8>(a, s);
  else
    launch<IO, 4, 1, 8>(a, s);
}

}  // namespace

cudaError_t launch_linattn_recurrent(const LinAttnArgs &a, bool bf16, int num_sms, cudaStream_t s) {
  if (bf16)
    launch_form<__nv_bfloat16>(a, num_sms, s);
  else
    launch_form<float>(a, num_sms, s);
  return cudaGetLastError();
}

}  // namespace gdn
