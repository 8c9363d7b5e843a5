// linattn_recurrent.cu -- linear attention with a decay for each head, token
// by token from the state (decode, and the prefill with fp32 io):
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t.
//
// Row i of S (value index i) needs only v_t[i], so the 128 rows are
// independent: a warp owns kRows of them in fp32 registers, lane L holding
// columns 4L .. 4L+3, and a CTA of 8 warps covers 8 kRows rows of one
// (sequence, value head).  The state is read once and written once per call,
// whatever the number of tokens.  Tokens are staged kTB at a time: while a
// block is worked on, the next one's q, k, v and decays are on their way into
// registers, then into the other half of a double buffer in shared memory.
//
// One token is bound by the state's traffic (128 KB per unit against 128 x 128
// fused multiply-adds); long runs by the fp32 multiply-adds.
#include "gdn_device.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTB = 8;  // tokens staged at a time: one 4-wide load of q and of k per thread

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

__device__ __forceinline__ float4 decayed(float4 s, float a, float v, float4 k) {
  const float2 x = __ffma2_rn(make_float2(a, a), make_float2(s.x, s.y),
                              __fmul2_rn(make_float2(v, v), make_float2(k.x, k.y)));
  const float2 y = __ffma2_rn(make_float2(a, a), make_float2(s.z, s.w),
                              __fmul2_rn(make_float2(v, v), make_float2(k.z, k.w)));
  return make_float4(x.x, x.y, y.x, y.y);
}

template <typename IO, int kRows>
__global__ void __launch_bounds__(kThreads) linattn_recurrent_kernel(LinAttnArgs a) {
  constexpr int kSplit = kD / (kWarps * kRows);  // CTAs per unit
  constexpr int kCtaRows = kWarps * kRows;
  __shared__ __align__(16) float s_q[2][kTB][kD], s_k[2][kTB][kD];
  __shared__ __align__(16) float s_v[2][kTB][kCtaRows];
  __shared__ float s_a[2][kTB];
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

  // This thread's share of a block's staging: token tb, columns c4 .. c4 + 3 of q and k.
  const int tb = tid / (kD / 4), c4 = 4 * (tid % (kD / 4));
  constexpr int kVLoads = kTB * kCtaRows / 4;  // 4-wide loads of v (at most one per thread)
  static_assert(kVLoads <= kThreads, "v staging");
  const int vb = tid / (kCtaRows / 4), v4 = 4 * (tid % (kCtaRows / 4));
  const IO *q = static_cast<const IO *>(a.q) + row0 * a.ldq + kh * kD;
  const IO *k = static_cast<const IO *>(a.k) + row0 * a.ldk + kh * kD;
  const IO *v = static_cast<const IO *>(a.v) + row0 * a.ldv + h * kD + part * kCtaRows;
  float4 nq, nk, nv;
  float na = 0.f;
  auto fetch = [&](int t0) {
    if (t0 + tb < T) {
      nq = ld_io4(q + (t0 + tb) * a.ldq + c4);
      nk = ld_io4(k + (t0 + tb) * a.ldk + c4);
    }
    if (tid < kVLoads && t0 + vb < T) nv = ld_io4(v + (t0 + vb) * a.ldv + v4);
    if (tid < kTB && t0 + tid < T) na = expf(a.g ? a.g[(row0 + t0 + tid) * a.Hv + h] : a.log_decay[h]);
  };
  auto stage = [&](int buf) {
    *reinterpret_cast<float4 *>(&s_q[buf][tb][c4]) = nq;
    *reinterpret_cast<float4 *>(&s_k[buf][tb][c4]) = nk;
    if (tid < kVLoads) *reinterpret_cast<float4 *>(&s_v[buf][vb][v4]) = nv;
    if (tid < kTB) s_a[buf][tid] = na;
  };
  nq = nk = nv = make_float4(0.f, 0.f, 0.f, 0.f);
  fetch(0);
  const long long s_at = ((long long)unit * kD + r0) * kD + 4 * lane;
  float4 S[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    S[r] = a.S0 ? ld_stream(a.S0 + s_at + r * kD) : make_float4(0.f, 0.f, 0.f, 0.f);
  stage(0);
  __syncthreads();
  IO *o = static_cast<IO *>(a.o) + row0 * a.ldo + h * kD + r0;
  const long long o_size = (total_rows - 1) * a.ldo + (long long)a.Hv * kD;
  for (int t0 = 0, buf = 0; t0 < T; t0 += kTB, buf ^= 1) {
    if (t0 + kTB < T) fetch(t0 + kTB);
    const int n = min(kTB, T - t0);
    for (int t = 0; t < n; ++t) {
      const float al = s_a[buf][t];
      const float4 kv = *reinterpret_cast<const float4 *>(&s_k[buf][t][4 * lane]);
      const float4 qv = *reinterpret_cast<const float4 *>(&s_q[buf][t][4 * lane]);
      float p[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        S[r] = decayed(S[r], al, s_v[buf][t][warp * kRows + r], kv);
        p[r] = dot4(S[r], qv);
      }
      const float sum = reduce_rows<kRows>(p, lane);
      constexpr int kPer = 32 / kRows;  // lanes per row
      const int r = lane / kPer;
      const long long at = (long long)(t0 + t) * a.ldo + r;
      if (lane % kPer == 0 && in_bounds(row0 * a.ldo + h * kD + r0 + at + 1, o_size, a.err)) st_io(o + at, sum * a.scale);
    }
    if (t0 + kTB < T) {
      stage(buf ^ 1);
      __syncthreads();
    }
  }
  const long long s_size = (long long)a.B * a.Hv * kD * kD;
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (in_bounds(s_at + r * kD + 4, s_size, a.err)) st_stream(a.S_T + s_at + r * kD, S[r]);
}

template <typename IO, int kRows>
void launch(const LinAttnArgs &a, cudaStream_t s) {
  const long long units = (long long)a.B * a.Hv;
  linattn_recurrent_kernel<IO, kRows><<<(unsigned)(units * (kD / (kWarps * kRows))), kThreads, 0, s>>>(a);
}

template <typename IO>
void launch_rows(const LinAttnArgs &a, int num_sms, cudaStream_t s) {
  // Few units: the rows of a unit over more CTAs, so that every SM has one.
  const long long units = (long long)a.B * a.Hv;
  if (units * 4 <= num_sms)
    launch<IO, 2>(a, s);
  else if (units <= num_sms)
    launch<IO, 4>(a, s);
  else
    launch<IO, 8>(a, s);
}

}  // namespace

cudaError_t launch_linattn_recurrent(const LinAttnArgs &a, bool bf16, int num_sms, cudaStream_t s) {
  if (bf16)
    launch_rows<__nv_bfloat16>(a, num_sms, s);
  else
    launch_rows<float>(a, num_sms, s);
  return cudaGetLastError();
}

}  // namespace gdn
