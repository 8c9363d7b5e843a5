// rope.cu -- rotary positions: the pair (a, b) of index i at position p becomes
//   m (a cos x - b sin x, b cos x + a sin x),   x = p f_i.
// The angle is kept as a 64-bit fraction of a turn, p * turns_i modulo 2^64: the
// integer product rounds nothing, however large p is.  What it has beyond the
// nearest quarter, an eighth of a turn at most, goes through fp32 to sincospi: within
// 2^-28 of a turn.
//
// Bound by memory traffic (in place that of the rotated elements alone; 8192 tokens,
// 28 heads, 64 of 256 elements, 59 MB: 12 us, 13 where they come from memory, 4.5 to 4.9 TB/s) and
// by instruction issue (49% active).  A block
// first forms the cosines and sines of its tokens, which all heads share; then
// its threads take items of 16 bytes (or, where an address or a width does not
// allow that, single pairs), two at a time, the first two asked for before that.
#include <algorithm>

#include "cache_device.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 2;

// n / d for n < 2^22, d <= 2^10 (and for n < d <= 2^11): n m / 2^32 with m = floor(2^32 / d) + 1 is too large by
// n (m d - 2^32) / (d 2^32) <= n / 2^32 < 1 / d.  (heads <= 2^12, D <= 2^10; a block of several tokens has at most 2^11
// items.)
struct FastDiv {
  uint32_t d, m;
};
FastDiv fast_div(uint32_t d) { return FastDiv{d, d == 1 ? 0u : (uint32_t)((1ull << 32) / d + 1)}; }
__device__ __forceinline__ uint32_t quotient(uint32_t n, FastDiv f) { return f.d == 1 ? n : __umulhi(n, f.m); }

struct Items {
  FastDiv of_token;            // items of a token, over all tensors
  FastDiv of_head[kRopeMaxX];  // of a head: pairs' vectors, then (out of place) those of the elements that stay
  int begin[kRopeMaxX];        // a tensor's first item of a token
  int rot;                     // items of a head that turn
  int per_block;               // tokens
  int pair_threads;            // of a token's angles: a power of two
};

template <bool kBf16, bool kVec, int kPairs>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Items n, const __grid_constant__ RopeTurns<kPairs> turns) {
  using X = Io<kBf16>;
  using T = typename X::T;
  constexpr int V = kVec ? X::V : 1;
  extern __shared__ float2 turn[];  // [per_block][rot / 2]: m cos, m sin
  const int pairs = a.rot >> 1;
  const int t0 = blockIdx.x * n.per_block, nt = min(n.per_block, a.tokens - t0);
  const uint32_t total = (uint32_t)nt * n.of_token.d;
  const T *src[kAtOnce];
  T *dst[kAtOnce];
  int what[kAtOnce];  // the item of its head, -1: none
  uint32_t token[kAtOnce];
  uint4 lo[kAtOnce], hi[kAtOnce];
  auto load = [&](uint32_t it0) {
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t it = it0 + u * kThreads;
      what[u] = -1;
      if (it >= total) continue;
      const uint32_t t = nt == 1 ? 0 : quotient(it, n.of_token), r = it - t * n.of_token.d;
      const int xi = ((int)r >= n.begin[1]) + ((int)r >= n.begin[2]) + ((int)r >= n.begin[3]);
      const FastDiv of_head = xi == 0 ? n.of_head[0] : xi == 1 ? n.of_head[1] : xi == 2 ? n.of_head[2] : n.of_head[3];
      const uint32_t in = r - (xi == 0 ? n.begin[0] : xi == 1 ? n.begin[1] : xi == 2 ? n.begin[2] : n.begin[3]);
      const uint32_t h = quotient(in, of_head);
      const int j = (int)(in - h * of_head.d);
      // chosen by comparisons: lanes that index the parameters each with its own number would take turns
      const RopeX x = xi == 0 ? a.x[0] : xi == 1 ? a.x[1] : xi == 2 ? a.x[2] : a.x[3];
      src[u] = static_cast<const T *>(x.x) + (long long)(t0 + t) * x.ldx + (long long)h * a.D;
      dst[u] = static_cast<T *>(x.y) + (long long)(t0 + t) * x.ldy + (long long)h * a.D;
      what[u] = j;
      token[u] = t;
      if constexpr (kVec) {
        const int at = j < n.rot ? j * V : a.rot + (j - n.rot) * V;
        lo[u] = *reinterpret_cast<const uint4 *>(src[u] + at);
        if (!a.interleaved && j < n.rot) hi[u] = *reinterpret_cast<const uint4 *>(src[u] + pairs + at);
      }
    }
  };
  load(threadIdx.x);  // on the way while the angles are formed
  // A thread keeps to one pair: its frequency is read once (lanes that read different parameters take turns).
  const int wide = n.pair_threads, i = threadIdx.x & (wide - 1);
  if (i < pairs) {
    const unsigned long long f = turns.at[i];
    for (int t = threadIdx.x / wide; t < nt; t += kThreads / wide) {
      const unsigned long long x = (unsigned long long)(long long)a.positions[t0 + t] * f;
      const uint32_t quarter = (uint32_t)((x + (1ull << 61)) >> 62);  // the nearest quarter of a turn; what is left is small
      float s, c;
      sincospif((float)(int)((x - ((unsigned long long)quarter << 62) + (1ull << 31)) >> 32) * 0x1p-31f, &s, &c);
      const float c1 = quarter & 1 ? -s : c, s1 = quarter & 1 ? c : s, m = quarter & 2 ? -a.m : a.m;
      turn[t * pairs + i] = make_float2(m * c1, m * a.sign * s1);
    }
  }
  __syncthreads();
  for (uint32_t it0 = threadIdx.x; it0 < total; it0 += kThreads * kAtOnce) {
    if (it0 != threadIdx.x) load(it0);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int j = what[u];
      if (j < 0) continue;
      T *const y = dst[u];
      const float2 *const cs = turn + token[u] * pairs;
      if constexpr (kVec) {
        if (j >= n.rot) {
          *reinterpret_cast<uint4 *>(y + a.rot + (j - n.rot) * V) = lo[u];
        } else if (a.interleaved) {
          float x[V], w[V];
          X::unpack(lo[u], x);
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float2 f = cs[(j * V + i) >> 1];
            w[i] = x[i] * f.x - x[i + 1] * f.y;
            w[i + 1] = x[i + 1] * f.x + x[i] * f.y;
          }
          X::store(y + j * V, w);
        } else {
          float x[V], w[V];
          X::unpack(lo[u], x);
          X::unpack(hi[u], w);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 f = cs[j * V + i];
            const float p = x[i] * f.x - w[i] * f.y;
            w[i] = w[i] * f.x + x[i] * f.y;
            x[i] = p;
          }
          X::store(y + j * V, x);
          X::store(y + pairs + j * V, w);
        }
      } else if (j >= n.rot) {
        y[a.rot + j - n.rot] = src[u][a.rot + j - n.rot];
      } else {
        const int ia = a.interleaved ? 2 * j : j, ib = a.interleaved ? 2 * j + 1 : j + pairs;
        const float x = X::get(src[u] + ia), w = X::get(src[u] + ib);
        const float2 f = cs[j];
        X::put(y + ia, x * f.x - w * f.y);
        X::put(y + ib, w * f.x + x * f.y);
      }
    }
  }
}

template <bool kBf16, bool kVec, int kPairs>
cudaError_t launch(const RopeArgs &a, const unsigned long long *turns, int num_sms, cudaStream_t s) {
  constexpr int V = kVec ? Io<kBf16>::V : 1;
  Items n{};
  n.rot = !kVec ? a.rot / 2 : a.interleaved ? a.rot / V : a.rot / (2 * V);
  int all = 0;
  for (int i = 0; i < a.n_x; ++i) {
    const int of_head = n.rot + (a.x[i].x == a.x[i].y ? 0 : (a.D - a.rot) / V);
    n.of_head[i] = fast_div(of_head);
    n.begin[i] = all;
    all += a.x[i].heads * of_head;
  }
  for (int i = a.n_x; i < kRopeMaxX; ++i) n.begin[i] = all;  // nothing is there
  n.of_token = fast_div(all);
  // Tokens of a block: what its threads take at once, if that leaves the GPU enough blocks.
  const int want = std::max(1, kAtOnce * kThreads / all), spread = std::max(1, a.tokens / (4 * num_sms));
  n.per_block = std::min({want, spread, 32});
  for (n.pair_threads = 1; n.pair_threads < a.rot / 2;) n.pair_threads *= 2;
  const int blocks = (a.tokens + n.per_block - 1) / n.per_block;
  RopeTurns<kPairs> f{};
  std::copy(turns, turns + a.rot / 2, f.at);
  rope_kernel<kBf16, kVec, kPairs><<<blocks, kThreads, (size_t)n.per_block * (a.rot / 2) * sizeof(float2), s>>>(a, n, f);
  return cudaGetLastError();
}
template <bool kBf16, bool kVec>
cudaError_t launch(const RopeArgs &a, const unsigned long long *turns, int num_sms, cudaStream_t s) {
  return a.rot <= 64 ? launch<kBf16, kVec, 32>(a, turns, num_sms, s) : launch<kBf16, kVec, kRopeMaxPairs>(a, turns, num_sms, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, const unsigned long long *turns, bool bf16, int num_sms, cudaStream_t s) {
  return bf16 ? (a.vec ? launch<true, true>(a, turns, num_sms, s) : launch<true, false>(a, turns, num_sms, s))
              : (a.vec ? launch<false, true>(a, turns, num_sms, s) : launch<false, false>(a, turns, num_sms, s));
}

}  // namespace gdn
