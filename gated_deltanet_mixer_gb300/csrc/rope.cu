// rope.cu -- rotary positions: the pair (a, b) of index i at position p becomes
//   m (a cos x - b sin x, b cos x + a sin x),   x = p f_i.
// The angle is kept as a 64-bit fraction of a turn, p * turns_i modulo 2^64: an
// integer product has no error that grows with p, and its upper bits are the
// angle in [-pi, pi) to fp32's precision for sincospi.
//
// Bound by memory traffic: a block first forms the cosines and sines of its
// tokens (shared by all heads), then its threads take 16-byte vectors.
#include "cache_device.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int per_block) {
  using X = Io<kBf16>;
  using T = typename X::T;
  constexpr int V = kVec ? X::V : 1;
  extern __shared__ float2 turn[];  // [per_block][rot / 2]: m cos, m sin
  const int pairs = a.rot >> 1;
  const long long t0 = (long long)blockIdx.x * per_block;
  const int nt = (int)min((long long)per_block, a.tokens - t0);
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const unsigned long long f = (unsigned long long)(long long)a.positions[t0 + i / pairs] * a.turns[i % pairs];
    float s, c;
    sincospif((float)(long long)f * 0x1p-63f, &s, &c);
    turn[i] = make_float2(a.m * c, a.m * a.sign * s);
  }
  __syncthreads();
  // items of a head: vectors of pairs (half: V pairs from two places; interleaved: V elements), then, out of place,
  // vectors of the elements that stay
  const int items_rot = !kVec ? pairs : a.interleaved ? a.rot / V : pairs / V;
  const int items_all = items_rot + (a.D - a.rot) / V;
  int xi = 0, h0 = 0;
  const int total = nt * a.heads * items_all;
  for (int it = threadIdx.x; it < total; it += kThreads) {
    const int j = it % items_all, th = it / items_all, h = th % a.heads, t = th / a.heads;
    for (xi = 0, h0 = 0; h - h0 >= a.x[xi].heads; ++xi) h0 += a.x[xi].heads;
    const RopeX &r = a.x[xi];
    const T *const x = static_cast<const T *>(r.x) + (t0 + t) * r.ldx + (long long)(h - h0) * a.D;
    T *const y = static_cast<T *>(r.y) + (t0 + t) * r.ldy + (long long)(h - h0) * a.D;
    if (j >= items_rot) {
      if (x == y) continue;
      const int e = a.rot + (j - items_rot) * V;
      if constexpr (kVec)
        *reinterpret_cast<uint4 *>(y + e) = *reinterpret_cast<const uint4 *>(x + e);
      else
        y[e] = x[e];
      continue;
    }
    const float2 *const cs = turn + t * pairs;
    if constexpr (kVec) {
      float u[V], w[V];
      if (a.interleaved) {
        X::load(x + j * V, u);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 f = cs[(j * V + i) >> 1];
          w[i] = u[i] * f.x - u[i + 1] * f.y;
          w[i + 1] = u[i + 1] * f.x + u[i] * f.y;
        }
        X::store(y + j * V, w);
      } else {
        X::load(x + j * V, u);
        X::load(x + pairs + j * V, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 f = cs[j * V + i];
          const float p = u[i] * f.x - w[i] * f.y;
          w[i] = w[i] * f.x + u[i] * f.y;
          u[i] = p;
        }
        X::store(y + j * V, u);
        X::store(y + pairs + j * V, w);
      }
    } else {
      const int ia = a.interleaved ? 2 * j : j, ib = a.interleaved ? 2 * j + 1 : j + pairs;
      const float u = X::get(x + ia), w = X::get(x + ib);
      const float2 f = cs[j];
      X::put(y + ia, u * f.x - w * f.y);
      X::put(y + ib, w * f.x + u * f.y);
    }
  }
}

template <bool kBf16, bool kVec>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
  const int per_block = a.tokens >= 4096 ? 4 : 1;
  const long long blocks = ((long long)a.tokens + per_block - 1) / per_block;
  rope_kernel<kBf16, kVec><<<(unsigned)blocks, kThreads, (size_t)per_block * (a.rot / 2) * sizeof(float2), s>>>(a, per_block);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool bf16, cudaStream_t s) {
  return bf16 ? (a.vec ? launch<true, true>(a, s) : launch<true, false>(a, s))
              : (a.vec ? launch<false, true>(a, s) : launch<false, false>(a, s));
}

}  // namespace gdn
