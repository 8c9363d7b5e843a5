// kv_append.cu -- new keys and values into the pages of the 8-bit cache:
//   s = 2^e, the smallest with max |x| <= 448 s over the page's new tokens, not
//   below the page's present scale where it holds older tokens;  byte = e4m3(x / s).
// A power of two loses no bits that e4m3 has (x / s is exact): where the scale
// of a half-filled page grows, its older bytes move by whole exponents and only
// those that become subnormal are rounded a second time.
//
// Bound by memory traffic: a block takes a page and head of k or v.
#include "cache_device.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kMinExp = -120, kMaxExp = 7;

// The smallest power of two s with 448 s >= the value of these bits (448 = 1.75 * 2^8), in its range.
__device__ __forceinline__ float scale_for(uint32_t bits) {
  if (bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(min(max(e, kMinExp), kMaxExp) + 127) << 23);
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a) {
  using X = Io<kBf16>;
  using T = typename X::T;
  const CacheArgs &c = a.cache;
  const int page = 1 << c.page_shift;
  int local = 0;
  const Seq s = find_seq(a.seq, blockIdx.x, 1, page, 2, &local);
  if (s.b < 0 || s.n == 0) return;
  if (s.n > s.kv) {
    if (threadIdx.x == 0) atomicOr(a.seq.err, kErrSeqlens);
    return;
  }
  const int start = s.kv - s.n, j = (start >> c.page_shift) + local;
  const long long first = (long long)j << c.page_shift;
  if (first >= s.kv) return;
  const int p = page_of(c, s.b, j, a.seq.err);
  if (p < 0) return;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int lo = (int)max((long long)start - first, 0ll), hi = (int)min((long long)s.kv - first, (long long)page);
  const int vecs = c.D >> 3;  // 8 elements each
  const long long ld = is_v ? a.ldv : a.ldk;
  const T *const src = static_cast<const T *>(is_v ? a.v : a.k) + (s.row0 + (first - start)) * ld + (long long)h * c.D;
  uint8_t *const dst = (is_v ? c.v : c.k) + ((long long)p * c.Hk + h) * page * c.D;
  float *const scale_at = (is_v ? c.vs : c.ks) + (long long)p * c.Hk + h;

  auto load8 = [&](int it, float (&x)[8]) {
    const T *const at = src + (long long)(it / vecs) * ld + (it % vecs) * 8;
    if constexpr (kBf16) {
      X::load(at, x);
    } else {
      float u[4], w[4];
      X::load(at, u);
      X::load(at + 4, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = u[i], x[4 + i] = w[i];
    }
  };
  uint32_t amax = 0;
  for (int it = lo * vecs + threadIdx.x; it < hi * vecs; it += kThreads) {
    float x[8];
    load8(it, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  __shared__ uint32_t warp_max[kThreads / 32];
  __shared__ float old_scale;
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  if (threadIdx.x == 0) old_scale = lo > 0 ? *scale_at : 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = max(amax, warp_max[w]);
  const float before = old_scale;
  float scale = scale_for(amax);
  if (!(before <= scale)) scale = before < __int_as_float(0x7f800000) && scale == scale ? before : __uint_as_float(0x7fc00000u);
  const bool nan = scale != scale;
  const float inv = 1.f / scale;
  for (int it = lo * vecs + threadIdx.x; it < hi * vecs; it += kThreads) {
    float x[8];
    load8(it, x);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = nan ? 0u : float2_to_e4m3(x[2 * i] * inv, x[2 * i + 1] * inv);
    *reinterpret_cast<uint2 *>(dst + (long long)it * 8) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
  if (lo > 0 && before < scale) {
    const float ratio = before * inv;
    for (int it = threadIdx.x; it < lo * vecs; it += kThreads) {
      const uint2 old = *reinterpret_cast<const uint2 *>(dst + (long long)it * 8);
      const uint32_t u[4] = {old.x & 0xffffu, old.x >> 16, old.y & 0xffffu, old.y >> 16};
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e4m3_to_float2(u[i]);
        w[i] = float2_to_e4m3(f.x * ratio, f.y * ratio);
      }
      *reinterpret_cast<uint2 *>(dst + (long long)it * 8) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
  }
  if (threadIdx.x == 0) *scale_at = scale;
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, bool bf16, cudaStream_t s) {
  const dim3 grid((unsigned)item_count(a.seq, 1, 1 << a.cache.page_shift, 2), a.cache.Hk, 2);
  if (bf16)
    kv_append_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else
    kv_append_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
