// kv_append.cu -- new keys and values into the pages of the 8-bit cache:
//   s = 2^e, the smallest with max |x| <= 448 s over the page's new tokens, not
//   below the page's present scale where it holds older tokens;  byte = e4m3(x / s).
// A power of two loses no bits that e4m3 has (x / s is exact): where the scale
// of a half-filled page grows, its older bytes move by whole exponents and only
// those that become subnormal are rounded a second time.
//
// Bound by memory traffic, of which few warps with a page each in flight do not
// reach all: 12 prompts (14,000 tokens, 4 heads of 256, 88 MB) take 19 us, 4.6 TB/s.  A warp
// takes a page and head of k or v, 8 elements to a lane and step; what 16 steps
// read (a page of 16 tokens at D = 256) stays in registers between the maximum and
// the rounding.  Larger pages are read twice: with 32, 64 and 128 tokens to a page the
// prompts take 24, 25 and 33 us (fp32 33 with 16, then 39, 42 and 51).  Every block looks
// at all offsets, which many sequences feel: 4096 of a token each, 2 heads of 64, 94 us.
#include <algorithm>

#include "cache_device.cuh"

namespace gdn {
namespace {

constexpr int kMaxWarps = 4, kBlocksSM = 5;  // 12 prompts: 18.9 us; blocks of 8 warps with 122 registers 20.8, and 3 of them to an SM, which spills, 30
constexpr int kMinExp = -120, kMaxExp = 7;

// The smallest power of two s with 448 s >= the value of these bits (448 = 1.75 * 2^8), in its range.
__device__ __forceinline__ float scale_for(uint32_t bits) {
  if (bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(min(max(e, kMinExp), kMaxExp) + 127) << 23);
}

// 8 elements of a row as they are in memory.
template <bool kBf16>
struct Eight;
template <>
struct Eight<true> {
  static constexpr int kSteps = 16;  // kept in registers
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void none() { w = make_uint4(0, 0, 0, 0); }
  // The largest size's bits, as those of an fp32 number (a NaN's are above infinity's).
  __device__ __forceinline__ uint32_t top(uint32_t m) const {
    const uint32_t u[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(u[i] << 16, u[i]));  // the upper 16 bits count
    return m;
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const { Io<true>::unpack(w, x); }
};
template <>
struct Eight<false> {
  static constexpr int kSteps = 8;
  uint4 w[2];
  __device__ __forceinline__ void load(const float *p) {
    w[0] = *reinterpret_cast<const uint4 *>(p);
    w[1] = *reinterpret_cast<const uint4 *>(p + 4);
  }
  __device__ __forceinline__ void none() { w[0] = w[1] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t top(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      m = max(max(max(m, w[i].x & 0x7fffffffu), max(w[i].y & 0x7fffffffu, w[i].z & 0x7fffffffu)), w[i].w & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x[4 * i] = __uint_as_float(w[i].x), x[4 * i + 1] = __uint_as_float(w[i].y), x[4 * i + 2] = __uint_as_float(w[i].z),
                x[4 * i + 3] = __uint_as_float(w[i].w);
  }
};

template <bool kBf16, int D>
__global__ void __launch_bounds__(32 * kMaxWarps, kBlocksSM) kv_append_kernel(const AppendArgs a) {
  using T = typename Io<kBf16>::T;
  constexpr int kSteps = Eight<kBf16>::kSteps, kLanes = D / 8, kRowsStep = 32 / kLanes;  // lanes of a row, rows of a step
  const CacheArgs &c = a.cache;
  const int page = 1 << c.page_shift, lane = threadIdx.x & 31;
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
  const int unit = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (unit >= 2 * c.Hk) return;
  const bool is_v = unit >= c.Hk;
  const int h = is_v ? unit - c.Hk : unit;
  const int lo = (int)max((long long)start - first, 0ll), hi = (int)min((long long)s.kv - first, (long long)page);
  const long long ld = is_v ? a.ldv : a.ldk;
  const int row_in = lane / kLanes, col = lane % kLanes * 8;
  const T *const src = static_cast<const T *>(is_v ? a.v : a.k) + (s.row0 + (first - start)) * ld + (long long)h * D + col;
  Eight<kBf16> x[kSteps];
  auto load = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = row0 + i * kRowsStep + row_in;
      if (row < hi)
        x[i].load(src + (long long)row * ld);
      else
        x[i].none();
    }
  };
  constexpr int kChunk = kSteps * kRowsStep;  // rows
  load(lo);  // on the way while the page is looked up
  const int p = page_of(c, s.b, j, a.seq.err);
  if (p < 0) return;
  uint8_t *const dst = (is_v ? c.v : c.k) + (((long long)p * c.Hk + h) << c.page_shift) * D + col;
  float *const scale_at = (is_v ? c.vs : c.ks) + (long long)p * c.Hk + h;
  const float before = lo > 0 ? *scale_at : 0.f;
  uint32_t top = 0;
  for (int row0 = lo; row0 < hi; row0 += kChunk) {
    if (row0 != lo) load(row0);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) top = x[i].top(top);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (kBf16) top &= 0xffff0000u;
  float scale = scale_for(top);
  if (!(before <= scale)) scale = before < __int_as_float(0x7f800000) && scale == scale ? before : __uint_as_float(0x7fc00000u);
  const bool nan = scale != scale;
  const float inv = 1.f / scale;
  for (int row0 = lo; row0 < hi; row0 += kChunk) {
    if (hi - lo > kChunk) load(row0);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = row0 + i * kRowsStep + row_in;
      if (row < hi) {
        float f[8];
        x[i].floats(f);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = nan ? 0u : float2_to_e4m3(f[2 * e] * inv, f[2 * e + 1] * inv);
        *reinterpret_cast<uint2 *>(dst + row * D) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      }
    }
  }
  if (lo > 0 && before < scale) {
    const float ratio = before * inv;
    for (int row = row_in; row < lo; row += kRowsStep) {
      const uint2 old = *reinterpret_cast<const uint2 *>(dst + row * D);
      const uint32_t u[4] = {old.x & 0xffffu, old.x >> 16, old.y & 0xffffu, old.y >> 16};
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e4m3_to_float2(u[i]);
        w[i] = float2_to_e4m3(f.x * ratio, f.y * ratio);
      }
      *reinterpret_cast<uint2 *>(dst + row * D) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
  }
  __syncwarp();
  if (lane == 0) *scale_at = scale;
}

template <bool kBf16>
cudaError_t launch(const AppendArgs &a, cudaStream_t s) {
  const int units = 2 * a.cache.Hk, warps = std::min(units, kMaxWarps);
  const dim3 grid((unsigned)item_count(a.seq, 1, 1 << a.cache.page_shift, 2), (units + warps - 1) / warps);
  switch (a.cache.D) {
    case 64: kv_append_kernel<kBf16, 64><<<grid, 32 * warps, 0, s>>>(a); break;
    case 128: kv_append_kernel<kBf16, 128><<<grid, 32 * warps, 0, s>>>(a); break;
    default: kv_append_kernel<kBf16, 256><<<grid, 32 * warps, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, bool bf16, cudaStream_t s) {
  return bf16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace gdn
