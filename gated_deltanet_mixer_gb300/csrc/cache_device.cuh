// cache_device.cuh -- the sequences and pages of a call on the paged 8-bit cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "launch.h"

namespace gdn {

struct Seq {
  int b;     // -1: none, or one to skip
  int row0;  // its first token row
  int n;     // new tokens
  int kv;    // tokens in all
};

// Sequence b with n rows from row0 on and kv tokens in all; b = -1 where the lengths are out of range.
__device__ __forceinline__ Seq checked_seq(const SeqArgs &g, int b, int row0, int n, int kv) {
  Seq s{b, row0, n, kv};
  if (n < 0 || n > g.max_new || s.kv < 0 || s.kv > g.max_kv) {
    atomicOr(g.err, kErrSeqlens);
    s.b = -1;
  }
  return s;
}
__device__ __forceinline__ Seq load_seq(const SeqArgs &g, int b, int row0, int n) { return checked_seq(g, b, row0, n, g.kv_lens[b]); }

// Work items are numbered over the sequences without a prefix sum: those of
// sequence b from base(b) = floor(cu[b] mul / div) + c b on, which leaves room for
// floor(n mul / div) + c of them.
__device__ __forceinline__ long long item_base(long long cu, int b, int mul, int div, int c) {
  return cu * mul / div + (long long)c * b;
}
inline long long item_count(const SeqArgs &g, int mul, int div, int c) {
  return g.cu ? (long long)g.T * mul / div + (long long)c * g.B : ((long long)g.T * mul / div + c) * g.B;
}
// The sequence of item `item` and its number there, for the whole block.  The
// offsets are all looked at, side by side: where they decrease or leave the
// rows, no item belongs to anyone.
__device__ __forceinline__ Seq find_seq(const SeqArgs &g, long long item, int mul, int div, int c, int *local) {
  if (!g.cu) {
    const long long per = (long long)g.T * mul / div + c;
    const int b = (int)(item / per);
    *local = (int)(item % per);
    return load_seq(g, b, b * g.T, g.T);
  }
  __shared__ Seq found;
  __shared__ int bad;
  if (threadIdx.x == 0) {
    found.b = -1;
    bad = 0;
  }
  __syncthreads();
  for (int b = threadIdx.x; b < g.B; b += blockDim.x) {
    const int lo = g.cu[b], hi = g.cu[b + 1], kv = g.kv_lens[b];
    if (lo < 0 || hi < lo || hi > g.T) {
      bad = 1;
    } else if (item >= item_base(lo, b, mul, div, c) && item < item_base(hi, b + 1, mul, div, c)) {
      found = Seq{b, lo, hi - lo, kv};
    }
  }
  __syncthreads();
  const Seq s = found;
  if (bad) {
    if (threadIdx.x == 0) atomicOr(g.err, kErrSeqlens);
    return Seq{-1, 0, 0, 0};
  }
  if (s.b < 0) return s;
  *local = (int)(item - item_base(s.row0, s.b, mul, div, c));
  return checked_seq(g, s.b, s.row0, s.n, s.kv);
}

// The page of block j of sequence b, or -1 (recorded) where the table has none.
__device__ __forceinline__ int page_of(const CacheArgs &c, int b, int j, unsigned int *err) {
  const int p = c.table[(long long)b * c.table_ld + j];
  if (p >= 0 && p < c.n_pages) return p;
  atomicOr(err, kErrSeqlens);
  return -1;
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&t);
}
// Two e4m3 bytes as floats (exact).
__device__ __forceinline__ float2 e4m3_to_float2(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// Two of a word's four e4m3 bytes, the lower or the upper ones, as fp16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w, int upper) {
  uint32_t o;
  if (upper)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(o) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(o) : "r"(w));
  return o;
}
// Two floats as e4m3 bytes, to nearest even, saturated to +-448.
__device__ __forceinline__ uint32_t float2_to_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// 2^x to about 2^-22, 0 below 2^-126.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// V consecutive elements (16 bytes) of an io tensor as floats.
template <bool kBf16>
struct Io;
template <>
struct Io<true> {
  static constexpr int V = 8;
  using T = __nv_bfloat16;
  static __device__ __forceinline__ void load(const T *p, float (&x)[8]) { unpack(*reinterpret_cast<const uint4 *>(p), x); }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_bf16(u[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store(T *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
  static __device__ __forceinline__ float get(const T *p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void put(T *p, float x) { *p = __float2bfloat16_rn(x); }
};
template <>
struct Io<false> {
  static constexpr int V = 4;
  using T = float;
  static __device__ __forceinline__ void load(const T *p, float (&x)[4]) { unpack(*reinterpret_cast<const uint4 *>(p), x); }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ void store(T *p, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
  static __device__ __forceinline__ float get(const T *p) { return *p; }
  static __device__ __forceinline__ void put(T *p, float x) { *p = x; }
};

}  // namespace gdn
