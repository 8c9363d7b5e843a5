// attn_rows.cu -- attention over the paged 8-bit cache in fp32 arithmetic (fp32 io):
//   o_i = sum_j p_ij v_j,  p_i = softmax_j(scale q_i . k_j), one pass over j with
// the running maximum and sum of each row.
//
// A block takes 16 rows (query tokens x the heads of one key head) and a range
// of tokens; tiles of 32 tokens become floats in shared memory, where a lane is
// a token for the scores and a set of columns for the values, and each value
// read serves the 4 rows of its warp.  Bound by the loads from shared memory
// and the shuffles that feed the multiply-adds: 64 tokens over 2000, 8/2 heads of 64,
// 128 and 256 take 47, 70 and 111 us, of which the multiply-adds alone are 3.4, 6.7 and 13
// at the fp32 rate.  Where rows are few, ranges of the tokens run side by side and a
// second launch joins them (1 token over 5000: 29, 39 and 53 us).
#include "cache_device.cuh"
#include "tma_host.h"

namespace gdn {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRowsWarp = 4, kRows = kWarps * kRowsWarp;
constexpr int kTile = 32;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
constexpr size_t smem_bytes() {
  return sizeof(float) * (kRows * D + kTile * (D + 4) + kTile * D + 2 * kTile);
}

// Where a block's rows lie.
struct RowSpan {
  Seq s;
  int first, count;  // of the sequence's n r rows for this key head
};
__device__ __forceinline__ RowSpan row_span(const AttnArgs &a) {
  int local = 0;
  RowSpan x;
  x.s = find_seq(a.seq, blockIdx.x, a.r, kRows, 1, &local);
  x.first = local * kRows;
  x.count = x.s.b < 0 ? 0 : (int)min((long long)kRows, (long long)x.s.n * a.r - x.first);
  return x;
}

// Partial results: [splits][rows][D] values, then [splits][rows] (maximum, sum).
__device__ __forceinline__ float *part_o(const AttnArgs &a, int z, long long row, int D) {
  const long long rows = (long long)a.seq.T * (a.seq.cu ? 1 : a.seq.B) * a.Hq;
  return static_cast<float *>(a.ws) + (z * rows + row) * D;
}
__device__ __forceinline__ float2 *part_ml(const AttnArgs &a, int splits, int z, long long row, int D) {
  const long long rows = (long long)a.seq.T * (a.seq.cu ? 1 : a.seq.B) * a.Hq;
  return reinterpret_cast<float2 *>(static_cast<float *>(a.ws) + splits * rows * D) + z * rows + row;
}

template <int D>
__global__ void __launch_bounds__(kThreads) attn_rows_kernel(const AttnArgs a, int chunk) {
  using X = Io<false>;
  using T = typename X::T;
  constexpr int C = D / 32;  // columns of a lane: 2 lane + 64 i, two at a time
  extern __shared__ float4 smem4[];
  float *const sq = reinterpret_cast<float *>(smem4), *const sk = sq + kRows * D, *const sv = sk + kTile * (D + 4);
  float *const sks = sv + kTile * D, *const svs = sks + kTile;
  const RowSpan span = row_span(a);
  if (span.count <= 0) return;
  const Seq s = span.s;
  const CacheArgs &c = a.cache;
  const int hk = blockIdx.y, z = blockIdx.z, splits = gridDim.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kRows * (D / X::V); i += kThreads) {
    const int row = i / (D / X::V), col = i % (D / X::V) * X::V, rr = span.first + row;
    float x[X::V];
#pragma unroll
    for (int u = 0; u < X::V; ++u) x[u] = 0.f;
    if (row < span.count)
      X::load(static_cast<const T *>(a.q) + (long long)(s.row0 + rr / a.r) * a.ldq + (long long)(hk * a.r + rr % a.r) * D + col, x);
#pragma unroll
    for (int u = 0; u < X::V; ++u) sq[row * D + col + u] = fabsf(x[u]) < INFINITY ? x[u] : __int_as_float(0x7fc00000);
  }
  int last[kRowsWarp];  // of the tokens each row sees
  float m[kRowsWarp], l[kRowsWarp], o[kRowsWarp][C];
#pragma unroll
  for (int i = 0; i < kRowsWarp; ++i) {
    const int row = warp * kRowsWarp + i;
    last[i] = row >= span.count ? -1 : a.causal ? s.kv - s.n + (span.first + row) / a.r : s.kv - 1;
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int u = 0; u < C; ++u) o[i][u] = 0.f;
  }
  const int last_row = span.first + span.count - 1;
  const int seen = a.causal ? s.kv - s.n + last_row / a.r + 1 : s.kv;  // by the block's last row
  const long long lo = (long long)z * chunk;
  const int hi = (int)min((long long)seen, lo + chunk);
  const float scale = a.scale * kLog2e;
  const int page = 1 << c.page_shift;
  for (int t0 = (int)lo; lo < hi && t0 < hi; t0 += kTile) {
    __syncthreads();
    for (int i = tid; i < 2 * kTile * (D / 16); i += kThreads) {
      const bool is_v = i >= kTile * (D / 16);
      const int i1 = is_v ? i - kTile * (D / 16) : i, tok = i1 / (D / 16), col = i1 % (D / 16) * 16, t = t0 + tok;
      uint4 w = make_uint4(0, 0, 0, 0);
      int p = -1;
      if (t < hi) p = page_of(c, s.b, t >> c.page_shift, a.seq.err);
      const long long head = (long long)p * c.Hk + hk;
      if (p >= 0)
        w = *reinterpret_cast<const uint4 *>((is_v ? c.v : c.k) + (head * page + (t & (page - 1))) * D + col);
      if (col == 0) {  // a key scale below 0: a token that is not there
        if (is_v)
          svs[tok] = p >= 0 ? c.vs[head] : 0.f;
        else
          sks[tok] = p >= 0 ? c.ks[head] : -1.f;
      }
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      float *const dst = is_v ? sv + tok * D + col : sk + tok * (D + 4) + col;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = e4m3_to_float2(u[e] & 0xffffu), g = e4m3_to_float2(u[e] >> 16);
        *reinterpret_cast<float4 *>(dst + 4 * e) = make_float4(f.x, f.y, g.x, g.y);
      }
    }
    __syncthreads();
    // scores: lane = token
    float sc[kRowsWarp] = {};
    const float *const kt = sk + lane * (D + 4), *const qw = sq + warp * kRowsWarp * D;
#pragma unroll 8
    for (int d = 0; d < D; d += 4) {
      const float4 kk = *reinterpret_cast<const float4 *>(kt + d);
#pragma unroll
      for (int i = 0; i < kRowsWarp; ++i) {
        const float4 qq = *reinterpret_cast<const float4 *>(qw + i * D + d);
        sc[i] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, sc[i]))));
      }
    }
    const float ks = sks[lane], vs = svs[lane];
    const int t = t0 + lane;
#pragma unroll
    for (int i = 0; i < kRowsWarp; ++i) {
      const bool sees = t <= last[i] && t < hi && !(ks < 0.f);
      const float x = sees ? sc[i] * scale * ks : -INFINITY;
      float top = x;
      bool nan = x != x;
#pragma unroll
      for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      nan = __any_sync(0xffffffffu, nan);
      if (top == -INFINITY && !nan) {
        sc[i] = 0.f;
        continue;
      }
      const float mn = nan ? __int_as_float(0x7fc00000) : fmaxf(m[i], top);
      const float alpha = m[i] == -INFINITY && !nan ? 0.f : exp2f(m[i] - mn);
      const float p = sees ? exp2f(x - mn) : 0.f;
      float sum = p;
#pragma unroll
      for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[i] = l[i] * alpha + sum;
      m[i] = mn;
#pragma unroll
      for (int u = 0; u < C; ++u) o[i][u] *= alpha;
      sc[i] = sees ? p * vs : 0.f;
    }
    // values: lane = columns
    for (int j = 0; j < kTile; ++j) {
      float p[kRowsWarp];
#pragma unroll
      for (int i = 0; i < kRowsWarp; ++i) p[i] = __shfl_sync(0xffffffffu, sc[i], j);
#pragma unroll
      for (int u = 0; u < C; u += 2) {
        const float2 v = *reinterpret_cast<const float2 *>(sv + j * D + 2 * lane + 32 * u);
#pragma unroll
        for (int i = 0; i < kRowsWarp; ++i) {
          o[i][u] = fmaf(p[i], v.x, o[i][u]);
          o[i][u + 1] = fmaf(p[i], v.y, o[i][u + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsWarp; ++i) {
    const int row = warp * kRowsWarp + i, rr = span.first + row;
    if (row >= span.count) continue;
    const int tok = s.row0 + rr / a.r, h = hk * a.r + rr % a.r;
    if (splits > 1) {
      const long long grow = (long long)tok * a.Hq + h;
      float *const dst = part_o(a, z, grow, D);
#pragma unroll
      for (int u = 0; u < C; u += 2) *reinterpret_cast<float2 *>(dst + 2 * lane + 32 * u) = make_float2(o[i][u], o[i][u + 1]);
      if (lane == 0) *part_ml(a, splits, z, grow, D) = make_float2(m[i], l[i]);
    } else {
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
      T *const dst = static_cast<T *>(a.o) + (long long)tok * a.ldo + (long long)h * D;
#pragma unroll
      for (int u = 0; u < C; ++u) X::put(dst + 2 * lane + 32 * (u & ~1) + (u & 1), o[i][u] * inv);
    }
  }
}

// Joins the partial results of a block's rows: o = sum_z 2^(m_z - m) o_z / sum_z 2^(m_z - m) l_z.
template <int D>
__global__ void __launch_bounds__(kThreads) attn_rows_join(const AttnArgs a, int splits) {
  using X = Io<false>;
  using T = typename X::T;
  constexpr int C = D / 32;
  const RowSpan span = row_span(a);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hk = blockIdx.y;
  for (int row = warp; row < span.count; row += kWarps) {
    const int rr = span.first + row, tok = span.s.row0 + rr / a.r, h = hk * a.r + rr % a.r;
    const long long grow = (long long)tok * a.Hq + h;
    float m = -INFINITY;
    bool nan = false;
    for (int z = 0; z < splits; ++z) {
      const float mz = part_ml(a, splits, z, grow, D)->x;
      nan |= mz != mz;
      m = fmaxf(m, mz);
    }
    if (nan) m = __int_as_float(0x7fc00000);
    float l = 0.f, o[C] = {};
    for (int z = 0; z < splits; ++z) {
      const float2 ml = *part_ml(a, splits, z, grow, D);
      if (ml.x == -INFINITY && !nan) continue;
      const float w = exp2f(ml.x - m);
      l += w * ml.y;
      const float *const src = part_o(a, z, grow, D);
#pragma unroll
      for (int u = 0; u < C; ++u) o[u] += w * src[lane + 32 * u];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *const dst = static_cast<T *>(a.o) + (long long)tok * a.ldo + (long long)h * D;
#pragma unroll
    for (int u = 0; u < C; ++u) X::put(dst + lane + 32 * u, o[u] * inv);
  }
}

template <int D>
struct RowsTag {};

template <int D>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
  cudaError_t e = allow_smem<RowsTag<D>>(attn_rows_kernel<D>, smem_bytes<D>());
  if (e != cudaSuccess) return e;
  const int splits = a.ws ? a.splits : 1;
  const int chunk = ((a.seq.max_kv + splits - 1) / splits + kTile - 1) / kTile * kTile;
  const dim3 grid((unsigned)item_count(a.seq, a.r, kRows, 1), a.cache.Hk, splits);
  attn_rows_kernel<D><<<grid, kThreads, smem_bytes<D>(), s>>>(a, chunk);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits < 2) return e;
  attn_rows_join<D><<<dim3(grid.x, grid.y), kThreads, 0, s>>>(a, splits);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t s) {
  return a.cache.D == 64 ? launch<64>(a, s) : a.cache.D == 128 ? launch<128>(a, s) : launch<256>(a, s);
}

}  // namespace gdn
