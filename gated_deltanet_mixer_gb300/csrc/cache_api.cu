// cache_api.cu -- the entry points of attention over the paged 8-bit cache, of
// what fills it and of rotary positions: argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "gdn.h"
#include "host_checks.h"
#include "launch.h"

namespace {

using gdn::aligned16;
using gdn::device_info;
using gdn::DeviceInfo;
using gdn::overlap;
using gdn::Range;
using gdn::range_of;
using gdn::rows_bytes;

constexpr long long kMaxLd = 1LL << 32;

int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }
bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Shape checks shared by gdn_kv_append and gdn_attn; rows: token rows of the call.
gdn_status check_attn_shape(const gdn_attn_shape *s, bool packed, long long *rows) {
  if (s->B < 1 || s->T < 1 || s->Hk < 1 || s->D < 1 || s->max_new < 0 || s->max_kv < 0) return GDN_ERR_INVALID_ARG;
  if (s->io_dtype != GDN_F32 && s->io_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (s->D != 64 && s->D != 128 && s->D != 256) return GDN_ERR_UNSUPPORTED_SHAPE;
  *rows = packed ? (long long)s->T : (long long)s->B * s->T;
  if (s->B > 65536 || s->Hk > 1024 || *rows > (1LL << 24)) return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}
gdn_status check_heads(const gdn_attn_shape *s) {
  if (s->Hq < 1) return GDN_ERR_INVALID_ARG;
  if (s->Hq % s->Hk != 0 || s->Hq / s->Hk > 64 || s->Hq > 4096) return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}

struct CacheRanges {
  Range k, v, ks, vs, table, lens;
};
gdn_status check_cache(const gdn_attn_shape *s, const gdn_kv_cache *c, gdn::CacheArgs *a, CacheRanges *r) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table || !c->kv_lens) return GDN_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->max_blocks < 1 || c->table_ld < c->max_blocks) return GDN_ERR_INVALID_ARG;
  const int shift = page_shift(c->page);
  if (shift < 0) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (c->table_ld > kMaxLd || c->n_pages > (1 << 27) || ((long long)c->max_blocks << shift) > (1LL << 30))
    return GDN_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4) ||
      !aligned_to(c->block_table, 4) || !aligned_to(c->kv_lens, 4))
    return GDN_ERR_ALIGNMENT;
  const size_t heads = (size_t)c->n_pages * s->Hk, bytes = heads * c->page * s->D;
  *r = CacheRanges{range_of(c->k, bytes), range_of(c->v, bytes), range_of(c->k_scale, heads * 4), range_of(c->v_scale, heads * 4),
                   range_of(c->block_table, rows_bytes(s->B, c->table_ld, c->max_blocks, 4)), range_of(c->kv_lens, (size_t)s->B * 4)};
  *a = gdn::CacheArgs{static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->k_scale, c->v_scale, c->n_pages, shift,
                      s->Hk, s->D, c->block_table, c->table_ld, c->max_blocks};
  return GDN_OK;
}
// The bounds on a sequence's new and cached tokens.
int bound_new(const gdn_attn_shape *s, bool packed) { return packed && s->max_new ? std::min(s->max_new, s->T) : s->T; }
int bound_kv(const gdn_attn_shape *s, int cap) { return s->max_kv ? std::min(s->max_kv, cap) : cap; }
gdn::SeqArgs seq_args(const gdn_attn_shape *s, const int *cu, const gdn_kv_cache *c, unsigned int *err) {
  return gdn::SeqArgs{s->B, s->T, bound_new(s, cu != nullptr), bound_kv(s, c->max_blocks * c->page), cu, c->kv_lens, err};
}

gdn_status check_rows(const void *p, long long ld, long long width, size_t el) {
  if (ld < width) return GDN_ERR_INVALID_ARG;
  if (ld > kMaxLd) return GDN_ERR_UNSUPPORTED_SHAPE;
  return aligned16(p) && ld * el % 16 == 0 ? GDN_OK : GDN_ERR_ALIGNMENT;
}

// How a call of gdn_attn runs, and the workspace it makes use of.
struct AttnPlan {
  int few_rows;  // rows of a tile of attn_few.cu, or 0
  bool tile;     // attn_tile.cu; neither: attn_rows.cu
  int splits;    // ranges of the tokens side by side (attn_few.cu cuts by itself)
  size_t bytes;
  gdn::TileCut cut;  // attn_tile.cu
};
const int kPacked = 0;  // stands for offsets where only their being there counts
gdn::SeqArgs plan_seqs(const gdn_attn_shape *s, bool packed) { return gdn::SeqArgs{s->B, s->T, 0, 0, packed ? &kPacked : nullptr, nullptr, nullptr}; }
// fp32: ranges of the tokens side by side, enough blocks to fill the GPU twice, none with less than 64 tokens
int rows_splits(long long blocks, int max_kv, int sms) {
  return (int)std::max(1LL, std::min({(2LL * sms + blocks - 1) / blocks, (max_kv + 63LL) / 64, 64LL}));
}
AttnPlan attn_plan(const gdn_attn_shape *s, bool packed, long long rows, int max_kv, int sms) {
  const int r = s->Hq / s->Hk;
  AttnPlan p{0, false, 1, 0, {}};
  if (s->io_dtype == GDN_BF16) {
    p.few_rows = gdn::attn_few_rows(s->D, (long long)bound_new(s, packed) * r);
    if (p.few_rows) {
      p.bytes = gdn::attn_few_ws_bytes(s->D, p.few_rows, sms);
      return p;
    }
    p.tile = true;
    p.cut = gdn::attn_tile_cut(plan_seqs(s, packed), r, s->Hk, s->D, max_kv, sms);
    p.splits = p.cut.parts;
    p.bytes = gdn::attn_tile_ws_bytes(p.cut, s->D);
    return p;
  }
  p.splits = rows_splits((packed ? rows * r / 16 + s->B : ((long long)s->T * r / 16 + 1) * s->B) * s->Hk, max_kv, sms);
  if (p.splits > 1) p.bytes = (size_t)p.splits * rows * s->Hq * (s->D + 2) * sizeof(float);
  return p;
}
// The most workspace of this call and of any with these heads and no more sequences, rows, new and cached tokens: what
// one call uses rises and falls with them, as its parts fill the GPU.
size_t attn_room(const gdn_attn_shape *s, bool packed, long long rows, int max_kv, int sms) {
  const int r = s->Hq / s->Hk;
  size_t most = 0;
  if (s->io_dtype == GDN_BF16) {
    bool all_few = true;
    for (int n = 1, top = bound_new(s, packed); n <= top && all_few; ++n) {
      const int few = gdn::attn_few_rows(s->D, (long long)n * r);
      all_few = few > 0;
      if (few) most = std::max(most, gdn::attn_few_ws_bytes(s->D, few, sms));
    }
    return all_few ? most : std::max(most, gdn::attn_tile_room(plan_seqs(s, packed), r, s->Hk, s->D, max_kv, sms));
  }
  for (long long n = 1; n <= rows; ++n) {
    const long long blocks = (n * r + 15) / 16 * s->Hk;  // so many at least, whatever the sequences
    if (blocks >= 2LL * sms) break;
    const int splits = rows_splits(blocks, max_kv, sms);
    if (splits > 1) most = std::max(most, (size_t)(splits * n) * s->Hq * (s->D + 2) * sizeof(float));
  }
  return most;
}

}  // namespace

extern "C" {

gdn_status gdn_kv_append(const gdn_attn_shape *shape, const gdn_kv_append_io *io, void *stream) {
  if (!shape || !io || !io->k || !io->v) return GDN_ERR_INVALID_ARG;
  long long rows = 0;
  gdn_status st = check_attn_shape(shape, io->cu_seqlens != nullptr, &rows);
  if (st != GDN_OK) return st;
  gdn::AppendArgs a{};
  CacheRanges r;
  if ((st = check_cache(shape, &io->cache, &a.cache, &r)) != GDN_OK) return st;
  const size_t el = shape->io_dtype == GDN_BF16 ? 2 : 4;
  const long long width = (long long)shape->Hk * shape->D;
  if ((st = check_rows(io->k, io->ldk, width, el)) != GDN_OK || (st = check_rows(io->v, io->ldv, width, el)) != GDN_OK) return st;
  if (!aligned_to(io->cu_seqlens, 4)) return GDN_ERR_ALIGNMENT;
  const Range in[] = {range_of(io->k, rows_bytes(rows, io->ldk, width, el)), range_of(io->v, rows_bytes(rows, io->ldv, width, el)),
                      r.table, r.lens, range_of(io->cu_seqlens, io->cu_seqlens ? ((size_t)shape->B + 1) * 4 : 0)};
  const Range out[] = {r.k, r.v, r.ks, r.vs};
  for (int i = 0; i < 4; ++i) {
    for (const Range &x : in)
      if (overlap(out[i], x)) return GDN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return GDN_ERR_ALIAS;
  }
  DeviceInfo dev;
  if ((st = device_info(&dev)) != GDN_OK) return st;
  a.seq = seq_args(shape, io->cu_seqlens, &io->cache, dev.err);
  a.k = io->k;
  a.v = io->v;
  a.ldk = io->ldk;
  a.ldv = io->ldv;
  return gdn::launch_kv_append(a, shape->io_dtype == GDN_BF16, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_attn_workspace_bytes(const gdn_attn_shape *shape, int packed) {
  long long rows = 0;
  DeviceInfo dev;
  if (!shape || check_attn_shape(shape, packed != 0, &rows) != GDN_OK || check_heads(shape) != GDN_OK || device_info(&dev) != GDN_OK)
    return 0;
  return attn_room(shape, packed != 0, rows, bound_kv(shape, 1 << 30), dev.sms);
}

gdn_status gdn_selftest_attn_form(const gdn_attn_shape *shape, int packed, int workspace, gdn_attn_form *form) {
  if (!shape || !form) return GDN_ERR_INVALID_ARG;
  long long rows = 0;
  DeviceInfo dev;
  gdn_status st = check_attn_shape(shape, packed != 0, &rows);
  if (st == GDN_OK) st = check_heads(shape);
  if (st == GDN_OK) st = device_info(&dev);
  if (st != GDN_OK) return st;
  const AttnPlan p = attn_plan(shape, packed != 0, rows, bound_kv(shape, 1 << 30), dev.sms);
  *form = gdn_attn_form{p.few_rows ? GDN_ATTN_FEW : p.tile ? GDN_ATTN_TILE : GDN_ATTN_ROWS, p.few_rows ? p.few_rows : p.tile ? 128 : 16,
                        p.few_rows ? 0 : workspace ? p.splits : 1};
  return GDN_OK;
}

gdn_status gdn_attn(const gdn_attn_shape *shape, const gdn_attn_io *io, void *stream) {
  if (!shape || !io || !io->q || !io->o) return GDN_ERR_INVALID_ARG;
  const bool packed = io->cu_seqlens != nullptr;
  long long rows = 0;
  gdn_status st = check_attn_shape(shape, packed, &rows);
  if (st == GDN_OK) st = check_heads(shape);
  if (st != GDN_OK) return st;
  if (!std::isfinite(io->scale)) return GDN_ERR_INVALID_ARG;
  gdn::AttnArgs a{};
  CacheRanges r;
  if ((st = check_cache(shape, &io->cache, &a.cache, &r)) != GDN_OK) return st;
  const size_t el = shape->io_dtype == GDN_BF16 ? 2 : 4;
  const long long width = (long long)shape->Hq * shape->D;
  if ((st = check_rows(io->q, io->ldq, width, el)) != GDN_OK || (st = check_rows(io->o, io->ldo, width, el)) != GDN_OK) return st;
  if (!aligned_to(io->cu_seqlens, 4) || !aligned_to(io->workspace, 256)) return GDN_ERR_ALIGNMENT;
  const Range ro = range_of(io->o, rows_bytes(rows, io->ldo, width, el)), rw = range_of(io->workspace, io->workspace_bytes);
  const Range rq = range_of(io->q, rows_bytes(rows, io->ldq, width, el));
  const Range in[] = {r.k, r.v, r.ks, r.vs, r.table, r.lens, range_of(io->cu_seqlens, io->cu_seqlens ? ((size_t)shape->B + 1) * 4 : 0)};
  for (const Range &x : in)
    if (overlap(ro, x) || overlap(rw, x)) return GDN_ERR_ALIAS;
  // q and o may be column blocks of one buffer
  if (overlap(ro, rq) && !(io->ldq == io->ldo && gdn::column_blocks(io->q, width * el, io->o, width * el, (size_t)io->ldo * el)))
    return GDN_ERR_ALIAS;
  if (overlap(rw, rq) || overlap(ro, rw)) return GDN_ERR_ALIAS;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != GDN_OK) return st;
  a.seq = seq_args(shape, io->cu_seqlens, &io->cache, dev.err);
  a.Hq = shape->Hq;
  a.r = shape->Hq / shape->Hk;
  a.q = io->q;
  a.o = io->o;
  a.ldq = io->ldq;
  a.ldo = io->ldo;
  a.causal = io->causal != 0;
  a.scale = io->scale != 0.f ? io->scale : 1.0f / std::sqrt((float)shape->D);
  const AttnPlan plan = attn_plan(shape, packed, rows, a.seq.max_kv, dev.sms);
  if (io->workspace && plan.bytes) {
    if (io->workspace_bytes < plan.bytes) return GDN_ERR_INVALID_ARG;
    a.ws = io->workspace;
  }
  a.splits = a.ws ? plan.splits : 1;
  a.blocks = plan.cut.blocks;
  a.whole = a.ws ? plan.cut.whole : plan.cut.blocks;
  const cudaError_t e = plan.few_rows ? gdn::launch_attn_few(a, plan.few_rows, dev.sms, (cudaStream_t)stream)
                        : plan.tile   ? gdn::launch_attn_tile(a, (cudaStream_t)stream)
                                      : gdn::launch_attn_rows(a, (cudaStream_t)stream);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_rope_plan_init(const gdn_rope_spec *spec, gdn_rope_plan *plan) {
  if (!spec || !plan) return GDN_ERR_INVALID_ARG;
  const int rot = spec->rot;
  if (rot < 2 || rot % 2 || (spec->layout != GDN_ROPE_HALF && spec->layout != GDN_ROPE_INTERLEAVED)) return GDN_ERR_INVALID_ARG;
  if (rot > 2 * GDN_ROPE_MAX_PAIRS) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (!(spec->base > 1.0) || !std::isfinite(spec->base)) return GDN_ERR_INVALID_ARG;
  if (spec->scaling != GDN_ROPE_PLAIN && (!(spec->factor >= 1.0) || !std::isfinite(spec->factor))) return GDN_ERR_INVALID_ARG;
  double base = spec->base, lo = 0, hi = 0;
  const double two_pi = 6.283185307179586476925286766559;
  switch (spec->scaling) {
    case GDN_ROPE_PLAIN:
    case GDN_ROPE_LINEAR: break;
    case GDN_ROPE_NTK:
      if (rot == 2) return GDN_ERR_INVALID_ARG;
      base *= std::pow(spec->factor, (double)rot / (rot - 2));
      if (!std::isfinite(base)) return GDN_ERR_INVALID_ARG;
      break;
    case GDN_ROPE_PARTS: {
      if (!(spec->original > 0) || !std::isfinite(spec->original) || !(spec->slow > 0) || !(spec->fast > spec->slow) ||
          !std::isfinite(spec->fast))
        return GDN_ERR_INVALID_ARG;
      const auto pair = [&](double n) { return rot * std::log(spec->original / (n * two_pi)) / (2 * std::log(base)); };
      lo = std::max(std::floor(pair(spec->fast)), 0.0);
      hi = std::min(std::ceil(pair(spec->slow)), rot - 1.0);
      break;
    }
    default: return GDN_ERR_INVALID_ARG;
  }
  std::memset(plan, 0, sizeof *plan);
  plan->rot = rot;
  plan->layout = spec->layout;
  plan->m = spec->scaling == GDN_ROPE_PARTS ? (float)(0.1 * std::log(spec->factor) + 1.0) : 1.f;
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (spec->scaling == GDN_ROPE_LINEAR) f /= spec->factor;
    if (spec->scaling == GDN_ROPE_PARTS) {
      const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
      f = f * (1 - ramp) + f / spec->factor * ramp;
    }
    plan->turns[i] = (unsigned long long)std::ldexp(f / two_pi, 64);  // f <= 1: below a sixth of a turn
  }
  return GDN_OK;
}

gdn_status gdn_rope(int tokens, int D, int io_dtype, const gdn_rope_plan *plan, const int *positions, int n_x,
                    const gdn_rope_x *x, int inverse, void *stream) {
  if (tokens < 1 || D < 1 || !plan || !positions || !x || n_x < 1 || n_x > gdn::kRopeMaxX) return GDN_ERR_INVALID_ARG;
  if (io_dtype != GDN_F32 && io_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (plan->rot < 2 || plan->rot % 2 || plan->rot > 2 * GDN_ROPE_MAX_PAIRS || plan->rot > D || !std::isfinite(plan->m) ||
      (plan->layout != GDN_ROPE_HALF && plan->layout != GDN_ROPE_INTERLEAVED))
    return GDN_ERR_INVALID_ARG;
  if (tokens > (1 << 24) || D > 1024) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (!aligned_to(positions, 4)) return GDN_ERR_ALIGNMENT;
  const size_t el = io_dtype == GDN_BF16 ? 2 : 4;
  const int V = (int)(16 / el);
  gdn::RopeArgs a{};
  a.tokens = tokens;
  a.D = D;
  a.rot = plan->rot;
  a.interleaved = plan->layout == GDN_ROPE_INTERLEAVED;
  a.n_x = n_x;
  a.m = plan->m;
  a.sign = inverse ? -1.f : 1.f;
  a.positions = positions;
  a.vec = D % V == 0 && plan->rot % (a.interleaved ? V : 2 * V) == 0;
  Range rx[gdn::kRopeMaxX], ry[gdn::kRopeMaxX];
  const Range rp = range_of(positions, (size_t)tokens * 4);
  for (int i = 0; i < n_x; ++i) {
    const long long width = (long long)x[i].heads * D;
    if (!x[i].x || !x[i].y || x[i].heads < 1 || x[i].ldx < width || x[i].ldy < width) return GDN_ERR_INVALID_ARG;
    if (x[i].heads > 4096 || x[i].ldx > kMaxLd || x[i].ldy > kMaxLd) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (!aligned_to(x[i].x, el) || !aligned_to(x[i].y, el)) return GDN_ERR_ALIGNMENT;
    if (!aligned16(x[i].x) || !aligned16(x[i].y) || x[i].ldx % V || x[i].ldy % V) a.vec = 0;
    rx[i] = range_of(x[i].x, rows_bytes(tokens, x[i].ldx, width, el));
    ry[i] = range_of(x[i].y, rows_bytes(tokens, x[i].ldy, width, el));
    a.x[i] = gdn::RopeX{x[i].x, x[i].y, x[i].ldx, x[i].ldy, x[i].heads};
  }
  for (int i = 0; i < n_x; ++i) {
    if (overlap(ry[i], rp)) return GDN_ERR_ALIAS;
    const size_t wi = (size_t)x[i].heads * D * el, pitch = (size_t)x[i].ldy * el;
    for (int j = 0; j < n_x; ++j) {
      const size_t wj = (size_t)x[j].heads * D * el;
      const bool in_place = i == j && x[i].x == x[i].y && x[i].ldx == x[i].ldy;
      if (!in_place && overlap(ry[i], rx[j]) &&
          !(x[j].ldx == x[i].ldy && gdn::column_blocks(x[i].y, wi, x[j].x, wj, pitch)))
        return GDN_ERR_ALIAS;
      if (j < i && overlap(ry[i], ry[j]) && !(x[j].ldy == x[i].ldy && gdn::column_blocks(x[i].y, wi, x[j].y, wj, pitch)))
        return GDN_ERR_ALIAS;
    }
  }
  DeviceInfo dev;
  const gdn_status st = device_info(&dev);
  if (st != GDN_OK) return st;
  return gdn::launch_rope(a, plan->turns, io_dtype == GDN_BF16, dev.sms, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv_pages(const gdn_kv_pages_io *io, void *stream) {
  if (!io || io->B < 1 || io->max_blocks < 1 || io->n_free < 0 || io->max_tokens < 0 || io->table_ld < io->max_blocks)
    return GDN_ERR_INVALID_ARG;
  if (!io->kv_lens || !io->new_tokens || !io->free_used || !io->block_table || !io->kv_lens_out || !io->free_used_out ||
      !io->cu_seqlens || (io->n_free > 0 && !io->free_pages))
    return GDN_ERR_INVALID_ARG;
  const int shift = page_shift(io->page);
  if (shift < 0 || io->B > gdn::kPagesMaxB || io->table_ld > kMaxLd || io->max_tokens > (1LL << 30) ||
      ((long long)io->max_blocks << shift) > (1LL << 30))
    return GDN_ERR_UNSUPPORTED_SHAPE;
  const void *const words[] = {io->kv_lens, io->new_tokens, io->free_pages, io->free_used, io->block_table,
                               io->kv_lens_out, io->free_used_out, io->cu_seqlens, io->positions};
  for (const void *p : words)
    if (!aligned_to(p, 4)) return GDN_ERR_ALIGNMENT;
  if (!aligned_to(io->slots, 8)) return GDN_ERR_ALIGNMENT;
  const size_t B = (size_t)io->B;
  const Range in[] = {range_of(io->kv_lens, B * 4), range_of(io->new_tokens, B * 4), range_of(io->free_pages, (size_t)io->n_free * 4),
                      range_of(io->free_used, 4)};
  const Range out[] = {range_of(io->kv_lens_out, B * 4), range_of(io->free_used_out, 4),
                       range_of(io->block_table, rows_bytes(io->B, io->table_ld, io->max_blocks, 4)),
                       range_of(io->cu_seqlens, (B + 1) * 4), range_of(io->slots, (size_t)io->max_tokens * 8),
                       range_of(io->positions, (size_t)io->max_tokens * 4)};
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < 4; ++j) {
      const bool same = (i == 0 && j == 0 && io->kv_lens == io->kv_lens_out) || (i == 1 && j == 3 && io->free_used == io->free_used_out);
      if (!same && overlap(out[i], in[j])) return GDN_ERR_ALIAS;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return GDN_ERR_ALIAS;
  }
  DeviceInfo dev;
  const gdn_status st = device_info(&dev);
  if (st != GDN_OK) return st;
  const gdn::PagesArgs a{io->B, shift, io->max_blocks, io->n_free, io->table_ld, io->max_tokens, io->kv_lens, io->new_tokens,
                         io->free_pages, io->free_used, io->block_table, io->kv_lens_out, io->free_used_out, io->cu_seqlens,
                         io->slots, io->positions, dev.err};
  return gdn::launch_kv_pages(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
