// C ABI of writing and reading a paged cache: argument checks before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include "cache.h"

namespace bd {

bitdelta_status status_of_hip(hipError_t e);

bitdelta_status check_kv_cache(const bitdelta_kv_cache* c, int32_t heads) {
  if (!c) return BITDELTA_ERR_INVALID_ARG;
  if (c->dtype != BITDELTA_KV_BF16 && c->dtype != BITDELTA_KV_FP8 && c->dtype != BITDELTA_KV_FP4)
    return BITDELTA_ERR_INVALID_ARG;
  const bool fp4 = c->dtype == BITDELTA_KV_FP4;
  if (fp4 && (!c->k_block_scales || !c->v_block_scales)) return BITDELTA_ERR_INVALID_ARG;
  if (!c->k || !c->v || c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || heads < 1)
    return BITDELTA_ERR_INVALID_ARG;
  if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || !isfinite(c->k_scale) || !isfinite(c->v_scale))
    return BITDELTA_ERR_INVALID_ARG;
  if (heads % c->kv_heads != 0) return BITDELTA_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return BITDELTA_ERR_UNSUPPORTED;
  if (heads / c->kv_heads > BITDELTA_ATTEND_MAX_GROUP) return BITDELTA_ERR_UNSUPPORTED;
  const int64_t unit = fp4 ? 32 : (c->dtype == BITDELTA_KV_FP8 ? 16 : 8);  // elements of 16 bytes
  // with 4 bits whole rows, so that the scale bytes of a row lie together
  const int64_t step = fp4 ? c->head_dim : unit;
  // strides of dimensions of one element are never stepped over: any value will do
  const struct { int64_t stride; int32_t n; } steps[] = {
      {c->k_stride_page, c->num_pages}, {c->k_stride_token, c->page_size}, {c->k_stride_head, c->kv_heads},
      {c->v_stride_page, c->num_pages}, {c->v_stride_token, c->page_size}, {c->v_stride_head, c->kv_heads}};
  for (const auto& s : steps) {
    if (s.n == 1) continue;
    if (s.stride < 0) return BITDELTA_ERR_INVALID_ARG;
    if (s.stride % step != 0) return BITDELTA_ERR_ALIGNMENT;
    if (s.stride / unit > 0xFFFFFFFFll) return BITDELTA_ERR_UNSUPPORTED;
  }
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return BITDELTA_ERR_ALIGNMENT;
  if (fp4 && (!aligned(c->k_block_scales, 4) || !aligned(c->v_block_scales, 4))) return BITDELTA_ERR_ALIGNMENT;
  return BITDELTA_OK;
}

PagedCache paged_cache(const bitdelta_kv_cache& c) {
  // bytes of n elements; strides of dimensions of one element, which may be anything, are never stepped
  // over and must not overflow on the way
  auto bytes = [&](int64_t n, int32_t size) -> int64_t {
    if (size == 1) return 0;
    return c.dtype == BITDELTA_KV_FP4 ? n / 2 : (c.dtype == BITDELTA_KV_FP8 ? n : n * 2);
  };
  PagedCache p{};
  p.k = static_cast<const unsigned char*>(c.k);
  p.v = static_cast<const unsigned char*>(c.v);
  p.k_page = (uint32_t)(bytes(c.k_stride_page, c.num_pages) / 16);
  p.k_token = (uint32_t)(bytes(c.k_stride_token, c.page_size) / 16);
  p.k_head = bytes(c.k_stride_head, c.kv_heads);
  p.v_page = (uint32_t)(bytes(c.v_stride_page, c.num_pages) / 16);
  p.v_token = (uint32_t)(bytes(c.v_stride_token, c.page_size) / 16);
  p.v_head = bytes(c.v_stride_head, c.kv_heads);
  p.alike = p.k_page == p.v_page && p.k_token == p.v_token && p.k_head == p.v_head;
  p.num_pages = c.num_pages;
  p.page_size = c.page_size;
  p.div = make_page_div((uint32_t)c.page_size);
  if (c.dtype == BITDELTA_KV_FP4) {
    p.k_blocks = static_cast<const unsigned char*>(c.k_block_scales);
    p.v_blocks = static_cast<const unsigned char*>(c.v_block_scales);
  }
  return p;
}

namespace {

bitdelta_status check(const bitdelta_kv_rows* r, const bitdelta_kv_cache* c, int32_t batch,
                      const int32_t* table, int32_t width, const int32_t* lens,
                      const int32_t* q_offsets) {
  bitdelta_status s = check_kv_cache(c, c ? c->kv_heads : 1);
  if (s != BITDELTA_OK) return s;
  if (!r->k || !r->v || !lens || width < 0 || (!table && width > 0)) return BITDELTA_ERR_INVALID_ARG;
  if (c->kv_heads > kCacheMaxHeads || batch > BITDELTA_ATTEND_MAX_SEQS ||
      r->tokens > kCacheMaxRows / c->kv_heads || (int64_t)width * c->page_size > (int64_t(1) << 30))
    return BITDELTA_ERR_UNSUPPORTED;
  if (!q_offsets && r->tokens != batch) return BITDELTA_ERR_SHAPE;
  const struct { int64_t stride; bool used; } steps[] = {{r->k_stride_token, r->tokens > 1},
                                                         {r->v_stride_token, r->tokens > 1},
                                                         {r->k_stride_head, c->kv_heads > 1},
                                                         {r->v_stride_head, c->kv_heads > 1}};
  for (const auto& x : steps)
    if (x.used && x.stride < 0) return BITDELTA_ERR_INVALID_ARG;
  for (const auto& x : steps)
    if (x.used && x.stride % 8 != 0) return BITDELTA_ERR_ALIGNMENT;
  if (!aligned(r->k, 16) || !aligned(r->v, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(q_offsets, 4))
    return BITDELTA_ERR_ALIGNMENT;
  return BITDELTA_OK;
}

// 1 / scale if every product with it is the quotient by scale: a power of two whose inverse is normal
float exact_inverse(float scale) {
  int e;
  const float inv = 1.0f / scale;
  return frexpf(scale, &e) == 0.5f && isnormal(scale) && isnormal(inv) ? inv : 0.0f;
}

// 1 / scale rounded, if Markstein's theorem holds with it (a fraction of scale that is not all ones) for
// quotients from 2^-20 to 2^9 without an underflow of what is left over (products 2^-48 of the value)
float near_inverse(float scale) {
  int e;
  const float f = frexpf(scale, &e);
  return e > -60 && e < 60 && f < 0.99999994f ? 1.0f / scale : 0.0f;
}

bitdelta_status run(bool write, const bitdelta_kv_rows* r, const bitdelta_kv_cache* c, int32_t batch,
                    const int32_t* table, int32_t width, const int32_t* lens,
                    const int32_t* q_offsets, bitdelta_stream stream) {
  if (!r || r->tokens < 0 || batch < 0) return BITDELTA_ERR_INVALID_ARG;
  if (r->tokens == 0 || batch == 0) return BITDELTA_OK;
  const bitdelta_status s = check(r, c, batch, table, width, lens, q_offsets);
  if (s != BITDELTA_OK) return s;
  CacheArgs a{};
  const bool tokens = r->tokens > 1, heads = c->kv_heads > 1;  // else the stride is never stepped over
  a.rows[0] = static_cast<uint16_t*>(r->k);
  a.rows[1] = static_cast<uint16_t*>(r->v);
  a.row_token[0] = tokens ? r->k_stride_token : 0;
  a.row_token[1] = tokens ? r->v_stride_token : 0;
  a.row_head[0] = heads ? r->k_stride_head : 0;
  a.row_head[1] = heads ? r->v_stride_head : 0;
  a.cache = paged_cache(*c);
  a.table = table;
  a.lens = lens;
  a.q_offsets = q_offsets;
  a.width = width;
  a.batch = batch;
  a.tokens = (int32_t)r->tokens;
  a.kv_heads = c->kv_heads;
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.inverse[0] = exact_inverse(c->k_scale);
  a.inverse[1] = exact_inverse(c->v_scale);
  a.near[0] = near_inverse(c->k_scale);
  a.near[1] = near_inverse(c->v_scale);
  hipStream_t st = static_cast<hipStream_t>(stream);
  return status_of_hip(write ? launch_cache_write(a, c->head_dim, c->dtype, st)
                             : launch_cache_read(a, c->head_dim, c->dtype, st));
}

}  // namespace
}  // namespace bd

extern "C" {

bitdelta_status bitdelta_cache_write(const bitdelta_kv_rows* rows, const bitdelta_kv_cache* cache,
                                     int32_t batch, const int32_t* table, int32_t table_width,
                                     const int32_t* lens, const int32_t* q_offsets,
                                     bitdelta_stream stream) {
  return bd::run(true, rows, cache, batch, table, table_width, lens, q_offsets, stream);
}

bitdelta_status bitdelta_cache_read(const bitdelta_kv_rows* rows, const bitdelta_kv_cache* cache,
                                    int32_t batch, const int32_t* table, int32_t table_width,
                                    const int32_t* lens, const int32_t* q_offsets,
                                    bitdelta_stream stream) {
  return bd::run(false, rows, cache, batch, table, table_width, lens, q_offsets, stream);
}

}  // extern "C"
