// C ABI of the paged-cache attention: argument checks, choice of kernels, workspace layout.
// Every argument error is detected here, on the host, before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/bitdelta.h"
#include "attend.h"
#include "cache.h"

namespace bd {
bitdelta_status status_of_hip(hipError_t e);
}

namespace {

constexpr int64_t kMaxKeys = int64_t(1) << 30;  // positions of a key list stay far below 2^31
// A launch holds fewer than 2^32 threads: 512 of each of at most 2^30 / 193 row tiles of a call's
// tokens (a tile of 256 rows is filled to 193 at least) and one more tile of each (sequence, kv head).
constexpr int64_t kMaxRows = int64_t(1) << 30;   // tokens x heads
constexpr int64_t kMaxUnits = int64_t(1) << 21;  // sequences x kv heads

// Workgroups of a split launch: as many as the 256 compute units hold at a time (more would start
// when the first have ended, and take as long again), which their registers decide.
int row_workers(int columns, int64_t max_q, const bitdelta_kv_cache& c) {
  if (columns == 1 && c.dtype == BITDELTA_KV_FP4) return 768;
  if (columns == 1 && max_q == 1 && (c.dtype == BITDELTA_KV_FP8 || c.head_dim == 64)) return 768;
  return columns <= 2 ? 512 : 256;
}
constexpr int kTileWorkers = 256;
// Steps of 64 keys that a part of a split unit has at least: it begins with three dependent readings.
constexpr int kPartSteps = 4;

// A unit (sequence, kv head) whose key list is at most this many 128-key steps long is done by one
// workgroup, without partials and the launch that joins them.  Few units: a step takes such a
// workgroup about 2 us, a split and joined short call 20 us in all (8 kv heads, bf16, head_dim 128,
// one sequence: 6 steps 18.0 against 20.7 us, 12 steps 30.6 against 21.0).  As many units as
// workgroups at a time fill the machine unsplit (64 sequences: 12 steps 77 against 84 us); beyond
// 12 steps one long list among short ones would be waited for.
// From 4 bits (64 sequences of up to the given length, 8 kv heads, one workgroup a unit against split and
// joined): 2000 keys 28 against 37 us, 4000 46 against 50, 6000 66 against 63; 256 of up to 3000 108 against
// 135.  Up to 32 steps one long list among short ones is waited for, which even batches and short ones in wide
// tables gain from: 64 of 100 keys 7 against 13 us, of 1000 18 against 27; but one of 4000 among 63 of 100 34
// against 17, among 63 of 1000 37 against 27, eight of 4000 among 56 of 500 36 against 27; one of 4000 among
// 255 of 100 37 against 33, among 255 of 700 45 against 57.
int direct_steps(int64_t units, int32_t dtype) {
  if (units < 512) return 6;
  return dtype == BITDELTA_KV_FP4 ? 32 : 12;
}

// Are prefixes worth a launch of their own?  Reading a prefix once per segment instead of once per
// sequence saves this many bytes, most of which the caches would have served; the tile launch and its
// pieces cost about 10 us.  Measured with 8 kv heads, bf16, head_dim 128, prefixes read by the tile
// against the row kernel: saving 67 MB 36.4 against 34.1 us, 101 MB 34.8 against 33.1, 201 MB 39.7
// against 47.9, 503 MB 61.3 against 92.8.
constexpr int64_t kShareBytes = int64_t(128) << 20;
// From 4 bits, whose row kernel reads 3.8 times the keys in that time, rows against tiles: saving 111 MB 42
// against 55 us, 134 MB 37 against 46, 267 MB 52 against 52, 446 MB 86 against 87, 508 MB 94 against 87,
// 561 MB 115 against 91, 1.0 GB 147 against 115.
constexpr int64_t kShareBytes4 = int64_t(400) << 20;

// Does a call with several rows a unit go to the tile kernel?  Beyond 64 rows always.  Below, a tile
// workgroup has idle rows, but reads a unit's keys at the same speed whatever its rows are, one unit a
// compute unit; the row kernel's time grows with its rows, and it splits a unit over workgroups.
// Rows x units at 4096 keys, bf16, head_dim 128, row against tile kernel: 64 x 8 39 against 86 us,
// 64 x 64 84 against 85, 64 x 256 286 against 100, 32 x 64 47 against 81, 32 x 256 136 against 100,
// 16 x 256 108 against 99.
// From 4 bits the tile kernel widens a tile's values once for its 8 waves and splits a unit's keys where
// units are few: row against tile kernel, with what joins them, 64 x 8 29 against 20 us, 64 x 64 47 against
// 40, 64 x 256 117 against 101, 32 x 8 20 against 18, 32 x 64 32 against 38, 32 x 256 80 against 97.
bool tiles_for_rows(int64_t rows, int64_t units, int32_t dtype) {
  if (dtype == BITDELTA_KV_FP4) return rows > 32;
  return rows > 64 || (rows > 32 && units >= 64) || (rows > 16 && units >= 192);
}

using bd::aligned;

enum class Kind { kRows, kRowsSplit, kPrefixTiles, kTiles };

struct Plan {
  Kind kind;
  int columns;         // row kernel: 16-column blocks
  int row_rows;        // rows of a row unit
  int64_t row_units, row_workers;
  int64_t tile_units, tile_workers;
  int tile_parts;      // 4 bits, window
  size_t scan_bytes, row_o, row_ml, segs_bytes, tile_o, tile_ml;
  size_t total;
};

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

void lay_out(Plan* p, int64_t batch, int dim) {
  p->scan_bytes = p->row_o = p->row_ml = p->segs_bytes = p->tile_o = p->tile_ml = 0;
  if (p->kind == Kind::kRowsSplit || p->kind == Kind::kPrefixTiles) {
    const size_t slots = (size_t)(p->row_units + p->row_workers) * p->row_rows;
    p->scan_bytes = up256((size_t)(batch + 1) * 4);
    p->row_o = up256(slots * dim * 4);
    p->row_ml = up256(slots * 8);
  }
  if (p->kind == Kind::kTiles && p->tile_parts > 1) {
    p->scan_bytes = up256((size_t)(batch + 1) * 4);
    const size_t slots = (size_t)p->tile_workers * bd::kTileRows;
    p->tile_o = up256(slots * dim * 4);
    p->tile_ml = up256(slots * 8);
  }
  if (p->kind == Kind::kPrefixTiles) {
    const size_t slots = (size_t)(p->tile_units + p->tile_workers) * bd::kTileRows;
    p->segs_bytes = up256((BITDELTA_MAX_SEGMENTS + 1) * 4);  // each of two
    p->tile_o = up256(slots * dim * 4);
    p->tile_ml = up256(slots * 8);
  }
  p->total = p->scan_bytes + p->row_o + p->row_ml + 2 * p->segs_bytes + p->tile_o + p->tile_ml;
}

// what scores are multiplied by to enter exp2
float score_factor(const bitdelta_attend_rows& r, const bitdelta_kv_cache& c) {
  return (float)((double)r.scale * c.k_scale * 1.4426950408889634);
}
// Each scale may be a number whose product is none: infinite, it makes a score of 0 NaN, and 0 a masked one.
bitdelta_status check_scales(const bitdelta_attend_rows& r, const bitdelta_kv_cache& c) {
  return isnormal(score_factor(r, c)) ? BITDELTA_OK : BITDELTA_ERR_INVALID_ARG;
}

bitdelta_status check_rows(const bitdelta_attend_rows* r, int64_t max_tokens) {
  if (!r || r->tokens < 0) return BITDELTA_ERR_INVALID_ARG;
  if (r->tokens > max_tokens) return BITDELTA_ERR_UNSUPPORTED;
  if (r->tokens == 0) return BITDELTA_OK;
  if (!r->q || !r->out || !(r->scale > 0.f) || !isfinite(r->scale)) return BITDELTA_ERR_INVALID_ARG;
  const bool tokens = r->tokens > 1, heads = r->heads > 1;  // else the stride is never stepped over
  if ((tokens && (r->q_stride_token < 0 || r->out_stride_token < 0)) ||
      (heads && (r->q_stride_head < 0 || r->out_stride_head < 0)))
    return BITDELTA_ERR_INVALID_ARG;
  if (!aligned(r->q, 16) || !aligned(r->out, 8) || !aligned(r->lse, 4) ||
      (tokens && (r->q_stride_token % 8 != 0 || r->out_stride_token % 4 != 0)) ||
      (heads && (r->q_stride_head % 8 != 0 || r->out_stride_head % 4 != 0)))
    return BITDELTA_ERR_ALIGNMENT;
  return BITDELTA_OK;
}

bitdelta_status check_segments(int64_t tokens, const int32_t* offs, int32_t n) {
  if (!offs || n < 0) return BITDELTA_ERR_INVALID_ARG;
  if (n > BITDELTA_MAX_SEGMENTS) return BITDELTA_ERR_INVALID_ARG;
  if (offs[0] != 0 || offs[n] != tokens) return BITDELTA_ERR_SHAPE;
  for (int i = 0; i < n; ++i)
    if (offs[i + 1] < offs[i]) return BITDELTA_ERR_SHAPE;
  return BITDELTA_OK;
}

int columns_for(int64_t rows) { return rows <= 16 ? 1 : (rows <= 32 ? 2 : 4); }

Plan plan_shared(int64_t batch, int32_t heads, const bitdelta_kv_cache& c, int32_t width,
                 int32_t pwidth, const int32_t* offs, int32_t nseg) {
  Plan p{};
  const int group = heads / c.kv_heads;
  p.row_rows = group;
  p.columns = columns_for(group);
  p.row_units = batch * c.kv_heads;
  const int64_t own = (int64_t)width * c.page_size, pre = (int64_t)pwidth * c.page_size;
  int used = 0;  // segments with sequences
  for (int i = 0; i < nseg; ++i) used += offs[i + 1] > offs[i];
  const int64_t row_bytes = c.dtype == BITDELTA_KV_FP4 ? c.head_dim + c.head_dim / 16
                                                       : 2 * (int64_t)c.head_dim * (c.dtype == BITDELTA_KV_FP8 ? 1 : 2);
  if (own + pre <= (int64_t)direct_steps(p.row_units, c.dtype) * bd::kRowStep) {
    p.kind = Kind::kRows;
  } else if ((batch - used) * pre * c.kv_heads * row_bytes <
             (c.dtype == BITDELTA_KV_FP4 ? kShareBytes4 : kShareBytes)) {
    p.kind = Kind::kRowsSplit;
  } else {
    p.kind = Kind::kPrefixTiles;
    const int tpt = bd::kTileRows / group;
    for (int i = 0; i < nseg; ++i) p.tile_units += (offs[i + 1] - offs[i] + tpt - 1) / tpt;
    p.tile_units *= c.kv_heads;
    const int64_t steps = (pre + bd::kTileKeys - 1) / bd::kTileKeys;
    p.tile_workers = std::min<int64_t>(kTileWorkers, std::max<int64_t>(1, p.tile_units * steps));
  }
  const int64_t keys = p.kind == Kind::kPrefixTiles ? own : own + pre;
  const int64_t steps = p.row_units * ((keys + bd::kRowStep - 1) / bd::kRowStep);
  p.row_workers = std::min<int64_t>(row_workers(p.columns, 1, c), std::max<int64_t>(1, steps));
  lay_out(&p, batch, c.head_dim);
  return p;
}

Plan plan_window(int32_t heads, const bitdelta_kv_cache& c, int32_t batch, int32_t width,
                 int32_t max_q, int32_t window, int32_t sinks) {
  Plan p{};
  const int group = heads / c.kv_heads;
  const int64_t rows = (int64_t)max_q * group;
  if (tiles_for_rows(rows, (int64_t)batch * c.kv_heads, c.dtype)) {
    p.kind = Kind::kTiles;
    if (c.dtype == BITDELTA_KV_FP4) {
      const int64_t keys = std::min<int64_t>((int64_t)width * c.page_size,
                                             (int64_t)window + bd::kTileRows / group - 1 + sinks);
      p.tile_workers = kTileWorkers;
      p.tile_parts = (int)std::min<int64_t>(kTileWorkers, keys / (kPartSteps * bd::kTileKeys));
      lay_out(&p, batch, c.head_dim);
    }
    return p;
  }
  p.row_rows = (int)rows;
  p.columns = columns_for(rows);
  p.row_units = (int64_t)batch * c.kv_heads;
  const int64_t keys = std::min<int64_t>((int64_t)width * c.page_size,
                                         (int64_t)window + max_q - 1 + sinks);
  const int64_t steps = (keys + bd::kRowStep - 1) / bd::kRowStep;
  p.kind = steps <= direct_steps(p.row_units, c.dtype) ? Kind::kRows : Kind::kRowsSplit;
  p.row_workers = std::min<int64_t>(row_workers(p.columns, max_q, c),
                                    std::max<int64_t>(1, p.row_units * steps));
  lay_out(&p, batch, c.head_dim);
  return p;
}

void fill(bd::AttendArgs* a, const bitdelta_attend_rows& r, const bitdelta_kv_cache& c) {
  a->q = static_cast<const uint16_t*>(r.q);
  a->q_token = r.q_stride_token;
  a->q_head = r.q_stride_head;
  a->out = static_cast<uint16_t*>(r.out);
  a->o_token = r.out_stride_token;
  a->o_head = r.out_stride_head;
  a->lse = r.lse;
  a->cache = bd::paged_cache(c);
  a->tokens = (int32_t)r.tokens;
  a->heads = r.heads;
  a->kv_heads = c.kv_heads;
  a->group = r.heads / c.kv_heads;
  a->c = score_factor(r, c);
  a->v_scale = c.v_scale;
}

bitdelta_status run(bd::AttendArgs* a, const Plan& p, const bitdelta_kv_cache& c, void* workspace,
                    bitdelta_stream stream) {
  const bool fp8 = c.dtype == BITDELTA_KV_FP8, fp4 = c.dtype == BITDELTA_KV_FP4;
  hipStream_t st = static_cast<hipStream_t>(stream);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a->rows = p.row_rows;
  a->workers = (int)p.row_workers;
  a->tile_workers = (int)p.tile_workers;
  a->tile_parts = p.tile_parts;
  a->halves = !fp8;
  a->direct = p.kind == Kind::kRows;
  a->row_prefix = a->nseg > 0 && p.kind != Kind::kPrefixTiles;
  auto take = [&](size_t bytes) {
    unsigned char* at = ws;
    ws += bytes;
    return at;
  };
  a->scan = reinterpret_cast<int32_t*>(take(p.scan_bytes));
  a->part_o = reinterpret_cast<float*>(take(p.row_o));
  a->part_ml = reinterpret_cast<float*>(take(p.row_ml));
  a->tile_segs = reinterpret_cast<int32_t*>(take(p.segs_bytes));
  a->tile_scan = reinterpret_cast<int32_t*>(take(p.segs_bytes));
  a->tile_o = reinterpret_cast<float*>(take(p.tile_o));
  a->tile_ml = reinterpret_cast<float*>(take(p.tile_ml));
  if (p.kind == Kind::kTiles) {
    const int tpt = bd::kTileRows / a->group;
    // each sequence rounds its tokens up to whole tiles
    const int64_t tiles = std::min<int64_t>(a->tokens / tpt + a->batch,
                                            a->batch * (((int64_t)a->max_q + tpt - 1) / tpt));
    const int units = (int)(tiles * a->kv_heads);
    if (!fp4) return bd::status_of_hip(bd::launch_attend_tiles(*a, c.head_dim, fp8, false, units, st));
    if (p.tile_parts < 2) return bd::status_of_hip(bd::launch_attend4_tiles(*a, c.head_dim, false, units, st));
    // of the units, at most these, the rest that does not fill the machine is split: to once its workgroups
    const int blocks = (units / kTileWorkers + 1) * kTileWorkers;
    const bitdelta_status s = bd::status_of_hip(bd::launch_attend4_tiles(*a, c.head_dim, false, blocks, st));
    if (s != BITDELTA_OK) return s;
    return bd::status_of_hip(bd::launch_attend4_join(*a, c.head_dim, std::min(units, kTileWorkers), st));
  }
  if (p.kind == Kind::kPrefixTiles) {
    // the grid holds whole runs of tile_workers / 8 per XCD
    const int per = (a->tile_workers + 7) / 8;
    const bitdelta_status s = bd::status_of_hip(
        fp4 ? bd::launch_attend4_tiles(*a, c.head_dim, true, per * 8, st)
            : bd::launch_attend_tiles(*a, c.head_dim, fp8, true, per * 8, st));
    if (s != BITDELTA_OK) return s;
  }
  const int blocks = (int)(p.kind == Kind::kRows ? p.row_units : p.row_workers);
  bitdelta_status s = bd::status_of_hip(
      fp4 ? bd::launch_attend4_rows(*a, c.head_dim, p.columns, blocks, st)
          : bd::launch_attend_rows(*a, c.head_dim, fp8, p.columns, blocks, st));
  if (s != BITDELTA_OK || p.kind == Kind::kRows) return s;
  // units of 32 pieces and more are few: 64 rows of 96 pieces 5 us instead of 11.  (The wider caches' would gain
  // as much, 64 rows of 64 pieces 4.9 against 8.3, but the order of their sums, and with it the last bits of
  // results they have had before, would be another.)
  const bool many = fp4 && p.row_workers >= 32 * p.row_units;
  return bd::status_of_hip(bd::launch_attend_combine(*a, c.head_dim, many, st));
}

bitdelta_status check_workspace(const Plan& p, const void* ws, size_t bytes) {
  if (p.total == 0) return BITDELTA_OK;
  if (!ws) return bytes == 0 ? BITDELTA_ERR_WORKSPACE : BITDELTA_ERR_INVALID_ARG;
  if (!aligned(ws, 16)) return BITDELTA_ERR_ALIGNMENT;
  return bytes < p.total ? BITDELTA_ERR_WORKSPACE : BITDELTA_OK;
}

bitdelta_status check_table(const void* table, int32_t width, const void* lens, int32_t page_size) {
  if (width < 0) return BITDELTA_ERR_INVALID_ARG;
  if (!lens || (!table && width > 0)) return BITDELTA_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(lens, 4)) return BITDELTA_ERR_ALIGNMENT;
  if ((int64_t)width * page_size > kMaxKeys) return BITDELTA_ERR_UNSUPPORTED;
  return BITDELTA_OK;
}

// Steps of all sequences are summed in 32 bits; the tables' capacity bounds them.  (The steps of prefixes
// in row tiles then fit, too: they have half the keys, but a tile holds at least 4 sequences, or the last
// ones of one of at most 65 segments.)
bool steps_fit(int64_t sequences, int64_t keys) {
  return sequences * ((keys + bd::kRowStep - 1) / bd::kRowStep) < int64_t(1) << 31;
}

bool shared_sizes_ok(int64_t tokens, int32_t heads, const bitdelta_kv_cache* cache, int32_t width,
                     int32_t pwidth, const int32_t* offs, int32_t nseg, bitdelta_status* s) {
  *s = bd::check_kv_cache(cache, heads);
  if (*s == BITDELTA_OK && (width < 0 || pwidth < 0)) *s = BITDELTA_ERR_INVALID_ARG;
  if (*s == BITDELTA_OK) *s = check_segments(tokens, offs, nseg);
  if (*s == BITDELTA_OK && (tokens > BITDELTA_ATTEND_MAX_SEQS || tokens * heads > kMaxRows ||
                            tokens * cache->kv_heads > kMaxUnits ||
                            ((int64_t)width + pwidth) * cache->page_size > kMaxKeys ||
                            !steps_fit(tokens, ((int64_t)width + pwidth) * cache->page_size)))
    *s = BITDELTA_ERR_UNSUPPORTED;
  return *s == BITDELTA_OK;
}

bitdelta_status check_window(int64_t tokens, int32_t heads, const bitdelta_kv_cache* cache,
                             int32_t batch, int32_t width, int32_t max_q, int32_t window,
                             int32_t sinks) {
  bitdelta_status s = bd::check_kv_cache(cache, heads);
  if (s != BITDELTA_OK) return s;
  if (batch < 0 || width < 0 || max_q < 1 || window < 1 || sinks < 0) return BITDELTA_ERR_INVALID_ARG;
  if (batch > BITDELTA_ATTEND_MAX_SEQS || (int64_t)width * cache->page_size > kMaxKeys ||
      tokens * heads > kMaxRows || (int64_t)batch * cache->kv_heads > kMaxUnits ||
      !steps_fit(batch, std::min<int64_t>((int64_t)width * cache->page_size, (int64_t)window + max_q - 1 + sinks)))
    return BITDELTA_ERR_UNSUPPORTED;
  return BITDELTA_OK;
}

}  // namespace

extern "C" {

size_t bitdelta_attend_shared_workspace_bytes(int64_t tokens, int32_t heads,
                                              const bitdelta_kv_cache* cache, int32_t table_width,
                                              int32_t prefix_width, const int32_t* seg_offsets,
                                              int32_t num_segments) {
  bitdelta_status s;
  if (tokens < 1 || !shared_sizes_ok(tokens, heads, cache, table_width, prefix_width, seg_offsets,
                                     num_segments, &s))
    return 0;
  return plan_shared(tokens, heads, *cache, table_width, prefix_width, seg_offsets, num_segments).total;
}

bitdelta_status bitdelta_attend_shared(const bitdelta_attend_rows* rows,
                                       const bitdelta_kv_cache* cache, const int32_t* table,
                                       int32_t table_width, const int32_t* lens,
                                       const int32_t* prefix_table, int32_t prefix_width,
                                       const int32_t* prefix_lens, const int32_t* seg_offsets,
                                       int32_t num_segments, void* workspace,
                                       size_t workspace_bytes, bitdelta_stream stream) {
  bitdelta_status s = check_rows(rows, BITDELTA_ATTEND_MAX_SEQS);
  if (s != BITDELTA_OK) return s;
  if (rows->tokens == 0) return BITDELTA_OK;
  if (!shared_sizes_ok(rows->tokens, rows->heads, cache, table_width, prefix_width, seg_offsets,
                       num_segments, &s))
    return s;
  s = check_scales(*rows, *cache);
  if (s == BITDELTA_OK) s = check_table(table, table_width, lens, cache->page_size);
  if (s == BITDELTA_OK && prefix_width > 0)
    s = check_table(prefix_table, prefix_width, prefix_lens, cache->page_size);
  if (s != BITDELTA_OK) return s;
  const Plan p = plan_shared(rows->tokens, rows->heads, *cache, table_width, prefix_width,
                             seg_offsets, num_segments);
  s = check_workspace(p, workspace, workspace_bytes);
  if (s != BITDELTA_OK) return s;
  bd::AttendArgs a{};
  fill(&a, *rows, *cache);
  a.table = table;
  a.lens = lens;
  a.prefix_table = prefix_table;
  a.prefix_lens = prefix_lens;
  a.width = table_width;
  a.pwidth = prefix_width;
  a.batch = a.tokens;
  a.max_q = 1;
  a.nseg = num_segments;
  for (int i = 0; i <= num_segments; ++i) a.seg_offsets[i] = seg_offsets[i];
  if (prefix_width == 0) {
    // no prefixes: one segment, with a length that counts as 0 in a table of width 0 whatever it is
    a.prefix_lens = lens;
    a.nseg = 1;
    a.seg_offsets[1] = a.tokens;
  }
  return run(&a, p, *cache, workspace, stream);
}

size_t bitdelta_attend_window_workspace_bytes(int64_t tokens, int32_t heads,
                                              const bitdelta_kv_cache* cache, int32_t batch,
                                              int32_t table_width, int32_t max_q_len,
                                              int32_t window, int32_t sinks) {
  if (tokens < 1 || batch < 1 ||
      check_window(tokens, heads, cache, batch, table_width, max_q_len, window, sinks) != BITDELTA_OK)
    return 0;
  return plan_window(heads, *cache, batch, table_width, max_q_len, window, sinks).total;
}

bitdelta_status bitdelta_attend_window(const bitdelta_attend_rows* rows,
                                       const bitdelta_kv_cache* cache, int32_t batch,
                                       const int32_t* table, int32_t table_width,
                                       const int32_t* lens, const int32_t* q_offsets,
                                       int32_t max_q_len, int32_t window, int32_t sinks,
                                       void* workspace, size_t workspace_bytes,
                                       bitdelta_stream stream) {
  bitdelta_status s = check_rows(rows, int64_t(1) << 30);
  if (s != BITDELTA_OK) return s;
  if (batch == 0 || rows->tokens == 0) return BITDELTA_OK;
  s = check_window(rows->tokens, rows->heads, cache, batch, table_width, max_q_len, window, sinks);
  if (s == BITDELTA_OK) s = check_scales(*rows, *cache);
  if (s == BITDELTA_OK) s = check_table(table, table_width, lens, cache->page_size);
  if (s != BITDELTA_OK) return s;
  if (!aligned(q_offsets, 4)) return BITDELTA_ERR_ALIGNMENT;
  if (!q_offsets && (max_q_len != 1 || rows->tokens != batch)) return BITDELTA_ERR_SHAPE;
  const Plan p = plan_window(rows->heads, *cache, batch, table_width, max_q_len, window, sinks);
  s = check_workspace(p, workspace, workspace_bytes);
  if (s != BITDELTA_OK) return s;
  bd::AttendArgs a{};
  fill(&a, *rows, *cache);
  a.table = table;
  a.lens = lens;
  a.q_offsets = q_offsets;
  a.width = table_width;
  a.batch = batch;
  a.max_q = max_q_len;
  a.window = window;
  a.sinks = sinks;
  return run(&a, p, *cache, workspace, stream);
}

}  // extern "C"
