// Internal declarations of the paged-cache attention kernels (attend.hip) and the index arithmetic
// they share with the host.  The index functions touch no GPU state, so that a host program can
// check them against its own buffers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bd {

constexpr int kAttendMaxSeqs = 1024;      // sequences per call: their step counts are summed in LDS
constexpr int kAttendMaxSegments = 65;
constexpr int kAttendMaxGroup = 64;       // query heads per kv head
constexpr int kTileRows = 256;            // query rows of a tile workgroup (8 waves of 32)
constexpr int kTileKeys = 64;             // keys per step of a tile workgroup
constexpr int kRowKeys = 32;              // keys per step of one wave of a row workgroup
constexpr int kRowWaves = 4;
constexpr int kRowStep = kRowKeys * kRowWaves;  // keys per step of a row workgroup

// Quotients by the page size for 0 <= n < 2^31: with s = ceil(log2 d) and
// mul = ceil(2^(31 + s) / d), which fits 32 bits, floor(n / d) = (n * mul) >> (31 + s) exactly.
struct PageDiv {
  uint32_t mul;
  int32_t shift;
};
inline PageDiv make_page_div(uint32_t d) {
  int s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t two = uint64_t(1) << (31 + s);
  return PageDiv{(uint32_t)((two + d - 1) / d), 31 + s};
}
__host__ __device__ __forceinline__ int page_quotient(int n, PageDiv d) {
  return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
}

// A paged cache: strides in 16-byte units, row bytes contiguous.
struct PagedCache {
  const unsigned char* k;
  const unsigned char* v;
  uint32_t k_page, k_token, v_page, v_token;
  int64_t k_head, v_head;       // bytes
  int32_t num_pages, page_size;
  PageDiv div;
};

// Where a key sits: page id and slot, id -1 when the table has no such page (entry out of range).
__host__ __device__ __forceinline__ int page_id_checked(int id, int num_pages) {
  return (uint32_t)id < (uint32_t)num_pages ? id : -1;
}
// Byte offset of a slot's row, from strides in 16-byte units: two 32 x 32 -> 64 bit products.
__host__ __device__ __forceinline__ int64_t page_row_bytes(int id, int slot, uint32_t page_stride,
                                                           uint32_t token_stride) {
  return (int64_t)(((uint64_t)(uint32_t)id * page_stride + (uint64_t)(uint32_t)slot * token_stride) << 4);
}

// The keys a set of queries reads, as one virtual list of n keys: the first na are positions
// 0 .. na - 1 of the table at row a, the rest positions lo, lo + 1, ... of the table at row b.
struct KeyList {
  const int32_t* ta;
  const int32_t* tb;
  int wa, wb;  // entries of the two table rows
  int na, lo, n;
};
__host__ __device__ __forceinline__ int key_position(const KeyList& l, int vp) {
  return vp < l.na ? vp : vp - l.na + l.lo;
}
// Index of vp's page in its table row, or -1 past the list's end or the table's width.
__host__ __device__ __forceinline__ int key_table_index(const KeyList& l, int vp, int page) {
  if ((uint32_t)vp >= (uint32_t)l.n) return -1;
  return page < (vp < l.na ? l.wa : l.wb) ? page : -1;
}
// Window keys of queries at positions p0 .. len - 1 (p0 may be negative): first na sinks, then
// the positions from lo on.
__host__ __device__ __forceinline__ KeyList window_keys(const int32_t* row, int width, int len,
                                                        int p0, int window, int sinks) {
  KeyList l;
  l.ta = l.tb = row;
  l.wa = l.wb = width;
  const int64_t lo = (int64_t)p0 - window + 1;
  l.lo = lo > 0 ? (lo < len ? (int)lo : len) : 0;
  l.na = sinks < l.lo ? sinks : l.lo;
  l.n = l.na + len - l.lo;
  return l;
}

// The query rows of a chunk that are computed: of the rows q0 .. q1 - 1 the first max_q, and of those
// the ones in [0, tokens).  Row q1 - 1 is the token at position len - 1, whether it is computed or not.
struct ChunkRows {
  int first, count;
  int p0;  // position of the first
};
__host__ __device__ __forceinline__ ChunkRows chunk_rows(int q0, int q1, int len, int max_q, int tokens) {
  const int64_t limit = (int64_t)q0 + max_q;
  const int first = q0 > 0 ? q0 : 0;
  int64_t end = q1 < limit ? q1 : limit;
  if (end > tokens) end = tokens;
  ChunkRows c;
  c.first = first;
  c.count = end > first ? (int)(end - first) : 0;
  // far below 0 (offsets that are none) every token is without keys, wherever it is
  const int64_t p0 = (int64_t)len - ((int64_t)q1 - first);
  c.p0 = p0 < -(1 << 30) ? -(1 << 30) : (int)(p0 < len ? p0 : len);
  return c;
}

// Work split: `total` steps over `workers` workgroups, worker w taking steps
// [w * total / workers, (w + 1) * total / workers).  Never more workers than steps, so that each
// worker has a step, and a unit's pieces are those of all workers from its first step's owner to
// its last step's.
__host__ __device__ __forceinline__ int split_workers(int64_t total, int workers) {
  return total < workers ? (int)total : workers;
}
// a / b of values that are not negative; 64-bit divisions cost hundreds of instructions
__host__ __device__ __forceinline__ int64_t split_quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
__host__ __device__ __forceinline__ int64_t split_begin(int64_t w, int64_t total, int workers) {
  return split_quotient(w * total, workers);
}
__host__ __device__ __forceinline__ int split_owner(int64_t step, int64_t total, int workers) {
  return (int)split_quotient((step + 1) * workers - 1, total);
}

struct AttendArgs {
  const uint16_t* q;
  int64_t q_token, q_head;      // strides in elements
  uint16_t* out;
  int64_t o_token, o_head;
  float* lse;                   // [tokens][heads] or null
  PagedCache cache;
  const int32_t* table;         // [batch][width]
  const int32_t* lens;          // [batch]
  const int32_t* q_offsets;     // [batch + 1], null: one token per sequence
  const int32_t* prefix_table;  // [segments][pwidth]
  const int32_t* prefix_lens;   // [segments]
  int32_t width, pwidth;
  int32_t batch, tokens, heads, kv_heads, group;
  int32_t max_q;                // tokens per sequence at most
  int32_t window, sinks;        // window op; shared op: no limit
  int32_t nseg;                 // 0: no prefixes (window op)
  int32_t rows;                 // partial rows per unit of the row kernel (max_q * group)
  float c;                      // scale * k_scale * log2(e): scores enter exp2
  float v_scale;
  int32_t workers;              // row kernel workgroups
  int32_t tile_workers;         // tile kernel workgroups that split the prefixes
  int32_t halves;               // tile kernel: units of up to 128 rows take two key tiles a step
  int32_t row_prefix;           // row kernel: 1 = a sequence's keys start with its prefix
  int32_t direct;               // row kernel: one workgroup per unit, written without partials
  // workspace
  int32_t* scan;                // [batch + 1] first step of each sequence, x kv_heads = of its units
  float* part_o;                // row partials [slot][rows][dim]
  float* part_ml;               // [slot][rows][2]: running maximum (log2 units) and sum
  int32_t* tile_segs;           // [segments + 1] row tiles before each segment
  int32_t* tile_scan;           // [segments + 1] steps before each segment, x kv_heads
  float* tile_o;                // tile partials [slot][kTileRows][dim]
  float* tile_ml;               // [slot][kTileRows][2]
  int32_t seg_offsets[kAttendMaxSegments + 1];
};

// dim: 64 or 128; fp8: e4m3 cache (else bf16); columns: 16-column blocks of the row kernel (1, 2, 4)
hipError_t launch_attend_rows(const AttendArgs& a, int dim, bool fp8, int columns, int blocks,
                              hipStream_t stream);
hipError_t launch_attend_tiles(const AttendArgs& a, int dim, bool fp8, bool prefix, int blocks,
                               hipStream_t stream);
hipError_t launch_attend_combine(const AttendArgs& a, int dim, hipStream_t stream);

}  // namespace bd
