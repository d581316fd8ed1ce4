// Attention over a paged cache: decode with prefixes shared by the segments of a batch, and causal
// attention with a sliding window and first tokens that stay visible.
//
// Mathematics, per query row q of kv head h and its visible keys j:
//   s_j = c * (q . k_j),  c = scale * k_scale * log2(e)
//   m = max_j s_j,  l = sum_j 2^(s_j - m),  o = v_scale / l * sum_j 2^(s_j - m) v_j
// in one pass: the running maximum m and sum l are kept in fp32 per row, and the fp32 output sums
// are rescaled when m grows.  Scores are computed transposed, S^T = K Q^T, so that the matrix
// instruction leaves each lane with scores of ONE query row: the softmax needs no shared memory,
// and the weights are already the B operand of O^T = V^T P^T.  The order of the keys inside a
// product is free as long as both operands agree, so the A operand V^T is read from LDS
// (transposed reads) in the key order the scores came out in.
#include <type_traits>

#include "attend_device.h"

namespace bd {
namespace {

// ---------------------------------------------------------------------------------------------
// Row kernel: up to 16 * NC query rows (the heads of one kv head, for one or a few tokens) against
// a key list.  Bound by reading the cache: each of a workgroup's 4 waves takes 32 keys of a
// 128-key step on its own (no barrier in the loop), its K rows straight from memory into operand
// registers (4 lanes take 64 bytes of a row) and its V rows through 8 KiB of its own LDS.  The
// waves' sums meet at the end of a piece.  A split launch gives each of as many workgroups as fit at
// a time an equal run of all units' steps, so unequal lengths leave none idle; more workgroups than
// fit took a second turn (145 against 120 us for the own keys of 256 sequences, bf16, dim 128).
// Measured: 64 sequences x 8 kv heads of 6.9k keys, e4m3, dim 128, 902 MB in 187 us, 4.8 TB/s, what a
// large copy reaches; the 448 MB of own keys of 256 sequences, bf16, in 121 us, 3.7 TB/s; one
// sequence's 4.3 MB 9 us, which is latency.  Registers decide how many fit; at dim 128 some variants
// spill: 8 for single tokens from e4m3 (36 bytes a lane), 23 to 87 with 2 and 4 column blocks from bf16,
// up to 47 from e4m3.
// ---------------------------------------------------------------------------------------------
template <int D, bool FP8, int NC>
struct RowLoop {
  static constexpr int kLoads = FP8 ? D / 64 : D / 32;  // 16-byte loads of a row per lane
  static constexpr int kSteps = D / 32;                 // matrix steps over D
  static constexpr int kTiles = D / 16;                 // 16-row tiles of O^T

  u32x4 q[NC][kSteps];
  f32x4 o[NC][kTiles];
  float m[NC], l[NC];
  int pos[NC];   // the column's token position (window op with several tokens)
  u32x4 kr[2][kLoads], vr[2][kLoads];
  int id[2], slot[2];
  bool ok[2];

  __device__ __forceinline__ void lookup(const AttendArgs& a, const KeyList& kl, int base, int j) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int p = base + 16 * r + j;
      const int kp = key_position(kl, p);
      const int page = page_quotient(kp < 0 ? 0 : kp, a.cache.div);
      const int at = key_table_index(kl, p, page);
      slot[r] = kp - page * a.cache.page_size;
      // the entry is only checked when it is used: the load stays in flight
      id[r] = at >= 0 ? (p < kl.na ? kl.ta : kl.tb)[at] : -1;
    }
  }
  __device__ __forceinline__ void fetch(const AttendArgs& a, int h, int g) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      // absent keys read page 0 and are cleared before they are used
      ok[r] = page_id_checked(id[r], a.cache.num_pages) >= 0;
      const int page = ok[r] ? id[r] : 0, at = ok[r] ? slot[r] : 0;
      const unsigned char* kp = a.cache.k + page_row_bytes(page, at, a.cache.k_page, a.cache.k_token) +
                                (int64_t)h * a.cache.k_head + 16 * g;
      const unsigned char* vp = a.cache.v + page_row_bytes(page, at, a.cache.v_page, a.cache.v_token) +
                                (int64_t)h * a.cache.v_head + 16 * g;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) kr[r][i] = *reinterpret_cast<const u32x4*>(kp + 64 * i);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) vr[r][i] = *reinterpret_cast<const u32x4*>(vp + 64 * i);
    }
  }
  // what the memory holds for an absent key must not reach the sums
  __device__ __forceinline__ void clear_absent() {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (!ok[r])
#pragma unroll
        for (int i = 0; i < kLoads; ++i) kr[r][i] = vr[r][i] = u32x4{0, 0, 0, 0};
  }
};

// MULTI: units may hold several tokens, which see different keys
template <int D, bool FP8, int NC, bool MULTI>
__global__ __launch_bounds__(256, NC == 1 && !MULTI && (FP8 || D == 64) ? 3 : (NC <= 2 ? 2 : 1))
void attend_row_kernel(const AttendArgs a) {
  using Loop = RowLoop<D, FP8, NC>;
  constexpr int kWaveLds = kRowKeys * D * 2;
  __shared__ __attribute__((aligned(16))) unsigned char vlds[kRowWaves * kWaveLds];
  __shared__ float ml[kRowWaves][16][2];
  __shared__ int scan[kAttendMaxSeqs + 1], lens[kAttendMaxSeqs];
  __shared__ int wave_sum[kRowWaves];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = lane & 15, g = lane >> 4;
  unsigned char* const vl = vlds + wave * kWaveLds;

  int64_t x, x_end, total = 0;
  if (a.direct) {
    x = 0;
    x_end = 1;
  } else {
    block_scan<256>(scan, wave_sum, a.batch, [&](int b) {
      lens[b] = a.lens[b];
      return row_steps(row_unit(a, b, lens[b]));
    });
    total = (int64_t)scan[a.batch] * a.kv_heads;
    if (blockIdx.x == 0)
      for (int i = tid; i <= a.batch; i += 256) a.scan[i] = scan[i];
    const int workers = split_workers(total, a.workers);
    if ((int)blockIdx.x >= workers) return;
    x = split_begin(blockIdx.x, total, workers);
    x_end = split_begin(blockIdx.x + 1, total, workers);
  }

  while (x < x_end) {
    int b, h, s_begin, s_end;
    RowUnit u;
    if (a.direct) {
      b = blockIdx.x / a.kv_heads;
      h = blockIdx.x - b * a.kv_heads;
      u = row_unit(a, b);
      s_begin = 0;
      s_end = row_steps(u);
      x = x_end;
    } else {
      b = scan_find(scan, a.batch, (int)(x / a.kv_heads));
      u = row_unit(a, b, lens[b]);
      const int s = row_steps(u);
      const int64_t x0 = (int64_t)scan[b] * a.kv_heads;
      h = (int)((x - x0) / s);
      s_begin = (int)(x - x0 - (int64_t)h * s);
      s_end = (int)(x_end - x < s - s_begin ? s_begin + (x_end - x) : s);
    }
    const int rows = u.nq * a.group;
    const KeyList kl = u.keys;
    Loop w;
    // ---- queries: column j of block c is row 16c + j, token (row / group), head (row % group)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int row = 16 * c + j;
      const int t = row / a.group, hh = row - t * a.group;
      w.pos[c] = u.p0 + t;
      w.m[c] = kNegInf;
      w.l[c] = 0.f;
#pragma unroll
      for (int i = 0; i < Loop::kTiles; ++i) w.o[c][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      const uint16_t* qp = a.q + (int64_t)(u.t0 + t) * a.q_token + (int64_t)(h * a.group + hh) * a.q_head;
#pragma unroll
      for (int s = 0; s < Loop::kSteps; ++s) {
        // the 8 dims of step s that K's register holds for this lane
        const int d = FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
        w.q[c][s] = row < rows ? *reinterpret_cast<const u32x4*>(qp + d) : u32x4{0, 0, 0, 0};
      }
    }

    int base = s_begin * kRowStep + wave * kRowKeys;
    const int end = s_end * kRowStep;
    if (base < end) {
      w.lookup(a, kl, base, j);
      w.fetch(a, h, g);
      if (base + kRowStep < end) w.lookup(a, kl, base + kRowStep, j);
    }
    for (; base < end; base += kRowStep) {
      const bool ok0 = w.ok[0], ok1 = w.ok[1];
      // keys of the tile that exist, bit (key): lanes 0..15 speak for keys 0..15 and 16..31
      const unsigned valid = (unsigned)(__ballot(ok0) & 0xFFFFull) |
                             ((unsigned)(__ballot(ok1) & 0xFFFFull) << 16);
      if (valid != 0xFFFFFFFFu) w.clear_absent();
      // keys whose values are not all finite: those values are taken out here and added below for
      // the tokens that see them, since their product with a zero weight would be NaN
      unsigned odd = 0;
      if constexpr (MULTI) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          bool f = false;
#pragma unroll
          for (int i = 0; i < Loop::kLoads; ++i) f |= clear_odd<FP8>(&w.vr[r][i]);
          uint64_t m = __ballot(f);
          m |= m >> 32;
          m |= m >> 16;
          odd |= (unsigned)(m & 0xFFFFull) << (16 * r);
        }
      }
      // ---- V into LDS, scores from K
      f32x4 s[NC][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int i = 0; i < Loop::kLoads; ++i) {
          const int row = 16 * r + j;
          if constexpr (FP8) {
            const u32x4 v = w.vr[r][i];
            *reinterpret_cast<u32x4*>(vl + v_unit<D>(row, 8 * i + 2 * g)) = fp8x8_to_bf16(v[0], v[1]);
            *reinterpret_cast<u32x4*>(vl + v_unit<D>(row, 8 * i + 2 * g + 1)) = fp8x8_to_bf16(v[2], v[3]);
          } else {
            *reinterpret_cast<u32x4*>(vl + v_unit<D>(row, 4 * i + g)) = w.vr[r][i];
          }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) s[c][r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < Loop::kLoads; ++i) {
          const u32x4 kv = w.kr[r][i];
          if constexpr (FP8) {
            const u32x4 k0 = fp8x8_to_bf16(kv[0], kv[1]), k1 = fp8x8_to_bf16(kv[2], kv[3]);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              s[c][r] = mfma16(k0, w.q[c][2 * i], s[c][r]);
              s[c][r] = mfma16(k1, w.q[c][2 * i + 1], s[c][r]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < NC; ++c) s[c][r] = mfma16(kv, w.q[c][i], s[c][r]);
          }
        }
      }
      // ---- the next tile's rows are on their way while this one is worked on
      if (base + kRowStep < end) {
        w.fetch(a, h, g);
        if (base + 2 * kRowStep < end) w.lookup(a, kl, base + 2 * kRowStep, j);
      }

      // ---- mask: lane (j, g) holds keys 4g + i (s[.][0]) and 16 + 4g + i (s[.][1]) of column j
      u32x4 p[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (valid != 0xFFFFFFFFu || MULTI) {
          const unsigned mine = valid >> (4 * g);
          const Sight at = sight(kl, w.pos[c], a.sinks, base + 4 * g);
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = 16 * r + i;  // + 4 g
              bool seen = (mine >> key) & 1u;
              if constexpr (MULTI) seen = seen & at.sees(key, a.window);
              const float v = s[c][r][i];
              s[c][r][i] = seen ? v : kNegInf;
            }
        }
        float t = kNegInf;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t = __builtin_elementwise_maximum(t, __builtin_elementwise_maximum((float)s[c][0][i], (float)s[c][1][i]));
        t = half_max(row_max(t)) * a.c;
        if (__any(t > w.m[c] + kRescale)) {
          const float mn = fmaxf(w.m[c], t);
          const float f = mn == kNegInf ? 1.f : exp2_fast(w.m[c] - mn);
          w.m[c] = mn;
          w.l[c] *= f;
#pragma unroll
          for (int i = 0; i < Loop::kTiles; ++i) w.o[c][i] *= f;
        }
        const float mb = w.m[c] == kNegInf ? 0.f : w.m[c];
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = exp2_fast(__builtin_fmaf(s[c][i >> 2][i & 3], a.c, -mb));
          w.l[c] += e[i];
        }
        // weights enter the product as bf16, the matrix instruction's operand type (off by at most 2^-8
        // of themselves, as the values they weigh were when stored); the sum l keeps them in fp32
        p[c] = u32x4{pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]),
                     pack_bf16(e[6], e[7])};
      }

      // ---- O^T += V^T P^T: the lane's 8 keys are 4g .. 4g + 3 and 16 + 4g .. 16 + 4g + 3
      const int vr0 = 4 * g + (j >> 2), vu = (j & 3) >> 1, vb = 8 * (j & 1);
#pragma unroll
      for (int i = 0; i < Loop::kTiles; ++i) {
        const u32x2 lo = lds_read_tr(vl + v_unit<D>(vr0, 2 * i + vu) + vb);
        const u32x2 hi = lds_read_tr(vl + v_unit<D>(16 + vr0, 2 * i + vu) + vb);
        const u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
        for (int c = 0; c < NC; ++c) w.o[c][i] = mfma16(v, p[c], w.o[c][i]);
      }
      if constexpr (MULTI) {
        for (; odd; odd &= odd - 1) {
          const int vp = base + __builtin_ctz(odd);
          const unsigned char* row = value_row(a.cache, kl, vp, h);
          if (!row) continue;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const bool seen = sees(kl, w.pos[c], a.window, a.sinks, vp);
#pragma unroll
            for (int i = 0; i < Loop::kTiles; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float x = w.o[c][i][e];
                w.o[c][i][e] = seen ? x + odd_value<FP8>(row, 16 * i + 4 * g + e) : x;
              }
          }
        }
      }
    }

    // ---- the waves' sums, block of columns by block of columns
    const int64_t slot = a.direct ? 0 : blockIdx.x + (int64_t)b * a.kv_heads + h;
    for (int c = 0; c < NC; ++c) {
      if (16 * c >= rows) break;
      float mc, lc;
      f32x4 oc[Loop::kTiles];
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
        if (cc == c) {
          mc = w.m[cc];
          lc = w.l[cc];
#pragma unroll
          for (int i = 0; i < Loop::kTiles; ++i) oc[i] = w.o[cc][i];
        }
      lc = half_sum(row_sum(lc));
      __syncthreads();  // the V tiles, or the last block's sums, are no longer read
      float* const ow = reinterpret_cast<float*>(vl);  // [16 columns][D]
#pragma unroll
      for (int i = 0; i < Loop::kTiles; ++i)
        *reinterpret_cast<f32x4*>(ow + j * D + 16 * i + 4 * g) = oc[i];
      if (g == 0) {
        ml[wave][j][0] = mc;
        ml[wave][j][1] = lc;
      }
      __syncthreads();
      constexpr int kQuads = 16 * D / 4 / 256;  // f32x4 per thread
#pragma unroll
      for (int e = 0; e < kQuads; ++e) {
        const int idx = tid + 256 * e, col = idx / (D / 4), d4 = idx - col * (D / 4);
        const int row = 16 * c + col;
        if (row < rows) {
          float mx = kNegInf;
#pragma unroll
          for (int v = 0; v < kRowWaves; ++v) mx = fmaxf(mx, ml[v][col][0]);
          const float mb = mx == kNegInf ? 0.f : mx;
          float lt = 0.f;
          f32x4 ot = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int v = 0; v < kRowWaves; ++v) {
            const float f = exp2_fast(ml[v][col][0] - mb);
            lt += f * ml[v][col][1];
            ot += f * *reinterpret_cast<const f32x4*>(
                          reinterpret_cast<const float*>(vlds + v * kWaveLds) + col * D + 4 * d4);
          }
          if (a.direct) {
            const int t = row / a.group, hh = h * a.group + row - t * a.group;
            const float inv = lt > 0.f ? a.v_scale / lt : (lt == 0.f ? 0.f : lt);
            u32x2 pk = {pack_bf16(ot[0] * inv, ot[1] * inv), pack_bf16(ot[2] * inv, ot[3] * inv)};
            *reinterpret_cast<u32x2*>(a.out + (int64_t)(u.t0 + t) * a.o_token +
                                      (int64_t)hh * a.o_head + 4 * d4) = pk;
            if (a.lse && d4 == 0)
              a.lse[(int64_t)(u.t0 + t) * a.heads + hh] = lt == 0.f ? kNegInf : (mb + __builtin_log2f(lt)) * kLn2;
          } else {
            *reinterpret_cast<f32x4*>(a.part_o + (slot * a.rows + row) * D + 4 * d4) = ot;
            if (d4 == 0) {
              a.part_ml[(slot * a.rows + row) * 2] = mx;
              a.part_ml[(slot * a.rows + row) * 2 + 1] = lt;
            }
          }
        }
      }
    }
    if (!a.direct) {
      __syncthreads();  // the sums are read before the next piece's V tiles land
      x += s_end - s_begin;
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Tile kernel: 256 query rows (tokens x the heads of one kv head) against a key list in 64-key
// steps.  8 waves of 32 rows; K and V tiles in LDS.  A bf16 cache's rows go straight from memory
// into LDS, three steps ahead, in four buffers; an e4m3 cache's rows pass through registers, which
// widen them, one step ahead, in two.  Where a segment's rows fill at most half the waves (and the
// cache is bf16), the other half takes a second key tile of the same step, and both halves' sums are
// joined later with the pieces (64 sequences of 14 segments: 70.0 -> 65.6 us).
//
// Bound by the chain of a step within a wave: scores (32 matrix instructions), softmax, values (32),
// about 2.2 us, with two waves a SIMD to fill each other's gaps; vector and matrix instructions each
// are busy 44% of the time, so that neither is at its limit.  Measured, bf16, dim 128, 64 heads on 8: 8192 new tokens of 16384, window
// 4096, 1.10 TFLOP in 1130 us, 970 TFLOP/s (a large matrix product reaches 1184); 4 requests of up to
// 2048 tokens, window 1024, 108 GFLOP in 168 us, 640 TFLOP/s; the same from an e4m3 cache 1156 and 172 us.
// Plain causal attention of 8192 tokens 1143 us, 960 TFLOP/s.  Prefixes of 256 sequences in 14 segments:
// 53 GFLOP on 300 MB in 110 us.  A unit's keys are not split: 16 tokens over 4096 keys, 8 units, take 88 us.
// Tried and slower or no faster: the next step's scores under this step's softmax (1133 in the
// compiler's order, 1171 to 1211 interleaved by hand), the second wave of each SIMD a third of a step
// late (4% slower),
// wave priorities around the products (1291 against 1225 us), a barrier every second step (1225
// against 1220), values with infinities or NaN multiplied key by key (spills, 5 times slower).
// ---------------------------------------------------------------------------------------------
// Byte offsets of a key's rows; bit 0 of k: there is no such key (offsets 0).
struct RowPlace {
  int64_t k, v;
};
// Where the lane's key sits: its table entry (null: no such key), and the rows' offsets from it.
struct KeyLookup {
  const int32_t* entry;
  int slot;
  __device__ __forceinline__ KeyLookup(const PagedCache& c, const KeyList& kl, int vp) {
    const int kp = key_position(kl, vp);
    const int page = page_quotient(kp < 0 ? 0 : kp, c.div);
    const int at = key_table_index(kl, vp, page);
    slot = kp - page * c.page_size;
    entry = at >= 0 ? (vp < kl.na ? kl.ta : kl.tb) + at : nullptr;
  }
  __device__ __forceinline__ RowPlace place(const PagedCache& c, int id) const {
    const bool ok = entry && page_id_checked(id, c.num_pages) >= 0;
    const int p = ok ? id : 0, t = ok ? slot : 0;
    return RowPlace{page_row_bytes(p, t, c.k_page, c.k_token) | (ok ? 0 : 1),
                    page_row_bytes(p, t, c.v_page, c.v_token)};
  }
};

template <int D, bool FP8>
struct TileStage {
  static constexpr int kUnits = FP8 ? D / 16 : D / 8;      // 16-byte units of a row in memory
  static constexpr int kPer = 2 * kTileKeys * kUnits / 512;  // of K and V, per thread
  static constexpr int kRows = kPer >= 4 ? kPer / 2 : 1;   // rows a thread serves
  static constexpr int kKV = kPer >= 2 ? 2 : 1;            // both tensors, or one by thread half
  static constexpr int kRowStride = 512 / kUnits;          // rows between a thread's rows

  u32x4 r[kPer];
  bool ok[kRows];

  __device__ __forceinline__ int row(int tid, int i) const {
    return (tid / kUnits + i * kRowStride) & (kTileKeys - 1);
  }
  // k, v: this thread's unit of the head's first row; places: RowPlace of each of the step's keys
  __device__ __forceinline__ void fetch(const unsigned char* k, const unsigned char* v,
                                        const RowPlace* places, int tid) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const RowPlace at = places[row(tid, i)];
      // absent keys read page 0 and are cleared before they are stored
      ok[i] = (at.k & 1) == 0;
      if constexpr (kKV == 2) {
        r[i] = *reinterpret_cast<const u32x4*>(k + (at.k & ~15ll));
        r[kRows + i] = *reinterpret_cast<const u32x4*>(v + at.v);
      } else {
        r[i] = *reinterpret_cast<const u32x4*>(tid < 256 ? k + (at.k & ~15ll) : v + at.v);
      }
    }
  }
  template <bool kIsV>
  __device__ __forceinline__ void put(unsigned char* t, int rw, int u, const u32x4& v) const {
    auto at = [&](int uu) { return kIsV ? v_unit<D>(rw, uu) : k_unit<D>(rw, uu); };
    if constexpr (FP8) {
      *reinterpret_cast<u32x4*>(t + at(2 * u)) = fp8x8_to_bf16(v[0], v[1]);
      *reinterpret_cast<u32x4*>(t + at(2 * u + 1)) = fp8x8_to_bf16(v[2], v[3]);
    } else {
      *reinterpret_cast<u32x4*>(t + at(u)) = v;
    }
  }
  // state: per key, bit 0: it exists; bit 1 (edge steps, where some row does not see some key):
  // some of its values are not finite.  Those are stored as zeros, since their product with a zero
  // weight would be NaN, and added later for the rows that see them.
  __device__ __forceinline__ void store(unsigned char* kt, unsigned char* vt, int* state, bool edge,
                                        int tid) {
    const int u = tid % kUnits;
    bool every = true;
#pragma unroll
    for (int i = 0; i < kRows; ++i) every &= ok[i];
    if (!__all(every)) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (!ok[i]) {
          r[i] = u32x4{0, 0, 0, 0};
          if constexpr (kKV == 2) r[kRows + i] = u32x4{0, 0, 0, 0};
        }
    }
    int bits[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) bits[i] = ok[i];
    if (edge) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        bool f = false;
        if (kKV == 2 || tid >= 256) f = clear_odd<FP8>(&r[kKV == 2 ? kRows + i : i]);
        const uint64_t m = __ballot(f) >> ((tid & 63) & ~(kUnits - 1));  // of this key's units
        if (m & ((1ull << kUnits) - 1)) bits[i] |= 2;
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int rw = row(tid, i);
      if constexpr (kKV == 2) {
        put<false>(kt, rw, u, r[i]);
        put<true>(vt, rw, u, r[kRows + i]);
      } else if (tid < 256) {
        put<false>(kt, rw, u, r[i]);
      } else {
        put<true>(vt, rw, u, r[i]);
      }
      if (u == 0 && (kKV == 2 || tid >= 256)) state[rw] = bits[i];
    }
  }
};

template <int D, bool FP8, bool PREFIX>
__global__ __launch_bounds__(512, 2) void attend_tile_kernel(const AttendArgs a) {
  constexpr int kTile = kTileKeys * D * 2;
  constexpr int kSteps = D / 16;   // matrix steps over D of a score tile
  constexpr int kOut = D / 32;     // 32-row tiles of O^T
  constexpr int kBuffers = FP8 ? 2 : 4;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // K tiles, then V tiles
  unsigned char* const vbuf = smem + kBuffers * kTile;
  __shared__ int state[FP8 ? 2 : 8][kTileKeys];
  __shared__ RowPlace places[4][kTileKeys];
  __shared__ int entries[8][kTileKeys];
  __shared__ int scan[kAttendMaxSeqs + 1];
  __shared__ int segs[PREFIX ? kAttendMaxSegments + 1 : 1];
  __shared__ int wave_sum[8];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane & 31, hf = lane >> 5;
  const int tpt = kTileRows / a.group;  // tokens per tile

  const unsigned smem_at = __builtin_amdgcn_readfirstlane(lds_address(smem));
  const unsigned entries_at = __builtin_amdgcn_readfirstlane(lds_address(entries));

  // ---- work: prefix: a share of all (segment, row tile, kv head) units' steps; window: one unit
  int64_t x = 0, x_end = 1, total = 1;
  int w_id = blockIdx.x;
  if constexpr (PREFIX) {
    // workgroups go round robin over the 8 XCDs: give each XCD one run of the work, so that the
    // row tiles and heads that read the same pages share its L2
    auto tiles_of = [&](int s) { return (a.seg_offsets[s + 1] - a.seg_offsets[s] + tpt - 1) / tpt; };
    block_scan<512>(segs, wave_sum, a.nseg, tiles_of);
    block_scan<512>(scan, wave_sum, a.nseg, [&](int s) { return tiles_of(s) * prefix_steps(a, s); });
    if (blockIdx.x == 0)  // for the joining kernel
      for (int i = tid; i <= a.nseg; i += 512) {
        a.tile_segs[i] = segs[i];
        a.tile_scan[i] = scan[i];
      }
    total = (int64_t)scan[a.nseg] * a.kv_heads;
    const int workers = split_workers(total, a.tile_workers);
    const int per = (workers + 7) / 8;
    w_id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || w_id >= workers) return;
    x = split_begin(w_id, total, workers);
    x_end = split_begin(w_id + 1, total, workers);
  } else {
    block_scan<512>(scan, wave_sum, a.batch, [&](int b) {
      const RowUnit u = row_unit(a, b);
      return (u.nq + tpt - 1) / tpt;
    });
  }

  while (x < x_end) {
    KeyList kl;
    int t0, nt, p0 = 0, h, s_begin, s_end;  // steps of one key tile
    int64_t slot = 0;
    bool half = false;
    if constexpr (PREFIX) {
      const int sg = scan_find(scan, a.nseg, (int)(x / a.kv_heads));
      const int n0 = a.seg_offsets[sg], n = a.seg_offsets[sg + 1] - n0;
      const int len = clamp_len(a.prefix_lens[sg], a.pwidth, a.cache.page_size);
      const int steps = prefix_steps(a, sg);
      const int tiles = (n + tpt - 1) / tpt;
      half = halved(a, sg);
      int64_t r = x - (int64_t)scan[sg] * a.kv_heads;  // units: kv head major, then row tile
      h = (int)(r / ((int64_t)tiles * steps));
      r -= (int64_t)h * tiles * steps;
      const int rt = (int)(r / steps);
      s_begin = (int)(r - (int64_t)rt * steps);
      s_end = (int)(x_end - x < steps - s_begin ? s_begin + (x_end - x) : steps);
      x += s_end - s_begin;
      if (half) {
        s_begin *= 2;
        s_end = min(2 * s_end, (len + kTileKeys - 1) / kTileKeys);
      }
      t0 = n0 + rt * tpt;
      nt = n - rt * tpt < tpt ? n - rt * tpt : tpt;
      slot = w_id + (int64_t)segs[sg] * a.kv_heads + h * tiles + rt;
      const int32_t* row = a.prefix_table + (int64_t)sg * a.pwidth;
      kl = KeyList{row, row, a.pwidth, a.pwidth, 0, 0, len};
    } else {
      // heads fastest: with a multiple of 8 kv heads each XCD serves its own heads.  Later tiles
      // see more keys: they start first.
      const int tiles = scan[a.batch];
      const int ti = tiles - 1 - (int)blockIdx.x / a.kv_heads;
      if (ti < 0) return;
      h = (int)blockIdx.x % a.kv_heads;
      const int b = scan_find(scan, a.batch, ti);
      const RowUnit u = row_unit(a, b);
      const int rt = ti - scan[b];
      t0 = u.t0 + rt * tpt;
      nt = u.nq - rt * tpt < tpt ? u.nq - rt * tpt : tpt;
      p0 = u.p0 + rt * tpt;
      // keys up to the tile's last token
      const int len = p0 + nt < 0 ? 0 : p0 + nt;
      kl = window_keys(a.table + (int64_t)b * a.width, a.width, len, p0, a.window, a.sinks);
      s_begin = 0;
      s_end = (kl.n + kTileKeys - 1) / kTileKeys;
    }

    // ---- this lane's query row: 32 * (wave's rows) + q of the tile
    const int wave_rows = half ? wave & 3 : wave;
    const int row = 32 * wave_rows + q;
    const int t = row / a.group, hh = h * a.group + row - t * a.group;
    const bool live = t < nt;
    const int pq = p0 + t;
    // positions of the wave's first and last live token
    const int wt0 = 32 * wave_rows / a.group;
    const int wt1 = (32 * wave_rows + 31) / a.group < nt ? (32 * wave_rows + 31) / a.group : nt - 1;
    const bool wave_live = wt0 < nt;
    u32x4 qf[kSteps];
    {
      const uint16_t* qp = a.q + (int64_t)(t0 + t) * a.q_token + (int64_t)hh * a.q_head + 8 * hf;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        qf[s] = live ? *reinterpret_cast<const u32x4*>(qp + 16 * s) : u32x4{0, 0, 0, 0};
      // wait for the queries here: left to their first use, in the loop, the wait would be for the
      // copies on their way, too
#pragma unroll
      for (int s = 0; s < kSteps; ++s) asm volatile("" : "+v"(qf[s]));
    }
    f32x16 o[kOut];
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[i][e] = 0.f;
    float m = kNegInf, l = 0.f;

    // The pipeline: the keys of step t are looked up by one wave (wave t mod 8, one lane a key).
    // Table entries are copied into LDS, so that no register waits for them; two steps later the
    // rows' offsets are worked out, and a step later the rows' loads begin.
    constexpr int kAhead = FP8 ? 2 : 3;  // steps from the loads to the step they are for
    auto look_begin = [&](int s) {
      if (((s - s_begin) & 7) == wave) {
        const KeyLookup look(a.cache, kl, s * kTileKeys + lane);
        if (look.entry) copy4(look.entry, entries_at + wave * kTileKeys * 4);
      }
    };
    auto look_end = [&](int s) {
      if (((s - s_begin) & 7) == wave) {
        const KeyLookup look(a.cache, kl, s * kTileKeys + lane);
        const RowPlace at = look.place(a.cache, entries[wave][lane]);
        places[(s - s_begin) & 3][lane] = at;
        if constexpr (!FP8) state[(s - s_begin) & 7][lane] = (at.k & 1) == 0;
      }
    };
    // edge step: some row of the tile does not see some key of it (the same for all waves)
    auto hides = [&](int base) {
      if constexpr (PREFIX) return false;
      const int f = key_position(kl, base), last = key_position(kl, base + kTileKeys - 1);
      return base < kl.na || last > p0 || p0 + nt - 1 - f >= a.window;
    };
    const unsigned char* const kh = a.cache.k + (int64_t)h * a.cache.k_head;
    const unsigned char* const vh = a.cache.v + (int64_t)h * a.cache.v_head;
    TileStage<D, FP8> st;
    // bf16: each wave moves 8 rows of K and of V, a lane 16 bytes: the stored unit lane % kU of row
    // r holds the row's unit (lane % kU) ^ swizzle(r)
    constexpr int kU = D / 8, kCopies = kU / 8;  // units of a row; copies of each tensor per wave
    auto copy_rows = [&](int s) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int r0 = 8 * wave + i * (64 / kU), r = r0 + lane / kU, u = lane % kU;
        const RowPlace at = places[(s - s_begin) & 3][r];
        const unsigned to = smem_at + ((s - s_begin) & 3) * kTile + r0 * (D * 2);
        copy16(kh + (at.k & ~15ll) + ((k_unit<D>(r, u) - r * (D * 2))), to);
        copy16(vh + at.v + (v_unit<D>(r, u) - r * (D * 2)), to + kBuffers * kTile);
      }
    };
    for (int i = 0; i < kAhead + 3; ++i) look_begin(s_begin + i);
    wait_copies<0>();
    __syncthreads();  // the last unit's tiles and notes are no longer read
    for (int i = 0; i <= kAhead; ++i) look_end(s_begin + i);
    __syncthreads();
    if constexpr (FP8) {
      const int unit = 16 * (tid % TileStage<D, FP8>::kUnits);
      st.fetch(kh + unit, vh + unit, places[0], tid);
      st.store(smem, vbuf, state[0], hides(s_begin * kTileKeys), tid);
      st.fetch(kh + unit, vh + unit, places[1], tid);
      __syncthreads();
    } else {
      copy_rows(s_begin);
      if (s_begin + 1 < s_end) copy_rows(s_begin + 1);
      if (!half && s_begin + 2 < s_end) copy_rows(s_begin + 2);
    }

    // O^T += V^T P^T of step s: of 16 keys the lane's 8 are 4 hf .. + 3 and 8 + 4 hf .. + 3
    u32x4 p[4];
    const int l16 = lane & 15;
    const int v_row = 4 * hf + (l16 >> 2), v_un = 2 * ((lane >> 4) & 1) + ((l16 & 3) >> 1);
    const int v_b = 8 * (l16 & 1);
    u32x4 vf[2][kOut];
    auto read_values = [&](int buf, int kb) {
      const unsigned char* vt = vbuf + buf * kTile;
#pragma unroll
      for (int i = 0; i < kOut; ++i) {
        const u32x2 lo = lds_read_tr(vt + v_unit<D>(16 * kb + v_row, 4 * i + v_un) + v_b);
        const u32x2 hi = lds_read_tr(vt + v_unit<D>(16 * kb + 8 + v_row, 4 * i + v_un) + v_b);
        vf[kb & 1][i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    };
    // rows of step s that are absent become zeros; values that are not finite, too, where some row
    // does not see them (added below for the rows that do): thread tid looks at units of row tid / 8
    auto mend = [&](int s, uint64_t valid, bool edge) {
      const int r = tid >> 3, u0 = (tid & 7) * kCopies, at = (s - s_begin) & 3;
      unsigned char* const vt = vbuf + at * kTile;
      if (!((valid >> r) & 1)) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          *reinterpret_cast<u32x4*>(smem + at * kTile + k_unit<D>(r, u0 + i)) = u32x4{0, 0, 0, 0};
          *reinterpret_cast<u32x4*>(vt + v_unit<D>(r, u0 + i)) = u32x4{0, 0, 0, 0};
        }
      } else if (edge) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          u32x4 v = *reinterpret_cast<const u32x4*>(vt + v_unit<D>(r, u0 + i));
          if (clear_odd<false>(&v)) {
            *reinterpret_cast<u32x4*>(vt + v_unit<D>(r, u0 + i)) = v;
            atomicOr(&state[(s - s_begin) & 7][r], 2);
          }
        }
      }
    };
    for (int s0 = s_begin; s0 < s_end; s0 += half ? 2 : 1) {
      const int s = s0 + (half ? wave >> 2 : 0);  // this wave's tile
      const int buf = (s - s_begin) & (kBuffers - 1), note = (s - s_begin) & (FP8 ? 1 : 7);
      const unsigned char* kt = smem + buf * kTile;
      const int base = s * kTileKeys;
      if constexpr (!FP8) {
        // this step's rows are in place once each wave's own copies are (at most the next two
        // steps' may still be on their way) and all waves have met; the last step's buffers are
        // free then
        if (!half && s + 2 < s_end) wait_copies<4 * kCopies>();
        else if (!half && s + 1 < s_end) wait_copies<2 * kCopies>();
        else wait_copies<0>();
        lds_barrier();
      }
      int key_state = state[note][lane];
      uint64_t valid = __ballot(key_state & 1);
      if constexpr (!FP8) {
        const bool edge = hides(base);
        if (half) {  // two tiles, of which the second may be past the end
          const uint64_t v0 = __ballot(state[(s0 - s_begin) & 7][lane] & 1);
          const uint64_t v1 = s0 + 1 < s_end ? __ballot(state[(s0 + 1 - s_begin) & 7][lane] & 1) : ~0ull;
          if (v0 != ~0ull) mend(s0, v0, false);
          if (v1 != ~0ull) mend(s0 + 1, v1, false);
          if ((v0 & v1) != ~0ull) lds_barrier();
          if (s >= s_end) valid = 0;
        } else if (valid != ~0ull || edge) {
          mend(s, valid, edge);
          lds_barrier();
          key_state = state[note][lane];
        }
        // (the entries of step s + 4, copied before the two newest steps' rows, are there)
        look_end(s0 + 4);
        look_begin(s0 + 6);
        if (half) {
          look_end(s0 + 5);
          look_begin(s0 + 7);
          if (s0 + 2 < s_end) copy_rows(s0 + 2);
        }
        if (s0 + 3 < s_end) copy_rows(s0 + 3);
      }
      uint64_t odd = PREFIX ? 0 : __ballot(key_state & 2);  // keys whose values were taken out
      // does the wave see anything, does every row see everything?
      bool any = wave_live && valid != 0, all = valid == ~0ull;
      if constexpr (!PREFIX) {
        const int f = key_position(kl, base), last = key_position(kl, base + kTileKeys - 1);
        const bool in_main = base >= kl.na;
        any = any && f <= p0 + wt1 && (f < a.sinks || p0 + wt0 - last < a.window);
        all = all && in_main && last <= p0 + wt0 && p0 + wt1 - f < a.window;
      }
      f32x16 sc[2];
      if (any) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) sc[i][e] = 0.f;
        // kDeep pairs of operand reads in flight ahead of the matrix instructions (left to itself
        // the compiler sinks each read to its use)
        constexpr int kDeep = kSteps < 4 ? kSteps : 4;
        u32x4 kf[kDeep][2];
        auto read_k = [&](int d) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            kf[d % kDeep][i] = *reinterpret_cast<const u32x4*>(kt + k_unit<D>(32 * i + q, 2 * d + hf));
        };
#pragma unroll
        for (int d = 0; d < kDeep; ++d) read_k(d);
#pragma unroll
        for (int d = 0; d < kSteps; ++d) {
          const u32x4 k0 = kf[d % kDeep][0], k1 = kf[d % kDeep][1];
          if (d + kDeep < kSteps) read_k(d + kDeep);
          sc[0] = mfma32(k0, qf[d], sc[0]);
          sc[1] = mfma32(k1, qf[d], sc[1]);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * kDeep, 0);
#pragma unroll
        for (int d = 0; d < kSteps - kDeep; ++d) {
          __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 2 * kDeep, 0);
      }
      if constexpr (FP8) {
        // ---- the next step's tiles; these buffers were last read before the barrier that began
        // this step
        if (s + 1 < s_end) {
          const int unit = 16 * (tid % TileStage<D, FP8>::kUnits);
          st.store(smem + (buf ^ 1) * kTile, vbuf + (buf ^ 1) * kTile, state[buf ^ 1],
                   hides(base + kTileKeys), tid);
          st.fetch(kh + unit, vh + unit, places[(s + 2 - s_begin) & 3], tid);
          // (the loads that st.store waited for are newer than the entries')
          look_end(s + 3);
          look_begin(s + 5);
        }
      }
      if (any) {
        // lane (q, hf) holds keys 32 i + 8 (e / 4) + 4 hf + e % 4 of its row
        if (!all) {
          const uint64_t mine = valid >> (4 * hf);
          const Sight at = sight(kl, pq, a.sinks, base + 4 * hf);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const unsigned bits = (unsigned)(mine >> (32 * i));
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int key = 8 * (e >> 2) + (e & 3);  // + 32 i + 4 hf
              bool seen = (bits >> key) & 1u;
              if constexpr (!PREFIX) seen = seen & at.sees(32 * i + key, a.window);
              const float v = sc[i][e];
              sc[i][e] = seen ? v : kNegInf;
            }
          }
        }
        // the first values are on their way while the weights are worked out
        read_values(buf, 0);
        __builtin_amdgcn_sched_barrier(0);
        // (elementwise maximum: a NaN among a row's scores passes, the row is NaN then)
        float tp[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          tp[e] = sc[0][e];
#pragma unroll
          for (int i = 4; i < 32; i += 4) tp[e] = __builtin_elementwise_maximum(tp[e], (float)sc[(i + e) >> 4][(i + e) & 15]);
        }
        float tm = __builtin_elementwise_maximum(__builtin_elementwise_maximum(tp[0], tp[1]),
                                                 __builtin_elementwise_maximum(tp[2], tp[3]));
        tm = half_max(tm) * a.c;
        if (__any(tm > m + kRescale)) {
          const float mn = fmaxf(m, tm);
          const float f = mn == kNegInf ? 1.f : exp2_fast(m - mn);
          m = mn;
          l *= f;
#pragma unroll
          for (int i = 0; i < kOut; ++i) o[i] *= f;
        }
        const float mb = m == kNegInf ? 0.f : m;
        float lp[4];
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = exp2_fast(__builtin_fmaf(sc[kb >> 1][8 * (kb & 1) + i], a.c, -mb));
          lp[kb] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
          // weights enter the product as bf16, the matrix instruction's operand type (off by at most
          // 2^-8 of themselves, as the values they weigh were when stored); the sum l keeps them in fp32
          p[kb] = u32x4{pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]),
                        pack_bf16(e[6], e[7])};
        }
        l += (lp[0] + lp[1]) + (lp[2] + lp[3]);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          if (kb < 3) read_values(buf, kb + 1);
#pragma unroll
          for (int i = 0; i < kOut; ++i) o[i] = mfma32(vf[kb & 1][i], p[kb], o[i]);
        }
        if constexpr (!PREFIX) {
          // (also where this wave's rows see all keys: the values were taken out for the whole tile)
          for (; odd; odd &= odd - 1) {
            const int vp = base + __builtin_ctzll(odd);
            const unsigned char* row_v = value_row(a.cache, kl, vp, h);
            if (!row_v) continue;
            const bool seen = sees(kl, pq, a.window, a.sinks, vp);
#pragma unroll
            for (int i = 0; i < kOut; ++i)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float x = o[i][e];
                o[i][e] = seen ? x + odd_value<FP8>(row_v, 32 * i + 8 * (e >> 2) + 4 * hf + (e & 3)) : x;
              }
          }
        }
      }
      if constexpr (FP8) __syncthreads();
    }
    // no copy into LDS outlives its use: the next unit, or workgroup, has these buffers
    wait_copies<0>();

    // ---- epilogue: lane (q, hf) holds dims 32 i + 8 (e / 4) + 4 hf + e % 4 of its row
    l = half_sum(l);
    if (live) {
      if constexpr (PREFIX) {
        const int64_t at = slot * kTileRows + row + (half ? (wave >> 2) * (kTileRows / 2) : 0);
        float* op = a.tile_o + at * D + 4 * hf;
#pragma unroll
        for (int i = 0; i < kOut; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f32x4*>(op + 32 * i + 8 * e) =
                f32x4{o[i][4 * e], o[i][4 * e + 1], o[i][4 * e + 2], o[i][4 * e + 3]};
        if (hf == 0) {
          a.tile_ml[at * 2] = m;
          a.tile_ml[at * 2 + 1] = l;
        }
      } else {
        const float inv = l > 0.f ? a.v_scale / l : (l == 0.f ? 0.f : l);
        uint16_t* op = a.out + (int64_t)(t0 + t) * a.o_token + (int64_t)hh * a.o_head + 4 * hf;
#pragma unroll
        for (int i = 0; i < kOut; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<u32x2*>(op + 32 * i + 8 * e) =
                u32x2{pack_bf16(o[i][4 * e] * inv, o[i][4 * e + 1] * inv),
                      pack_bf16(o[i][4 * e + 2] * inv, o[i][4 * e + 3] * inv)};
        if (a.lse && hf == 0)
          a.lse[(int64_t)(t0 + t) * a.heads + hh] =
              l == 0.f ? kNegInf : (m + __builtin_log2f(l)) * kLn2;
      }
    }
    if constexpr (!PREFIX) break;
  }
}

// ---------------------------------------------------------------------------------------------
// Combine: one wave per query row adds the row's partials of both kernels, in a fixed order: lanes of
// 4 dims each, 64 / (dim / 4) pieces side by side, four loads each in flight.  Bound by finding the
// pieces (divisions) and the loads' latency: 16384 rows of 3 to 5 pieces 16 to 18 us, 64 rows of 96 10.7, of 64
// 8.3.  Two rows a wave were 13% faster for the first, but half as much again for few rows of many pieces.
// W = 4: a workgroup's waves take one row's pieces between them: 64 rows of 96 5.0 to 5.4 us, of 64 4.9.
// ---------------------------------------------------------------------------------------------
template <int D, int W>
__global__ __launch_bounds__(256) void attend_combine_kernel(const AttendArgs a) {
  const int tpt = kTileRows / a.group;
  constexpr int kQ = D / 4, kWays = W * (64 / kQ);  // lanes of a row, pieces side by side
  const int lane = threadIdx.x & 63;
  const int rest = W == 1 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x, b = blockIdx.y;
  if (rest >= a.max_q * a.heads) return;
  const int tq = rest / a.heads, hh = rest - tq * a.heads;
  const int h = hh / a.group;
  const RowUnit u = row_unit(a, b);
  if (tq >= u.nq) return;
  const int d4 = lane % kQ, way = lane / kQ + (W == 1 ? 0 : (threadIdx.x >> 6) * (64 / kQ));

  float mx = kNegInf, lt = 0.f;
  f32x4 ot = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](float pm, float pl, const f32x4& po) {
    const float mn = fmaxf(mx, pm);
    const float mb = mn == kNegInf ? 0.f : mn;
    const float f0 = exp2_fast(mx - mb), f1 = exp2_fast(pm - mb);
    lt = lt * f0 + pl * f1;
    ot = ot * f0 + po * f1;
    mx = mn;
  };
  // own pieces: of workers own_w .. own_w + own_n - 1
  int own_n = 0;
  int64_t own_at = 0;  // the first one's row
  {
    const int64_t total = (int64_t)a.scan[a.batch] * a.kv_heads;
    const int steps = a.scan[b + 1] - a.scan[b];
    if (steps > 0) {
      const int64_t x0 = (int64_t)a.scan[b] * a.kv_heads + (int64_t)h * steps;
      const int workers = split_workers(total, a.workers);
      const int w0 = split_owner(x0, total, workers);
      own_n = split_owner(x0 + steps - 1, total, workers) + 1 - w0;
      own_at = (w0 + (int64_t)b * a.kv_heads + h) * a.rows + tq * a.group + hh - h * a.group;
    }
  }
  // the prefix's
  int pre_n = 0, pre_all = 0;  // workers, pieces: two per worker if the unit is halved
  int64_t pre_at = 0;
  if (a.nseg > 0 && !a.row_prefix) {
    // the sequence's segment: how many segments end at or before it (at most 64: the last does not)
    const int sg = __popcll(__ballot(lane < a.nseg && a.seg_offsets[lane + 1] <= b));
    const int n0 = a.seg_offsets[sg];
    const int ub = a.tile_segs[sg], tiles = a.tile_segs[sg + 1] - ub;
    const int before = a.tile_scan[sg], seg_steps = a.tile_scan[sg + 1] - before;
    if (seg_steps > 0) {
      const int64_t total = (int64_t)a.tile_scan[a.nseg] * a.kv_heads;
      const int steps = seg_steps / tiles;
      const int rt = (b - n0) / tpt;
      const int row = (b - n0 - rt * tpt) * a.group + hh - h * a.group;
      const int64_t x0 = (int64_t)before * a.kv_heads + ((int64_t)h * tiles + rt) * steps;
      const int workers = split_workers(total, a.tile_workers);
      const int w0 = split_owner(x0, total, workers);
      pre_n = split_owner(x0 + steps - 1, total, workers) + 1 - w0;
      pre_all = halved(a, sg) ? 2 * pre_n : pre_n;
      pre_at = (w0 + (int64_t)ub * a.kv_heads + h * tiles + rt) * kTileRows + row;
    }
  }
  // all pieces, four loads in flight
  const int pieces = own_n + pre_all;
  for (int i0 = way; i0 < pieces; i0 += 4 * kWays) {
    f32x2 pm[4];
    f32x4 po[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(i0 + i * kWays, pieces - 1), t = n - own_n;
      const bool own = t < 0;
      const int64_t at = own ? own_at + (int64_t)n * a.rows
                             : pre_at + (int64_t)(t < pre_n ? t : t - pre_n) * kTileRows +
                                   (t < pre_n ? 0 : kTileRows / 2);
      pm[i] = *reinterpret_cast<const f32x2*>((own ? a.part_ml : a.tile_ml) + at * 2);
      po[i] = *reinterpret_cast<const f32x4*>((own ? a.part_o : a.tile_o) + at * D + 4 * d4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i0 + i * kWays < pieces) add(pm[i][0], pm[i][1], po[i]);
  }
  // the ways' sums
#pragma unroll
  for (int d = kQ; d < 64; d <<= 1) {
    const float om = __shfl_xor(mx, d, 64), ol = __shfl_xor(lt, d, 64);
    f32x4 oo;
#pragma unroll
    for (int i = 0; i < 4; ++i) oo[i] = __shfl_xor(ot[i], d, 64);
    const float mn = fmaxf(mx, om);
    const float mb = mn == kNegInf ? 0.f : mn;
    const float f0 = exp2_fast(mx - mb), f1 = exp2_fast(om - mb);
    lt = lt * f0 + ol * f1;
    ot = ot * f0 + oo * f1;
    mx = mn;
  }
  if constexpr (W > 1) {  // the waves' sums
    __shared__ f32x4 wave_o[W][kQ];
    __shared__ float wave_ml[W][2];
    const int wave = threadIdx.x >> 6;
    if (lane < kQ) wave_o[wave][lane] = ot;
    if (lane == 0) {
      wave_ml[wave][0] = mx;
      wave_ml[wave][1] = lt;
    }
    __syncthreads();
    if (way == 0)
      for (int v = 1; v < W; ++v) add(wave_ml[v][0], wave_ml[v][1], wave_o[v][d4]);
  }
  if (way == 0) {
    const float inv = lt > 0.f ? a.v_scale / lt : (lt == 0.f ? 0.f : lt);
    const int64_t tok = u.t0 + tq;
    *reinterpret_cast<u32x2*>(a.out + tok * a.o_token + (int64_t)hh * a.o_head + 4 * d4) =
        u32x2{pack_bf16(ot[0] * inv, ot[1] * inv), pack_bf16(ot[2] * inv, ot[3] * inv)};
    if (a.lse && d4 == 0)
      a.lse[tok * a.heads + hh] = lt == 0.f ? kNegInf : (mx + __builtin_log2f(lt)) * kLn2;
  }
}

template <int D, bool FP8>
hipError_t rows_for(const AttendArgs& a, int columns, int blocks, hipStream_t stream) {
  clear_stale_error();
  const dim3 grid(blocks), block(256);
  const bool multi = a.max_q > 1;
  if (columns == 1 && !multi) hipLaunchKernelGGL((attend_row_kernel<D, FP8, 1, false>), grid, block, 0, stream, a);
  else if (columns == 2 && !multi) hipLaunchKernelGGL((attend_row_kernel<D, FP8, 2, false>), grid, block, 0, stream, a);
  else if (columns == 4 && !multi) hipLaunchKernelGGL((attend_row_kernel<D, FP8, 4, false>), grid, block, 0, stream, a);
  else if (columns == 1) hipLaunchKernelGGL((attend_row_kernel<D, FP8, 1, true>), grid, block, 0, stream, a);
  else if (columns == 2) hipLaunchKernelGGL((attend_row_kernel<D, FP8, 2, true>), grid, block, 0, stream, a);
  else if (columns == 4) hipLaunchKernelGGL((attend_row_kernel<D, FP8, 4, true>), grid, block, 0, stream, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

template <int D, bool FP8, bool PREFIX>
hipError_t tiles_for(const AttendArgs& a, int blocks, hipStream_t stream) {
  constexpr int lds = (FP8 ? 4 : 8) * kTileKeys * D * 2;
  static DeviceOnce once;
  const hipError_t e = set_dynamic_lds_once(
      once, reinterpret_cast<const void*>(&attend_tile_kernel<D, FP8, PREFIX>), lds);
  if (e != hipSuccess) return e;
  clear_stale_error();
  hipLaunchKernelGGL((attend_tile_kernel<D, FP8, PREFIX>), dim3(blocks), dim3(512), lds, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_rows(const AttendArgs& a, int dim, bool fp8, int columns, int blocks,
                              hipStream_t stream) {
  if (blocks < 1 || a.batch > kAttendMaxSeqs || a.rows > 16 * columns) return hipErrorInvalidValue;
  if (dim == 64) return fp8 ? rows_for<64, true>(a, columns, blocks, stream)
                            : rows_for<64, false>(a, columns, blocks, stream);
  if (dim == 128) return fp8 ? rows_for<128, true>(a, columns, blocks, stream)
                             : rows_for<128, false>(a, columns, blocks, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_attend_tiles(const AttendArgs& a, int dim, bool fp8, bool prefix, int blocks,
                               hipStream_t stream) {
  if (blocks < 1 || a.batch > kAttendMaxSeqs || a.nseg > kAttendMaxSegments)
    return hipErrorInvalidValue;
  if (dim == 64)
    return prefix ? (fp8 ? tiles_for<64, true, true>(a, blocks, stream)
                         : tiles_for<64, false, true>(a, blocks, stream))
                  : (fp8 ? tiles_for<64, true, false>(a, blocks, stream)
                         : tiles_for<64, false, false>(a, blocks, stream));
  if (dim == 128)
    return prefix ? (fp8 ? tiles_for<128, true, true>(a, blocks, stream)
                         : tiles_for<128, false, true>(a, blocks, stream))
                  : (fp8 ? tiles_for<128, true, false>(a, blocks, stream)
                         : tiles_for<128, false, false>(a, blocks, stream));
  return hipErrorInvalidValue;
}

hipError_t launch_attend_combine(const AttendArgs& a, int dim, bool many, hipStream_t stream) {
  const unsigned rows = (unsigned)a.max_q * a.heads;  // at most 64 per kv head
  const dim3 grid(many ? rows : (rows + 3) / 4, a.batch);
  clear_stale_error();
  if (dim == 64 && many) hipLaunchKernelGGL((attend_combine_kernel<64, 4>), grid, dim3(256), 0, stream, a);
  else if (dim == 64) hipLaunchKernelGGL((attend_combine_kernel<64, 1>), grid, dim3(256), 0, stream, a);
  else if (dim == 128 && many) hipLaunchKernelGGL((attend_combine_kernel<128, 4>), grid, dim3(256), 0, stream, a);
  else if (dim == 128) hipLaunchKernelGGL((attend_combine_kernel<128, 1>), grid, dim3(256), 0, stream, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace bd
