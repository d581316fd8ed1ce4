// Attention over a paged cache of 4-bit keys and values: decode with prefixes shared by the segments of a
// batch, and causal attention with a sliding window and first tokens that stay visible.
//
// Mathematics, per query row q of kv head h and its visible keys j (k_j and v_j: e2m1 codes times their
// block's power of two):
//   s_j = c * (q . k_j),  c = scale * k_scale * log2(e)
//   m = max_j s_j,  l = sum_j 2^(s_j - m),  o = v_scale / l * sum_j 2^(s_j - m) v_j
// in one pass over the keys, with a running maximum and sum.
#include "attend_device.h"

namespace bd {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 8 codes -> 8 bf16, times a power of two; exact
__device__ __forceinline__ u32x4 fp4x8_to_bf16(unsigned v, float step) {
  return u32x4{__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, step, 0)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, step, 1)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, step, 2)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, step, 3))};
}
__device__ __forceinline__ float block_step(unsigned byte) { return __uint_as_float(byte << 23); }

// ---------------------------------------------------------------------------------------------
// Queries.  The scaled matrix instruction takes K's codes and scale bytes as they lie in memory; its
// other operand is 8 bits wide, so a query row q goes in as two e4m3 rows of 4 significant bits each:
// q / 2^e = hi + lo / 16, hi = q / 2^e rounded, lo what is left of it, times 16, rounded, with 2^e such
// that the row's largest |q| / 2^e is in [128, 256).  A bf16 value has 8 bits: values down to 2^-9 of the
// largest are exact, smaller ones off by at most 2^-20 of it.  A row with an infinity or NaN has the scale
// byte 255, which makes its scores NaN.
// ---------------------------------------------------------------------------------------------
// 16 values (x: bf16 pairs) of a row -> their bytes of both parts; scales: bytes of e + 127 and e - 4 + 127
__device__ __forceinline__ void split_query(const u32x4* x, unsigned scales, int* hi, int* lo) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  const float step = block_step(scales & 0xFF), fine = block_step((scales >> 8) & 0xFF);
#pragma unroll
  for (int w = 0; w < 4; ++w) {  // 4 values a word
    s16x2 h = {0, 0}, l = {0, 0};
    const unsigned a = x[w >> 1][2 * (w & 1)], b = x[w >> 1][2 * (w & 1) + 1];
    const float f0 = bf16lo_to_f32(a), f1 = bf16hi_to_f32(a), f2 = bf16lo_to_f32(b), f3 = bf16hi_to_f32(b);
    h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, f0, f1, step, false);
    h = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(h, f2, f3, step, true);
    hi[w] = __builtin_bit_cast(int, h);
    const f32x2 u = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi[w], step, false);
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi[w], step, true);
    l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, f0 - u[0], f1 - u[1], fine, false);
    l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, f2 - v[0], f3 - v[1], fine, true);
    lo[w] = __builtin_bit_cast(int, l);
  }
}
// largest |x| of 8 bf16 values, as its bits
__device__ __forceinline__ unsigned top_bits(const u32x4& x) {
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[i] & 0x7FFF7FFFu));
  return max((unsigned)m[0], (unsigned)m[1]);
}
// scale bytes of the two parts of a row whose largest value has these bits
__device__ __forceinline__ unsigned query_scales(unsigned top) {
  const int p = (int)(top >> 7);
  const int hi = p == 255 ? 255 : max(p - 7, 5);
  return (unsigned)hi | (unsigned)(p == 255 ? 255 : hi - 4) << 8;
}

__device__ __forceinline__ f32x4 mfma_k16(const u32x4& k, int k_byte, const i32x8& q, int q_bytes, bool low,
                                          const f32x4& c) {
  const i32x8 a = {(int)k[0], (int)k[1], (int)k[2], (int)k[3], 0, 0, 0, 0};
  return low ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, q, c, 4, 0, 0, k_byte, 1, q_bytes)
             : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, q, c, 4, 0, 0, k_byte, 0, q_bytes);
}

// NaN if the block of dim d of a value row is NaN, else 0; blocks: the row's scale bytes
__device__ __forceinline__ float odd_block(const unsigned char* blocks, int d) {
  return blocks[d >> 5] == 255 ? __builtin_nanf("") : 0.f;
}

// ---------------------------------------------------------------------------------------------
// Row kernel: up to 16 * NC query rows (the heads of one kv head, for one or a few tokens) against a key
// list, each of a workgroup's 4 waves 32 keys of a 128-key step on its own.  A lane's 16 bytes of a K row
// are one block of 32 dims, as the scaled matrix instruction wants its operand (dim 64: one row in the
// first two lane groups, another, 16 keys on, in the last two; each is met by a query operand that is zero
// in the other half).  V rows are widened to bf16 into 8 KiB of the wave's LDS, and read transposed.
// ---------------------------------------------------------------------------------------------
template <int D, int NC>
struct Row4Loop {
  static constexpr int kLoads = D / 64;   // keys a lane has a block of, per step
  static constexpr int kTiles = D / 16;   // 16-row tiles of O^T
  static constexpr int kWords = D / 16;   // dwords of a query operand (dim 64: its half that is not zero)

  int hi[NC][kWords], lo[NC][kWords];
  int scales[NC];
  f32x4 o[NC][kTiles];
  float m[NC], l[NC];
  int pos[NC];   // the column's token position (window op with several tokens)
  u32x4 kr[kLoads], vr[kLoads];
  int kb[kLoads], vb[kLoads];  // scale bytes
  int id[kLoads], slot[kLoads];
  bool ok[kLoads];

  // the key of load i within a step, and the block
  static __device__ __forceinline__ int key(int i, int j, int g) { return D == 128 ? 16 * i + j : j + 16 * (g >> 1); }
  static __device__ __forceinline__ int block(int g) { return D == 128 ? g : g & 1; }

  __device__ __forceinline__ void lookup(const AttendArgs& a, const KeyList& kl, int base, int j, int g) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int p = base + key(i, j, g);
      const int kp = key_position(kl, p);
      const int page = page_quotient(kp < 0 ? 0 : kp, a.cache.div);
      const int at = key_table_index(kl, p, page);
      slot[i] = kp - page * a.cache.page_size;
      // the entry is only checked when it is used: the load stays in flight
      id[i] = at >= 0 ? (p < kl.na ? kl.ta : kl.tb)[at] : -1;
    }
  }
  __device__ __forceinline__ void fetch(const AttendArgs& a, int h, int g) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // absent keys read page 0 and are cleared before they are used
      ok[i] = page_id_checked(id[i], a.cache.num_pages) >= 0;
      const int page = ok[i] ? id[i] : 0, at = ok[i] ? slot[i] : 0;
      const int64_t ko = page_row_bytes(page, at, a.cache.k_page, a.cache.k_token) + (int64_t)h * a.cache.k_head;
      const int64_t vo = page_row_bytes(page, at, a.cache.v_page, a.cache.v_token) + (int64_t)h * a.cache.v_head;
      kr[i] = *reinterpret_cast<const u32x4*>(a.cache.k + ko + 16 * block(g));
      vr[i] = *reinterpret_cast<const u32x4*>(a.cache.v + vo + 16 * block(g));
      kb[i] = a.cache.k_blocks[(ko >> 4) + block(g)];
      vb[i] = a.cache.v_blocks[(vo >> 4) + block(g)];
    }
  }
  // keys of the step that exist, bit (key)
  __device__ __forceinline__ unsigned valid() const {
    if constexpr (D == 128) {
      return (unsigned)(__ballot(ok[0]) & 0xFFFFull) | ((unsigned)(__ballot(ok[kLoads - 1]) & 0xFFFFull) << 16);
    } else {
      const uint64_t b = __ballot(ok[0]);
      return (unsigned)(b & 0xFFFFull) | ((unsigned)((b >> 32) & 0xFFFFull) << 16);
    }
  }
  // what the memory holds for an absent key must not reach the sums (of its scores, the masks see to it)
  __device__ __forceinline__ void clear_absent() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (!ok[i]) {
        vr[i] = u32x4{0, 0, 0, 0};
        vb[i] = 127;
      }
  }
  // keys with a block of NaN among their values, bit (key); those blocks become zeros
  __device__ __forceinline__ unsigned clear_odd_blocks() {
    unsigned odd = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool f = vb[i] == 255;
      uint64_t m = __ballot(f);
      if (m) {
        if (f) {
          vr[i] = u32x4{0, 0, 0, 0};
          vb[i] = 127;
        }
        m |= m >> 16;  // lane groups 0, 1 and 2, 3
        if constexpr (D == 128) odd |= (unsigned)((m | (m >> 32)) & 0xFFFFull) << (16 * i);
        else odd |= (unsigned)(m & 0xFFFFull) | ((unsigned)((m >> 32) & 0xFFFFull) << 16);
      }
    }
    return odd;
  }
  // dim 64: a product has two keys in it, one met by zeros, which a block of NaN would pass through: such
  // blocks become zeros.  Returns their keys, bit (key), whose scores are NaN.
  __device__ __forceinline__ unsigned clear_odd_keys() {
    if constexpr (D == 128) return 0;
    const bool f = kb[0] == 255;
    uint64_t m = __ballot(f);
    if (!m) return 0;
    if (f) kb[0] = 0, kr[0] = u32x4{0, 0, 0, 0};
    m |= m >> 16;
    return (unsigned)(m & 0xFFFFull) | ((unsigned)((m >> 32) & 0xFFFFull) << 16);
  }
  // column j of block c is query row 16 c + j; row: this lane's, or null
  __device__ __forceinline__ void load_query(int c, const uint16_t* row, int g) {
    constexpr int kHalves = D / 64;
    u32x4 x[kHalves][2];
    unsigned top = 0;
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[h][i] = row ? *reinterpret_cast<const u32x4*>(row + 64 * h + 16 * g + 8 * i) : u32x4{0, 0, 0, 0};
        top = max(top, top_bits(x[h][i]));
      }
    // (bits of values that are not negative order as they do)
    top = __float_as_uint(half_max(row_max(__uint_as_float(top << 16)))) >> 16;
    scales[c] = (int)query_scales(top);
#pragma unroll
    for (int h = 0; h < kHalves; ++h) split_query(x[h], (unsigned)scales[c], hi[c] + 4 * h, lo[c] + 4 * h);
  }
  // scores of the keys 16 r .. 16 r + 15 (lane (j, g): keys 4 g .. + 3) with block c's queries
  __device__ __forceinline__ f32x4 scores(int c, int r) const {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    auto operand = [&](const int* w) {
      if constexpr (D == 128) return i32x8{w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
      else return r == 0 ? i32x8{w[0], w[1], w[2], w[3], 0, 0, 0, 0} : i32x8{0, 0, 0, 0, w[0], w[1], w[2], w[3]};
    };
    const int i = D == 128 ? r : 0;
    s = mfma_k16(kr[i], kb[i], operand(hi[c]), scales[c], false, s);
    return mfma_k16(kr[i], kb[i], operand(lo[c]), scales[c], true, s);
  }
};

// The sums of a row workgroup's waves for the 16 query rows of column block c, lane (j, g) of a wave with
// maximum mc, its part lc of the sum and the dims 16 i + 4 g .. + 3 of row 16 c + j in oc[i]; joined
// through the waves' LDS and written as results (a.direct) or as partials of `slot`.
template <int D>
__device__ __forceinline__ void join_waves(const AttendArgs& a, unsigned char* vlds, float (*ml)[16][2], int wave,
                                           int tid, float mc, float lc, const f32x4* oc, int c, int rows,
                                           int t0, int h, int64_t slot) {
  constexpr int kWaveLds = kRowKeys * D * 2;
  const int lane = tid & 63, j = lane & 15, g = lane >> 4;
  lc = half_sum(row_sum(lc));
  __syncthreads();  // the V tiles, or the last block's sums, are no longer read
  float* const ow = reinterpret_cast<float*>(vlds + wave * kWaveLds);  // [16 columns][D]
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
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
        *reinterpret_cast<u32x2*>(a.out + (int64_t)(t0 + t) * a.o_token + (int64_t)hh * a.o_head + 4 * d4) = pk;
        if (a.lse && d4 == 0)
          a.lse[(int64_t)(t0 + t) * a.heads + hh] = lt == 0.f ? kNegInf : (mb + __builtin_log2f(lt)) * kLn2;
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

// MULTI: units may hold several tokens, which see different keys
template <int D, int NC, bool MULTI>
__global__ __launch_bounds__(256, NC == 1 ? 3 : (NC == 2 ? 2 : 1)) void attend4_row_kernel(const AttendArgs a) {
  using Loop = Row4Loop<D, NC>;
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
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int row = 16 * c + j;
      const int t = row / a.group, hh = row - t * a.group;
      w.pos[c] = u.p0 + t;
      w.m[c] = kNegInf;
      w.l[c] = 0.f;
#pragma unroll
      for (int i = 0; i < Loop::kTiles; ++i) w.o[c][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      w.load_query(c, row < rows ? a.q + (int64_t)(u.t0 + t) * a.q_token + (int64_t)(h * a.group + hh) * a.q_head
                                 : nullptr, g);
    }

    int base = s_begin * kRowStep + wave * kRowKeys;
    const int end = s_end * kRowStep;
    if (base < end) {
      w.lookup(a, kl, base, j, g);
      w.fetch(a, h, g);
      if (base + kRowStep < end) w.lookup(a, kl, base + kRowStep, j, g);
    }
    for (; base < end; base += kRowStep) {
      const unsigned valid = w.valid();
      if (valid != 0xFFFFFFFFu) w.clear_absent();
      // keys whose values are not all numbers: those values are taken out here and added below for the
      // tokens that see them, since their product with a zero weight would be NaN
      unsigned odd = 0;
      if constexpr (MULTI) odd = w.clear_odd_blocks();
      // ---- V into LDS, scores from K
#pragma unroll
      for (int i = 0; i < Loop::kLoads; ++i) {
        const float step = block_step(w.vb[i]);
        const int row = Loop::key(i, j, g), unit = 4 * Loop::block(g);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<u32x4*>(vl + v_unit<D>(row, unit + e)) = fp4x8_to_bf16(w.vr[i][e], step);
      }
      const unsigned odd_keys = w.clear_odd_keys();
      f32x4 s[NC][2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c) s[c][r] = w.scores(c, r);
      if (D == 64 && odd_keys) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((odd_keys >> (16 * r + 4 * g + i)) & 1u) s[c][r][i] = __builtin_nanf("");
      }
      // ---- the next tile's rows are on their way while this one is worked on
      if (base + kRowStep < end) {
        w.fetch(a, h, g);
        if (base + 2 * kRowStep < end) w.lookup(a, kl, base + 2 * kRowStep, j, g);
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
        // of themselves); the sum l keeps them in fp32
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
          const unsigned char* blocks = a.cache.v_blocks + ((row - a.cache.v) >> 4);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const bool seen = sees(kl, w.pos[c], a.window, a.sinks, vp);
#pragma unroll
            for (int i = 0; i < Loop::kTiles; ++i) {
              const float odd_one = seen ? odd_block(blocks, 16 * i) : 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) w.o[c][i][e] = w.o[c][i][e] + odd_one;
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
      join_waves<D>(a, vlds, ml, wave, tid, mc, lc, oc, c, rows, u.t0, h, slot);
    }
    if (!a.direct) {
      __syncthreads();  // the sums are read before the next piece's V tiles land
      x += s_end - s_begin;
    }
  }
}

// One wave per query row: a lane takes a key of 64 at a time, its whole score; then the wave goes through
// the 64 values, a lane two dims.
template <int D>
__global__ __launch_bounds__(64) void attend4_plain_kernel(const AttendArgs a) {
  __shared__ float qs[D];
  const int lane = threadIdx.x;
  const int64_t rows = (int64_t)a.tokens * a.heads;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int t = (int)(r / a.heads), hh = (int)(r - (int64_t)t * a.heads), h = hh / a.group;
    // the row's sequence and keys
    KeyList kl{};
    bool found = false;
    if (a.nseg > 0) {
      const RowUnit u = row_unit(a, t);
      kl = u.keys;
      found = true;
    } else {
      for (int b0 = 0; b0 < a.batch && !found; b0 += 64) {
        const int b = b0 + lane;
        RowUnit u{};
        if (b < a.batch) u = row_unit(a, b);
        const uint64_t mine = __ballot(b < a.batch && t >= u.t0 && t < u.t0 + u.nq);
        if (!mine) continue;
        const int bb = b0 + __builtin_ctzll(mine);
        u = row_unit(a, bb);
        const int pos = u.p0 + t - u.t0;
        kl = window_keys(a.table + (int64_t)bb * a.width, a.width, pos < 0 ? 0 : pos + 1, pos, a.window, a.sinks);
        found = true;
      }
    }
    if (!found) continue;
    const uint16_t* qp = a.q + (int64_t)t * a.q_token + (int64_t)hh * a.q_head;
    __syncthreads();
    for (int d = lane; d < D; d += 64) qs[d] = __uint_as_float((unsigned)qp[d] << 16);
    __syncthreads();
    float m = kNegInf, l = 0.f, o0 = 0.f, o1 = 0.f;
    for (int base = 0; base < kl.n; base += 64) {
      const int vp = base + lane;
      const int kp = key_position(kl, vp);
      const int page = page_quotient(kp < 0 ? 0 : kp, a.cache.div);
      const int at = key_table_index(kl, vp, page);
      const int id = at >= 0 ? page_id_checked((vp < kl.na ? kl.ta : kl.tb)[at], a.cache.num_pages) : -1;
      float s = kNegInf;
      int64_t vo = -1;
      if (id >= 0) {
        const int slot = kp - page * a.cache.page_size;
        vo = page_row_bytes(id, slot, a.cache.v_page, a.cache.v_token) + (int64_t)h * a.cache.v_head;
        const int64_t ko = page_row_bytes(id, slot, a.cache.k_page, a.cache.k_token) + (int64_t)h * a.cache.k_head;
        s = 0.f;
        for (int i = 0; i < D / 32; ++i) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(a.cache.k + ko + 16 * i);
          const float step = __uint_as_float((unsigned)a.cache.k_blocks[(ko >> 4) + i] << 23);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float* qd = qs + 32 * i + 8 * w;
            auto add = [&](unsigned pair, int d) {
              s = __builtin_fmaf(bf16lo_to_f32(pair), qd[d], s);
              s = __builtin_fmaf(bf16hi_to_f32(pair), qd[d + 1], s);
            };
            add(__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x[w], step, 0)), 0);
            add(__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x[w], step, 1)), 2);
            add(__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x[w], step, 2)), 4);
            add(__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x[w], step, 3)), 6);
          }
        }
        s *= a.c;
      }
      float t0 = s;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) t0 = __builtin_elementwise_maximum(t0, __shfl_xor(t0, d, 64));
      const float mn = __builtin_elementwise_maximum(m, t0);
      const float mb = mn == kNegInf ? 0.f : mn;
      const float f = m == kNegInf ? 0.f : exp2_fast(m - mb);
      m = mn;
      const float p = exp2_fast(s - mb);
      float sum = p;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
      l = l * f + sum;
      o0 *= f;
      o1 *= f;
      for (uint64_t left = __ballot(id >= 0); left; left &= left - 1) {
        const int j = __builtin_ctzll(left);
        const float w = __shfl(p, j, 64);
        const int64_t off = __shfl(vo, j, 64);
        if (2 * lane < D) {
          const unsigned x = a.cache.v[off + lane];
          const float step = __uint_as_float((unsigned)a.cache.v_blocks[(off >> 4) + lane / 16] << 23);
          const unsigned pair = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, step, 0));
          o0 = __builtin_fmaf(w, bf16lo_to_f32(pair), o0);
          o1 = __builtin_fmaf(w, bf16hi_to_f32(pair), o1);
        }
      }
    }
    const float inv = l > 0.f ? a.v_scale / l : (l == 0.f ? 0.f : l);
    if (2 * lane < D) {
      uint16_t* op = a.out + (int64_t)t * a.o_token + (int64_t)hh * a.o_head + 2 * lane;
      *reinterpret_cast<unsigned*>(op) = pack_bf16(o0 * inv, o1 * inv);
    }
    if (a.lse && lane == 0)
      a.lse[(int64_t)t * a.heads + hh] = l == 0.f ? kNegInf : (m + __builtin_log2f(l)) * kLn2;
  }
}

template <int D>
hipError_t rows_for(const AttendArgs& a, int columns, int blocks, hipStream_t stream) {
  clear_stale_error();
  const dim3 grid(blocks), block(256);
  const bool multi = a.max_q > 1;
  if (columns == 1 && !multi) hipLaunchKernelGGL((attend4_row_kernel<D, 1, false>), grid, block, 0, stream, a);
  else if (columns == 2 && !multi) hipLaunchKernelGGL((attend4_row_kernel<D, 2, false>), grid, block, 0, stream, a);
  else if (columns == 4 && !multi) hipLaunchKernelGGL((attend4_row_kernel<D, 4, false>), grid, block, 0, stream, a);
  else if (columns == 1) hipLaunchKernelGGL((attend4_row_kernel<D, 1, true>), grid, block, 0, stream, a);
  else if (columns == 2) hipLaunchKernelGGL((attend4_row_kernel<D, 2, true>), grid, block, 0, stream, a);
  else if (columns == 4) hipLaunchKernelGGL((attend4_row_kernel<D, 4, true>), grid, block, 0, stream, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend4_rows(const AttendArgs& a, int dim, int columns, int blocks, hipStream_t stream) {
  if (blocks < 1 || a.batch > kAttendMaxSeqs || a.rows > 16 * columns) return hipErrorInvalidValue;
  if (dim == 64) return rows_for<64>(a, columns, blocks, stream);
  if (dim == 128) return rows_for<128>(a, columns, blocks, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_attend4(const AttendArgs& a, int dim, hipStream_t stream) {
  const int64_t rows = (int64_t)a.tokens * a.heads;
  const dim3 grid((unsigned)(rows < (1 << 22) ? rows : (1 << 22)));
  clear_stale_error();
  if (dim == 64) hipLaunchKernelGGL(attend4_plain_kernel<64>, grid, dim3(64), 0, stream, a);
  else if (dim == 128) hipLaunchKernelGGL(attend4_plain_kernel<128>, grid, dim3(64), 0, stream, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace bd
