// Attention over a paged cache of 4-bit keys and values: decode with prefixes shared by the segments of a
// batch, and causal attention with a sliding window and first tokens that stay visible.
//
// Mathematics, per query row q of kv head h and its visible keys j (k_j and v_j: e2m1 codes times their
// block's power of two):
//   s_j = c * (q . k_j),  c = scale * k_scale * log2(e)
//   m = max_j s_j,  l = sum_j 2^(s_j - m),  o = v_scale / l * sum_j 2^(s_j - m) v_j
// in one pass over the keys: the running maximum m and sum l are kept in fp32 per row, and the fp32 output
// sums are rescaled when m grows.  As from the wider caches, scores are computed transposed, S^T = K Q^T, so
// that each lane has scores of one query row and the weights are the B operand of O^T = V^T P^T as they are.
// K goes into the scaled matrix instruction in 4 bits (no widening, a quarter of the LDS bytes), V is
// widened to bf16, exactly: its blocks lie along the dims, not along the keys that the second product sums.
#include <type_traits>

#include "attend_device.h"

namespace bd {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x6 __attribute__((ext_vector_type(6)));
typedef float f32x32 __attribute__((ext_vector_type(32)));

// 8 codes -> 8 bf16, times a power of two; exact
__device__ __forceinline__ u32x4 fp4x8_to_bf16(unsigned v, float step) {
  return u32x4{__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, step, 0)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, step, 1)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, step, 2)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, step, 3))};
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float block_step(unsigned byte) { return __uint_as_float(byte << 23); }

// ---------------------------------------------------------------------------------------------
// Queries.  The scaled matrix instruction takes K's codes and scale bytes as they lie in memory, against
// another operand of at most 8 bits a value, so a query goes in as four rows of e2m3 (4 significant bits, or
// steps of 1/8 below 2): by blocks of 32 dims, q / 2^e = x0 + 2^-4 x1 + 2^-9 x2 + 2^-14 x3, where 2^e is the
// smallest power of two with max |q| <= 7.5 * 2^e, and each x is what those before it leave, in its unit,
// rounded.  x0 leaves at most 2^-2 (2^-4 of values below 2), x1 2^-8, x2 2^-13, x3 2^-18: a bf16 value's 8
// bits are exact down to 2^-10, and smaller values off by at most 2^-19 of the block's largest: log-sums of
// normal queries come out 4e-8 off, as from a bf16 cache (two rows of e4m3, which take the same time, left those
// over few keys 5e-6 off, three of e2m3 3e-6 in 98% of the time).  A block with an infinity or NaN has scale bytes 255,
// which make its row's scores NaN.
// ---------------------------------------------------------------------------------------------
constexpr int kParts = 4;
__device__ constexpr int part_shift(int k) { return k == 0 ? 0 : 5 * k - 1; }  // 0, 4, 9, 14
struct Query {
  i32x6 part[kParts];
  int scales;  // bytes: e - part_shift(k) + 127
};
// 32 values / scale as e2m3 codes, to nearest even, at most 7.5: code 2 i from even[i], 2 i + 1 from odd[i].
// (In assembly: the compiler gives its builtin's result registers that overlap the sources.)
__device__ __forceinline__ i32x6 to_e2m3(const f32x16& even, const f32x16& odd, float scale) {
  i32x6 r;
  asm("v_cvt_scalef32_2xpk16_fp6_f32 %0, %1, %2, %3" : "=&v"(r) : "v"(even), "v"(odd), "v"(scale));
  return r;
}
__device__ __forceinline__ f32x32 e2m3_values(const i32x6& codes, float scale) {
  f32x32 r;
  asm("v_cvt_scalef32_pk32_f32_fp6 %0, %1, %2" : "=&v"(r) : "v"(codes), "v"(scale));
  return r;
}
// x: 32 bf16 values
__device__ __forceinline__ Query split_query(const u32x4* x) {
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[i >> 2][i & 3] & 0x7FFF7FFFu));
  const int top = max((int)m[0], (int)m[1]);  // bits of the largest |value|
  const int exponent = top >> 7;
  // (larger than need be where all values are below 2^-110, so that all scales are numbers)
  const int e = max(exponent - 2 + ((top & 0x7F) > 0x70 ? 1 : 0), part_shift(kParts - 1) + 1);
  Query q;
  q.scales = 0;
#pragma unroll
  for (int k = 0; k < kParts; ++k) q.scales |= (exponent == 255 ? 255 : e - part_shift(k)) << (8 * k);
  f32x16 even, odd;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    even[i] = bf16lo_to_f32(x[i >> 2][i & 3]);
    odd[i] = bf16hi_to_f32(x[i >> 2][i & 3]);
  }
#pragma unroll
  for (int k = 0; k < kParts; ++k) {
    const float scale = block_step((unsigned)(e - part_shift(k)));
    q.part[k] = to_e2m3(even, odd, scale);
    if (k == kParts - 1) break;
    const f32x32 v = e2m3_values(q.part[k], scale);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      even[i] -= v[2 * i];
      odd[i] -= v[2 * i + 1];
    }
  }
  return q;
}

// Part SEL of the queries against 16 (32) keys: c + K q, K's scale byte in byte BYTE of k_bytes
template <int SEL>
__device__ __forceinline__ f32x4 mfma_k16(const u32x4& k, int k_byte, const Query& q, const f32x4& c) {
  const i32x8 a = {(int)k[0], (int)k[1], (int)k[2], (int)k[3], 0, 0, 0, 0};
  const i32x6& p = q.part[SEL];
  const i32x8 b = {p[0], p[1], p[2], p[3], p[4], p[5], 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 2, 0, k_byte, SEL, q.scales);
}
template <int SEL, int BYTE>
__device__ __forceinline__ f32x16 mfma_k32(const u32x4& k, int k_bytes, const Query& q, const f32x16& c) {
  const i32x8 a = {(int)k[0], (int)k[1], (int)k[2], (int)k[3], 0, 0, 0, 0};
  const i32x6& p = q.part[SEL];
  const i32x8 b = {p[0], p[1], p[2], p[3], p[4], p[5], 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 2, BYTE, k_bytes, SEL, q.scales);
}

// Values that are no finite number once they are bf16: all of a block of NaN (byte 255), and under the largest
// scales 2^128 and more (4 and 6 * 2^126 of byte 253, 2 and more * 2^127 of byte 254), which the conversion
// makes infinities.  Their codes' bits among those of v; byte: the block's scale.
constexpr unsigned kOddByte = 253;  // the first scale with such values
__device__ __forceinline__ unsigned odd_codes(unsigned v, unsigned byte) {
  const unsigned ones = 0x11111111u;
  const unsigned m = byte == 255 ? ones : (byte == 254 ? (v >> 2) & ones : (byte == 253 ? (v >> 2) & (v >> 1) & ones : 0));
  return 15u * m;
}
// Values d .. d + 3 of a value row that are such, else 0; d is a multiple of 4, byte: their block's scale
__device__ __forceinline__ f32x4 odd_values(const unsigned char* row, unsigned byte, int d) {
  const unsigned codes = *reinterpret_cast<const uint16_t*>(row + (d >> 1)), odd = odd_codes(codes, byte);
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = byte == 255 ? __builtin_nanf("") : ((codes >> (4 * e + 3)) & 1u ? kNegInf : -kNegInf);
    r[e] = (odd >> (4 * e)) & 15u ? x : 0.f;
  }
  return r;
}

// ---------------------------------------------------------------------------------------------
// Row kernel: up to 16 * NC query rows (the heads of one kv head, for one or a few tokens) against a key
// list, each of a workgroup's 4 waves 32 keys of a 128-key step on its own.  A lane's 16 bytes of a K row
// are one block of 32 dims, as the scaled matrix instruction wants its operand (dim 64: one row in the
// first two lane groups, another, 16 keys on, in the last two, whose queries are zeros; for the others' turn
// the halves change places).  V rows are widened to bf16 into 8 KiB of the wave's LDS, and read transposed,
// four 16-row tiles ahead of the product.  The work split, and what joins its pieces, are those of the wider
// caches' row kernel.
//
// Bound by reading the cache: 64 sequences x 8 kv heads of up to 8208 keys, dim 128, 480 MB in 100 us, 4.8
// TB/s (a large copy's 5.2); one sequence's 131072 keys, 143 MB in 33.5 us, 4.3 TB/s, 4 us of them to begin.
// Vector instructions are busy 50% of the time, matrix instructions 13%, the LDS 33% (bank conflicts 13%).
// Where the keys come from the caches (64 sequences in 14 segments, 100 MB of readings, 43 MB of them from
// memory: 31 us) it is the chain of a step within a wave.  Tried and no faster: rows two steps ahead in two
// sets of registers, queries in LDS; two workgroups a compute unit instead of three, with rows one or two
// steps ahead; keys' lists in vector registers and byte loads of the scales, which the compiler widens at
// once and so waits for; a unit's first rows fetched during the last step of the unit before it; up to 8 rows
// in two columns each, with two of the query's parts and one of a wave's two key tiles, which halves the
// score products and the exponentials.  At dim 128 four column blocks spill 41 registers.
// ---------------------------------------------------------------------------------------------
// The aligned word with the scale bytes of the row at byte o of the scale bytes (dim 64: a row has two, at
// bits 0 or 16; the word's other half is a neighbour's, or behind the array's end in the same word, and is
// not looked at).
template <int D>
__device__ __forceinline__ unsigned block_word(const unsigned char* blocks, int64_t o, int* at) {
  *at = D == 128 ? 0 : 8 * (int)(o & 2);
  return *reinterpret_cast<const unsigned*>(blocks + (D == 128 ? o : o & ~3ll));
}

template <int D, int NC>
struct Row4Loop {
  static constexpr int kLoads = D / 64;   // keys a lane has a block of, per step
  static constexpr int kTiles = D / 16;   // 16-row tiles of O^T

  Query q[NC];
  f32x4 o[NC][kTiles];
  float m[NC], l[NC];
  int pos[NC];   // the column's token position (window op with several tokens)
  u32x4 kr[kLoads], vr[kLoads];
  unsigned kb[kLoads], vb[kLoads];  // words that hold the rows' scale bytes
  int kat[kLoads], vat[kLoads];     // (dim 64) where in them this row's begin, bits
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
      // (most caches lay keys and values out alike: then their offsets are worked out once)
      int64_t vo = ko;
      if (!a.cache.alike)
        vo = page_row_bytes(page, at, a.cache.v_page, a.cache.v_token) + (int64_t)h * a.cache.v_head;
      kr[i] = *reinterpret_cast<const u32x4*>(a.cache.k + ko + 16 * block(g));
      vr[i] = *reinterpret_cast<const u32x4*>(a.cache.v + vo + 16 * block(g));
      // (whole words: the compiler widens a loaded byte at once, and waits for it there)
      kb[i] = block_word<D>(a.cache.k_blocks, ko >> 4, &kat[i]);
      vb[i] = block_word<D>(a.cache.v_blocks, vo >> 4, &vat[i]);
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
        vb[i] = 0;
      }
  }
  // the lane's blocks' scale bytes, K's in the low byte
  __device__ __forceinline__ int k_byte(int i, int g) const { return (int)(kb[i] >> (kat[i] + 8 * block(g))); }
  __device__ __forceinline__ unsigned v_byte(int i, int g) const {
    return __builtin_amdgcn_ubfe(vb[i], vat[i] + 8 * block(g), 8);
  }
  // keys with values that may be no finite numbers, bit (key); those that are none become zeros
  __device__ __forceinline__ unsigned clear_odd_blocks(int g) {
    unsigned odd = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const unsigned byte = v_byte(i, g);
      const bool f = byte >= kOddByte;
      uint64_t m = __ballot(f);
      if (m) {
        if (f) {
#pragma unroll
          for (int e = 0; e < 4; ++e) vr[i][e] &= ~odd_codes(vr[i][e], byte);
          if (byte == 255) vb[i] = 0;
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
  __device__ __forceinline__ unsigned clear_odd_keys(int g) {
    if constexpr (D == 128) return 0;
    const bool f = (k_byte(0, g) & 255) == 255;
    uint64_t m = __ballot(f);
    if (!m) return 0;
    if (f) kb[0] = 0, kr[0] = u32x4{0, 0, 0, 0};
    m |= m >> 16;
    return (unsigned)(m & 0xFFFFull) | ((unsigned)((m >> 32) & 0xFFFFull) << 16);
  }
  // column j of block c is query row 16 c + j; row: this lane's, or null
  __device__ __forceinline__ void load_query(int c, const uint16_t* row, int g) {
    u32x4 x[4];
    const bool live = row && (D == 128 || g < 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = live ? *reinterpret_cast<const u32x4*>(row + 32 * block(g) + 8 * i) : u32x4{0, 0, 0, 0};
    q[c] = split_query(x);
  }
  // scores of the keys 16 r .. 16 r + 15 (lane (j, g): keys 4 g .. + 3) with all queries
  __device__ __forceinline__ void scores(int r, int g, f32x4 (*s)[2]) const {
    u32x4 k = kr[D == 128 ? r : 0];
    int byte = k_byte(D == 128 ? r : 0, g);
    if (D == 64 && r == 1) {  // the last two lane groups' keys to the first two, which have the queries
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = __builtin_amdgcn_permlane32_swap(k[i], k[i], false, false)[1];
      byte = (int)__builtin_amdgcn_permlane32_swap((unsigned)byte, (unsigned)byte, false, false)[1];
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
      x = mfma_k16<0>(k, byte, q[c], x);
      x = mfma_k16<1>(k, byte, q[c], x);
      x = mfma_k16<2>(k, byte, q[c], x);
      s[c][r] = mfma_k16<3>(k, byte, q[c], x);
    }
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
  // [16 columns][D], dims by fours, four n of column j at n ^ j: a column's length is a multiple of all
  // banks (256 sequences' own keys, in short units, 51 us instead of 58)
  auto fours = [](int col, int n) { return col * D + 4 * (n ^ col); };
  float* const ow = reinterpret_cast<float*>(vlds + wave * kWaveLds);
  const bool live = 16 * c + j < rows;
  if (live) {
    int col = j;  // (opaque: the addresses are worked out here, not before the steps, which lack the registers)
    asm volatile("" : "+v"(col));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *reinterpret_cast<f32x4*>(ow + fours(col, 4 * i + g)) = oc[i];
  }
  if (live && g == 0) {
    ml[wave][j][0] = mc;
    ml[wave][j][1] = lc;
  }
  __syncthreads();
  constexpr int kQuads = 16 * D / 4 / 256;  // f32x4 per thread
#pragma unroll
  for (int e = 0; e < kQuads; ++e) {
    int idx = tid + 256 * e;
    asm volatile("" : "+v"(idx));
    const int col = idx / (D / 4), d4 = idx - col * (D / 4);
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
                      reinterpret_cast<const float*>(vlds + v * kWaveLds) + fours(col, d4));
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
    // (values from LDS are the same for all lanes, which the compiler does not know: told so, it keeps what
    // comes of them, the key list above all, in scalar registers)
    total = (int64_t)uniform(scan[a.batch]) * a.kv_heads;
    if (blockIdx.x == 0)
      for (int i = tid; i <= a.batch; i += 256) a.scan[i] = scan[i];
    const int workers = split_workers(total, a.workers);
    if ((int)blockIdx.x >= workers) return;
    x = split_begin(blockIdx.x, total, workers);
    x_end = split_begin(blockIdx.x + 1, total, workers);
  }

  int b = -1, h = 0;
  while (x < x_end) {
    int s_begin, s_end;
    RowUnit u;
    if (a.direct) {
      b = blockIdx.x / a.kv_heads;
      h = blockIdx.x - b * a.kv_heads;
      u = row_unit(a, b);
      s_begin = 0;
      s_end = row_steps(u);
      x = x_end;
    } else {
      int s;
      if (b < 0) {
        b = uniform(scan_find(scan, a.batch, (int)(x / a.kv_heads)));
        u = row_unit(a, b, uniform(lens[b]));
        s = row_steps(u);
        const int64_t x0 = (int64_t)uniform(scan[b]) * a.kv_heads;
        h = (int)((x - x0) / s);
        s_begin = (int)(x - x0 - (int64_t)h * s);
      } else {
        // the next unit: there is one, x being before the end of all (looked up anew, 256 sequences' own
        // keys took 63 us instead of 59)
        if (++h == a.kv_heads) {
          h = 0;
          do ++b;
          while (uniform(scan[b + 1] - scan[b]) == 0);
        }
        u = row_unit(a, b, uniform(lens[b]));
        s = row_steps(u);
        s_begin = 0;
      }
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
      if constexpr (MULTI) odd = w.clear_odd_blocks(g);
      // ---- V into LDS, scores from K
#pragma unroll
      for (int i = 0; i < Loop::kLoads; ++i) {
        const float step = block_step(w.v_byte(i, g));
        const int row = Loop::key(i, j, g), unit = 4 * Loop::block(g);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<u32x4*>(vl + v_unit<D>(row, unit + e)) = fp4x8_to_bf16(w.vr[i][e], step);
      }
      const unsigned odd_keys = w.clear_odd_keys(g);
      f32x4 s[NC][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) w.scores(r, g, s);
      if (D == 64 && odd_keys) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((odd_keys >> (16 * r + 4 * g + i)) & 1u) s[c][r][i] = __builtin_nanf("");
      }
      // ---- the next tile's rows are on their way while this one is worked on (not before the products have
      // their operands: the compiler would keep those in copies)
      __builtin_amdgcn_sched_barrier(0);
      if (base + kRowStep < end) {
        w.fetch(a, h, g);
        if (base + 2 * kRowStep < end) w.lookup(a, kl, base + 2 * kRowStep, j, g);
      }

      // ---- V^T from LDS, the first half on its way while the weights are worked out: the lane's 8 keys are
      // 4g .. 4g + 3 and 16 + 4g .. 16 + 4g + 3
      u32x4 vt[Loop::kTiles];
      const int vr0 = 4 * g + (j >> 2), vu = (j & 3) >> 1, vb = 8 * (j & 1);
      auto read_values = [&](int i0) {
#pragma unroll
        for (int i = i0; i < i0 + Loop::kTiles / 2; ++i) {
          const u32x2 lo = lds_read_tr(vl + v_unit<D>(vr0, 2 * i + vu) + vb);
          const u32x2 hi = lds_read_tr(vl + v_unit<D>(16 + vr0, 2 * i + vu) + vb);
          vt[i] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
      };
      read_values(0);
      __builtin_amdgcn_sched_barrier(0);
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

      // ---- O^T += V^T P^T
      read_values(Loop::kTiles / 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < Loop::kTiles; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) w.o[c][i] = mfma16(vt[i], p[c], w.o[c][i]);
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
              const unsigned byte = (unsigned)uniform(blocks[i >> 1]);
              if (byte < kOddByte) continue;
              int d = 16 * i + 4 * g;
              // (opaque: else its part of the lane is kept in a register over the steps, one too many at dim 128)
              if constexpr (NC == 1) asm volatile("" : "+v"(d));
              const f32x4 x = odd_values(row, byte, d);
#pragma unroll
              for (int e = 0; e < 4; ++e) w.o[c][i][e] = w.o[c][i][e] + (seen ? x[e] : 0.f);
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

// ---------------------------------------------------------------------------------------------
// Tile kernel: 256 query rows (tokens x the heads of one kv head) against a key list in 64-key steps.  8
// waves of 32 rows; K codes and scale bytes in LDS as they are, V widened to bf16 on the way there, each a
// step ahead.  Prefixes: work cut into equal runs, and where a segment's rows fill at most half the waves,
// the others take a second key tile of the same step (256 sequences in 14 segments 118 -> 106 us).  Windows:
// tile_work below.
//
// Bound by matrix and vector instructions, which take turns on a SIMD rather than overlap: of a step's about
// 5400 cycles the two waves of a SIMD have 2000 of products (16 scaled ones for the scores, 16 of bf16 for the
// values, a wave) and 2300 of weights (32 exponentials a lane, at a quarter of the rate, are half of that).
// Dim 128, 64 heads on 8: 4 chunks of up to 2048 tokens behind 4096, window 4096, 689 GFLOP in 720 to 800 us
// by the machine, 860 to 960 TFLOP/s (a large matrix product reaches 1192).  Tried and slower or no faster (that
// call, 761 us at the time): the late half of the waves a phase behind, so that products meet weights, 861
// us; a barrier that leaves the next rows' loads on their way, no change; scores by two e4m3 products or
// three of e2m3 instead of four, within 2%.
// ---------------------------------------------------------------------------------------------
// Byte offset of 16-byte unit u (32 dims) of row r in a K tile: a wave's reads take one unit of 32 rows
template <int D>
__device__ __forceinline__ unsigned k4_unit(int r, int u) {
  return D == 128 ? (unsigned)(r * 64 + ((u ^ ((r >> 1) & 3)) << 4)) : (unsigned)(r * 32 + (u << 4));
}

// Byte offsets of a key's rows; bit 0 of k: there is no such key (offsets 0).
struct Row4Place {
  int64_t k, v;
};
// Where the lane's key sits: its table entry (null: no such key), and the rows' offsets from it.
struct Key4Lookup {
  const int32_t* entry;
  int slot;
  __device__ __forceinline__ Key4Lookup(const PagedCache& c, const KeyList& kl, int vp) {
    const int kp = key_position(kl, vp);
    const int page = page_quotient(kp < 0 ? 0 : kp, c.div);
    const int at = key_table_index(kl, vp, page);
    slot = kp - page * c.page_size;
    entry = at >= 0 ? (vp < kl.na ? kl.ta : kl.tb) + at : nullptr;
  }
  __device__ __forceinline__ Row4Place place(const PagedCache& c, int id) const {
    const bool ok = entry && page_id_checked(id, c.num_pages) >= 0;
    const int p = ok ? id : 0, t = ok ? slot : 0;
    return Row4Place{page_row_bytes(p, t, c.k_page, c.k_token) | (ok ? 0 : 1),
                     page_row_bytes(p, t, c.v_page, c.v_token)};
  }
};

// Work of a tile launch over `units` (sequence, row tile, kv head) on `workers` compute units: as many whole
// units as fill them a number of times, then the rest's keys cut into as many parts as fill them once more
// (at most `most`): few units use the whole machine, and many end together (the last 8 of 1288 units, left
// whole, kept 8 compute units busy for a sixth of the time).
struct TileWork {
  int unit;  // -1: none
  int part, parts;
  int slot;  // of the part's sums
};
__device__ __forceinline__ TileWork tile_work(int units, int workers, int most, int w) {
  const int rest = most > 1 ? units % workers : 0, whole = units - rest;
  if (w < whole) return TileWork{w, 0, 1, 0};
  const int j = w - whole;
  if (rest == 0) return TileWork{-1, 0, 1, 0};
  const int parts = min(workers / rest, most);
  if (j >= rest * parts) return TileWork{-1, 0, 1, 0};
  const int part = j / rest, unit = j - part * rest;
  return TileWork{whole + unit, part, parts, unit * parts + part};
}

// What a thread moves of a step: an eighth of a key's rows, D / 16 bytes each of K and V, and the key's scale
// bytes.
template <int D>
struct Tile4Stage {
  static constexpr int kBytes = D / 16;
  u32x2 k, v;
  unsigned vb, kb;  // words that hold the rows' scale bytes
  int vat, kat;     // (dim 64) where in them, bits
  bool ok;

  __device__ __forceinline__ void fetch(const AttendArgs& a, int64_t k_head, int64_t v_head,
                                        const Row4Place* places, int tid) {
    const Row4Place at = places[tid >> 3];
    const int part = tid & 7;
    // absent keys read page 0; their values are cleared before they are stored, their scores masked
    ok = (at.k & 1) == 0;
    const int64_t ko = (at.k & ~15ll) + k_head, vo = at.v + v_head;
    const unsigned char* kp = a.cache.k + ko + kBytes * part;
    const unsigned char* vp = a.cache.v + vo + kBytes * part;
    if constexpr (D == 128) {
      k = *reinterpret_cast<const u32x2*>(kp);
      v = *reinterpret_cast<const u32x2*>(vp);
    } else {
      k[0] = *reinterpret_cast<const unsigned*>(kp);
      v[0] = *reinterpret_cast<const unsigned*>(vp);
    }
    vb = block_word<D>(a.cache.v_blocks, vo >> 4, &vat);
    kb = block_word<D>(a.cache.k_blocks, ko >> 4, &kat);
  }
  // state: per key, bit 0: it exists; bit 1 (edge steps, where some row does not see some key): some of its
  // values may be no finite numbers.  Those that are none are stored as zeros, since their product with a zero
  // weight would be NaN, and added later for the rows that see them.
  __device__ __forceinline__ void store(unsigned char* kt, unsigned* kbt, unsigned char* vt, int* state, bool edge,
                                        int tid) {
    const int r = tid >> 3, part = tid & 7;
    int bits = ok;
    unsigned byte = __builtin_amdgcn_ubfe(vb, vat + 8 * (part * (D / 8) / 32), 8);
    if (!ok) {
      v = u32x2{0, 0};
      byte = 0;
    }
    if (edge) {
      const bool f = byte >= kOddByte;
      if (f) {
        v[0] &= ~odd_codes(v[0], byte);
        v[1] &= ~odd_codes(v[1], byte);
        if (byte == 255) byte = 0;
      }
      const uint64_t m = __ballot(f) >> (tid & 56);  // of this key's eighths
      if (m & 0xFF) bits |= 2;
    }
    const float step = block_step(byte);
    if constexpr (D == 128) {
      *reinterpret_cast<u32x2*>(kt + k4_unit<D>(r, part >> 1) + 8 * (part & 1)) = k;
      *reinterpret_cast<u32x4*>(vt + v_unit<D>(r, 2 * part)) = fp4x8_to_bf16(v[0], step);
      *reinterpret_cast<u32x4*>(vt + v_unit<D>(r, 2 * part + 1)) = fp4x8_to_bf16(v[1], step);
    } else {
      *reinterpret_cast<unsigned*>(kt + k4_unit<D>(r, part >> 2) + 4 * (part & 3)) = k[0];
      *reinterpret_cast<u32x4*>(vt + v_unit<D>(r, part)) = fp4x8_to_bf16(v[0], step);
    }
    if (part == 0) {
      kbt[r] = kb >> kat;
      state[r] = bits;
    }
  }
};

// prefixes may take two key tiles a step
constexpr int tile4_buffers(bool prefix) { return prefix ? 4 : 2; }
constexpr int tile4_lds(int D, bool prefix) { return tile4_buffers(prefix) * kTileKeys * (D * 2 + D / 2); }

template <int D, bool PREFIX>
__global__ __launch_bounds__(512, 2) void attend4_tile_kernel(const AttendArgs a) {
  constexpr int kTile = kTileKeys * D * 2;   // bytes of a V tile
  constexpr int kTileK = kTileKeys * D / 2;
  constexpr int kSteps = D / 64;   // matrix steps over D of a score tile
  constexpr int kOut = D / 32;     // 32-row tiles of O^T
  constexpr int kBuffers = tile4_buffers(PREFIX);
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // K tiles, then V tiles
  unsigned char* const vbuf = smem + kBuffers * kTileK;
  __shared__ unsigned kbytes[kBuffers][kTileKeys];
  __shared__ int state[kBuffers][kTileKeys];
  __shared__ Row4Place places[4][kTileKeys];
  __shared__ int entries[8][kTileKeys];
  __shared__ int scan[kAttendMaxSeqs + 1];
  __shared__ int segs[PREFIX ? kAttendMaxSegments + 1 : 1];
  __shared__ int wave_sum[8];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane & 31, hf = lane >> 5;
  const int tpt = kTileRows / a.group;  // tokens per tile
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
    if (blockIdx.x == 0 && a.tile_parts > 1)  // for the joining kernel
      for (int i = tid; i <= a.batch; i += 512) a.scan[i] = scan[i];
  }

  while (x < x_end) {
    KeyList kl;
    int t0, nt, p0 = 0, h, s_begin, s_end;
    int64_t slot = 0;
    int parts = 1;  // that the unit's keys are split into
    bool half = false;  // the unit's rows fill at most half the waves: the others take a second key tile
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
      const TileWork w = tile_work(uniform(scan[a.batch]) * a.kv_heads, a.tile_workers, a.tile_parts, blockIdx.x);
      if (w.unit < 0) return;
      const int ti = uniform(scan[a.batch]) - 1 - w.unit / a.kv_heads;
      h = w.unit % a.kv_heads;
      parts = w.parts;
      slot = w.slot;
      const int b = scan_find(scan, a.batch, ti);
      const RowUnit u = row_unit(a, b);
      const int rt = ti - scan[b];
      t0 = u.t0 + rt * tpt;
      nt = u.nq - rt * tpt < tpt ? u.nq - rt * tpt : tpt;
      p0 = u.p0 + rt * tpt;
      // keys up to the tile's last token
      const int len = p0 + nt < 0 ? 0 : p0 + nt;
      kl = window_keys(a.table + (int64_t)b * a.width, a.width, len, p0, a.window, a.sinks);
      const int steps = (kl.n + kTileKeys - 1) / kTileKeys;
      s_begin = (int)((int64_t)steps * w.part / parts);
      s_end = (int)((int64_t)steps * (w.part + 1) / parts);
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
    Query qs[kSteps];  // of step d: the lane's dims 64 d + 32 hf .. + 31
    {
      const uint16_t* qp = a.q + (int64_t)(t0 + t) * a.q_token + (int64_t)hh * a.q_head + 32 * hf;
#pragma unroll
      for (int d = 0; d < kSteps; ++d) {
        u32x4 x4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x4[i] = live ? *reinterpret_cast<const u32x4*>(qp + 64 * d + 8 * i) : u32x4{0, 0, 0, 0};
        qs[d] = split_query(x4);
      }
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
    auto look_begin = [&](int s) {
      if (((s - s_begin) & 7) == wave) {
        const Key4Lookup look(a.cache, kl, s * kTileKeys + lane);
        if (look.entry) copy4(look.entry, entries_at + wave * kTileKeys * 4);
      }
    };
    auto look_end = [&](int s) {
      if (((s - s_begin) & 7) == wave) {
        const Key4Lookup look(a.cache, kl, s * kTileKeys + lane);
        places[(s - s_begin) & 3][lane] = look.place(a.cache, entries[wave][lane]);
      }
    };
    // edge step: some row of the tile does not see some key of it (the same for all waves)
    auto hides = [&](int base) {
      if constexpr (PREFIX) return false;
      const int f = key_position(kl, base), last = key_position(kl, base + kTileKeys - 1);
      return base < kl.na || last > p0 || p0 + nt - 1 - f >= a.window;
    };
    const int64_t k_head = (int64_t)h * a.cache.k_head, v_head = (int64_t)h * a.cache.v_head;
    Tile4Stage<D> st[PREFIX ? 2 : 1];
    auto fetch = [&](int s) {
      st[0].fetch(a, k_head, v_head, places[(s - s_begin) & 3], tid);
      if (PREFIX && half) st[PREFIX].fetch(a, k_head, v_head, places[(s + 1 - s_begin) & 3], tid);
    };
    auto store_one = [&](Tile4Stage<D>& t, int s) {
      const int buf = (s - s_begin) & (kBuffers - 1);
      t.store(smem + buf * kTileK, kbytes[buf], vbuf + buf * kTile, state[buf], hides(s * kTileKeys), tid);
    };
    auto store = [&](int s) {
      store_one(st[0], s);
      if (PREFIX && half) store_one(st[PREFIX], s + 1);
    };
    const int take = PREFIX && half ? 2 : 1;  // key tiles a step
    for (int i = 0; i < (take == 2 ? 8 : 5); ++i) look_begin(s_begin + i);
    wait_copies<0>();
    __syncthreads();  // the last unit's tiles and notes are no longer read
    for (int i = 0; i < (take == 2 ? 4 : 3); ++i) look_end(s_begin + i);
    __syncthreads();
    fetch(s_begin);
    store(s_begin);
    fetch(s_begin + take);
    __syncthreads();
    if (take == 2) {
      for (int i = 4; i < 6; ++i) look_end(s_begin + i);
      for (int i = 8; i < 10; ++i) look_begin(s_begin + i);
      lds_barrier();
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
    for (int s0 = s_begin; s0 < s_end; s0 += take) {
      const int s = s0 + (half ? wave >> 2 : 0);  // this wave's tile
      const int buf = (s - s_begin) & (kBuffers - 1);
      const int base = s * kTileKeys;
      const int key_state = state[buf][lane];
      uint64_t valid = __ballot(key_state & 1);
      if (PREFIX && s >= s_end) valid = 0;
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
        u32x4 kf[2][kSteps];
        int kb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // the lane's scale bytes: of block hf in byte 0, of block 2 + hf in byte 2
          kb[i] = (int)(kbytes[buf][32 * i + q] >> (8 * hf));
#pragma unroll
          for (int d = 0; d < kSteps; ++d)
            kf[i][d] = *reinterpret_cast<const u32x4*>(smem + buf * kTileK + k4_unit<D>(32 * i + q, 2 * d + hf));
        }
        auto products = [&](auto byte) {
          constexpr int d = byte / 2;
          sc[0] = mfma_k32<0, byte>(kf[0][d], kb[0], qs[d], sc[0]);
          sc[1] = mfma_k32<0, byte>(kf[1][d], kb[1], qs[d], sc[1]);
          sc[0] = mfma_k32<1, byte>(kf[0][d], kb[0], qs[d], sc[0]);
          sc[1] = mfma_k32<1, byte>(kf[1][d], kb[1], qs[d], sc[1]);
          sc[0] = mfma_k32<2, byte>(kf[0][d], kb[0], qs[d], sc[0]);
          sc[1] = mfma_k32<2, byte>(kf[1][d], kb[1], qs[d], sc[1]);
          sc[0] = mfma_k32<3, byte>(kf[0][d], kb[0], qs[d], sc[0]);
          sc[1] = mfma_k32<3, byte>(kf[1][d], kb[1], qs[d], sc[1]);
        };
        products(std::integral_constant<int, 0>{});
        if constexpr (kSteps == 2) products(std::integral_constant<int, 2>{});
      }
      // ---- the next step's tiles; these buffers were last read before the barrier that began
      // this step
      if (s0 + take < s_end) {
        store(s0 + take);
        fetch(s0 + 2 * take);
        // (the loads that the store waited for are newer than the entries')
        for (int i = 0; i < take; ++i) look_end(s0 + 3 * take + i);
        for (int i = 0; i < take; ++i) look_begin(s0 + 5 * take + i);
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
          // 2^-8 of themselves); the sum l keeps them in fp32
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
            const unsigned char* blocks = a.cache.v_blocks + ((row_v - a.cache.v) >> 4);
            const bool seen = sees(kl, pq, a.window, a.sinks, vp);
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
              const unsigned byte = (unsigned)uniform(blocks[i]);
              if (byte < kOddByte) continue;
#pragma unroll
              for (int e4 = 0; e4 < 4; ++e4) {
                const f32x4 x = odd_values(row_v, byte, 32 * i + 8 * e4 + 4 * hf);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][4 * e4 + e] = o[i][4 * e4 + e] + (seen ? x[e] : 0.f);
              }
            }
          }
        }
      }
      __syncthreads();
    }
    // no copy into LDS outlives its use: the next unit, or workgroup, has these buffers
    wait_copies<0>();

    // ---- epilogue: lane (q, hf) holds dims 32 i + 8 (e / 4) + 4 hf + e % 4 of its row
    l = half_sum(l);
    if (live) {
      if (PREFIX || parts > 1) {
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

// Joins the parts of split units: a wave per query row, lanes of 4 dims, 64 / (D / 4) parts side by side,
// four loads each in flight, in a fixed order.
template <int D>
__global__ __launch_bounds__(256) void attend4_join_kernel(const AttendArgs a) {
  constexpr int kQ = D / 4, kWays = 64 / kQ;
  const int lane = threadIdx.x & 63;
  const int i = blockIdx.x / (kTileRows / 4);  // of the split units
  const int row = (blockIdx.x % (kTileRows / 4)) * 4 + (threadIdx.x >> 6);
  const int tpt = kTileRows / a.group;
  const int tiles = a.scan[a.batch], units = tiles * a.kv_heads;
  const int rest = units % a.tile_workers, whole = units - rest;
  if (i >= rest) return;
  const int parts = min(a.tile_workers / rest, a.tile_parts);
  if (parts == 1) return;
  const int unit = whole + i, h = unit % a.kv_heads;
  const int ti = tiles - 1 - unit / a.kv_heads;
  const int b = scan_find(a.scan, a.batch, ti);
  const RowUnit u = row_unit(a, b);
  const int t = (ti - a.scan[b]) * tpt + row / a.group, hh = h * a.group + row % a.group;
  if (row >= tpt * a.group || t >= u.nq) return;
  const int d4 = lane % kQ, way = lane / kQ;
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
  for (int p0 = way; p0 < parts; p0 += 4 * kWays) {
    f32x2 pm[4];
    f32x4 po[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = (int64_t)(i * parts + min(p0 + k * kWays, parts - 1)) * kTileRows + row;
      pm[k] = *reinterpret_cast<const f32x2*>(a.tile_ml + at * 2);
      po[k] = *reinterpret_cast<const f32x4*>(a.tile_o + at * D + 4 * d4);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (p0 + k * kWays < parts) add(pm[k][0], pm[k][1], po[k]);
  }
#pragma unroll
  for (int d = kQ; d < 64; d <<= 1) {
    const float om = __shfl_xor(mx, d, 64), ol = __shfl_xor(lt, d, 64);
    f32x4 oo;
#pragma unroll
    for (int e = 0; e < 4; ++e) oo[e] = __shfl_xor(ot[e], d, 64);
    add(om, ol, oo);
  }
  if (way == 0) {
    const float inv = lt > 0.f ? a.v_scale / lt : (lt == 0.f ? 0.f : lt);
    const int64_t tok = u.t0 + t;
    *reinterpret_cast<u32x2*>(a.out + tok * a.o_token + (int64_t)hh * a.o_head + 4 * d4) =
        u32x2{pack_bf16(ot[0] * inv, ot[1] * inv), pack_bf16(ot[2] * inv, ot[3] * inv)};
    if (a.lse && d4 == 0)
      a.lse[tok * a.heads + hh] = lt == 0.f ? kNegInf : (mx + __builtin_log2f(lt)) * kLn2;
  }
}

template <int D>
hipError_t rows_for(const AttendArgs& a, int columns, int blocks, hipStream_t stream) {
  clear_stale_error();
  const dim3 grid(blocks), block(256);
  const bool multi = a.max_q > 1;  // (with more than 32 rows: the tile kernel)
  if (columns == 1 && !multi) hipLaunchKernelGGL((attend4_row_kernel<D, 1, false>), grid, block, 0, stream, a);
  else if (columns == 2 && !multi) hipLaunchKernelGGL((attend4_row_kernel<D, 2, false>), grid, block, 0, stream, a);
  else if (columns == 4 && !multi) hipLaunchKernelGGL((attend4_row_kernel<D, 4, false>), grid, block, 0, stream, a);
  else if (columns == 1) hipLaunchKernelGGL((attend4_row_kernel<D, 1, true>), grid, block, 0, stream, a);
  else if (columns == 2) hipLaunchKernelGGL((attend4_row_kernel<D, 2, true>), grid, block, 0, stream, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

template <int D, bool PREFIX>
hipError_t tiles_for(const AttendArgs& a, int blocks, hipStream_t stream) {
  constexpr int lds = tile4_lds(D, PREFIX);
  static DeviceOnce once;
  const hipError_t e =
      set_dynamic_lds_once(once, reinterpret_cast<const void*>(&attend4_tile_kernel<D, PREFIX>), lds);
  if (e != hipSuccess) return e;
  clear_stale_error();
  hipLaunchKernelGGL((attend4_tile_kernel<D, PREFIX>), dim3(blocks), dim3(512), lds, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend4_rows(const AttendArgs& a, int dim, int columns, int blocks, hipStream_t stream) {
  if (blocks < 1 || a.batch > kAttendMaxSeqs || a.rows > 16 * columns) return hipErrorInvalidValue;
  if (dim == 64) return rows_for<64>(a, columns, blocks, stream);
  if (dim == 128) return rows_for<128>(a, columns, blocks, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_attend4_tiles(const AttendArgs& a, int dim, bool prefix, int blocks, hipStream_t stream) {
  if (blocks < 1 || a.batch > kAttendMaxSeqs || a.nseg > kAttendMaxSegments) return hipErrorInvalidValue;
  if (dim == 64) return prefix ? tiles_for<64, true>(a, blocks, stream) : tiles_for<64, false>(a, blocks, stream);
  if (dim == 128) return prefix ? tiles_for<128, true>(a, blocks, stream) : tiles_for<128, false>(a, blocks, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_attend4_join(const AttendArgs& a, int dim, int units, hipStream_t stream) {
  if (units < 1 || units > a.tile_workers) return hipErrorInvalidValue;
  const dim3 grid((unsigned)units * (kTileRows / 4));
  clear_stale_error();
  if (dim == 64) hipLaunchKernelGGL(attend4_join_kernel<64>, grid, dim3(256), 0, stream, a);
  else if (dim == 128) hipLaunchKernelGGL(attend4_join_kernel<128>, grid, dim3(256), 0, stream, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace bd
