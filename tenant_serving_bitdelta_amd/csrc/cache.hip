// Writing new keys and values into a paged cache, quantised on the way, and reading tokens back.
//
// Mathematics, per value x of a row, y = x / scale in fp32:
//   bf16  y rounded;   e4m3  min(max(y, -448), 448) rounded;
//   4 bits, per 32 consecutive values: 2^e = the smallest power of two with max |y| <= 7 * 2^e, code = y /
//   2^e rounded to the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, by the conversion
//   instruction.  No value is then off by more than half a step of that grid (with 2^e the largest power of
//   two below max |y| / 4, as is common, values near 8 would become 6).
// The quotient is a product where 1 / scale is exact, else a correctly rounded division.
//
// Bound by memory where tokens are many: 4 bytes of bf16 and 2 * 17/32 (4 bits) to 4 stored bytes per pair
// of a key and a value.  A thread takes 8 values (16 bytes of bf16) of one row at a time, so that a wave's
// loads and stores are whole lines, and 4 lanes hold a block of 32 (its largest value by two lane moves);
// each of a workgroup's tokens is looked up once, by one thread, while the rows to write are on their way.
// Measured, dim 128: 14 prompts of up to 8192 tokens, 8 heads, read from 4 bits, 363 MB in 58 us, 6.2 TB/s;
// 4.6 thousand tokens of 8 heads written in 4 bits, 24 MB in 10.7 us, and read back in 7.8; 7 thousand of 4
// heads written in e4m3, 22 MB in 9.2 us; four single tokens 3.5 us.  Of the short calls' times 3 us are the
// launch and the chain offsets -> length -> table -> place; a workgroup per token took 15 us for the 10.7.
// 65536 tokens of 8 heads: written in bf16 537 MB in 108 us (5.0 TB/s), e4m3 403 MB in 87 (4.6), 4 bits 340 MB
// in 77 (4.4; 89 with a scale that is no power of two), read back in 101 (5.3), 77 (5.2) and 54 us (6.3).
#include "bd_internal.h"
#include "cache.h"

namespace bd {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;  // of a workgroup at a time
constexpr int kAhead = 4;       // loads of a thread in flight

// Where a token's head 0 rows sit in the pages, byte offsets; row: some sequence has it; placed: it has a
// place (else the offsets are those of page 0, which may be read).
struct TokenPlace {
  int64_t k, v;
  int row, placed;
};

// offsets: the call's q_offsets in LDS
__device__ __forceinline__ TokenPlace token_place(const CacheArgs& a, const int* offsets, int t) {
  TokenPlace at{0, 0, 0, 0};
  int b = t;
  int64_t pos;
  if (a.q_offsets) {
    // the last sequence that begins at or before row t; empty ones end before it
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (offsets[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    const int end = offsets[b + 1];
    if (t < offsets[b] || t >= end) return at;
    pos = (int64_t)a.lens[b] - ((int64_t)end - t);
  } else {
    pos = (int64_t)a.lens[b] - 1;
  }
  at.row = 1;
  if (pos < 0) return at;
  const int page = page_quotient((int)pos, a.cache.div);
  if (page >= a.width) return at;
  const int id = page_id_checked(a.table[(int64_t)b * a.width + page], a.cache.num_pages);
  if (id < 0) return at;
  const int slot = (int)pos - page * a.cache.page_size;
  at.k = page_row_bytes(id, slot, a.cache.k_page, a.cache.k_token);
  at.v = page_row_bytes(id, slot, a.cache.v_page, a.cache.v_token);
  at.placed = 1;
  return at;
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  f32x2 f;
  f[0] = a;
  f[1] = b;
  return __builtin_bit_cast(unsigned, __builtin_convertvector(f, bf16x2));
}

__device__ __forceinline__ u16x2 max2(u16x2 a, u16x2 b) { return __builtin_elementwise_max(a, b); }
// max over the 4 lanes of a block, in each
__device__ __forceinline__ unsigned block_max(unsigned m) {
  const unsigned x = max(m, (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
  return max(x, (unsigned)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true));
}
__device__ __forceinline__ float quotient(float x, float scale, float inverse) {
  return inverse != 0.f ? x * inverse : x / scale;
}

// 8 bf16 values -> what is stored of them, at unit `part` of row `to` (blocks: its scale bytes)
template <int KV>
__device__ __forceinline__ void store8(const u32x4& x, unsigned char* to, unsigned char* blocks, int part,
                                       float scale, float inverse, float near) {
  if constexpr (KV == BITDELTA_KV_BF16) {
    u32x4 r = x;
    if (scale != 1.f) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = pack_bf16(quotient(bf16lo_to_f32(x[i]), scale, inverse),
                         quotient(bf16hi_to_f32(x[i]), scale, inverse));
    }
    *reinterpret_cast<u32x4*>(to + 16 * part) = r;
  } else if constexpr (KV == BITDELTA_KV_FP8) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = e & 1 ? bf16hi_to_f32(x[e >> 1]) : bf16lo_to_f32(x[e >> 1]);
    bool odd[8];  // infinities and NaN, which the bounds below would turn into 448
#pragma unroll
    for (int e = 0; e < 8; ++e) odd[e] = !__builtin_isfinite(y[e]);
    if (inverse != 0.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= inverse;
    } else if (near != 0.f) {
      // Markstein's division: with near = 1 / scale rounded and q within a unit of the quotient, what q
      // leaves over, times near, corrects q to the rounded quotient (the 22 MB of 7 thousand tokens of 4
      // heads of dim 128 in 9.5 us instead of 11.8)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = fminf(fmaxf(y[e] * near, -512.f), 512.f);
        // (the sign again: the correction of -0 is +0)
        y[e] = __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, scale, y[e]), near, q), y[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] / scale;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = odd[e] ? __builtin_nanf("") : fminf(fmaxf(y[e], -448.f), 448.f);
    u32x2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
      r[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w, true);
    }
    *reinterpret_cast<u32x2*>(to + 8 * part) = r;
  } else {
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max2(m, __builtin_bit_cast(u16x2, x[i] & 0x7FFF7FFFu));
    const unsigned top = block_max(max((unsigned)m[0], (unsigned)m[1]));  // bf16 bits of max |x|
    // division is monotonic: the quotient of the largest is the largest quotient
    const float q = fminf(quotient(__uint_as_float(top << 16), scale, inverse), 3.402823466e38f);
    // the exponent of q, one more where its fraction is above 1.75, two less
    int byte = (int)((__float_as_uint(q) + 0x1FFFFFu) >> 23) - 2;
    byte = min(max(byte, 2), 252);
    const float step = __uint_as_float((unsigned)byte << 23);
    unsigned r = 0;
    if (top < 0x7F80u) {
      auto lo = [&](int i) { return quotient(bf16lo_to_f32(x[i]), scale, inverse); };
      auto hi = [&](int i) { return quotient(bf16hi_to_f32(x[i]), scale, inverse); };
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, lo(0), hi(0), step, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, lo(1), hi(1), step, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, lo(2), hi(2), step, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, lo(3), hi(3), step, 3);
    } else {
      byte = 255;
    }
    *reinterpret_cast<unsigned*>(to + 4 * part) = r;
    if ((part & 3) == 0) blocks[part >> 2] = (unsigned char)byte;
  }
}

// what 8 values of a row are read as: the stored bytes, and with 4 bits the block's scale byte
struct Stored {
  u32x4 r;
  unsigned byte;
};
template <int KV>
__device__ __forceinline__ Stored load8(const unsigned char* from, const unsigned char* blocks, int part) {
  Stored s{};
  if constexpr (KV == BITDELTA_KV_BF16) {
    s.r = *reinterpret_cast<const u32x4*>(from + 16 * part);
  } else if constexpr (KV == BITDELTA_KV_FP8) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(from + 8 * part);
    s.r[0] = x[0];
    s.r[1] = x[1];
  } else {
    s.r[0] = *reinterpret_cast<const unsigned*>(from + 4 * part);
    s.byte = blocks[part >> 2];
  }
  return s;
}
template <int KV>
__device__ __forceinline__ u32x4 values8(const Stored& s, float scale) {
  u32x4 r;
  if constexpr (KV == BITDELTA_KV_BF16) {
    r = s.r;
  } else if constexpr (KV == BITDELTA_KV_FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = i & 1 ? __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(s.r[i >> 1], 1.0f, true))
                   : __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(s.r[i >> 1], 1.0f, false));
  } else {
    const float step = __uint_as_float(s.byte << 23);
    r[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.r[0], step, 0));
    r[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.r[0], step, 1));
    r[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.r[0], step, 2));
    r[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.r[0], step, 3));
  }
  if (scale != 1.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16(bf16lo_to_f32(r[i]) * scale, bf16hi_to_f32(r[i]) * scale);
  }
  return r;
}

// One workgroup takes `per` tokens at a time.  A token's rows are 2 * kv_heads * D / 8 units of 8 values, its
// key rows, then its value rows.  A thread keeps its unit and goes over the tokens, or, where a token has
// fewer units than the workgroup has threads, over every `groups`-th token; so what a unit's place within a
// token costs is paid once.
template <int D, int KV, bool WRITE>
__global__ __launch_bounds__(kThreads) void cache_kernel(const CacheArgs a, int per) {
  constexpr int kUnits = D / 8;
  __shared__ int offsets[kAttendMaxSeqs + 1];
  __shared__ TokenPlace places[kMaxTokens];
  const int tid = threadIdx.x;
  if (a.q_offsets) {
    for (int i = tid; i <= a.batch; i += kThreads) offsets[i] = a.q_offsets[i];
    __syncthreads();
  }
  const int units = 2 * a.kv_heads * kUnits;
  const int groups = units < kThreads ? kThreads / units : 1;
  const int group = groups > 1 ? tid / units : 0, first = tid - group * units;
  const int64_t stride = (int64_t)gridDim.x * per;
  for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < a.tokens; t0 += stride) {
    const int n = a.tokens - t0 < per ? (int)(a.tokens - t0) : per;
    int u = first, tok = group, part;
    bool v;
    unsigned char *pages, *blocks;
    int64_t head, row_step;
    uint16_t* row;  // of token tok
    auto unit = [&] {
      const int r = u / kUnits;
      part = u & (kUnits - 1);
      v = r >= a.kv_heads;
      const int h = v ? r - a.kv_heads : r;
      pages = const_cast<unsigned char*>(v ? a.cache.v : a.cache.k);
      blocks = const_cast<unsigned char*>(v ? a.cache.v_blocks : a.cache.k_blocks);
      head = (int64_t)h * (v ? a.cache.v_head : a.cache.k_head);
      row_step = v ? a.row_token[1] : a.row_token[0];
      row = (v ? a.rows[1] : a.rows[0]) + (int64_t)h * (v ? a.row_head[1] : a.row_head[0]) + 8 * part +
            (t0 + tok) * row_step;
    };
    // the token of load i; no branches around loads: one under a condition would wait for those before it
    auto token = [&](int i) { return tok + i * groups < n ? tok + i * groups : n - 1; };
    u32x4 x[kAhead];
    auto load_rows = [&] {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) x[i] = *reinterpret_cast<const u32x4*>(row + (token(i) - tok) * row_step);
    };
    bool more = group < groups && u < units && tok < n;
    if (more) {
      unit();
      if constexpr (WRITE) load_rows();  // on their way while the tokens are looked up
    }
    if (tid < n) places[tid] = token_place(a, offsets, (int)t0 + tid);
    __syncthreads();
    while (more) {
      const float scale = v ? a.scale[1] : a.scale[0], inverse = v ? a.inverse[1] : a.inverse[0];
      const float near = v ? a.near[1] : a.near[0];
      int64_t o[kAhead];
      bool live[kAhead], placed[kAhead];
      Stored s[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const TokenPlace p = places[token(i)];
        o[i] = (v ? p.v : p.k) + head;
        placed[i] = p.placed;
        live[i] = tok + i * groups < n && (WRITE ? p.placed : p.row);
        if constexpr (!WRITE) s[i] = load8<KV>(pages + o[i], blocks + (o[i] >> 4), part);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (!live[i]) continue;
        if constexpr (WRITE)
          store8<KV>(x[i], pages + o[i], blocks + (o[i] >> 4), part, scale, inverse, near);
        else  // (not to be kept in the caches: 14 prompts of up to 8192 tokens, 363 MB, 58 us instead of 79)
          __builtin_nontemporal_store(placed[i] ? values8<KV>(s[i], scale) : u32x4{0, 0, 0, 0},
                                      reinterpret_cast<u32x4*>(row + i * groups * row_step));
      }
      tok += kAhead * groups;
      row += kAhead * groups * row_step;
      if (tok >= n) {
        tok = group;
        u += kThreads;
        if (u >= units) break;
        unit();
      }
      if constexpr (WRITE) load_rows();
    }
    __syncthreads();  // the places are read
  }
}

template <int D, int KV, bool WRITE>
hipError_t launch(const CacheArgs& a, hipStream_t stream) {
  // about 8 units a thread, fewer where that would leave compute units without a workgroup
  int64_t per = 2048 / ((int64_t)a.kv_heads * (D / 4));
  if (per > a.tokens / 512) per = a.tokens / 512;
  per = per < 1 ? 1 : (per > kMaxTokens ? kMaxTokens : per);
  int64_t blocks = (a.tokens + per - 1) / per;
  if (blocks > (1 << 20)) blocks = 1 << 20;  // a launch holds fewer than 2^32 threads
  clear_stale_error();
  hipLaunchKernelGGL((cache_kernel<D, KV, WRITE>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a,
                     (int)per);
  return hipGetLastError();
}

template <bool WRITE>
hipError_t launch_for(const CacheArgs& a, int dim, int dtype, hipStream_t stream) {
  if (dim != 64 && dim != 128) return hipErrorInvalidValue;
  if (dtype == BITDELTA_KV_BF16)
    return dim == 64 ? launch<64, BITDELTA_KV_BF16, WRITE>(a, stream)
                     : launch<128, BITDELTA_KV_BF16, WRITE>(a, stream);
  if (dtype == BITDELTA_KV_FP8)
    return dim == 64 ? launch<64, BITDELTA_KV_FP8, WRITE>(a, stream)
                     : launch<128, BITDELTA_KV_FP8, WRITE>(a, stream);
  if (dtype == BITDELTA_KV_FP4)
    return dim == 64 ? launch<64, BITDELTA_KV_FP4, WRITE>(a, stream)
                     : launch<128, BITDELTA_KV_FP4, WRITE>(a, stream);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_cache_write(const CacheArgs& a, int dim, int dtype, hipStream_t stream) {
  return launch_for<true>(a, dim, dtype, stream);
}
hipError_t launch_cache_read(const CacheArgs& a, int dim, int dtype, hipStream_t stream) {
  return launch_for<false>(a, dim, dtype, stream);
}

}  // namespace bd
