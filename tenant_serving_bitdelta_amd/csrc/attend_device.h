// Device code that the attention kernels share (attend.hip: bf16 and e4m3 caches, attend4.hip: 4 bits):
// lane moves, conversions, LDS layouts, copies into LDS, key lists, sums over the units of a launch.
#pragma once

#include "attend.h"
#include "bd_internal.h"

namespace bd {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kNegInf = -__builtin_inff();
constexpr float kLn2 = 0.6931471805599453f;
// Output sums are rescaled only when a row's maximum grows by more than this many powers of two:
// weights then stay below 2^8, far from fp32 overflow, and their bf16 rounding is relative.
constexpr float kRescale = 8.0f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// max over the two halves of a wave, in every lane
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// the same over the lanes l, l ^ 16
__device__ __forceinline__ float row_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float row_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  f32x2 f;
  f[0] = a;
  f[1] = b;
  return __builtin_bit_cast(unsigned, __builtin_convertvector(f, bf16x2));
}

// 4 e4m3 values -> 4 bf16, exact
__device__ __forceinline__ u32x2 fp8x4_to_bf16(unsigned v) {
  u32x2 r;
  r[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
  r[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true));
  return r;
}
__device__ __forceinline__ u32x4 fp8x8_to_bf16(unsigned a, unsigned b) {
  const u32x2 x = fp8x4_to_bf16(a), y = fp8x4_to_bf16(b);
  return u32x4{x[0], x[1], y[0], y[1]};
}

// Clears the bf16 (e4m3) values of v that are infinite or NaN; true if there were any.
template <bool FP8>
__device__ __forceinline__ bool clear_odd(u32x4* v) {
  unsigned any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned x = (*v)[i];
    unsigned m = 0;
    if constexpr (FP8) {  // e4m3 has no infinity; NaN is all ones below the sign
#pragma unroll
      for (int b = 0; b < 32; b += 8) m |= ((x >> b) & 0x7Fu) == 0x7Fu ? 0xFFu << b : 0u;
    } else {
      m = ((x & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
    }
    (*v)[i] = x & ~m;
    any |= m;
  }
  return any != 0;
}
// Element d of a value row as fp32, if it is infinite or NaN, else 0.
template <bool FP8>
__device__ __forceinline__ float odd_value(const unsigned char* row, int d) {
  if constexpr (FP8) return (row[d] & 0x7F) == 0x7F ? __builtin_nanf("") : 0.f;
  const unsigned x = reinterpret_cast<const uint16_t*>(row)[d];
  return (x & 0x7F80u) == 0x7F80u ? __uint_as_float(x << 16) : 0.f;
}
// Where the value row of key vp sits, or null when it has none.
__device__ __forceinline__ const unsigned char* value_row(const PagedCache& c, const KeyList& kl, int vp,
                                                          int h) {
  const int kp = key_position(kl, vp);
  const int page = page_quotient(kp, c.div);
  const int at = key_table_index(kl, vp, page);
  if (at < 0) return nullptr;
  const int id = page_id_checked((vp < kl.na ? kl.ta : kl.tb)[at], c.num_pages);
  if (id < 0) return nullptr;
  return c.v + page_row_bytes(id, kp - page * c.page_size, c.v_page, c.v_token) + (int64_t)h * c.v_head;
}

__device__ __forceinline__ u32x2 lds_read_tr(const unsigned char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (lds_s16x4*)(const_cast<unsigned char*>(p))));
}

// Copies straight from memory into LDS: 16 (4) bytes per lane, lane l's to the LDS address
// `to` + 16 l (4 l), the same `to` for the wave.  In assembly because the compiler, which knows what
// the builtin does, puts a wait for all copies before every transposed LDS read; here each step waits
// for its own (wait_copies).  The instruction has no result register, and its address is read as it issues.
__device__ __forceinline__ unsigned lds_address(const void* p) {
  return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void copy16(const unsigned char* from, unsigned to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(to)
               : "memory", "m0");
}
__device__ __forceinline__ void copy4(const int32_t* from, unsigned to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "s"(to)
               : "memory", "m0");
}
// until at most n of the wave's memory operations, the newest, are not done
template <int n>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}
// The workgroup meets, its LDS accesses done; copies into LDS may still be on their way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Byte offset of 16-byte unit u of row r in a V tile (D bf16 a row).  A transposed read takes 32
// bytes of each of 8 consecutive rows at a time; the XOR spreads those over all banks.
template <int D>
__device__ __forceinline__ unsigned v_unit(int r, int u) {
  const int x = D == 128 ? 2 * (r & 7) : 2 * ((r >> 1) & 3);
  return (unsigned)(r * (D * 2) + ((u ^ x) << 4));
}
// The same for a K tile, whose reads take one 16-byte unit of 16 consecutive rows at a time.
template <int D>
__device__ __forceinline__ unsigned k_unit(int r, int u) {
  const int x = D == 128 ? (r & 15) : ((r >> 1) & 7);
  return (unsigned)(r * (D * 2) + ((u ^ x) << 4));
}

__device__ __forceinline__ int clamp_len(int len, int width, int page_size) {
  const int64_t cap = (int64_t)width * page_size;
  return len < 0 ? 0 : (len > cap ? (int)cap : len);
}

// Does the token at position pos see key vp of its list?  In vp, the list's second part ends at
// pos + (na - lo) for this token and begins a window before; the first tokens are the vp below
// min(sinks, pos + 1) (when lo < sinks the list has no gap, else the token sees all na of them).
// Sight holds both relative to a vp, so that a tile's keys are constants beyond it: one subtraction
// and one comparison per bound, no branches.
struct Sight {
  int end, first;
  __device__ __forceinline__ bool sees(int k, int window) const {
    return ((unsigned)(end - k) < (unsigned)window) | (k < first);
  }
};
__device__ __forceinline__ Sight sight(const KeyList& l, int pos, int sinks, int vp) {
  return Sight{pos + (l.na - l.lo) - vp, min(sinks, pos + 1) - vp};
}
__device__ __forceinline__ bool sees(const KeyList& l, int pos, int window, int sinks, int vp) {
  return sight(l, pos, sinks, vp).sees(0, window);
}

// What one unit (sequence, kv head) of the row kernel reads and for which query rows.
struct RowUnit {
  KeyList keys;
  int t0, nq;   // first token row of q, tokens
  int p0;       // position of the first token (window op)
};
__device__ __forceinline__ RowUnit row_unit(const AttendArgs& a, int b, int len) {
  RowUnit u;
  len = clamp_len(len, a.width, a.cache.page_size);
  const int32_t* row = a.table + (int64_t)b * a.width;
  if (a.nseg > 0) {
    u.t0 = b;
    u.nq = 1;
    u.p0 = 0;
    u.keys = KeyList{row, row, a.width, a.width, 0, 0, len};
    if (a.row_prefix) {
      int g = 0;
      while (g + 1 < a.nseg && a.seg_offsets[g + 1] <= b) ++g;
      const int plen = clamp_len(a.prefix_lens[g], a.pwidth, a.cache.page_size);
      u.keys.ta = a.prefix_table + (int64_t)g * a.pwidth;
      u.keys.wa = a.pwidth;
      u.keys.na = plen;
      // positions of both parts together stay below 2^31 (checked on the host)
      u.keys.n = plen + len;
    }
  } else {
    u.t0 = b;
    u.nq = 1;
    u.p0 = len - 1;
    if (a.q_offsets) {
      const ChunkRows c = chunk_rows(a.q_offsets[b], a.q_offsets[b + 1], len, a.max_q, a.tokens);
      u.t0 = c.first;
      u.nq = c.count;
      u.p0 = c.p0;
    }
    // keys up to the last token: a unit of one token has no masks
    const int end = u.p0 + u.nq;
    u.keys = window_keys(row, a.width, end < 0 ? 0 : end, u.p0, a.window, a.sinks);
  }
  return u;
}
__device__ __forceinline__ RowUnit row_unit(const AttendArgs& a, int b) {
  return row_unit(a, b, a.lens[b]);
}
__device__ __forceinline__ int row_steps(const RowUnit& u) {
  return u.nq > 0 ? (u.keys.n + kRowStep - 1) / kRowStep : 0;
}

// Running sums of `count` values (value(i) >= 0) into scan[0 .. count] in LDS, by all threads of
// the workgroup; scan[0] = 0.
template <int kThreads, class F>
__device__ void block_scan(int* scan, int* wave_sum, int count, F value) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) scan[0] = 0;
  int carry = 0;
  for (int base = 0; base < count; base += kThreads) {
    const int i = base + tid;
    int x = i < count ? value(i) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(x, d, 64);
      if (lane >= d) x += y;
    }
    if (lane == 63) wave_sum[wave] = x;
    __syncthreads();
    int before = carry, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) before += wave_sum[w];
      total += wave_sum[w];
    }
    if (i < count) scan[i + 1] = before + x;
    carry += total;
    __syncthreads();
  }
}
// largest i with scan[i] <= x, for 0 <= x < scan[count]
__device__ __forceinline__ int scan_find(const int* scan, int count, int x) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (scan[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// segments whose rows fit half a tile: their units take two 64-key tiles a step
__device__ __forceinline__ bool halved(const AttendArgs& a, int sg) {
  return a.halves && (a.seg_offsets[sg + 1] - a.seg_offsets[sg]) * a.group <= kTileRows / 2;
}
__device__ __forceinline__ int prefix_steps(const AttendArgs& a, int sg) {
  const int len = clamp_len(a.prefix_lens[sg], a.pwidth, a.cache.page_size);
  const int keys = halved(a, sg) ? 2 * kTileKeys : kTileKeys;
  return (len + keys - 1) / keys;
}

}  // namespace
}  // namespace bd
