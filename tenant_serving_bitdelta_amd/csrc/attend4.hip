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

}  // namespace

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
