// Sampling the next token of each row from given uniform numbers.
//
// Mathematics.  A row's tokens are ordered by descending logit, ties by ascending index; token j
// of that order weighs w_j = exp((l_j - l_0) / T).  Top-k, top-p and min-p each keep a prefix of
// the order: the first k; the shortest prefix whose weight reaches p times the weight of the first
// k; those with w_j >= min_p.  With n the shortest of the three (at least 1), the token drawn is
// the first whose running sum of weights exceeds u times the sum of the first n.
//
// Only a prefix of the order is ever needed.  A workgroup reads its row once and keeps, per
// thread, the largest value of each of 8 stretches.  The k-th largest of the threads' maxima is a
// bound that at least k tokens reach and few more do: the stretches whose maximum reaches it are
// read again and the tokens at or above it collected, ranked by counting, weighed and summed.
// Weights and sums are fp64, so that a draw next to a border between two tokens falls on the side
// where the definition puts it.  When the answer lies outside the collected tokens (a flat
// distribution and no top-k), the borders are found by bisection over (logit, index), one pass
// over the row per step.
#include <limits.h>

#include "bd_internal.h"
#include "sample.h"

namespace bd {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kSegments = 8;    // stretches of a thread's part of the row
constexpr int kCap = 2048;      // collected tokens at most
constexpr int kMaxK = 1024;     // top-k up to this goes by the threads' maxima (one per thread)
constexpr int kGuess = 256;     // tokens to collect when no top-k says how many

constexpr float kNegInf = -__builtin_inff();

// Order-preserving map of floats to unsigned; -0 and +0 are one value, NaN counts as -inf.
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.0f : kNegInf; }
__device__ __forceinline__ unsigned to_key(float x) {
  const unsigned b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_key(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

template <bool F32>
struct Row {
  static constexpr int kE = F32 ? 4 : 8;  // elements of a 16-byte vector
  const unsigned char* p;                 // first element
  int vocab;
  int head, nv, extra;  // elements before the first aligned vector, vectors, head + tail elements

  __device__ __forceinline__ Row(const SampleArgs& a, int row) {
    p = static_cast<const unsigned char*>(a.logits) + (int64_t)row * a.row_stride * (F32 ? 4 : 2);
    vocab = a.vocab;
    const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    head = min(vocab, mis ? (16 - mis) / (F32 ? 4 : 2) : 0);
    nv = (vocab - head) / kE;
    extra = vocab - nv * kE;
  }
  __device__ __forceinline__ int extra_index(int i) const { return i < head ? i : nv * kE + i; }
  __device__ __forceinline__ float one(int i) const {
    if constexpr (F32) return clean(reinterpret_cast<const float*>(p)[i]);
    return clean(__uint_as_float((unsigned)reinterpret_cast<const uint16_t*>(p)[i] << 16));
  }
  __device__ __forceinline__ u32x4 raw(int v) const {
    return *reinterpret_cast<const u32x4*>(p + (int64_t)head * (F32 ? 4 : 2) + (int64_t)v * 16);
  }
  __device__ __forceinline__ static float part(const u32x4& r, int e) {
    if constexpr (F32) return clean(__uint_as_float(r[e]));
    const unsigned x = r[e >> 1];
    return clean((e & 1) ? bf16hi_to_f32(x) : bf16lo_to_f32(x));
  }
};

// ln w and w; the largest logit weighs 1, also where it is infinite
__device__ __forceinline__ double log_weight(float l, float top, double inv_t) {
  return l == top ? 0.0 : ((double)l - (double)top) * inv_t;
}
__device__ __forceinline__ double weight(float l, float top, double inv_t) {
  return l == kNegInf ? 0.0 : exp(log_weight(l, top, inv_t));
}

__device__ __forceinline__ uint64_t composite(float l, int idx) {
  return ((uint64_t)to_key(l) << 32) | (0xFFFFFFFFu - (unsigned)idx);
}

__device__ __forceinline__ double shfl_xor_f64(double x, int d) { return __shfl_xor(x, d, 64); }

struct Shared {
  union {
    uint64_t cand[kCap];
    unsigned maxima[kThreads];
  };
  uint64_t sorted[kCap];
  double cum[kCap];
  double wave_d[kWaves];
  uint64_t wave_u[kWaves];
  float wave_f[kWaves];
  int wave_i[kWaves];
  int count;
  int best;
};

__device__ double block_sum(Shared& sh, double x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += shfl_xor_f64(x, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.wave_d[threadIdx.x >> 6] = x;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) t += sh.wave_d[w];
  return t;
}
__device__ int block_count(Shared& sh, int x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.wave_i[threadIdx.x >> 6] = x;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) t += sh.wave_i[w];
  return t;
}
__device__ float block_max(Shared& sh, float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.wave_f[threadIdx.x >> 6] = x;
  __syncthreads();
  float t = kNegInf;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) t = fmaxf(t, sh.wave_f[w]);
  return t;
}

// Count and weight of the row's tokens at or above a composite.
template <bool F32>
__device__ void above(Shared& sh, const Row<F32>& row, uint64_t c, float top, double inv_t,
                      int* count, double* mass) {
  int n = 0;
  double s = 0;
  auto one = [&](float l, int idx) {
    if (composite(l, idx) >= c) {
      ++n;
      s += weight(l, top, inv_t);
    }
  };
  for (int v = threadIdx.x; v < row.nv; v += kThreads) {
    const u32x4 r = row.raw(v);
#pragma unroll
    for (int e = 0; e < Row<F32>::kE; ++e) one(row.part(r, e), row.head + v * Row<F32>::kE + e);
  }
  if ((int)threadIdx.x < row.extra) {
    const int idx = row.extra_index(threadIdx.x);
    one(row.one(idx), idx);
  }
  *count = block_count(sh, n);
  *mass = block_sum(sh, s);
}

// The largest composite c for which reached(count above c, weight above c) holds; it does for 0.
template <bool F32, class Reached>
__device__ uint64_t bisect(Shared& sh, const Row<F32>& row, float top, double inv_t, Reached reached) {
  uint64_t lo = 0, hi = ((uint64_t)to_key(top) << 32) | 0xFFFFFFFFull;
  while (lo < hi) {
    const uint64_t mid = lo + (hi - lo) / 2 + 1;
    int n;
    double s;
    above<F32>(sh, row, mid, top, inv_t, &n, &s);
    if (reached(n, s)) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a) {
  __shared__ Shared sh;
  constexpr int kE = Row<F32>::kE;
  const int tid = threadIdx.x, lane = tid & 63;
  const int b = blockIdx.x;
  const Row<F32> row(a, b);
  const int vocab = a.vocab;

  const float temp = a.temperature ? a.temperature[b] : 1.0f;
  int k = a.top_k ? a.top_k[b] : 0;
  if (k <= 0 || k > vocab) k = vocab;
  const float pf = a.top_p ? a.top_p[b] : 1.0f;
  const double p = pf < 1.0f ? (double)pf : 2.0;   // 2: off (NaN too)
  const float mf = a.min_p ? a.min_p[b] : 0.0f;
  const double minp = mf > 0.0f ? (double)mf : 0.0;
  const float uf = a.u[b];
  const double u = uf > 0.0f ? (double)uf : 0.0;
  // one token is kept whatever the others weigh
  const bool greedy = !(temp > 0.0f) || k == 1 || p <= 0.0 || minp > 1.0;
  const double inv_t = greedy ? 1.0 : 1.0 / (double)temp;
  const bool known_k = k <= kMaxK;
  const bool need_z = !greedy && !known_k && (p < 1.0 || minp == 0.0);

  // ---- one pass: maxima of stretches, and the row's weight where the filters need it
  float seg[kSegments], mt = kNegInf;
  double st = 0;
  const int iters = (row.nv + kThreads - 1) / kThreads;
  const int seglen = (iters + kSegments - 1) / kSegments;
#pragma unroll
  for (int s = 0; s < kSegments; ++s) {
    float sm = kNegInf;
    const int end = min((s + 1) * seglen, iters);
    for (int i = s * seglen; i < end; i += 4) {
      u32x4 r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = row.raw(min(tid + (i + q) * kThreads, row.nv - 1));
      float vm = kNegInf;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool in = i + q < end && tid + (i + q) * kThreads < row.nv;
        float m4 = kNegInf;
#pragma unroll
        for (int e = 0; e < kE; ++e) m4 = fmaxf(m4, row.part(r[q], e));
        vm = fmaxf(vm, in ? m4 : kNegInf);
      }
      sm = fmaxf(sm, vm);
      if (need_z) {
        if (vm > mt) {
          st *= weight(mt, vm, inv_t);
          mt = vm;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (i + q < end && tid + (i + q) * kThreads < row.nv)
#pragma unroll
            for (int e = 0; e < kE; ++e) {
              const float l = row.part(r[q], e);
              if (l > kNegInf) st += weight(l, mt, inv_t);
            }
      }
    }
    seg[s] = sm;
  }
  const int ei = tid < row.extra ? row.extra_index(tid) : 0;
  const float ev = tid < row.extra ? row.one(ei) : kNegInf;
  if (need_z && ev > kNegInf) {
    if (ev > mt) {
      st *= weight(mt, ev, inv_t);
      mt = ev;
    }
    st += weight(ev, mt, inv_t);
  }
  float mine = ev;
#pragma unroll
  for (int s = 0; s < kSegments; ++s) mine = fmaxf(mine, seg[s]);
  if (tid == 0) {
    sh.count = 0;
    sh.best = vocab;
  }
  const float top = block_max(sh, mine);
  if (top == kNegInf) {  // every token is masked
    if (tid == 0) {
      a.tokens[b] = -1;
      if (a.logprob) a.logprob[b] = kNegInf;
    }
    return;
  }
  double z = 0;
  if (need_z) z = block_sum(sh, mt == kNegInf ? 0.0 : st * weight(mt, top, inv_t));

  // ---- the bound: at least `want` tokens reach it
  float tau;
  bool all_min_p = false;  // the collected tokens include every one with w >= min_p
  if (greedy) {
    tau = top;
  } else {
    const int want = known_k ? k : min(kGuess, vocab);
    __syncthreads();
    sh.maxima[tid] = to_key(mine);
    __syncthreads();
    // every wave bisects the keys on its own, 16 a lane
    unsigned key[kThreads / 64];
    unsigned lo = 0, hi = to_key(top);
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) key[i] = sh.maxima[lane + 64 * i];
    while (lo < hi) {
      const unsigned mid = lo + (hi - lo) / 2 + 1;
      int n = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 64; ++i) n += __popcll(__ballot(key[i] >= mid));
      if (n >= want) lo = mid;
      else hi = mid - 1;
      if (n >= want && n <= want + (want >> 3)) break;
    }
    // fewer maxima than wanted (a short row, or masked tokens): every token
    tau = lo <= to_key(kNegInf) ? kNegInf : from_key(lo);
    if (!known_k && minp > 0.0) {
      // every token that min_p keeps (and a margin for the rounding of this bound)
      const float t2 = (float)((double)top + log(minp) / inv_t);
      tau = t2 - fabsf(t2) * 1e-5f - 1e-30f;
      all_min_p = true;
    }
    __syncthreads();
  }

  // ---- collect the tokens at or above the bound
  auto collect = [&](float l, int idx) {
    if (l >= tau) {
      if (greedy) {
        atomicMin(&sh.best, idx);
      } else {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kCap) sh.cand[at] = composite(l, idx);
      }
    }
  };
#pragma unroll
  for (int s = 0; s < kSegments; ++s) {
    if (seg[s] >= tau && seg[s] > kNegInf) {
      const int end = min((s + 1) * seglen, iters);
      for (int i = s * seglen; i < end; ++i) {
        const int v = tid + i * kThreads;
        if (v < row.nv) {
          const u32x4 r = row.raw(v);
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const float l = row.part(r, e);
            if (l > kNegInf) collect(l, row.head + v * kE + e);
          }
        }
      }
    }
  }
  if (ev > kNegInf) collect(ev, ei);
  __syncthreads();
  if (greedy) {
    if (tid == 0) {
      a.tokens[b] = sh.best;
      if (a.logprob) a.logprob[b] = 0.0f;
    }
    return;
  }
  const int n = sh.count;
  bool solved = false;
  if (n <= kCap) {
    // ---- order by counting the greater ones
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t c = sh.cand[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += sh.cand[j] > c;
      sh.sorted[rank] = c;
    }
    __syncthreads();
    // ---- weights and their running sums: thread t holds tokens 2t and 2t + 1
    double w0 = 0, w1 = 0;
    if (2 * tid < n) w0 = weight(from_key((unsigned)(sh.sorted[2 * tid] >> 32)), top, inv_t);
    if (2 * tid + 1 < n) w1 = weight(from_key((unsigned)(sh.sorted[2 * tid + 1] >> 32)), top, inv_t);
    double x = w0 + w1;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double y = __shfl_up(x, d, 64);
      if (lane >= d) x += y;
    }
    if (lane == 63) sh.wave_d[tid >> 6] = x;
    __syncthreads();
    double before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (w < (tid >> 6)) before += sh.wave_d[w];
    const double c1 = before + x, c0 = c1 - w1;
    sh.cum[2 * tid] = c0;
    sh.cum[2 * tid + 1] = c1;
    __syncthreads();
    // everything collected, or the tokens beyond weigh nothing (they are masked)?
    const bool complete = tau == kNegInf;
    const int full = complete ? n : vocab;      // tokens of the order that count
    const int kk = min(k, full);
    // shortest of the prefixes; one that ends beyond the collected tokens only counts as "beyond"
    bool ok = true;
    int keep = kk;
    if (p < 1.0) {
      // the weight of the first k: collected, or the row's when k is off
      ok = kk <= n || k == vocab;
      const double t = p * (kk <= n ? sh.cum[kk - 1] : z);
      const int lim = min(kk, n);
      const int np = block_count(sh, (2 * tid < lim && c0 < t) + (2 * tid + 1 < lim && c1 < t));
      keep = np < lim ? np + 1 : (kk <= n ? kk : INT_MAX);
    }
    if (minp > 0.0) {
      const int nm = block_count(sh, (2 * tid < n && w0 >= minp) + (2 * tid + 1 < n && w1 >= minp));
      if (nm < n || complete || all_min_p) keep = min(keep, nm);
      else if (keep > n) keep = INT_MAX;
    }
    keep = max(keep, 1);
    if (keep > n && (keep != vocab || p < 1.0 || minp > 0.0)) ok = false;
    if (ok) {
      const double zn = keep <= n ? sh.cum[keep - 1] : z;
      const double t = u * zn;
      const int lim = min(keep, n);
      int j = block_count(sh, (2 * tid < lim && c0 <= t) + (2 * tid + 1 < lim && c1 <= t));
      if (j < lim || keep <= n) {
        j = min(j, keep - 1);
        solved = true;
        if (tid == 0) {
          const uint64_t c = sh.sorted[j];
          a.tokens[b] = (int)(0xFFFFFFFFu - (unsigned)c);
          if (a.logprob) {
            a.logprob[b] = (float)(log_weight(from_key((unsigned)(c >> 32)), top, inv_t) - log(zn));
          }
        }
      }
    }
  }
  if (solved) return;

  // ---- outside the collected tokens: borders by bisection over the whole row
  uint64_t border = 0;
  if (k < vocab)
    border = bisect<F32>(sh, row, top, inv_t, [&](int c, double) { return c >= k; });
  if (p < 1.0) {
    int c;
    double zk;
    above<F32>(sh, row, border, top, inv_t, &c, &zk);
    const uint64_t bp = bisect<F32>(sh, row, top, inv_t, [&](int, double s) { return s >= p * zk; });
    border = max(border, bp);
  }
  if (minp > 0.0) {
    unsigned lo = 0, hi = to_key(top);  // the smallest key with w >= min_p
    while (lo < hi) {
      const unsigned mid = lo + (hi - lo) / 2;
      if (weight(clean(from_key(mid)), top, inv_t) >= minp) hi = mid;
      else lo = mid + 1;
    }
    border = max(border, (uint64_t)lo << 32);
  }
  int c;
  double zn;
  above<F32>(sh, row, border, top, inv_t, &c, &zn);
  uint64_t hit = bisect<F32>(sh, row, top, inv_t, [&](int, double s) { return s > u * zn; });
  if (hit < border || hit == 0) {
    // u * zn rounded up to zn: the last token kept that weighs something
    hit = bisect<F32>(sh, row, top, inv_t, [&](int, double s) { return s >= zn; });
  }
  if (tid == 0) {
    a.tokens[b] = (int)(0xFFFFFFFFu - (unsigned)hit);
    if (a.logprob) {
      a.logprob[b] = (float)(log_weight(from_key((unsigned)(hit >> 32)), top, inv_t) - log(zn));
    }
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, bool f32, hipStream_t stream) {
  if (a.rows < 1 || a.vocab < 1) return hipErrorInvalidValue;
  clear_stale_error();
  if (f32) hipLaunchKernelGGL(sample_kernel<true>, dim3(a.rows), dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL(sample_kernel<false>, dim3(a.rows), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace bd
