// Sampling the next token of each row from given uniform numbers.
//
// Mathematics.  A row's tokens are ordered by descending logit, ties by ascending index; token j
// of that order weighs w_j = exp((l_j - l_0) / T).  Top-k, top-p and min-p each keep a prefix of
// the order: the first k; the shortest prefix whose weight reaches p times the weight of the first
// k; those with w_j >= min_p.  With n the shortest of the three (at least 1), the token drawn is
// the first whose running sum of weights exceeds u times the sum of the first n.
//
// Only a prefix of the order is ever needed.  A workgroup reads its row once and keeps, per
// thread, the largest value of each of 8 parts.  The k-th largest of the threads' maxima is a
// bound that at least k tokens reach and few more do: the parts whose maximum reaches it are read
// again and the tokens at or above it collected, ordered, weighed and summed.  Weights and sums
// are fp64, so that a draw next to a border between two tokens falls on the side where the
// definition puts it.
//
// When the answer lies outside the collected tokens (a flat distribution and no top-k), a second
// reading counts and weighs the tokens in bins of 1/128 in (l_0 - l) / T, which confines each
// border (top-k, top-p, min-p, the draw) to a bin or few; a third reading collects the tokens of
// those bins, and the borders are resolved as before.  Where even that collects
// too many (thousands of equal logits), the borders are found by bisection over (logit, index), one
// reading per step.
#include <limits.h>

#include "bd_internal.h"
#include "sample.h"

namespace bd {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kParts = 8;       // a thread's vectors i, i + 8, ... make its part i
constexpr int kCap = 4096;      // collected tokens at most
constexpr int kBins = 4096;     // of 1/kBinScale each in (l_0 - l) / T; the last takes the rest
constexpr int kBinScale = 128;
constexpr int kMaxK = 1024;     // top-k up to this goes by the threads' maxima (one per thread)
constexpr int kGuess = 128;     // tokens to collect when no top-k says how many
constexpr int kFewK = 128;      // up to this many go by one maximum per thread, more by kParts

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
// e^x for x <= 0 in fp64: x = n ln 2 + r with |r| <= ln 2 / 2, and the Taylor series of e^r to
// r^12 (the next term is below 2e-16).  About 20 fp64 instructions.
__device__ __forceinline__ double exp_f64(double x) {
  x = fmax(x, -745.0);
  const double n = __builtin_rint(x * 1.4426950408889634074);
  double r = __builtin_fma(n, -0.693147180369123816490, x);  // ln 2 in two parts, the first short
  r = __builtin_fma(n, -1.90821492927058770002e-10, r);
  double e = 1.0 / 479001600.0;
  e = __builtin_fma(e, r, 1.0 / 39916800.0);
  e = __builtin_fma(e, r, 1.0 / 3628800.0);
  e = __builtin_fma(e, r, 1.0 / 362880.0);
  e = __builtin_fma(e, r, 1.0 / 40320.0);
  e = __builtin_fma(e, r, 1.0 / 5040.0);
  e = __builtin_fma(e, r, 1.0 / 720.0);
  e = __builtin_fma(e, r, 1.0 / 120.0);
  e = __builtin_fma(e, r, 1.0 / 24.0);
  e = __builtin_fma(e, r, 1.0 / 6.0);
  e = __builtin_fma(e, r, 0.5);
  e = __builtin_fma(e, r, 1.0);
  e = __builtin_fma(e, r, 1.0);
  return __builtin_ldexp(e, (int)n);
}
__device__ __forceinline__ double weight(float l, float top, double inv_t) {
  return l == kNegInf ? 0.0 : exp_f64(log_weight(l, top, inv_t));
}
// Where a logit falls among the bins, in fp64 (bin = its whole part): never less for a smaller
// logit.  scale: kBinScale / T; what lies beyond the bins counts as the last one's lower end.
__device__ __forceinline__ double bin_place(float l, double top, double scale) {
  return fmin((top - (double)l) * scale, (double)(kBins - 1));
}

// One reading of the row by the workgroup, kParts vectors a thread in flight ahead of the ones that
// are worked on: each(vectors, i0) gets the vectors tid + (i0 + q) * kThreads, q < kParts (past the
// row's end: its last one); one(l, idx) the elements before and after the vectors.
template <bool F32, class Each, class One>
__device__ __forceinline__ void read_batches(const Row<F32>& row, Each each, One one) {
  const int tid = threadIdx.x;
  const int iters = (row.nv + kThreads - 1) / kThreads;
  u32x4 r[kParts], nx[kParts];
  auto fetch = [&](int i0, u32x4* v) {
#pragma unroll
    for (int q = 0; q < kParts; ++q) v[q] = row.raw(min(tid + (i0 + q) * kThreads, row.nv - 1));
  };
  if (iters > 0) fetch(0, r);
  if (tid < row.extra) {
    const int idx = row.extra_index(tid);
    one(row.one(idx), idx);
  }
  for (int i0 = 0; i0 < iters; i0 += kParts) {
    if (i0 + kParts < iters) fetch(i0 + kParts, nx);
    each(r, i0);
#pragma unroll
    for (int q = 0; q < kParts; ++q) r[q] = nx[q];
  }
}
// The same, element by element: one(l, idx).
template <bool F32, class One>
__device__ __forceinline__ void read_row(const Row<F32>& row, One one) {
  constexpr int kE = Row<F32>::kE;
  read_batches<F32>(
      row,
      [&](const u32x4* r, int i0) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          const int v = (int)threadIdx.x + (i0 + q) * kThreads;
          if (v < row.nv)
#pragma unroll
            for (int e = 0; e < kE; ++e) one(row.part(r[q], e), row.head + v * kE + e);
        }
      },
      one);
}

// Sums of e^((l - top) / T) over many tokens: with y the exponent in powers of two, y = n + r, |r| <= 1/2, and the series of 2^r to r^11 (the next term is below 1e-14).  n comes
// out of the low bits of y + 1.5 * 2^52.  Weights below 2^-1000 (0 among them) count as 2^-1000,
// which does not reach the sums.
struct Exp2 {
  double a, top;
  __device__ __forceinline__ Exp2(float l0, double inv_t) {
    a = inv_t * 1.4426950408889634074;
    top = l0;
  }
  __device__ __forceinline__ double operator()(float l) const {
    const double kMagic = 6755399441055744.0;
    const double y = fmax(((double)l - top) * a, -1000.0);
    const double t = y + kMagic;
    const double r = y - (t - kMagic);
    double e = 4.446e-10;                           // ln2^11 / 11! and so on
    e = __builtin_fma(e, r, 7.0549116208011233e-9);
    e = __builtin_fma(e, r, 1.0178086009239699e-7);
    e = __builtin_fma(e, r, 1.3215486790144309e-6);
    e = __builtin_fma(e, r, 1.5252733804059841e-5);
    e = __builtin_fma(e, r, 1.5403530393381610e-4);
    e = __builtin_fma(e, r, 1.3333558146428443e-3);
    e = __builtin_fma(e, r, 9.6181291076284772e-3);
    e = __builtin_fma(e, r, 5.5504108664821580e-2);
    e = __builtin_fma(e, r, 0.24022650695910071);
    e = __builtin_fma(e, r, 0.69314718055994531);
    e = __builtin_fma(e, r, 1.0);
    return __builtin_ldexp(e, (int)__double_as_longlong(t));
  }
};

__device__ __forceinline__ uint64_t composite(float l, int idx) {
  return ((uint64_t)to_key(l) << 32) | (0xFFFFFFFFu - (unsigned)idx);
}

__device__ __forceinline__ double shfl_xor_f64(double x, int d) { return __shfl_xor(x, d, 64); }

// A stretch of the order whose tokens are collected: bins lo .. hi (none: hi < 0), the count and
// weight of all tokens before it, and its tokens first .. first + size - 1 of the collected ones.
struct Interval {
  int lo, hi, count0, first, size;
  double mass0;
};

struct Shared {
  uint64_t cand[kCap];
  union {
    double cum[kCap];
    struct {
      unsigned long long mass[kBins];
      int bins[kBins];
    };
    uint16_t hits[kParts * kThreads];  // parts to read again: thread + kThreads * part
  };
  int rank[256];
  int wave_n[2][kWaves];
  float wave_g[kWaves];
  double wave_d[kWaves];
  float wave_f[kWaves];
  int wave_i[kWaves];
  Interval iv[4];
  int count, nhits;
  int best;
  int solved;
  int found[4];
  double found_d;
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
// the largest x, and the smallest in *least
__device__ float block_max(Shared& sh, float x, float* least) {
  float y = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    x = fmaxf(x, __shfl_xor(x, d, 64));
    y = fminf(y, __shfl_xor(y, d, 64));
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    sh.wave_f[threadIdx.x >> 6] = x;
    sh.wave_g[threadIdx.x >> 6] = y;
  }
  __syncthreads();
  float t = sh.wave_f[0], u = sh.wave_g[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    t = fmaxf(t, sh.wave_f[w]);
    u = fminf(u, sh.wave_g[w]);
  }
  *least = u;
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
  read_row<F32>(row, one);
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

// Sorts sh.cand[0 .. n) in descending order (all threads).  Up to 256 tokens by rank, the number of
// greater ones, which all waves count (each a slice of the comparisons); more by a bitonic network,
// whose steps of up to 64 stay within 128 tokens of one wave and need no barrier.
__device__ void sort_candidates(Shared& sh, int n) {
  const int tid = threadIdx.x;
  if (n <= 256) {
    const int width = n <= 64 ? 64 : (n <= 128 ? 128 : 256);
    if (tid < width) sh.rank[tid] = 0;
    __syncthreads();
    const int i = tid & (width - 1), slices = kThreads / width, s = tid / width;
    const uint64_t c = i < n ? sh.cand[i] : 0;
    int rank = 0;
    for (int j = n * s / slices; j < n * (s + 1) / slices; ++j) rank += sh.cand[j] > c;
    if (i < n && rank) atomicAdd(&sh.rank[i], rank);
    __syncthreads();
    if (tid < n) sh.cand[sh.rank[tid]] = c;
    __syncthreads();
    return;
  }
  int size = 512;
  while (size < n) size <<= 1;
  for (int i = n + tid; i < size; i += kThreads) sh.cand[i] = 0;
  __syncthreads();
  for (int len = 2; len <= size; len <<= 1)
    for (int step = len >> 1; step > 0; step >>= 1) {
      for (int i = tid; i < size / 2; i += kThreads) {
        const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
        const uint64_t x = sh.cand[lo], y = sh.cand[hi];
        const bool down = (lo & len) == 0;
        if ((x < y) == down) {
          sh.cand[lo] = y;
          sh.cand[hi] = x;
        }
      }
      // the next step (step / 2, or the first of the next length) crosses waves?
      const int next = step > 1 ? step >> 1 : len;
      if (next > 64 || step > 64) __syncthreads();
      else __builtin_amdgcn_wave_barrier();
    }
  __syncthreads();
}

constexpr int kPer = kCap / kThreads;  // sorted tokens per thread: kPer t .. kPer t + kPer - 1

// Weights of the sorted tokens and their running sums (c, sh.cum).
__device__ void weigh(Shared& sh, int n, float top, double inv_t, double* w, double* c) {
  const int tid = threadIdx.x, lane = tid & 63;
  double x = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = kPer * tid + i;
    w[i] = j < n ? weight(from_key((unsigned)(sh.cand[j] >> 32)), top, inv_t) : 0.0;
    x += w[i];
    c[i] = x;
  }
  double y = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double z = __shfl_up(y, d, 64);
    if (lane >= d) y += z;
  }
  if (lane == 63) sh.wave_d[tid >> 6] = y;
  __syncthreads();
  double before = y - x;
#pragma unroll
  for (int v = 0; v < kWaves; ++v)
    if (v < (tid >> 6)) before += sh.wave_d[v];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    c[i] += before;
    sh.cum[kPer * tid + i] = c[i];
  }
  __syncthreads();
}

// How many of this thread's sorted tokens from `from` up to `to` satisfy f(i), summed over all.
template <class F>
__device__ int count_tokens(Shared& sh, int from, int to, F f) {
  int x = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = kPer * (int)threadIdx.x + i;
    x += j >= from && j < to && f(i);
  }
  return block_count(sh, x);
}

// A row's settings.
struct Filters {
  int k, vocab;        // k = vocab: off
  double p, minp, u;   // p >= 1, minp = 0: off
  double inv_t;
};

// Second way: bins, then the tokens of the bins that hold a border.  False: too many of those.
template <bool F32>
__device__ bool by_bins(Shared& sh, const Row<F32>& row, const Filters& f, float top,
                        uint64_t* token, double* kept) {
  const int tid = threadIdx.x, lane = tid & 63;
  const double scale = f.inv_t * kBinScale;
  const bool open = top == __builtin_inff();  // only infinite logits weigh anything
  const double dtop = open ? (double)__FLT_MAX__ : (double)top;
  constexpr int kOwn = kBins / kThreads;
  __syncthreads();
  for (int i = tid; i < kBins; i += kThreads) {
    sh.bins[i] = 0;
    sh.mass[i] = 0;
  }
  if (tid == 0) sh.count = 0;
  if (tid < 4) {
    sh.found[tid] = kBins - 1;
    sh.iv[tid].lo = kBins;
    sh.iv[tid].hi = -1;
    sh.iv[tid].size = 0;
  }
  __syncthreads();
  // A token at place b + x of bin b weighs e^(-b / 128) (1 - y), y = 1 - e^(-x / 128) < 2^-7.  The
  // bins sum the y, as integers in units of 2^-38 (so that the sums do not depend on the order of
  // the additions), from fp32: y is off by at most about 2^-31.
  read_row<F32>(row, [&](float l, int) {
    if (l > kNegInf && !open) {
      const double place = bin_place(l, dtop, scale);
      const int b = (int)place;
      const float x = (float)(place - (double)b) * (1.0f / kBinScale);
      const float y = x * __builtin_fmaf(x, __builtin_fmaf(x, 1.0f / 6.0f, -0.5f), 1.0f);
      atomicAdd(&sh.bins[b], 1);
      atomicAdd(&sh.mass[b], (unsigned long long)(unsigned)(y * 274877906944.0f));
    } else if (l > kNegInf) {
      atomicAdd(&sh.bins[l == top ? 0 : kBins - 1], 1);
    }
  });
  __syncthreads();

  // ---- running counts and weights at the end of each of this thread's bins
  int cnt[kOwn];
  double mass[kOwn];
  {
    int cn = 0;
    double m = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int b = kOwn * tid + i, n = sh.bins[b];
      cn += n;
      const double e = open ? (b == 0 ? 1.0 : 0.0) : exp_f64(-(double)b / kBinScale);
      m += e * ((double)n - (double)sh.mass[b] * 3.637978807091713e-12);
      cnt[i] = cn;
      mass[i] = m;
    }
    int xc = cn;
    double xm = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int yc = __shfl_up(xc, d, 64);
      const double ym = __shfl_up(xm, d, 64);
      if (lane >= d) {
        xc += yc;
        xm += ym;
      }
    }
    if (lane == 63) {
      sh.wave_i[tid >> 6] = xc;
      sh.wave_d[tid >> 6] = xm;
    }
    __syncthreads();
    xc -= cn;
    xm -= m;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (w < (tid >> 6)) {
        xc += sh.wave_i[w];
        xm += sh.wave_d[w];
      }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      cnt[i] += xc;
      mass[i] += xm;
    }
  }
  // the first bin that passes, the last bin if none does
  auto first_bin = [&](int slot, auto passes) {
#pragma unroll
    for (int i = kOwn - 1; i >= 0; --i)
      if (passes(i)) atomicMin(&sh.found[slot], kOwn * tid + i);
    __syncthreads();
    const int b = sh.found[slot];
    __syncthreads();
    if (tid == 0) sh.found[slot] = kBins - 1;
    return b;
  };
  auto mass_to = [&](int bin) {  // the weight up to and including a bin, to all threads
    if (bin >= 0 && bin / kOwn == tid) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (bin % kOwn == i) sh.found_d = mass[i];
    }
    __syncthreads();
    const double r = bin < 0 ? 0.0 : sh.found_d;
    __syncthreads();
    return r;
  };
  // ---- the bins of each border: top-k, top-p, min-p, the draw.  Bounds of what a border depends
  // on (the weight of the first k, of the kept tokens) may spread it over several.
  constexpr double kSlack = 1e-10;
  int blo[4], bhi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    blo[i] = kBins;
    bhi[i] = -1;
  }
  const double z = mass_to(kBins - 1);
  double zk_lo = z, zk_hi = z;
  if (f.k < f.vocab) {
    blo[0] = bhi[0] = first_bin(0, [&](int i) { return cnt[i] >= f.k; });
    zk_lo = mass_to(blo[0] - 1);
    zk_hi = mass_to(bhi[0]);
  }
  double zn_lo = zk_lo, zn_hi = zk_hi;
  if (f.p < 1.0) {
    const double t0 = f.p * zk_lo * (1.0 - kSlack), t1 = f.p * zk_hi * (1.0 + kSlack);
    blo[1] = first_bin(1, [&](int i) { return mass[i] >= t0; });
    bhi[1] = first_bin(1, [&](int i) { return mass[i] >= t1; });
    zn_lo = fmin(zn_lo, fmax(t0, mass_to(blo[1] - 1)));
    zn_hi = fmin(zn_hi, mass_to(bhi[1]));
  }
  if (f.minp > 0.0) {
    const double d = -log(f.minp) * kBinScale;
    blo[2] = (int)fmin(fmax(d * (1.0 - 1e-5) - 0.01, 0.0), (double)(kBins - 1));
    bhi[2] = (int)fmin(d * (1.0 + 1e-5) + 0.01, (double)(kBins - 1));
    zn_lo = fmin(zn_lo, mass_to(blo[2] - 1));
    zn_hi = fmin(zn_hi, mass_to(bhi[2]));
  }
  {
    const double t0 = f.u * zn_lo * (1.0 - kSlack), t1 = f.u * zn_hi * (1.0 + kSlack);
    blo[3] = first_bin(3, [&](int i) { return mass[i] > t0; });
    bhi[3] = first_bin(3, [&](int i) { return mass[i] > t1; });
  }
  // ---- as disjoint intervals, in order: sort by lo, join those that touch
  if (tid == 0) {
    int ilo[4], ihi[4], m = 0;
    for (int i = 0; i < 4; ++i)
      if (bhi[i] >= 0) {
        int j = m++;
        for (; j > 0 && ilo[j - 1] > blo[i]; --j) {
          ilo[j] = ilo[j - 1];
          ihi[j] = ihi[j - 1];
        }
        ilo[j] = blo[i];
        ihi[j] = bhi[i];
      }
    int n = 0;
    for (int i = 0; i < m; ++i) {
      if (n > 0 && ilo[i] <= sh.iv[n - 1].hi + 1) {
        if (ihi[i] > sh.iv[n - 1].hi) sh.iv[n - 1].hi = ihi[i];
      } else {
        sh.iv[n].lo = ilo[i];
        sh.iv[n].hi = ihi[i];
        sh.iv[n].count0 = 0;
        sh.iv[n].mass0 = 0.0;
        ++n;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int b = kOwn * tid + i;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (b == sh.iv[v].lo - 1) {
        sh.iv[v].count0 = cnt[i];
        sh.iv[v].mass0 = mass[i];
      }
      if (b == sh.iv[v].hi) sh.iv[v].size = cnt[i];
    }
  }
  __syncthreads();
  if (tid == 0) {
    int first = 0;
    for (int v = 0; v < 4; ++v) {
      Interval& I = sh.iv[v];
      if (I.hi >= 0) I.size -= I.count0;
      I.first = first;
      first += I.size;
    }
    sh.found[0] = first;
  }
  __syncthreads();
  const int n = sh.found[0];
  if (n > kCap || n == 0) return false;

  // ---- third reading: collect the intervals' tokens
  const int lo0 = sh.iv[0].lo, hi0 = sh.iv[0].hi, lo1 = sh.iv[1].lo, hi1 = sh.iv[1].hi;
  const int lo2 = sh.iv[2].lo, hi2 = sh.iv[2].hi, lo3 = sh.iv[3].lo, hi3 = sh.iv[3].hi;
  const int nint = hi3 >= 0 ? 4 : (hi2 >= 0 ? 3 : (hi1 >= 0 ? 2 : 1));
  read_row<F32>(row, [&](float l, int idx) {
    const int b = open ? (l == top ? 0 : kBins - 1) : (int)bin_place(l, dtop, scale);
    bool in = b >= lo0 && b <= hi0;
    if (nint > 1) in |= b >= lo1 && b <= hi1;
    if (nint > 2) in |= (b >= lo2 && b <= hi2) || (b >= lo3 && b <= hi3);
    if (in && l > kNegInf) sh.cand[atomicAdd(&sh.count, 1)] = composite(l, idx);
  });
  __syncthreads();
  sort_candidates(sh, n);
  double w[kPer], c[kPer];
  weigh(sh, n, top, f.inv_t, w, c);
  // the interval that holds a border's bins, and what its running sums lack
  auto home = [&](int bin) { return bin <= hi0 ? 0 : (bin <= hi1 ? 1 : (bin <= hi2 ? 2 : 3)); };
  auto lacks = [&](const Interval& I) { return I.mass0 - (I.first > 0 ? sh.cum[I.first - 1] : 0.0); };
  // ---- the filters' prefixes: counts and weights
  int keep = f.vocab;
  double zk = z, zn = z;
  if (f.k < f.vocab) {
    const Interval& I = sh.iv[home(blo[0])];
    const int j = I.first + f.k - I.count0 - 1;
    if (j < I.first || j >= I.first + I.size) {
      if (f.k <= I.count0) return false;
      // fewer than k tokens are not masked: all of them
    } else {
      zk = zn = sh.cum[j] + lacks(I);
      keep = f.k;
    }
  }
  if (f.p < 1.0) {
    const Interval& I = sh.iv[home(blo[1])];
    const double t = f.p * zk - lacks(I);
    int m = count_tokens(sh, I.first, I.first + I.size, [&](int i) { return c[i] < t; });
    m = min(m, I.size - 1);  // (running sums rounded below the bin's)
    if (I.count0 + m + 1 < keep) {
      keep = I.count0 + m + 1;
      zn = sh.cum[I.first + m] + lacks(I);
    }
  }
  if (f.minp > 0.0) {
    const Interval& I = sh.iv[home(blo[2])];
    const int m = count_tokens(sh, I.first, I.first + I.size, [&](int i) { return w[i] >= f.minp; });
    if (I.count0 + m < keep) {
      keep = I.count0 + m;
      zn = m > 0 ? sh.cum[I.first + m - 1] + lacks(I) : I.mass0;
    }
  }
  const Interval& I = sh.iv[home(blo[3])];
  const double t = f.u * zn - lacks(I);
  int m = count_tokens(sh, I.first, I.first + I.size, [&](int i) { return c[i] <= t; });
  m = min(min(m, I.size - 1), keep - 1 - I.count0);
  if (m < 0) return false;
  *token = sh.cand[I.first + m];
  *kept = zn;
  return true;
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
  const bool need_z = !greedy && k == vocab && !known_k && (p < 1.0 || minp == 0.0);

  // ---- one reading: maxima of the parts, and the row's weight where the filters need it
  float part[kParts], ev = kNegInf, mt = kNegInf;
  double st = 0;
  const int iters = (row.nv + kThreads - 1) / kThreads;
#pragma unroll
  for (int q = 0; q < kParts; ++q) part[q] = kNegInf;
  read_batches<F32>(
      row,
      [&](const u32x4* r, int i0) {
        float vm = mt;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          // a vector past the end repeats the row's last one: it adds no weight, and must not
          // become this part's maximum
          const bool in = tid + (i0 + q) * kThreads < row.nv;
          float m4 = row.part(r[q], 0);
#pragma unroll
          for (int e = 1; e < kE; ++e) m4 = fmaxf(m4, row.part(r[q], e));
          m4 = in ? m4 : kNegInf;
          part[q] = fmaxf(part[q], m4);
          vm = fmaxf(vm, m4);
        }
        if (need_z && vm > kNegInf) {
          // weights relative to the thread's largest logit so far
          if (vm > mt) {
            st *= weight(mt, vm, inv_t);
            mt = vm;
          }
          if (mt < __builtin_inff()) {
            const Exp2 w(mt, inv_t);
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
              double v = 0;
#pragma unroll
              for (int e = 0; e < kE; ++e) v += w(row.part(r[q], e));
              st += tid + (i0 + q) * kThreads < row.nv ? v : 0.0;
            }
          } else {
#pragma unroll
            for (int q = 0; q < kParts; ++q)
#pragma unroll
              for (int e = 0; e < kE; ++e)
                st += tid + (i0 + q) * kThreads < row.nv && row.part(r[q], e) == mt ? 1.0 : 0.0;
          }
        }
      },
      [&](float l, int) { ev = l; });
  const int ei = tid < row.extra ? row.extra_index(tid) : 0;
  if (need_z && ev > kNegInf) {
    if (ev > mt) {
      st *= weight(mt, ev, inv_t);
      mt = ev;
    }
    st += weight(ev, mt, inv_t);
  }
  float mine = ev;
#pragma unroll
  for (int s = 0; s < kParts; ++s) mine = fmaxf(mine, part[s]);
  if (tid == 0) {
    sh.count = 0;
    sh.nhits = 0;
    sh.best = vocab;
  }
  float least;  // of the threads' maxima
  const float top = block_max(sh, mine, &least);
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
    // the want-th largest of the maxima, by bisection over their keys: every wave counts its own.
    // A bound that a few more reach will do.  All kThreads >= want threads reach the least.
    const bool few = want <= kFewK;
    unsigned key[kParts];
#pragma unroll
    for (int q = 0; q < kParts; ++q) key[q] = to_key(q == 0 && few ? mine : part[q]);
    unsigned lo = to_key(least), hi = to_key(top);
    for (int turn = 0; lo < hi; turn ^= 1) {
      const unsigned mid = lo + (hi - lo) / 2 + 1;
      int n = __popcll(__ballot(key[0] >= mid));
      if (!few)
#pragma unroll
        for (int q = 1; q < kParts; ++q) n += __popcll(__ballot(key[q] >= mid));
      if (lane == 0) sh.wave_n[turn][tid >> 6] = n;
      __syncthreads();
      n = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) n += sh.wave_n[turn][w];
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

  // ---- collect the tokens at or above the bound: the parts that reach it, read again by all
  // threads alike
  auto collect = [&](float l, int idx) {
    if (l >= tau && l > kNegInf) {
      if (greedy) {
        atomicMin(&sh.best, idx);
      } else {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kCap) sh.cand[at] = composite(l, idx);
      }
    }
  };
#pragma unroll
  for (int q = 0; q < kParts; ++q)
    if (part[q] >= tau && part[q] > kNegInf)
      sh.hits[atomicAdd(&sh.nhits, 1)] = (uint16_t)(tid + kThreads * q);
  collect(ev, ei);
  __syncthreads();
  {
    const int per = (iters + kParts - 1) / kParts, total = sh.nhits * per;
    for (int e0 = tid; e0 < total; e0 += kThreads) {
      const int hit = sh.hits[e0 / per];
      const int v = (hit & (kThreads - 1)) + (hit / kThreads + kParts * (e0 % per)) * kThreads;
      if (v < row.nv) {
        const u32x4 r = row.raw(v);
#pragma unroll
        for (int e = 0; e < kE; ++e) collect(row.part(r, e), row.head + v * kE + e);
      }
    }
  }
  __syncthreads();
  if (greedy) {
    if (tid == 0) {
      a.tokens[b] = sh.best;
      if (a.logprob) a.logprob[b] = 0.0f;
    }
    return;
  }
  auto answer = [&](uint64_t token, double kept) {
    if (tid == 0) {
      a.tokens[b] = (int)(0xFFFFFFFFu - (unsigned)token);
      if (a.logprob)
        a.logprob[b] = (float)(log_weight(from_key((unsigned)(token >> 32)), top, inv_t) - log(kept));
    }
  };
  const int n = sh.count;
  if (n <= kCap) {
    sort_candidates(sh, n);
    double w[kPer], c[kPer];
    weigh(sh, n, top, inv_t, w, c);
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
      const int np = count_tokens(sh, 0, lim, [&](int i) { return c[i] < t; });
      keep = np < lim ? np + 1 : (kk <= n ? kk : INT_MAX);
    }
    if (minp > 0.0) {
      const int nm = count_tokens(sh, 0, n, [&](int i) { return w[i] >= minp; });
      if (nm < n || complete || all_min_p) keep = min(keep, nm);
      else if (keep > n) keep = INT_MAX;
    }
    keep = max(keep, 1);
    if (keep > n && (keep != vocab || p < 1.0 || minp > 0.0)) ok = false;
    if (ok) {
      const double zn = keep <= n ? sh.cum[keep - 1] : z;
      const double t = u * zn;
      const int lim = min(keep, n);
      const int j = count_tokens(sh, 0, lim, [&](int i) { return c[i] <= t; });
      if (j < lim || keep <= n) {
        answer(sh.cand[min(j, keep - 1)], zn);
        return;
      }
    }
  }
  {
    const Filters f = {k, vocab, p, minp, u, inv_t};
    uint64_t token;
    double kept;
    if (by_bins<F32>(sh, row, f, top, &token, &kept)) {
      answer(token, kept);
      return;
    }
  }

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
  answer(hit, zn);
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
