// Sampling the next token of each row from given uniform numbers.
//
// Mathematics.  A row's tokens are ordered by descending logit, ties by ascending index; token j
// of that order weighs w_j = exp((l_j - l_0) / T).  Top-k, top-p and min-p each keep a prefix of
// the order: the first k; the shortest prefix whose weight reaches p times the weight of the first
// k; those with w_j >= min_p.  With n the shortest of the three (at least 1), the token drawn is
// the first whose running sum of weights exceeds u times the sum of the first n.
//
// Only a prefix of the order is ever needed.  A workgroup reads its row once and keeps, per
// thread, the largest value of each of 4 parts.  The k-th largest of the parts' maxima is a
// bound that at least k tokens reach and few more do: the parts whose maximum reaches it are read
// again and the tokens at or above it collected, ordered, weighed and summed.  Weights and sums
// are fp64, so that a draw next to a border between two tokens falls on the side where the
// definition puts it.
//
// Where no top-k says how many tokens to collect (top-p alone, or no filter at all), the reading
// instead counts and weighs the tokens in bins of 1/64 in (l_0 - l) / T, which gives the row's
// weight (to about 1e-9 of it) and confines each border (top-k, top-p, min-p, the draw) to a bin;
// the tokens of that bin are collected, and the border is resolved as before.  Where even that
// collects too many (thousands of tokens in a bin: nearly or quite equal logits), each border is found
// among the (logit, index) of all tokens, 12 bits a reading; a row of more than 2^20 tokens by bisection
// over them.
//
// What bounds it.  One workgroup a row: the rows are few (a decode batch), a row is small (512 KiB)
// and a second launch to join parts of rows costs as much as a row's reading.  A row of 131072 fp32
// logits: greedy 8 us (6.5 of them the reading, the rate of one compute unit), top-k 50 11, top-k
// 1000 27, top-p 0.9 29 (18 the reading with its tallies: vector instructions and LDS atomics), no
// filter 50 (13 of them reading the row again for a bin of thousands).  256 such rows with mixed
// settings, 134 MB: 64 us, 2.1 TB/s; 64 x 128000 bf16, top-k 50 with top-p: 16 us.
// Histograms by LDS atomics in the first reading without the maxima, every weight in fp64, took 158 us
// a row and more.
#include "bd_internal.h"
#include "sample.h"

namespace bd {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kParts = 4;       // a thread's vectors i, i + 4, ... make its part i
constexpr int kCap = 4096;      // collected tokens at most
constexpr int kPer = kCap / kThreads;  // of them per thread: kPer t .. kPer t + kPer - 1
// Top-k up to this goes by the maxima of the threads' parts, beyond by the bins (32 rows of 131072:
// k = 200 24.9 against 36.5 us, 1000 34.7 against 39.4, 2000 59.0 against 45.5).
constexpr int kMaxK = 1024;
constexpr int kBins = 4096;     // of 1/kBinScale each in logit / T; the last takes the rest
constexpr int kBinScale = 64;
constexpr int kMaxBinVocab = 1 << 20;

constexpr float kNegInf = -__builtin_inff();

// The workgroup's shared memory, at file scope so that functions that are not inlined address it
// directly: the kernel's time is largely latency, and much code run once costs fetches.
struct Shared {
  uint64_t cand[kCap];
  double cum[kCap];
  union {
    unsigned long long bins[kBins + 64];  // tallies; the last 64, one a lane, are not used
    double bin_mass[kBins];  // running weights, once the tallies have been read
  };
  int bin_count[kBins];  // running counts
  uint16_t hits[kParts * kThreads];  // parts to read again: thread + kThreads * part
  int bucket[kThreads];
  double wave_d[kWaves];
  float wave_f[kWaves], wave_g[kWaves];
  int wave_i[kWaves], wave_n[2][kWaves];
  int count, nhits, best, most;
  int found;
  uint64_t few_token;
  double few_mass;
  int few_keep;
};
__shared__ Shared sh;

// Order-preserving map of floats to unsigned; -0 and +0 are one value, NaN counts as -inf.
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.0f : kNegInf; }
__device__ __forceinline__ unsigned to_key(float x) {
  const unsigned b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_key(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// A token in the order: larger logits first, then smaller indices.
__device__ __forceinline__ uint64_t composite(float l, int idx) {
  return ((uint64_t)to_key(l) << 32) | (0xFFFFFFFFu - (unsigned)idx);
}
__device__ __forceinline__ float logit_of(uint64_t c) { return from_key((unsigned)(c >> 32)); }

template <bool F32>
struct Row {
  static constexpr int kE = F32 ? 4 : 8;  // elements of a 16-byte vector
  const unsigned char* p;                 // first element
  int head, nv, extra;  // elements before the first aligned vector, vectors, head + tail elements
  int iters;            // vectors per thread, at most

  __device__ __forceinline__ Row(const SampleArgs& a, int row) {
    p = static_cast<const unsigned char*>(a.logits) + (int64_t)row * a.row_stride * (F32 ? 4 : 2);
    const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    head = min(a.vocab, mis ? (16 - mis) / (F32 ? 4 : 2) : 0);
    nv = (a.vocab - head) / kE;
    extra = a.vocab - nv * kE;
    iters = (nv + kThreads - 1) / kThreads;
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
  __device__ __forceinline__ static float plain(const u32x4& r, int e) {  // NaN and -0 as they are
    if constexpr (F32) return __uint_as_float(r[e]);
    const unsigned x = r[e >> 1];
    return (e & 1) ? bf16hi_to_f32(x) : bf16lo_to_f32(x);
  }
};

// e^x for x <= 0 in fp64: x = n ln 2 + r with |r| <= ln 2 / 2, and the Taylor series of e^r to
// r^12 (the next term is below 2e-16).
__device__ __noinline__ double exp_f64(double x) {
  x = fmax(x, -745.0);
  const double n = __builtin_rint(x * 1.4426950408889634074);
  // ln 2 in two parts: its first 40 bits, of which n (11 bits) times is exact, and the rest
  double r = __builtin_fma(n, -0x1.62e42fefa2p-1, x);
  r = __builtin_fma(n, -0x1.9ef35793c7673p-41, r);
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
__device__ __noinline__ double log_f64(double x) { return log(x); }
// ln w and w; the largest logit weighs 1, also where it is infinite
__device__ __forceinline__ double log_weight(float l, float top, double inv_t) {
  return l == top ? 0.0 : ((double)l - (double)top) * inv_t;
}
__device__ __forceinline__ double weight(float l, float top, double inv_t) {
  return l == kNegInf ? 0.0 : exp_f64(log_weight(l, top, inv_t));
}

// The bins.  A logit's place is (ref - l) * 64 / T, kept as a fixed-point number: the bin, and 32
// bits of the place within it.  Never less for a smaller logit; what lies beyond the bins counts as
// the last one's.  One fused product and sum in fp64 with an offset of 1.5 * 2^20 leaves the bin in
// the low bits of the upper half, the place within it in the lower half.
//
// A token at place b + 64 x of bin b weighs e^(-b / 64) (1 - y), y = 1 - e^-x < 2^-6.  A bin's
// tally is one 64-bit integer, count * 2^low + sum of y in units: additions of integers do not
// depend on their order.  y is a cubic in fp32 (x - x^2 / 2 + x^3 / 6 - x^4 / 24 with the last term
// replaced by the cubic nearest to it over [0, 2^-6]), so a weight is off by about 1e-9 of itself
// at most; these errors average out over a sum.
constexpr double kOffset = 1572864.0;
constexpr unsigned kOffsetHigh = 0x41380000u;  // its upper half
struct Bins {
  double offset, scale;  // of the place
  int low;               // bits below the count, at least 42
  float units;           // units of y in 1, a power of two up to 2^36: y in units fits 32 bits
  double unit;           // 1 / units
  float c1, c2, c3;      // y in units as a polynomial of the 32 bits
  // false: places do not fit (T is so small that only the largest logit counts), or there are none (T
  // is infinite: all in one bin whose width in logits has no number)
  __device__ __forceinline__ bool begin_at(double ref) {
    offset = ref * scale + kOffset;
    return scale > 0.0 && fabs(ref * scale) < 1073741824.0;
  }
  __device__ __forceinline__ Bins(int vocab, double inv_t) {
    scale = inv_t * kBinScale;
    offset = 0;
    const int cb = 32 - __builtin_clz((unsigned)vocab);  // a count takes up to cb bits
    low = 63 - cb;
    units = __builtin_ldexpf(1.0f, min(low - cb + 6, 36));
    unit = 1.0 / (double)units;
    constexpr double a = 1.0 / kBinScale, x1 = a / 4294967296.0;  // 2^-6, and x of the lowest bit
    c1 = (float)((1.0 - a * a * a / 96.0) * x1) * units;
    c2 = (float)((-0.5 + a * a * (1.25 / 24.0)) * x1 * x1) * units;
    c3 = (float)((1.0 / 6.0 - a / 12.0) * x1 * x1 * x1) * units;
  }
  // bin (or more than that, where it is beyond the bins) * 2^32 + place within it
  __device__ __forceinline__ uint64_t place(float l) const {
    const uint64_t x = (uint64_t)__double_as_longlong(__builtin_fma(-(double)l, scale, offset));
    return x - ((uint64_t)kOffsetHigh << 32);
  }
  __device__ __forceinline__ static unsigned bin(uint64_t place) {
    return min((unsigned)(place >> 32), (unsigned)kBins - 1);
  }
  __device__ __forceinline__ unsigned long long tally(uint64_t place) const {
    const float f = (float)(unsigned)place;
    const float y = __builtin_fmaf(f, __builtin_fmaf(f, __builtin_fmaf(f, c3, c2), c1), 0.5f);
    return (unsigned long long)(1u << (low - 32)) << 32 | (unsigned)y;
  }
  __device__ __forceinline__ int count(unsigned long long t) const { return (int)(t >> low); }
  // of a bin whose upper logit weighs 1
  __device__ __forceinline__ double weight(unsigned long long t) const {
    return (double)count(t) - (double)(t & ((1ull << low) - 1)) * unit;
  }
};

// ---- within a wave: lane i's sum of the lanes up to it (lane 63: of all), by moves between lanes
// that need no shared memory.  kCtrl 0x110 + n: from n lanes below in the row of 16; 0x142, 0x143:
// the last lane of the row, of the half, below to the next one.
template <int kCtrl, int kRows>
__device__ __forceinline__ int lane_move(int x, int otherwise) {
  return __builtin_amdgcn_update_dpp(otherwise, x, kCtrl, kRows, 0xF, false);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ double lane_move(double x) {
  const long long b = __double_as_longlong(x);
  const unsigned lo = (unsigned)lane_move<kCtrl, kRows>((int)b, 0);
  const unsigned hi = (unsigned)lane_move<kCtrl, kRows>((int)(b >> 32), 0);
  return __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
}
__device__ __forceinline__ double wave_scan(double x) {
  x += lane_move<0x111, 0xF>(x);
  x += lane_move<0x112, 0xF>(x);
  x += lane_move<0x114, 0xF>(x);
  x += lane_move<0x118, 0xF>(x);
  x += lane_move<0x142, 0xA>(x);
  return x + lane_move<0x143, 0xC>(x);
}
__device__ __forceinline__ int wave_scan(int x) {
  x += lane_move<0x111, 0xF>(x, 0);
  x += lane_move<0x112, 0xF>(x, 0);
  x += lane_move<0x114, 0xF>(x, 0);
  x += lane_move<0x118, 0xF>(x, 0);
  x += lane_move<0x142, 0xA>(x, 0);
  return x + lane_move<0x143, 0xC>(x, 0);
}
__device__ __forceinline__ double last_lane(double x) {
  const long long b = __double_as_longlong(x);
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)b, 63);
  const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(b >> 32), 63);
  return __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
}
template <int kCtrl, int kRows>
__device__ __forceinline__ float lane_move(float x) {  // where there is none: its own
  return __int_as_float(lane_move<kCtrl, kRows>(__float_as_int(x), __float_as_int(x)));
}
__device__ __forceinline__ float wave_most(float x) {  // lane 63: of all
  x = fmaxf(x, lane_move<0x111, 0xF>(x));
  x = fmaxf(x, lane_move<0x112, 0xF>(x));
  x = fmaxf(x, lane_move<0x114, 0xF>(x));
  x = fmaxf(x, lane_move<0x118, 0xF>(x));
  x = fmaxf(x, lane_move<0x142, 0xA>(x));
  return fmaxf(x, lane_move<0x143, 0xC>(x));
}

// ---- sums over the workgroup, in a fixed order, to all threads
__device__ __noinline__ double block_sum(double x) {
  x = wave_scan(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) sh.wave_d[threadIdx.x >> 6] = x;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) t += sh.wave_d[w];
  return t;
}
__device__ __noinline__ int block_count(int x) {
  x = wave_scan(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) sh.wave_i[threadIdx.x >> 6] = x;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) t += sh.wave_i[w];
  return t;
}
struct Range {
  float most, least;
};
__device__ __noinline__ Range block_range(float x) {
  const float y = -wave_most(-x);
  x = wave_most(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) {
    sh.wave_f[threadIdx.x >> 6] = x;
    sh.wave_g[threadIdx.x >> 6] = y;
  }
  __syncthreads();
  Range r = {sh.wave_f[0], sh.wave_g[0]};
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    r.most = fmaxf(r.most, sh.wave_f[w]);
    r.least = fminf(r.least, sh.wave_g[w]);
  }
  return r;
}
// Running sums of one count and one weight per thread, without its own.
struct Before {
  int count;
  double mass;
};
__device__ __noinline__ Before block_prefix(int n, double m) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int y = wave_scan(n);
  const double z = wave_scan(m);
  __syncthreads();
  if (lane == 63) {
    sh.wave_i[wave] = y;
    sh.wave_d[wave] = z;
  }
  __syncthreads();
  Before r = {0, 0.0};
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w) {
    const bool in = w < wave;
    r.count += in ? sh.wave_i[w] : 0;
    r.mass += in ? sh.wave_d[w] : 0.0;
  }
  r.count += y - n;
  r.mass += z - m;
  return r;
}

// One reading of the row by the workgroup, kParts vectors a thread in flight ahead of the ones that
// are worked on: each(vectors, i0) gets the vectors tid + (i0 + q) * kThreads, q < kParts (past the
// row's end: its last one); one(l, idx) the elements before and after the vectors.
template <bool F32, class Each, class One>
__device__ __forceinline__ void read_batches(const Row<F32>& row, Each each, One one) {
  const int tid = threadIdx.x;
  u32x4 r[kParts], nx[kParts];
  auto fetch = [&](int i0, u32x4* v) {
#pragma unroll
    for (int q = 0; q < kParts; ++q) v[q] = row.raw(min(tid + (i0 + q) * kThreads, row.nv - 1));
  };
  if (row.iters > 0) fetch(0, r);
  if (tid < row.extra) {
    const int idx = row.extra_index(tid);
    one(row.one(idx), idx);
  }
  for (int i0 = 0; i0 < row.iters; i0 += kParts) {
    if (i0 + kParts < row.iters) fetch(i0 + kParts, nx);
    each(r, i0);
#pragma unroll
    for (int q = 0; q < kParts; ++q) r[q] = nx[q];
  }
}

// Puts the tokens with lo <= logit <= hi that `keep` confirms into sh.cand (sh.count counts them,
// also beyond kCap), the row read in full: a mask of a batch's elements first, so that the many that
// fail cost two comparisons each.
template <bool F32, class Keep>
__device__ __forceinline__ void collect_row(const Row<F32>& row, float lo, float hi, Keep keep) {
  constexpr int kE = Row<F32>::kE;
  auto take = [&](float l, int idx) {
    if (l >= lo && l <= hi && l > kNegInf && keep(l)) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kCap) sh.cand[at] = composite(l, idx);
    }
  };
  read_batches<F32>(
      row,
      [&](const u32x4* r, int i0) {
        unsigned mask = 0;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          unsigned m = 0;
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const float l = row.part(r[q], e);
            m |= (unsigned)((l >= lo) & (l <= hi)) << e;
          }
          if ((int)threadIdx.x + (i0 + q) * kThreads < row.nv) mask |= m << (kE * q);
        }
        while (mask) {
          const int bit = __builtin_ctz(mask);
          mask &= mask - 1;
          const int v = (int)threadIdx.x + (i0 + bit / kE) * kThreads;
          const int idx = row.head + v * kE + bit % kE;
          take(row.one(idx), idx);
        }
      },
      take);
}
// The same, reading only the parts listed in sh.hits (by all threads alike) and this thread's own
// element ev at ei.
template <bool F32, class Keep>
__device__ __forceinline__ void collect_hits(const Row<F32>& row, float ev, int ei, float lo, float hi,
                                             Keep keep) {
  constexpr int kE = Row<F32>::kE;
  auto take = [&](float l, int idx) {
    if (l >= lo && l <= hi && l > kNegInf && keep(l)) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kCap) sh.cand[at] = composite(l, idx);
    }
  };
  take(ev, ei);
  const int per = (row.iters + kParts - 1) / kParts, total = sh.nhits * per;
  for (int e0 = threadIdx.x; e0 < total; e0 += kThreads) {
    const int item = e0 / per, hit = sh.hits[item];
    const int v = (hit & (kThreads - 1)) + (hit / kThreads + kParts * (e0 - item * per)) * kThreads;
    if (v < row.nv) {
      const u32x4 r = row.raw(v);
#pragma unroll
      for (int e = 0; e < kE; ++e) take(row.part(r, e), row.head + v * kE + e);
    }
  }
}
// Lists the parts whose maximum is at least lo.
__device__ __forceinline__ void list_hits(const float* part, float lo) {
#pragma unroll
  for (int q = 0; q < kParts; ++q)
    if (part[q] >= lo && part[q] > kNegInf)
      sh.hits[atomicAdd(&sh.nhits, 1)] = (uint16_t)(threadIdx.x + kThreads * q);
}

// Sorts sh.cand[0 .. n) in descending order (all threads).  Up to 256 tokens by rank, the number of
// greater ones, which all waves count (each a slice of the comparisons; 100 tokens 22.3 us a call
// against 24.8 by buckets, 200 24.7 against 26.1).  More: kThreads buckets of equal width from the
// largest logit down to the least, and the rank within the bucket; a bitonic network where a bucket
// gets too many for that.
__device__ __noinline__ void sort_candidates(int n) {
  const int tid = threadIdx.x;
  sh.bucket[tid] = 0;
  if (tid == 0) sh.most = 0;
  __syncthreads();
  if (n <= 256) {
    const int width = n <= 64 ? 64 : (n <= 128 ? 128 : 256);
    const int i = tid & (width - 1), slices = kThreads / width, s = tid / width;
    const uint64_t c = i < n ? sh.cand[i] : 0;
    int rank = 0;
    for (int j = n * s / slices; j < n * (s + 1) / slices; ++j) rank += sh.cand[j] > c;
    if (i < n && rank) atomicAdd(&sh.bucket[i], rank);
    __syncthreads();
    if (tid < n) sh.cand[sh.bucket[tid]] = c;
    __syncthreads();
    return;
  }
  float least = __builtin_inff(), most = kNegInf;
  for (int j = tid; j < n; j += kThreads) {
    const float l = logit_of(sh.cand[j]);
    least = fminf(least, l);
    most = fmaxf(most, l);
  }
  most = block_range(most).most;
  least = block_range(least).least;
  const float width = (most - least) * (1.0f / kThreads);
  const float inv = width > 0.f && width < __FLT_MAX__ ? 1.0f / width : 0.f;
  uint64_t c[kPer];
  int place[kPer];  // bucket * 2^16 + slot
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = tid + kThreads * i;
    c[i] = 0;
    place[i] = 0;
    if (j < n) {
      c[i] = sh.cand[j];
      const int b = (int)fminf((most - logit_of(c[i])) * inv, (float)(kThreads - 1));
      place[i] = (b << 16) + atomicAdd(&sh.bucket[b], 1);
    }
  }
  __syncthreads();
  const int size = sh.bucket[tid];
  if (size > 256) sh.most = 1;
  const int begin = block_prefix(size, 0.0).count;
  if (sh.most == 0) {
    sh.bucket[tid] = begin;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (tid + kThreads * i < n) sh.cand[sh.bucket[place[i] >> 16] + (place[i] & 0xFFFF)] = c[i];
    __syncthreads();
    int rank[kPer];
    for (int i = 0; i < kPer; ++i) {
      rank[i] = 0;
      if (tid + kThreads * i < n) {
        const int b = place[i] >> 16;
        const int first = sh.bucket[b], last = b + 1 < kThreads ? sh.bucket[b + 1] : n;
        rank[i] = first;
        for (int j = first; j < last; ++j) rank[i] += sh.cand[j] > c[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (tid + kThreads * i < n) sh.cand[rank[i]] = c[i];
    __syncthreads();
    return;
  }
  int pow2 = 512;
  while (pow2 < n) pow2 <<= 1;
  for (int i = n + tid; i < pow2; i += kThreads) sh.cand[i] = 0;
  __syncthreads();
  for (int len = 2; len <= pow2; len <<= 1)
    for (int step = len >> 1; step > 0; step >>= 1) {
      for (int i = tid; i < pow2 / 2; i += kThreads) {
        const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
        const uint64_t x = sh.cand[lo], y = sh.cand[hi];
        const bool down = (lo & len) == 0;
        if ((x < y) == down) {
          sh.cand[lo] = y;
          sh.cand[hi] = x;
        }
      }
      __syncthreads();
    }
}

// Running sums of the sorted tokens' weights into sh.cum.
__device__ __noinline__ void weigh(int n, float top, double inv_t) {
  const int first = kPer * (int)threadIdx.x;
  double x = 0;
#pragma unroll 1
  for (int j = first; j < min(first + kPer, n); ++j) {
    const double w = weight(logit_of(sh.cand[j]), top, inv_t);
    sh.cum[j] = w;
    x += w;
  }
  x = block_prefix(0, x).mass;
#pragma unroll 1
  for (int j = first; j < min(first + kPer, n); ++j) {
    x += sh.cum[j];
    sh.cum[j] = x;
  }
  __syncthreads();
}
// How many of the first n running sums are below t (or equal, too).
__device__ __noinline__ int count_below(int n, double t, bool or_equal) {
  int x = 0;
#pragma unroll 1
  for (int j = threadIdx.x; j < n; j += kThreads) x += or_equal ? sh.cum[j] <= t : sh.cum[j] < t;
  return block_count(x);
}
// How many of the first n sorted tokens weigh at least m.
__device__ __noinline__ int count_heavy(int n, double m, float top, double inv_t) {
  int x = 0;
#pragma unroll 1
  for (int j = threadIdx.x; j < n; j += kThreads) x += weight(logit_of(sh.cand[j]), top, inv_t) >= m;
  return block_count(x);
}

// ---- up to 64 collected tokens: one wave orders and weighs them, a lane each, with no barriers
// (32 rows of 131072 with top-p 0.9: 31.7 us, 35.0 with the workgroup's sort and sums)
struct Few {
  uint64_t c;     // the lane's token in the order; 0: none
  double w, cum;  // its weight, and the running sum
};
__device__ __noinline__ Few order_few(int n, float top, double inv_t) {
  const int lane = threadIdx.x & 63;
  uint64_t c = lane < n ? sh.cand[lane] : 0;
  int rank = 0;  // tokens before it
#pragma unroll
  for (int j = 0; j < 64; ++j) {  // (the lanes past n hold 0, which is before no token)
    if (j % 16 == 0 && j >= n) break;
    const uint64_t lo = (unsigned)__builtin_amdgcn_readlane((int)c, j);
    const uint64_t hi = (unsigned)__builtin_amdgcn_readlane((int)(c >> 32), j);
    rank += (hi << 32 | lo) > c;
  }
  if (lane >= n) rank = lane;
  const unsigned lo = (unsigned)__builtin_amdgcn_ds_permute(4 * rank, (int)c);
  const unsigned hi = (unsigned)__builtin_amdgcn_ds_permute(4 * rank, (int)(c >> 32));
  c = (uint64_t)hi << 32 | lo;
  const double w = lane < n ? weight(logit_of(c), top, inv_t) : 0.0;
  return Few{c, w, wave_scan(w)};
}
__device__ __forceinline__ int lanes_below(int n, double t, bool or_equal, const Few& f) {
  return __popcll(__ballot((int)(threadIdx.x & 63) < n && (or_equal ? f.cum <= t : f.cum < t)));
}

// ---- the last resort: borders as (logit, index), whatever the logits are
// one(l, idx) for every token, a few loads in flight ahead of it
template <bool F32, class One>
__device__ __forceinline__ void each_token(const Row<F32>& row, One one) {
  constexpr int kAhead = 4;
  const int vocab = row.nv * Row<F32>::kE + row.extra;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < vocab; i0 += kAhead * kThreads) {
    float l[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) l[j] = row.one(min(i0 + j * kThreads, vocab - 1));
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j * kThreads < vocab) one(l[j], i0 + j * kThreads);
  }
}
// Count and weight of the row's tokens at or above a composite.
template <bool F32>
__device__ __noinline__ Before above(const Row<F32> row, uint64_t c, float top, double inv_t) {
  int n = 0;
  double s = 0;
  auto one = [&](float l, int idx) {
    if (composite(l, idx) >= c) {
      ++n;
      s += weight(l, top, inv_t);
    }
  };
  each_token(row, one);
  const Before r = {block_count(n), block_sum(s)};
  return r;
}
// The largest composite c at or above which there are `count` tokens, a weight of `mass`, or (strict)
// a weight of more than `mass`; 0 if there is none.
template <bool F32>
__device__ __noinline__ uint64_t bisect(const Row<F32> row, float top, double inv_t, int count, double mass,
                                        bool strict) {
  uint64_t lo = 0, hi = ((uint64_t)to_key(top) << 32) | 0xFFFFFFFFull;
  while (lo < hi) {
    const uint64_t mid = lo + (hi - lo) / 2 + 1;
    const Before x = above<F32>(row, mid, top, inv_t);
    const bool reached = count > 0 ? x.count >= count : (strict ? x.mass > mass : x.mass >= mass);
    if (reached) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The same for rows up to kMaxBinVocab, 12 bits of the composite at a time: one reading per 12 bits
// tallies the tokens that agree with the bits found so far, as counts or as weights in units as fine as
// the row's tokens let them be (integers: no order of additions matters; n tokens of weight 1 fit 64
// bits, so that n rounded weights are off by at most n^2 2^-64 together: 1e-9 at 2^17, 6e-8 at 2^20),
// and the bits of the border are those where the running sum from the top passes the target.  A row of 131072 nearly equal logits, no filter:
// 0.32 ms, bisection 3.8; all equal, where additions to one tally take turns: 0.75 against 3.8.
template <bool F32>
__device__ __noinline__ uint64_t select(const Row<F32> row, float top, double inv_t, int count, double mass,
                                        bool strict) {
  constexpr int kOwn = kBins / kThreads;
  const int tid = threadIdx.x;
  const int vocab = row.nv * Row<F32>::kE + row.extra;
  const double units = __builtin_ldexp(1.0, 32 + __builtin_clz((unsigned)vocab));
  const double target = count > 0 ? (double)count : mass * units;
  double before = 0;    // the sum above the bits found so far
  uint64_t found = 0;   // those bits
#pragma unroll 1
  for (int shift = 52; shift >= 0; shift = shift == 4 ? 0 : shift - 12) {
    const int bits = shift == 0 ? 4 : 12;
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) sh.bins[i] = 0;
    if (tid == 0) {
      sh.found = -1;
      sh.most = kBins;
    }
    __syncthreads();
    auto one = [&](float l, int idx) {
      const uint64_t c = composite(l, idx);
      if (shift < 52 && c >> (shift + bits) != found) return;
      const unsigned long long u =
          count > 0 ? 1 : (unsigned long long)(weight(l, top, inv_t) * units + 0.5);
      atomicAdd(&sh.bins[(unsigned)(c >> shift) & ((1u << bits) - 1)], u);
    };
    each_token(row, one);
    __syncthreads();
    // thread t has the digits kBins - 1 - kOwn t and the kOwn - 1 below
    const int first = kBins - 1 - kOwn * tid;
    double sum = 0;
    for (int i = 0; i < kOwn; ++i) sum += (double)sh.bins[first - i];
    const double start = before + block_prefix(0, sum).mass;
    sum = start;
    for (int i = 0; i < kOwn; ++i) {
      const unsigned long long u = sh.bins[first - i];
      if (u) atomicMin(&sh.most, first - i);
      sum += (double)u;
      if (strict ? sum > target : sum >= target) {
        atomicMax(&sh.found, first - i);
        break;
      }
    }
    __syncthreads();
    int digit = sh.found;
    if (digit < 0) {
      // the whole row does not reach it: none does, or (a sum of weights, rounded) its last token
      if (strict && shift == 52) return 0;
      digit = min(sh.most, kBins - 1);
    }
    if (digit <= first && digit > first - kOwn) {
      sum = start;
      for (int i = first; i > digit; --i) sum += (double)sh.bins[i];
      sh.few_mass = sum;
    }
    __syncthreads();
    before = sh.few_mass;
    found = found << bits | (unsigned)digit;
  }
  __syncthreads();
  return found;
}

// A row's settings.
struct Filters {
  int k, vocab;        // k = vocab: off
  double p, minp, u;   // p >= 1, minp = 0: off
  double inv_t;
};
struct Answer {
  uint64_t token;
  double kept;  // the weight of the tokens kept
  bool found;
};

template <bool F32>
__device__ __noinline__ Answer by_rank(const Row<F32> row, const Filters f, float top) {
  auto find = [&](int count, double mass, bool strict) {
    return f.vocab <= kMaxBinVocab ? select<F32>(row, top, f.inv_t, count, mass, strict)
                                   : bisect<F32>(row, top, f.inv_t, count, mass, strict);
  };
  uint64_t border = 0;
  if (f.k < f.vocab) border = find(f.k, 0.0, false);
  if (f.p < 1.0) {
    const double zk = above<F32>(row, border, top, f.inv_t).mass;
    const uint64_t c = find(0, f.p * zk, false);
    border = c > border ? c : border;
  }
  if (f.minp > 0.0) {
    unsigned lo = 0, hi = to_key(top);  // the smallest key with w >= min_p
    while (lo < hi) {
      const unsigned mid = lo + (hi - lo) / 2;
      if (weight(clean(from_key(mid)), top, f.inv_t) >= f.minp) hi = mid;
      else lo = mid + 1;
    }
    const uint64_t c = (uint64_t)lo << 32;
    border = c > border ? c : border;
  }
  const Before kept = above<F32>(row, border, top, f.inv_t);
  const double zn = kept.mass;
  uint64_t hit = find(0, f.u * zn, true);
  // u * zn rounded up to zn: the last token kept that weighs something
  if (hit < border || hit == 0) {
    hit = find(0, zn, false);
    if (hit < border) hit = find(kept.count, 0.0, false);  // (a rounding of the sums)
  }
  return Answer{hit, zn, true};
}

// The answer from the tallied bins: each border in turn (top-k,
// top-p, min-p, the draw) lies in one bin, whose tokens are collected and sorted.  part: this
// thread's maxima; ev, ei: its single element.  Not found: too many tokens in a bin (or not those that
// were tallied).
template <bool F32>
__device__ __forceinline__ Answer by_bins(const Row<F32>& row, const Filters& f, float top,
                                          const Bins& bins, const float* part, float ev, int ei) {
  constexpr int kOwn = kBins / kThreads;
  const int tid = threadIdx.x;
  const double inv_scale = 1.0 / bins.scale, ref = (bins.offset - kOffset) * inv_scale;
  const double lead = (double)bins.place(top) * (1.0 / 4294967296.0);  // of the largest
  // running counts and weights (of the largest logit: 1) before and after this thread's bins
  int cnt0 = 0, cnt1 = 0;
  double mass0 = 0, mass1 = 0;
  {
    unsigned long long t[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) t[i] = sh.bins[kOwn * tid + i];
    // a bin's upper logit weighs e^(-1/64) of the one's before (bins above the largest are empty)
    double e = exp_f64((lead - (double)(kOwn * tid)) * (1.0 / kBinScale) - 1.0) * 2.718281828459045235;
    double m[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      cnt1 += bins.count(t[i]);
      // (what lies beyond the bins weighs less than e^-39.9 each, 4e-12 together: nothing, among sums)
      m[i] = mass1 += kOwn * tid + i < kBins - 1 ? e * bins.weight(t[i]) : 0.0;
      e *= 0.98449643700540840596;  // e^(-1/64)
    }
    const Before b = block_prefix(cnt1, mass1);
    cnt0 = cnt1 = b.count;
    mass0 = b.mass;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      sh.bin_count[kOwn * tid + i] = cnt1 += bins.count(t[i]);
      sh.bin_mass[kOwn * tid + i] = mass1 = mass0 + m[i];
    }
  }
  if (tid == 0) sh.found = kBins - 1;
  __syncthreads();
  // the value before is the one that the thread before ends with, to the last bit
  mass0 = tid ? sh.bin_mass[kOwn * tid - 1] : 0.0;
  int keep = f.vocab;                         // tokens kept
  double zk = sh.bin_mass[kBins - 1], zn = zk;  // weight of the first k, of the tokens kept
  int whole = kBins;  // the bins before this one are in zk and zn as tallied, this one token by token
  Answer r = {0, 0.0, false};
#pragma unroll 1
  for (int stage = 0; stage < 4; ++stage) {
    if (stage == 0 ? f.k == f.vocab : (stage == 1 ? f.p >= 1.0 : (stage == 2 && f.minp == 0.0))) continue;
    // the border's bin: the first whose value passes the target, the last bin if none does
    double target = f.k;
    bool here = cnt0 < f.k && cnt1 >= f.k;  // among this thread's bins?
    if (stage == 1) {
      target = f.p * zk;
      here = mass0 < target && mass1 >= target;
    } else if (stage == 2) {
      target = fmin(fmax(floor(lead - log_f64(f.minp) * kBinScale), 0.0), kBins - 1.0);
      here = (int)target / kOwn == tid;
    } else if (stage == 3) {
      target = f.u * zn;
      here = mass0 <= target && mass1 > target;
    }
    if (here) {
      int at = kOwn * tid;
      for (; at < kOwn * tid + kOwn - 1; ++at) {
        const double x = stage == 0 ? (double)sh.bin_count[at] : (stage == 2 ? (double)at : sh.bin_mass[at]);
        if (stage == 3 ? x > target : x >= target) break;
      }
      atomicMin(&sh.found, at);  // (by rounding, running weights may pass a target twice)
    }
    if (tid == 0) sh.count = sh.nhits = 0;
    __syncthreads();
    const int bin = sh.found, before = bin ? sh.bin_count[bin - 1] : 0, n = sh.bin_count[bin] - before;
    const double mass_before = bin ? sh.bin_mass[bin - 1] : 0.0;
    if (n > kCap) return r;
    // the bin's tokens; bounds in logits, with a margin for their rounding, pass over most others
    const double up = ref - (double)bin * inv_scale, down = up - inv_scale;
    const double slack = 1e-6 * (fabs(up) + fabs(down)) + 1e-3 * inv_scale;
    const float hi = (float)(up + slack), lo = bin == kBins - 1 ? kNegInf : (float)(down - slack);
    auto keep_it = [&](float l) { return (int)Bins::bin(bins.place(l)) == bin; };
    list_hits(part, lo);
    __syncthreads();
    // (32 rows of 131072: top-p 0.9, few parts: hits 31.4, row 48.3 us; top-p 0.99 at T = 1.3, most
    // parts: 84.4 against 68.2)
    if (sh.nhits > kParts * kThreads / 4) collect_row<F32>(row, lo, hi, keep_it);
    else collect_hits<F32>(row, ev, ei, lo, hi, keep_it);
    __syncthreads();
    // only what was collected is ordered: a token that was tallied but lies outside the bounds would
    // leave a place that nobody wrote
    if (sh.count != n) return r;
    // sums of weights before the border are those of the bins before and of the bin's own tokens
    int last = -1;    // the last of the bin's tokens that is kept
    double sum = 0;   // their weight up to it
    uint64_t token = 0;
    const int limit = min(n, keep - before);  // tokens of the bin that a draw may take
    // A target takes the bin's weight as its tokens have it, too: where they hold the row's weight, a
    // border between equal tokens (half of them, say) is then exactly where the definition has it.  (Up
    // to 64 tokens it is wave 0 that has them, and zn then: the wave that writes the answer.)
    const double tallied = bin < whole ? sh.bin_mass[bin] - mass_before : 0.0;
    auto own_target = [&](double weight) {
      const double more = bin < whole ? weight - tallied : 0.0;
      if (stage == 3) zn += more;
      return (stage == 3 ? f.u * zn : f.p * (zk + more)) - mass_before;
    };
    const bool few = n <= 64;
    if (few) {
      if (tid < 64) {
        const Few c = order_few(n, top, f.inv_t);
        const double t = own_target(last_lane(c.cum));
        if (stage == 0) last = f.k - before <= n ? f.k - before - 1 : -1;
        else if (stage == 1) last = min(lanes_below(n, t, false, c), n - 1);
        else if (stage == 2) last = __popcll(__ballot(tid < n && c.w >= f.minp)) - 1;
        else last = min(lanes_below(n, t, true, c), limit - 1);
        sum = __shfl(c.cum, max(last, 0), 64);
        token = __shfl(c.c, max(last, 0), 64);
        if (tid == 0) {
          sh.few_keep = last;
          sh.few_mass = sum;
          sh.few_token = token;
        }
      }
      __syncthreads();
      last = sh.few_keep;
      sum = sh.few_mass;
      token = sh.few_token;
    } else {
      sort_candidates(n);
      weigh(n, top, f.inv_t);
      const double t = own_target(sh.cum[n - 1]);
      if (stage == 0) last = f.k - before <= n ? f.k - before - 1 : -1;
      else if (stage == 1) last = min(count_below(n, t, false), n - 1);
      else if (stage == 2) last = count_heavy(n, f.minp, top, f.inv_t) - 1;
      else last = min(count_below(n, t, true), limit - 1);
      sum = sh.cum[max(last, 0)];
      token = sh.cand[max(last, 0)];
    }
    sum = mass_before + (last >= 0 ? sum : 0.0);
    if (stage == 0) {
      if (last >= 0) {  // (else fewer than k tokens are not masked: all of them)
        keep = f.k;
        zk = zn = sum;
        whole = bin;
      }
    } else if (stage == 3) {
      if (last >= 0) r = Answer{token, zn, true};
    } else if (before + last + 1 < keep) {
      keep = max(before + last + 1, 1);
      whole = bin;
      zn = stage == 2 ? fmax(sum, 1.0) : sum;
    }
    if (tid == 0) sh.found = kBins - 1;
    __syncthreads();
  }
  return r;
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a) {
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
  // no filter says how many tokens to collect: tally the bins while reading
  const bool binned = !greedy && !known_k && (k < vocab || p < 1.0 || minp == 0.0) &&
                      vocab <= kMaxBinVocab;
  Bins bins(vocab, inv_t);

  // ---- one reading: maxima of the parts
  float part[kParts], ev = kNegInf;
#pragma unroll
  for (int q = 0; q < kParts; ++q) part[q] = kNegInf;
  auto maxima = [&](const u32x4* r, int i0) {
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      // a vector past the end repeats the row's last one, which must not become this part's maximum
      const bool in = tid + (i0 + q) * kThreads < row.nv;
      float m4 = row.part(r[q], 0);
#pragma unroll
      for (int e = 1; e < kE; ++e) m4 = fmaxf(m4, row.part(r[q], e));
      part[q] = fmaxf(part[q], in ? m4 : kNegInf);
    }
  };
  // a logit beyond the bins (many, if T is small) is counted by its thread and added at the end
  int beyond = 0;
  auto tally_one = [&](float l) {
    // (no branch: what lies beyond goes to a place of the lane's own)
    const uint64_t at = bins.place(l);
    const bool in = (unsigned)(at >> 32) < kBins - 1;
    atomicAdd(&sh.bins[in ? (unsigned)(at >> 32) : kBins + lane], bins.tally(at));
    beyond += (int)(!in & (l > kNegInf));
  };
  auto tally_batch = [&](const u32x4* r, int i0) {
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      if (tid + (i0 + q) * kThreads < row.nv)
#pragma unroll
        for (int e = 0; e < kE; ++e) tally_one(row.plain(r[q], e));
  };
  bool bins_ready = binned;
  if (binned)
    for (int i = tid; i < kBins; i += kThreads) sh.bins[i] = 0;
  read_batches<F32>(
      row,
      [&](const u32x4* r, int i0) {
        maxima(r, i0);
        if (binned) {
          if (i0 == 0) {
            // the bins (64 T of logits) begin a margin above the largest logit of the first batch
            float m = ev;
#pragma unroll
            for (int q = 0; q < kParts; ++q) m = fmaxf(m, part[q]);
            m = block_range(m).most;
            bins_ready = m > kNegInf && bins.begin_at((double)m + fmin(12.0, 24.0 / inv_t));
          }
          if (bins_ready) tally_batch(r, i0);
        }
      },
      [&](float l, int) { ev = l; });
  if (binned && bins_ready && ev > kNegInf) tally_one(ev);
  const int ei = tid < row.extra ? row.extra_index(tid) : 0;
  float mine = ev;
#pragma unroll
  for (int s = 0; s < kParts; ++s) mine = fmaxf(mine, part[s]);
  if (tid == 0) {
    sh.count = 0;
    sh.nhits = 0;
    sh.best = vocab;
  }
  const Range range = block_range(mine);
  const float top = range.most;
  if (top == kNegInf) {  // every token is masked
    if (tid == 0) {
      a.tokens[b] = -1;
      if (a.logprob) a.logprob[b] = kNegInf;
    }
    return;
  }
  Answer r = {0, 0.0, false};
  if (!binned) {
    // ---- a bound that at least k tokens reach
    float tau = top;
    if (!greedy && known_k) {
      // the k-th largest of the maxima, by bisection over their keys: every wave counts its own.  A
      // bound that a few more reach will do.  All threads reach the least of their
      // largest ones.
      unsigned key[kParts];
#pragma unroll
      for (int q = 0; q < kParts; ++q) key[q] = to_key(part[q]);
      unsigned lo = to_key(range.least), hi = to_key(top);  // kMaxK = kThreads maxima reach the least
#pragma unroll 1
      for (int turn = 0; lo < hi; turn ^= 1) {
        const unsigned mid = lo + (hi - lo) / 2 + 1;
        int n = 0;
#pragma unroll
        for (int q = 0; q < kParts; ++q) n += __popcll(__ballot(key[q] >= mid));
        if (lane == 0) sh.wave_n[turn][tid >> 6] = n;
        __syncthreads();
        n = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) n += sh.wave_n[turn][w];
        if (n >= k) lo = mid;
        else hi = mid - 1;
        if (n >= k && n <= k + (k >> 3)) break;
      }
      // fewer maxima than k (a short row, or masked tokens): every token
      tau = lo <= to_key(kNegInf) ? kNegInf : from_key(lo);
    } else if (!greedy) {
      tau = kNegInf;
      if (p >= 1.0 && minp > 0.0 && inv_t > 0.0) {
        // every token that min_p keeps (and margins for the rounding of its weight and of this bound;
        // where T is infinite, every token that is not masked)
        const float t = (float)((double)top + (log_f64(minp) - 0x1p-52) / inv_t);
        tau = top < __builtin_inff() ? t - fabsf(t) * 1e-5f - 1e-30f : top;
      }
    }
    // ---- the tokens that reach it: the first k, every token with w >= min_p, or every token that
    // is not masked
    list_hits(part, tau);
    __syncthreads();
    collect_hits<F32>(row, ev, ei, tau, top, [](float) { return true; });
    __syncthreads();
    const int n = sh.count;
    if (n <= kCap) {
      if (greedy) {
        // the first of the tokens at the top
        for (int j = tid; j < n; j += kThreads)
          atomicMin(&sh.best, (int)(0xFFFFFFFFu - (unsigned)sh.cand[j]));
        __syncthreads();
        r = Answer{composite(top, sh.best), 1.0, true};
      } else if (n <= 64) {
        if (tid >= 64) return;
        const Few c = order_few(n, top, inv_t);
        const int kk = min(k, n);
        int keep = kk;
        if (p < 1.0) keep = min(lanes_below(kk, p * __shfl(c.cum, kk - 1, 64), false, c) + 1, kk);
        if (minp > 0.0) keep = min(keep, __popcll(__ballot(lane < n && c.w >= minp)));
        keep = max(keep, 1);
        const double zn = __shfl(c.cum, keep - 1, 64);
        const int j = lanes_below(keep, u * zn, true, c);
        r = Answer{(uint64_t)__shfl((unsigned long long)c.c, min(j, keep - 1), 64), zn, true};
      } else {
        sort_candidates(n);
        weigh(n, top, inv_t);
        const int kk = min(k, n);
        int keep = kk;
        if (p < 1.0) keep = min(count_below(kk, p * sh.cum[kk - 1], false) + 1, kk);
        if (minp > 0.0) keep = min(keep, count_heavy(n, minp, top, inv_t));
        keep = max(keep, 1);
        const double zn = sh.cum[keep - 1];
        const int j = count_below(keep, u * zn, true);
        r = Answer{sh.cand[min(j, keep - 1)], zn, true};
      }
    }
  }
  const Filters f = {greedy ? 1 : k, vocab, greedy ? 2.0 : p, greedy ? 0.0 : minp, u, inv_t};
  if (!r.found && vocab <= kMaxBinVocab && top < __builtin_inff()) {
    if (!bins_ready || __builtin_fma(-(double)top, bins.scale, bins.offset) < kOffset) {
      // too many tokens for the first way, or bins that began too low: tally from the top
      __syncthreads();
      for (int i = tid; i < kBins; i += kThreads) sh.bins[i] = 0;
      beyond = 0;
      __syncthreads();
      bins_ready = bins.begin_at((double)top);
      if (bins_ready) read_batches<F32>(row, tally_batch, [&](float l, int) { if (l > kNegInf) tally_one(l); });
    }
    if (beyond) atomicAdd(&sh.bins[kBins - 1], (unsigned long long)beyond << bins.low);
    __syncthreads();
    if (bins_ready) r = by_bins<F32>(row, f, top, bins, part, ev, ei);
  }
  if (!r.found) r = by_rank<F32>(row, f, top);
  if (tid == 0) {
    a.tokens[b] = (int)(0xFFFFFFFFu - (unsigned)r.token);
    if (a.logprob)
      a.logprob[b] = greedy ? 0.0f : (float)(log_weight(logit_of(r.token), top, inv_t) - log_f64(r.kept));
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, bool f32, hipStream_t stream) {
  if (a.rows < 1 || a.vocab < 1) return hipErrorInvalidValue;
  clear_stale_error();
  constexpr int kMost = 1 << 21;  // rows of a launch, which holds fewer than 2^32 threads
  for (int first = 0; first < a.rows; first += kMost) {
    SampleArgs part = a;
    part.rows = min(a.rows - first, kMost);
    part.logits = static_cast<const unsigned char*>(a.logits) + first * a.row_stride * (f32 ? 4 : 2);
    part.u += first;
    if (a.temperature) part.temperature += first;
    if (a.top_k) part.top_k += first;
    if (a.top_p) part.top_p += first;
    if (a.min_p) part.min_p += first;
    part.tokens += first;
    if (a.logprob) part.logprob += first;
    if (f32) hipLaunchKernelGGL(sample_kernel<true>, dim3(part.rows), dim3(kThreads), 0, stream, part);
    else hipLaunchKernelGGL(sample_kernel<false>, dim3(part.rows), dim3(kThreads), 0, stream, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bd
