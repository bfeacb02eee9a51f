// Sampling from logits with temperature, top-k, top-p and min-p.
//
// Entries are ordered by falling logit, equal ones by rising index.  With
// w_v = exp((l_v - max) / T) an entry is kept if fewer than k are before it, if
// the mass (sum of w) before it is below p times the mass of the first k, and
// if w_v >= min_p; the first always is.  The token is argmax w_v / e_v over the
// kept entries with given exponential e_v: it is drawn in proportion to w.
//
// Nothing is sorted.  What is kept is a head of the order, so only its border
// has to be found: logits are put into buckets of an eighth of T on one grid
// for the whole row, and a bucket's number and mass of entries say which one
// the border lies in.  Three launches, a fourth for probabilities:
//   scan     a slice's entries in registers: its largest, and its histogram in
//            LDS relative to that one (one atomic an entry: number and mass in
//            one word);
//   collect  adds a row's histograms, finds the border's bucket, draws among
//            the entries before it and lists those in it (the candidates);
//   finish   one workgroup a row: the border among the candidates, the token;
//   write    probabilities, where they are asked for.
//
// Whether an entry is kept depends on a sum over the whole row, and binary32
// exponentials would let one of some thousand rows keep one entry more or
// less.  So masses are computed in binary64, whose products the vector unit
// does at binary32's pace, and summed as integers, which do not depend on the
// order of the atomics: in a bucket l grid = q + f, w is exp((f - 1/2) / 8), a
// short series, times a factor of the bucket.
//
// Measured on MI355X, latency throughout (logits are read at 5 TB/s in 4 us by 64
// rows of 151,936 bf16): 1 row of 32,001: 19.4 us (scan 3.7, collect 8.0, finish 8.4);
// 64 rows of 151,936 bf16, all rules mixed: 60 us (14, 26, 17-21); 40 rows of
// 128,256 with top-p and probabilities: 64 us (9, 21, 23, write 14, which moves 41 MB).
//   scan: an LDS atomic an entry, and binary64 masses.
//   collect: the sum of the histograms is a chain of loads, exponentials and a
//     prefix sum (most of a single row's 8 us), then the logits once more, from the
//     caches; loading them a piece ahead gave nothing.
//   finish: a workgroup a row; how often it counts depends on the candidates (64
//     rows without rules: 48 us, with top-k 38, with top-p 69).
#include "attention_common.hpp"
#include "serving_args.hpp"

#include <type_traits>

namespace qlk {

constexpr int kSampleThreads = 512;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kSampleCopies = 4;         // of a histogram: lanes of equal buckets add one after the other
constexpr int kMassBits = 49;            // 16384 entries of up to e^(1/16) 2^34
constexpr uint64_t kMassMask = (uint64_t(1) << kMassBits) - 1;
constexpr double kMassOne = 17179869184.0;   // 2^34
constexpr double kLog2E = 1.44269504088896340736;

// 2^y as m 2^e with m in [0.7, 1.42): the exponential's own series (6 10^-15).
__device__ __forceinline__ double exp2_parts(double y, int* e) {
  y = fmin(fmax(y, -1000.0), 1000.0);
  const double n = rint(y), f = (y - n) * 0.69314718055994530942;
  double p = 1.0 / 39916800.0;
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  *e = (int)n;
  return p;
}

__device__ __forceinline__ double exp2_of(double y) {
  int e;
  const double m = exp2_parts(y, &e);
  return ldexp(m, e);
}

// One row's rules.
struct Rules {
  double rate;       // log2(e) / T
  double grid;       // buckets per unit of the logits: 8 / T
  int k;             // 0: off
  float p, m;        // 1, 0: off
};

__device__ __forceinline__ Rules rules_of(const SampleArgs& a, int row) {
  Rules r;
  const float t = a.temperature ? a.temperature[row] : 1.0f;
  const bool greedy = !(t > 0.0f);
  const double inv = greedy ? 1.0 : 1.0 / (double)fmaxf(t, 1e-6f);
  r.rate = inv * kLog2E;
  r.grid = 8.0 * inv;
  r.k = greedy ? 1 : a.top_k ? max(a.top_k[row], 0) : 0;
  r.p = greedy || !a.top_p ? 1.0f : a.top_p[row];
  r.m = greedy || !a.min_p ? 0.0f : a.min_p[row];
  r.p = r.p < 1.0f ? fmaxf(r.p, 0.0f) : 1.0f;  // NaN: off
  r.m = r.m > 0.0f ? fminf(r.m, 1.0f) : 0.0f;
  return r;
}

// The grid's line below a logit.  (Beyond 2^53 lines neighbouring binary32
// logits are more than 2^29 of them apart: a bucket then holds equal ones.)
__device__ __forceinline__ double line_of(float l, double grid) { return floor((double)l * grid); }

// exp((f - 1/2) / 8) in steps of 2^-34, and `above` more, for f in [0, 1): the
// polynomial that meets it at the six Chebyshev nodes (off by 3 10^-12 at most).
__device__ __forceinline__ double mass_of(double f, double above = 0.0) {
  double p = kMassOne * 2.54348632162432e-07;
  p = fma(p, f, kMassOne * 9.53864143867337e-06);
  p = fma(p, f, kMassOne * 0.0003058076755491678);
  p = fma(p, f, kMassOne * 0.007339162402444752);
  p = fma(p, f, kMassOne * 0.11742663303627268);
  return fma(p, f, kMassOne * 0.9394130628109114 + above);
}

// An entry's mass in its bucket, that of the part of l grid above the line.  The
// low bits of 2^52 + x are x rounded.
__device__ __forceinline__ uint64_t mass_word(float l, double grid) {
  const double p = mass_of(__builtin_amdgcn_fract((double)l * grid), 4503599627370496.0);
  return (uint64_t)__double_as_longlong(p) - (uint64_t(0x433) << 52);
}

// Values that order as binary32 logits do, and their inverse.
__device__ __forceinline__ uint32_t order_of(float l) {
  const uint32_t u = __float_as_uint(l);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// The place of an entry in the order: larger is earlier.
__device__ __forceinline__ uint64_t key_of(float l, int v) { return (uint64_t)order_of(l) << 32 | (0xffffffffu - (uint32_t)v); }
__device__ __forceinline__ int index_of(uint64_t key) { return (int)(0xffffffffu - (uint32_t)key); }

typedef unsigned u32x4b __attribute__((ext_vector_type(4), aligned(2)));

// 8 entries from v on (as many as there are; the others -inf).  NaN is no entry,
// and zeros are alike.
template <bool BF16>
__device__ __forceinline__ void load_logits(const SampleArgs& a, int row, int v, float (&x)[8]) {
  if (v + 8 <= a.vocab) {
    if constexpr (BF16) {
      const u32x4 t = *reinterpret_cast<const u32x4b*>(static_cast<const uint16_t*>(a.logits) + row * a.row + v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(t[i] << 16);
        x[2 * i + 1] = __uint_as_float(t[i] & 0xffff0000u);
      }
    } else {
      const f32x4u* p = reinterpret_cast<const f32x4u*>(static_cast<const float*>(a.logits) + row * a.row + v);
      const f32x4u t = p[0], u = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = t[i];
        x[4 + i] = u[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = kNegInf;
      if (v + i < a.vocab)
        x[i] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[row * a.row + v + i])
                    : static_cast<const float*>(a.logits)[row * a.row + v + i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] == x[i] ? x[i] + 0.0f : kNegInf;
}

// Where a row has +inf, that is its only value: as 0 here.
__device__ __forceinline__ float beside_inf(float l) { return l == -kNegInf ? 0.0f : kNegInf; }

// Reductions over a wave by lane shifts (v_mov_dpp: no trip to LDS), returned in
// every lane; `none` is what lanes without a neighbour add.
template <class T, class F>
__device__ __forceinline__ T wave_reduce(T v, T none, F add) {
  auto shifted = [&](auto ctrl, auto rows) {
    constexpr int C = decltype(ctrl)::value, R = decltype(rows)::value;
    if constexpr (sizeof(T) == 8) {
      const uint64_t x = __builtin_bit_cast(uint64_t, v), o = __builtin_bit_cast(uint64_t, none);
      const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)x, C, R, 0xf, false);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(o >> 32), (int)(x >> 32), C, R, 0xf, false);
      v = add(v, __builtin_bit_cast(T, (uint64_t)hi << 32 | lo));
    } else {
      v = add(v, __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), C, R, 0xf, false)));
    }
  };
  shifted(std::integral_constant<int, 0x111>(), std::integral_constant<int, 0xf>());   // row_shr 1, 2, 4, 8
  shifted(std::integral_constant<int, 0x112>(), std::integral_constant<int, 0xf>());
  shifted(std::integral_constant<int, 0x114>(), std::integral_constant<int, 0xf>());
  shifted(std::integral_constant<int, 0x118>(), std::integral_constant<int, 0xf>());
  shifted(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());   // row_bcast 15 into rows 1 and 3
  shifted(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());   // row_bcast 31 into rows 2 and 3
  if constexpr (sizeof(T) == 8) {
    const uint64_t x = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(T, (uint64_t)(uint32_t)lane_i32((int)(x >> 32), 63) << 32 | (uint32_t)lane_i32((int)x, 63));
  } else {
    return __builtin_bit_cast(T, lane_i32(__builtin_bit_cast(int, v), 63));
  }
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, kNegInf, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ uint64_t wave_max_key(uint64_t v) { return wave_reduce(v, uint64_t(0), max_u64); }
__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
  return wave_reduce(v, uint64_t(0), [](uint64_t a, uint64_t b) { return a + b; });
}

// A value that is the same in all lanes, as such (a scalar register).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float uniform(float v) { return __uint_as_float(uniform((int)__float_as_uint(v))); }
__device__ __forceinline__ double uniform(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)(uint32_t)uniform((int)(u >> 32)) << 32 | (uint32_t)uniform((int)u)));
}

// A score and its index as one word: the larger score, between equals the
// lower index.
__device__ __forceinline__ uint64_t score_of(double w, float noise, int v) {
  const float s = __fdiv_rn((float)w, noise);
  return (uint64_t)__float_as_uint(s > 0.0f ? s : 0.0f) << 32 | (0xffffffffu - (uint32_t)v);
}

// Slice blockIdx.x of row blockIdx.y; PIECES pieces of 8 entries a thread.
template <bool BF16, int PIECES>
__global__ void __launch_bounds__(kSampleThreads) sample_scan_kernel(SampleArgs a) {
  const int row = blockIdx.y, slice = blockIdx.x, first = slice * PIECES * 8 * kSampleThreads, t = threadIdx.x;
  __shared__ unsigned long long hist[kSampleBuckets * kSampleCopies];
  __shared__ float tops[kSampleWaves];
  float x[PIECES][8], top = kNegInf;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) load_logits<BF16>(a, row, first + (i * kSampleThreads + t) * 8, x[i]);
  const Rules r = rules_of(a, row);
#pragma unroll
  for (int i = 0; i < kSampleCopies; ++i) hist[i * kSampleThreads + t] = 0;
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, x[i][j]);
  top = wave_max(top);
  if ((t & 63) == 0) tops[t >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSampleWaves; ++i) top = fmaxf(top, tops[i]);
  if (t == 0) {
    a.top[(int64_t)row * a.slices + slice] = top;
    if (slice == 0) a.count[row * kSampleCountStep] = 0;
  }
  if (top == -kNegInf) {
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = beside_inf(x[i][j]);
  }
  const double line = line_of(top, r.grid);
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!(x[i][j] > kNegInf)) continue;
      const int bucket = (int)fmin(line - line_of(x[i][j], r.grid), kSampleBuckets - 1.0);
      // (the last bucket and what is beyond weigh less than 2^-90 of the largest: no mass)
      const uint64_t mass = bucket < kSampleBuckets - 1 ? mass_word(x[i][j], r.grid) : 0;
      atomicAdd(&hist[bucket * kSampleCopies + (t & (kSampleCopies - 1))], (unsigned long long)(mass + (uint64_t(1) << kMassBits)));
    }
  __syncthreads();
  uint64_t sum = 0;
#pragma unroll
  for (int i = 0; i < kSampleCopies; ++i) sum += hist[t * kSampleCopies + i];
  a.hist[((int64_t)row * a.slices + slice) * kSampleBuckets + t] = sum;
}

// Sums over the threads before this one, in their order.
struct Before {
  int count;
  double mass;
};

// What a row's histograms say; the same in every thread of its workgroups.
__device__ __forceinline__ SampleRow settle_row(const SampleArgs& a, int row, const Rules& r) {
  static_assert(kSampleThreads == kSampleBuckets, "a thread a bucket");
  constexpr int W = kSampleWaves, U = 10;
  __shared__ int shift[kSampleThreads];
  __shared__ float tops[W];
  __shared__ Before waves[W];
  __shared__ int k_bucket, p_lo, p_hi, lo_count;
  __shared__ double k_mass[2], lo_mass;
  const int b = threadIdx.x, lane = b & 63, wave = b >> 6;
  const float* part = a.top + (int64_t)row * a.slices;
  SampleRow s;
  float mine = b < a.slices ? part[b] : kNegInf, top = mine;
  for (int i = b + kSampleThreads; i < a.slices; i += kSampleThreads) top = fmaxf(top, part[i]);
  top = wave_max(top);
  if (lane == 0) tops[wave] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) top = fmaxf(top, tops[i]);
  top = uniform(top);
  s.inf = top == -kNegInf;
  s.top = s.inf ? 0.0f : top;
  s.line = uniform(line_of(s.top, r.grid));
  // a thread adds one bucket over the slices
  int count = 0;
  uint64_t sum = 0;
  for (int i0 = 0; i0 < a.slices; i0 += kSampleThreads) {
    if (i0) {
      __syncthreads();
      mine = i0 + b < a.slices ? part[i0 + b] : kNegInf;
    }
    // slices without an entry, or without +inf beside one that has it: none
    const bool there = s.inf ? mine == -kNegInf : mine > kNegInf;
    shift[b] = there ? (int)fmin(s.line - line_of(s.inf ? 0.0f : mine, r.grid), (double)kSampleBuckets) : 2 * kSampleBuckets;
    __syncthreads();
    const int n = min(kSampleThreads, a.slices - i0);
    const uint64_t* h = a.hist + ((int64_t)row * a.slices + i0) * kSampleBuckets;
    for (int i = 0; i < n; i += U) {
      uint64_t x[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int at = b - shift[min(i + k, n - 1)];
        x[k] = i + k < n && at >= 0 && at < kSampleBuckets - 1 ? h[(int64_t)(i + k) * kSampleBuckets + at] : 0;
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        count += (int)(x[k] >> kMassBits);
        sum += x[k] & kMassMask;
      }
    }
  }
  // w of the middle of bucket b is exp((1/2 - f - b) / 8), f of the largest
  const double middle = (0.5 - __builtin_amdgcn_fract((double)s.top * r.grid) - b) * (0.125 * kLog2E);
  double mass = sum ? (double)sum / kMassOne * exp2_of(middle) : 0.0;
  int c = count;
  double m = mass;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int c2 = __shfl_up(c, o, 64);
    const double m2 = __shfl_up(m, o, 64);
    if (lane >= o) {
      c += c2;
      m += m2;
    }
  }
  if (lane == 63) waves[wave] = Before{c, m};
  if (b == 0) {
    k_bucket = p_lo = p_hi = kSampleBuckets - 1;
    k_mass[0] = k_mass[1] = -1.0;
  }
  __syncthreads();
  Before before = {0, 0.0}, all = {0, 0.0};
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w == wave) before = all;
    all.count += waves[w].count;
    all.mass += waves[w].mass;
  }
  const double end = before.mass + m;
  before.count += c - count;
  before.mass = fmax(end - mass, 0.0);
  // the last bucket holds what all others do not: no mass, and any number of entries
  const bool p_on = r.p < 1.0f, m_on = r.m > 0.0f;
  s.all = all.mass;
  if (r.k > 0 && before.count < r.k && before.count + count >= r.k) {
    k_bucket = b;
    k_mass[0] = before.mass;
    k_mass[1] = end;
  }
  __syncthreads();
  // the border lies where the mass reaches p of the first k's, which is known up to the k-th's bucket: the first
  // bucket that reaches it (rounding of these sums allowed for).  Ends are compared with the limits, and with nothing
  // else: a bucket's start is worked out apart from the end before it, and a limit may lie between the two.
  const bool k_found = k_mass[1] >= 0.0;
  if (p_on) {
    const double least = (double)r.p * (k_found ? k_mass[0] : all.mass) * (1.0 - 1e-10),
                 most = (double)r.p * (k_found ? k_mass[1] : all.mass) * (1.0 + 1e-10);
    const uint64_t reach = __ballot(end >= least), pass = __ballot(end >= most);
    if (lane == 0) {
      if (reach) atomicMin(&p_lo, b + __ffsll((unsigned long long)reach) - 1);
      if (pass) atomicMin(&p_hi, b + __ffsll((unsigned long long)pass) - 1);
    }
  }
  __syncthreads();
  // a k beyond the entries that have mass cuts nothing that top-p has not
  s.k = p_on && !k_found ? 0 : r.k;
  s.lo = kSampleBuckets;
  s.hi = kSampleBuckets - 1;
  if (s.k) s.lo = s.hi = k_bucket;
  if (p_on) {
    s.lo = min(s.lo, p_lo);
    if (!s.k) s.hi = min(s.hi, p_hi);
  }
  if (m_on) {
    const float at = floorf(-8.0f * logf(r.m));
    s.lo = min(s.lo, (int)fminf(fmaxf(at - 1.0f, 0.0f), kSampleBuckets - 1.0f));
    if (!(s.k && p_on)) s.hi = min(s.hi, (int)fminf(at + 2.0f, kSampleBuckets - 1.0f));
  }
  if (b == s.lo) {
    lo_count = before.count;
    lo_mass = before.mass;
  }
  if (s.lo == kSampleBuckets && b == 0) {
    lo_count = all.count;
    lo_mass = all.mass;
  }
  __syncthreads();
  s.lo = uniform(s.lo);
  s.hi = uniform(s.hi);
  s.k = uniform(s.k);
  s.all = uniform(s.all);
  s.count = uniform(lo_count);
  s.mass = uniform(lo_mass);
  s.unit = (0.5 - __builtin_amdgcn_fract((double)s.top * r.grid) - s.lo) * (0.125 * kLog2E);
  return s;
}

// An entry's weight, relative to the largest's.
__device__ __forceinline__ double weight_of(float l, float top, double rate) {
  return exp2_of(((double)l - (double)top) * rate);
}
// A candidate's mass, in steps of 2^-34 of the middle of the first candidates'
// bucket: in that one the number that the histogram has.
__device__ __forceinline__ uint64_t cand_mass(float l, const SampleRow& s, double grid) {
  const double below = s.line - line_of(l, grid) - s.lo;
  const uint64_t m = mass_word(l, grid);
  return below == 0.0 ? m : (uint64_t)rint((double)m * exp2_of(-below * (0.125 * kLog2E)));
}

// The best score among many entries, a wave together: few can be the best one,
// so binary32's exponential and reciprocal pick out those that come within 10^-4
// of the best so far (what these can be off by).  Both end in 0 below 2^-126:
// weights are taken 2^60 times as large, which reaches below binary32's smallest
// number, and only bounds that no such reciprocal passes are made.
struct BestScore {
  uint64_t best = 0;   // this lane's
  float bound = 0.0f;  // of the wave's, 2^60 times
  __device__ __forceinline__ void add(const bool (&in)[4], const uint64_t (&key)[4], const float (&noise)[4], float top, double rate) {
    float about[4], most = 0.0f;
    bool near = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      about[u] = __builtin_amdgcn_exp2f(fmaf(logit_of(key[u]) - top, (float)rate, 60.0f)) * __builtin_amdgcn_rcpf(noise[u]);
      near |= in[u] && !(about[u] < bound);
      most = in[u] ? fmaxf(most, about[u]) : most;
    }
    if (!__any(near)) return;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (in[u] && !(about[u] < bound)) {
        const uint64_t score = score_of(weight_of(logit_of(key[u]), top, rate), noise[u], index_of(key[u]));
        best = score > best ? score : best;
      }
    most = wave_max(most) * (1.0f - 1e-4f);
    bound = most > 0x1p-60f && most < 0x1p120f ? fmaxf(bound, most) : bound;
  }
};

constexpr int kWaveList = 640;   // entries that a wave notes before it works on them: a piece's 512 and some more

template <bool BF16, int PIECES>
__global__ void __launch_bounds__(kSampleThreads, 6) sample_collect_kernel(SampleArgs a) {
  constexpr int E = PIECES * 8 * kSampleThreads;
  const int row = blockIdx.y, slice = blockIdx.x, first = slice * E, t = threadIdx.x, lane = t & 63;
  // a wave's surely kept entries from the front, its candidates from the back
  __shared__ uint64_t lists[kSampleWaves][kWaveList], bests[kSampleWaves];
  __shared__ int left[kSampleWaves], row_base;
  float x[8];
  load_logits<BF16>(a, row, first + t * 8, x);
  const Rules r = rules_of(a, row);
  const SampleRow s = settle_row(a, row, r);
  if (slice == 0 && t == 0) a.state[row] = s;
  if (s.top == kNegInf) return;   // no entry at all
  // (no buckets after the last one: the comparisons are with lines as they lie)
  const double sure = s.lo == kSampleBuckets ? __builtin_huge_val() : s.lo;
  const double maybe = s.hi == kSampleBuckets - 1 ? __builtin_huge_val() : s.hi;
  uint64_t* list = lists[t >> 6];
  int found[2] = {0, 0};   // entries of the wave's list
  BestScore score;
#pragma unroll 1
  for (int i = 0; i < PIECES; ++i) {
    const int v = first + (i * kSampleThreads + t) * 8;
    unsigned bits[2] = {0, 0};
    if (i) load_logits<BF16>(a, row, v, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (s.inf) x[j] = beside_inf(x[j]);
      const double below = s.line - line_of(x[j], r.grid);
      const bool there = x[j] > kNegInf;
      bits[0] |= (unsigned)(there && below < sure) << j;
      bits[1] |= (unsigned)(there && below >= sure && below <= maybe) << j;
    }
    const float* noise = a.noise + (int64_t)row * a.vocab;
    // places in the list: sums over the lanes
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      if (!__any(bits[kind] != 0)) continue;
      const int n = __popc(bits[kind]), upto = inclusive_sum(n);
      int at = found[kind] + upto - n;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (bits[kind] >> j & 1) {
          list[kind ? kWaveList - 1 - at : at] = key_of(x[j], v + j);
          ++at;
        }
      found[kind] += lane_i32(upto, 63);
    }
    const bool end = i + 1 == PIECES;
    if (!end && found[0] + found[1] <= kWaveList - 512) continue;
    // the candidates' place in the row's list: as a rule all of the workgroup's at the end, by one atomic (those of one
    // address come one after the other; 8 rows of 151,936: 71 us with one a wave)
    const bool flush = end || found[1] > 128;
    int base = 0;
    if (end) {
      if (lane == 0) left[t >> 6] = found[1];
      __syncthreads();
      int all = 0;
#pragma unroll
      for (int w = 0; w < kSampleWaves; ++w) {
        base += w < (t >> 6) ? left[w] : 0;
        all += left[w];
      }
      if (t == 0) row_base = all ? atomicAdd(&a.count[row * kSampleCountStep], all) : 0;
    } else if (flush && lane == 0) {
      base = atomicAdd(&a.count[row * kSampleCountStep], found[1]);
    }
#pragma unroll 1
    for (int k = 0; k < found[0]; k += 256) {
      uint64_t key[4];
      float e[4];
      bool in[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        in[u] = k + 64 * u + lane < found[0];
        key[u] = list[min(k + 64 * u + lane, found[0] - 1)];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) e[u] = noise[index_of(key[u])];
      score.add(in, key, e, s.top, r.rate);
    }
    found[0] = 0;
    if (end) {
      __syncthreads();
      base += row_base;
    }
    if (flush) {
      base = lane_i32(base, 0);
#pragma unroll 1
      for (int k = lane; k < found[1]; k += 64) a.cand[(int64_t)row * a.vocab + base + k] = list[kWaveList - 1 - k];
      found[1] = 0;
    }
  }
  const uint64_t best = wave_max_key(score.best);
  if (lane == 0) bests[t >> 6] = best;
  __syncthreads();
  if (t < 64) {
    const uint64_t all = wave_max_key(bests[t % kSampleWaves]);
    if (t == 0) a.best[(int64_t)row * a.slices + slice] = all;
  }
}

constexpr int kFinishLast = 64;     // candidates that one wave orders by itself
constexpr int kFinishParts = 256;   // parts that a range of candidates is counted into
constexpr int kFinishCopies = 2;    // of the counts: lanes of equal parts add one after the other
constexpr int kFinishThreads = 512;
constexpr int kFinishWaves = kFinishThreads / 64;
constexpr int kHeld = 16384;        // candidates that LDS holds

struct FinishSpace {
  uint64_t held[kHeld];
  unsigned long long mass[kFinishCopies][kFinishParts];
  unsigned count[kFinishCopies][kFinishParts];
  unsigned long long keys[kFinishLast], own[kFinishLast], mat[kFinishLast];   // what is left: masses, and those before
  int at[kFinishLast];
  uint64_t tops[kFinishWaves], sums[kFinishWaves];
  uint64_t b_mass;
  int b_count, part, listed;
};

// f(keys, which are there) for the candidates of a row, four a lane at a time
// with all lanes of a wave together: from LDS, where they are loaded to in turns
// if they are very many.
constexpr int kEach = 4;
template <class F>
__device__ __forceinline__ void each(const uint64_t* list, int n, uint64_t* held, bool loaded, F f) {
#pragma unroll 1
  for (int c0 = 0; c0 < n; c0 += kHeld) {
    const int m = min(n - c0, kHeld);
    if (!loaded) {
      __syncthreads();
#pragma unroll 4
      for (int i = threadIdx.x; i < m; i += kFinishThreads) held[i] = list[c0 + i];
      __syncthreads();
    }
#pragma unroll 1
    for (int i0 = 0; i0 < m; i0 += kEach * kFinishThreads) {
      uint64_t key[kEach];
      bool in[kEach];
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        const int i = i0 + u * kFinishThreads + (int)threadIdx.x;
        in[u] = i < m;
        key[u] = held[min(i, m - 1)];
      }
      f(key, in);
    }
  }
}

// The token of row blockIdx.x.  The border among the candidates is looked for by rank (top-k), then by
// mass (top-p): the last one that is kept has fewer than `most` of them before
// it, or less than `limit` of their mass.  They are counted into parts of their
// range, again within the part that the border lies in, until one wave orders
// what is left.  (The code is run once a row, from a cold instruction cache: it
// is kept short.  Unrolled to five times its length it took 2 to 3 times as long.)
template <bool BF16>
__global__ void __launch_bounds__(kFinishThreads) sample_finish_kernel(SampleArgs a) {
  __shared__ FinishSpace sp;
  const int row = blockIdx.x, t = threadIdx.x, copy = t % kFinishCopies;
  const SampleRow s = a.state[row];
  if (s.top == kNegInf) {   // no entry at all
    if (t == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = kNegInf;
    }
    return;
  }
  const Rules r = rules_of(a, row);
  const uint64_t* list = a.cand + (int64_t)row * a.vocab;
  const int n = a.count[row * kSampleCountStep];
  uint64_t best = 0;
  for (int i = t; i < a.slices; i += kFinishThreads) best = max_u64(best, a.best[(int64_t)row * a.slices + i]);
  const bool held = n <= kHeld;
  if (held) {
#pragma unroll 4
    for (int i = t; i < n; i += kFinishThreads) sp.held[i] = list[i];
    __syncthreads();
  }
  const double step = exp2_of(s.unit) / kMassOne;   // of candidates' masses
  // a mass that reaches the limit but for these products' rounding does; the first entry is kept whatever it is
  double limit = (double)r.p * s.all;
  uint64_t least = 0, upto = 0;   // smallest kept candidate, and the mass up to it
#pragma unroll 1
  for (int by_mass = 0; by_mass < 2; ++by_mass) {
    if (n == 0 || !(by_mass ? r.p < 1.0f : s.k > 0)) continue;
    const int most = s.k - s.count;
    if (by_mass) {
      limit = (limit * (1.0 - 1e-13) - s.mass) / step;
      if (s.count == 0) limit = fmax(limit, 0.5);
    }
    // the range of keys that the border is among: at first the candidates' buckets and a line more to each side
    // (rounding to binary32 passes no logit)
    uint64_t hi = key_of((float)((s.line - s.lo + 2.0) / r.grid), 0), lo = 0;
    if (s.hi < kSampleBuckets - 1) lo = key_of((float)((s.line - s.hi - 1.0) / r.grid), 0) & ~uint64_t(0xffffffff);
    int before = 0, inside = n;   // candidates before that range, and in it
    uint64_t before_mass = 0;
#pragma unroll 1
    while (inside > kFinishLast) {
      if (t == 0) sp.part = -1;
      if (t < kFinishCopies * kFinishParts) (&sp.mass[0][0])[t] = (&sp.count[0][0])[t] = 0;
      __syncthreads();
      const int shift = max(0, 56 - __clzll((long long)(hi - lo)));
      each(list, n, sp.held, held, [&](uint64_t (&key)[kEach], bool (&there)[kEach]) {
        uint64_t mass[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) mass[u] = cand_mass(logit_of(key[u]), s, r.grid);
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
          const uint64_t k = key[u];
          const bool in = there[u] && k >= lo && k <= hi;
          const int i = (int)((hi - k) >> shift);
          if (in) {
            atomicAdd(&sp.count[copy][i], 1u);
            atomicAdd(&sp.mass[copy][i], (unsigned long long)mass[u]);
          }
        }
      });
      __syncthreads();
      // wave 0: the last part whose first entry is kept, four of them a lane
      if (t < 64) {
        constexpr int L = kFinishParts / 64;
        int c[L], sum = 0;
        uint64_t m[L], msum = 0;
#pragma unroll
        for (int i = 0; i < L; ++i) {
          c[i] = (int)(sp.count[0][L * t + i] + sp.count[1][L * t + i]);
          m[i] = sp.mass[0][L * t + i] + sp.mass[1][L * t + i];
          sum += c[i];
          msum += m[i];
        }
        int at = sum;
        uint64_t mat = msum;
#pragma unroll 1
        for (int o = 1; o < 64; o <<= 1) {
          const int x = __shfl_up(at, o, 64);
          const uint64_t y = (uint64_t)__shfl_up((unsigned long long)mat, o, 64);
          if (t >= o) {
            at += x;
            mat += y;
          }
        }
        at += before - sum;
        mat += before_mass - msum;
        int mine = -1, mine_at = 0;
        uint64_t mine_mass = 0;
#pragma unroll
        for (int i = 0; i < L; ++i) {
          if (c[i] > 0 && (by_mass ? (double)mat < limit : at < most)) {
            mine = L * t + i;
            mine_at = at;
            mine_mass = mat;
          }
          at += c[i];
          mat += m[i];
        }
        const uint64_t any = __ballot(mine >= 0);
        if (any && t == 63 - __clzll((long long)any)) {
          sp.part = mine;
          sp.b_count = mine_at;
          sp.b_mass = mine_mass;
        }
      }
      __syncthreads();
      const int p = sp.part;
      if (p < 0) {   // not even the first one is kept
        inside = 0;
      } else {
        before = sp.b_count;
        before_mass = sp.b_mass;
        inside = (int)(sp.count[0][p] + sp.count[1][p]);
        const uint64_t top = hi - ((uint64_t)p << shift), wide = (uint64_t(1) << shift) - 1;
        lo = top - lo > wide ? top - wide : lo;
        hi = top;
        // the ends of the range come to the next keys that there can be: bf16 logits have but a few values (their
        // orders end in 16 zeros, below 0 ones), equal logits the vocabulary's indices
        uint32_t l = (uint32_t)(lo >> 32), h = (uint32_t)(hi >> 32);
        if (BF16) {
          l = l & 0x80000000u ? (l + 0xffffu) & 0xffff0000u : l | 0xffffu;
          h = h & 0x80000000u ? h & 0xffff0000u : ((h + 1u) & 0xffff0000u) - 1u;
        }
        lo = max_u64(lo, (uint64_t)l << 32 | (0xffffffffu - (uint32_t)(a.vocab - 1)));
        hi = ~max_u64(~hi, ~((uint64_t)h << 32 | 0xffffffffu));
      }
      __syncthreads();
    }
    if (t == 0) sp.listed = 0;
    __syncthreads();
    if (inside > 0)
      each(list, n, sp.held, held, [&](uint64_t (&key)[kEach], bool (&there)[kEach]) {
#pragma unroll
        for (int u = 0; u < kEach; ++u)
          if (there[u] && key[u] >= lo && key[u] <= hi) sp.keys[atomicAdd(&sp.listed, 1)] = key[u];
      });
    __syncthreads();
    // an entry a lane in every wave, which compares with its share of the entries
    const int m = uniform(sp.listed), lane = t & 63;
    const uint64_t key = lane < m ? sp.keys[lane] : 0, mass = lane < m ? cand_mass(logit_of(key), s, r.grid) : 0;
    if (t < 64) {
      sp.own[lane] = mass;
      sp.mat[lane] = before_mass;
      sp.at[lane] = before;
    }
    __syncthreads();
    int ahead = 0;
    uint64_t ahead_mass = 0;
#pragma unroll 2
    for (int j = t >> 6; j < m; j += kFinishWaves) {
      const bool first = sp.keys[j] > key;
      ahead += first;
      ahead_mass += first ? sp.own[j] : 0;
    }
    if (ahead) {
      atomicAdd(&sp.at[lane], ahead);
      atomicAdd(&sp.mat[lane], (unsigned long long)ahead_mass);
    }
    __syncthreads();
    const int at = sp.at[lane];
    const uint64_t mat = sp.mat[lane];
    const bool kept = lane < m && (by_mass ? (double)mat < limit : at < most);
    const uint64_t last = ~wave_max_key(kept ? ~key : 0);   // the smallest kept key; none: all ones
    upto = wave_max_key(kept ? mat + mass : before_mass);
    if (!by_mass) limit = (double)r.p * (s.mass + (double)upto * step);
    least = last > least ? last : least;
    __syncthreads();
  }
  // the kept candidates' scores; their mass anew where min-p drops some
  uint64_t sum = 0;
  BestScore score;
  const float* noise = a.noise + (int64_t)row * a.vocab;
  each(list, n, sp.held, held, [&](uint64_t (&key)[kEach], bool (&there)[kEach]) {
    float e[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      there[u] = there[u] && key[u] >= least;
      e[u] = there[u] ? noise[index_of(key[u])] : 1.0f;
    }
    if (r.m > 0.0f) {
#pragma unroll
      for (int u = 0; u < kEach; ++u) {
        there[u] = there[u] && weight_of(logit_of(key[u]), s.top, r.rate) >= (double)r.m;
        if (there[u]) sum += cand_mass(logit_of(key[u]), s, r.grid);
      }
    }
    score.add(there, key, e, s.top, r.rate);
  });
  best = score.best > best ? score.best : best;
  best = wave_max_key(best);
  sum = wave_sum_u64(sum);
  if ((t & 63) == 0) {
    sp.tops[t >> 6] = best;
    sp.sums[t >> 6] = sum;
  }
  __syncthreads();
  if (t == 0) {
    for (int i = 1; i < kFinishWaves; ++i) {
      best = sp.tops[i] > best ? sp.tops[i] : best;
      sum += sp.sums[i];
    }
    const double total = s.mass + (double)(r.m > 0.0f ? sum : upto) * step;
    const int v = index_of(best);
    a.tokens[row] = v;
    if (a.logprobs) {
      const int64_t at = row * a.row + v;
      const float l = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
      a.logprobs[row] = (float)log(weight_of(s.inf ? 0.0f : l, s.top, r.rate) / total);
    }
    a.state[row].total = total;
    a.state[row].least = least;
  }
}

constexpr int kWriteThreads = 256;

// Probabilities: w over the mass of the kept entries.
//
// w of (l - top) grid = n + f is exp((f - 1/2) / 8), the series of mass_word, times
// exp((n + 1/2) / 8) in two factors, of n / 32 and n % 32, that a workgroup works out once:
// half the binary64 operations of an exponential of each entry's own (40 rows of 128,256,
// top-p: 14.3 us, 15.9 so).
template <bool BF16>
__global__ void __launch_bounds__(kWriteThreads) sample_write_kernel(SampleArgs a) {
  const int row = blockIdx.y, t = threadIdx.x, v = ((int)blockIdx.x * kWriteThreads + t) * 8;
  __shared__ double factors[48];   // of 32 k lines below (k 0 .. 15), over the total; of 0 .. 31 lines
  float x[8], p[8];
  if (v < a.vocab) load_logits<BF16>(a, row, v, x);
  const SampleRow s = a.state[row];
  const Rules r = rules_of(a, row);
  const double per = 1.0 / s.total;
  if (t < 48) {
    const double f = exp2_of((t < 16 ? -32.0 * t : 16.5 - t) * (0.125 * kLog2E));
    factors[t] = t < 16 ? f * (per / kMassOne) : f;
  }
  __syncthreads();
  if (v >= a.vocab) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j] = 0.0f;
    if (s.inf) x[j] = beside_inf(x[j]);
    if (!(x[j] > kNegInf)) continue;
    const double below = s.line - line_of(x[j], r.grid);
    const bool in = below < s.lo || s.lo == kSampleBuckets;
    if (in || ((below <= s.hi || s.hi == kSampleBuckets - 1) && key_of(x[j], v + j) >= s.least)) {
      const double d = ((double)x[j] - (double)s.top) * r.grid, n = floor(d);
      if (n > -(double)kSampleBuckets && (in || !(r.m > 0.0f))) {
        const int k = (int)-n;
        p[j] = (float)(mass_of(d - n) * (factors[k / 32] * factors[16 + k % 32]));
      } else {
        const double w = weight_of(x[j], s.top, r.rate);
        if (in || w >= (double)r.m) p[j] = (float)(w * per);
      }
    }
  }
  float* out = a.probs + (int64_t)row * a.vocab + v;
  if (v + 8 <= a.vocab) {
    reinterpret_cast<f32x4u*>(out)[0] = f32x4u{p[0], p[1], p[2], p[3]};
    reinterpret_cast<f32x4u*>(out)[1] = f32x4u{p[4], p[5], p[6], p[7]};
  } else {
    for (int j = 0; v + j < a.vocab; ++j) out[j] = p[j];
  }
}

template <bool BF16, int PIECES>
static hipError_t launch_rows(const SampleArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.slices, (unsigned)a.rows);
  hipLaunchKernelGGL((sample_scan_kernel<BF16, PIECES>), grid, dim3(kSampleThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((sample_collect_kernel<BF16, PIECES>), grid, dim3(kSampleThreads), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((sample_finish_kernel<BF16>), dim3((unsigned)a.rows), dim3(kFinishThreads), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess || !a.probs) return e;
  const int per = 8 * kWriteThreads;
  hipLaunchKernelGGL((sample_write_kernel<BF16>), dim3((unsigned)((a.vocab + per - 1) / per), (unsigned)a.rows),
                     dim3(kWriteThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_sample(const SampleArgs& a, bool bf16, hipStream_t s) {
  constexpr int WIDE = kSampleWide / (8 * kSampleThreads), NARROW = kSampleNarrow / (8 * kSampleThreads);
  if (a.entries == kSampleWide) return bf16 ? launch_rows<true, WIDE>(a, s) : launch_rows<false, WIDE>(a, s);
  if (a.entries == kSampleWide / 2) return bf16 ? launch_rows<true, WIDE / 2>(a, s) : launch_rows<false, WIDE / 2>(a, s);
  return bf16 ? launch_rows<true, NARROW>(a, s) : launch_rows<false, NARROW>(a, s);
}

}  // namespace qlk
