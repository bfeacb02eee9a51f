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
// the border lies in.  Four launches:
//   scan     a slice's entries in registers: its largest, and its histogram in
//            LDS relative to that one (one atomic an entry: number and mass in
//            one word);
//   collect  adds a row's histograms, finds the border's bucket, draws among
//            the entries before it and lists those in it (the candidates);
//   finish   one workgroup a row: the border among the candidates, the token;
//   write    probabilities, where they are asked for.
//
// Mass is a sum of integers, w in steps of 2^-36 of a slice's largest: sums do
// not depend on the order of the atomics.  w itself is computed in binary64
// (10^-11): whether an entry is kept depends on a sum over the whole row, and
// binary32 exponentials would let one of some thousand rows keep one entry
// more or less.  The vector unit does binary64 products at binary32's pace.
#include "attention_common.hpp"
#include "serving_args.hpp"

namespace qlk {

constexpr int kSampleThreads = 256;
constexpr int kMassBits = 50;
constexpr uint64_t kMassMask = (uint64_t(1) << kMassBits) - 1;
constexpr int kMassScale = 36;   // w in steps of 2^-36

// 2^y for y <= 0 as m 2^e with m in [0.7, 1.42): the exponential's own series.
__device__ __forceinline__ double exp2_parts(double y, int* e) {
  y = fmax(y, -1000.0);
  const double n = rint(y), f = (y - n) * 0.69314718055994530942;
  double p = 1.0 / 362880.0;
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

// An entry's weight relative to `top`: 1 for top itself (also where that is
// infinite), 0 for what is infinitely far from it.
__device__ __forceinline__ double weight_of(float l, float top, double rate) {
  int e;
  const double m = exp2_parts(((double)l - (double)top) * rate, &e);
  return l == top ? 1.0 : ldexp(m, e);
}

// The same in steps of 2^-36, rounded to nearest (the low bits of 2^52 + w).
__device__ __forceinline__ uint64_t mass_of(float l, float top, double rate) {
  const double w = ldexp(weight_of(l, top, rate), kMassScale) + 4503599627370496.0;
  return (uint64_t)__double_as_longlong(w) & ((uint64_t(1) << 52) - 1);
}

// One row's rules.
struct Rules {
  double rate;       // log2(e) / T
  float grid;        // buckets per unit of the logits
  float span;        // buckets an e-fold of w takes
  int k;             // 0: off
  float p, m;        // 1, 0: off
  bool greedy;
};

__device__ __forceinline__ Rules rules_of(const SampleArgs& a, int row) {
  Rules r;
  const float t = a.temperature ? a.temperature[row] : 1.0f;
  r.greedy = !(t > 0.0f);
  const double inv = r.greedy ? 1.0 : 1.0 / (double)t;
  r.rate = inv * 1.44269504088896340736;
  // an eighth of T; wider where logits of up to 10^4 would leave 2^23 buckets
  r.grid = (float)fmin(8.0 * inv, 800.0);
  r.span = r.greedy ? r.grid : r.grid * t;
  r.k = r.greedy ? 1 : a.top_k ? a.top_k[row] : 0;
  r.p = r.greedy || !a.top_p ? 1.0f : a.top_p[row];
  r.m = r.greedy || !a.min_p ? 0.0f : a.min_p[row];
  r.k = max(r.k, 0);
  r.p = r.p < 1.0f ? r.p : 1.0f;               // NaN: off
  r.m = r.m > 0.0f ? fminf(r.m, 1.0f) : 0.0f;
  return r;
}

__device__ __forceinline__ int bucket_of(float l, float grid) {
  return (int)fminf(fmaxf(floorf(__fmul_rn(l, grid)), -8388608.0f), 8388608.0f);
}

// Values that order as binary32 logits do, and their inverse.
__device__ __forceinline__ uint32_t order_of(float l) {
  const uint32_t u = __float_as_uint(l);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// The place of an entry in the order: larger is earlier.
__device__ __forceinline__ uint64_t key_of(float l, int v) { return (uint64_t)order_of(l) << 32 | (0xffffffffu - (uint32_t)v); }

typedef unsigned u32x4b __attribute__((ext_vector_type(4), aligned(2)));

// N entries from v on (as many as there are; the others -inf).  NaN is no entry,
// and zeros are alike.
template <bool BF16, int N>
__device__ __forceinline__ void load_logits(const SampleArgs& a, int row, int v, float (&x)[N]) {
  static_assert(N == 8, "two or one 16-byte loads");
  if (v + N <= a.vocab) {
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
    for (int i = 0; i < N; ++i) {
      x[i] = kNegInf;
      if (v + i < a.vocab)
        x[i] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[row * a.row + v + i])
                    : static_cast<const float*>(a.logits)[row * a.row + v + i];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = x[i] == x[i] ? x[i] + 0.0f : kNegInf;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ uint64_t wave_max_key(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t w = (uint64_t)__shfl_xor((unsigned long long)v, o, 64);
    v = v > w ? v : w;
  }
  return v;
}
__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += (uint64_t)__shfl_xor((unsigned long long)v, o, 64);
  return v;
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
  const int row = blockIdx.y, slice = blockIdx.x, first = slice * PIECES * 8 * kSampleThreads;
  __shared__ unsigned long long hist[kSampleBuckets];
  __shared__ float tops[kSampleThreads / 64];
  __shared__ unsigned long long all;
  float x[PIECES][8], top = kNegInf;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) load_logits<BF16>(a, row, first + (i * kSampleThreads + (int)threadIdx.x) * 8, x[i]);
  const Rules r = rules_of(a, row);
  hist[threadIdx.x] = 0;
  if (threadIdx.x == 0) all = 0;
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, x[i][j]);
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSampleThreads / 64; ++i) top = fmaxf(top, tops[i]);
  const int most = bucket_of(top, r.grid);
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (x[i][j] > kNegInf)
        atomicAdd(&hist[min(most - bucket_of(x[i][j], r.grid), kSampleBuckets - 1)],
                  (unsigned long long)(uint64_t(1) << kMassBits | mass_of(x[i][j], top, r.rate)));
  __syncthreads();
  const uint64_t mine = hist[threadIdx.x], sum = wave_sum_u64(mine);
  const int64_t at = (int64_t)row * a.slices + slice;
  a.hist[at * kSampleBuckets + threadIdx.x] = mine;
  if ((threadIdx.x & 63) == 0) atomicAdd(&all, (unsigned long long)sum);
  __syncthreads();
  if (threadIdx.x == 0) a.slice[at] = SampleSlice{top, most, all};
}

// Sums over the threads before this one, in their order.
struct Before {
  int count;
  double mass;
};
__device__ __forceinline__ Before sum_before(int count, double mass, Before* waves) {
  const int lane = threadIdx.x & 63;
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
  if (lane == 63) waves[threadIdx.x >> 6] = Before{c, m};
  __syncthreads();
  Before b = {c - count, m - mass};
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) {
    b.count += waves[w].count;
    b.mass += waves[w].mass;
  }
  return b;
}

// What the row's histograms say; the same in every thread of every workgroup.
__device__ __forceinline__ SampleRow settle_row(const SampleArgs& a, int row, const Rules& r) {
  static_assert(kSampleThreads == kSampleBuckets, "a thread a bucket");
  __shared__ double scale[kSampleThreads];
  __shared__ int shift[kSampleThreads];
  __shared__ float tops[kSampleThreads / 64];
  __shared__ Before waves[kSampleThreads / 64];
  __shared__ int all_count, k_bucket, p_lo, p_hi, lo_count;
  __shared__ double all_mass, k_mass[2], lo_mass;
  const int b = threadIdx.x;
  const SampleSlice* part = a.slice + (int64_t)row * a.slices;
  SampleRow s;
  float top = kNegInf;
  for (int i = b; i < a.slices; i += kSampleThreads) top = fmaxf(top, part[i].top);
  top = wave_max(top);
  if ((b & 63) == 0) tops[b >> 6] = top;
  __syncthreads();
  for (int i = 0; i < kSampleThreads / 64; ++i) top = fmaxf(top, tops[i]);
  s.top = top;
  s.bucket = bucket_of(top, r.grid);
  // a thread adds one bucket over the slices; the last one, what is left of all
  int count = 0, all_c = 0;
  double mass = 0.0, all_m = 0.0;
  for (int i0 = 0; i0 < a.slices; i0 += kSampleThreads) {
    __syncthreads();
    if (i0 + b < a.slices) {
      const SampleSlice p = part[i0 + b];
      scale[b] = p.top > kNegInf ? ldexp(weight_of(p.top, top, r.rate), -kMassScale) : 0.0;
      shift[b] = p.top > kNegInf ? s.bucket - p.bucket : kSampleBuckets;
    }
    __syncthreads();
    const int n = min(kSampleThreads, a.slices - i0);
    const uint64_t* h = a.hist + ((int64_t)row * a.slices + i0) * kSampleBuckets;
    for (int i = 0; i < n; ++i) {
      const int at = b - shift[i];
      uint64_t x = 0;
      if (b == kSampleBuckets - 1)
        x = part[i0 + i].all;
      else if (at >= 0)
        x = h[(int64_t)i * kSampleBuckets + at];
      count += (int)(x >> kMassBits);
      mass += (double)(x & kMassMask) * scale[i];
    }
  }
  if (b == kSampleBuckets - 1) {
    all_c = count;
    all_m = mass;
    count = 0;
    mass = 0.0;
  }
  Before before = sum_before(count, mass, waves);
  if (b == kSampleBuckets - 1) {
    count = all_c - before.count;
    mass = fmax(all_m - before.mass, 0.0);
    all_count = all_c;
    all_mass = before.mass + mass;
    k_bucket = p_lo = p_hi = kSampleBuckets - 1;
    lo_count = 0;
    lo_mass = 0.0;
  }
  __syncthreads();
  const bool k_on = r.k > 0 && r.k < all_count, p_on = r.p < 1.0f, m_on = r.m > 0.0f;
  if (k_on && before.count < r.k && before.count + count >= r.k) {
    k_bucket = b;
    k_mass[0] = before.mass;
    k_mass[1] = before.mass + mass;
  }
  __syncthreads();
  // the border lies where the mass reaches p of the first k's, which is known up to the k-th's bucket: the first
  // bucket that reaches it (rounding of these sums allowed for)
  if (p_on) {
    const double p = fmax((double)r.p, 0.0), least = p * (k_on ? k_mass[0] : all_mass) * (1.0 - 1e-9),
                 most = p * (k_on ? k_mass[1] : all_mass) * (1.0 + 1e-9);
    const double end = before.mass + mass;
    if (end >= least && (b == 0 || before.mass < least)) atomicMin(&p_lo, b);
    if (end >= most && (b == 0 || before.mass < most)) atomicMin(&p_hi, b);
  }
  __syncthreads();
  s.lo = kSampleBuckets;
  s.hi = kSampleBuckets - 1;
  if (k_on) {
    s.lo = min(s.lo, k_bucket);
    s.hi = min(s.hi, k_bucket);
  }
  if (p_on) {
    s.lo = min(s.lo, p_lo);
    if (!k_on) s.hi = min(s.hi, p_hi);
  }
  if (m_on) {
    // (logits beyond the grid's ends share a bucket: nothing is sure then)
    const float at = abs(s.bucket) < 8388608 - 1024 ? floorf(-logf(r.m) * r.span) : __uint_as_float(0x7fc00000u);
    s.lo = min(s.lo, (int)fminf(fmaxf(at - 2.0f, 0.0f), kSampleBuckets - 1.0f));
    if (!(k_on && p_on)) s.hi = min(s.hi, (int)fminf(at + 3.0f, kSampleBuckets - 1.0f));
  }
  if (b == s.lo) {
    lo_count = before.count;
    lo_mass = before.mass;
  }
  if (s.lo == kSampleBuckets && b == 0) {
    lo_count = all_count;
    lo_mass = all_mass;
  }
  __syncthreads();
  s.count = lo_count;
  s.mass = (uint64_t)rint(ldexp(lo_mass, kMassScale));
  s.greedy = r.greedy;
  s.rate = r.rate;
  s.limit = fmax((double)r.p, 0.0) * ldexp(all_mass, kMassScale);
  s.top_k = k_on ? r.k : 0;
  s.top_p = r.p;
  s.min_p = r.m;
  s.least = 0;
  s.total = 0;
  return s;
}

template <bool BF16, int PIECES>
__global__ void __launch_bounds__(kSampleThreads) sample_collect_kernel(SampleArgs a) {
  const int row = blockIdx.y, slice = blockIdx.x, first = slice * PIECES * 8 * kSampleThreads;
  __shared__ uint64_t tops[kSampleThreads / 64];
  __shared__ int found;
  const Rules r = rules_of(a, row);
  if (threadIdx.x == 0) found = 0;
  const SampleRow s = settle_row(a, row, r);
  const int64_t at = (int64_t)row * a.slices + slice;
  uint64_t best = 0, *list = a.cand + at * a.entries;
  for (int i = 0; i < PIECES; ++i) {
    const int v = first + (i * kSampleThreads + (int)threadIdx.x) * 8;
    float x[8];
    load_logits<BF16>(a, row, v, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!(x[j] > kNegInf)) continue;
      const int bucket = min(s.bucket - bucket_of(x[j], r.grid), kSampleBuckets - 1);
      if (bucket < s.lo) {
        const uint64_t score = score_of(weight_of(x[j], s.top, s.rate), a.noise[(int64_t)row * a.vocab + v + j], v + j);
        best = score > best ? score : best;
      } else if (bucket <= s.hi) {
        list[atomicAdd(&found, 1)] = key_of(x[j], v + j);
      }
    }
  }
  best = wave_max_key(best);
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kSampleThreads / 64; ++i) best = tops[i] > best ? tops[i] : best;
    a.best[at] = best;
    a.found[at] = found;
    if (slice == 0) a.state[row] = s;
  }
}

constexpr int kFinishThreads = 512;
constexpr int kFinishHeld = 2048;   // candidates that a workgroup keeps in LDS
constexpr int kFinishLast = 64;     // candidates that one wave orders by itself

// A row's candidates.
struct Candidates {
  const SampleArgs& a;
  int row, n;
  uint64_t* held;
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    if (n <= kFinishHeld) {
      for (int i = threadIdx.x; i < n; i += kFinishThreads) f(held[i]);
    } else {
      for (int s = threadIdx.x >> 6; s < a.slices; s += kFinishThreads / 64) {
        const int64_t at = (int64_t)row * a.slices + s;
        for (int i = threadIdx.x & 63; i < a.found[at]; i += 64) f(a.cand[at * a.entries + i]);
      }
    }
  }
};

// The last candidate in the order that is kept: by rank (fewer than `most`
// entries before it) or, most < 0, by mass (less than `limit` before it).
// -> its key (all ones: none is kept) and the mass up to and with it.  Candidates
// are counted into 256 parts of their range, again within the part that the
// border lies in, until one wave orders what is left.
__device__ __forceinline__ uint64_t border(const Candidates& c, const SampleRow& s, int most, double limit, uint64_t* upto) {
  __shared__ unsigned long long mass[256], low, high, keys[kFinishLast];
  __shared__ unsigned count[256];
  __shared__ uint64_t b_mass, out_key, out_mass;
  __shared__ int b_count, part, listed;
  const int t = threadIdx.x;
  uint64_t lo = 0, hi = ~uint64_t(0);   // range of keys that the border is among
  int before = s.count;                 // entries before that range, and their mass
  uint64_t before_mass = s.mass;
  int inside = c.n;
  while (inside > kFinishLast) {
    // the range that is in use
    if (t == 0) {
      low = ~0ull;
      high = 0;
      part = -1;
    }
    if (t < 256) {
      mass[t] = 0;
      count[t] = 0;
    }
    __syncthreads();
    uint64_t a = ~uint64_t(0), b = 0;
    c.each([&](uint64_t k) {
      if (k >= lo && k <= hi) {
        a = k < a ? k : a;
        b = k > b ? k : b;
      }
    });
    b = wave_max_key(b);
    a = ~wave_max_key(~a);
    if ((t & 63) == 0) {
      atomicMin(&low, (unsigned long long)a);
      atomicMax(&high, (unsigned long long)b);
    }
    __syncthreads();
    lo = low;
    hi = high;
    const int shift = max(0, 56 - __clzll((long long)(hi - lo)));
    c.each([&](uint64_t k) {
      if (k >= lo && k <= hi) {
        const int i = (int)((hi - k) >> shift);
        atomicAdd(&count[i], 1u);
        atomicAdd(&mass[i], (unsigned long long)mass_of(logit_of((uint32_t)(k >> 32)), s.top, s.rate));
      }
    });
    __syncthreads();
    // wave 0: the part of the border, four a lane
    if (t < 64) {
      int n[4], sum = 0;
      uint64_t m[4], msum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        n[i] = (int)count[4 * t + i];
        m[i] = mass[4 * t + i];
        sum += n[i];
        msum += m[i];
      }
      int at = sum;
      uint64_t mat = msum;
#pragma unroll
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
      for (int i = 0; i < 4; ++i) {
        // the last part whose first entry is kept
        if (n[i] > 0 && (most >= 0 ? at < most : (double)mat < limit)) {
          mine = 4 * t + i;
          mine_at = at;
          mine_mass = mat;
        }
        at += n[i];
        mat += m[i];
      }
      const uint64_t any = __ballot(mine >= 0);
      if (any && t == 63 - __clzll((long long)any)) {
        part = mine;
        b_count = mine_at;
        b_mass = mine_mass;
      }
    }
    __syncthreads();
    const int p = part;
    if (p < 0) {   // not even the first one
      *upto = before_mass;
      __syncthreads();
      return ~uint64_t(0);
    }
    before = b_count;
    before_mass = b_mass;
    inside = (int)count[p];
    const uint64_t top = hi - ((uint64_t)p << shift);
    const uint64_t wide = (uint64_t(1) << shift) - 1;
    lo = top - lo > wide ? top - wide : lo;
    hi = top;
    __syncthreads();
  }
  if (t == 0) listed = 0;
  __syncthreads();
  c.each([&](uint64_t k) {
    if (k >= lo && k <= hi) keys[atomicAdd(&listed, 1)] = k;
  });
  __syncthreads();
  if (t < 64) {
    const bool in = t < listed;
    const uint64_t key = in ? keys[t] : 0;
    const uint64_t own = in ? mass_of(logit_of((uint32_t)(key >> 32)), s.top, s.rate) : 0;
    int at = before;
    uint64_t mat = before_mass;
    for (int j = 0; j < listed; ++j) {
      const uint64_t k = (uint64_t)__shfl((unsigned long long)key, j, 64), m = (uint64_t)__shfl((unsigned long long)own, j, 64);
      if (k > key) {
        ++at;
        mat += m;
      }
    }
    const bool kept = in && (most >= 0 ? at < most : (double)mat < limit);
    const uint64_t last = ~wave_max_key(kept ? ~key : 0);   // the smallest kept key; none: all ones
    const uint64_t sum = wave_max_key(kept ? mat + own : before_mass);
    if (t == 0) {
      out_key = last;
      out_mass = sum;
    }
  }
  __syncthreads();
  const uint64_t key = out_key;
  *upto = out_mass;
  __syncthreads();
  return key;
}

template <bool BF16>
__global__ void __launch_bounds__(kFinishThreads) sample_finish_kernel(SampleArgs a) {
  __shared__ uint64_t held[kFinishHeld], tops[kFinishThreads / 64], sums[kFinishThreads / 64];
  __shared__ int n, listed;
  const int row = blockIdx.x, t = threadIdx.x;
  SampleRow s = a.state[row];
  if (s.top == kNegInf) {   // no entry at all
    if (t == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = kNegInf;
    }
    return;
  }
  if (t == 0) n = listed = 0;
  __syncthreads();
  uint64_t best = 0;
  for (int i = t; i < a.slices; i += kFinishThreads) {
    const int64_t at = (int64_t)row * a.slices + i;
    const uint64_t b = a.best[at];
    best = b > best ? b : best;
    atomicAdd(&n, a.found[at]);
  }
  __syncthreads();
  const Candidates c = {a, row, n, held};
  if (n <= kFinishHeld) {
    for (int i = t >> 6; i < a.slices; i += kFinishThreads / 64) {
      const int64_t at = (int64_t)row * a.slices + i;
      for (int j = t & 63; j < a.found[at]; j += 64) held[atomicAdd(&listed, 1)] = a.cand[at * a.entries + j];
    }
    __syncthreads();
  }
  uint64_t least = 0, upto;
  if (c.n > 0) {
    if (s.top_k) {
      least = border(c, s, s.top_k, 0.0, &upto);
      s.limit = (double)s.top_p * (double)upto;
    }
    if (s.top_p < 1.0f) {
      // the first entry is kept whatever the limit
      const uint64_t k = border(c, s, -1, fmax(s.limit, 0.5), &upto);
      least = k > least ? k : least;
    }
  }
  uint64_t sum = 0;
  if (c.n > 0)
    c.each([&](uint64_t k) {
      if (k < least) return;
      const float l = logit_of((uint32_t)(k >> 32));
      const double w = weight_of(l, s.top, s.rate);
      if (w < (double)s.min_p) return;
      const int v = (int)(0xffffffffu - (uint32_t)k);
      sum += mass_of(l, s.top, s.rate);
      const uint64_t score = score_of(w, a.noise[(int64_t)row * a.vocab + v], v);
      best = score > best ? score : best;
    });
  best = wave_max_key(best);
  sum = wave_sum_u64(sum);
  if ((t & 63) == 0) {
    tops[t >> 6] = best;
    sums[t >> 6] = sum;
  }
  __syncthreads();
  if (t == 0) {
    sum += s.mass;
    for (int i = 1; i < kFinishThreads / 64; ++i) {
      best = tops[i] > best ? tops[i] : best;
      sum += sums[i];
    }
    s.least = least;
    s.total = sum;
    a.state[row] = s;
    const int v = (int)(0xffffffffu - (uint32_t)best);
    a.tokens[row] = v;
    if (a.logprobs) {
      const int64_t at = row * a.row + v;
      const float l = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
      a.logprobs[row] = (float)log(ldexp(weight_of(l + 0.0f, s.top, s.rate), kMassScale) / (double)sum);
    }
  }
}

// Probabilities: w over the mass of the kept entries.
template <bool BF16>
__global__ void __launch_bounds__(kSampleThreads) sample_write_kernel(SampleArgs a) {
  const int row = blockIdx.y, v = ((int)blockIdx.x * kSampleThreads + (int)threadIdx.x) * 8;
  if (v >= a.vocab) return;
  const SampleRow s = a.state[row];
  const Rules r = rules_of(a, row);
  const double per = s.top > kNegInf ? ldexp(1.0, kMassScale) / (double)s.total : 0.0;
  float x[8], p[8];
  load_logits<BF16>(a, row, v, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    p[j] = 0.0f;
    if (!(x[j] > kNegInf)) continue;
    const int bucket = min(s.bucket - bucket_of(x[j], r.grid), kSampleBuckets - 1);
    if (bucket < s.lo || (bucket <= s.hi && key_of(x[j], v + j) >= s.least)) {
      const double w = weight_of(x[j], s.top, s.rate);
      if (bucket < s.lo || w >= (double)s.min_p) p[j] = (float)(w * per);
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
  const int per = 8 * kSampleThreads;
  hipLaunchKernelGGL((sample_write_kernel<BF16>), dim3((unsigned)((a.vocab + per - 1) / per), (unsigned)a.rows),
                     dim3(kSampleThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_sample(const SampleArgs& a, bool bf16, hipStream_t s) {
  constexpr int WIDE = kSampleWide / (8 * kSampleThreads), NARROW = kSampleNarrow / (8 * kSampleThreads);
  if (a.entries == kSampleWide) return bf16 ? launch_rows<true, WIDE>(a, s) : launch_rows<false, WIDE>(a, s);
  return bf16 ? launch_rows<true, NARROW>(a, s) : launch_rows<false, NARROW>(a, s);
}

}  // namespace qlk
