// Verification of drafted tokens against the target's probabilities.
//
// A sequence has n drafted tokens x_i with the draft's distributions q_i and
// the target's p_0 .. p_n.  With given uniforms u_i it accepts x_0, x_1, ...
// while u_i q_i(x_i) < p_i(x_i), i.e. with probability min(1, p_i / q_i).  At
// the first rejection k the next token is drawn from max(p_k - q_k, 0)
// normalised, after n acceptances from p_n: the argmax over v of weight_v /
// e_v with given exponential e_v, which draws v with probability in
// proportion to its weight and needs no sum, so neither the order of a sum
// nor its rounding can change the token.  Ties go to the lowest index.  Where
// p_k - q_k is nowhere positive (rounding only) the weights are p_k's own.
//
// One pass over one row of p, q and e of each sequence (12 bytes an entry,
// one division): bound by memory, by the launches for few sequences.  A row
// is cut into slices so that a single sequence also fills the card, short
// enough for a workgroup to hold its slice in registers: e, which no decision
// chooses, is on its way while the drafts are walked (three dependent loads),
// then p and q are requested at once.  Every workgroup walks its sequence's
// drafts itself instead of waiting for a launch that would.  A second launch
// takes the maximum over the slices.
// Measured: 64 sequences of 5 drafts, 151,936 entries: 21.3 us
// (107 MB, 5.0 TB/s with both launches); 24.6 and 27.1 us with 8,192 and 10,240
// entries a workgroup, which leave too few of them a compute unit.
#include "attention_args.hpp"
#include "attention_common.hpp"

namespace qlk {

constexpr int kVerifyThreads = 256;

// A draft's probability; NaN counts as 0.  (The target's needs no test: as 0 it
// accepts nothing and leaves no weight, and so do the comparisons with NaN.)
__device__ __forceinline__ float draft_prob(float q) { return q == q ? q : 0.0f; }

// Accepted drafts of a sequence, by the lanes of a wave: drafts in groups of
// 64, one a lane, the first rejection by ballot.
__device__ __forceinline__ int accepted_drafts(const VerifyArgs& a, int64_t first, int n, int b) {
  const int lane = threadIdx.x & 63;
  for (int i0 = 0; i0 < n; i0 += 64) {
    const int i = i0 + lane;
    bool ok = true;
    if (i < n) {
      const int64_t x = a.tokens[first + i];
      const bool known = x >= 0 && x < a.vocab;  // a token outside the vocabulary is rejected
      const float p = known ? a.target[(first + i + b) * a.vocab + x] : 0.0f;
      const float q = known && a.draft ? draft_prob(a.draft[(first + i) * a.vocab + x]) : 1.0f;
      ok = __fmul_rn(a.uniforms[first + i], q) < p;
    }
    const unsigned long long no = __ballot(!ok);
    if (no) return i0 + __ffsll(no) - 1;
  }
  return n;
}

// The drafts [first, first + n) of sequence b, kept inside the arrays.
__device__ __forceinline__ int draft_range(const VerifyArgs& a, int b, int64_t* first) {
  int64_t f = a.cu[b], e = a.cu[b + 1];
  f = f < 0 ? 0 : f > a.n_drafts ? a.n_drafts : f;
  e = e < f ? f : e > a.n_drafts ? a.n_drafts : e;
  *first = f;
  return (int)(e - f < a.max_drafts ? e - f : a.max_drafts);
}

// A weight's score and index as one word whose maximum is the larger score
// and, between equals, the lower index; 0 for no positive score.  Positive
// binary32 values order as their bit patterns.
__device__ __forceinline__ uint64_t score_key(float s, uint32_t v) {
  return s > 0.0f ? ((uint64_t)__float_as_uint(s) << 32) | (0xffffffffu - v) : 0u;
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  for (int o = 32; o > 0; o >>= 1) v = max_u64(v, (uint64_t)__shfl_xor((unsigned long long)v, o, 64));
  return v;
}

// The weights of one place: p, or what is left of it above q.
struct Weights {
  const float* p;
  const float* q;  // null: nothing is subtracted but `certain`
  int certain;     // a certain draft (q = 1), else -1
  __device__ __forceinline__ float at(float p, float q, int v) const {
    return fmaxf(p - (v == certain ? 1.0f : draft_prob(q)), 0.0f);
  }
};

__device__ __forceinline__ Weights weights_of(const VerifyArgs& a, int64_t first, int n, int k, int b, bool diff) {
  Weights w = {a.target + (first + k + b) * a.vocab, nullptr, -1};
  if (diff && k < n) {  // rejected: the draft's row is subtracted
    if (a.draft)
      w.q = a.draft + (first + k) * a.vocab;
    else
      w.certain = a.tokens[first + k];
  }
  return w;
}

// Workgroup (slice, b): the best score of a slice of sequence b's row.  The
// first slice's also writes the accepted drafts.
__global__ void __launch_bounds__(kVerifyThreads) verify_scan_kernel(VerifyArgs a) {
  constexpr int U = kVerifySlice / (4 * kVerifyThreads);  // 16-byte pieces a thread holds of each array
  const int b = blockIdx.y;
  const int per = ((a.vocab + a.slices - 1) / a.slices + 3) / 4 * 4;
  const int v0 = min((int)blockIdx.x * per, a.vocab), v1 = min(v0 + per, a.vocab);
  // a piece that would pass the row's end is moved back: entries seen twice
  // do not change a maximum
  const int last = max(a.vocab - 4, 0);
  const float* e = a.noise + (int64_t)b * a.vocab;
  const bool wide = a.vocab >= 4;
  auto piece = [&](const float* row, int v) {
    if (wide) return __builtin_nontemporal_load(reinterpret_cast<const f32x4u*>(row + v));
    f32x4u x = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < a.vocab; ++i) x[i] = row[i];
    return x;
  };
  f32x4u noise[U], p[U], q[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int v = v0 + (i * kVerifyThreads + (int)threadIdx.x) * 4;
    if (v < v1) noise[i] = piece(e, min(v, last));
  }
  int64_t first;
  const int n = draft_range(a, b, &first);
  const int k = accepted_drafts(a, first, n, b);
  const Weights w = weights_of(a, first, n, k, b, true);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int v = v0 + (i * kVerifyThreads + (int)threadIdx.x) * 4;
    if (v < v1) {
      p[i] = piece(w.p, min(v, last));
      if (w.q) q[i] = piece(w.q, min(v, last));
    }
  }
  if (blockIdx.x == 0) {
    int32_t* out = a.out_tokens + (int64_t)b * (a.max_drafts + 1);
    for (int i = threadIdx.x; i <= a.max_drafts; i += kVerifyThreads)
      if (i != k) out[i] = i < k ? a.tokens[first + i] : -1;
    if (threadIdx.x == 0) a.accepted[b] = k;
  }
  // a thread's entries come in rising order: the first of the largest is kept
  float top = 0.0f;
  int top_at = 0;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int v = v0 + (i * kVerifyThreads + (int)threadIdx.x) * 4;
    if (v >= v1) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = min(v, last) + j;
      const float s = __fdiv_rn(w.at(p[i][j], w.q ? q[i][j] : 0.0f, at), noise[i][j]);
      if (at < a.vocab && s > top) {
        top = s;
        top_at = at;
      }
    }
  }
  uint64_t best = wave_max_u64(score_key(top, (uint32_t)top_at));
  __shared__ uint64_t part[kVerifyThreads / 64];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kVerifyThreads / 64; ++i) best = max_u64(best, part[i]);
    a.part[(int64_t)b * a.slices + blockIdx.x] = best;
  }
}

// One wave a sequence: the maximum over the slices is the next token.  Where p - q
// is nowhere positive this wave reads the whole of p by itself: 333 us for a
// sequence of 151,936 entries, 1.1 ms for 64 of them.  Rounding alone leads there,
// or a drafted token outside the vocabulary with p = q.
__global__ void __launch_bounds__(64) verify_pick_kernel(VerifyArgs a) {
  const int b = blockIdx.x, lane = threadIdx.x;
  const int k = a.accepted[b];
  uint64_t best = 0;
  for (int i = lane; i < a.slices; i += 64) best = max_u64(best, a.part[(int64_t)b * a.slices + i]);
  best = wave_max_u64(best);
  if (best == 0) {  // p - q nowhere positive (rounding alone), or p: p itself, by this wave
    int64_t first;
    const int n = draft_range(a, b, &first);
    const Weights w = weights_of(a, first, n, k, b, false);
    for (int v = lane; v < a.vocab; v += 64)
      best = max_u64(best, score_key(__fdiv_rn(w.at(w.p[v], 0.0f, v), a.noise[(int64_t)b * a.vocab + v]), (uint32_t)v));
    best = wave_max_u64(best);
  }
  if (lane == 0)
    a.out_tokens[(int64_t)b * (a.max_drafts + 1) + k] = best ? (int)(0xffffffffu - (uint32_t)best) : 0;
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(verify_scan_kernel, dim3((unsigned)a.slices, (unsigned)a.batch), dim3(kVerifyThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_pick_kernel, dim3((unsigned)a.batch), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlk
