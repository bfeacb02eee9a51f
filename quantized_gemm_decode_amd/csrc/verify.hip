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
// is cut into slices so that a single sequence also fills the card; every
// workgroup walks its sequence's drafts itself (a few dependent-free loads)
// instead of waiting for a launch that would.  A second launch takes the
// maximum over the slices and writes the tokens.
#include "attention_args.hpp"
#include "device_common.hpp"

namespace qlk {

constexpr int kVerifyThreads = 256;

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
      const float q = known && a.draft ? a.draft[(first + i) * a.vocab + x] : 1.0f;
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
__device__ __forceinline__ uint64_t score_key(float weight, float noise, uint32_t v) {
  const float s = __fdiv_rn(weight, noise);
  return s > 0.0f ? ((uint64_t)__float_as_uint(s) << 32) | (0xffffffffu - v) : 0u;
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  for (int o = 32; o > 0; o >>= 1) v = max_u64(v, (uint64_t)__shfl_xor((unsigned long long)v, o, 64));
  return v;
}

// Four binary32 values at a 4-byte aligned address: rows of an odd vocabulary
// start anywhere.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// The weights of one place: p, or what is left of it above q.
struct Weights {
  const float* p;
  const float* q;  // null: nothing is subtracted but `certain`
  int certain;     // a certain draft (q = 1), else -1
  __device__ __forceinline__ float at(float p, float q, int v) const { return fmaxf(p - (v == certain ? 1.0f : q), 0.0f); }
};

// Best score of entries [v0, v1) of a row, over one workgroup's (or wave's)
// `threads` threads.
__device__ __forceinline__ uint64_t scan(const Weights& w, const float* e, int v0, int v1, int thread, int threads) {
  constexpr int U = 2;
  uint64_t best = 0;
  int v = v0 + thread * 4;
  for (; v + 4 * threads * (U - 1) + 4 <= v1; v += 4 * threads * U) {
    f32x4u p[U], q[U], n[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      p[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4u*>(w.p + v + 4 * threads * i));
      n[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4u*>(e + v + 4 * threads * i));
      if (w.q) q[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4u*>(w.q + v + 4 * threads * i));
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = v + 4 * threads * i + j;
        best = max_u64(best, score_key(w.at(p[i][j], w.q ? q[i][j] : 0.0f, at), n[i][j], (uint32_t)at));
      }
  }
  for (; v < v1; v += 4 * threads)
    for (int at = v; at < v + 4 && at < v1; ++at)
      best = max_u64(best, score_key(w.at(w.p[at], w.q ? w.q[at] : 0.0f, at), e[at], (uint32_t)at));
  return best;
}

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

__global__ void __launch_bounds__(kVerifyThreads) verify_scan_kernel(VerifyArgs a) {
  const int b = blockIdx.y;
  int64_t first;
  const int n = draft_range(a, b, &first);
  const int k = accepted_drafts(a, first, n, b);
  const int per = ((a.vocab + a.slices - 1) / a.slices + 3) / 4 * 4;
  const int v0 = min((int)blockIdx.x * per, a.vocab), v1 = min(v0 + per, a.vocab);
  uint64_t best = wave_max_u64(scan(weights_of(a, first, n, k, b, true), a.noise + (int64_t)b * a.vocab, v0, v1,
                                    threadIdx.x, kVerifyThreads));
  __shared__ uint64_t part[kVerifyThreads / 64];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kVerifyThreads / 64; ++w) best = max_u64(best, part[w]);
    a.part[(int64_t)b * a.slices + blockIdx.x] = best;
  }
}

// One wave a sequence: the maximum over the slices, then the row of tokens.
__global__ void __launch_bounds__(64) verify_pick_kernel(VerifyArgs a) {
  const int b = blockIdx.x, lane = threadIdx.x;
  uint64_t best = 0;
  for (int i = lane; i < a.slices; i += 64) best = max_u64(best, a.part[(int64_t)b * a.slices + i]);
  int64_t first;
  const int n = draft_range(a, b, &first);
  const int k = accepted_drafts(a, first, n, b);
  best = wave_max_u64(best);
  // p - q nowhere positive (rounding alone): p itself, by this wave
  if (best == 0 && k < n)
    best = wave_max_u64(scan(weights_of(a, first, n, k, b, false), a.noise + (int64_t)b * a.vocab, 0, a.vocab, lane, 64));
  const int next = best ? (int)(0xffffffffu - (uint32_t)best) : 0;
  for (int i = lane; i <= a.max_drafts; i += 64)
    a.out_tokens[(int64_t)b * (a.max_drafts + 1) + i] = i < k ? a.tokens[first + i] : i == k ? next : -1;
  if (lane == 0) a.accepted[b] = k;
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(verify_scan_kernel, dim3((unsigned)a.slices, (unsigned)a.batch), dim3(kVerifyThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(verify_pick_kernel, dim3((unsigned)a.batch), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlk
