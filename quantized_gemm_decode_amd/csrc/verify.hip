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

// Entry v of one slice: the best of the difference's and of p's own scores.
__device__ __forceinline__ void take(float p, float q, float e, uint32_t v, bool diff, uint64_t* best, uint64_t* own) {
  *own = max_u64(*own, score_key(p, e, v));
  if (diff) *best = max_u64(*best, score_key(fmaxf(p - q, 0.0f), e, v));
}

__global__ void __launch_bounds__(kVerifyThreads) verify_scan_kernel(VerifyArgs a) {
  const int b = blockIdx.y;
  int64_t first;
  const int n = draft_range(a, b, &first);
  const int k = accepted_drafts(a, first, n, b);
  const bool diff = k < n;  // rejected: the draft's row is subtracted
  const float* p = a.target + (first + k + b) * a.vocab;
  const float* q = diff && a.draft ? a.draft + (first + k) * a.vocab : nullptr;
  const int certain = diff && !a.draft ? a.tokens[first + k] : -1;
  const float* e = a.noise + (int64_t)b * a.vocab;
  const int per = (a.vocab + a.slices - 1) / a.slices;
  const int v0 = (int)blockIdx.x * per, v1 = v0 + per < a.vocab ? v0 + per : a.vocab;
  uint64_t best = 0, own = 0;
  for (int v = v0 + (int)threadIdx.x; v < v1; v += kVerifyThreads)
    take(p[v], q ? q[v] : (v == certain ? 1.0f : 0.0f), e[v], (uint32_t)v, diff, &best, &own);
  best = wave_max_u64(best);
  own = wave_max_u64(own);
  __shared__ uint64_t part[2][kVerifyThreads / 64];
  if ((threadIdx.x & 63) == 0) {
    part[0][threadIdx.x >> 6] = best;
    part[1][threadIdx.x >> 6] = own;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    uint64_t m = 0;
    for (int w = 0; w < kVerifyThreads / 64; ++w) m = max_u64(m, part[threadIdx.x][w]);
    a.part[((int64_t)b * a.slices + blockIdx.x) * 2 + threadIdx.x] = m;
  }
}

// One wave a sequence: the maximum over the slices, then the row of tokens.
__global__ void __launch_bounds__(64) verify_pick_kernel(VerifyArgs a) {
  const int b = blockIdx.x, lane = threadIdx.x;
  int64_t first;
  const int n = draft_range(a, b, &first);
  const int k = accepted_drafts(a, first, n, b);
  uint64_t best = 0, own = 0;
  for (int i = lane; i < a.slices; i += 64) {
    best = max_u64(best, a.part[((int64_t)b * a.slices + i) * 2]);
    own = max_u64(own, a.part[((int64_t)b * a.slices + i) * 2 + 1]);
  }
  best = wave_max_u64(best);
  own = wave_max_u64(own);
  const uint64_t w = best ? best : own;
  const int next = w ? (int)(0xffffffffu - (uint32_t)w) : 0;
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
