// Launch arguments of the operators of a server of many requests: low-rank
// adapters beside a projection, and sampling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlk {

constexpr int kLoraSlices = 4;      // most slices of a merged projection
constexpr int kLoraBlock = 64;      // tokens among which equal adapters are looked for: one a lane
constexpr int kLoraMostRank = 128;

struct LoraArgs {
  const uint8_t* x;        // bf16 [tokens, K]; strides in bytes
  const uint8_t* y;        // bf16 [tokens, N]
  uint8_t* out;            // bf16 [tokens, N]
  const uint8_t* a;        // bf16 [adapters, slices * rank, K]
  const uint8_t* b;        // bf16 [adapters, N, rank]
  const float* scales;     // [adapters] or null
  const int32_t* adapter;  // [tokens]; outside [0, adapters): none
  float* part;             // [chunks, tokens, slices * rank]: sums over chunks of K
  int64_t x_row, y_row, out_row, a_step, b_step;
  int tokens, adapters, rank, k, slices;
  int width[kLoraSlices];
  int chunk, chunks;       // K of a partial sum (a multiple of 256: 64 a step of each wave), their number
  int wide;                // first product: tiles of 32 tokens, not 16
  int down_slots, up_slots;  // workgroups that share a block's tiles of tokens, of each product
  int tiles_wg;            // 64-wide column tiles of a workgroup of the second product
  int ranges;              // of all slices together
};

constexpr int kSampleBuckets = 512;
constexpr int kSampleWide = 16384, kSampleNarrow = 4096;   // entries of a slice
constexpr int kSampleCountStep = 32;   // a row's counter has a 128-byte line to itself

// What a row's histograms say of it, and what is kept at last.
struct SampleRow {
  double line;       // the grid's line below the largest logit
  double mass;       // of the buckets before lo, of the largest's weight
  double unit;       // log2 of the weight that candidates' masses refer to: the middle of bucket lo
  double all;        // mass of all entries
  double total;      // of the kept ones
  uint64_t least;    // smallest kept candidate
  float top;         // largest logit (0 where that is +inf); -inf: no entry
  int inf;
  int lo, hi;        // buckets before lo are kept whole, those after hi are not; between them the candidates
  int count;         // entries of the buckets before lo
  int k;             // top-k, 0: off or without effect
};

struct SampleArgs {
  const void* logits;      // binary32 or bf16 [rows, vocab]
  int64_t row;             // entries between rows
  const float* noise;      // [rows, vocab]
  const float* temperature;  // [rows] each, or null
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;         // [rows]
  float* logprobs;         // [rows] or null
  float* probs;            // [rows, vocab] or null
  uint64_t* hist;          // [rows, slices, kSampleBuckets]: entries (high bits) and their mass
  float* top;              // [rows, slices]: a slice's largest logit
  uint64_t* best;          // [rows, slices]: best score among a slice's surely kept entries
  uint64_t* cand;          // [rows, vocab]: candidates
  int32_t* count;          // [rows, kSampleCountStep], the first: candidates
  SampleRow* state;        // [rows]
  int rows, vocab, slices, entries;
};

hipError_t launch_lora(const LoraArgs& a, hipStream_t s);
hipError_t launch_sample(const SampleArgs& a, bool bf16, hipStream_t s);

}  // namespace qlk
