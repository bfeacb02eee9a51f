// C ABI of the adapters and of sampling: argument checks, sizes, launches.
#include "../../include/qlinear.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.hpp"
#include "serving_args.hpp"

using qlapi::aligned;
using qlapi::aligned16;
using qlapi::fail;
using qlapi::hip_fail;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxStride = int64_t(1) << 40;  // elements
constexpr int64_t kMaxWorkgroups = int64_t(1) << 24;

// Sizes and launch shape of an adapter call; the pointers stay unset.
ql_status lora_shape(const ql_lora* l, int64_t tokens, qlk::LoraArgs* a) {
  if (!l) return fail(QL_E_INVALID, "lora is NULL");
  if (tokens < 0 || l->adapters < 0) return fail(QL_E_INVALID, "negative size");
  if (tokens > kMaxTokens || l->adapters > 65536) return fail(QL_E_UNSUPPORTED, "more than 2^24 tokens or 2^16 adapters");
  if (l->slices < 1 || l->slices > qlk::kLoraSlices)
    return fail(QL_E_UNSUPPORTED, "slices %d must be in [1, %d]", l->slices, qlk::kLoraSlices);
  if (l->rank < 8 || l->rank > qlk::kLoraMostRank || l->rank % 8)
    return fail(QL_E_UNSUPPORTED, "rank %d must be a multiple of 8 in [8, %d]", l->rank, qlk::kLoraMostRank);
  if (l->in_features < 8 || l->in_features % 8 || l->in_features > (int64_t(1) << 20))
    return fail(QL_E_UNSUPPORTED, "in_features must be a multiple of 8 in [8, 2^20]");
  int64_t wide = 0, tiles = 0;
  for (int i = 0; i < l->slices; ++i) {
    if (l->widths[i] < 8 || l->widths[i] % 8 || l->widths[i] > (int64_t(1) << 20))
      return fail(QL_E_UNSUPPORTED, "widths must be multiples of 8 in [8, 2^20]");
    wide += l->widths[i];
    tiles += (l->widths[i] + 63) / 64;
    a->width[i] = (int)l->widths[i];
  }
  const int64_t rows = (int64_t)l->slices * l->rank;
  if (l->a_adapter_stride < 0 || l->b_adapter_stride < 0 || l->a_adapter_stride > kMaxStride || l->b_adapter_stride > kMaxStride)
    return fail(QL_E_INVALID, "adapter strides must be in [0, 2^40]");
  if (l->adapters > 1 && (l->a_adapter_stride < rows * l->in_features || l->b_adapter_stride < wide * l->rank))
    return fail(QL_E_INVALID, "adapter strides are shorter than an adapter");
  if (l->a_adapter_stride % 8 || l->b_adapter_stride % 8) return fail(QL_E_ALIGN, "adapter strides must be multiples of 8 elements");
  a->tokens = (int)tokens;
  a->adapters = l->adapters;
  a->rank = l->rank;
  a->k = (int)l->in_features;
  a->slices = l->slices;
  a->a_step = l->a_adapter_stride * 2;
  a->b_step = l->b_adapter_stride * 2;
  const int64_t blocks = (tokens + qlk::kLoraBlock - 1) / qlk::kLoraBlock;
  // a decode batch can hold as many tiles as adapters (and tokens without one),
  // and one more for every 16 tokens; a prompt's block of 64 tokens has four, or two
  // of 32 in the first product, which then reads A half as often (4,093 tokens: 57.2 us,
  // 63.7 in tiles of 16).  (Batches of more than 64 tokens that mix their adapters token by
  // token hold more tiles than that, and wait for them: 65 tokens of 32 adapters 63 us, 64
  // 13; in runs of 16 tokens 12.5 and 9.7.)
  a->wide = blocks > 1;
  const int64_t few = std::max<int64_t>(1, std::min<int64_t>(tokens, l->adapters + 1 + tokens / 16));
  a->down_slots = (int)(a->wide ? 2 : few);
  a->up_slots = (int)(a->wide ? 4 : few);
  const int64_t groups = (rows + 63) / 64, down = std::max<int64_t>(1, blocks * a->down_slots * groups),
                up = std::max<int64_t>(1, blocks * a->up_slots);
  // K is cut until there are four workgroups a compute unit, in parts of 512 at least,
  // 128 a wave (4,093 tokens: 57.2 us, 59.0 with two and 57.4 with eight; a decode batch does not mind)
  int64_t chunks = std::max<int64_t>(1, std::min<int64_t>((l->in_features + 511) / 512, 1024 / down));
  const int64_t chunk = ((l->in_features + chunks - 1) / chunks + 255) / 256 * 256;
  chunks = (l->in_features + chunk - 1) / chunk;
  a->chunk = (int)chunk;
  a->chunks = (int)chunks;
  // columns of a workgroup: h is summed and laid out once for them, so prompts take as many as leave four
  // workgroups a compute unit (4,093 tokens: 57.2 us, 62.6 with two), decode batches, of whose slots
  // many stay empty, two (64 tokens of 24 adapters: 20.3 us, 20.8 with four)
  a->tiles_wg = (int)std::max<int64_t>(4, std::min<int64_t>(32, up * tiles / (a->wide ? 1024 : 512) / 4 * 4));
  int64_t ranges = 0;
  for (int i = 0; i < l->slices; ++i) ranges += ((l->widths[i] + 63) / 64 + a->tiles_wg - 1) / a->tiles_wg;
  a->ranges = (int)ranges;
  if (down * chunks >= kMaxWorkgroups || up * ranges >= kMaxWorkgroups)
    return fail(QL_E_UNSUPPORTED, "2^24 workgroups or more");
  return QL_OK;
}

// The most partial sums (chunks of K of all tokens) that a call of up to a.tokens
// tokens has: up to a block of tokens any number of chunks; with more of them 1024 /
// (2 blocks groups), 512 a block and group over its 64 tokens.
int64_t most_parts(const qlk::LoraArgs& a) {
  const int64_t tokens = a.tokens, cut = (a.k + 511) / 512, groups = (a.slices * a.rank + 63) / 64;
  return std::max(tokens, std::min(tokens * cut, std::max<int64_t>(cut, 512 / groups) * qlk::kLoraBlock));
}

ql_status check_matrix(const void* p, int64_t stride, int64_t width, int64_t tokens, const char* name) {
  if (!p) return fail(QL_E_INVALID, "%s is NULL", name);
  if (!aligned16(p)) return fail(QL_E_ALIGN, "%s is not 16-byte aligned", name);
  if (stride < 0 || stride > kMaxStride) return fail(QL_E_INVALID, "%s stride must be in [0, 2^40]", name);
  if (tokens > 1 && stride < width) return fail(QL_E_INVALID, "%s stride is shorter than a row", name);
  if (stride % 8) return fail(QL_E_ALIGN, "%s stride must be a multiple of 8 elements", name);
  return QL_OK;
}

// Entries of a vocabulary row that a workgroup takes: long slices, which leave
// fewer histograms to add, where they still give every compute unit two.  (4,096,
// 8,192 and 16,384 entries; 8 rows of 32,000: 24, 27 and 34 us; 8 of 151,936: 38, 37
// and 43; 64 of 151,936: 82, 64 and 61.)
constexpr int64_t kSampleFill = 512;

int64_t slices_of(int64_t vocab, int entries) { return (vocab + entries - 1) / entries; }

int sample_entries(int64_t rows, int64_t vocab) {
  int entries = qlk::kSampleWide;
  while (entries > qlk::kSampleNarrow && rows * slices_of(vocab, entries) < kSampleFill) entries /= 2;
  return entries;
}

// The most slices of all rows together that a call of up to that many rows and
// entries has.  (Those shorter than kSampleWide are at most twice as many as the
// longer ones that were too few.)
int64_t most_slices(int64_t rows, int64_t vocab) {
  return std::max(rows * slices_of(vocab, qlk::kSampleWide),
                  std::min(2 * (kSampleFill - 1), rows * slices_of(vocab, qlk::kSampleNarrow)));
}

// Places in the workspace; `end` does not fall with fewer rows or a shorter
// vocabulary, so the largest call's workspace serves all.
struct SampleSpace {
  int64_t slices, entries, hist, cand, best, state, top, count, end;
};

SampleSpace sample_space(int64_t rows, int64_t vocab) {
  SampleSpace s;
  s.entries = sample_entries(rows, vocab);
  s.slices = slices_of(vocab, (int)s.entries);
  const int64_t all = rows * s.slices;
  s.hist = 0;
  s.cand = s.hist + all * qlk::kSampleBuckets * 8;
  s.best = s.cand + rows * vocab * 8;
  s.state = s.best + all * 8;
  s.top = s.state + rows * (int64_t)sizeof(qlk::SampleRow);
  s.count = s.top + all * 4;
  const int64_t more = most_slices(rows, vocab) - all;   // room of smaller calls
  s.end = (s.count + rows * qlk::kSampleCountStep * 4 + more * (qlk::kSampleBuckets * 8 + 8 + 4) + 15) / 16 * 16;
  return s;
}

ql_status sample_size(int64_t rows, int64_t vocab) {
  if (rows < 0 || vocab < 0) return fail(QL_E_INVALID, "negative size");
  if (rows > 65535 || vocab > (int64_t(1) << 24)) return fail(QL_E_UNSUPPORTED, "more than 65535 rows or 2^24 tokens of vocabulary");
  return QL_OK;
}

}  // namespace

extern "C" {

int64_t qlinear_lora_workspace_bytes(const ql_lora* lora, int64_t tokens) {
  qlk::LoraArgs a{};
  if (lora_shape(lora, tokens, &a) != QL_OK) return 0;
  return most_parts(a) * a.slices * a.rank * 4;
}

ql_status qlinear_lora(const ql_lora* lora, int64_t tokens, const void* x, int64_t x_stride, const void* y, int64_t y_stride,
                       const int32_t* adapter, void* out, int64_t out_stride, void* workspace, void* stream) {
  qlk::LoraArgs a{};
  ql_status st = lora_shape(lora, tokens, &a);
  if (st != QL_OK) return st;
  if (tokens == 0) return QL_OK;
  int64_t wide = 0;
  for (int i = 0; i < a.slices; ++i) wide += a.width[i];
  if ((st = check_matrix(x, x_stride, a.k, tokens, "x")) != QL_OK || (st = check_matrix(y, y_stride, wide, tokens, "y")) != QL_OK ||
      (st = check_matrix(out, out_stride, wide, tokens, "out")) != QL_OK)
    return st;
  if (out == y && out_stride != y_stride && tokens > 1) return fail(QL_E_INVALID, "out is y with another stride");
  if (!adapter) return fail(QL_E_INVALID, "adapter is NULL");
  if (lora->adapters > 0 && (!lora->a || !lora->b)) return fail(QL_E_INVALID, "a or b is NULL");
  if (!aligned16(lora->a) || !aligned16(lora->b)) return fail(QL_E_ALIGN, "a and b must be 16-byte aligned");
  if (!aligned(lora->scales, 4) || !aligned(adapter, 4)) return fail(QL_E_ALIGN, "scales and adapter must be 4-byte aligned");
  if (!workspace) return fail(QL_E_INVALID, "workspace is NULL");
  if (!aligned16(workspace)) return fail(QL_E_ALIGN, "workspace is not 16-byte aligned");
  a.x = static_cast<const uint8_t*>(x);
  a.y = static_cast<const uint8_t*>(y);
  a.out = static_cast<uint8_t*>(out);
  a.a = static_cast<const uint8_t*>(lora->a);
  a.b = static_cast<const uint8_t*>(lora->b);
  a.scales = lora->scales;
  a.adapter = adapter;
  a.part = static_cast<float*>(workspace);
  a.x_row = x_stride * 2;
  a.y_row = y_stride * 2;
  a.out_row = out_stride * 2;
  hipError_t e = qlk::launch_lora(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? QL_OK : hip_fail(e, "adapter launch");
}

int64_t qlinear_sample_workspace_bytes(int64_t rows, int64_t vocab) {
  if (sample_size(rows, vocab) != QL_OK || rows == 0 || vocab == 0) return 0;
  return sample_space(rows, vocab).end;
}

ql_status qlinear_sample(const ql_sampling* rules, int64_t rows, int64_t vocab, const void* logits, int64_t logits_stride,
                         int32_t logits_type, const float* noise, int32_t* tokens, float* logprobs, float* probs,
                         void* workspace, void* stream) {
  ql_status st = sample_size(rows, vocab);
  if (st != QL_OK) return st;
  if (rows == 0) return QL_OK;
  if (vocab == 0) return fail(QL_E_INVALID, "the vocabulary is empty");
  if (logits_type != QL_LOGITS_F32 && logits_type != QL_LOGITS_BF16) return fail(QL_E_INVALID, "unknown logits type %d", logits_type);
  if (logits_stride < 0 || logits_stride > kMaxStride) return fail(QL_E_INVALID, "logits stride must be in [0, 2^40]");
  if (rows > 1 && logits_stride < vocab) return fail(QL_E_INVALID, "logits stride is shorter than a row");
  if (!logits || !noise || !tokens || !workspace) return fail(QL_E_INVALID, "NULL pointer");
  if (!aligned(logits, logits_type == QL_LOGITS_F32 ? 4 : 2)) return fail(QL_E_ALIGN, "logits is not aligned to its type");
  for (const void* p : {(const void*)noise, (const void*)tokens, (const void*)logprobs, (const void*)probs,
                        (const void*)(rules ? rules->temperature : nullptr), (const void*)(rules ? rules->top_k : nullptr),
                        (const void*)(rules ? rules->top_p : nullptr), (const void*)(rules ? rules->min_p : nullptr)})
    if (!aligned(p, 4)) return fail(QL_E_ALIGN, "pointers must be 4-byte aligned");
  if (!aligned16(workspace)) return fail(QL_E_ALIGN, "workspace is not 16-byte aligned");
  const SampleSpace w = sample_space(rows, vocab);
  char* base = static_cast<char*>(workspace);
  qlk::SampleArgs a{};
  a.logits = logits;
  a.row = logits_stride;
  a.noise = noise;
  if (rules) {
    a.temperature = rules->temperature;
    a.top_k = rules->top_k;
    a.top_p = rules->top_p;
    a.min_p = rules->min_p;
  }
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.probs = probs;
  a.hist = reinterpret_cast<uint64_t*>(base + w.hist);
  a.top = reinterpret_cast<float*>(base + w.top);
  a.state = reinterpret_cast<qlk::SampleRow*>(base + w.state);
  a.best = reinterpret_cast<uint64_t*>(base + w.best);
  a.count = reinterpret_cast<int32_t*>(base + w.count);
  a.cand = reinterpret_cast<uint64_t*>(base + w.cand);
  a.rows = (int)rows;
  a.vocab = (int)vocab;
  a.slices = (int)w.slices;
  a.entries = (int)w.entries;
  hipError_t e = qlk::launch_sample(a, logits_type == QL_LOGITS_BF16, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? QL_OK : hip_fail(e, "sampling launch");
}

}  // extern "C"
