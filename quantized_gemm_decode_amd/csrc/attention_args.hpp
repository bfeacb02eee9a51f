// Launch arguments of the serving operators around the linears: per-head
// norm and rotation, append to a paged cache, attention over it, and the
// verification of drafted tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlk {

// bf16 rows [tokens, heads, head_dim], head_dim contiguous; strides in bytes.
struct Rows {
  uint8_t* p;
  int64_t token, head;
};

// One tensor of the paged cache, [pages, page_size, kv_heads, head_dim] with
// head_dim contiguous; strides in bytes.
struct Pages {
  uint8_t* p;
  int64_t page, token, head;
  const float* scale;  // [kv_heads], null: 1 (E4M3 caches: value = code * scale)
};

struct HeadArgs {
  Rows q, k, v;          // inputs (v: append only)
  Rows q_out, k_out;     // outputs (k_out: without a cache)
  Pages kc, vc;          // cache (append only)
  const uint16_t* q_w;   // norm weights [head_dim] bf16; null: no norm
  const uint16_t* k_w;
  const float* table;    // [max_pos, rot]: rot/2 cosines, then rot/2 sines
  const int64_t* pos;    // [tokens]
  const int64_t* slots;  // [tokens], append only
  int64_t max_pos, num_slots;
  uint64_t page_magic;   // ceil(2^36 / (page_size / 16)) (see page_of)
  float eps;
  int tokens, q_heads, kv_heads, page_size, rot, interleaved;
};

struct AttnArgs {
  Rows q, out;
  Pages kc, vc;
  const int32_t* table;  // page of each (sequence, page column)
  int64_t table_row;     // entries between the rows of the table
  const int32_t* seq_lens;
  const int32_t* cu_q;
  float* lse;            // [tokens, q_heads] or null
  float* part_o;         // partial outputs of head_dim values a row: [kv_heads, splits, tokens * group] rows of
                         // the tile kernel, [slots, 2, kv_heads, R] rows of the stream kernel (trees: [shares, waves,
                         // registers and one of maxima and sums, lanes] pairs)
  float* part_ml;        // their rows' maxima (base 2) and sums
  uint64_t page_magic;
  const uint64_t* sees;  // trees of drafts: [tokens, words] new tokens of its sequence that a token sees, one a bit
  float scale_log2;      // softmax scale * log2(e)
  int batch, tokens, q_heads, kv_heads, group, page_size, num_pages, max_kv, causal, window;
  int words;             // of a row of `sees`
  // tile kernel
  int row_blocks;        // most blocks of R (token, head of the group) rows of a sequence and KV head
  int by_rows;           // numbering of the units (see unit_at)
  int splits, chunk;     // most chunks of keys of a unit, and their length
  int min_rows;          // sequences with fewer rows are left to the stream kernel
  // trees: the keys are cut on the device (see tree_cut)
  int32_t* cut;          // [batch, 2]: a sequence's first share (of one KV head), shares of a unit
  int shares;            // workgroups there are at most
  // stream kernel
  int slots;             // shares that all sequences' keys are cut into, for each KV head
  int heads_wg;          // KV heads of a workgroup (1, 2 or 4); its other waves take other slots
  int max_rows;          // sequences with more rows are left to the tile kernel
};

struct VerifyArgs {
  const float* target;    // [drafts + batch, vocab]
  const float* draft;     // [drafts, vocab], null: the drafts were certain
  const int32_t* tokens;  // [drafts]
  const int32_t* cu;      // [batch + 1]
  const float* uniforms;  // [drafts]
  const float* noise;     // [batch, vocab]
  int32_t* out_tokens;    // [batch, max_drafts + 1]
  int32_t* accepted;      // [batch]
  uint64_t* part;         // [batch, slices]
  int64_t n_drafts;       // rows of draft / tokens / uniforms
  int batch, vocab, max_drafts, slices;
};

constexpr int kCommitLayers = 32;     // caches of one launch
constexpr int kCommitDepth = 1024;    // most accepted tokens of a sequence

struct CommitLayer {
  Pages k, v;
  int kv_heads, head_bytes;
};

struct CommitArgs {
  const int32_t* table;        // page of each (sequence, page column)
  int64_t table_row;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const int32_t* node_tokens;  // [tokens]
  const int32_t* parents;
  const int32_t* sampled;
  int32_t* out_tokens;         // [batch, max_depth + 1]; null: not this launch's to write
  int32_t* accepted;           // [batch]
  int32_t* new_lens;           // [batch] or null
  int64_t num_pages;           // of the smallest cache
  int batch, tokens, max_depth, max_kv, page_size, layers;
  CommitLayer layer[kCommitLayers];
};

constexpr int kPageMagicShift = 36;

// The page column of the 16-key group `sub` (page_size / 16 groups a page):
// floor(sub / groups) as a multiplication by ceil(2^36 / groups), exact for
// sub < 2^27 and at most 512 groups a page.
__host__ __device__ __forceinline__ int page_of(int sub, uint64_t magic) {
  return (int)(((uint64_t)(uint32_t)sub * magic) >> kPageMagicShift);
}

// Tiles of 32 keys that a slot of the stream kernel has at least: 2^kStreamPad.
// Up to 64 sequences, if the slots suffice for it, have slots of their own.
constexpr int kStreamPad = 1;

// Most entries of a vocabulary row that one workgroup of the verification takes.
constexpr int kVerifySlice = 4096;

hipError_t launch_heads(const HeadArgs& a, int head_dim, bool append, bool e4m3, hipStream_t s);
// Slots of the stream kernel: as many as the card holds waves for each KV head.
int attn_stream_slots(int head_dim, bool e4m3, int rows, int kv_heads, int heads_wg);
// (Attention for trees where a.sees is given.)
hipError_t launch_attn_stream(const AttnArgs& a, int head_dim, bool e4m3, int rows, hipStream_t s);
hipError_t launch_attn_stream_join(const AttnArgs& a, int head_dim, int rows, int most_rows, hipStream_t s);
hipError_t launch_attn_tile(const AttnArgs& a, int head_dim, bool e4m3, int units, hipStream_t s);
hipError_t launch_attn_join(const AttnArgs& a, int head_dim, int rows, hipStream_t s);
hipError_t launch_attn_tree_join(const AttnArgs& a, int head_dim, int units, hipStream_t s);
// Workgroups of the tile kernel that the card holds at once.
int attn_tile_slots(int head_dim);
hipError_t launch_verify(const VerifyArgs& a, hipStream_t s);
hipError_t launch_tree_commit(const CommitArgs& a, hipStream_t s);

}  // namespace qlk
