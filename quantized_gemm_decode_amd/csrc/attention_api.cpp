// C ABI of the serving operators around the linears: argument checks, the
// attention planner, launches.
#include "../../include/qlinear.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "api_common.hpp"
#include "attention_args.hpp"

using qlapi::aligned;
using qlapi::aligned16;
using qlapi::fail;
using qlapi::hip_fail;

namespace {

// One kernel's share of a plan.
struct Part {
  bool used;
  int rows;                              // rows of a unit
  int row_blocks, splits, chunk, units;  // tile kernel
  bool by_rows;
  int slots, heads_wg, most;             // stream kernel; most rows of its sequences
  int64_t o_at, ml_at, end;              // partial outputs, their maxima and sums, in the workspace (bytes)
};

}  // namespace

struct ql_attention_plan_s {
  ql_attention_shape shape;
  Part stream, tile;
  int tile_from;  // rows of a sequence from which it goes to the tile kernel
};

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxStride = int64_t(1) << 40;  // elements

ql_status check_rows(const ql_rows* r, const char* name, int64_t heads, qlk::Rows* out) {
  if (!r || !r->data) return fail(QL_E_INVALID, "%s is NULL", name);
  if (!aligned16(r->data)) return fail(QL_E_ALIGN, "%s is not 16-byte aligned", name);
  if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride > kMaxStride || r->head_stride > kMaxStride)
    return fail(QL_E_INVALID, "%s strides must be in [0, 2^40]", name);
  if (r->token_stride % 8 || r->head_stride % 8)
    return fail(QL_E_ALIGN, "%s strides must be multiples of 8 elements", name);
  if (r->head_stride * 2 * heads >= (int64_t(1) << 31))
    return fail(QL_E_UNSUPPORTED, "%s heads span 2^31 bytes or more", name);
  *out = qlk::Rows{static_cast<uint8_t*>(r->data), r->token_stride * 2, r->head_stride * 2};
  return QL_OK;
}

ql_status check_pages(void* p, const float* scale, int64_t page, int64_t token, int64_t head, int size,
                      const char* name, qlk::Pages* out) {
  if (!p) return fail(QL_E_INVALID, "cache %s is NULL", name);
  if (!aligned16(p)) return fail(QL_E_ALIGN, "cache %s is not 16-byte aligned", name);
  if (!aligned(scale, 4)) return fail(QL_E_ALIGN, "cache %s_scale is not 4-byte aligned", name);
  if (page < 0 || token < 0 || head < 0 || page > kMaxStride || token > kMaxStride || head > kMaxStride)
    return fail(QL_E_INVALID, "cache %s strides must be in [0, 2^40]", name);
  if (page * size % 16 || token * size % 16 || head * size % 16)
    return fail(QL_E_ALIGN, "cache %s strides must be multiples of 16 bytes", name);
  if (token * size * 16 >= (int64_t(1) << 31))
    return fail(QL_E_UNSUPPORTED, "cache %s token stride beyond 2^27 bytes", name);
  *out = qlk::Pages{static_cast<uint8_t*>(p), page * size, token * size, head * size, scale};
  return QL_OK;
}

ql_status check_page_size(int32_t page_size) {
  if (page_size < 16 || page_size % 16 || page_size > 8192)
    return fail(QL_E_UNSUPPORTED, "page_size %d must be a multiple of 16 in [16, 8192]", page_size);
  return QL_OK;
}

uint64_t page_magic(int32_t page_size) {
  const uint64_t groups = (uint64_t)page_size / 16;
  return ((uint64_t(1) << qlk::kPageMagicShift) + groups - 1) / groups;
}

ql_status check_cache(const ql_kv_cache* c, qlk::Pages* k, qlk::Pages* v) {
  if (!c) return fail(QL_E_INVALID, "cache is NULL");
  if (c->type != QL_KV_BF16 && c->type != QL_KV_E4M3) return fail(QL_E_INVALID, "unknown cache type %d", c->type);
  if (c->kv_heads < 1 || c->num_pages < 1)
    return fail(QL_E_INVALID, "the cache needs at least one page and one head");
  ql_status st = check_page_size(c->page_size);
  if (st != QL_OK) return st;
  if (c->num_pages > (int64_t(1) << 31) / c->page_size || c->num_pages * c->page_size >= (int64_t(1) << 31))
    return fail(QL_E_UNSUPPORTED, "the cache holds 2^31 tokens or more");
  const int size = c->type == QL_KV_E4M3 ? 1 : 2;
  if (c->type == QL_KV_BF16 && (c->k_scale || c->v_scale))
    return fail(QL_E_INVALID, "a bf16 cache has no scales");
  st = check_pages(c->k, c->k_scale, c->k_page_stride, c->k_token_stride, c->k_head_stride, size, "k", k);
  if (st != QL_OK) return st;
  return check_pages(c->v, c->v_scale, c->v_page_stride, c->v_token_stride, c->v_head_stride, size, "v", v);
}

bool norm_dim(int32_t d) { return d == 64 || d == 128 || d == 256; }

ql_status check_rule(const ql_norm_rope* r, int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                     const int64_t* positions, qlk::HeadArgs* a) {
  if (!r) return fail(QL_E_INVALID, "rule is NULL");
  if (tokens < 0 || q_heads < 0 || kv_heads < 0) return fail(QL_E_INVALID, "negative size");
  if (tokens > kMaxTokens || q_heads > 65536 || kv_heads > 65536)
    return fail(QL_E_UNSUPPORTED, "more than 2^24 tokens or 2^16 heads");
  if (!norm_dim(head_dim)) return fail(QL_E_UNSUPPORTED, "head_dim %d must be 64, 128 or 256", head_dim);
  if (r->rot_dim < 0 || r->rot_dim > head_dim || r->rot_dim % 16)
    return fail(QL_E_INVALID, "rot_dim %d must be a multiple of 16 in [0, head_dim]", r->rot_dim);
  if (r->interleaved != 0 && r->interleaved != 1) return fail(QL_E_INVALID, "interleaved must be 0 or 1");
  if (!(r->eps >= 0.0f)) return fail(QL_E_INVALID, "eps must be >= 0");
  if (r->max_pos < 0 || r->max_pos > (int64_t(1) << 40)) return fail(QL_E_INVALID, "max_pos outside [0, 2^40]");
  if (!aligned16(r->q_weight) || !aligned16(r->k_weight))
    return fail(QL_E_ALIGN, "norm weights must be 16-byte aligned");
  if (tokens > 0 && (q_heads > 0 || kv_heads > 0)) {
    if (r->rot_dim > 0 && r->max_pos > 0 && !r->cos_sin) return fail(QL_E_INVALID, "cos_sin is NULL");
    if (!positions) return fail(QL_E_INVALID, "positions is NULL");
  }
  if (!aligned(r->cos_sin, 4) || !aligned(positions, 8)) return fail(QL_E_ALIGN, "cos_sin or positions misaligned");
  a->q_w = static_cast<const uint16_t*>(r->q_weight);
  a->k_w = static_cast<const uint16_t*>(r->k_weight);
  a->table = r->cos_sin;
  a->pos = positions;
  a->max_pos = r->max_pos;
  a->eps = r->eps;
  a->tokens = (int)tokens;
  a->q_heads = q_heads;
  a->kv_heads = kv_heads;
  a->rot = r->rot_dim;
  a->interleaved = r->interleaved;
  return QL_OK;
}

// Rows (new tokens x query heads of a KV head) of a sequence up to which the
// stream kernel serves it; in a batch that has longer ones too, up to which
// sequences get a stream launch of their own.  More than 32 rows it would not hold
// in registers.  With 17 to 32 rows the tile kernel is the faster one where all
// sequences are about as long as the plan's bound, the slower one where they are
// not, as in a server's batches and captured steps.  Stream and tile kernel, us, 5
// new tokens of 32 / 8 heads of 128: 16 sequences of 500 keys 19.7 and 13.7 (bf16),
// of 4,000 60.1 and 56.8 (E4M3: 40.4 and 46.7); 64 of 1,000 59.5 and 50.6; with 8
// new tokens 64.9 and 51.6.  16 of 515 .. 4,099 38.7 and 50.0, 64 of 200 .. 8,000 192
// and 240 (64-wide: 110 and 181); 16 of 4,000 under a bound of 32,768 59.8 and 106.
// The stream kernel also holds the weights more exactly.
constexpr int64_t kStreamRows = 32;
constexpr int64_t kMixedRows = 16;

constexpr int kTileRows = 128;

// A grid's extent is a 32-bit number of threads, 256 a workgroup.
constexpr int64_t kMaxWorkgroups = int64_t(1) << 24;

// Chunk of the tile kernel.  A workgroup runs at its own pace, 512 of them at a
// time (two a compute unit).  Measured in ns a key: 19 while every workgroup has
// a compute unit to itself, 33 when two share one (64-wide heads: 14 and 23.5);
// 4 us around that; for a cut the join's launch (6 us) and its traffic (0.02 us a
// workgroup's partial result, more where they outgrow the caches).  The plan
// knows the longest context only: a batch is taken to have 3/4 of that on
// average, and the last round to be half full.  Takes the number of chunks that
// this makes cheapest.  Best and taken in us, over 1 .. 16 chunks: 9 x 475 new
// tokens at 2,732 .. 7,023, 16 / 16 heads, 192 and 192 (1 chunk; 2: 294); 512 at 8,192
// 85 and 85 (4; 1: 157); 64 at 8,192 25 and 26 (16); 4 x 140 at 507 .. 2,506, 64-wide, 33
// and 33 (2; 1: 40); 8 x 1,024 at 4,096 492 and 492 (1; 2: 675).
int64_t tile_chunk(int head_dim, int64_t batch, int64_t units, int64_t span) {
  const double alone = head_dim == 64 ? 0.0142 : 0.019, shared = head_dim == 64 ? 0.0235 : 0.033;
  int64_t best = span;
  double least = 0;
  for (int64_t s = 1; s == 1 || (s <= 64 && span / s >= 256); ++s) {
    const int64_t chunk = ((span + s - 1) / s + 63) / 64 * 64;
    const double groups = (double)(units * s) * (batch > 1 ? 0.75 : 1.0), x = groups / 512;
    const double rounds = x <= 1.0 ? 1.0 : (x + std::ceil(x)) / 2;
    // between 256 and 512 the units that share take longest, unless they are the short ones
    const double both = batch > 1 ? std::min(1.0, std::max(0.0, groups / 256 - 1.0)) : groups > 256 ? 1.0 : 0.0;
    const double pace = alone + (shared - alone) * both;
    const double us = rounds * (4.0 + (double)chunk * pace) + (s > 1 ? 6.0 + groups * 0.02 : 0.0);
    if (s == 1 || us < least) {
      least = us;
      best = chunk;
    }
  }
  return std::max<int64_t>(best, 64);
}

// The most keys that a unit's rows can see, from the 64-aligned start of
// their window.
int64_t tile_span(const ql_attention_shape& s) {
  if (!s.window) return s.max_kv;
  return std::min<int64_t>(s.max_kv, (int64_t)s.window + kTileRows / (s.q_heads / s.kv_heads) + 2 + 64);
}

// Cuts a batch into units of kTileRows rows and their keys into chunks.
// `at`: free workspace.  Units are numbered in whichever way takes fewer numbers
// (the others' workgroups end at once): by the rows there are for batches of
// mixed lengths, so that neither the grid nor the workspace grows with batch
// times the longest sequence; sequence by sequence where all may be full (4 x
// 512 new tokens at 2,000, 64-wide: 49.2 us so, 54.3 by rows; 256 x 5 of 8 heads
// at 100 .. 700: 100.7 and 106.3; 12 x up to 701, 64-wide E4M3: 83.0 and 82.3).
// Partial results are kept for rows that exist (a chunk of 2,048 tokens beside
// 31 single ones, 32 / 8 heads, contexts of up to 32,768: 277 MB; 8.7 GB for
// every sequence's units).
ql_status plan_tile(const ql_attention_shape& s, int64_t rows, int64_t at, Part* p) {
  const int64_t group = s.q_heads / s.kv_heads, R = kTileRows;
  const int64_t blocks = (rows + R - 1) / R;
  const int64_t by_rows = s.tokens * group / R + s.batch;
  const int64_t units = std::min(s.batch * blocks, by_rows) * s.kv_heads;
  const int64_t span = tile_span(s);
  const int64_t chunk = tile_chunk(s.head_dim, s.batch, units, span);
  const int64_t splits = std::max<int64_t>(1, (span + chunk - 1) / chunk);
  if (s.tokens * s.q_heads >= (int64_t(1) << 31)) return fail(QL_E_UNSUPPORTED, "tokens * q_heads exceeds 2^31");
  const int64_t parts = splits > 1 ? s.tokens * s.q_heads * splits : 0;
  // both launches fit a grid (the join's: a wave a row), or neither is made
  if (units * splits >= kMaxWorkgroups || (parts && s.tokens * s.q_heads / 4 + s.kv_heads >= kMaxWorkgroups))
    return fail(QL_E_UNSUPPORTED, "2^24 workgroups or more");
  p->used = true;
  p->rows = (int)R;
  p->row_blocks = (int)blocks;
  p->splits = (int)splits;
  p->chunk = (int)chunk;
  p->units = (int)units;
  p->by_rows = by_rows < s.batch * blocks;
  p->o_at = at;
  p->ml_at = at + parts * s.head_dim * 4;
  p->end = p->ml_at + parts * 2 * 4;
  return QL_OK;
}

// The stream kernel for sequences of at most `rows` rows: the shares of the
// keys are cut on the device, the plan fixes how many there can be.
ql_status plan_stream(const ql_attention_shape& s, int64_t rows, Part* p) {
  const int64_t tiles = s.batch * (s.max_kv / 32 + 1);
  if (tiles >= (int64_t(1) << 31)) return fail(QL_E_UNSUPPORTED, "batch * max_kv / 32 exceeds 2^31");
  p->used = true;
  p->rows = rows <= 16 ? 16 : 32;
  p->most = (int)rows;
  p->heads_wg = s.kv_heads % 4 == 0 ? 4 : s.kv_heads % 2 == 0 ? 2 : 1;
  p->slots = qlk::attn_stream_slots(s.head_dim, s.kv_type == QL_KV_E4M3, p->rows, s.kv_heads, p->heads_wg);
  if ((int64_t)p->slots * s.kv_heads >= (int64_t(1) << 31) || rows * s.kv_heads >= (int64_t(1) << 31))
    return fail(QL_E_UNSUPPORTED, "more than 2^31 workgroups");
  // sequences that fit a slot each are never cut
  const int64_t whole = s.batch <= std::min(64, p->slots) ? 32 << qlk::kStreamPad : 32;
  const int64_t parts = s.max_kv > whole ? (int64_t)p->slots * 2 * s.kv_heads * p->rows : 0;
  p->splits = parts ? 2 : 1;
  p->ml_at = parts * s.head_dim * 4;
  p->end = p->ml_at + parts * 2 * 4;
  return QL_OK;
}

}  // namespace

extern "C" {

ql_status qlinear_qk_norm_rope(const ql_norm_rope* rule, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                               int32_t head_dim, const ql_rows* q, const ql_rows* k, const int64_t* positions,
                               const ql_rows* q_out, const ql_rows* k_out, void* stream) {
  qlk::HeadArgs a{};
  ql_status st = check_rule(rule, tokens, q_heads, kv_heads, head_dim, positions, &a);
  if (st != QL_OK) return st;
  if (tokens == 0 || q_heads + kv_heads == 0) return QL_OK;
  if (q_heads && ((st = check_rows(q, "q", q_heads, &a.q)) != QL_OK || (st = check_rows(q_out, "q_out", q_heads, &a.q_out)) != QL_OK))
    return st;
  if (kv_heads && ((st = check_rows(k, "k", a.kv_heads, &a.k)) != QL_OK || (st = check_rows(k_out, "k_out", a.kv_heads, &a.k_out)) != QL_OK))
    return st;
  hipError_t e = qlk::launch_heads(a, head_dim, false, false, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? QL_OK : hip_fail(e, "norm and rotation launch");
}

ql_status qlinear_qkv_append(const ql_norm_rope* rule, int64_t tokens, int32_t q_heads, const ql_rows* q,
                             const ql_rows* k, const ql_rows* v, const int64_t* positions, const int64_t* slots,
                             const ql_rows* q_out, const ql_kv_cache* cache, void* stream) {
  qlk::HeadArgs a{};
  ql_status st = check_cache(cache, &a.kc, &a.vc);
  if (st != QL_OK) return st;
  st = check_rule(rule, tokens, q_heads, cache->kv_heads, cache->head_dim, positions, &a);
  if (st != QL_OK) return st;
  if (tokens == 0) return QL_OK;
  if (q_heads && ((st = check_rows(q, "q", q_heads, &a.q)) != QL_OK || (st = check_rows(q_out, "q_out", q_heads, &a.q_out)) != QL_OK))
    return st;
  if ((st = check_rows(k, "k", a.kv_heads, &a.k)) != QL_OK || (st = check_rows(v, "v", a.kv_heads, &a.v)) != QL_OK) return st;
  if (!slots) return fail(QL_E_INVALID, "slots is NULL");
  if (!aligned(slots, 8)) return fail(QL_E_ALIGN, "slots is not 8-byte aligned");
  a.slots = slots;
  a.num_slots = cache->num_pages * cache->page_size;
  a.page_size = cache->page_size;
  a.page_magic = page_magic(cache->page_size);
  hipError_t e = qlk::launch_heads(a, cache->head_dim, true, cache->type == QL_KV_E4M3, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? QL_OK : hip_fail(e, "cache append launch");
}

ql_status qlinear_attention_plan(const ql_attention_shape* s, ql_attention_plan* out) {
  if (!out) return fail(QL_E_INVALID, "out_plan is NULL");
  *out = nullptr;
  if (!s) return fail(QL_E_INVALID, "shape is NULL");
  if (s->batch < 0 || s->tokens < 0 || s->max_q < 0 || s->max_kv < 0) return fail(QL_E_INVALID, "negative size");
  if (s->tokens > kMaxTokens || s->max_q > kMaxTokens || s->batch > 65536 || s->max_kv > (int64_t(1) << 30))
    return fail(QL_E_UNSUPPORTED, "more than 2^24 new tokens, 2^16 sequences or 2^30 cached tokens");
  if (s->kv_heads < 1 || s->q_heads < 1 || s->q_heads % s->kv_heads)
    return fail(QL_E_INVALID, "q_heads %d must be a positive multiple of kv_heads %d", s->q_heads, s->kv_heads);
  if (s->q_heads > 65536) return fail(QL_E_UNSUPPORTED, "more than 2^16 heads");
  if (s->head_dim != 64 && s->head_dim != 128) return fail(QL_E_UNSUPPORTED, "head_dim %d must be 64 or 128", s->head_dim);
  if (s->kv_type != QL_KV_BF16 && s->kv_type != QL_KV_E4M3) return fail(QL_E_INVALID, "unknown cache type %d", s->kv_type);
  ql_status st = check_page_size(s->page_size);
  if (st != QL_OK) return st;
  if (s->causal != 0 && s->causal != 1) return fail(QL_E_INVALID, "causal must be 0 or 1");
  if (s->window < 0 || (s->window && !s->causal)) return fail(QL_E_INVALID, "a window is >= 0 and causal");
  if (!std::isfinite(s->scale) || s->scale < 0.0f) return fail(QL_E_INVALID, "scale must be finite and >= 0");
  const int64_t group = s->q_heads / s->kv_heads;
  const int64_t max_q = std::min(s->max_q, s->tokens);  // no sequence has more new tokens than there are
  const int64_t rows = max_q * group;
  if (rows > (int64_t(1) << 30)) return fail(QL_E_UNSUPPORTED, "max_q * q_heads / kv_heads exceeds 2^30");
  ql_attention_plan_s* p = new (std::nothrow) ql_attention_plan_s();
  if (!p) return fail(QL_E_INVALID, "out of host memory");
  p->shape = *s;
  // as long as any context: no window (and no position minus the window leaves 32 bits)
  if (s->window >= s->max_kv) p->shape.window = 0;
  s = &p->shape;
  const bool chunks = rows > kStreamRows;
  // Sequences of few rows among longer ones get a launch of their own where
  // there can be many of them with long contexts: to the tile kernel each is a
  // workgroup of mostly idle rows for each KV head.  By the (sequence, KV head,
  // key) triples that this would take, apart and together, us: 48 k (a chunk of 64
  // and 7 x 1,000) 34 and 24; 84 k (12 sequences, 701 new tokens at most, window
  // 2048, 64-wide) 103 and 93; 240 k (4 x 128 and 60 x 500, 64-wide) 35 and 35; 480 k
  // (256 and 15 x 4,000) 116 and 112; 504 k (100 and 63 x 1,000) 76 and 118; 744 k
  // (1,024 and 31 x 3,000) 116 and 227; 4 M (512 and 63 x 8,000) 491 and 974.
  const int64_t few = max_q > 0 ? s->batch - (s->tokens + max_q - 1) / max_q : 0;
  // (More query heads a KV head than that launch takes rows: none would go there.)
  const bool mixed = chunks && group <= kMixedRows && few * s->kv_heads * tile_span(*s) > 160000;
  p->tile_from = mixed ? kMixedRows + 1 : 0;
  if (!chunks || mixed) st = plan_stream(*s, mixed ? kMixedRows : rows, &p->stream);
  if (st == QL_OK && chunks) st = plan_tile(*s, rows, p->stream.end, &p->tile);
  if (st != QL_OK) {
    delete p;
    return st;
  }
  *out = p;
  return QL_OK;
}

ql_status qlinear_attention_plan_info(ql_attention_plan p, ql_attention_facts* facts) {
  if (!p || !facts) return fail(QL_E_INVALID, "NULL argument");
  *facts = ql_attention_facts{p->stream.used ? p->stream.rows : 0, p->stream.slots, p->tile.used ? p->tile.rows : 0,
                              p->tile.row_blocks, p->tile.splits, p->tile.chunk,
                              qlinear_attention_workspace_bytes(p)};
  return QL_OK;
}

int64_t qlinear_attention_workspace_bytes(ql_attention_plan p) { return p ? std::max(p->stream.end, p->tile.end) : 0; }

void qlinear_attention_plan_destroy(ql_attention_plan p) { delete p; }

ql_status qlinear_attention(ql_attention_plan p, const ql_rows* q, const ql_kv_cache* cache,
                            const int32_t* page_table, int64_t table_stride, const int32_t* seq_lens,
                            const int32_t* cu_q, const ql_rows* out, float* lse, void* workspace, void* stream) {
  if (!p) return fail(QL_E_INVALID, "plan is NULL");
  const ql_attention_shape& s = p->shape;
  qlk::AttnArgs a{};
  ql_status st = check_cache(cache, &a.kc, &a.vc);
  if (st != QL_OK) return st;
  if (cache->type != s.kv_type || cache->kv_heads != s.kv_heads || cache->head_dim != s.head_dim ||
      cache->page_size != s.page_size)
    return fail(QL_E_INVALID, "the cache is not of the plan's type, heads, head_dim and page_size");
  if (s.batch == 0 || s.tokens == 0 || s.max_q == 0) return QL_OK;
  if ((st = check_rows(q, "q", s.q_heads, &a.q)) != QL_OK || (st = check_rows(out, "out", s.q_heads, &a.out)) != QL_OK) return st;
  if ((!page_table && s.max_kv > 0) || !seq_lens || !cu_q) return fail(QL_E_INVALID, "page_table, seq_lens or cu_q is NULL");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(lse, 4))
    return fail(QL_E_ALIGN, "page_table, seq_lens, cu_q and lse must be 4-byte aligned");
  if (s.batch > 1 && table_stride < (s.max_kv + s.page_size - 1) / s.page_size)
    return fail(QL_E_INVALID, "page_table rows hold fewer than ceil(max_kv / page_size) entries");
  if (qlinear_attention_workspace_bytes(p) > 0 && !workspace) return fail(QL_E_INVALID, "this plan needs a workspace");
  if (!aligned16(workspace)) return fail(QL_E_ALIGN, "workspace is not 16-byte aligned");
  // without any context the table may have no entry, but the decode kernel looks
  // up a page for every sequence (and clamps it)
  a.table = s.max_kv > 0 ? page_table : seq_lens;
  a.table_row = s.max_kv > 0 ? table_stride : 0;
  a.seq_lens = seq_lens;
  a.cu_q = cu_q;
  a.lse = lse;
  a.page_magic = page_magic(s.page_size);
  const float scale = s.scale != 0.0f ? s.scale : 1.0f / std::sqrt((float)s.head_dim);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.batch = (int)s.batch;
  a.tokens = (int)s.tokens;
  a.q_heads = s.q_heads;
  a.kv_heads = s.kv_heads;
  a.group = s.q_heads / s.kv_heads;
  a.page_size = s.page_size;
  a.num_pages = (int)cache->num_pages;
  a.max_kv = (int)s.max_kv;
  a.causal = s.causal;
  a.window = s.window;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  const bool e4m3 = s.kv_type == QL_KV_E4M3;
  auto partials = [&](const Part& x) {
    a.part_o = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + x.o_at) : nullptr;
    a.part_ml = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + x.ml_at) : nullptr;
  };
  hipError_t e = hipSuccess;
  if (p->stream.used) {
    const Part& x = p->stream;
    partials(x);
    a.slots = x.slots;
    a.heads_wg = x.heads_wg;
    a.max_rows = x.most;
    e = qlk::launch_attn_stream(a, s.head_dim, e4m3, x.rows, hs);
    if (e == hipSuccess && x.splits > 1) e = qlk::launch_attn_stream_join(a, s.head_dim, x.rows, x.most, hs);
  }
  if (e == hipSuccess && p->tile.used) {
    const Part& x = p->tile;
    partials(x);
    a.row_blocks = x.row_blocks;
    a.by_rows = x.by_rows;
    a.splits = x.splits;
    a.chunk = x.chunk;
    a.min_rows = p->tile_from;
    e = qlk::launch_attn_tile(a, s.head_dim, e4m3, x.units, hs);
    if (e == hipSuccess && x.splits > 1) e = qlk::launch_attn_join(a, s.head_dim, x.rows, hs);
  }
  return e == hipSuccess ? QL_OK : hip_fail(e, "attention launch");
}

// Slices of a vocabulary row: enough workgroups for the card with few
// sequences, at least 1024 entries (4 a thread) each, at most kVerifySlice.  With
// 512, 1,024 and 2,048 workgroups, us: 4 x 151,936 entries 7.4, 7.9, 7.9; 16 x 151,936
// 10.9, 10.2, 10.5; 64 x 32,001 9.8, 9.4, 10.1.
static int verify_slices(int64_t batch, int64_t vocab) {
  const int64_t most = std::max<int64_t>(1, vocab / 1024), least = (vocab + qlk::kVerifySlice - 8) / (qlk::kVerifySlice - 4);
  return (int)std::max<int64_t>({1, least, std::min<int64_t>(most, 1024 / std::max<int64_t>(1, batch))});
}

int64_t qlinear_verify_workspace_bytes(int64_t batch, int64_t vocab) {
  if (batch <= 0 || vocab <= 0) return 0;
  return (batch * verify_slices(batch, vocab) * 8 + 15) / 16 * 16;
}

ql_status qlinear_verify_draft(int64_t batch, int64_t n_drafts, int64_t max_drafts, int64_t vocab,
                               const float* target_probs, const float* draft_probs, const int32_t* draft_tokens,
                               const int32_t* cu_drafts, const float* uniforms, const float* noise,
                               int32_t* out_tokens, int32_t* accepted, void* workspace, void* stream) {
  if (batch < 0 || n_drafts < 0 || max_drafts < 0 || vocab < 0) return fail(QL_E_INVALID, "negative size");
  if (batch > 65535 || n_drafts > kMaxTokens || max_drafts > 65536 || vocab > (int64_t(1) << 30))
    return fail(QL_E_UNSUPPORTED, "more than 65535 sequences, 2^24 drafts or 2^30 tokens of vocabulary");
  if (batch == 0) return QL_OK;
  if (vocab == 0) return fail(QL_E_INVALID, "the vocabulary is empty");
  if (!target_probs || !cu_drafts || !noise || !out_tokens || !accepted || !workspace)
    return fail(QL_E_INVALID, "NULL pointer");
  if (n_drafts > 0 && (!draft_tokens || !uniforms)) return fail(QL_E_INVALID, "draft_tokens or uniforms is NULL");
  for (const void* p : {(const void*)target_probs, (const void*)draft_probs, (const void*)draft_tokens,
                        (const void*)cu_drafts, (const void*)uniforms, (const void*)noise, (const void*)out_tokens,
                        (const void*)accepted})
    if (!aligned(p, 4)) return fail(QL_E_ALIGN, "pointers must be 4-byte aligned");
  if (!aligned16(workspace)) return fail(QL_E_ALIGN, "workspace is not 16-byte aligned");
  qlk::VerifyArgs a{};
  a.target = target_probs;
  a.draft = draft_probs;
  a.tokens = draft_tokens;
  a.cu = cu_drafts;
  a.uniforms = uniforms;
  a.noise = noise;
  a.out_tokens = out_tokens;
  a.accepted = accepted;
  a.part = static_cast<uint64_t*>(workspace);
  a.n_drafts = n_drafts;
  a.batch = (int)batch;
  a.vocab = (int)vocab;
  a.max_drafts = (int)max_drafts;
  a.slices = verify_slices(batch, vocab);
  hipError_t e = qlk::launch_verify(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? QL_OK : hip_fail(e, "draft verification launch");
}

}  // extern "C"
