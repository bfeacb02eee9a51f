// Attention over the paged cache for few rows a sequence: the decode kernel.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale q_r.k_j - m_r),
// in one pass over the keys with the running maximum m_r and sum of each row.
//
// Few rows (new tokens x query heads of a KV head) read long K and V, 2
// bytes (E4M3: 1) for 2 flops a row and value: bound by memory up to about
// 150 rows.  So the kernel is built as a stream.
//
// All sequences' keys, in tiles of 32, are laid end to end and cut into equal
// slots, one a wave and KV head, as many as the card holds at once: every wave
// starts at once, reads the same amount and ends at the same time, whatever
// the lengths.  (Chunks of one length in a grid of all sequences' longest left
// the compute units idle for 40 % of the time: sequences end at different
// chunks.)  A wave that passes from one sequence to the next writes the first
// one's result and starts over; where a sequence lies in several slots their
// results are partial and the join kernel adds them.  There are no barriers
// and no LDS; waves of a workgroup take the heads of the same keys, which lie
// next to each other in memory, and workgroups of the same slot follow each
// other on one XCD.
//
// Operands (16x16x32 bf16; lane l = 16 g + r):
//   S^T = K Q^T: the first operand is 16 keys (key r of the group in lane r)
//     with 8 of their values each, so a lane loads 16 contiguous bytes of a
//     key; Q is held with the same values in the same places.
//   The result has keys 4g .. 4g+3 of query row r in lane l.  With the keys of
//   two groups next to each other that is the second operand of
//   O^T = V^T P^T as it stands: P never moves between lanes.
//   V^T: a lane loads D/16 contiguous values of the 8 keys that its P has
//     (whole rows of V per 16 lanes), and the 8 x D/16 transposition into
//     operands stays inside the lane (one byte permutation per two values).
//     So output value d sits in operand row d / (D/16) of product d % (D/16).
// The maximum that a row's weights refer to moves where a new one exceeds it by
// more than 8 (in base 2): its tests need no exchange between lanes, and most
// tiles leave the outputs as they are.
// P enters the product as two bf16 numbers, itself rounded and what that left
// out, so that its error is 2^-16 of a term and an output's own rounding is the
// only one to 16 bits.  The second product is behind the memory: 32 x 8,190 keys
// 101.0 us without and 101.3 with it, 64 x 16,001 in E4M3 214.9 and 215.4, 16 x 5
// at 4,000 59.6 and 60.3; at most 3 % (32 x 5 at 4,000, E4M3, 70.2 and 72.5).
// Row sums take P in binary32, and all sums and maxima are binary32.
//
// Measured on MI355X, against 7.05 TB/s of a streaming read: 32 sequences of
// 1,021 .. 8,190 keys, 64 / 8 heads of 128, bf16 (605 MB) 97 us and the join's 5; 64
// of 4,003 .. 16,001, 40 / 8 heads, E4M3 (1.31 GB) 210 and 6; 5 x 4 rows of each of 16
// sequences of 515 .. 4,099, bf16 (153 MB) 33 and 6; one of 1,031 keys 7 and 4, all
// of it latency.
#include "attention_common.hpp"

namespace qlk {

constexpr int kStreamWaves = 4;

// A sequence has kMostPieces slots at most, a slot 2^kStreamPad tiles at least:
// shorter slots, more partial results.  One sequence of 1,000 keys: 10.6, 11.3,
// 12.4 us with 1, 2, 3 tiles; of 2,000: 13.5, 12.7, 13.7 (30 sequences of 44 keys,
// 4 x 7 rows: 15.0, 11.0 with 1, 2).  One of 16,000, E4M3: 21.2, 17.4, 19.2 us with
// 256, 128, 80 slots; 8 new tokens of it 24.8, 25.0, 23.7.
constexpr int kMostPieces = 128;

// One wave's 32 keys: K operands and V rows as they come from memory.
template <int D, bool E4M3>
struct KvTile {
  static constexpr int KP = E4M3 ? D / 64 : D / 32;  // 16-byte pieces of a key a lane holds
  static constexpr int VW = E4M3 ? D / 64 : D / 32;  // words of a value row a lane holds (D/16 values)
  u32x4 k[2][KP];
  uint32_t v[8][VW];
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* o) {
  if constexpr (N == 4) {
    const u32x4 t = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = t[i];
  } else if constexpr (N == 2) {
    const u32x2 t = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    o[0] = t.x;
    o[1] = t.y;
  } else {
    o[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
  }
}

// Loads a tile's K or V: its two 16-key groups are entries i and i + 1 of `at`.
template <int D, bool E4M3>
__device__ __forceinline__ void load_k(const AttnArgs& a, const Groups& at, int i, uint32_t lane, KvTile<D, E4M3>* t) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* k = a.kc.p + pick(at.k_lo, at.k_hi, i + u);
#pragma unroll
    for (int s = 0; s < KvTile<D, E4M3>::KP; ++s) t->k[u][s] = *reinterpret_cast<const u32x4*>(k + lane + 64 * s);
  }
}

template <int D, bool E4M3>
__device__ __forceinline__ void load_v(const AttnArgs& a, const Groups& at, int i, uint32_t lane, KvTile<D, E4M3>* t) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* v = a.vc.p + pick(at.v_lo, at.v_hi, i + u);
#pragma unroll
    for (int j = 0; j < 4; ++j) load_words<KvTile<D, E4M3>::VW>(v + j * (int)a.vc.token + lane, t->v[4 * u + j]);
  }
}

// One sequence of the stream: its new tokens, cached length and tiles.  lo is
// the first key that any of its rows sees.
struct Seq {
  int first, n, len, lo, tiles;
};

// Sequence b as this lane's own (b < batch; no tiles if it has no rows here).
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  Seq s = {0, 0, 0, 0, 0};
  if (b < a.batch) {
    const int q0 = min(max(a.cu_q[b], 0), a.tokens);
    const int q1 = min(max(a.cu_q[b + 1], q0), a.tokens);
    s.first = q0;
    s.n = q1 - q0;
    s.len = min(max(a.seq_lens[b], 0), a.max_kv);
    s.lo = a.window ? min(s.len, max(0, s.len - s.n - a.window + 1)) : 0;
    // rows without any key still need one tile to be written
    if (s.n > 0 && s.n * a.group <= a.max_rows) s.tiles = max(1, (s.len - (s.lo & ~31) + 31) >> 5);
  }
  return s;
}

// All sequences' tiles, and how they are cut: `slots` slots of `each` tiles,
// the first `more` of them one longer.  A sequence takes room for a multiple of
// 2^pad tiles.
struct Cut {
  int slots, each, more, pad;
  __device__ __forceinline__ int start(int j) const { return j * each + min(j, more); }
  __device__ __forceinline__ int slot_of(int t) const {
    if (pad) return t >> pad;
    const int longer = more * (each + 1);
    return t < longer ? t / (each + 1) : more + (t - longer) / each;
  }
  __device__ __forceinline__ int room(int tiles) const { return (tiles + (1 << pad) - 1) >> pad << pad; }
};

// The cut of a batch whose first sequences the lanes hold, and the tiles up to
// theirs.  Where the slots suffice, each lies in one sequence: a slot that
// passes to a second one waits for its page table, then for its keys (15
// sequences of 400 keys, E4M3: 17.5 us so, 15.1 with a sequence a slot; 8 of 30
// keys: 11.3 and 6.9).  Else all slots are equally long.
__device__ __forceinline__ Cut cut_of(const AttnArgs& a, const Seq& mine, int* upto) {
  int most = a.slots;
  if (a.batch <= 64) {
    most = min(most, kMostPieces * a.batch);
    const int pieces = inclusive_sum((mine.tiles + (1 << kStreamPad) - 1) >> kStreamPad), slots = lane_i32(pieces, 63);
    if (slots <= most) {
      *upto = pieces << kStreamPad;
      return Cut{slots, 1 << kStreamPad, 0, kStreamPad};
    }
  }
  *upto = inclusive_sum(mine.tiles);
  int total = lane_i32(*upto, 63);
  for (int b0 = 64; b0 < a.batch; b0 += 64) total += lane_i32(inclusive_sum(seq_of(a, b0 + (threadIdx.x & 63)).tiles), 63);
  Cut c;
  c.slots = min(most, (total + (1 << kStreamPad) - 1) >> kStreamPad);
  c.each = total / max(1, c.slots);
  c.more = total - c.each * c.slots;
  c.pad = 0;
  return c;
}

// The 16-key groups of the 32 tiles of a sequence from key `key` on: lane i
// holds group i % 2 of tile i / 2.
__device__ __forceinline__ Groups tile_groups(const AttnArgs& a, const int32_t* table, int h, int key, int last) {
  return groups_at(a, table, h, (key >> 4) + (threadIdx.x & 63), last);
}

// Operand k of the products over D for the 16 keys v: 8 values of one key.
template <int D, bool E4M3>
__device__ __forceinline__ u32x4 k_operand(const KvTile<D, E4M3>& t, int v, int k) {
  if constexpr (!E4M3) return t.k[v][k];
  const uint32_t c0 = t.k[v][k / 2][k % 2 * 2], c1 = t.k[v][k / 2][k % 2 * 2 + 1];
  return u32x4{e4m3_to_bf16<false>(c0), e4m3_to_bf16<true>(c0), e4m3_to_bf16<false>(c1), e4m3_to_bf16<true>(c1)};
}

// V^T operand of product dt from a tile's value rows: 8 keys of one value.
template <int D, bool E4M3>
__device__ __forceinline__ u32x4 v_operand(const KvTile<D, E4M3>& t, int dt) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E4M3) {  // the same permutation serves products dt and dt ^ 1
      const uint32_t c = __builtin_amdgcn_perm(t.v[2 * i + 1][dt / 4], t.v[2 * i][dt / 4],
                                               dt % 4 < 2 ? 0x05010400u : 0x07030602u);
      o[i] = dt % 2 ? e4m3_to_bf16<true>(c) : e4m3_to_bf16<false>(c);
    } else {
      o[i] = __builtin_amdgcn_perm(t.v[2 * i + 1][dt / 2], t.v[2 * i][dt / 2], dt % 2 ? 0x07060302u : 0x05040100u);
    }
  }
  return o;
}

// Whether a tile's values (of this lane) have infinities or NaNs: the exponent
// (E4M3: the code's lower seven bits) all ones.  And without them.
template <int D, bool E4M3>
__device__ __forceinline__ bool has_nonfinite(const KvTile<D, E4M3>& t) {
  uint32_t any = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int w = 0; w < KvTile<D, E4M3>::VW; ++w)
      any |= E4M3 ? (t.v[j][w] & 0x7f7f7f7fu) + 0x01010101u : (t.v[j][w] & 0x7f807f80u) + 0x00800080u;
  return any & (E4M3 ? 0x80808080u : 0x80008000u);
}
template <int D, bool E4M3>
__device__ __forceinline__ void drop_nonfinite(KvTile<D, E4M3>& t) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int w = 0; w < KvTile<D, E4M3>::VW; ++w) t.v[j][w] &= finite_mask<E4M3>(t.v[j][w]);
}

// Workgroups a compute unit gets.  Measured, one and two: 32 sequences of 4,600
// keys, 64 / 8 heads, bf16 99.2 and 106.0 us (16 of 4,000, 64-wide heads: 29.3 and
// 31.2); E4M3, 64 of 9,000 200.3 and 201.0 us, 64-wide heads of 3,000 56.4 and 47.0,
// of 8,000 134.8 and 109.7, 5 x 4 rows of 32 of 4,000 46.1 and 43.0.  More requests on
// their way than that only queue; E4M3's are half as large.  With 32 rows the sums
// of 128-wide heads leave one workgroup its registers (32 sequences of 5 x 4 rows,
// 4,000 keys, E4M3: 71.6 us, 72.7 with two; bf16 100.6 and 118.1).
constexpr int stream_workgroups(int D, bool e4m3, int row_tiles) { return e4m3 && (row_tiles == 1 || D == 64) ? 2 : 1; }

// Tiles that a wave has in its registers: a compute unit's only workgroup asks
// for a second one while it works on the first (32 sequences of 5 x 4 rows and
// 4,000 keys, with one and two: E4M3 75.0 and 71.6 us, 64-wide bf16 62.2 and
// 58.8); where there are two, they cover each other (64-wide E4M3, 64 single tokens:
// 3,000 keys 47.0 and 47.9 us, 8,000 keys 109.7 and 109.6).
constexpr int stream_depth(int D, bool e4m3, int row_tiles) { return stream_workgroups(D, e4m3, row_tiles) == 1 ? 2 : 1; }

template <int D, bool E4M3, int NR, bool TREE>
__global__ void __launch_bounds__(kStreamWaves * 64, stream_workgroups(D, E4M3, NR)) attn_stream_kernel(AttnArgs a) {
  constexpr int R = 16 * NR, DT = D / 16;
  constexpr int KS = D / 32;  // products over D of one 16-key group
  using Tile = KvTile<D, E4M3>;
  constexpr int DEPTH = stream_depth(D, E4M3, NR);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int head_groups = a.kv_heads / a.heads_wg;
  const int h = (int)(blockIdx.x / 8) % head_groups * a.heads_wg + wave % a.heads_wg;
  const int slot = ((int)(blockIdx.x / 8) / head_groups * 8 + (int)blockIdx.x % 8) * (kStreamWaves / a.heads_wg) +
                   wave / a.heads_wg;

  // the tiles of all sequences, 64 sequences at a time; `before`: of those
  // before the ones the lanes hold
  Seq mine = seq_of(a, lane);
  int upto, before = 0, base = 0;
  const Cut cut = cut_of(a, mine, &upto);
  if (slot >= cut.slots) return;
  int t = cut.start(slot);
  const int t_begin = t, t_end = cut.start(slot + 1);

  const float scale = a.scale_log2 * (E4M3 && a.kc.scale ? a.kc.scale[h] : 1.0f);
  const float v_scale = E4M3 && a.vc.scale ? a.vc.scale[h] : 1.0f;
  const uint32_t k_lane = (uint32_t)(r * (int)a.kc.token + g * 16);
  const uint32_t v_lane = (uint32_t)(4 * g * (int)a.vc.token + r * Tile::VW * 4);

  while (t < t_end) {
    // the sequence that tile t belongs to
    while (before + lane_i32(upto, 63) <= t) {
      before += lane_i32(upto, 63);
      base += 64;
      mine = seq_of(a, base + lane);
      upto = inclusive_sum(mine.tiles);  // more than 64 sequences: without padding
    }
    const int i = __ffsll((unsigned long long)__ballot(before + upto > t)) - 1;
    const int b = base + i;
    const Seq s = {lane_i32(mine.first, i), lane_i32(mine.n, i), lane_i32(mine.len, i), lane_i32(mine.lo, i),
                   lane_i32(mine.tiles, i)};
    const int seq_end = before + lane_i32(upto, i), seq_begin = seq_end - cut.room(s.tiles);
    const int t_stop = min(t_end, seq_begin + s.tiles);
    const int rows = min(s.n * a.group, R), pos0 = s.len - s.n;
    int key = (s.lo & ~31) + (t - seq_begin) * 32;
    const int end = (s.lo & ~31) + (t_stop - seq_begin) * 32;

    const int32_t* table = a.table + (int64_t)b * a.table_row;
    const int last_sub = max(s.len - 1, 0) >> 4;
    Groups at = tile_groups(a, table, h, key, last_sub);

    // Q operands, and the keys each of this lane's rows sees
    u32x4 q[NR][KS];
    int lo[NR], hi[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int row = 16 * n + r, tok = row / a.group, head = h * a.group + row % a.group;
      hi[n] = row < rows ? a.causal ? min(s.len, max(0, pos0 + tok + 1)) : s.len : 0;
      lo[n] = a.window ? max(0, pos0 + tok - a.window + 1) : 0;
      const uint8_t* p = a.q.p + (int64_t)(s.first + tok) * a.q.token + (int64_t)head * a.q.head;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int d0 = E4M3 ? ((k / 2) * 4 + g) * 16 + (k % 2) * 8 : (k * 4 + g) * 8;
        q[n][k] = row < rows ? *reinterpret_cast<const u32x4*>(p + d0 * 2) : u32x4{0u, 0u, 0u, 0u};
      }
    }
    // keys that every row sees
    const int full_lo = a.window ? max(0, pos0 + (rows - 1) / a.group - a.window + 1) : 0;
    const int full_hi = TREE ? min(s.len, max(0, pos0)) : a.causal ? min(s.len, max(0, pos0 + 1)) : s.len;
    auto is_whole = [&](int key) { return key >= full_lo && key + 32 <= full_hi; };
    const int key0 = key;
    bool dropped = false;

    f32x4 o[NR][DT];
    float m[NR], l[NR], base[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      m[n] = kNegInf;
      l[n] = base[n] = 0.0f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[n][dt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // K of a later tile is on its way while the weights and sums of this one
    // are made, V while the next one's scores are
    int tile = DEPTH - 1;
    Tile ahead[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
      if (i == 0 || key + 32 * i < end) {
        load_k<D, E4M3>(a, at, 2 * i, k_lane, &ahead[i]);
        load_v<D, E4M3>(a, at, 2 * i, v_lane, &ahead[i]);
      }
    auto step = [&](Tile& cur) {
      float x[NR][8];
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < KS; ++k) c = mma_bf16(k_operand<D, E4M3>(cur, v, k), q[n][k], c);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[n][4 * v + j] = c[j];
        }
      const bool more = key + 32 * DEPTH < end;
      if (more) {
        if ((++tile & 31) == 0) at = tile_groups(a, table, h, key + 32 * DEPTH, last_sub);
        load_k<D, E4M3>(a, at, 2 * (tile & 31), k_lane, &cur);
      }
      if (key + 32 > s.len) {  // the cache beyond the sequence may hold anything: 0 * NaN would reach every row
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (key + 16 * (j / 4) + 4 * g + j % 4 >= s.len)
#pragma unroll
            for (int w = 0; w < Tile::VW; ++w) cur.v[j][w] = 0u;
      }
      const bool whole = is_whole(key);
      if (!whole && __any(has_nonfinite<D, E4M3>(cur))) {
        drop_nonfinite<D, E4M3>(cur);
        dropped = true;
      }
      u32x4 p[NR], rest[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        if (!whole) {
          int first = key + 4 * g;
          pin(first);
          uint32_t bits = 0xffffffffu;
          if (TREE) bits = tree_bits(a, s.first + min(16 * n + r, rows - 1) / a.group, key - pos0) >> 4 * g;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int k = first + 16 * (j / 4) + j % 4;
            x[n][j] = k >= lo[n] && k < hi[n] && (!TREE || bits >> (16 * (j / 4) + j % 4) & 1) ? x[n][j] : kNegInf;
          }
        }
        float top = x[n][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, x[n][j]);
        top *= scale;
        if (__any(top > m[n] + kRescaleAt)) {
          top = fmaxf(m[n], row4_max(top));
          base[n] = top == kNegInf ? 0.0f : top;  // a row that has seen no key yet
          const float keep = __builtin_amdgcn_exp2f(m[n] - base[n]);
          m[n] = top;
          l[n] *= keep;
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) o[n][dt] *= keep;
        }
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[n][j] = __builtin_amdgcn_exp2f(__fmaf_rn(x[n][j], scale, -base[n]));
          sum += x[n][j];
        }
        l[n] += sum;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = bf16_pair(x[n][2 * j], x[n][2 * j + 1]);
          p[n][j] = w;
          rest[n][j] = bf16_pair(x[n][2 * j] - __uint_as_float(w << 16), x[n][2 * j + 1] - __uint_as_float(w & 0xffff0000u));
        }
      }
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        const u32x4 v = v_operand<D, E4M3>(cur, dt);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          o[n][dt] = mma_bf16(v, rest[n], o[n][dt]);
          o[n][dt] = mma_bf16(v, p[n], o[n][dt]);
        }
      }
      if (more) load_v<D, E4M3>(a, at, 2 * (tile & 31), v_lane, &cur);
    };
    while (key < end) {
#pragma unroll
      for (int i = 0; i < DEPTH; ++i)
        if (key < end) {
          step(ahead[i]);
          key += 32;
        }
    }

    // the outputs that dropped values would have reached
    if (dropped) {
      for (key = key0; key < end; key += 32) {
        if (is_whole(key)) continue;
        for_nonfinite<D, E4M3>(a, table, h, key, min(32, s.len - key), [&](int k, const uint64_t (&bad)[D / 64]) {
          int d0 = 4 * g * DT;
          pin(d0);
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const bool named = !TREE || (tree_bits(a, s.first + min(16 * n + r, rows - 1) / a.group, k - pos0) & 1);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (named && k >= lo[n] && k < hi[n] && bad_at<D>(bad, d0 + j * DT + dt)) o[n][dt][j] = __uint_as_float(0x7fc00000u);
          }
        });
      }
    }

    // the sequence's output if all of it lies in this slot, else this slot's
    // share: number 0 if it is the slot's first sequence, else 1
    const bool alone = t_stop - t == s.tiles;
    const int64_t part = (((int64_t)slot * 2 + (t == t_begin ? 0 : 1)) * a.kv_heads + h) * R;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int row = 16 * n + r;
      const float sum = row4_sum(l[n]);
      if (row < rows) {
        const int tok = s.first + row / a.group, head = h * a.group + row % a.group;
        const float f = alone ? (sum > 0.0f || sum != sum ? v_scale / sum : 0.0f) : v_scale;  // no key seen: zero
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int d0 = (4 * g + j) * DT;
          float x[DT];
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) x[dt] = o[n][dt][j] * f;
          if (alone) {
            uint8_t* out = a.out.p + (int64_t)tok * a.out.token + (int64_t)head * a.out.head + d0 * 2;
            if constexpr (DT == 8)
              *reinterpret_cast<u32x4*>(out) = u32x4{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]),
                                                     bf16_pair(x[6], x[7])};
            else
              *reinterpret_cast<u32x2*>(out) = u32x2{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
          } else {
#pragma unroll
            for (int w = 0; w < DT; w += 4)
              *reinterpret_cast<f32x4*>(a.part_o + (part + row) * D + d0 + w) = f32x4{x[w], x[w + 1], x[w + 2], x[w + 3]};
          }
        }
        if (g == 0) {
          if (!alone) {
            a.part_ml[(part + row) * 2] = m[n];
            a.part_ml[(part + row) * 2 + 1] = sum;
          } else if (a.lse) {
            a.lse[(int64_t)tok * a.q_heads + head] = lse_of(m[n], sum);
          }
        }
      }
    }
    t = t_stop == seq_begin + s.tiles ? seq_end : t_stop;
  }
}

// A running softmax sum: maximum (base 2), sum and 4 values of the output.
struct Partial {
  float m, l;
  f32x4 x;
  __device__ __forceinline__ void add(float m2, float l2, const f32x4& x2) {
    const float top = fmaxf(m, m2), base = top == kNegInf ? 0.0f : top;
    const float e = __builtin_amdgcn_exp2f(m - base), e2 = __builtin_amdgcn_exp2f(m2 - base);
    m = top;
    l = l * e + l2 * e2;
    x = x * e + x2 * e2;
  }
};

// Adds `n` partial results of one row, by WAVES waves.  Entry 0 lies at row
// `first` of the partial results, entry c at second + (c - 1) step.  D/4 lanes
// take an entry, 16 bytes each, four entries on their way at once: what this
// costs is latency.
template <int D, int WAVES>
__device__ __forceinline__ void join_row(const AttnArgs& a, int64_t first, int64_t second, int64_t step, int n, int tok,
                                         int head) {
  constexpr int L = D / 4, P = 64 * WAVES / L;
  const int id = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x, d0 = id % L * 4;
  Partial p = {kNegInf, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
  for (int c = id / L; c < n; c += 4 * P) {
    float m[4], l[4];
    f32x4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = min(c + k * P, n - 1);
      const int64_t at = i == 0 ? first : second + (int64_t)(i - 1) * step;
      m[k] = a.part_ml[at * 2];
      l[k] = a.part_ml[at * 2 + 1];
      x[k] = *reinterpret_cast<const f32x4*>(a.part_o + at * D + d0);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k * P < n) p.add(m[k], l[k], x[k]);
  }
#pragma unroll
  for (int s = L; s < 64; s *= 2) {
    const float m = __shfl_xor(p.m, s, 64), l = __shfl_xor(p.l, s, 64);
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __shfl_xor(p.x[i], s, 64);
    p.add(m, l, x);
  }
  if constexpr (WAVES > 1) {
    __shared__ Partial shared[WAVES][L];
    if ((id & 63) < L) shared[id >> 6][id & 63] = p;
    __syncthreads();
    if (id >= L) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) p.add(shared[w][id].m, shared[w][id].l, shared[w][id].x);
  }
  const float inv = p.l > 0.0f || p.l != p.l ? 1.0f / p.l : 0.0f;
  if (id < L)
    *reinterpret_cast<u32x2*>(a.out.p + (int64_t)tok * a.out.token + (int64_t)head * a.out.head + d0 * 2) =
        u32x2{bf16_pair(p.x[0] * inv, p.x[1] * inv), bf16_pair(p.x[2] * inv, p.x[3] * inv)};
  if (a.lse && id == 0)
    a.lse[(int64_t)tok * a.q_heads + head] = lse_of(p.m, p.l);
}

constexpr int kJoinWaves = 4;

// The stream kernel's sequences that lie in several slots: WAVES waves a row.
// grid.y: sequences; grid.x: rows of all KV heads.
template <int D, int WAVES>
__global__ void __launch_bounds__(kJoinWaves * 64) attn_stream_join_kernel(AttnArgs a, int R) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int id = WAVES == 1 ? (int)blockIdx.x * kJoinWaves + wave : blockIdx.x;
  const int h = id % a.kv_heads, row = id / a.kv_heads, b = blockIdx.y;
  Seq s = seq_of(a, lane), mine = {0, 0, 0, 0, 0};
  int upto, seq_begin = 0;
  const Cut cut = cut_of(a, s, &upto);
  for (int b0 = 0;; b0 += 64, s = seq_of(a, b0 + lane), upto = inclusive_sum(s.tiles)) {
    if (b < b0 + 64) {
      const int i = b - b0;
      mine = Seq{lane_i32(s.first, i), lane_i32(s.n, i), 0, 0, lane_i32(s.tiles, i)};
      seq_begin += lane_i32(upto, i) - cut.room(mine.tiles);
      break;
    }
    seq_begin += lane_i32(upto, 63);
  }
  if (mine.tiles == 0 || row >= mine.n * a.group) return;
  const int s0 = cut.slot_of(seq_begin), s1 = cut.slot_of(seq_begin + mine.tiles - 1);
  if (s0 == s1) return;  // written by the stream kernel
  const int64_t step = (int64_t)a.kv_heads * R;
  const int64_t first = ((int64_t)s0 * 2 + (seq_begin == cut.start(s0) ? 0 : 1)) * step + (int64_t)h * R + row;
  join_row<D, WAVES>(a, first, (int64_t)(s0 + 1) * 2 * step + (int64_t)h * R + row, 2 * step, s1 - s0 + 1,
                     mine.first + row / a.group, h * a.group + row % a.group);
}

// The tile kernel's units that were cut into chunks: one wave a row of a KV
// head (new token, query head of the group).
template <int D>
__global__ void __launch_bounds__(kJoinWaves * 64) attn_join_kernel(AttnArgs a, int R) {
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int h = (int)blockIdx.x % a.kv_heads, at = (int)blockIdx.x / a.kv_heads * kJoinWaves + wave;
  if (at >= a.tokens * a.group) return;
  const Sequence s = sequence_at(a, at, [&](int, int q0) { return q0 * a.group; });
  const int row = at - s.first * a.group;  // of the sequence
  const Unit u = unit_of(a, s, row / R, R);
  if (row - u.row0 >= u.rows || u.chunks <= 1) return;
  const int64_t first = part_at(a, h, 0, at), step = (int64_t)a.tokens * a.group;
  join_row<D, 1>(a, first, first + step, step, min(u.chunks, a.splits), at / a.group, h * a.group + at % a.group);
}

template <int D, bool E4M3, int NR>
static hipError_t launch_stream(const AttnArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)(a.slots / (kStreamWaves / a.heads_wg)) * (unsigned)(a.kv_heads / a.heads_wg);
  if (a.sees)
    hipLaunchKernelGGL((attn_stream_kernel<D, E4M3, NR, true>), dim3(grid), dim3(kStreamWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL((attn_stream_kernel<D, E4M3, NR, false>), dim3(grid), dim3(kStreamWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int D, bool E4M3>
static hipError_t launch_stream_d(const AttnArgs& a, int rows, hipStream_t s) {
  return rows == 16 ? launch_stream<D, E4M3, 1>(a, s) : launch_stream<D, E4M3, 2>(a, s);
}

hipError_t launch_attn_stream(const AttnArgs& a, int head_dim, bool e4m3, int rows, hipStream_t s) {
  if (head_dim == 64) return e4m3 ? launch_stream_d<64, true>(a, rows, s) : launch_stream_d<64, false>(a, rows, s);
  return e4m3 ? launch_stream_d<128, true>(a, rows, s) : launch_stream_d<128, false>(a, rows, s);
}

int attn_stream_slots(int head_dim, bool e4m3, int rows, int kv_heads, int heads_wg) {
  const int per_cu = stream_workgroups(head_dim, e4m3, rows / 16), head_groups = kv_heads / heads_wg;
  const int workgroups = 256 * per_cu / head_groups / 8 * 8;  // of one group of heads; a multiple of the XCDs
  return (workgroups < 8 ? 8 : workgroups) * (kStreamWaves / heads_wg);
}

template <int D>
static void launch_stream_join(const AttnArgs& a, int rows, int most_rows, hipStream_t s) {
  const unsigned all = (unsigned)(most_rows * a.kv_heads);
  // Sequences in more than 16 slots on average: a workgroup a row, else a wave.  A
  // wave's and a workgroup's join, 32 / 8 heads, bf16, us: 1 x 16,000 keys 31.9 and
  // 21.2, 4 x 4,000 22.9 and 20.1, 7 x 4,000 28.4 and 26.9, 8 x 4,000 (16 slots) 29.8
  // and 28.6, 16 x 4,000 50.6 and 50.1, 24 x 2,000 39.5 and 40.0, 64 x 1,000 49.2 and
  // 50.8; 16 x 5 tokens at 515 .. 4,099 38.5 and 40.4; 200 x 300, 64 / 8 heads, 64.8
  // and 82.7.
  if (a.slots > 16 * a.batch)
    hipLaunchKernelGGL((attn_stream_join_kernel<D, kJoinWaves>), dim3(all, (unsigned)a.batch), dim3(kJoinWaves * 64), 0, s,
                       a, rows);
  else
    hipLaunchKernelGGL((attn_stream_join_kernel<D, 1>), dim3((all + kJoinWaves - 1) / kJoinWaves, (unsigned)a.batch),
                       dim3(kJoinWaves * 64), 0, s, a, rows);
}

hipError_t launch_attn_stream_join(const AttnArgs& a, int head_dim, int rows, int most_rows, hipStream_t s) {
  if (head_dim == 64)
    launch_stream_join<64>(a, rows, most_rows, s);
  else
    launch_stream_join<128>(a, rows, most_rows, s);
  return hipGetLastError();
}

hipError_t launch_attn_join(const AttnArgs& a, int head_dim, int rows, hipStream_t s) {
  const unsigned grid = (unsigned)((a.tokens * a.group + kJoinWaves - 1) / kJoinWaves) * (unsigned)a.kv_heads;
  if (head_dim == 64)
    hipLaunchKernelGGL((attn_join_kernel<64>), dim3(grid), dim3(kJoinWaves * 64), 0, s, a, rows);
  else
    hipLaunchKernelGGL((attn_join_kernel<128>), dim3(grid), dim3(kJoinWaves * 64), 0, s, a, rows);
  return hipGetLastError();
}

}  // namespace qlk
