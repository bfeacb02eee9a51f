// What the attention kernels share: the rows of a unit, the range of keys
// they see, page look-up, and the conversion of cache codes to matrix-core
// operands.
//
// One unit is a sequence b, a KV head h and a block of R rows; row r of the
// sequence's n * group rows is new token r / group, query head h * group + r
// % group, so the rows of a block share the keys and values they read.  The
// new token t of n stands at position p = len - n + t and sees the keys
// j <= p (causal) with j > p - window (window > 0).
#pragma once

#include "attention_args.hpp"
#include "device_common.hpp"
#include "tree_cut.hpp"

namespace qlk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Four binary32 values at a 4-byte aligned address: rows of an odd vocabulary,
// or a caller's table, start anywhere.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr float kNegInf = -__builtin_huge_valf();

// How far (base 2) a new maximum exceeds the one that a row's weights refer to
// before that moves: weights stay below 2^8, exact in relative terms.
constexpr float kRescaleAt = 8.0f;

__device__ __forceinline__ f32x4 mma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two binary32 values as a pair of bf16, round to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  bf16x2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

// Two E4M3 codes (the low or high half of w) as a pair of bf16: exact.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_to_bf16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// Pins a value's computation to this place: without it the compiler turns a
// rarely taken branch into arithmetic that is always done, or sinks work out
// of the block whose products are to cover it.
template <class T>
__device__ __forceinline__ void pin(T& x) {
  asm volatile("" : "+v"(x));
}

// Maximum over a lane and the lane 32 away.
__device__ __forceinline__ float half_max(float v) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
}

// Maximum and sum over lanes l, l^16, l^32, l^48: the four lanes that hold
// one row's keys.
__device__ __forceinline__ float row4_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float row4_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Sum over lanes 0 .. l, by lane shifts inside 16 lanes, then the rows' last
// lanes to the rows behind them.
__device__ __forceinline__ int inclusive_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr 1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);   // row_shr 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);   // row_shr 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);   // row_shr 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast 31 into rows 2 and 3
  return v;
}

// A row's lse from its maximum (base 2, -inf: no score above -inf) and sum.  Where
// all scores are NaN the maximum has not moved either, but the sum is NaN.
__device__ __forceinline__ float lse_of(float m, float sum) {
  return m == kNegInf && sum == sum ? kNegInf : (m + log2f(sum)) * 0.6931471805599453f;
}

// A table or length entry at a wave-uniform address.
__device__ __forceinline__ int uniform_i32(const int32_t* p) { return __builtin_amdgcn_readfirstlane(*p); }

__device__ __forceinline__ int lane_i32(int v, int i) { return __builtin_amdgcn_readlane(v, i); }

// Sequence b of the batch: its new tokens [first, end) of q and its cached
// length; every field is wave-uniform.  b < 0: none.
struct Sequence {
  int b, first, end, len;
};

// The last sequence with start(b, its first token) <= n, for starts that do
// not fall from one sequence to the next: 64 probes at once, so one round of
// loads for up to 64 sequences, two up to 4,096.  Whatever cu_q holds, the
// answer is a sequence of the batch or none.
template <class F>
__device__ __forceinline__ Sequence sequence_at(const AttnArgs& a, int n, F start) {
  const int lane = threadIdx.x & 63;
  for (int lo = 0, width = a.batch;;) {
    const int step = (width + 63) >> 6, b = min(lo + lane * step, a.batch - 1);
    const int q0 = min(max(a.cu_q[b], 0), a.tokens), q1 = min(max(a.cu_q[b + 1], q0), a.tokens);
    const int len = min(max(a.seq_lens[b], 0), a.max_kv);
    const unsigned long long before = __ballot(lane * step < width && start(b, q0) <= n);
    if (before == 0) return Sequence{-1, 0, 0, 0};
    const int i = 63 - __clzll((long long)before);
    if (step == 1) return Sequence{lo + i, lane_i32(q0, i), lane_i32(q1, i), lane_i32(len, i)};
    lo += i * step;
    width = min(step, width - i * step);
  }
}

// The rows and keys of one unit; every field is wave-uniform.
struct Unit {
  int b;         // its sequence
  int first;     // the sequence's first token in q
  int rows;      // rows of this block (0: nothing to do)
  int row0;      // first row of the block
  int pos0;      // position of the sequence's first new token
  int len;       // cached length (keys beyond it are never read)
  int lo, hi;    // keys any row of the block sees: [lo, hi)
  int chunks;    // chunks of keys, from lo rounded down to 64
};

// Block `block` of sequence s.  Sequences that are left to the stream kernel,
// and blocks beyond the plan's, have no rows.
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, const Sequence& s, int block, int R) {
  Unit u;
  const int n = s.end - s.first, all = n * a.group;
  u.b = s.b;
  u.len = s.len;
  u.first = s.first;
  u.row0 = block * R;
  u.rows = s.b < 0 || all < a.min_rows || block < 0 || block >= a.row_blocks ? 0 : min(max(all - u.row0, 0), R);
  u.pos0 = u.len - n;
  u.hi = u.len;
  u.lo = 0;
  if (u.rows > 0) {
    const int t0 = u.row0 / a.group, t1 = (u.row0 + u.rows - 1) / a.group;
    if (a.causal) u.hi = min(u.len, max(0, u.pos0 + t1 + 1));
    if (a.window) u.lo = min(u.hi, max(0, u.pos0 + t0 - a.window + 1));
  } else {
    u.hi = 0;
  }
  const int lo64 = u.lo & ~63;
  u.chunks = u.hi > u.lo ? (u.hi - lo64 + a.chunk - 1) / a.chunk : 0;
  return u;
}

// Unit n of the batch, in one of two numberings, a sequence's last block (the
// longest) first.  Sequence by sequence, row_blocks numbers each.  Or by the
// rows before them (a.by_rows): sequence b's numbers follow from floor(rows
// before it / R) + b, which leaves room for every sequence's ceil(rows / R)
// blocks in rows / R + batch numbers, whatever the lengths, and a number's
// sequence is found by search.
__device__ __forceinline__ Unit unit_at(const AttnArgs& a, int n, int R) {
  if (!a.by_rows) {
    const int b = n / a.row_blocks;
    const int q0 = min(max(uniform_i32(a.cu_q + b), 0), a.tokens), q1 = min(max(uniform_i32(a.cu_q + b + 1), q0), a.tokens);
    const Sequence s = {b, q0, q1, min(max(uniform_i32(a.seq_lens + b), 0), a.max_kv)};
    return unit_of(a, s, a.row_blocks - 1 - n % a.row_blocks, R);
  }
  auto start = [&](int b, int q0) { return q0 * a.group / R + b; };
  const Sequence s = sequence_at(a, n, start);
  const int blocks = min(((s.end - s.first) * a.group + R - 1) / R, a.row_blocks);
  return unit_of(a, s, blocks - 1 - (n - start(s.b, s.first)), R);
}

__device__ __forceinline__ int tree_blocks(const AttnArgs& a, const Sequence& s, int R) {
  return min(((s.end - s.first) * a.group + R - 1) / R, a.row_blocks);
}

// Sequence b as this lane's own; none beyond the batch.
__device__ __forceinline__ Sequence tree_sequence(const AttnArgs& a, int b) {
  if (b >= a.batch) return Sequence{-1, 0, 0, 0};
  const int q0 = min(max(a.cu_q[b], 0), a.tokens), q1 = min(max(a.cu_q[b + 1], q0), a.tokens);
  return Sequence{b, q0, q1, min(max(a.seq_lens[b], 0), a.max_kv)};
}

// The cut of a batch, a sequence a lane.
__device__ __forceinline__ TreeCut tree_cut(const AttnArgs& a, const Sequence& mine, int R, int slots) {
  const int lane = threadIdx.x & 63;
  auto each = [&](auto f) {
#pragma unroll 1
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
      const Sequence s = b0 ? tree_sequence(a, b0 + lane) : mine;
      f(tree_blocks(a, s, R), s.len);
    }
  };
  return tree_cut_of(each, [](int x) { return lane_i32(inclusive_sum(x), 63); }, a.kv_heads, a.max_kv, slots);
}

// The shares of this lane's sequence, and those before them (of one KV head).  Where
// they start one after the other: by falling length of a share, so that the last ones to start
// are the short ones (32 sequences of 1,021 .. 8,190 keys, 33 .. 64 nodes of 40 / 8
// heads, E4M3, 1,024 shares: 175 us, 184 in the sequences' order, three runs in turn).
struct TreeShares {
  int each, all, before;   // of a unit, of all its units
};
__device__ __forceinline__ TreeShares tree_shares_of(const AttnArgs& a, const TreeCut& cut, const Sequence& s, int R, int before) {
  TreeShares t;
  t.each = tree_shares(s.len, cut);
  t.all = tree_blocks(a, s, R) * t.each;
  t.before = before + inclusive_sum(t.all) - t.all;
  if (cut.rounds && a.batch <= 64) {
    const int lane = threadIdx.x & 63, size = s.len / t.each;
    t.before = 0;
#pragma unroll 1
    for (int j = 0; j < a.batch; ++j) {
      const int other = lane_i32(size, j), n = lane_i32(t.all, j);
      t.before += other > size || (other == size && j < lane) ? n : 0;
    }
  }
  return t;
}

// Share n of one KV head: its unit, the share of the unit's keys and their number.
__device__ __forceinline__ Unit tree_unit(const AttnArgs& a, const TreeCut& cut, const Sequence& mine, int n, int R, int* share,
                                         int* shares) {
  const int lane = threadIdx.x & 63;
  int before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const Sequence s = b0 ? tree_sequence(a, b0 + lane) : mine;
    const TreeShares t = tree_shares_of(a, cut, s, R, before);
    const uint64_t here = __ballot(n >= t.before && n - t.before < t.all);
    if (here) {
      const int i = __ffsll((unsigned long long)here) - 1;
      const Sequence own = {b0 + i, lane_i32(s.first, i), lane_i32(s.end, i), lane_i32(s.len, i)};
      *shares = lane_i32(t.each, i);
      const int at = n - lane_i32(t.before, i);
      *share = at % *shares;
      return unit_of(a, own, at / *shares, R);
    }
    before = lane_i32(t.before + t.all, 63);
  }
  Unit none{};
  return none;
}

// Where the partial results of one row over chunk `split` lie: rows of all
// tokens, for each chunk and KV head.
__device__ __forceinline__ int64_t part_at(const AttnArgs& a, int h, int split, int row) {
  return ((int64_t)h * a.splits + split) * ((int64_t)a.tokens * a.group) + row;
}

// Keys [lo, hi) that row r of the block sees.
__device__ __forceinline__ void row_range(const AttnArgs& a, const Unit& u, int r, int* lo, int* hi) {
  const int p = u.pos0 + (u.row0 + r) / a.group;
  *hi = a.causal ? min(u.len, max(0, p + 1)) : u.len;
  *lo = a.window ? max(0, p - a.window + 1) : 0;
}

// Trees of drafted tokens (TREE; a.causal and a.window are 0 then): a row sees
// the keys before the sequence's new tokens and those of these that its token's
// bits name.  Which of the 32 keys from the `node`-th new token on (below 0:
// keys before them) token `tok` sees, one a bit.
__device__ __forceinline__ uint32_t tree_bits(const AttnArgs& a, int tok, int node) {
  const uint64_t* bits = a.sees + (int64_t)tok * a.words;
  if (node < 0) return node <= -32 ? 0xffffffffu : (uint32_t)(bits[0] << -node) | ((1u << -node) - 1);
  const int w = node >> 6, s = node & 63;
  uint64_t x = w < a.words ? bits[w] >> s : 0;
  if (s > 32 && w + 1 < a.words) x |= bits[w + 1] << (64 - s);
  return (uint32_t)x;
}

// Where 64 16-key groups of a sequence lie: lane i holds the byte offsets of
// group `group` of its own in K and V.  One gather of page numbers and one
// round of address arithmetic serve 64 groups; a wave then picks a group by
// its lane number, without a dependent scalar load per tile.  Columns past
// the sequence's last page are never read, and a page number out of range is
// taken into range (a wrong answer for a broken table, never a read outside
// the cache).
struct Groups {
  uint32_t k_lo, k_hi, v_lo, v_hi;
};

__device__ __forceinline__ Groups groups_at(const AttnArgs& a, const int32_t* row, int h, int group, int last) {
  const int sub = min(group, last);
  const int col = page_of(sub, a.page_magic);
  const int64_t at = sub * 16 - col * a.page_size;
  const int64_t page = min((uint32_t)row[col], (uint32_t)(a.num_pages - 1));
  const uint64_t k = (uint64_t)(page * a.kc.page + at * a.kc.token + h * a.kc.head);
  const uint64_t v = (uint64_t)(page * a.vc.page + at * a.vc.token + h * a.vc.head);
  return Groups{(uint32_t)k, (uint32_t)(k >> 32), (uint32_t)v, (uint32_t)(v >> 32)};
}

__device__ __forceinline__ uint64_t pick(uint32_t lo, uint32_t hi, int i) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)lo, i) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, i) << 32;
}

// Infinities and NaNs in values that some rows see and others do not: in a
// product a hidden value's weight is 0, and 0 * NaN would reach the rows that do
// not see it.  So where a tile is hidden in part they are dropped from it, and
// at the end the outputs that they reach are found by reading the values again.

// Ones where a word's values (two bf16, or four E4M3 codes) are finite: the sum
// has a field's top bit exactly where its exponent (its code) is all ones.
template <bool E4M3>
__device__ __forceinline__ uint32_t finite_mask(uint32_t w) {
  const uint32_t top = E4M3 ? ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u : ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
  return ~((top << 1) - (top >> (E4M3 ? 7 : 15)));
}

// `seen(key, bad)` is called for each key of [key, key + n) with non-finite
// values, bad[i] holding value d = 2 l + i (D = 64: l) in bit l.
template <int D, bool E4M3, class F>
__device__ __forceinline__ void for_nonfinite(const AttnArgs& a, const int32_t* table, int h, int key, int n, F seen) {
  constexpr int W = D / 64;
  const int lane = threadIdx.x & 63;
  for (int k = key; k < key + n; ++k) {
    const int col = page_of(k >> 4, a.page_magic);
    const int64_t page = min((uint32_t)uniform_i32(table + col), (uint32_t)(a.num_pages - 1));
    const uint8_t* p = a.vc.p + page * a.vc.page + (int64_t)(k - col * a.page_size) * a.vc.token + h * a.vc.head;
    uint64_t bad[W];
    bool any = false;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int d = lane * W + i;
      bad[i] = __ballot(E4M3 ? (p[d] & 0x7f) == 0x7f : (reinterpret_cast<const uint16_t*>(p)[d] & 0x7f80) == 0x7f80);
      any |= bad[i] != 0;
    }
    if (any) seen(k, bad);
  }
}

template <int D>
__device__ __forceinline__ bool bad_at(const uint64_t (&bad)[D / 64], int d) {
  return D == 128 ? (bad[d & (D / 64 - 1)] >> (d >> 1)) & 1 : (bad[0] >> d) & 1;
}

}  // namespace qlk
