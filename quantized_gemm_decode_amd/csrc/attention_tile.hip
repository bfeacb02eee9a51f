// Attention over the paged cache for many rows a sequence: chunks of new
// tokens.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale q_r.k_j - m_r),
// in one pass over the keys with the running maximum m_r and sum of each row.
//
// 4 D flops a row and key: with hundreds of rows bound by the matrix cores.
// Four waves share tiles of 64 keys in LDS; each holds 32 rows of Q and of the
// output in registers, two or three workgroups a compute unit.  Products are 32x32x16
// bf16 (lane l = 32 g + r):
//   S^T = K Q^T: a lane ends with 16 of 32 keys of one row, so maximum and
//     sum of a row are in-lane, with one exchange between the lane halves;
//   O^T = V^T P^T: S's registers 8i .. 8i+7 hold the 8 keys of a lane's
//     operand as they stand, P never moves between lanes; V^T comes out of
//     LDS by transposing reads (ds_read_b64_tr_b16: 4 keys of one value).
// The three parts of the work on 32 keys -- scores, weights, sums -- run one
// 32-key step apart, so that every product has exponentials of another step
// and the next operands' LDS reads behind it (inner_step).
//
// LDS holds K and V rows in 16-byte pieces with their place in the row
// exchanged by row, so that the 16 rows (K) or 4 rows (V) that one read
// touches lie in different banks (no bank conflicts counted).
// The maximum a row's weights refer to is only moved when a row's new maximum
// exceeds it by more than 8 (in base 2): weights then stay below 2^8, exact in
// relative terms, and the outputs need no rescaling for most tiles.
//
// P is rounded to bf16 for the product, 2^-8 of a term at most: against 64 bits
// outputs are off by 2.3e-3 of their root mean square, 1.7e-3 of it their own
// rounding.  Sums take it in binary32.  A second product over what the rounding
// left out (as the decode kernel has behind its memory) would cost 26 % of a
// chunk of 2,048 at 10,240 and 13 % with 64-wide heads.
//
// Values that some rows do not see: 0 * NaN would reach them.  A tile that is
// hidden in part loses its infinities and NaNs on the way into LDS; where there
// were any (none, as a rule), the outputs that they reach are found by reading
// the values again.
//
// Measured on MI355X, 2048 new tokens at the end of 10,240 cached ones, 32 / 8
// heads of 128: 304-375 us by card, 820-1020 TFLOP/s of the visible pairs' flops
// (a traced run's median 335),
// against 1140-1380 that a large library product reaches.  With the exponentials, the
// LDS reads or the staging left out it is 1, 3 or 13 % faster, with all of
// them 33 %: no single part bounds it, the products' own rate does at last.
// (Nor the tests of the reference maximum: made behind the products instead of
// ahead of the weights, 344 us.)  64-wide heads have half the products for the
// same weights: 512 new tokens of each of 4 sequences of 2,000, bf16: 49 us, 597
// TFLOP/s.  No unit bounds them alone (12 sequences with 4,327 new tokens, window
// 2048, E4M3: vector unit busy 56 % of the time, matrix cores 27 %).
//
// Trees of drafted tokens (TREE) are the same but for the mask of the new tokens and
// the cut of the keys (tree_cut); their partial results lie as the registers do
// and have a join of their own.  1 sequence of 1,031 keys, 26 nodes, 32 / 8 heads of
// 128: 15.5 us, latency (10) and the join (6); 16 of 515 .. 4,099, 32 nodes: 55 us, 46 of
// them reading at 3.3 TB/s behind a start of about 8 us, 9 the join of 35 MB of
// partial results; 32 of 1,021 .. 8,190, 33 .. 64 nodes of 40 / 8 heads, E4M3: 174 .. 178 us
// (160 .. 166 and the join's 15), 640 .. 650 TFLOP/s of the visible pairs' flops.
#include "attention_common.hpp"

#include <type_traits>

namespace qlk {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kTileKeys = 64;
constexpr int kTileWaves = 4;
constexpr int kTileRows = kTileWaves * 32;

__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Place of 16-byte piece c of K row `row` and of 64-byte block c of V row
// `row` (rows of D bf16).
template <int D>
__device__ __forceinline__ int k_piece(int row, int c) {
  return c ^ ((D == 128 ? row : row >> 1) & (D / 8 - 1));
}
template <int D>
__device__ __forceinline__ int v_block(int row, int c) {
  return c ^ ((D == 128 ? row : row >> 1) & (D / 32 - 1));
}

// 4 keys of one value: lane 4j + c of 16 names 4 values of key j.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// What a thread carries of a tile from memory to LDS: wave w brings the
// tile's keys 16w .. 16w + 15, whole rows in contiguous pieces.
template <int D, bool E4M3>
struct Staged {
  static constexpr int CH = D * (E4M3 ? 1 : 2) / 16;  // 16-byte pieces of a row
  static constexpr int RP = 64 / CH;                  // rows a wave's load covers
  static constexpr int PASSES = 16 / RP;
  u32x4 x[PASSES];
};

template <int D, bool E4M3>
__device__ __forceinline__ void load_k(const AttnArgs& a, const Groups& at, int i, uint32_t lane, Staged<D, E4M3>* t) {
  const uint8_t* k = a.kc.p + pick(at.k_lo, at.k_hi, i);
#pragma unroll
  for (int j = 0; j < Staged<D, E4M3>::PASSES; ++j)
    t->x[j] = *reinterpret_cast<const u32x4*>(k + j * (Staged<D, E4M3>::RP * (int)a.kc.token) + lane);
}

template <int D, bool E4M3>
__device__ __forceinline__ void load_v(const AttnArgs& a, const Groups& at, int i, uint32_t lane, Staged<D, E4M3>* t) {
  const uint8_t* v = a.vc.p + pick(at.v_lo, at.v_hi, i);
#pragma unroll
  for (int j = 0; j < Staged<D, E4M3>::PASSES; ++j)
    t->x[j] = *reinterpret_cast<const u32x4*>(v + j * (Staged<D, E4M3>::RP * (int)a.vc.token) + lane);
}

// 16 E4M3 codes as two pieces of bf16.
__device__ __forceinline__ void widen(const u32x4& c, u32x4* lo, u32x4* hi) {
  *lo = u32x4{e4m3_to_bf16<false>(c.x), e4m3_to_bf16<true>(c.x), e4m3_to_bf16<false>(c.y), e4m3_to_bf16<true>(c.y)};
  *hi = u32x4{e4m3_to_bf16<false>(c.z), e4m3_to_bf16<true>(c.z), e4m3_to_bf16<false>(c.w), e4m3_to_bf16<true>(c.w)};
}

// The tile's rows this thread carries, j-th pass.
template <int D, bool E4M3>
__device__ __forceinline__ int staged_row(int j) {
  using S = Staged<D, E4M3>;
  return (threadIdx.x >> 6) * 16 + j * S::RP + (threadIdx.x & 63) / S::CH;
}

template <int D, bool E4M3>
__device__ __forceinline__ void store_k(const Staged<D, E4M3>& t, uint8_t* kl) {
  using S = Staged<D, E4M3>;
  const int piece = threadIdx.x % S::CH;
#pragma unroll
  for (int j = 0; j < S::PASSES; ++j) {
    const int row = staged_row<D, E4M3>(j);
    if constexpr (E4M3) {
      u32x4 x[2];
      widen(t.x[j], &x[0], &x[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<u32x4*>(kl + row * D * 2 + k_piece<D>(row, 2 * piece + i) * 16) = x[i];
    } else {
      *reinterpret_cast<u32x4*>(kl + row * D * 2 + k_piece<D>(row, piece) * 16) = t.x[j];
    }
  }
}

// V rows of keys beyond the sequence are stored as zero: the cache there may
// hold anything, and 0 * NaN would reach every row.  From a tile that is hidden
// from some rows (`part`) infinities and NaNs are dropped; `mark` is then set.
template <int D, bool E4M3>
__device__ __forceinline__ void store_v(Staged<D, E4M3>& t, int key, int len, uint8_t* vl, bool part, int* mark) {
  using S = Staged<D, E4M3>;
  const int piece = threadIdx.x % S::CH;
  if (part && key + kTileKeys > len) {
    pin(key);
#pragma unroll
    for (int j = 0; j < S::PASSES; ++j)
      if (key + staged_row<D, E4M3>(j) >= len) t.x[j] = u32x4{0u, 0u, 0u, 0u};
  }
  if (part) {
    bool dropped = false;
#pragma unroll
    for (int j = 0; j < S::PASSES; ++j) {
      pin(t.x[j]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t keep = finite_mask<E4M3>(t.x[j][w]);
        dropped |= keep != 0xffffffffu;
        t.x[j][w] &= keep;
      }
    }
    if (__any(dropped)) *mark = 1;
  }
#pragma unroll
  for (int j = 0; j < S::PASSES; ++j) {
    const int row = staged_row<D, E4M3>(j);
    constexpr int N = E4M3 ? 2 : 1;
    u32x4 x[N];
    if constexpr (E4M3)
      widen(t.x[j], &x[0], &x[1]);
    else
      x[0] = t.x[j];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = N * piece + i;
      *reinterpret_cast<u32x4*>(vl + row * D * 2 + v_block<D>(row, c / 4) * 64 + (c % 4) * 16) = x[i];
    }
  }
}

// One K operand (values 16 i .. 16 i + 15 of 32 keys of half t) and one V
// operand (16 keys c / DT of half t, values 32 (c % DT) ..).
template <int D>
__device__ __forceinline__ u32x4 k_operand(const uint8_t* kl, int t, int i) {
  const int row = t * 32 + (threadIdx.x & 31), g = (threadIdx.x >> 5) & 1;
  return *reinterpret_cast<const u32x4*>(kl + row * D * 2 + k_piece<D>(row, 2 * i + g) * 16);
}
template <int D>
__device__ __forceinline__ u32x4 v_operand(const uint8_t* vl, int t, int c) {
  const int lane = threadIdx.x & 63, g = lane >> 5, j = (lane & 15) >> 2;
  const uint8_t* vp = vl + (t * 32 + c / (D / 32) * 16 + 4 * g + j) * D * 2 +
                      v_block<D>(4 * g + j, c % (D / 32)) * 64 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
  const u32x2 v0 = read_transposed(vp), v1 = read_transposed(vp + 8 * D * 2);
  return u32x4{v0.x, v0.y, v1.x, v1.y};
}

// S^T of 32 keys (half t of a K tile) and the wave's 32 rows.
template <int D>
__device__ __forceinline__ f32x16 qk(const uint8_t* kl, int t, const u32x4 (&q)[D / 16]) {
  f32x16 s;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) s = mma32(k_operand<D>(kl, t, i), q[i], s);
  return s;
}

// O^T += V^T P^T over the 32 keys of half t of a V tile.
template <int D>
__device__ __forceinline__ void pv(const uint8_t* vl, int t, const u32x4 (&p)[2], f32x16 (&o)[D / 32]) {
#pragma unroll
  for (int c = 0; c < D / 16; ++c) o[c % (D / 32)] = mma32(v_operand<D>(vl, t, c), p[c / (D / 32)], o[c % (D / 32)]);
}

// One row's running softmax (row = lane & 31; the lane halves hold different
// keys): the maximum its weights refer to (scaled, base 2; -inf: no key yet)
// and this lane's share of the sum.
struct Soft {
  float m, base, l, scale;
};

// Weights of 32 keys, rounded to bf16 in the order of O's operand.
__device__ __forceinline__ void weights(const f32x16& s, Soft* w, u32x4 (&p)[2]) {
  float e[16], sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    e[i] = __builtin_amdgcn_exp2f(__fmaf_rn(s[i], w->scale, -w->base));
    sum[i % 4] += e[i];
  }
  w->l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) p[i][k] = bf16_pair(e[8 * i + 2 * k], e[8 * i + 2 * k + 1]);
}

// The inner step: next = S^T of half kt of the K tile kl, O^T += V^T P^T over
// half vt of the V tile vl, and p_out = the weights of s.  The three do not
// depend on each other, so the order below lays a share of the exponentials
// and the next operands' LDS reads behind every product; the barriers keep
// the compiler from gathering the products again (it then runs the matrix
// cores and the vector unit one after the other).
template <int D>
__device__ __forceinline__ void inner_step(const uint8_t* kl, int kt, const uint8_t* vl, int vt, const u32x4 (&q)[D / 16],
                                           const f32x16& s, Soft* w, const u32x4 (&p)[2], f32x16 (&o)[D / 32],
                                           f32x16* next, u32x4 (&p_out)[2]) {
  constexpr int N = D / 16, E = 16 / (2 * N);  // products of each kind; exponentials behind one
  // ahead of the compute unit's other wave while that loads, masks or stores
  // (128-wide heads: 363 -> 351 us; with 64-wide ones the exponentials bound it
  // and there is nothing to be ahead for)
  if (D == 128) __builtin_amdgcn_s_setprio(1);
  u32x4 kf[2], vf[2];
  kf[0] = k_operand<D>(kl, kt, 0);
  vf[0] = v_operand<D>(vl, vt, 0);
  f32x16 c;
#pragma unroll
  for (int i = 0; i < 16; ++i) c[i] = 0.0f;
  float e[16], sum[2] = {0.0f, 0.0f};
  auto share = [&](int first) {
#pragma unroll
    for (int i = first; i < first + E; ++i) {
      e[i] = __builtin_amdgcn_exp2f(__fmaf_rn(s[i], w->scale, -w->base));
      sum[i & 1] += e[i];
      if (i & 1) {
        uint32_t pair = bf16_pair(e[i - 1], e[i]);
        pin(pair);
        p_out[i / 8][i % 8 / 2] = pair;
      }
    }
  };
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + 1 < N) {
      kf[(i + 1) & 1] = k_operand<D>(kl, kt, i + 1);
      vf[(i + 1) & 1] = v_operand<D>(vl, vt, i + 1);
    }
    c = mma32(kf[i & 1], q[i], c);
    share(2 * i * E);
    __builtin_amdgcn_sched_barrier(0);
    o[i % (D / 32)] = mma32(vf[i & 1], p[i / (D / 32)], o[i % (D / 32)]);
    share((2 * i + 1) * E);
    __builtin_amdgcn_sched_barrier(0);
  }
  w->l += sum[0] + sum[1];
  pin(w->l);
  *next = c;
  if (D == 128) __builtin_amdgcn_s_setprio(0);
}

// Workgroups a compute unit gets: what the registers allow.  (64-wide heads, 12
// sequences with 4,327 new tokens, window 2048, E4M3: 101 us with three, 109 us
// with two; 8 chunks of 512 at 2,000, bf16: 96 and 102 us.)
constexpr int tile_workgroups(int D) { return D == 64 ? 3 : 2; }

// How the keys of trees were cut, for the join.
__device__ __forceinline__ void tell_cut(const AttnArgs& a, const TreeCut& cut) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const Sequence s = tree_sequence(a, b0 + lane);
    const TreeShares t = tree_shares_of(a, cut, s, kTileRows, before);
    if (threadIdx.x < 64 && s.b >= 0) {
      a.cut[2 * s.b] = t.before;
      a.cut[2 * s.b + 1] = t.each;
    }
    before = lane_i32(t.before + t.all, 63);
  }
}

template <int D, bool E4M3, bool TREE>
__global__ void __launch_bounds__(kTileWaves * 64, tile_workgroups(D)) attn_tile_kernel(AttnArgs a) {
  constexpr int R = kTileRows, DT = D / 32, KS = D / 16;
  constexpr int kBytes = kTileKeys * D * 2;  // one tensor's tile
  __shared__ __align__(16) uint8_t k_lds[2][kBytes], v_lds[2][kBytes];
  __shared__ int dropped;  // values were, from a tile hidden in part
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  int id = blockIdx.x;
  const int h = id % a.kv_heads;
  id /= a.kv_heads;
  int split, chunk, chunks;
  Unit u;
  if constexpr (TREE) {
    split = 0;
    chunks = 1;
    if (a.splits > 1) {
      const Sequence mine = tree_sequence(a, lane);
      const TreeCut cut = tree_cut(a, mine, R, 256 * tile_workgroups(D));
      if (blockIdx.x == 0) tell_cut(a, cut);
      u = tree_unit(a, cut, mine, id, R, &split, &chunks);
    } else {
      u = unit_at(a, id, R);
    }
    if (u.rows == 0) return;
    chunk = ((u.len + chunks - 1) / chunks + 63) / 64 * 64;   // the shares as equal as whole tiles are
  } else {
    split = id % a.splits;
    u = unit_at(a, id / a.splits, R);
    if (u.rows == 0) return;
    if (u.chunks == 0 ? split != 0 : split >= u.chunks) return;
    chunk = a.chunk;
    chunks = u.chunks;
  }
  const int begin = (u.lo & ~63) + split * chunk;
  const int end = min(u.hi, begin + chunk);
  const int tiles = end > begin ? (end - begin + kTileKeys - 1) / kTileKeys : 0;

  // this lane's row, and what follows from it, is worked out again where it is
  // used: kept through the loop its registers cost 64-wide heads a workgroup
  auto own_row = [&]() {
    int x = wave * 32 + r;
    pin(x);
    return x;
  };
  int row = own_row(), place = u.row0 + row;
  u32x4 q[KS];
  {
    const int tok = u.first + place / a.group, head = h * a.group + place % a.group;
    const uint8_t* p = a.q.p + (int64_t)tok * a.q.token + (int64_t)head * a.q.head + g * 16;
#pragma unroll
    for (int s = 0; s < KS; ++s)
      q[s] = row < u.rows ? *reinterpret_cast<const u32x4*>(p + s * 32) : u32x4{0u, 0u, 0u, 0u};
  }
  Soft w = {kNegInf, 0.0f, 0.0f, a.scale_log2 * (E4M3 && a.kc.scale ? a.kc.scale[h] : 1.0f)};
  f32x16 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] = 0.0f;

  if (tiles > 0) {
    // keys that every row of the block sees
    int full_lo, full_hi, x;
    row_range(a, u, u.rows - 1, &full_lo, &x);
    row_range(a, u, 0, &x, &full_hi);
    full_hi = min(TREE ? max(0, u.pos0) : full_hi, end);
    const int32_t* table = a.table + u.b * a.table_row;
    const int last_sub = (u.len - 1) >> 4;
    using S = Staged<D, E4M3>;
    const uint32_t k_lane = (uint32_t)(lane / S::CH * (int)a.kc.token + lane % S::CH * 16);
    const uint32_t v_lane = (uint32_t)(lane / S::CH * (int)a.vc.token + lane % S::CH * 16);
    // places of 64 tiles' groups at a time; K runs a tile ahead of V
    Groups at = groups_at(a, table, h, (begin >> 4) + wave + 4 * lane, last_sub);

    auto own_range = [&](int* lo, int* hi) {
      const int x = own_row();
      row_range(a, u, x, lo, hi);
      *hi = x < u.rows ? min(*hi, end) : 0;
    };
    // trees: which of the keys [key, key + 32) the lane's row sees
    auto own_bits = [&](int key) {
      return tree_bits(a, u.first + (u.row0 + min(own_row(), u.rows - 1)) / a.group, key - u.pos0);
    };
    // masks the scores of keys [key, key + 32) where some row does not see all of them
    auto mask = [&](f32x16& s, int key) {
      if (key < full_lo || key + 32 > full_hi) {
        int first = key + 4 * g, lo, hi;
        pin(first);
        own_range(&lo, &hi);
        uint32_t bits = 0xffffffffu;
        if (TREE) bits = own_bits(key) >> 4 * g;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = first + 8 * (i / 4) + i % 4;
          s[i] = j >= lo && j < hi && (!TREE || bits >> (8 * (i / 4) + i % 4) & 1) ? s[i] : kNegInf;
        }
      }
    };
    // moves the reference maximum where 32 new scores exceed it by far; what
    // is not in O yet (p over half t of vl) is added first
    auto refer = [&](const f32x16& s, const uint8_t* vl, int t, u32x4 (&p)[2]) {
      float top = s[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
      top *= w.scale;
      if (__any(top > w.m + kRescaleAt)) {
        top = half_max(top);
        if (vl) pv<D>(vl, t, p, o);
        p[0] = p[1] = u32x4{0u, 0u, 0u, 0u};
        const float now = fmaxf(w.m, top);
        const float keep = __builtin_amdgcn_exp2f(w.m - (now == kNegInf ? 0.0f : now));
        w.m = now;
        w.base = now == kNegInf ? 0.0f : now;
        w.l *= keep;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] *= keep;
      }
    };

    // whether tile T is hidden from some row
    auto part = [&](int T) {
      const int key = begin + T * kTileKeys;
      return key < full_lo || key + kTileKeys > full_hi;
    };
    S staged;
    if (threadIdx.x == 0) dropped = 0;
    lds_barrier();
    load_k<D, E4M3>(a, at, 0, k_lane, &staged);
    store_k<D, E4M3>(staged, k_lds[0]);
    load_v<D, E4M3>(a, at, 0, v_lane, &staged);
    store_v<D, E4M3>(staged, begin, u.len, v_lds[0], part(0), &dropped);
    if (tiles > 1) load_k<D, E4M3>(a, at, 1, k_lane, &staged);
    lds_barrier();
    // a wave without rows only brings in its share of the tiles (64 x 9 tokens of 4
    // heads at 3,000: 145 -> 140 us; 24 x 8 of 5 at 500: 19.5 -> 16.9)
    if (wave * 32 >= u.rows) {
      if (tiles > 1) store_k<D, E4M3>(staged, k_lds[1]);
      lds_barrier();
      for (int T = 0; T < tiles - 1; ++T) {
        const int key = begin + (T + 1) * kTileKeys;
        load_v<D, E4M3>(a, at, (T + 1) & 63, v_lane, &staged);
        store_v<D, E4M3>(staged, key, u.len, v_lds[(T + 1) & 1], part(T + 1), &dropped);
        if (T + 2 < tiles) {
          if (((T + 2) & 63) == 0) at = groups_at(a, table, h, ((key + kTileKeys) >> 4) + wave + 4 * lane, last_sub);
          load_k<D, E4M3>(a, at, (T + 2) & 63, k_lane, &staged);
          store_k<D, E4M3>(staged, k_lds[T & 1]);
        }
        lds_barrier();
      }
      return;
    }
    u32x4 p0[2], p1[2];
    p1[0] = p1[1] = u32x4{0u, 0u, 0u, 0u};
    f32x16 s0 = qk<D>(k_lds[0], 0, q);
    mask(s0, begin);
    refer(s0, nullptr, 0, p1);
    f32x16 s1 = qk<D>(k_lds[0], 1, q);
    weights(s0, &w, p0);
    if (tiles > 1) store_k<D, E4M3>(staged, k_lds[1]);
    lds_barrier();

    // step T: scores of tile T + 1, weights of keys 32 .. 95 and sums over
    // keys 0 .. 63 of tile T; meanwhile K of tile T + 2 and V of tile T + 1
    // come in, one after the other through the same registers
    // (trees of few nodes, bf16, 128-wide heads: both at once, straight into LDS,
    // is no faster; 16 sequences of 515 .. 4,099 keys, 32 nodes of 32 / 8 heads: 45 us either way)
    auto step = [&](int T, auto hidden) {
      constexpr bool HIDDEN = decltype(hidden)::value;
      const int key = begin + T * kTileKeys;
      const uint8_t* kl = k_lds[(T + 1) & 1];
      const uint8_t* vl = v_lds[T & 1];
      load_v<D, E4M3>(a, at, (T + 1) & 63, v_lane, &staged);
      if (HIDDEN) mask(s1, key + 32);
      refer(s1, vl, 0, p0);
      inner_step<D>(kl, 0, vl, 0, q, s1, &w, p0, o, &s0, p1);
      store_v<D, E4M3>(staged, key + kTileKeys, u.len, v_lds[(T + 1) & 1], HIDDEN && part(T + 1), &dropped);
      if (T + 2 < tiles) {
        if (((T + 2) & 63) == 0) at = groups_at(a, table, h, ((key + 2 * kTileKeys) >> 4) + wave + 4 * lane, last_sub);
        load_k<D, E4M3>(a, at, (T + 2) & 63, k_lane, &staged);
      }
      if (HIDDEN) mask(s0, key + kTileKeys);
      refer(s0, vl, 1, p1);
      inner_step<D>(kl, 1, vl, 1, q, s0, &w, p1, o, &s1, p0);
      if (T + 2 < tiles) store_k<D, E4M3>(staged, k_lds[T & 1]);
      lds_barrier();
    };
    // tiles [first, last) are seen whole; a loop each, for the hidden ones' work
    // in the whole tiles' loop cost 3 % there (and one loop with both bodies spills)
    const int first = max(0, full_lo - begin + kTileKeys - 1) / kTileKeys, last = max(0, full_hi - begin) / kTileKeys;
    int T = 0;
    for (; T < min(first, tiles - 1); ++T) step(T, std::true_type());
    for (; T < last - 1; ++T) step(T, std::false_type());
    for (; T < tiles - 1; ++T) step(T, std::true_type());
    const uint8_t* vl = v_lds[(tiles - 1) & 1];
    mask(s1, begin + (tiles - 1) * kTileKeys + 32);
    refer(s1, vl, 0, p0);
    weights(s1, &w, p1);
    pv<D>(vl, 0, p0, o);
    pv<D>(vl, 1, p1, o);

    // the outputs that dropped values would have reached
    if (__builtin_amdgcn_readfirstlane(dropped)) {
      int lo, hi;
      own_range(&lo, &hi);
      for (int T = 0; T < tiles; ++T) {
        const int key = begin + T * kTileKeys;
        if (!part(T)) continue;
        for_nonfinite<D, E4M3>(a, table, h, key, min(kTileKeys, u.len - key), [&](int k, const uint64_t (&bad)[D / 64]) {
          int g4 = 4 * g;
          pin(g4);
          const bool named = !TREE || (own_bits(k) & 1);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (named && k >= lo && k < hi && bad_at<D>(bad, 32 * dt + 8 * (i / 4) + g4 + i % 4))
                o[dt][i] = __uint_as_float(0x7fc00000u);
        });
      }
    }
  }

  const float sum = w.l + __shfl_xor(w.l, 32, 64);
  row = own_row();
  if (row >= u.rows) return;
  place = u.row0 + row;
  const int tok = u.first + place / a.group, head = h * a.group + place % a.group;
  const float v_scale = E4M3 && a.vc.scale ? a.vc.scale[h] : 1.0f;
  if (chunks <= 1) {
    const float inv = sum > 0.0f || sum != sum ? v_scale / sum : 0.0f;  // a row that saw no key is zero
    uint8_t* out = a.out.p + (int64_t)tok * a.out.token + (int64_t)head * a.out.head + g * 8;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x16& c = o[dt];
        *reinterpret_cast<u32x2*>(out + (32 * dt + 8 * i) * 2) =
            u32x2{bf16_pair(c[4 * i] * inv, c[4 * i + 1] * inv), bf16_pair(c[4 * i + 2] * inv, c[4 * i + 3] * inv)};
      }
    if (a.lse && g == 0)
      a.lse[(int64_t)tok * a.q_heads + head] = lse_of(w.m, sum);
  } else {
    if constexpr (TREE) {
      // as the registers lie, for the join's lanes to read in the same way
      uint64_t* out = reinterpret_cast<uint64_t*>(a.part_o) + ((int64_t)blockIdx.x * kTileWaves + wave) * (DT * 8 + 1) * 64 + lane;
      auto put = [&](int i, float x, float y) {
        out[i * 64] = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
      };
      put(0, w.m, sum);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 8; ++i) put(1 + dt * 8 + i, o[dt][2 * i] * v_scale, o[dt][2 * i + 1] * v_scale);
      return;
    }
    const int64_t part = part_at(a, h, split, u.first * a.group + place);
    float* out = a.part_o + part * D + 4 * g;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x16& c = o[dt];
        *reinterpret_cast<f32x4*>(out + 32 * dt + 8 * i) =
            f32x4{c[4 * i] * v_scale, c[4 * i + 1] * v_scale, c[4 * i + 2] * v_scale, c[4 * i + 3] * v_scale};
      }
    if (g == 0) {
      a.part_ml[part * 2] = w.m;
      a.part_ml[part * 2 + 1] = sum;
    }
  }
}

// Joins the shares of a tree's units.  grid.x: units of all KV heads, as unit_at
// numbers them; grid.y: 32 of the values.  A lane has the row and the values that
// it had in the tile kernel, and adds its shares in their order.
template <int D>
__global__ void __launch_bounds__(kTileWaves * 64) attn_tree_join_kernel(AttnArgs a) {
  constexpr int R = kTileRows, DT = D / 32, kAtOnce = 8;   // shares on their way
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), dt = blockIdx.y;
  const int h = (int)blockIdx.x % a.kv_heads;
  const Unit u = unit_at(a, (int)blockIdx.x / a.kv_heads, R);
  if (u.rows == 0) return;
  const int shares = uniform_i32(a.cut + 2 * u.b + 1);
  const int before = tree_first_share(uniform_i32(a.cut + 2 * u.b), u.row0 / R, shares, a.kv_heads, a.shares);
  if (before < 0) return;
  const int row = wave * 32 + (lane & 31), place = u.row0 + row;
  if (row >= u.rows) return;
  constexpr int64_t wide = (DT * 8 + 1) * 64;
  const uint64_t* p = reinterpret_cast<const uint64_t*>(a.part_o) + (((int64_t)before * a.kv_heads + h) * kTileWaves + wave) * wide + lane;
  const int64_t step = (int64_t)a.kv_heads * kTileWaves * wide;
  float m = kNegInf, l = 0.0f, x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  for (int c = 0; c < shares; c += kAtOnce) {
    uint64_t ml[kAtOnce], y[kAtOnce][8];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (c + k >= shares) break;
      const uint64_t* q = p + (c + k) * step;
      ml[k] = q[0];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[k][i] = q[(1 + dt * 8 + i) * 64];
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (c + k >= shares) break;
      const float m2 = __uint_as_float((uint32_t)ml[k]), l2 = __uint_as_float((uint32_t)(ml[k] >> 32));
      const float top = fmaxf(m, m2), base = top == kNegInf ? 0.0f : top;
      const float e = __builtin_amdgcn_exp2f(m - base), e2 = __builtin_amdgcn_exp2f(m2 - base);
      m = top;
      l = l * e + l2 * e2;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] = x[2 * i] * e + __uint_as_float((uint32_t)y[k][i]) * e2;
        x[2 * i + 1] = x[2 * i + 1] * e + __uint_as_float((uint32_t)(y[k][i] >> 32)) * e2;
      }
    }
  }
  const int tok = u.first + place / a.group, head = h * a.group + place % a.group;
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  uint8_t* out = a.out.p + (int64_t)tok * a.out.token + (int64_t)head * a.out.head + (32 * dt + 4 * (lane >> 5)) * 2;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<u32x2*>(out + 16 * i) =
        u32x2{bf16_pair(x[4 * i] * inv, x[4 * i + 1] * inv), bf16_pair(x[4 * i + 2] * inv, x[4 * i + 3] * inv)};
  if (a.lse && dt == 0 && lane < 32) a.lse[(int64_t)tok * a.q_heads + head] = lse_of(m, l);
}

hipError_t launch_attn_tree_join(const AttnArgs& a, int head_dim, int units, hipStream_t s) {
  if (head_dim == 64)
    hipLaunchKernelGGL((attn_tree_join_kernel<64>), dim3((unsigned)units, 2), dim3(kTileWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL((attn_tree_join_kernel<128>), dim3((unsigned)units, 4), dim3(kTileWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int D, bool E4M3>
static hipError_t launch_tile(const AttnArgs& a, int units, hipStream_t s) {
  const dim3 grid((unsigned)units * (unsigned)a.splits), threads(kTileWaves * 64);
  if (a.sees)
    hipLaunchKernelGGL((attn_tile_kernel<D, E4M3, true>), dim3((unsigned)a.shares), threads, 0, s, a);
  else
    hipLaunchKernelGGL((attn_tile_kernel<D, E4M3, false>), grid, threads, 0, s, a);
  return hipGetLastError();
}

int attn_tile_slots(int head_dim) { return 256 * tile_workgroups(head_dim); }

hipError_t launch_attn_tile(const AttnArgs& a, int head_dim, bool e4m3, int units, hipStream_t s) {
  if (head_dim == 64) return e4m3 ? launch_tile<64, true>(a, units, s) : launch_tile<64, false>(a, units, s);
  return e4m3 ? launch_tile<128, true>(a, units, s) : launch_tile<128, false>(a, units, s);
}

}  // namespace qlk
