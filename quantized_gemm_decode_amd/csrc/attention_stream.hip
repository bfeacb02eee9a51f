// Attention over the paged cache for few rows a sequence: the decode kernel.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale q_r.k_j - m_r),
// in one pass over the keys with the running maximum m_r and sum of each row.
//
// Few rows (new tokens x query heads of a KV head) read long K and V, 2
// bytes (E4M3: 1) for 2 flops a row and value: bound by memory up to about
// 150 rows.  So the kernel is built as a stream.  Every wave takes tiles of
// 32 keys of its own and loads them straight into matrix-core operands, the
// next tile's loads in flight while it works on one; there is no barrier and
// no LDS until the workgroup's four waves join at the end.  Long contexts are
// cut into chunks over many workgroups; attention_join adds their partial
// results.
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
// P is rounded to bf16 for the product (its error, 2^-9 of a term at most,
// averages out below the output's own rounding); the row sums take P in
// binary32 before that, and all sums and maxima are binary32.
#include "attention_common.hpp"

namespace qlk {

constexpr int kStreamWaves = 4;

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
    const u32x4 t = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = t[i];
  } else if constexpr (N == 2) {
    const u32x2 t = *reinterpret_cast<const u32x2*>(p);
    o[0] = t.x;
    o[1] = t.y;
  } else {
    o[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Loads a tile: its two 16-key groups are entries i and i + 1 of `at`.
template <int D, bool E4M3>
__device__ __forceinline__ void load_tile(const AttnArgs& a, const Groups& at, int i, uint32_t k_lane, uint32_t v_lane,
                                          KvTile<D, E4M3>* t) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* k = a.kc.p + pick(at.k_lo, at.k_hi, i + u);
    const uint8_t* v = a.vc.p + pick(at.v_lo, at.v_hi, i + u);
#pragma unroll
    for (int s = 0; s < KvTile<D, E4M3>::KP; ++s) t->k[u][s] = *reinterpret_cast<const u32x4*>(k + k_lane + 64 * s);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_words<KvTile<D, E4M3>::VW>(v + j * (int)a.vc.token + v_lane, t->v[4 * u + j]);
  }
}

// The groups of a wave's next 32 tiles, the first at key `key`.
__device__ __forceinline__ Groups tile_groups(const AttnArgs& a, const int32_t* table, int h, int key, int last) {
  const int lane = threadIdx.x & 63;
  return groups_at(a, table, h, (key >> 4) + 2 * kStreamWaves * (lane >> 1) + (lane & 1), last);
}

// V^T operand of product dt from a tile's value rows: 8 keys of one value.
template <int D, bool E4M3>
__device__ __forceinline__ u32x4 v_operand(const KvTile<D, E4M3>& t, int dt) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E4M3) {
      const uint32_t c = __builtin_amdgcn_perm(t.v[2 * i + 1][dt / 4], t.v[2 * i][dt / 4],
                                               0x0c0c0000u | (uint32_t)((dt % 4) | ((4 + dt % 4) << 8)));
      o[i] = e4m3_to_bf16<false>(c);
    } else {
      o[i] = __builtin_amdgcn_perm(t.v[2 * i + 1][dt / 2], t.v[2 * i][dt / 2], dt % 2 ? 0x07060302u : 0x05040100u);
    }
  }
  return o;
}

template <int D, bool E4M3, int NR>
__global__ void __launch_bounds__(kStreamWaves * 64, NR == 4 ? 1 : 2) attn_stream_kernel(AttnArgs a) {
  constexpr int R = 16 * NR, DT = D / 16;
  constexpr int KS = D / 32;  // products over D of one 16-key group
  using Tile = KvTile<D, E4M3>;
  // the next tile's registers fit beside the sums of few rows only
  constexpr bool AHEAD = NR == 1 || E4M3;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  int id = blockIdx.x;
  const int h = id % a.kv_heads;
  id /= a.kv_heads;
  const int split = id % a.splits;
  id /= a.splits;
  const int block = id % a.row_blocks, b = id / a.row_blocks;
  const Unit u = unit_of(a, b, block, R);
  if (u.rows == 0 || u.all > a.max_rows) return;
  if (u.chunks == 0 ? split != 0 : split >= u.chunks) return;
  const int begin = (u.lo & ~63) + split * a.chunk;
  const int end = min(u.hi, begin + a.chunk);

  // Q operands, and the keys each of this lane's rows sees
  u32x4 q[NR][KS];
  int lo[NR], hi[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int row = 16 * n + r;
    row_range(a, u, row, &lo[n], &hi[n]);
    if (row >= u.rows) lo[n] = hi[n] = 0;
    const int at = u.row0 + row, tok = at / a.group, head = h * a.group + at % a.group;
    const uint8_t* p = a.q.p + (int64_t)(u.first + tok) * a.q.token + (int64_t)head * a.q.head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d0 = E4M3 ? ((s / 2) * 4 + g) * 16 + (s % 2) * 8 : (s * 4 + g) * 8;
      q[n][s] = row < u.rows ? *reinterpret_cast<const u32x4*>(p + d0 * 2) : u32x4{0u, 0u, 0u, 0u};
    }
  }
  const float scale = a.scale_log2 * (E4M3 && a.kc.scale ? a.kc.scale[h] : 1.0f);

  f32x4 o[NR][DT];
  float m[NR], l[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    m[n] = kNegInf;
    l[n] = 0.0f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[n][dt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // tiles every row of the block sees whole need no mask
  int full_lo, full_hi, x;
  row_range(a, u, u.rows - 1, &full_lo, &x);
  row_range(a, u, 0, &x, &full_hi);
  const int32_t* table = a.table + b * a.table_row;
  const int last_sub = (u.len - 1) >> 4;
  const uint32_t k_lane = (uint32_t)(r * (int)a.kc.token + g * 16);
  const uint32_t v_lane = (uint32_t)(4 * g * (int)a.vc.token + r * Tile::VW * 4);

  // this wave's tiles are every fourth: lane i holds group i % 2 of its tile
  // i / 2, 32 tiles at a time
  int key = begin + 32 * wave, tile = 0;
  Groups at;
  Tile cur;
  if (key < end) {
    at = tile_groups(a, table, h, key, last_sub);
    if (AHEAD) load_tile<D, E4M3>(a, at, 0, k_lane, v_lane, &cur);
  }
  for (; key < end; key += 32 * kStreamWaves) {
    Tile next;
    if (!AHEAD) load_tile<D, E4M3>(a, at, 2 * (tile & 31), k_lane, v_lane, &cur);
    if (key + 32 * kStreamWaves < end) {
      if ((++tile & 31) == 0) at = tile_groups(a, table, h, key + 32 * kStreamWaves, last_sub);
      if (AHEAD) load_tile<D, E4M3>(a, at, 2 * (tile & 31), k_lane, v_lane, &next);
    }
    if (key + 32 > u.len) {  // the cache beyond the sequence may hold anything: 0 * NaN would reach every row
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (key + 16 * (j / 4) + 4 * g + j % 4 >= u.len)
#pragma unroll
          for (int w = 0; w < Tile::VW; ++w) cur.v[j][w] = 0u;
    }
    const bool whole = key >= full_lo && key + 32 <= full_hi;
    u32x4 p[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float s[8];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          u32x4 k;
          if constexpr (E4M3) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t codes = cur.k[v][i / 2][(i % 2) * 2 + w];
              k[2 * w] = e4m3_to_bf16<false>(codes);
              k[2 * w + 1] = e4m3_to_bf16<true>(codes);
            }
          } else {
            k = cur.k[v][i];
          }
          c = mma_bf16(k, q[n][i], c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * v + i] = c[i];
      }
      if (whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] *= scale;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = key + 16 * (i / 4) + 4 * g + i % 4;
          s[i] = at >= lo[n] && at < hi[n] ? s[i] * scale : kNegInf;
        }
      }
      float top = s[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i]);
      top = fmaxf(m[n], row4_max(top));
      const float base = top == kNegInf ? 0.0f : top;  // a row that has seen no key yet
      const float keep = __builtin_amdgcn_exp2f(m[n] - base);
      m[n] = top;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[i] = __builtin_amdgcn_exp2f(s[i] - base);
        sum += s[i];
      }
      l[n] = l[n] * keep + sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[n][i] = bf16_pair(s[2 * i], s[2 * i + 1]);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[n][dt] *= keep;
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const u32x4 v = v_operand<D, E4M3>(cur, dt);
#pragma unroll
      for (int n = 0; n < NR; ++n) o[n][dt] = mma_bf16(v, p[n], o[n][dt]);
    }
    if (AHEAD) cur = next;
  }

  // join the four waves: each scales its sums to the common maximum, then a
  // thread adds 8 values of a row over the waves
  constexpr int LD = D + 4;  // floats between rows
  extern __shared__ float lds[];
  float* const ml = lds + kStreamWaves * 16 * LD;  // [wave][NR][16][2]
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    l[n] = row4_sum(l[n]);
    if (g == 0) {
      ml[((wave * NR + n) * 16 + r) * 2] = m[n];
      ml[((wave * NR + n) * 16 + r) * 2 + 1] = l[n];
    }
  }
  __syncthreads();
  const float v_scale = E4M3 && a.vc.scale ? a.vc.scale[h] : 1.0f;
  const bool alone = u.chunks <= 1;
  const int64_t unit = ((int64_t)b * a.row_blocks + block) * a.kv_heads + h;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float top = kNegInf, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kStreamWaves; ++w) top = fmaxf(top, ml[((w * NR + n) * 16 + r) * 2]);
    const float base = top == kNegInf ? 0.0f : top;
    const float keep = __builtin_amdgcn_exp2f(m[n] - base);
    if (n) __syncthreads();
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) lds[(wave * 16 + r) * LD + (4 * g + i) * DT + dt] = o[n][dt][i] * keep;
    __syncthreads();
    // 16 threads a row, D/16 values each
    const int row = threadIdx.x / 16, d0 = (threadIdx.x % 16) * DT;
    const int mine = 16 * n + row;
    if (mine < u.rows) {
      float acc[DT];
#pragma unroll
      for (int i = 0; i < DT; ++i) acc[i] = 0.0f;
      float rt = kNegInf;
#pragma unroll
      for (int w = 0; w < kStreamWaves; ++w) rt = fmaxf(rt, ml[((w * NR + n) * 16 + row) * 2]);
      const float rb = rt == kNegInf ? 0.0f : rt;
#pragma unroll
      for (int w = 0; w < kStreamWaves; ++w) {
        sum += ml[((w * NR + n) * 16 + row) * 2 + 1] * __builtin_amdgcn_exp2f(ml[((w * NR + n) * 16 + row) * 2] - rb);
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[i] += lds[(w * 16 + row) * LD + d0 + i];
      }
      const int at = u.row0 + mine, tok = u.first + at / a.group, head = h * a.group + at % a.group;
      if (alone) {
        // a row that saw no key is zero
        const float inv = sum > 0.0f || sum != sum ? v_scale / sum : 0.0f;
        uint32_t w[DT / 2];
#pragma unroll
        for (int i = 0; i < DT / 2; ++i) w[i] = bf16_pair(acc[2 * i] * inv, acc[2 * i + 1] * inv);
        uint8_t* out = a.out.p + (int64_t)tok * a.out.token + (int64_t)head * a.out.head + d0 * 2;
        if constexpr (DT == 8)
          *reinterpret_cast<u32x4*>(out) = u32x4{w[0], w[1], w[2], w[3]};
        else
          *reinterpret_cast<u32x2*>(out) = u32x2{w[0], w[1]};
        if (a.lse && d0 == 0)
          a.lse[(int64_t)tok * a.q_heads + head] = rt == kNegInf ? kNegInf : (rt + log2f(sum)) * 0.6931471805599453f;
      } else {
        const int64_t part = (unit * a.splits + split) * R + mine;
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[i] *= v_scale;
#pragma unroll
        for (int i = 0; i < DT; i += 4)
          *reinterpret_cast<f32x4*>(a.part_o + part * D + d0 + i) = f32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
        if (d0 == 0) {
          a.part_ml[part * 2] = rt;
          a.part_ml[part * 2 + 1] = sum;
        }
      }
    }
  }
}

// Adds the chunks of a unit: one wave a row.  o = sum_c e_c o_c / sum_c e_c
// l_c with e_c = exp(m_c - max m).  Rows whose unit had one chunk were
// written by the attention kernel.
constexpr int kJoinWaves = 4;

template <int D>
__global__ void __launch_bounds__(kJoinWaves * 64) attn_join_kernel(AttnArgs a, int R) {
  constexpr int W = D / 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int id = blockIdx.x;
  const int h = id % a.kv_heads;
  id /= a.kv_heads;
  const int per = R / kJoinWaves;
  const int row = (id % per) * kJoinWaves + wave;
  id /= per;
  const int block = id % a.row_blocks, b = id / a.row_blocks;
  const Unit u = unit_of(a, b, block, R);
  if (row >= u.rows || u.chunks <= 1 || u.all > a.max_rows || u.all < a.min_rows) return;
  const int64_t unit = ((int64_t)b * a.row_blocks + block) * a.kv_heads + h;
  const float* ml = a.part_ml + (unit * a.splits * R + row) * 2;
  const int n = min(u.chunks, a.splits);
  float top = kNegInf;
  for (int c = lane; c < n; c += 64) top = fmaxf(top, ml[(int64_t)c * R * 2]);
  for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
  const float base = top == kNegInf ? 0.0f : top;
  float sum = 0.0f, acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.0f;
  const float* po = a.part_o + (unit * a.splits * R + row) * D + lane * W;
  for (int c = 0; c < n; ++c) {
    const float e = __builtin_amdgcn_exp2f(ml[(int64_t)c * R * 2] - base);
    sum = __fmaf_rn(e, ml[(int64_t)c * R * 2 + 1], sum);
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = __fmaf_rn(e, po[(int64_t)c * R * D + i], acc[i]);
  }
  const int at = u.row0 + row, tok = u.first + at / a.group, head = h * a.group + at % a.group;
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  uint8_t* out = a.out.p + (int64_t)tok * a.out.token + (int64_t)head * a.out.head + lane * W * 2;
  if constexpr (W == 2)
    *reinterpret_cast<uint32_t*>(out) = bf16_pair(acc[0] * inv, acc[1] * inv);
  else
    *reinterpret_cast<uint16_t*>(out) = (uint16_t)bf16_rne(acc[0] * inv);
  if (a.lse && lane == 0)
    a.lse[(int64_t)tok * a.q_heads + head] = top == kNegInf ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool E4M3, int NR>
static hipError_t launch_stream(const AttnArgs& a, int units, hipStream_t s) {
  const unsigned grid = (unsigned)units * (unsigned)a.splits;
  const size_t lds = (kStreamWaves * 16 * (D + 4) + kStreamWaves * NR * 16 * 2) * sizeof(float);
  hipLaunchKernelGGL((attn_stream_kernel<D, E4M3, NR>), dim3(grid), dim3(kStreamWaves * 64), lds, s, a);
  return hipGetLastError();
}

template <int D, bool E4M3>
static hipError_t launch_stream_d(const AttnArgs& a, int rows, int units, hipStream_t s) {
  if (rows == 16) return launch_stream<D, E4M3, 1>(a, units, s);
  if (rows == 32) return launch_stream<D, E4M3, 2>(a, units, s);
  return launch_stream<D, E4M3, 4>(a, units, s);
}

hipError_t launch_attn_stream(const AttnArgs& a, int head_dim, bool e4m3, int rows, int units, hipStream_t s) {
  if (head_dim == 64)
    return e4m3 ? launch_stream_d<64, true>(a, rows, units, s) : launch_stream_d<64, false>(a, rows, units, s);
  return e4m3 ? launch_stream_d<128, true>(a, rows, units, s) : launch_stream_d<128, false>(a, rows, units, s);
}

hipError_t launch_attn_join(const AttnArgs& a, int head_dim, int rows, int batch, hipStream_t s) {
  const unsigned grid = (unsigned)batch * (unsigned)a.row_blocks * (unsigned)a.kv_heads * (unsigned)(rows / kJoinWaves);
  if (head_dim == 64)
    hipLaunchKernelGGL((attn_join_kernel<64>), dim3(grid), dim3(kJoinWaves * 64), 0, s, a, rows);
  else
    hipLaunchKernelGGL((attn_join_kernel<128>), dim3(grid), dim3(kJoinWaves * 64), 0, s, a, rows);
  return hipGetLastError();
}

}  // namespace qlk
