// Per-head norm and position rotation of queries and keys, and their append
// to a paged cache.
//
// One row is the head_dim values x of one head of one token:
//   n = x * w / sqrt(mean(x^2) + eps)       (w given; else n = x)
//   y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin
// over the pairs (a, b) of the first `rot` values -- (i, rot/2 + i), or
// (2i, 2i+1) interleaved -- with the token's row of the cosine / sine table.
// All in binary32, rounded once to the output's type (bf16, or E4M3 of
// y / scale as the library's quantizers round it).
//
// 8 flops a value against 4 bytes moved: bound by memory, and by the launch
// for few tokens.  A row is held by head_dim/8 lanes, 8 values (16 bytes)
// each, so a wave reads and writes whole rows in contiguous pieces, the sum
// of squares stays inside a 16-lane row of the wave, and a pair's other half
// is one exchange away.  Norm weight and rotation are folded into two factors
// a value, kept for all heads of a token by the wave that has the token: made
// anew for every head they are most of the arithmetic, which then bounds it.
// Two rows a lane are on their way while the two before are worked on.
// Measured: 8,191 tokens of 40 + 8 heads of 128 (206 MB) 42.1 us, 4.9 TB/s, what a
// large copy reaches here; 43.1 and 43.6 us with three and four rows ahead.
// Append of 4,096 tokens of 32 + 2 x 8 heads as E4M3 (94 MB) 24.6 us, 3.8 TB/s:
// with one token a wave 4,096 waves do not fill the card, and with half a token
// each (27.1 us) the factors are made twice.
#include <algorithm>
#include <type_traits>

#include "attention_common.hpp"
#include "quant_common.hpp"

namespace qlk {

// Sum over the L lanes that hold one row (L = 8, 16 or 32, aligned): lane
// swaps inside 16 lanes (xor 1, xor 2, half-row mirror, row mirror).
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  auto swap = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  v += swap(v, std::integral_constant<int, 0xB1>());
  v += swap(v, std::integral_constant<int, 0x4E>());
  v += swap(v, std::integral_constant<int, 0x141>());
  if (L >= 16) v += swap(v, std::integral_constant<int, 0x140>());
  if (L >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

__device__ __forceinline__ void unpack8(const u32x4& v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ u32x4 pack8(const float* f) {
  return u32x4{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
}

// y / s as E4M3, the quantizers' rule: the quotient clamped to +-448 and
// rounded to nearest even; a NaN stays one.  The quotient comes from the
// rounded reciprocal with the exact remainder put right (div_fast), which
// needs y within reach of the clamp and s a normal number with a normal
// reciprocal; any other scale takes the division.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b, float s, float r) {
  const float reach = 512.0f * s;
  const float qa = r != 0.0f ? div_fast(__builtin_amdgcn_fmed3f(a, -reach, reach), s, r) : __fdiv_rn(a, s);
  const float qb = r != 0.0f ? div_fast(__builtin_amdgcn_fmed3f(b, -reach, reach), s, r) : __fdiv_rn(b, s);
  const uint32_t c = e4m3_pk2<false>(clamp448(qa), clamp448(qb), 0u) & 0xffffu;
  return (a != a ? (c & 0xff00u) | 0x7fu : c) | (b != b ? 0x7f00u : 0u);
}

__device__ __forceinline__ u32x2 e4m3_row8(const float* y, float s) {
  const float r = s >= FAST_DIV_MIN_SCALE && s <= 1.0f / FAST_DIV_MIN_SCALE ? __fdiv_rn(1.0f, s) : 0.0f;
  u32x2 o = {e4m3_pair(y[0], y[1], s, r) | (e4m3_pair(y[2], y[3], s, r) << 16),
             e4m3_pair(y[4], y[5], s, r) | (e4m3_pair(y[6], y[7], s, r) << 16)};
  return o;
}

constexpr int kHeadThreads = 256;
constexpr int kHeadWaves = 4096;  // waves up to which a token's rows go to several
constexpr int kHeadRows = 2;      // rows a lane has on their way at once

// Requests a round of rows: kHeadRows of them, `step` apart.
__device__ __forceinline__ void load_rows(u32x4 (&raw)[kHeadRows], int r0, int step, int rows, int first_k, int first_v,
                                          const uint8_t* in_q, const uint8_t* in_k, const uint8_t* in_v, uint32_t head_q,
                                          uint32_t head_k, uint32_t head_v, int d) {
#pragma unroll
  for (int i = 0; i < kHeadRows; ++i) {
    const int r = r0 + i * step;
    if (r >= rows) continue;
    const bool is_q = r < first_k, is_v = r >= first_v;
    const uint8_t* in = is_v ? in_v : in_k;
    in = is_q ? in_q : in;
    const uint32_t head = is_q ? head_q : is_v ? head_v : head_k;
    const uint32_t h = (uint32_t)(r - (is_q ? 0 : is_v ? first_v : first_k));
    raw[i] = *reinterpret_cast<const u32x4*>(in + h * head + d);
  }
}

// Wave (t, part) of tokens x parts: token t, rows part*G + g, + G*parts, ... of
// its heads, G = 64 / L rows at a time.  Head order: queries, keys, values.
// Many tokens: a wave has a whole token, so that its cosines, sines and
// weights serve all heads; few: a token's rows over several waves.
template <int D, bool APPEND, bool E4M3>
__global__ void __launch_bounds__(kHeadThreads) heads_kernel(HeadArgs a, int parts) {
  constexpr int L = D / 8, G = 64 / L;
  const int w = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * (kHeadThreads / 64) + threadIdx.x / 64));
  const int t = w / parts, part = w - t * parts;
  if (t >= a.tokens) return;
  const int lane = threadIdx.x % L;
  const int d0 = lane * 8;
  // a round of rows is on its way before the tables' values that it waits for
  // (which hang on the position), later rounds while the one before is worked on
  const int rows = a.q_heads + (APPEND ? 2 : 1) * a.kv_heads;
  const int step = G * parts;
  const uint8_t* in_q = a.q.p + t * a.q.token;
  const uint8_t* in_k = a.k.p + t * a.k.token;
  const uint8_t* in_v = a.v.p + t * a.v.token;
  const uint32_t head_q = (uint32_t)a.q.head, head_k = (uint32_t)a.k.head, head_v = (uint32_t)a.v.head;
  const int first_k = a.q_heads, first_v = a.q_heads + a.kv_heads;
  u32x4 raw[kHeadRows];
  int r0 = part * G + (int)(threadIdx.x & 63) / L;
  const int half = a.rot / 2;
  const bool turned = d0 < a.rot, low = d0 < half;
  // the lane of a pair's other halves
  const int other = !turned || a.interleaved ? lane : low ? lane + half / 8 : lane - half / 8;
  const int64_t pos = a.pos[t];
  load_rows(raw, r0, step, rows, first_k, first_v, in_q, in_k, in_v, head_q, head_k, head_v, d0 * 2);
  u32x4 weight[2][2] = {};
  if (a.q_w) {
    weight[0][0] = *reinterpret_cast<const u32x4*>(a.q_w + d0);
    weight[0][1] = *reinterpret_cast<const u32x4*>(a.q_w + other * 8);
  }
  if (a.k_w) {
    weight[1][0] = *reinterpret_cast<const u32x4*>(a.k_w + d0);
    weight[1][1] = *reinterpret_cast<const u32x4*>(a.k_w + other * 8);
  }
  const bool known = pos >= 0 && pos < a.max_pos;
  int64_t slot = -1;
  int64_t k_at = 0, v_at = 0;
  if constexpr (APPEND) {
    slot = a.slots[t];
    if (slot < 0 || slot >= a.num_slots) slot = -1;
    const int64_t page = slot < 0 ? 0 : page_of((int)(slot / 16), a.page_magic);
    const int64_t at = slot < 0 ? 0 : slot - page * a.page_size;
    k_at = page * a.kc.page + at * a.kc.token;
    v_at = page * a.vc.page + at * a.vc.token;
  }
  // y = inv (x A + x' B) with x' the pair's other half: A = w cos, B = w' sin
  // with the sign of this lane's side, once a token for its queries and keys
  float c[8], s[8];
  if (turned && known) {
    const float* row = a.table + pos * a.rot;
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = (*reinterpret_cast<const f32x4u*>(row + d0 / 2))[i];
        s[2 * i + 1] = (*reinterpret_cast<const f32x4u*>(row + half + d0 / 2))[i];
        s[2 * i] = -s[2 * i + 1];
      }
    } else {
      const int at = low ? d0 : d0 - half;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const f32x4u x = *reinterpret_cast<const f32x4u*>(row + at + i);
        const f32x4u z = *reinterpret_cast<const f32x4u*>(row + half + at + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[i + j] = x[j];
          s[i + j] = low ? -z[j] : z[j];
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
  }
  if (!known && a.rot) {
    // a position outside the table has no rotation: its rows become NaN
    // instead of a read out of the table's range
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __uint_as_float(0x7fc00000u);
  }
  float A[2][8], B[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bool given = (k ? a.k_w : a.q_w) != nullptr;
    float mine[8], far[8];
    unpack8(weight[k][0], mine);
    unpack8(weight[k][1], far);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      A[k][i] = given ? mine[i] * c[i] : c[i];
      B[k][i] = given ? far[a.interleaved ? i ^ 1 : i] * s[i] : s[i];
    }
  }
  uint8_t* const out_q = a.q_out.p + t * a.q_out.token;
  uint8_t* const out_k = a.k_out.p + t * a.k_out.token;
  const uint32_t out_head_q = (uint32_t)a.q_out.head, out_head_k = (uint32_t)a.k_out.head;
  uint8_t* const cache_k = a.kc.p + k_at;
  uint8_t* const cache_v = a.vc.p + v_at;
  const int64_t cache_head_k = a.kc.head, cache_head_v = a.vc.head;
  const float *const scale_k = a.kc.scale, *const scale_v = a.vc.scale;
  const bool some = a.rot < D && !turned;  // values beyond the rotation: not even 0 times the partner
  for (; r0 < rows; r0 += step * kHeadRows) {
    u32x4 now[kHeadRows];
#pragma unroll
    for (int i = 0; i < kHeadRows; ++i) now[i] = raw[i];
    if (r0 + step * kHeadRows < rows)
      load_rows(raw, r0 + step * kHeadRows, step, rows, first_k, first_v, in_q, in_k, in_v, head_q, head_k, head_v, d0 * 2);
#pragma unroll
    for (int i = 0; i < kHeadRows; ++i) {
      const int r = r0 + i * step;
      if (r >= rows) continue;  // a row's lanes leave together
      const bool is_q = r < a.q_heads, is_v = r >= a.q_heads + a.kv_heads;
      const int h = is_q ? r : is_v ? r - a.q_heads - a.kv_heads : r - a.q_heads;
      if (APPEND && !is_q && slot < 0) continue;
      float y[8];
      unpack8(now[i], y);
      if (!is_v) {
        float o[8];
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = y[j ^ 1];
        } else {
          u32x4 far;
#pragma unroll
          for (int j = 0; j < 4; ++j) far[j] = (uint32_t)__shfl((int)now[i][j], other, L);
          unpack8(far, o);
        }
        float inv = 1.0f;
        if (is_q ? a.q_w != nullptr : a.k_w != nullptr) {
          float ss = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = __fmaf_rn(y[j], y[j], ss);
          inv = rsqrtf(__fmaf_rn(row_sum<L>(ss), 1.0f / D, a.eps));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float b = is_q ? B[0][j] : B[1][j], z = y[j] * (is_q ? A[0][j] : A[1][j]);
          y[j] = inv * (some ? z : __fmaf_rn(o[j], b, z));
        }
      }
      if (is_q || !APPEND) {
        uint8_t* at = (is_q ? out_q : out_k) + (uint32_t)h * (is_q ? out_head_q : out_head_k) + d0 * 2;
        *reinterpret_cast<u32x4*>(at) = pack8(y);
      } else {
        uint8_t* at = (is_v ? cache_v : cache_k) + (int64_t)h * (is_v ? cache_head_v : cache_head_k);
        const float* scale = is_v ? scale_v : scale_k;
        if constexpr (E4M3)
          *reinterpret_cast<u32x2*>(at + d0) = e4m3_row8(y, scale ? scale[h] : 1.0f);
        else
          *reinterpret_cast<u32x4*>(at + d0 * 2) = pack8(y);
      }
    }
  }
}

template <int D>
static hipError_t launch_heads_d(const HeadArgs& a, bool append, bool e4m3, hipStream_t s) {
  const int rows = a.q_heads + (append ? 2 : 1) * a.kv_heads;
  const int passes = (rows + 64 / (D / 8) - 1) / (64 / (D / 8));
  // a few waves for each SIMD before a wave gets more than one pass
  const int parts = std::max(1, std::min(passes, kHeadWaves / a.tokens));
  const int waves = kHeadThreads / 64;
  const dim3 grid((unsigned)(((int64_t)a.tokens * parts + waves - 1) / waves)), block(kHeadThreads);
  if (!append)
    hipLaunchKernelGGL((heads_kernel<D, false, false>), grid, block, 0, s, a, parts);
  else if (e4m3)
    hipLaunchKernelGGL((heads_kernel<D, true, true>), grid, block, 0, s, a, parts);
  else
    hipLaunchKernelGGL((heads_kernel<D, true, false>), grid, block, 0, s, a, parts);
  return hipGetLastError();
}

hipError_t launch_heads(const HeadArgs& a, int head_dim, bool append, bool e4m3, hipStream_t s) {
  if (head_dim == 64) return launch_heads_d<64>(a, append, e4m3, s);
  if (head_dim == 128) return launch_heads_d<128>(a, append, e4m3, s);
  return launch_heads_d<256>(a, append, e4m3, s);
}

}  // namespace qlk
