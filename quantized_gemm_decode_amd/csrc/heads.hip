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
// is one exchange away.  A lane keeps its 8 cosines and sines for every head
// of its token: read per head they would be four times a row's own bytes.
#include "attention_args.hpp"
#include "quant_common.hpp"

namespace qlk {

// Sum over the L lanes that hold one row (L = 8, 16 or 32, aligned).
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < L; o *= 2) v += __shfl_xor(v, o, 64);
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
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = bf16_rne(f[2 * i]) | (bf16_rne(f[2 * i + 1]) << 16);
  return o;
}

// y / scale as E4M3, the quantizers' rule: the quotient clamped to +-448 and
// rounded to nearest even; a NaN stays one.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b, float s) {
  const float qa = __fdiv_rn(a, s), qb = __fdiv_rn(b, s);
  const uint32_t c = e4m3_pk2<false>(clamp448(qa), clamp448(qb), 0u) & 0xffffu;
  return (qa != qa ? (c & 0xff00u) | 0x7fu : c) | (qb != qb ? 0x7f00u : 0u);
}

__device__ __forceinline__ u32x2 e4m3_row8(const float* y, float s) {
  u32x2 o = {e4m3_pair(y[0], y[1], s) | (e4m3_pair(y[2], y[3], s) << 16),
             e4m3_pair(y[4], y[5], s) | (e4m3_pair(y[6], y[7], s) << 16)};
  return o;
}

constexpr int kHeadThreads = 256;

// Workgroup (t, part): token t, rows part*G + g, + G*gridDim.y ... of its
// heads, G = 256 / L rows at a time.  Head order: queries, keys, values.
template <int D, bool APPEND, bool E4M3>
__global__ void __launch_bounds__(kHeadThreads) heads_kernel(HeadArgs a) {
  constexpr int L = D / 8, G = kHeadThreads / L;
  const int t = blockIdx.x, lane = threadIdx.x % L;
  const int d0 = lane * 8;
  const int64_t pos = a.pos[t];
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
  // this lane's cosines and sines; for the half-split pairs with the sign of
  // its own side, so that y = n * cos + other * sin on either side
  const int half = a.rot / 2;
  const bool turned = d0 < a.rot;
  float c[8], s[8];
  int other = lane;
  if (turned) {
    const float* row = a.table + (known ? pos : 0) * a.rot;
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = row[d0 / 2 + i];
        s[2 * i + 1] = row[half + d0 / 2 + i];
        s[2 * i] = -s[2 * i + 1];
      }
    } else {
      const bool low = d0 < half;
      const int at = low ? d0 : d0 - half;
      other = low ? lane + half / 8 : lane - half / 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = row[at + i];
        const float v = row[half + at + i];
        s[i] = low ? -v : v;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
  }
  // a position outside the table has no rotation: its rows become NaN
  // instead of a read out of the table's range
  const float nan = __uint_as_float(0x7fc00000u);
  const int rows = a.q_heads + (APPEND ? 2 : 1) * a.kv_heads;
  for (int r = (int)blockIdx.y * G + (int)threadIdx.x / L; r < rows; r += G * (int)gridDim.y) {
    const bool is_q = r < a.q_heads, is_v = r >= a.q_heads + a.kv_heads;
    const int h = is_q ? r : is_v ? r - a.q_heads - a.kv_heads : r - a.q_heads;
    if (APPEND && !is_q && slot < 0) continue;  // whole rows: a row's lanes leave together
    const Rows& in = is_q ? a.q : is_v ? a.v : a.k;
    const u32x4 raw = *reinterpret_cast<const u32x4*>(in.p + t * in.token + h * in.head + d0 * 2);
    float y[8];
    unpack8(raw, y);
    if (!is_v) {
      const uint16_t* w = is_q ? a.q_w : a.k_w;
      u32x4 far;
#pragma unroll
      for (int i = 0; i < 4; ++i) far[i] = (uint32_t)__shfl((int)raw[i], other, L);
      float o[8];
      unpack8(far, o);
      if (w) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(y[i], y[i], ss);
        const float inv = rsqrtf(__fmaf_rn(row_sum<L>(ss), 1.0f / D, a.eps));
        float wy[8], wo[8];
        unpack8(*reinterpret_cast<const u32x4*>(w + d0), wy);
        unpack8(*reinterpret_cast<const u32x4*>(w + other * 8), wo);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = y[i] * inv * wy[i];
          o[i] = o[i] * inv * wo[i];
        }
      }
      if (turned) {
        float z[8];
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = y[i] * c[i] + y[i ^ 1] * s[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = y[i] * c[i] + o[i] * s[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = z[i];
      }
      if (!known && a.rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = nan;
      }
    }
    if (is_q || !APPEND) {
      const Rows& out = is_q ? a.q_out : a.k_out;
      *reinterpret_cast<u32x4*>(out.p + t * out.token + h * out.head + d0 * 2) = pack8(y);
    } else {
      const Pages& to = is_v ? a.vc : a.kc;
      uint8_t* at = to.p + (is_v ? v_at : k_at) + h * to.head;
      if constexpr (E4M3)
        *reinterpret_cast<u32x2*>(at + d0) = e4m3_row8(y, to.scale ? to.scale[h] : 1.0f);
      else
        *reinterpret_cast<u32x4*>(at + d0 * 2) = pack8(y);
    }
  }
}

template <int D>
static hipError_t launch_heads_d(const HeadArgs& a, bool append, bool e4m3, hipStream_t s) {
  const int rows = a.q_heads + (append ? 2 : 1) * a.kv_heads;
  const int passes = (rows + kHeadThreads / (D / 8) - 1) / (kHeadThreads / (D / 8));
  // few tokens: a token's rows over as many workgroups as it takes
  const int parts = (int64_t)a.tokens * passes <= 1024 ? passes : 1;
  const dim3 grid((unsigned)a.tokens, (unsigned)parts), block(kHeadThreads);
  if (!append)
    hipLaunchKernelGGL((heads_kernel<D, false, false>), grid, block, 0, s, a);
  else if (e4m3)
    hipLaunchKernelGGL((heads_kernel<D, true, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((heads_kernel<D, true, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_heads(const HeadArgs& a, int head_dim, bool append, bool e4m3, hipStream_t s) {
  if (head_dim == 64) return launch_heads_d<64>(a, append, e4m3, s);
  if (head_dim == 128) return launch_heads_d<128>(a, append, e4m3, s);
  return launch_heads_d<256>(a, append, e4m3, s);
}

}  // namespace qlk
