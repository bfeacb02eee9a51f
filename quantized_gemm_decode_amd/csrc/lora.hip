// Low-rank adapters of many requests beside a shared projection.
//
//   out[t, n] = y[t, n] + s_i sum_r B_i[n, r] h[t, j R + r],
//   h[t, j R + r] = sum_k A_i[j R + r, k] x[t, k],
// i = adapter[t], j the slice of the merged projection that column n lies in.
//
// Bytes bound it: a decode step reads each adapter in use once (4 flops a
// byte), a prompt chunk reads x and reads and writes y.  Two launches.
//
// Tokens of one adapter share its weights: of 64 tokens, one a lane, a wave
// finds the j-th adapter among them by ballots and takes that adapter's tokens,
// 16 at a time, as the columns of 16x16x32 products (lane l = 16 g + r holds 8
// values of K, or of the ranks, of row r).  Other tokens' columns never meet
// its weights, so nothing an adapter holds reaches them.
//
// First product: a wave takes one chunk of K of one adapter; partial sums are
// binary32 and are added in their order by the second product's waves, so
// results do not depend on timing.
// Second product: h enters as two bf16 numbers, itself rounded and what that
// left out (2^-16 of it), in the same instruction where the ranks leave room
// (R = 16: 16 of its 32 places each).  out is rounded to bf16 once.
#include "attention_common.hpp"
#include "serving_args.hpp"

namespace qlk {

constexpr int kLoraWaves = 4;

// The adapter of this lane's token of block `block`, -1 without one; lanes
// beyond the tokens are not in `there`.
__device__ __forceinline__ int lane_adapter(const LoraArgs& a, int block, uint64_t* there) {
  const int t = block * kLoraBlock + (threadIdx.x & 63);
  const bool in = t < a.tokens;
  const int i = in ? a.adapter[t] : -1;
  *there = __ballot(in);
  return i >= 0 && i < a.adapters ? i : -1;
}

// Calls f(adapter, mask of its tokens) for adapters number slot, slot + slots,
// ... among the lanes of `left`.
template <class F>
__device__ __forceinline__ void for_adapters(int mine, uint64_t left, int slot, int slots, F f) {
  for (int n = 0; left; ++n) {
    const int i = lane_i32(mine, __ffsll((unsigned long long)left) - 1);
    const uint64_t same = __ballot(mine == i) & left;
    left &= ~same;
    if (n == slot) {
      f(i, same);
      slot += slots;
    }
  }
}

// Lane c gets the c-th lane of `mask` (those after them: the other lanes).
__device__ __forceinline__ int nth_lane(uint64_t mask) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int at = mask >> lane & 1 ? __popcll(mask & below) : __popcll(mask) + __popcll(~mask & below);
  return __builtin_amdgcn_ds_permute(at * 4, lane);
}

// h of one adapter's tokens, one chunk of K, TW tiles of 16 ranks.
template <int NT, int TW>
__global__ void __launch_bounds__(kLoraWaves * 64) lora_down_kernel(LoraArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int rows = a.slices * a.rank;
  const int groups = (rows + 16 * TW - 1) / (16 * TW);
  int id = (int)blockIdx.x * kLoraWaves + wave;
  const int chunk = id % a.chunks;
  id /= a.chunks;
  const int row0 = id % groups * 16 * TW;
  id /= groups;
  const int slot = id % a.down_slots, block = id / a.down_slots;
  if (block * kLoraBlock >= a.tokens) return;
  uint64_t there;
  const int mine = lane_adapter(a, block, &there);
  const int k0 = chunk * a.chunk, k1 = min(a.k, k0 + a.chunk);
  for_adapters(mine, __ballot(mine >= 0), slot, a.down_slots, [&](int i, uint64_t mask) {
    const int n = __popcll(mask), order = nth_lane(mask);
    const uint8_t* wp[TW];
#pragma unroll
    for (int v = 0; v < TW; ++v)
      wp[v] = a.a + i * a.a_step + (int64_t)min(row0 + 16 * v + r, rows - 1) * a.k * 2 + g * 32;
    for (int c0 = 0; c0 < n; c0 += 16 * NT) {
      const uint8_t* xp[NT];
      int tok[NT];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        tok[u] = block * kLoraBlock + __shfl(order, min(c0 + 16 * u + r, n - 1), 64);
        xp[u] = a.x + tok[u] * a.x_row + g * 32;
      }
      f32x4 h[NT][TW];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int v = 0; v < TW; ++v) h[u][v] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      // 64 values of K a step, 16 a lane: whole 128-byte lines of a row
      auto step = [&](int k, bool tail) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const bool in = !tail || k + 16 * g + 8 * half < k1;
          const u32x4 zero = {0u, 0u, 0u, 0u};
          u32x4 w[TW];
#pragma unroll
          for (int v = 0; v < TW; ++v)
            w[v] = in ? *reinterpret_cast<const u32x4*>(wp[v] + (int64_t)k * 2 + half * 16) : zero;
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            const u32x4 x = in ? *reinterpret_cast<const u32x4*>(xp[u] + (int64_t)k * 2 + half * 16) : zero;
#pragma unroll
            for (int v = 0; v < TW; ++v) h[u][v] = mma_bf16(w[v], x, h[u][v]);
          }
        }
      };
      int k = k0;
#pragma unroll 4
      for (; k + 64 <= k1; k += 64) step(k, false);
      if (k < k1) step(k, true);
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int v = 0; v < TW; ++v)
          if (c0 + 16 * u + r < n && row0 + 16 * v + 4 * g < rows)
            *reinterpret_cast<f32x4*>(a.part + ((int64_t)chunk * a.tokens + tok[u]) * rows + row0 + 16 * v + 4 * g) = h[u][v];
    }
  });
}

// out = y + s B h for one adapter's tokens and a range of column tiles of one
// slice.  STEPS: products over the ranks, 2 R / 32 rounded up.
template <int NT, int STEPS>
__global__ void __launch_bounds__(kLoraWaves * 64) lora_up_kernel(LoraArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  int id = (int)blockIdx.x * kLoraWaves + wave;
  int range = id % a.ranges, slice = 0, first = 0;
  id /= a.ranges;
  const int slot = id % a.up_slots, block = id / a.up_slots;
  if (block * kLoraBlock >= a.tokens) return;
  // the slice, and its first column
  const int wide = a.tiles_wave * 64;
  for (;; ++slice) {
    const int here = (a.width[slice] + wide - 1) / wide;
    if (range < here) break;
    range -= here;
    first += a.width[slice];
  }
  const int width = a.width[slice], rows = a.slices * a.rank, octets = a.rank / 8;
  const int n0 = range * wide, n1 = min(width, n0 + wide);
  uint64_t there;
  const int mine = lane_adapter(a, block, &there);
  for_adapters(mine, there, slot, a.up_slots, [&](int i, uint64_t mask) {
    if (i < 0 && a.out == a.y) return;
    const int n = __popcll(mask), order = nth_lane(mask);
    const float scale = i >= 0 && a.scales ? a.scales[i] : 1.0f;
    const uint8_t* b = a.b + (i >= 0 ? i * a.b_step : 0) + (int64_t)first * a.rank * 2;
    for (int c0 = 0; c0 < n; c0 += 16 * NT) {
      int tok[NT];
      u32x4 h[NT][STEPS];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        tok[u] = block * kLoraBlock + __shfl(order, min(c0 + 16 * u + r, n - 1), 64);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          // places 0 .. octets - 1: h rounded, then what that left out
          const int place = 4 * s + g, octet = place < octets ? place : place - octets;
          h[u][s] = u32x4{0u, 0u, 0u, 0u};
          if (i >= 0 && octet < octets) {
            f32x4 x[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
            const float* p = a.part + (int64_t)tok[u] * rows + slice * a.rank + octet * 8;
            for (int c = 0; c < a.chunks; ++c, p += (int64_t)a.tokens * rows) {
              x[0] += *reinterpret_cast<const f32x4*>(p);
              x[1] += *reinterpret_cast<const f32x4*>(p + 4);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float e = x[k / 2][k % 2 * 2] * scale, f = x[k / 2][k % 2 * 2 + 1] * scale;
              const uint32_t w = bf16_pair(e, f);
              h[u][s][k] = place < octets ? w : bf16_pair(e - __uint_as_float(w << 16), f - __uint_as_float(w & 0xffff0000u));
            }
          }
        }
      }
      for (int t = n0; t < n1; t += 64) {
        // product j's row m is column (m / 4) 16 + 4 j + m % 4 of the tile: a lane ends with 16 columns of its token
        f32x4 o[NT][4];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[u][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (i >= 0) {
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const int place = 4 * s + g, octet = place < octets ? place : place - octets;
            if (4 * s >= 2 * octets) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int col = min(t + r / 4 * 16 + 4 * j + r % 4, width - 1);
              const u32x4 w = octet < octets ? *reinterpret_cast<const u32x4*>(b + (int64_t)col * a.rank * 2 + octet * 16)
                                             : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
              for (int u = 0; u < NT; ++u) o[u][j] = mma_bf16(w, h[u][s], o[u][j]);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          if (c0 + 16 * u + r >= n) continue;
          const int64_t at = (int64_t)(first + t + 16 * g) * 2;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (t + 16 * g + 8 * half >= n1) continue;
            u32x4 v = *reinterpret_cast<const u32x4*>(a.y + tok[u] * a.y_row + at + half * 16);
            if (i >= 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const f32x4& d = o[u][2 * half + k / 2];
                v[k] = bf16_pair(__uint_as_float(v[k] << 16) + d[k % 2 * 2], __uint_as_float(v[k] & 0xffff0000u) + d[k % 2 * 2 + 1]);
              }
            }
            *reinterpret_cast<u32x4*>(a.out + tok[u] * a.out_row + at + half * 16) = v;
          }
        }
      }
    }
  });
}

template <int NT>
static hipError_t launch_up(const LoraArgs& a, int blocks, hipStream_t s) {
  const unsigned grid = (unsigned)((blocks * a.up_slots * a.ranges + kLoraWaves - 1) / kLoraWaves);
  const dim3 threads(kLoraWaves * 64);
  if (a.rank <= 16)
    hipLaunchKernelGGL((lora_up_kernel<NT, 1>), dim3(grid), threads, 0, s, a);
  else if (a.rank <= 32)
    hipLaunchKernelGGL((lora_up_kernel<NT, 2>), dim3(grid), threads, 0, s, a);
  else if (a.rank <= 64)
    hipLaunchKernelGGL((lora_up_kernel<NT, 4>), dim3(grid), threads, 0, s, a);
  else
    hipLaunchKernelGGL((lora_up_kernel<(NT > 2 ? 2 : NT), 8>), dim3(grid), threads, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int blocks = (a.tokens + kLoraBlock - 1) / kLoraBlock, rows = a.slices * a.rank;
  const bool wide = a.tokens > kLoraBlock;
  const int groups = wide ? (rows + 63) / 64 : (rows + 15) / 16;
  const unsigned grid = (unsigned)((blocks * a.down_slots * groups * a.chunks + kLoraWaves - 1) / kLoraWaves);
  if (wide)
    hipLaunchKernelGGL((lora_down_kernel<4, 4>), dim3(grid), dim3(kLoraWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL((lora_down_kernel<1, 1>), dim3(grid), dim3(kLoraWaves * 64), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return wide ? launch_up<4>(a, blocks, s) : launch_up<1>(a, blocks, s);
}

}  // namespace qlk
