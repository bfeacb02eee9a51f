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
//
// Measured on MI355X (copy 5.2 TB/s, a launch 4.4 us back to back):
//   8 tokens of as many adapters, R 16, K 4096, widths 4096 + 1024 + 1024: 9 us, both
//     launches at their floor (4.7 + 4.9);
//   64 tokens of 24 adapters, R 32, K 5120, widths 17408 twice, 79 MB: 20.4 us (5.9 + 14),
//     3.9 TB/s over both launches, 4.5 in the second;
//   4,093 tokens of 8 adapters, R 16, widths 4096 + 1024 + 1024, 138 MB: 57 us (17.5 + 38).
//     The second launch reads y and writes out (100 MB) at 2.7 TB/s: without the reads it
//     is 17 us shorter, without the writes 16; deeper prefetch, other orders
//     of the columns and non-temporal accesses gave nothing (accesses through LDS, of
//     whole runs of a row for 64 bytes of 16 rows, have not been tried).
#include "attention_common.hpp"
#include "serving_args.hpp"

namespace qlk {

constexpr int kLoraWaves = 4;
constexpr float kMostBf16 = 0x1.fep127f;

// The adapter of this lane's token of block `block`, -1 without one; lanes
// beyond the tokens are not in `there`.
__device__ __forceinline__ int lane_adapter(const LoraArgs& a, int block, uint64_t* there) {
  const int t = block * kLoraBlock + (threadIdx.x & 63);
  const bool in = t < a.tokens;
  const int i = in ? a.adapter[t] : -1;
  *there = __ballot(in);
  return i >= 0 && i < a.adapters ? i : -1;
}

// Calls f(adapter, mask of its tokens, first of its tile) for the tiles number
// slot, slot + slots, ... of the lanes of `left`: up to `size` tokens of one adapter.
template <class F>
__device__ __forceinline__ void for_tiles(int mine, uint64_t left, int size, int slot, int slots, F f) {
  for (int n = 0; left;) {
    const int i = lane_i32(mine, __ffsll((unsigned long long)left) - 1);
    const uint64_t same = __ballot(mine == i) & left;
    left &= ~same;
    const int end = n + (__popcll(same) + size - 1) / size;
    for (; slot < end; slot += slots) f(i, same, (slot - n) * size);
    n = end;
  }
}

// Lane c gets the c-th lane of `mask` (those after them: the other lanes).
__device__ __forceinline__ int nth_lane(uint64_t mask) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int at = mask >> lane & 1 ? __popcll(mask & below) : __popcll(mask) + __popcll(~mask & below);
  return __builtin_amdgcn_ds_permute(at * 4, lane);
}

// h of tiles of 16 NT tokens, one chunk of K, TW tiles of 16 ranks: four waves a
// quarter of the chunk each.
template <int NT, int TW>
__global__ void __launch_bounds__(kLoraWaves * 64) lora_down_kernel(LoraArgs a) {
  __shared__ f32x4 sums[kLoraWaves][NT * TW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int rows = a.slices * a.rank, groups = (rows + 63) / 64;
  int id = blockIdx.x;
  const int chunk = id % a.chunks;
  id /= a.chunks;
  const int row0 = id % groups * 64;
  id /= groups;
  const int slot = id % a.down_slots, block = id / a.down_slots;
  uint64_t there;
  const int mine = lane_adapter(a, block, &there);
  const int k0 = chunk * a.chunk + wave * (a.chunk / kLoraWaves), k1 = min(a.k, k0 + a.chunk / kLoraWaves);
  for_tiles(mine, there, 16 * NT, slot, a.down_slots, [&](int i, uint64_t mask, int c0) {
    if (i < 0) return;
    const int n = __popcll(mask), order = nth_lane(mask);
    int tok[NT];
    const uint8_t *wp[TW], *xp[NT];
#pragma unroll
    for (int v = 0; v < TW; ++v)
      wp[v] = a.a + i * a.a_step + (int64_t)min(row0 + 16 * v + r, rows - 1) * a.k * 2 + g * 32;
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
        u32x4 x[NT];
#pragma unroll
        for (int u = 0; u < NT; ++u) x[u] = in ? *reinterpret_cast<const u32x4*>(xp[u] + (int64_t)k * 2 + half * 16) : zero;
#pragma unroll
        for (int v = 0; v < TW; ++v) {
          const u32x4 w = in ? *reinterpret_cast<const u32x4*>(wp[v] + (int64_t)k * 2 + half * 16) : zero;
#pragma unroll
          for (int u = 0; u < NT; ++u) h[u][v] = mma_bf16(w, x[u], h[u][v]);
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
      for (int v = 0; v < TW; ++v) sums[wave][u * TW + v][lane] = h[u][v];
    __syncthreads();
    // one wave's place of the product for each tile of tokens and ranks
    for (int p = wave; p < NT * TW; p += kLoraWaves) {
      f32x4 x = sums[0][p][lane];
#pragma unroll
      for (int w = 1; w < kLoraWaves; ++w) x += sums[w][p][lane];
      const int u = p / TW, row = row0 + 16 * (p % TW) + 4 * g;
      int t = tok[0];
#pragma unroll
      for (int k = 1; k < NT; ++k) t = u == k ? tok[k] : t;
      if (c0 + 16 * u + r < n && row < rows)
        *reinterpret_cast<f32x4*>(a.part + ((int64_t)chunk * a.tokens + t) * rows + row) = x;
    }
    __syncthreads();
  });
}

// The column of a 64-wide tile that row m of product j stands for: a lane ends
// with 8 columns of its token from 8 g on and 8 from 32 + 8 g on, so a load or
// store of 16 bytes a lane covers 64 in a row.
__device__ __forceinline__ int tile_column(int j, int m) { return j / 2 * 32 + m / 4 * 8 + j % 2 * 4 + m % 4; }

// out = y + s B h for tiles of 16 tokens and a range of column tiles of one slice.
// BS products of 32 ranks for h rounded and as many for what that left out; ranks
// of up to 16 have both in one (PACKED).
template <int BS, bool PACKED>
__global__ void __launch_bounds__(kLoraWaves * 64, BS == 1 ? 4 : BS == 2 ? 3 : 2) lora_up_kernel(LoraArgs a) {
  constexpr int HS = PACKED ? 1 : 2 * BS, PS = PACKED ? 1 : BS;
  __shared__ u32x4 h_lds[HS][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  int id = blockIdx.x;
  int range = id % a.ranges, slice = 0, first = 0;
  id /= a.ranges;
  const int slot = id % a.up_slots, block = id / a.up_slots;
  // the slice, and its first column
  const int wide = a.tiles_wg * 64;
  for (;; ++slice) {
    const int here = (a.width[slice] + wide - 1) / wide;
    if (range < here) break;
    range -= here;
    first += a.width[slice];
  }
  const int width = a.width[slice], rows = a.slices * a.rank, octets = a.rank / 8;
  const int n0 = range * wide + wave * 64, n1 = min(width, range * wide + wide);
  uint64_t there;
  const int mine = lane_adapter(a, block, &there);
  for_tiles(mine, there, 16, slot, a.up_slots, [&](int i, uint64_t mask, int c0) {
    if (i < 0 && a.out == a.y) return;
    const int n = __popcll(mask), order = nth_lane(mask);
    const int tok = block * kLoraBlock + __shfl(order, min(c0 + r, n - 1), 64);
    const bool live = c0 + r < n;
    const uint8_t* b = a.b + (i >= 0 ? i * a.b_step : 0) + (int64_t)first * a.rank * 2;
    const uint8_t* y = a.y + tok * a.y_row + (int64_t)(first + 8 * g) * 2;
    uint8_t* out = a.out + tok * a.out_row + (int64_t)(first + 8 * g) * 2;
    u32x4 w[4][BS], v[2];
    auto load = [&](int t) {
#pragma unroll
      for (int half = 0; half < 2; ++half)
        if (live && t + 32 * half + 8 * g < n1) v[half] = *reinterpret_cast<const u32x4*>(y + (t + 32 * half) * 2);
      if (i >= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (an adapter of a slice is shorter than 2^31 bytes)
          const uint32_t at = (uint32_t)(min(t + tile_column(j, r), width - 1) * a.rank * 2);
#pragma unroll
          for (int s = 0; s < BS; ++s) {
            const int octet = PACKED ? (g < octets ? g : g - octets) : 4 * s + g;
            w[j][s] = octet < octets ? *reinterpret_cast<const u32x4*>(b + (at + octet * 16)) : u32x4{0u, 0u, 0u, 0u};
          }
        }
      }
    };
    if (n0 < n1) load(n0);
    if (i >= 0) {
      // h of the tile's tokens, in the order of the products' operands
      const float scale = a.scales ? a.scales[i] : 1.0f;
      for (int s = wave; s < PS; s += kLoraWaves) {
        const int place = 4 * s + g, octet = PACKED && place >= octets ? place - octets : place;
        u32x4 hi = {0u, 0u, 0u, 0u}, lo = {0u, 0u, 0u, 0u};
        if (octet < octets) {
          f32x4 x[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
          const float* p = a.part + (int64_t)tok * rows + slice * a.rank + octet * 8;
          const int64_t step = (int64_t)a.tokens * rows;
          int c = 0;
          for (; c + 4 <= a.chunks; c += 4, p += 4 * step) {
            f32x4 e[4], f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              e[k] = *reinterpret_cast<const f32x4*>(p + k * step);
              f[k] = *reinterpret_cast<const f32x4*>(p + k * step + 4);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[0] += e[k];
              x[1] += f[k];
            }
          }
          for (; c < a.chunks; ++c, p += step) {
            x[0] += *reinterpret_cast<const f32x4*>(p);
            x[1] += *reinterpret_cast<const f32x4*>(p + 4);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float e = x[k / 2][k % 2 * 2] * scale, f = x[k / 2][k % 2 * 2 + 1] * scale;
            // (no larger than bf16 holds: what is beyond, infinities and NaN are left to the second number)
            hi[k] = bf16_pair(fminf(fmaxf(e, -kMostBf16), kMostBf16), fminf(fmaxf(f, -kMostBf16), kMostBf16));
            lo[k] = bf16_pair(e - __uint_as_float(hi[k] << 16), f - __uint_as_float(hi[k] & 0xffff0000u));
          }
        }
        if (PACKED) {
          h_lds[0][lane] = place < octets ? hi : lo;
        } else {
          h_lds[s][lane] = hi;
          h_lds[BS + s][lane] = lo;
        }
      }
      lds_barrier();
    }
    for (int t = n0; t < n1; t += 64 * kLoraWaves) {
      f32x4 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (i >= 0) {
#pragma unroll
        for (int s = 0; s < HS; ++s) {
          const u32x4 h = h_lds[s][lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = mma_bf16(w[j][s % BS], h, o[j]);
        }
      }
      const u32x4 now[2] = {v[0], v[1]};
      if (t + 64 * kLoraWaves < n1) load(t + 64 * kLoraWaves);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!live || t + 32 * half + 8 * g >= n1) continue;
        u32x4 x = now[half];
        if (i >= 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const f32x4& d = o[2 * half + k / 2];
            x[k] = bf16_pair(__uint_as_float(x[k] << 16) + d[k % 2 * 2],
                             __uint_as_float(x[k] & 0xffff0000u) + d[k % 2 * 2 + 1]);
          }
        }
        *reinterpret_cast<u32x4*>(out + (t + 32 * half) * 2) = x;
      }
    }
    lds_barrier();
  });
}

template <int NT>
static void launch_down(const LoraArgs& a, int blocks, hipStream_t s) {
  const int rows = a.slices * a.rank, groups = (rows + 63) / 64, tiles = rows >= 64 ? 4 : (rows + 15) / 16;
  const dim3 grid((unsigned)(blocks * a.down_slots * groups * a.chunks)), threads(kLoraWaves * 64);
  if (tiles == 1)
    hipLaunchKernelGGL((lora_down_kernel<NT, 1>), grid, threads, 0, s, a);
  else if (tiles == 2)
    hipLaunchKernelGGL((lora_down_kernel<NT, 2>), grid, threads, 0, s, a);
  else if (tiles == 3)
    hipLaunchKernelGGL((lora_down_kernel<NT, 3>), grid, threads, 0, s, a);
  else
    hipLaunchKernelGGL((lora_down_kernel<NT, 4>), grid, threads, 0, s, a);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int blocks = (a.tokens + kLoraBlock - 1) / kLoraBlock;
  if (a.wide)
    launch_down<2>(a, blocks, s);
  else
    launch_down<1>(a, blocks, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)(blocks * a.up_slots * a.ranges)), threads(kLoraWaves * 64);
  if (a.rank <= 16)
    hipLaunchKernelGGL((lora_up_kernel<1, true>), grid, threads, 0, s, a);
  else if (a.rank <= 32)
    hipLaunchKernelGGL((lora_up_kernel<1, false>), grid, threads, 0, s, a);
  else if (a.rank <= 64)
    hipLaunchKernelGGL((lora_up_kernel<2, false>), grid, threads, 0, s, a);
  else if (a.rank <= 96)
    hipLaunchKernelGGL((lora_up_kernel<3, false>), grid, threads, 0, s, a);
  else
    hipLaunchKernelGGL((lora_up_kernel<4, false>), grid, threads, 0, s, a);
  return hipGetLastError();
}

}  // namespace qlk
