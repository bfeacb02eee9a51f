// How the keys of a batch of trees are cut into shares: the arithmetic alone, for
// a wave of the GPU (see tree_cut) and for its check on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlk {

// Trees: the units' keys are cut by the lengths found, into equal shares of a
// unit that are as many as the card takes at once (or for more units than that, a
// multiple).  A host's bound of the lengths would leave the card idle behind the
// longest ones (16 sequences of 515 .. 4,099 keys, 32 nodes of 32 / 8 heads: 54 us so
// cut, 46 by the lengths found).
struct TreeCut {
  float per_key;   // shares a key
  bool rounds;     // more of them than the card takes at once
};

// Shares of a unit.  (Rounding of the product only moves a border between counts.)
__host__ __device__ __forceinline__ int tree_shares(int len, const TreeCut& cut) {
  const int n = (int)ceilf((float)len * cut.per_key);
  return n > 1 ? n : 1;
}

// Workgroups that `units` units of all KV heads are cut for at most: units / slots +
// 1/4, rounded up, times the slots.
__host__ __device__ __forceinline__ int64_t tree_most(int64_t units, int slots) {
  return (4 * units + 5 * (int64_t)slots - 1) / (4 * (int64_t)slots) * slots;
}

// Cuts a batch.  each(f) calls f(blocks of rows, length) for its sequences, a
// lane's at a time, total(x) adds x over the lanes.  Chunks are the shortest
// whose shares fit in tree_most: with chunks of c 64-key tiles a KV head has at most
// tiles / c + units of them, so c = tiles / (most - units) is enough, and the
// search is between that and tiles / most.  Blocks times tiles take more than 32
// bits at long contexts: they are added in halves of 24 bits, then as binary32
// (within 2^-18 of their sum; a thousandth more has room for that and for the products' rounding).
template <class Each, class Total>
__host__ __device__ __forceinline__ TreeCut tree_cut_of(Each each, Total total, int kv_heads, int max_kv, int slots) {
  int64_t units = 0;    // of one KV head
  float tiles = 0.0f;   // and theirs
  each([&](int blocks, int len) {
    const int64_t n = (int64_t)blocks * ((len + 63) >> 6);
    units += total(blocks);
    tiles += (float)total((int)(n >> 24)) * 16777216.0f + (float)total((int)(n & 0xffffff));
  });
  const int64_t all = tree_most(units * kv_heads, slots);
  const int most = (int)(all < 0x7fffffff ? all : 0x7fffffff) / kv_heads;   // (beyond 2^24: no batch of a plan's)
  // shares of one KV head
  auto count = [&](int c) {
    const TreeCut cut = {1.0f / (64.0f * (float)c), false};
    int64_t n = 0;
    each([&](int blocks, int len) { n += total(blocks * tree_shares(len, cut)); });
    return n;
  };
  const int longest = (max_kv + 63) / 64;   // a share a unit
  int lo = (int)fminf(tiles / (float)most, (float)longest), hi = longest;
  if (most > units) hi = (int)fminf(tiles / (float)(most - (int)units) * 1.001f + 1.0f, (float)longest);
  lo = lo > 2 ? lo : 2;
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (count(mid) <= most)
      hi = mid;
    else
      lo = mid + 1;
  }
  return TreeCut{1.0f / (64.0f * (float)lo), (int64_t)most * kv_heads > slots};
}

// The first of the shares of block `block` of a sequence (before: shares before the
// sequence, of one KV head, as the tile kernel counted them); -1: not cut, or not
// among the shares that were launched.  (Sequences that overlap, as no cu_q has
// them, may count more than 32 bits hold.)
__host__ __device__ __forceinline__ int tree_first_share(int before, int block, int shares, int kv_heads, int launched) {
  const int64_t first = before + (int64_t)block * shares;
  if (shares <= 1 || first < 0 || first + shares > launched / kv_heads) return -1;
  return (int)first;
}

}  // namespace qlk
