// Commit of the branch of a drafted tree that the drawn tokens agree with.
//
// From the root (node 0, the newest token) the walk goes to the first child
// whose token is the one drawn at the node, as long as there is one.  The keys
// and values of the d-th node reached move from its place among the nodes to
// the d-th place behind the root, so that the sequence's cache is without gaps.
//
// A few kilobytes a sequence and layer: bound by latency.  One launch for all
// layers: every workgroup walks its sequence's tree itself, nodes in lanes (a
// step is a comparison and a ballot), then moves its layer's rows.  The d-th
// node's number is at least d, and rises along the branch, so rows moved in
// their order never overwrite one that is still to be moved; a thread moves
// the same 16 bytes of every row, so that order needs no barrier.
//
// Measured on MI355X: 4 sequences of 13 nodes 4.5 us, 64 of 64 nodes (4.4 MB moved)
// 5.8 us; a launch alone takes 4.4.
#include "attention_args.hpp"
#include "device_common.hpp"

namespace qlk {

constexpr int kCommitThreads = 256;

// The first child of `node` with token `draw`, -1 without one.  Lanes hold the
// first 64 nodes' parents and tokens.
__device__ __forceinline__ int child_of(const CommitArgs& a, int64_t first, int n, int node, int draw, int parent, int token) {
  const int lane = threadIdx.x & 63;
  uint64_t hit = __ballot(lane > node && lane < n && parent == node && token == draw);
  if (hit) return __ffsll((unsigned long long)hit) - 1;
  for (int i0 = 64; i0 < n; i0 += 64) {
    const int i = i0 + lane;
    hit = __ballot(i > node && i < n && a.parents[first + i] == node && a.node_tokens[first + i] == draw);
    if (hit) return i0 + __ffsll((unsigned long long)hit) - 1;
  }
  return -1;
}

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(CommitArgs a) {
  __shared__ int path[kCommitDepth], from[kCommitDepth], to[kCommitDepth];   // nodes; places as page * page_size + place
  const int b = blockIdx.x, lane = threadIdx.x & 63;
  const int first = min(max(a.cu_q[b], 0), a.tokens), end = min(max(a.cu_q[b + 1], first), a.tokens), n = end - first;
  const int len = min(max(a.seq_lens[b], 0), a.max_kv);
  const bool tells = blockIdx.y == 0 && a.out_tokens;
  // every wave walks
  int parent = -1, token = 0, draws = 0;
  if (lane < n) {
    parent = a.parents[first + lane];
    token = a.node_tokens[first + lane];
    draws = a.sampled[first + lane];
  }
  int node = 0, depth = 0;
  while (n > 0) {
    const int draw = node < 64 ? __builtin_amdgcn_readlane(draws, node) : a.sampled[first + node];
    if (tells && threadIdx.x == 0) a.out_tokens[(int64_t)b * (a.max_depth + 1) + depth] = draw;
    const int next = depth < a.max_depth ? child_of(a, first, n, node, draw, parent, token) : -1;
    if (next < 0) break;
    node = __builtin_amdgcn_readfirstlane(next);
    if (threadIdx.x == 0) path[depth] = node;
    ++depth;
  }
  if (tells) {
    for (int i = (n > 0 ? depth + 1 : 0) + (int)threadIdx.x; i <= a.max_depth; i += kCommitThreads)
      a.out_tokens[(int64_t)b * (a.max_depth + 1) + i] = -1;
    if (threadIdx.x == 0) {
      a.accepted[b] = depth;
      if (a.new_lens) a.new_lens[b] = n > 0 ? len - n + 1 + depth : len;
    }
  }
  if ((int)blockIdx.y >= a.layers) return;
  __syncthreads();
  for (int d = threadIdx.x; d < depth; d += kCommitThreads) {
    // -1: stays where it is, or lies outside the context
    const int src = len - n + path[d], dst = len - n + d + 1;
    from[d] = -1;
    if (src != dst && dst >= 0 && src < a.max_kv) {
      const int32_t* table = a.table + (int64_t)b * a.table_row;
      const int p = src / a.page_size, q = dst / a.page_size;
      const int64_t sp = table[p], dp = table[q];
      if (sp >= 0 && sp < a.num_pages && dp >= 0 && dp < a.num_pages) {
        from[d] = (int)(sp * a.page_size + src - p * a.page_size);
        to[d] = (int)(dp * a.page_size + dst - q * a.page_size);
      }
    }
  }
  __syncthreads();
  const CommitLayer& l = a.layer[blockIdx.y];
  const int head_pieces = l.head_bytes / 16, pieces = l.kv_heads * head_pieces;
  for (int i = threadIdx.x; i < 2 * pieces; i += kCommitThreads) {
    const bool v = i >= pieces;
    const int at = v ? i - pieces : i;
    const Pages& c = v ? l.v : l.k;
    uint8_t* p = c.p + (int64_t)(at / head_pieces) * c.head + at % head_pieces * 16;
    auto place = [&](int slot) {
      const int page = slot / a.page_size;
      return reinterpret_cast<u32x4*>(p + page * c.page + (int64_t)(slot - page * a.page_size) * c.token);
    };
    for (int d0 = 0; d0 < depth; d0 += 4) {
      u32x4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (d0 + k < depth && from[d0 + k] >= 0) x[k] = *place(from[d0 + k]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (d0 + k < depth && from[d0 + k] >= 0) *place(to[d0 + k]) = x[k];
    }
  }
}

hipError_t launch_tree_commit(const CommitArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.batch, (unsigned)(a.layers > 1 ? a.layers : 1));
  hipLaunchKernelGGL(tree_commit_kernel, grid, dim3(kCommitThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace qlk
