// Reads batches of trees from stdin and prints how their keys are cut:
//   kv_heads max_kv slots sequences, then blocks and length of each sequence;
// out: shares of all KV heads together, the longest share of a sequence in 64-key
// tiles, whether they come in rounds.
#include <math.h>
#include <stdio.h>

#include <vector>

#include "tree_cut.hpp"

int main(void) {
  int heads, max_kv, slots, n;
  while (scanf("%d %d %d %d", &heads, &max_kv, &slots, &n) == 4) {
    std::vector<int> blocks(n), lens(n);
    for (int i = 0; i < n; ++i)
      if (scanf("%d %d", &blocks[i], &lens[i]) != 2) return 1;
    auto each = [&](auto f) {
      for (int i = 0; i < n; ++i) f(blocks[i], lens[i]);
    };
    const qlk::TreeCut cut = qlk::tree_cut_of(each, [](int x) { return x; }, heads, max_kv, slots);
    long long shares = 0, longest = 0;
    for (int i = 0; i < n; ++i) {
      const long long each = qlk::tree_shares(lens[i], cut), tiles = (lens[i] + 63) / 64;
      shares += blocks[i] * each;
      if (blocks[i] && (tiles + each - 1) / each > longest) longest = (tiles + each - 1) / each;
    }
    printf("%lld %lld %d\n", shares * heads, longest, (int)cut.rounds);
  }
  return 0;
}
