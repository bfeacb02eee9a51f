// Reads "before block shares kv_heads launched" from stdin and prints where a unit's
// first partial result lies, -1 where its shares are not among those launched.
#include <stdio.h>

#include "tree_cut.hpp"

int main(void) {
  int before, block, shares, heads, launched;
  while (scanf("%d %d %d %d %d", &before, &block, &shares, &heads, &launched) == 5)
    printf("%d\n", qlk::tree_first_share(before, block, shares, heads, launched));
  return 0;
}
