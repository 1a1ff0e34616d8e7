// The key list of tree_rule.cuh on the host: reads "len depths nodes k pi S cap ring" lines and prints,
// for each, every (depth, position, kind, cache row) that the rule gives for the list's cache entries.
#include <cstdio>

#include "tree_rule.cuh"

int main() {
  int len, depths, nodes, ring;
  pia::TreeArgs a = {};
  while (scanf("%d %d %d %d %d %d %d %d", &len, &depths, &nodes, &a.kwin, &a.pi, &a.S, &a.cap, &ring) == 8) {
    a.ring = ring;
    pia::TreeList tl;
    tl.init(a, len, nodes, depths);
    for (int e = 0; e < tl.cached(); ++e) {
      const int rel = tl.rel_of(e), mod = tl.mod_of(rel);
      for (int x = 0; x < depths; ++x) {
        const int kind = pia::tree_kind(x, tl.mod_of(x), rel, mod, tl.kwin, tl.reach);
        if (kind) printf("%d,%lld,%d,%d ", x, (long long)len + rel, kind, tl.row_of(rel));
      }
    }
    printf("\n");
  }
  return 0;
}
