// Host harness: which split records the merges follow, by the library's own
// header, for a test that checks them against unbounded integers.  Input lines:
// "x y z bound stride"; output lines: is_split(bound) has_pieces(stride, bound).
#include <cstdio>

#include "splits.cuh"

int main() {
  int x, y, z, bound, stride;
  while (std::scanf("%d %d %d %d %d", &x, &y, &z, &bound, &stride) == 5) {
    const int4 info = make_int4(x, y, z, 0);
    std::printf("%d %d\n", mla::is_split(info, bound) ? 1 : 0, mla::has_pieces(info, stride, bound) ? 1 : 0);
  }
  return 0;
}
