// Reads "first step width rows" from stdin and walks csrc/row_walk.cuh to the end of the
// rows: prints how many places there were, the last one, and whether each was the one
// that 64-bit arithmetic gives.
#define __host__
#define __device__
#define __forceinline__ inline
#include <cstdio>

#include "row_walk.cuh"

int main() {
  int first, step, width, rows;
  while (std::scanf("%d %d %d %d", &first, &step, &width, &rows) == 4) {
    long long n = 0, place = first;
    bool same = true;
    int row = -1, at = -1;
    for (g3::RowWalk e(first, step, width); e.within(rows); e.next(), ++n, place += step) {
      same &= e.row == place / width && e.at == place % width;
      row = (int)e.row;
      at = e.at;
    }
    std::printf("%lld %d %d %d\n", n, row, at, (int)same);
  }
  return 0;
}
