// Prints the positions that a sliding-window decode reads, run by run
// (csrc/window_run.h).  Input lines: sinks window max_seq n_splits chunk seq_len.
#include <cstdio>

#include "window_run.h"

int main() {
  sgl::dec::Window w;
  int chunk, len;
  while (std::scanf("%d %d %d %d %d %d", &w.sinks, &w.window, &w.max_seq, &w.n_splits, &chunk, &len) == 6) {
    const sgl::dec::WindowRun r(w, chunk, len);
    std::printf("%d %d", r.n, r.ns);
    // the ends, and all of it where it is short
    for (int i = 0; i < r.n; ++i)
      if (r.n <= 400 || i < 200 || i >= r.n - 200) std::printf(" %d", r.pos(i));
    std::printf("\n");
  }
  return 0;
}
