// The keys of a request that a sliding-window decode reads, and their cutting
// into runs (plain C++: the host tests compile it as it is).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SGL_HD __host__ __device__ __forceinline__
#else
#define SGL_HD inline
#endif

namespace sgl {
namespace dec {

// The query of a request of len keys is at position len - 1 and sees positions
// [0, sinks) and [len - window, len); those below max_seq are read.  In order
// they are its visible keys 0 .. n - 1, cut into at most n_splits near-equal
// runs; run s of request r is item r * n_splits + s.
struct Window {
  int32_t sinks, window;
  int32_t max_seq;   // positions from it on are left out (lengths above the host's)
  int32_t n_splits;  // runs of at most Params::chunk visible keys
};

struct WindowRun {
  int32_t first, lo;  // visible: [0, first) and from lo on
  int32_t n;          // visible keys (none of a padding row, of length 0 or less)
  int32_t ns;         // runs

  // The window counts from the true length, also where that passes max_seq: a
  // window counted from the cut one would reach positions that the query does
  // not see, whose entries of req_to_token may hold anything.
  SGL_HD WindowRun(const Window& w, int32_t chunk, int32_t seq_len) {
    const int32_t len = seq_len > 0 ? seq_len : 0;
    const int32_t end = len < w.max_seq ? len : w.max_seq;
    lo = len > w.window ? len - w.window : 0;
    const int32_t before = lo < end ? lo : end;
    first = w.sinks < before ? w.sinks : before;
    n = first + (end > lo ? end - lo : 0);
    ns = n > 0 ? 1 + (n - 1) / chunk : 0;
  }
  SGL_HD int32_t pos(int32_t i) const { return i < first ? i : lo + (i - first); }
};

}  // namespace dec
}  // namespace sgl
