// Which request owns a packed row, run on the host.  Built by tests/test_packed_rows.py as a shared library.
#include <cuda_runtime.h>

#include "packed_rows.cuh"

// As the warp does it: the request, bs for none, -1 for a list that is none.
extern "C" __attribute__((visibility("default"))) int request_of(const int* cu, int bs, int rows, int row) {
  int r = 0;
  bool bad = false, before_all = false;
  for (int i = 0; i < (bs + 31) / 32 * 32; ++i) {
    const dspark::WindowEnd e = dspark::window_end(cu, bs, rows, row, i);
    r += e.passed, bad |= e.bad, before_all |= e.before_all;
  }
  return bad ? -1 : before_all ? bs : r;
}
