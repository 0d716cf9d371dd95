// The packed batch as the target model's kernels see it: which request a packed row belongs to,
// and the paged cache's addressing.
#pragma once

#include <stdint.h>

namespace dspark {

// The request that owns packed row `row`: the count of window ends cu[1 .. bs] that are <= row (bs
// if no request owns it), or -1 when cu is no list of windows of `rows` rows (it decreases, starts
// below 0 or ends beyond rows).  A whole warp calls it; all lanes get the answer.
__device__ __forceinline__ int warp_request_of(const int32_t* __restrict__ cu, int bs, int rows, int row, int lane) {
  int r = 0;
  bool bad = false;
  for (int i = lane; i - lane < bs; i += 32) {
    const int a = i < bs ? cu[i] : 0, b = i < bs ? cu[i + 1] : rows;
    bad |= a < 0 || b < a || b > rows;
    r += __popc(__ballot_sync(~0u, i < bs && b <= row));
  }
  return __any_sync(~0u, bad) ? -1 : r;
}

}  // namespace dspark
