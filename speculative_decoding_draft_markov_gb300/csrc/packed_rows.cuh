// The packed batch as the target model's kernels see it: which request a packed row belongs to.
#pragma once

#include <stdint.h>

namespace dspark {

// What entry i of a list of windows cu[0 .. bs] (i < bs; i >= bs: nothing) says about packed row `row`: whether its
// window ends before the row, whether the row lies before all windows, and whether the list is none of windows of `rows`
// rows there (it decreases, starts below 0 or ends beyond rows).
struct WindowEnd {
  bool passed, before_all, bad;
};
__host__ __device__ __forceinline__ WindowEnd window_end(const int32_t* __restrict__ cu, int bs, int rows, int row, int i) {
  if (i >= bs) return {false, false, false};
  const int a = cu[i], b = cu[i + 1];
  return {b <= row, i == 0 && row < a, a < 0 || b < a || b > rows};
}

// The request that owns packed row `row`: the count of window ends cu[1 .. bs] that are <= row; bs if no request owns
// it (the row lies before cu[0] or from cu[bs] on), -1 when cu is no list of windows of `rows` rows.  A whole warp
// calls it; all lanes get the answer.
__device__ __forceinline__ int warp_request_of(const int32_t* __restrict__ cu, int bs, int rows, int row, int lane) {
  int r = 0;
  bool bad = false, before_all = false;
  for (int i = lane; i - lane < bs; i += 32) {
    const WindowEnd e = window_end(cu, bs, rows, row, i);
    bad |= e.bad, before_all |= e.before_all;
    r += __popc(__ballot_sync(~0u, e.passed));
  }
  if (__any_sync(~0u, bad)) return -1;
  return __any_sync(~0u, before_all) ? bs : r;
}

}  // namespace dspark
