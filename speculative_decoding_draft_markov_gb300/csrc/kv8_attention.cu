// dspark_window_attention_kv8: the packed rows' attention over an 8-bit paged cache.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "packed_rows.cuh"
#include "pdl.h"

namespace dspark {
namespace {

struct Kv8Args {
  const __nv_bfloat16* q;
  int64_t q_stride, cache_limit;
  const uint8_t *k_cache, *v_cache, *kv_scale;
  const int32_t *page_table, *cu, *ctx;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  float scale;
  int max_pages, n_pages, page_shift, bs, rows, Hq, Hkv, window, n_sink;
};

// One warp per (row, query head), a position at a time under a running maximum.
template <int D>
__global__ void __launch_bounds__(128) kv8_rows_kernel(const __grid_constant__ Kv8Args a) {
  constexpr int E = D / 32;
  pdl_enter();
  const int lane = threadIdx.x & 31, row = blockIdx.x, head = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int r = warp_request_of(a.cu, a.bs, a.rows, row, lane);
  if (r < 0) {
    if (lane == 0) set_status(a.status, DSPARK_EINVAL);
    return;
  }
  if (r >= a.bs || head >= a.Hq) return;
  const int c = a.ctx[r], n = a.cu[r + 1] - a.cu[r], p = c + row - a.cu[r];
  if (c < 0 || int64_t(c) + n > a.cache_limit) {
    if (lane == 0) set_status(a.status, DSPARK_EINVAL);
    return;
  }
  const int h = head / (a.Hq / a.Hkv);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[int64_t(row) * a.q_stride + head * D + lane * E + e]) * a.scale;
    o[e] = 0.f;
  }
  const int lo = a.window ? max(0, p - a.window + 1) : 0, sinks = a.window ? min(a.n_sink, lo) : 0;
  for (int j = 0; j <= p; ++j) {
    if (j == sinks) j = max(j, lo);
    const int page = a.page_table[int64_t(r) * a.max_pages + (j >> a.page_shift)];
    float k[E], v[E];
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) set_status(a.status, DSPARK_EINVAL);
#pragma unroll
      for (int e = 0; e < E; ++e) k[e] = v[e] = 0.f;
    } else {
      const int64_t slot = ((int64_t(page) * a.Hkv + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
      const float kf = kv8::factor(a.kv_scale[2 * slot]), vf = kv8::factor(a.kv_scale[2 * slot + 1]);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 kk = kv8::values(*reinterpret_cast<const uint16_t*>(a.k_cache + slot * D + lane * E + e));
        const float2 vv = kv8::values(*reinterpret_cast<const uint16_t*>(a.v_cache + slot * D + lane * E + e));
        k[e] = kk.x * kf, k[e + 1] = kk.y * kf, v[e] = vv.x * vf, v[e + 1] = vv.y * vf;
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = warp_sum(s);
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
    const float keep = expf(m - base), w = expf(s - base);
    m = top;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + (w == 0.f ? 0.f : w * v[e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = int64_t(row) * a.Hq + head;
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[at * D + lane * E + e] = __float2bfloat16(o[e] * inv);
  if (a.lse && lane == 0) a.lse[at] = m + logf(l);
}

}  // namespace

cudaError_t launch_window_attention_kv8(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                        const uint8_t* kv_scale, const int32_t* page_table, int max_pages, int n_pages,
                                        int page_shift, const int32_t* cu, const int32_t* ctx, int bs, int rows,
                                        int max_rows, int Hq, int Hkv, int D, float scale, int window, int n_sink,
                                        void* out, float* lse, void* k_scratch, void* v_scratch, void* ws,
                                        cudaStream_t s) {
  Kv8Args a;
  a.q = static_cast<const __nv_bfloat16*>(q), a.q_stride = q_stride;
  a.cache_limit = std::min(int64_t(max_pages) << page_shift, int64_t(1) << 30);
  a.k_cache = static_cast<const uint8_t*>(k_cache), a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.kv_scale = kv_scale, a.page_table = page_table, a.cu = cu, a.ctx = ctx;
  a.out = static_cast<__nv_bfloat16*>(out), a.lse = lse, a.status = static_cast<uint32_t*>(ws), a.scale = scale;
  a.max_pages = max_pages, a.n_pages = n_pages, a.page_shift = page_shift, a.bs = bs, a.rows = rows, a.Hq = Hq, a.Hkv = Hkv;
  a.window = window >= a.cache_limit ? 0 : window, a.n_sink = n_sink;
  const dim3 grid(rows, (Hq + 3) / 4);
  return D == 64 ? launch_pdl(kv8_rows_kernel<64>, grid, dim3(128), 0, s, a)
                 : launch_pdl(kv8_rows_kernel<128>, grid, dim3(128), 0, s, a);
}

}  // namespace dspark
