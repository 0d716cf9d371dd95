// dspark_window_attention: attention of the packed rows over the paged cache.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "packed_rows.cuh"
#include "pdl.h"

namespace dspark {
namespace {

struct AttnArgs {
  const __nv_bfloat16 *q, *k_cache, *v_cache;
  int64_t q_stride;
  const int32_t *page_table, *cu, *ctx;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  float scale;
  int max_pages, n_pages, page_shift, bs, rows, Hq, Hkv, window, n_sink;
};

constexpr int kAttnWarps = 4;

// One warp per (row, query head); lane l holds lanes l, l + 32, .. of the head.  The plain form of
// one pass with the running maximum and sum.
template <int D>
__global__ void __launch_bounds__(32 * kAttnWarps) attention_kernel(AttnArgs a) {
  constexpr int E = D / 32;
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x, h = blockIdx.y * kAttnWarps + (threadIdx.x >> 5);
  if (h >= a.Hq) return;
  const int r = warp_request_of(a.cu, a.bs, a.rows, row, lane);
  if (r >= a.bs) return;
  const int c = r < 0 ? -1 : a.ctx[r], first = r < 0 ? 0 : a.cu[r], n = r < 0 ? 0 : a.cu[r + 1] - first;
  const int i = row - first;
  if (c < 0 || int64_t(c) + n > int64_t(a.max_pages) << a.page_shift) {
    if (lane == 0) set_status(a.status, DSPARK_EINVAL);
    return;
  }
  const int p = c + i, hk = h / (a.Hq / a.Hkv);
  const int lo = a.window ? max(0, p - a.window + 1) : 0, sinks = min(lo, a.window ? a.n_sink : 0);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[row * a.q_stride + h * D + e * 32 + lane]) * a.scale;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < sinks + p + 1 - lo; ++t) {
    const int j = t < sinks ? t : lo + t - sinks;
    const int page = a.page_table[int64_t(r) * a.max_pages + (j >> a.page_shift)];
    const bool good = page >= 0 && page < a.n_pages;
    if (!good && lane == 0) set_status(a.status, DSPARK_EINVAL);
    const int64_t at = (((int64_t(page) * a.Hkv + hk) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += good ? q[e] * __bfloat162float(a.k_cache[at + e * 32 + lane]) : 0.f;
    s = warp_sum(s);
    s = __shfl_sync(~0u, s, 0);
    const float mn = fmaxf(m, s), al = expf(m - mn), w = expf(s - mn);
    l = l * al + w;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * al + (good ? w * __bfloat162float(a.v_cache[at + e * 32 + lane]) : 0.f);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[(int64_t(row) * a.Hq + h) * D + e * 32 + lane] = __float2bfloat16(o[e] / l);
  if (a.lse && lane == 0) a.lse[int64_t(row) * a.Hq + h] = m + logf(l);
}

}  // namespace

size_t window_attention_ws_bytes(int Hq, int Hkv, int D) { return 256; }

cudaError_t launch_window_attention(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                    const int32_t* page_table, int max_pages, int n_pages, int page_shift,
                                    const int32_t* cu, const int32_t* ctx, int bs, int rows, int max_rows, int Hq,
                                    int Hkv, int D, float scale, int window, int n_sink, void* out, float* lse,
                                    void* ws, cudaStream_t s) {
  AttnArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q), a.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<const __nv_bfloat16*>(v_cache), a.q_stride = q_stride;
  a.page_table = page_table, a.cu = cu, a.ctx = ctx, a.out = static_cast<__nv_bfloat16*>(out), a.lse = lse;
  a.status = static_cast<uint32_t*>(ws), a.scale = scale;
  a.max_pages = max_pages, a.n_pages = n_pages, a.page_shift = page_shift, a.bs = bs, a.rows = rows, a.Hq = Hq;
  a.Hkv = Hkv, a.window = window, a.n_sink = n_sink;
  const dim3 grid(rows, (Hq + kAttnWarps - 1) / kAttnWarps), block(32 * kAttnWarps);
  return D == 64 ? launch_pdl(attention_kernel<64>, grid, block, 0, s, a)
                 : launch_pdl(attention_kernel<128>, grid, block, 0, s, a);
}

}  // namespace dspark
