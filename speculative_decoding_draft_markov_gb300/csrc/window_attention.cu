// dspark_window_attention, host side and join: which kernel takes a call, and the kernel that joins the
// partial rows of units that a cut between CTAs runs through.
#include <algorithm>
#include <cmath>

#include "attention_common.cuh"

namespace dspark {
namespace {

using namespace attn;

// Joins the partial rows of the units that a cut between ranges runs through: block v takes the unit that
// range v began and did not finish, in the order of its KV tiles.  One warp per row:
//     out = sum_i 2^(lse_i - M) out_i / sum_i 2^(lse_i - M),   M = max_i lse_i
// A chain of trips to memory (the unit, its parts, the row), so the parts' loads are issued kTogether at a time with
// their log-sum-exps, under a running maximum: two with few registers, so that more rows are under way, or sixteen.
// GB300, prompts of 4000 rows each: 13 us of the call's 306 (40 MB of partial rows), and 6 for the launch; 64 windows 3 and 5
// of 83; one token 1 and 2 of 9.  Slower: blocks of 1024 threads that take a range's rows in turn (64 windows 88 us), and the warps of
// a block sharing a row's parts (20.2 us where one token has 40 of them, against 15.9).
template <int D, int kTogether>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ AttnArgs a, int unit_rows) {
  constexpr int E = D / 32;
  pdl_enter();
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5), c = blockIdx.x;
  const int4 info = a.info[c];
  const int n = info.x;  // part 0 is the unit's rows in range c, part i those in range c + i
  const int tok = (row / kTile) * a.tokens + (row % kTile) / a.g, hh = (row % kTile) % a.g;
  if (n == 0 || row % kTile >= a.tokens * a.g || tok >= info.z) return;
  float ref = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += kTogether) {
    float v[kTogether][E], lse[kTogether];
#pragma unroll
    for (int k = 0; k < kTogether; ++k) {
      lse[k] = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = 0.f;
      if (i0 + k >= n) continue;
      const int64_t at = int64_t(i0 + k == 0 ? 2 * c + 1 : 2 * (c + i0 + k)) * unit_rows + row;
      lse[k] = a.plse[at];
      if constexpr (E == 4)
        *reinterpret_cast<float4*>(v[k]) = *reinterpret_cast<const float4*>(a.partial + at * D + lane * E);
      else
        *reinterpret_cast<float2*>(v[k]) = *reinterpret_cast<const float2*>(a.partial + at * D + lane * E);
    }
    float top = ref;
#pragma unroll
    for (int k = 0; k < kTogether; ++k) top = fmaxf(top, lse[k]);
    const float base = top == -INFINITY ? 0.f : top, keep = exp2f(ref - base);
    ref = top;
    sum *= keep;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= keep;
#pragma unroll
    for (int k = 0; k < kTogether; ++k) {
      const float w = exp2f(lse[k] - base);  // 0: nothing seen there; NaN: no number seen there
      sum += w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = w == 0.f ? acc[e] : fmaf(w, v[k][e], acc[e]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t at = int64_t(info.y + tok) * a.Hq + info.w * a.g + hh;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(a.out + at * D + lane * E + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[at] = (ref + log2f(sum)) * kLn2;
}

// The cache is read in blocks of 32 slots, or of a smaller page: fewer that nobody sees at a window's ends than with
// blocks of up to 128 (page 128: 256 windows of 8 rows, window 1024, 187 us against 217; prompts with a window of 500
// 118 against 152, without 318 against 326).
constexpr int kMaxBlockShift = 5;

// Workspace: status block | what each range left | partial rows | their log-sum-exps.
struct AttnWs {
  size_t info, partial, plse, total;
};
AttnWs attn_ws(int D, int unit_rows, int n_ranges) {
  AttnWs w;
  w.info = 256;
  w.partial = w.info + align256(n_ranges * sizeof(int4));
  w.plse = w.partial + align256(size_t(2) * n_ranges * unit_rows * D * sizeof(float));
  w.total = w.plse + align256(size_t(2) * n_ranges * unit_rows * sizeof(float));
  return w;
}

// The cache as a 4-D tensor [page, head, slot, lane]; a box is one block's 64 columns.
bool encode_cache(CUtensorMap* map, const void* base, int n_pages, int Hkv, int page, int D, int block) {
  const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(page), cuuint64_t(Hkv), cuuint64_t(n_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(D) * 2, cuuint64_t(page) * D * 2, cuuint64_t(Hkv) * page * D * 2};
  const cuuint32_t box[4] = {64u, cuuint32_t(block), 1u, 1u}, es[4] = {1, 1, 1, 1};
  return tch::encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Q as [row, head, lane]; a box is 64 columns of the g heads of `tokens` rows: the tile's rows in order.
bool encode_q(CUtensorMap* map, const void* base, int rows, int Hq, int D, int64_t stride, int g, int tokens) {
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(Hq), cuuint64_t(rows)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(stride) * 2};
  const cuuint32_t box[3] = {64u, cuuint32_t(g), cuuint32_t(tokens)}, es[3] = {1, 1, 1};
  return tch::encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t window_attention_ws_bytes(int Hq, int Hkv, int D) {
  size_t most = attn_ws(D, 2 * kTile, tch::sm_count()).total;  // any tiling
  for (int rows = 16; rows <= attention_window_rows(D); rows *= 2)
    most = std::max(most, attn_ws(D, rows, attention_window_sets(D, rows) * tch::sm_count()).total);
  return most;
}

cudaError_t launch_window_attention(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                    const int32_t* page_table, int max_pages, int n_pages, int page_shift,
                                    const int32_t* cu, const int32_t* ctx, int bs, int rows, int max_rows, int Hq,
                                    int Hkv, int D, float scale, int window, int n_sink, void* out, float* lse,
                                    void* ws, cudaStream_t s) {
  AttnArgs a;
  const int n_cta = tch::sm_count(), g = Hq / Hkv, fit = kTile / g;
  // GB300, 64 requests over 3000 .. 5000 positions, 8 KV heads, D 128: 132 rows to a KV head, the prompts' kernel 192 us, the
  // windows' 319; 128 rows 182 and 181; 80 rows 175 and 172 (256 requests, window 256: 152 and 128).  D 64: 80 rows
  // 131 and 153 (window 256: 140 and 128); 64 rows 131 and 95.
  const bool prompts = max_rows > attention_window_rows(D) / g;
  // short windows: the narrowest tile that holds the expected rows.  256 requests, window 256, D 128, a row to a
  // request (4 to a KV head): R = 16 58 us, 32 59, 64 88, 128 123
  int unit_rows = 16;
  while (!prompts && unit_rows < max_rows * g) unit_rows *= 2;
  if (prompts) unit_rows = 2 * kTile;
  a.cache_limit = std::min(int64_t(max_pages) << page_shift, int64_t(1) << 30);  // positions: well inside 32 bits
  a.page_table = page_table, a.cu = cu, a.ctx = ctx, a.out = static_cast<__nv_bfloat16*>(out), a.lse = lse;
  char* w = static_cast<char*>(ws);
  const int n_ranges = n_cta * (prompts ? 1 : attention_window_sets(D, unit_rows));
  const AttnWs L = attn_ws(D, unit_rows, n_ranges);
  a.status = reinterpret_cast<uint32_t*>(w), a.diag = reinterpret_cast<uint32_t*>(w + 16);
  a.info = reinterpret_cast<int4*>(w + L.info);
  a.partial = reinterpret_cast<float*>(w + L.partial), a.plse = reinterpret_cast<float*>(w + L.plse);
  a.timeout_ns = g_wait_timeout_ns;
  a.c2 = std::fabs(scale) * kLog2e;
  a.negate_q = scale < 0.f ? tc::kIdescNegateA : 0u;
  // a hidden score is -inf before the scale: a scale of 0 becomes one that gives equal weights all the same
  // (2^(1e-30 s) is 1)
  if (a.c2 == 0.f) a.c2 = 1e-30f;
  a.max_pages = max_pages, a.n_pages = n_pages, a.page_shift = page_shift, a.block_shift = std::min(page_shift, kMaxBlockShift);
  a.bs = bs, a.rows = rows, a.Hq = Hq, a.Hkv = Hkv, a.g = g, a.tokens = prompts ? fit : std::min(unit_rows / g, std::max(max_rows, 1));
  a.window = window >= a.cache_limit ? 0 : window, a.n_sink = n_sink;
  CUtensorMap mq, mk, mv;
  const int page = 1 << page_shift, block = 1 << a.block_shift;
  if (!tch::encode_fn() || !encode_q(&mq, q, rows, Hq, D, q_stride, a.g, a.tokens) ||
      !encode_cache(&mk, k_cache, n_pages, Hkv, page, D, block) ||
      !encode_cache(&mv, v_cache, n_pages, Hkv, page, D, block))
    return cudaErrorInvalidValue;
  const cudaError_t e = prompts ? launch_attention_prompts(D, mq, mk, mv, a, n_cta, s)
                                : launch_attention_windows(D, unit_rows, mq, mk, mv, a, n_cta, s);
  if (e != cudaSuccess) return e;
  // A unit is cut about once where units outnumber the ranges (64 windows over up to 32000 positions: two parts at a time 83.2
  // us, eight 85.1; prompts 306 and 316), and often where there are few (one token over 5000 positions: two 20.4, four 19.1,
  // eight 16.9).  A prompt has so many rows that their number counts for more than their parts (500 rows: two 22.8, sixteen
  // 28.0; 100 over 50000 positions: 42.7 and 40.3).  The number of units says nothing of a long context among short ones: 1 of
  // 30000 positions among 15 of 300, 8 KV heads, D 128, takes two parts (36.2) though sixteen were better (29.4), 1 of 100000
  // among 63 of 500 as well (91.7 and 85.9); with one KV head both take sixteen (18.0, two 41.1; 28.6, two 66.2).
  const bool many_parts = !prompts && n_ranges > int64_t(4) * Hkv * std::max(bs, rows / a.tokens);
  const dim3 grid(n_ranges, ((prompts ? kTile : 0) + a.tokens * g + 7) / 8);
  auto join = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, s, a, unit_rows); };
  if (many_parts) return D == 64 ? join(attention_join_kernel<64, kJoinTogether>) : join(attention_join_kernel<128, kJoinTogether>);
  return D == 64 ? join(attention_join_kernel<64, 2>) : join(attention_join_kernel<128, 2>);
}

}  // namespace dspark
