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
// A chain of trips to memory (what the ranges left, the log-sum-exps, the rows), so each step's loads are issued
// together, eight rows' pieces at a time.
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ AttnArgs a, int n_ranges, int unit_rows) {
  constexpr int E = D / 32, kTogether = 8;
  pdl_enter();
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5), c = blockIdx.x;
  const int4 info = a.info[c];
  int flags = c + 1 + lane < n_ranges ? a.info[c + 1 + lane].x : 0;
  if (!(info.x & kHeadUsed)) return;
  const int tok = (row / kTile) * a.tokens + (row % kTile) / a.g, hh = (row % kTile) % a.g;
  if (row % kTile >= a.tokens * a.g || tok >= info.z) return;
  // part 0 is the head of c, part i the tail of c + i, up to the first range that finished the unit
  int n = 0;
  for (int base = c + 1;; base += 32) {
    const uint32_t ends = __ballot_sync(~0u, flags & kTailEnds);
    if (ends || base + 32 >= n_ranges) {
      n = (ends ? base + __ffs(ends) - 1 : n_ranges - 1) - c + 1;
      break;
    }
    flags = base + 32 + lane < n_ranges ? a.info[base + 32 + lane].x : 0;
  }
  auto part_row = [&](int i) { return int64_t(i == 0 ? 2 * c + 1 : 2 * (c + i)) * unit_rows + row; };
  auto part_lse = [&](int i) {  // every range between has worked on the unit and on nothing else
    return i < n ? a.plse[part_row(i)] : -INFINITY;
  };
  const float mine = part_lse(lane);
  float top = mine;
  for (int i = lane + 32; i < n; i += 32) top = fmaxf(top, part_lse(i));
  top = __shfl_sync(~0u, warp_max(top), 0);
  const float ref = top == -INFINITY ? 0.f : top;
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int base = 0; base < n; base += 32) {
    const float w_mine = exp2f((base == 0 ? mine : part_lse(base + lane)) - ref);  // 0: nothing seen there
    for (int i0 = 0; i0 < min(32, n - base); i0 += kTogether) {
      float v[kTogether][E], w[kTogether];
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        w[k] = __shfl_sync(~0u, w_mine, i0 + k);  // beyond the last part: 0, and the last part's row again
        const float* src = a.partial + part_row(min(base + i0 + k, n - 1)) * D + lane * E;
        if constexpr (E == 4)
          *reinterpret_cast<float4*>(v[k]) = *reinterpret_cast<const float4*>(src);
        else
          *reinterpret_cast<float2*>(v[k]) = *reinterpret_cast<const float2*>(src);
      }
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        sum += w[k];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = w[k] == 0.f ? acc[e] : fmaf(w[k], v[k][e], acc[e]);
      }
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
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
  const dim3 grid(n_ranges, ((prompts ? kTile : 0) + a.tokens * g + 7) / 8);
  return D == 64 ? launch_pdl(attention_join_kernel<64>, grid, dim3(256), 0, s, a, n_ranges, unit_rows)
                 : launch_pdl(attention_join_kernel<128>, grid, dim3(256), 0, s, a, n_ranges, unit_rows);
}

}  // namespace dspark
