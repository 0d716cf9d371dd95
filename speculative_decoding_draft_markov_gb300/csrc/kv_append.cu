// dspark_append_kv: rotate q and k of the packed rows by their positions and put k and v into the
// paged cache.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "packed_rows.cuh"
#include "pdl.h"

namespace dspark {
namespace {

constexpr int kMaxAppendThreads = 256;

struct AppendArgs {
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *cu, *ctx;
  const float* cos_sin;
  const int32_t* page_table;
  __nv_bfloat16 *q_out, *k_cache, *v_cache;
  uint32_t* status;
  int bs, rows, max_pos, rot, max_pages, n_pages, page_shift, Hq, Hkv, D;
};

struct RowPlace {
  int pos;        // position in its sequence; < 0: the row is skipped
  int64_t slot;   // element offset of (page, KV head 0, slot) in the cache
};

__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
  x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// A memory-bound copy with two multiplications per element.  A block has one row; an item is 16 lanes of one head, as
// two 16-byte loads and stores: rotated by halves, lanes t .. t+7 and their partners t + rot/2 ..;
// otherwise 16 lanes in a row (8 interleaved pairs, or lanes that pass).  So each thread holds both
// lanes of its pairs and q_out may be q.
// GB300, Hq 32, Hkv 8, D 128: 8191 rows 31.8 us (90% of the measured copy bandwidth); 256 windows of 1 .. 8 rows
// 7.1 us (4.2 by their bytes); one row 3.0 us, a launch and five dependent trips to memory (window, length, page, row, store).
// Four rows to a block took 33.9, 7.0 and 3.3 us, eight 41.5, 9.0 and 3.8; a thread's first two items asked for
// before the row's place is known 36.5, 9.4 and 3.0 (twice the registers); 40 registers in place of 32 34.0 and 8.3.
template <bool kInterleaved>
__global__ void __launch_bounds__(kMaxAppendThreads, 8) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ RowPlace place;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_enter();
  const int row = blockIdx.x;
  if (tid < 32) {
    const int r = warp_request_of(a.cu, a.bs, a.rows, row, lane);
    if (lane == 0) {
      RowPlace pl{-1, 0};
      if (r < 0) {
        set_status(a.status, DSPARK_EINVAL);
      } else if (r < a.bs) {
        const int c = a.ctx[r];
        const int64_t p = int64_t(c) + row - a.cu[r];
        const int64_t pi = p >> a.page_shift;
        int page = -1;
        if (c >= 0 && p >= 0 && p < a.max_pos && pi < a.max_pages)
          page = a.page_table[int64_t(r) * a.max_pages + pi];
        if (page >= 0 && page < a.n_pages) {
          pl.pos = int(p);
          pl.slot = ((int64_t(page) * a.Hkv << a.page_shift) + (p & ((1 << a.page_shift) - 1))) * a.D;
        } else {
          set_status(a.status, DSPARK_EINVAL);
        }
      }
      place = pl;
    }
  }
  __syncthreads();

  const int per_head = a.D / 16, turned = a.rot / 16;
  const RowPlace pl = place;
  if (pl.pos < 0) return;
  for (int it = tid; it < (a.Hq + 2 * a.Hkv) * per_head; it += int(blockDim.x)) {
    const int hh = it / per_head, c = it - hh * per_head;
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    const int64_t head_step = int64_t(a.D) << a.page_shift;
    if (hh < a.Hq) {
      src = a.q + int64_t(row) * a.q_stride + hh * a.D;
      dst = a.q_out + (int64_t(row) * a.Hq + hh) * a.D;
    } else if (hh < a.Hq + a.Hkv) {
      src = a.k + int64_t(row) * a.k_stride + (hh - a.Hq) * a.D;
      dst = a.k_cache + pl.slot + (hh - a.Hq) * head_step;
    } else {
      src = a.v + int64_t(row) * a.v_stride + (hh - a.Hq - a.Hkv) * a.D;
      dst = a.v_cache + pl.slot + (hh - a.Hq - a.Hkv) * head_step;
    }
    const bool rotates = hh < a.Hq + a.Hkv && c < turned;
    const int lo = !kInterleaved && rotates ? c * 8 : c * 16;
    const int hi = !kInterleaved && rotates ? lo + a.rot / 2 : lo + 8;
    uint4 x = *reinterpret_cast<const uint4*>(src + lo), y = *reinterpret_cast<const uint4*>(src + hi);
    if (rotates) {
      // pairs t0 .. t0+7 of this position: cosines and sines
      const float* cs = a.cos_sin + int64_t(pl.pos) * a.rot + c * 8;
      float co[8], si[8], u[8], w[8];
      *reinterpret_cast<float4*>(co) = *reinterpret_cast<const float4*>(cs);
      *reinterpret_cast<float4*>(co + 4) = *reinterpret_cast<const float4*>(cs + 4);
      *reinterpret_cast<float4*>(si) = *reinterpret_cast<const float4*>(cs + a.rot / 2);
      *reinterpret_cast<float4*>(si + 4) = *reinterpret_cast<const float4*>(cs + a.rot / 2 + 4);
      unpack8(x, u);
      unpack8(y, w);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        float& p0 = kInterleaved ? (t < 4 ? u[2 * t] : w[2 * t - 8]) : u[t];
        float& p1 = kInterleaved ? (t < 4 ? u[2 * t + 1] : w[2 * t - 7]) : w[t];
        const float n0 = p0 * co[t] - p1 * si[t], n1 = p1 * co[t] + p0 * si[t];
        p0 = n0, p1 = n1;
      }
      x = pack8(u);
      y = pack8(w);
    }
    *reinterpret_cast<uint4*>(dst + lo) = x;
    *reinterpret_cast<uint4*>(dst + hi) = y;
  }
}

}  // namespace

cudaError_t launch_append_kv(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, const int32_t* cu, const int32_t* ctx, int bs, int rows,
                             const float* cos_sin, int max_pos, int rot, int interleaved, const int32_t* page_table,
                             int max_pages, int n_pages, int page_shift, int Hq, int Hkv, int D, void* q_out,
                             void* k_cache, void* v_cache, uint32_t* status, cudaStream_t s) {
  AppendArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q), a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.cu = cu, a.ctx = ctx, a.cos_sin = cos_sin, a.page_table = page_table;
  a.q_out = static_cast<__nv_bfloat16*>(q_out), a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  a.status = status;
  a.bs = bs, a.rows = rows, a.max_pos = max_pos, a.rot = rot, a.max_pages = max_pages, a.n_pages = n_pages;
  a.page_shift = page_shift, a.Hq = q ? Hq : 0, a.Hkv = Hkv, a.D = D;
  const int items = (a.Hq + 2 * Hkv) * (D / 16);
  const dim3 block(std::min((items + 31) / 32 * 32, kMaxAppendThreads));
  return launch_pdl(interleaved ? append_kernel<true> : append_kernel<false>, dim3(rows), block, 0, s, a);
}

}  // namespace dspark
