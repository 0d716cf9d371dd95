// dspark_append_kv8 and dspark_read_kv8: rotate, quantise and append the packed rows to an 8-bit paged cache, and read what
// they see of it back to pages of bf16.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "packed_rows.cuh"
#include "pdl.h"
#include "tc_host.h"

namespace dspark {
namespace {

constexpr int kMaxAppendThreads = 128;

struct AppendArgs {
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *cu, *ctx;
  const float* cos_sin;
  const int32_t* page_table;
  __nv_bfloat16* q_out;
  uint8_t *k_cache, *v_cache, *kv_scale;
  uint32_t* status;
  int bs, rows, max_pos, rot, max_pages, n_pages, page_shift, Hq, Hkv, D;
};

struct RowPlace {
  int pos;       // position in its sequence; < 0: the row is skipped
  int64_t slot;  // slots of the cache before (page, KV head 0, slot)
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
// 8 values times `by` (a power of two) as codes
__device__ __forceinline__ uint2 codes8(const float* x, float by) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = kv8::code2(x[2 * i] * by, x[2 * i + 1] * by);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// A memory-bound copy: two multiplications per element, and for K and V the largest magnitude of a head.  A block has one
// row; an item is 16 lanes of one head: rotated by halves, lanes t .. t+7 and their partners t + rot/2 ..; otherwise 16
// lanes in a row (8 interleaved pairs, or lanes that pass).  So each thread holds both lanes of its pairs and q_out may be q,
// and a head's D / 16 items lie in neighbouring lanes of one warp, which agree on the head's power of two.
// GB300, Hq 32, Hkv 8, D 128: 8191 rows 36.3 us (26.8 by their bytes), one row 6.2, of which most is the call.  Bound by a
// block's chain (its row's place, an item's lanes, the head's maximum) and by the instructions between (half of the issue
// slots).  A thread's next item is asked for before this one is turned; without that 37.4, with the first one alone asked for
// early 38.3 (10 blocks an SM) and 39.7 (12).  256 threads, which leave half of them idle in a row's second turn, took 45.6
// where 128 took 37.7, 192 threads 38.7, two items at a time 45.1, registers for 16 blocks 54.8, for 8 36.9.
// The rotated K goes into 8 bits from fp32, with one rounding.  Products and sums of a pair are rounded one by one (no fused
// multiply-add), so that the powers of two are those of any plain fp32 evaluation.
template <bool kInterleaved>
__global__ void __launch_bounds__(kMaxAppendThreads, 10) append8_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ RowPlace place;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_enter();
  const int row = blockIdx.x;
  const int per_head = a.D / 16, turned = a.rot / 16, items = (a.Hq + 2 * a.Hkv) * per_head;
  uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
  auto fetch = [&](int it) {  // an item's lanes: in time for a thread's next turn, the first while the row's place is looked up
    if (it >= items) return;
    const int hh = it / per_head, c = it - hh * per_head;
    const bool is_q = hh < a.Hq, is_k = !is_q && hh < a.Hq + a.Hkv;
    const int kv = is_q ? 0 : hh - a.Hq - (is_k ? 0 : a.Hkv);
    const __nv_bfloat16* src = is_q   ? a.q + int64_t(row) * a.q_stride + hh * a.D
                               : is_k ? a.k + int64_t(row) * a.k_stride + kv * a.D
                                      : a.v + int64_t(row) * a.v_stride + kv * a.D;
    const bool halves = !kInterleaved && !(hh >= a.Hq + a.Hkv) && c < turned;
    const int lo = halves ? c * 8 : c * 16, hi = halves ? lo + a.rot / 2 : lo + 8;
    x = *reinterpret_cast<const uint4*>(src + lo), y = *reinterpret_cast<const uint4*>(src + hi);
  };
  fetch(tid);
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
          pl.slot = (int64_t(page) * a.Hkv << a.page_shift) + (p & ((1 << a.page_shift) - 1));
        } else {
          set_status(a.status, DSPARK_EINVAL);
        }
      }
      place = pl;
    }
  }
  __syncthreads();

  const RowPlace pl = place;
  if (pl.pos < 0) return;
  for (int first = tid - lane; first < items; first += int(blockDim.x)) {  // the warp's: all its lanes agree below
    const int it = first + lane;
    const bool live = it < items;
    const int hh = live ? it / per_head : 0, c = live ? it - hh * per_head : 0;
    const bool is_q = hh < a.Hq, is_k = !is_q && hh < a.Hq + a.Hkv;
    const int kv = is_q ? 0 : hh - a.Hq - (is_k ? 0 : a.Hkv);
    const bool rotates = (is_q || is_k) && c < turned;
    const int lo = !kInterleaved && rotates ? c * 8 : c * 16;
    const int hi = !kInterleaved && rotates ? lo + a.rot / 2 : lo + 8;
    float u[8], w[8];
    unpack8(x, u);
    unpack8(y, w);
    fetch(it + int(blockDim.x));
    if (live && rotates) {
      // pairs t0 .. t0+7 of this position: cosines and sines
      const float* cs = a.cos_sin + int64_t(pl.pos) * a.rot + c * 8;
      float co[8], si[8];
      *reinterpret_cast<float4*>(co) = *reinterpret_cast<const float4*>(cs);
      *reinterpret_cast<float4*>(co + 4) = *reinterpret_cast<const float4*>(cs + 4);
      *reinterpret_cast<float4*>(si) = *reinterpret_cast<const float4*>(cs + a.rot / 2);
      *reinterpret_cast<float4*>(si + 4) = *reinterpret_cast<const float4*>(cs + a.rot / 2 + 4);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        float& p0 = kInterleaved ? (t < 4 ? u[2 * t] : w[2 * t - 8]) : u[t];
        float& p1 = kInterleaved ? (t < 4 ? u[2 * t + 1] : w[2 * t - 7]) : w[t];
        const float n0 = __fsub_rn(__fmul_rn(p0, co[t]), __fmul_rn(p1, si[t]));
        const float n1 = __fadd_rn(__fmul_rn(p1, co[t]), __fmul_rn(p0, si[t]));
        p0 = n0, p1 = n1;
      }
    }
    if (live && is_q) {
      __nv_bfloat16* dst = a.q_out + (int64_t(row) * a.Hq + hh) * a.D;
      *reinterpret_cast<uint4*>(dst + lo) = pack8(u);
      *reinterpret_cast<uint4*>(dst + hi) = pack8(w);
    }
    if (__all_sync(~0u, is_q || !live)) continue;
    // the head's largest magnitude: as bits, so that a NaN is larger than everything
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) top = max(top, max(__float_as_uint(u[t]) & 0x7FFFFFFFu, __float_as_uint(w[t]) & 0x7FFFFFFFu));
    for (int o = 1; o < per_head; o <<= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
    if (!live || is_q) continue;
    const uint32_t byte = kv8::exponent_byte(top);
    const float by = byte == kv8::kNan ? 0.f : kv8::power(127 - int(byte));
    if (byte == kv8::kNan) {
#pragma unroll
      for (int t = 0; t < 8; ++t) u[t] = w[t] = 0.f;
    }
    const int64_t slot = pl.slot + (int64_t(kv) << a.page_shift);
    uint8_t* dst = (is_k ? a.k_cache : a.v_cache) + slot * a.D;
    *reinterpret_cast<uint2*>(dst + lo) = codes8(u, by);
    *reinterpret_cast<uint2*>(dst + hi) = codes8(w, by);
    if (c == 0) a.kv_scale[slot * 2 + (is_k ? 0 : 1)] = uint8_t(byte);
  }
}

// ------------------------------------------------------------------------------- reading back

struct ReadArgs {
  const uint8_t *k_cache, *v_cache, *kv_scale;
  const int32_t *page_table, *cu, *ctx, *out_table;
  __nv_bfloat16 *k_out, *v_out;
  uint32_t* status;
  int64_t cache_limit;
  int max_pages, n_pages, page_shift, block_shift, bs, rows, Hkv, D, window, n_sink, n_out_pages;
  bool attended;  // by products over whole tiles, next
};

constexpr int kReadThreads = 256;

// 16 codes to 16 values of bf16: exact, but for values below bf16's normal range.
__device__ __forceinline__ void widen16(uint4 w, float by, uint4* out) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = kv8::values(in[i] & 0xFFFFu), b = kv8::values(in[i] >> 16);
    r[2 * i] = pack2(a.x * by, a.y * by), r[2 * i + 1] = pack2(b.x * by, b.y * by);
  }
  out[0] = make_uint4(r[0], r[1], r[2], r[3]), out[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// What a request's packed rows see, in blocks of the cache (pages, or 32-slot pieces of larger pages): those that hold
// sinks, then those of the window.  Blocks are counted over the requests; a unit is a block of one KV head, and the units are
// dealt out to the grid's warps in turn.
// A copy that doubles in size: bound by memory.  GB300, what 64 windows of 4096 see, D 64: 118 us (92 by
// its bytes); a block for each unit 142, five blocks on an SM 138, three 134.
template <int D>
__global__ void __launch_bounds__(kReadThreads, 4) read8_kernel(const __grid_constant__ ReadArgs a) {
  __shared__ long long before[DSPARK_MAX_BS + 1];  // blocks of the requests before
  __shared__ long long warp_total[DSPARK_MAX_BS / 32];
  __shared__ int2 first[DSPARK_MAX_BS];  // the first position of a request's window, and behind its last
  __shared__ int bad;
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bsh = a.block_shift;
  if (tid == 0) bad = 0;
  __syncthreads();
  int mine = 0;
  if (tid < a.bs) {
    const int row = a.cu[tid], next = a.cu[tid + 1], c = a.ctx[tid];
    if (row < 0 || next < row || next > a.rows) {
      bad = 1;
    } else if (next > row) {
      const int n = next - row;
      if (c < 0 || int64_t(c) + n > a.cache_limit) {
        if (blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
      } else {
        const int lo = a.window ? max(0, c - a.window + 1) : 0;
        const int sinks = a.window ? min(a.n_sink, lo) : 0;
        first[tid] = make_int2(lo, c + n);
        mine = ((c + n - 1) >> bsh) - (lo >> bsh) + 1;
        // sink blocks that the window's do not reach
        mine += min((sinks + (1 << bsh) - 1) >> bsh, lo >> bsh);
      }
    }
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  for (int i = 0; i < warp; ++i) incl += warp_total[i];
  if (tid == 0) before[0] = 0;
  before[tid + 1] = incl;
  __syncthreads();
  if (bad) {
    if (tid == 0 && blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
    return;
  }
  const int64_t units = before[a.bs] * a.Hkv;
  constexpr int kPerSlot = D / 16, kRounds = 32 * kPerSlot / 32;  // 16-byte pieces; rounds of a warp over a whole block
  for (int64_t u = int64_t(blockIdx.x) * (kReadThreads / 32) + warp; u < units; u += int64_t(gridDim.x) * (kReadThreads / 32)) {
    const long long block = u / a.Hkv;
    const int h = int(u - block * a.Hkv);
    int r = 0;
    for (int step = DSPARK_MAX_BS / 2; step > 0; step >>= 1)
      if (r + step < a.bs && before[r + step] <= block) r += step;
    const int lo = first[r].x, end = first[r].y, sinks = a.window ? min(a.n_sink, lo) : 0;
    const int sb = min((sinks + (1 << bsh) - 1) >> bsh, lo >> bsh), v = int(block - before[r]);
    const int pos0 = (v < sb ? v : v - sb + (lo >> bsh)) << bsh;
    const int64_t at = int64_t(r) * a.max_pages + (pos0 >> a.page_shift);
    const int page = a.page_table[at], to = a.out_table[at];
    if (page < 0 || page >= a.n_pages || to < 0 || to >= a.n_out_pages) {
      if (lane == 0) set_status(a.status, DSPARK_EINVAL);
      continue;
    }
    const int slot0 = pos0 & ((1 << a.page_shift) - 1);
    const int64_t src = ((int64_t(page) * a.Hkv + h) << a.page_shift) + slot0;
    const int64_t dst = ((int64_t(to) * a.Hkv + h) << a.page_shift) + slot0;
    // lane i has slot i's exponents, and whether some row sees it
    const int pos = pos0 + lane;
    const bool mine = lane < 1 << bsh && pos < end && (pos >= lo || pos < sinks);
    const uint32_t seen = __ballot_sync(~0u, mine);
    uint32_t bytes = mine ? reinterpret_cast<const uint16_t*>(a.kv_scale)[src + lane] : 0u;
    // A V of NaN would reach rows that do not see it, as 0 * NaN, and leave the log-sum-exp: its K is NaN instead
    if (a.attended && ((bytes & 0xFFu) == kv8::kNan || bytes >> 8 == kv8::kNan)) bytes = 127u << 8 | kv8::kNan;
    const uint4* ks = reinterpret_cast<const uint4*>(a.k_cache) + src * kPerSlot + lane;
    const uint4* vs = reinterpret_cast<const uint4*>(a.v_cache) + src * kPerSlot + lane;
    uint4* ko = reinterpret_cast<uint4*>(a.k_out) + (dst * kPerSlot + lane) * 2;
    uint4* vo = reinterpret_cast<uint4*>(a.v_out) + (dst * kPerSlot + lane) * 2;
#pragma unroll
    for (int k0 = 0; k0 < kRounds; k0 += 4) {  // eight loads under way
      uint4 k[4], x[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int s = ((k0 + b) * 32 + lane) / kPerSlot;
        if (seen >> s & 1u) k[b] = __ldcs(ks + (k0 + b) * 32), x[b] = __ldcs(vs + (k0 + b) * 32);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int s = ((k0 + b) * 32 + lane) / kPerSlot;
        const uint32_t e = __shfl_sync(~0u, bytes, s);
        if (seen >> s & 1u) {
          widen16(k[b], kv8::factor(e & 0xFFu), ko + (k0 + b) * 64);
          widen16(x[b], kv8::factor(e >> 8), vo + (k0 + b) * 64);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_append_kv8(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* cu, const int32_t* ctx, int bs, int rows,
                              const float* cos_sin, int max_pos, int rot, int interleaved, const int32_t* page_table,
                              int max_pages, int n_pages, int page_shift, int Hq, int Hkv, int D, void* q_out,
                              void* k_cache, void* v_cache, uint8_t* kv_scale, uint32_t* status, cudaStream_t s) {
  AppendArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q), a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.cu = cu, a.ctx = ctx, a.cos_sin = cos_sin, a.page_table = page_table;
  a.q_out = static_cast<__nv_bfloat16*>(q_out), a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache), a.kv_scale = kv_scale;
  a.status = status;
  a.bs = bs, a.rows = rows, a.max_pos = max_pos, a.rot = rot, a.max_pages = max_pages, a.n_pages = n_pages;
  a.page_shift = page_shift, a.Hq = q ? Hq : 0, a.Hkv = Hkv, a.D = D;
  const int items = (a.Hq + 2 * Hkv) * (D / 16);
  // as many threads as share the items evenly: 384 items, 8191 rows, 128 threads 37.7 us, 192 38.7, 256 45.6
  const int rounds = (items + kMaxAppendThreads - 1) / kMaxAppendThreads;
  const dim3 block(((items + rounds - 1) / rounds + 31) / 32 * 32);
  return launch_pdl(interleaved ? append8_kernel<true> : append8_kernel<false>, dim3(rows), block, 0, s, a);
}

cudaError_t launch_read_kv8(const void* k_cache, const void* v_cache, const uint8_t* kv_scale, const int32_t* page_table,
                            int max_pages, int n_pages, int page_shift, const int32_t* cu, const int32_t* ctx, int bs,
                            int rows, int Hkv, int D, int window, int n_sink, const int32_t* out_table, int n_out_pages,
                            void* k_out, void* v_out, bool attended, uint32_t* status, cudaStream_t s) {
  ReadArgs a;
  a.k_cache = static_cast<const uint8_t*>(k_cache), a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.kv_scale = kv_scale, a.page_table = page_table, a.cu = cu, a.ctx = ctx, a.out_table = out_table;
  a.k_out = static_cast<__nv_bfloat16*>(k_out), a.v_out = static_cast<__nv_bfloat16*>(v_out), a.status = status;
  a.cache_limit = std::min(int64_t(max_pages) << page_shift, int64_t(1) << 30);  // positions: well inside 32 bits
  a.max_pages = max_pages, a.n_pages = n_pages, a.page_shift = page_shift, a.block_shift = std::min(page_shift, 5);
  a.bs = bs, a.rows = rows, a.Hkv = Hkv, a.D = D, a.window = window >= a.cache_limit ? 0 : window, a.n_sink = n_sink;
  a.n_out_pages = n_out_pages, a.attended = attended;
  // a warp for each block that the page table can hold, where that is fewer
  const int64_t most = (int64_t(bs) * (a.cache_limit >> a.block_shift) * Hkv + kReadThreads / 32 - 1) / (kReadThreads / 32);
  const dim3 grid(unsigned(std::min(int64_t(tch::sm_count()) * 4, std::max(most, int64_t(1)))));
  return D == 64 ? launch_pdl(read8_kernel<64>, grid, dim3(kReadThreads), 0, s, a)
                 : launch_pdl(read8_kernel<128>, grid, dim3(kReadThreads), 0, s, a);
}

}  // namespace dspark
