// dspark_process_logits (penalties, biases and grammar masks on the packed target rows) and the
// token history that its penalties read.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "pdl.h"
#include "tc_host.h"

namespace dspark {
namespace {

constexpr int kRuleThreads = 256;
constexpr int kRuleIds = 8;                          // ids per thread
constexpr int kRuleChunk = kRuleThreads * kRuleIds;  // ids per block

struct RuleArgs {
  const void* logits;
  void* out;
  const int32_t *cu, *ids;
  const int16_t* hist;
  const float *repetition, *frequency, *presence;
  const int32_t *bias_start, *bias_ids;
  const float* bias_vals;
  const uint8_t* mask;
  uint32_t* status;
  int rows, V, n_bias, mask_row_bytes;
};

template <typename T> struct Pack8;  // 8 logits of a row
template <> struct Pack8<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void get(float* x) const {
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
  }
  static __device__ uint32_t two(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // store x, with -inf where a bit of `allowed` is 0
  static __device__ void store(__nv_bfloat16* p, const float* x, uint32_t allowed) {
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t m;  // bits 2k and 2k + 1, as the signs of two low bytes, spread over 16 bits each
      asm("prmt.b32 %0, %1, %2, 0xCC88;" : "=r"(m) : "r"(allowed << (7 - 2 * k)), "r"(k == 3 ? allowed : allowed << (6 - 2 * k)));
      v[k] = (two(x[2 * k], x[2 * k + 1]) & m) | (0xFF80FF80u & ~m);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(v[0], v[1], v[2], v[3]));
  }
};
template <> struct Pack8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ void store(float* p, const float* x, uint32_t allowed) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = allowed >> k & 1u ? x[k] : -INFINITY;
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
  }
};

// One streaming pass: read the row, write the row; bound by memory as long as a warp spends fewer than
// about 170 instructions on the 1 KB of a row that it reads and writes.  A block owns 2048 ids of one request
// and walks the request's rows (with few requests, blockIdx.z takes a share of them).  Per id the rules are
// one product and one sum, l * (l > 0 ? up : down) + add, which a thread keeps in registers for its 8 ids: the
// history and the biases are read once for all rows of a window, a drafted token changes one thread's
// registers.  The first rows are asked for before the history and the biases.  Each warp finds its own
// biases in the request's sorted list, so no barrier stands in the way.
// GB300, V 151936, bf16, history, 300 biases and a mask, 256 requests: windows of 8 rows 212 us (95% of the
// measured copy bandwidth); of 1 .. 8 rows 147 us (82%); of one row 69 us (51%).  A warp executes 360
// instructions (83 for the biases) before a window's first row and 81 for each row, at 2.0 to 2.1 a
// cycle and SM: short windows are bound by the instructions before the first row.  Slower, each measured there: the factors worked out per
// row; rows through shared memory by asynchronous copies (238 us where registers took 212); the biases asked for before the
// search (153 us for 146); one wave of blocks, each over many windows (197 for 146).
// In place a row's logits are asked for when its rules are known, for the groups of 8 ids that a rule changes (under a
// mask nearly all of them): 256 windows of 1 .. 8 rows 200 us with the mask, 180 without (out of place 147 and 139), of 8
// rows 303 (218), of one row 91 (69); 8 windows of 16 rows in fp32 without a mask 16.0 (26.1), with one 27.4 (27.1); one
// row 3.3 (3.1).  The sectors that the rules touch are worth 120, 42, 201, 35, 1.3, 19 and 0.1 us.
// kAhead: rows in flight; kBlocks: blocks on an SM, which sets the registers.
template <typename T, bool kInPlace, int kAhead, int kBlocks>
__global__ void __launch_bounds__(kRuleThreads, kBlocks) rules_kernel(const __grid_constant__ RuleArgs a) {
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, r = blockIdx.y;
  const int lo = blockIdx.x * kRuleChunk, base = lo + tid * kRuleIds;  // V is a multiple of 8
  const int row0 = a.cu[r], row1 = a.cu[r + 1], n = row1 - row0;
  if (row0 < 0 || n < 0 || row1 > a.rows) {
    if (tid == 0 && blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
    return;
  }
  // this block's rows of the window
  const int share = (n + gridDim.z - 1) / gridDim.z, i0 = blockIdx.z * share, i1 = min(n, i0 + share);
  if (i0 >= i1) return;
  const bool live = base < a.V, checks = blockIdx.x == 0 && blockIdx.z == 0;

  const size_t at0 = size_t(row0 + i0) * a.V + base;
  const T* ask_src = static_cast<const T*>(a.logits) + at0;
  const T* src = ask_src;
  T* dst = static_cast<T*>(a.out) + at0;
  const uint8_t* ask_mask = a.mask ? a.mask + size_t(row0 + i0) * a.mask_row_bytes + (base >> 3) : nullptr;
  Pack8<T> x[kAhead];
  uint32_t allowed[kAhead];
  auto ask = [&](int b) {
    if (!kInPlace) x[b].load(ask_src), ask_src += a.V;
    if (ask_mask) allowed[b] = __ldcs(ask_mask), ask_mask += a.mask_row_bytes;
  };
#pragma unroll
  for (int b = 0; b < kAhead; ++b) {
    allowed[b] = 0xFFu;
    if (live && b < i1 - i0) ask(b);
  }
  uint4 words = make_uint4(0u, 0u, 0u, 0u);
  if (a.hist && live) words = __ldcs(reinterpret_cast<const uint4*>(a.hist + size_t(r) * a.V + base));
  const float rho = a.repetition ? a.repetition[r] : 1.f;
  const float inv_rho = 1.f / rho;  // l / rho as a product: within 1.5 ulp of fp32 of the quotient
  const float freq = a.frequency ? a.frequency[r] : 0.f, pres = a.presence ? a.presence[r] : 0.f;

  // whether a drafted id of the window is one of the block's
  const int32_t* ids = a.ids + row0;
  bool touched = false;
  if (a.hist) {
    for (int i = 1 + lane; i < n; i += 32) {
      const int id = ids[i];
      touched |= id >= lo && id < lo + kRuleChunk;
      if (checks && (id < 0 || id >= a.V)) set_status(a.status, DSPARK_EINVAL);
    }
    touched = __any_sync(~0u, touched);
  }

  float up[kRuleIds], down[kRuleIds], add[kRuleIds];  // factors of l > 0 and l <= 0, and what is added
  uint32_t said = 0, acts = 0;                        // bit j: id j was said; some rule but the mask changes it
#pragma unroll
  for (int j = 0; j < kRuleIds; ++j) add[j] = 0.f;
  if (a.bias_start) {
    const int e0 = max(a.bias_start[r], 0), e1 = min(a.bias_start[r + 1], a.n_bias);
    if (checks && tid == 0 && (a.bias_start[r] < 0 || a.bias_start[r + 1] < e0 || a.bias_start[r + 1] > a.n_bias))
      set_status(a.status, DSPARK_EINVAL);
    if (checks)
      for (int e = e0 + tid; e < e1; e += kRuleThreads) {
        const int id = a.bias_ids[e];
        if (id < 0 || id >= a.V || (e > e0 && a.bias_ids[e - 1] >= id)) set_status(a.status, DSPARK_EINVAL);
      }
    // the warp's ids are wb .. wb + 255: from the last sampled entry below wb on, to the first beyond
    const int wb = lo + (tid - lane) * kRuleIds;
    int first = e0;
    for (int len = e1 - e0; len > 64;) {
      const int step = (len + 31) / 32, e = first + lane * step;
      const int below = __popc(__ballot_sync(~0u, lane * step < len && a.bias_ids[min(e, e1 - 1)] < wb));
      first += max(0, below - 1) * step;
      len = min(step, e1 - first);
    }
    for (int e = first + lane; e1 > e0; e += 32) {
      const int id = e < e1 ? a.bias_ids[e] : 0x7FFFFFFF;
      const bool in = id >= wb && id < wb + 32 * kRuleIds;
      const float val = in ? a.bias_vals[e] : 0.f;
      for (uint32_t m = __ballot_sync(~0u, in); m; m &= m - 1) {
        const int who = __ffs(m) - 1, d = __shfl_sync(~0u, id, who) - base;
        const float v = __shfl_sync(~0u, val, who);
        if (d >= 0 && d < kRuleIds) acts |= 1u << d;
#pragma unroll
        for (int j = 0; j < kRuleIds; ++j)
          if (j == d) add[j] = v;
      }
      if (__any_sync(~0u, id >= wb + 32 * kRuleIds)) break;
    }
  }
  if (!live) return;

  const uint32_t h[4] = {words.x, words.y, words.z, words.w};
#pragma unroll
  for (int j = 0; j < kRuleIds; ++j) {
    const uint32_t word = (h[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, count = word & 0x7FFFu;
    if (count) add[j] -= fmaf(freq, float(count), pres), said |= 1u << j;
    up[j] = word ? inv_rho : 1.f, down[j] = word ? rho : 1.f;
    if (kInPlace && word) acts |= 1u << j;
  }
  auto say = [&](int id) {  // one more of `id`
    const int d = id - base;
    if (d >= 0 && d < kRuleIds) {
#pragma unroll
      for (int j = 0; j < kRuleIds; ++j)
        if (j == d) add[j] -= said >> j & 1u ? freq : freq + pres, up[j] = inv_rho, down[j] = rho;
      said |= 1u << d, acts |= 1u << d;
    }
  };
  if (touched)
    for (int i = 1; i < i0; ++i) say(ids[i]);  // drafted before this block's rows
  for (int first = i0; first < i1; first += kAhead) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int i = first + b;
      if (i >= i1) break;
      if (touched && i > 0) say(ids[i]);
      if (!kInPlace || acts != 0 || allowed[b] != 0xFFu) {  // in place, nothing else changes
        if (kInPlace) x[b].load(src);
        float v[kRuleIds];
        x[b].get(v);
#pragma unroll
        for (int j = 0; j < kRuleIds; ++j) v[j] = fmaf(v[j], v[j] > 0.f ? up[j] : down[j], add[j]);
        Pack8<T>::store(dst, v, allowed[b]);
      }
      if (kInPlace) src += a.V;
      dst += a.V;
      if (i + kAhead < i1) ask(b);
    }
  }
}

// ---------------------------------------------------------------------------- history

constexpr int kHistThreads = 512, kHistAhead = 8;  // and tokens that a thread asks for at once
constexpr int kHistMaxChunk = 36 * 1024;  // ids of a block: 72 KB of words, three blocks on an SM

// One more of the 16-bit word at `sh` of *w: a saturating add on its 15-bit count.
__device__ __forceinline__ void count_up(uint32_t* w, int sh) {
  uint32_t old = *w;
  while (((old >> sh) & 0x7FFFu) != 0x7FFFu) {
    const uint32_t got = atomicCAS(w, old, old + (1u << sh));
    if (got == old) break;
    old = got;
  }
}

// A block counts one request's tokens that fall into its `chunk` ids in shared memory, in the words that it
// then writes once.  A list of up to 2^15 - 1 generated tokens cannot overflow a count: plain adds.
// Bound by the latency of its steps (launch, list, counts, words): GB300, one list of 2500 tokens, V
// 151936, 3.7 us with the commit after it; 64 lists of up to 8000 tokens, V 129280, 9.2 us (2.6 by its bytes),
// of 100 tokens each 6.5.  A word per id (twice the blocks, each reading its list) took 12.4, four loads at a time 11.0,
// 1024 threads 9.5.
__global__ void __launch_bounds__(kHistThreads)
    history_build_kernel(const int32_t* __restrict__ tokens, int n_tokens, const int32_t* __restrict__ start,
                         const int32_t* __restrict__ n_prompt, int V, int chunk, int16_t* __restrict__ hist,
                         uint32_t* status) {
  extern __shared__ __align__(16) uint32_t cell[];  // two ids each
  pdl_enter();
  const int tid = threadIdx.x, r = blockIdx.y;
  const int lo = blockIdx.x * chunk, n = min(chunk, V - lo);  // multiples of 8
  int t0 = start[r], t1 = start[r + 1];
  const int asked = n_prompt[r];
  for (int i = tid; i < n / 8; i += kHistThreads) reinterpret_cast<uint4*>(cell)[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  if (t0 < 0 || t1 < t0 || t1 > n_tokens) {
    if (tid == 0 && blockIdx.x == 0) set_status(status, DSPARK_EINVAL);
    t0 = t1 = 0;
  }
  const bool fits = int64_t(t1) - t0 - max(asked, 0) <= 0x7FFF;
  for (int64_t first = int64_t(t0) + tid; first < t1; first += kHistThreads * kHistAhead) {
    int ids[kHistAhead];
#pragma unroll
    for (int k = 0; k < kHistAhead; ++k) {
      const int64_t t = first + k * kHistThreads;
      ids[k] = t < t1 ? tokens[t] : 0;
    }
#pragma unroll
    for (int k = 0; k < kHistAhead; ++k) {
      const int64_t t = first + k * kHistThreads;
      if (t >= t1) break;
      const int id = ids[k], d = id - lo, sh = (d & 1) * 16;
      if (d >= 0 && d < n) {
        if (t - t0 < asked)
          atomicOr(&cell[d >> 1], 0x8000u << sh);
        else if (fits)
          atomicAdd(&cell[d >> 1], 1u << sh);
        else
          count_up(&cell[d >> 1], sh);
      }
      if (blockIdx.x == 0 && (id < 0 || id >= V)) set_status(status, DSPARK_EINVAL);
    }
  }
  __syncthreads();
  uint4* out = reinterpret_cast<uint4*>(hist + size_t(r) * V + lo);
  for (int i = tid; i < n / 8; i += kHistThreads) out[i] = reinterpret_cast<const uint4*>(cell)[i];
}

// One thread per committed token; the latency of a launch and three trips to memory (2.5 us in a row of calls).
__global__ void history_commit_kernel(const int32_t* __restrict__ out_tokens, int n, int per_request, int V,
                                      int16_t* __restrict__ hist, uint32_t* status) {
  pdl_enter();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int id = out_tokens[i];
  if (id == -1) return;
  if (id < 0 || id >= V) {
    set_status(status, DSPARK_EINVAL);
    return;
  }
  const size_t at = size_t(i / per_request) * V + id;
  count_up(reinterpret_cast<uint32_t*>(hist) + (at >> 1), int(at & 1) * 16);
}

}  // namespace

cudaError_t launch_process_logits(const void* logits, int dtype, int rows, int V, const int32_t* cu,
                                  const int32_t* ids, int bs, const int16_t* hist, const float* repetition,
                                  const float* frequency, const float* presence, const int32_t* bias_start,
                                  const int32_t* bias_ids, const float* bias_vals, int n_bias, const uint32_t* mask,
                                  void* out, uint32_t* status, cudaStream_t s) {
  RuleArgs a;
  a.logits = logits, a.out = out, a.cu = cu, a.ids = ids, a.hist = hist;
  a.repetition = repetition, a.frequency = frequency, a.presence = presence;
  a.bias_start = bias_start, a.bias_ids = bias_ids, a.bias_vals = bias_vals;
  a.mask = reinterpret_cast<const uint8_t*>(mask);  // little-endian words: byte i holds ids 8i .. 8i+7
  a.status = status, a.rows = rows, a.V = V, a.n_bias = n_bias, a.mask_row_bytes = (V + 31) / 32 * 4;
  // A window's rows are shared out over z blocks where that fills the SMs better: the z with the least waves x (set-up,
  // worth about four rows, + rows).  8 windows of 16 rows in fp32, V 129280: z = 2 26.3 us, 1 29.8; in bf16, V
  // 151936: z = 1 15.6, 2 17.3; one of 8 rows: z = 4 4.2, 8 4.5, 1 4.8.
  const int blocks = (V + kRuleChunk - 1) / kRuleChunk, slots = (dtype == DSPARK_F32 ? 3 : 4) * tch::sm_count();
  int z = 1;
  auto cost = [&](int n) {
    return int64_t((int64_t(blocks) * bs * n + slots - 1) / slots) * (4 + (rows + bs * n - 1) / (bs * n));
  };
  for (int n = 2; n <= 4; n *= 2)
    if (cost(n) < cost(z)) z = n;
  const dim3 grid(blocks, bs, z), block(kRuleThreads);
  // Windows of one or two rows have nothing to ask for ahead: fewer registers and a fifth block on each SM, once there
  // are more blocks than an SM holds.  256 windows of one row, bf16: 69 us against 79 (64 in fp32: 19.7
  // against 24.6); of 1 .. 8 rows 157 against 146; 8 windows of one row 4.3 against 3.9.
  const bool few = rows < 2 * bs && blocks * bs > 4 * tch::sm_count();
  auto launch = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, s, a); };
  using bf16 = __nv_bfloat16;
  if (dtype == DSPARK_F32)
    return launch(logits == out ? rules_kernel<float, true, 2, 3> : few ? rules_kernel<float, false, 1, 5> : rules_kernel<float, false, 2, 3>);
  return launch(logits == out ? rules_kernel<bf16, true, 3, 4> : few ? rules_kernel<bf16, false, 1, 5> : rules_kernel<bf16, false, 3, 4>);
}

cudaError_t launch_history_build(const int32_t* tokens, int n_tokens, const int32_t* start, const int32_t* n_prompt,
                                 int bs, int V, int16_t* hist, uint32_t* status, cudaStream_t s) {
  // every block of a request reads the request's whole list, so no more blocks than SMs, except as
  // shared memory asks for (four blocks an SM: 64 lists of up to 8000 tokens, V 129280, 10.6 us against 9.2)
  const int most = std::max(1, tch::sm_count() / bs), least = (V + kHistMaxChunk - 1) / kHistMaxChunk;
  const int n = std::max(least, std::min(most, (V + 2047) / 2048));
  const int chunk = ((V + n - 1) / n + 7) / 8 * 8;
  static bool done[tch::kMaxDevices] = {};
  static std::mutex mu;
  const cudaError_t e = tch::set_smem_once(history_build_kernel, kHistMaxChunk * 2, done, &mu);
  if (e != cudaSuccess) return e;
  return launch_pdl(history_build_kernel, dim3((V + chunk - 1) / chunk, bs), dim3(kHistThreads),
                    chunk * 2, s, tokens, n_tokens, start, n_prompt, V, chunk, hist, status);
}

cudaError_t launch_history_commit(const int32_t* out_tokens, int bs, int gamma, int V, int16_t* hist, uint32_t* status,
                                  cudaStream_t s) {
  const int n = bs * (gamma + 1);
  return launch_pdl(history_commit_kernel, dim3((n + 127) / 128), dim3(128), 0, s, out_tokens, n, gamma + 1, V, hist,
                    status);
}

}  // namespace dspark
