// dspark_process_logits (penalties, biases and grammar masks on the packed target rows) and the
// token history that its penalties read.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "pdl.h"

namespace dspark {
namespace {

constexpr int kRuleThreads = 256;
constexpr int kRuleIds = 8;                            // ids per thread
constexpr int kRuleChunk = kRuleThreads * kRuleIds;    // ids per block
constexpr int kRowBatch = 4;                           // rows whose loads are in flight together

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
  int rows, V, mask_row_bytes;
  bool in_place;
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
  static __device__ void store(__nv_bfloat16* p, const float* x) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7])));
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
  static __device__ void store(float* p, const float* x) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  }
};

// One streaming pass, bound by memory: read the row, write the row.  A block owns 2048 ids of one
// request and walks the request's rows; each thread keeps what the rules say of its 8 ids (their
// counts, and the sum of bias and penalties) in registers, so the history and the biases are read
// once for all rows of a window, and a drafted token changes one thread's registers.
template <typename T>
__global__ void __launch_bounds__(kRuleThreads) rules_kernel(RuleArgs a) {
  __shared__ float sbias[kRuleChunk];
  pdl_enter();
  const int tid = threadIdx.x, r = blockIdx.y;
  const int lo = blockIdx.x * kRuleChunk, base = lo + tid * kRuleIds;
  const int row0 = a.cu[r], row1 = a.cu[r + 1];
  if (row0 < 0 || row1 < row0 || row1 > a.rows) {
    if (tid == 0 && blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
    return;
  }
  if (row0 == row1) return;

  float bias[kRuleIds];
#pragma unroll
  for (int j = 0; j < kRuleIds; ++j) bias[j] = 0.f;
  if (a.bias_start) {
    const int e0 = a.bias_start[r], e1 = a.bias_start[r + 1];
    if (e1 > e0) {  // the same for the whole block
      for (int i = tid; i < kRuleChunk; i += kRuleThreads) sbias[i] = 0.f;
      __syncthreads();
      for (int e = e0 + tid; e < e1; e += kRuleThreads) {
        const int id = a.bias_ids[e];
        if (id >= lo && id < lo + kRuleChunk) sbias[id - lo] = a.bias_vals[e];
        if (blockIdx.x == 0 && (id < 0 || id >= a.V || (e > e0 && a.bias_ids[e - 1] >= id)))
          set_status(a.status, DSPARK_EINVAL);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kRuleIds; ++j) bias[j] = sbias[tid * kRuleIds + j];
    }
  }
  if (base >= a.V) return;  // V is a multiple of 8

  const float rho = a.repetition ? a.repetition[r] : 1.f;
  const float inv_rho = 1.f / rho;  // l / rho as a product: within 1.5 ulp of fp32 of the quotient
  const float freq = a.frequency ? a.frequency[r] : 0.f, pres = a.presence ? a.presence[r] : 0.f;
  int count[kRuleIds];
  uint32_t seen = 0, acts = 0;  // bit j: id j was seen; a rule but the mask can change id j
  float add[kRuleIds];
  auto weigh = [&](int j) {
    add[j] = bias[j] - freq * float(count[j]) - (count[j] > 0 ? pres : 0.f);
    if (add[j] != 0.f || ((seen >> j & 1u) && rho != 1.f)) acts |= 1u << j;
  };
  {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (a.hist) w = *reinterpret_cast<const uint4*>(a.hist + size_t(r) * a.V + base);
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < kRuleIds; ++j) {
      const uint32_t word = (h[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
      count[j] = int(word & 0x7FFFu);
      if (word) seen |= 1u << j;
      weigh(j);
    }
  }

  const T* src = static_cast<const T*>(a.logits) + size_t(row0) * a.V + base;
  T* dst = static_cast<T*>(a.out) + size_t(row0) * a.V + base;
  const uint8_t* mk = a.mask ? a.mask + size_t(row0) * a.mask_row_bytes + (base >> 3) : nullptr;
  for (int first = 0; first < row1 - row0; first += kRowBatch) {
    Pack8<T> x[kRowBatch];
    uint32_t allowed[kRowBatch];
    int drafted[kRowBatch];
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      const int i = first + b;
      allowed[b] = 0xFFu, drafted[b] = -1;
      if (i >= row1 - row0) continue;
      if (!a.in_place) x[b].load(src + size_t(i) * a.V);
      if (mk) allowed[b] = mk[size_t(i) * a.mask_row_bytes];
      if (a.hist && i > 0) drafted[b] = a.ids[row0 + i];
    }
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      const int i = first + b;
      if (i >= row1 - row0) break;
      if (a.hist && i > 0) {
        const int d = drafted[b] - base;
        if (d >= 0 && d < kRuleIds) {
#pragma unroll
          for (int j = 0; j < kRuleIds; ++j)
            if (j == d) {
              ++count[j];
              seen |= 1u << j;
              weigh(j);
            }
        }
        if (base == 0 && (drafted[b] < 0 || drafted[b] >= a.V)) set_status(a.status, DSPARK_EINVAL);
      }
      if (a.in_place) {
        if (acts == 0 && allowed[b] == 0xFFu) continue;  // nothing changes here
        x[b].load(src + size_t(i) * a.V);
      }
      float v[kRuleIds];
      x[b].get(v);
#pragma unroll
      for (int j = 0; j < kRuleIds; ++j) {
        float l = v[j];
        if (seen >> j & 1u) l *= l > 0.f ? inv_rho : rho;
        l += add[j];
        v[j] = allowed[b] >> j & 1u ? l : -INFINITY;
      }
      Pack8<T>::store(dst + size_t(i) * a.V, v);
    }
  }
}

// ---------------------------------------------------------------------------- history

constexpr int kHistThreads = 512;

// A block counts one request's tokens that fall into its `chunk` ids in shared memory (32-bit:
// a list can be longer than the 15-bit count) and writes the chunk once.
__global__ void __launch_bounds__(kHistThreads)
    history_build_kernel(const int32_t* __restrict__ tokens, int n_tokens, const int32_t* __restrict__ start,
                         const int32_t* __restrict__ n_prompt, int V, int chunk, int16_t* __restrict__ hist,
                         uint32_t* status) {
  extern __shared__ uint32_t cell[];
  pdl_enter();
  const int tid = threadIdx.x, r = blockIdx.y;
  const int lo = blockIdx.x * chunk, n = min(chunk, V - lo);
  for (int i = tid; i < n; i += kHistThreads) cell[i] = 0u;
  __syncthreads();
  int t0 = start[r], t1 = start[r + 1];
  if (t0 < 0 || t1 < t0 || t1 > n_tokens) {
    if (tid == 0 && blockIdx.x == 0) set_status(status, DSPARK_EINVAL);
    t0 = t1 = 0;
  }
  const int said0 = t0 + n_prompt[r];
  for (int t = t0 + tid; t < t1; t += kHistThreads) {
    const int id = tokens[t];
    const int d = id - lo;
    if (d >= 0 && d < n) {
      if (t < said0)
        atomicOr(&cell[d], 0x80000000u);
      else
        atomicAdd(&cell[d], 1u);
    }
    if (blockIdx.x == 0 && (id < 0 || id >= V)) set_status(status, DSPARK_EINVAL);
  }
  __syncthreads();
  uint32_t* out = reinterpret_cast<uint32_t*>(hist + size_t(r) * V + lo);
  auto word = [](uint32_t c) { return min(c & 0x7FFFFFFFu, 0x7FFFu) | (c >> 16 & 0x8000u); };
  for (int i = tid; 2 * i < n; i += kHistThreads) out[i] = word(cell[2 * i]) | word(cell[2 * i + 1]) << 16;
}

// One thread per committed token: a saturating add on its half of a 32-bit word.
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
  uint32_t* w = reinterpret_cast<uint32_t*>(hist) + (at >> 1);
  const int sh = int(at & 1) * 16;
  uint32_t old = *w;
  while (((old >> sh) & 0x7FFFu) != 0x7FFFu) {
    const uint32_t got = atomicCAS(w, old, old + (1u << sh));
    if (got == old) break;
    old = got;
  }
}

}  // namespace

cudaError_t launch_process_logits(const void* logits, int dtype, int rows, int V, const int32_t* cu,
                                  const int32_t* ids, int bs, const int16_t* hist, const float* repetition,
                                  const float* frequency, const float* presence, const int32_t* bias_start,
                                  const int32_t* bias_ids, const float* bias_vals, const uint32_t* mask, void* out,
                                  uint32_t* status, cudaStream_t s) {
  RuleArgs a;
  a.logits = logits, a.out = out, a.cu = cu, a.ids = ids, a.hist = hist;
  a.repetition = repetition, a.frequency = frequency, a.presence = presence;
  a.bias_start = bias_start, a.bias_ids = bias_ids, a.bias_vals = bias_vals;
  a.mask = reinterpret_cast<const uint8_t*>(mask);  // little-endian words: byte i holds ids 8i .. 8i+7
  a.status = status, a.rows = rows, a.V = V, a.mask_row_bytes = (V + 31) / 32 * 4;
  a.in_place = logits == out;
  const dim3 grid((V + kRuleChunk - 1) / kRuleChunk, bs);
  return dtype == DSPARK_F32 ? launch_pdl(rules_kernel<float>, grid, dim3(kRuleThreads), 0, s, a)
                             : launch_pdl(rules_kernel<__nv_bfloat16>, grid, dim3(kRuleThreads), 0, s, a);
}

cudaError_t launch_history_build(const int32_t* tokens, int n_tokens, const int32_t* start, const int32_t* n_prompt,
                                 int bs, int V, int16_t* hist, uint32_t* status, cudaStream_t s) {
  const int chunk = 2048;
  return launch_pdl(history_build_kernel, dim3((V + chunk - 1) / chunk, bs), dim3(kHistThreads),
                    chunk * sizeof(uint32_t), s, tokens, n_tokens, start, n_prompt, V, chunk, hist, status);
}

cudaError_t launch_history_commit(const int32_t* out_tokens, int bs, int gamma, int V, int16_t* hist, uint32_t* status,
                                  cudaStream_t s) {
  const int n = bs * (gamma + 1);
  return launch_pdl(history_commit_kernel, dim3((n + 127) / 128), dim3(128), 0, s, out_tokens, n, gamma + 1, V, hist,
                    status);
}

}  // namespace dspark
