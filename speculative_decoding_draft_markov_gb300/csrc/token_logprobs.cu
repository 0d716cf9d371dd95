// dspark_token_logprobs: log probabilities of given tokens, with the rows' entropies, the tokens' ranks and the
// likeliest alternatives.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "pdl.h"

namespace dspark {
namespace {

struct LogprobArgs {
  const void* logits;
  const int32_t *cu, *tokens;
  float *logprob, *entropy;
  int32_t *rank, *top_ids;
  float* top_logprobs;
  uint32_t* status;
  float by;  // 1 / temperature
  int rows, V, per, top_n;
};

// The packed row of item i and its token; row < 0: the item reports nothing.
struct Item {
  int row, token;
};
__device__ __forceinline__ Item item_of(const LogprobArgs& a, int i, bool reports) {
  Item t{-1, a.tokens[i]};
  if (t.token == -1) return t;
  int row = i;
  bool ok = t.token >= 0 && t.token < a.V;
  if (a.cu) {
    const int r = i / a.per, first = a.cu[r], end = a.cu[r + 1];
    row = first + (i - r * a.per);
    ok = ok && first >= 0 && end <= a.rows && row < end;
  }
  if (ok)
    t.row = row;
  else if (reports)
    set_status(a.status, DSPARK_EINVAL);
  return t;
}

constexpr int kThreads = 512;

// A value and its id as one number that orders by value, then by the lower id; 0: nothing (NaN and -inf among it).
__device__ __forceinline__ unsigned long long key_of(float x, int id) {
  if (!(x > -INFINITY)) return 0ull;
  const uint32_t b = __float_as_uint(x + 0.f);  // one zero
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(o) << 32) | uint32_t(~id);
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const uint32_t o = uint32_t(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ unsigned long long warp_top(unsigned long long k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(~0u, k, o);
    k = y > k ? y : k;
  }
  return k;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ float scratch[kThreads / 32];
  __shared__ unsigned long long keys[kThreads / 32];
  pdl_enter();
  const int tid = threadIdx.x, i = blockIdx.x;
  const Item it = item_of(a, i, tid == 0);
  if (it.row < 0) {
    if (tid == 0) {
      a.logprob[i] = 0.f;
      if (a.entropy) a.entropy[i] = 0.f;
      if (a.rank) a.rank[i] = 0;
    }
    for (int k = tid; k < a.top_n; k += kThreads)
      a.top_ids[int64_t(i) * a.top_n + k] = -1, a.top_logprobs[int64_t(i) * a.top_n + k] = -INFINITY;
    return;
  }
  const T* x = static_cast<const T*>(a.logits) + size_t(it.row) * a.V;
  const float chosen = ld_f32(x, it.token);
  float top = -INFINITY;
  bool nan = false;
  for (int v = tid; v < a.V; v += kThreads) {
    const float l = ld_f32(x, v);
    top = fmaxf(top, l), nan |= l != l;
  }
  top = block_max<kThreads>(top, scratch);
  if (__syncthreads_or(nan)) top = __uint_as_float(0x7FFFFFFFu);
  float sum = 0.f, dot = 0.f, ahead = 0.f;
  for (int v = tid; v < a.V; v += kThreads) {
    const float l = ld_f32(x, v), d = (l - top) * a.by, w = expf(d);
    sum += w;
    dot += w == 0.f ? 0.f : w * d;
    ahead += l > chosen || (l == chosen && v < it.token) ? 1.f : 0.f;
  }
  sum = block_sum<kThreads>(sum, scratch);
  __syncthreads();
  dot = block_sum<kThreads>(dot, scratch);
  __syncthreads();
  ahead = block_sum<kThreads>(ahead, scratch);
  const float log_sum = logf(sum);
  if (tid == 0) {
    a.logprob[i] = (chosen - top) * a.by - log_sum;
    if (a.entropy) a.entropy[i] = log_sum - dot / sum;
    if (a.rank) a.rank[i] = 1 + int(ahead);
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.top_n; ++k) {
    unsigned long long best = 0;
    for (int v = tid; v < a.V; v += kThreads) {
      const unsigned long long key = key_of(ld_f32(x, v), v);
      if (key < last && key > best) best = key;
    }
    best = warp_top(best);
    __syncthreads();
    if ((tid & 31) == 0) keys[tid >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) best = max(best, keys[w]);
    last = best;
    if (tid == 0) {
      const int64_t at = int64_t(i) * a.top_n + k;
      a.top_ids[at] = best ? int(~uint32_t(best)) : -1;
      a.top_logprobs[at] = best ? (value_of(best) - top) * a.by - log_sum : -INFINITY;
    }
  }
}

}  // namespace

size_t token_logprobs_ws_bytes(int items, int V, int top_n) { return 256; }

cudaError_t launch_token_logprobs(const void* logits, int dtype, int rows, int V, const int32_t* cu, int bs,
                                  const int32_t* tokens, int per, float temperature, float* logprob, float* entropy,
                                  int32_t* rank, int32_t* top_ids, float* top_logprobs, int top_n, void* ws,
                                  cudaStream_t s) {
  LogprobArgs a;
  a.logits = logits, a.cu = cu, a.tokens = tokens, a.logprob = logprob, a.entropy = entropy, a.rank = rank;
  a.top_ids = top_ids, a.top_logprobs = top_logprobs, a.status = static_cast<uint32_t*>(ws);
  a.by = 1.f / temperature, a.rows = rows, a.V = V, a.per = per, a.top_n = top_n;
  const dim3 grid(bs * per);
  return dtype == DSPARK_F32 ? launch_pdl(logprobs_kernel<float>, grid, dim3(kThreads), 0, s, a)
                             : launch_pdl(logprobs_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace dspark
