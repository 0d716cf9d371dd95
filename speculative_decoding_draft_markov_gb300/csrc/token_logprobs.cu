// dspark_token_logprobs: log probabilities of given tokens, with the rows' entropies, the tokens' ranks and the
// likeliest alternatives.
//
// One pass over the row: with d = (l - m) log2(e) / T and a reference m of the thread's own,
//     S = sum 2^d,  W = sum 2^d d      logprob of t = d_t - log2 S,  entropy = log2 S - W / S      (times ln 2)
// The alternatives come from a threshold that n ids at least reach: each warp's share of n among its lanes' maxima, the
// least over the warps.  Each thread keeps the maxima of four parts of its ids, so that only parts that reach the threshold,
// some dozen of 1024, are looked at again; what reaches it there (some dozen ids) is ranked by counting.
//
// GB300, V 151936, bf16, 761 tokens (256 windows of 1 to 8 rows) with rank and 20 alternatives: 69 us (34.6 by their bytes; 67.7 with
// d as one fma under a rounded m log2(e) / T, an error that grows with the logits); of tokens drawn evenly from the allowed ids,
// which many ids stand before, 78 (96 by comparing each of them twice).  Bound by
// instructions (12 or 13 a logit) that the SMs have unevenly: five blocks each on average, the busiest a third more.
// Slower, where this form took 70 to 73: half rows 78, quarters 90; equal ranges over persistent blocks 113; a second look for
// the rank too 94; 2 or 3 blocks an SM with eight loads ahead 79 and 71, 5 to 8 blocks 76 to 150; 512 threads 74 to 82; a maximum
// over two loads before the next are asked for 85.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "pdl.h"
#include "tc_host.h"
#include "tc_ptx.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kParts = 4;    // of a thread's ids, each with a maximum of its own
constexpr int kRoom = 512;   // ids that may reach the threshold; with more, the alternatives are found one by one
constexpr int kMaxSegments = 128;
constexpr float kSlack = 20.f;  // what d may grow to before m moves; at the end m is a thread's maximum
// Logits below -kPlain count as that, so that no mask's value (-inf times the weight 0 is NaN) needs care; a segment without
// any above it, or a temperature under which it would weigh something, is summed with care.
constexpr float kPlain = 0x1.9200000000000p+99f;  // 9.95e29, exact in bf16
constexpr float kLowest = -3.402823466e38f;  // m before there is a logit

struct LogprobArgs {
  const void* logits;
  const int32_t *cu, *tokens;
  float *logprob, *entropy;
  int32_t *rank, *top_ids;
  float* top_logprobs;
  uint32_t* status;
  float4* part;              // [items][segments]: m, S, W, and the ids before the token (as an int)
  unsigned long long* best;  // [items][segments][top_n] keys, 0: none
  float c2, slack;           // log2(e) / temperature; kSlack of it
  int rows, V, per, top_n, segments, segment;  // ids of a segment
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
    const int r = i / a.per, j = i - r * a.per, first = a.cu[r], end = a.cu[r + 1];
    ok = ok && first >= 0 && first <= end && end <= a.rows && j < end - first;
    row = ok ? first + j : 0;
  }
  if (ok)
    t.row = row;
  else if (reports)
    set_status(a.status, DSPARK_EINVAL);
  return t;
}

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

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The next number below a finite x, in fp32.
__device__ __forceinline__ float number_below(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // one zero
  return __uint_as_float(b == 0u ? 0x80000001u : b & 0x80000000u ? b + 1u : b - 1u);
}

template <typename T> struct Eight;  // 8 logits of a row
template <> struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ void raise() {  // to -kPlain at least; a NaN stays
    const uint32_t to = 0xF149F149u;
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.x) : "r"(to));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.y) : "r"(to));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.z) : "r"(to));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.w) : "r"(to));
  }
  __device__ void get(float* x) const {
    x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
  }
};
template <> struct Eight<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void raise() {
    a.x = max_or_nan(a.x, -kPlain), a.y = max_or_nan(a.y, -kPlain), a.z = max_or_nan(a.z, -kPlain), a.w = max_or_nan(a.w, -kPlain);
    b.x = max_or_nan(b.x, -kPlain), b.y = max_or_nan(b.y, -kPlain), b.z = max_or_nan(b.z, -kPlain), b.w = max_or_nan(b.w, -kPlain);
  }
  __device__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

// Sums of a row or of a part of it, under a reference of their own.
struct Sums {
  float m, s, w;
  int before;
};
__device__ __forceinline__ Sums joined(const Sums& a, const Sums& b, float c2) {
  const float m = a.m > b.m ? a.m : b.m;  // references are numbers or +inf
  const float da = (a.m - m) * c2, db = (b.m - m) * c2, fa = tc::ex2_approx(da), fb = tc::ex2_approx(db);
  // W under another reference is f (W + S d), where f is not 0
  const float wa = fa == 0.f ? 0.f : fa * fmaf(a.s, da, a.w), wb = fb == 0.f ? 0.f : fb * fmaf(b.s, db, b.w);
  return Sums{m, fmaf(a.s, fa, b.s * fb), wa + wb, a.before + b.before};
}
__device__ __forceinline__ Sums warp_joined(Sums v, float c2) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sums y{__shfl_xor_sync(~0u, v.m, o), __shfl_xor_sync(~0u, v.s, o), __shfl_xor_sync(~0u, v.w, o),
                 __shfl_xor_sync(~0u, v.before, o)};
    v = (threadIdx.x & o) ? joined(y, v, c2) : joined(v, y, c2);  // the same sum in both lanes
  }
  return v;
}

__device__ __forceinline__ void report_sums(const LogprobArgs& a, int64_t i, const Sums& t, float chosen) {
  const float log_sum = log2f(t.s);
  a.logprob[i] = ((chosen - t.m) * a.c2 - log_sum) * kLn2;
  if (a.entropy) a.entropy[i] = (log_sum - t.w / t.s) * kLn2;
  if (a.rank) a.rank[i] = 1 + t.before;
}
__device__ __forceinline__ void report_top(const LogprobArgs& a, int64_t at, unsigned long long key, const Sums& t) {
  a.top_ids[at] = key ? int(~uint32_t(key)) : -1;
  a.top_logprobs[at] = key ? ((value_of(key) - t.m) * a.c2 - log2f(t.s)) * kLn2 : -INFINITY;
}
__device__ __forceinline__ void report_nothing(const LogprobArgs& a, int64_t i, int tid, int threads) {
  if (tid == 0) {
    a.logprob[i] = 0.f;
    if (a.entropy) a.entropy[i] = 0.f;
    if (a.rank) a.rank[i] = 0;
  }
  for (int k = tid; k < a.top_n; k += threads) a.top_ids[i * a.top_n + k] = -1, a.top_logprobs[i * a.top_n + k] = -INFINITY;
}

struct Scan {
  Sums warp_sums[kWarps];
  float warp_least[kWarps];
  float most[kParts][kThreads];  // maxima
  unsigned long long key[kRoom], warp_key[kWarps];
  uint16_t reach[kParts * kThreads];  // the parts that reach the threshold
  int n_reach, n_key;
};

// A block takes one item's segment of the vocabulary.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ Scan sh;
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t i = blockIdx.x / uint32_t(a.segments);
  const int seg = int(blockIdx.x - i * a.segments);
  const Item it = item_of(a, int(i), tid == 0 && seg == 0);
  if (it.row < 0) {
    if (a.segments == 1) report_nothing(a, i, tid, kThreads);
    return;
  }
  if (tid == 0) sh.n_reach = sh.n_key = 0;
  const int lo = seg * a.segment, hi = min(a.V, lo + a.segment);  // multiples of 8
  const T* row = static_cast<const T*>(a.logits) + size_t(it.row) * a.V;
  const float chosen = ld_f32(row, it.token), chosen_raised = a.rank ? max_or_nan(chosen, -kPlain) : INFINITY;
  const float below = number_below(chosen);
  const int packs = (hi - lo) / 8, mine = (packs + kThreads - 1) / kThreads;  // of the segment, of a thread
  constexpr int kAhead = 4;
  const int part = ((mine + kParts - 1) / kParts + kAhead - 1) / kAhead * kAhead;
  const float c2 = a.c2;
  const unsigned long long cc = pack_f32x2(c2, c2);
  float m = kLowest, most = -INFINITY, all = -INFINITY;  // the largest of a part, of all
  int q = 0;
  unsigned long long s2 = 0ull, w2 = 0ull;
  int before = 0;
  auto refer = [&](float top) {  // a new reference
    const float d = (m - top) * c2, f = tc::ex2_approx(d);
    float s0, s1, w0, w1;
    unpack_f32x2(s2, s0, s1);
    unpack_f32x2(w2, w0, w1);
    w0 = f == 0.f ? 0.f : f * fmaf(s0, d, w0), w1 = f == 0.f ? 0.f : f * fmaf(s1, d, w1);
    s2 = pack_f32x2(s0 * f, s1 * f), w2 = pack_f32x2(w0, w1), m = top;
  };
  if (a.top_n > 0)
    for (int k = 0; k < kParts; ++k) sh.most[k][tid] = -INFINITY;
  Eight<T> x[kAhead];
#pragma unroll
  for (int b = 0; b < kAhead; ++b)
    if (b * kThreads + tid < packs) x[b].load(row + lo + (b * kThreads + tid) * 8);
#pragma unroll 1
  for (int k0 = 0; k0 < mine; k0 += kAhead) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int p = (k0 + b) * kThreads + tid, next = p + kAhead * kThreads;
      if (p >= packs) break;
      float l[8];
      x[b].raise();
      x[b].get(l);
      if (next < packs) x[b].load(row + lo + next * 8);
      const float top = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
      most = fmaxf(most, top);
      if (top > m + a.slack && top > -kPlain) refer(top);
      if (top >= chosen_raised) {
        const int id0 = lo + p * 8;
        if (chosen_raised > -kPlain && (id0 > it.token || id0 + 8 <= it.token)) {
          // how many lie above the logit, or the number below it (ids before the token stand before it with its own logit
          // too): by the differences' signs; a NaN's is positive
          const float over = id0 > it.token ? chosen + 0.f : below;
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float d0, d1;
            unpack_f32x2(fma_f32x2(pack_f32x2(l[j], l[j + 1]), pack_f32x2(-1.f, -1.f), pack_f32x2(over, over)), d0, d1);
            before += int(__float_as_uint(d0) >> 31), before += int(__float_as_uint(d1) >> 31);
          }
        } else {
          Eight<T> raw = {};  // as they are, not raised
          raw.load(row + id0);
          float r[8];
          raw.get(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) before += r[j] > chosen || (r[j] == chosen && id0 + j < it.token);
        }
      }
      const float neg = m == kLowest ? 0.f : -m;  // nothing but raised ones so far: they weigh nothing
      const unsigned long long mm = pack_f32x2(neg, neg);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float d0, d1;
        // the difference first: under a rounded m c2, d would be off by up to 2^-24 |m| / T
        const unsigned long long d = mul_f32x2(add_f32x2(pack_f32x2(l[j], l[j + 1]), mm), cc);
        unpack_f32x2(d, d0, d1);
        const unsigned long long e = pack_f32x2(tc::ex2_approx(d0), tc::ex2_approx(d1));
        s2 = add_f32x2(s2, e);
        w2 = fma_f32x2(e, d, w2);
      }
    }
    if (k0 + kAhead == (q + 1) * part || k0 + kAhead >= mine) {
      if (a.top_n > 0) sh.most[q][tid] = most;
      all = fmaxf(all, most), most = -INFINITY;
      ++q;
    }
  }
  if (all > m && all > -kPlain) refer(all);
  const bool some = __syncthreads_or(all > -kPlain), huge = __syncthreads_or(all >= kPlain);
  if (!some || huge || c2 * kPlain < 400.f || c2 > 1e7f) {  // (c2 beyond: d would overflow, and 0 * -inf is NaN)
    m = kLowest, s2 = w2 = 0ull;
    float high = -INFINITY;
    for (int p = tid; p < packs; p += kThreads) {
      float l[8];
      x[0].load(row + lo + p * 8);
      x[0].get(l);
      const float top = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
      high = fmaxf(high, top);
      if (top > m + a.slack) refer(top);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float d0 = max_or_nan((l[j] - m) * c2, -200.f), d1 = max_or_nan((l[j + 1] - m) * c2, -200.f);  // 2^-200 is 0
        const unsigned long long e = pack_f32x2(tc::ex2_approx(d0), tc::ex2_approx(d1));
        s2 = add_f32x2(s2, e);
        w2 = fma_f32x2(e, pack_f32x2(d0, d1), w2);
      }
    }
    if (high > m) refer(high);
  }
  float s0, s1, w0, w1;
  unpack_f32x2(s2, s0, s1);
  unpack_f32x2(w2, w0, w1);
  Sums t = warp_joined(Sums{m, s0 + s1, w0 + w1, before}, c2);
  if (lane == 0) sh.warp_sums[warp] = t;
  const int n = a.top_n;
  if (n > 0) {
    // a value that the warp's share of n lanes reach
    float best = fmaxf(fmaxf(sh.most[0][tid], sh.most[1][tid]), fmaxf(sh.most[2][tid], sh.most[3][tid])), least = -INFINITY;
    static_assert(kParts == 4, "parts");
    for (int k = 0; k < (n + kWarps - 1) / kWarps; ++k) {
      asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(least) : "f"(best));
      const uint32_t who = __ballot_sync(~0u, best == least);
      if (who == 0 || least == -INFINITY) break;
      if (lane == __ffs(who) - 1) best = -INFINITY;
    }
    if (lane == 0) sh.warp_least[warp] = least;
  }
  __syncthreads();
  t = sh.warp_sums[0];
#pragma unroll
  for (int k = 1; k < kWarps; ++k) t = joined(t, sh.warp_sums[k], c2);
  const bool whole = a.segments == 1;
  if (tid == 0) {
    if (whole)
      report_sums(a, i, t, chosen);
    else
      a.part[i * a.segments + seg] = make_float4(t.m, t.s, t.w, __int_as_float(t.before));
  }
  if (n == 0) return;
  float least = sh.warp_least[0];
#pragma unroll
  for (int k = 1; k < kWarps; ++k) least = fminf(least, sh.warp_least[k]);
  if (least <= -kPlain) least = -INFINITY;  // raised: what it was is to be seen
#pragma unroll
  for (int q = 0; q < kParts; ++q) {
    const bool in = sh.most[q][tid] >= least && sh.most[q][tid] > -INFINITY;
    const uint32_t all = __ballot_sync(~0u, in);
    int at = 0;
    if (lane == 0 && all) at = atomicAdd(&sh.n_reach, __popc(all));
    at = __shfl_sync(~0u, at, 0) + __popc(all & ((1u << lane) - 1u));
    if (in) sh.reach[at] = uint16_t(q * kThreads + tid);
  }
  __syncthreads();
  const int looks = sh.n_reach * part;
  for (int k = tid; k < looks; k += kThreads) {
    const int what = sh.reach[k / part], q = what / kThreads;
    const int kk = q * part + k % part, p = kk * kThreads + what % kThreads;
    if (kk >= mine || p >= packs) continue;
    Eight<T> x;
    x.load(row + lo + p * 8);
    float l[8];
    x.get(l);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (l[j] >= least && l[j] > -INFINITY) {
        const int at = atomicAdd(&sh.n_key, 1);
        if (at < kRoom) sh.key[at] = key_of(l[j], lo + p * 8 + j);
      }
  }
  __syncthreads();
  const int found = sh.n_key;
  auto give = [&](int place, unsigned long long key) {
    if (whole)
      report_top(a, i * n + place, key, t);
    else
      a.best[(i * a.segments + seg) * n + place] = key;
  };
  if (found <= kRoom) {
    for (int k = tid; k < found; k += kThreads) {
      const unsigned long long key = sh.key[k];
      int place = 0;
      for (int j = 0; j < found; ++j) place += sh.key[j] > key;
      if (place < n) give(place, key);
    }
    for (int k = found + tid; k < n; k += kThreads) give(k, 0ull);
    return;
  }
  // More ids reach the threshold than there is room for: one alternative after the other, over the whole segment.  The threshold is the
  // least of eight warps', so a warp without a logit above -kPlain leaves every id that is a number: rows of less than some 2000 ids,
  // and masks that leave no id to a warp (few allowed ids, or ids side by side) where more than kRoom numbers are left, as beside a
  // mask of finite value.  GB300, V 151936, 761 rows, 5 / 20 alternatives: 10 allowed ids beside -1e9 719 / 2108 us, 1000 side by
  // side beside -infinity 635 / 2035; scattered 110 / 114, 10 beside -infinity 148 / 148, no mask 72 / 76.  One row 15 / 33, no mask
  // 9.4 / 12.5.  16 rows of 1000 ids 7.5 (of 2200 5.2).
  unsigned long long last = ~0ull;
  for (int k = 0; k < n; ++k) {
    unsigned long long best = 0;
    for (int p = tid; p < packs; p += kThreads) {
      Eight<T> x;
      x.load(row + lo + p * 8);
      float l[8];
      x.get(l);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned long long key = key_of(l[j], lo + p * 8 + j);
        if (key < last && key > best) best = key;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(~0u, best, o));
    __syncthreads();
    if (lane == 0) sh.warp_key[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = max(best, sh.warp_key[w]);
    last = best;
    if (tid == 0) give(k, best);
  }
}

// Joins an item's segments: their sums in order, and n times the largest of their lists' heads.
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) logprobs_join_kernel(const __grid_constant__ LogprobArgs a, int dtype) {
  extern __shared__ __align__(16) unsigned long long list[];  // [segments][top_n]
  __shared__ float4 part[kMaxSegments];
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, n = a.top_n, S = a.segments;
  const int64_t i = blockIdx.x;
  const Item it = item_of(a, int(i), false);
  if (it.row < 0) {
    report_nothing(a, i, tid, kJoinThreads);
    return;
  }
  for (int k = tid; k < S; k += kJoinThreads) part[k] = a.part[i * S + k];
  for (int k = tid; k < S * n; k += kJoinThreads) list[k] = a.best[i * S * n + k];
  const size_t at = size_t(it.row) * a.V + it.token;
  const float chosen = dtype == DSPARK_F32 ? static_cast<const float*>(a.logits)[at]
                                           : ld_f32(static_cast<const __nv_bfloat16*>(a.logits), at);
  __syncthreads();
  if (tid >= 32) return;
  Sums t{kLowest, 0.f, 0.f, 0};
  for (int k = lane; k < S; k += 32) t = joined(t, Sums{part[k].x, part[k].y, part[k].z, __float_as_int(part[k].w)}, a.c2);
  t = warp_joined(t, a.c2);
  if (lane == 0) report_sums(a, i, t, chosen);
  constexpr int kHeads = kMaxSegments / 32;
  int head[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) head[h] = 0;
  unsigned long long mine = 0;  // the key of rank `lane`
  for (int k = 0; k < n; ++k) {
    unsigned long long best = 0;
    int from = -1;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      const int seg = h * 32 + lane;
      const unsigned long long key = seg < S && head[h] < n ? list[seg * n + head[h]] : 0ull;
      if (key > best) best = key, from = h;
    }
    const uint32_t high = __reduce_max_sync(~0u, uint32_t(best >> 32));
    const uint32_t low = __reduce_max_sync(~0u, uint32_t(best >> 32) == high ? uint32_t(best) : 0u);
    const unsigned long long top = (static_cast<unsigned long long>(high) << 32) | low;
    if (top != 0 && top == best) {
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h == from) ++head[h];
    }
    if (lane == k) mine = top;
  }
  if (lane < n) report_top(a, i * n + lane, mine, t);
}
static_assert(DSPARK_MAX_TOP <= 32, "a lane has one alternative");

// How many segments a row is cut into: as many as it takes to fill the SMs, of 6144 ids at least.  GB300, 16 rows of 151936 with
// 20 alternatives 14.9 us, by 2048 ids 17.3, by 12288 14.6; one row with 5 alternatives 8.6, 8.6 and 8.8; one row of 8000 5.3, cut
// in three 7.8.
int most_segments(int V) { return std::min(kMaxSegments, std::max(1, V / (24 * kThreads))); }
int segments_of(int items, int V) {
  const int most = most_segments(V);
  return std::max(1, std::min(most, 4 * tch::sm_count() / items));
}

}  // namespace

size_t token_logprobs_ws_bytes(int items, int V, int top_n) {
  size_t most = 256;
  // any number of items up to that: fewer are cut into more segments
  const size_t parts = std::min(size_t(items) * most_segments(V), std::max(size_t(items), size_t(4) * tch::sm_count()));
  most += align256(parts * sizeof(float4)) + align256(parts * top_n * sizeof(unsigned long long));
  return most;
}

cudaError_t launch_token_logprobs(const void* logits, int dtype, int rows, int V, const int32_t* cu, int bs,
                                  const int32_t* tokens, int per, float temperature, float* logprob, float* entropy,
                                  int32_t* rank, int32_t* top_ids, float* top_logprobs, int top_n, void* ws,
                                  cudaStream_t s) {
  LogprobArgs a;
  const int items = bs * per;
  a.logits = logits, a.cu = cu, a.tokens = tokens, a.logprob = logprob, a.entropy = entropy, a.rank = rank;
  a.top_ids = top_ids, a.top_logprobs = top_logprobs, a.status = static_cast<uint32_t*>(ws);
  a.c2 = kLog2e / temperature, a.slack = std::min(kSlack / a.c2, 1e37f), a.rows = rows, a.V = V, a.per = per, a.top_n = top_n;
  a.segments = segments_of(items, V);
  a.segment = ((V + a.segments - 1) / a.segments + 7) / 8 * 8;
  a.segments = (V + a.segment - 1) / a.segment;
  char* w = static_cast<char*>(ws) + 256;
  a.part = reinterpret_cast<float4*>(w);
  a.best = reinterpret_cast<unsigned long long*>(w + align256(size_t(items) * a.segments * sizeof(float4)));
  const dim3 grid(a.segments * items);
  const cudaError_t e = dtype == DSPARK_F32
                            ? launch_pdl(logprobs_kernel<float>, grid, dim3(kThreads), 0, s, a)
                            : launch_pdl(logprobs_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, a);
  if (e != cudaSuccess || a.segments == 1) return e;
  return launch_pdl(logprobs_join_kernel, dim3(items), dim3(kJoinThreads),
                    size_t(a.segments) * std::max(top_n, 1) * sizeof(unsigned long long), s, a, dtype);
}

}  // namespace dspark
