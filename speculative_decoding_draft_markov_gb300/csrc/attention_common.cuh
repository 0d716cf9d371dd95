// What the two attention kernels share: the call's arguments, the KV tiles of a unit of work, how the work
// is cut over the CTAs, bounded waits, and the row masks.
//
// A unit of work is one KV head of one request and a run of its rows: the rows' query heads of that KV head
// are stacked into a tile of (token, head) rows, so that K and V are read once for all of them.  The
// work of a call, counted in KV tiles of 128 slots, is cut into one equal range per CTA (one CTA per SM),
// whatever the lengths are; a unit that crosses a cut leaves partial rows in the workspace, which a small
// kernel joins in a fixed order.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "pdl.h"
#include "tc_host.h"
#include "tc_ptx.cuh"

namespace dspark {
namespace attn {

constexpr int kTile = 128;  // KV slots per tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnArgs {
  int64_t cache_limit;  // positions that the page table can hold
  const int32_t *page_table, *cu, *ctx;
  __nv_bfloat16* out;
  float* lse;
  uint32_t *status, *diag;
  int4* info;       // per CTA: which partials it left (Info)
  float* partial;   // [2 grid][rows of a unit][D] partial outputs, normalised
  float* plse;      // [2 grid][rows of a unit] their log2-sum-exp
  uint64_t timeout_ns;
  float c2;         // scale * log2(e), never 0
  int max_pages, n_pages, page_shift, block_shift, bs, rows, Hq, Hkv, g, tokens, window, n_sink;
};

// What a CTA left for the join, as an int4: x = flags, then the unit that it began and did not finish.
enum : int { kTailUsed = 1, kTailEnds = 2, kHeadUsed = 4 };
// tail: the range began inside a unit (partial slot 2 cta); head: it ends inside one that it began (slot
// 2 cta + 1).  y = packed row of the unit's first token, z = its tokens, w = its KV head.

// The work of a call and where the range of this CTA begins.
struct Range {
  uint32_t pre[DSPARK_MAX_BS + 1];  // work before each request, in KV tiles
  int bad, n_long;
  int r, h, t, tile;
  uint32_t count;
};

// The KV tiles of one unit: its rows sit at positions p0 .. p1 and see, as a whole, the sinks and
// lo .. p1.  Its blocks (pages, or 128-slot pieces of larger pages) in order: sink blocks 0 .. sb - 1,
// then wb0 onwards.
struct Geom {
  int p0, p1, lo, sb, wb0, nblk, ntiles;
};

__device__ __forceinline__ Geom unit_geom(const AttnArgs& a, int c, int n, int t, int unit_tokens) {
  Geom u;
  u.p0 = c + t * unit_tokens;
  u.p1 = c + min((t + 1) * unit_tokens, n) - 1;
  u.lo = a.window ? max(0, u.p0 - a.window + 1) : 0;
  u.wb0 = u.lo >> a.block_shift;
  u.sb = a.window ? (min(a.n_sink, u.lo) + (1 << a.block_shift) - 1) >> a.block_shift : 0;
  if (u.sb >= u.wb0) u.sb = 0, u.wb0 = 0;  // the sinks' blocks meet the window's
  u.nblk = u.sb + (u.p1 >> a.block_shift) - u.wb0 + 1;
  u.ntiles = ((u.nblk << a.block_shift) + kTile - 1) / kTile;
  return u;
}
// Position of the first slot of block v of a unit.
__device__ __forceinline__ int block_pos(const AttnArgs& a, const Geom& u, int v) {
  return (v < u.sb ? v : v - u.sb + u.wb0) << a.block_shift;
}

struct Segment {
  Geom u;
  int r, h, row0, ntok;     // request, KV head, packed row of the unit's first token, its tokens
  int tile0, n;             // KV tiles tile0 .. tile0 + n - 1 of the unit
};

// Walks a CTA's range; every role walks the same one.
struct Walk {
  int r, h, t, tile, unit_tokens;
  uint32_t left;
  int loaded, row, n, c;
  __device__ Walk(const Range& g, int ut)
      : r(g.r), h(g.h), t(g.t), tile(g.tile), unit_tokens(ut), left(g.count), loaded(-1), row(0), n(0), c(0) {}
  __device__ __forceinline__ bool next(const AttnArgs& a, const Range& g, Segment& s) {
    if (left == 0) return false;
    while (g.pre[r + 1] == g.pre[r]) ++r;  // requests with nothing to do
    if (loaded != r) {
      row = a.cu[r];
      n = a.cu[r + 1] - row;
      c = a.ctx[r];
      loaded = r;
    }
    s.u = unit_geom(a, c, n, t, unit_tokens);
    s.r = r, s.h = h, s.row0 = row + t * unit_tokens, s.ntok = s.u.p1 - s.u.p0 + 1;
    s.tile0 = tile;
    s.n = int(min(left, uint32_t(s.u.ntiles - tile)));
    left -= uint32_t(s.n);
    tile += s.n;
    if (tile == s.u.ntiles) {
      tile = 0;
      if (++t * unit_tokens >= n) {
        t = 0;
        if (++h == a.Hkv) h = 0, ++r;
      }
    }
    return true;
  }
};

// A position in a ring of N slots.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) slot = 0, phase ^= 1;
  }
};

struct Waiter {
  volatile int* abort;
  uint64_t timeout_ns;
  // A whole warp waits; one answer for all lanes (false: given up).
  __device__ __forceinline__ bool operator()(const uint64_t* bar, uint32_t parity) const {
    const uint32_t b = tc::smem_u32(bar);
    bool ok = tc::mbar_try_wait(b, parity);
    if (!ok) ok = tc::mbar_wait_bounded(b, parity, tc::deadline_after_ns(timeout_ns), abort);
    return __all_sync(~0u, ok);
  }
};


// The range of this CTA: the call's KV tiles, counted over (request, KV head, unit), are cut into one
// equal range per CTA.  The whole block calls it (g.bad and g.n_long zeroed before); long_req: scratch
// of DSPARK_MAX_BS bytes.
__device__ __forceinline__ void plan_range(const AttnArgs& a, Range& g, uint8_t* long_req, int unit_tokens) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < a.bs) {
    const int r0 = a.cu[tid], r1 = a.cu[tid + 1], c = a.ctx[tid];
    uint32_t cost = 0;
    if (r0 < 0 || r1 < r0 || r1 > a.rows) {
      g.bad = 1;
    } else if (r1 > r0) {
      const int n = r1 - r0;
      if (c < 0 || int64_t(c) + n > a.cache_limit) {
        if (blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
      } else {
        const int nt = (n + unit_tokens - 1) / unit_tokens;
        if (nt > 4)  // many units: summed by the whole block below
          long_req[atomicAdd(&g.n_long, 1)] = uint8_t(tid);
        else
          for (int t = 0; t < nt; ++t) cost += unit_geom(a, c, n, t, unit_tokens).ntiles;
      }
    }
    g.pre[tid + 1] = cost;
  }
  if (tid == 0) g.pre[0] = 0;
  __syncthreads();
  for (int i = 0; i < g.n_long; ++i) {
    const int r = long_req[i], n = a.cu[r + 1] - a.cu[r], c = a.ctx[r];
    uint32_t part = 0;
    for (int t = tid; t * unit_tokens < n; t += int(blockDim.x)) part += unit_geom(a, c, n, t, unit_tokens).ntiles;
    part = __reduce_add_sync(~0u, part);
    if (lane == 0) atomicAdd(&g.pre[r + 1], part);
  }
  __syncthreads();
  if (warp == 0) {
    constexpr int kPer = DSPARK_MAX_BS / 32;
    long long x[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = lane * kPer + i;
      sum += r < a.bs && !g.bad ? static_cast<long long>(g.pre[r + 1]) * a.Hkv : 0;
      x[i] = sum;
    }
    long long before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, before, o);
      if (lane >= o) before += y;
    }
    const bool too_much = __shfl_sync(~0u, before, 31) >> 32 != 0;  // counted in 32 bits below
    before -= sum;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane * kPer + i < a.bs) g.pre[lane * kPer + i + 1] = too_much ? 0u : uint32_t(before + x[i]);
    __syncwarp();
    const long long total = g.pre[a.bs];
    const long long w0 = total * blockIdx.x / gridDim.x, w1 = total * (blockIdx.x + 1) / gridDim.x;
    int r = 0;
    for (int i = lane; i - lane < a.bs; i += 32) r += __popc(__ballot_sync(~0u, i < a.bs && g.pre[i + 1] <= w0));
    int h = 0, t = 0, tile = 0;
    if (w1 > w0) {
      const long long per_head = (g.pre[r + 1] - g.pre[r]) / a.Hkv;
      long long rem = w0 - g.pre[r];
      h = int(rem / per_head);
      rem -= h * per_head;
      const int n = a.cu[r + 1] - a.cu[r], c = a.ctx[r], nt = (n + unit_tokens - 1) / unit_tokens;
      for (int base = 0;; base += 32) {  // the unit that holds tile `rem` of this head
        const int mine = base + lane < nt ? unit_geom(a, c, n, base + lane, unit_tokens).ntiles : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(~0u, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(~0u, incl > rem);
        if (past != 0 || base + 32 >= nt) {
          const int at = past ? __ffs(past) - 1 : 31;
          t = base + at;
          tile = int(rem) - __shfl_sync(~0u, incl - mine, at);
          break;
        }
        rem -= __shfl_sync(~0u, incl, 31);
      }
    }
    if (lane == 0) {
      g.r = r, g.h = h, g.t = t, g.tile = tile;
      g.count = uint32_t(w1 - w0);
      if ((g.bad || too_much) && blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
    }
  }
  __syncthreads();
}

// One tile of a unit as the TMA warp loads it: lane i's block of the tile.
struct TileLoad {
  int page;      // as the page table has it
  int slot, head;
  int n_blocks;  // blocks of the tile
};
__device__ __forceinline__ TileLoad tile_load(const AttnArgs& a, const Segment& s, int j, int lane) {
  const int per_tile = kTile >> a.block_shift, v0 = (s.tile0 + j) * per_tile;
  TileLoad t;
  t.n_blocks = min(per_tile, s.u.nblk - v0);
  t.head = s.h;
  t.page = t.slot = 0;
  if (lane < t.n_blocks) {
    const int pos = block_pos(a, s.u, v0 + lane);
    t.slot = pos & ((1 << a.page_shift) - 1);
    t.page = a.page_table[int64_t(s.r) * a.max_pages + (pos >> a.page_shift)];
  }
  return t;
}
// Issue its loads into the tile at `dst` (column blocks of 64 lanes, 128-byte swizzled).
template <int kHalves>
__device__ __forceinline__ void issue_tile(const AttnArgs& a, const CUtensorMap* map, const TileLoad& t, uint32_t dst,
                                           uint32_t bar, uint64_t policy, int lane) {
  const int block_bytes = 128 << a.block_shift;
  if (lane == 0) tc::mbar_arrive_expect_tx(bar, uint32_t(t.n_blocks * block_bytes * kHalves));
  __syncwarp();
  if (lane >= t.n_blocks) return;
  int page = t.page;
  if (page < 0 || page >= a.n_pages) {
    set_status(a.status, DSPARK_EINVAL);
    page = a.n_pages;  // outside the tensor: reads as zeros
  }
#pragma unroll
  for (int hf = 0; hf < kHalves; ++hf)
    tc::tma_load_4d(dst + lane * block_bytes + hf * (kTile * 128), map, bar, hf * 64, t.slot, t.head, page, policy);
}

// Tiles j0 .. j1 - 1 of a segment whose every slot is seen by all rows at positions q0 .. q1 of the unit
// (q0 = p1, q1 = p0: by some row or other).
__device__ __forceinline__ void whole_tiles(const AttnArgs& a, const Segment& s, int q0, int q1, int& j0, int& j1) {
  const int per_tile = kTile >> a.block_shift, shift = s.u.sb - s.u.wb0;
  // in blocks of the unit: past the sinks and not before the window of q1; ending by q0
  int in0 = s.u.sb;
  if (a.window) in0 = max(in0, ((q1 - a.window + (1 << a.block_shift)) >> a.block_shift) + shift);
  const int in1 = ((q0 + 1) >> a.block_shift) + shift;
  j0 = (in0 + per_tile - 1) / per_tile - s.tile0, j1 = in1 / per_tile - s.tile0;
}

// Slots that no row of the unit sees hold whatever was there, NaN included, and 0 * NaN is NaN: their rows of
// the V tile are cleared.  A whole warp, 16-byte stores, rotated so that the lanes spread over the banks.
template <int kHalves>
__device__ __forceinline__ void clear_unseen(const AttnArgs& a, const Segment& s, int j, uint8_t* tile, int lane) {
  const int first = (s.tile0 + j) * (kTile >> a.block_shift);
  for (int i = lane; i < kTile; i += 32) {
    const int pos = block_pos(a, s.u, first + (i >> a.block_shift)) + (i & ((1 << a.block_shift) - 1));
    if (pos <= s.u.p1 && (pos >= s.u.lo || pos < a.n_sink)) continue;
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4*>(tile + i * 128 + hf * (kTile * 128) + (((k + lane) & 7) << 4)) =
            make_uint4(0u, 0u, 0u, 0u);
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
}
// The clearing warp and the warp that issues the product with V agree on the tiles that need it; their
// barriers are counted over those tiles alone (more barriers than V slots, so that neither can lap the other).
constexpr int kReady = 8;

}  // namespace attn

cudaError_t launch_attention_prompts(int D, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                     const attn::AttnArgs& a, int n_cta, cudaStream_t s);
cudaError_t launch_attention_windows(int D, int unit_rows, const CUtensorMap& q, const CUtensorMap& k,
                                     const CUtensorMap& v, const attn::AttnArgs& a, int n_cta, cudaStream_t s);

}  // namespace dspark
