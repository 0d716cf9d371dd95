// What the two attention kernels share: the call's arguments, the KV tiles of a unit of work, how the work
// is cut over the CTAs, bounded waits, and the row masks.
//
// A unit of work is one KV head of one request and a run of its rows: the rows' query heads of that KV head
// are stacked into a tile of (token, head) rows, so that K and V are read once for all of them.  The
// work of a call, counted in KV tiles of 128 slots, is cut into equal ranges, one or two per CTA (one CTA per
// SM), whatever the lengths are; a unit that crosses a cut leaves partial rows in the workspace, which a
// small kernel joins in a fixed order.
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
constexpr int kJoinTogether = 16;  // parts of a row that the join reads at a time, where they are many
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The exponentials' reference m (log2 units) before a row has one, and by how much a score may outgrow it before it moves
// and O and l are rescaled.  It costs range in O, which holds up to 2^16 n |v| for n positions: |v| of
// 2^90 is safe with 2^21 of them; scores hardly ever outgrow the first tile's by more.
constexpr float kUnset = -1e30f, kRescaleAt = 16.f;

struct AttnArgs {
  int64_t cache_limit;  // positions that the page table can hold
  const int32_t *page_table, *cu, *ctx;
  __nv_bfloat16* out;
  float* lse;
  uint32_t *status, *diag;
  int4* info;       // per range: the unit that it began and did not finish
  float* partial;   // [2 ranges][rows of a unit][D] partial outputs, normalised
  float* plse;      // [2 ranges][rows of a unit] their log2-sum-exp
  uint64_t timeout_ns;
  float c2;           // |scale| log2(e), never 0
  uint32_t negate_q;  // instruction descriptor bit: the first operand's sign, for a negative scale
  int max_pages, n_pages, page_shift, block_shift, bs, rows, Hq, Hkv, g, tokens, window, n_sink;
};

// What a range v leaves for the join.  Its rows of a unit that it began and did not finish are partial slot 2 v + 1,
// those of a unit that an earlier range began slot 2 v.  info[v] is the unit that it began and did not finish: x =
// how many ranges from v on have a part of it (0: there is no such unit), y = packed row of its first token,
// z = its tokens, w = its KV head.

// The KV tiles of one unit: its rows sit at positions p0 .. p1 and see, as a whole, the sinks and
// lo .. p1.  Its blocks (pages, or 32-slot pieces of larger pages) in order: sink blocks 0 .. sb - 1,
// then wb0 onwards.
struct Geom {
  int p0, p1, lo, sb, wb0, nblk, ntiles;
};

__host__ __device__ __forceinline__ Geom unit_geom(const AttnArgs& a, int c, int n, int t, int unit_tokens) {
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
__host__ __device__ __forceinline__ int block_pos(const AttnArgs& a, const Geom& u, int v) {
  return (v < u.sb ? v : v - u.sb + u.wb0) << a.block_shift;
}

struct Segment {
  Geom u;
  int r, h, row0, ntok;     // request, KV head, packed row of the unit's first token, its tokens
  int tile0, n;             // KV tiles tile0 .. tile0 + n - 1 of the unit
};

// Where a range begins: request (its first packed row, rows and tokens cached before), KV head, unit, KV tile.
struct Start {
  int r, h, t, tile, row, n, c;
  uint32_t count;  // KV tiles
};

// Walks a range; every role of a pipeline walks the same one.  After its end it stays at its end.
struct Walk {
  int r, h, t, tile, unit_tokens;
  uint32_t left;
  int loaded, row, n, c;
  __host__ __device__ Walk(const Start& g, int ut)
      : r(g.r), h(g.h), t(g.t), tile(g.tile), unit_tokens(ut), left(g.count), loaded(g.r), row(g.row), n(g.n), c(g.c) {}
  __host__ __device__ __forceinline__ bool next(const AttnArgs& a, Segment& s) {
    if (left == 0) return false;
    while (loaded != r) {  // the next request with something to do
      if (r >= a.bs) return false;
      row = a.cu[r];
      n = a.cu[r + 1] - row;
      c = a.ctx[r];
      if (n > 0 && c >= 0 && int64_t(c) + n <= a.cache_limit)
        loaded = r;
      else
        ++r;
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

// The tiles of a range one by one.  After the last tile `next` is false however often it is called.
struct Cursor {
  Walk walk;
  Segment s = {};
  int j = 0;
  __host__ __device__ Cursor(const Start& g, int unit_tokens) : walk(g, unit_tokens) {}
  __host__ __device__ __forceinline__ bool next(const AttnArgs& a) {
    if (j + 1 < s.n) {
      ++j;
      return true;
    }
    if (!walk.next(a, s)) return false;
    j = 0;
    return true;
  }
  __host__ __device__ __forceinline__ bool first() const { return j == 0; }
  __host__ __device__ __forceinline__ bool last() const { return j + 1 == s.n; }
};

// The order in which the tiles of a range are loaded: K 0, K 1, then V t, K t + 2.  fetch() describes the next tile
// (`there` false after the last, as often as it is asked), three tiles before its V is put; put_k and put_v say
// whether to go on.  Every load is waited for by the products, which take the same tiles in the same order.
#pragma nv_exec_check_disable
template <typename Fetch, typename PutK, typename PutV>
__host__ __device__ __forceinline__ bool load_in_order(Fetch fetch, PutK put_k, PutV put_v) {
  auto f0 = fetch(), f1 = fetch(), f2 = fetch(), f3 = fetch();
  bool ok = (!f0.there || put_k(f0)) && (!f1.there || put_k(f1));
  while (ok && f0.there) {
    ok = put_v(f0) && (!f2.there || put_k(f2));
    f0 = f1, f1 = f2, f2 = f3, f3 = fetch();
  }
  return ok;
}

// A position in a ring of N slots.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) slot = 0, phase ^= 1;
  }
};

// The parity of the phase in which a ring's slot was used last, after n > slot uses of the ring in order.
__host__ __device__ __forceinline__ uint32_t last_phase(int n, int slots, int slot) {
  return uint32_t((n - 1 - slot) / slots) & 1;
}
// A block whose roles gave up, whichever of them did, may not end with copies into its shared memory under way: wait
// (bounded) for the last one into each slot of a ring that n copies went to.
__device__ __forceinline__ void drain_copies(const uint64_t* full, int slots, int n, long long deadline) {
  const volatile int never = 0;
  for (int i = 0; i < min(n, slots); ++i)
    tc::mbar_wait_bounded(tc::smem_u32(&full[i]), last_phase(n, slots, i), deadline, &never);
}
constexpr uint64_t kDrainNs = 200000000ull;

// A whole warp waits; one answer for all lanes (false: given up).  The limit holds for each wait by itself: a
// call over a long cache may take its time.
struct Waiter {
  volatile int* abort;
  uint64_t timeout_ns;
  __device__ __forceinline__ bool operator()(const uint64_t* bar, uint32_t parity) const {
    const uint32_t b = tc::smem_u32(bar);
    bool ok = tc::mbar_try_wait(b, parity);
    if (!ok) ok = tc::mbar_wait_bounded(b, parity, tc::deadline_after_ns(timeout_ns), abort);
    return __all_sync(~0u, ok);
  }
};
// The same for the TMA warps.  try_wait itself sleeps for a while, so with a limit shorter than that they look
// instead, and the other warps learn of it by the abort flag.  (In the MMA warps' loops the longer code of this
// wait cost the prompts' kernel a tenth.)
struct TmaWaiter {
  Waiter wait;
  __device__ __forceinline__ bool operator()(const uint64_t* bar, uint32_t parity) const {
    if (wait.timeout_ns >= 1000000) return wait(bar, parity);
    const long long deadline = tc::deadline_after_ns(wait.timeout_ns);
    bool ok = tc::mbar_test_wait(tc::smem_u32(bar), parity);
    while (!ok && !*wait.abort && clock64() <= deadline) ok = tc::mbar_test_wait(tc::smem_u32(bar), parity);
    return __all_sync(~0u, ok);
  }
};

// The call's KV tiles, counted over (request, KV head, unit), are cut into kSets * gridDim.x ranges that differ
// by one tile at most; this CTA has ranges blockIdx.x + set * gridDim.x.
struct PlanScratch {
  long long warp_total[DSPARK_MAX_BS / 32];
  unsigned long long long_cost[DSPARK_MAX_BS];
  uint8_t long_req[DSPARK_MAX_BS];
  int n_long, bad;
};
// The whole block calls it, after one thread has cleared n_long, bad and the starts' counts and a
// __syncthreads; the starts are there after the next one.
struct Cut {
  uint32_t each, extra;  // tiles of a range, and how many ranges (the first) have one more
  // how many ranges from v on `tiles` tiles take
  __device__ __forceinline__ int ranges(uint32_t v, uint32_t tiles) const {
    const uint32_t big = v < extra ? extra - v : 0u;
    if (tiles <= big * (each + 1)) return int((tiles + each) / (each + 1));
    return int(big + (tiles - big * (each + 1) + each - 1) / each);
  }
};
template <int kSets>
__device__ __forceinline__ Cut plan_ranges(const AttnArgs& a, Start* start, PlanScratch& p, int unit_tokens) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int row = 0, n = 0, c = 0;
  uint32_t cost = 0;  // KV tiles of one KV head; from kTooMany on the call is refused
  constexpr uint32_t kTooMany = 1u << 31;
  bool is_long = false;
  if (tid < a.bs) {
    row = a.cu[tid], n = a.cu[tid + 1] - row, c = a.ctx[tid];
    if (row < 0 || n < 0 || row + n > a.rows) {
      p.bad = 1;
    } else if (n > 0) {
      if (c < 0 || int64_t(c) + n > a.cache_limit) {
        if (blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
      } else if (n > 4 * unit_tokens) {  // many units: summed by the whole block below
        is_long = true;
        p.long_cost[tid] = 0;
        p.long_req[atomicAdd(&p.n_long, 1)] = uint8_t(tid);
      } else {
        for (int t = 0; t * unit_tokens < n; ++t) cost += unit_geom(a, c, n, t, unit_tokens).ntiles;
      }
    }
  }
  __syncthreads();
  if (p.n_long > 0) {
    for (int i = 0; i < p.n_long; ++i) {
      const int r = p.long_req[i], rn = a.cu[r + 1] - a.cu[r], rc = a.ctx[r];
      unsigned long long part = 0;  // 2^20 rows over 2^29 positions pass 32 bits
      for (int t = tid; t * unit_tokens < rn; t += int(blockDim.x)) part += unit_geom(a, rc, rn, t, unit_tokens).ntiles;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(~0u, part, o);
      if (lane == 0) atomicAdd(&p.long_cost[r], part);
    }
    __syncthreads();
    if (is_long) cost = uint32_t(min(p.long_cost[tid], static_cast<unsigned long long>(kTooMany)));
  }
  const long long mine = p.bad ? 0 : static_cast<long long>(cost) * a.Hkv;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31 && warp < DSPARK_MAX_BS / 32) p.warp_total[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < DSPARK_MAX_BS / 32; ++i) {
    if (i < warp) before += p.warp_total[i];
    total += p.warp_total[i];
  }
  const bool too_much = total >= kTooMany;  // counted in 32 bits from here on
  if (tid == 0 && blockIdx.x == 0 && (p.bad || too_much)) set_status(a.status, DSPARK_EINVAL);
  const uint32_t all = too_much ? 0u : uint32_t(total);
  // A unit of T tiles in ranges of m has T / m parts, which the join reads kJoinTogether at a time, one trip to memory each, and
  // a trip takes about as long as a tile: m >= sqrt(T / kJoinTogether), T the mean over requests and KV heads.  GB300, one
  // token over 50000 positions, 1 KV head: 18.0 us, cut as finely as there are CTAs 30.3; 8 KV heads over 5000 14.2 and 16.4,
  // over 1500 the same.  Those batches are uniform: a long context among short ones is cut by the mean as well.
  const uint32_t least = max(1u, uint32_t(ceilf(sqrtf(float(all) / (float(a.Hkv) * float(a.bs * kJoinTogether))))));
  const uint32_t n_ranges = min(kSets * gridDim.x, (all + least - 1) / least), some = max(n_ranges, 1u);
  const uint32_t each = all / some, extra = all - each * some, first = uint32_t(before + incl - mine);
#pragma unroll
  for (int set = 0; set < kSets; ++set) {
    const uint32_t v = blockIdx.x + set * gridDim.x, w0 = each * v + min(v, extra);
    const uint32_t count = v < n_ranges ? each + (v < extra ? 1u : 0u) : 0u;
    if (count > 0 && w0 >= first && w0 - first < uint32_t(mine)) {  // this thread's request
      const uint32_t h = (w0 - first) / cost;
      start[set] = Start{tid, int(h), 0, int(w0 - first - h * cost), row, n, c, count};
    }
  }
  __syncthreads();
  if (warp < kSets && start[warp].count > 0 && start[warp].n > unit_tokens) {  // the unit that holds that tile of the head
    Start& g = start[warp];
    int rem = g.tile, t = 0;
    for (int base = 0;; base += 32) {
      const int tiles = (base + lane) * unit_tokens < g.n ? unit_geom(a, g.c, g.n, base + lane, unit_tokens).ntiles : 0;
      int sum = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t past = __ballot_sync(~0u, sum > rem);
      if (past != 0 || (base + 32) * unit_tokens >= g.n) {
        const int at = past ? __ffs(past) - 1 : 31;
        t = base + at;
        rem -= __shfl_sync(~0u, sum - tiles, at);
        break;
      }
      rem -= __shfl_sync(~0u, sum, 31);
    }
    __syncwarp();
    if (lane == 0) g.t = t, g.tile = rem;
  }
  return Cut{each, extra};
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
}  // namespace attn

// The most (token, head) rows of a unit of the short windows' kernel, and its ranges per CTA (partial rows in the workspace are
// per range).
constexpr int attention_window_rows(int D) { return D == 64 ? 64 : 128; }
int attention_window_sets(int D, int unit_rows);
cudaError_t launch_attention_prompts(int D, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                     const attn::AttnArgs& a, int n_cta, cudaStream_t s);
cudaError_t launch_attention_windows(int D, int unit_rows, const CUtensorMap& q, const CUtensorMap& k,
                                     const CUtensorMap& v, const attn::AttnArgs& a, int n_cta, cudaStream_t s);

}  // namespace dspark
