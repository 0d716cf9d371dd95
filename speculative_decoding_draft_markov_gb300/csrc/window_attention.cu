// dspark_window_attention: attention of the packed rows over the paged cache, on the tensor cores.
//
// A unit of work is one KV head of one request and a run of its rows: the rows' query heads of that
// KV head are stacked into a tile of 128 (token, head) rows, so that a K or V tile is read once for
// all of them.  Per KV tile of 128 slots
//     S = Q K^T (tcgen05, fp32 in TMEM)  ->  P = exp2(c S - m), running m and l = sum P (registers)
//     O += P V  (tcgen05, P in bf16 in TMEM, O in fp32 in TMEM)
// with one thread per row.  m is only a reference that keeps the exponentials in range: it moves (and O
// and l are rescaled) when a row's maximum has outgrown it by 2^8, which is exact in the end because the
// sum is divided out.
//
// Two streams of tiles A and B keep the tensor cores busy while the other's softmax runs.  Short windows
// (kPair false): one Q tile, A and B take alternate KV tiles and their sums are merged at the end of
// the unit.  Prompts (kPair true): two Q tiles that read the same KV tiles.
//
// The work of the whole call, counted in KV tiles, is cut into one equal range per CTA (one CTA per SM),
// whatever the lengths are: a unit that crosses a cut leaves partial rows in the workspace, which a
// second small kernel joins in a fixed order.
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

constexpr int kThreads = 384;  // warps 0-3: softmax A, 4-7: softmax B, 8: TMA, 9: MMA, 10 and 11: idle
// Registers: launched with 384 x 168; the softmax warps hold a whole row of S and take what the others
// give back (256 x 208 + 128 x 80 <= 384 x 168).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
constexpr int kTile = 128;     // KV slots per tile, and rows of a Q tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleAt = 8.f;  // log2 of how far a row's maximum may outgrow its reference

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;              // 128-byte swizzled column blocks of a row
  static constexpr int kHalfBytes = kTile * 128;      // one column block of a tile
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kSlots = D == 128 ? 5 : 10;    // ring of K and V tiles: 160 KB either way
};

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

struct Shared {
  uint64_t q_full[2], q_empty[2], kv_full[10], kv_empty[10], s_full[2], p_full[2], o_full[2], m_full, m_empty, drain;
  float2 ml[kTile];  // (m, l) of stream B's rows, for the merge
  uint32_t pre[DSPARK_MAX_BS + 1];  // work before each request, in KV tiles
  uint32_t tmem_base;
  volatile int abort;
  int bad, n_long, mma_pending;
  int r, h, t, tile;  // where this CTA's range begins
  uint32_t count;
  uint8_t long_req[DSPARK_MAX_BS];
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
  __device__ Walk(const Shared* sh, int ut) : r(sh->r), h(sh->h), t(sh->t), tile(sh->tile), unit_tokens(ut),
                                              left(sh->count), loaded(-1), row(0), n(0), c(0) {}
  __device__ __forceinline__ bool next(const AttnArgs& a, const Shared* sh, Segment& s) {
    if (left == 0) return false;
    while (sh->pre[r + 1] == sh->pre[r]) ++r;  // requests with nothing to do
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

// Bits k = 0 .. 7 with lo <= k <= hi.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  const uint32_t below = hi >= 7 ? 0xFFu : hi < 0 ? 0u : (2u << hi) - 1u;
  const uint32_t from = lo <= 0 ? 0xFFu : lo > 7 ? 0u : 0xFFu << lo;
  return below & from;
}

template <int D, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                            // two Q tiles
  uint8_t* sKV = smem + 2 * C::kTileBytes;       // ring
  Shared* sh = reinterpret_cast<Shared*>(sKV + C::kSlots * C::kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit_tokens = kPair ? 2 * a.tokens : a.tokens;
  const int tile_rows = a.tokens * a.g;
  const int active = (tile_rows + 31) / 32;      // softmax warps of a stream that hold rows
  const Waiter wait{&sh->abort, a.timeout_ns};

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->q_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->q_empty[i]), kPair ? 1 : active);
      tc::mbar_init(tc::smem_u32(&sh->s_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->p_full[i]), active);
      tc::mbar_init(tc::smem_u32(&sh->o_full[i]), 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->kv_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->kv_empty[i]), 1);
    }
    tc::mbar_init(tc::smem_u32(&sh->m_full), active);
    tc::mbar_init(tc::smem_u32(&sh->m_empty), active);
    tc::mbar_init(tc::smem_u32(&sh->drain), 1);
    tc::fence_mbar_init();
    sh->abort = 0, sh->bad = 0, sh->n_long = 0, sh->mma_pending = 0;
    tc::prefetch_tensormap(&map_q);
    tc::prefetch_tensormap(&map_k);
    tc::prefetch_tensormap(&map_v);
  }
  if (warp == 9) {
    tc::tmem_alloc(tc::smem_u32(&sh->tmem_base), 512);
    tc::tmem_relinquish();
  }
  __syncthreads();
  pdl_enter();

  // ------------------------------------------------------------- the range of this CTA
  if (tid < a.bs) {
    const int r0 = a.cu[tid], r1 = a.cu[tid + 1], c = a.ctx[tid];
    uint32_t cost = 0;
    if (r0 < 0 || r1 < r0 || r1 > a.rows) {
      sh->bad = 1;
    } else if (r1 > r0) {
      const int n = r1 - r0;
      if (c < 0 || int64_t(c) + n > a.cache_limit) {
        if (blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
      } else {
        const int nt = (n + unit_tokens - 1) / unit_tokens;
        if (nt > 4)  // many units: summed by the whole block below
          sh->long_req[atomicAdd(&sh->n_long, 1)] = uint8_t(tid);
        else
          for (int t = 0; t < nt; ++t) cost += unit_geom(a, c, n, t, unit_tokens).ntiles;
      }
    }
    sh->pre[tid + 1] = cost;
  }
  if (tid == 0) sh->pre[0] = 0;
  __syncthreads();
  for (int i = 0; i < sh->n_long; ++i) {
    const int r = sh->long_req[i], n = a.cu[r + 1] - a.cu[r], c = a.ctx[r];
    uint32_t part = 0;
    for (int t = tid; t * unit_tokens < n; t += kThreads) part += unit_geom(a, c, n, t, unit_tokens).ntiles;
    part = __reduce_add_sync(~0u, part);
    if (lane == 0) atomicAdd(&sh->pre[r + 1], part);
  }
  __syncthreads();
  if (warp == 0) {
    constexpr int kPer = DSPARK_MAX_BS / 32;
    long long x[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = lane * kPer + i;
      sum += r < a.bs && !sh->bad ? static_cast<long long>(sh->pre[r + 1]) * a.Hkv : 0;
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
      if (lane * kPer + i < a.bs) sh->pre[lane * kPer + i + 1] = too_much ? 0u : uint32_t(before + x[i]);
    __syncwarp();
    const long long total = sh->pre[a.bs];
    const long long w0 = total * blockIdx.x / gridDim.x, w1 = total * (blockIdx.x + 1) / gridDim.x;
    int r = 0;
    for (int i = lane; i - lane < a.bs; i += 32) r += __popc(__ballot_sync(~0u, i < a.bs && sh->pre[i + 1] <= w0));
    int h = 0, t = 0, tile = 0;
    if (w1 > w0) {
      const long long per_head = (sh->pre[r + 1] - sh->pre[r]) / a.Hkv;
      long long rem = w0 - sh->pre[r];
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
      sh->r = r, sh->h = h, sh->t = t, sh->tile = tile;
      sh->count = uint32_t(w1 - w0);
      if ((sh->bad || too_much) && blockIdx.x == 0) set_status(a.status, DSPARK_EINVAL);
    }
  }
  __syncthreads();
  const uint32_t tmem = sh->tmem_base;

  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 8) {
    // --------------------------------------------------------------------- TMA producer
    const uint64_t policy = kPair ? tc::policy_evict_last() : tc::policy_evict_first();
    const int per_tile = kTile >> a.block_shift;  // blocks in a tile
    const int block_bytes = 128 << a.block_shift;
    int slot = 0, seg_i = 0, flags = 0;
    uint32_t phase = 0;
    int q_issued[2] = {-1, -1};
    uint32_t issued = 0;  // slots that hold or held a load
    int4 info = make_int4(0, 0, 0, 0);
    bool ok = true;
    Walk walk(sh, unit_tokens);
    Segment s = {};
    // the page of this lane's block of tile j: loaded a tile ahead of its use
    auto page_of = [&](int j) {
      const int v = (s.tile0 + j) * per_tile + lane;
      if (lane >= per_tile || v >= s.u.nblk || j >= s.n) return -2;  // no block
      const int pos = block_pos(a, s.u, v);
      const int pg = a.page_table[int64_t(s.r) * a.max_pages + (pos >> a.page_shift)];
      if (pg < 0 || pg >= a.n_pages) {
        set_status(a.status, DSPARK_EINVAL);
        return a.n_pages;  // outside the tensor: reads as zeros
      }
      return pg;
    };
    auto load = [&](const CUtensorMap* map, int j, int pg) {
      if (!wait(&sh->kv_empty[slot], phase ^ 1)) return false;
      const uint32_t bar = tc::smem_u32(&sh->kv_full[slot]);
      const int n_blocks = min(per_tile, s.u.nblk - (s.tile0 + j) * per_tile);
      if (lane == 0) tc::mbar_arrive_expect_tx(bar, uint32_t(n_blocks * block_bytes * C::kHalves));
      __syncwarp();
      if (pg != -2) {
        const int pos = block_pos(a, s.u, (s.tile0 + j) * per_tile + lane);
        const uint32_t dst = tc::smem_u32(sKV + slot * C::kTileBytes) + lane * block_bytes;
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tc::tma_load_4d(dst + hf * C::kHalfBytes, map, bar, hf * 64, pos & ((1 << a.page_shift) - 1), s.h, pg, policy);
      }
      issued |= 1u << slot;
      if (++slot == C::kSlots) slot = 0, phase ^= 1;
      return true;
    };
    auto load_q = [&](int b, int parity, int row) {
      if (!wait(&sh->q_empty[b], parity ^ 1)) return false;
      if (lane == 0) {
        const uint32_t bar = tc::smem_u32(&sh->q_full[b]);
        tc::mbar_arrive_expect_tx(bar, uint32_t(tile_rows * 128 * C::kHalves));
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tc::tma_load_3d(tc::smem_u32(sQ + b * C::kTileBytes + hf * C::kHalfBytes), &map_q, bar, hf * 64, s.h * a.g,
                          row, tc::policy_evict_last());
      }
      q_issued[b] = parity;
      return true;
    };
    int q_use[2] = {0, 0};
    while (ok && walk.next(a, sh, s)) {
      if (s.tile0 > 0) flags |= kTailUsed | (s.tile0 + s.n == s.u.ntiles ? kTailEnds : 0);
      if (s.tile0 == 0 && s.n < s.u.ntiles) flags |= kHeadUsed, info = make_int4(0, s.row0, s.ntok, s.h);
      int pg0 = page_of(0), pg1 = page_of(1);
      if (kPair) {
        ok = load(&map_k, 0, pg0) && load_q(0, q_use[0]++ & 1, s.row0) &&
             (s.ntok <= a.tokens || load_q(1, q_use[1]++ & 1, s.row0 + a.tokens));
        for (int j = 0; ok && j < s.n; ++j) {
          const int pg2 = page_of(j + 2);
          ok = load(&map_v, j, pg0) && (j + 1 >= s.n || load(&map_k, j + 1, pg1));
          pg0 = pg1, pg1 = pg2;
        }
      } else {
        const int b = seg_i & 1;
        ok = load(&map_k, 0, pg0) && load_q(b, q_use[b]++ & 1, s.row0) && (s.n < 2 || load(&map_k, 1, pg1));
        int pg2 = page_of(2);
        for (int j = 0; ok && j < s.n; ++j) {
          const int pg3 = page_of(j + 3);
          ok = load(&map_v, j, pg0) && (j + 2 >= s.n || load(&map_k, j + 2, pg2));
          pg0 = pg1, pg1 = pg2, pg2 = pg3;
        }
      }
      ++seg_i;
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 1u, uint32_t(seg_i));
      // wait (bounded) for every copy in flight before the CTA exits
      const volatile int never = 0;
      const long long dl = tc::deadline_after_ns(200000000ull);
      for (int i = 0; i < C::kSlots; ++i)  // the last use of a slot before `slot` is in this round, of the others in the last
        if (issued >> i & 1u)
          tc::mbar_wait_bounded(tc::smem_u32(&sh->kv_full[i]), i < slot ? phase : phase ^ 1, dl, &never);
      for (int b = 0; b < 2; ++b)
        if (q_issued[b] >= 0) tc::mbar_wait_bounded(tc::smem_u32(&sh->q_full[b]), q_issued[b], dl, &never);
    }
    if (lane == 0) {
      info.x = ok ? flags : 0;
      a.info[blockIdx.x] = info;
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(kTile, kTile);
    constexpr uint32_t idesc_pv = tc::idesc_bf16_f32(kTile, D) | tc::kIdescBMajorMN;
    int slot = 0, seg_i = 0, q_use[2] = {0, 0}, p_use[2] = {0, 0};
    uint32_t phase = 0;
    bool ok = true, any = false;
    Walk walk(sh, unit_tokens);
    Segment s = {};
    // S_st = Q_b K^T for the tile in ring slot `ks`
    auto issue_qk = [&](int st, int b, int ks) {
      const uint32_t q = tc::smem_u32(sQ + b * C::kTileBytes), k = tc::smem_u32(sKV + ks * C::kTileBytes);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t off = (i / 4) * C::kHalfBytes + (i % 4) * 32;
        tc::mma_bf16(tmem + st * kTile, tc::sdesc_kmajor_sw128(q + off), tc::sdesc_kmajor_sw128(k + off), idesc_qk, i != 0);
      }
    };
    // O_st (+)= P_st V; P_st lies over the first 64 columns of S_st
    auto issue_pv = [&](int st, int vs, bool add) {
      const uint32_t v = tc::smem_u32(sKV + vs * C::kTileBytes);
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i)
        tc::mma_bf16_ts(tmem + 2 * kTile + st * D, tmem + st * kTile + 8 * i,
                        tc::sdesc_mnmajor_sw128(v + i * 2048, C::kHalfBytes), idesc_pv, add || i != 0);
    };
    auto take = [&](int& which) {  // the next filled slot of the ring
      which = slot;
      if (!wait(&sh->kv_full[slot], phase)) return false;
      if (++slot == C::kSlots) slot = 0, phase ^= 1;
      return true;
    };
    // Slots that no row of the unit sees hold whatever was there, NaN included, and 0 * NaN is NaN: their V
    // rows are cleared.  All lanes, 16-byte stores, rotated so that the lanes spread over the banks.
    auto clear_unseen = [&](int j, int vs) {
      const int first = (s.tile0 + j) * (kTile >> a.block_shift);
      const int last = first + (kTile >> a.block_shift) - 1;
      const int b0 = block_pos(a, s.u, first);
      const int end = block_pos(a, s.u, last) + (1 << a.block_shift) - 1;
      if (end <= s.u.p1 && (first >= s.u.sb ? b0 >= s.u.lo : end < a.n_sink)) return;
      for (int i = lane; i < kTile; i += 32) {
        const int pos = block_pos(a, s.u, first + (i >> a.block_shift)) + (i & ((1 << a.block_shift) - 1));
        if (pos <= s.u.p1 && (pos >= s.u.lo || pos < a.n_sink)) continue;
        uint8_t* row = sKV + vs * C::kTileBytes + i * 128;
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(row + hf * C::kHalfBytes + (((k + lane) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
    };
    while (ok && walk.next(a, sh, s)) {
      const bool both = kPair ? s.ntok > a.tokens : s.n > 1;
      int ks, vs;
      if (kPair) {
        ok = take(ks) && wait(&sh->q_full[0], q_use[0]++ & 1) && (!both || wait(&sh->q_full[1], q_use[1]++ & 1));
        if (!ok) break;
        tc::tc_fence_after();
        if (lane == 0) {
          issue_qk(0, 0, ks);
          tc::mma_commit(tc::smem_u32(&sh->s_full[0]));
          if (s.n == 1) tc::mma_commit(tc::smem_u32(&sh->q_empty[0]));
          if (both) {
            issue_qk(1, 1, ks);
            tc::mma_commit(tc::smem_u32(&sh->s_full[1]));
            if (s.n == 1) tc::mma_commit(tc::smem_u32(&sh->q_empty[1]));
          }
          tc::mma_commit(tc::smem_u32(&sh->kv_empty[ks]));
        }
        any = true;
        for (int j = 0; ok && j < s.n; ++j) {
          ok = take(vs);
          if (!ok) break;
          clear_unseen(j, vs);
          const bool more = j + 1 < s.n;
          for (int st = 0; ok && st < (both ? 2 : 1); ++st) {
            ok = wait(&sh->p_full[st], p_use[st]++ & 1) && (st != 0 || !more || take(ks));
            if (!ok) break;
            tc::tc_fence_after();
            if (lane == 0) {
              issue_pv(st, vs, j > 0);
              if (!more) tc::mma_commit(tc::smem_u32(&sh->o_full[st]));
              if (st == (both ? 1 : 0)) tc::mma_commit(tc::smem_u32(&sh->kv_empty[vs]));
              if (more) {
                issue_qk(st, st, ks);
                tc::mma_commit(tc::smem_u32(&sh->s_full[st]));
                if (j + 2 == s.n) tc::mma_commit(tc::smem_u32(&sh->q_empty[st]));
                if (st == (both ? 1 : 0)) tc::mma_commit(tc::smem_u32(&sh->kv_empty[ks]));
              }
            }
            __syncwarp();
          }
        }
      } else {
        const int b = seg_i & 1;
        auto qk = [&](int j) {  // tile j on its stream
          if (!take(ks)) return false;
          tc::tc_fence_after();
          if (lane == 0) {
            issue_qk(j & 1, b, ks);
            tc::mma_commit(tc::smem_u32(&sh->s_full[j & 1]));
            tc::mma_commit(tc::smem_u32(&sh->kv_empty[ks]));
          }
          any = true;
          __syncwarp();
          return true;
        };
        // the ring holds K 0, K 1, then V j, K j + 2, ..
        ok = wait(&sh->q_full[b], q_use[b]++ & 1) && qk(0) && (!both || qk(1));
        for (int j = 0; ok && j < s.n; ++j) {
          const int st = j & 1;
          ok = take(vs);
          if (!ok) break;
          clear_unseen(j, vs);
          ok = wait(&sh->p_full[st], p_use[st]++ & 1);
          if (!ok) break;
          tc::tc_fence_after();
          if (lane == 0) {
            issue_pv(st, vs, j > 1);
            tc::mma_commit(tc::smem_u32(&sh->kv_empty[vs]));
            if (j + 2 >= s.n) tc::mma_commit(tc::smem_u32(&sh->o_full[st]));
          }
          __syncwarp();
          if (j + 2 < s.n) ok = qk(j + 2);
        }
      }
      ++seg_i;
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 2u, uint32_t(seg_i));
    }
    if (lane == 0) sh->mma_pending = any;
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    if ((warp & 3) < active) {
    // ------------------------------------------------------------------------- softmax
    const int st = warp >> 2, row = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t t_s = lane_base + st * kTile, t_o = lane_base + 2 * kTile + st * D;
    const int tok = row / a.g, hh = row - tok * a.g;
    const float c2 = a.c2;
    int seg_i = 0, s_use = 0, o_use = 0, m_use = 0;
    bool ok = true;
    Walk walk(sh, unit_tokens);
    Segment s = {};
    while (ok && walk.next(a, sh, s)) {
      const bool both = kPair ? s.ntok > a.tokens : s.n > 1;
      const bool partial = s.n < s.u.ntiles;
      if (st == 1 && !both) {
        ++seg_i;
        continue;
      }
      // this stream's rows and tiles
      const int tok0 = kPair ? st * a.tokens : 0;
      const int p = s.u.p0 + tok0 + tok;                                       // this row's position
      const int q0 = s.u.p0 + tok0, q1 = kPair ? min(q0 + a.tokens - 1, s.u.p1) : s.u.p1;
      const bool valid = row < tile_rows && tok0 + tok < s.ntok;
      float m = -INFINITY;  // reference of the exponentials, log2 units
      unsigned long long l2[2] = {0ull, 0ull};
      float l = 0.f;
      for (int j = kPair ? 0 : st; j < s.n; j += kPair ? 1 : 2) {
        ok = wait(&sh->s_full[st], s_use++ & 1);
        if (!ok) break;
        tc::tc_fence_after();
        float x[kTile];
#pragma unroll
        for (int i = 0; i < 4; ++i) tc::tmem_ld32(t_s + 32 * i, reinterpret_cast<uint32_t*>(x + 32 * i));
        tc::tmem_ld_wait();
        const int first = (s.tile0 + j) * (kTile >> a.block_shift);
        const int c0 = block_pos(a, s.u, first);
        const bool inside = (first >= s.u.sb) && c0 + kTile - 1 <= q0 && (a.window == 0 || c0 > q1 - a.window);
        if (!inside) {
          // what the row does not see takes no part: -inf after the scale
          const float out = c2 > 0.f ? -INFINITY : INFINITY;
#pragma unroll
          for (int gr = 0; gr < kTile / 8; ++gr) {  // 8 slots of one block
            const int pos = block_pos(a, s.u, first + ((8 * gr) >> a.block_shift)) + ((8 * gr) & ((1 << a.block_shift) - 1));
            uint32_t see = bits_between(a.window ? p - a.window + 1 - pos : 0, p - pos);
            if (a.window) see |= bits_between(0, min(p, a.n_sink - 1) - pos);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (!(see >> k & 1u)) x[8 * gr + k] = out;
          }
        }
        float t4[4];
        if (c2 > 0.f) {
#pragma unroll
          for (int i = 0; i < 4; ++i) t4[i] = x[i];
#pragma unroll
          for (int i = 4; i < kTile; ++i) t4[i & 3] = fmaxf(t4[i & 3], x[i]);
          t4[0] = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) t4[i] = x[i];
#pragma unroll
          for (int i = 4; i < kTile; ++i) t4[i & 3] = fminf(t4[i & 3], x[i]);
          t4[0] = fminf(fminf(t4[0], t4[1]), fminf(t4[2], t4[3]));
        }
        const float top = t4[0] * c2;
        const bool first_tile = kPair ? j == 0 : j < 2;
        float alpha = 1.f;
        if (top > m + kRescaleAt) {
          alpha = tc::ex2_approx(m - top);
          m = top;
        }
        if (__any_sync(~0u, alpha != 1.f)) {
          l *= alpha;
          if (!first_tile) {  // PV of the stream's last tile was issued before this tile's S: complete
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              uint32_t o[32];
              tc::tmem_ld32(t_o + 32 * i, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tc::tmem_st32(t_o + 32 * i, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const unsigned long long cc = pack_f32x2(c2, c2), mm = pack_f32x2(-ref, -ref);
        l2[0] = l2[1] = 0ull;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int i = 64 * hf + 2 * k;
            float e0, e1;
            unpack_f32x2(fma_f32x2(pack_f32x2(x[i], x[i + 1]), cc, mm), e0, e1);
            e0 = tc::ex2_approx(e0);
            e1 = tc::ex2_approx(e1);
            l2[k & 1] = add_f32x2(l2[k & 1], pack_f32x2(e0, e1));
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(e0, e1);
            pk[k] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          tc::tmem_st32(t_s + 32 * hf, pk);
        }
        {
          float u0, u1;
          unpack_f32x2(add_f32x2(l2[0], l2[1]), u0, u1);
          l += u0 + u1;
        }
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->p_full[st]));
      }
      if (!ok) break;
      ok = wait(&sh->o_full[st], o_use++ & 1);
      if (!ok) break;
      tc::tc_fence_after();
      // ---------------------------------------------------------------- the unit's rows
      const int orow = s.row0 + tok0 + tok;
      const int64_t oat = int64_t(orow) * a.Hq + s.h * a.g + hh;
      const int pslot = 2 * blockIdx.x + (s.tile0 > 0 ? 0 : 1);
      const int64_t prow = int64_t(pslot) * ((kPair ? 2 : 1) * kTile) + (kPair ? st * kTile : 0) + row;
      // 32 columns of the row from `cols` on
      auto put = [&](const float* v, int cols) {
        if (!valid) return;
        if (partial) {
          float4* dst = reinterpret_cast<float4*>(a.partial + prow * D + cols);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(a.out + oat * D + cols);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[8 * k + 2 * z], v[8 * k + 2 * z + 1]);
              w[z] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      };
      auto put_lse = [&](float mx, float sum) {
        if (!valid) return;
        const float lse2 = sum > 0.f ? mx + log2f(sum) : -INFINITY;
        if (partial)
          a.plse[prow] = lse2;
        else if (a.lse)
          a.lse[oat] = lse2 * kLn2;
      };
      if (kPair || !both) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float v[32];
          tc::tmem_ld32(t_o + 32 * i, reinterpret_cast<uint32_t*>(v));
          tc::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] *= inv;
          put(v, 32 * i);
        }
        put_lse(m, l);
      } else {
        // the other stream's half of the tiles: through this segment's Q tile (its last MMA is done), half
        // of the columns at a time; a row's 16-byte pieces are rotated over the banks
        constexpr int kRound = D / 2, kPieces = kRound / 4;
        uint8_t* buf = sQ + (seg_i & 1) * C::kTileBytes;
        float4* mine = reinterpret_cast<float4*>(buf + row * (kRound * 4));
        float2* ml = sh->ml + row;
        if (st == 1) *ml = make_float2(m, l);
        float w_own = 1.f, w_other = 0.f, mx = m, sum = l;
#pragma unroll
        for (int rd = 0; rd < 2; ++rd) {
          if (st == 1) {
            if (rd == 1) {
              ok = wait(&sh->m_empty, m_use & 1);
              if (!ok) break;
            }
#pragma unroll
            for (int i = 0; i < kRound / 32; ++i) {
              float v[32];
              tc::tmem_ld32(t_o + rd * kRound + 32 * i, reinterpret_cast<uint32_t*>(v));
              tc::tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mine[(8 * i + k) ^ (row & (kPieces - 1))] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->m_full));
          } else {
            ok = wait(&sh->m_full, rd);
            if (!ok) break;
            if (rd == 0) {
              const float2 o = *ml;
              mx = fmaxf(m, o.x);
              const float ref = mx == -INFINITY ? 0.f : mx;
              w_own = tc::ex2_approx(m - ref), w_other = tc::ex2_approx(o.x - ref);
              sum = l * w_own + o.y * w_other;
              const float inv = sum > 0.f ? 1.f / sum : 0.f;
              w_own *= inv, w_other *= inv;
            }
#pragma unroll
            for (int i = 0; i < kRound / 32; ++i) {
              float v[32];
              tc::tmem_ld32(t_o + rd * kRound + 32 * i, reinterpret_cast<uint32_t*>(v));
              tc::tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 o = mine[(8 * i + k) ^ (row & (kPieces - 1))];
                v[4 * k] = v[4 * k] * w_own + o.x * w_other;
                v[4 * k + 1] = v[4 * k + 1] * w_own + o.y * w_other;
                v[4 * k + 2] = v[4 * k + 2] * w_own + o.z * w_other;
                v[4 * k + 3] = v[4 * k + 3] * w_own + o.w * w_other;
              }
              put(v, rd * kRound + 32 * i);
            }
            if (rd == 0) {
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->m_empty));
            }
          }
        }
        if (!ok) break;
        ++m_use;
        if (st == 0) put_lse(mx, sum);
      }
      tc::tc_fence_before();  // O has been read: the next unit's first PV may follow this stream's next P
      if (!kPair && st == 0) {
        tc::fence_proxy_async_smem();  // the merge's reads and writes before the next TMA into this Q tile
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->q_empty[seg_i & 1]));
      }
      ++seg_i;
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 3u, uint32_t(seg_i) | uint32_t(warp) << 24);
    }
    }
  }

  __syncthreads();
  if (warp == 9) {
    if (lane == 0 && sh->mma_pending && sh->abort) {  // MMAs may still be in flight: wait (bounded) before TMEM is freed
      tc::mma_commit(tc::smem_u32(&sh->drain));
      const volatile int never = 0;
      tc::mbar_wait_bounded(tc::smem_u32(&sh->drain), 0, tc::deadline_after_ns(200000000ull), &never);
    }
    __syncwarp();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the partial rows of the units that a cut between CTAs runs through: the block of CTA c takes the
// unit that c began and did not finish, in the order of its KV tiles.  One warp per row:
//     out = sum_i 2^(lse_i - M) out_i / sum_i 2^(lse_i - M),   M = max_i lse_i
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttnArgs a, int n_cta, int unit_rows) {
  constexpr int E = D / 32;
  pdl_enter();
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5), c = blockIdx.x;
  const int4 info = a.info[c];
  if (!(info.x & kHeadUsed)) return;
  const int tok = (row / kTile) * a.tokens + (row % kTile) / a.g, hh = (row % kTile) % a.g;
  if (row % kTile >= a.tokens * a.g || tok >= info.z) return;
  // the CTAs after c that worked on the unit: up to the first that finished it
  int last = c;
  for (int base = c + 1; base < n_cta; base += 32) {
    const int fl = base + lane < n_cta ? a.info[base + lane].x : 0;
    const uint32_t ends = __ballot_sync(~0u, fl & kTailEnds);
    if (ends) {
      last = base + __ffs(ends) - 1;
      break;
    }
    last = min(base + 31, n_cta - 1);
  }
  // part i: the head of c, then the tails of c + 1 ..; CTAs without work in between have none
  auto part_row = [&](int i) { return int64_t(i == 0 ? 2 * c + 1 : 2 * (c + i)) * unit_rows + row; };
  auto part_lse = [&](int i) {
    if (c + i > last || (i > 0 && !(a.info[c + i].x & kTailUsed))) return -INFINITY;
    return a.plse[part_row(i)];
  };
  const int n = last - c + 1;
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, part_lse(i));
  top = warp_max(top);
  top = __shfl_sync(~0u, top, 0);
  const float ref = top == -INFINITY ? 0.f : top;
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int base = 0; base < n; base += 32) {
    const float w_mine = exp2f(part_lse(base + lane) - ref);
#pragma unroll 4
    for (int i = 0; i < min(32, n - base); ++i) {
      const float w = __shfl_sync(~0u, w_mine, i);
      if (w == 0.f) continue;  // nothing seen there (and nothing written by a CTA without work)
      sum += w;
      const float* src = a.partial + part_row(base + i) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = *reinterpret_cast<const float2*>(src + e);
        acc[e] += w * v.x;
        acc[e + 1] += w * v.y;
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

// Workspace: status block | Info of each CTA | partial rows | their log-sum-exps.
struct AttnWs {
  size_t info, partial, plse, total;
};
AttnWs attn_ws(int D, int unit_rows, int n_cta) {
  AttnWs w;
  w.info = 256;
  w.partial = w.info + align256(n_cta * sizeof(int4));
  w.plse = w.partial + align256(size_t(2) * n_cta * unit_rows * D * sizeof(float));
  w.total = w.plse + align256(size_t(2) * n_cta * unit_rows * sizeof(float));
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

template <int D, bool kPair>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a, int n_cta,
                   cudaStream_t s) {
  using C = Cfg<D>;
  constexpr int kSmem = (2 + C::kSlots) * C::kTileBytes + int(sizeof(Shared));
  static_assert(kSmem <= 232448, "dynamic shared memory beyond the 227 KB per-block limit");
  static bool done[tch::kMaxDevices] = {};
  static std::mutex mu;
  cudaError_t e = tch::set_smem_once(attention_kernel<D, kPair>, kSmem, done, &mu);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attention_kernel<D, kPair>, dim3(n_cta), dim3(kThreads), kSmem, s, mq, mk, mv, a);
  if (e != cudaSuccess) return e;
  const int unit_rows = (kPair ? 2 : 1) * kTile;
  return launch_pdl(attention_join_kernel<D>, dim3(n_cta, ((kPair ? kTile : 0) + a.tokens * a.g + 7) / 8), dim3(256), 0, s, a,
                    n_cta, unit_rows);
}

}  // namespace

size_t window_attention_ws_bytes(int Hq, int Hkv, int D) {
  return attn_ws(D, 2 * kTile, tch::sm_count()).total;  // either tiling
}

cudaError_t launch_window_attention(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                    const int32_t* page_table, int max_pages, int n_pages, int page_shift,
                                    const int32_t* cu, const int32_t* ctx, int bs, int rows, int max_rows, int Hq,
                                    int Hkv, int D, float scale, int window, int n_sink, void* out, float* lse,
                                    void* ws, cudaStream_t s) {
  AttnArgs a;
  const int n_cta = tch::sm_count(), fit = kTile / (Hq / Hkv);
  const bool pair = max_rows > fit;  // more rows than one Q tile holds: two tiles that share K and V
  a.cache_limit = std::min(int64_t(max_pages) << page_shift, int64_t(1) << 30);  // positions: well inside 32 bits
  a.page_table = page_table, a.cu = cu, a.ctx = ctx, a.out = static_cast<__nv_bfloat16*>(out), a.lse = lse;
  char* w = static_cast<char*>(ws);
  const AttnWs L = attn_ws(D, pair ? 2 * kTile : kTile, n_cta);
  a.status = reinterpret_cast<uint32_t*>(w), a.diag = reinterpret_cast<uint32_t*>(w + 16);
  a.info = reinterpret_cast<int4*>(w + L.info);
  a.partial = reinterpret_cast<float*>(w + L.partial), a.plse = reinterpret_cast<float*>(w + L.plse);
  a.timeout_ns = g_wait_timeout_ns;
  a.c2 = scale * kLog2e;
  // the kernel hides a score by an infinity before the scale: a scale of 0 becomes one that gives equal weights
  // all the same (2^(1e-30 s) is 1)
  if (a.c2 == 0.f) a.c2 = 1e-30f;
  a.max_pages = max_pages, a.n_pages = n_pages, a.page_shift = page_shift, a.block_shift = std::min(page_shift, 7);
  a.bs = bs, a.rows = rows, a.Hq = Hq, a.Hkv = Hkv, a.g = Hq / Hkv, a.tokens = std::min(fit, max_rows);
  a.window = window >= a.cache_limit ? 0 : window, a.n_sink = n_sink;
  CUtensorMap mq, mk, mv;
  const int page = 1 << page_shift, block = 1 << a.block_shift;
  if (!tch::encode_fn() || !encode_q(&mq, q, rows, Hq, D, q_stride, a.g, a.tokens) ||
      !encode_cache(&mk, k_cache, n_pages, Hkv, page, D, block) ||
      !encode_cache(&mv, v_cache, n_pages, Hkv, page, D, block))
    return cudaErrorInvalidValue;
  if (D == 64) return pair ? launch<64, true>(mq, mk, mv, a, n_cta, s) : launch<64, false>(mq, mk, mv, a, n_cta, s);
  return pair ? launch<128, true>(mq, mk, mv, a, n_cta, s) : launch<128, false>(mq, mk, mv, a, n_cta, s);
}

}  // namespace dspark
