// The attention of short windows: all (token, head) rows of a unit fit one tile of R = 16, 32, 64 or 128.
//
// Bound by reading K and V once, so a KV tile's way through the SM has to be short: the products are taken
// transposed,
//     S^T = K Q^T        [128 slots x R]   (tcgen05, M = 128, N = R; fp32 in TMEM)
//     P^T = 2^(c S^T - m)                   (bf16, shared memory), partial sums of P per slot in registers
//     O^T += V^T P^T     [D x R]            (tcgen05, fp32 in TMEM)
// so that a thread holds one KV slot and some of the rows, and all softmax warps have work however few the rows
// are.  (With the rows on TMEM lanes instead, 32 rows sat in one warp per stream: a unit of 10 tiles at 32
// rows took 24 us per CTA; it takes 12.)  A tile's way through the softmax is a chain of latencies, so two sets of
// softmax warps take alternate tiles, each with its own S^T, P^T, O^T and references; a unit's two halves
// are merged when its rows are written.  At R = 128 one set takes all tiles (its registers allow no more,
// and it has twice the work per tile).
//
// m is a reference that only keeps the exponentials in range, the same for all slots of a row: any value
// within 2^60 of the maximum gives the same result, since the sum is divided out and neither fp32 nor bf16 loses
// bits there.  So it is set from a set's first tile of a unit and checked, not recomputed, on the others.
#include <type_traits>

#include "attention_common.cuh"

namespace dspark {
namespace {

using namespace attn;

constexpr int kMaxSlots = 6;
constexpr float kUnset = -1e30f, kRescaleAt = 60.f;  // log2 units

// Sixteen softmax warps in groups of four; a group takes R / kRowGroups rows of its set's tiles.  Then one warp
// each for TMA, S^T, O^T and the clearing of what must not be seen of V.
constexpr int kGroups = 4, kThreads = (kGroups + 1) * 128;
constexpr int kTma = 4 * kGroups, kSWarp = kTma + 1, kOWarp = kTma + 2, kClearWarp = kTma + 3;
// Registers: launched with 640 x 96; the softmax warps take what the others give back (512 x 104 + 128 x 56 <= 640 x 96).
constexpr int kSoftmaxRegs = 104, kOtherRegs = 56;

template <int R>
struct Split {
  static constexpr int kSets = R == 128 ? 1 : 2, kRowGroups = kGroups / kSets, kRows = R / kRowGroups;
};

template <int R>
struct Shared {
  static constexpr int kSets = Split<R>::kSets, kRowGroups = Split<R>::kRowGroups, kRows = Split<R>::kRows;
  uint64_t q_full[2], q_empty[2], k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
  uint64_t v_ready[kReady];
  uint64_t s_full[2], p_full[2], p_empty[2];
  uint64_t o_full[kSets], o_read[kSets];           // a set's O^T is complete; has been read by all that do
  uint64_t group[kGroups];                          // the four warps of a group
  uint64_t pair_put[kRowGroups], pair_got[kRowGroups];  // the two sets' groups of the same rows
  uint64_t drain[2];
  uint32_t tmem_base;
  volatile int abort;
  int pending[2];                                   // the MMA warps have issued something
  int need[kGroups][2];                             // [parity]: the last tile at which a warp asked for a new reference
  Range range;
  float warp_part[kGroups][4][kRows];               // by warp: the rows' maxima of a tile, sums of a unit
  alignas(16) float ref[kSets][R];                  // the rows' references, read four at a time
  float scale[kSets][R];                            // what a new reference scales the old sums by
};

template <int D, int R>
struct Cfg {
  static constexpr int kHalves = D / 64;                   // 128-byte swizzled column blocks of a tile
  static constexpr int kSlotBytes = kTile * D * 2;
  static constexpr int kQBytes = R * D * 2, kQBufs = R == 128 || R * D == 64 * 128 ? 1 : 2;
  static constexpr int kPPitch = R < 64 ? R * 2 : 128;      // bytes of a slot's row of P, R > 64: in two chunks
  static constexpr int kPBytes = kTile * R * 2, kPBufs = Split<R>::kSets;
  // O^T has M = 128 also where D = 64: its lanes 64 .. 127 come from the 16 KB behind the V tile, whatever
  // they hold, and are not read
  static constexpr int kBehind = kQBytes * kQBufs + kPBytes * kPBufs;
  static constexpr int kPad = D == 64 && kBehind < 16384 ? 16384 - kBehind : 0;
  // rings of K and V tiles; K runs two tiles ahead of V
  static constexpr int kRoom = (232448 - int(sizeof(Shared<R>)) - kBehind - kPad) / kSlotBytes;
  static constexpr int kVSlots = (kRoom + 1) / 2 < kMaxSlots ? (kRoom + 1) / 2 : kMaxSlots;
  static constexpr int kKSlots = kRoom / 2 < kMaxSlots ? kRoom / 2 : kMaxSlots;
  static constexpr int kSmem = (kKSlots + kVSlots) * kSlotBytes + kBehind + kPad + int(sizeof(Shared<R>));
  static constexpr int kTmemCols = 4 * R;  // S^T twice, the sets' O^T; a power of two
  static_assert(kKSlots >= 2 && kVSlots >= 2 && kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "shared memory layout");
};

// The tiles of a CTA's range one by one.
struct Cursor {
  Walk walk;
  Segment s = {};
  int j = 0;
  __device__ Cursor(const Range& g, int unit_tokens) : walk(g, unit_tokens) {}
  __device__ __forceinline__ bool next(const AttnArgs& a, const Range& g) {
    if (++j < s.n) return true;
    j = 0;
    return walk.next(a, g, s);
  }
  __device__ __forceinline__ bool first() const { return j == 0; }
  __device__ __forceinline__ bool last() const { return j + 1 == s.n; }
};

// Folds N values of each lane over the 32 lanes (kMax: maxima, else sums, in a fixed order), halving the values with the
// lanes; N = 8, 16 or 32.  Afterwards lane l holds the result of value l / (32 / N) in v[0].
template <int N, bool kMax>
__device__ __forceinline__ float fold_lanes(float* v, int lane) {
  static_assert(N == 8 || N == 16 || N == 32, "values");
  int cnt = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (cnt > 1) {
      cnt >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < cnt) {
          const float got = __shfl_xor_sync(~0u, up ? v[i] : v[i + cnt], o), keep = up ? v[i + cnt] : v[i];
          v[i] = kMax ? fmaxf(keep, got) : keep + got;
        }
    } else {
      const float got = __shfl_xor_sync(~0u, v[0], o);
      v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
    }
  }
  return v[0];
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
    window_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttnArgs a) {
  using C = Cfg<D, R>;
  constexpr int kSets = Split<R>::kSets, kRowGroups = Split<R>::kRowGroups, RW = Split<R>::kRows;  // RW: rows per thread
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::kKSlots * C::kSlotBytes;
  uint8_t* sQ = sV + C::kVSlots * C::kSlotBytes;
  uint8_t* sP = sQ + C::kQBytes * C::kQBufs;
  Shared<R>* sh = reinterpret_cast<Shared<R>*>(sP + C::kPBytes * C::kPBufs + C::kPad);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // the same for the warp, and known to be
  const int tile_rows = a.tokens * a.g;
  const Waiter wait{&sh->abort, a.timeout_ns};

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->q_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->q_empty[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->s_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->p_full[i]), 4 * kRowGroups);
      tc::mbar_init(tc::smem_u32(&sh->p_empty[i]), 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->group[i]), 4);
      sh->need[i][0] = sh->need[i][1] = 0;
    }
    for (int i = 0; i < kMaxSlots; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->k_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->k_empty[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->v_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->v_empty[i]), 2);  // the product, and the clearing warp
    }
    for (int i = 0; i < kReady; ++i) tc::mbar_init(tc::smem_u32(&sh->v_ready[i]), 1);
    for (int i = 0; i < kSets; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->o_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->o_read[i]), 4 * kGroups);
    }
    for (int i = 0; i < kRowGroups; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->pair_put[i]), 8);
      tc::mbar_init(tc::smem_u32(&sh->pair_got[i]), 8);
    }
    tc::mbar_init(tc::smem_u32(&sh->drain[0]), 1);
    tc::mbar_init(tc::smem_u32(&sh->drain[1]), 1);
    tc::fence_mbar_init();
    sh->abort = 0, sh->pending[0] = sh->pending[1] = 0, sh->range.bad = 0, sh->range.n_long = 0;
    tc::prefetch_tensormap(&map_q);
    tc::prefetch_tensormap(&map_k);
    tc::prefetch_tensormap(&map_v);
  }
  if (warp == kSWarp) {
    tc::tmem_alloc(tc::smem_u32(&sh->tmem_base), C::kTmemCols);
    tc::tmem_relinquish();
  }
  // rows of Q past the unit's last are never loaded: zeros, so that their scores are 0
  for (int i = tid; i < C::kQBytes * C::kQBufs / 16; i += kThreads)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc::fence_proxy_async_smem();
  __syncthreads();
  pdl_enter();
  plan_range(a, sh->range, reinterpret_cast<uint8_t*>(sh->warp_part), a.tokens);
  __syncthreads();
  const uint32_t tmem = sh->tmem_base;

  if (warp >= kTma) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kTma) {
    // --------------------------------------------------------------------- TMA producer
    // In order: K 0, K 1, then V t, K t + 2, over all tiles of the range; a unit's Q with its first K.
    const uint64_t keep = tc::policy_evict_last(), stream = tc::policy_evict_first();
    Ring<C::kKSlots> kr;
    Ring<C::kVSlots> vr;
    int n_seg = 0, flags = 0, n_k = 0, n_v = 0;
    int q_uses[2] = {0, 0};
    int4 info = make_int4(0, 0, 0, 0);
    Cursor cur(sh->range, a.tokens);
    struct Ahead {
      TileLoad t;
      int row0;  // >= 0: the unit's first tile here
      bool there;
    };
    auto fetch = [&]() {  // the next tile's pages; used three tiles later
      Ahead f = {};
      f.there = cur.next(a, sh->range);
      if (!f.there) return f;
      const Segment& s = cur.s;
      f.t = tile_load(a, s, cur.j, lane);
      f.row0 = cur.first() ? s.row0 : -1;
      if (cur.first()) {
        if (s.tile0 > 0) flags |= kTailUsed | (s.tile0 + s.n == s.u.ntiles ? kTailEnds : 0);
        if (s.tile0 == 0 && s.n < s.u.ntiles) flags |= kHeadUsed, info = make_int4(0, s.row0, s.ntok, s.h);
      }
      return f;
    };
    auto put_v = [&](const Ahead& f) {
      if (!wait(&sh->v_empty[vr.slot], vr.phase ^ 1)) return false;
      issue_tile<C::kHalves>(a, &map_v, f.t, tc::smem_u32(sV + vr.slot * C::kSlotBytes), tc::smem_u32(&sh->v_full[vr.slot]),
                             stream, lane);
      ++n_v;
      vr.step();
      return true;
    };
    auto put_k = [&](const Ahead& f) {
      if (!wait(&sh->k_empty[kr.slot], kr.phase ^ 1)) return false;
      issue_tile<C::kHalves>(a, &map_k, f.t, tc::smem_u32(sK + kr.slot * C::kSlotBytes), tc::smem_u32(&sh->k_full[kr.slot]),
                             stream, lane);
      ++n_k;
      kr.step();
      if (f.row0 < 0) return true;
      const int b = n_seg++ % C::kQBufs;
      if (!wait(&sh->q_empty[b], (q_uses[b] & 1) ^ 1)) return false;
      if (lane == 0) {
        const uint32_t bar = tc::smem_u32(&sh->q_full[b]);
        tc::mbar_arrive_expect_tx(bar, uint32_t(tile_rows * 128 * C::kHalves));
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tc::tma_load_3d(tc::smem_u32(sQ + b * C::kQBytes + hf * (R * 128)), &map_q, bar, hf * 64, f.t.head * a.g,
                          f.row0, keep);
      }
      ++q_uses[b];
      return true;
    };
    Ahead f0 = fetch(), f1 = fetch(), f2 = fetch(), f3 = fetch();
    bool ok = (!f0.there || put_k(f0)) && (!f1.there || put_k(f1));
    while (ok && f0.there) {
      ok = put_v(f0) && (!f2.there || put_k(f2));
      f0 = f1, f1 = f2, f2 = f3, f3 = fetch();
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 1u, uint32_t(n_seg));
      // wait (bounded) for every copy in flight before the CTA exits
      const volatile int never = 0;
      const long long dl = tc::deadline_after_ns(200000000ull);
      // slots before the ring's position were last used in this round, the others in the last one
      for (int i = 0; i < min(n_k, C::kKSlots); ++i)
        tc::mbar_wait_bounded(tc::smem_u32(&sh->k_full[i]), i < kr.slot ? kr.phase : kr.phase ^ 1, dl, &never);
      for (int i = 0; i < min(n_v, C::kVSlots); ++i)
        tc::mbar_wait_bounded(tc::smem_u32(&sh->v_full[i]), i < vr.slot ? vr.phase : vr.phase ^ 1, dl, &never);
      for (int b = 0; b < 2; ++b)
        if (q_uses[b] > 0) tc::mbar_wait_bounded(tc::smem_u32(&sh->q_full[b]), (q_uses[b] - 1) & 1, dl, &never);
    }
    if (lane == 0) {
      info.x = ok ? flags : 0;
      a.info[blockIdx.x] = info;
    }
  } else if (warp == kSWarp) {
    // ------------------------------------------------------------------ S^T = K Q^T of each tile
    constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, R);
    const uint64_t dk = tc::sdesc_kmajor_sw128(tc::smem_u32(sK)), dq = tc::sdesc_kmajor_sw128(tc::smem_u32(sQ));
    Ring<C::kKSlots> ring;
    int n_seg = 0, t = 0;
    bool ok = true;
    Cursor cur(sh->range, a.tokens);
    for (; cur.next(a, sh->range); ++t) {
      const int b = n_seg % C::kQBufs;
      ok = (!cur.first() || wait(&sh->q_full[b], (n_seg / C::kQBufs) & 1)) && wait(&sh->k_full[ring.slot], ring.phase) &&
           (t < 2 || wait(&sh->p_full[t & 1], ((t - 2) >> 1) & 1));  // the S before last has been read
      if (!ok) break;
      tc::tc_fence_after();
      const uint64_t dk_t = dk + uint32_t(ring.slot * (C::kSlotBytes >> 4)), dq_t = dq + uint32_t(b * (C::kQBytes >> 4));
      const bool last = cur.last();
      if (tc::elect_one()) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          tc::mma_bf16(tmem + (t & 1) * R, dk_t + (((i / 4) * (kTile * 128) + (i % 4) * 32) >> 4),
                       dq_t + (((i / 4) * (R * 128) + (i % 4) * 32) >> 4), idesc, i != 0);
        tc::mma_commit(tc::smem_u32(&sh->s_full[t & 1]));
        tc::mma_commit(tc::smem_u32(&sh->k_empty[ring.slot]));
        if (last) tc::mma_commit(tc::smem_u32(&sh->q_empty[b]));
      }
      __syncwarp();
      ring.step();
      if (last) ++n_seg;
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 2u, uint32_t(t));
    }
    if (lane == 0) sh->pending[0] = t > 0;
  } else if (warp == kOWarp) {
    // -------------------------------------------------------------- O^T += V^T P^T of each tile
    constexpr uint32_t idesc = tc::idesc_bf16_f32(128, R) | tc::kIdescAMajorMN | tc::kIdescBMajorMN;
    const uint64_t dv = tc::sdesc_mnmajor<128>(tc::smem_u32(sV), kTile * 128);
    const uint64_t dp = tc::sdesc_mnmajor<C::kPPitch>(tc::smem_u32(sP), kTile * 128);
    Ring<C::kVSlots> ring;
    int t = 0, o_uses[kSets] = {}, j0 = 0, j1 = 0;
    Ring<kReady> ready;
    bool ok = true;
    Cursor cur(sh->range, a.tokens);
    for (; cur.next(a, sh->range); ++t) {
      if (cur.first()) whole_tiles(a, cur.s, cur.s.u.p1, cur.s.u.p0, j0, j1);
      const int set = kSets == 2 ? t & 1 : 0;
      const bool first = cur.j < kSets, last = cur.j + kSets >= cur.s.n;  // of the set's tiles of the unit
      ok = wait(&sh->v_full[ring.slot], ring.phase);
      if (ok && (cur.j < j0 || cur.j >= j1)) {
        ok = wait(&sh->v_ready[ready.slot], ready.phase);
        ready.step();
      }
      ok = ok && wait(&sh->p_full[t & 1], (t >> 1) & 1);
      // the set's O^T of the unit before has been read
      if (ok && first) ok = wait(&sh->o_read[set], ((kSets == 2 && set ? o_uses[kSets - 1]++ : o_uses[0]++) & 1) ^ 1);
      if (!ok) break;
      tc::tc_fence_after();
      const uint64_t dv_t = dv + uint32_t(ring.slot * (C::kSlotBytes >> 4));
      const uint64_t dp_t = dp + uint32_t((t % C::kPBufs) * (C::kPBytes >> 4));
      if (tc::elect_one()) {
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
          tc::mma_bf16(tmem + 2 * R + set * R, dv_t + ((i * 2048) >> 4), dp_t + ((i * 16 * C::kPPitch) >> 4), idesc, !first || i != 0);
        tc::mma_commit(tc::smem_u32(&sh->p_empty[t % C::kPBufs]));
        tc::mma_commit(tc::smem_u32(&sh->v_empty[ring.slot]));
        if (last) tc::mma_commit(tc::smem_u32(&sh->o_full[set]));
      }
      __syncwarp();
      ring.step();
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 4u, uint32_t(t));
    }
    if (lane == 0) sh->pending[1] = t > 0;
  } else if (warp == kClearWarp) {
    // ------------------------------------------- V tiles: unseen slots cleared, then ready for O^T
    Ring<C::kVSlots> ring;
    Ring<kReady> ready;
    int t = 0, j0 = 0, j1 = 0;
    bool ok = true;
    Cursor cur(sh->range, a.tokens);
    for (; cur.next(a, sh->range); ++t, ring.step()) {
      if (cur.first()) whole_tiles(a, cur.s, cur.s.u.p1, cur.s.u.p0, j0, j1);
      ok = wait(&sh->v_full[ring.slot], ring.phase);
      if (!ok) break;
      if (cur.j < j0 || cur.j >= j1) {
        clear_unseen<C::kHalves>(a, cur.s, cur.j, sV + ring.slot * C::kSlotBytes, lane);
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->v_ready[ready.slot]));
        ready.step();
      }
      // every tile, so that the ring never turns more than once past this warp (a parity tells no more)
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->v_empty[ring.slot]));
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 5u, uint32_t(t));
    }
  } else if (warp < kTma) {
    // ------------------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int grp = warp >> 2, w4 = warp & 3;
    const int kv = w4 * 32 + lane;  // this thread's slot of each tile = TMEM lane
    const int set = kSets == 2 ? grp & 1 : 0, rg = grp / kSets, row0 = rg * RW;  // and its rows
    const uint32_t lane_base = tmem + (uint32_t(w4 * 32) << 16) + row0;
    const uint32_t t_o = lane_base + 2 * R;  // the first set's O^T
    const float c2 = a.c2, hidden = c2 > 0.f ? -INFINITY : INFINITY;  // 2^-infinity after the scale
    const unsigned long long cc = pack_f32x2(c2, c2);
    float* ref = sh->ref[set] + row0;
    float* scale = sh->scale[set] + row0;
    // where this thread's row of P goes: 16-byte pieces, from the first row of the group on
    uint8_t* p_row = sP + (R == 128 ? (row0 / 64) * (kTile * 128) : 0);
    const int piece0 = (R == 128 ? row0 % 64 : row0) / 8;
    // the row that this lane holds after a fold (the lanes of a row hold the same)
    const int fold_row = lane / (32 / RW);
    int t0 = 0, sync = 0, n_pair = 0, n_unit[2] = {0, 0};  // tiles before; meetings; units merged; units of each set
    bool ok = true;
    Walk walk(sh->range, a.tokens);
    Segment s = {};
    // the group's four warps: everything before on all of them is visible after
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->group[grp]));
      return wait(&sh->group[grp], sync++ & 1);
    };
    while (ok && walk.next(a, sh->range, s)) {
      const bool both = kSets == 2 && s.n > 1;
      const int begin = kSets == 2 ? (set ^ t0) & 1 : 0;  // this set's first tile of the unit
      const int units0 = n_unit[0], units1 = n_unit[1];
      if (both || kSets == 1 || (t0 & 1) == 0) ++n_unit[0];
      if (both || (kSets == 2 && (t0 & 1) == 1)) ++n_unit[1];
      t0 += s.n;
      if (begin >= s.n) continue;  // a single tile, the other set's
      const int per_tile = kTile >> a.block_shift;
      int j_in0, j_in1;  // the tiles that every row sees whole
      whole_tiles(a, s, s.u.p0, s.u.p1, j_in0, j_in1);
      float l[RW];  // this slot's share of the rows' sums
#pragma unroll
      for (int i = 0; i < RW; ++i) l[i] = 0.f;
      bool fresh = true;  // a new reference is needed
      for (int j = begin; j < s.n; j += kSets) {
        const int t = t0 - s.n + j;
        const bool inside = j >= j_in0 && j < j_in1;
        int from = 0, to = R;  // the rows that see this thread's slot
        if (!inside) {
          // the token at p0 + tok sees the slot from tok = pos - p0 on, for `window` tokens, a sink always
          const int v = (s.tile0 + j) * per_tile + (kv >> a.block_shift);
          const int pos = block_pos(a, s.u, v) + (kv & ((1 << a.block_shift) - 1));
          const int d = pos - s.u.p0;
          from = d <= 0 ? 0 : d >= a.tokens ? R : d * a.g;
          if (a.window && pos >= a.n_sink) to = d + a.window <= 0 ? 0 : d + a.window >= a.tokens ? R : (d + a.window) * a.g;
        }
        ok = wait(&sh->s_full[t & 1], (t >> 1) & 1);
        if (!ok) break;
        tc::tc_fence_after();
        float x[RW];
        tc::tmem_ld<RW>(lane_base + (t & 1) * R, x);
        tc::tmem_ld_wait();
        if (!inside) {
#pragma unroll
          for (int i = 0; i < RW; ++i)
            if (row0 + i < from || row0 + i >= to) x[i] = hidden;
        }
        const bool head = j == begin;
        fresh = head;
        float y[RW];
        if (!head) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < RW; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(ref + i);
            unpack_f32x2(fma_f32x2(pack_f32x2(x[i], x[i + 1]), cc, pack_f32x2(-m.x, -m.y)), y[i], y[i + 1]);
            unpack_f32x2(fma_f32x2(pack_f32x2(x[i + 2], x[i + 3]), cc, pack_f32x2(-m.z, -m.w)), y[i + 2], y[i + 3]);
            top = fmaxf(fmaxf(top, fmaxf(y[i], y[i + 1])), fmaxf(y[i + 2], y[i + 3]));
          }
          const int at = sync & 1;
          if (__any_sync(~0u, top > kRescaleAt) && lane == 0) sh->need[grp][at] = t + 1;
          ok = meet();
          if (!ok) break;
          fresh = sh->need[grp][at] == t + 1;
          if (fresh) {  // the scores once more (S is still there: P has not been written)
            tc::tmem_ld<RW>(lane_base + (t & 1) * R, x);
            tc::tmem_ld_wait();
            if (!inside) {
#pragma unroll
              for (int i = 0; i < RW; ++i)
                if (row0 + i < from || row0 + i >= to) x[i] = hidden;
            }
          }
        }
        if (fresh) {
          // each row's maximum over the tile's 128 slots, by warp then over the group's warps
#pragma unroll
          for (int i = 0; i < RW; ++i) y[i] = x[i] * c2;
          const float mine = fold_lanes<RW, true>(y, lane);
          // the other set's group has read this one's last sums
          if (head && kSets == 2 && n_pair > 0) ok = wait(&sh->pair_got[rg], (n_pair - 1) & 1);
          if (!ok) break;
          const float old = head ? kUnset : ref[fold_row];
          sh->warp_part[grp][w4][fold_row] = mine;
          ok = meet();
          if (!ok) break;
          const float (*part)[RW] = sh->warp_part[grp];
          const float m = fmaxf(fmaxf(old, fmaxf(part[0][fold_row], part[1][fold_row])),
                                fmaxf(part[2][fold_row], part[3][fold_row]));
          ref[fold_row] = m;  // the four warps write the same values
          scale[fold_row] = tc::ex2_approx(old - m);
          __syncwarp();
          if (!head) {
            // the sums so far and this thread's lane of O^T, after the set's last product
            const int last = t - kSets;
            ok = wait(&sh->p_empty[last % C::kPBufs], (last / C::kPBufs) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            tc::tmem_ld<RW>(t_o + set * R, y);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < RW; ++i) l[i] *= scale[i], y[i] *= scale[i];
            tc::tmem_st<RW>(t_o + set * R, y);
            tc::tmem_st_wait();
          }
#pragma unroll
          for (int i = 0; i < RW; ++i) y[i] = fmaf(x[i], c2, -ref[i]);
        }
        uint32_t pk[RW / 2];
#pragma unroll
        for (int i = 0; i < RW; i += 2) {
          const float e0 = tc::ex2_approx(y[i]), e1 = tc::ex2_approx(y[i + 1]);
          l[i] += e0, l[i + 1] += e1;
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(e0, e1);
          pk[i / 2] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        ok = wait(&sh->p_empty[t % C::kPBufs], ((t / C::kPBufs) & 1) ^ 1);
        if (!ok) break;
        uint8_t* p = p_row + (t % C::kPBufs) * C::kPBytes;
#pragma unroll
        for (int i = 0; i < RW / 8; ++i)
          *reinterpret_cast<uint4*>(p + tc::swizzled<C::kPPitch>(kv, piece0 + i)) =
              make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->p_full[t & 1]));
      }
      if (!ok) break;
      // ---------------------------------------------------------------- the unit's rows
      // rows' sums over the 128 slots: lanes, then the group's warps in order
      if (fresh) ok = meet();  // the last tile's maxima, in the same place, have been read
      if (!ok) break;
      const float mine = fold_lanes<RW, false>(l, lane);
      sh->warp_part[grp][w4][fold_row] = mine;
      auto row_sum = [&](int of) {
        const float (*part)[RW] = sh->warp_part[of];
        return (part[0][fold_row] + part[1][fold_row]) + (part[2][fold_row] + part[3][fold_row]);
      };
      float lse2, f0, f1 = 0.f;  // the row's log2-sum-exp; the factors of its O^T, of the first and second set's
      if (both) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->pair_put[rg]));
        ok = wait(&sh->pair_put[rg], n_pair & 1);
        if (!ok) break;
        const int g0 = rg * 2;
        const float r0 = sh->ref[0][row0 + fold_row], r1 = sh->ref[kSets - 1][row0 + fold_row], m = fmaxf(r0, r1);
        f0 = tc::ex2_approx(r0 - m), f1 = tc::ex2_approx(r1 - m);
        const float sum = row_sum(g0) * f0 + row_sum(g0 + 1) * f1, inv = sum > 0.f ? 1.f / sum : 0.f;
        f0 *= inv, f1 *= inv;
        lse2 = sum > 0.f ? m + log2f(sum) : -INFINITY;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->pair_got[rg]));
        ++n_pair;
      } else {
        ok = meet();
        if (!ok) break;
        const float sum = row_sum(grp);
        f0 = sum > 0.f ? 1.f / sum : 0.f;
        lse2 = sum > 0.f ? ref[fold_row] + log2f(sum) : -INFINITY;
        ok = meet();  // read by all four before the next unit writes there
        if (!ok) break;
      }
      const bool partial = s.n < s.u.ntiles;
      const int64_t pbase = (int64_t(2) * blockIdx.x + (s.tile0 > 0 ? 0 : 1)) * R + row0;
      const int n_rows = s.ntok * a.g - row0;  // of this group's
      if (w4 == 0 && (set == 0 || !both) && fold_row * (32 / RW) == lane && fold_row < n_rows) {
        const int row = row0 + fold_row;
        if (partial)
          a.plse[pbase + fold_row] = lse2;
        else if (a.lse)
          a.lse[int64_t(s.row0 + row / a.g) * a.Hq + s.h * a.g + row % a.g] = lse2 * kLn2;
      }
      ok = (both || set == 0 ? wait(&sh->o_full[0], units0 & 1) : true) &&
           (both || set == 1 ? wait(&sh->o_full[kSets - 1], units1 & 1) : true);
      if (!ok) break;
      tc::tc_fence_after();
      // N rows from row r of the group's on, already divided, this thread's lane of the head
      auto put = [&](auto n_of, int r, const float* o) {
        constexpr int N = decltype(n_of)::value;
        if (partial) {
          float* dst = a.partial + (pbase + r) * D + kv;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (r + i < n_rows) dst[i * D] = o[i];
        } else {
          const int tok = (row0 + r) / a.g;
          int hh = row0 + r - tok * a.g;
          __nv_bfloat16* dst = a.out + (int64_t(s.row0 + tok) * a.Hq + s.h * a.g + hh) * D + kv;
          const int64_t wrap = int64_t(a.Hq - a.g) * D;  // from a token's last head to the next token's first
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (r + i < n_rows) *dst = __float2bfloat16(o[i]);
            dst += D;
            if (++hh == a.g) hh = 0, dst += wrap;
          }
        }
      };
      // O^T has been read: the sets' next units may overwrite it
      auto read = [&](int of, uint32_t count) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_n(tc::smem_u32(&sh->o_read[of]), count);
      };
      // TMEM lane = lane of the head; lanes from D on hold nothing
      if (both) {  // the sets' groups of the same rows write half of them each
        constexpr int N = RW / 2;
        const int r = set * N;
        float o[N], o1[N];
        tc::tmem_ld<N>(t_o + r, o);
        tc::tmem_ld<N>(t_o + R + r, o1);
        tc::tmem_ld_wait();
        read(0, 1);
        read(kSets - 1, 1);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float a0 = __shfl_sync(~0u, f0, (r + i) * (32 / RW)), a1 = __shfl_sync(~0u, f1, (r + i) * (32 / RW));
          o[i] = o[i] * a0 + o1[i] * a1;
        }
        if (kv < D) put(std::integral_constant<int, N>(), r, o);
      } else {
        float o[RW];
        tc::tmem_ld<RW>(t_o + set * R, o);
        tc::tmem_ld_wait();
        read(set, kSets);
#pragma unroll
        for (int i = 0; i < RW; ++i) o[i] *= __shfl_sync(~0u, f0, i * (32 / RW));
        if (kv < D) put(std::integral_constant<int, RW>(), 0, o);
      }
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 3u, uint32_t(t0) | uint32_t(warp) << 24);
    }
  }

  __syncthreads();
  if (sh->abort) {  // MMAs may be in flight: wait (bounded) before TMEM is freed
    if ((warp == kSWarp || warp == kOWarp) && sh->pending[warp - kSWarp]) {
      if (tc::elect_one()) tc::mma_commit(tc::smem_u32(&sh->drain[warp - kSWarp]));
      __syncwarp();
      const volatile int never = 0;
      tc::mbar_wait_bounded(tc::smem_u32(&sh->drain[warp - kSWarp]), 0, tc::deadline_after_ns(200000000ull), &never);
    }
    __syncthreads();
  }
  if (warp == kSWarp) tc::tmem_dealloc(tmem, C::kTmemCols);
}

template <int D, int R>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int n_cta,
                   cudaStream_t s) {
  static bool done[tch::kMaxDevices] = {};
  static std::mutex mu;
  constexpr int kSmem = Cfg<D, R>::kSmem;
  const cudaError_t e = tch::set_smem_once(window_kernel<D, R>, kSmem, done, &mu);
  return e != cudaSuccess ? e : launch_pdl(window_kernel<D, R>, dim3(n_cta), dim3(kThreads), kSmem, s, q, k, v, a);
}

}  // namespace

cudaError_t launch_attention_windows(int D, int unit_rows, const CUtensorMap& q, const CUtensorMap& k,
                                     const CUtensorMap& v, const attn::AttnArgs& a, int n_cta, cudaStream_t s) {
  if (D == 64) switch (unit_rows) {
      case 16: return launch<64, 16>(q, k, v, a, n_cta, s);
      case 32: return launch<64, 32>(q, k, v, a, n_cta, s);
      case 64: return launch<64, 64>(q, k, v, a, n_cta, s);
      default: return launch<64, 128>(q, k, v, a, n_cta, s);
    }
  switch (unit_rows) {
    case 16: return launch<128, 16>(q, k, v, a, n_cta, s);
    case 32: return launch<128, 32>(q, k, v, a, n_cta, s);
    case 64: return launch<128, 64>(q, k, v, a, n_cta, s);
    default: return launch<128, 128>(q, k, v, a, n_cta, s);
  }
}

}  // namespace dspark
