// The attention of short windows: all (token, head) rows of a unit fit one tile of R = 16, 32, 64 or (D = 128) 128.
//
// Bound by reading K and V once, so a KV tile's way through the SM has to be short: the products are taken
// transposed,
//     S^T = K Q^T        [128 slots x R]   (tcgen05, M = 128, N = R; fp32 in TMEM)
//     P^T = 2^(c S^T - m)                   (bf16, shared memory), partial sums of P per slot in registers
//     O^T += V^T P^T     [D x R]            (tcgen05, fp32 in TMEM)
// so that a thread holds one KV slot and some of the rows, and all softmax warps have work however few the rows
// are.  (With the rows on TMEM lanes instead, 32 rows sat in one warp per stream: a unit of 10 tiles at 32
// rows took 24 us per CTA.)  A tile's way is a chain of latencies, and so are the first and the last tile of
// a unit.  So an SM runs two pipelines side by side, each with its own range of the work, ring, S^T, P^T and O^T;
// where tensor memory (R = 128) or shared memory (R = 64 with D = 128) does not allow two, one pipeline has all
// sixteen softmax warps.
//
// m is a reference that only keeps the exponentials in range, the same for all slots of a row: weights of up to
// 2^16 give the same result, since the sum is divided out and neither fp32 nor bf16 loses bits there.  So it is
// set from a unit's first tile and checked against kRescaleAt, not recomputed, on the others.
// P is rounded to bf16 for the second product (relative 2^-9 a weight), its sum is taken before that, in fp32: the
// outputs' error against 64 bits is 0.0023 of their size, that of a product with fp32 weights and one rounding
// 0.0017.
//
// GB300, D 128, 8 KV heads: 2 requests of 16 rows over 125000 positions 152 us (1.02 GB of K and V, 6.7 TB/s: 99% of the
// measured copy bandwidth); 256 of 8 rows, window 4096, 636 us; window 1024, 184 us (90%), where the ~20 us of
// launches, the cut of the work, first loads and join are a tenth; one token over 1500 positions 9 us, nearly all of
// it those.  D 64, 64 rows to a KV head: 135 us of 85 (61%): softmax-bound, a warp's chain through a tile (its
// stalls: tensor memory and barriers 3.5 cycles an instruction, fixed latencies 1.8).  Slower there, each measured: sums in packed pairs and
// three-way maxima (140 us); a unit's rows read after the next one's first tile (139); each step of a tile once, in a loop of rounds
// (154); sums after P is handed on (144); one pipeline in place of two (window 4096: 417 us, 344).  With rows on lanes, window 1024: 304 us,
// transposed 206, all before the second pipeline.
#include "attention_common.cuh"

namespace dspark {
namespace {

using namespace attn;

// Sixteen softmax warps in groups of four; a group takes a share of the rows of its pipeline's tiles.  Then a
// TMA warp for each pipeline, and an MMA warp for each.
constexpr int kGroups = 4, kThreads = (kGroups + 1) * 128;
constexpr int kTmaWarp = 4 * kGroups, kMmaWarp = kTmaWarp + 2;
// Registers: launched with 640 x 96; the softmax warps take what the others give back (512 x 104 + 128 x 56 <= 640 x 96).
constexpr int kSoftmaxRegs = 104, kOtherRegs = 56;
constexpr int kMaxSlots = 8;

constexpr int sets_of(int D, int R) { return R * D >= 64 * 128 ? 1 : 2; }

template <int D, int R>
struct Shared {
  static constexpr int kSets = sets_of(D, R), kRowGroups = kGroups / kSets, kRows = R / kRowGroups;
  uint64_t q_full[kSets][2], q_empty[kSets][2], full[kSets][kMaxSlots], empty[kSets][kMaxSlots];
  uint64_t s_full[kSets][2], p_full[kSets], p_empty[kSets], o_full[kSets], o_read[kSets];
  uint64_t group[kGroups], drain[kSets];
  uint32_t tmem_base;
  volatile int abort;
  int pending[kSets];        // the MMA warp has issued something
  int n_put[kSets], n_q[kSets];  // copies issued: tiles, units' Q
  int need[kGroups][2];      // [parity]: the last tile at which a warp asked for a new reference
  Start start[kSets];
  float warp_max[kGroups][4][kRows], warp_sum[kGroups][4][kRows];  // by warp: the rows' maxima of a tile, sums of a unit
  alignas(16) float ref[kSets][R];                                 // the rows' references, read four at a time
};

template <int D, int R>
struct Cfg {
  static constexpr int kSets = sets_of(D, R), kRowGroups = kGroups / kSets;
  static constexpr int kHalves = D / 64;                    // 128-byte swizzled column blocks of a tile
  static constexpr int kSlotBytes = kTile * D * 2;
  static constexpr int kQBytes = R * D * 2, kQBufs = R * D < 32 * 128 || (R == 64 && D == 128) ? 2 : 1;  // where they fit
  static constexpr int kPPitch = R < 64 ? R * 2 : 128;       // bytes of a slot's row of P, R > 64: in two chunks
  static constexpr int kPBytes = kTile * R * 2;
  // O^T has M = 128 also where D = 64: its lanes 64 .. 127 come from the 16 KB behind the V tile, whatever
  // they hold, and are not read
  static constexpr int kBehind = kSets * (kQBytes * kQBufs + kPBytes);
  static constexpr int kPad = D == 64 && kBehind < 16384 ? 16384 - kBehind : 0;
  static constexpr int kRoom = (232448 - int(sizeof(Shared<D, R>)) - kBehind - kPad) / kSlotBytes / kSets;
  static constexpr int kSlots = kRoom < kMaxSlots ? kRoom : kMaxSlots;  // ring of a pipeline
  static constexpr int kSmem = kSets * kSlots * kSlotBytes + kBehind + kPad + int(sizeof(Shared<D, R>));
  static constexpr int kUsedCols = kSets * 3 * R;            // per pipeline: S^T twice, O^T
  static constexpr int kTmemCols = kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
  static_assert(kSlots >= 3 && kUsedCols <= 512 && kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "layout");
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
  constexpr int kSets = C::kSets, kRowGroups = C::kRowGroups, RW = R / kRowGroups;  // RW: rows per thread
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sRing = smem;
  uint8_t* sQ = sRing + kSets * C::kSlots * C::kSlotBytes;
  uint8_t* sP = sQ + kSets * C::kQBufs * C::kQBytes;
  Shared<D, R>* sh = reinterpret_cast<Shared<D, R>*>(sP + kSets * C::kPBytes + C::kPad);
  PlanScratch& plan = *reinterpret_cast<PlanScratch*>(sRing);  // before the first load
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // the same for the warp, and known to be
  const int tile_rows = a.tokens * a.g;

  if (warp == 0) {  // barriers: lane i those of number i
    for (int z = 0; z < kSets; ++z) {
      if (lane < 2) {
        tc::mbar_init(tc::smem_u32(&sh->q_full[z][lane]), 1);
        tc::mbar_init(tc::smem_u32(&sh->q_empty[z][lane]), 1);
        tc::mbar_init(tc::smem_u32(&sh->s_full[z][lane]), 1);
      }
      if (lane < C::kSlots) {
        tc::mbar_init(tc::smem_u32(&sh->full[z][lane]), 1);
        tc::mbar_init(tc::smem_u32(&sh->empty[z][lane]), 1);
      }
    }
    if (lane < kSets) {
      tc::mbar_init(tc::smem_u32(&sh->p_full[lane]), 4 * kRowGroups);
      tc::mbar_init(tc::smem_u32(&sh->p_empty[lane]), 1);
      tc::mbar_init(tc::smem_u32(&sh->o_full[lane]), 1);
      tc::mbar_init(tc::smem_u32(&sh->o_read[lane]), 4 * kRowGroups);
      tc::mbar_init(tc::smem_u32(&sh->drain[lane]), 1);
      sh->pending[lane] = 0;
      sh->start[lane].count = 0;
    }
    if (lane < kGroups) {
      tc::mbar_init(tc::smem_u32(&sh->group[lane]), 4);
      sh->need[lane][0] = sh->need[lane][1] = 0;
    }
    if (lane == 0) sh->abort = 0, plan.bad = 0, plan.n_long = 0;
    tc::fence_mbar_init();
  }
  if (tid == 32) {
    tc::prefetch_tensormap(&map_q);
    tc::prefetch_tensormap(&map_k);
    tc::prefetch_tensormap(&map_v);
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tc::smem_u32(&sh->tmem_base), C::kTmemCols);
    tc::tmem_relinquish();
  }
  // A unit's Q is always `tokens` rows, beyond its last the next request's (or zeros past the last packed row), whose
  // results nobody stores.  Rows of the tile beyond those are never loaded: zeros, so that their scores are 0.
  for (int i = tid; i < kSets * C::kQBufs * C::kQBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  pdl_enter();
  const Cut cut = plan_ranges<kSets>(a, sh->start, plan, a.tokens);
  tc::fence_proxy_async_smem();  // the zeros, and the plan's scratch, which lies where TMA writes
  __syncthreads();
  const uint32_t tmem = sh->tmem_base;

  if (warp >= kTmaWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp >= kTmaWarp && warp < kTmaWarp + kSets) {
    // --------------------------------------------------------------------- TMA producer
    // In the order of load_in_order over all tiles of the range; a unit's Q with its first K.
    const int set = warp - kTmaWarp;
    const uint32_t range = blockIdx.x + set * gridDim.x;
    const TmaWaiter wait{{&sh->abort, a.timeout_ns}};
    const uint64_t keep = tc::policy_evict_last(), stream = tc::policy_evict_first();
    uint8_t* ring_mem = sRing + set * C::kSlots * C::kSlotBytes;
    Ring<C::kSlots> ring;
    int n_seg = 0, n_put = 0;
    int4 info = make_int4(0, 0, 0, 0);
    Cursor cur(sh->start[set], a.tokens);
    struct Ahead {
      TileLoad t;
      int row0;  // >= 0: the unit's first tile here
      bool there;
    };
    auto fetch = [&]() {  // the next tile's pages
      Ahead f = {};
      f.there = cur.next(a);
      if (!f.there) return f;
      const Segment& s = cur.s;
      f.t = tile_load(a, s, cur.j, lane);
      f.row0 = cur.first() ? s.row0 : -1;
      if (cur.first() && s.tile0 == 0 && s.n < s.u.ntiles)
        info = make_int4(1 + cut.ranges(range + 1, uint32_t(s.u.ntiles - s.n)), s.row0, s.ntok, s.h);
      return f;
    };
    auto put = [&](const CUtensorMap* map, const Ahead& f) {
      if (!wait(&sh->empty[set][ring.slot], ring.phase ^ 1)) return false;
      issue_tile<C::kHalves>(a, map, f.t, tc::smem_u32(ring_mem + ring.slot * C::kSlotBytes),
                             tc::smem_u32(&sh->full[set][ring.slot]), stream, lane);
      ++n_put;
      ring.step();
      return true;
    };
    auto put_k = [&](const Ahead& f) {
      if (!put(&map_k, f)) return false;
      if (f.row0 < 0) return true;
      const int b = n_seg % C::kQBufs;
      if (!wait(&sh->q_empty[set][b], ((n_seg / C::kQBufs) & 1) ^ 1)) return false;
      if (lane == 0) {
        const uint32_t bar = tc::smem_u32(&sh->q_full[set][b]);
        tc::mbar_arrive_expect_tx(bar, uint32_t(tile_rows * 128 * C::kHalves));
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tc::tma_load_3d(tc::smem_u32(sQ + (set * C::kQBufs + b) * C::kQBytes + hf * (R * 128)), &map_q, bar, hf * 64,
                          f.t.head * a.g, f.row0, keep);
      }
      ++n_seg;
      return true;
    };
    const bool ok = load_in_order(fetch, put_k, [&](const Ahead& f) { return put(&map_v, f); });
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 1u, uint32_t(n_seg));
    }
    if (lane == 0) {
      if (!ok) info.x = 0;
      a.info[range] = info;
      sh->n_put[set] = n_put, sh->n_q[set] = n_seg;
    }
  } else if (warp >= kMmaWarp && warp < kMmaWarp + kSets) {
    // ------------------------------------------------------------ the two products of each tile
    const uint32_t idesc_s = tc::idesc_bf16_f32(kTile, R) | a.negate_q << 1;  // Q is the second operand here
    constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, R) | tc::kIdescAMajorMN | tc::kIdescBMajorMN;
    const int set = warp - kMmaWarp;
    const Waiter wait{&sh->abort, a.timeout_ns};
    uint8_t* ring_mem = sRing + set * C::kSlots * C::kSlotBytes;
    const uint32_t t_s = tmem + set * 3 * R, t_o = t_s + 2 * R;
    const uint64_t dk = tc::sdesc_kmajor_sw128(tc::smem_u32(ring_mem));
    const uint64_t dq = tc::sdesc_kmajor_sw128(tc::smem_u32(sQ + set * C::kQBufs * C::kQBytes));
    const uint64_t dv = tc::sdesc_mnmajor<128>(tc::smem_u32(ring_mem), kTile * 128);
    const uint64_t dp = tc::sdesc_mnmajor<C::kPPitch>(tc::smem_u32(sP + set * C::kPBytes), kTile * 128);
    Ring<C::kSlots> ring;
    int n_seg = 0, n_s = 0, t = 0, units = 0, j0 = 0, j1 = 0;
    Cursor kc(sh->start[set], a.tokens), vc(sh->start[set], a.tokens);
    auto s_product = [&]() {  // S^T of the tile at kc; the S before last has been read (its P is there)
      const int b = n_seg % C::kQBufs;
      if (kc.first() && !wait(&sh->q_full[set][b], (n_seg / C::kQBufs) & 1)) return false;
      if (!wait(&sh->full[set][ring.slot], ring.phase)) return false;
      tc::tc_fence_after();
      const uint64_t dk_t = dk + uint32_t(ring.slot * (C::kSlotBytes >> 4)), dq_t = dq + uint32_t(b * (C::kQBytes >> 4));
      const bool last = kc.last();
      if (tc::elect_one()) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          tc::mma_bf16(t_s + (n_s & 1) * R, dk_t + (((i / 4) * (kTile * 128) + (i % 4) * 32) >> 4),
                       dq_t + (((i / 4) * (R * 128) + (i % 4) * 32) >> 4), idesc_s, i != 0);
        tc::mma_commit(tc::smem_u32(&sh->s_full[set][n_s & 1]));
        tc::mma_commit(tc::smem_u32(&sh->empty[set][ring.slot]));
        if (last) tc::mma_commit(tc::smem_u32(&sh->q_empty[set][b]));
      }
      __syncwarp();
      ring.step();
      ++n_s;
      if (last) ++n_seg;
      return true;
    };
    bool more = kc.next(a);
    bool ok = !more || s_product();
    if (ok && more) {
      more = kc.next(a);
      ok = !more || s_product();
    }
    for (; ok && vc.next(a); ++t) {
      const bool first = vc.first(), last = vc.last();
      ok = wait(&sh->full[set][ring.slot], ring.phase);
      if (!ok) break;
      if (first) whole_tiles(a, vc.s, vc.s.u.p1, vc.s.u.p0, j0, j1);
      // while the softmax works on this tile
      if (vc.j < j0 || vc.j >= j1) clear_unseen<C::kHalves>(a, vc.s, vc.j, ring_mem + ring.slot * C::kSlotBytes, lane);
      ok = wait(&sh->p_full[set], t & 1);
      if (ok && first) ok = wait(&sh->o_read[set], (units++ & 1) ^ 1);  // the unit before has been read
      if (!ok) break;
      tc::tc_fence_after();
      const uint64_t dv_t = dv + uint32_t(ring.slot * (C::kSlotBytes >> 4));
      if (tc::elect_one()) {
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
          tc::mma_bf16(t_o, dv_t + ((i * 2048) >> 4), dp + ((i * 16 * C::kPPitch) >> 4), idesc_o, !first || i != 0);
        tc::mma_commit(tc::smem_u32(&sh->p_empty[set]));
        tc::mma_commit(tc::smem_u32(&sh->empty[set][ring.slot]));
        if (last) tc::mma_commit(tc::smem_u32(&sh->o_full[set]));
      }
      __syncwarp();
      ring.step();
      if (more) {
        more = kc.next(a);
        ok = !more || s_product();
      }
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 2u, uint32_t(t));
    }
    if (lane == 0) sh->pending[set] = n_s > 0;
  } else if (warp < kTmaWarp) {
    // ------------------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const Waiter wait{&sh->abort, a.timeout_ns};
    const int grp = warp >> 2, w4 = warp & 3;
    const int kv = w4 * 32 + lane;  // this thread's slot of each tile = TMEM lane
    const int set = grp % kSets, row0 = grp / kSets * RW;  // and its rows
    const uint32_t t_s = tmem + (uint32_t(w4 * 32) << 16) + set * 3 * R + row0, t_o = t_s + 2 * R;
    const float c2 = a.c2;
    const unsigned long long cc = pack_f32x2(c2, c2);
    float* ref = sh->ref[set] + row0;
    // where this thread's row of P goes: 16-byte pieces, from the first row of the group on
    uint8_t* p_row = sP + set * C::kPBytes + (R == 128 ? (row0 / 64) * (kTile * 128) : 0);
    const int piece0 = (R == 128 ? row0 % 64 : row0) / 8;
    // the row that this lane holds after a fold (the lanes of a row hold the same)
    const int fold_row = lane / (32 / RW);
    int t = 0, sync = 0, units = 0;
    bool ok = true;
    Walk walk(sh->start[set], a.tokens);
    Segment s = {};
    // the group's four warps: everything before on all of them is visible after
    auto arrive = [&]() {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->group[grp]));
    };
    auto meet = [&]() {
      arrive();
      return wait(&sh->group[grp], sync++ & 1);
    };
    while (ok && walk.next(a, s)) {
      const int per_tile = kTile >> a.block_shift;
      int j_in0, j_in1;  // the tiles that every row sees whole
      whole_tiles(a, s, s.u.p0, s.u.p1, j_in0, j_in1);
      float l[RW];  // this slot's share of the rows' sums
#pragma unroll
      for (int i = 0; i < RW; ++i) l[i] = 0.f;
      for (int j = 0; j < s.n; ++j, ++t) {
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
        ok = wait(&sh->s_full[set][t & 1], (t >> 1) & 1);
        if (!ok) break;
        tc::tc_fence_after();
        float y[RW];  // the only array beside l: what is needed once more is loaded once more (S is there until P is)
        auto load_scores = [&]() {
          tc::tmem_ld<RW>(t_s + (t & 1) * R, y);
          tc::tmem_ld_wait();
          if (!inside) {
#pragma unroll
            for (int i = 0; i < RW; ++i)
              if (row0 + i < from || row0 + i >= to) y[i] = -INFINITY;
          }
        };
        auto refer = [&]() {  // scores to exponents; the largest
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < RW; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(ref + i);
            unpack_f32x2(fma_f32x2(pack_f32x2(y[i], y[i + 1]), cc, pack_f32x2(-m.x, -m.y)), y[i], y[i + 1]);
            unpack_f32x2(fma_f32x2(pack_f32x2(y[i + 2], y[i + 3]), cc, pack_f32x2(-m.z, -m.w)), y[i + 2], y[i + 3]);
            top = fmaxf(fmaxf(top, fmaxf(y[i], y[i + 1])), fmaxf(y[i + 2], y[i + 3]));
          }
          return top;
        };
        auto weigh = [&]() {
#pragma unroll
          for (int i = 0; i < RW; ++i) y[i] = tc::ex2_approx(y[i]);
        };
        load_scores();
        bool fresh = j == 0;  // a new reference is needed
        if (j > 0) {
          const float top = refer();
          const int at = sync & 1;
          if (__any_sync(~0u, top > kRescaleAt) && lane == 0) sh->need[grp][at] = t + 1;
          arrive();
          weigh();  // while the others arrive; done again where the reference moves
          ok = wait(&sh->group[grp], sync++ & 1);
          if (!ok) break;
          fresh = sh->need[grp][at] == t + 1;
          if (fresh) load_scores();
        }
        if (fresh) {
          // each row's maximum over the tile's 128 slots, by warp then over the group's warps
#pragma unroll
          for (int i = 0; i < RW; ++i) y[i] *= c2;
          const float mine = fold_lanes<RW, true>(y, lane);
          const float old = j == 0 ? kUnset : ref[fold_row];
          sh->warp_max[grp][w4][fold_row] = mine;
          ok = meet();
          if (!ok) break;
          const float (*part)[RW] = sh->warp_max[grp];
          const float m = fmaxf(fmaxf(old, fmaxf(part[0][fold_row], part[1][fold_row])),
                                fmaxf(part[2][fold_row], part[3][fold_row]));
          ref[fold_row] = m;  // the four warps write the same values
          __syncwarp();
          if (j > 0) {
            // the sums so far and this thread's lane of O^T, after the last product
            ok = wait(&sh->p_empty[set], (t - 1) & 1);
            if (!ok) break;
            tc::tc_fence_after();
            const float alpha = tc::ex2_approx(old - m);
            tc::tmem_ld<RW>(t_o, y);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < RW; ++i) {
              const float al = __shfl_sync(~0u, alpha, i * (32 / RW));
              l[i] *= al, y[i] *= al;
            }
            tc::tmem_st<RW>(t_o, y);
            tc::tmem_st_wait();
          }
          load_scores();
          refer();
          weigh();
        }
        uint32_t pk[RW / 2];
#pragma unroll
        for (int i = 0; i < RW; i += 2) {
          l[i] += y[i], l[i + 1] += y[i + 1];
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(y[i], y[i + 1]);
          pk[i / 2] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        ok = wait(&sh->p_empty[set], (t & 1) ^ 1);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < RW / 8; ++i)
          *reinterpret_cast<uint4*>(p_row + tc::swizzled<C::kPPitch>(kv, piece0 + i)) =
              make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->p_full[set]));
      }
      if (!ok) break;
      // ---------------------------------------------------------------- the unit's rows
      // rows' sums over the 128 slots: lanes, then the group's warps in order
      const float mine = fold_lanes<RW, false>(l, lane);
      sh->warp_sum[grp][w4][fold_row] = mine;
      ok = meet();
      if (!ok) break;
      const float (*part)[RW] = sh->warp_sum[grp];
      const float sum = (part[0][fold_row] + part[1][fold_row]) + (part[2][fold_row] + part[3][fold_row]);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN, in the log-sum-exp too
      const bool partial = s.n < s.u.ntiles;
      const int64_t pbase = (int64_t(2) * (blockIdx.x + set * gridDim.x) + (s.tile0 > 0 ? 0 : 1)) * R + row0;
      const int n_rows = s.ntok * a.g - row0;  // of this group's
      if (w4 == 0 && fold_row * (32 / RW) == lane && fold_row < n_rows) {
        const float lse2 = sum == 0.f ? -INFINITY : ref[fold_row] + log2f(sum);
        const int row = row0 + fold_row;
        if (partial)
          a.plse[pbase + fold_row] = lse2;
        else if (a.lse)
          a.lse[int64_t(s.row0 + row / a.g) * a.Hq + s.h * a.g + row % a.g] = lse2 * kLn2;
      }
      ok = wait(&sh->o_full[set], units++ & 1);
      if (!ok) break;
      tc::tc_fence_after();
      float o[RW];
      tc::tmem_ld<RW>(t_o, o);
      tc::tmem_ld_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->o_read[set]));  // the next unit may overwrite it
      if (kv < D) {  // TMEM lane = lane of the head; lanes from D on hold nothing
#pragma unroll
        for (int i = 0; i < RW; ++i) o[i] *= __shfl_sync(~0u, inv, i * (32 / RW));
        if (partial) {
          float* dst = a.partial + pbase * D + kv;
#pragma unroll
          for (int i = 0; i < RW; ++i)
            if (i < n_rows) dst[i * D] = o[i];
        } else {
          const int tok = row0 / a.g;
          int hh = row0 - tok * a.g;
          __nv_bfloat16* dst = a.out + (int64_t(s.row0 + tok) * a.Hq + s.h * a.g + hh) * D + kv;
          const int64_t wrap = int64_t(a.Hq - a.g) * D;  // from a token's last head to the next token's first
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            if (i < n_rows) *dst = __float2bfloat16(o[i]);
            dst += D;
            if (++hh == a.g) hh = 0, dst += wrap;
          }
        }
      }
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 3u, uint32_t(t) | uint32_t(warp) << 24);
    }
  }

  __syncthreads();
  if (sh->abort) {  // MMAs and copies may be in flight: wait (bounded) before TMEM is freed and the block ends
    const long long deadline = tc::deadline_after_ns(kDrainNs);
    const int set = (warp - kTmaWarp) % 2;
    if (warp >= kMmaWarp && set < kSets && sh->pending[set]) {
      if (tc::elect_one()) tc::mma_commit(tc::smem_u32(&sh->drain[set]));
      __syncwarp();
      const volatile int never = 0;
      tc::mbar_wait_bounded(tc::smem_u32(&sh->drain[set]), 0, deadline, &never);
    } else if (warp >= kTmaWarp && warp < kMmaWarp && set < kSets) {
      drain_copies(sh->full[set], C::kSlots, sh->n_put[set], deadline);
      drain_copies(sh->q_full[set], C::kQBufs, sh->n_q[set], deadline);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, C::kTmemCols);
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

int attention_window_sets(int D, int unit_rows) { return sets_of(D, unit_rows); }

cudaError_t launch_attention_windows(int D, int unit_rows, const CUtensorMap& q, const CUtensorMap& k,
                                     const CUtensorMap& v, const attn::AttnArgs& a, int n_cta, cudaStream_t s) {
  if (D == 64) switch (unit_rows) {
      case 16: return launch<64, 16>(q, k, v, a, n_cta, s);
      case 32: return launch<64, 32>(q, k, v, a, n_cta, s);
      default: return launch<64, 64>(q, k, v, a, n_cta, s);
    }
  switch (unit_rows) {
    case 16: return launch<128, 16>(q, k, v, a, n_cta, s);
    case 32: return launch<128, 32>(q, k, v, a, n_cta, s);
    case 64: return launch<128, 64>(q, k, v, a, n_cta, s);
    default: return launch<128, 128>(q, k, v, a, n_cta, s);
  }
}

}  // namespace dspark
