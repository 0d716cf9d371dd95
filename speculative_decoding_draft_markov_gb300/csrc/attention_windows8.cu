// The attention of short windows over the 8-bit cache: attention_windows.cu's pipelines with half the bytes to read.
//
//     S^T = K8 (Qh + Ql)^T      [128 slots x R]   (tcgen05 kind::f8f6f4, fp32 in TMEM)
//     x = S^T 2^(ek + eq) c,  P^T = 2^(x - m) 2^(ev - f) = Ph + Pl / 16   (e4m3, shared memory), sums of 2^(x - m) in registers
//     Oh^T | Ol^T += V8^T (Ph | Pl)^T  [D x 2R]   (tcgen05, fp32 in TMEM),   out = (Oh + Ol / 16) 2^f / l
//
// K and V go into the products as they lie in the cache; nothing is converted but the other operands, which one code of e4m3
// (relative error 2^-4) would be too little for, so each is a sum of two.
// Q's row is taken under a power of two of its own, 2^eq: the first part has the upper four of bf16's eight bits, the second
// what is left, exact for lanes down to 2^-9.8 of the row's largest, which lies above 224 = 2^7.8 of that power; smaller ones are
// off by at most half of the second part's least step, 2^-10 of the power, i.e. 2^-17.8 of the row's largest.  The slots'
// powers, ek, are one factor per thread, the rows' one per score.
// A weight has eight bits, as bf16 has (relative 2^-8), down to 2^-12 of the largest and an error of 2^-20 of it
// below; the second part is kept times 16 and in accumulators of its own for that.  V's contraction runs over slots, so its
// powers 2^ev have to go into P, and a V that lies 2^k below their reference has k bits fewer of its weight.
// P is kept inside e4m3's range by two references, a row's m, which lies kTop below its maximum of a unit's first tile, and f,
// the largest ev of a tile's slots.  Both are checked on each tile against kMost, f also for lying above all of the tile's ev by
// more than kFall (else a large V would take the weights' bits from all tiles behind it); they are set anew where they have to
// be, O^T and the sums with them.  The last check takes 2% (256 windows 117.6 us without it).
//
// GB300, 8 KV heads: D 128, 256 windows of 8 rows, window 1024, 120 us (81.5 by its bytes; over a bf16 cache 175); 2 requests of
// 16 rows over 125000 positions 104 us (77; 154); one token over 1500 positions 10.4 (9.7); D 64, 64 windows of 64 rows to a KV
// head, window 4096, 97 us (33; 83).  What bounds it is the chain of a tile's steps, some 3200 cycles for a pipeline with 64
// rows, and the softmax warps' instructions (0.6 of the issue slots): a satisfied wait costs about 200 cycles, a TMA load its
// warp 180, so K and V have a warp each (one for both took 3000 cycles a tile) and the exponent bytes come by 8-byte
// asynchronous copies (1000 cycles of bulk copies before).  The code has to stay small: with every step inlined where it is used
// (172 KB of instructions) the first three took 201 us, with each step there once 147.
// Slower, in us for 256 windows / 125000 positions / 64 rows: V converted to fp16 by four warps and P in fp16 237 / 178 / 178;
// eight softmax warps of 184 registers 129 / 116 / 109 where sixteen took 123 / 105 / 98; blocks of 64 slots 126 / 104 / 98
// beside the same; waits that may sleep 123 / 105 / 98 beside 118 / 102 / 94 (all of these without the last check).  Q split by plain loads took 33000 cycles for 64
// rows, copied to where it is split 20000.
#include "attention_common.cuh"
#include "kv8.cuh"

namespace dspark {
namespace {

using namespace attn;

// Sixteen softmax warps in groups of four; a group takes a share of the rows of its pipeline's tiles.  Then for each pipeline a
// warp that loads K, one that issues the products and one that loads V, and two warps that split Q (both for a lone pipeline).
constexpr int kGroups = 4, kThreads = (kGroups + 2) * 128;
constexpr int kKWarp = 4 * kGroups, kMmaWarp = kKWarp + 2, kVWarp = kMmaWarp + 2, kSplitWarp = kVWarp + 2;
// Registers: launched with 768 x 80; the softmax warps take what the others give back (512 x 96 + 256 x 48 = 768 x 80).
constexpr int kSoftmaxRegs = 96, kOtherRegs = 48;
constexpr int kMaxSlots = 8;
constexpr int kQBufs = 2, kQRing = 4;  // units whose Q, whose rows' factors are kept
// m lies kTop below a maximum; a score and a value's power together may outgrow the references up to kMost (e4m3 ends at
// 448 = 2^8.8)
constexpr float kTop = 6.f, kMost = 8.75f;
// V's reference may lie above a tile's largest power of two by this much.
constexpr int kFall = 4;

constexpr int sets_of(int D, int R) { return R == 128 ? 1 : 2; }

template <int D, int R>
struct Shared {
  static constexpr int kSets = sets_of(D, R), kRowGroups = kGroups / kSets, kRows = R / kRowGroups;
  // tiles whose exponent bytes are kept: a slot of the ring ahead of the products, which are two tiles ahead of the softmax
  static constexpr int kScales = 16;
  static_assert(kScales >= kMaxSlots + 3, "a tile's bytes are written anew when its softmax is over");
  uint64_t q_ready[kSets][kQRing], q_empty[kSets][kQBufs], full[kSets][kMaxSlots], empty[kSets][kMaxSlots];
  uint64_t sc_full[kSets][kScales];
  uint64_t s_full[kSets][2], p_full[kSets], p_empty[kSets], o_full[kSets], o_read[kSets];
  uint64_t group[kGroups], drain[kSets];
  uint32_t tmem_base;
  volatile int abort;
  int pending[kSets];          // the MMA warp has issued something
  int need[kGroups][2];        // [parity]: the last tile at which a warp asked for new references
  alignas(16) int low[kGroups][2][4];  // [parity], by warp: the last tile whose V it found to lie far below the reference
  Start start[kSets];
  int warp_byte[kGroups][4];   // by warp: the largest exponent byte of V in a tile
  float warp_max[kGroups][4][kRows], warp_sum[kGroups][4][kRows];  // by warp: the rows' maxima of a tile, sums of a unit
  alignas(16) float neg_ref[kSets][R];         // the rows' references, negated; read four at a time
  alignas(16) float row_by[kSets][R];          // what a row's sums, and its output, are to be multiplied by
  alignas(16) int row_at[kSets][R];            // where a row's output lies behind the unit's first; -1: nowhere
  alignas(16) float zeros[kRows];
  alignas(16) float row_factor[kSets][kQRing][R];  // 2^eq c
  alignas(16) uint16_t scales[kSets][kScales][kTile];
};

template <int D, int R>
struct Cfg {
  static constexpr int kSets = sets_of(D, R), kRowGroups = kGroups / kSets;
  static constexpr int kSplitWarps = 2 / kSets;              // of a pipeline
  static constexpr int kSlotBytes = kTile * D;               // a tile of codes: rows of D bytes, D-byte swizzled
  static constexpr int kQPart = R * D, kQBytes = 2 * kQPart;
  static constexpr int kPPitch = R < 64 ? R * 2 : 128;       // bytes of a slot's row of P, R > 64: in two chunks
  static constexpr int kPBytes = kTile * R * 2;
  static constexpr int kRoom = (232448 - int(sizeof(Shared<D, R>)) - kSets * (kQBytes * kQBufs + kPBytes)) / kSlotBytes / kSets;
  static constexpr int kSlots = kRoom < kMaxSlots ? kRoom : kMaxSlots;  // ring of a pipeline
  static constexpr int kSmem = kSets * (kSlots * kSlotBytes + kQBytes * kQBufs + kPBytes) + int(sizeof(Shared<D, R>));
  static constexpr int kUsedCols = kSets * 4 * R;            // per pipeline: S^T twice, Oh^T, Ol^T
  static constexpr int kTmemCols = kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
  static_assert(kSlots >= 3 && kUsedCols <= 512 && kQPart % 1024 == 0 && kPBytes % 1024 == 0, "layout");
};

// V's slots that no row of the unit sees hold whatever was there, NaN included, and 0 * NaN is NaN: their codes are
// cleared.  A whole warp, 16-byte stores, rotated so that the lanes spread over the banks.
template <int D>
__device__ __forceinline__ void clear_unseen_codes(const AttnArgs& a, const Segment& s, int j, uint8_t* tile, int lane) {
  const int first = (s.tile0 + j) * (kTile >> a.block_shift);
  for (int i = lane; i < kTile; i += 32) {
    const int pos = block_pos(a, s.u, first + (i >> a.block_shift)) + (i & ((1 << a.block_shift) - 1));
    if (pos <= s.u.p1 && (pos >= s.u.lo || pos < a.n_sink)) continue;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      *reinterpret_cast<uint4*>(tile + i * D + (((k + lane) & (D / 16 - 1)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
}

// Bits i = 0 .. 31 with from <= i < to.
__device__ __forceinline__ uint32_t bits32(int from, int to) {
  const uint32_t below = to >= 32 ? ~0u : to <= 0 ? 0u : (1u << to) - 1u;
  return from >= 32 ? 0u : from <= 0 ? below : below & (~0u << from);
}
// The largest of the lanes' values (NaN where all are).
__device__ __forceinline__ float warp_max_f32(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// A whole warp waits, as Waiter does, in fewer instructions: the limit begins with the first look that fails.
struct ShortWaiter {
  volatile int* abort;
  long long cycles;
  __device__ __forceinline__ bool operator()(const uint64_t* bar, uint32_t parity) const {
    const uint32_t b = tc::smem_u32(bar);
    bool ok = true;
    long long deadline = 0;
    while (!tc::mbar_try_wait(b, parity)) {
      const long long now = clock64();
      if (deadline == 0) deadline = now + cycles;
      if (*abort || now > deadline) {
        ok = false;
        break;
      }
    }
    return __all_sync(~0u, ok);
  }
  // Two barriers at once: a wait that finds its phase complete takes some 200 cycles all the same.
  __device__ __forceinline__ bool both(const uint64_t* bar, uint32_t parity, const uint64_t* bar2, uint32_t parity2) const {
    const uint32_t b = tc::smem_u32(bar), b2 = tc::smem_u32(bar2);
    bool ok = true;
    long long deadline = 0;
    while (!(tc::mbar_try_wait(b, parity) & tc::mbar_try_wait(b2, parity2))) {
      const long long now = clock64();
      if (deadline == 0) deadline = now + cycles;
      if (*abort || now > deadline) {
        ok = false;
        break;
      }
    }
    return __all_sync(~0u, ok);
  }
};
__device__ __forceinline__ long long cycles_of(uint64_t ns) { return tc::deadline_after_ns(ns) - clock64(); }

// Issue a tile's loads of codes.  One lane issues them all: issued by the blocks' own lanes, a load takes some 180 cycles.
template <int D>
__device__ __forceinline__ void issue_codes(const AttnArgs& a, const CUtensorMap* map, const TileLoad& t, uint32_t dst,
                                            uint32_t bar, uint64_t policy, int lane) {
  const int block_bytes = D << a.block_shift;
  int page = t.page;
  if (lane < t.n_blocks && (page < 0 || page >= a.n_pages)) {
    set_status(a.status, DSPARK_EINVAL);
    page = a.n_pages;  // outside the tensor: reads as zeros
  }
  const int head = __shfl_sync(~0u, t.head, 0), n = __shfl_sync(~0u, t.n_blocks, 0);
  if (lane == 0) tc::mbar_arrive_expect_tx(bar, uint32_t(n * block_bytes));
  __syncwarp();
  for (int i = 0; i < n; ++i) {
    const int to = __shfl_sync(~0u, page, i), slot = __shfl_sync(~0u, t.slot, i);
    if (tc::elect_one()) tc::tma_load_4d(dst + i * block_bytes, map, bar, 0, slot, head, to, policy);
    __syncwarp();
  }
}
// The exponent bytes of a tile's slots, four slots to a lane; zeros of any power of two where there is no page.  Every lane
// arrives at `bar` when its own are there: by its copy's end, or itself behind its store, which an arrival by copies does not order.
__device__ __forceinline__ void issue_scales(const Attn8Args& p, const TileLoad& t, uint16_t* dst, uint32_t bar, int lane) {
  const AttnArgs& a = p.a;
  const int block = (lane * 4) >> a.block_shift, in = (lane * 4) & ((1 << a.block_shift) - 1);
  const int page = __shfl_sync(~0u, t.page, block), slot = __shfl_sync(~0u, t.slot, block) + in;
  uint16_t* to = dst + lane * 4;
  if (block < t.n_blocks && page >= 0 && page < a.n_pages) {
    tc::async_copy_8(tc::smem_u32(to), p.kv_scale + 2 * (((int64_t(page) * a.Hkv + t.head) << a.page_shift) + slot));
    tc::async_copies_arrive(bar);
  } else {
    *reinterpret_cast<uint2*>(to) = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    tc::mbar_arrive(bar);
  }
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
    window8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ Attn8Args args) {
  using C = Cfg<D, R>;
  using Sh = Shared<D, R>;
  constexpr int kSets = C::kSets, kRowGroups = C::kRowGroups, RW = R / kRowGroups;  // RW: rows per thread
  const AttnArgs& a = args.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sRing = smem;
  uint8_t* sQ = sRing + kSets * C::kSlots * C::kSlotBytes;
  uint8_t* sP = sQ + kSets * kQBufs * C::kQBytes;
  Sh* sh = reinterpret_cast<Sh*>(sP + kSets * C::kPBytes);
  PlanScratch& plan = *reinterpret_cast<PlanScratch*>(sRing);  // before the first load
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // the same for the warp, and known to be

  if (warp == 0) {  // barriers: lane i those of number i
    for (int z = 0; z < kSets; ++z) {
      if (lane < kQRing) tc::mbar_init(tc::smem_u32(&sh->q_ready[z][lane]), C::kSplitWarps);
      if (lane < 2) {
        if (lane < kQBufs) tc::mbar_init(tc::smem_u32(&sh->q_empty[z][lane]), 1);
        tc::mbar_init(tc::smem_u32(&sh->s_full[z][lane]), 1);
      }
      if (lane < C::kSlots) {
        tc::mbar_init(tc::smem_u32(&sh->full[z][lane]), 1);
        tc::mbar_init(tc::smem_u32(&sh->empty[z][lane]), 1);
      }
      if (lane < Sh::kScales) tc::mbar_init(tc::smem_u32(&sh->sc_full[z][lane]), 32);
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
      for (int i = 0; i < 8; ++i) sh->low[lane][i / 4][i % 4] = 0;
    }
    for (int i = lane; i < Sh::kRows; i += 32) sh->zeros[i] = 0.f;
    if (lane == 0) sh->abort = 0, plan.bad = 0, plan.n_long = 0;
    tc::fence_mbar_init();
  }
  if (tid == 32) {
    tc::prefetch_tensormap(&map_k);
    tc::prefetch_tensormap(&map_v);
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tc::smem_u32(&sh->tmem_base), C::kTmemCols);
    tc::tmem_relinquish();
  }
  __syncthreads();
  pdl_enter();
  const Cut cut = plan_ranges<kSets>(a, sh->start, plan, a.tokens);
  tc::fence_proxy_async_smem();  // the plan's scratch lies where TMA writes
  __syncthreads();
  const uint32_t tmem = sh->tmem_base;

  int n_put = 0;  // loads that this warp has issued
  if (warp >= kKWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if ((warp >= kKWarp && warp < kKWarp + kSets) || (warp >= kVWarp && warp < kVWarp + kSets)) {
    // ------------------------------------------------------------------ K, and V, into the ring
    // Two warps, since a load costs the warp that issues it some 180 cycles.
    const bool loads_v = warp >= kVWarp;
    const int set = warp - (loads_v ? kVWarp : kKWarp);
    const uint32_t range = blockIdx.x + set * gridDim.x;
    const TmaWaiter wait{{&sh->abort, a.timeout_ns}};
    const uint64_t stream = tc::policy_evict_first();
    uint8_t* ring_mem = sRing + set * C::kSlots * C::kSlotBytes;
    const CUtensorMap* map = loads_v ? &map_v : &map_k;
    const uint32_t n_tiles = sh->start[set].count;
    int4 info = make_int4(0, 0, 0, 0);
    Cursor cur(sh->start[set], a.tokens);
    // The tiles' pages are looked up two tiles before they are wanted
    struct Ahead {
      TileLoad t;
      bool there;
    };
    Ahead now = {}, next = {}, last = {};
    bool ok = true;
    int i = -3;
    for (;; ++i) {
      if (i >= 0) {
        if (!now.there) break;
        const uint32_t at = ring_place(loads_v, uint32_t(i), n_tiles), slot = at % C::kSlots;
        ok = wait(&sh->empty[set][slot], (at / C::kSlots & 1) ^ 1);
        if (!ok) break;
        issue_codes<D>(a, map, now.t, tc::smem_u32(ring_mem + slot * C::kSlotBytes), tc::smem_u32(&sh->full[set][slot]), stream,
                       lane);
        if (!loads_v) {
          const int b = i % Sh::kScales;
          issue_scales(args, now.t, sh->scales[set][b], tc::smem_u32(&sh->sc_full[set][b]), lane);
        }
      }
      now = next, next = last;
      last.there = cur.next(a);
      if (last.there) {
        const Segment& s = cur.s;
        last.t = tile_load(a, s, cur.j, lane);
        if (cur.first() && s.tile0 == 0 && s.n < s.u.ntiles)
          info = make_int4(1 + cut.ranges(range + 1, uint32_t(s.u.ntiles - s.n)), s.row0, s.ntok, s.h);
      }
    }
    if (!ok) {
      sh->abort = 1;
      info.x = 0;
      if (lane == 0) note_timeout(a.status, a.diag, loads_v ? 5u : 1u, uint32_t(i));
    }
    if (lane == 0 && !loads_v) a.info[range] = info;
    n_put = max(i, 0);
  } else if (warp >= kMmaWarp && warp < kMmaWarp + kSets) {
    // ------------------------------------------------------------ the two products of each tile
    constexpr uint32_t idesc_s = tc::idesc_e4m3_f32(kTile, R);
    constexpr uint32_t idesc_o = tc::idesc_e4m3_f32(128, 2 * R) | tc::kIdescAMajorMN | tc::kIdescBMajorMN;
    const int set = warp - kMmaWarp;
    const ShortWaiter wait{&sh->abort, cycles_of(a.timeout_ns)};
    uint8_t* ring_mem = sRing + set * C::kSlots * C::kSlotBytes;
    const uint32_t t_s = tmem + set * 4 * R, t_o = t_s + 2 * R;
    const uint64_t dk = tc::sdesc_kmajor<D>(tc::smem_u32(ring_mem));
    const uint64_t dq = tc::sdesc_kmajor<D>(tc::smem_u32(sQ + set * kQBufs * C::kQBytes));
    // O^T has M = 128 also where D = 64: its lanes 64 .. 127 come from the tile behind, whatever it holds, and are not read
    const uint64_t dv = tc::sdesc_mnmajor<D>(tc::smem_u32(ring_mem), C::kSlotBytes);
    const uint64_t dp = tc::sdesc_mnmajor<C::kPPitch>(tc::smem_u32(sP + set * C::kPBytes), kTile * 128);
    Ring<C::kSlots> ring;
    int n_seg = 0, n_s = 0, t = 0, units = 0, j0 = 0, j1 = 0;
    Cursor kc(sh->start[set], a.tokens), vc(sh->start[set], a.tokens);
    auto s_product = [&]() {  // S^T of the tile at kc; the S before last has been read (its P is there)
      const int b = n_seg % kQBufs;
      if (kc.first() && !wait(&sh->q_ready[set][n_seg % kQRing], (n_seg / kQRing) & 1)) return false;
      if (!wait(&sh->full[set][ring.slot], ring.phase)) return false;
      tc::tc_fence_after();
      // shuffled, so that the compiler knows them to be the same for the warp
      const uint64_t dk_t = dk + uint32_t(__shfl_sync(~0u, ring.slot, 0) * (C::kSlotBytes >> 4));
      const uint64_t dq_t = dq + uint32_t(__shfl_sync(~0u, b, 0) * (C::kQBytes >> 4));
      const bool last = kc.last();
      if (tc::elect_one()) {
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            tc::mma_f8(t_s + (n_s & 1) * R, dk_t + ((i * 32) >> 4), dq_t + ((part * C::kQPart + i * 32) >> 4), idesc_s,
                       part != 0 || i != 0);
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
    bool ok = true, more = true;
    for (t = -2; ok; ++t) {  // O^T of tile t, then S^T of tile t + 2
      if (t >= 0) {
        if (!vc.next(a)) break;
        const bool first = vc.first(), last = vc.last();
        if (first) whole_tiles(a, vc.s, vc.s.u.p1, vc.s.u.p0, j0, j1);
        if (vc.j < j0 || vc.j >= j1) {  // while the softmax works on this tile
          ok = wait(&sh->full[set][ring.slot], ring.phase);
          if (!ok) break;
          clear_unseen_codes<D>(a, vc.s, vc.j, ring_mem + ring.slot * C::kSlotBytes, lane);
        }
        ok = wait.both(&sh->full[set][ring.slot], ring.phase, &sh->p_full[set], t & 1);
        if (ok && first) ok = wait(&sh->o_read[set], (units++ & 1) ^ 1);  // the unit before has been read
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t dv_t = dv + uint32_t(__shfl_sync(~0u, ring.slot, 0) * (C::kSlotBytes >> 4));
        if (tc::elect_one()) {
#pragma unroll
          for (int i = 0; i < kTile / 32; ++i)
            tc::mma_f8(t_o, dv_t + ((i * 32 * D) >> 4), dp + ((i * 32 * C::kPPitch) >> 4), idesc_o, !first || i != 0);
          tc::mma_commit(tc::smem_u32(&sh->p_empty[set]));
          tc::mma_commit(tc::smem_u32(&sh->empty[set][ring.slot]));
          if (last) tc::mma_commit(tc::smem_u32(&sh->o_full[set]));
        }
        __syncwarp();
        ring.step();
      }
      more = more && kc.next(a);
      if (more) ok = s_product();
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 2u, uint32_t(t));
    }
    if (lane == 0) sh->pending[set] = n_s > 0;
  } else if (warp >= kSplitWarp) {
    // ---------------------------------------------------------------- Q into two parts of e4m3
    const int set = (warp - kSplitWarp) / C::kSplitWarps, w = (warp - kSplitWarp) % C::kSplitWarps;
    const ShortWaiter wait{&sh->abort, cycles_of(a.timeout_ns)};
    constexpr int kLanes = D / 16, kPass = 32 / kLanes * C::kSplitWarps;  // threads to a row, rows at a time
    const int piece = lane % kLanes;
    int n_seg = 0;
    bool ok = true;
    Walk walk(sh->start[set], a.tokens);
    Segment s = {};
    for (; walk.next(a, s); ++n_seg) {
      const int b = n_seg % kQBufs;
      ok = wait(&sh->q_empty[set][b], ((n_seg / kQBufs) & 1) ^ 1);
      if (!ok) break;
      uint8_t* q_mem = sQ + (set * kQBufs + b) * C::kQBytes;
      // A thread's 16 lanes of a row are copied to where their two parts will lie, all rows at once, and then split in place.
      const __nv_bfloat16* src = args.q + int64_t(s.row0) * args.q_stride + int64_t(s.h) * a.g * D + piece * 16;
#pragma unroll 1
      for (int row = w * (32 / kLanes) + lane / kLanes; row < R; row += kPass) {
        const int tok = row / a.g, hh = row - tok * a.g;
        uint8_t* to = q_mem + tc::swizzled<D>(row, piece);
        if (tok < s.ntok) {
          const __nv_bfloat16* from = src + tok * args.q_stride + hh * D;
          tc::async_copy_16(tc::smem_u32(to), from);
          tc::async_copy_16(tc::smem_u32(to + C::kQPart), from + 8);
        } else {  // rows behind the unit's are 0
          *reinterpret_cast<uint4*>(to) = *reinterpret_cast<uint4*>(to + C::kQPart) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      tc::async_copies_wait();
#pragma unroll 1
      for (int row = w * (32 / kLanes) + lane / kLanes; row < R; row += kPass) {
        uint8_t* at = q_mem + tc::swizzled<D>(row, piece);
        uint32_t word[8];
        *reinterpret_cast<uint4*>(word) = *reinterpret_cast<const uint4*>(at);
        *reinterpret_cast<uint4*>(word + 4) = *reinterpret_cast<const uint4*>(at + C::kQPart);
        uint32_t top = 0;  // the row's largest magnitude, as bits of fp32
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, max(word[i] & 0x7FFF0000u, (word[i] << 16) & 0x7FFF0000u));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
        const uint32_t byte = kv8::exponent_byte(top);
        const float by = byte == kv8::kNan ? 0.f : kv8::power(127 - int(byte)) * (args.negate ? -1.f : 1.f);
        const unsigned long long by2 = pack_f32x2(by, by);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t h[2], l[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y0, y1;  // at most 448: exact in fp16, but for what lies 2^-25 below
            unpack_f32x2(mul_f32x2(pack_f32x2(bf16lo(word[2 * i + k]), bf16hi(word[2 * i + k])), by2), y0, y1);
            kv8::split2<false>(__floats2half2_rn(y0, y1), h[k], l[k]);
          }
          hi[i] = h[0] | h[1] << 16, lo[i] = l[0] | l[1] << 16;
        }
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + C::kQPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (piece == 0) sh->row_factor[set][n_seg % kQRing][row] = kv8::factor(byte) * a.c2;
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->q_ready[set][n_seg % kQRing]));
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 4u, uint32_t(n_seg));
    }
  } else if (warp < kKWarp) {
    // ------------------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const ShortWaiter wait{&sh->abort, cycles_of(a.timeout_ns)};
    const int grp = warp >> 2, w4 = warp & 3;
    const int kv = w4 * 32 + lane;  // this thread's slot of each tile = TMEM lane
    const int set = grp % kSets, row0 = grp / kSets * RW;  // and its rows
    const uint32_t t_s = tmem + (uint32_t(w4 * 32) << 16) + set * 4 * R + row0, t_o = t_s + 2 * R;
    float* neg_ref = sh->neg_ref[set] + row0;
    // a slot's row of P: its R first parts, then its second parts (R = 128: in a chunk of their own)
    uint8_t* p_mem = sP + set * C::kPBytes;
    // the rows that this lane holds after a fold, of 32 rows or all of them at a time (the lanes of a row hold the same)
    constexpr int kFolds = RW > 32 ? RW / 32 : 1, kFold = RW / kFolds;
    const int fold_row = lane / (32 / kFold);
    float* row_by = sh->row_by[set] + row0;
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
      const float* factor = sh->row_factor[set][units % kQRing] + row0;
      ok = wait(&sh->q_ready[set][units % kQRing], (units / kQRing) & 1);
      if (!ok) break;
      int f = 1, f_top = 1;  // the reference of V's powers of two, as an exponent byte, and the largest one so far
      float l[RW];  // this slot's share of the rows' sums
#pragma unroll
      for (int i = 0; i < RW; ++i) l[i] = 0.f;
      for (int j = 0; j < s.n; ++j, ++t) {
        const bool inside = j >= j_in0 && j < j_in1;
        int from = 0, to = RW;  // the rows of this thread's that see its slot
        if (!inside) {
          // the token at p0 + tok sees the slot from tok = pos - p0 on, for `window` tokens, a sink always.  Rows behind the
          // unit's see nothing here: a slot for them alone holds whatever was there, and may not set V's reference
          const int v = (s.tile0 + j) * per_tile + (kv >> a.block_shift);
          const int pos = block_pos(a, s.u, v) + (kv & ((1 << a.block_shift) - 1));
          const int d = pos - s.u.p0;
          from = d <= 0 ? 0 : min(d, a.tokens) * a.g;
          to = s.ntok * a.g;
          if (a.window && pos >= a.n_sink) to = min(max(d + a.window, 0), s.ntok) * a.g;
          from = max(from - row0, 0), to = min(to - row0, RW);
        }
        const bool seen = from < to;
        ok = wait.both(&sh->s_full[set][t & 1], (t >> 1) & 1, &sh->sc_full[set][t % Sh::kScales], (t / Sh::kScales) & 1);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t bytes = sh->scales[set][t % Sh::kScales][kv];
        // a V of NaN makes the rows that see it NaN by way of their scores: a weight of 0 would not do
        const bool v_nan = bytes >> 8 == kv8::kNan;
        const float kf = kv8::factor(v_nan ? kv8::kNan : bytes & 0xFFu);
        const unsigned long long kk = pack_f32x2(kf, kf);
        const int v_byte = seen && !v_nan ? max(1, int(bytes >> 8)) : 0;  // a slot that no row sees counts for nothing
        float y[RW];  // the only array beside l: what is needed once more is loaded once more (S is there until P is)
        // First by the references as they stand; where they are outgrown, and on a unit's first tile, once more without, and by
        // new ones.  (Rounds of one loop: a tile's code has to stay in the instruction cache.)
        for (bool fresh = j == 0;; fresh = true) {
          const float* minus = fresh ? sh->zeros : neg_ref;
          tc::tmem_ld<RW>(t_s + (t & 1) * R, y);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < RW; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(minus + i), c = *reinterpret_cast<const float4*>(factor + i);
            unpack_f32x2(fma_f32x2(mul_f32x2(pack_f32x2(y[i], y[i + 1]), kk), pack_f32x2(c.x, c.y), pack_f32x2(m.x, m.y)), y[i], y[i + 1]);
            unpack_f32x2(fma_f32x2(mul_f32x2(pack_f32x2(y[i + 2], y[i + 3]), kk), pack_f32x2(c.z, c.w), pack_f32x2(m.z, m.w)), y[i + 2], y[i + 3]);
          }
          if (__builtin_expect(!inside, 0)) {
#pragma unroll
            for (int k = 0; k < RW; k += 32) {
              const uint32_t see = bits32(from - k, to - k);
#pragma unroll
              for (int i = k; i < k + 32 && i < RW; ++i)
                if (!(see >> (i - k) & 1u)) y[i] = -INFINITY;
            }
          }
          if (__builtin_expect(fresh, 0)) {
            // each row's maximum over the tile's 128 slots, by warp then over the group's warps; lane i has row i, and 32 + i
#pragma unroll
            for (int k = 0; k < kFolds; ++k) {
              float mine = -INFINITY;
#pragma unroll
              for (int i = 0; i < kFold; ++i) {
                const float top = warp_max_f32(y[k * 32 + i]);
                if (lane == i) mine = top;
              }
              if (lane < kFold) sh->warp_max[grp][w4][k * 32 + lane] = mine;
            }
            float old[kFolds];  // before any warp writes the new ones
#pragma unroll
            for (int k = 0; k < kFolds; ++k) old[k] = j == 0 || lane >= kFold ? kUnset : -neg_ref[k * 32 + lane];
            const int my_byte = __reduce_max_sync(~0u, v_byte);
            if (lane == 0) sh->warp_byte[grp][w4] = my_byte;
            ok = meet();
            if (!ok) break;
            const float (*part)[RW] = sh->warp_max[grp];
            const int* byte = sh->warp_byte[grp];
            const int f_old = f;
            // f may fall, too, so that this tile's weights keep their place in e4m3, but not so far that O^T leaves fp32: its terms
            // are below 2^18 2^70
            f = max(max(max(byte[0], byte[1]), max(byte[2], byte[3])), max(f_top - 70, 1));
            f_top = max(f_top, f);
#pragma unroll
            for (int k = 0; k < kFolds; ++k) {
              const int row = k * 32 + lane;
              if (lane >= kFold) break;
              const float m = fmaxf(old[k], fmaxf(fmaxf(part[0][row], part[1][row]), fmaxf(part[2][row], part[3][row])) - kTop);
              row_by[row] = tc::ex2_approx(old[k] - m);  // the four warps write the same values
              neg_ref[row] = row0 + row < s.ntok * a.g ? -m : -INFINITY;  // rows behind the unit's weigh nothing
            }
            __syncwarp();
            ok = wait(&sh->p_empty[set], (t & 1) ^ 1);  // the last product is over
            if (!ok) break;
            if (j > 0) {  // the sums so far and this thread's lane of O^T
              tc::tc_fence_after();
              const float fewer = tc::ex2_approx(float(f_old - f));
#pragma unroll
              for (int i = 0; i < RW; i += 4) {
                const float4 by = *reinterpret_cast<const float4*>(row_by + i);
                l[i] *= by.x, l[i + 1] *= by.y, l[i + 2] *= by.z, l[i + 3] *= by.w;
              }
#pragma unroll 1
              for (int i = 0; i < 2 * RW; i += 8) {
                const int col = i < RW ? i : R + i - RW;
                const float* by = row_by + (i < RW ? i : i - RW);
                float o[8];
                tc::tmem_ld<8>(t_o + col, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= by[k] * fewer;
                tc::tmem_st<8>(t_o + col, o);
              }
              tc::tmem_st_wait();
            }
#pragma unroll
            for (int i = 0; i < RW; i += 4) {
              const float4 m = *reinterpret_cast<const float4*>(neg_ref + i);
              y[i] += m.x, y[i + 1] += m.y, y[i + 2] += m.z, y[i + 3] += m.w;
            }
          }
          const int at = sync & 1;
          if (!fresh) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < RW; i += 4) top = fmaxf(fmaxf(top, fmaxf(y[i], y[i + 1])), fmaxf(y[i + 2], y[i + 3]));
            // (a V far beyond f is looked at however little it weighs: its weight would leave fp32)
            if (__any_sync(~0u, top + float(max(0, v_byte - f)) > kMost || v_byte - f > 60) && lane == 0) sh->need[grp][at] = t + 1;
            // V's powers far below f: this warp's slots; the tile's where the others say so too
            if (!__any_sync(~0u, v_byte >= f - kFall)) {
              const int seen_by = __any_sync(~0u, v_byte > 0);
              if (lane == 0) sh->low[grp][at][w4] = 2 * (t + 1) + seen_by;
            }
            arrive();
          }
#pragma unroll
          for (int i = 0; i < RW; ++i) y[i] = tc::ex2_approx(y[i]);  // while the others arrive; done again where a reference moves
          if (fresh) break;
          // and the last product, which reads P, is over
          ok = wait.both(&sh->group[grp], sync++ & 1, &sh->p_empty[set], (t & 1) ^ 1);
          if (!ok) break;
          bool again = sh->need[grp][at] == t + 1;
          if (__builtin_expect(!__any_sync(~0u, v_byte >= f - kFall), 0)) {
            const int4 low = *reinterpret_cast<const int4*>(sh->low[grp][at]);
            again |= low.x / 2 == t + 1 && low.y / 2 == t + 1 && low.z / 2 == t + 1 && low.w / 2 == t + 1 &&
                     ((low.x | low.y | low.z | low.w) & 1) && f > f_top - 70;
          }
          if (!again) break;
        }
        if (!ok) break;
        const float vf = kv8::power(max(v_byte - f, -126));  // 2^(ev - f)
        const unsigned long long vv = pack_f32x2(vf, vf);
        uint32_t hi[RW / 4], lo[RW / 4];
#pragma unroll
        for (int i = 0; i < RW; i += 2) {
          const unsigned long long p2 = pack_f32x2(y[i], y[i + 1]);
          unpack_f32x2(add_f32x2(pack_f32x2(l[i], l[i + 1]), p2), l[i], l[i + 1]);
          unpack_f32x2(mul_f32x2(p2, vv), y[i], y[i + 1]);
        }
#pragma unroll
        for (int i = 0; i < RW / 4; ++i) {
          uint32_t h[2], r[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) kv8::split2<true>(__floats2half2_rn(y[4 * i + 2 * k], y[4 * i + 2 * k + 1]), h[k], r[k]);
          hi[i] = h[0] | h[1] << 16, lo[i] = r[0] | r[1] << 16;
        }
        auto put_p = [&](const uint32_t* w, int at) {  // at byte `at` of the slot's row
          uint8_t* dst = p_mem + (at / C::kPPitch) * (kTile * C::kPPitch);
          const int in = at % C::kPPitch;
          if constexpr (RW == 8) {
            *reinterpret_cast<uint2*>(dst + tc::swizzled<C::kPPitch>(kv, in / 16) + in % 16) = make_uint2(w[0], w[1]);
          } else {
#pragma unroll
            for (int i = 0; i < RW / 16; ++i)
              *reinterpret_cast<uint4*>(dst + tc::swizzled<C::kPPitch>(kv, in / 16 + i)) =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        };
        put_p(hi, row0);
        put_p(lo, R + row0);
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->p_full[set]));
      }
      if (!ok) break;
      // ---------------------------------------------------------------- the unit's rows
      // rows' sums over the 128 slots: lanes, then the group's warps in order
#pragma unroll
      for (int k = 0; k < kFolds; ++k) sh->warp_sum[grp][w4][k * 32 + fold_row] = fold_lanes<kFold, false>(l + k * 32, lane);
      ok = meet();
      if (!ok) break;
      const float (*part)[RW] = sh->warp_sum[grp];
      const float of = kv8::power(f - 127);
      const bool partial = s.n < s.u.ntiles;
      const int64_t pbase = (int64_t(2) * (blockIdx.x + set * gridDim.x) + (s.tile0 > 0 ? 0 : 1)) * R + row0;
      const int n_rows = s.ntok * a.g - row0;  // of this group's
      int* row_at = sh->row_at[set] + row0;
      for (int mine = lane; mine < RW; mine += 32) {  // the four warps write the same values
        const int tok = (row0 + mine) / a.g, at = tok * (a.Hq - a.g) + row0 + mine;  // heads from the unit's first
        const float sum = (part[0][mine] + part[1][mine]) + (part[2][mine] + part[3][mine]);
        row_by[mine] = (sum == 0.f ? 0.f : 1.f / sum) * of;  // NaN stays NaN, in the log-sum-exp too
        row_at[mine] = mine < n_rows ? at * D : -1;
        if (w4 == 0 && mine < n_rows) {
          const float lse2 = sum == 0.f ? -INFINITY : log2f(sum) - neg_ref[mine];
          if (partial)
            a.plse[pbase + mine] = lse2;
          else if (a.lse)
            a.lse[int64_t(s.row0) * a.Hq + s.h * a.g + at] = lse2 * kLn2;
        }
      }
      __syncwarp();
      ok = wait(&sh->o_full[set], units++ & 1);
      if (!ok) break;
      tc::tc_fence_after();
      if (w4 * 32 < D) {  // TMEM lane = lane of the head; lanes from D on hold nothing
        __nv_bfloat16* dst = a.out + (int64_t(s.row0) * a.Hq + s.h * a.g) * D + kv;
        float* pdst = a.partial + pbase * D + kv;
#pragma unroll 1
        for (int i = 0; i < RW; i += 8) {
          float o[8], o2[8], by[8];
          int to[8];
          tc::tmem_ld<8>(t_o + i, o);
          tc::tmem_ld<8>(t_o + R + i, o2);
          *reinterpret_cast<float4*>(by) = *reinterpret_cast<const float4*>(row_by + i);
          *reinterpret_cast<float4*>(by + 4) = *reinterpret_cast<const float4*>(row_by + i + 4);
          *reinterpret_cast<int4*>(to) = *reinterpret_cast<const int4*>(row_at + i);
          *reinterpret_cast<int4*>(to + 4) = *reinterpret_cast<const int4*>(row_at + i + 4);
          tc::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = fmaf(o2[k], 1.f / 16, o[k]) * by[k];
          if (partial) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (to[k] >= 0) pdst[(i + k) * D] = o[k];
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (to[k] >= 0) dst[to[k]] = __float2bfloat16(o[k]);
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->o_read[set]));  // the next unit may overwrite it
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 3u, uint32_t(t) | uint32_t(warp) << 24);
    }
  }

  __syncthreads();
  if (sh->abort) {  // MMAs and copies may be in flight: wait (bounded) before TMEM is freed and the block ends
    const long long deadline = tc::deadline_after_ns(kDrainNs);
    const int set = warp - kMmaWarp;
    if (set >= 0 && set < kSets && sh->pending[set]) {
      if (tc::elect_one()) tc::mma_commit(tc::smem_u32(&sh->drain[set]));
      __syncwarp();
      const volatile int never = 0;
      tc::mbar_wait_bounded(tc::smem_u32(&sh->drain[set]), 0, deadline, &never);
    }
    // a loading warp's last copies, the newest first; of one whose slot has been filled anew since the barrier may tell or not
    const bool loads_v = warp >= kVWarp;
    const int from = loads_v ? kVWarp : kKWarp;
    if (n_put > 0) {
      const volatile int never = 0;
      for (int i = n_put - 1; i >= 0 && i >= n_put - C::kSlots; --i) {
        const uint32_t at = ring_place(loads_v, uint32_t(i), sh->start[warp - from].count);
        tc::mbar_wait_bounded(tc::smem_u32(&sh->full[warp - from][at % C::kSlots]), at / C::kSlots & 1, deadline, &never);
      }
    }
    tc::async_copies_wait();
    __syncthreads();
  }
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, C::kTmemCols);
}

template <int D, int R>
cudaError_t launch(const CUtensorMap& k, const CUtensorMap& v, const Attn8Args& a, int n_cta, cudaStream_t s) {
  static bool done[tch::kMaxDevices] = {};
  static std::mutex mu;
  constexpr int kSmem = Cfg<D, R>::kSmem;
  const cudaError_t e = tch::set_smem_once(window8_kernel<D, R>, kSmem, done, &mu);
  return e != cudaSuccess ? e : launch_pdl(window8_kernel<D, R>, dim3(n_cta), dim3(kThreads), kSmem, s, k, v, a);
}

}  // namespace

int attention_window8_sets(int D, int unit_rows) { return sets_of(D, unit_rows); }

cudaError_t launch_attention_windows8(int D, int unit_rows, const CUtensorMap& k, const CUtensorMap& v,
                                      const attn::Attn8Args& a, int n_cta, cudaStream_t s) {
  if (D == 64) switch (unit_rows) {
      case 16: return launch<64, 16>(k, v, a, n_cta, s);
      case 32: return launch<64, 32>(k, v, a, n_cta, s);
      case 64: return launch<64, 64>(k, v, a, n_cta, s);
      default: return launch<64, 128>(k, v, a, n_cta, s);
    }
  switch (unit_rows) {
    case 16: return launch<128, 16>(k, v, a, n_cta, s);
    case 32: return launch<128, 32>(k, v, a, n_cta, s);
    case 64: return launch<128, 64>(k, v, a, n_cta, s);
    default: return launch<128, 128>(k, v, a, n_cta, s);
  }
}

}  // namespace dspark
