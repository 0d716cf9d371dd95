// The attention of prompts: windows of more (token, head) rows than one tile of 128 holds.
//
// Bound by the two products and the exponentials.  A unit is two Q tiles of 128 rows that read the same KV tiles:
//     S = Q K^T  (tcgen05, fp32 in TMEM)  ->  P = 2^(c S - m), l += sum P  (registers, one thread per row)
//     O += P V   (tcgen05; P in bf16 in TMEM over S, O in fp32 in TMEM)
// While one tile's softmax runs, the tensor cores work for the other.  The softmax of a tile has to be done within
// the other tile's two products, so its first half is handed on as soon as it is there, computed by the
// reference m as it stands while the row's maximum is found: m only keeps the exponentials in range, and
// weights of up to 2^16 give the same result, since the sum is divided out and neither fp32 nor bf16 loses bits
// there.  It moves, and O and l are rescaled, when a maximum has outgrown it by more (kRescaleAt).  P is rounded to
// bf16 for the second product, its sum is taken before that, in fp32.
//
// GB300, 2 prompts of about 4000 rows over 1000 .. 5000 cached positions, window 4096, Hq 32, Hkv 8: D 128 304 us of 238 at the
// measured matrix rate (78%), 19 us of it the join and its launch; D 64 296 us (132 by its products, 206 by its exponentials at
// 16 a cycle and SM).  What holds it is the chain of one tile, S into registers, maximum, exponentials, P, product,
// next S, which two tiles in turn do not quite hide (tensor pipes 62% busy, 4.4 instructions an exponential).  Slower or the
// same, each measured on D 128: P handed on in 4 or 8 parts (338, 389 us); all eight warps on each tile together
// (356); a polynomial for an eighth to a half of the exponentials (319 .. 365; D 64, then 292 us, 280 with an eighth and 279
// with a quarter); the first half's store waited for later, and the MMA loop in one thread (no change).
#include <type_traits>

#include "attention_common.cuh"

namespace dspark {
namespace {

using namespace attn;

constexpr int kThreads = 384;  // warps 0-3: softmax of the first tile, 4-7: of the second, 8: TMA, 9: MMA,
                               // 10: clears what must not be seen of V
// Registers: launched with 384 x 168; the softmax warps hold a whole row of S and take what the others
// give back (256 x 208 + 128 x 80 <= 384 x 168).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;            // 128-byte swizzled column blocks of a tile
  static constexpr int kHalfBytes = kTile * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kKSlots = D == 128 ? 2 : 5, kVSlots = D == 128 ? 3 : 5;  // rings: 160 KB either way
};

// The clearing warp and the MMA warp agree on the tiles that need clearing; their barriers are counted over those
// tiles alone (more barriers than V slots, so that neither can lap the other).
constexpr int kReady = 8;

struct Shared {
  uint64_t q_full[2], q_empty[2], k_full[5], k_empty[5], v_full[5], v_empty[5], v_ready[kReady], s_full[2], p_full[2][2], o_full[2], drain;
  uint32_t tmem_base;
  volatile int abort;
  int mma_pending;
  int n_k, n_v, n_q[2];  // copies issued
  Start start;
};

// Bits k = 0 .. 7 with lo <= k <= hi.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  const uint32_t below = hi >= 7 ? 0xFFu : hi < 0 ? 0u : (2u << hi) - 1u;
  const uint32_t from = lo <= 0 ? 0xFFu : lo > 7 ? 0u : 0xFFu << lo;
  return below & from;
}

__device__ __forceinline__ void store_32b(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void store_2x16b(void* p, const uint32_t* v) {
  uint4* to = static_cast<uint4*>(p);
  to[0] = make_uint4(v[0], v[1], v[2], v[3]), to[1] = make_uint4(v[4], v[5], v[6], v[7]);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                       // two Q tiles
  uint8_t* sK = smem + 2 * C::kTileBytes;
  uint8_t* sV = sK + C::kKSlots * C::kTileBytes;
  Shared* sh = reinterpret_cast<Shared*>(sV + C::kVSlots * C::kTileBytes);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // the same for the warp, and known to be
  const int unit_tokens = 2 * a.tokens, tile_rows = a.tokens * a.g;
  const int active = (tile_rows + 31) / 32;  // softmax warps of a tile that hold rows
  PlanScratch& plan = *reinterpret_cast<PlanScratch*>(sK);  // before the first load

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->q_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->q_empty[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->s_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->p_full[i][0]), active);
      tc::mbar_init(tc::smem_u32(&sh->p_full[i][1]), active);
      tc::mbar_init(tc::smem_u32(&sh->o_full[i]), 1);
    }
    for (int i = 0; i < 5; ++i) {
      tc::mbar_init(tc::smem_u32(&sh->k_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->k_empty[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->v_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh->v_empty[i]), 2);  // the product, and the clearing warp
    }
    for (int i = 0; i < kReady; ++i) tc::mbar_init(tc::smem_u32(&sh->v_ready[i]), 1);
    tc::mbar_init(tc::smem_u32(&sh->drain), 1);
    tc::fence_mbar_init();
    sh->abort = 0, sh->mma_pending = 0, sh->start.count = 0, plan.bad = 0, plan.n_long = 0;
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
  const Cut cut = plan_ranges<1>(a, &sh->start, plan, unit_tokens);
  tc::fence_proxy_async_smem();  // the plan's scratch lies where TMA writes
  __syncthreads();
  const uint32_t tmem = sh->tmem_base;

  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 8) {
    // --------------------------------------------------------------------- TMA producer
    // In order: a unit's K 0 and Q, then V j, K j + 1.  K and V are read by every unit of the head: kept in L2.
    const TmaWaiter wait{{&sh->abort, a.timeout_ns}};
    const uint64_t keep = tc::policy_evict_last();
    Ring<C::kKSlots> kr;
    Ring<C::kVSlots> vr;
    int seg_i = 0, n_k = 0, n_v = 0, q_use0 = 0, q_use1 = 0;
    int4 info = make_int4(0, 0, 0, 0);
    bool ok = true;
    Walk walk(sh->start, unit_tokens);
    Segment s = {};
    auto put_k = [&](const TileLoad& t) {
      if (!wait(&sh->k_empty[kr.slot], kr.phase ^ 1)) return false;
      issue_tile<C::kHalves>(a, &map_k, t, tc::smem_u32(sK + kr.slot * C::kTileBytes), tc::smem_u32(&sh->k_full[kr.slot]), keep,
                             lane);
      ++n_k;
      kr.step();
      return true;
    };
    auto put_v = [&](const TileLoad& t) {
      if (!wait(&sh->v_empty[vr.slot], vr.phase ^ 1)) return false;
      issue_tile<C::kHalves>(a, &map_v, t, tc::smem_u32(sV + vr.slot * C::kTileBytes), tc::smem_u32(&sh->v_full[vr.slot]), keep,
                             lane);
      ++n_v;
      vr.step();
      return true;
    };
    auto put_q = [&](int b, int& use, int row) {
      if (!wait(&sh->q_empty[b], (use & 1) ^ 1)) return false;
      if (lane == 0) {
        const uint32_t bar = tc::smem_u32(&sh->q_full[b]);
        tc::mbar_arrive_expect_tx(bar, uint32_t(tile_rows * 128 * C::kHalves));
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tc::tma_load_3d(tc::smem_u32(sQ + b * C::kTileBytes + hf * C::kHalfBytes), &map_q, bar, hf * 64, s.h * a.g, row, keep);
      }
      ++use;
      return true;
    };
    while (ok && walk.next(a, s)) {
      if (s.tile0 == 0 && s.n < s.u.ntiles)
        info = make_int4(1 + cut.ranges(blockIdx.x + 1, uint32_t(s.u.ntiles - s.n)), s.row0, s.ntok, s.h);
      TileLoad t0 = tile_load(a, s, 0, lane), t1 = t0;
      if (s.n > 1) t1 = tile_load(a, s, 1, lane);
      ok = put_k(t0) && put_q(0, q_use0, s.row0) && (s.ntok <= a.tokens || put_q(1, q_use1, s.row0 + a.tokens));
      for (int j = 0; ok && j < s.n; ++j) {
        TileLoad t2 = t1;
        if (j + 2 < s.n) t2 = tile_load(a, s, j + 2, lane);
        ok = put_v(t0) && (j + 1 >= s.n || put_k(t1));
        t0 = t1, t1 = t2;
      }
      ++seg_i;
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 1u, uint32_t(seg_i));
    }
    if (lane == 0) {
      if (!ok) info.x = 0;
      a.info[blockIdx.x] = info;
      sh->n_k = n_k, sh->n_v = n_v, sh->n_q[0] = q_use0, sh->n_q[1] = q_use1;
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------------- MMA issuer
    const Waiter wait{&sh->abort, a.timeout_ns};
    const uint32_t idesc_qk = tc::idesc_bf16_f32(kTile, kTile) | a.negate_q;
    constexpr uint32_t idesc_pv = tc::idesc_bf16_f32(kTile, D) | tc::kIdescBMajorMN;
    Ring<C::kKSlots> kr;
    Ring<C::kVSlots> vr;
    Ring<kReady> ready;
    int seg_i = 0;
    uint32_t use0 = 0, use1 = 0, p0 = 0, p1 = 0;  // parities: the tiles' Q, their P
    bool ok = true, any = false;
    Walk walk(sh->start, unit_tokens);
    Segment s = {};
    const uint64_t dq = tc::sdesc_kmajor_sw128(tc::smem_u32(sQ)), dk = tc::sdesc_kmajor_sw128(tc::smem_u32(sK));
    const uint64_t dv = tc::sdesc_mnmajor(tc::smem_u32(sV), C::kHalfBytes);
    // S_st = Q_st K^T for the tile in ring slot `ks`
    auto issue_qk = [&](int st, int ks) {
      const uint64_t q = dq + uint32_t(st * (C::kTileBytes >> 4)), k = dk + uint32_t(ks * (C::kTileBytes >> 4));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        constexpr int kHalf = C::kHalfBytes;
        tc::mma_bf16(tmem + st * kTile, q + (((i / 4) * kHalf + (i % 4) * 32) >> 4),
                     k + (((i / 4) * kHalf + (i % 4) * 32) >> 4), idesc_qk, i != 0);
      }
      tc::mma_commit(tc::smem_u32(&sh->s_full[st]));
    };
    // O_st (+)= P_st V; P_st lies over the first 64 columns of S_st
    auto issue_pv = [&](int st, int vs, int hf, bool add) {  // of half of the tile's slots
      const uint64_t v = dv + uint32_t(vs * (C::kTileBytes >> 4));
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i)
        tc::mma_bf16_ts(tmem + 2 * kTile + st * D, tmem + st * kTile + 32 * hf + 8 * i,
                        v + uint32_t(hf * (kTile / 2 * 128 >> 4)) + ((i * 2048) >> 4), idesc_pv, add || i != 0);
    };
    while (ok && walk.next(a, s)) {
      const int n_st = s.ntok > a.tokens ? 2 : 1;
      const bool two = n_st == 2;
      ok = wait(&sh->k_full[kr.slot], kr.phase) && wait(&sh->q_full[0], use0) && (!two || wait(&sh->q_full[1], use1));
      if (!ok) break;
      use0 ^= 1, use1 ^= two;
      tc::tc_fence_after();
      if (tc::elect_one()) {
        issue_qk(0, kr.slot);
        if (s.n == 1) tc::mma_commit(tc::smem_u32(&sh->q_empty[0]));
        if (two) {
          issue_qk(1, kr.slot);
          if (s.n == 1) tc::mma_commit(tc::smem_u32(&sh->q_empty[1]));
        }
        tc::mma_commit(tc::smem_u32(&sh->k_empty[kr.slot]));
      }
      __syncwarp();
      kr.step();
      any = true;
      int j0, j1;  // the tiles that need no clearing
      whole_tiles(a, s, s.u.p1, s.u.p0, j0, j1);
      // P_st V of this tile, then S_st of the next; `last` of the unit's Q tiles frees V and K
      auto step = [&](auto st_of, uint32_t parity, int j, bool more, bool last) {
        constexpr int st = decltype(st_of)::value;
        if (!wait(&sh->p_full[st][0], parity)) return false;
        tc::tc_fence_after();
        if (tc::elect_one()) issue_pv(st, vr.slot, 0, j > 0);
        __syncwarp();
        if (!wait(&sh->p_full[st][1], parity)) return false;
        tc::tc_fence_after();
        if (tc::elect_one()) {
          issue_pv(st, vr.slot, 1, true);
          if (more) issue_qk(st, kr.slot);
          if (!more) tc::mma_commit(tc::smem_u32(&sh->o_full[st]));
          if (last) {
            tc::mma_commit(tc::smem_u32(&sh->v_empty[vr.slot]));
            if (more) tc::mma_commit(tc::smem_u32(&sh->k_empty[kr.slot]));
          }
          if (j + 2 == s.n) tc::mma_commit(tc::smem_u32(&sh->q_empty[st]));
        }
        __syncwarp();
        return true;
      };
      for (int j = 0; ok && j < s.n; ++j) {
        const bool more = j + 1 < s.n;
        ok = wait(&sh->v_full[vr.slot], vr.phase) && (!more || wait(&sh->k_full[kr.slot], kr.phase));
        if (ok && (j < j0 || j >= j1)) {
          ok = wait(&sh->v_ready[ready.slot], ready.phase);
          ready.step();
        }
        ok = ok && step(std::integral_constant<int, 0>(), p0, j, more, !two);
        p0 ^= 1;
        if (two) {
          ok = ok && step(std::integral_constant<int, 1>(), p1, j, more, true);
          p1 ^= 1;
        }
        vr.step();
        if (more) kr.step();
      }
      ++seg_i;
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 2u, uint32_t(seg_i));
    }
    if (lane == 0) sh->mma_pending = any;
  } else if (warp == 10) {
    // ------------------------------------------- V tiles: unseen slots cleared, then ready for the MMA
    const Waiter wait{&sh->abort, a.timeout_ns};
    Ring<C::kVSlots> ring;
    Ring<kReady> ready;
    int seg_i = 0;
    bool ok = true;
    Walk walk(sh->start, unit_tokens);
    Segment s = {};
    while (ok && walk.next(a, s)) {
      int j0, j1;
      whole_tiles(a, s, s.u.p1, s.u.p0, j0, j1);
      for (int j = 0; j < s.n; ++j, ring.step()) {
        ok = wait(&sh->v_full[ring.slot], ring.phase);
        if (!ok) break;
        if (j < j0 || j >= j1) {
          clear_unseen<C::kHalves>(a, s, j, sV + ring.slot * C::kTileBytes, lane);
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->v_ready[ready.slot]));
          ready.step();
        }
        // every tile, so that the ring never turns more than once past this warp (a parity tells no more)
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->v_empty[ring.slot]));
      }
      ++seg_i;
    }
    if (!ok) {
      sh->abort = 1;
      if (lane == 0) note_timeout(a.status, a.diag, 4u, uint32_t(seg_i));
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    if ((warp & 3) < active) {
      const Waiter wait{&sh->abort, a.timeout_ns};
      const int st = warp >> 2, row = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
      const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16);
      const uint32_t t_s = lane_base + st * kTile, t_o = lane_base + 2 * kTile + st * D;
      const int tok = row / a.g, hh = row - tok * a.g, tok0 = st * a.tokens;
      const float c2 = a.c2;
      int seg_i = 0, s_use = 0, o_use = 0;
      bool ok = true;
      Walk walk(sh->start, unit_tokens);
      Segment s = {};
      while (ok && walk.next(a, s)) {
        ++seg_i;
        if (tok0 >= s.ntok) continue;  // the unit has no second tile
        const int p = s.u.p0 + tok0 + tok;  // this row's position; the tile's: q0 .. q1
        const int q0 = s.u.p0 + tok0, q1 = min(q0 + a.tokens - 1, s.u.p1);
        const bool valid = row < tile_rows && tok0 + tok < s.ntok;
        const int per_tile = kTile >> a.block_shift;
        int j_in0, j_in1;  // the KV tiles that every row of this Q tile sees whole
        whole_tiles(a, s, q0, q1, j_in0, j_in1);
        float m = kUnset, l = 0.f;  // the reference (log2 units) and the sum
        for (int j = 0; j < s.n; ++j) {
          ok = wait(&sh->s_full[st], s_use++ & 1);
          if (!ok) break;
          tc::tc_fence_after();
          float x[kTile];
          tc::tmem_ld<kTile>(t_s, x);
          tc::tmem_ld_wait();
          if (j < j_in0 || j >= j_in1) {
            const int first = (s.tile0 + j) * per_tile;
            constexpr float hidden = -INFINITY;
            if (first >= s.u.sb) {  // one run of positions: slots from .. to are seen
              const int begin = block_pos(a, s.u, first);
              const int to = p - begin, from = a.window ? p - a.window + 1 - begin : 0;
              if (__any_sync(~0u, to < kTile - 1)) {
#pragma unroll
                for (int i = 0; i < kTile; ++i)
                  if (i > to) x[i] = hidden;
              }
              if (__any_sync(~0u, from > 0)) {  // a slot below n_sink stays: none here, unless sinks meet the window
                const int keep = a.n_sink - begin;
#pragma unroll
                for (int i = 0; i < kTile; ++i)
                  if (i < from && i >= keep) x[i] = hidden;
              }
            } else {
#pragma unroll
              for (int gr = 0; gr < kTile / 8; ++gr) {  // 8 slots of one block
                const int pos = block_pos(a, s.u, first + ((8 * gr) >> a.block_shift)) + ((8 * gr) & ((1 << a.block_shift) - 1));
                const uint32_t see = bits_between(p - a.window + 1 - pos, p - pos) | bits_between(0, min(p, a.n_sink - 1) - pos);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (!(see >> k & 1u)) x[8 * gr + k] = hidden;
              }
            }
          }
          // The first half's weights by the reference as it stands, and the row's maximum beside them; a new
          // reference only where that has been outgrown (and at a unit's first tile)
          const unsigned long long cc = pack_f32x2(c2, c2);
          unsigned long long l2[2] = {0ull, 0ull};
          uint32_t pk[32];
          auto weigh = [&](int hf) {
            const unsigned long long mm = pack_f32x2(-m, -m);
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
          };
          auto give = [&](int hf) {  // the product with V may begin
            tc::tmem_st32(t_s + 32 * hf, pk);
            tc::tmem_st_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh->p_full[st][hf]));
          };
          float t4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t4[i] = x[i];
#pragma unroll
          for (int i = 4; i < kTile; ++i) t4[i & 3] = fmaxf(t4[i & 3], x[i]);
          t4[0] = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          const float top = t4[0] * c2;
          weigh(0);
          if (__any_sync(~0u, top > m + kRescaleAt)) {
            const float old = m;
            if (top > m) m = top;
            const float alpha = tc::ex2_approx(old - m);
            l *= alpha;
            if (j > 0) {  // the product with the last tile was issued before this tile's S: it is complete
#pragma unroll
              for (int i = 0; i < D; i += 32) {
                float o[32];
                tc::tmem_ld<32>(t_o + i, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= alpha;
                tc::tmem_st<32>(t_o + i, o);
              }
            }
            l2[0] = l2[1] = 0ull;
            weigh(0);
          }
          give(0);
          weigh(1);
          give(1);
          float u0, u1;
          unpack_f32x2(add_f32x2(l2[0], l2[1]), u0, u1);
          l += u0 + u1;
        }
        if (!ok) break;
        ok = wait(&sh->o_full[st], o_use++ & 1);
        if (!ok) break;
        tc::tc_fence_after();
        // -------------------------------------------------------------- the tile's rows
        const int64_t oat = int64_t(s.row0 + tok0 + tok) * a.Hq + s.h * a.g + hh;
        const int64_t prow = (int64_t(2) * blockIdx.x + (s.tile0 > 0 ? 0 : 1)) * (2 * kTile) + st * kTile + row;
        const bool partial = s.n < s.u.ntiles;
        const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN, in the log-sum-exp too
        float o[D];
        tc::tmem_ld<D>(t_o, o);
        tc::tmem_ld_wait();
        tc::tc_fence_before();  // O has been read: the next unit's first product may follow its first P
        // 32-byte stores: a thread's row is D lanes in a row, other lanes' rows lie elsewhere.  The caller's tensor may
        // begin at any multiple of 16 bytes, and then takes two stores (the branch: 2 us of 296 with D 64, none with D 128; each kind in a loop of its own 315 and 313).
        const bool out_32b = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
        if (valid && partial) {
#pragma unroll
          for (int i = 0; i < D; i += 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = o[i + k] * inv;
            store_32b(a.partial + prow * D + i, reinterpret_cast<const uint32_t*>(v));
          }
        } else if (valid) {
#pragma unroll
          for (int i = 0; i < D; i += 16) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(o[i + 2 * k] * inv, o[i + 2 * k + 1] * inv);
              w[k] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            if (out_32b)
              store_32b(a.out + oat * D + i, w);
            else
              store_2x16b(a.out + oat * D + i, w);
          }
        }
        if (valid) {
          const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
          if (partial)
            a.plse[prow] = lse2;
          else if (a.lse)
            a.lse[oat] = lse2 * kLn2;
        }
      }
      if (!ok) {
        sh->abort = 1;
        if (lane == 0) note_timeout(a.status, a.diag, 3u, uint32_t(seg_i) | uint32_t(warp) << 24);
      }
    }
  }

  __syncthreads();
  if (sh->abort) {  // MMAs and copies may be in flight: wait (bounded) before TMEM is freed and the block ends
    const long long deadline = tc::deadline_after_ns(kDrainNs);
    if (warp == 9 && sh->mma_pending) {
      if (tc::elect_one()) tc::mma_commit(tc::smem_u32(&sh->drain));  // by the thread that issued them
      __syncwarp();
      const volatile int never = 0;
      tc::mbar_wait_bounded(tc::smem_u32(&sh->drain), 0, deadline, &never);
    } else if (warp == 8) {
      drain_copies(sh->k_full, C::kKSlots, sh->n_k, deadline);
      drain_copies(sh->v_full, C::kVSlots, sh->n_v, deadline);
      drain_copies(&sh->q_full[0], 1, sh->n_q[0], deadline);
      drain_copies(&sh->q_full[1], 1, sh->n_q[1], deadline);
    }
    __syncthreads();
  }
  if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int n_cta,
                   cudaStream_t s) {
  using C = Cfg<D>;
  constexpr int kSmem = (2 + C::kKSlots + C::kVSlots) * C::kTileBytes + int(sizeof(Shared));
  static_assert(kSmem <= 232448, "dynamic shared memory beyond the 227 KB per-block limit");
  static bool done[tch::kMaxDevices] = {};
  static std::mutex mu;
  const cudaError_t e = tch::set_smem_once(prompt_kernel<D>, kSmem, done, &mu);
  return e != cudaSuccess ? e : launch_pdl(prompt_kernel<D>, dim3(n_cta), dim3(kThreads), kSmem, s, q, k, v, a);
}

}  // namespace

cudaError_t launch_attention_prompts(int D, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                     const attn::AttnArgs& a, int n_cta, cudaStream_t s) {
  return D == 64 ? launch<64>(q, k, v, a, n_cta, s) : launch<128>(q, k, v, a, n_cta, s);
}

}  // namespace dspark
