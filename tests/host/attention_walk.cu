// The attention kernels' walk over their work, run on the host: which KV tiles a range loads, in which order.
// Built by tests/test_attention_walk.py as a shared library.
#include <vector>

#include "attention_common.cuh"

using namespace dspark::attn;

namespace {

AttnArgs args_of(const int* cu, const int* ctx, int bs, int Hkv, int window, int n_sink, int block_shift) {
  AttnArgs a = {};
  a.cu = cu, a.ctx = ctx, a.bs = bs, a.Hkv = Hkv, a.window = window, a.n_sink = n_sink, a.block_shift = block_shift;
  a.cache_limit = int64_t(1) << 30;
  return a;
}

struct Out {
  int* to;
  int n, room;
  void put(int what, int r, int h, int row0, int tile) {
    if (n < room) to[5 * n] = what, to[5 * n + 1] = r, to[5 * n + 2] = h, to[5 * n + 3] = row0, to[5 * n + 4] = tile;
    ++n;
  }
};

}  // namespace

extern "C" {

// The loads of the range of `count` tiles that begins at (r, h, t, tile), as five numbers each: 0 = K or 1 = V, request,
// KV head, packed row of the unit's first token, tile.  Returns how many there are.
__attribute__((visibility("default"))) int loads_of_range(const int* cu, const int* ctx, int bs, int Hkv, int window, int n_sink, int block_shift, int unit_tokens,
                              int r, int h, int t, int tile, unsigned count, int* to, int room) {
  const AttnArgs a = args_of(cu, ctx, bs, Hkv, window, n_sink, block_shift);
  Out out{to, 0, room};
  Cursor cur(Start{r, h, t, tile, cu[r], cu[r + 1] - cu[r], ctx[r], count}, unit_tokens);
  struct Ahead {
    int r, h, row0, tile;
    bool there;
  };
  auto fetch = [&]() {
    Ahead f = {};
    f.there = cur.next(a);
    if (f.there) f.r = cur.s.r, f.h = cur.s.h, f.row0 = cur.s.row0, f.tile = cur.s.tile0 + cur.j;
    return f;
  };
  auto put = [&](int what) {
    return [&out, what](const Ahead& f) {
      out.put(what, f.r, f.h, f.row0, f.tile);
      return out.n < 1 << 20;
    };
  };
  load_in_order(fetch, put(0), put(1));
  return out.n;
}

// KV tiles of unit t of a request.
__attribute__((visibility("default"))) int tiles_of_unit(int c, int n, int t, int window, int n_sink, int block_shift, int unit_tokens) {
  const AttnArgs a = args_of(nullptr, nullptr, 1, 1, window, n_sink, block_shift);
  return unit_geom(a, c, n, t, unit_tokens).ntiles;
}

// Parity of the last use of a ring's slot after n uses.
__attribute__((visibility("default"))) int last_use(int n, int slots, int slot) { return int(last_phase(n, slots, slot)); }

}  // extern "C"
