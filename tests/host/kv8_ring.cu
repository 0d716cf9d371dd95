// Host copies of what the 8-bit cache's kernels count with: a load's place in the ring, a vector's exponent byte.
#include "attention_common.cuh"
#include "kv8.cuh"

#define EXPORT extern "C" __attribute__((visibility("default")))

EXPORT unsigned ring_place(int v, unsigned i, unsigned n_tiles) { return dspark::attn::ring_place(v != 0, i, n_tiles); }
EXPORT unsigned exponent_byte(unsigned top) { return dspark::kv8::exponent_byte(top); }
