// Operators on a paged cache of keys and values in 4 bits, as bpe_plan_blocks
// plans it: rotary positions (rotary.cuh), rows into their slots and back
// (cache_rows.cuh, layout in cache.cuh). The attention over it is attend.cu.
// The source pages end at the ids; these have no counterpart there.

#include <cmath>

#include "ops.cuh"
#include "vec.cuh"
#include "cache.cuh"
#include "rotary.cuh"
#include "cache_rows.cuh"
