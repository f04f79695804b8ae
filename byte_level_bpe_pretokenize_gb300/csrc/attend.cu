// Attention over a paged cache in 4 bits (attend.cuh). A translation unit of
// its own: its kernels take longest to compile.

#include <cmath>

#include "ops.cuh"
#include "vec.cuh"
#include "cache.cuh"
#include "attend.cuh"
