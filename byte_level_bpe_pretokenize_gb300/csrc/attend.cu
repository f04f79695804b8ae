// Attention over a paged cache in 4 bits: single tokens and short runs of new
// ones (attend.cuh), long runs (attend_wide.cuh), and what chooses between them
// (attend_entry.cuh). A translation unit of its own: its kernels take longest to
// compile.

#include <cmath>

#include "ops.cuh"
#include "vec.cuh"
#include "cache.cuh"
#include "attend.cuh"
#include "attend_wide.cuh"
#include "attend_entry.cuh"
