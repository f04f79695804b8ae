// Attention of long runs of new tokens over a paged cache in 4 bits: the same
// sums as attend.cuh, on tcgen05 tensor cores.
//
// Included once by attend.cu, behind attend.cuh; not a standalone header.
//
// A block takes up to T x 128 columns (a column: a query head of a new token) of
// one cache head. Keys and values become halves in shared memory, 128 tokens at
// a time; scores, weights (as the left factor of the values' product) and
// results live in tensor memory, a row a column.
//
//   scores [128 columns x 128 tokens] = queries x keys^T
//   results [128 columns x dim] += weights x values
//
// Keys and values are halves, off by up to 2^-11 of themselves, in units of 2^e
// that the first 128 tokens give. What does not fit that (an infinity, a NaN,
// sizes 2^9 larger or 2^15 smaller than the largest of those tokens) marks the
// request, which attend.cuh then computes again: so masked tokens spoil no column
// here that may not see them. 16 prompts with such sizes in one block of 50: 5.9 ms
// in place of 0.54.
//
// A step (128 tokens, two tiles of columns, dim 128) takes 3,700 clocks. Its
// 2 x 16 products take 2,450 of them, 76 each where 64 are the tensor cores'
// own: both factors of the scores come from shared memory, 8 KB a product at 128
// bytes a clock, beside what fills it. A tile's softmax, 1,200 to 1,900, is
// hidden behind the other tile's products but for the waits on either side. A
// block's beginning and end take 18,000 clocks (its place among the requests,
// queries, results), so that runs behind little cost more than their products.
// 8,000 new tokens of 16 prompts behind 3,000 each (8 x 128, 4 query heads each):
// 538 us, 855 TFLOP/s, 45% of the measured rate.

namespace {

constexpr int kWideTile = 128;
// Warps: 8 for the softmax of each tile of columns, 4 for each half of 128 tokens; 4 that fill in keys, 4 values; and
// one that issues products.
constexpr int kWideSoftmax = 8, kWideFill = 16, kWideIssue = 24;
constexpr int kWideThreads = 25 * 32;
constexpr uint64_t kPatience = 2000000000;  // nanoseconds of a wait, which lasts microseconds

__device__ __forceinline__ void barrier_init(uint32_t at, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(at), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t at) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(at) : "memory");
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
// Whether the phase of this parity ended; gives up after kPatience or when
// another thread of the block gave up.
__device__ __forceinline__ bool barrier_wait(uint32_t at, uint32_t parity, volatile int* gave_up) {
  uint64_t since = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(at), "r"(parity)
        : "memory");
    if (done) return true;
    if (*gave_up) return false;
    if (i % 16 == 15) {
      const uint64_t now = now_ns();
      if (since == 0) since = now;
      if (now - since > kPatience) break;
    }
  }
  *gave_up = 1;
  return false;
}

// Matrix in shared memory in rows of 128 bytes, swizzled in groups of 8 rows,
// as the low word of its description. K-major (a row: 64 elements of the summed
// dimension): groups of rows are 1024 bytes apart. MN-major (a row: 64 elements
// of the other one): groups of 8 along the sum 1024 bytes, blocks of 64 elements
// `block` bytes apart. Steps within the matrix are added in units of 16 bytes.
__device__ __forceinline__ uint32_t matrix_at(uint32_t at, uint32_t block) { return (at & 0x3FFFF) >> 4 | block >> 4 << 16; }
constexpr uint32_t kMatrixHigh = 1024 >> 4 | 1 << 14 | 2u << 29;

// d (+)= a b, by one thread.
__device__ __forceinline__ void product_smem(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(shape), "r"((uint32_t)add), "r"(kMatrixHigh)
      : "memory");
}
__device__ __forceinline__ void product_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.u32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(shape), "r"((uint32_t)add), "r"(kMatrixHigh)
      : "memory");
}
// Arrives at a barrier when the products issued so far are done.
__device__ __forceinline__ void products_done(uint32_t barrier) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(barrier) : "memory");
}
// Whether this is the one thread of its warp that issues.
__device__ __forceinline__ bool elected() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
  return yes != 0;
}

// 32 columns of a thread's row of tensor memory.
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_store8(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Two additions, or products and sums, at once.
__device__ __forceinline__ float2 add_two(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 c, a, b;\n mov.b64 {%0, %1}, c;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 fma_two(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float max_three(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// What this thread wrote to shared memory is there for the tensor cores.
__device__ __forceinline__ void publish() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int G, int T>
struct WideShape {
  static constexpr int kTiles = T;                // of 128 columns
  static constexpr int kStages = G <= 4 ? 2 : 1;  // of 128 tokens
  static constexpr int kSubs = (G + 1) / 2;       // blocks of 64 elements
  static constexpr int kSub = kWideTile * 128;    // bytes of one
  static constexpr int kBytes = kSubs * kSub;     // of 128 rows
  static constexpr int kDim = 32 * G;
  static constexpr int kQueries = 0, kKeys = kTiles * kBytes, kValues = kKeys + kStages * kBytes;
  static constexpr int kEnd = kValues + kStages * kBytes;
  // more than half of an SM's, for a block has all of its tensor memory
  static constexpr int kSmem = (kEnd > 118 * 1024 ? kEnd : 118 * 1024) + 1024;
  static constexpr int kScoresAt = 0, kResultsAt = kTiles * kWideTile;  // columns of tensor memory
};

struct WideShared {
  uint64_t keys_full[2], values_full[2];
  // of each tile of columns, for even and odd steps; those of the last tile also say that a stage is free: of keys
  // when its scores are there, of values when the next step's are, which are made behind its results
  uint64_t scores_full[2][2];
  uint64_t weights_full[2], results_full[2], queries_full, units_full, drained;
  uint32_t tmem;
  int power[2];      // of keys and of values: they are stored in units of 2^power
  float largest[2][4];
  float half_row[2][2][kWideTile];  // of each tile: what the halves of a row tell each other
  int query_size[2][kWideTile];  // the largest element of a column's query, as bits
  int gave_up;
};

// Keys (or values) of 128 tokens at a time, a thread a token, 64 elements after
// another with the next ones on their way. A code gets the exponent of 1024
// before it, becomes n by one exact operation, and base + step n by another that
// rounds.
template <int G, int T>
__device__ void wide_fill(const AttendArgs& a, WideShared& sm, int which, uint32_t tile0, int r, int h, int limit,
                          int n_tiles, int last_tile, int* redo) {
  using Shape = WideShape<G, T>;
  constexpr int U = Shape::kSubs;
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const uint32_t full = (uint32_t)__cvta_generic_to_shared(which ? sm.values_full : sm.keys_full);
  const uint32_t free = (uint32_t)__cvta_generic_to_shared(sm.scores_full[last_tile]);
  const unsigned char* pages = a.cache + ((int64_t)which * a.heads + h) * a.page_bytes;
  const int32_t* table = a.table + (int64_t)r * a.table_stride;
  bool bad = false;
  const unsigned char* codes = nullptr;  // of the token's row, or null
  const uint32_t* words = nullptr;       // its pairs
  int32_t entry = -1;
  auto look_up = [&](int i) {
    const int t = i * kWideTile + tid;
    entry = t < limit ? __ldg(table + a.block((uint32_t)t)) : -1;
  };
  auto find = [&](int i) {
    const int t = i * kWideTile + tid;
    codes = nullptr;
    if (t >= limit) return;
    if ((uint32_t)entry >= (uint32_t)a.n_blocks || entry < 0) {
      bad = true;  // reported by the other kernel, which leaves its tokens out
      return;
    }
    const uint32_t row = (uint32_t)t - a.block((uint32_t)t) * a.block.d;
    const unsigned char* page = pages + (int64_t)entry * a.block_stride;
    codes = page + (int64_t)row * (16 * G);
    words = reinterpret_cast<const uint32_t*>(page + ((int64_t)a.block.d * 16 + (int64_t)row * 4) * G);
  };
  look_up(0);
  find(0);
  // the unit: the largest of the first 128 tokens becomes 2^6 to 2^7
  float most = 0.f;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const uint32_t z = codes ? __ldg(words + j) : 0;
    most = fmaxf(most, fabsf(bf16_high(z)) + 16.f * bf16_low(z));
  }
  if (!(most < INFINITY)) most = 0.f;
  most = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most)));
  if (lane == 0) sm.largest[which][tid >> 5] = most;
  asm volatile("bar.sync %0, 128;" ::"r"(1 + which) : "memory");
#pragma unroll
  for (int w = 0; w < 4; ++w) most = fmaxf(most, sm.largest[which][w]);
  const int power = most > 0.f ? min(max((__float_as_int(most) >> 23) - 127 - 6, -100), 100) : 0;
  if (tid == 0) sm.power[which] = power;
  const float unit = power_of_2(-power);
  barrier_arrive((uint32_t)__cvta_generic_to_shared(&sm.units_full));

  uint4 next[2];
  uint32_t next_pair[2];
  auto load = [&](int u) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool there = codes && 2 * u + k < G;
      next[k] = there ? __ldg(reinterpret_cast<const uint4*>(codes) + 2 * u + k) : make_uint4(0, 0, 0, 0);
      next_pair[k] = there ? __ldg(words + 2 * u + k) : 0;
    }
  };
  load(0);
  if (n_tiles > 1) look_up(1);
  const __half2 less = __float2half2_rn(-1024.f), by = __float2half2_rn(0.0625f), less16 = __float2half2_rn(-64.f);
  for (int i = 0; i < n_tiles; ++i) {
    const int stage = i % Shape::kStages;
    const uint32_t to = tile0 + stage * Shape::kBytes + tid * 128;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t now[8] = {next[0].x, next[0].y, next[0].z, next[0].w, next[1].x, next[1].y, next[1].z, next[1].w};
      const uint32_t z[2] = {next_pair[0], next_pair[1]};
      if (u + 1 < U) {
        load(u + 1);
      } else if (i + 1 < n_tiles) {
        find(i + 1);
        load(0);
        if (i + 2 < n_tiles) look_up(i + 2);
      }
      if (u == 0 && i >= Shape::kStages) {  // which step's scores say that the stage is free
        const int step = i - Shape::kStages + which;
        if (!barrier_wait(free + 8 * (step & 1), step >> 1 & 1, &sm.gave_up)) return;
      }
      __half2 st[2], ba[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x = bf16_low(z[k]) * unit, y = bf16_high(z[k]) * unit, size = fabsf(y) + 16.f * x;
        // too large for halves or no number, or too small for what is left of their bits (of keys too: a query may ask
        // for a small group alone)
        if (!(size < 32768.f) || (size > 0.f && size < 0x1p-9f)) bad = true;
        st[k] = __float2half2_rn(x);
        ba[k] = __float2half2_rn(y);
      }
      const bool pair = 2 * u + 1 < G;  // else a group by itself
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (!pair && w >= 4) break;
        const int k = pair ? w & 1 : 0, chunk = pair ? 4 * (w & 1) + w / 2 : w;  // group, and 8 elements of 64
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = e < 2 ? now[w] : now[w] >> 8;
          const uint32_t y = (x & (e & 1 ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
          const __half2 n = e & 1 ? __hfma2(*reinterpret_cast<const __half2*>(&y), by, less16)
                                  : __hadd2(*reinterpret_cast<const __half2*>(&y), less);
          const __half2 v = __hfma2(n, st[k], ba[k]);
          out[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        const uint32_t at = to + u * Shape::kSub + ((chunk ^ (tid & 7)) << 4);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(out[0]), "r"(out[1]), "r"(out[2]), "r"(out[3])
                     : "memory");
      }
    }
    publish();
    barrier_arrive(full + 8 * stage);
  }
  if (bad) atomicOr(redo + r, 1);
}

template <int G, int T>
__global__ void __launch_bounds__(kWideThreads, 1) k_attend_wide(AttendArgs a, int* redo) {
  using Shape = WideShape<G, T>;
  constexpr int kCols = Shape::kTiles * kWideTile;
  extern __shared__ unsigned char raw[];
  __shared__ WideShared sm;
  __shared__ int64_t upto[kWideThreads + 1];
  __shared__ int64_t warp_sum[kWideThreads / 32];
  __shared__ int found[4];  // request, head, first column
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- this block's columns: requests in order, each from its last columns on, heads in turn ----
  const int each = (a.n + kWideThreads - 1) / kWideThreads;
  const int r0 = min(a.n, tid * each), r1 = min(a.n, r0 + each);
  auto blocks_of = [&](int r) -> int64_t {
    const AttendRequest q = attend_request(a, r, false);
    const int64_t cols = (int64_t)q.fresh * a.group.d;
    return cols < kWideMin ? 0 : (cols + kCols - 1) / kCols * a.heads;
  };
  int64_t x = 0;
  for (int r = r0; r < r1; ++r) x += blocks_of(r);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += o;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += warp_sum[w];
  upto[tid + 1] = x;
  if (tid == 0) upto[0] = 0;
  __syncthreads();
  const int64_t me = blockIdx.x;
  if (me == 0 && upto[kWideThreads] > gridDim.x) {
    // Offsets fall, so that requests share tokens and have more columns than the tokens. Those that the blocks do not
    // reach are left to attend.cuh.
    int64_t end = upto[tid];
    for (int r = r0; r < r1; ++r) {
      const int64_t n = blocks_of(r);
      end += n;
      if (n > 0 && end > gridDim.x) atomicOr(redo + r, 1);
    }
  }
  if (me >= upto[kWideThreads]) return;
  if (upto[tid] <= me && me < upto[tid + 1]) {
    int64_t rest = me - upto[tid];
    for (int r = r0; r < r1; ++r) {
      const int64_t n = blocks_of(r);
      if (rest < n) {
        const int tiles = (int)(n / a.heads);
        found[0] = r;
        found[1] = (int)(rest % a.heads);
        found[2] = (tiles - 1 - (int)(rest / a.heads)) * kCols;
        break;
      }
      rest -= n;
    }
  }
  if (tid == 0) {
    auto at = [&](uint64_t& b) { return (uint32_t)__cvta_generic_to_shared(&b); };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      barrier_init(at(sm.keys_full[s]), 128);
      barrier_init(at(sm.values_full[s]), 128);
      barrier_init(at(sm.scores_full[s][0]), 1);
      barrier_init(at(sm.scores_full[s][1]), 1);
      barrier_init(at(sm.weights_full[s]), 256);
      barrier_init(at(sm.results_full[s]), 1);
    }
    barrier_init(at(sm.queries_full), 256 * Shape::kTiles);
    barrier_init(at(sm.units_full), 256);
    barrier_init(at(sm.drained), 1);
    sm.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWideIssue) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    before_sync();
  }
  __syncthreads();
  after_sync();
  constexpr uint32_t tmem = 0;  // all of it: it begins at its beginning
  const int r = found[0], h = found[1], first_col = found[2], group = (int)a.group.d;
  const AttendRequest q = attend_request(a, r, false);
  const int cols = min(kCols, q.fresh * group - first_col);
  const int tiles = (cols + kWideTile - 1) / kWideTile;  // of columns that there are
  // tokens that the last column sees
  const int limit = max(0, q.len - q.fresh + (first_col + cols - 1) / group + 1);
  const int n_tiles = (limit + kWideTile - 1) / kWideTile;
  const uint32_t smem = ((uint32_t)__cvta_generic_to_shared(raw) + 1023u) & ~1023u;
  auto bar = [&](uint64_t& b) { return (uint32_t)__cvta_generic_to_shared(&b); };

  if (n_tiles == 0) {
    // nothing is seen: zeros below
  } else if (warp == kWideIssue) {
    constexpr uint32_t kToScores = 1u << 4 | (kWideTile / 8) << 17 | (kWideTile / 16) << 24;
    constexpr uint32_t kToResults = 1u << 4 | 1u << 16 | (uint32_t)(Shape::kDim / 8) << 17 | (kWideTile / 16) << 24;
    const uint32_t queries = matrix_at(smem + Shape::kQueries, 16), keys = matrix_at(smem + Shape::kKeys, 16);
    const uint32_t values = matrix_at(smem + Shape::kValues, Shape::kSub);
    auto scores = [&](int t, int i) {
      const uint32_t qs = queries + t * (Shape::kBytes / 16), ks = keys + i % Shape::kStages * (Shape::kBytes / 16);
      const uint32_t d = tmem + Shape::kScoresAt + t * kWideTile;
#pragma unroll
      for (int k = 0; k < 2 * G; ++k)
        product_smem(d, qs + (k / 4 * Shape::kSub + k % 4 * 32) / 16, ks + (k / 4 * Shape::kSub + k % 4 * 32) / 16,
                     kToScores, k > 0);
      products_done(bar(sm.scores_full[t][i & 1]));
    };
    if (elected()) {
      bool ok = barrier_wait(bar(sm.queries_full), 0, &sm.gave_up) && barrier_wait(bar(sm.keys_full[0]), 0, &sm.gave_up);
      if (ok) {
        after_sync();
        for (int t = 0; t < tiles; ++t) scores(t, 0);
      }
      for (int i = 0; ok && i < n_tiles; ++i) {
        const int stage = i % Shape::kStages, next = (i + 1) % Shape::kStages;
        ok = barrier_wait(bar(sm.values_full[stage]), i / Shape::kStages & 1, &sm.gave_up);
        for (int t = 0; ok && t < tiles; ++t) {
          ok = barrier_wait(bar(sm.weights_full[t]), i & 1, &sm.gave_up);
          if (!ok) break;
          after_sync();
          const uint32_t vs = values + stage * (Shape::kBytes / 16);
          const uint32_t d = tmem + Shape::kResultsAt + t * Shape::kDim, w = tmem + Shape::kScoresAt + t * kWideTile;
#pragma unroll
          for (int k = 0; k < kWideTile / 16; ++k)
            product_tmem(d, w + k / 4 * 64 + k % 4 * 8, vs + k * 2048 / 16, kToResults, i > 0 || k > 0);
          if (i + 1 < n_tiles) {
            if (t == 0) {
              ok = barrier_wait(bar(sm.keys_full[next]), (i + 1) / Shape::kStages & 1, &sm.gave_up);
              if (!ok) break;
              after_sync();
            }
            scores(t, i + 1);
          } else {
            products_done(bar(sm.results_full[t]));
          }
        }
      }
      if (!ok) {  // products must not outlive the block
        int alone = 0;
        products_done(bar(sm.drained));
        barrier_wait(bar(sm.drained), 0, &alone);
      }
    }
    __syncwarp();
  } else if (warp >= kWideFill) {
    const int which = (warp - kWideFill) / 4;
    wide_fill<G, T>(a, sm, which, smem + (which ? Shape::kValues : Shape::kKeys), r, h, limit, n_tiles, tiles - 1, redo);
  } else if (warp / kWideSoftmax >= tiles) {
    if (warp / kWideSoftmax < Shape::kTiles) barrier_arrive(bar(sm.queries_full));
  } else {
    // ---- two threads a column: each has half of every 128 tokens, and of the results ----
    const int t = warp / kWideSoftmax, half = warp >> 2 & 1, row = tid & 127, col = first_col + t * kWideTile + row;
    const bool real = t * kWideTile + row < cols;
    const int token = (int)a.group((uint32_t)col);
    const int sees = real ? max(0, q.len - q.fresh + token + 1) : 0;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // of tensor memory
    const uint32_t s_at = tmem + lanes + Shape::kScoresAt + t * kWideTile + half * 64;
    const uint32_t o_at = tmem + lanes + Shape::kResultsAt + t * Shape::kDim;
    float* const mine = &sm.half_row[t][half][row];
    const float* const other = &sm.half_row[t][1 - half][row];
    auto meet = [&] { asm volatile("bar.sync %0, 256;" ::"r"(3 + t) : "memory"); };  // all threads of the tile
    float to_score;
    {
      // The tile's queries, 8 elements a thread at a time, neighbours in a row: read once for each row's largest
      // element, and again, from the caches, to be scaled and stored.
      const int in_tile = tid & 255;
      sm.query_size[t][row] = 0;
      meet();
      auto scale_of = [&](int of) {  // the largest element in [2^6, 2^7)
        return power_of_2(min(max(6 - ((sm.query_size[t][of] >> 23) - 127), -120), 120));
      };
      auto queries = [&](auto type, auto wide_tag) {
        using TQ = decltype(type);
        constexpr bool kVectors = decltype(wide_tag)::value;
        // without branches where rows are vectors, so that loads are in flight together
        auto get = [&](int k, int& of, int& at, float (&e)[8]) {
          const int i = k * 256 + in_tile;
          of = i / (4 * G);
          at = i % (4 * G);
          const bool there = t * kWideTile + of < cols && 8 * at < a.dim;
          const int c = first_col + (there ? t * kWideTile + of : 0), of_token = (int)a.group((uint32_t)c);
          const TQ* x = static_cast<const TQ*>(a.queries) + (int64_t)(q.first + of_token) * a.q_token +
                       (h * group + c - of_token * group) * a.q_head + (there ? 8 * at : 0);
          if constexpr (kVectors) {
            Vec<TQ, 8> v;
            v.template load<true>(x);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = there ? to_f32(v.x[j]) : 0.f;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = there && 8 * at + j < a.dim ? to_f32(x[j]) : 0.f;
          }
        };
        constexpr int kAtOnce = kVectors && G % 2 == 0 ? 4 : kVectors ? 2 : 1;
        int of[kAtOnce], at[kAtOnce];
        float e[kAtOnce][8];
        for (int k0 = 0; k0 < 2 * G; k0 += kAtOnce) {
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) get(k0 + k, of[k], at[k], e[k]);
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(e[k][j]));
            if constexpr (32 % (4 * G) == 0) {  // a row's threads are neighbours
#pragma unroll
              for (int d = 1; d < 4 * G; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
              if (at[k] == 0) sm.query_size[t][of[k]] = __float_as_int(most);
            } else {
              atomicMax(&sm.query_size[t][of[k]], __float_as_int(most));
            }
          }
        }
        meet();
        const uint32_t to = smem + Shape::kQueries + t * Shape::kBytes;
        for (int k0 = 0; k0 < 2 * G; k0 += kAtOnce) {
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) get(k0 + k, of[k], at[k], e[k]);
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            const float by = a.scale < 0.f ? -scale_of(of[k]) : scale_of(of[k]);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_halves(e[k][i] * by, e[k][i + 4] * by);
            const uint32_t place = to + (at[k] >> 3) * Shape::kSub + of[k] * 128 + (((at[k] & 7) ^ (of[k] & 7)) << 4);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(place), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          }
        }
      };
      if (a.q_type == BPE_F16) {
        if (a.q_wide) queries(__half{}, std::true_type{});
        else queries(__half{}, std::false_type{});
      } else {
        if (a.q_wide) queries(__nv_bfloat16{}, std::true_type{});
        else queries(__nv_bfloat16{}, std::false_type{});
      }
      to_score = fabsf(a.scale) / scale_of(row);
    }
    publish();
    barrier_arrive(bar(sm.queries_full));
    bool ok = barrier_wait(bar(sm.units_full), 0, &sm.gave_up);
    to_score *= power_of_2(sm.power[0]);
    // weights are 2^6 at the reference, which follows the maximum only when it is 2^8 behind
    float reference = -INFINITY, total = 0.f;
    for (int i = 0; i < n_tiles; ++i) {  // to the end even where a wait gave up: the threads of a tile meet in each step
      ok = ok && barrier_wait(bar(sm.scores_full[t][i & 1]), i >> 1 & 1, &sm.gave_up);
      ok = __all_sync(0xFFFFFFFFu, ok);
      after_sync();
      const int left = sees - i * kWideTile - half * 64;  // tokens of this half that the column sees
      const bool all = __all_sync(0xFFFFFFFFu, left >= 64);
      // the scores, 16 at a time, the next ones on their way
      auto scores = [&](auto use) {
        uint32_t s[2][16];
        tmem_load16(s[0], s_at);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          tmem_loaded();
          if (k < 3) tmem_load16(s[(k + 1) & 1], s_at + 16 * (k + 1));
          use(k, s[k & 1]);
        }
      };
      float most = -INFINITY;
      if (ok && all) {
        scores([&](int, const uint32_t* s) {
#pragma unroll
          for (int j = 0; j < 16; j += 2) most = max_three(most, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
        });
      } else if (ok) {
        scores([&](int k, const uint32_t* s) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (16 * k + j < left) most = fmaxf(most, __uint_as_float(s[j]));
        });
      }
      *mine = most;
      meet();
      if (!ok) continue;
      most = fmaxf(most, *other) * to_score;
      if (__any_sync(0xFFFFFFFFu, most > reference + 8.f)) {
        const float next = fmaxf(reference, most), f = next > reference ? exp2_fast(reference - next) : 1.f;
        total *= f;
        reference = next;
        if (i > 0) {
          for (int k = half; k < G; k += 2) {
            uint32_t o[32];
            tmem_load(o, o_at + 32 * k);
            tmem_loaded();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_store(o_at + 32 * k, o);
          }
        }
      }
      const float minus = 6.f - (reference == -INFINITY ? 0.f : reference);
      const float2 by = make_float2(to_score, to_score), less = make_float2(minus, minus);
      float2 sum = make_float2(0.f, 0.f);
      auto weigh = [&](auto all_tag) {
        scores([&](int k, const uint32_t* s) {
          uint32_t p[8];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float2 z = fma_two(make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), by, less);
            float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
            if (!decltype(all_tag)::value) {
              if (16 * k + j >= left) e.x = 0.f;
              if (16 * k + j + 1 >= left) e.y = 0.f;
            }
            sum = add_two(sum, e);
            p[j / 2] = pack_halves(e.x, e.y);
          }
          tmem_store8(s_at + 8 * k, p);  // over scores that were read
        });
      };
      if (all) weigh(std::true_type{});
      else weigh(std::false_type{});
      total += sum.x + sum.y;
      tmem_stored();
      before_sync();
      barrier_arrive(bar(sm.weights_full[t]));
    }
    meet();  // what the halves told each other is read
    *mine = total;
    meet();
    total += *other;
    ok = ok && barrier_wait(bar(sm.results_full[t]), 0, &sm.gave_up);
    if (__all_sync(0xFFFFFFFFu, ok)) {
      after_sync();
      const float by = total == 0.f ? 0.f : power_of_2(sm.power[1]) / total;
      // 32 columns at a time through shared memory, where the queries are needed no more, so that a row's neighbours
      // are stored together
      constexpr bool kBoth = Shape::kBytes >= 8 * 4096;  // room for both halves' threads
      const uint32_t stage = smem + Shape::kQueries + t * Shape::kBytes + (warp & (kBoth ? 7 : 3)) * 4096;
      int64_t to[8];  // rows that this thread stores in
      uint32_t there = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int in_block = t * kWideTile + (warp & 3) * 32 + 4 * i + lane / 8;
        const int at = first_col + in_block, of_token = (int)a.group((uint32_t)at);
        to[i] = (int64_t)(q.first + of_token) * a.o_token + (h * group + at - of_token * group) * a.o_head;
        there |= (uint32_t)(in_block < cols) << i;
      }
      for (int k = kBoth || !half ? half : G; k < G; k += kBoth ? 2 : 1) {
        uint32_t o[32];
        tmem_load(o, o_at + 32 * k);
        tmem_loaded();
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // in each 8 in the order 0, 4, 1, 5, 2, 6, 3, 7
          auto e = [&](int i) { return __uint_as_float(o[8 * (c / 2) + 2 * i + c % 2]) * by; };
          asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(stage + lane * 128 + ((c ^ (lane & 7)) << 4)),
                       "f"(e(0)), "f"(e(1)), "f"(e(2)), "f"(e(3))
                       : "memory");
        }
        __syncwarp();
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int of = 4 * i + lane / 8;
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(v[i].x), "=f"(v[i].y), "=f"(v[i].z), "=f"(v[i].w)
                       : "r"(stage + of * 128 + (((lane % 8) ^ (of & 7)) << 4)));
        }
        const int at = 32 * k + 4 * (lane % 8);
        if (a.o_wide && a.out_type != BPE_F32) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint2 w;
            if (a.out_type == BPE_F16) {
              w = make_uint2(pack_halves(v[i].x, v[i].y), pack_halves(v[i].z, v[i].w));
            } else {
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v[i].y), "f"(v[i].x));
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v[i].w), "f"(v[i].z));
            }
            if (there >> i & 1 && at < a.dim)
              __stcs(reinterpret_cast<uint2*>(static_cast<unsigned short*>(a.out) + to[i] + at), w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (there >> i & 1) attend_store(a, to[i], at, v[i]);
        }
        __syncwarp();
      }
      before_sync();
    }
  }
  if (n_tiles == 0) {
    for (int i = tid; i < cols * (Shape::kDim / 4); i += kWideThreads) {
      const int col = first_col + i / (Shape::kDim / 4), token = col / group, head = h * group + col - token * group;
      attend_store(a, (int64_t)(q.first + token) * a.o_token + head * a.o_head, i % (Shape::kDim / 4) * 4,
                   make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
  __syncthreads();
  if (tid == 0 && sm.gave_up) atomicOr(&a.small->op_status, kStTimeout);
  after_sync();
  if (warp == kWideIssue) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace
