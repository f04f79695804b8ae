// Attention of new tokens over a paged cache in 4 bits (cache.cuh).
//
// Included once by attend.cu; not a standalone header.
//
//   s_t = scale * (query . key_t),  out = sum_t e^(s_t - m) value_t / sum_t e^(s_t - m)
//
// over the tokens t that the query sees, in one pass with the running maximum m.
// With the codes n, the steps S and bases B of group j,
//   query . key_t = sum_j S_tj (sum_i q_i n_ti) + B_tj (sum_i q_i)
//   out_i = sum_t (p_t S_tj) (n_ti - 8) + sum_t p_t (B_tj + 8 S_tj)
// All sums over i and t run on the tensor cores. A code is its own bits there: a
// mask leaves it in the lowest or the next four of a half's mantissa, where it
// is the subnormal n 2^-24 or n 2^-20, exactly; queries and weights carry what
// is lacking. Keys' steps stay outside, in 32 bits; values' steps go to the
// weights, whose mean with n - 8 loses less to their rounding than with n.

namespace {

constexpr int kUnit = 32;      // tokens of a step
constexpr int kItemCost = 3;   // what beginning and ending an item takes, in steps
constexpr int kAttMaxWarps = 16;  // workers of an SM
// Sizes of values, |base| + 16 step, are compared as the bits of floats. Those that a worker takes as halves lie below a
// cap, a power of two, which becomes 2^8, and at most kApart powers of two below it. Weights are 2^11 at most and off by
// 2^-25 where that is more than their own rounding, so a token loses at most 2^(kApart - 36) of the largest part of a
// sum. Where sizes are further apart a step is added up in 32 bits (below). 2^12 leaves room for first tokens of next to
// nothing among others; 32-bit queries expect more of their sums. 384 requests of 4,000 tokens (8 x 128, 8 query heads
// each) with one group of every value 2^20 smaller: 2,450 us, with all values of one block in 50 2^20 larger 840,
// without either 427. No look at sizes: 417, and what is 2^20 smaller is off by 2^-8, what is 2^30 smaller lost.
template <int P>
constexpr int kApart = P == 1 ? 12 : 8;
constexpr int kLeastCap = 16 << 23;    // so that 1 / unit is a float
constexpr int kFarApart = 32 << 23;    // above the cap, where sums are in 32 bits
constexpr int kNoLow = 0x7FFFFFFF;
// The unit of values below a cap, and what divides by it.
__device__ __forceinline__ float unit_of(int cap) { return __int_as_float(cap - (8 << 23)); }
__device__ __forceinline__ float per_unit(int cap) { return __uint_as_float((262u << 23) - (uint32_t)cap); }
constexpr int kWideMin = BPE_ATTEND_LONG;  // columns of a request from which attend_wide.cuh takes it

struct AttendArgs {
  const void* queries;
  void* out;
  int q_type, out_type;
  int64_t q_token, q_head, o_token, o_head;
  int64_t n_tokens;
  int heads, dim;
  FastDiv group;
  const unsigned char* cache;
  int64_t n_blocks, block_stride, page_bytes;
  FastDiv block;
  const int32_t* table;
  int64_t table_stride, capacity;  // capacity: tokens of a table row
  const int32_t* seq_lens;
  const int64_t* offsets;
  int n;
  float scale;            // times log2 e
  bool q_wide, o_wide;    // rows are aligned for vectors
  bool centre;            // codes of values count from their middle
  bool near;              // the cache lies within 2^32 times 16 bytes
  float* partial;
  int4* record;
  const int* redo;        // requests of kWideMin columns on that are computed here all the same; null: all of them
  DevSmall* small;
};

struct AttendRequest {
  int first, fresh, len;  // first new token, new tokens, tokens in the cache
};

__device__ __forceinline__ AttendRequest attend_request(const AttendArgs& a, int r, bool report) {
  AttendRequest q;
  const int64_t first = a.offsets ? __ldg(a.offsets + r) : r, end = a.offsets ? __ldg(a.offsets + r + 1) : r + 1;
  q.len = __ldg(a.seq_lens + r);
  const bool ok = first >= 0 && end >= first && end <= a.n_tokens, fits = q.len >= 0 && q.len <= a.capacity;
  q.first = ok ? (int)first : 0;
  q.fresh = ok ? (int)(end - first) : 0;
  if (!fits) q.len = 0;
  if (report && !(ok && fits)) atomicOr(&a.small->op_status, kStBadInput);
  return q;
}

// The request as far as it is computed here.
__device__ __forceinline__ AttendRequest attend_mine(const AttendArgs& a, int r, bool report) {
  AttendRequest q = attend_request(a, r, report);
  if (a.redo && (int64_t)q.fresh * a.group.d >= kWideMin && !__ldg(a.redo + r)) q.fresh = 0;
  return q;
}

// d = a b, and d += a b. The first needs no zeros in registers.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The codes of a word's halves, e = 0 and 1 of the word itself or e = 2 and 3 of
// the word shifted by 8. As subnormal halves, n 2^-24 and n 2^-20, they cost one
// operation, but the tensor cores cut sums off some 24 bits below a product's
// exponent, which for a subnormal is 2^-14: that leaves 2^-15 of a sum, enough for
// results of 16 bits. For 32-bit ones (P = 2) they become n - kFrom in the normal
// range, two operations more.
template <int P, int kFrom>
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
  if (P == 1) return w & 0x000F000Fu;
  const uint32_t x = (w & 0x000F000Fu) | 0x64006400u;  // 1024 + n
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(1024.f + kFrom));
  return *reinterpret_cast<const uint32_t*>(&y);
}
template <int P, int kFrom>
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
  if (P == 1) return w & 0x00F000F0u;
  const uint32_t x = (w & 0x00F000F0u) | 0x64006400u;  // 1024 + 16 n
  const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(0.0625f), __float2half2_rn(-64.f - kFrom));
  return *reinterpret_cast<const uint32_t*>(&y);
}
// what brings them back
template <int P>
constexpr float kCodesEven = P == 1 ? 0x1p24f : 1.f;
template <int P>
constexpr float kCodesOdd = P == 1 ? 0x1p20f : 1.f;
constexpr uint32_t kMinus8Even = 0x80088008u, kMinus8Odd = 0x80808080u;  // of the subnormals

// 2^x for whole x in [-126, 127].
__device__ __forceinline__ float power_of_2(int x) { return __int_as_float((x + 127) << 23); }

__device__ __forceinline__ uint32_t pack_halves(float low, float high) {
  const __half2 h = __floats2half2_rn(low, high);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_halves(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int kBytes, bool kThere>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool there) {
  if constexpr (kThere) {
    if constexpr (kBytes == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(kBytes) : "memory");
  } else {
    const int size = there ? kBytes : 0;  // else zeros
    if constexpr (kBytes == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(size) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(kBytes), "r"(size) : "memory");
  }
}

// Cuts x and y into kParts halves each that add up to them: two leave 2^-24 of a
// number that stays above 2^-2.
template <int kParts>
__device__ __forceinline__ void split_halves(float x, float y, uint32_t (&part)[kParts]) {
  part[0] = pack_halves(x, y);
  if (kParts == 2) {
    const float2 lead = unpack_halves(part[0]);
    part[kParts - 1] = pack_halves(x - lead.x, y - lead.y);
  }
}

// Where the tokens of all requests are cut. A request with new tokens has
// heads x tiles items (a tile: 8 NT columns, a column a query head of a new
// token), each of its tokens in steps of kUnit (one at least, so that every row
// is written), before which kItemCost places count for its beginning and end.
// The places of all items in a row are dealt out evenly.
struct AttendCursor {
  int r, h, tile;    // request, head, tile
  int tiles, units;  // of the request; steps of the item
  AttendRequest q;
};

template <int kCols>
__device__ __forceinline__ void attend_sizes(const AttendArgs& a, AttendCursor& c) {
  c.units = max(1, (c.q.len + kUnit - 1) / kUnit);
  c.tiles = (int)(((int64_t)c.q.fresh * a.group.d + kCols - 1) / kCols);
}

template <int kCols>
__device__ __forceinline__ int64_t attend_units(const AttendArgs& a, int r, bool report) {
  AttendCursor c;
  c.q = attend_mine(a, r, report);
  attend_sizes<kCols>(a, c);
  return (int64_t)(c.units + kItemCost) * c.tiles * a.heads;
}

// The next item.
template <int kCols>
__device__ __forceinline__ void attend_next(const AttendArgs& a, AttendCursor& c) {
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.h < a.heads) return;
  c.h = 0;
  do {
    ++c.r;
    c.q.fresh = 0;
    if (c.r < a.n) c.q = attend_mine(a, c.r, false);
  } while (c.q.fresh == 0 && c.r < a.n);
  attend_sizes<kCols>(a, c);
}

template <int G, int kParts, int NT>
struct AttendShape {
  static constexpr int kCols = 8 * NT;
  static constexpr int kUnits = (G + 1) / 2;                         // pairs of groups
  static constexpr int kRow = 16 * G, kPair = 4 * G;                 // bytes of a row's codes, of its pairs
  static constexpr int kHalfStage = kUnit * (kRow + kPair);          // keys, or values
  static constexpr int kStage = 2 * kHalfStage;
  static constexpr int kScores = NT * kUnit * 8 * 4;
  static constexpr int kSteps = G * kUnit * 2;                       // values' steps as halves, and mids likewise
  // As many warps an SM as registers allow: 8 x 2 of 128, 6 x 2 of 168 or 8 of 255. The queries, which only the first
  // half of a step needs, stay in shared memory where it has room for them.
  static constexpr bool kSmall = G <= 4 && NT == 1 && kParts == 1;
  static constexpr bool kMiddle = kParts == 1 && (NT == 1 ? G == 3 || G == 4 : G <= 2);
  static constexpr bool kQueriesShared = kParts == 1 && G <= 6;
  static constexpr int kQueries = kQueriesShared ? NT * G * 512 : 0;
  static constexpr int kWarp = 2 * kStage + kScores + (1 + kParts) * kSteps + kQueries;
  static constexpr int kBlocks = kSmall || kMiddle ? 2 : 1;
  static constexpr int kWarps = kMiddle ? 6 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kSmem = kWarps * kWarp;
  static constexpr int kPartial = kCols * (32 * G + 2);              // floats of an item's partial sums
  static constexpr int kBaseMmas = (3 * kUnits + 7) / 8;             // products of keys' bases
};

// Rows of 64 and of 128 bytes lie on two and on one set of banks: their 32-byte
// pieces are exchanged, so that the eight-byte loads of four rows meet no other.
template <int G>
__device__ __forceinline__ uint32_t attend_piece(uint32_t row, uint32_t piece) {
  if (G == 4) return piece ^ (row >> 1 & 1);
  if (G == 8) return piece ^ (row & 3);
  return piece;
}

// Four elements of a row from `at` on, rounded to the output's type.
__device__ __forceinline__ void attend_store(const AttendArgs& a, int64_t row, int at, float4 r) {
  if (at >= a.dim) return;
  auto put = [&](auto type) {
    using T = decltype(type);
    T* to = static_cast<T*>(a.out) + row + at;
    Vec<T, 4> v;
    v.x[0] = from_f32<T>(r.x), v.x[1] = from_f32<T>(r.y), v.x[2] = from_f32<T>(r.z), v.x[3] = from_f32<T>(r.w);
    if (a.o_wide) {
      v.store(to);
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (at + e < a.dim) to[e] = v.x[e];
  };
  if (a.out_type == BPE_F32) put(float{});
  else if (a.out_type == BPE_F16) put(__half{});
  else put(__nv_bfloat16{});
}

// A warp is a worker: it walks its share of the steps with the next step's codes
// on their way into its own half of shared memory, and waits for no other warp.
// What it has of an item that other workers share goes to the workspace
// (k_attend_join). Keys are the left factor of a product (16 tokens x 16
// elements) and so are values (16 elements x 16 tokens), both straight from
// their codes into registers; the few columns are the right factor. So the tiles
// of 8 columns of mma.sync leave little unused, where tcgen05 would take 128 rows
// of keys from shared memory in 16 bits, four times the bytes that a code has
// there.
//
// Bound by issue and latency: 373 instructions for 16 tokens of 128 elements (80
// of them take the codes apart, 25 are products, 45 the copies, 60 the softmax),
// at 56% of the slots with the 12 warps that 168 registers leave; 8 x 2 warps of
// 128 registers spill and take 455 us where 6 x 2 take 428, 7 x 2 450. 384
// requests of 4,000 tokens (8 x 128, 8 query heads each): 427 us, 4.7 TB/s of
// codes and pairs. Weights in two bfloat16 parts outside the codes' products, and
// codes as 1 + n / 16, took 868 us.
//
// P is 1 for 16-bit queries, which a half holds without loss once they are
// scaled by a power of two, and 2 for 32-bit ones. Weights are halves too (P of
// them), and their products with steps once more: off by up to 2^-11 each, about
// what a result of 11 bits rounds away, and for 32-bit results of 16-bit queries as well.
template <int P, int G, int NT>
__global__ void __launch_bounds__(AttendShape<G, P, NT>::kThreads, AttendShape<G, P, NT>::kBlocks) k_attend(AttendArgs a) {
  using Shape = AttendShape<G, P, NT>;
  constexpr int kWarps = Shape::kWarps, kThreads = Shape::kThreads;
  constexpr int U = Shape::kUnits;
  constexpr float kEven = kCodesEven<P>, kOdd = kCodesOdd<P>;
  constexpr int kCols = Shape::kCols;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int64_t upto[kThreads + 1];
  __shared__ int64_t warp_sum[kWarps];
  __shared__ AttendCursor items[kWarps][2];  // each warp's, of its copies and of their use: seldom needed
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

  // steps of all requests: each thread adds up a run of them
  const int each = (a.n + kThreads - 1) / kThreads;
  const int r0 = min(a.n, (int)threadIdx.x * each), r1 = min(a.n, r0 + each);
  int64_t sum = 0;
  for (int r = r0; r < r1; ++r) sum += attend_units<kCols>(a, r, blockIdx.x == 0);
  int64_t x = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += o;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += warp_sum[w];
  upto[threadIdx.x + 1] = x;
  if (threadIdx.x == 0) upto[0] = 0;
  __syncthreads();
  const int64_t total = upto[kThreads];

  // neighbours in the row of steps are on different SMs
  const int64_t all = (int64_t)gridDim.x * kWarps, workers = min(all, total);
  const int64_t me = (int64_t)warp * gridDim.x + blockIdx.x;
  if (lane < 2) a.record[2 * me + lane] = make_int4(-1, 0, 0, 0);
  __syncwarp();
  if (me >= workers) return;
  const int64_t from = total * me / workers;
  const int count = (int)(total * (me + 1) / workers - from);  // places of this worker

  AttendCursor* const item_ahead = &items[warp][0];
  AttendCursor* const item = &items[warp][1];
  int place;          // of the step, in this worker's share
  int u, units;       // step of the item, of so many
  {
    AttendCursor use;
    int lo = 0, hi = kThreads;  // upto[lo] <= from < upto[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (upto[mid] <= from) lo = mid;
      else hi = mid;
    }
    int64_t rest = from - upto[lo];
    int r = lo * each;
    for (;; r += 32) {  // 32 requests at a time
      const int64_t mine = r + lane < a.n ? attend_units<kCols>(a, r + lane, false) : 0;
      int64_t s = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += o;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, s > rest);
      if (past || r + 32 >= a.n) {
        const int k = past ? __ffs(past) - 1 : 0;
        rest -= __shfl_sync(0xFFFFFFFFu, s - mine, k);
        r += k;
        break;
      }
      rest -= __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    use.r = min(r, a.n - 1);
    use.q = attend_mine(a, use.r, false);
    attend_sizes<kCols>(a, use);
    const int64_t before = rest / (use.units + kItemCost);
    units = use.units;
    u = (int)(rest - before * (use.units + kItemCost)) - kItemCost;
    place = max(0, -u);
    u = max(0, u);
    use.h = (int)(before / use.tiles);
    use.tile = (int)(before - (int64_t)use.h * use.tiles);
    if (lane < 2) items[warp][lane] = use;
    __syncwarp();
  }
  if (place >= count) return;  // the beginning of an item alone

  // in registers for good: a quadruple made anew costs four moves at each of its products
  uint32_t minus8[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("mov.b32 %0, %1;" : "=r"(minus8[i]) : "r"(i & 1 ? kMinus8Odd : kMinus8Even));
  // places in shared memory, from its first byte on
  const uint32_t smem_at = (uint32_t)__cvta_generic_to_shared(smem), ring = warp * Shape::kWarp;
  auto lds64 = [&](uint32_t at) { return *reinterpret_cast<const uint2*>(smem + at); };
  auto lds32 = [&](uint32_t at) { return *reinterpret_cast<const uint32_t*>(smem + at); };
  const uint32_t scores = ring + 2 * Shape::kStage, steps = scores + Shape::kScores;

  // ---- the copies of a step, one ahead of its use ----
  const int64_t values = (int64_t)a.heads * a.page_bytes;
  const uint64_t stride16 = (uint64_t)a.block_stride / 16;
  uint64_t head16 = 0;  // the head's first page in a block
  auto next_item = [&](AttendCursor* at) {
    AttendCursor c = *at;
    attend_next<kCols>(a, c);
    __syncwarp();
    if (lane == 0) *at = c;
    __syncwarp();
  };
  int ahead_place = place, ahead_u = u, ahead_units = units, ahead_len = item_ahead->q.len;
  head16 = (uint64_t)item_ahead->h * (uint64_t)(a.page_bytes / 16);
  int entry = 0;  // of the lane's token in the next step to copy
  auto look_up = [&] {
    const int t = ahead_u * kUnit + lane;
    entry = t < ahead_len ? __ldg(a.table + (int64_t)item_ahead->r * a.table_stride + a.block((uint32_t)t)) : -1;
  };
  // Goes on to the next step, if this worker has one.
  auto step_ahead = [&] {
    const bool last = ahead_u + 1 == ahead_units;
    ahead_place += last ? 1 + kItemCost : 1;
    if (ahead_place >= count) return;
    ++ahead_u;
    if (last) {
      next_item(item_ahead);
      ahead_u = 0;
      ahead_units = item_ahead->units;
      ahead_len = item_ahead->q.len;
      head16 = (uint64_t)item_ahead->h * (uint64_t)(a.page_bytes / 16);
    }
    look_up();
  };
  auto copy = [&](int stage) -> uint32_t {
    const int t = ahead_u * kUnit + lane;
    const bool there = (uint32_t)entry < (uint32_t)a.n_blocks && entry >= 0;
    if (!there && t < ahead_len) atomicOr(&a.small->op_status, kStBadInput);
    const uint32_t row = (uint32_t)t - a.block((uint32_t)t) * a.block.d;
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, there);
    const uint32_t to = smem_at + ring + stage * Shape::kStage;
    // Addresses are counted in 16 bytes from the cache's first, in 32 bits where it is below 64 GB.
    auto get = [&](auto type, auto whole_tag) {
      using T = decltype(type);
      constexpr bool kWhole = decltype(whole_tag)::value;
      constexpr bool kSteady = G != 3 && G != 6;  // a lane has the same chunk of rows 32 / G apart
      const T head = (T)(there ? entry : 0) * (T)stride16 + (T)head16, codes = head + (T)row * G;
      const unsigned char* pairs = a.cache + (uint64_t)head * 16 + (a.block.d * 4 + row) * (uint32_t)Shape::kPair;
      const uint32_t d0 = to + (lane / G) * Shape::kRow + (attend_piece<G>(lane / G, lane % G >> 1) * 2 + (lane % G & 1)) * 16;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int at = i * 32 + lane, src = at / G, chunk = at % G;
        const uint64_t from = __shfl_sync(0xFFFFFFFFu, codes, src);
        const bool ok = kWhole || (all >> src & 1);
        const unsigned char* p = a.cache + chunk * 16 + from * 16;
        const unsigned char* v = a.cache + values + chunk * 16 + from * 16;
        const uint32_t d = kSteady ? d0 + i * (32 / G) * Shape::kRow
                                   : to + src * Shape::kRow + (attend_piece<G>(src, chunk >> 1) * 2 + (chunk & 1)) * 16;
        copy_async<16, kWhole>(d, ok ? p : a.cache, ok);
        copy_async<16, kWhole>(d + Shape::kHalfStage, ok ? v : a.cache, ok);
      }
      const bool ok = kWhole || there;
      constexpr int kPiece = G % 4 == 0 ? 16 : G % 2 == 0 ? 8 : 4;
#pragma unroll
      for (int i = 0; i < Shape::kPair / kPiece; ++i) {
        const uint32_t d = to + kUnit * Shape::kRow + lane * Shape::kPair + i * kPiece;
        copy_async<kPiece, kWhole>(d, ok ? pairs + i * kPiece : a.cache, ok);
        copy_async<kPiece, kWhole>(d + Shape::kHalfStage, ok ? pairs + values + i * kPiece : a.cache, ok);
      }
    };
    if (all == 0xFFFFFFFFu && a.near) get(uint32_t{}, std::true_type{});
    else get(uint64_t{}, std::false_type{});
    asm volatile("cp.async.commit_group;" ::: "memory");
    return all;
  };

  // ---- an item's state ----
  uint32_t q_kept[NT][G][P][4];  // unless in shared memory
  const uint32_t queries = steps + (1 + P) * Shape::kSteps + lane * 16;
  uint32_t qbase[NT][Shape::kBaseMmas][2];  // sums of a group's query elements, in three parts of bfloat16
  float to_score[NT];     // of column g: what makes a score of its products
  float acc[NT][2 * G][4];
  float mid[NT][4];       // of group g (and nothing), columns 2 c and 2 c + 1
  float top[NT], total_p[NT];  // of column g; the weights of this thread's tokens
  int sees[NT];           // tokens that column g sees
  int cap, low;           // of sizes of values: what all are below, and the smallest that this lane met (zeros aside)
  bool whole = false;     // the item begins with this worker's first step of it
  // the pairs of groups whose bases this thread has in the products of bases
  auto base_unit = [&](int m, int half) { return (m * 8 + half * 4 + c) % U; };

  auto begin = [&] {
    const AttendCursor use = *item;
    cap = kLeastCap;
    low = kNoLow;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = use.tile * kCols + 8 * n + g;
      const bool real = col < use.q.fresh * (int)a.group.d;
      const int token = (int)a.group((uint32_t)col), head = use.h * (int)a.group.d + col - token * (int)a.group.d;
      const int64_t row = (int64_t)(use.q.first + token) * a.q_token + head * a.q_head;
      // columns without a token ask for no masks
      sees[n] = real ? use.q.len - use.q.fresh + token + 1 : INT32_MAX;
      top[n] = -INFINITY;
      total_p[n] = 0.f;
      float e[G][8], most = 0.f;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int at = 32 * j + 8 * c;
        auto get = [&](auto type) {
          using T = decltype(type);
          const T* from = static_cast<const T*>(a.queries) + row;
          if (real && a.q_wide && at < a.dim) {
            Vec<T, 8> v;
            v.template load<true>(from + at);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[j][i] = to_f32(v.x[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[j][i] = real && at + i < a.dim ? to_f32(from[at + i]) : 0.f;
          }
        };
        if (P == 2) get(float{});
        else if (a.q_type == BPE_F16) get(__half{});
        else get(__nv_bfloat16{});
#pragma unroll
        for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(e[j][i]));
      }
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      // the largest element in [2^14, 2^15): elements down to 2^-28 of it are normal halves
      const int by = min(14 - ((__float_as_int(most) >> 23) - 127), 126);
      const float scale = power_of_2(max(by, -113));
      to_score[n] = a.scale * kEven / scale;
      float sum[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[j][i] *= scale;
          s += e[j][i];
        }
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
        sum[j] = s * (1.f / kEven);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = i & 1 ? kOdd / kEven : 1.f;
          uint32_t part[P];
          split_halves<P>(e[j][i] * f, e[j][i + 4] * f, part);
#pragma unroll
          for (int p = 0; p < P; ++p) q_kept[n][j][p][i] = part[p];
        }
        if (Shape::kQueriesShared)
          *reinterpret_cast<uint4*>(smem + queries + (n * G + j) * 512) =
              make_uint4(q_kept[n][j][0][0], q_kept[n][j][0][1], q_kept[n][j][0][2], q_kept[n][j][0][3]);
      }
      // the products of bases: part s / U of the sums of groups 2 (s % U) and the next, in place s
#pragma unroll
      for (int m = 0; m < Shape::kBaseMmas; ++m) qbase[n][m][0] = qbase[n][m][1] = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x = sum[2 * u], y = 2 * u + 1 < G ? sum[(2 * u + 1) % G] : 0.f;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const int s = p * U + u;
          uint32_t w;
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y), "f"(x));
          x -= bf16_low(w);
          y -= bf16_high(w);
          if (c == s % 4) qbase[n][s / 8][s / 4 % 2] = w;
        }
      }
#pragma unroll
      for (int j = 0; j < 2 * G; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][j][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) mid[n][i] = 0.f;
    }
  };

  // ---- a step ----
  // Its values are added up by themselves and then to those before it: the tensor
  // cores cut sums off where an addition rounds them, so that a long row of
  // weights above zero would lose a little at each of its products (f32, 700
  // tokens: 9e-6 of the result).
  auto step = [&](uint32_t at, uint32_t there, auto partial_tag) {
    constexpr bool kPartial = decltype(partial_tag)::value;
    constexpr bool kOddGroups = G % 2 == 1;
    const uint32_t key_pairs = at + kUnit * Shape::kRow;
    float s[NT][2][4];  // scores: of tokens g and g + 8 of each half of the step, columns 2 c and 2 c + 1
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const uint32_t k0 = tile * 16 + g, k1 = k0 + 8;
#pragma unroll
      for (int m = 0; m < Shape::kBaseMmas; ++m) {
        uint32_t b[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half == 1 && 4 % U == 0) {  // the same pair of groups again
            b[2] = b[0];
            b[3] = b[1];
            break;
          }
          const int u = base_unit(m, half);
          if (!kOddGroups) {
            const uint2 x = lds64(key_pairs + k0 * Shape::kPair + u * 8), y = lds64(key_pairs + k1 * Shape::kPair + u * 8);
            b[2 * half] = __byte_perm(x.x, x.y, 0x7632);
            b[2 * half + 1] = __byte_perm(y.x, y.y, 0x7632);
          } else {
            const uint32_t x = lds32(key_pairs + k0 * Shape::kPair + u * 8);
            const uint32_t y = lds32(key_pairs + k1 * Shape::kPair + u * 8);
            uint32_t x2 = 0, y2 = 0;
            if (u + 1 < U) {
              x2 = lds32(key_pairs + k0 * Shape::kPair + u * 8 + 4);
              y2 = lds32(key_pairs + k1 * Shape::kPair + u * 8 + 4);
            }
            b[2 * half] = __byte_perm(x, x2, 0x7632);
            b[2 * half + 1] = __byte_perm(y, y2, 0x7632);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (m == 0) mma_bf16_first(s[n][tile], b, qbase[n][m][0], qbase[n][m][1]);
          else mma_bf16(s[n][tile], b, qbase[n][m][0], qbase[n][m][1]);
        }
      }
    }
    // The step's two halves side by side, with the query's words of one group at a time. One half after the
    // other took 422 us for 384 requests of 128 elements (so 417) and 146 for 16 query heads a head (so 143).
#pragma unroll
    for (int two = 0; two < U; ++two) {
      const bool pair = !kOddGroups || two < G / 2;
      uint2 w[2][2] = {}, p[2][2] = {};
#pragma unroll
      for (int tile = 0; tile < 2; ++tile)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t k = tile * 16 + g + 8 * i;
          if (pair) w[tile][i] = lds64(at + k * Shape::kRow + attend_piece<G>(k, two) * 32 + c * 8);
          else w[tile][i].x = lds32(at + k * Shape::kRow + two * 32 + c * 4);
          if (!kOddGroups) {
            p[tile][i] = lds64(key_pairs + k * Shape::kPair + two * 8);
          } else {
            p[tile][i].x = lds32(key_pairs + k * Shape::kPair + two * 8);
            if (pair) p[tile][i].y = lds32(key_pairs + k * Shape::kPair + two * 8 + 4);
          }
        }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int j = 2 * two + half;
        if (j >= G) break;
        uint32_t q[NT][P][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (Shape::kQueriesShared) {
            const uint4 x = *reinterpret_cast<const uint4*>(smem + queries + (n * G + j) * 512);
            q[n][0][0] = x.x, q[n][0][1] = x.y, q[n][0][2] = x.z, q[n][0][3] = x.w;
          } else {
#pragma unroll
            for (int k = 0; k < P; ++k)
#pragma unroll
              for (int i = 0; i < 4; ++i) q[n][k][i] = q_kept[n][j][k][i];
          }
        }
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          const uint32_t x0 = half ? w[tile][0].y : w[tile][0].x, x1 = half ? w[tile][1].y : w[tile][1].x;
          const uint32_t z0 = x0 >> 8, z1 = x1 >> 8;
          const float s0 = bf16_low(half ? p[tile][0].y : p[tile][0].x), s1 = bf16_low(half ? p[tile][1].y : p[tile][1].x);
          const uint32_t lo[4] = {codes_even<P, 0>(x0), codes_even<P, 0>(x1), codes_odd<P, 0>(x0), codes_odd<P, 0>(x1)};
          const uint32_t hi[4] = {codes_even<P, 0>(z0), codes_even<P, 0>(z1), codes_odd<P, 0>(z0), codes_odd<P, 0>(z1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float d[4];
            mma_f16_first(d, lo, q[n][P - 1][0], q[n][P - 1][1]);
            mma_f16(d, hi, q[n][P - 1][2], q[n][P - 1][3]);
            if (P == 2) {  // leading parts by themselves
              float d0[4], d1[4];
              mma_f16_first(d0, lo, q[n][0][0], q[n][0][1]);
              mma_f16_first(d1, hi, q[n][0][2], q[n][0][3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) d[i] += d0[i] + d1[i];
            }
            s[n][tile][0] += s0 * d[0];
            s[n][tile][1] += s0 * d[1];
            s[n][tile][2] += s1 * d[2];
            s[n][tile][3] += s1 * d[3];
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
        const uint32_t to = scores + n * (kUnit * 32) + c * 8 + (tile * 16 + g) * 32;
        *reinterpret_cast<float2*>(smem + to) = make_float2(s[n][tile][0], s[n][tile][1]);
        *reinterpret_cast<float2*>(smem + to + 8 * 32) = make_float2(s[n][tile][2], s[n][tile][3]);
      }
    // the pairs of values of token `lane`, meanwhile
    const uint32_t codes = at + Shape::kHalfStage, value_pairs = codes + kUnit * Shape::kRow + lane * Shape::kPair;
    uint32_t z[G];
    if (!kOddGroups) {
#pragma unroll
      for (int u = 0; u < G / 2; ++u) {
        const uint2 x = lds64(value_pairs + u * 8);
        z[2 * u] = x.x;
        z[(2 * u + 1) % G] = x.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < G; ++j) z[j] = lds32(value_pairs + j * 4);
    }
    // the largest and the smallest size of what they stand for, but of groups behind the row's end
    auto size_of = [](uint32_t pair) { return __float_as_int(fabsf(bf16_high(pair)) + 16.f * bf16_low(pair)); };
    const bool padded = G > 4 && a.dim <= 32 * (G - 1);
    int largest = 0, smallest = kNoLow;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (j == G - 1 && padded) break;
      const int size = size_of(z[j]);
      largest = max(largest, size);
      smallest = min(smallest, size);
    }
    // Whether the sizes lie where this worker's do. Tokens that no column sees do not count.
    uint32_t all = 0xFFFFFFFFu;
    if (kPartial) {
      int furthest = 0;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (sees[n] != INT32_MAX) furthest = max(furthest, sees[n]);
      const int k = __reduce_max_sync(0xFFFFFFFFu, furthest) - u * kUnit;
      all = there & (k >= kUnit ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << k) - 1u);
    }
    const bool mine = !kPartial || (all >> lane & 1);
    constexpr int kSpan = (kApart<P> + 1) << 23;
    const bool odd = mine && (largest >= cap || smallest < cap - kSpan);
    __syncwarp();
    // from here on a thread has column g and tokens c, c + 4, .. of the step
    float p[NT][8];
    uint32_t seen[NT];
    bool grows = false;
    float most[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      seen[n] = 0;
      float m = top[n];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[n][i] = to_score[n] * __uint_as_float(lds32(scores + n * (kUnit * 32) + (c + 4 * i) * 32 + g * 4));
        if (kPartial) {
          const bool see = u * kUnit + c + 4 * i < sees[n] && (there >> (c + 4 * i) & 1);
          if (see) seen[n] |= 1u << i;
          else p[n][i] = -INFINITY;
        }
        m = fmaxf(m, p[n][i]);
      }
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      most[n] = m;
      grows |= m > top[n];
    }
    bool close = true;
    if (__any_sync(0xFFFFFFFFu, grows || odd)) {
      if (__any_sync(0xFFFFFFFFu, odd)) {
        // seldom: the same without zeros and what is no number, which spoils its own group in any unit
        largest = 0, smallest = kNoLow;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const int size = size_of(z[j]);
          if (!mine || (j == G - 1 && padded) || (uint32_t)size - 1u >= 0x7F7FFFFFu) continue;
          largest = max(largest, size);
          smallest = min(smallest, size);
        }
        const int most_here = (int)(__reduce_max_sync(0xFFFFFFFFu, (uint32_t)largest) >> 23) + 1 << 23;
        const int least_met = (int)__reduce_min_sync(0xFFFFFFFFu, (uint32_t)low);
        const int least = min(least_met, (int)__reduce_min_sync(0xFFFFFFFFu, (uint32_t)smallest));
        // (a cap that no halves have gone by may fall, but not so far that sums pass the largest float)
        int then = max(most_here, least_met == kNoLow && cap - most_here <= kFarApart ? kLeastCap : cap);
        close = least >= then - kSpan;
        if (!close) then = most_here - cap > kFarApart ? most_here : cap;
        if (then != cap) {
          const int by = (cap - then) >> 23;
          const float f = by < -126 ? 0.f : power_of_2(by);
          cap = then;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 2 * G; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[n][j][i] *= f;
            mid[n][0] *= f;
            mid[n][1] *= f;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float f = most[n] > top[n] ? exp2_fast(top[n] - most[n]) : 1.f;
        top[n] = most[n];
        total_p[n] *= f;
        const float f0 = __shfl_sync(0xFFFFFFFFu, f, 8 * c), f1 = __shfl_sync(0xFFFFFFFFu, f, 8 * c + 4);
        mid[n][0] *= f0;
        mid[n][1] *= f1;
#pragma unroll
        for (int j = 0; j < 2 * G; ++j) {
          acc[n][j][0] *= f0;
          acc[n][j][1] *= f1;
          acc[n][j][2] *= f0;
          acc[n][j][3] *= f1;
        }
      }
    }
    // weights of at most 2^11: those down to 2^-25 of the largest are normal halves
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float m = (top[n] == -INFINITY ? 0.f : top[n]) - 11.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[n][i] = exp2_fast(p[n][i] - m);
        total_p[n] += p[n][i];
      }
    }

    uint32_t ph[NT][P][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t part[P];
        split_halves<P>(p[n][2 * i], p[n][2 * i + 1], part);
#pragma unroll
        for (int k = 0; k < P; ++k) ph[n][k][i] = part[k];
      }
    }
    if (!close) {
      // in 32 bits, a token after another: no size matters to another
      // weights where the scores are, those of columns that do not see a token below zero
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m = (top[n] == -INFINITY ? 0.f : top[n]) - 11.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float* const at = reinterpret_cast<float*>(smem + scores + n * (kUnit * 32) + (c + 4 * i) * 32 + g * 4);
          *at = kPartial && !(seen[n] >> i & 1) ? -1.f : exp2_fast(to_score[n] * *at - m);
        }
      }
      __syncwarp();
      const float unit = per_unit(cap);
      const uint32_t pairs = codes + kUnit * Shape::kRow;
#pragma unroll 1
      for (int t = 0; t < kUnit; ++t) {
        if (kPartial && !(all >> t & 1)) continue;
        float2 weight[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          weight[n] = *reinterpret_cast<const float2*>(smem + scores + n * (kUnit * 32) + t * 32 + c * 8);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const bool paired = !kOddGroups || j < G - 1;
          const uint32_t row = codes + t * Shape::kRow + (paired ? attend_piece<G>(t, j / 2) * 32 + (g >> 1) * 8 + (j & 1) * 4
                                                                 : j * 16 + (g >> 1) * 4);
          const uint32_t word = lds32(row) >> (g & 1) * 16, pair = lds32(pairs + t * Shape::kPair + j * 4);
          const float st = bf16_low(pair) * unit, ba = bf16_high(pair) * unit;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float code = __uint_as_float((word >> 4 * i & 15u) | 0x4B000000u) - 0x1p23f;
            const float value = fmaf(st, code, ba) * (i & 1 ? 1.f / kOdd : 1.f / kEven);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float* const to = acc[n][2 * j + i / 2] + (i & 1) * 2;
              if (!(weight[n].x < 0.f)) to[0] = fmaf(weight[n].x, value, to[0]);
              if (!(weight[n].y < 0.f)) to[1] = fmaf(weight[n].y, value, to[1]);
            }
          }
        }
      }
      return;
    }
    if (mine) low = min(low, smallest);
    {
      const float unit = per_unit(cap), middle = P == 2 || a.centre ? 8.f : 0.f;
      // in the order of a thread's tokens: c, c + 4, c + 8, c + 12 of each half of the step are neighbours
      const uint32_t place = ((lane & 16) | (lane & 3) << 2 | (lane >> 2 & 3)) * 2;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const float st = bf16_low(z[j]), ba = bf16_high(z[j]);
        float m = (ba + middle * st) * unit, w = st * unit;
        if (kPartial) {
          // what is no number comes in with the steps, by the weights of those that see it
          const bool good = mine && fabsf(ba) + 16.f * st < INFINITY;
          m = good ? m : 0.f;
          w = good ? w : mine ? NAN : 0.f;
        }
        const uint32_t to = steps + j * (kUnit * 2) + place;
        const __half wh = __float2half_rn(w), mh = __float2half_rn(m);
        *reinterpret_cast<__half*>(smem + to) = wh;
        *reinterpret_cast<__half*>(smem + to + Shape::kSteps) = mh;
        if (P == 2) {
          const __half ml = __float2half_rn(m - __half2float(mh));
          *reinterpret_cast<__half*>(smem + to + 2 * Shape::kSteps) = ml;
        }
      }
      __syncwarp();
      float om[NT][4];
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
        const uint32_t row = steps + Shape::kSteps + (G < 8 ? min(g, G - 1) : g) * (kUnit * 2) + tile * 32 + c * 8;
        const uint2 x = lds64(row);
        const uint32_t lead[4] = {x.x, 0u, x.y, 0u};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < P; ++k) {
            if (tile == 0 && k == 0) mma_f16_first(om[n], lead, ph[n][k][2 * tile], ph[n][k][2 * tile + 1]);
            else mma_f16(om[n], lead, ph[n][k][2 * tile], ph[n][k][2 * tile + 1]);
          }
        if (P == 2) {
          const uint2 y = lds64(row + Shape::kSteps);
          const uint32_t rest[4] = {y.x, 0u, y.y, 0u};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(om[n], rest, ph[n][0][2 * tile], ph[n][0][2 * tile + 1]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mid[n][0] += om[n][0];
        mid[n][1] += om[n][1];
      }
      const uint32_t select = g & 1 ? 0x7632 : 0x5410;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float o[NT][4][4];
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          const bool pair = !kOddGroups || u < G / 2;
          uint2 w[4] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t t = tile * 16 + c + 4 * i;
            if (pair) w[i] = lds64(codes + t * Shape::kRow + attend_piece<G>(t, u) * 32 + (g >> 1) * 8);
            else w[i].x = lds32(codes + t * Shape::kRow + u * 32 + (g >> 1) * 4);
          }
          uint32_t b0[NT][2][P], b1[NT][2][P];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int j = 2 * u + half;
            if (j >= G) break;
            const uint2 st = lds64(steps + j * (kUnit * 2) + tile * 32 + c * 8);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (P == 1) {
                const __half2 w0 = __hmul2(*reinterpret_cast<const __half2*>(&ph[n][0][2 * tile]),
                                           *reinterpret_cast<const __half2*>(&st.x));
                const __half2 w1 = __hmul2(*reinterpret_cast<const __half2*>(&ph[n][0][2 * tile + 1]),
                                           *reinterpret_cast<const __half2*>(&st.y));
                b0[n][half][0] = *reinterpret_cast<const uint32_t*>(&w0);
                b1[n][half][0] = *reinterpret_cast<const uint32_t*>(&w1);
              } else {
                const float2 s0 = unpack_halves(st.x), s1 = unpack_halves(st.y);
                split_halves<P>(p[n][4 * tile] * s0.x, p[n][4 * tile + 1] * s0.y, b0[n][half]);
                split_halves<P>(p[n][4 * tile + 2] * s1.x, p[n][4 * tile + 3] * s1.y, b1[n][half]);
              }
              if (kPartial) {  // whatever the steps of tokens are that a column does not see
                const uint32_t bits = seen[n] >> (4 * tile);
                const uint32_t m0 = (bits & 1 ? 0xFFFFu : 0u) | (bits & 2 ? 0xFFFF0000u : 0u);
                const uint32_t m1 = (bits & 4 ? 0xFFFFu : 0u) | (bits & 8 ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                  b0[n][half][k] &= m0;
                  b1[n][half][k] &= m1;
                }
              }
            }
            const uint32_t x0 = __byte_perm(half ? w[0].y : w[0].x, half ? w[1].y : w[1].x, select);
            const uint32_t x1 = __byte_perm(half ? w[2].y : w[2].x, half ? w[3].y : w[3].x, select);
            const uint32_t z0 = x0 >> 8, z1 = x1 >> 8;
            const uint32_t lo[4] = {codes_even<P, 8>(x0), codes_odd<P, 8>(x0), codes_even<P, 8>(x1), codes_odd<P, 8>(x1)};
            const uint32_t hi[4] = {codes_even<P, 8>(z0), codes_odd<P, 8>(z0), codes_even<P, 8>(z1), codes_odd<P, 8>(z1)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              auto add = [&](float (&d)[4], const uint32_t (&codes)[4], int k) {
                if (tile == 0) mma_f16_first(d, codes, b0[n][half][k], b1[n][half][k]);
                else mma_f16(d, codes, b0[n][half][k], b1[n][half][k]);
              };
              add(o[n][2 * half], lo, P - 1);
              add(o[n][2 * half + 1], hi, P - 1);
              if (P == 2) {  // leading parts by themselves
                float lead[2][4];
                mma_f16_first(lead[0], lo, b0[n][half][0], b1[n][half][0]);
                mma_f16_first(lead[1], hi, b0[n][half][0], b1[n][half][0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  o[n][2 * half][i] += lead[0][i];
                  o[n][2 * half + 1][i] += lead[1][i];
                }
              }
            }
          }
          if (P == 1 && a.centre) {  // n to n - 8
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (4 * u + i < 2 * G) mma_f16(o[n][i], minus8, b0[n][i / 2][0], b1[n][i / 2][0]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (4 * u + i < 2 * G) acc[n][4 * u + i][e] += o[n][i][e];
      }
    }
  };

  // ---- an item's end, or the end of this worker's share of it ----
  auto finish = [&](bool last) {
    const AttendCursor use = *item;
    const bool done = whole && last;
    float* part = a.partial + (2 * me + (whole ? 1 : 0)) * Shape::kPartial;
    const float unit = unit_of(cap);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float l = total_p[n];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
      if (!done && c == 0) {
        part[kCols * 32 * G + 8 * n + g] = top[n];
        part[kCols * (32 * G + 1) + 8 * n + g] = l;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sum_p = __shfl_sync(0xFFFFFFFFu, l, 8 * c + 4 * e);
        const float by = sum_p == 0.f ? 0.f : unit / sum_p;
        const int col = use.tile * kCols + 8 * n + 2 * c + e;
        const bool real = col < use.q.fresh * (int)a.group.d;
        const int token = (int)a.group((uint32_t)col), head = use.h * (int)a.group.d + col - token * (int)a.group.d;
        const int64_t row = (int64_t)(use.q.first + token) * a.o_token + head * a.o_head;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float m = __shfl_sync(0xFFFFFFFFu, mid[n][e], 4 * j + c);
          float4 r = make_float4(acc[n][2 * j][e] * kEven + m, acc[n][2 * j][2 + e] * kOdd + m,
                                 acc[n][2 * j + 1][e] * kEven + m, acc[n][2 * j + 1][2 + e] * kOdd + m);
          r.x *= by, r.y *= by, r.z *= by, r.w *= by;  // partial sums too, which large values would take past a float
          if (!done) *reinterpret_cast<float4*>(part + (8 * n + 2 * c + e) * 32 * G + 32 * j + 4 * g) = r;
          else if (real) attend_store(a, row, 32 * j + 4 * g, r);
        }
      }
    }
    if (!done && lane == 0) {
      // the workers among which the item's steps lie
      const int64_t total = upto[kThreads], workers = min((int64_t)gridDim.x * kWarps, total);
      const int64_t i0 = total * me / workers + place - u, i1 = i0 + use.units - 1;
      a.record[2 * me + (whole ? 1 : 0)] =
          make_int4((int)(((i0 + 1) * workers - 1) / total), (int)(((i1 + 1) * workers - 1) / total), use.r,
                    use.h * use.tiles + use.tile);
    }
  };
  look_up();
  uint32_t there = copy(0), there_next = 0;
  step_ahead();
  begin();
  whole = u == 0;
  for (int stage = 0;; stage ^= 1) {
    const bool more = ahead_place < count;
    if (more) {
      there_next = copy(stage ^ 1);
      step_ahead();
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    bool part = there != 0xFFFFFFFFu;
#pragma unroll
    for (int n = 0; n < NT; ++n) part |= sees[n] < (u + 1) * kUnit;
    if (__any_sync(0xFFFFFFFFu, part)) step(ring + stage * Shape::kStage, there, std::true_type{});
    else step(ring + stage * Shape::kStage, there, std::false_type{});
    __syncwarp();  // before the stage is filled again
    there = there_next;
    const bool last = u + 1 == units;
    if (last || !more) finish(last);
    if (!more) return;
    ++place;
    ++u;
    if (last) {
      place += kItemCost;
      next_item(item);
      u = 0;
      units = item->units;
      begin();
      whole = true;
    }
  }
}

// Adds up what several workers' shares have of an item (the mean of the values by
// its weights, their sum and maximum), in the order of the shares or by a fixed
// tree. Block b looks at the border between workers b and b + 1; of an item that
// spans k borders each of their blocks takes columns. With few parts a thread
// reads all parts of its four elements; with many, parts are spread over the
// threads, their factors first.
constexpr int kJoinThreads = 256;
constexpr int kJoinFew = 8;
constexpr float kJoinUnit = 0x1p-44f;  // all weights of 2^31 tokens add up to less than 1
template <int G, int NT>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(AttendArgs a) {
  using Shape = AttendShape<G, 1, NT>;
  constexpr int kCols = Shape::kCols, kVecs = 8 * G;  // vectors of 4 of a column
  constexpr int kTop = kCols * 32 * G, kTotal = kTop + kCols;
  await_previous();
  const int64_t b = blockIdx.x + 1;
  const int4 rec = a.record[2 * b];
  if (rec.x < 0) return;
  const int w0 = rec.x, w1 = rec.y, parts = w1 - w0 + 1;
  AttendCursor cur;
  cur.q = attend_mine(a, rec.z, false);
  attend_sizes<kCols>(a, cur);
  const int h = rec.w / cur.tiles, tile = rec.w - h * cur.tiles, group = (int)a.group.d;
  const int cols = min(kCols, cur.q.fresh * group - tile * kCols);
  // this block's columns
  const int first = (int)b - w0 - 1, step = w1 - w0, tid = threadIdx.x;
  auto part = [&](int k) { return a.partial + (2 * (int64_t)(w0 + k) + (k == 0 ? 1 : 0)) * Shape::kPartial; };
  auto put = [&](int col, int vec, float4 sum, float total) {
    const float by = total == 0.f ? 0.f : 1.f / total;
    sum.x *= by, sum.y *= by, sum.z *= by, sum.w *= by;
    const int at = tile * kCols + col, token = at / group, head = h * group + at - token * group;
    attend_store(a, (int64_t)(cur.q.first + token) * a.o_token + head * a.o_head, 4 * vec, sum);
  };
  auto add = [](float4& sum, float f, const float* from) {
    const float4 v = *reinterpret_cast<const float4*>(from);
    sum.x += f * v.x, sum.y += f * v.y, sum.z += f * v.z, sum.w += f * v.w;
  };
  if (parts <= kJoinFew) {
    const int mine = (cols - first + step - 1) / step;  // none where first >= cols
    for (int i = tid; i < mine * kVecs; i += kJoinThreads) {
      const int col = first + i / kVecs * step, vec = i % kVecs;
      float top[kJoinFew], m = -INFINITY, total = 0.f;
#pragma unroll
      for (int k = 0; k < kJoinFew; ++k) {
        top[k] = k < parts ? part(k)[kTop + col] : -INFINITY;
        m = fmaxf(m, top[k]);
      }
      if (m == -INFINITY) m = 0.f;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kJoinFew; ++k) {
        if (k >= parts) break;
        const float f = exp2_fast(top[k] - m) * (part(k)[kTotal + col] * kJoinUnit);
        total += f;
        add(sum, f, part(k) + col * 32 * G + 4 * vec);
      }
      put(col, vec, sum, total);
    }
    return;
  }
  constexpr int kSlices = kJoinThreads / kVecs, kRound = 512;  // parts whose factors are held at once
  __shared__ float factor[kRound];
  __shared__ float of_warp[kJoinThreads / 32];
  __shared__ float4 sums[kJoinThreads];
  const int slice = tid / kVecs, vec = tid % kVecs;
  auto all_of = [&](float x, auto join) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = join(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    __syncthreads();  // of_warp and sums may still be read
    if (tid % 32 == 0) of_warp[tid / 32] = x;
    __syncthreads();
    x = of_warp[0];
#pragma unroll
    for (int w = 1; w < kJoinThreads / 32; ++w) x = join(x, of_warp[w]);
    return x;
  };
  for (int col = first; col < cols; col += step) {
    float m = -INFINITY;
    for (int k = tid; k < parts; k += kJoinThreads) m = fmaxf(m, part(k)[kTop + col]);
    m = all_of(m, [](float x, float y) { return fmaxf(x, y); });
    if (m == -INFINITY) m = 0.f;
    float total = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += kRound) {
      if (k0) __syncthreads();  // factors may still be read
      for (int k = k0 + tid; k < min(parts, k0 + kRound); k += kJoinThreads) {
        const float f = exp2_fast(part(k)[kTop + col] - m) * (part(k)[kTotal + col] * kJoinUnit);
        factor[k - k0] = f;
        total += f;
      }
      __syncthreads();
      if (slice < kSlices) {
        const int end = min(parts, k0 + kRound);
#pragma unroll 8
        for (int k = k0 + slice; k < end; k += kSlices) add(sum, factor[k - k0], part(k) + col * 32 * G + 4 * vec);
      }
    }
    total = all_of(total, [](float x, float y) { return x + y; });
    sums[tid] = sum;
    __syncthreads();
    if (slice == 0) {
#pragma unroll
      for (int s = 1; s < kSlices; ++s) {
        const float4 v = sums[vec + s * kVecs];
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      }
      put(col, vec, sum, total);
    }
  }
}

}  // namespace
