// Attention of new tokens over a paged cache in 4 bits (cache.cuh).
//
// Included once by attend.cu; not a standalone header.
//
//   s_t = scale * (query . key_t),  out = sum_t e^(s_t - m) value_t / sum_t e^(s_t - m)
//
// over the tokens t that the query sees, in one pass with the running maximum m.
// With the codes n, the steps S and bases B of group j,
//   query . key_t = sum_j 16 S_tj (sum_i q_i (1 + n_ti / 16)) + (B_tj - 16 S_tj) (sum_i q_i)
//   out_i = sum_t (p_t 16 S_tj) (1 + n_ti / 16) + sum_t p_t (B_tj - 16 S_tj)
// The sums over i and t in which codes take part run on the tensor cores:
// 1 + n / 16 is a code with an exponent put before it, exact in 16 bits and made
// by a shift and one logical operation for two codes; steps and bases stay
// outside, in 32 bits.

namespace {

constexpr int kAttWarps = 8;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kUnit = 32;  // tokens of a step

struct AttendArgs {
  const void* queries;
  void* out;
  int out_type;
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
  float* partial;
  int4* record;
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

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 1 + n / 16 of the codes at bits 4 e and 16 + 4 e of a word, as two 16-bit floats.
template <bool kHalf>
__device__ __forceinline__ uint32_t codes_to_floats(uint32_t w, int e) {
  if (kHalf) return ((e == 0 ? w << 6 : e == 1 ? w << 2 : e == 2 ? w >> 2 : w >> 6) & 0x03C003C0u) | 0x3C003C00u;
  return ((e == 0 ? w << 3 : w >> (4 * e - 3)) & 0x00780078u) | 0x3F803F80u;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool there) {
  const int size = there ? kBytes : 0;  // else zeros
  if (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(size) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(kBytes), "r"(size) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Cuts x into kParts bfloat16 numbers that add up to it (to 2^-9 of the last):
// the leading ones by cutting bits off, the last rounded.
template <int kParts>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&part)[kParts]) {
#pragma unroll
  for (int p = 0; p + 1 < kParts; ++p) {
    part[p] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    x -= __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    y -= __uint_as_float(__float_as_uint(y) & 0xFFFF0000u);
  }
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(part[kParts - 1]) : "f"(y), "f"(x));
}

// Where the tokens of all requests are cut. A request with new tokens has
// heads x tiles items (a tile: 8 NT columns, a column a query head of a new
// token), each of its tokens in steps of kUnit (one at least, so that every row
// is written). The steps of all items in a row are dealt out evenly.
struct AttendCursor {
  int r, h, tile, u;          // request, head, tile, step
  int tiles, units;
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
  c.q = attend_request(a, r, report);
  attend_sizes<kCols>(a, c);
  return (int64_t)c.units * c.tiles * a.heads;
}

template <int kCols>
__device__ __forceinline__ void attend_next(const AttendArgs& a, AttendCursor& c) {
  if (++c.u < c.units) return;
  c.u = 0;
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.h < a.heads) return;
  c.h = 0;
  do {
    ++c.r;
    c.q.fresh = 0;
    if (c.r < a.n) c.q = attend_request(a, c.r, false);
  } while (c.q.fresh == 0 && c.r < a.n);
  attend_sizes<kCols>(a, c);
}

template <int G, int kParts, int NT>
struct AttendShape {
  static constexpr int kCols = 8 * NT;
  static constexpr int kRow = 16 * G, kPair = 4 * G;                 // bytes of a row's codes, of its pairs
  static constexpr int kHalfStage = kUnit * (kRow + kPair);          // keys, or values
  static constexpr int kStage = 2 * kHalfStage;
  static constexpr int kScores = NT * kUnit * 8 * 4;
  static constexpr int kWarp = 2 * kStage + kScores;
  static constexpr int kSmem = kAttWarps * kWarp;
  static constexpr int kPartial = kCols * (32 * G + 2);              // floats of an item's partial sums
};

// Rows of 64 and of 128 bytes lie on two and on one set of banks: their 32-byte
// pieces are exchanged, so that the eight-byte loads of four rows meet no other.
template <int G>
__device__ __forceinline__ uint32_t attend_piece(int row, int piece) {
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
template <class TQ, int G, int NT>
__global__ void __launch_bounds__(kAttThreads, (G <= 4 && NT == 1 && sizeof(TQ) == 2) ? 2 : 1) k_attend(AttendArgs a) {
  constexpr bool kHalf = std::is_same<TQ, __half>::value;
  constexpr int QP = sizeof(TQ) == 4 ? 3 : 1;  // parts of a query
  constexpr int PP = sizeof(TQ) == 4 ? 3 : 2;  // parts of a weight
  using Shape = AttendShape<G, QP, NT>;
  constexpr int kCols = Shape::kCols;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int64_t upto[kAttThreads + 1];
  __shared__ int64_t warp_sum[kAttWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

  // steps of all requests: each thread adds up a run of them
  const int each = (a.n + kAttThreads - 1) / kAttThreads;
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
  const int64_t total = upto[kAttThreads];

  // neighbours in the row of steps are on different SMs
  const int64_t all = (int64_t)gridDim.x * kAttWarps, workers = min(all, total);
  const int64_t me = (int64_t)warp * gridDim.x + blockIdx.x;
  if (lane < 2) a.record[2 * me + lane] = make_int4(-1, 0, 0, 0);
  __syncwarp();
  if (me >= workers) return;
  const int64_t from = total * me / workers, count = total * (me + 1) / workers - from;

  AttendCursor use;
  int64_t passed = 0;  // steps taken
  {
    int lo = 0, hi = kAttThreads;  // upto[lo] <= from < upto[hi]
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
    use.q = attend_request(a, use.r, false);
    attend_sizes<kCols>(a, use);
    const int64_t item = rest / use.units;
    use.u = (int)(rest - item * use.units);
    use.h = (int)(item / use.tiles);
    use.tile = (int)(item - (int64_t)use.h * use.tiles);
  }

  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * Shape::kWarp;
  const uint32_t scores = ring + 2 * Shape::kStage;

  // ---- the copies of a step, one ahead of its use ----
  AttendCursor ahead = use;
  int entry = 0;  // of the lane's token in the next step to copy
  auto look_up = [&] {
    const int t = ahead.u * kUnit + lane;
    entry = t < ahead.q.len ? __ldg(a.table + (int64_t)ahead.r * a.table_stride + a.block((uint32_t)t)) : -1;
  };
  auto copy = [&](int stage) -> uint32_t {
    const int t = ahead.u * kUnit + lane;
    const bool there = (uint32_t)entry < (uint32_t)a.n_blocks && entry >= 0;
    if (!there && t < ahead.q.len) atomicOr(&a.small->op_status, kStBadInput);
    const uint32_t row = (uint32_t)t - a.block((uint32_t)t) * a.block.d;
    const unsigned char* page =
        there ? a.cache + (int64_t)entry * a.block_stride + (int64_t)ahead.h * a.page_bytes : a.cache;
    const int64_t values = there ? (int64_t)a.heads * a.page_bytes : 0;
    const unsigned char* codes = there ? page + (int64_t)row * Shape::kRow : page;
    const uint32_t to = ring + stage * Shape::kStage;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int at = i * 32 + lane, src = at / G, chunk = at % G;
      const unsigned char* p =
          reinterpret_cast<const unsigned char*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(codes), src));
      const int64_t v = __shfl_sync(0xFFFFFFFFu, (unsigned long long)values, src);
      const bool ok = v != 0;
      const uint32_t d = to + src * Shape::kRow + (attend_piece<G>(src, chunk >> 1) * 2 + (chunk & 1)) * 16;
      copy_async<16>(d, p + (ok ? chunk * 16 : 0), ok);
      copy_async<16>(d + Shape::kHalfStage, p + (ok ? v + chunk * 16 : 0), ok);
    }
    const unsigned char* pairs =
        there ? page + ((int64_t)a.block.d * 16 + (int64_t)row * 4) * G : page;
    constexpr int kPiece = G % 4 == 0 ? 16 : G % 2 == 0 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < Shape::kPair / kPiece; ++i) {
      const uint32_t d = to + kUnit * Shape::kRow + lane * Shape::kPair + i * kPiece;
      copy_async<kPiece>(d, pairs + (there ? i * kPiece : 0), there);
      copy_async<kPiece>(d + Shape::kHalfStage, pairs + (there ? values + i * kPiece : 0), there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return __ballot_sync(0xFFFFFFFFu, there);
  };

  // ---- an item's state ----
  uint32_t q[NT][G][QP][4];
  float qsum[NT][G][2];   // of columns 2 c and 2 c + 1
  float acc[NT][2 * G][4];
  float off[NT][G], top[NT], total_p[NT];  // of column g, this thread's tokens
  int sees[NT];           // tokens that column g sees
  bool whole = false;     // the item begins with this worker's first step of it

  auto begin = [&] {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = use.tile * kCols + 8 * n + g;
      const bool real = col < use.q.fresh * (int)a.group.d;
      const int token = (int)a.group((uint32_t)col), head = use.h * (int)a.group.d + col - token * (int)a.group.d;
      const TQ* row = static_cast<const TQ*>(a.queries) + (int64_t)(use.q.first + token) * a.q_token + head * a.q_head;
      sees[n] = real ? use.q.len - use.q.fresh + token + 1 : INT32_MAX;  // columns without a token ask for no masks
      top[n] = -INFINITY;
      total_p[n] = 0.f;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float e[8];
        const int at = 32 * j + 8 * c;
        if (real && a.q_wide && at < a.dim) {
          Vec<TQ, 8> v;
          v.template load<true>(row + at);
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = to_f32(v.x[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = real && at + i < a.dim ? to_f32(row[at + i]) : 0.f;
        }
        float s = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
        qsum[n][j][0] = __shfl_sync(0xFFFFFFFFu, s, 8 * c);
        qsum[n][j][1] = __shfl_sync(0xFFFFFFFFu, s, 8 * c + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kHalf) {
            const __half2 h = __floats2half2_rn(e[i], e[i + 4]);
            q[n][j][0][i] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            uint32_t part[QP];
            split_pair<QP>(e[i], e[i + 4], part);
#pragma unroll
            for (int p = 0; p < QP; ++p) q[n][j][p][i] = part[p];
          }
        }
        off[n][j] = 0.f;
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][2 * j + s2][i] = 0.f;
      }
    }
  };

  // ---- a step ----
  auto step = [&](uint32_t at, uint32_t there, auto partial_tag) {
    constexpr bool kPartial = decltype(partial_tag)::value;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const int k0 = tile * 16 + g, k1 = k0 + 8;
      float s[NT][4] = {};
#pragma unroll
      for (int u = 0; u < (G + 1) / 2; ++u) {
        constexpr bool kOdd = G % 2 == 1;
        const bool pair = !kOdd || u < G / 2;
        uint2 w0, w1, p0, p1;
        const uint32_t codes = at, pairs = at + kUnit * Shape::kRow;
        if (pair) {
          w0 = lds64(codes + k0 * Shape::kRow + attend_piece<G>(k0, u) * 32 + c * 8);
          w1 = lds64(codes + k1 * Shape::kRow + attend_piece<G>(k1, u) * 32 + c * 8);
        } else {
          w0.x = lds32(codes + k0 * Shape::kRow + u * 32 + c * 4);
          w1.x = lds32(codes + k1 * Shape::kRow + u * 32 + c * 4);
        }
        if (!kOdd) {
          p0 = lds64(pairs + k0 * Shape::kPair + u * 8);
          p1 = lds64(pairs + k1 * Shape::kPair + u * 8);
        } else {
          p0.x = lds32(pairs + k0 * Shape::kPair + u * 8);
          p1.x = lds32(pairs + k1 * Shape::kPair + u * 8);
          if (pair) {
            p0.y = lds32(pairs + k0 * Shape::kPair + u * 8 + 4);
            p1.y = lds32(pairs + k1 * Shape::kPair + u * 8 + 4);
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int j = 2 * u + half;
          if (j >= G) break;
          const uint32_t x0 = half ? w0.y : w0.x, x1 = half ? w1.y : w1.x;
          const uint32_t y0 = half ? p0.y : p0.x, y1 = half ? p1.y : p1.x;
          const float s0 = 16.f * bf16_low(y0), s1 = 16.f * bf16_low(y1);
          const float b0 = bf16_high(y0) - s0, b1 = bf16_high(y1) - s1;
          uint32_t lo[4], hi[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            lo[2 * i] = codes_to_floats<kHalf>(x0, i);
            lo[2 * i + 1] = codes_to_floats<kHalf>(x1, i);
            hi[2 * i] = codes_to_floats<kHalf>(x0, i + 2);
            hi[2 * i + 1] = codes_to_floats<kHalf>(x1, i + 2);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < QP; ++p) {
              if (kHalf) {
                mma_f16(d, lo, q[n][j][p][0], q[n][j][p][1]);
                mma_f16(d, hi, q[n][j][p][2], q[n][j][p][3]);
              } else {
                mma_bf16(d, lo, q[n][j][p][0], q[n][j][p][1]);
                mma_bf16(d, hi, q[n][j][p][2], q[n][j][p][3]);
              }
            }
            s[n][0] += s0 * d[0] + b0 * qsum[n][j][0];
            s[n][1] += s0 * d[1] + b0 * qsum[n][j][1];
            s[n][2] += s1 * d[2] + b1 * qsum[n][j][0];
            s[n][3] += s1 * d[3] + b1 * qsum[n][j][1];
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t to = scores + n * (kUnit * 32) + c * 8;
        asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(to + k0 * 32), "f"(s[n][0]), "f"(s[n][1]) : "memory");
        asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(to + k1 * 32), "f"(s[n][2]), "f"(s[n][3]) : "memory");
      }
    }
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
        p[n][i] = a.scale * __uint_as_float(lds32(scores + n * (kUnit * 32) + (c + 4 * i) * 32 + g * 4));
        if (kPartial) {
          const bool see = use.u * kUnit + c + 4 * i < sees[n] && (there >> (c + 4 * i) & 1);
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
    if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float f = most[n] > top[n] ? exp2_fast(top[n] - most[n]) : 1.f;
        top[n] = most[n];
        total_p[n] *= f;
        const float f0 = __shfl_sync(0xFFFFFFFFu, f, 8 * c), f1 = __shfl_sync(0xFFFFFFFFu, f, 8 * c + 4);
#pragma unroll
        for (int j = 0; j < G; ++j) off[n][j] *= f;
#pragma unroll
        for (int j = 0; j < 2 * G; ++j) {
          acc[n][j][0] *= f0;
          acc[n][j][1] *= f1;
          acc[n][j][2] *= f0;
          acc[n][j][3] *= f1;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float m = top[n] == -INFINITY ? 0.f : top[n];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[n][i] = exp2_fast(p[n][i] - m);
        total_p[n] += p[n][i];
      }
    }
    const uint32_t codes = at + Shape::kHalfStage, pairs = codes + kUnit * Shape::kRow;
    const uint32_t select = g & 1 ? 0x7632 : 0x5410;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
#pragma unroll
      for (int u = 0; u < (G + 1) / 2; ++u) {
        constexpr bool kOdd = G % 2 == 1;
        const bool pair = !kOdd || u < G / 2;
        uint2 w[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = tile * 16 + c + 4 * i;
          if (pair) w[i] = lds64(codes + t * Shape::kRow + attend_piece<G>(t, u) * 32 + (g >> 1) * 8);
          else w[i].x = lds32(codes + t * Shape::kRow + u * 32 + (g >> 1) * 4);
          if (!kOdd) {
            y[i] = lds64(pairs + t * Shape::kPair + u * 8);
          } else {
            y[i].x = lds32(pairs + t * Shape::kPair + u * 8);
            if (pair) y[i].y = lds32(pairs + t * Shape::kPair + u * 8 + 4);
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int j = 2 * u + half;
          if (j >= G) break;
          const uint32_t x0 = __byte_perm(half ? w[0].y : w[0].x, half ? w[1].y : w[1].x, select);
          const uint32_t x1 = __byte_perm(half ? w[2].y : w[2].x, half ? w[3].y : w[3].x, select);
          uint32_t v[2][4];
#pragma unroll
          for (int s2 = 0; s2 < 2; ++s2) {
            v[s2][0] = codes_to_floats<false>(x0, 2 * s2);
            v[s2][1] = codes_to_floats<false>(x0, 2 * s2 + 1);
            v[s2][2] = codes_to_floats<false>(x1, 2 * s2);
            v[s2][3] = codes_to_floats<false>(x1, 2 * s2 + 1);
          }
          float st[4], ba[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t z = half ? y[i].y : y[i].x;
            st[i] = 16.f * bf16_low(z);
            ba[i] = bf16_high(z) - st[i];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float wt[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w1 = p[n][4 * tile + i];
              wt[i] = w1 * st[i];
              float b = w1 * ba[i];
              if (kPartial && !(seen[n] >> (4 * tile + i) & 1)) wt[i] = b = 0.f;  // whatever is stored there
              off[n][j] += b;
            }
            uint32_t b0[PP], b1[PP];
            split_pair<PP>(wt[0], wt[1], b0);
            split_pair<PP>(wt[2], wt[3], b1);
#pragma unroll
            for (int k = 0; k < PP; ++k) {
              mma_bf16(acc[n][2 * j], v[0], b0[k], b1[k]);
              mma_bf16(acc[n][2 * j + 1], v[1], b0[k], b1[k]);
            }
          }
        }
      }
    }
  };

  // ---- an item's end, or the end of this worker's share of it ----
  auto finish = [&](bool last) {
    const bool done = whole && last;
    float* part = a.partial + (2 * me + (whole ? 1 : 0)) * Shape::kPartial;
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
      for (int j = 0; j < G; ++j) {
        off[n][j] += __shfl_xor_sync(0xFFFFFFFFu, off[n][j], 1);
        off[n][j] += __shfl_xor_sync(0xFFFFFFFFu, off[n][j], 2);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from_lane = 8 * c + 4 * e;
        const float sum_p = __shfl_sync(0xFFFFFFFFu, l, from_lane);
        const float by = sum_p == 0.f ? 0.f : 1.f / sum_p;
        const int col = use.tile * kCols + 8 * n + 2 * c + e;
        const bool real = col < use.q.fresh * (int)a.group.d;
        const int token = (int)a.group((uint32_t)col), head = use.h * (int)a.group.d + col - token * (int)a.group.d;
        const int64_t row = (int64_t)(use.q.first + token) * a.o_token + head * a.o_head;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float o = __shfl_sync(0xFFFFFFFFu, off[n][j], from_lane);
          float4 r = make_float4(acc[n][2 * j][e] + o, acc[n][2 * j][2 + e] + o, acc[n][2 * j + 1][e] + o,
                                 acc[n][2 * j + 1][2 + e] + o);
          if (!done) {
            *reinterpret_cast<float4*>(part + (8 * n + 2 * c + e) * 32 * G + 32 * j + 4 * g) = r;
          } else if (real) {
            r.x *= by, r.y *= by, r.z *= by, r.w *= by;
            attend_store(a, row, 32 * j + 4 * g, r);
          }
        }
      }
    }
    if (!done && lane == 0) {
      // the workers among which the item's steps lie
      const int64_t i0 = from + passed - use.u, i1 = i0 + use.units - 1;
      a.record[2 * me + (whole ? 1 : 0)] =
          make_int4((int)(((i0 + 1) * workers - 1) / total), (int)(((i1 + 1) * workers - 1) / total), use.r,
                    use.h * use.tiles + use.tile);
    }
  };
  look_up();
  uint32_t there = copy(0), there_next = 0;
  if (count > 1) {
    attend_next<kCols>(a, ahead);
    look_up();
  }
  begin();
  whole = use.u == 0;
  for (; passed < count; ++passed) {
    const int stage = passed & 1;
    if (passed + 1 < count) {
      there_next = copy(stage ^ 1);
      if (passed + 2 < count) {
        attend_next<kCols>(a, ahead);
        look_up();
      }
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    bool part = there != 0xFFFFFFFFu;
#pragma unroll
    for (int n = 0; n < NT; ++n) part |= sees[n] < (use.u + 1) * kUnit;
    if (__any_sync(0xFFFFFFFFu, part)) step(ring + stage * Shape::kStage, there, std::true_type{});
    else step(ring + stage * Shape::kStage, there, std::false_type{});
    __syncwarp();  // before the stage is filled again
    there = there_next;
    const bool last = use.u + 1 == use.units;
    if (last || passed + 1 == count) finish(last);
    if (passed + 1 < count) {
      attend_next<kCols>(a, use);
      if (last) {
        begin();
        whole = true;
      }
    }
  }
}

// Adds up the partial sums of items that lie in several workers' shares, in the
// order of the shares. Block b looks at the border between workers b and b + 1;
// of an item that spans k borders each of their blocks takes columns.
constexpr int kJoinThreads = 256;
template <int G, int NT>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(AttendArgs a) {
  using Shape = AttendShape<G, 1, NT>;
  constexpr int kCols = Shape::kCols, kVecs = 8 * G;  // vectors of 4 of a column
  __shared__ float4 part_sum[kJoinThreads];
  __shared__ float part_total[kJoinThreads];
  await_previous();
  const int64_t b = blockIdx.x + 1;
  const int4 rec = a.record[2 * b];
  if (rec.x < 0) return;
  const int w0 = rec.x, w1 = rec.y, parts = w1 - w0 + 1;
  const AttendRequest q = attend_request(a, rec.z, false);
  AttendCursor cur;
  cur.q = q;
  attend_sizes<kCols>(a, cur);
  const int h = rec.w / cur.tiles, tile = rec.w - h * cur.tiles, group = (int)a.group.d;
  const int cols = min(kCols, q.fresh * group - tile * kCols);
  // this block's columns, and for each of its vectors as many threads as there are
  const int first = (int)b - w0 - 1, step = w1 - w0;
  if (first >= cols) return;
  const int mine = (cols - first + step - 1) / step;
  const int slices = max(1, min(parts, kJoinThreads / (mine * kVecs)));
  const int lanes = min(mine * kVecs, kJoinThreads);
  for (int base = 0; base < mine * kVecs; base += lanes) {
    const int slice = threadIdx.x / lanes, item = base + threadIdx.x % lanes;
    const bool here = slice < slices && item < mine * kVecs;
    const int col = first + (item / kVecs) * step, at = 4 * (item % kVecs);
    auto slot = [&](int k) { return a.partial + (2 * (int64_t)(w0 + k) + (k == 0 ? 1 : 0)) * Shape::kPartial; };
    float top = -INFINITY;
    if (here)
#pragma unroll 8
      for (int k = 0; k < parts; ++k) top = fmaxf(top, slot(k)[kCols * 32 * G + col]);
    const float m = top == -INFINITY ? 0.f : top;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    if (here)
#pragma unroll 4
      for (int k = slice; k < parts; k += slices) {
        const float* p = slot(k);
        const float f = exp2_fast(p[kCols * 32 * G + col] - m);
        const float4 v = *reinterpret_cast<const float4*>(p + col * 32 * G + at);
        sum.x += f * v.x, sum.y += f * v.y, sum.z += f * v.z, sum.w += f * v.w;
        total += f * p[kCols * (32 * G + 1) + col];
      }
    part_sum[threadIdx.x] = sum;
    part_total[threadIdx.x] = total;
    __syncthreads();
    if (here && slice == 0) {
      for (int k = 1; k < slices; ++k) {
        const float4 v = part_sum[threadIdx.x + k * lanes];
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        total += part_total[threadIdx.x + k * lanes];
      }
      const float by = total == 0.f ? 0.f : 1.f / total;
      sum.x *= by, sum.y *= by, sum.z *= by, sum.w *= by;
      const int at_col = tile * kCols + col, token = at_col / group, head = h * group + at_col - token * group;
      attend_store(a, (int64_t)(q.first + token) * a.o_token + head * a.o_head, at, sum);
    }
    __syncthreads();
  }
}

template <class F>
int with_groups(int64_t groups, F f) {
  using std::integral_constant;
  switch (groups) {
    case 1: return f(integral_constant<int, 1>{});
    case 2: return f(integral_constant<int, 2>{});
    case 3: return f(integral_constant<int, 3>{});
    case 4: return f(integral_constant<int, 4>{});
    case 6: return f(integral_constant<int, 6>{});
    default: return f(integral_constant<int, 8>{});
  }
}

}  // namespace

extern "C" {

int bpe_attend(bpe_handle* h, const bpe_attend_args* args, bpe_stream_t stream) {
  return guarded("bpe_attend", [&]() -> int {
    auto bad = [&](const char* what) { return fail(BPE_ERR_INVALID_ARG, std::string("bpe_attend: ") + what); };
    if (!h) return bad("null handle");
    if (!args) return bad("null arguments");
    const bpe_attend_args& p = *args;
    int rc = cache_check("bpe_attend", h, p.cache, p.n_blocks, p.block_stride, p.block_size, p.n_heads, p.dim);
    if (rc) return rc;
    if (!type_ok(p.query_type) || !type_ok(p.out_type)) return bad("unknown element type");
    if (p.n_requests < 0 || p.n_requests >= INT32_MAX || p.n_tokens < 0 || p.n_tokens >= INT32_MAX || p.group < 1 ||
        p.group > 256 || p.n_tokens * p.group >= INT32_MAX / p.n_heads || p.max_blocks < 0 || p.max_blocks > INT32_MAX ||
        p.query_token_stride < 0 || p.query_head_stride < 0 || p.out_token_stride < 0 || p.out_head_stride < 0)
      return bad("a size or stride is negative or too large");
    if (!std::isfinite(p.scale)) return bad("scale is not finite");
    if (p.n_requests > 1 && p.table_stride < p.max_blocks) return bad("table rows overlap");
    if (!p.offsets && p.n_tokens < p.n_requests) return bad("n_tokens is below one new token a request");
    if (p.n_requests == 0 || p.n_tokens == 0) return BPE_OK;
    if (!p.queries || !p.out || !p.seq_lens || (p.max_blocks > 0 && !p.table)) return bad("null pointer");
    if (!aligned(p.queries, type_size(p.query_type)) || !aligned(p.out, type_size(p.out_type)) ||
        !aligned(p.table, 4) || !aligned(p.seq_lens, 4) || !aligned(p.offsets, 8))
      return bad("a pointer is not aligned to its elements");
    const int64_t n_rows = p.n_heads * p.group;
    if (rows_meet(p.n_tokens, p.out_token_stride, n_rows, p.out_head_stride, p.dim)) return bad("output rows overlap");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t groups = cache_groups(p.dim);
    const size_t records = align256((size_t)h->n_sms * 2 * kAttWarps * 2 * sizeof(int4));
    rc = ensure_ws(h, records + (size_t)h->n_sms * BPE_ATTEND_PARTIALS * (32 * groups + 2) * sizeof(float), st);
    if (rc) return rc;
    auto fits = [&](const void* q, int64_t token, int64_t head, int64_t size, int64_t V) {
      return p.dim % V == 0 && vec_ok(q, p.n_tokens > 1 ? token : 0, size, V) &&
             vec_ok(q, n_rows > 1 ? head : 0, size, V);
    };
    // absent tokens are zeros copied from nowhere, but from an address that is one
    const void* cache = p.cache ? p.cache : h->d_ws;
    AttendArgs a{p.queries, p.out, p.out_type, p.query_token_stride, p.query_head_stride, p.out_token_stride,
                 p.out_head_stride, p.n_tokens, (int)p.n_heads, (int)p.dim, FastDiv(p.group),
                 static_cast<const unsigned char*>(cache), p.n_blocks, p.block_stride,
                 cache_page_bytes(p.block_size, p.dim), FastDiv(p.block_size), p.table, p.table_stride,
                 std::min<int64_t>(p.max_blocks * p.block_size, INT32_MAX - 2 * kUnit), p.seq_lens, p.offsets, (int)p.n_requests,
                 p.scale * 1.4426950408889634f,
                 fits(p.queries, p.query_token_stride, p.query_head_stride, type_size(p.query_type), 8),
                 fits(p.out, p.out_token_stride, p.out_head_stride, type_size(p.out_type), 4),
                 reinterpret_cast<float*>(static_cast<char*>(h->d_ws) + records), static_cast<int4*>(h->d_ws), h->d_small};
    // 16 columns share the work on a code; a request with at most 8 has no use for the second half
    const bool wide = p.query_type != BPE_F32 &&
                      (p.offsets ? p.n_tokens * p.group > 8 * p.n_requests : p.group > 8);
    return with_groups(groups, [&](auto gs) {
      return with_type(p.query_type, [&](auto tq) -> int {
        constexpr int G = decltype(gs)::value;
        using TQ = decltype(tq);
        auto launch = [&](auto nt) -> int {
          constexpr int NT = decltype(nt)::value;
          constexpr int kSmem = AttendShape<G, 1, NT>::kSmem;
          constexpr int kBlocks = (G <= 4 && NT == 1 && sizeof(TQ) == 2) ? 2 : 1;
          int ok = once_per_device(h->device, [&] {
            return cudaFuncSetAttribute(k_attend<TQ, G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
          });
          if (ok) return ok;
          const unsigned blocks = (unsigned)h->n_sms * kBlocks;
          k_attend<TQ, G, NT><<<blocks, kAttThreads, kSmem, st>>>(a);
          CK(cudaGetLastError());
          CK(launch_after(k_attend_join<G, NT>, dim3(blocks * kAttWarps - 1), kJoinThreads, 0, st, a));
          return BPE_OK;
        };
        if constexpr (sizeof(TQ) == 2)
          if (wide) return launch(std::integral_constant<int, 2>{});
        return launch(std::integral_constant<int, 1>{});
      });
    });
  });
}

}  // extern "C"
