// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Included once by model_ops.cu; not a standalone header.
//
//   out[i, :] = round(scale * W[ids[i], :])
//   dW[r, :]  = round([dW[r, :] +] scale * sum over {i : ids[i] = r} of dOut[i, :])
//
// Sums run in 32 bits over ascending i, so a gradient does not depend on the
// order in which CTAs run.

namespace {

constexpr int kEmbThreads = 128;
constexpr int64_t kEmbMaxDim = 1 << 22;  // columns of a block times the grid's limit

__device__ __forceinline__ bool emb_row_ok(int32_t id, int64_t n_rows) { return id >= 0 && id < n_rows; }

// ---------------------------------------------------------------- lookup --

// A block takes rows of tokens x tx threads: each thread holds kEmbRows tokens'
// vectors of V elements in flight at one column and walks the columns in steps
// of tx vectors. V is 8 where rows are aligned for it, else 2 or 1.
//
// One product an element: bound by HBM, and by the L2 from which frequent rows
// come again, so rows are kept there and the output streams past. 65,536 tokens
// of a Zipf law, 4,096 columns, f32 to bf16: 123 us for the 731 MB of distinct
// rows and output, 5.9 TB/s. With blocks of 256 threads it took 131 us, with
// more tokens a thread up to 152, with 512 threads 159.
constexpr int kEmbRows = 2;

template <class TW, class TO, int V>
__global__ void __launch_bounds__(kEmbThreads) k_embed(const int32_t* ids, int64_t n_ids, const TW* weight,
                                                       int64_t n_rows, int dim, int64_t weight_stride, float scale,
                                                       int32_t skip_id, TO* out, int64_t out_stride, int tx_log2,
                                                       DevSmall* small) {
  const int tx = 1 << tx_log2, ty = kEmbThreads >> tx_log2;
  const int64_t first = (int64_t)blockIdx.x * (kEmbRows * ty) + (threadIdx.x >> tx_log2);
  const int x = threadIdx.x & (tx - 1);
  const TW* w[kEmbRows];
  bool have[kEmbRows], ok[kEmbRows];
#pragma unroll
  for (int q = 0; q < kEmbRows; ++q) {
    const int64_t i = first + q * ty;
    have[q] = i < n_ids;
    const int32_t id = have[q] ? ids[i] : skip_id;
    ok[q] = have[q] && id != skip_id && emb_row_ok(id, n_rows);
    if (have[q] && !ok[q] && id != skip_id && x == 0 && blockIdx.y == 0) atomicOr(&small->op_status, kStBadInput);
    w[q] = weight + (ok[q] ? id : 0) * weight_stride;
  }
  TO* o = out + first * out_stride;
  for (int c = ((int)blockIdx.y * tx + x) * V; c < dim; c += (int)gridDim.y * tx * V) {
    Vec<TW, V> v[kEmbRows];
#pragma unroll
    for (int q = 0; q < kEmbRows; ++q)
      if (ok[q]) v[q].template load<true>(w[q] + c);
#pragma unroll
    for (int q = 0; q < kEmbRows; ++q) {
      if (!have[q]) continue;
      Vec<TO, V> r;
#pragma unroll
      for (int e = 0; e < V; ++e) r.x[e] = from_f32<TO>(ok[q] ? scale * to_f32(v[q].x[e]) : 0.f);
      r.store(o + q * ty * out_stride + c);
    }
  }
}

// ------------------------------------------------------- zero rows and sort --

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBits = 10;  // a bin for each thread
constexpr int kSortCluster = 16;
constexpr int kSortBatch = 4;     // tokens that a lane holds
constexpr int kFillRows = 2048;   // rows a CTA marks at once
constexpr int kFillPage = 16384;  // bytes of a bulk store
constexpr int kFillThreads = 512;

// Rows [r0, r1) without a token become zeros: the CTA reads every id and marks
// the rows that are met; then each thread takes a row and stores its 16-byte
// aligned inside in bulk from a page of zeros in shared memory, which leaves
// the SM's issue slots free, and its ragged ends by element. Alone, with eight
// blocks an SM, 6.5 to 7.0 TB/s; with one 4.4, since SMs differ in what they
// can write and one of two neighbours may get two blocks.
struct FillArgs {
  const int32_t* ids;
  int64_t n, n_rows;
  int32_t skip_id;
  unsigned char* out;
  int64_t row_bytes, stride_bytes, row_step;  // row_step: rows of a CTA at once, at most kFillRows
  int element;                                // bytes of an element
};

struct FillSmem {
  __align__(16) unsigned char zeros[kFillPage];
  uint8_t met[kFillRows];
};

__device__ void fill_absent(const FillArgs& a, int64_t r0, int64_t r1, FillSmem& sm) {
  const int tid = threadIdx.x, threads = blockDim.x;
  for (int b = tid; b < kFillRows; b += threads) sm.met[b] = 0;
  for (int b = tid; b < kFillPage / 16; b += threads) reinterpret_cast<uint4*>(sm.zeros)[b] = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  each_id<4>(a.ids, a.n, tid, threads, [&](uint32_t id) {
    if (id - (uint32_t)r0 < (uint32_t)(r1 - r0) && (int32_t)id != a.skip_id) sm.met[id - (uint32_t)r0] = 1;
  });
  __syncthreads();
  const uint32_t page = (uint32_t)__cvta_generic_to_shared(sm.zeros);
  for (int64_t r = r0 + tid; r < r1; r += threads) {
    if (sm.met[r - r0]) continue;
    unsigned char* row = a.out + r * a.stride_bytes;
    unsigned char* end = row + a.row_bytes;
    unsigned char* from = row + (-reinterpret_cast<uintptr_t>(row) & 15);
    unsigned char* to = end - (reinterpret_cast<uintptr_t>(end) & 15);
    if (from >= to) from = to = end;
    auto element = [&](unsigned char* at) {
      if (a.element == 4) *reinterpret_cast<uint32_t*>(at) = 0;
      else *reinterpret_cast<uint16_t*>(at) = 0;
    };
    for (unsigned char* at = row; at < from; at += a.element) element(at);
    for (unsigned char* at = from; at < to; at += kFillPage) {
      const uint32_t size = (uint32_t)min((int64_t)kFillPage, (int64_t)(to - at));
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(at), "r"(page), "r"(size)
                   : "memory");
    }
    for (unsigned char* at = to; at < end; at += a.element) element(at);
  }
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  // the page is read; the grid's end completes the writes
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncthreads();
}

// The rows of filler `who` of `fillers`.
__device__ __forceinline__ void fill_rows(const FillArgs& a, int64_t who, int64_t fillers, FillSmem& sm) {
  for (int64_t r = who * a.row_step; r < a.n_rows; r += fillers * a.row_step)
    fill_absent(a, r, min(r + a.row_step, a.n_rows), sm);
}

// Runs on the SMs that the sort leaves free: the zeros are most of what a
// gradient writes, and need only the ids.
__global__ void __launch_bounds__(kFillThreads) k_emb_fill(FillArgs a) {
  __shared__ FillSmem sm;
  let_next_begin();
  fill_rows(a, blockIdx.x, gridDim.x, sm);
  await_previous();
}

struct SortArgs {
  const int32_t* ids;
  int64_t n, n_rows;
  int32_t skip_id;
  int passes, bits;    // passes of `bits` bits each, lowest first
  int64_t per_warp;    // tokens of a warp, a multiple of 32
  uint2* ping[2];      // (key, token); the last pass p writes ping[p & 1]
  DevSmall* small;
};

// Tokens sorted by row, equal rows in token order: a counting sort by `bits`
// bits a pass, by the CTAs of one cluster. Tokens without a row (skip_id, and
// ids out of range, which are reported) get the key n_rows and sort last.
//
// A pass: each warp counts the digits of its run of tokens in its own bins;
// the bins' prefix over warps, over the cluster's CTAs (read through
// distributed shared memory) and over digits gives each warp its first place
// for each digit; then the warp walks its run again, 32 tokens at a time, and
// a match of equal digits ranks them in token order.
//
// Bound by the latency of its steps, not by bytes: 65,536 tokens into 69,424
// rows take 21 us, most of which the zeroing of rows hides. A cluster's barrier
// costs less than the launches that it saves.
__global__ void __launch_bounds__(kSortThreads) k_emb_sort(SortArgs a) {
  extern __shared__ __align__(16) int32_t sort_smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int n_ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t n = a.n, n_rows = a.n_rows;
  let_next_begin();
  const int bins = 1 << a.bits;
  int32_t* hist = sort_smem;                  // [kSortWarps][bins]
  int32_t* total = hist + kSortWarps * bins;  // [bins]: of this CTA
  int32_t* base = total + bins;               // [bins]: this CTA's first place
  int32_t* warp_sum = base + bins;            // [kSortWarps]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = ((int64_t)rank * kSortWarps + warp) * a.per_warp;
  const int64_t last = min(first + a.per_warp, n);
  const bool held = a.per_warp <= 32 * kSortBatch;  // a warp's tokens stay in its registers
  int32_t* mine = hist + warp * bins;
  for (int p = 0; p < a.passes; ++p) {
    const int shift = p * a.bits;
    const uint2* from = a.ping[(p + 1) & 1];
    // tokens i0 + 32 q + lane; past `last` the key is none
    auto tokens = [&](int64_t i0, uint2 (&t)[kSortBatch]) {
#pragma unroll
      for (int q = 0; q < kSortBatch; ++q) {
        const int64_t i = i0 + 32 * q + lane;
        t[q] = make_uint2(0xFFFFFFFFu, 0);
        if (i >= last) continue;
        if (p > 0) {
          t[q] = __ldcg(from + i);
        } else {
          const int32_t id = __ldg(a.ids + i);
          const bool ok = id != a.skip_id && emb_row_ok(id, n_rows);
          if (!ok && id != a.skip_id) atomicOr(&a.small->op_status, kStBadInput);
          t[q] = make_uint2(ok ? (uint32_t)id : (uint32_t)n_rows, (uint32_t)i);
        }
      }
    };
    uint2 t[kSortBatch];
    for (int b = tid; b < kSortWarps * bins; b += kSortThreads) hist[b] = 0;
    __syncthreads();
    for (int64_t i0 = first; i0 < last; i0 += 32 * kSortBatch) {
      tokens(i0, t);
#pragma unroll
      for (int q = 0; q < kSortBatch; ++q)
        if (t[q].x != 0xFFFFFFFFu) atomicAdd(&mine[(t[q].x >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    if (tid < bins) {
      int32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int32_t c = hist[w * bins + tid];
        hist[w * bins + tid] = sum;
        sum += c;
      }
      total[tid] = sum;
    }
    cluster.sync();
    int32_t lower = 0, all = 0;
    if (tid < bins) {
#pragma unroll
      for (int r = 0; r < kSortCluster; ++r) {
        const int32_t v = r < n_ctas ? *cluster.map_shared_rank(total + tid, r) : 0;
        all += v;
        if (r < rank) lower += v;
      }
    }
    int32_t upto = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    if (warp == 0) {
      int32_t s = warp_sum[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += o;
      }
      warp_sum[lane] = s;
    }
    __syncthreads();
    if (warp > 0) upto += warp_sum[warp - 1];
    if (tid < bins) base[tid] = upto - all + lower;
    __syncthreads();
    for (int64_t i0 = first; i0 < last; i0 += 32 * kSortBatch) {
      if (!held) tokens(i0, t);
#pragma unroll
      for (int q = 0; q < kSortBatch; ++q) {
        if (i0 + 32 * q >= last) break;
        const bool have = t[q].x != 0xFFFFFFFFu;
        const int digit = have ? (int)((t[q].x >> shift) & (uint32_t)(bins - 1)) : bins;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, digit);
        const int leader = __ffs(same) - 1;
        int32_t before = 0;
        if (have && lane == leader) before = base[digit] + atomicAdd(&mine[digit], __popc(same));
        before = __shfl_sync(0xFFFFFFFFu, before, leader);
        if (have) a.ping[p & 1][before + __popc(same & ((1u << lane) - 1))] = t[q];
      }
    }
    cluster.sync();
  }
}

// Up to kRankTokens tokens: the blocks share the tokens out, and each finds the
// places of its own. It counts all tokens into buckets of neighbouring rows,
// which gives each bucket's first place, and in its token's bucket it counts
// the keys below the token's. All blocks count the same, but none waits for
// another: the passes of a sort do, twice each. 9,001 tokens: 8.0 us, against
// 20 for comparing every token with every other, without buckets.
constexpr int kRankEach = 24;  // tokens of a thread
constexpr int kRankThreads = 512;
constexpr int kRankTokens = kRankEach * kRankThreads;
constexpr int kRankOwn = 64;   // tokens whose place a block finds
constexpr int kRankShare = kRankThreads / kRankOwn;
constexpr int kRankBits = 10;  // buckets: two a thread
constexpr int kRankBuckets = 1 << kRankBits;

struct RankArgs {
  const int32_t* ids;
  int n;
  uint32_t n_rows, by;  // by: a row times this, plus the token, sorts as (row, token)
  int32_t skip_id, shift;  // shift: the rows of a bucket, as a power of two
  uint2* sorted;
  DevSmall* small;
};

__global__ void __launch_bounds__(kRankThreads) k_emb_rank(RankArgs a) {
  static_assert(kRankBuckets == 2 * kRankThreads);
  extern __shared__ uint32_t rank_keys[];  // [n] by bucket
  __shared__ int next[kRankBuckets];       // a bucket's next place: once all are taken, its end
  __shared__ uint32_t mine[kRankOwn];
  __shared__ int part[kRankShare][kRankOwn], warp_sum[kRankThreads / 32];
  let_next_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, first = (int)blockIdx.x * kRankOwn;
  int32_t id[kRankEach];
#pragma unroll
  for (int q = 0; q < kRankEach; ++q) id[q] = tid + q * kRankThreads < a.n ? __ldg(a.ids + tid + q * kRankThreads) : 0;
  next[tid] = next[tid + kRankThreads] = 0;
  __syncthreads();
  uint32_t row[kRankEach];
#pragma unroll
  for (int q = 0; q < kRankEach; ++q) {
    const int i = tid + q * kRankThreads;
    const bool ok = id[q] != a.skip_id && (uint32_t)id[q] < a.n_rows;
    row[q] = ok ? (uint32_t)id[q] : a.n_rows;
    if (i >= a.n) continue;
    atomicAdd(&next[row[q] >> a.shift], 1);
    if (i >= first && i < first + kRankOwn) {
      if (!ok && id[q] != a.skip_id) atomicOr(&a.small->op_status, kStBadInput);
      mine[i - first] = row[q];
    }
  }
  __syncthreads();
  const int c0 = next[2 * tid], c1 = next[2 * tid + 1];
  int upto = c0 + c1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRankThreads / 32; ++w)
    if (w < warp) upto += warp_sum[w];
  next[2 * tid] = upto - c0 - c1;
  next[2 * tid + 1] = upto - c1;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kRankEach; ++q) {
    const int i = tid + q * kRankThreads;
    if (i < a.n) rank_keys[atomicAdd(&next[row[q] >> a.shift], 1)] = row[q] * a.by + (uint32_t)i;
  }
  __syncthreads();
  const int own = tid % kRankOwn, share = tid / kRankOwn, i = first + own;
  int begin = 0, below = 0;
  uint32_t r = 0;
  if (i < a.n) {
    r = mine[own];
    const uint32_t bucket = r >> a.shift, k = r * a.by + (uint32_t)i;
    begin = bucket > 0 ? next[bucket - 1] : 0;
    const int end = next[bucket];
#pragma unroll 4
    for (int j = begin + share; j < end; j += kRankShare) below += rank_keys[j] < k;
  }
  part[share][own] = below;
  __syncthreads();
  if (share == 0 && i < a.n) {
#pragma unroll
    for (int q = 1; q < kRankShare; ++q) below += part[q][own];
    a.sorted[begin + below] = make_uint2(r, (uint32_t)i);
  }
}

// ------------------------------------------------------------------- sum --

constexpr int kSumWarps = 8;
constexpr int kSumCols = 512;     // columns of a block
constexpr int kSumMaxRun = 32;    // tokens of a warp, at most
constexpr int kSumMinRun = 2;     // and at least
constexpr int kSmallTokens = 512; // most tokens of the single launch
constexpr int64_t kSmallRows = (1ll << 32) / kSmallTokens - 1;  // and rows: a key and a token fit 32 bits
constexpr int kSumRing = 8320;    // bytes of a warp's tokens in flight

template <class TG, class TW>
struct SumArgs {
  const uint2* sorted;   // (key, token)
  int64_t n, n_rows;
  const TG* grad;
  int64_t grad_stride;
  float scale;
  int dim, run;          // run: tokens of a warp
  TW* out;
  int64_t out_stride;
  int accumulate;
  float* partial;        // [chunks][2][dim]: what a chunk adds to the row that it begins in and that began before,
                         // and to the row that it ends in and that goes on
};

// V columns of row r from their sums.
template <class TG, class TW, int V>
__device__ __forceinline__ void sum_write(const SumArgs<TG, TW>& a, int64_t r, int col, const float* x) {
  TW* o = a.out + r * a.out_stride + col;
  Vec<TW, V> v;
  if (a.accumulate) v.load(o);
#pragma unroll
  for (int e = 0; e < V; ++e)
    v.x[e] = from_f32<TW>(a.accumulate ? to_f32(v.x[e]) + a.scale * x[e] : a.scale * x[e]);
  v.store(o);
}

// acc += v: two 32-bit sums an instruction where V is even.
template <class T, int V>
__device__ __forceinline__ void add_vec(float (&acc)[V], const Vec<T, V>& v) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2)
      asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
          "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
          : "+f"(acc[e]), "+f"(acc[e + 1])
          : "f"(to_f32(v.x[e])), "f"(to_f32(v.x[e + 1])));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] += to_f32(v.x[e]);
  }
}

// A block sums kSumCols columns of a chunk of kSumWarps runs of sorted tokens;
// a warp its run, a lane V adjacent columns in each of kSlabs slabs. Every warp
// has the same number of tokens, however they are spread over the rows:
//   * a row that begins and ends inside a run is written by the warp;
//   * the sums of a run's first and last row go to shared memory, where the
//     block joins them over its runs in order and writes the rows that begin
//     and end inside its chunk;
//   * what the chunk adds to a row that reaches past it goes to `partial`,
//     which k_emb_join adds up in order.
// Tokens come through a ring of asynchronous copies in shared memory (8 KB a
// warp in flight without registers for them), and sums run two an instruction.
// Bound by HBM: 65,536 tokens of 4,096 bf16 columns, 537 MB, and the rows that
// they meet written once: 111 us, beside which the zeros of the other rows are
// written (190 us in all, 1.1 GB). With one warp a row, and long rows cut in
// pieces, the kernel before took 301 us.
template <class TG, class TW, int V>
__device__ __forceinline__ void sum_chunk(const SumArgs<TG, TW>& a, const uint2* sorted, int64_t c0, int64_t c1,
                                          int run, unsigned char* sum_smem) {
  constexpr int kSlabs = kSumCols / (32 * V);
  constexpr bool kVectors = V * sizeof(TG) == 16;
  constexpr int kSlot = kSumCols * (int)sizeof(TG) + (kVectors ? 0 : 16);  // of a token in the ring
  constexpr int kAhead = kSumRing / kSlot;                                 // tokens in flight
  const int ring_bytes = min(kAhead, run) * kSlot;                         // a run has no more
  __shared__ __align__(16) float part[kSumWarps][2][kSumCols];
  __shared__ int32_t part_key[kSumWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col0 = (int)blockIdx.y * kSumCols;
  const int64_t j0 = min(c0 + warp * run, c1), j1 = min(j0 + run, c1);
  const int32_t before = c0 > 0 ? (int32_t)sorted[c0 - 1].x : -1;
  const int32_t after = c1 < a.n ? (int32_t)sorted[c1].x : -1;
  // up to 32 tokens of the run, a lane each; those without a row are the last
  uint2 mine = make_uint2(0xFFFFFFFFu, 0);
  int len = 0;
  auto take = [&](int64_t from) {
    mine = from + lane < j1 ? sorted[from + lane] : make_uint2(0xFFFFFFFFu, 0);
    len = __popc(__ballot_sync(0xFFFFFFFFu, mine.x < (uint32_t)a.n_rows));
  };
  take(j0);
  const bool any = len > 0;
  float acc[kSlabs][V] = {};
  int32_t row = (int32_t)__shfl_sync(0xFFFFFFFFu, mine.x, 0);
  bool begun = false;  // the run's first row has ended
  auto stash = [&](int which) {
#pragma unroll
    for (int s = 0; s < kSlabs; ++s) {
      float* to = &part[warp][which][(s * 32 + lane) * V];
      if constexpr (V >= 4) {
#pragma unroll
        for (int e = 0; e < V; e += 4)
          *reinterpret_cast<float4*>(to + e) = make_float4(acc[s][e], acc[s][e + 1], acc[s][e + 2], acc[s][e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) to[e] = acc[s][e];
      }
    }
    if (lane == 0) part_key[warp][which] = row;
  };
  const TG* grad = a.grad + col0 + lane * V;
  const int cols = a.dim - col0 - lane * V;  // this lane's slab s exists if s * 32 * V < cols
  // the row that ended leaves, and `key` begins
  auto next_row = [&](int32_t key) {
    if (!begun) {
      stash(0);
    } else {
#pragma unroll
      for (int s = 0; s < kSlabs; ++s)
        if (s * 32 * V < cols) sum_write<TG, TW, V>(a, row, col0 + (s * 32 + lane) * V, acc[s]);
    }
    begun = true;
    row = key;
#pragma unroll
    for (int s = 0; s < kSlabs; ++s)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[s][e] = 0.f;
  };
  for (int64_t from = j0;;) {
    if constexpr (kVectors) {
      // Each lane copies its own vectors into its warp's ring and reads them
      // back itself, so no barrier is needed; a token is one group of copies.
      const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sum_smem) + warp * ring_bytes + lane * 16;
      auto fetch = [&](int j, uint32_t slot) {
        if (j < len) {
          const TG* g = grad + (int64_t)__shfl_sync(0xFFFFFFFFu, mine.y, j) * a.grad_stride;
#pragma unroll
          for (int s = 0; s < kSlabs; ++s)
            if (s * 32 * V < cols)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + slot + s * 512), "l"(g + s * 32 * V)
                           : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(j, j * kSlot);
      uint32_t slot = 0;
      for (int j = 0; j < len; ++j) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const int32_t key = (int32_t)__shfl_sync(0xFFFFFFFFu, mine.x, j);
        Vec<TG, V> v[kSlabs];
#pragma unroll
        for (int s = 0; s < kSlabs; ++s)
          v[s] = *reinterpret_cast<const Vec<TG, V>*>(__cvta_shared_to_generic(ring + slot + s * 512));
        if (key != row) next_row(key);
#pragma unroll
        for (int s = 0; s < kSlabs; ++s) add_vec<TG, V>(acc[s], v[s]);
        fetch(j + kAhead, slot);
        slot = slot + kSlot == kAhead * kSlot ? 0 : slot + kSlot;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      // Rows that are not aligned: the warp copies the 16-byte granules that a
      // token's columns lie in, and the lanes read theirs from inside them.
      unsigned char* ring = sum_smem + warp * ring_bytes;
      const int bytes = min(kSumCols, a.dim - col0) * (int)sizeof(TG);
      const char* from0 = reinterpret_cast<const char*>(a.grad + col0);
      auto source = [&](int j) {
        return from0 + (int64_t)__shfl_sync(0xFFFFFFFFu, mine.y, j & 31) * a.grad_stride * (int64_t)sizeof(TG);
      };
      auto fetch = [&](int j, int slot) {
        const char* from = source(j);
        if (j < len) {
          const int off = (int)(reinterpret_cast<uintptr_t>(from) & 15);
          const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring + slot * kSlot);
          for (int g = lane * 16; g < off + bytes; g += 512) {
            const int size = min(16, off + bytes - g);  // nothing past the row is read
            const char* at = from - off + g;
            if (at < reinterpret_cast<const char*>(a.grad)) {  // nor before the first one
              for (int e = off; e < size; e += sizeof(TG))
                *reinterpret_cast<TG*>(ring + slot * kSlot + e) = *reinterpret_cast<const TG*>(at + e);
              continue;
            }
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + g), "l"(at), "r"(size) : "memory");
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(j, j);
      int slot = 0;
      for (int j = 0; j < len; ++j) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        __syncwarp();
        const int32_t key = (int32_t)__shfl_sync(0xFFFFFFFFu, mine.x, j);
        const int off = (int)(reinterpret_cast<uintptr_t>(source(j)) & 15);
        const TG* v = reinterpret_cast<const TG*>(ring + slot * kSlot + off) + lane;
        if (key != row) next_row(key);
#pragma unroll
        for (int s = 0; s < kSlabs; ++s)
          if (s * 32 < cols) acc[s][0] += to_f32(v[s * 32]);
        __syncwarp();
        fetch(j + kAhead, slot);
        slot = slot + 1 == kAhead ? 0 : slot + 1;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    }
    from += 32;
    if (len < 32 || from >= j1) break;
    take(from);
  }
  // a run of one row has only the first part, an empty run none (key -1)
  if (any) stash(begun ? 1 : 0);
  if (lane == 0) {
    if (!any) part_key[warp][0] = -1;
    if (!begun) part_key[warp][1] = -1;
  }
  __syncthreads();
  constexpr int kPer = kSumCols / (kSumWarps * 32);  // columns of a thread
  constexpr int kW = V < kPer ? V : kPer;
  const int c = threadIdx.x * kPer;
  int32_t cur = part_key[0][0];
  if (col0 + c >= a.dim || cur < 0) return;
  float sum[kPer] = {};
  bool at_start = true;  // cur is the chunk's first row
  auto emit = [&](bool at_end) {
    const bool from = at_start && cur == before, on = at_end && cur == after;
    if (from || on) {
      float* to = a.partial + (2 * (int64_t)blockIdx.x + (at_start ? 0 : 1)) * a.dim + col0 + c;
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (col0 + c + e < a.dim) to[e] = sum[e];
    } else {
#pragma unroll
      for (int e = 0; e < kPer; e += kW)
        if (col0 + c + e < a.dim) sum_write<TG, TW, kW>(a, cur, col0 + c + e, sum + e);
    }
  };
  for (int w = 0; w < kSumWarps; ++w) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int32_t k = part_key[w][which];
      if (k < 0) continue;
      if (k != cur) {
        emit(false);
        cur = k;
        at_start = false;
#pragma unroll
        for (int e = 0; e < kPer; ++e) sum[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) sum[e] += part[w][which][c + e];
    }
  }
  emit(true);
}

template <class TG, class TW, int V>
__global__ void __launch_bounds__(kSumWarps * 32) k_emb_sum(SumArgs<TG, TW> a) {
  extern __shared__ __align__(16) unsigned char sum_smem[];
  await_previous();
  let_next_begin();
  const int64_t c0 = (int64_t)blockIdx.x * kSumWarps * a.run;
  sum_chunk<TG, TW, V>(a, a.sorted, c0, min(c0 + kSumWarps * a.run, a.n), a.run, sum_smem);
}

// Up to kSmallTokens tokens in one launch: blocks [0, chunks) rank the tokens
// by comparing each with every other, all of them in each block, which is
// sooner done than another kernel is begun, and sum a chunk of whole rows; the
// others zero rows without a token. 300 tokens of 512 f32 columns into 768
// rows: 8.6 us, latency (14.8 as sort, sums and join); 7 tokens into 69,424 rows
// of 1,600: 64 us, the rate of the zeros.
template <class TG, class TW, int V>
__global__ void __launch_bounds__(kSumWarps * 32) k_emb_small(SumArgs<TG, TW> a, FillArgs f, int64_t n_chunks,
                                                              DevSmall* small) {
  extern __shared__ __align__(16) unsigned char sum_smem[];
  __shared__ uint2 sorted[kSmallTokens];
  __shared__ __align__(16) uint32_t key[kSmallTokens];
  __shared__ int bound[2];
  if (blockIdx.x >= n_chunks) {
    if (blockIdx.y == 0)
      fill_rows(f, blockIdx.x - n_chunks, gridDim.x - n_chunks, *reinterpret_cast<FillSmem*>(sum_smem));
    return;
  }
  // key * kSmallTokens + token: distinct, and in sorted order
  const int n = (int)a.n, tid = threadIdx.x;
  for (int i = tid; i < kSmallTokens; i += kSumWarps * 32) {
    uint32_t k = 0xFFFFFFFFu;
    if (i < n) {
      const int32_t id = __ldg(f.ids + i);
      const bool ok = id != f.skip_id && emb_row_ok(id, a.n_rows);
      if (!ok && id != f.skip_id && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(&small->op_status, kStBadInput);
      k = (ok ? (uint32_t)id : (uint32_t)a.n_rows) * kSmallTokens + (uint32_t)i;
    }
    key[i] = k;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kSumWarps * 32) {
    const uint32_t k = key[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(key + j);
      rank += (o.x < k) + (o.y < k) + (o.z < k) + (o.w < k);
    }
    sorted[rank] = make_uint2(k / kSmallTokens, (uint32_t)i);
  }
  if (tid == 0) bound[0] = bound[1] = n;
  __syncthreads();
  // the block's share of the places, moved to where rows begin
  const int c0 = (int)blockIdx.x * kSumWarps * a.run, c1 = c0 + kSumWarps * a.run;
  for (int p = tid; p < n; p += kSumWarps * 32)
    if (p == 0 || sorted[p].x != sorted[p - 1].x) {
      if (p >= c0) atomicMin(&bound[0], p);
      if (p >= c1) atomicMin(&bound[1], p);
    }
  __syncthreads();
  const int b0 = bound[0], b1 = bound[1];
  if (b0 < b1) sum_chunk<TG, TW, V>(a, sorted, b0, b1, (b1 - b0 + kSumWarps - 1) / kSumWarps, sum_smem);
}

// The parts of a row that reaches past a chunk, joined in order by the block
// of the chunk that it begins in. A chunk's part is its second one if the row
// begins inside it, and its first one otherwise. The sorted tokens are older
// than the kernel before, so they are read before it ends. 11 us for the 256
// chunks of 65,536 tokens, most of it the latency of a few dependent reads.
template <class TG, class TW, int V>
__global__ void __launch_bounds__(kSumWarps * 32) k_emb_join(SumArgs<TG, TW> a) {
  constexpr int kPer = kSumCols / 32;
  __shared__ float part[kSumWarps][kSumCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t chunk = kSumWarps * a.run;
  const int64_t c = blockIdx.x, c0 = c * chunk, c1 = min(c0 + chunk, a.n);
  const uint32_t r = a.sorted[c1 - 1].x, first = a.sorted[c0].x;
  const uint32_t before = c0 > 0 ? a.sorted[c0 - 1].x : 0xFFFFFFFFu;
  const bool whole = first == r;
  // chunks after this one that begin with r
  int64_t parts = 1;
  for (;; parts += 32) {
    const int64_t at = (c + parts + lane) * chunk;
    const unsigned other = __ballot_sync(0xFFFFFFFFu, at >= a.n || a.sorted[min(at, a.n - 1)].x != r);
    if (other) {
      parts += __ffs(other) - 1;
      break;
    }
  }
  await_previous();
  if (parts == 1 || r >= a.n_rows || (whole && before == r)) return;
  const int64_t per = (parts + kSumWarps - 1) / kSumWarps;
  const int64_t p0 = min(warp * per, parts), p1 = min(p0 + per, parts);
  const int col0 = (int)blockIdx.y * kSumCols;
  float acc[kPer] = {};
#pragma unroll 4
  for (int64_t p = p0; p < p1; ++p) {
    const float* from = a.partial + (2 * (c + p) + (p == 0 && !whole ? 1 : 0)) * a.dim + col0 + lane;
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (col0 + q * 32 + lane < a.dim) acc[q] += __ldcg(from + q * 32);
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q) part[warp][q * 32 + lane] = acc[q];
  __syncthreads();
  constexpr int kOut = kSumCols / (kSumWarps * 32), kW = V < kOut ? V : kOut;
  const int col = threadIdx.x * kOut;
#pragma unroll
  for (int e = 0; e < kOut; e += kW) {
    if (col0 + col + e >= a.dim) break;
    float x[kW];
#pragma unroll
    for (int f = 0; f < kW; ++f) {
      x[f] = part[0][col + e + f];
#pragma unroll
      for (int w = 1; w < kSumWarps; ++w) x[f] += part[w][col + e + f];
    }
    sum_write<TG, TW, kW>(a, r, col0 + col + e, x);
  }
}

// Tokens of a warp of k_emb_sum: as many as leave a block for every SM, at most
// 32 (65,536 tokens took 199 us with 16, which doubles the parts to join).
int emb_run(int64_t n_ids, int64_t groups, int n_sms) {
  int run = kSumMaxRun;
  while (run > kSumMinRun && (n_ids / (kSumWarps * run)) * groups < n_sms) run /= 2;
  return run;
}

// At least chunks * dim for the chunks that emb_run cuts, and never less for
// fewer tokens or columns, so that the workspace of a call is enough for every
// smaller one. Shorter runs, which fewer tokens get, make more chunks: below 32
// tokens a run, twice the run would leave an SM without a block, which bounds
// the chunks of all column groups by 2 n_sms + 3 groups.
int64_t emb_chunk_columns(int64_t n_ids, int64_t dim, int64_t groups, int n_sms) {
  auto chunks = [&](int64_t run) { return (n_ids + kSumWarps * run - 1) / (kSumWarps * run); };
  return std::max(chunks(kSumMaxRun) * dim, std::min(chunks(kSumMinRun) * dim, (2 * n_sms + 3 * groups) * kSumCols));
}

int emb_check(const char* what, bpe_handle* h, const int32_t* ids, int64_t n_ids, const void* rows, int rows_type,
              int64_t n_rows, int64_t dim, int64_t rows_stride, const void* toks, int toks_type, int64_t toks_stride) {
  const std::string name(what);
  if (!h) return fail(BPE_ERR_INVALID_ARG, name + ": null handle");
  if (!type_ok(rows_type) || !type_ok(toks_type)) return fail(BPE_ERR_INVALID_ARG, name + ": unknown type");
  if (n_ids < 0 || n_ids > INT32_MAX - 1024 || n_rows < 0 || n_rows > INT32_MAX - 1024 || dim < 0 || dim > kEmbMaxDim)
    return fail(BPE_ERR_INVALID_ARG, name + ": a size is negative or too large");
  if ((n_ids > 0 && !ids) || (n_rows > 0 && dim > 0 && !rows) || (n_ids > 0 && dim > 0 && !toks))
    return fail(BPE_ERR_INVALID_ARG, name + ": null pointer");
  if (rows_stride < 0 || toks_stride < 0) return fail(BPE_ERR_INVALID_ARG, name + ": negative stride");
  if (!aligned(ids, 4) || !aligned(rows, type_size(rows_type)) || !aligned(toks, type_size(toks_type)))
    return fail(BPE_ERR_INVALID_ARG, name + ": a pointer is not aligned to its elements");
  return BPE_OK;
}

}  // namespace

extern "C" {

int bpe_embed(bpe_handle* h, const int32_t* d_ids, int64_t n_ids, const void* d_weight, int weight_type,
              int64_t n_rows, int64_t dim, int64_t weight_stride, float scale, int32_t skip_id, void* d_out,
              int out_type, int64_t out_stride, bpe_stream_t stream) {
  return guarded("bpe_embed", [&]() -> int {
    int rc = emb_check("bpe_embed", h, d_ids, n_ids, d_weight, weight_type, n_rows, dim, weight_stride, d_out,
                       out_type, out_stride);
    if (rc) return rc;
    if (n_ids > 1 && out_stride < dim) return fail(BPE_ERR_INVALID_ARG, "bpe_embed: output rows overlap");
    if (n_ids == 0 || dim == 0) return BPE_OK;
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    return with_type(weight_type, [&](auto w) {
      return with_type(out_type, [&](auto o) -> int {
        using TW = decltype(w);
        using TO = decltype(o);
        auto launch = [&](auto width) {
          constexpr int V = decltype(width)::value;
          const int64_t vecs = dim / V;
          int tx_log2 = 0;
          while ((1 << tx_log2) < kEmbThreads && (1 << tx_log2) < vecs) ++tx_log2;
          const int64_t tokens = kEmbRows * (kEmbThreads >> tx_log2);
          const int64_t blocks = (n_ids + tokens - 1) / tokens;
          // few tokens: several blocks share their columns
          const int64_t steps = (vecs + (1 << tx_log2) - 1) >> tx_log2;
          const int64_t share = std::max<int64_t>(1, std::min<int64_t>(steps, 2 * h->n_sms / blocks));
          k_embed<TW, TO, V><<<dim3((unsigned)blocks, (unsigned)std::min<int64_t>(share, 65535)), kEmbThreads, 0, st>>>(
              d_ids, n_ids, static_cast<const TW*>(d_weight), n_rows, (int)dim, weight_stride, scale, skip_id,
              static_cast<TO*>(d_out), out_stride, tx_log2, h->d_small);
        };
        auto fits = [&](int64_t V) {
          return dim % V == 0 && vec_ok(d_weight, weight_stride, sizeof(TW), V) &&
                 vec_ok(d_out, out_stride, sizeof(TO), V);
        };
        if (fits(8)) launch(std::integral_constant<int, 8>{});
        else if (fits(2)) launch(std::integral_constant<int, 2>{});
        else launch(std::integral_constant<int, 1>{});
        CK(cudaGetLastError());
        return BPE_OK;
      });
    });
  });
}

int bpe_embed_grad(bpe_handle* h, const int32_t* d_ids, int64_t n_ids, const void* d_grad_out, int grad_out_type,
                   int64_t grad_out_stride, float scale, int32_t skip_id, int64_t n_rows, int64_t dim,
                   void* d_grad_weight, int grad_weight_type, int64_t grad_weight_stride, int accumulate,
                   bpe_stream_t stream) {
  return guarded("bpe_embed_grad", [&]() -> int {
    int rc = emb_check("bpe_embed_grad", h, d_ids, n_ids, d_grad_weight, grad_weight_type, n_rows, dim,
                       grad_weight_stride, d_grad_out, grad_out_type, grad_out_stride);
    if (rc) return rc;
    if (n_rows > 1 && grad_weight_stride < dim) return fail(BPE_ERR_INVALID_ARG, "bpe_embed_grad: output rows overlap");
    if (n_rows == 0 || dim == 0) return BPE_OK;
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t groups = (dim + kSumCols - 1) / kSumCols;
    const int run = emb_run(n_ids, groups, h->n_sms);
    const int64_t chunk = kSumWarps * run, n_chunks = (n_ids + chunk - 1) / chunk;
    // The single launch's rank takes n^2 / 1,024 steps of a thread; placing by
    // rank counts all keys in every block, n / 512 steps of a thread, which
    // shared memory bounds too (8 us against the sort's 18 at 9,001).
    const bool small = n_ids <= kSmallTokens && (n_rows < kSmallRows || n_ids == 0);
    const bool rank = !small && n_ids <= kRankTokens && (n_rows + 1) * n_ids < (1ll << 32);
    uint2* ping[2] = {nullptr, nullptr};
    float* partial = nullptr;
    if (!small) {  // the single launch orders its tokens in shared memory and joins no parts
      const size_t pair = align256((size_t)n_ids * 8);
      const size_t parts = (size_t)emb_chunk_columns(n_ids, dim, groups, h->n_sms) * 2 * sizeof(float);
      rc = ensure_ws(h, 2 * pair + parts, st);
      if (rc) return rc;
      unsigned char* ws = static_cast<unsigned char*>(h->d_ws);
      ping[0] = reinterpret_cast<uint2*>(ws);
      ping[1] = reinterpret_cast<uint2*>(ws + pair);
      partial = reinterpret_cast<float*>(ws + 2 * pair);
    }
    FillArgs f{};
    f.ids = d_ids;
    f.n = n_ids;
    f.n_rows = n_rows;
    f.skip_id = skip_id;
    f.out = static_cast<unsigned char*>(d_grad_weight);
    f.element = (int)type_size(grad_weight_type);
    f.row_bytes = dim * f.element;
    f.stride_bytes = grad_weight_stride * f.element;
    const int ctas = n_ids <= 2048 ? 1 : kSortCluster;  // of a sort, where a few tokens' rows are too many to rank
    // Zeros beside the kernels that find and sum the tokens, fewer blocks where
    // each would have under 32 KB to write. Where they take longer than the
    // sort they go on a stream of their own, so that the sums need not wait
    // for them; that costs four calls on the host, 5 us (where tokens are
    // placed by rank it would gain 1: 31.9 us against 32.8 for 9,001 tokens).
    const bool aside = !small && !rank && !accumulate && n_rows * f.row_bytes >= (64ll << 20);
    int64_t fillers = 0;
    if (!accumulate) {
      // more blocks even out the SMs' rates, but each reads all ids
      const int64_t most = small ? 8 * h->n_sms : 2 * (rank || aside ? h->n_sms : h->n_sms - ctas);
      fillers = std::min<int64_t>(most, std::max<int64_t>(1, n_rows * f.row_bytes / 32768));
      f.row_step = std::min<int64_t>(kFillRows, (n_rows + fillers - 1) / fillers);
    }
    int passes = 1;
    if (aside) {
      if (!h->s_side) {
        int low = 0, high = 0;
        CK(cudaDeviceGetStreamPriorityRange(&low, &high));
        CK(cudaStreamCreateWithPriority(&h->s_side, cudaStreamNonBlocking, low));
      }
      if (!h->ev_fork) CK(cudaEventCreateWithFlags(&h->ev_fork, cudaEventDisableTiming));
      if (!h->ev_join) CK(cudaEventCreateWithFlags(&h->ev_join, cudaEventDisableTiming));
      CK(cudaEventRecord(h->ev_fork, st));
    }
    if (rank) {
      int shift = 0;
      while (n_rows >> shift >= kRankBuckets) ++shift;
      const RankArgs q{d_ids, (int)n_ids, (uint32_t)n_rows, (uint32_t)n_ids, skip_id, shift, ping[0], h->d_small};
      rc = once_per_device(h->device, [] {
        return cudaFuncSetAttribute(k_emb_rank, cudaFuncAttributeMaxDynamicSharedMemorySize, kRankTokens * 4);
      });
      if (rc) return rc;
      k_emb_rank<<<(unsigned)((n_ids + kRankOwn - 1) / kRankOwn), kRankThreads, (size_t)n_ids * 4, st>>>(q);
      CK(cudaGetLastError());
    } else if (!small) {
      SortArgs q{};
      q.ids = d_ids;
      q.n = n_ids;
      q.n_rows = n_rows;
      q.skip_id = skip_id;
      int bits = 1;
      while (n_rows >> bits) ++bits;
      passes = q.passes = (bits + kSortMaxBits - 1) / kSortMaxBits;
      q.bits = (bits + q.passes - 1) / q.passes;
      q.per_warp = (n_ids + ctas * kSortThreads - 1) / (ctas * kSortThreads) * 32;
      q.ping[0] = ping[0];
      q.ping[1] = ping[1];
      q.small = h->d_small;
      rc = once_per_device(h->device, [] {
        cudaError_t e = cudaFuncSetAttribute(k_emb_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             ((kSortWarps + 2) * (1 << kSortMaxBits) + kSortWarps) * 4);
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(k_emb_sort, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      });
      if (rc) return rc;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3((unsigned)ctas);
      cfg.blockDim = dim3(kSortThreads);
      cfg.dynamicSmemBytes = ((size_t)(kSortWarps + 2) * (1 << q.bits) + kSortWarps) * 4;
      cfg.stream = st;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)ctas;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      CK(cudaLaunchKernelEx(&cfg, k_emb_sort, q));
    }
    if (aside) {
      CK(cudaStreamWaitEvent(h->s_side, h->ev_fork, 0));
      k_emb_fill<<<(unsigned)fillers, kFillThreads, 0, h->s_side>>>(f);
      CK(cudaGetLastError());
      CK(cudaEventRecord(h->ev_join, h->s_side));
    } else if (fillers && !small) {
      CK(launch_after(k_emb_fill, dim3((unsigned)fillers), kFillThreads, 0, st, f));
    }
    if (n_chunks + fillers == 0) return BPE_OK;
    return with_type(grad_out_type, [&](auto g_) {
      return with_type(grad_weight_type, [&](auto w) -> int {
        using TG = decltype(g_);
        using TW = decltype(w);
        const SumArgs<TG, TW> a{ping[(passes - 1) & 1], n_ids, n_rows, static_cast<const TG*>(d_grad_out),
                                grad_out_stride, scale, (int)dim, run, static_cast<TW*>(d_grad_weight),
                                grad_weight_stride, accumulate, partial};
        auto launch = [&](auto width) {
          constexpr int V = decltype(width)::value;
          constexpr size_t kSmem = kSumWarps * kSumRing, kSmallSmem = std::max(kSmem, sizeof(FillSmem));
          constexpr int kSlot = kSumCols * (int)sizeof(TG) + (V * sizeof(TG) == 16 ? 0 : 16);
          const size_t smem = kSumWarps * (size_t)std::min(kSumRing / kSlot, run) * kSlot;
          int rc = once_per_device(h->device, [=] {
            cudaError_t e = cudaFuncSetAttribute(k_emb_sum<TG, TW, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)kSmem);
            if (e != cudaSuccess) return e;
            return cudaFuncSetAttribute(k_emb_small<TG, TW, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)kSmallSmem);
          });
          if (rc) return rc;
          const dim3 grid((unsigned)n_chunks, (unsigned)groups);
          if (small) {
            k_emb_small<TG, TW, V><<<dim3((unsigned)(n_chunks + fillers), (unsigned)groups), kSumWarps * 32,
                                     kSmallSmem, st>>>(a, f, n_chunks, h->d_small);
            CK(cudaGetLastError());
          } else {
            CK(launch_after(k_emb_sum<TG, TW, V>, grid, kSumWarps * 32, smem, st, a));
          }
          if (n_chunks > 1 && !small) CK(launch_after(k_emb_join<TG, TW, V>, grid, kSumWarps * 32, 0, st, a));
          if (aside) CK(cudaStreamWaitEvent(st, h->ev_join, 0));
          return (int)BPE_OK;
        };
        auto fits = [&](int64_t V) {
          return dim % V == 0 && vec_ok(d_grad_out, grad_out_stride, sizeof(TG), V) &&
                 vec_ok(d_grad_weight, grad_weight_stride, sizeof(TW), V);
        };
        constexpr int kWide = 16 / (int)sizeof(TG);
        if (fits(kWide)) return launch(std::integral_constant<int, kWide>{});
        return launch(std::integral_constant<int, 1>{});
      });
    });
  });
}

}  // extern "C"
