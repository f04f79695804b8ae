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

constexpr int kEmbThreads = 256;
constexpr int64_t kEmbMaxDim = 1 << 22;  // columns of a block times the grid's limit

__device__ __forceinline__ bool emb_row_ok(int32_t id, int64_t n_rows) { return id >= 0 && id < n_rows; }

// ---------------------------------------------------------------- lookup --

// A block takes rows of tokens x tx threads: each thread holds kEmbRows tokens'
// vectors of V elements in flight at one column and walks the columns in steps
// of tx vectors.
constexpr int kEmbRows = 4;

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

// ------------------------------------------------------------------ sort --

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBits = 10;  // a bin for each thread
constexpr int kSortCluster = 16;

struct SortArgs {
  const int32_t* ids;
  int64_t n, n_rows;
  int32_t skip_id;
  int passes, bits;       // passes of `bits` bits each, lowest first
  int64_t per_warp;       // tokens of a warp, a multiple of 32
  uint2* ping[2];         // (key, token) between passes
  int32_t *key, *pos;     // the sorted keys and tokens
  int32_t* row_start;     // [n_rows + 1]
  DevSmall* small;
};

// Tokens sorted by row, equal rows in token order: a counting sort by `bits`
// bits a pass, by the CTAs of one cluster. Tokens without a row (skip_id, and
// ids out of range, which are reported) get the key n_rows and sort last.
// row_start[r] is the first sorted place whose key is at least r.
//
// A pass: each warp counts the digits of its run of tokens in its own bins;
// the bins' prefix over warps, over the cluster's CTAs (read through
// distributed shared memory) and over digits gives each warp its first place
// for each digit; then the warp walks its run again, 32 tokens at a time, and
// a match of equal digits ranks them in token order.
__global__ void __launch_bounds__(kSortThreads) k_emb_sort(SortArgs a) {
  extern __shared__ int32_t sort_smem[];
  const int bins = 1 << a.bits;
  int32_t* hist = sort_smem;                       // [kSortWarps][bins]
  int32_t* total = hist + kSortWarps * bins;       // [bins]: of this CTA
  int32_t* base = total + bins;                    // [bins]: this CTA's first place
  int32_t* start = base + bins;                    // [bins + 1]: the cluster's first place
  int32_t* warp_sum = start + bins + 1;            // [kSortWarps]
  cg::cluster_group cluster = cg::this_cluster();
  const int n_ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = ((int64_t)rank * kSortWarps + warp) * a.per_warp;
  const int64_t last = min(first + a.per_warp, a.n);
  int32_t* mine = hist + warp * bins;
  for (int p = 0; p < a.passes; ++p) {
    const int shift = p * a.bits;
    const uint2* from = a.ping[(p + 1) & 1];
    const bool final_pass = p + 1 == a.passes;
    auto token = [&](int64_t i) -> uint2 {
      if (p > 0) return __ldcg(from + i);
      const int32_t id = __ldg(a.ids + i);
      const bool ok = id != a.skip_id && emb_row_ok(id, a.n_rows);
      if (!ok && id != a.skip_id) atomicOr(&a.small->op_status, kStBadInput);
      return make_uint2(ok ? (uint32_t)id : (uint32_t)a.n_rows, (uint32_t)i);
    };
    for (int b = tid; b < kSortWarps * bins; b += kSortThreads) hist[b] = 0;
    __syncthreads();
#pragma unroll 4
    for (int64_t i = first + lane; i < last; i += 32) atomicAdd(&mine[(token(i).x >> shift) & (bins - 1)], 1);
    __syncthreads();
    if (tid < bins) {
      int32_t sum = 0;
#pragma unroll 8
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
      for (int r = 0; r < n_ctas; ++r) {
        const int32_t v = *cluster.map_shared_rank(total + tid, r);
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
    if (tid < bins) {
      start[tid] = upto - all;
      base[tid] = upto - all + lower;
      if (tid == bins - 1) start[bins] = upto;
    }
    __syncthreads();
    for (int64_t i0 = first; i0 < last; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool have = i < last;
      const uint2 t = have ? token(i) : make_uint2(0, 0);
      const int digit = have ? (int)((t.x >> shift) & (uint32_t)(bins - 1)) : bins;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, digit);
      const int leader = __ffs(same) - 1;
      int32_t before = 0;
      if (have && lane == leader) before = atomicAdd(&mine[digit], __popc(same));
      before = __shfl_sync(0xFFFFFFFFu, before, leader);
      if (have) {
        const int32_t to = base[digit] + before + __popc(same & ((1u << lane) - 1));
        if (final_pass) {
          a.key[to] = (int32_t)t.x;
          a.pos[to] = (int32_t)t.y;
        } else {
          a.ping[p & 1][to] = t;
        }
      }
    }
    cluster.sync();
  }
  // Each row's first place, in the range of its last digit; a thread's rows
  // step together, so that their loads overlap.
  const int shift = (a.passes - 1) * a.bits;
  constexpr int kRows = 8;
  const int64_t threads = (int64_t)n_ctas * kSortThreads;
  for (int64_t r0 = (int64_t)rank * kSortThreads + tid; r0 <= a.n_rows; r0 += kRows * threads) {
    int32_t lo[kRows], hi[kRows];
    bool more = false;
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const int64_t r = r0 + q * threads;
      const int64_t d = r >> shift;
      lo[q] = r <= a.n_rows ? start[d] : 0;
      hi[q] = r <= a.n_rows && shift > 0 ? start[d + 1] : lo[q];
      more |= lo[q] < hi[q];
    }
    while (more) {
      more = false;
      int32_t k[kRows];
#pragma unroll
      for (int q = 0; q < kRows; ++q)
        if (lo[q] < hi[q]) k[q] = __ldcg(a.key + lo[q] + ((hi[q] - lo[q]) >> 1));
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        if (lo[q] < hi[q]) {
          const int32_t mid = lo[q] + ((hi[q] - lo[q]) >> 1);
          if (k[q] < r0 + q * threads) lo[q] = mid + 1;
          else hi[q] = mid;
        }
        more |= lo[q] < hi[q];
      }
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q)
      if (r0 + q * threads <= a.n_rows) a.row_start[r0 + q * threads] = lo[q];
  }
}

// ------------------------------------------------------------------- sum --

constexpr int kSumWarps = 8;
constexpr int kSumSlabs = 4;    // a lane holds this many vectors of a row
constexpr int kSumAlone = 16;   // a row of up to this many tokens is one warp's
constexpr int kSumChunk = 128;  // a row of up to this many is one block's; longer ones are cut at its multiples

template <class TG, class TW>
struct SumArgs {
  const int32_t *key, *pos, *row_start;
  int64_t n, n_rows;
  const TG* grad;
  int64_t grad_stride;
  float scale;
  int dim;
  TW* out;
  int64_t out_stride;
  int accumulate;
  float* partial;  // [chunks][2][dim]: what a chunk adds to a long row that it begins in, and to one that begins in it
  int64_t n_chunks;
};

// acc[s] += the vectors of tokens pos[j0 .. j1) at column col + s * 32 * V.
template <class TG, int V>
__device__ __forceinline__ void sum_tokens(float (&acc)[kSumSlabs][V], const int32_t* pos, int32_t j0, int32_t j1,
                                           const TG* grad, int64_t stride, int col, int dim) {
  for (int32_t j = j0; j < j1; j += 2) {
    const bool two = j + 1 < j1;
    const TG* g0 = grad + (int64_t)__ldg(pos + j) * stride + col;
    const TG* g1 = grad + (int64_t)__ldg(pos + (two ? j + 1 : j)) * stride + col;
    Vec<TG, V> a[kSumSlabs], b[kSumSlabs];
#pragma unroll
    for (int s = 0; s < kSumSlabs; ++s)
      if (col + s * 32 * V < dim) {
        a[s].load(g0 + s * 32 * V);
        if (two) b[s].load(g1 + s * 32 * V);
      }
#pragma unroll
    for (int s = 0; s < kSumSlabs; ++s)
      if (col + s * 32 * V < dim) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          acc[s][e] += to_f32(a[s].x[e]);
          if (two) acc[s][e] += to_f32(b[s].x[e]);
        }
      }
  }
}

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

// The block's warps share the tokens pos[j0 .. j1); write(col, x) gets the
// sums of V columns, added in warp order.
template <class TG, int V, class W>
__device__ __forceinline__ void sum_by_block(float* smem, const int32_t* pos, int32_t j0, int32_t j1, const TG* grad,
                                             int64_t stride, int col0, int dim, W write) {
  constexpr int kCols = kSumSlabs * 32 * V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t per = (j1 - j0 + kSumWarps - 1) / kSumWarps;
  float acc[kSumSlabs][V] = {};
  sum_tokens<TG, V>(acc, pos, min(j0 + warp * per, j1), min(j0 + (warp + 1) * per, j1), grad, stride,
                    col0 + lane * V, dim);
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kSumSlabs; ++s)
#pragma unroll
    for (int e = 0; e < V; ++e) smem[warp * kCols + (s * V + e) * 32 + lane] = acc[s][e];
  __syncthreads();
  for (int v = threadIdx.x; v < kSumSlabs * 32; v += kSumWarps * 32) {
    const int s = v >> 5, l = v & 31, col = col0 + (s * 32 + l) * V;
    if (col >= dim) continue;
    float x[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[e] = smem[(s * V + e) * 32 + l];
#pragma unroll
      for (int w = 1; w < kSumWarps; ++w) x[e] += smem[w * kCols + (s * V + e) * 32 + l];
    }
    write(col, x);
  }
}

// Blocks [0, n_chunks): the parts of long rows in a chunk of kSumChunk sorted
// places. The others: 8 rows each, far apart, so that frequent rows that are
// neighbours meet different blocks.
template <class TG, class TW, int V>
__global__ void __launch_bounds__(kSumWarps * 32) k_emb_sum(SumArgs<TG, TW> a) {
  __shared__ float smem[kSumWarps * kSumSlabs * 32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col0 = (int)blockIdx.y * kSumSlabs * 32 * V;
  if (blockIdx.x < a.n_chunks) {
    const int64_t c0 = (int64_t)blockIdx.x * kSumChunk, c1 = min(c0 + kSumChunk, a.n);
    const int32_t ra = a.key[c0], rb = a.key[c1 - 1];
    for (int part = 0; part < 2; ++part) {
      const int32_t r = part ? rb : ra;
      if (r >= a.n_rows || (part && ra == rb)) continue;
      const int32_t s = a.row_start[r], e = a.row_start[r + 1];
      if (e - s <= kSumChunk) continue;
      float* to = a.partial + (2 * (int64_t)blockIdx.x + part) * a.dim;
      sum_by_block<TG, V>(smem, a.pos, (int32_t)max((int64_t)s, c0), (int32_t)min((int64_t)e, c1), a.grad,
                          a.grad_stride, col0, a.dim, [&](int col, const float* x) {
#pragma unroll
                            for (int q = 0; q < V; ++q) to[col + q] = x[q];
                          });
    }
    return;
  }
  const int64_t blocks = gridDim.x - a.n_chunks, block = blockIdx.x - a.n_chunks;
  __shared__ int32_t row_from[kSumWarps], row_to[kSumWarps];
  const int64_t r = warp * blocks + block;
  int32_t s = 0, e = 0;
  if (r < a.n_rows) {
    s = a.row_start[r];
    e = a.row_start[r + 1];
  }
  if (lane == 0) {
    row_from[warp] = s;
    row_to[warp] = e;
  }
  if (r < a.n_rows && e - s <= kSumAlone && !(s == e && a.accumulate)) {
    const int col = col0 + lane * V;
    float acc[kSumSlabs][V] = {};
    sum_tokens<TG, V>(acc, a.pos, s, e, a.grad, a.grad_stride, col, a.dim);
#pragma unroll
    for (int q = 0; q < kSumSlabs; ++q)
      if (col + q * 32 * V < a.dim) sum_write<TG, TW, V>(a, r, col + q * 32 * V, acc[q]);
  }
  __syncthreads();
  for (int w = 0; w < kSumWarps; ++w) {
    const int32_t len = row_to[w] - row_from[w];
    if (len <= kSumAlone || len > kSumChunk) continue;
    const int64_t row = w * blocks + block;
    sum_by_block<TG, V>(smem, a.pos, row_from[w], row_to[w], a.grad, a.grad_stride, col0, a.dim,
                        [&](int col, const float* x) { sum_write<TG, TW, V>(a, row, col, x); });
  }
}

// The parts of a long row, joined in order by the block of the chunk that it
// begins in.
template <class TG, class TW, int V>
__global__ void __launch_bounds__(kSumWarps * 32) k_emb_join(SumArgs<TG, TW> a) {
  __shared__ float smem[kSumWarps * kSumSlabs * 32 * V];
  constexpr int kCols = kSumSlabs * 32 * V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col0 = (int)blockIdx.y * kCols;
  const int64_t c = blockIdx.x, c0 = c * kSumChunk;
  const int32_t r = a.key[min(c0 + kSumChunk, a.n) - 1];
  if (r >= a.n_rows) return;
  const int64_t s = a.row_start[r], e = a.row_start[r + 1];
  if (e - s <= kSumChunk || s < c0) return;
  const int64_t parts = (e - 1) / kSumChunk - c + 1;
  const int64_t per = (parts + kSumWarps - 1) / kSumWarps;
  const int64_t p0 = min(warp * per, parts), p1 = min(p0 + per, parts);
  float acc[kSumSlabs * V] = {};
#pragma unroll 4
  for (int64_t p = p0; p < p1; ++p) {
    const float* from = a.partial + (2 * (c + p) + (p == 0 && s > c0 ? 1 : 0)) * a.dim + col0;
#pragma unroll
    for (int q = 0; q < kSumSlabs * V; ++q)
      if (col0 + q * 32 + lane < a.dim) acc[q] += __ldcs(from + q * 32 + lane);
  }
#pragma unroll
  for (int q = 0; q < kSumSlabs * V; ++q) smem[warp * kCols + q * 32 + lane] = acc[q];
  __syncthreads();
  for (int col = threadIdx.x; col < kCols && col0 + col < a.dim; col += kSumWarps * 32) {
    float x = smem[col];
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w) x += smem[w * kCols + col];
    sum_write<TG, TW, 1>(a, r, col0 + col, &x);
  }
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
          k_embed<TW, TO, V><<<(unsigned)blocks, kEmbThreads, 0, st>>>(
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
    SortArgs q{};
    q.ids = d_ids;
    q.n = n_ids;
    q.n_rows = n_rows;
    q.skip_id = skip_id;
    q.small = h->d_small;
    int bits = 1;
    while (n_rows >> bits) ++bits;
    q.passes = (bits + kSortMaxBits - 1) / kSortMaxBits;
    q.bits = (bits + q.passes - 1) / q.passes;
    // One CTA sorts a small batch by itself; the cluster's barriers cost more than it saves.
    const int ctas = n_ids <= 2048 && n_rows <= 8192 ? 1 : kSortCluster;
    q.per_warp = (n_ids + ctas * kSortThreads - 1) / (ctas * kSortThreads) * 32;
    const int64_t n_chunks = (n_ids + kSumChunk - 1) / kSumChunk;
    const size_t pair = align256((size_t)n_ids * 8), list = align256((size_t)n_ids * 4),
                 rows = align256((size_t)(n_rows + 1) * 4), parts = align256((size_t)n_chunks * 2 * (size_t)dim * 4);
    rc = ensure_ws(h, 2 * pair + 2 * list + rows + parts);
    if (rc) return rc;
    unsigned char* ws = static_cast<unsigned char*>(h->d_ws);
    q.ping[0] = reinterpret_cast<uint2*>(ws);
    q.ping[1] = reinterpret_cast<uint2*>(ws + pair);
    q.key = reinterpret_cast<int32_t*>(ws + 2 * pair);
    q.pos = reinterpret_cast<int32_t*>(ws + 2 * pair + list);
    q.row_start = reinterpret_cast<int32_t*>(ws + 2 * pair + 2 * list);
    float* partial = reinterpret_cast<float*>(ws + 2 * pair + 2 * list + rows);
    const size_t smem = ((size_t)(kSortWarps + 3) * (1 << q.bits) + 1 + kSortWarps) * 4;
    CK(cudaFuncSetAttribute(k_emb_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    CK(cudaFuncSetAttribute(k_emb_sort, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    CK(cudaLaunchKernelEx(&cfg, k_emb_sort, q));
    return with_type(grad_out_type, [&](auto g_) {
      return with_type(grad_weight_type, [&](auto w) -> int {
        using TG = decltype(g_);
        using TW = decltype(w);
        const SumArgs<TG, TW> a{q.key, q.pos, q.row_start, n_ids, n_rows, static_cast<const TG*>(d_grad_out),
                                grad_out_stride, scale, (int)dim, static_cast<TW*>(d_grad_weight),
                                grad_weight_stride, accumulate, partial, n_chunks};
        auto launch = [&](auto width) {
          constexpr int V = decltype(width)::value;
          const unsigned groups = (unsigned)((dim + kSumSlabs * 32 * V - 1) / (kSumSlabs * 32 * V));
          k_emb_sum<TG, TW, V><<<dim3((unsigned)(n_chunks + (n_rows + kSumWarps - 1) / kSumWarps), groups),
                                 kSumWarps * 32, 0, st>>>(a);
          if (n_ids > kSumChunk)
            k_emb_join<TG, TW, V><<<dim3((unsigned)n_chunks, groups), kSumWarps * 32, 0, st>>>(a);
        };
        auto fits = [&](int64_t V) {
          return dim % V == 0 && vec_ok(d_grad_out, grad_out_stride, sizeof(TG), V) &&
                 vec_ok(d_grad_weight, grad_weight_stride, sizeof(TW), V);
        };
        constexpr int kWide = 16 / (int)sizeof(TG), kNarrow = 4 / (int)sizeof(TG);
        if (dim > 32 * kNarrow && fits(kWide)) launch(std::integral_constant<int, kWide>{});
        else if (fits(kNarrow)) launch(std::integral_constant<int, kNarrow>{});
        else launch(std::integral_constant<int, 1>{});
        CK(cudaGetLastError());
        return BPE_OK;
      });
    });
  });
}

}  // extern "C"
