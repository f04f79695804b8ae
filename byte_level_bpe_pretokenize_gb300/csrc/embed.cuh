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

__device__ __forceinline__ bool emb_row_ok(int32_t id, int64_t n_rows) { return id >= 0 && id < n_rows; }

template <class TW, class TO>
__global__ void __launch_bounds__(kEmbThreads) k_embed(const int32_t* ids, int64_t n_ids, const TW* weight,
                                                       int64_t n_rows, int64_t dim, int64_t weight_stride, float scale,
                                                       int32_t skip_id, TO* out, int64_t out_stride, DevSmall* small) {
  for (int64_t i = blockIdx.x; i < n_ids; i += gridDim.x) {
    const int32_t id = ids[i];
    const bool ok = id != skip_id && emb_row_ok(id, n_rows);
    if (!ok && id != skip_id && threadIdx.x == 0) atomicOr(&small->op_status, kStBadInput);
    const TW* w = weight + (ok ? id : 0) * weight_stride;
    TO* o = out + i * out_stride;
    for (int64_t c = threadIdx.x; c < dim; c += kEmbThreads) o[c] = from_f32<TO>(ok ? scale * to_f32(w[c]) : 0.f);
  }
}

// ------------------------------------------------------------------ sort --

constexpr int kSortThreads = 1024;
constexpr int kSortBits = 8;
constexpr int kSortBins = 1 << kSortBits;

// Tokens sorted by row, equal rows in token order: a counting sort by 8 bits
// a pass, lowest first, by one CTA. Tokens without a row (skip_id, and ids out
// of range, which are reported) get the key n_rows and sort last.
// row_start[r] is the first sorted place whose key is at least r.
__global__ void __launch_bounds__(kSortThreads) k_emb_sort(const int32_t* ids, int64_t n, int64_t n_rows,
                                                           int32_t skip_id, int passes, int32_t* key_a, int32_t* pos_a,
                                                           int32_t* key_b, int32_t* pos_b, int32_t* row_start,
                                                           DevSmall* small) {
  constexpr int kWarps = kSortThreads / 32;
  __shared__ int32_t total[kSortBins], base[kSortBins];
  __shared__ uint16_t warp_count[kWarps][kSortBins];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t i = tid; i < n; i += kSortThreads) {
    const int32_t id = ids[i];
    const bool ok = id != skip_id && emb_row_ok(id, n_rows);
    if (!ok && id != skip_id) atomicOr(&small->op_status, kStBadInput);
    key_a[i] = ok ? id : (int32_t)n_rows;
    pos_a[i] = (int32_t)i;
  }
  __syncthreads();
  for (int p = 0; p < passes; ++p) {
    const int shift = p * kSortBits;
    if (tid < kSortBins) total[tid] = 0;
    __syncthreads();
    for (int64_t i = tid; i < n; i += kSortThreads) atomicAdd(&total[(key_a[i] >> shift) & (kSortBins - 1)], 1);
    __syncthreads();
    if (tid == 0) {
      int32_t sum = 0;
      for (int b = 0; b < kSortBins; ++b) {
        base[b] = sum;
        sum += total[b];
      }
    }
    for (int64_t i0 = 0; i0 < n; i0 += kSortThreads) {
      for (int b = tid; b < kWarps * kSortBins; b += kSortThreads) (&warp_count[0][0])[b] = 0;
      __syncthreads();
      const int64_t i = i0 + tid;
      const bool have = i < n;
      const int32_t key = have ? key_a[i] : 0, pos = have ? pos_a[i] : 0;
      const int digit = have ? (key >> shift) & (kSortBins - 1) : kSortBins;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, digit);
      const int rank = __popc(same & ((1u << lane) - 1));
      if (have && rank == 0) warp_count[warp][digit] = (uint16_t)__popc(same);
      __syncthreads();
      if (tid < kSortBins) {
        int32_t sum = base[tid];
        for (int w = 0; w < kWarps; ++w) {
          const int c = warp_count[w][tid];
          warp_count[w][tid] = (uint16_t)(sum - base[tid]);
          sum += c;
        }
        total[tid] = sum;
      }
      __syncthreads();
      if (have) {
        const int64_t to = base[digit] + warp_count[warp][digit] + rank;
        key_b[to] = key;
        pos_b[to] = pos;
      }
      __syncthreads();
      if (tid < kSortBins) base[tid] = total[tid];
    }
    __syncthreads();
    int32_t* t = key_a;
    key_a = key_b;
    key_b = t;
    t = pos_a;
    pos_a = pos_b;
    pos_b = t;
  }
  for (int64_t i = tid; i <= n; i += kSortThreads) {
    const int64_t k0 = i > 0 ? key_a[i - 1] : -1, k1 = i < n ? key_a[i] : n_rows;
    for (int64_t r = k0 + 1; r <= k1; ++r) row_start[r] = (int32_t)i;
  }
}

template <class TG, class TW>
__global__ void __launch_bounds__(kEmbThreads) k_emb_sum(const int32_t* pos, const int32_t* row_start, const TG* grad,
                                                         int64_t grad_stride, float scale, int64_t n_rows, int64_t dim,
                                                         TW* out, int64_t out_stride, int accumulate) {
  for (int64_t r = blockIdx.x; r < n_rows; r += gridDim.x) {
    const int32_t s = row_start[r], e = row_start[r + 1];
    if (s == e && accumulate) continue;
    TW* o = out + r * out_stride;
    for (int64_t c = threadIdx.x; c < dim; c += kEmbThreads) {
      float sum = 0.f;
      for (int32_t j = s; j < e; ++j) sum += to_f32(grad[pos[j] * grad_stride + c]);
      sum *= scale;
      o[c] = from_f32<TW>(accumulate ? to_f32(o[c]) + sum : sum);
    }
  }
}

int emb_check(const char* what, bpe_handle* h, const int32_t* ids, int64_t n_ids, const void* rows, int rows_type,
              int64_t n_rows, int64_t dim, int64_t rows_stride, const void* toks, int toks_type, int64_t toks_stride) {
  const std::string name(what);
  if (!h) return fail(BPE_ERR_INVALID_ARG, name + ": null handle");
  if (!type_ok(rows_type) || !type_ok(toks_type)) return fail(BPE_ERR_INVALID_ARG, name + ": unknown type");
  if (n_ids < 0 || n_ids > INT32_MAX - 1024 || n_rows < 0 || n_rows > INT32_MAX - 1024 || dim < 0 || dim > INT32_MAX)
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
        k_embed<TW, TO><<<(unsigned)std::min<int64_t>(n_ids, 65535), kEmbThreads, 0, st>>>(
            d_ids, n_ids, static_cast<const TW*>(d_weight), n_rows, dim, weight_stride, scale, skip_id,
            static_cast<TO*>(d_out), out_stride, h->d_small);
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
    const size_t list = align256((size_t)n_ids * 4), rows = align256((size_t)(n_rows + 1) * 4);
    rc = ensure_ws(h, 4 * list + rows);
    if (rc) return rc;
    unsigned char* ws = static_cast<unsigned char*>(h->d_ws);
    int32_t* key_a = reinterpret_cast<int32_t*>(ws);
    int32_t* pos_a = reinterpret_cast<int32_t*>(ws + list);
    int32_t* key_b = reinterpret_cast<int32_t*>(ws + 2 * list);
    int32_t* pos_b = reinterpret_cast<int32_t*>(ws + 3 * list);
    int32_t* row_start = reinterpret_cast<int32_t*>(ws + 4 * list);
    int passes = 1;
    while (passes * kSortBits < 32 && (n_rows >> (passes * kSortBits)) != 0) ++passes;
    k_emb_sort<<<1, kSortThreads, 0, st>>>(d_ids, n_ids, n_rows, skip_id, passes, key_a, pos_a, key_b, pos_b,
                                           row_start, h->d_small);
    CK(cudaGetLastError());
    const int32_t* pos = passes % 2 ? pos_b : pos_a;
    return with_type(grad_out_type, [&](auto g_) {
      return with_type(grad_weight_type, [&](auto w) -> int {
        using TG = decltype(g_);
        using TW = decltype(w);
        k_emb_sum<TG, TW><<<(unsigned)std::min<int64_t>(n_rows, 65535), kEmbThreads, 0, st>>>(
            pos, row_start, static_cast<const TG*>(d_grad_out), grad_out_stride, scale, n_rows, dim,
            static_cast<TW*>(d_grad_weight), grad_weight_stride, accumulate);
        CK(cudaGetLastError());
        return BPE_OK;
      });
    });
  });
}

}  // extern "C"
