// Keys and values into the slots of a cache in 4 bits (cache.cuh), and back.
//
// Included once by paged_ops.cu; not a standalone header.

namespace {

constexpr int kCacheThreads = 256;

struct CacheRows {
  const void* in[2];     // keys and values
  void* out[2];
  int64_t token[2], head[2];  // strides in elements
};

// Eight elements of a row from `at` on; those past dim are not there. V is 8
// where they lie in aligned vectors, else 1.
template <class T, int V>
__device__ __forceinline__ int cache_load(const T* row, int at, int dim, float (&x)[8]) {
  const int n = min(8, dim - at);
  if constexpr (V == 8) {
    if (n <= 0) return 0;
    Vec<T, 8> v;
    v.load(row + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = to_f32(v.x[e]);
    return 8;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = e < n ? to_f32(row[at + e]) : 0.f;
    return max(n, 0);
  }
}

// A thread quantises 8 elements of a key and of a value, four threads a group.
// Halves of the elements are subtracted, for the difference of two finite ones
// may pass the largest float, and multiplied by the step's reciprocal, one
// division a group.
template <class T, int V>
__global__ void __launch_bounds__(kCacheThreads) k_cache_write(CacheArgs a, CacheRows r, uint32_t total) {
  const uint32_t index = blockIdx.x * kCacheThreads + threadIdx.x;
  const bool here = index < total;
  const uint32_t line = a.words(here ? index : 0), word = (here ? index : 0) - line * a.words.d;
  const uint32_t token = a.heads(line), h = line - token * a.heads.d;
  const int64_t slot = here ? __ldg(a.slots + token) : -1;
  const bool ok = slot >= 0 && slot < a.n_slots;
  if (here && !ok && slot != -1 && word == 0) atomicOr(&a.small->op_status, kStBadInput);
  float x[2][8];
  int n[2] = {0, 0};
#pragma unroll
  for (int w = 0; w < 2; ++w)
    if (ok)
      n[w] = cache_load<T, V>(static_cast<const T*>(r.in[w]) + token * r.token[w] + h * r.head[w], word * 8, a.dim, x[w]);
  uint32_t row = 0;
  unsigned char* page = a.cache;
  if (ok) page = cache_page(a, slot, h, &row);
  const int j = word >> 2, c = word & 3;
#pragma unroll
  for (int w = 0; w < 2; ++w, page += (int64_t)a.heads.d * a.page_bytes) {
    float low = INFINITY, high = -INFINITY;
    bool lost = false;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n[w]) {
        low = fminf(low, x[w][e]);
        high = fmaxf(high, x[w][e]);
        lost |= !(fabsf(x[w][e]) <= kBf16Max);
      }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
      high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
      lost |= (bool)__shfl_xor_sync(0xFFFFFFFFu, (int)lost, d);
    }
    if (!ok) continue;
    const bool empty = !(low <= high);  // padding behind dim
    __nv_bfloat16 base = __float2bfloat16_rn(empty ? 0.f : low);
    const float half = 0.5f * __bfloat162float(base);
    __nv_bfloat16 step = __float2bfloat16_rn(fmaxf((0.5f * (empty ? 0.f : high) - half) / 7.5f, 0.f));
    if (__bfloat162float(step) < 0x1p-100f) step = __float2bfloat16_rn(0.f);
    const float half_step = 0.5f * __bfloat162float(step), by = half_step > 0.f ? 1.f / half_step : 0.f;
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = fminf(fmaxf(rintf((0.5f * x[w][e] - half) * by), 0.f), 15.f);
      if (e < n[w]) codes |= (uint32_t)q << (4 * e);
    }
    uint32_t pair = (uint32_t)__bfloat16_as_ushort(step) | (uint32_t)__bfloat16_as_ushort(base) << 16;
    if (lost) pair = 0x7FC00000u;
    reinterpret_cast<uint32_t*>(page + (int64_t)row * a.groups * 16)[cache_word(a.groups, j, c)] = codes;
    if (c == 0)
      reinterpret_cast<uint32_t*>(page + ((int64_t)a.block.d * 16 + (int64_t)row * 4) * a.groups)[j] = pair;
  }
}

// A thread reads the words of 8 elements of a key and of a value.
template <class T, int V>
__global__ void __launch_bounds__(kCacheThreads) k_cache_read(CacheArgs a, CacheRows r, uint32_t total) {
  const uint32_t index = blockIdx.x * kCacheThreads + threadIdx.x;
  if (index >= total) return;
  const uint32_t line = a.words(index), word = index - line * a.words.d;
  const uint32_t token = a.heads(line), h = line - token * a.heads.d;
  const int64_t slot = __ldg(a.slots + token);
  const bool ok = slot >= 0 && slot < a.n_slots;
  if (!ok && slot != -1 && word == 0) atomicOr(&a.small->op_status, kStBadInput);
  uint32_t row = 0, codes[2] = {0, 0}, pair[2] = {0, 0};
  if (ok) {
    const unsigned char* page = cache_page(a, slot, h, &row);
#pragma unroll
    for (int w = 0; w < 2; ++w, page += (int64_t)a.heads.d * a.page_bytes) {
      codes[w] = __ldg(reinterpret_cast<const uint32_t*>(page + (int64_t)row * a.groups * 16) +
                       cache_word(a.groups, word >> 2, word & 3));
      pair[w] = __ldg(reinterpret_cast<const uint32_t*>(page + ((int64_t)a.block.d * 16 + (int64_t)row * 4) * a.groups) +
                      (word >> 2));
    }
  }
  const int n = min(8, a.dim - (int)word * 8);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    T* out = static_cast<T*>(r.out[w]) + token * r.token[w] + h * r.head[w] + word * 8;
    const float step = bf16_low(pair[w]), base = bf16_high(pair[w]);
    Vec<T, 8> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.x[e] = from_f32<T>(base + step * (float)((codes[w] >> (4 * e)) & 15));
    if constexpr (V == 8) {
      if (n > 0) v.store(out);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) out[e] = v.x[e];
    }
  }
}

// Runs launch(args, tokens before, total threads) in parts of fewer than 2^31 threads.
template <class F>
int cache_parts(int64_t n_tokens, int64_t n_heads, int64_t words, F launch) {
  const int64_t at_once = std::min(n_tokens, (int64_t)INT32_MAX / 2 / (n_heads * words));
  for (int64_t t = 0; t < n_tokens; t += at_once) {
    launch(t, (uint32_t)(std::min(at_once, n_tokens - t) * n_heads * words));
    CK(cudaGetLastError());
  }
  return BPE_OK;
}

}  // namespace

extern "C" {

int bpe_cache_page_bytes(int64_t block_size, int64_t dim, int64_t* bytes) {
  if (!bytes || block_size < 1 || block_size > BPE_CACHE_MAX_BLOCK || dim < 1 || dim > BPE_CACHE_MAX_DIM)
    return guarded("bpe_cache_page_bytes", [&] {
      return fail(BPE_ERR_INVALID_ARG, "bpe_cache_page_bytes: block_size or dim out of range");
    });
  *bytes = cache_page_bytes(block_size, dim);
  return BPE_OK;
}

int bpe_cache_write(bpe_handle* h, const int64_t* d_slots, int64_t n_tokens, const void* d_keys, const void* d_values,
                    int type, int64_t n_heads, int64_t dim, int64_t key_token_stride, int64_t key_head_stride,
                    int64_t value_token_stride, int64_t value_head_stride, void* d_cache, int64_t n_blocks,
                    int64_t block_stride, int64_t block_size, bpe_stream_t stream) {
  return guarded("bpe_cache_write", [&]() -> int {
    int rc = cache_check("bpe_cache_write", h, d_cache, n_blocks, block_stride, block_size, n_heads, dim);
    if (rc) return rc;
    if (!type_ok(type)) return fail(BPE_ERR_INVALID_ARG, "bpe_cache_write: unknown element type");
    if (n_tokens < 0 || n_tokens >= INT32_MAX || key_token_stride < 0 || key_head_stride < 0 || value_token_stride < 0 ||
        value_head_stride < 0)
      return fail(BPE_ERR_INVALID_ARG, "bpe_cache_write: a size or stride is negative or too large");
    if (n_tokens == 0) return BPE_OK;
    if (!d_slots || !d_keys || !d_values) return fail(BPE_ERR_INVALID_ARG, "bpe_cache_write: null pointer");
    if (!aligned(d_slots, 8) || !aligned(d_keys, type_size(type)) || !aligned(d_values, type_size(type)))
      return fail(BPE_ERR_INVALID_ARG, "bpe_cache_write: a pointer is not aligned to its elements");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t groups = cache_groups(dim), words = groups * 4;
    CacheArgs a{static_cast<unsigned char*>(d_cache), block_stride, cache_page_bytes(block_size, dim),
                n_blocks * block_size, FastDiv(block_size), FastDiv(words), FastDiv(n_heads), (int)groups, (int)dim,
                d_slots, h->d_small};
    CacheRows r{{d_keys, d_values}, {}, {key_token_stride, value_token_stride}, {key_head_stride, value_head_stride}};
    return with_type(type, [&](auto t) -> int {
      using T = decltype(t);
      bool wide = dim % 8 == 0;
      for (int w = 0; w < 2; ++w)
        wide = wide && vec_ok(r.in[w], n_tokens > 1 ? r.token[w] : 0, sizeof(T), 8) &&
               vec_ok(r.in[w], n_heads > 1 ? r.head[w] : 0, sizeof(T), 8);
      return cache_parts(n_tokens, n_heads, words, [&](int64_t from, uint32_t total) {
        CacheArgs b = a;
        b.slots += from;
        CacheRows s = r;
        for (int w = 0; w < 2; ++w) s.in[w] = static_cast<const T*>(r.in[w]) + from * r.token[w];
        const unsigned blocks = (total + kCacheThreads - 1) / kCacheThreads;
        if (wide) k_cache_write<T, 8><<<blocks, kCacheThreads, 0, st>>>(b, s, total);
        else k_cache_write<T, 1><<<blocks, kCacheThreads, 0, st>>>(b, s, total);
      });
    });
  });
}

int bpe_cache_read(bpe_handle* h, const int64_t* d_slots, int64_t n_tokens, const void* d_cache, int64_t n_blocks,
                   int64_t block_stride, int64_t block_size, int64_t n_heads, int64_t dim, void* d_keys,
                   void* d_values, int type, int64_t key_token_stride, int64_t key_head_stride,
                   int64_t value_token_stride, int64_t value_head_stride, bpe_stream_t stream) {
  return guarded("bpe_cache_read", [&]() -> int {
    int rc = cache_check("bpe_cache_read", h, d_cache, n_blocks, block_stride, block_size, n_heads, dim);
    if (rc) return rc;
    if (!type_ok(type)) return fail(BPE_ERR_INVALID_ARG, "bpe_cache_read: unknown element type");
    if (n_tokens < 0 || n_tokens >= INT32_MAX) return fail(BPE_ERR_INVALID_ARG, "bpe_cache_read: a size is negative or too large");
    if (n_tokens == 0) return BPE_OK;
    if (rows_meet(n_tokens, key_token_stride, n_heads, key_head_stride, dim) ||
        rows_meet(n_tokens, value_token_stride, n_heads, value_head_stride, dim))
      return fail(BPE_ERR_INVALID_ARG, "bpe_cache_read: output rows overlap");
    if (!d_slots || !d_keys || !d_values) return fail(BPE_ERR_INVALID_ARG, "bpe_cache_read: null pointer");
    if (!aligned(d_slots, 8) || !aligned(d_keys, type_size(type)) || !aligned(d_values, type_size(type)))
      return fail(BPE_ERR_INVALID_ARG, "bpe_cache_read: a pointer is not aligned to its elements");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t groups = cache_groups(dim), words = (dim + 7) / 8;
    CacheArgs a{static_cast<unsigned char*>(const_cast<void*>(d_cache)), block_stride,
                cache_page_bytes(block_size, dim), n_blocks * block_size, FastDiv(block_size), FastDiv(words),
                FastDiv(n_heads), (int)groups, (int)dim, d_slots, h->d_small};
    CacheRows r{{}, {d_keys, d_values}, {key_token_stride, value_token_stride}, {key_head_stride, value_head_stride}};
    return with_type(type, [&](auto t) -> int {
      using T = decltype(t);
      bool wide = dim % 8 == 0;
      for (int w = 0; w < 2; ++w)
        wide = wide && vec_ok(r.out[w], n_tokens > 1 ? r.token[w] : 0, sizeof(T), 8) &&
               vec_ok(r.out[w], n_heads > 1 ? r.head[w] : 0, sizeof(T), 8);
      return cache_parts(n_tokens, n_heads, words, [&](int64_t from, uint32_t total) {
        CacheArgs b = a;
        b.slots += from;
        CacheRows s = r;
        for (int w = 0; w < 2; ++w) s.out[w] = static_cast<T*>(r.out[w]) + from * r.token[w];
        const unsigned blocks = (total + kCacheThreads - 1) / kCacheThreads;
        if (wide) k_cache_read<T, 8><<<blocks, kCacheThreads, 0, st>>>(b, s, total);
        else k_cache_read<T, 1><<<blocks, kCacheThreads, 0, st>>>(b, s, total);
      });
    });
  });
}

}  // extern "C"
