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

// The smallest and the largest of numbers: as halves of one word (the second
// negative, so that both are minima), or as floats. A NaN spoils both.
__device__ __forceinline__ float min_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
template <class T>
struct Span;
template <>
struct Span<float> {
  float low = INFINITY, minus_high = INFINITY;
  __device__ __forceinline__ void add(const float* x) {  // two of them
    low = min_nan(low, min_nan(x[0], x[1]));
    minus_high = min_nan(minus_high, min_nan(-x[0], -x[1]));
  }
  __device__ __forceinline__ void close() {}
  __device__ __forceinline__ void meet_lane(int d) {
    low = min_nan(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
    minus_high = min_nan(minus_high, __shfl_xor_sync(0xFFFFFFFFu, minus_high, d));
  }
  __device__ __forceinline__ float2 ends() const { return make_float2(low, -minus_high); }
};
template <class T, class T2>
struct SpanOfTwo {
  T2 low, high, both;
  __device__ __forceinline__ SpanOfTwo() {
    low.x = low.y = from_f32<T>(INFINITY);
    high = low;
  }
  __device__ __forceinline__ void add(const T* x) {
    const T2 v = *reinterpret_cast<const T2*>(x);
    low = __hmin2_nan(low, v);
    high = __hmin2_nan(high, __hneg2(v));
  }
  __device__ __forceinline__ void close() {
    both.x = __hmin_nan(low.x, low.y);
    both.y = __hmin_nan(high.x, high.y);
  }
  __device__ __forceinline__ void meet_lane(int d) { both = __hmin2_nan(both, __shfl_xor_sync(0xFFFFFFFFu, both, d)); }
  __device__ __forceinline__ float2 ends() const { return make_float2(to_f32(both.x), -to_f32(both.y)); }
};
template <>
struct Span<__half> : SpanOfTwo<__half, __half2> {};
template <>
struct Span<__nv_bfloat16> : SpanOfTwo<__nv_bfloat16, __nv_bfloat162> {};

// Elements of a row that a thread takes: half a group.
constexpr int kCacheTake = 16;

// Whole numbers cut to [0, 15] as codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t pack_codes(const int (&n)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 6; e >= 0; e -= 2)
    asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %3;" : "=r"(w) : "r"(n[e + 1]), "r"(n[e]), "r"(w));
  return w;
}

// The first n of 16 elements from any address on, by the 16-byte granules that
// hold them (what else lies in a granule is read, but not used).
template <class T>
__device__ __forceinline__ void load_granules(T (&x)[kCacheTake], const T* from, int n) {
  constexpr int kBytes = kCacheTake * (int)sizeof(T), kGranules = kBytes / 16 + 1, kWords = kBytes / 4 + 1;
  const uintptr_t at = reinterpret_cast<uintptr_t>(from), first = at & ~(uintptr_t)15, end = at + n * sizeof(T);
  uint32_t w[4 * kGranules + 3];  // three more, so that every choice below has both sides
#pragma unroll
  for (int g = 0; g < kGranules; ++g) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (first + 16 * g < end) v = __ldcs(reinterpret_cast<const uint4*>(first) + g);
    w[4 * g] = v.x, w[4 * g + 1] = v.y, w[4 * g + 2] = v.z, w[4 * g + 3] = v.w;
  }
#pragma unroll
  for (int i = 4 * kGranules; i < 4 * kGranules + 3; ++i) w[i] = 0;
  const bool one = at & 4, two = at & 8;
#pragma unroll
  for (int i = 0; i < kWords + 2; ++i) w[i] = one ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < kWords; ++i) w[i] = two ? w[i + 2] : w[i];
  const uint32_t select = at & 2 ? 0x5432 : 0x3210;
#pragma unroll
  for (int i = 0; i < kBytes / 4; ++i) {
    const uint32_t v = sizeof(T) == 2 ? __byte_perm(w[i], w[i + 1], select) : w[i];
    reinterpret_cast<uint32_t*>(x)[i] = v;
  }
}

// 16 halves to any address, in words where they lie in them.
template <class T>
__device__ __forceinline__ void store_words(T* to, const T (&x)[kCacheTake]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
  if (reinterpret_cast<uintptr_t>(to) & 2) {
    to[0] = x[0];
#pragma unroll
    for (int i = 0; i < kCacheTake / 2 - 1; ++i)
      __stcs(reinterpret_cast<unsigned int*>(to + 1) + i, __byte_perm(w[i], w[i + 1], 0x5432));
    to[kCacheTake - 1] = x[kCacheTake - 1];
  } else {
#pragma unroll
    for (int i = 0; i < kCacheTake / 2; ++i) __stcs(reinterpret_cast<unsigned int*>(to) + i, w[i]);
  }
}

// A thread quantises 16 elements of a key and of a value, two threads a group.
// Halves of the elements are subtracted, for the difference of two finite ones
// may pass the largest float, and multiplied by the step's reciprocal, the
// one division of a group. Rounding is an addition: below 2^22 the lowest bits of
// x + 1.5 2^23 are the whole number next to x, ties to even. (|x| stays below
// 2^20: the base is at most 2^-9 of an element above it, the step at least
// 2^-24 of one over 15.) V is 8 where elements lie in aligned vectors, else 1.
//
// Bound by issue: 84% of the slots, 12 instructions an element. 131,072 tokens of
// 8 x 128 in bf16 take 143 us, 4.9 TB/s. With 8 elements a thread, four threads a
// group, what is done once a group took as long as all else: 332 us.
template <class T, int V>
__global__ void __launch_bounds__(kCacheThreads) k_cache_write(CacheArgs a, CacheRows r, uint32_t total) {
  const uint32_t index = blockIdx.x * kCacheThreads + threadIdx.x;
  const bool here = index < total;
  const uint32_t line = a.parts(here ? index : 0), part = (here ? index : 0) - line * a.parts.d;
  const uint32_t token = a.heads(line), h = line - token * a.heads.d;
  const int64_t slot = here ? __ldg(a.slots + token) : -1;
  const bool ok = slot >= 0 && slot < a.n_slots;
  if (here && !ok && slot != -1 && part == 0) atomicOr(&a.small->op_status, kStBadInput);
  const int at = part * kCacheTake, n = ok ? min(kCacheTake, a.dim - at) : 0;
  __align__(16) T x[2][kCacheTake];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const T* row = static_cast<const T*>(r.in[w]) + token * r.token[w] + h * r.head[w] + at;
    if constexpr (V == 8) {
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (v * 8 < n) reinterpret_cast<Vec<T, 8>*>(x[w])[v].load(row + v * 8);
    } else if (n > 0) {
      load_granules(x[w], row, n);
    }
  }
  uint32_t row = 0;
  unsigned char* page = a.cache;
  if (ok) page = cache_page(a, slot, h, &row);
  const int j = part >> 1, c = part & 1;
#pragma unroll
  for (int w = 0; w < 2; ++w, page += (int64_t)a.heads.d * a.page_bytes) {
    // what is not there does as the first element does
    if (n > 0 && n < kCacheTake) {
#pragma unroll
      for (int e = 1; e < kCacheTake; ++e)
        if (e >= n) x[w][e] = x[w][0];
    }
    Span<T> span;
    if (n > 0) {
#pragma unroll
      for (int e = 0; e < kCacheTake; e += 2) span.add(x[w] + e);
    }
    span.close();
    span.meet_lane(1);
    if (!ok) continue;
    const float2 ends = span.ends();
    const bool empty = n <= 0 && ends.x == INFINITY && ends.y == -INFINITY;  // padding behind dim
    const bool lost = !empty && !(fabsf(ends.x) <= kBf16Max && fabsf(ends.y) <= kBf16Max);
    const __nv_bfloat16 base = __float2bfloat16_rn(empty ? 0.f : ends.x);
    const float half = 0.5f * __bfloat162float(base);
    __nv_bfloat16 step = __float2bfloat16_rn(fmaxf((0.5f * (empty ? 0.f : ends.y) - half) * (1.f / 7.5f), 0.f));
    if (__bfloat162float(step) < 0x1p-100f) step = __float2bfloat16_rn(0.f);
    const float half_step = 0.5f * __bfloat162float(step), by = half_step > 0.f ? 1.f / half_step : 0.f;
    uint32_t* codes = reinterpret_cast<uint32_t*>(page + (int64_t)row * a.groups * 16);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      int q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        q[e] = __float_as_int(__fadd_rn((0.5f * to_f32(x[w][8 * v + e]) - half) * by, 0x1.8p23f)) - 0x4B400000;
      uint32_t word = pack_codes(q);
      if (n < 8 * v + 8) word &= n <= 8 * v ? 0u : (1u << (4 * (n - 8 * v))) - 1u;
      codes[cache_word(a.groups, j, 2 * c + v)] = lost ? 0u : word;
    }
    if (c == 0)
      reinterpret_cast<uint32_t*>(page + ((int64_t)a.block.d * 16 + (int64_t)row * 4) * a.groups)[j] =
          lost ? 0x7FC00000u : (uint32_t)__bfloat16_as_ushort(step) | (uint32_t)__bfloat16_as_ushort(base) << 16;
  }
}

// A thread reads what 16 elements of a key and of a value stand for. A code
// becomes a float by the bits of 2^23 put before it, exactly. 131,072 tokens of
// 8 x 128 in bf16: 133 us, 5.3 TB/s, bound by loads and stores in flight.
template <class T, int V>
__global__ void __launch_bounds__(kCacheThreads) k_cache_read(CacheArgs a, CacheRows r, uint32_t total) {
  const uint32_t index = blockIdx.x * kCacheThreads + threadIdx.x;
  if (index >= total) return;
  const uint32_t line = a.parts(index), part = index - line * a.parts.d;
  const uint32_t token = a.heads(line), h = line - token * a.heads.d;
  const int64_t slot = __ldg(a.slots + token);
  const bool ok = slot >= 0 && slot < a.n_slots;
  if (!ok && slot != -1 && part == 0) atomicOr(&a.small->op_status, kStBadInput);
  uint32_t row = 0, codes[2][2] = {}, pair[2] = {};
  if (ok) {
    const unsigned char* page = cache_page(a, slot, h, &row);
#pragma unroll
    for (int w = 0; w < 2; ++w, page += (int64_t)a.heads.d * a.page_bytes) {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(page + (int64_t)row * a.groups * 16);
#pragma unroll
      for (int v = 0; v < 2; ++v) codes[w][v] = __ldg(from + cache_word(a.groups, part >> 1, 2 * (part & 1) + v));
      pair[w] = __ldg(reinterpret_cast<const uint32_t*>(page + ((int64_t)a.block.d * 16 + (int64_t)row * 4) * a.groups) +
                      (part >> 1));
    }
  }
  const int at = part * kCacheTake, n = a.dim - at;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    T* out = static_cast<T*>(r.out[w]) + token * r.token[w] + h * r.head[w] + at;
    const float step = bf16_low(pair[w]), base = bf16_high(pair[w]);
    __align__(16) T y[kCacheTake];
#pragma unroll
    for (int e = 0; e < kCacheTake; ++e) {
      const float code = __uint_as_float(((codes[w][e / 8] >> (4 * (e % 8))) & 15u) | 0x4B000000u) - 0x1p23f;
      y[e] = from_f32<T>(base + step * code);
    }
    if constexpr (V == 8) {
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (8 * v < n) reinterpret_cast<const Vec<T, 8>*>(y)[v].store(out + 8 * v);
    } else if (sizeof(T) == 2 && n >= kCacheTake) {
      if constexpr (sizeof(T) == 2) store_words(out, y);
    } else {
#pragma unroll
      for (int e = 0; e < kCacheTake; ++e)
        if (e < n) out[e] = y[e];
    }
  }
}

// Runs launch(args, tokens before, total threads) in parts of fewer than 2^31 threads.
template <class F>
int cache_parts(int64_t n_tokens, int64_t n_heads, int64_t parts, F launch) {
  const int64_t at_once = std::min(n_tokens, (int64_t)INT32_MAX / 2 / (n_heads * parts));
  for (int64_t t = 0; t < n_tokens; t += at_once) {
    launch(t, (uint32_t)(std::min(at_once, n_tokens - t) * n_heads * parts));
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
    const int64_t groups = cache_groups(dim), parts = groups * 2;
    CacheArgs a{static_cast<unsigned char*>(d_cache), block_stride, cache_page_bytes(block_size, dim),
                n_blocks * block_size, FastDiv(block_size), FastDiv(parts), FastDiv(n_heads), (int)groups, (int)dim,
                d_slots, h->d_small};
    CacheRows r{{d_keys, d_values}, {}, {key_token_stride, value_token_stride}, {key_head_stride, value_head_stride}};
    return with_type(type, [&](auto t) -> int {
      using T = decltype(t);
      bool wide = dim % 8 == 0;
      for (int w = 0; w < 2; ++w)
        wide = wide && vec_ok(r.in[w], n_tokens > 1 ? r.token[w] : 0, sizeof(T), 8) &&
               vec_ok(r.in[w], n_heads > 1 ? r.head[w] : 0, sizeof(T), 8);
      return cache_parts(n_tokens, n_heads, parts, [&](int64_t from, uint32_t total) {
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
    const int64_t groups = cache_groups(dim), parts = (dim + kCacheTake - 1) / kCacheTake;
    CacheArgs a{static_cast<unsigned char*>(const_cast<void*>(d_cache)), block_stride,
                cache_page_bytes(block_size, dim), n_blocks * block_size, FastDiv(block_size), FastDiv(parts),
                FastDiv(n_heads), (int)groups, (int)dim, d_slots, h->d_small};
    CacheRows r{{}, {d_keys, d_values}, {key_token_stride, value_token_stride}, {key_head_stride, value_head_stride}};
    return with_type(type, [&](auto t) -> int {
      using T = decltype(t);
      bool wide = dim % 8 == 0;
      for (int w = 0; w < 2; ++w)
        wide = wide && vec_ok(r.out[w], n_tokens > 1 ? r.token[w] : 0, sizeof(T), 8) &&
               vec_ok(r.out[w], n_heads > 1 ? r.head[w] : 0, sizeof(T), 8);
      return cache_parts(n_tokens, n_heads, parts, [&](int64_t from, uint32_t total) {
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
