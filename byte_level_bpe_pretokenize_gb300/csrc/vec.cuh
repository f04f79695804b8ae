// Vector loads and stores of 32- and 16-bit elements as 32-bit floats.
//
// Included once by model_ops.cu; not a standalone header.
//
// A vector of V elements moves in accesses of at most 16 bytes, so its address
// needs an alignment of min(16, V * size) only. Both directions use the
// streaming cache policy unless kKeep: data that a call touches once should
// not push out of the L2 what it reads again (table rows, lists).

namespace {

template <int kBytes>
struct Raw;
template <>
struct Raw<2> { using type = unsigned short; };
template <>
struct Raw<4> { using type = unsigned int; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<16> { using type = uint4; };

template <class T, int V>
struct __align__(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Vec {
  static constexpr int kAccess = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;
  static constexpr int kParts = V * (int)sizeof(T) / kAccess;
  using R = typename Raw<kAccess>::type;
  T x[V];

  template <bool kKeep = false>
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const R* q = reinterpret_cast<const R*>(p) + i;
      reinterpret_cast<R*>(x)[i] = kKeep ? __ldg(q) : __ldcs(q);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) __stcs(reinterpret_cast<R*>(p) + i, reinterpret_cast<const R*>(x)[i]);
  }
};

// f(id) for each id of a list, by `threads` threads of which this is tid;
// whole 16-byte vectors of ids are loaded as such, kLoads at a time.
template <int kLoads, class F>
__device__ __forceinline__ void each_id(const int32_t* ids, int64_t count, int tid, int threads, F f) {
  const int64_t head = min((int64_t)((-reinterpret_cast<uintptr_t>(ids) & 15) / 4), count);
  const int64_t vecs = (count - head) / 4, tail = head + vecs * 4;
  // at most three ids before the vectors and three after
  const int64_t edge = tid < head ? tid : tail + tid - head;
  const bool has_edge = edge < count;
  const uint32_t edge_id = has_edge ? (uint32_t)__ldg(ids + edge) : 0;
  const uint4* from = reinterpret_cast<const uint4*>(ids + head);
  for (int64_t j = tid; j < vecs; j += kLoads * threads) {
    uint4 id[kLoads];
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      if (j + q * threads < vecs) id[q] = __ldg(from + j + q * threads);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      if (j + q * threads >= vecs) break;
      f(id[q].x);
      f(id[q].y);
      f(id[q].z);
      f(id[q].w);
    }
  }
  if (has_edge) f(edge_id);
}

// Whether V elements of `size` bytes at every multiple of V from p, and from p
// plus multiples of stride elements, are aligned for Vec.
inline bool vec_ok(const void* p, int64_t stride, int64_t size, int64_t V) {
  const int64_t to = std::min<int64_t>(16, V * size);
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)to == 0 && (stride * size) % to == 0;
}

}  // namespace
