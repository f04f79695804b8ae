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

// f(id, second) for each id of two lists, by `threads` threads of which this
// is tid; whole 16-byte vectors of ids are loaded as such, kLoads at a time.
template <int kLoads, class F>
__device__ __forceinline__ void each_id(const int32_t* a, int64_t n_a, const int32_t* b, int64_t n_b, int tid,
                                        int threads, F f) {
  const int64_t head_a = min((int64_t)((-reinterpret_cast<uintptr_t>(a) & 15) / 4), n_a), vecs_a = (n_a - head_a) / 4;
  const int64_t head_b = min((int64_t)((-reinterpret_cast<uintptr_t>(b) & 15) / 4), n_b), vecs_b = (n_b - head_b) / 4;
  // at most three ids before the vectors of a list and three after: a's by
  // threads 0 to 7, b's by threads 8 to 15
  const int e = tid & 7;
  const bool edge_b = tid & 8;
  const int64_t head = edge_b ? head_b : head_a, count = edge_b ? n_b : n_a;
  const int64_t edge = e < head ? e : e + 4 * (edge_b ? vecs_b : vecs_a);
  const bool has_edge = tid < 16 && edge < count;
  const uint32_t edge_id = has_edge ? (uint32_t)__ldg((edge_b ? b : a) + edge) : 0;
  const uint4* from_a = reinterpret_cast<const uint4*>(a + head_a);
  const uint4* from_b = reinterpret_cast<const uint4*>(b + head_b) - vecs_a;
  const int64_t vecs = vecs_a + vecs_b;
  for (int64_t j = tid; j < vecs; j += kLoads * threads) {
    uint4 id[kLoads];
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int64_t k = j + q * threads;
      if (k < vecs) id[q] = __ldg((k < vecs_a ? from_a : from_b) + k);
    }
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int64_t k = j + q * threads;
      if (k >= vecs) break;
      f(id[q].x, k >= vecs_a);
      f(id[q].y, k >= vecs_a);
      f(id[q].z, k >= vecs_a);
      f(id[q].w, k >= vecs_a);
    }
  }
  if (has_edge) f(edge_id, edge_b);
}

// f(id) for each id of one list.
template <int kLoads, class F>
__device__ __forceinline__ void each_id(const int32_t* ids, int64_t count, int tid, int threads, F f) {
  each_id<kLoads>(ids, count, nullptr, 0, tid, threads, [&](uint32_t id, bool) { f(id); });
}

// Whether V elements of `size` bytes at every multiple of V from p, and from p
// plus multiples of stride elements, are aligned for Vec.
inline bool vec_ok(const void* p, int64_t stride, int64_t size, int64_t V) {
  const int64_t to = std::min<int64_t>(16, V * size);
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)to == 0 && (stride * size) % to == 0;
}

}  // namespace
