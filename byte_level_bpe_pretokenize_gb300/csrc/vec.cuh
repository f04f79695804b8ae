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

// Whether V elements of `size` bytes at every multiple of V from p, and from p
// plus multiples of stride elements, are aligned for Vec.
inline bool vec_ok(const void* p, int64_t stride, int64_t size, int64_t V) {
  const int64_t to = std::min<int64_t>(16, V * size);
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)to == 0 && (stride * size) % to == 0;
}

}  // namespace
