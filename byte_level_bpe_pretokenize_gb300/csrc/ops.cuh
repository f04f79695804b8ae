// What the operators around a language model share: element types, launches
// and the guard of their C entries.
//
// Included once by each of their translation units; not a standalone header.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "handle.cuh"

using namespace bpe_impl;
namespace cg = cooperative_groups;

namespace {

size_t type_size(int type) { return type == BPE_F32 ? 4 : 2; }
bool type_ok(int type) { return type == BPE_F32 || type == BPE_F16 || type == BPE_BF16; }
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Rounds to nearest even, once, at the end of a 32-bit computation.
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }

// f(T{}) with the C++ type of a BPE_F32, BPE_F16 or BPE_BF16.
template <class F>
int with_type(int type, F f) {
  if (type == BPE_F32) return f(float{});
  if (type == BPE_F16) return f(__half{});
  return f(__nv_bfloat16{});
}

// Runs f (kernel attributes, which last as long as the process) once per device
// for each place that calls this; the caller has the device current. Racing
// first calls both run it.
template <class F>
int once_per_device(int device, F f) {
  static std::atomic<bool> done[64];
  if (device < 64 && done[device].load(std::memory_order_acquire)) return BPE_OK;
  CK(f());
  if (device < 64) done[device].store(true, std::memory_order_release);
  return BPE_OK;
}

// Programmatic dependent launch. A kernel launched by launch_after may begin
// once every block of the kernel before it has called let_next_begin or ended;
// what it does before await_previous must not depend on that kernel. Each
// kernel of such a chain awaits the one before it, so the end of the last one
// is the end of all; the first is an ordinary launch.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Exact division of numbers below 2^31 by d in [1, 2^31): with 2^(l-1) < d <=
// 2^l and m = ceil(2^(31+l) / d), the excess e = m d - 2^(31+l) is below 2^l,
// so x m / 2^(31+l) = x / d + (x / 2^31) (e / 2^l) / d, which is less than 1/d
// above x / d and has the same floor.
struct FastDiv {
  uint32_t d, m, l;
  explicit FastDiv(int64_t by = 1) : d((uint32_t)by), l(0) {
    while ((1ll << l) < by) ++l;
    m = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return (uint32_t)(((uint64_t)x * m) >> (31 + l)); }
};

// Whether two of n x m rows of dim elements, at multiples of the strides s and t, meet.
inline bool rows_meet(int64_t n, int64_t s, int64_t m, int64_t t, int64_t dim) {
  if (n <= 1 && m <= 1) return false;
  if (n <= 1) return t < dim;
  if (m <= 1) return s < dim;
  return !(t >= dim && s >= (m - 1) * t + dim) && !(s >= dim && t >= (n - 1) * s + dim);
}

// n x m rows of `row` bytes from `at` on, s and t bytes apart (>= 0).
struct Rows {
  uintptr_t at;
  int64_t n, m, s, t, row;
  int64_t reach() const { return (n - 1) * s + (m - 1) * t + row; }
  bool gapless() const {
    return (m <= 1 || t <= row) && (n <= 1 || s <= (m - 1) * t + row);
  }
};

// Whether two such tensors share a byte, as far as that shows without looking at every pair of rows: always where
// their strides are equal, and where one of them has no gaps and an end of the other lies in it.
inline bool rows_share(const Rows& a, const Rows& b) {
  if (a.n < 1 || a.m < 1 || b.n < 1 || b.m < 1) return false;
  const int64_t d = (int64_t)(b.at - a.at);  // rows meet where -b.row < d + i s + j t < a.row
  if (d >= a.reach() || -d >= b.reach()) return false;
  if (a.gapless() && b.gapless()) return true;
  if (a.n == b.n && a.m == b.m && (a.n == 1 || a.s == b.s) && (a.m == 1 || a.t == b.t)) {
    for (int64_t j = 1 - a.m; j < a.m; ++j) {
      const int64_t e = d + j * a.t;  // the smallest e + i s above -b.row
      int64_t i = 0;
      if (a.n > 1 && a.s > 0) {
        const int64_t over = e + b.row - 1;
        i = -(over >= 0 ? over / a.s : -((-over + a.s - 1) / a.s));
        i = std::max(i, 1 - a.n);
        if (i > a.n - 1) continue;
      }
      if (e + i * a.s > -b.row && e + i * a.s < a.row) return true;
    }
    return false;
  }
  auto in = [](const Rows& whole, const Rows& other) {
    if (!whole.gapless()) return false;
    const int64_t first = (int64_t)(other.at - whole.at), last = first + other.reach() - other.row;
    auto meets = [&](int64_t at) { return at < whole.reach() && at + other.row > 0; };
    return meets(first) || meets(last);
  };
  return in(a, b) || in(b, a);
}

// No exception (an allocation for an error message, say) leaves a C entry.
template <class F>
int guarded(const char* what, F f) noexcept {
  try {
    return f();
  } catch (const std::exception& e) {
    try {
      return fail(BPE_ERR_INTERNAL, std::string(what) + ": " + e.what());
    } catch (...) {
      return BPE_ERR_INTERNAL;
    }
  }
}

}  // namespace
