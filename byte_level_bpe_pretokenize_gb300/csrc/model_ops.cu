// Operators between the encoder and a language model, on packed ids: block
// plans of a paged cache (blocks.cuh), embedding lookup and its gradient
// (embed.cuh), penalties, biases and grammar masks on logits (logits.cuh).
// The source pages end at the ids; these have no counterpart there.
//
// They share the handle's device, workspace and status with the encoder
// (handle.cuh). No kernel waits on another CTA outside its own cluster.

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

#include "vec.cuh"
#include "blocks.cuh"
#include "embed.cuh"
#include "logits.cuh"
