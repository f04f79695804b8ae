// What the translation units of the library share: the handle, its device
// workspace and status words, error messages and host helpers.
#ifndef BPE_HANDLE_CUH_
#define BPE_HANDLE_CUH_

#include <cuda_runtime.h>

#include <cstdint>
#include <exception>
#include <string>
#include <vector>

#include "../../include/bpe_gb300.h"

namespace bpe_impl {

// device status bits
constexpr uint32_t kStBadInput = 1u;
constexpr uint32_t kStTimeout = 2u;
constexpr uint32_t kStInternal = 4u;
constexpr uint32_t kStCapacity = 8u;

struct DevSmall {
  uint32_t status;
  uint32_t op_status;                // the same bits, set by kernels outside the encoder, whose
                                     // own act on status
  int64_t total;                     // ids of the call
  unsigned long long tile_ctr;       // tiles taken by k_tiles' warps
  unsigned long long n_misses;       // cache misses handed to k_misses
  unsigned long long n_giants;       // pre-tokens deferred to k_giants
  unsigned long long giant_ctr;      // deferred pre-tokens taken by k_giants' CTAs
  unsigned long long n_ranges;       // long runs of tiles for k_prep_long
};

// Message of the last failing call on this thread (bpe_last_error).
std::string& last_error();

inline int fail(int code, const std::string& msg) {
  last_error() = msg;
  return code;
}

inline int cuda_fail(cudaError_t e, const char* what) {
  return fail(BPE_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

#define CK(call)                                        \
  do {                                                  \
    cudaError_t e_ = (call);                            \
    if (e_ != cudaSuccess) return cuda_fail(e_, #call); \
  } while (0)

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    cudaGetDevice(&prev);
    if (prev != dev) cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    int cur = -1;
    cudaGetDevice(&cur);
    if (prev >= 0 && cur != prev) cudaSetDevice(prev);
  }
};

constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace bpe_impl

struct bpe_handle {
  int device = 0;
  int n_sms = 1;  // multiprocessors of the device (grids of persistent kernels)
  int64_t n_merges = 0, n_vocab = 0;
  int monotone = 1;  // every merge's operands are made by lower ranks (bpe_merges_monotone)
  uint4* d_ht = nullptr;
  uint32_t hmask = 0;
  int32_t* d_mrows = nullptr;
  int32_t* d_byte_id = nullptr;
  uint8_t* d_vbytes = nullptr;
  int64_t* d_voffs = nullptr;
  uint4* d_vent = nullptr;  // per token: its first 12 bytes and its length (decoding)
  uint4* d_cache = nullptr;
  uint32_t cache_mask = 0;
  int64_t cache_entries = 0;
  int cache_enabled = 1;
  int call_memo = BPE_MEMO_AUTO;  // bpe_set_call_memo
  bpe_impl::DevSmall* d_small = nullptr;
  bpe_impl::DevSmall* h_small = nullptr;  // pinned
  void* d_ws = nullptr;
  size_t ws_bytes = 0;
  bool ws_captured = false;    // a graph may hold d_ws
  std::vector<void*> kept_ws;  // outgrown blocks that a graph may hold, freed with the handle
  size_t kept_bytes = 0;
  bool smem_set = false;
  cudaEvent_t ev_start = nullptr, ev_stop = nullptr;
  cudaEvent_t* ev_phase = nullptr;  // BPE_ENCODE_LAUNCHES + 1 caller-owned events, or null
  // bpe_encode_batch_host: kHostSlots slots of device buffers, copy streams,
  // events
  static constexpr int kHostSlots = 4;
  struct HostSlot {
    uint8_t* bytes = nullptr;
    int64_t* offs = nullptr;
    int32_t* ids = nullptr;
    int64_t* out_offs = nullptr;
    cudaEvent_t in = nullptr, done = nullptr, free = nullptr;
  } slot[kHostSlots];
  int64_t slot_bytes = 0, slot_docs = 0;  // capacity of each slot
  cudaStream_t s_h2d = nullptr, s_d2h = nullptr;
  // bpe_embed_grad: zeros written beside its other kernels
  cudaStream_t s_side = nullptr;
  cudaEvent_t ev_fork = nullptr, ev_join = nullptr;
  int64_t* h_totals = nullptr;  // pinned, one per slice
  int64_t* d_totals = nullptr;  // the same memory as the device addresses it
  int64_t h_totals_cap = 0;
};

namespace bpe_impl {

// The handle's workspace, grown to at least `need` bytes, for a call on st. A
// block that a call under stream capture has used stays until the handle is
// destroyed, for the graph's replays use it again.
inline int ensure_ws(bpe_handle* h, size_t need, cudaStream_t st) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  CK(cudaStreamIsCapturing(st, &capture));
  if (need > h->ws_bytes) {
    if (h->ws_captured) {
      try {
        h->kept_ws.push_back(h->d_ws);
      } catch (const std::exception& e) {
        return fail(BPE_ERR_INTERNAL, e.what());
      }
      h->kept_bytes += h->ws_bytes;
    } else if (h->d_ws) {
      CK(cudaFree(h->d_ws));
    }
    h->d_ws = nullptr;
    h->ws_bytes = 0;
    h->ws_captured = false;
    const size_t sz = need + need / 4 + 4096;
    CK(cudaMalloc(&h->d_ws, sz));
    h->ws_bytes = sz;
  }
  if (capture != cudaStreamCaptureStatusNone && need > 0) h->ws_captured = true;
  return BPE_OK;
}

}  // namespace bpe_impl

#endif  // BPE_HANDLE_CUH_
