// Penalties for repeated tokens, biases and grammar masks on logits.
//
// Included once by model_ops.cu; not a standalone header.
//
// For row b and token v, with k the times v occurs in the row's output and
// "seen" whether it occurs in its prompt or output:
//   x = logits[b, v]
//   seen:   x = x > 0 ? x / repetition_b : x * repetition_b
//   k > 0:  x = x - frequency_b * k - presence_b
//   biased: x = x + (the sum of its biases)
//   shut by the row's mask: x = -inf, whatever it was

namespace {

constexpr int kLogThreads = 256;
constexpr int kLogChunk = 4096;  // tokens of a CTA
constexpr uint32_t kLogPrompt = 0x80000000u, kLogBias = 0x40000000u, kLogCount = 0x3FFFFFFFu;

// Adds v to bias[at], equal places in lane order; at < 0 for none. One warp.
__device__ __forceinline__ void log_add_bias(float* bias, uint32_t* seen, int at, float v, int lane) {
  const unsigned same = __match_any_sync(0xFFFFFFFFu, at);
  float sum = at >= 0 ? bias[at] : 0.f;
  if (__any_sync(0xFFFFFFFFu, at >= 0 && (same & (same - 1)))) {
    for (int k = 0; k < 32; ++k) {
      const float vk = __shfl_sync(0xFFFFFFFFu, v, k);
      if (same >> k & 1) sum += vk;
    }
  } else {
    sum += v;
  }
  if (at >= 0 && (same & ((1u << lane) - 1)) == 0) {
    bias[at] = sum;
    atomicOr(&seen[at], kLogBias);
  }
  __syncwarp();
}

template <class TI, class TO>
__global__ void __launch_bounds__(kLogThreads) k_logits(bpe_logits_args a, DevSmall* small) {
  __shared__ uint32_t seen[kLogChunk];
  __shared__ float bias[kLogChunk];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.y, v0 = (int64_t)blockIdx.x * kLogChunk;
  const int n = (int)min((int64_t)kLogChunk, a.n_vocab - v0);
  bool bad = false;
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f, pres = a.presence ? a.presence[b] : 0.f;
  for (int v = tid; v < n; v += kLogThreads) {
    seen[v] = 0;
    bias[v] = 0.f;
  }
  __syncthreads();
  if (rep != 1.f && a.prompt_ids) {
    const int64_t s = a.prompt_offsets[b], e = a.prompt_offsets[b + 1];
    if (s < 0 || e < s || e > a.n_prompt_ids) bad = true;
    else
      for (int64_t j = s + tid; j < e; j += kLogThreads) {
        const int64_t id = a.prompt_ids[j];
        if (id < 0 || id >= a.n_vocab) bad = true;
        else if (id >= v0 && id < v0 + n) atomicOr(&seen[id - v0], kLogPrompt);
      }
  }
  if ((rep != 1.f || freq != 0.f || pres != 0.f) && a.output_ids) {
    const int64_t len = a.output_lens[b];
    if (len < 0 || len > a.output_capacity) bad = true;
    else
      for (int64_t j = tid; j < len; j += kLogThreads) {
        const int64_t id = a.output_ids[b * a.output_stride + j];
        if (id < 0 || id >= a.n_vocab) bad = true;
        else if (id >= v0 && id < v0 + n) atomicAdd(&seen[id - v0], 1u);
      }
  }
  __syncthreads();
  if (tid < 32 && a.bias_ids) {
    const int64_t s = a.bias_offsets[b], e = a.bias_offsets[b + 1];
    if (s < 0 || e < s || e > a.n_bias) bad = true;
    else
      for (int64_t j = s; j < e; j += 32) {
        int at = -1;
        float v = 0.f;
        if (j + tid < e) {
          const int64_t id = a.bias_ids[j + tid];
          if (id < 0 || id >= a.n_vocab) bad = true;
          else if (id >= v0 && id < v0 + n) at = (int)(id - v0);
          v = a.bias_values[j + tid];
        }
        log_add_bias(bias, seen, at, v, tid);
      }
  }
  __syncthreads();
  int64_t mask_row = -1;
  if (a.mask) {
    mask_row = a.mask_rows ? a.mask_rows[b] : b;
    if (mask_row < -1 || mask_row >= a.n_masks) {
      bad = true;
      mask_row = -1;
    }
  }
  const TI* in = static_cast<const TI*>(a.logits) + b * a.logits_stride + v0;
  TO* out = static_cast<TO*>(a.out) + b * a.out_stride + v0;
  for (int v = tid; v < n; v += kLogThreads) {
    float x = to_f32(in[v]);
    const uint32_t q = seen[v];
    if (q) {
      const uint32_t k = q & kLogCount;
      if (k || (q & kLogPrompt)) x = x > 0.f ? x / rep : x * rep;
      if (k) x = x - freq * (float)k - pres;
      if (q & kLogBias) x += bias[v];
    }
    if (mask_row >= 0 && !(a.mask[mask_row * a.mask_stride + ((v0 + v) >> 5)] >> ((v0 + v) & 31) & 1)) x = -INFINITY;
    out[v] = from_f32<TO>(x);
  }
  if (bad) atomicOr(&small->op_status, kStBadInput);
}

}  // namespace

extern "C" int bpe_adjust_logits(bpe_handle* h, const bpe_logits_args* args, bpe_stream_t stream) {
  return guarded("bpe_adjust_logits", [&]() -> int {
    if (!h || !args) return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: null handle or arguments");
    const bpe_logits_args& a = *args;
    if (!type_ok(a.logits_type) || !type_ok(a.out_type))
      return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: unknown type");
    if (a.n_rows < 0 || a.n_rows > 65535 || a.n_vocab < 0 || a.n_vocab >= INT32_MAX || a.n_prompt_ids < 0 ||
        a.output_capacity < 0 || a.output_capacity > (int64_t)kLogCount || a.n_bias < 0 || a.n_masks < 0)
      return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: a size is negative or too large");
    if (a.n_rows == 0 || a.n_vocab == 0) return BPE_OK;
    if (!a.logits || !a.out || (a.prompt_ids && !a.prompt_offsets) || (a.output_ids && !a.output_lens) ||
        (a.bias_ids && (!a.bias_values || !a.bias_offsets)))
      return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: null pointer");
    const int64_t words = (a.n_vocab + 31) / 32;
    if (a.logits_stride < 0 || a.output_stride < 0 || a.mask_stride < 0 || (a.n_rows > 1 && a.out_stride < a.n_vocab) ||
        (a.mask && a.n_masks > 1 && a.mask_stride < words))
      return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: a stride is negative or below its row's length");
    if (a.mask && !a.mask_rows && a.n_masks < a.n_rows)
      return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: fewer masks than rows, and no mask_rows");
    if (!aligned(a.logits, type_size(a.logits_type)) || !aligned(a.out, type_size(a.out_type)) ||
        !aligned(a.prompt_ids, 4) || !aligned(a.prompt_offsets, 8) || !aligned(a.output_ids, 4) ||
        !aligned(a.output_lens, 4) || !aligned(a.repetition, 4) || !aligned(a.frequency, 4) ||
        !aligned(a.presence, 4) || !aligned(a.bias_ids, 4) || !aligned(a.bias_values, 4) ||
        !aligned(a.bias_offsets, 8) || !aligned(a.mask, 4) || !aligned(a.mask_rows, 4))
      return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: a pointer is not aligned to its elements");
    if (a.logits == a.out && (a.logits_type != a.out_type || a.logits_stride != a.out_stride) )
      return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: in place needs one type and one stride");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    return with_type(a.logits_type, [&](auto i) {
      return with_type(a.out_type, [&](auto o) -> int {
        const dim3 grid((unsigned)((a.n_vocab + kLogChunk - 1) / kLogChunk), (unsigned)a.n_rows);
        k_logits<decltype(i), decltype(o)><<<grid, kLogThreads, 0, st>>>(a, h->d_small);
        CK(cudaGetLastError());
        return BPE_OK;
      });
    });
  });
}
