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
constexpr int kLogWarps = kLogThreads / 32;
constexpr int kLogGroup = 8;         // tokens of a vector
constexpr int kLogAhead = 2;         // vectors of a thread in flight
constexpr int kLogIds = 2;           // 16-byte loads of ids of a thread in flight
constexpr int kLogBlocks = 2;        // CTAs an SM at least, while chunks can be halved
constexpr int kLogMinChunk = 2048;   // tokens of a CTA
constexpr int kLogMaxChunk = 16384;
constexpr int kLogDenseChunk = 8192; // with a count for each token
constexpr int kLogWords = 2;         // words of bits of a thread
constexpr int kLogList = 1024;       // concerned tokens that a CTA lists at once
constexpr int kLogBiases = 512;      // biases of a chunk that it lists
constexpr int kLogShare = kLogBiases / kLogWarps;
constexpr int kLogSaid = 2048;       // output tokens of a chunk that it lists

// Bits 15 and 31 of word w of the result, moved down by w: whether the halves of
// p's word w equal those of `twice`. (In their difference the half that is 0 is
// the one whose low 15 bits carry nothing into its top bit, which is 0 too.)
__device__ __forceinline__ uint32_t log_equal(const uint4& p, uint32_t twice) {
  auto zero = [](uint32_t x) { return ~(((x & 0x7FFF7FFFu) + 0x7FFF7FFFu) | x | 0x7FFF7FFFu); };
  return zero(p.x ^ twice) | zero(p.y ^ twice) >> 1 | zero(p.z ^ twice) >> 2 | zero(p.w ^ twice) >> 3;
}

// What a row's history says about a chunk, in shared memory: a bit for each
// token that occurs in it, one for each that has a bias, and the times a token
// occurs in the output. Outputs of up to kLogSaid tokens have a bit for a
// token's first occurrence and one for whether there are more; those are listed
// and counted when they are asked for. Longer outputs have a count for each
// token (in 16 bits where that is enough), and shorter chunks. All but the first
// bit are added to without a look at what was there, so that nothing waits for
// shared memory.
struct LogTable {
  uint32_t* bits;    // [chunk / 32]
  uint32_t* biased;  // [chunk / 32]
  uint32_t* twice;   // [chunk / 32] tokens with more than one bias
  uint32_t* said;    // [chunk / 32], where the output is listed
  uint32_t* again;   // [chunk / 32] said more than once, likewise
  uint16_t* list;    // [kLogSaid] the chunk's output tokens but for the first of each, in any order
  int* listed;       // how many
  uint32_t* counts;  // [chunk] or, in 16 bits, [chunk / 2]; where the output is counted
  int wide;          // bits of a count; 0: the output is listed

  __host__ __device__ static constexpr int bytes(int chunk, bool by_output, int wide) {
    return 3 * chunk / 8 + (!by_output ? 0 : wide ? chunk * wide / 8 : chunk / 4 + 2 * kLogSaid);
  }
  __device__ __forceinline__ LogTable(uint32_t* smem, int chunk, int wide_, int* listed_)
      : bits(smem), biased(smem + chunk / 32), twice(smem + 2 * chunk / 32), said(smem + 3 * chunk / 32),
        again(smem + 4 * chunk / 32), list(reinterpret_cast<uint16_t*>(smem + 5 * chunk / 32)), listed(listed_),
        counts(smem + 3 * chunk / 32), wide(wide_) {}
  __device__ __forceinline__ void clear(int chunk, bool by_output) const {
    const int words = 3 * chunk / 32 + (!by_output ? 0 : wide ? chunk * wide / 32 : chunk / 16);
    for (int v = threadIdx.x; v < words / 4; v += kLogThreads)
      reinterpret_cast<uint4*>(bits)[v] = make_uint4(0, 0, 0, 0);
    // no token of a chunk is 0xFFFF, which fills the last vector of the list
    if (by_output && !wide)
      for (int i = threadIdx.x; i < kLogSaid / 8; i += kLogThreads)
        reinterpret_cast<uint4*>(list)[i] = make_uint4(0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu);
    if (threadIdx.x == 0) *listed = 0;
  }
  __device__ __forceinline__ void see(int v) const { atomicOr(&bits[v >> 5], 1u << (v & 31)); }
  __device__ __forceinline__ void say(int v) const {
    if (wide == 16) {
      atomicAdd(&counts[v >> 1], (v & 1) ? 0x10000u : 1u);
    } else if (wide) {
      atomicAdd(&counts[v], 1u);
    } else {
      const uint32_t bit = 1u << (v & 31);
      if (atomicOr(&said[v >> 5], bit) & bit) {
        atomicOr(&again[v >> 5], bit);
        list[atomicAdd(listed, 1)] = (uint16_t)v;
      }
    }
  }
  __device__ __forceinline__ bool seen(int v) const { return bits[v >> 5] >> (v & 31) & 1; }
  __device__ __forceinline__ uint32_t times(int v) const {
    if (wide == 16) return counts[v >> 1] >> ((v & 1) * 16) & 0xFFFFu;
    if (wide) return counts[v];
    uint32_t k = said[v >> 5] >> (v & 31) & 1;
    if (!(again[v >> 5] >> (v & 31) & 1)) return k;
    const int vecs = (*listed + 7) / 8;
    const uint32_t twice = (uint32_t)v * 0x10001u;
    const uint4* from = reinterpret_cast<const uint4*>(list);
#pragma unroll 4
    for (int i = 0; i < vecs; ++i) k += __popc(log_equal(from[i], twice));
    return k;
  }
};

// A row's parameters, and where its history and biases are.
struct LogRow {
  float rep, freq, pres;
  const int32_t *prompt, *output, *bias_ids;
  const float* bias_values;
  int64_t n_prompt, n_output, n_bias;
  const uint32_t* mask;  // its words, or null
  bool concerned;        // anything but the mask concerns it
};

__device__ __forceinline__ LogRow log_row(const bpe_logits_args& a, int64_t b, bool table, bool* bad) {
  LogRow r{1.f, 0.f, 0.f, nullptr, nullptr, nullptr, nullptr, 0, 0, 0, nullptr, false};
  if (table) {
    // all loads first, so that they overlap
    const int64_t p0 = a.prompt_ids ? __ldg(a.prompt_offsets + b) : 0;
    const int64_t p1 = a.prompt_ids ? __ldg(a.prompt_offsets + b + 1) : 0;
    const int64_t len = a.output_ids ? __ldg(a.output_lens + b) : 0;
    const int64_t b0 = a.bias_ids ? __ldg(a.bias_offsets + b) : 0;
    const int64_t b1 = a.bias_ids ? __ldg(a.bias_offsets + b + 1) : 0;
    if (a.repetition) r.rep = __ldg(a.repetition + b);
    if (a.frequency) r.freq = __ldg(a.frequency + b);
    if (a.presence) r.pres = __ldg(a.presence + b);
    if (r.rep != 1.f) {
      if (p0 < 0 || p1 < p0 || p1 > a.n_prompt_ids) *bad = true;
      else r.prompt = a.prompt_ids + p0, r.n_prompt = p1 - p0;
    }
    if (r.rep != 1.f || r.freq != 0.f || r.pres != 0.f) {
      if (len < 0 || len > a.output_capacity) *bad = true;
      else r.output = a.output_ids + b * a.output_stride, r.n_output = len;
    }
    if (b0 < 0 || b1 < b0 || b1 > a.n_bias) *bad = true;
    else r.bias_ids = a.bias_ids + b0, r.bias_values = a.bias_values + b0, r.n_bias = b1 - b0;
    r.concerned = r.n_prompt + r.n_output + r.n_bias > 0;
  }
  if (a.mask) {
    const int64_t row = a.mask_rows ? __ldg(a.mask_rows + b) : b;
    if (row < -1 || row >= a.n_masks) *bad = true;
    else if (row >= 0) r.mask = a.mask + row * a.mask_stride;
  }
  return r;
}

// Adds x to sums[v], equal tokens in lane order; v < 0 for none. One warp.
__device__ __noinline__ void log_add_bias(float* sums, int v, float x, int lane) {
  const unsigned same = __match_any_sync(0xFFFFFFFFu, v);
  float sum = v >= 0 ? sums[v] : 0.f;
  for (unsigned m = v >= 0 ? same : 0; __any_sync(0xFFFFFFFFu, m); m &= m - 1) {
    const float xk = __shfl_sync(0xFFFFFFFFu, x, m ? __ffs(m) - 1 : lane);
    if (m) sum += xk;
  }
  if (v >= 0 && (same & ((1u << lane) - 1)) == 0) sums[v] = sum;
  __syncwarp();
}

// sums[k] = the sum, in order, of the biases of the token of [low, low + n) whose
// number among those with several is first + k, for k < kLogShare. One warp.
__device__ __noinline__ void log_sum_several(float* sums, const uint16_t* number, const uint32_t* twice,
                                             const int32_t* ids, const float* values, int64_t n_ids, uint32_t low,
                                             uint32_t n, int first, int lane) {
  constexpr int kLook = 4;
  for (int k = lane; k < kLogShare; k += 32) sums[k] = 0.f;
  __syncwarp();
  for (int64_t j = lane; j - lane < n_ids; j += 32 * kLook) {
    uint32_t v[kLook];
#pragma unroll
    for (int q = 0; q < kLook; ++q) v[q] = j + 32 * q < n_ids ? (uint32_t)__ldg(ids + j + 32 * q) - low : 0xFFFFFFFFu;
#pragma unroll
    for (int q = 0; q < kLook; ++q) {
      int at = -1;
      if (v[q] < n) {
        const uint32_t word = twice[v[q] >> 5], bit = v[q] & 31;
        if (word >> bit & 1) at = number[v[q] >> 5] + __popc(word & ((1u << bit) - 1)) - first;
        if (at >= kLogShare) at = -1;
      }
      if (__any_sync(0xFFFFFFFFu, at >= 0))
        log_add_bias(sums, max(at, -1), at >= 0 ? __ldg(values + j + 32 * q) : 0.f, lane);
    }
  }
}

// The bits of the tokens from v on, 8 of them at least; `words` of the mask may
// be read.
__device__ __forceinline__ uint32_t log_open(const uint32_t* mask, int v, int words) {
  const int w = v >> 5;
  return __funnelshift_r(__ldg(mask + w), __ldg(mask + min(w + 1, words - 1)), v & 31);
}

// A seen token's logit.
__device__ __forceinline__ float log_penalty(const LogRow& r, float x, uint32_t times) {
  x = x > 0.f ? x / r.rep : x * r.rep;
  return times ? x - r.freq * (float)times - r.pres : x;
}

// A byte of x's top bit in each place, for the two bytes that kSelect names.
template <uint32_t kSelect>
__device__ __forceinline__ uint32_t log_halves(uint32_t x) {
  uint32_t y;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(y) : "r"(x), "n"(kSelect));
  return y;
}

// Tokens [v0, v0 + n) of a row pass through registers once, 16 bytes of input
// at a time, and leave with the mask applied; by kThreads threads, of which
// this is tid. The first vectors are loaded before row() gives the row's mask.
template <class TI, class TO, int kThreads, class R>
__device__ __forceinline__ void log_pass(const bpe_logits_args& a, int64_t b, int64_t v0, int n, int tid, R row) {
  const int words = (int)((a.n_vocab + 31) >> 5);
  const TI* in = static_cast<const TI*>(a.logits) + b * a.logits_stride + v0;
  TO* out = static_cast<TO*>(a.out) + b * a.out_stride + v0;
  // vectors start at the first 16-byte boundary of the input; if the output
  // has none there, every token goes by itself
  int head = (int)((-reinterpret_cast<uintptr_t>(in) & 15) / sizeof(TI));
  if (reinterpret_cast<uintptr_t>(out + head) & 15) head = n;
  head = min(head, n);
  if (!a.mask && a.logits == a.out) {  // in place, nothing to do but what row() prepares
    row();
    return;
  }
  const int groups = (n - head) / kLogGroup;
  constexpr int kAhead = sizeof(TI) == 4 ? kLogAhead / 2 : kLogAhead;
  Vec<TI, kLogGroup> x[kAhead];
#pragma unroll
  for (int q = 0; q < kAhead; ++q)
    if (tid + q * kThreads < groups) x[q].load(in + head + (tid + q * kThreads) * kLogGroup);
  const uint32_t* mask = row();
  for (int g0 = tid; g0 < groups; g0 += kAhead * kThreads) {
    if (g0 != tid) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        if (g0 + q * kThreads < groups) x[q].load(in + head + (g0 + q * kThreads) * kLogGroup);
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (g0 + q * kThreads >= groups) break;
      const int v = head + (g0 + q * kThreads) * kLogGroup;
      const uint32_t bits = mask ? log_open(mask, (int)v0 + v, words) : 0xFFFFFFFFu;
      Vec<TO, kLogGroup> o;
      if constexpr (std::is_same_v<TI, TO> && sizeof(TI) == 2) {
        // pairs of bit patterns, without a conversion; the product puts four
        // bits into the top bits of its bytes, which become halves of a mask
        const uint32_t* from = reinterpret_cast<const uint32_t*>(x[q].x);
        constexpr uint32_t kShut = std::is_same_v<TI, __half> ? 0xFC00FC00u : 0xFF80FF80u;  // twice -infinity
#pragma unroll
        for (int e = 0; e < kLogGroup / 2; e += 2) {
          const uint32_t four = (bits >> (2 * e) & 15) * 0x10204080u;
          const uint32_t open[2] = {log_halves<0x9988>(four), log_halves<0xBBAA>(four)};
#pragma unroll
          for (int f = 0; f < 2; ++f)
            reinterpret_cast<uint32_t*>(o.x)[e + f] = (from[e + f] & open[f]) | (kShut & ~open[f]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kLogGroup; ++e)
          o.x[e] = from_f32<TO>(bits >> e & 1 ? to_f32(x[q].x[e]) : -INFINITY);
      }
      o.store(out + v);
    }
  }
  // what is before the first vector and after the last
  const int tail = head + groups * kLogGroup;
  for (int k = tid; k < head + n - tail; k += kThreads) {
    const int v = k < head ? k : tail + k - head;
    out[v] = from_f32<TO>(!mask || (log_open(mask, (int)v0 + v, words) & 1) ? to_f32(in[v]) : -INFINITY);
  }
}

// A CTA takes `chunk` tokens of one row. With kTable, what the row's history
// and biases say about them is gathered in shared memory, and after the pass
// the few tokens that are concerned are written again, each once: the pass has
// left a token that the mask shuts at -infinity, and in place it has left the
// bits of every other one. Bits and counts do not depend on the order in which
// they are made, and biases are listed in theirs: nothing depends on timing.
//
// All CTAs of a row read its whole history, which is L2 traffic and a few
// instructions an id. Bound by HBM for the pass (384 rows of 113,645 bf16 with a
// mask for each: 28.5 us, 6.3 TB/s) and, with a history, by issue and by the
// latency of a CTA's steps: lists, barrier, pass, barrier, the tokens again
// (48 us with 3,000 prompt and 450 output tokens a row on average; without the
// last step 41). What was slower for that case: a word for each token looked at
// in the pass (most warps hold a concerned token, and the whole warp waits for
// its division: 135 us), a hash table filled by atomics that return a value (a
// chain of waits for each id: 84 us), warps that gather while others pass
// (152 us), the last CTA of a row writing for all (119 us), a second launch a
// row (82 us), logits changed in shared memory between asynchronous copies and
// one store (67 us, and 33 without a history: fewer CTAs fit an SM), all outputs
// listed and not only the repeated ones (57 us).
template <class TI, class TO, bool kTable, bool kBias, bool kByToken>
__global__ void __launch_bounds__(kLogThreads, 8) k_logits(bpe_logits_args a, int chunk, int wide, DevSmall* small) {
  extern __shared__ __align__(16) uint32_t log_smem[];
  __shared__ uint16_t list[kTable ? kLogList : 1];
  __shared__ int warp_sum[kLogWarps], n_biases, n_said;
  const LogTable t(log_smem, chunk, wide, &n_said);
  // biases: with kByToken (the shortest chunks) a sum for each token, else a list
  float* bias_value = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(log_smem) +
                                               LogTable::bytes(chunk, a.output_ids != nullptr, wide));
  uint16_t* bias_token = reinterpret_cast<uint16_t*>(bias_value + kLogBiases);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.y, v0 = (int64_t)blockIdx.x * chunk;
  const int n = (int)min((int64_t)chunk, a.n_vocab - v0);
  const uint32_t low = (uint32_t)v0, vocab = (uint32_t)a.n_vocab;
  bool bad = false;
  LogRow r;
  log_pass<TI, TO, kLogThreads>(a, b, v0, n, tid, [&] {
    if (kTable) t.clear(chunk, a.output_ids != nullptr);
    if constexpr (kByToken)
      for (int v = tid; v < kLogMinChunk; v += kLogThreads) bias_value[v] = 0.f;
    r = log_row(a, b, kTable, &bad);
    if (!kTable || !r.concerned) return r.mask;
    __syncthreads();
    each_id<kLogIds>(r.prompt, r.n_prompt, r.output, r.n_output, tid, kLogThreads, [&](uint32_t id, bool said) {
      if (id - low < (uint32_t)n) {
        t.see((int)(id - low));
        if (said) t.say((int)(id - low));
      }
      bad |= id >= vocab;
    });
    if (kBias && warp == kLogWarps - 1) {
      // the chunk's biases in their order: added up by token, or listed; past kLogBiases they are only counted
      int m = 0;
      constexpr int kLook = 4;
      for (int64_t j = lane; j - lane < r.n_bias; j += 32 * kLook) {
        uint32_t id[kLook];
        float value[kLook];
#pragma unroll
        for (int q = 0; q < kLook; ++q) {
          const bool have = j + 32 * q < r.n_bias;
          id[q] = have ? (uint32_t)__ldg(r.bias_ids + j + 32 * q) : 0;
          value[q] = have ? __ldg(r.bias_values + j + 32 * q) : 0.f;
          bad |= have && id[q] >= vocab;
          if (!have || id[q] - low >= (uint32_t)n) id[q] = 0xFFFFFFFFu;
        }
#pragma unroll
        for (int q = 0; q < kLook; ++q) {
          const unsigned in_chunk = __ballot_sync(0xFFFFFFFFu, id[q] != 0xFFFFFFFFu);
          const int at = m + __popc(in_chunk & ((1u << lane) - 1));
          if (id[q] != 0xFFFFFFFFu) {
            const int v = (int)(id[q] - low);
            const uint32_t bit = 1u << (v & 31);
            if (atomicOr(&t.biased[v >> 5], bit) & bit) atomicOr(&t.twice[v >> 5], bit);
            if (!kByToken && at < kLogBiases) {
              bias_token[at] = (uint16_t)v;
              bias_value[at] = value[q];
            }
          }
          if constexpr (kByToken)
            if (in_chunk) log_add_bias(bias_value, id[q] != 0xFFFFFFFFu ? (int)(id[q] - low) : -1, value[q], lane);
          m += __popc(in_chunk);
        }
      }
      if (lane == 0) n_biases = m;
      // no token of a chunk is 0xFFFF, which fills the last vector of the list
      if (!kByToken && m + lane < min((m + 7) & ~7, kLogBiases)) bias_token[m + lane] = 0xFFFF;
    }
    return r.mask;
  });
  if (bad) atomicOr(&small->op_status, kStBadInput);
  if (!kTable || !r.concerned) return;
  const int words = (int)((a.n_vocab + 31) >> 5);
  const TI* in = static_cast<const TI*>(a.logits) + b * a.logits_stride + v0;
  TO* out = static_cast<TO*>(a.out) + b * a.out_stride + v0;
  auto open = [&](int v) { return !r.mask || (log_open(r.mask, (int)v0 + v, words) & 1); };
  auto penalised = [&](int v) {
    const float x = to_f32(in[v]);
    return t.seen(v) ? log_penalty(r, x, a.output_ids ? t.times(v) : 0) : x;
  };
  __syncthreads();
  if (r.n_prompt + r.n_output > 0 || kByToken) {
    // list the tokens that are concerned and not shut, but for those with a
    // listed bias, from kLogWords words of bits a thread, and share them out
    static_assert(kLogMaxChunk <= 32 * kLogWords * kLogThreads);
    uint32_t bits[kLogWords];
    int mine = 0;
#pragma unroll
    for (int q = 0; q < kLogWords; ++q) {
      const int w = tid + q * kLogThreads;
      bits[q] = w >= (n + 31) / 32 ? 0 : kByToken ? t.bits[w] | t.biased[w] : t.bits[w] & ~t.biased[w];
      if (r.mask && bits[q]) bits[q] &= __ldg(r.mask + (v0 >> 5) + w);
      mine += __popc(bits[q]);
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int k = 0; k < kLogWarps; ++k) {
      if (k < warp) upto += warp_sum[k];
      total += warp_sum[k];
    }
    for (int k0 = 0; k0 < total; k0 += kLogList) {
      int at = upto - mine - k0;
#pragma unroll
      for (int q = 0; q < kLogWords; ++q)
        for (uint32_t m = bits[q]; m; m &= m - 1, ++at)
          if ((uint32_t)at < kLogList) list[at] = (uint16_t)((tid + q * kLogThreads) * 32 + __ffs(m) - 1);
      __syncthreads();
      for (int k = tid; k < min(total - k0, kLogList); k += kLogThreads) {
        const int v = list[k];
        out[v] = from_f32<TO>(kByToken ? penalised(v) + bias_value[v] : penalised(v));
      }
      if (k0 + kLogList < total) __syncthreads();
    }
  }
  if (!kBias || kByToken) return;
  const int m = n_biases;
  if (m <= kLogBiases) {
    // whoever has a token's first bias adds up all of them; from the last
    // thread on, since the first ones have most of the list above
    for (int k = kLogThreads - 1 - tid; k < m; k += kLogThreads) {
      const int v = bias_token[k];
      float sum = bias_value[k];
      bool first = true;
      if (t.twice[v >> 5] >> (v & 31) & 1) {
        for (int o0 = 0; o0 < m && first; o0 += 8) {
          if (!log_equal(*reinterpret_cast<const uint4*>(bias_token + o0), (uint32_t)v * 0x10001u)) continue;
          for (int o = o0; o < min(o0 + 8, m); ++o) {
            if (bias_token[o] != v) continue;
            first &= o >= k;
            if (o > k) sum += bias_value[o];
          }
        }
      }
      if (first && open(v)) out[v] = from_f32<TO>(penalised(v) + sum);
    }
  } else {
    // more than the list holds: tokens with one bias from the row's own list ...
    for (int64_t k = tid; k < r.n_bias; k += kLogThreads) {
      const uint32_t v = (uint32_t)__ldg(r.bias_ids + k) - low;
      if (v >= (uint32_t)n || (t.twice[v >> 5] >> (v & 31) & 1)) continue;
      if (open((int)v)) out[v] = from_f32<TO>(penalised((int)v) + __ldg(r.bias_values + k));
    }
    // ... and those with more, numbered in the order of their ids, kLogBiases at
    // a time: each warp adds up its share of them in one walk over that list, so
    // the work is linear in it. 64 rows of 113,645 bf16, one of them with 30,000
    // biases in pairs: 0.86 ms (0.2 with a token each); a search for each took 149.
    __syncthreads();
    uint16_t* number = list;  // [n / 32] how many there are before a word's
    const int n_words = (n + 31) / 32;
    if (warp == 0) {
      int before = 0;
      for (int w0 = 0; w0 < n_words; w0 += 32) {
        const int here = w0 + lane < n_words ? __popc(t.twice[w0 + lane]) : 0;
        int upto = here;
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
          if (lane >= d) upto += o;
        }
        if (w0 + lane < n_words) number[w0 + lane] = (uint16_t)(before + upto - here);
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
      if (lane == 0) n_biases = before;
    }
    __syncthreads();
    const int several = n_biases;
    for (int s0 = 0; s0 < several; s0 += kLogBiases) {
      log_sum_several(bias_value + warp * kLogShare, number, t.twice, r.bias_ids, r.bias_values, r.n_bias, low,
                      (uint32_t)n, s0 + warp * kLogShare, lane);
      __syncthreads();
      for (int w = tid; w < n_words; w += kLogThreads) {
        int at = number[w] - s0;
        for (uint32_t m = t.twice[w]; m; m &= m - 1, ++at) {
          const int v = w * 32 + __ffs(m) - 1;
          if ((uint32_t)at < kLogBiases && open(v)) out[v] = from_f32<TO>(penalised(v) + bias_value[at]);
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace

extern "C" int bpe_adjust_logits(bpe_handle* h, const bpe_logits_args* args, bpe_stream_t stream) {
  return guarded("bpe_adjust_logits", [&]() -> int {
    if (!h || !args) return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: null handle or arguments");
    const bpe_logits_args& a = *args;
    if (!type_ok(a.logits_type) || !type_ok(a.out_type))
      return fail(BPE_ERR_INVALID_ARG, "bpe_adjust_logits: unknown type");
    if (a.n_rows < 0 || a.n_rows > 65535 || a.n_vocab < 0 || a.n_vocab >= INT32_MAX || a.n_prompt_ids < 0 ||
        a.output_capacity < 0 || a.output_capacity >= (1 << 29) || a.n_bias < 0 || a.n_bias > INT32_MAX ||
        a.n_masks < 0)
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
    const bool by_bias = a.bias_ids && a.n_bias > 0;
    const bool table = by_bias || (a.prompt_ids && a.repetition) ||
                       (a.output_ids && (a.repetition || a.frequency || a.presence));
    if (!table && !a.mask && a.logits == a.out) return BPE_OK;
    // Tokens of a CTA: long chunks read the history less often and hide its
    // latency behind a longer pass; short ones spread few rows over more SMs,
    // and leave room for counts. At least 2 CTAs an SM: 100 rows of 32,256 f16
    // take 8.3 us, with 5 at least 9.4, with 1 9.2; 48 rows of 69,424 bf16 take
    // 12.2 us either way, with 1 at least 14.
    const int wide = !a.output_ids || a.output_capacity <= kLogSaid ? 0 : a.output_capacity <= 0xFFFF ? 16 : 32;
    int chunk = !table || !wide ? kLogMaxChunk : wide == 16 ? kLogDenseChunk : kLogDenseChunk / 2;
    while (chunk > kLogMinChunk && a.n_rows * ((a.n_vocab + chunk - 1) / chunk) < kLogBlocks * h->n_sms) chunk /= 2;
    // four times the mean biases of a chunk fit its list
    if (by_bias)
      while (chunk > kLogMinChunk &&
             4 * (a.n_bias / a.n_rows) * chunk / std::max<int64_t>(a.n_vocab, chunk) > kLogBiases)
        chunk /= 2;
    const dim3 grid((unsigned)((a.n_vocab + chunk - 1) / chunk), (unsigned)a.n_rows);
    return with_type(a.logits_type, [&](auto i) {
      return with_type(a.out_type, [&](auto o) -> int {
        using TI = decltype(i);
        using TO = decltype(o);
        auto launch = [&](auto with_table, auto with_bias, auto by_token) {
          constexpr bool kTable = decltype(with_table)::value, kBias = decltype(with_bias)::value,
                         kByToken = decltype(by_token)::value;
          const int smem = (kTable ? LogTable::bytes(chunk, a.output_ids != nullptr, wide) : 0) +
                           (!kBias ? 0 : kByToken ? 4 * kLogMinChunk : 6 * kLogBiases);
          k_logits<TI, TO, kTable, kBias, kByToken><<<grid, kLogThreads, smem, st>>>(a, chunk, wide, h->d_small);
          CK(cudaGetLastError());
          return (int)BPE_OK;
        };
        using Yes = std::true_type;
        using No = std::false_type;
        if (!table) return launch(No{}, No{}, No{});
        if (!by_bias) return launch(Yes{}, No{}, No{});
        return chunk <= kLogMinChunk ? launch(Yes{}, Yes{}, Yes{}) : launch(Yes{}, Yes{}, No{});
      });
    });
  });
}
