// Block tables, cache slots and positions of a batch of requests, from their
// lengths on the device.
//
// Included once by model_ops.cu; not a standalone header.
//
// Request i has c_i tokens in the cache, in h_i = ceil(c_i / s) blocks of s
// slots, and m_i new ones, so it needs g_i = ceil((c_i + m_i) / s) - h_i more
// blocks. They are dealt from the free list in request order: with
// G_i = g_0 + .. + g_i and A blocks left in the list, request i is served if
// g_i = 0 or G_i <= A, and takes the list's entries [G_i - g_i, G_i).

namespace {

constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int64_t* offsets;  // [n + 1] or null: one new token each
  const int32_t* cached;   // [n] or null: none
  int64_t n, block, n_free, max_blocks, table_stride, n_slots;
  const int32_t* free_list;
  const int64_t* head;     // entries of the free list already taken, or null: none
  int32_t* table;
  int32_t* seq_lens;
  int64_t* slots;
  int32_t* positions;
  int64_t* info;
  int64_t* base;           // [n] workspace: G_i - g_i, or -1 where not served
  DevSmall* small;
};

struct PlanRequest {
  int64_t first, cached, fresh;  // first new token, tokens in the cache, new tokens
  int64_t held, gets;            // blocks it has, blocks it needs
  bool ok;
};

__device__ __forceinline__ PlanRequest plan_request(const PlanArgs& a, int64_t i) {
  PlanRequest r;
  const int64_t end = a.offsets ? a.offsets[i + 1] : i + 1;
  r.first = a.offsets ? a.offsets[i] : i;
  r.cached = a.cached ? a.cached[i] : 0;
  r.fresh = end - r.first;
  r.ok = r.first >= 0 && end >= r.first && end <= a.n_slots && r.cached >= 0 && r.cached + r.fresh <= INT32_MAX;
  if (r.ok) {
    r.held = (r.cached + a.block - 1) / a.block;
    const int64_t want = (r.cached + r.fresh + a.block - 1) / a.block;
    r.gets = want - r.held;
    r.ok = want <= a.max_blocks;
  }
  if (!r.ok) r.held = r.gets = 0;
  return r;
}

// One CTA: the blocks of every request, its length and its table entries.
__global__ void __launch_bounds__(kPlanThreads) k_plan_requests(PlanArgs a) {
  __shared__ int64_t warp_sum[kPlanThreads / 32];
  __shared__ int64_t carry, taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t head = a.head ? *a.head : 0;
  if (head < 0 || head > a.n_free) {
    if (tid == 0) atomicOr(&a.small->op_status, kStBadInput);
    head = a.n_free;
  }
  const int64_t room = a.n_free - head;
  if (tid == 0) carry = taken = 0;
  for (int64_t i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int64_t i = i0 + tid;
    PlanRequest r{};
    if (i < a.n) {
      r = plan_request(a, i);
      if (!r.ok) atomicOr(&a.small->op_status, kStBadInput);
    }
    int64_t upto = r.gets;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += warp_sum[w];
    upto += carry;
    __syncthreads();
    if (tid == kPlanThreads - 1) carry = upto;
    if (i < a.n) {
      const bool served = r.ok && (r.gets == 0 || upto <= room);
      const int64_t base = upto - r.gets;
      if (upto <= room) atomicMax((unsigned long long*)&taken, (unsigned long long)upto);
      a.base[i] = served ? base : -1;
      a.seq_lens[i] = (int32_t)(served ? r.cached + r.fresh : r.cached > 0 ? r.cached : 0);
      if (served)
        for (int64_t k = 0; k < r.gets; ++k) a.table[i * a.table_stride + r.held + k] = a.free_list[head + base + k];
    }
    __syncthreads();
  }
  if (tid == 0) {
    a.info[0] = head + taken;
    a.info[1] = carry > room ? carry - room : 0;
  }
}

__global__ void __launch_bounds__(256) k_plan_tokens(PlanArgs a) {
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < a.n_slots; t += (int64_t)gridDim.x * 256) {
    int64_t slot = -1, position = 0;
    // the last request that starts at or before t
    int64_t lo = 0, hi = a.n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if ((a.offsets ? a.offsets[mid] : mid) <= t) lo = mid + 1;
      else hi = mid;
    }
    if (lo > 0) {
      const int64_t i = lo - 1;
      const PlanRequest r = plan_request(a, i);
      if (r.ok && t >= r.first && t < r.first + r.fresh) {
        position = r.cached + t - r.first;
        if (a.base[i] >= 0) {
          const int64_t b = position / a.block;
          slot = (int64_t)a.table[i * a.table_stride + b] * a.block + (position - b * a.block);
        }
      }
    }
    a.slots[t] = slot;
    a.positions[t] = (int32_t)position;
  }
}

}  // namespace

extern "C" {

int bpe_plan_blocks(bpe_handle* h, const int64_t* d_offsets, const int32_t* d_cached, int64_t n_requests,
                    int64_t block_size, const int32_t* d_free, int64_t n_free, const int64_t* d_head,
                    int32_t* d_table, int64_t max_blocks, int64_t table_stride, int32_t* d_seq_lens, int64_t* d_slots,
                    int32_t* d_positions, int64_t n_slots, int64_t* d_info, bpe_stream_t stream) {
  return guarded("bpe_plan_blocks", [&]() -> int {
    if (!h) return fail(BPE_ERR_INVALID_ARG, "bpe_plan_blocks: null handle");
    if (n_requests < 0 || n_requests >= INT32_MAX || block_size < 1 || block_size > INT32_MAX || n_free < 0 ||
        max_blocks < 0 || n_slots < 0 || n_slots >= INT32_MAX)
      return fail(BPE_ERR_INVALID_ARG, "bpe_plan_blocks: a size is negative or too large");
    if (n_requests > 1 && table_stride < max_blocks)
      return fail(BPE_ERR_INVALID_ARG, "bpe_plan_blocks: table rows overlap");
    if (!d_offsets && n_slots < n_requests)
      return fail(BPE_ERR_INVALID_ARG, "bpe_plan_blocks: n_slots is below one new token a request");
    if (!d_info || (n_requests > 0 && (!d_seq_lens || (max_blocks > 0 && !d_table))) ||
        (n_slots > 0 && (!d_slots || !d_positions)) || (n_free > 0 && !d_free))
      return fail(BPE_ERR_INVALID_ARG, "bpe_plan_blocks: null pointer");
    if (!aligned(d_offsets, 8) || !aligned(d_cached, 4) || !aligned(d_free, 4) || !aligned(d_head, 8) ||
        !aligned(d_table, 4) || !aligned(d_seq_lens, 4) || !aligned(d_slots, 8) || !aligned(d_positions, 4) ||
        !aligned(d_info, 8))
      return fail(BPE_ERR_INVALID_ARG, "bpe_plan_blocks: a pointer is not aligned to its elements");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    int rc = ensure_ws(h, (size_t)n_requests * sizeof(int64_t));
    if (rc) return rc;
    const PlanArgs a{d_offsets, d_cached, n_requests, block_size, n_free, max_blocks, table_stride, n_slots, d_free,
                     d_head, d_table, d_seq_lens, d_slots, d_positions, d_info, static_cast<int64_t*>(h->d_ws),
                     h->d_small};
    k_plan_requests<<<1, kPlanThreads, 0, st>>>(a);
    CK(cudaGetLastError());
    if (n_slots > 0) {
      k_plan_tokens<<<(unsigned)std::min<int64_t>((n_slots + 255) / 256, 65535), 256, 0, st>>>(a);
      CK(cudaGetLastError());
    }
    return BPE_OK;
  });
}

}  // extern "C"
