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

struct PlanArgs {
  const int64_t* offsets;  // [n + 1] or null: one new token each
  const int32_t* cached;   // [n] or null: none
  int64_t n, n_free, max_blocks, table_stride, n_slots;
  FastDiv block;
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
  int64_t first, fresh;       // first new token, new tokens
  int32_t cached;             // tokens in the cache
  uint32_t held, gets;        // blocks it has, blocks it needs
  bool ok;
};

__device__ __forceinline__ PlanRequest plan_request(const PlanArgs& a, int64_t i) {
  PlanRequest r;
  const int64_t end = a.offsets ? __ldg(a.offsets + i + 1) : i + 1;
  r.first = a.offsets ? __ldg(a.offsets + i) : i;
  r.cached = a.cached ? __ldg(a.cached + i) : 0;
  r.fresh = end - r.first;
  // the sum below INT32_MAX - block + 1, so that rounding up to blocks stays below 2^31
  r.ok = r.first >= 0 && end >= r.first && end <= a.n_slots && r.cached >= 0 &&
         r.cached + r.fresh <= (int64_t)INT32_MAX - (int64_t)a.block.d + 1;
  r.held = r.gets = 0;
  if (r.ok) {
    r.held = a.block((uint32_t)r.cached + a.block.d - 1);
    const uint32_t want = a.block((uint32_t)(r.cached + r.fresh) + a.block.d - 1);
    r.ok = want <= a.max_blocks;
    if (r.ok) r.gets = want - r.held;
    else r.held = 0;
  }
  return r;
}

__device__ __forceinline__ int64_t plan_head(const PlanArgs& a, bool* bad) {
  const int64_t head = a.head ? __ldg(a.head) : 0;
  *bad = head < 0 || head > a.n_free;
  return *bad ? a.n_free : head;
}

// Inclusive sum over a block of kWarps warps, and the block's total.
template <int kWarps>
__device__ __forceinline__ int64_t plan_scan(int64_t x, int64_t* total, int64_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += o;
  }
  __syncthreads();  // warp_sum may still be read from the last call
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int64_t w = lane < kWarps ? warp_sum[lane] : 0;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, w, d);
    if (lane >= d) w += o;
  }
  const int64_t below = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
  *total = __shfl_sync(0xFFFFFFFFu, w, kWarps - 1);
  return warp > 0 ? x + below : x;
}

// Raises *to to the largest x of the block's threads.
__device__ __forceinline__ void plan_max(unsigned long long* to, unsigned long long x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = max(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
  if ((threadIdx.x & 31) == 0 && x) atomicMax(to, x);
}

// What the tokens [t0, t1) of a tile need of their requests: the last request
// that starts at or before t, for each. Requests that start inside the tile
// have their first token in shared memory if they are no more than kPlanTile;
// else (many empty ones) a token searches the offsets themselves.
constexpr int kPlanThreads = 256;
constexpr int kPlanTile = 1024;  // tokens of a block

__device__ __forceinline__ int64_t plan_upper(const int64_t* offsets, int64_t lo, int64_t hi, int64_t t) {
  while (lo < hi) {
    const int64_t mid = lo + ((hi - lo) >> 1);
    if (__ldg(offsets + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// The same by a warp, 32 offsets a step.
__device__ __forceinline__ int64_t plan_upper_warp(const int64_t* offsets, int64_t n, int64_t t) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = n;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;
    const bool below = at < hi && __ldg(offsets + at) <= t;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, below));  // offsets rise, so these are the first k
    hi = min(hi, lo + (k + 1) * step - 1);
    lo = min(lo + k * step, hi);
  }
  return lo;
}

struct PlanTile {
  int64_t low, count;  // requests before the tile's first that starts in it; how many start in it
  int32_t start[kPlanTile];
};

__device__ __forceinline__ void plan_tile(const PlanArgs& a, int64_t t0, int64_t t1, PlanTile& p) {
  const int warp = threadIdx.x >> 5;
  if (a.offsets && warp < 2) {
    const int64_t u = plan_upper_warp(a.offsets, a.n, warp == 0 ? t0 : t1 - 1);
    if ((threadIdx.x & 31) == 0) (warp == 0 ? p.low : p.count) = u;
  }
  __syncthreads();
  if (a.offsets && p.count - p.low <= kPlanTile)
    for (int64_t k = threadIdx.x; k < p.count - p.low; k += kPlanThreads)
      p.start[k] = (int32_t)(__ldg(a.offsets + p.low + k) - t0);
  __syncthreads();
}

// Slots, positions and table entries of the tile's tokens; base(i) is G_i -
// g_i of request i, or -1 where it is not served. A block that is dealt has
// one token in its first slot, and that token writes its table entry.
template <class B>
__device__ __forceinline__ void plan_tokens(const PlanArgs& a, int64_t t0, int64_t t1, const PlanTile& p, int64_t head,
                                            B base) {
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kPlanThreads) {
    int64_t i = t;
    if (a.offsets) {
      const int64_t count = p.count - p.low;
      if (count >= 0 && count <= kPlanTile) {
        int lo = 0, hi = (int)count;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (p.start[mid] <= t - t0) lo = mid + 1;
          else hi = mid;
        }
        i = p.low + lo - 1;
      } else {
        i = plan_upper(a.offsets, 0, a.n, t) - 1;
      }
    }
    int64_t slot = -1;
    uint32_t position = 0;
    if (i >= 0 && i < a.n) {
      const PlanRequest r = plan_request(a, i);
      if (r.ok && t >= r.first && t < r.first + r.fresh) {
        position = (uint32_t)(r.cached + (t - r.first));
        const int64_t dealt = base(i);
        if (dealt >= 0) {
          const uint32_t b = a.block(position), in = position - b * a.block.d;
          int32_t* entry = a.table + i * a.table_stride + b;
          int32_t q;
          if (b < r.held) {
            q = *entry;
          } else {
            q = __ldg(a.free_list + head + dealt + (b - r.held));
            if (in == 0) *entry = q;
          }
          slot = (int64_t)q * a.block.d + in;
        }
      }
    }
    __stcs(a.slots + t, slot);
    __stcs(a.positions + t, (int32_t)position);
  }
}

// Up to kPlanOne requests: every block adds up all requests' blocks itself,
// which takes less time than a launch, and plans its tile of tokens.
constexpr int kPlanOne = 2048;

__global__ void __launch_bounds__(kPlanThreads) k_plan_one(PlanArgs a) {
  constexpr int kPer = kPlanOne / kPlanThreads;
  __shared__ PlanTile tile;
  __shared__ int64_t base[kPlanOne];
  __shared__ int64_t warp_sum[kPlanThreads / 32];
  __shared__ unsigned long long taken;
  const int tid = threadIdx.x, n = (int)a.n;
  const bool lead = blockIdx.x == 0;
  bool bad;
  const int64_t head = plan_head(a, &bad), room = a.n_free - head;
  if (tid == 0) taken = 0;
  PlanRequest r[kPer];
  int64_t mine = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = tid * kPer + q;
    if (i >= n) continue;
    r[q] = plan_request(a, i);
    mine += r[q].gets;
    bad |= !r[q].ok;
  }
  int64_t total;
  int64_t upto = plan_scan<kPlanThreads / 32>(mine, &total, warp_sum) - mine;
  unsigned long long best = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = tid * kPer + q;
    if (i >= n) continue;
    upto += r[q].gets;
    const bool served = r[q].ok && (r[q].gets == 0 || upto <= room);
    base[i] = served ? upto - r[q].gets : -1;
    if (upto <= room) best = (unsigned long long)upto;
    if (lead) a.seq_lens[i] = served ? (int32_t)(r[q].cached + r[q].fresh) : max(r[q].cached, 0);
  }
  if (lead) plan_max(&taken, best);
  if (lead && bad) atomicOr(&a.small->op_status, kStBadInput);
  const int64_t t0 = (int64_t)blockIdx.x * kPlanTile, t1 = min(t0 + kPlanTile, a.n_slots);
  plan_tile(a, t0, t1, tile);  // its barriers also publish base and taken
  if (lead && tid == 0) {
    a.info[0] = head + (int64_t)taken;
    a.info[1] = max((int64_t)0, total - room);
  }
  plan_tokens(a, t0, t1, tile, head, [&](int64_t i) { return base[i]; });
}

// More requests: one cluster adds up their blocks (a CTA a contiguous part, the
// parts' totals read through distributed shared memory) ...
constexpr int kPlanCluster = 8;
constexpr int kPlanSumThreads = 1024;

__global__ void __cluster_dims__(kPlanCluster, 1, 1) __launch_bounds__(kPlanSumThreads) k_plan_requests(PlanArgs a) {
  constexpr int kWarps = kPlanSumThreads / 32;
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int64_t part;
  __shared__ unsigned long long taken;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster.block_rank();
  let_next_begin();
  bool bad;
  const int64_t head = plan_head(a, &bad), room = a.n_free - head;
  const int64_t per = (a.n + kPlanCluster - 1) / kPlanCluster;
  const int64_t i0 = min(rank * per, a.n), i1 = min(i0 + per, a.n);
  int64_t mine = 0, total;
  for (int64_t i = i0 + tid; i < i1; i += kPlanSumThreads) mine += plan_request(a, i).gets;
  plan_scan<kWarps>(mine, &total, warp_sum);
  if (tid == 0) {
    part = total;
    taken = 0;
  }
  cluster.sync();
  int64_t carry = 0, all = 0;
#pragma unroll
  for (int q = 0; q < kPlanCluster; ++q) {
    const int64_t v = *cluster.map_shared_rank(&part, q);
    all += v;
    if (q < rank) carry += v;
  }
  unsigned long long best = 0;
  for (int64_t j = i0; j < i1; j += kPlanSumThreads) {
    const int64_t i = j + tid;
    PlanRequest r{};
    if (i < i1) {
      r = plan_request(a, i);
      bad |= !r.ok;
    }
    const int64_t upto = carry + plan_scan<kWarps>(r.gets, &total, warp_sum);
    carry += total;
    if (i < i1) {
      const bool served = r.ok && (r.gets == 0 || upto <= room);
      if (upto <= room) best = max(best, (unsigned long long)upto);
      a.base[i] = served ? upto - r.gets : -1;
      a.seq_lens[i] = served ? (int32_t)(r.cached + r.fresh) : max(r.cached, 0);
    }
  }
  plan_max(&taken, best);
  if (bad) atomicOr(&a.small->op_status, kStBadInput);
  cluster.sync();
  if (rank == 0 && tid == 0) {
    best = 0;
#pragma unroll
    for (int q = 0; q < kPlanCluster; ++q) best = max(best, *cluster.map_shared_rank(&taken, q));
    a.info[0] = head + (int64_t)best;
    a.info[1] = max((int64_t)0, all - room);
  }
  cluster.sync();  // the others' shared memory stays until it is read
}

// ... and the blocks of a second launch plan their tiles of tokens, having
// found their requests while the first one ran.
__global__ void __launch_bounds__(kPlanThreads) k_plan_tokens(PlanArgs a) {
  __shared__ PlanTile tile;
  bool bad;
  const int64_t head = plan_head(a, &bad);
  const int64_t t0 = (int64_t)blockIdx.x * kPlanTile, t1 = min(t0 + kPlanTile, a.n_slots);
  plan_tile(a, t0, t1, tile);
  await_previous();
  plan_tokens(a, t0, t1, tile, head, [&](int64_t i) { return __ldcg(a.base + i); });
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
    auto overlap = [](const void* p, int64_t n, const void* q, int64_t m) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
      return p && q && x < y + (uintptr_t)m && y < x + (uintptr_t)n;
    };
    // blocks read the head and the lengths while others write their successors
    if (overlap(d_info, 16, d_head, 8) || overlap(d_seq_lens, n_requests * 4, d_cached, n_requests * 4))
      return fail(BPE_ERR_INVALID_ARG, "bpe_plan_blocks: d_info and d_seq_lens cannot replace d_head and d_cached in place");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    PlanArgs a{d_offsets, d_cached, n_requests, n_free, max_blocks, table_stride, n_slots, FastDiv(block_size), d_free,
               d_head, d_table, d_seq_lens, d_slots, d_positions, d_info, nullptr, h->d_small};
    const unsigned tiles = (unsigned)((n_slots + kPlanTile - 1) / kPlanTile);
    if (n_requests <= kPlanOne) {
      k_plan_one<<<std::max(1u, tiles), kPlanThreads, 0, st>>>(a);
      CK(cudaGetLastError());
      return BPE_OK;
    }
    int rc = ensure_ws(h, (size_t)n_requests * sizeof(int64_t));
    if (rc) return rc;
    a.base = static_cast<int64_t*>(h->d_ws);
    k_plan_requests<<<kPlanCluster, kPlanSumThreads, 0, st>>>(a);
    CK(cudaGetLastError());
    if (tiles) CK(launch_after(k_plan_tokens, dim3(tiles), kPlanThreads, 0, st, a));
    return BPE_OK;
  });
}

}  // extern "C"
