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
//
// Where offsets fall, a request that begins below an earlier offset is refused,
// for its tokens may be another's too. One that is left begins at the largest
// offset so far, and a search of these largest offsets finds its tokens as a
// search of the offsets does where none falls.

namespace {

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
  int64_t* high;           // [n] workspace, where offsets fall: the largest of offsets[0 .. i]
  int64_t* falls;          // [1] workspace: whether they do
  DevSmall* small;
};

struct PlanRequest {
  int64_t first, fresh;       // first new token, new tokens
  int32_t cached;             // tokens in the cache
  uint32_t held, gets;        // blocks it has, blocks it needs
  bool ok, falls;             // falls: its end is below its first token
};

__device__ __forceinline__ PlanRequest plan_request(const PlanArgs& a, int64_t i) {
  PlanRequest r;
  const int64_t end = a.offsets ? __ldg(a.offsets + i + 1) : i + 1;
  r.first = a.offsets ? __ldg(a.offsets + i) : i;
  r.cached = a.cached ? __ldg(a.cached + i) : 0;
  r.fresh = (int64_t)((uint64_t)end - (uint64_t)r.first);  // of any two numbers
  r.falls = end < r.first;
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

// Inclusive sum over a block of kWarps warps, and the block's total. kFirst: no
// thread can still be reading warp_sum.
template <int kWarps, bool kFirst = false>
__device__ __forceinline__ int64_t plan_scan(int64_t x, int64_t* total, int64_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += o;
  }
  if (!kFirst) __syncthreads();  // warp_sum may still be read from the last call
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

// The largest x of the threads before this one (INT64_MIN for the first), and of
// a block of kWarps warps.
template <int kWarps>
__device__ __noinline__ int64_t plan_highest_before(int64_t x, int64_t* block_most, int64_t* warp_most) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x = max(x, o);
  }
  int64_t before = __shfl_up_sync(0xFFFFFFFFu, x, 1);
  if (lane == 0) before = INT64_MIN;
  __syncthreads();  // warp_most may still be read from the last call
  if (lane == 31) warp_most[warp] = x;
  __syncthreads();
  *block_most = INT64_MIN;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before = max(before, warp_most[w]);
    *block_most = max(*block_most, warp_most[w]);
  }
  return before;
}

// Raises *to to the largest x of the block's threads.
__device__ __forceinline__ void plan_max(unsigned long long* to, unsigned long long x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = max(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
  if ((threadIdx.x & 31) == 0 && x) atomicMax(to, x);
}

constexpr int kPlanThreads = 256;
constexpr int kPlanPairs = 4;                                // pairs of tokens of a thread, at most
constexpr int kPlanTile = kPlanThreads * 2 * kPlanPairs;     // tokens of a block, at most
constexpr int kPlanList = 2048;                              // requests that a block lists

// Consecutive requests, in shared memory.
struct PlanList {
  int32_t start[kPlanList + 1];  // first new token (the largest offset so far), relative to the tile's
  int32_t cached[kPlanList];     // -1 - (what is in the cache) for a request that is not ok
  int32_t held[kPlanList];
  int32_t base[kPlanList];       // G_i - g_i, -1 where not served
};

__device__ __forceinline__ int32_t plan_relative(int64_t offset, int64_t t0) {
  return (int32_t)min(max(offset - t0, (int64_t)INT32_MIN), (int64_t)INT32_MAX);
}

// Slots, positions and table entries of the tokens [t0, t1), whose requests
// are `first` and the next ones in the list. A thread takes pairs of
// neighbours: one search finds both, and they are stored as one vector. Its
// pairs step together, so that their loads overlap. A block that is dealt has
// one token in its first slot, and that token writes its table entry.
__device__ __forceinline__ void plan_tokens(const PlanArgs& a, int64_t t0, int64_t t1, int64_t head, int64_t first,
                                            int count, const PlanList& list) {
  const int len = (int)(t1 - t0);
  const bool vectors =
      ((reinterpret_cast<uintptr_t>(a.slots + t0) & 15) | (reinterpret_cast<uintptr_t>(a.positions + t0) & 7)) == 0;
  const int32_t* free_list = a.free_list + head;
  int32_t position[kPlanPairs][2], in[kPlanPairs][2], entry[kPlanPairs][2];
  int32_t* dealt[kPlanPairs][2];  // the table entry that the token writes, or null
#pragma unroll
  for (int q = 0; q < kPlanPairs; ++q) {
    const int at = 2 * (int)threadIdx.x + 2 * kPlanThreads * q;
    int l = 0;
    if (at < len) {
      if (a.offsets) {
        int h = count;
        while (l < h) {
          const int mid = (l + h) >> 1;
          if (list.start[mid] <= at) l = mid + 1;
          else h = mid;
        }
      } else {
        l = (int)min(t0 - first + at + 1, (int64_t)count);  // request t is token t's
      }
    }
    --l;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = at + e;
      while (e == 1 && x < len && l + 1 < count && list.start[l + 1] <= x) ++l;
      position[q][e] = 0;
      in[q][e] = -1;
      dealt[q][e] = nullptr;
      if (x >= len || l < 0) continue;
      const int32_t from = list.start[l], c = list.cached[l];
      if (c < 0 || x < from || x >= list.start[l + 1]) continue;
      const uint32_t p = (uint32_t)(c + (x - from));
      position[q][e] = (int32_t)p;
      const int32_t base = list.base[l];
      if (base < 0) continue;
      const uint32_t b = a.block(p);
      in[q][e] = (int32_t)(p - b * a.block.d);
      const int32_t fresh = (int32_t)b - list.held[l];
      int32_t* row = a.table + (first + l) * a.table_stride + b;
      entry[q][e] = *(fresh < 0 ? row : free_list + base + fresh);
      if (fresh >= 0 && in[q][e] == 0) dealt[q][e] = row;
    }
  }
#pragma unroll
  for (int q = 0; q < kPlanPairs; ++q) {
    const int at = 2 * (int)threadIdx.x + 2 * kPlanThreads * q;
    if (at >= len) break;
    int64_t slot[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      slot[e] = in[q][e] < 0 ? -1 : (int64_t)entry[q][e] * a.block.d + in[q][e];
      if (dealt[q][e]) *dealt[q][e] = entry[q][e];
    }
    if (vectors && at + 1 < len) {
      __stcs(reinterpret_cast<longlong2*>(a.slots + t0 + at), make_longlong2(slot[0], slot[1]));
      __stcs(reinterpret_cast<int2*>(a.positions + t0 + at), make_int2(position[q][0], position[q][1]));
    } else {
      for (int e = 0; e < 2 && at + e < len; ++e) {
        a.slots[t0 + at + e] = slot[e];
        a.positions[t0 + at + e] = position[q][e];
      }
    }
  }
}

// Takes the requests that begin below an earlier offset out of a list of all n,
// `per` a thread: their cached becomes -1 - cached. All starts become the
// largest offset so far. seq_lens may be null.
__device__ __noinline__ void plan_refuse(const int64_t* offsets, int32_t* seq_lens, int n, int per, int64_t t0,
                                         PlanList& list, int64_t* warp_most) {
  const int i0 = min((int)threadIdx.x * per, n), i1 = min(i0 + per, n);
  int64_t high = INT64_MIN, most;
  for (int i = i0; i < i1; ++i) high = max(high, __ldg(offsets + i));
  high = plan_highest_before<kPlanThreads / 32>(high, &most, warp_most);
  for (int i = i0; i < i1; ++i) {
    const int64_t first = __ldg(offsets + i);
    high = max(high, first);
    list.start[i] = plan_relative(high, t0);
    if (first >= high) continue;
    if (list.cached[i] >= 0) list.cached[i] = -1 - list.cached[i];
    if (seq_lens) seq_lens[i] = -1 - list.cached[i];
  }
  if (threadIdx.x == 0) list.start[n] = plan_relative(max(most, __ldg(offsets + n)), t0);
  __syncthreads();  // warp_most is read
}

// Up to kPlanList requests: every block adds up all requests' blocks itself,
// which takes less time than a launch, and plans its tile of tokens from the
// list that it then has. Latency: 3.1 us for 8 single tokens, 3.9 us for 500
// requests with 8,000 tokens (8.0 with a search of the offsets for each token).
__global__ void __launch_bounds__(kPlanThreads) k_plan_one(PlanArgs a, int tile) {
  constexpr int kPer = kPlanList / kPlanThreads;
  __shared__ PlanList list;
  __shared__ int64_t warp_sum[kPlanThreads / 32];
  __shared__ unsigned long long taken;
  const int tid = threadIdx.x, n = (int)a.n;
  const int64_t t0 = (int64_t)blockIdx.x * tile, t1 = min(t0 + tile, a.n_slots);
  const bool lead = blockIdx.x == 0;
  bool bad;
  const int64_t head = plan_head(a, &bad), room = a.n_free - head;
  if (tid == 0) taken = 0;
  // thread t has requests [t * per, t * per + per)
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  uint32_t gets[kPer];
  int64_t mine = 0;
  bool falls = false;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = tid * per + q;
    if (q >= per || i >= n) break;
    const PlanRequest r = plan_request(a, i);
    list.start[i] = plan_relative(r.first, t0);
    list.cached[i] = r.ok ? r.cached : -1 - max(r.cached, 0);
    list.held[i] = (int32_t)r.held;
    gets[q] = r.gets;
    mine += r.gets;
    bad |= !r.ok;
    falls |= r.falls;
    if (lead) a.seq_lens[i] = r.ok ? (int32_t)(r.cached + r.fresh) : max(r.cached, 0);
  }
  if (tid == 0) list.start[n] = plan_relative(a.offsets ? __ldg(a.offsets + n) : a.n, t0);
  if (__syncthreads_or(falls)) {
    plan_refuse(a.offsets, lead ? a.seq_lens : nullptr, n, per, t0, list, warp_sum);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (q >= per || tid * per + q >= n || list.cached[tid * per + q] >= 0) continue;
      mine -= gets[q];
      gets[q] = 0;
    }
  }
  int64_t total;
  int64_t upto = plan_scan<kPlanThreads / 32, true>(mine, &total, warp_sum) - mine;
  unsigned long long best = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = tid * per + q;
    if (q >= per || i >= n) break;
    upto += gets[q];
    // a request without new blocks takes no entry, and its sum may be past the list
    const bool served = gets[q] == 0 || upto <= room;
    list.base[i] = served ? (gets[q] ? (int32_t)(upto - gets[q]) : 0) : -1;
    if (upto <= room) best = (unsigned long long)upto;
    if (lead && !served) a.seq_lens[i] = list.cached[i];
  }
  if (lead) plan_max(&taken, best);
  if (lead && bad) atomicOr(&a.small->op_status, kStBadInput);
  __syncthreads();
  if (lead && tid == 0) {
    a.info[0] = head + (int64_t)taken;
    a.info[1] = max((int64_t)0, total - room);
  }
  if (t0 < t1) plan_tokens(a, t0, t1, head, 0, n, list);
}

// More requests: one cluster adds up their blocks (a CTA a contiguous part, the
// parts' totals read through distributed shared memory) ...
constexpr int kPlanCluster = 8;
constexpr int kPlanSumThreads = 1024;

__global__ void __cluster_dims__(kPlanCluster, 1, 1) __launch_bounds__(kPlanSumThreads) k_plan_requests(PlanArgs a) {
  constexpr int kWarps = kPlanSumThreads / 32;
  __shared__ int64_t warp_sum[kWarps];
  __shared__ longlong2 part;  // blocks of this part's requests, and whether offsets fall in it
  __shared__ int64_t part_high;
  __shared__ unsigned long long taken;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, rank = (int)cluster.block_rank();
  let_next_begin();
  bool bad;
  const int64_t head = plan_head(a, &bad), room = a.n_free - head;
  const int64_t per = (a.n + kPlanCluster - 1) / kPlanCluster;
  const int64_t i0 = min(rank * per, a.n), i1 = min(i0 + per, a.n);
  int64_t mine = 0, total;
  bool falls = false;
  for (int64_t i = i0 + tid; i < i1; i += kPlanSumThreads) {
    const PlanRequest r = plan_request(a, i);
    mine += r.gets;
    falls |= r.falls;
  }
  const int any = __syncthreads_or(falls);
  plan_scan<kWarps, true>(mine, &total, warp_sum);
  if (tid == 0) {
    part = make_longlong2(total, any);
    taken = 0;
  }
  cluster.sync();
  int64_t carry = 0, all = 0;
  falls = false;
#pragma unroll
  for (int q = 0; q < kPlanCluster; ++q) {
    const longlong2 v = *cluster.map_shared_rank(&part, q);
    all += v.x;
    if (q < rank) carry += v.x;
    falls |= v.y != 0;
  }
  if (rank == 0 && tid == 0) *a.falls = falls;
  if (falls) {
    // the sums once more, without the requests that begin below an earlier offset
    int64_t high = INT64_MIN, most;
    for (int64_t i = i0 + tid; i < i1; i += kPlanSumThreads) high = max(high, __ldg(a.offsets + i));
    plan_highest_before<kWarps>(high, &most, warp_sum);
    if (tid == 0) part_high = most;
    cluster.sync();
    high = INT64_MIN;
    for (int q = 0; q < rank; ++q) high = max(high, *cluster.map_shared_rank(&part_high, q));
    mine = 0;
    for (int64_t j = i0; j < i1; j += kPlanSumThreads) {
      const int64_t i = j + tid, first = i < i1 ? __ldg(a.offsets + i) : INT64_MIN;
      const int64_t before = max(high, plan_highest_before<kWarps>(first, &most, warp_sum));
      high = max(high, most);
      if (i < i1) {
        a.high[i] = max(before, first);
        if (first >= before) mine += plan_request(a, i).gets;
      }
    }
    plan_scan<kWarps>(mine, &total, warp_sum);
    if (tid == 0) part.x = total;  // all have read what was there: they are past a cluster barrier since
    cluster.sync();
    carry = all = 0;
    for (int q = 0; q < kPlanCluster; ++q) {
      const int64_t v = cluster.map_shared_rank(&part, q)->x;
      all += v;
      if (q < rank) carry += v;
    }
  }
  unsigned long long best = 0;
  for (int64_t j = i0; j < i1; j += kPlanSumThreads) {
    const int64_t i = j + tid;
    PlanRequest r{};
    if (i < i1) {
      r = plan_request(a, i);
      if (falls && r.first < a.high[i]) r.ok = false, r.gets = 0;
      bad |= !r.ok;
    }
    const int64_t upto = carry + plan_scan<kWarps>(r.gets, &total, warp_sum);
    carry += total;
    if (i < i1) {
      const bool served = r.ok && (r.gets == 0 || upto <= room);
      if (upto <= room) best = max(best, (unsigned long long)upto);
      // a request without new blocks takes no entry, and its sum may be past the list
      a.base[i] = served ? (r.gets ? upto - r.gets : 0) : -1;
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
// listed their requests while the first one ran: the last that starts at or
// before the tile, and those that start inside it. Where these are more than
// a list holds (many are empty), the tile's tokens search the offsets.
// 16,384 prompts with 1.5 million tokens: 18.6 us, of which the sums take 9 (a
// cluster's two passes over the lengths) and the tokens 14 alone, bound by the
// latency of a tile's steps rather than by their 18 MB; the first form, with a
// search of the offsets for each token, took 126 us.
__global__ void __launch_bounds__(kPlanThreads) k_plan_tokens(PlanArgs a, int tile) {
  __shared__ PlanList list;
  const int tid = threadIdx.x;
  bool bad;
  const int64_t head = plan_head(a, &bad);
  const int64_t t0 = (int64_t)blockIdx.x * tile, t1 = min(t0 + tile, a.n_slots);
  // the number of requests that start at or before t0, by as many probes a step as threads
  int64_t lo = a.offsets ? 0 : min(t0 + 1, a.n), hi = a.offsets ? a.n : lo;
  while (lo < hi) {
    const int64_t step = (hi - lo + kPlanThreads - 1) / kPlanThreads, at = lo + (tid + 1) * step - 1;
    const int k = __syncthreads_count(at < hi && __ldg(a.offsets + at) <= t0);  // offsets rise: these are the first k
    hi = min(hi, lo + (k + 1) * step - 1);
    lo = min(lo + k * step, hi);
  }
  const int64_t first = max(lo - 1, (int64_t)0);
  int count = 0;      // requests listed
  bool whole = false; // and no other one is the tile's
  while (count < kPlanList && !whole) {
    const int64_t i = first + count + tid;
    bool inside = false;
    if (i < a.n) {
      const PlanRequest r = plan_request(a, i);
      list.start[count + tid] = plan_relative(r.first, t0);
      list.cached[count + tid] = r.ok ? r.cached : -1;
      list.held[count + tid] = (int32_t)r.held;
      inside = r.first < t1;
    } else if (i == a.n) {
      list.start[count + tid] = plan_relative(a.offsets ? __ldg(a.offsets + i) : i, t0);
    }
    const int k = __syncthreads_count(inside);
    whole = k < kPlanThreads;
    count += k;
  }
  // the start after the last listed request, which bounds it
  if (!whole && tid == 0) {
    const int64_t i = min(first + count, a.n);
    list.start[count] = plan_relative(a.offsets ? __ldg(a.offsets + i) : i, t0);
  }
  await_previous();
  const bool falls = __ldcg(a.falls) != 0;  // then the list may lack requests
  for (int k = tid; k < count; k += kPlanThreads) list.base[k] = (int32_t)__ldcg(a.base + first + k);
  __syncthreads();
  whole |= list.start[count] >= t1 - t0 || first + count >= a.n;
  if (whole && !falls) {
    plan_tokens(a, t0, t1, head, first, count, list);
    return;
  }
  const int64_t* starts = falls ? a.high : a.offsets;
  for (int64_t t = t0 + tid; t < t1; t += kPlanThreads) {
    int64_t l = 0, h = a.n;
    while (l < h) {
      const int64_t mid = l + ((h - l) >> 1);
      if (__ldcg(starts + mid) <= t) l = mid + 1;
      else h = mid;
    }
    int64_t slot = -1, position = 0;
    const int64_t i = l - 1;
    if (i >= 0) {
      const PlanRequest r = plan_request(a, i);
      if (r.ok && r.first >= __ldcg(starts + i) && t < r.first + r.fresh) {
        position = r.cached + (t - r.first);
        const int64_t base = __ldcg(a.base + i);
        if (base >= 0) {
          const uint32_t b = a.block((uint32_t)position);
          const int32_t in = (int32_t)((uint32_t)position - b * a.block.d), fresh = (int32_t)b - (int32_t)r.held;
          int32_t* row = a.table + i * a.table_stride + b;
          const int32_t entry = *(fresh < 0 ? row : a.free_list + head + base + fresh);
          if (fresh >= 0 && in == 0) *row = entry;
          slot = (int64_t)entry * a.block.d + in;
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
        n_free > INT32_MAX ||
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
      return fail(BPE_ERR_INVALID_ARG, "bpe_plan_blocks: d_info and d_seq_lens cannot replace d_head and d_cached");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    PlanArgs a{d_offsets, d_cached, n_requests, n_free, max_blocks, table_stride, n_slots, FastDiv(block_size), d_free,
               d_head, d_table, d_seq_lens, d_slots, d_positions, d_info, nullptr, nullptr, nullptr, h->d_small};
    // tokens of a thread: as few as leave at most two blocks an SM, and at most
    // kPlanPairs pairs (1.5 million tokens: 733 blocks)
    const int64_t each = (n_slots + kPlanThreads * 4 * h->n_sms - 1) / (kPlanThreads * 4 * h->n_sms);
    const int tile = 2 * kPlanThreads * (int)std::min<int64_t>(kPlanPairs, std::max<int64_t>(1, each));
    const unsigned tiles = (unsigned)((n_slots + tile - 1) / tile);
    if (n_requests <= kPlanList) {
      k_plan_one<<<std::max(1u, tiles), kPlanThreads, 0, st>>>(a, tile);
      CK(cudaGetLastError());
      return BPE_OK;
    }
    int rc = ensure_ws(h, (2 * (size_t)n_requests + 1) * sizeof(int64_t), st);
    if (rc) return rc;
    a.base = static_cast<int64_t*>(h->d_ws);
    a.high = a.base + n_requests;
    a.falls = a.high + n_requests;
    k_plan_requests<<<kPlanCluster, kPlanSumThreads, 0, st>>>(a);
    CK(cudaGetLastError());
    if (tiles) CK(launch_after(k_plan_tokens, dim3(tiles), kPlanThreads, 0, st, a, tile));
    return BPE_OK;
  });
}

}  // extern "C"
