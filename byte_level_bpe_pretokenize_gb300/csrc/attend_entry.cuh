// bpe_attend: which kernels take a call.
//
// Included once by attend.cu, behind attend.cuh and attend_wide.cuh; not a standalone header.

namespace {

template <class F>
int with_groups(int64_t groups, F f) {
  using std::integral_constant;
  switch (groups) {
    case 1: return f(integral_constant<int, 1>{});
    case 2: return f(integral_constant<int, 2>{});
    case 3: return f(integral_constant<int, 3>{});
    case 4: return f(integral_constant<int, 4>{});
    case 6: return f(integral_constant<int, 6>{});
    default: return f(integral_constant<int, 8>{});
  }
}

}  // namespace

extern "C" {

int bpe_attend(bpe_handle* h, const bpe_attend_args* args, bpe_stream_t stream) {
  return guarded("bpe_attend", [&]() -> int {
    auto bad = [&](const char* what) { return fail(BPE_ERR_INVALID_ARG, std::string("bpe_attend: ") + what); };
    if (!h) return bad("null handle");
    if (!args) return bad("null arguments");
    const bpe_attend_args& p = *args;
    int rc = cache_check("bpe_attend", h, p.cache, p.n_blocks, p.block_stride, p.block_size, p.n_heads, p.dim);
    if (rc) return rc;
    if (!type_ok(p.query_type) || !type_ok(p.out_type)) return bad("unknown element type");
    if (p.n_requests < 0 || p.n_requests >= INT32_MAX || p.n_tokens < 0 || p.n_tokens >= INT32_MAX || p.group < 1 ||
        p.group > 256 || p.n_tokens * p.group >= INT32_MAX / p.n_heads || p.max_blocks < 0 || p.max_blocks > INT32_MAX ||
        p.query_token_stride < 0 || p.query_head_stride < 0 || p.out_token_stride < 0 || p.out_head_stride < 0)
      return bad("a size or stride is negative or too large");
    const float scale = p.scale * 1.4426950408889634f;  // scores are powers of two
    if (!std::isfinite(scale)) return bad("scale is not finite, or too large");
    if (p.n_requests > 1 && p.table_stride < p.max_blocks) return bad("table rows overlap");
    if (!p.offsets && p.n_tokens < p.n_requests) return bad("n_tokens is below one new token a request");
    if (p.n_requests == 0 || p.n_tokens == 0) return BPE_OK;
    if (!p.queries || !p.out || !p.seq_lens || (p.max_blocks > 0 && !p.table)) return bad("null pointer");
    if (!aligned(p.queries, type_size(p.query_type)) || !aligned(p.out, type_size(p.out_type)) ||
        !aligned(p.table, 4) || !aligned(p.seq_lens, 4) || !aligned(p.offsets, 8))
      return bad("a pointer is not aligned to its elements");
    const int64_t n_rows = p.n_heads * p.group;
    if (rows_meet(p.n_tokens, p.out_token_stride, n_rows, p.out_head_stride, p.dim)) return bad("output rows overlap");
    // (a long run that is computed again reads its queries again)
    auto rows = [&](const void* at, int64_t token, int64_t head, int64_t size) {
      return Rows{reinterpret_cast<uintptr_t>(at), p.n_tokens, n_rows, token * size, head * size, p.dim * size};
    };
    if (rows_share(rows(p.queries, p.query_token_stride, p.query_head_stride, type_size(p.query_type)),
                   rows(p.out, p.out_token_stride, p.out_head_stride, type_size(p.out_type))))
      return bad("out overlaps queries");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t groups = cache_groups(p.dim);
    const size_t records = align256((size_t)h->n_sms * kAttMaxWarps * 2 * sizeof(int4));
    const size_t partials = align256((size_t)h->n_sms * BPE_ATTEND_PARTIALS * (32 * groups + 2) * sizeof(float));
    // The host knows how many columns there are, not whose. Where all heads' are below 8192, long runs keep too few
    // SMs busy (2 requests of 256 behind 4,000 tokens, 8 heads: 110 us, here 83; 2 of 512: 109 and 144). Few a request
    // (drafted tokens of many): that one has kWideMin of them is not worth the launch, 10 us.
    const int64_t columns = p.n_tokens * p.group;
    const bool wide = p.query_type != BPE_F32 && p.offsets && columns >= kWideMin && columns * p.n_heads >= 8192 &&
                      (columns >= 4096 || columns >= 16 * p.n_requests);
    rc = ensure_ws(h, records + partials + (wide ? (size_t)p.n_requests * sizeof(int) : 0), st);
    if (rc) return rc;
    auto fits = [&](const void* q, int64_t token, int64_t head, int64_t size, int64_t V) {
      return p.dim % V == 0 && vec_ok(q, p.n_tokens > 1 ? token : 0, size, V) &&
             vec_ok(q, n_rows > 1 ? head : 0, size, V);
    };
    // absent tokens are zeros copied from nowhere, but from an address that is one
    const void* cache = p.cache ? p.cache : h->d_ws;
    AttendArgs a{p.queries, p.out, p.query_type, p.out_type, p.query_token_stride, p.query_head_stride, p.out_token_stride,
                 p.out_head_stride, p.n_tokens, (int)p.n_heads, (int)p.dim, FastDiv(p.group),
                 static_cast<const unsigned char*>(cache), p.n_blocks, p.block_stride,
                 cache_page_bytes(p.block_size, p.dim), FastDiv(p.block_size), p.table, p.table_stride,
                 std::min<int64_t>(p.max_blocks * p.block_size, INT32_MAX - 2 * kUnit), p.seq_lens, p.offsets, (int)p.n_requests,
                 scale,
                 fits(p.queries, p.query_token_stride, p.query_head_stride, type_size(p.query_type), 8),
                 fits(p.out, p.out_token_stride, p.out_head_stride, type_size(p.out_type), 4),
                 p.query_type != BPE_BF16 || p.out_type != BPE_BF16,
                 std::max(p.block_stride, 2 * p.n_heads * cache_page_bytes(p.block_size, p.dim)) / 16 <=
                     (int64_t)UINT32_MAX / std::max<int64_t>(1, p.n_blocks),
                 reinterpret_cast<float*>(static_cast<char*>(h->d_ws) + records), static_cast<int4*>(h->d_ws), nullptr, h->d_small};
    // 16 columns share the work on a code; a request with at most 8 has no use for the second half
    const bool two_tiles = p.offsets ? p.n_tokens * p.group > 8 * p.n_requests : p.group > 8;
    int* redo = reinterpret_cast<int*>(static_cast<char*>(h->d_ws) + records + partials);
    return with_groups(groups, [&](auto gs) {
      constexpr int G = decltype(gs)::value;
      auto launch = [&](auto parts, auto nt) -> int {
        constexpr int P = decltype(parts)::value, NT = decltype(nt)::value;
        constexpr int kSmem = AttendShape<G, P, NT>::kSmem;
        int ok = once_per_device(h->device, [&] {
          return cudaFuncSetAttribute(k_attend<P, G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        });
        if (ok) return ok;
        using Shape = AttendShape<G, P, NT>;
        static_assert(Shape::kBlocks * Shape::kWarps * 2 * Shape::kCols <= BPE_ATTEND_PARTIALS &&
                      Shape::kBlocks * Shape::kWarps <= kAttMaxWarps, "the workspace");
        const unsigned blocks = (unsigned)(h->n_sms * Shape::kBlocks);
        k_attend<P, G, NT><<<blocks, Shape::kThreads, kSmem, st>>>(a);
        CK(cudaGetLastError());
        CK(launch_after(k_attend_join<G, NT>, dim3(blocks * Shape::kWarps - 1), kJoinThreads, 0, st, a));
        return BPE_OK;
      };
      constexpr std::integral_constant<int, 1> one{};
      constexpr std::integral_constant<int, 2> two{};
      if (p.query_type == BPE_F32) return launch(two, one);
      if (wide) {
        CK(cudaMemsetAsync(redo, 0, (size_t)p.n_requests * sizeof(int), st));
        auto launch_wide = [&](auto tiles) -> int {
          constexpr int T = decltype(tiles)::value;
          using Wide = WideShape<G, T>;
          int ok = once_per_device(h->device, [&] {
            return cudaFuncSetAttribute(k_attend_wide<G, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide::kSmem);
          });
          if (ok) return ok;
          // as many blocks as requests of kWideMin columns on can need
          const int64_t blocks = (columns / (T * kWideTile) + std::min(p.n_requests, columns / kWideMin)) * p.n_heads;
          k_attend_wide<G, T><<<(unsigned)std::min<int64_t>(blocks, INT32_MAX), kWideThreads, Wide::kSmem, st>>>(a, redo);
          CK(cudaGetLastError());
          return BPE_OK;
        };
        int ok;
        // two tiles share what is filled in, one takes less time a step: where blocks of two leave SMs idle
        if constexpr (G <= 4) ok = columns / (2 * kWideTile) * p.n_heads >= h->n_sms ? launch_wide(two) : launch_wide(one);
        else ok = launch_wide(one);
        if (ok) return ok;
        a.redo = redo;
      }
      return two_tiles ? launch(one, two) : launch(one, one);
    });
  });
}

}  // extern "C"
