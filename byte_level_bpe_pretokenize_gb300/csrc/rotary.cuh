// Rotary positions: pairs of a head's elements turned by angles that grow with
// the token's position.
//
// Included once by paged_ops.cu; not a standalone header.
//
//   (y1, y2) = scale * (x1 cos a - x2 sin a, x1 sin a + x2 cos a),  a = 2 pi f_i p
//
// of pair i, at position p. The table holds f_i, in turns a position, as a
// fraction of 2^64, so p f_i modulo a turn is one wrapping product of integers:
// its error is p 2^-65 turns, below that of the 32-bit angle that its upper
// half becomes, at every position. (In 32-bit floats a fast pair is off by a
// radian after some million positions, and 64-bit ones are slow here.) What f_i
// itself is off by, 2^-53 of it where it is computed, p multiplies too.

namespace {

constexpr int kRotThreads = 256;
constexpr int64_t kRotMaxDim = 65536, kRotMaxHeads = 65536;

struct RotateArgs {
  const void* x;
  void* out;
  int64_t x_token, x_head, out_token, out_head;  // strides in elements
  const int32_t* positions;
  const uint64_t* turns;
  uint32_t total;        // threads that have work: tokens x shares x items
  FastDiv items, shares; // of a head; threads that divide a token's heads
  int heads, pairs, dim;
  int turning;           // items of a head that turn pairs; the others copy
  float scale;
  bool inverse;
};

// A thread takes one item (V elements of each half, or V elements that pairs
// lie next to each other in) of every shares-th head of a token, so that sines
// and cosines, 40 instructions a pair, are computed once for these heads. A is
// the elements of an access: 1 where addresses are aligned for no more.
//
// Bound by HBM where tokens are many: two bytes in and two out for six
// operations a pair. 65,536 tokens of 40 heads of 128 in bf16: 198 us, 6.8 TB/s,
// the rate of a copy. 8 tokens: 2.8 to 3.4 us.
template <class TI, class TO, int V, int A, bool kAdjacent>
__global__ void __launch_bounds__(kRotThreads) k_rotate(RotateArgs a) {
  constexpr int kPairs = kAdjacent ? V / 2 : V, kVecs = kAdjacent ? 1 : 2;
  constexpr int kRotHeads = V * sizeof(TI) * kVecs >= 32 ? 4 : 8;  // heads that a thread holds in flight
  const uint32_t index = blockIdx.x * kRotThreads + threadIdx.x;
  if (index >= a.total) return;
  const uint32_t row = a.items(index), item = index - row * a.items.d;
  const uint32_t token = a.shares(row), share = row - token * a.shares.d;
  const TI* x = static_cast<const TI*>(a.x) + (int64_t)token * a.x_token;
  TO* y = static_cast<TO*>(a.out) + (int64_t)token * a.out_token;
  // the first n elements (single ones only: the last of an odd dim has no partner)
  auto get = [](Vec<TI, V>& v, const TI* p, int n = V) {
    if constexpr (A == V) {
      v.load(p);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < n) v.x[e] = p[e];
    }
  };
  auto put = [](const Vec<TO, V>& v, TO* p, int n = V) {
    if constexpr (A == V) {
      v.store(p);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < n) p[e] = v.x[e];
    }
  };
  if ((int)item >= a.turning) {  // behind the turned part
    const int at = (kAdjacent ? 0 : 2 * a.pairs) + ((int)item - (kAdjacent ? 0 : a.turning)) * V;
    for (int h0 = share; h0 < a.heads; h0 += kRotHeads * a.shares.d) {
      Vec<TI, V> v[kRotHeads];
#pragma unroll
      for (int q = 0; q < kRotHeads; ++q) {
        const int h = h0 + q * a.shares.d;
        if (h < a.heads) get(v[q], x + h * a.x_head + at, a.dim - at);
      }
#pragma unroll
      for (int q = 0; q < kRotHeads; ++q) {
        const int h = h0 + q * a.shares.d;
        if (h >= a.heads) break;
        Vec<TO, V> r;
#pragma unroll
        for (int e = 0; e < V; ++e) r.x[e] = from_f32<TO>(to_f32(v[q].x[e]));
        put(r, y + h * a.out_head + at, a.dim - at);
      }
    }
    return;
  }
  const int64_t position = a.positions[token];
  float c[kPairs], s[kPairs];
  bool turned[kPairs];  // an item of adjacent pairs may reach past the last one
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int pair = (int)item * kPairs + i;
    turned[i] = !kAdjacent || pair < a.pairs;
    const uint64_t turn = turned[i] ? __ldg(a.turns + pair) : 0;
    // half turns in [-1, 1): to 2^-25 of the angle
    const float half = (float)(int32_t)(uint32_t)(((uint64_t)position * turn) >> 32) * 0x1p-31f;
    sincospif(half, &s[i], &c[i]);
    if (a.inverse) s[i] = -s[i];
    s[i] *= a.scale;
    c[i] *= a.scale;
  }
  const int first = item * V, second = a.pairs + item * V;
  for (int h0 = share; h0 < a.heads; h0 += kRotHeads * a.shares.d) {
    Vec<TI, V> v[kRotHeads][kVecs];
#pragma unroll
    for (int q = 0; q < kRotHeads; ++q) {
      const int h = h0 + q * a.shares.d;
      if (h >= a.heads) break;
      get(v[q][0], x + h * a.x_head + first);
      if (!kAdjacent) get(v[q][kVecs - 1], x + h * a.x_head + second);
    }
#pragma unroll
    for (int q = 0; q < kRotHeads; ++q) {
      const int h = h0 + q * a.shares.d;
      if (h >= a.heads) break;
      Vec<TO, V> r[kVecs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float x1 = to_f32(kAdjacent ? v[q][0].x[(2 * i) % V] : v[q][0].x[i % V]);
        const float x2 = to_f32(kAdjacent ? v[q][0].x[(2 * i + 1) % V] : v[q][kVecs - 1].x[i % V]);
        const float y1 = turned[i] ? x1 * c[i] - x2 * s[i] : x1, y2 = turned[i] ? x1 * s[i] + x2 * c[i] : x2;
        (kAdjacent ? r[0].x[(2 * i) % V] : r[0].x[i % V]) = from_f32<TO>(y1);
        (kAdjacent ? r[0].x[(2 * i + 1) % V] : r[kVecs - 1].x[i % V]) = from_f32<TO>(y2);
      }
      put(r[0], y + h * a.out_head + first);
      if (!kAdjacent) put(r[kVecs - 1], y + h * a.out_head + second);
    }
  }
}

// 1 / (2 pi) as a sum of three doubles, to 2^-163.
constexpr double kPerTurn = 0x1.45f306dc9c883p-3, kPerTurn2 = -0x1.6b01ec5417056p-57, kPerTurn3 = -0x1.6447e493ad4cep-111;

// f / (2 pi) modulo 1 as a fraction of 2^64, rounded, for f up to 2^90: f times each part is a sum of two doubles, and
// a double modulo 1 is exact. So far positions turn by what f says, to p 2^-65 turns, where f / (2 pi) in 64 bits would
// be off by up to p 2^-56, and p 2^-54 for a negative f.
inline uint64_t fraction_of_turn(double f) {
  auto fraction = [](double x) -> uint64_t {  // x modulo 1 in units of 2^-64, cut off below them
    const double whole = std::trunc(x), part = std::fabs(x - whole);
    const uint64_t u = (uint64_t)std::ldexp(part, 64);
    return x < 0 ? 0 - u : u;
  };
  auto rest = [](double x) {  // what that cut off, in units
    const double part = std::ldexp(x - std::trunc(x), 64);
    return part - std::trunc(part);
  };
  uint64_t sum = 0;
  double below = 0;
  for (double c : {kPerTurn, kPerTurn2, kPerTurn3}) {
    const double high = f * c, low = std::fma(f, c, -high);
    for (double x : {high, low}) {
      sum += fraction(x);
      below += rest(x);
    }
  }
  return sum + (uint64_t)(int64_t)std::nearbyint(below);
}

}  // namespace

extern "C" {

int bpe_rotary_table(const double* frequencies, int64_t n_pairs, double base, double factor, double original,
                     double low, double high, uint64_t* turns) {
  return guarded("bpe_rotary_table", [&]() -> int {
    if (n_pairs < 0 || n_pairs > kRotMaxDim / 2 || (n_pairs > 0 && !turns))
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotary_table: bad number of pairs or null pointer");
    if (!(factor > 0) || !std::isfinite(factor) || (!frequencies && (!(base > 0) || !std::isfinite(base))))
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotary_table: base and factor must be positive and finite");
    if (original != 0 && (!(original > 0) || !std::isfinite(original) || !(low < high) || !std::isfinite(high - low)))
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotary_table: needs original > 0 and low < high");
    for (int64_t i = 0; i < n_pairs; ++i) {
      double f = frequencies ? frequencies[i] : std::pow(base, -(double)i / (double)n_pairs);
      if (!std::isfinite(f)) return fail(BPE_ERR_INVALID_ARG, "bpe_rotary_table: a frequency is not finite");
      if (original > 0) {
        const double turns_over = original * (std::fabs(f) * kPerTurn);
        const double keep = std::min(1.0, std::max(0.0, (turns_over - low) / (high - low)));
        f *= keep + (1.0 - keep) / factor;
      } else {
        f /= factor;
      }
      if (!std::isfinite(f)) return fail(BPE_ERR_INVALID_ARG, "bpe_rotary_table: a stretched frequency is not finite");
      turns[i] = fraction_of_turn(f);
    }
    return BPE_OK;
  });
}

int bpe_rotate(bpe_handle* h, const void* d_x, int x_type, int64_t n_tokens, int64_t n_heads, int64_t dim,
               int64_t x_token_stride, int64_t x_head_stride, const int32_t* d_positions, const uint64_t* d_turns,
               int64_t n_pairs, int interleaved, int inverse, float scale, void* d_out, int out_type,
               int64_t out_token_stride, int64_t out_head_stride, bpe_stream_t stream) {
  return guarded("bpe_rotate", [&]() -> int {
    if (!h) return fail(BPE_ERR_INVALID_ARG, "bpe_rotate: null handle");
    if (!type_ok(x_type) || !type_ok(out_type)) return fail(BPE_ERR_INVALID_ARG, "bpe_rotate: unknown element type");
    if (n_tokens < 0 || n_tokens >= INT32_MAX || n_heads < 0 || n_heads > kRotMaxHeads || dim < 0 ||
        dim > kRotMaxDim || n_pairs < 0 || 2 * n_pairs > dim || x_token_stride < 0 || x_head_stride < 0 ||
        out_token_stride < 0 || out_head_stride < 0)
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotate: a size or stride is negative or too large");
    if (n_tokens == 0 || n_heads == 0 || dim == 0) return BPE_OK;
    if (!d_x || !d_out || (n_pairs > 0 && (!d_positions || !d_turns)))
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotate: null pointer");
    if (!aligned(d_x, type_size(x_type)) || !aligned(d_out, type_size(out_type)) || !aligned(d_positions, 4) ||
        !aligned(d_turns, 8))
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotate: a pointer is not aligned to its elements");
    if (rows_meet(n_tokens, out_token_stride, n_heads, out_head_stride, dim))
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotate: output rows overlap");
    const bool same = d_x == d_out;
    if (same && (x_type != out_type || (n_tokens > 1 && x_token_stride != out_token_stride) ||
                 (n_heads > 1 && x_head_stride != out_head_stride)))
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotate: in place needs one type and the same strides");
    auto rows = [&](const void* at, int64_t token, int64_t head, int64_t size) {
      return Rows{reinterpret_cast<uintptr_t>(at), n_tokens, n_heads, token * size, head * size, dim * size};
    };
    if (!same && rows_share(rows(d_x, x_token_stride, x_head_stride, type_size(x_type)),
                            rows(d_out, out_token_stride, out_head_stride, type_size(out_type))))
      return fail(BPE_ERR_INVALID_ARG, "bpe_rotate: out overlaps x");
    DeviceGuard g(h->device);
    cudaStream_t st = (cudaStream_t)stream;
    return with_type(x_type, [&](auto ti) {
      return with_type(out_type, [&](auto to) -> int {
        using TI = decltype(ti);
        using TO = decltype(to);
        // elements [from, from + dim) of each head, of which the first 2 * n_pairs turn
        auto launch = [&](auto width, auto access, auto adjacent, int64_t from, int64_t dim, int64_t n_pairs) -> int {
          constexpr int V = decltype(width)::value, A = decltype(access)::value;
          constexpr bool kAdjacent = decltype(adjacent)::value;
          int64_t turning = kAdjacent ? (2 * n_pairs + V - 1) / V : n_pairs / V;
          // in place, what is behind the turned part stays
          const int64_t items = same ? turning : kAdjacent ? (dim + V - 1) / V : turning + (dim - 2 * n_pairs) / V;
          // adjacent pairs that do not turn go with those that do: lanes of a warp have both (but where none turn
          // there may be no positions)
          if (kAdjacent && A == V && n_pairs > 0) turning = items;
          if (items == 0) return BPE_OK;
          // As many threads share a token's heads as give the GPU half of the threads that it holds: with
          // more, sines are computed again, with fewer, loads are too few.
          const int64_t want = (int64_t)h->n_sms * 1024;
          const int64_t shares = std::max<int64_t>(1, std::min(n_heads, want / std::max<int64_t>(1, n_tokens * items)));
          const int64_t at_once = std::min(n_tokens, (int64_t)INT32_MAX / 2 / (items * shares));
          for (int64_t t = 0; t < n_tokens; t += at_once) {
            const int64_t n = std::min(at_once, n_tokens - t);
            RotateArgs a{static_cast<const TI*>(d_x) + t * x_token_stride + from,
                         static_cast<TO*>(d_out) + t * out_token_stride + from,
                         x_token_stride, x_head_stride, out_token_stride, out_head_stride,
                         d_positions ? d_positions + t : nullptr, d_turns, (uint32_t)(n * items * shares),
                         FastDiv(items), FastDiv(shares), (int)n_heads, (int)n_pairs, (int)dim, (int)turning, scale,
                         inverse != 0};
            k_rotate<TI, TO, V, A, kAdjacent><<<(a.total + kRotThreads - 1) / kRotThreads, kRotThreads, 0, st>>>(a);
            CK(cudaGetLastError());
          }
          return BPE_OK;
        };
        auto rows_fit = [&](int64_t V) {
          auto rows = [&](const void* p, int64_t token, int64_t head, int64_t size) {
            return vec_ok(p, n_tokens > 1 ? token : 0, size, V) && vec_ok(p, n_heads > 1 ? head : 0, size, V);
          };
          return dim % V == 0 && rows(d_x, x_token_stride, x_head_stride, sizeof(TI)) &&
                 rows(d_out, out_token_stride, out_head_stride, sizeof(TO));
        };
        auto fits = [&](int64_t V) { return rows_fit(V) && (interleaved || n_pairs % V == 0); };
        using std::integral_constant;
        constexpr integral_constant<int, 8> c8{};
        constexpr integral_constant<int, 4> c4{};
        constexpr integral_constant<int, 2> c2{};
        constexpr integral_constant<int, 1> c1{};
        if (interleaved) {
          if (fits(8)) return launch(c8, c8, std::true_type{}, 0, dim, n_pairs);
          if (fits(4)) return launch(c4, c4, std::true_type{}, 0, dim, n_pairs);
          if (fits(2)) return launch(c2, c2, std::true_type{}, 0, dim, n_pairs);
          return launch(c2, c1, std::true_type{}, 0, dim, n_pairs);
        }
        if (fits(8)) return launch(c8, c8, std::false_type{}, 0, dim, n_pairs);
        // Rows are aligned, but not the second halves of their pairs: what is behind the turned part is copied by
        // itself, where it is enough for a launch.
        const int64_t behind = (2 * n_pairs + 7) / 8 * 8;
        if (!same && rows_fit(8) && n_tokens * n_heads * (dim - behind) >= (1 << 20)) {
          const int rc = launch(c8, c8, std::false_type{}, behind, dim - behind, 0);
          if (rc) return rc;
          if (n_pairs % 4 == 0) return launch(c4, c4, std::false_type{}, 0, behind, n_pairs);
          if (n_pairs % 2 == 0) return launch(c2, c2, std::false_type{}, 0, behind, n_pairs);
          return launch(c1, c1, std::false_type{}, 0, behind, n_pairs);
        }
        if (fits(4)) return launch(c4, c4, std::false_type{}, 0, dim, n_pairs);
        if (fits(2)) return launch(c2, c2, std::false_type{}, 0, dim, n_pairs);
        return launch(c1, c1, std::false_type{}, 0, dim, n_pairs);
      });
    });
  });
}

}  // extern "C"
