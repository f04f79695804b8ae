// A paged cache of keys and values in 4 bits: its layout, and what writes and
// reads rows by slot.
//
// Included by paged_ops.cu and attend.cu; not a standalone header.
//
// A row (a token's key or value of one head) is cut into groups of 32 elements,
// each with a base and a step in bfloat16:
//   base = bf16(smallest),  step = bf16((largest - base) / 15), 0 below 2^-100,
//   code = round((x - base) / step) in [0, 15],   x is read back as base + step * code.
// (Both quotients are products in 32 bits, of halves, with 1 / 7.5 and 2 / step. Where
// (largest - base) / 15 is next to a tie of two bfloat16 numbers, as of one f16 group
// in a thousand, the step may so be the other one of them; the codes follow it.)
// Base and step are rounded first and the codes follow them, so the step's
// rounding costs nothing but the largest element's last 2^-9 of the range, and the
// base's is no worse than a bfloat16 of the same elements. A group with a NaN or
// an element beyond bfloat16 reads back as NaN.
//
// A page (one head's keys, or values, in one block of s slots) holds the s rows'
// codes, 16 bytes a group, then the s rows' (step, base) words, one a group, and
// ends at a multiple of 16 bytes. A block is [keys, values][heads][page].
// The 8 codes of elements 32 j + 8 c .. + 7 make a 32-bit word, the first in its
// lowest bits. Words of two groups alternate (word 2 c + (j & 1) of the pair's
// 32 bytes), so that one 8-byte load gives a thread of an attention tile its
// elements of both; a last group without a partner has word c at c.

namespace {

constexpr int kGroup = 32;
constexpr int kMaxGroups = 8;
constexpr float kBf16Max = 0x1.FEp127f;

// Groups of a row of dim elements: even beyond four, so that the attention has fewer shapes.
inline int64_t cache_groups(int64_t dim) {
  const int64_t g = (dim + kGroup - 1) / kGroup;
  return g > 4 ? g + g % 2 : g;
}

inline int64_t cache_page_bytes(int64_t block_size, int64_t dim) {
  return (block_size * cache_groups(dim) * 20 + 15) / 16 * 16;
}

// The word of group j's codes 8 c .. 8 c + 7 in a row of `groups` groups.
__device__ __forceinline__ int cache_word(int groups, int j, int c) {
  return (j | 1) < groups ? (j >> 1) * 8 + 2 * c + (j & 1) : j * 4 + c;
}

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

struct CacheArgs {
  unsigned char* cache;
  int64_t block_stride, page_bytes, n_slots;
  FastDiv block;     // slots of a block
  FastDiv parts, heads;  // threads of a row; heads of a token
  int groups, dim;
  const int64_t* slots;
  DevSmall* small;
};

// The page of head h's keys that a slot lies in, and its row there.
__device__ __forceinline__ unsigned char* cache_page(const CacheArgs& a, int64_t slot, int h, uint32_t* row) {
  int64_t page;
  if (slot < INT32_MAX) {
    page = a.block((uint32_t)slot);
    *row = (uint32_t)slot - (uint32_t)page * a.block.d;
  } else {
    page = slot / a.block.d;
    *row = (uint32_t)(slot - page * a.block.d);
  }
  return a.cache + page * a.block_stride + h * a.page_bytes;
}

inline int cache_check(const char* who, const bpe_handle* h, const void* d_cache, int64_t n_blocks,
                       int64_t block_stride, int64_t block_size, int64_t n_heads, int64_t dim) {
  auto bad = [&](const char* what) { return fail(BPE_ERR_INVALID_ARG, std::string(who) + ": " + what); };
  if (!h) return bad("null handle");
  if (n_blocks < 0 || n_blocks > INT32_MAX || block_size < 1 || block_size > BPE_CACHE_MAX_BLOCK || n_heads < 1 ||
      n_heads > BPE_CACHE_MAX_HEADS || dim < 1 || dim > BPE_CACHE_MAX_DIM)
    return bad("blocks, block_size, heads or dim out of range");
  if (n_blocks > 0 && !d_cache) return bad("null cache");
  if (!aligned(d_cache, 16) || block_stride % 16 != 0) return bad("cache and block_stride need multiples of 16 bytes");
  if (n_blocks > 1 && block_stride < 2 * n_heads * cache_page_bytes(block_size, dim)) return bad("blocks overlap");
  return BPE_OK;
}

}  // namespace
