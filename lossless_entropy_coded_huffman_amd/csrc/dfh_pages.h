// The pages of a cache and the sequences in them, as kernels see them: shared by the
// cache's writes and reads and by the attention over it (gfx950).
//
// Keys and values lie in pages of page_size tokens, [pages, kv_heads, page_size,
// head_dim] each, so that one head's tokens of a page are contiguous.  A sequence's
// position p lies in page tables[p / page_size], row p % page_size.  What the device
// holds is not trusted: a page number outside the pool, or a position outside the
// table, is a token that is not there.
#ifndef DFH_PAGES_H
#define DFH_PAGES_H

#include "dfh.h"
#include "dfh_gemm.h"

namespace dfh {
namespace {

struct Pages {
  uint8_t *k, *v;
  float *k_scales, *v_scales;  // 8 bits
  uint32_t pages, shift;       // page_size = 1 << shift
  uint32_t heads, dim;         // of keys
};
struct Sequences {
  const int32_t *tables, *lengths, *starts;
  uint64_t stride;  // of tables
  uint32_t count, width;
  uint32_t tokens;  // rows of new tokens in the call
};

// A sequence's new tokens, rows first .. last - 1 of the call's, and its length; row r
// is position r + ahead.
struct Span {
  int32_t first, last, length, ahead;
};
__device__ __forceinline__ Span span_of(const Sequences &b, uint32_t s) {
  const int32_t n = (int32_t)b.tokens;
  Span p;
  p.first = b.starts[s];
  p.last = b.starts[s + 1];
  p.first = p.first < 0 ? 0 : p.first < n ? p.first : n;
  p.last = p.last < p.first ? p.first : p.last < n ? p.last : n;
  p.length = b.lengths[s];
  // positions stay below 2^30, tables hold fewer
  p.length = p.length < 0 ? 0 : p.length < (1 << 30) ? p.length : 1 << 30;
  p.ahead = p.length - p.last;
  return p;
}

// How many of starts[0 .. count] are at most t, by a whole wave: each round looks at 64
// places at equal distances, so 64 sequences take one load, 4096 two.
template <class I>
__device__ __forceinline__ uint32_t starts_up_to(const I *starts, uint32_t count, I t) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0, n = count;  // the answer lies in lo .. lo + n
  while (n) {
    const uint32_t step = (n + 63) / 64, at = lo + lane * step;
    const bool in = lane * step < n && starts[at] <= t;
    const uint32_t c = __popcll(__ballot(in));  // of those places, in order
    if (c == 0) return lo;
    const uint32_t before = lo + n;
    lo = lo + (c - 1) * step + 1;
    n = lo + step - 1 < before ? step - 1 : before - lo;
  }
  return lo;
}
// The sequence that row t belongs to, or none (count).
__device__ __forceinline__ uint32_t sequence_of(const Sequences &b, int32_t t) {
  if (b.count == 0) return 0;
  const uint32_t c = starts_up_to(b.starts, b.count + 1, t);
  return c == 0 || c > b.count ? b.count : c - 1;
}

// The token that position p of a sequence is, counted over the pool's pages: page *
// page_size + row, or -1 where there is none.
__device__ __forceinline__ int64_t token_at(const Pages &c, const Sequences &b, uint32_t s, int32_t p) {
  if (p < 0 || (uint32_t)p >> c.shift >= b.width) return -1;
  const int32_t page = b.tables[s * b.stride + ((uint32_t)p >> c.shift)];
  if ((uint32_t)page >= c.pages) return -1;
  return ((int64_t)page << c.shift) + (p & ((1 << c.shift) - 1));
}
// Row of a head's token in [pages, heads, page_size].
__device__ __forceinline__ uint64_t row_of(const Pages &c, int64_t token, uint32_t head) {
  const uint64_t page = (uint64_t)token >> c.shift;
  return ((page * c.heads + head) << c.shift) + ((uint64_t)token & ((1u << c.shift) - 1));
}

// ------------------------------------------------------------------- host
inline bool cache_ok(const df_cache *c) {
  if (!c || !c->k || !c->v || ((uintptr_t)c->k & 15) || ((uintptr_t)c->v & 15)) return false;
  if (c->type != DF_TYPE_BF16 && c->type != DF_TYPE_F16) return false;
  if (c->bits != 16 && c->bits != 8) return false;
  if (c->bits == 8 && (!c->k_scales || !c->v_scales || ((uintptr_t)c->k_scales & 3) || ((uintptr_t)c->v_scales & 3)))
    return false;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return false;
  if (c->kv_heads == 0 || c->kv_heads > 256 || c->pages == 0 || c->pages > (1u << 26)) return false;
  return c->head_dim == 32 || c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256;
}
inline bool batch_ok(const df_cache_batch *b, uint64_t tokens) {
  if (!b || tokens > (1u << 24) || b->seqs > (1u << 16)) return false;
  if (b->seqs == 0) return true;
  if (!b->tables || !b->lengths || !b->starts || (((uintptr_t)b->tables | (uintptr_t)b->lengths | (uintptr_t)b->starts) & 3))
    return false;
  return b->width >= 1 && b->width <= (1u << 22) && b->table_stride >= b->width && b->table_stride <= (1u << 30);
}
inline Pages pages_of(const df_cache *c) {
  return Pages{(uint8_t *)c->k, (uint8_t *)c->v, c->k_scales, c->v_scales, (uint32_t)c->pages,
               (uint32_t)__builtin_ctz(c->page_size), c->kv_heads, c->head_dim};
}
inline Sequences sequences_of(const df_cache_batch *b, uint64_t tokens) {
  return Sequences{b->tables, b->lengths, b->starts, b->table_stride, b->seqs, b->width, (uint32_t)tokens};
}

}  // namespace
}  // namespace dfh

#endif
