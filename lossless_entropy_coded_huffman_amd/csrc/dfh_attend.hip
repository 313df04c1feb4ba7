// Attention of the new tokens of several sequences over a paged cache (gfx950).
//
//   o[t, h] = sum_j p_j v[j] / sum_j p_j,   p_j = exp(scale q[t, h] . k[j] - max),
//
// over the positions j of the token's sequence with j <= position and, with a window,
// position - j < window.  Keys and values of 8 bits are codes times a token's scale.
//
// One pass over the keys with the running maximum and sum of the softmax, in FP32, on
// v_mfma_f32_32x32x16: S^T = K Q^T leaves a lane 16 keys of one query, so the maximum
// and the sum are taken in registers with one exchange between the two halves of the
// wave, and the same registers, rounded to 16 bits, are the operand P^T of
// O^T = V^T P^T, whose columns are the same queries: what a new maximum takes off is one
// factor a lane.  The order of the summed keys is the one that P^T's registers have
// (key_of), V^T's columns are read in it by transposing LDS loads.
// The heads that share a key head are rows of one tile, so a key is read once for them.
//
// attend_few takes sequences with at most 32 rows (tokens times heads a key head),
// whose time is the reading of the cache: each wave has tiles of 32 keys of its own,
// read straight to LDS, and the key range is split over workgroups too.  attend_tile takes the
// others: 128 rows share tiles of 64 keys.  attend_join adds up what splits leave.
//
// Roundings: q and 16-bit keys and values are taken as they are, codes of 8 bits are
// exact in both 16-bit types.  A token's scale of keys multiplies the FP32 scores; its
// scale of values multiplies p before that is rounded to 16 bits where the type is BF16
// (p times scale is the one rounding), while in FP16, whose range p times scale may leave,
// the value is rounded to FP16 as cache_read gives it.  p is rounded to 16 bits (half a step:
// 2^-9 or 2^-12 of it), sums are FP32.
#include <hip/hip_runtime.h>

#include "dfh.h"
#include "dfh_gemm.h"
#include "dfh_pages.h"
#include "dfh_quant.h"

namespace {

using namespace dfh;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x16 mfma32(BF16, u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ f32x16 mfma32(F16, u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
// Two floats as 16 bits each, to nearest even, in one instruction.
__device__ __forceinline__ uint32_t pair(BF16, float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ uint32_t pair(F16, float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
// A value and its lane's in the other half of the wave.
__device__ __forceinline__ f32x2 both_halves(float v) {
  const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return f32x2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

// Eight codes as 16-bit floats, exactly.  FP16: a byte of offset 128 in the mantissa of
// 1024, then 1152 off; BF16 has no bits for that and goes by FP32.
__device__ __forceinline__ u32x4 widen8(F16, u32x2 w) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t u = w[i] ^ 0x80808080u;
    const f16x2 off = {(_Float16)-1152.f, (_Float16)-1152.f};
    o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + off);
    o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + off);
  }
  return o;
}
__device__ __forceinline__ u32x4 widen8(BF16, u32x2 w) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t v = w[i / 2] >> (16 * (i & 1));
    o[i] = pair(BF16{}, (float)(int8_t)v, (float)(int8_t)(v >> 8));
  }
  return o;
}
// Eight codes times a scale each, rounded.
template <class T>
__device__ __forceinline__ u32x4 widen8_by(T, u32x2 w, const float *f) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t v = w[i / 2] >> (16 * (i & 1));
    o[i] = pair(T{}, (float)(int8_t)v * f[2 * i], (float)(int8_t)(v >> 8) * f[2 * i + 1]);
  }
  return o;
}

struct Attend {
  const uint16_t *q;
  uint64_t q_token, q_head;  // strides in elements
  uint16_t *out;             // [tokens, heads, D]
  float *lse;                // [tokens, heads], or null
  uint32_t heads, group;     // heads a key head
  int32_t window;            // INT32_MAX: none
  float c;                   // scale times log2 e
  // few rows
  uint32_t cap, few_splits;
  uint32_t alone;            // no attend_tile follows: sequences of more rows are taken too
  float *few_o, *few_ml;     // [splits][seqs][kv heads][cap][D], [..][2]
  // tiles
  uint32_t tiles, tile_splits;
  float *tile_o, *tile_ml;   // [splits][tokens][heads][D], [..][2]
};

// The keys that rows at positions first .. last see, in units of 2^shift, cut into
// `count` parts of `per`.
struct Cuts {
  int32_t begin, end, per, count, stop;  // stop: the first position that is not seen
};
__device__ __forceinline__ Cuts cuts_of(const Pages &c, const Sequences &b, int32_t first, int32_t last, int32_t length,
                                        int32_t window, int shift, uint32_t splits, int32_t least) {
  Cuts k;
  const uint64_t held = (uint64_t)b.width << c.shift;
  k.stop = last + 1 < length ? last + 1 : length;
  if ((uint64_t)(k.stop < 0 ? 0 : k.stop) > held) k.stop = (int32_t)held;
  const int64_t before = (int64_t)first - window + 1;  // first may lie before position 0
  const int32_t from = before > 0 ? (int32_t)before : 0;
  k.begin = from >> shift;
  k.end = k.stop > from ? (k.stop + (1 << shift) - 1) >> shift : k.begin;
  const int32_t n = k.end - k.begin;
  int32_t want = (n + least - 1) / least;
  want = want < (int32_t)splits ? want : (int32_t)splits;
  k.per = want > 0 ? (n + want - 1) / want : 0;
  k.count = k.per > 0 ? (n + k.per - 1) / k.per : 0;
  return k;
}
constexpr int kFewShift = 5, kFewLeast = 4, kTileShift = 6, kTileLeast = 8;

// A tile of keys or values in LDS: rows of D values of BITS, 16-byte chunks exchanged
// within a row (in the source address, since a load writes LDS linearly).  Keys are
// read 16 bytes at one chunk of 32 rows: 8 rows in a row fall into 8 places.  Values are
// read transposed, 64 (BITS 8: 32) bytes of 8 (16) rows: neighbours fall into different ones.
template <int BITS, int D>
struct Rows {
  static constexpr int kBytes = D * BITS / 8, kChunks = kBytes / 16;
  static constexpr int kPer = kBytes >= 128 ? 1 : 128 / kBytes;  // rows in 128 bytes
  static constexpr int kKeyPlaces = kChunks < 8 ? kChunks : 8;
  static constexpr int kUnit = BITS == 16 ? 4 : 2;
  static constexpr int kUnits = kChunks / kUnit < 1 ? 1 : kChunks / kUnit < 16 / kUnit ? kChunks / kUnit : 16 / kUnit;
  static __device__ __forceinline__ uint32_t key_swap(uint32_t r) { return (r / kPer) & (kKeyPlaces - 1); }
  static __device__ __forceinline__ uint32_t value_swap(uint32_t r) { return ((r / kPer) & (kUnits - 1)) * kUnit; }
};

// Key of a lane's register r (of 16) in a block of 32, without the 4 * (lane / 32).
__device__ __forceinline__ constexpr int key_of(int r) { return 8 * (r / 4) + r % 4; }

// What 32 queries of a wave gather: lane l has query l % 32.
template <class T, int BITS, int D>
struct Wave {
  u32x4 q[D / 16];
  f32x16 o[D / 32];
  float m, l;  // maximum (times c), and this half's sum
  int32_t pos;

  // row: this lane's query
  __device__ __forceinline__ void init(const uint16_t *row, int32_t position) {
    const uint32_t h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int s = 0; s < D / 16; s++) {
      // a step's 16 elements: 8 of each half; of keys of 8 bits a lane reads two steps' at once
      const uint32_t chunk = BITS == 8 ? (s / 2) * 4 + h * 2 + (s & 1) : s * 2 + h;
      q[s] = *(const u32x4 *)(row + chunk * 8);
    }
#pragma unroll
    for (int d = 0; d < D / 32; d++) o[d] = f32x16{};
    m = -__builtin_huge_valf();
    l = 0.f;
    pos = position;
  }
};

// Whether a query at pos sees the key at pos - gap.
__device__ __forceinline__ bool sees(int32_t gap, int32_t window) { return (uint32_t)gap < (uint32_t)window; }

// NB blocks of 32 keys at position `base` in LDS (LB bits a value there): adds them to w.
// SCALED: scales of the keys (times c) and of the values in LDS, `there` bit j of a block: the key
// exists; whole: every query sees every key.  BARE: values are codes, p takes their
// scale.
template <class T, int BITS, int LB, int D, int NB, bool SCALED, bool BARE, class Mask>
__device__ __forceinline__ void add_keys(Wave<T, BITS, D> &w, const uint8_t *lk, const uint8_t *lv, const float *ks,
                                         const float *vs, int32_t base, Mask there, bool whole, float c, int32_t window) {
  typedef Rows<LB, D> R;
  const uint32_t lane = threadIdx.x & 63, h = lane >> 5, row = lane & 31;
  // scores
  f32x16 s[NB];
#pragma unroll
  for (int n = 0; n < NB; n++) {
    s[n] = f32x16{};
    const uint8_t *p = lk + (n * 32 + row) * R::kBytes;
    const uint32_t f = R::key_swap(row);
    if constexpr (LB == 16) {
#pragma unroll
      for (int st = 0; st < D / 16; st++) {
        // the order of a lane's 8 elements is q's
        const uint32_t chunk = BITS == 8 ? (st / 2) * 4 + h * 2 + (st & 1) : st * 2 + h;
        s[n] = mfma32(T{}, *(const u32x4 *)(p + ((chunk ^ f) * 16)), w.q[st], s[n]);
      }
    } else {
#pragma unroll
      for (int st = 0; st < D / 32; st++) {
        const u32x4 k = *(const u32x4 *)(p + (((st * 2 + h) ^ f) * 16));
        s[n] = mfma32(T{}, widen8(T{}, u32x2{k[0], k[1]}), w.q[2 * st], s[n]);
        s[n] = mfma32(T{}, widen8(T{}, u32x2{k[2], k[3]}), w.q[2 * st + 1], s[n]);
      }
    }
  }
  if constexpr (SCALED) {
#pragma unroll
    for (int n = 0; n < NB; n++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const f32x4 k = *(const f32x4 *)(ks + n * 32 + 8 * i + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; e++) s[n][4 * i + e] *= k[e];
      }
  }
  const int32_t gap = w.pos - base - 4 * (int32_t)h;  // to the key of register 0 of block 0
  if (!whole) {
#pragma unroll
    for (int n = 0; n < NB; n++) {
      const uint32_t t = there(n) >> (4 * h);
#pragma unroll
      for (int r = 0; r < 16; r++)
        if (!(sees(gap - n * 32 - key_of(r), window) && (t >> key_of(r) & 1))) s[n][r] = -__builtin_huge_valf();
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int n = 0; n < NB; n++)
#pragma unroll
    for (int r = 0; r < 16; r++) top = __builtin_fmaxf(top, s[n][r]);
  const f32x2 tops = both_halves(top);
  top = __builtin_fmaxf(tops[0], tops[1]);
  if constexpr (!SCALED) top *= c;
  top = __builtin_fmaxf(top, w.m);
  const float ref = top == -__builtin_huge_valf() ? 0.f : top;
  if (__ballot(top > w.m)) {
    const float back = exp2_of(w.m - ref);
    w.l *= back;
#pragma unroll
    for (int d = 0; d < D / 32; d++) w.o[d] *= back;
    w.m = top;
  }
  float sum = 0.f;
#pragma unroll
  for (int n = 0; n < NB; n++)
#pragma unroll
    for (int r = 0; r < 16; r++) {
      s[n][r] = exp2_of(SCALED ? s[n][r] - ref : __builtin_fmaf(s[n][r], c, -ref));
      sum += s[n][r];
    }
  w.l += sum;
  // values
  float f[SCALED ? NB * 16 : 1];
  if constexpr (SCALED) {
#pragma unroll
    for (int n = 0; n < NB; n++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const f32x4 v = *(const f32x4 *)(vs + n * 32 + 8 * i + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; e++) f[n * 16 + 4 * i + e] = v[e];
      }
    if constexpr (BARE) {
#pragma unroll
      for (int n = 0; n < NB; n++)
#pragma unroll
        for (int r = 0; r < 16; r++) {
          float p = s[n][r] * f[n * 16 + r];
          // a scale that is no number belongs to the queries that see its key alone
          if (!whole && !(sees(gap - n * 32 - key_of(r), window) && (there(n) >> (4 * h) >> key_of(r) & 1))) p = 0.f;
          s[n][r] = p;
        }
    }
  }
  const uint32_t l16 = lane & 15, dh = (lane >> 4) & 1;
  auto value = [&](int st, int d) -> u32x4 {  // 16 keys, 32 of D
    if constexpr (LB == 16) {
      const uint32_t r = 4 * h + l16 / 4, fs = R::value_swap(r);
      const uint8_t *p = lv + (st * 16 + r) * R::kBytes + (((d * 4 + dh * 2 + ((l16 >> 1) & 1)) ^ fs) * 16) + (l16 & 1) * 8;
      const u32x2 lo = read_turned(p), hi = read_turned(p + 8 * R::kBytes);
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
      const uint32_t slot = l16 / 2, r = 8 * (slot / 4) + 4 * h + slot % 4, fs = R::value_swap(r);
      const uint8_t *p = lv + (st * 16 + r) * R::kBytes + (((d * 2 + dh) ^ fs) * 16) + (l16 & 1) * 8;
      const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) i32x2 *)(__attribute__((address_space(3))) void *)p);
      const u32x2 u = __builtin_bit_cast(u32x2, v);
      if constexpr (BARE) return widen8(T{}, u);
      return widen8_by(T{}, u, f + st * 8);
    }
  };
  u32x4 p[2 * NB];
#pragma unroll
  for (int st = 0; st < 2 * NB; st++)
#pragma unroll
    for (int i = 0; i < 4; i++) p[st][i] = pair(T{}, s[st / 2][8 * (st & 1) + 2 * i], s[st / 2][8 * (st & 1) + 2 * i + 1]);
  if constexpr (!BARE) {
    // Values that are not finite count for the queries that see them, and zero times one
    // is no number: a tile in which some query does not see every key is looked
    // through, and where there is one, those are left out of the products and
    // come after, key by key.  The other queries' sums keep their bits.
    if (!whole) {
      uint32_t most = 0;
#pragma unroll
      for (int st = 0; st < 2 * NB; st++)
#pragma unroll
        for (int d = 0; d < D / 32; d++) most = most_bits(value(st, d), most);
      if (__ballot(joined(most) > finite_bits(T{}))) {
        auto finite = [](u32x4 v) {
#pragma unroll
          for (int i = 0; i < 4; i++)
            v[i] &= ((v[i] & 0x7FFFu) > finite_bits(T{}) ? 0u : 0xFFFFu) | ((v[i] >> 16 & 0x7FFFu) > finite_bits(T{}) ? 0u : 0xFFFF0000u);
          return v;
        };
#pragma unroll
        for (int st = 0; st < 2 * NB; st++) {
#pragma unroll
          for (int d = 0; d < D / 32; d++) w.o[d] = mfma32(T{}, finite(value(st, d)), p[st], w.o[d]);
#pragma unroll 1
          for (uint32_t e = 0; e < 16; e++) {
            const uint32_t half = e >> 3, word = (e & 7) >> 1, at = st * 16 + 8 * ((e & 7) / 4) + 4 * half + (e & 3);
            const uint32_t bits = h == half ? ((e & 1) ? 0xFFFF0000u : 0xFFFFu) : 0u;
            const u32x4 only = {word == 0 ? bits : 0u, word == 1 ? bits : 0u, word == 2 ? bits : 0u, word == 3 ? bits : 0u};
            const bool seen = sees(w.pos - base - (int32_t)at, window) && (there(at / 32) >> (at % 32) & 1);
#pragma unroll
            for (int d = 0; d < D / 32; d++) {
              const u32x4 v = value(st, d);
              const f32x16 t = mfma32(T{}, (v ^ finite(v)) & only, p[st] & only, f32x16{});
#pragma unroll
              for (int r = 0; r < 16; r++) w.o[d][r] += seen ? t[r] : 0.f;
            }
          }
        }
        return;
      }
    }
  }
#pragma unroll
  for (int st = 0; st < 2 * NB; st++)
#pragma unroll
    for (int d = 0; d < D / 32; d++) w.o[d] = mfma32(T{}, value(st, d), p[st], w.o[d]);
}

// The address of a head's row in the pool.
__device__ __forceinline__ uint64_t pool_row(const Pages &c, uint32_t page, uint32_t head, uint32_t at) {
  return (((uint64_t)page * c.heads + head) << c.shift) + (at & ((1u << c.shift) - 1));
}
// Page of a position below stop, -1 where there is none.
__device__ __forceinline__ int32_t page_at(const Pages &c, const int32_t *table, int32_t pos, int32_t stop) {
  if (pos >= stop) return -1;
  const int32_t page = table[(uint32_t)pos >> c.shift];
  return (uint32_t)page < c.pages ? page : -1;
}

// Four outputs of a row, as they are or for attend_join.
template <class T>
__device__ __forceinline__ void store4(uint16_t *out, T, f32x4 v) {
  *(u32x2 *)out = u32x2{pair(T{}, v[0], v[1]), pair(T{}, v[2], v[3])};
}
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -__builtin_huge_valf() : (m + __builtin_log2f(l)) * 0.693147180559945309f;
}

template <class T, int BITS, int D, int W>
__global__ __launch_bounds__(64 * W) void attend_few(const Pages c, const Sequences b, const Attend a) {
  typedef Rows<BITS, D> R;
  constexpr int kTile = 32 * R::kBytes, kLoads = kTile / 1024, kRowsPer = 32 / kLoads;
  constexpr bool SCALED = BITS == 8, BARE = SCALED && T::kRange;
  extern __shared__ __align__(1024) uint8_t lds[];  // [W][2][keys, values], then joined
  __shared__ float scales[W][64], ms[W][32], ls[W][32];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t *buf = lds + wave * (4 * kTile);
  const uint64_t units = (uint64_t)b.count * c.heads * a.few_splits;
  for (uint64_t id = blockIdx.x; id < units; id += gridDim.x) {
    const uint32_t head = (uint32_t)(id % c.heads), s = (uint32_t)(id / c.heads % b.count), z = (uint32_t)(id / c.heads / b.count);
    const Span sp = span_of(b, s);
    const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
    if (s == 0 && z == 0) {
      // rows of no sequence
      const int32_t begin = sp.first, end = span_of(b, b.count - 1).last;
      const uint32_t per = a.group * (D / 8);
      const uint64_t all = ((uint64_t)begin + (b.tokens - end)) * per;
      for (uint64_t i = threadIdx.x; i < all; i += 64 * W) {
        const uint64_t t = i / per < (uint64_t)begin ? i / per : i / per - begin + end, e = i % per;
        ((u32x4 *)(a.out + (t * a.heads + head * a.group) * D))[e] = u32x4{0, 0, 0, 0};
        if (a.lse && e < a.group) a.lse[t * a.heads + head * a.group + e] = -__builtin_huge_valf();
      }
    }
    if (rows == 0 || (!a.alone && rows > a.cap)) continue;
    const int32_t *table = b.tables + s * b.stride;
    for (uint32_t r0 = 0; r0 < rows; r0 += r0 ? 32 : a.cap) {
      if (r0 && z) break;  // rows behind the capacity are not split
      const uint32_t most = r0 ? 32 : a.cap, count = rows - r0 < most ? rows - r0 : most;
      const int32_t first = sp.first + (int32_t)(r0 / a.group), last = sp.first + (int32_t)((r0 + count - 1) / a.group);
      const Cuts k = cuts_of(c, b, first + sp.ahead, last + sp.ahead, sp.length, a.window, kFewShift, r0 ? 1 : a.few_splits, kFewLeast);
      if (z >= (uint32_t)k.count && z) break;
      const int32_t t0 = k.begin + (int32_t)z * k.per, t1 = t0 + k.per < k.end ? t0 + k.per : k.end;
      const uint32_t mine = r0 + ((lane & 31) < count ? (lane & 31) : count - 1);
      const int32_t token = sp.first + (int32_t)(mine / a.group);
      Wave<T, BITS, D> w;
      w.init(a.q + token * a.q_token + (head * a.group + mine % a.group) * a.q_head, token + sp.ahead);
      // a tile's pages and scales come a tile ahead of its rows
      int32_t page = -1;
      float scale = 0.f;
      auto look = [&](int32_t t) { page = t < t1 ? page_at(c, table, t * 32 + (int32_t)(lane & 31), k.stop) : -1; };
      auto request = [&](int32_t t, uint8_t *dst) {
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
          const uint32_t row = i * kRowsPer + lane / R::kChunks;
          const int32_t pg = kRowsPer <= 16 ? __builtin_amdgcn_readlane(page, i * kRowsPer) : __shfl(page, (int)row);
          // (the last tile's pages begin in it, and its rows end in it)
          const bool in = pg >= 0 && t * 32 + (int32_t)row < k.stop;
          const uint64_t at = pool_row(c, (uint32_t)pg, head, (uint32_t)(t * 32) + row) * R::kBytes;
          const void *none = &g_zero16;
          to_lds(in ? c.k + at + (((lane % R::kChunks) ^ R::key_swap(row)) * 16) : none, dst + i * 1024);
          to_lds(in ? c.v + at + (((lane % R::kChunks) ^ R::value_swap(row)) * 16) : none, dst + kTile + i * 1024);
        }
        if constexpr (SCALED) {
          scale = 0.f;
          if (page >= 0) scale = (lane < 32 ? c.k_scales : c.v_scales)[pool_row(c, (uint32_t)page, head, (uint32_t)(t * 32) + (lane & 31))];
        }
      };
      const int32_t mine0 = t0 + (int32_t)wave;
      look(mine0);
      uint32_t there = (uint32_t)__ballot(page >= 0), next = 0;
      if (mine0 < t1) {
        request(mine0, buf);
        look(mine0 + W);
      }
      for (int32_t t = mine0; t < t1; t += W) {
        const uint32_t odd = ((t - mine0) / W) & 1;
        wait_but<0>();
        if constexpr (SCALED) scales[wave][lane] = lane < 32 ? scale * a.c : scale;
        next = (uint32_t)__ballot(page >= 0);
        if (t + W < t1) {
          request(t + W, buf + (odd ^ 1) * (2 * kTile));
          look(t + 2 * W);
        }
        const bool whole = there == 0xFFFFFFFFu && t * 32 + 31 <= first + sp.ahead && last + sp.ahead - t * 32 < a.window;
        const uint8_t *p = buf + odd * (2 * kTile);
        add_keys<T, BITS, BITS, D, 1, SCALED, BARE>(w, p, p + kTile, scales[wave], scales[wave] + 32, t * 32,
                                                    [=](int) { return there; }, whole, a.c, a.window);
        there = next;
        wait_reads();  // the buffer is asked for again
      }
      // the waves' sums: [W][32][D] in place of the tiles, 16-byte chunks exchanged
      const f32x2 sums = both_halves(w.l);
      __syncthreads();
      float *part = (float *)lds;
      if ((lane & 31) < count) {
#pragma unroll
        for (int d = 0; d < D / 32; d++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const uint32_t chunk = d * 8 + i * 2 + (lane >> 5);
            *(f32x4 *)(part + (wave * 32 + (lane & 31)) * D + ((chunk ^ (lane & 7)) * 4)) =
                f32x4{w.o[d][4 * i], w.o[d][4 * i + 1], w.o[d][4 * i + 2], w.o[d][4 * i + 3]};
          }
        ms[wave][lane & 31] = w.m;
        ls[wave][lane & 31] = sums[0] + sums[1];
      }
      __syncthreads();
      const bool direct = k.count <= 1;
      for (uint32_t i = threadIdx.x; i < count * (D / 4); i += 64 * W) {
        const uint32_t r = i / (D / 4), chunk = i % (D / 4);
        float m = ms[0][r];
#pragma unroll
        for (int q = 1; q < W; q++) m = __builtin_fmaxf(m, ms[q][r]);
        const float ref = m == -__builtin_huge_valf() ? 0.f : m;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        float l = 0.f;
#pragma unroll
        for (int q = 0; q < W; q++) {
          const float f = exp2_of(ms[q][r] - ref);
          v += *(const f32x4 *)(part + (q * 32 + r) * D + ((chunk ^ (r & 7)) * 4)) * f;
          l += ls[q][r] * f;
        }
        const uint32_t row = r0 + r;
        const uint64_t to = (uint64_t)(sp.first + row / a.group) * a.heads + head * a.group + row % a.group;
        if (direct) {
          store4(a.out + to * D + chunk * 4, T{}, l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : v * (1.f / l));
          if (a.lse && chunk == 0) a.lse[to] = lse_of(m, l);
        } else {
          const uint64_t at = (((uint64_t)z * b.count + s) * c.heads + head) * a.cap + row;
          *(f32x4 *)(a.few_o + at * D + chunk * 4) = v;
          if (chunk == 0) *(f32x2 *)(a.few_ml + at * 2) = f32x2{m, l};
        }
      }
      __syncthreads();
    }
  }
}

// Tile i of 128 rows lies in sequence s, whose tiles begin at starts[s] * group / 128
// (rounded down) + s: no two sequences' overlap, and what lies between them is empty.
__device__ __forceinline__ int64_t first_tile(const Sequences &b, uint32_t s, uint32_t group) {
  const int32_t at = b.starts[s];
  return (int64_t)((uint64_t)(at < 0 ? 0 : at) * group / 128) + s;
}
__device__ __forceinline__ uint32_t tile_owner(const Sequences &b, uint32_t group, int64_t tile) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0, n = b.count;  // as starts_up_to
  while (n) {
    const uint32_t step = (n + 63) / 64;
    const bool in = lane * step < n && first_tile(b, lo + lane * step, group) <= tile;
    const uint32_t k = __popcll(__ballot(in));
    if (k == 0) break;
    const uint32_t before = lo + n;
    lo = lo + (k - 1) * step + 1;
    n = lo + step - 1 < before ? step - 1 : before - lo;
  }
  return lo ? lo - 1 : b.count;
}

template <class T, int BITS, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attend_tile(const Pages c, const Sequences b, const Attend a) {
  typedef Rows<16, D> R;  // in LDS
  constexpr int kTile = 64 * R::kBytes, kLoads = kTile / 4096, kRowsPer = 1024 / R::kBytes;
  constexpr bool SCALED = BITS == 8, BARE = SCALED && T::kRange;
  constexpr int kRaw = D < 64 ? 1 : D / 64;  // 16 bytes of codes a thread
  extern __shared__ __align__(1024) uint8_t lds[];  // [2][keys, values]
  __shared__ float scales[2][128];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t units = (uint64_t)a.tiles * c.heads * a.tile_splits;
  for (uint64_t id = blockIdx.x; id < units; id += gridDim.x) {
    // the last tiles of a prompt see the most keys: they go first
    const uint32_t head = (uint32_t)(id % c.heads), z = (uint32_t)(id / c.heads % a.tile_splits);
    const int64_t tile = (int64_t)a.tiles - 1 - (int64_t)(id / c.heads / a.tile_splits);
    const uint32_t s = tile_owner(b, a.group, tile);
    if (s >= b.count) continue;
    const Span sp = span_of(b, s);
    const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
    const int64_t r0 = (tile - first_tile(b, s, a.group)) * 128;
    if (rows <= a.cap || r0 >= (int64_t)rows) continue;
    const uint32_t count = rows - (uint32_t)r0 < 128 ? rows - (uint32_t)r0 : 128;
    const int32_t first = sp.first + (int32_t)((uint32_t)r0 / a.group), last = sp.first + (int32_t)(((uint32_t)r0 + count - 1) / a.group);
    const Cuts k = cuts_of(c, b, first + sp.ahead, last + sp.ahead, sp.length, a.window, kTileShift, a.tile_splits, kTileLeast);
    if (z && z >= (uint32_t)k.count) continue;
    const int32_t t0 = k.begin + (int32_t)z * k.per, t1 = t0 + k.per < k.end ? t0 + k.per : k.end;
    const int32_t *table = b.tables + s * b.stride;
    const uint32_t in_tile = wave * 32 + (lane & 31), mine = (uint32_t)r0 + (in_tile < count ? in_tile : count - 1);
    const int32_t token = sp.first + (int32_t)(mine / a.group);
    // this wave's positions
    const uint32_t w0 = wave * 32 < count ? wave * 32 : count - 1, w1 = wave * 32 + 31 < count ? wave * 32 + 31 : count - 1;
    const int32_t wfirst = sp.first + (int32_t)(((uint32_t)r0 + w0) / a.group) + sp.ahead, wlast = sp.first + (int32_t)(((uint32_t)r0 + w1) / a.group) + sp.ahead;
    Wave<T, BITS, D> w;
    w.init(a.q + token * a.q_token + (head * a.group + mine % a.group) * a.q_head, token + sp.ahead);
    int32_t page = -1;  // of key `lane` of the tile to be asked for next
    auto look = [&](int32_t t) { page = t < t1 ? page_at(c, table, t * 64 + (int32_t)lane, k.stop) : -1; };
    u32x4 raw_k[kRaw], raw_v[kRaw];
    float raw_f[kRaw], scale = 0.f;
    auto request = [&](int32_t t, uint8_t *dst) {
      const void *none = &g_zero16;
      if constexpr (BITS == 16) {
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
          const uint32_t r = (i * 4 + wave) * kRowsPer, row = r + lane / R::kChunks;
          const int32_t pg = __builtin_amdgcn_readlane(page, r);
          const bool in = pg >= 0 && t * 64 + (int32_t)row < k.stop;
          const uint64_t at = pool_row(c, (uint32_t)pg, head, (uint32_t)(t * 64) + row) * R::kBytes;
          to_lds(in ? c.k + at + (((lane % R::kChunks) ^ R::key_swap(row)) * 16) : none, dst + (i * 4 + wave) * 1024);
          to_lds(in ? c.v + at + (((lane % R::kChunks) ^ R::value_swap(row)) * 16) : none,
                 dst + kTile + (i * 4 + wave) * 1024);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kRaw; i++) {
          const uint32_t at16 = i * 256 + threadIdx.x, row = at16 / (D / 16) & 63;
          const int32_t pg = __shfl(page, (int)row);
          const bool in = pg >= 0 && at16 < 64 * (D / 16);
          const uint64_t r = pool_row(c, (uint32_t)pg, head, (uint32_t)(t * 64) + row);
          raw_k[i] = raw_v[i] = u32x4{0, 0, 0, 0};
          raw_f[i] = 0.f;
          if (in) {
            raw_k[i] = *(const u32x4 *)(c.k + r * D + (at16 % (D / 16)) * 16);
            raw_v[i] = *(const u32x4 *)(c.v + r * D + (at16 % (D / 16)) * 16);
            if constexpr (!BARE) raw_f[i] = c.v_scales[r];
          }
        }
        scale = 0.f;
        if (wave < 2 && page >= 0) scale = (wave ? c.v_scales : c.k_scales)[pool_row(c, (uint32_t)page, head, (uint32_t)(t * 64) + lane)];
      }
    };
    // codes of 8 bits become 16-bit values on their way to LDS, once for all waves
    auto spread = [&](uint8_t *dst, float *sc) {
      if constexpr (BITS == 8) {
#pragma unroll
        for (int i = 0; i < kRaw; i++) {
          const uint32_t at16 = i * 256 + threadIdx.x, row = at16 / (D / 16), chunk = at16 % (D / 16) * 2;
          if (at16 >= 64 * (D / 16)) break;
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; e++) f[e] = raw_f[i];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const u32x2 kc = {raw_k[i][2 * e], raw_k[i][2 * e + 1]}, vc = {raw_v[i][2 * e], raw_v[i][2 * e + 1]};
            *(u32x4 *)(dst + row * R::kBytes + (((chunk + e) ^ R::key_swap(row)) * 16)) = widen8(T{}, kc);
            *(u32x4 *)(dst + kTile + row * R::kBytes + (((chunk + e) ^ R::value_swap(row)) * 16)) =
                BARE ? widen8(T{}, vc) : widen8_by(T{}, vc, f);
          }
        }
        if (wave < 2) sc[wave * 64 + lane] = wave ? scale : scale * a.c;
      }
    };
    look(t0);
    uint64_t there = __ballot(page >= 0), next = 0;
    if (t0 < t1) {
      request(t0, lds);
      look(t0 + 1);
      if constexpr (BITS == 8) {
        spread(lds, scales[0]);
        next = __ballot(page >= 0);
        if (t0 + 1 < t1) {
          request(t0 + 1, nullptr);
          look(t0 + 2);
        }
      }
    }
    for (int32_t t = t0; t < t1; t++) {
      const uint32_t odd = (t - t0) & 1;
      uint8_t *p = lds + odd * (2 * kTile), *other = lds + (odd ^ 1) * (2 * kTile);
      uint64_t after = 0;
      if constexpr (BITS == 16) {
        wait_but<0>();
        meet();  // tile t is whole, and tile t - 1 read by all
        next = __ballot(page >= 0);
        if (t + 1 < t1) {
          request(t + 1, other);
          look(t + 2);
        }
      } else {
        __syncthreads();
        if (t + 1 < t1) {
          spread(other, scales[odd ^ 1]);
          after = __ballot(page >= 0);
          if (t + 2 < t1) {
            request(t + 2, nullptr);
            look(t + 3);
          }
        }
      }
      if (t * 64 <= wlast && wfirst - (t * 64 + 63) < a.window) {  // some row of this wave sees some key
        const bool whole = there == ~0ull && t * 64 + 63 <= wfirst && wlast - t * 64 < a.window;
        const uint32_t lo = (uint32_t)there, hi = (uint32_t)(there >> 32);
        add_keys<T, BITS, 16, D, 2, SCALED, BARE>(w, p, p + kTile, scales[odd], scales[odd] + 64, t * 64,
                                                  [=](int n) { return n ? hi : lo; }, whole, a.c, a.window);
      }
      there = next;
      if constexpr (BITS == 8) next = after;
    }
    __syncthreads();  // the buffers are read
    const f32x2 sums = both_halves(w.l);
    const float l = sums[0] + sums[1];
    if (in_tile < count) {
      const uint64_t to = (uint64_t)token * a.heads + head * a.group + mine % a.group;
      const bool direct = k.count <= 1;
      const float f = direct ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const uint64_t at = (uint64_t)z * b.tokens * a.heads + to;
#pragma unroll
      for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const uint32_t e = d * 32 + i * 8 + (lane >> 5) * 4;
          const f32x4 v = f32x4{w.o[d][4 * i], w.o[d][4 * i + 1], w.o[d][4 * i + 2], w.o[d][4 * i + 3]} * f;
          if (direct) {
            store4(a.out + to * D + e, T{}, v);
          } else {
            *(f32x4 *)(a.tile_o + at * D + e) = v;
          }
        }
      if (lane < 32) {
        if (!direct) {
          *(f32x2 *)(a.tile_ml + at * 2) = f32x2{w.m, l};
        } else if (a.lse) {
          a.lse[to] = lse_of(w.m, l);
        }
      }
    }
  }
}

// A row's parts added up, D / 4 lanes to a row: the rows of few (sequence, key head,
// row), then those of tiles (token, head), where either was split.
template <class T, int D>
__global__ __launch_bounds__(256) void attend_join(const Pages c, const Sequences b, const Attend a) {
  constexpr uint32_t kLanes = D / 4;
  const uint64_t few = a.few_splits > 1 ? (uint64_t)b.count * c.heads * a.cap : 0;
  const uint64_t tiled = a.tile_splits > 1 ? (uint64_t)b.tokens * a.heads : 0;
  const uint32_t chunk = threadIdx.x % kLanes;
  // a wave's rows go together: the search below is the whole wave's
  const uint64_t all = (few + tiled) * kLanes;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i - (threadIdx.x & 63) < all; i += (uint64_t)gridDim.x * 256) {
    const bool in = i < all;
    uint64_t row = (in ? i : all - 1) / kLanes;
    const float *o, *ml;
    uint64_t to, stride;
    int32_t parts = 0;
    const uint64_t base = (i - (threadIdx.x & 63)) / kLanes, top = base + 64 / kLanes - 1;  // the wave's first and last row
    uint32_t owner = b.count;
    if (top >= few) {
      // rows of a wave may lie in several sequences: each looks for its own in turn
#pragma unroll 1
      for (uint32_t r = 0; r < 64 / kLanes; r++) {
        const uint64_t rr = base + r;
        if (rr < few || rr >= few + tiled) continue;
        const uint32_t s = sequence_of(b, (int32_t)((rr - few) / a.heads));
        if (row == rr) owner = s;
      }
    }
    if (row < few) {
      const uint32_t r = (uint32_t)(row % a.cap), head = (uint32_t)(row / a.cap % c.heads), s = (uint32_t)(row / a.cap / c.heads);
      const Span sp = span_of(b, s);
      const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
      o = a.few_o;
      ml = a.few_ml;
      stride = few;
      to = (uint64_t)(sp.first + r / a.group) * a.heads + head * a.group + r % a.group;
      if (r < rows && (a.alone || rows <= a.cap)) {
        const uint32_t count = rows < a.cap ? rows : a.cap;
        parts = cuts_of(c, b, sp.first + sp.ahead, sp.first + (int32_t)((count - 1) / a.group) + sp.ahead, sp.length, a.window, kFewShift,
                        a.few_splits, kFewLeast).count;
      }
    } else {
      row -= few;
      o = a.tile_o;
      ml = a.tile_ml;
      stride = tiled;
      to = row;
      const int32_t t = (int32_t)(row / a.heads);
      if (owner < b.count) {
        const Span sp = span_of(b, owner);
        const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
        if (t >= sp.first && t < sp.last && rows > a.cap) {
          const uint32_t r = (uint32_t)(t - sp.first) * a.group + (uint32_t)(row % a.heads) % a.group, r0 = r & ~127u;
          const uint32_t count = rows - r0 < 128 ? rows - r0 : 128;
          parts = cuts_of(c, b, sp.first + (int32_t)(r0 / a.group) + sp.ahead, sp.first + (int32_t)((r0 + count - 1) / a.group) + sp.ahead,
                          sp.length, a.window, kTileShift, a.tile_splits, kTileLeast).count;
        }
      }
    }
    if (!in || parts <= 1) continue;
    float m = -__builtin_huge_valf();
    for (int32_t p = 0; p < parts; p++) m = __builtin_fmaxf(m, ml[(p * stride + row) * 2]);
    const float ref = m == -__builtin_huge_valf() ? 0.f : m;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll 4
    for (int32_t p = 0; p < parts; p++) {
      const f32x2 t = *(const f32x2 *)(ml + (p * stride + row) * 2);
      const float f = exp2_of(t[0] - ref);
      v += *(const f32x4 *)(o + (p * stride + row) * D + chunk * 4) * f;
      l += t[1] * f;
    }
    store4(a.out + to * D + chunk * 4, T{}, l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : v * (1.f / l));
    if (a.lse && chunk == 0) a.lse[to] = lse_of(m, l);
  }
}

// ------------------------------------------------------------------- host
// What a call launches, by what the host knows: rows and table widths, not lengths.
struct Plan {
  Attend a;
  bool tile;
  uint64_t few_o, few_ml, tile_o, tile_ml, all;  // workspace offsets
};
constexpr uint64_t kMostParts = 256u << 20;  // bytes of partial sums

Plan plan_of(const df_cache *cache, const df_cache_batch *batch, uint64_t tokens, uint32_t heads, int64_t window) {
  Plan p = {};
  Attend &a = p.a;
  const uint64_t kv = cache->kv_heads, seqs = batch->seqs, dim = cache->head_dim;
  a.heads = heads;
  a.group = heads / cache->kv_heads;
  a.window = window <= 0 || window > INT32_MAX ? INT32_MAX : (int32_t)window;
  const uint64_t hint = batch->max_new && batch->max_new < tokens ? batch->max_new : tokens;
  p.tile = hint * a.group > 32;
  a.alone = !p.tile;
  const uint64_t fit = 32 / a.group;
  a.cap = (uint32_t)((hint < fit ? hint : fit) * a.group);
  a.few_splits = a.tile_splits = 1;
  // the most keys that a sequence's rows may see
  const uint64_t held = (uint64_t)batch->width * cache->page_size;
  const uint64_t seen = held < (uint64_t)a.window + hint ? held : (uint64_t)a.window + hint;
  if (a.cap) {
    // a round or two of workgroups, and no part longer than 2048 keys
    const uint64_t units = seqs * kv, most = (seen + 31) / 32 + 1, slots = cache->bits == 16 ? 512 : 1024;
    uint64_t n = (slots + units - 1) / units;
    if (n < (most + 63) / 64) n = (most + 63) / 64;
    if (n > (most + kFewLeast - 1) / kFewLeast) n = (most + kFewLeast - 1) / kFewLeast;
    const uint64_t part = units * a.cap * (dim + 2) * 4;
    if (n * part > kMostParts) n = kMostParts / part;
    if (n > 512) n = 512;
    a.few_splits = n < 1 ? 1 : (uint32_t)n;
  }
  if (p.tile) {
    a.tiles = (uint32_t)(tokens * a.group / 128 + seqs);
    const uint64_t units = (tokens * a.group + 127) / 128 * kv, most = (seen + 63) / 64 + 1;
    uint64_t n = units >= 512 ? 1 : 512 / units;
    if (n > most / kTileLeast) n = most / kTileLeast;
    const uint64_t part = tokens * heads * (dim + 2) * 4;
    if (n * part > kMostParts) n = kMostParts / part;
    if (n > 16) n = 16;
    a.tile_splits = n < 1 ? 1 : (uint32_t)n;
  }
  uint64_t at = 0;
  if (a.few_splits > 1) {
    const uint64_t rows = a.few_splits * seqs * kv * a.cap;
    p.few_o = at;
    at += up(rows * dim * 4, 256);
    p.few_ml = at;
    at += up(rows * 8, 256);
  }
  if (a.tile_splits > 1) {
    const uint64_t rows = a.tile_splits * tokens * heads;
    p.tile_o = at;
    at += up(rows * dim * 4, 256);
    p.tile_ml = at;
    at += up(rows * 8, 256);
  }
  p.all = at;
  return p;
}

constexpr uint32_t kDeclared = 4096;  // LDS that the kernels declare beside what a launch gives, at most
uint32_t grid_of(uint64_t units) { return (uint32_t)(units < (1u << 20) ? units : 1u << 20); }

template <class T, int BITS, int D>
hipError_t attend(const Plan &p, const Pages &c, const Sequences &b, hipStream_t s) {
  // attend_few goes always: it clears the rows of no sequence
  constexpr int W = BITS == 16 && D == 256 ? 2 : 4;
  constexpr uint32_t few = W * 4 * 32 * Rows<BITS, D>::kBytes;
  static_assert(few >= W * 32 * D * 4, "the waves' sums lie in the tiles' place");
  const hipError_t e = allow_lds((const void *)attend_few<T, BITS, D, W>, few, kDeclared);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attend_few<T, BITS, D, W>), dim3(grid_of((uint64_t)b.count * c.heads * p.a.few_splits)), dim3(64 * W), few, s, c,
                     b, p.a);
  const hipError_t launched = hipGetLastError();
  if (launched != hipSuccess) return launched;
  if (p.tile) {
    constexpr uint32_t lds = 4 * 64 * Rows<16, D>::kBytes;
    const hipError_t st0 = allow_lds((const void *)attend_tile<T, BITS, D>, lds, kDeclared);
    if (st0 != hipSuccess) return st0;
    hipLaunchKernelGGL((attend_tile<T, BITS, D>), dim3(grid_of((uint64_t)p.a.tiles * c.heads * p.a.tile_splits)), dim3(256), lds, s, c,
                       b, p.a);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  const uint64_t rows = (p.a.few_splits > 1 ? (uint64_t)b.count * c.heads * p.a.cap : 0) +
                        (p.a.tile_splits > 1 ? (uint64_t)b.tokens * p.a.heads : 0);
  if (rows) {
    hipLaunchKernelGGL((attend_join<T, D>), dim3(grid_of((rows * (D / 4) + 255) / 256)), dim3(256), 0, s, c, b, p.a);
    return hipGetLastError();
  }
  return hipSuccess;
}
template <class T, int BITS>
hipError_t attend_dim(const Plan &p, const Pages &c, const Sequences &b, hipStream_t s) {
  switch (c.dim) {
    case 32: return attend<T, BITS, 32>(p, c, b, s);
    case 64: return attend<T, BITS, 64>(p, c, b, s);
    case 128: return attend<T, BITS, 128>(p, c, b, s);
    default: return attend<T, BITS, 256>(p, c, b, s);
  }
}

__global__ __launch_bounds__(256) void no_sequences(uint16_t *out, float *lse, uint64_t rows, uint32_t dim) {
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < rows * (dim / 8); i += (uint64_t)gridDim.x * 256) {
    ((u32x4 *)out)[i] = u32x4{0, 0, 0, 0};
    if (lse && i < rows) lse[i] = -__builtin_huge_valf();
  }
}

bool call_ok(const df_cache *cache, const df_cache_batch *batch, uint64_t tokens, uint32_t heads) {
  if (!cache_ok(cache) || !batch_ok(batch, tokens)) return false;
  if (heads == 0 || heads % cache->kv_heads || heads / cache->kv_heads > 256) return false;
  return tokens * (heads / cache->kv_heads) <= (1u << 30);
}

}  // namespace

extern "C" {

uint64_t df_cached_attention_workspace_bytes(const df_cache *cache, const df_cache_batch *batch, uint64_t tokens, uint32_t heads,
                                             int64_t window) {
  if (!call_ok(cache, batch, tokens, heads) || tokens == 0 || batch->seqs == 0) return 0;
  return plan_of(cache, batch, tokens, heads, window).all;
}

df_status df_cached_attention(const df_cache *cache, const df_cache_batch *batch, const void *q, uint64_t q_token_stride,
                              uint64_t q_head_stride, uint64_t tokens, uint32_t heads, float scale, int64_t window, void *out,
                              float *lse, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
  if (!call_ok(cache, batch, tokens, heads) || !(scale > 0.f) || !(scale < __builtin_huge_valf()) || window < 0) return DF_ERR_ARG;
  if (tokens == 0) return DF_OK;
  if (!q || !out || (((uintptr_t)q | (uintptr_t)out) & 15) || ((uintptr_t)lse & 3) || q_token_stride % 8 || q_head_stride % 8 ||
      q_token_stride > (1u << 30) || q_head_stride > (1u << 30))
    return DF_ERR_ARG;
  if (batch->seqs == 0) {
    hipLaunchKernelGGL(no_sequences, dim3(1024), dim3(256), 0, stream, (uint16_t *)out, lse, tokens * heads, cache->head_dim);
    return hipGetLastError() == hipSuccess ? DF_OK : DF_ERR_HIP;
  }
  Plan p = plan_of(cache, batch, tokens, heads, window);
  if (p.all && (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < p.all)) return DF_ERR_ARG;
  Attend &a = p.a;
  uint8_t *ws = (uint8_t *)workspace;
  a.q = (const uint16_t *)q;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.out = (uint16_t *)out;
  a.lse = lse;
  a.c = scale * 1.44269504088896341f;
  a.few_o = (float *)(ws + p.few_o);
  a.few_ml = (float *)(ws + p.few_ml);
  a.tile_o = (float *)(ws + p.tile_o);
  a.tile_ml = (float *)(ws + p.tile_ml);
  const Pages c = pages_of(cache);
  const Sequences b = sequences_of(batch, tokens);
  const hipError_t e = cache->type == DF_TYPE_BF16
                           ? (cache->bits == 8 ? attend_dim<BF16, 8>(p, c, b, stream) : attend_dim<BF16, 16>(p, c, b, stream))
                           : (cache->bits == 8 ? attend_dim<F16, 8>(p, c, b, stream) : attend_dim<F16, 16>(p, c, b, stream));
  return e == hipSuccess ? DF_OK : DF_ERR_HIP;
}

}  // extern "C"
