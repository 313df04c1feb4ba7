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
// others: 128 or 256 rows share tiles of 64 keys.  join_few and join_tiles add up what splits
// leave.
//
// Roundings: q and 16-bit keys and values are taken as they are, codes of 8 bits are
// exact in both 16-bit types.  A token's scale of keys multiplies the FP32 scores; its
// scale of values multiplies p before that is rounded to 16 bits: the one rounding (half a
// step, up to 2^-8 or 2^-11 of it) beside the output's.  Sums are FP32.
#include <hip/hip_runtime.h>

#include <type_traits>

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

// Infinities and NaN made zero.
template <class T>
__device__ __forceinline__ u32x4 finite_part(T, u32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; i++)
    v[i] &= ((v[i] & 0x7FFFu) > finite_bits(T{}) ? 0u : 0xFFFFu) | ((v[i] >> 16 & 0x7FFFu) > finite_bits(T{}) ? 0u : 0xFFFF0000u);
  return v;
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
struct Attend {
  const uint16_t *q;
  uint64_t q_token, q_head;  // strides in elements
  uint16_t *out;             // [tokens, heads, D]
  float *lse;                // [tokens, heads], or null
  uint32_t heads, group;     // heads a key head
  int32_t window;            // INT32_MAX: none
  float c;                   // scale times log2 e
  // few rows
  uint32_t cap;
  uint32_t alone;            // no attend_tile follows: sequences of more rows are taken too
  uint32_t few_splits;       // whether rows may be split
  float *few_o, *few_ml;     // [workgroups + seqs * kv heads][cap][D], [..][2]
  uint32_t *few_parts;       // [seqs][kv heads][2]: parts, and the first one's place in few_o
  // tiles
  uint32_t tiles, tile_rows, tile_splits;
  float *tile_o, *tile_ml;   // [splits][tokens][heads][D], [..][2]
};

// The keys that rows at positions first .. last see, in units of 2^shift, cut into
// `count` parts of `per`: `splits` of them, of `least` units or more.
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

// What codes of 8 bits become to multiply q: FP16, which is made of bytes with half of the
// instructions that BF16 takes, for a lifted q (lift_q).
template <class T, int BITS>
struct KeyType {
  typedef T type;
};
template <class T>
struct KeyType<T, 8> {
  typedef F16 type;
};

// A tile of keys or values in LDS, 16 bits a value: rows of D, 16-byte chunks exchanged
// within a row (in the source address, where a load writes LDS linearly).  Keys are
// read 16 bytes at one chunk of 32 rows, 16 rows at once: those in a row fall into 16 places of
// 256 bytes (of heads of 256 only 8: all of a wave's loads have one exchange).  Values are read
// transposed, 64 bytes of 8 rows: neighbours fall into different ones.
template <int D>
struct Rows {
  static constexpr int kBytes = D * 2, kChunks = kBytes / 16;
  static constexpr int kPer = kBytes >= 128 ? 1 : 128 / kBytes;  // rows in 128 bytes
  static constexpr int kKeyPer = kBytes >= 256 ? 1 : 256 / kBytes;
  static constexpr int kKeyPlaces = kChunks <= 16 ? kChunks : 8;
  static constexpr int kUnits = kChunks < 4 ? 1 : kChunks / 4 < 4 ? kChunks / 4 : 4;
  static __device__ __forceinline__ uint32_t key_swap(uint32_t r) { return (r / kKeyPer) & (kKeyPlaces - 1); }
  static __device__ __forceinline__ uint32_t value_swap(uint32_t r) { return ((r / kPer) & (kUnits - 1)) * 4; }
};

// Key of a lane's register r (of 16) in a block of 32, without the 4 * (lane / 32).
__device__ __forceinline__ constexpr int key_of(int r) { return 8 * (r / 4) + r % 4; }

// 16 bytes a lane from base + off (of each lane) to LDS address at + 16 lane.  The
// compiler is not told of these loads: before a transposing read it would wait for all that it
// knows of, the next tile's among them (4096 x 16384 x 32 heads 1038 us, unknown 967).  A load
// of this kind writes no register but m0, which nothing else here uses; what it writes in LDS is
// waited for by wait_but.
__device__ __forceinline__ uint32_t same(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t same(uint64_t v) { return (uint64_t)same((uint32_t)(v >> 32)) << 32 | same((uint32_t)v); }
__device__ __forceinline__ void ask(const uint8_t *base, uint32_t off, uint32_t at) {
  base = (const uint8_t *)same((uint64_t)base);
  at = same(at);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void ask(const uint8_t *src, uint32_t at) {
  at = same(at);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "memory");
}
__device__ __forceinline__ void ask_word(const uint8_t *src, uint32_t at) {  // 4 bytes a lane
  at = same(at);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(src) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// q's elements lifted into FP16 by a power of two that brings the row's largest (most) to
// 2^14 .. 2^15, so that what is 2^-28 of that keeps all its bits; returns what takes it back.
template <int N>
__device__ __forceinline__ float lift_q(u32x4 (&q)[N], float most) {
  const int up = lift_bits(most, 14);
#pragma unroll
  for (int st = 0; st < N; st++)
#pragma unroll
    for (int i = 0; i < 4; i++)
      q[st][i] = pair(F16{}, __builtin_ldexpf(from_bits(BF16{}, (uint16_t)q[st][i]), up),
                      __builtin_ldexpf(from_bits(BF16{}, (uint16_t)(q[st][i] >> 16)), up));
  return power_of_two(-up);
}

// What 32 queries of a wave gather: lane l has query l % 32.
template <class T, int BITS, int D>
struct Wave {
  u32x4 q[D / 16];
  f32x16 o[D / 32];
  float m, l;       // reference of the exponentials (times log2 e), this half's sum
  float z, lift;    // the largest score, where m lies below it
  float mul;        // what a score is multiplied by
  int32_t pos;
  uint32_t key_at, value_at;  // this lane's part of a tile in LDS

  // row: this lane's query
  __device__ __forceinline__ void init(const uint16_t *row, int32_t position, float c) {
    const uint32_t h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int s = 0; s < D / 16; s++) q[s] = *(const u32x4 *)(row + (s * 2 + h) * 8);
    mul = BITS == 8 ? 1.f : c;
    if constexpr (BITS == 8 && T::kRange) {
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < D / 16; s++) top = most_bits(q[s], top);
      const f32x2 tops = both_halves(from_bits(T{}, (uint16_t)joined(top)));
      mul = lift_q(q, __builtin_fmaxf(tops[0], tops[1]));
    }
#pragma unroll
    for (int d = 0; d < D / 32; d++) o[d] = f32x16{};
    m = z = -__builtin_huge_valf();
    l = 0.f;
    lift = 64.f;
    pos = position;
    // chunk h of row lane % 32 (step st: that ^ 2 st); of 4 rows by 16 values a group of 16 lanes, 8 bytes
    // (of values 32 d on: that ^ 4 d chunks)
    typedef Rows<D> R;
    const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, r = 4 * h + l16 / 4;
    key_at = (lane & 31) * R::kBytes + (h ^ R::key_swap(lane & 31)) * 16;
    value_at = r * R::kBytes + ((((lane >> 4) & 1) * 2 + ((l16 >> 1) & 1)) ^ R::value_swap(r)) * 16 + (l16 & 1) * 8;
  }
};

// FP16 with codes: exponentials are taken off a reference that lies `lift` below the row's
// largest score, the least lift of the tiles so far that brings the largest scale of the
// values it sees to 2^14 .. 2^15, so p times a scale neither overflows nor loses
// bits until it is 2^-28 of the largest.  Values of FP16 span 2^40, so what is lost below lies under
// their own steps.  The sum of p is off by the same power of two.
constexpr bool lifts(bool range, int bits) { return bits == 8 && !range; }
__device__ __forceinline__ float value_lift(float largest, float so_far) {
  const int up = lift_bits(largest, 14);
  const float f = (float)(up < -64 ? -64 : up > 64 ? 64 : up);
  return largest > 0.f && f < so_far ? f : so_far;
}

// Whether a query at pos sees the key at pos - gap.
__device__ __forceinline__ bool sees(int32_t gap, int32_t window) { return (uint32_t)gap < (uint32_t)window; }

// LDS by address.
template <class V>
__device__ __forceinline__ V read_lds(uint32_t at) {
  return *(const __attribute__((address_space(3))) V *)at;
}
__device__ __forceinline__ u32x2 turned_lds(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)at));
}
// The same value, in a register that the compiler knows nothing of: what is made of it is
// made again where it is used, not kept from one tile to the next in registers that the
// sums need.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Blocks of 32 keys in LDS, 16 bits a value, go through four steps: scores (matrix), settle (scale,
// mask, maximum), weigh (exponentials) and gather (matrix).  BITS 8: ks are scales of the
// keys times c, vs of the values.  Not MASKED: every query sees every key.
template <class T, int BITS, int D>
__device__ __forceinline__ f32x16 scores(const Wave<T, BITS, D> &w, uint32_t lk) {
  typedef typename KeyType<T, BITS>::type K;
  const uint32_t at = lk + fresh(w.key_at);
  f32x16 s = {};
#pragma unroll
  for (int st = 0; st < D / 16; st++) s = mfma32(K{}, read_lds<u32x4>(at ^ st * 32), w.q[st], s);
  return s;
}

// Which of a lane's keys, by register, its query sees.  there: bit j: key j of the block exists.
struct Seen {
  int32_t gap, window;
  uint32_t there;
  template <class W>
  __device__ __forceinline__ Seen(const W &w, int32_t base, uint32_t all, int32_t win) {
    const uint32_t h = (threadIdx.x >> 5) & 1;
    gap = w.pos - base - 4 * (int32_t)h;
    there = all >> (4 * h);
    window = win;
  }
  __device__ __forceinline__ bool operator()(int r) const { return sees(gap - key_of(r), window) && (there >> key_of(r) & 1); }
};

// The reference that a row's largest score asks for, where that is lifted.
template <class W, class S>
__device__ __forceinline__ float lifted(W &w, float top, const float *vs, S seen) {
  const uint32_t h = (threadIdx.x >> 5) & 1;
  float largest = 0.f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const f32x4 v = *(const f32x4 *)(vs + 8 * i + 4 * h);
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (seen(4 * i + e)) largest = __builtin_fmaxf(largest, __builtin_fabsf(v[e]));
  }
  const f32x2 both = both_halves(largest);
  w.lift = value_lift(__builtin_fmaxf(both[0], both[1]), w.lift);
  w.z = __builtin_fmaxf(top, w.z);
  return w.z - w.lift;
}

// Scores times the keys' scales, -inf where a key is not seen; returns the row's largest (times log2 e).
template <class T, int BITS, int D, bool MASKED>
__device__ __forceinline__ float settle(Wave<T, BITS, D> &w, f32x16 &s, const float *ks, const float *vs, const Seen &seen) {
  const uint32_t h = (threadIdx.x >> 5) & 1;
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const f32x4 k = *(const f32x4 *)(ks + 8 * i + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; e++) s[4 * i + e] *= k[e];
    }
  }
  if constexpr (MASKED) {
#pragma unroll
    for (int r = 0; r < 16; r++)
      if (!seen(r)) s[r] = -__builtin_huge_valf();
  }
  float top = s[0];
#pragma unroll
  for (int r = 1; r < 16; r++) top = __builtin_fmaxf(top, s[r]);
  const f32x2 tops = both_halves(top);
  top = __builtin_fmaxf(tops[0], tops[1]) * w.mul;
  if constexpr (lifts(T::kRange, BITS)) top = lifted(w, top, vs, [&](int r) { return !MASKED || seen(r); });
  return top;
}

// A row's reference stays while no score is more than 2^8 above it (codes of FP16: none): p and
// its sums bear that, and most tiles take nothing off (32 rows with a maximum of their own
// would in every third of 256).
template <class T, int BITS, int D>
__device__ __forceinline__ void refer(Wave<T, BITS, D> &w, float top) {
  constexpr float kSlack = lifts(T::kRange, BITS) ? 0.f : 8.f;
  if (__ballot(top > w.m + kSlack)) {
    const float up = top > w.m + kSlack ? top : w.m, back = exp2_of(w.m - (up == -__builtin_huge_valf() ? 0.f : up));
    w.l *= back;
#pragma unroll
    for (int d = 0; d < D / 32; d++) w.o[d] *= back;
    w.m = up;
  }
}

// Exponentials of settled scores, as the operand of gather.
template <class T, int BITS, int D, bool MASKED>
__device__ __forceinline__ void weigh(Wave<T, BITS, D> &w, const f32x16 &s, u32x4 (&p)[2], const float *vs, const Seen &seen) {
  const uint32_t h = (threadIdx.x >> 5) & 1;
  const float ref = w.m == -__builtin_huge_valf() ? 0.f : w.m;
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int st = 0; st < 2; st++) {
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
      z[e] = exp2_of(__builtin_fmaf(s[8 * st + e], w.mul, -ref));
      sum[e & 1] += z[e];
    }
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const f32x4 v = *(const f32x4 *)(vs + st * 16 + 8 * i + 4 * h);
        // a scale that is no number belongs to the queries that see its key alone
#pragma unroll
        for (int e = 0; e < 4; e++) z[4 * i + e] = !MASKED || seen(8 * st + 4 * i + e) ? z[4 * i + e] * v[e] : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) p[st][i] = pair(T{}, z[2 * i], z[2 * i + 1]);
  }
  w.l += sum[0] + sum[1];
}

// Sixteen keys (from 16 st on, in the order of p) of 32 values (from 32 d on), turned.
// at: of a lane's part of the tile (value_at).
template <int D>
__device__ __forceinline__ u32x4 turned_values(uint32_t at, int st, int d) {
  typedef Rows<D> R;
  const uint32_t p = (at ^ d * 64) + st * 16 * R::kBytes;
  const u32x2 lo = turned_lds(p), hi = turned_lds(p + 8 * R::kBytes);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}
template <class T, int BITS, int D, bool MASKED>
__device__ __forceinline__ void gather(Wave<T, BITS, D> &w, const u32x4 (&p)[2], uint32_t lv, int32_t base, uint32_t there,
                                       int32_t window) {
  const uint32_t at = lv + fresh(w.value_at);
  // Values that are not finite count for the queries that see them, and zero times one is no
  // number: a block in which some query does not see every key is looked through, and where
  // there is one, those are left out of the products and come after, key by key.  The
  // other queries' sums keep their bits.  (One after the other: a rare way does not need the
  // registers that the usual one lives on.)
  bool odd = false;
  if constexpr (BITS == 16 && MASKED) {
    uint32_t most = 0;
#pragma unroll
    for (int st = 0; st < 2; st++)
#pragma unroll
      for (int d = 0; d < D / 32; d++) {
        most = most_bits(turned_values<D>(at, st, d), most);
        __builtin_amdgcn_sched_barrier(0);
      }
    odd = __ballot(joined(most) > finite_bits(T{})) != 0;
  }
#pragma unroll
  for (int st = 0; st < 2; st++)
#pragma unroll
    for (int d = 0; d < D / 32; d++) {
      u32x4 v = turned_values<D>(at, st, d);
      if (odd) v = finite_part(T{}, v);
      w.o[d] = mfma32(T{}, v, p[st], w.o[d]);
    }
  if (odd) {
    const uint32_t h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int st = 0; st < 2; st++) {
#pragma unroll 1
      for (uint32_t e = 0; e < 16; e++) {
        const uint32_t half = e >> 3, word = (e & 7) >> 1, key = st * 16 + 8 * ((e & 7) / 4) + 4 * half + (e & 3);
        const uint32_t bits = h == half ? ((e & 1) ? 0xFFFF0000u : 0xFFFFu) : 0u;
        const u32x4 only = {word == 0 ? bits : 0u, word == 1 ? bits : 0u, word == 2 ? bits : 0u, word == 3 ? bits : 0u};
        const bool is = sees(w.pos - base - (int32_t)key, window) && (there >> key & 1);
#pragma unroll
        for (int d = 0; d < D / 32; d++) {
          const u32x4 v = turned_values<D>(at, st, d);
          const f32x16 t = mfma32(T{}, (v ^ finite_part(T{}, v)) & only, p[st] & only, f32x16{});
#pragma unroll
          for (int r = 0; r < 16; r++) w.o[d][r] += is ? t[r] : 0.f;
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
}

// All of that at once for keys that every query sees: the scores of the next 32 keys (at lk, left
// settled in next; returns their largest) beside the weights of these (settled scores s) and
// their sums (values at lv).  Products and vector instructions are dealt out by
// hand, a slot to a product: in slots of the scores the first half of the exponentials, in those
// of the sums the second half, which the later sums take, then the maximum; reads
// run two slots ahead.  (Left to itself the compiler puts the parts one after the other:
// 4096 x 16384 x 32 heads 1101 us where this order took 967.)
template <class T, int BITS, int D>
__device__ __forceinline__ float half_step(Wave<T, BITS, D> &w, const f32x16 &s, f32x16 &next, uint32_t lk, uint32_t lv, const float *vs,
                                           const float *next_ks, const float *next_vs) {
  typedef typename KeyType<T, BITS>::type K;
  constexpr int N = D / 16;  // products of the scores, and of the sums
  const uint32_t h = (threadIdx.x >> 5) & 1;
  const float ref = w.m == -__builtin_huge_valf() ? 0.f : w.m;
  const uint32_t ka = lk + fresh(w.key_at), va = lv + fresh(w.value_at);
  u32x4 kf[N], vf[N], p[2];
  f32x4 by[BITS == 8 ? 4 : 1], keys[BITS == 8 ? 4 : 1];
  float z[16], sum[2] = {0.f, 0.f}, top = -__builtin_huge_valf();
  auto weight = [&](int e) {
    z[e] = exp2_of(__builtin_fmaf(s[e], w.mul, -ref));
    sum[e & 1] += z[e];
    if constexpr (BITS == 8) z[e] *= by[e / 4][e % 4];
    if (e & 1) p[e / 8][e % 8 / 2] = pair(T{}, z[e - 1], z[e]);
  };
  // what a slot makes stays in it
  auto slot_ends = [&] {
    asm volatile("" : "+v"(sum[0]), "+v"(sum[1]), "+v"(top));
    __builtin_amdgcn_sched_barrier(0);
  };
  auto read_key = [&](int i) { kf[i] = read_lds<u32x4>(ka ^ i * 32); };
  auto read_value = [&](int i) { vf[i] = turned_values<D>(va, i / (D / 32), i % (D / 32)); };
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 4; i++) by[i] = *(const f32x4 *)(vs + 8 * i + 4 * h);
  }
  next = f32x16{};
  __builtin_amdgcn_s_setprio(1);
  __builtin_amdgcn_sched_barrier(0);
  read_key(0);
  if (N > 1) read_key(1);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; i++) {
    if (i + 2 < N) read_key(i + 2);
    else read_value(i + 2 - N);
    next = mfma32(K{}, kf[i], w.q[i], next);
#pragma unroll
    for (int e = 8 * i / N; e < 8 * (i + 1) / N; e++) weight(e);
    slot_ends();
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    if (i + 2 < N) read_value(i + 2);
    if (BITS == 8 && i == N / 2 - 1) {
#pragma unroll
      for (int j = 0; j < 4; j++) keys[j] = *(const f32x4 *)(next_ks + 8 * j + 4 * h);
    }
    w.o[i % (D / 32)] = mfma32(T{}, vf[i], p[i / (D / 32)], w.o[i % (D / 32)]);
    if (i < N / 2) {
#pragma unroll
      for (int e = 8 + 16 * i / N; e < 8 + 16 * (i + 1) / N; e++) weight(e);
    } else {
#pragma unroll
      for (int r = 32 * (i - N / 2) / N; r < 32 * (i + 1 - N / 2) / N; r++) {
        if constexpr (BITS == 8) next[r] *= keys[r / 4][r % 4];
        top = __builtin_fmaxf(top, next[r]);
      }
    }
    slot_ends();
  }
  __builtin_amdgcn_s_setprio(0);
  w.l += sum[0] + sum[1];
  const f32x2 tops = both_halves(top);
  top = __builtin_fmaxf(tops[0], tops[1]) * w.mul;
  if constexpr (lifts(T::kRange, BITS)) top = lifted(w, top, next_vs, [](int) { return true; });
  return top;
}

// The address of a head's row in the pool.
__device__ __forceinline__ uint64_t pool_row(const Pages &c, uint32_t page, uint32_t head, uint32_t at) {
  return (((uint64_t)page * c.heads + head) << c.shift) + (at & ((1u << c.shift) - 1));
}

// Four outputs of a row, as they are or for the join.
template <class T>
__device__ __forceinline__ void store4(uint16_t *out, T, f32x4 v) {
  *(u32x2 *)out = u32x2{pair(T{}, v[0], v[1]), pair(T{}, v[2], v[3])};
}
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -__builtin_huge_valf() : (m + __builtin_log2f(l)) * 0.693147180559945309f;
}

// The largest of the four lanes of a query (l % 16), and their sum.
__device__ __forceinline__ float most_of_four(float v) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  const f32x2 b = both_halves(__builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
  return __builtin_fmaxf(b[0], b[1]);
}
__device__ __forceinline__ float sum_of_four(float v) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  const f32x2 b = both_halves(__uint_as_float(a[0]) + __uint_as_float(a[1]));
  return b[0] + b[1];
}

// What 16 NQ queries of a wave gather: lane l has queries l % 16 (+ 16).  As Wave, on
// v_mfma_f32_16x16x32, whose results leave a lane 8 keys of 32: with a few queries a tile
// half of the exponentials, and of the registers, that 32 columns take.
template <class T, int BITS, int D, int NQ>
struct Few {
  u32x4 q[NQ][D / 32];
  f32x4 o[NQ][D / 16];
  float m[NQ], l[NQ], z[NQ], lift[NQ], mul[NQ];
  int32_t pos[NQ];

  // the element of D that q's step st, part u (of 8) starts at in lane group g
  static __device__ __forceinline__ uint32_t chunk_of(int st, uint32_t g) {
    return BITS == 8 && D >= 64 ? (st / 2) * 8 + g * 2 + (st & 1) : st * 4 + g;
  }
  __device__ __forceinline__ void init(int n, const uint16_t *row, int32_t position, float c) {
    const uint32_t g = (threadIdx.x >> 4) & 3;
#pragma unroll
    for (int st = 0; st < D / 32; st++) q[n][st] = *(const u32x4 *)(row + chunk_of(st, g) * 8);
    mul[n] = c;
    if constexpr (BITS == 8 && T::kRange) {
      uint32_t top = 0;
#pragma unroll
      for (int st = 0; st < D / 32; st++) top = most_bits(q[n][st], top);
      const float most = most_of_four(from_bits(T{}, (uint16_t)joined(top)));
      mul[n] *= lift_q(q[n], most);
    }
#pragma unroll
    for (int d = 0; d < D / 16; d++) o[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    m[n] = z[n] = -__builtin_huge_valf();
    l[n] = 0.f;
    lift[n] = 64.f;
    pos[n] = position;
  }
};
// Key of a lane's register r (of 8) among 32, without the 4 * (lane / 16).
__device__ __forceinline__ constexpr int few_key(int r) { return 16 * (r / 4) + r % 4; }

// A tile of 32 rows of D values of BITS in LDS.  As Rows; values are read transposed
// in 32 (16) bytes of 16 (32) rows.
template <int BITS, int D>
struct FewRows {
  static constexpr int kBytes = D * BITS / 8, kChunks = kBytes / 16;
  static constexpr int kPer = kBytes >= 128 ? 1 : 128 / kBytes;
  static constexpr int kPlaces = kChunks < 8 ? kChunks : 8;
  static constexpr int kUnit = BITS == 16 ? 2 : 1;
  static constexpr int kUnits = kChunks / kUnit < 16 / kUnit ? kChunks / kUnit : 16 / kUnit;
  static __device__ __forceinline__ uint32_t key_swap(uint32_t r) { return (r / kPer) & (kPlaces - 1); }
  static __device__ __forceinline__ uint32_t value_swap(uint32_t r) { return ((r / kPer) & (kUnits - 1)) * kUnit; }
};

// 32 keys at position `base` in LDS: the weights p of their values.  BITS 8: ks are scales of the
// keys, vs of the values; there: bit j: key j exists.  Not MASKED: every query sees all.
template <class T, int BITS, int D, int NQ, bool MASKED>
__device__ __forceinline__ void weigh_few(Few<T, BITS, D, NQ> &w, u32x4 (&p)[NQ], const uint8_t *lk, const float *ks, const float *vs,
                                          int32_t base, uint32_t there, int32_t window) {
  typedef FewRows<BITS, D> R;
  const uint32_t lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  f32x4 s[NQ][2];
#pragma unroll
  for (int b = 0; b < 2; b++) {
#pragma unroll
    for (int n = 0; n < NQ; n++) s[n][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint8_t *row = lk + (b * 16 + l16) * R::kBytes;
    const uint32_t f = R::key_swap(b * 16 + l16);
    if constexpr (BITS == 16) {
#pragma unroll
      for (int st = 0; st < D / 32; st++) {
        const u32x4 k = *(const u32x4 *)(row + (((st * 4 + g) ^ f) * 16));
#pragma unroll
        for (int n = 0; n < NQ; n++) s[n][b] = mfma(T{}, k, w.q[n][st], s[n][b]);
      }
    } else if constexpr (D == 32) {
      const u32x4 k = widen8(F16{}, *(const u32x2 *)(row + (((g >> 1) ^ f) * 16) + (g & 1) * 8));
#pragma unroll
      for (int n = 0; n < NQ; n++) s[n][b] = mfma(F16{}, k, w.q[n][0], s[n][b]);
    } else {
#pragma unroll
      for (int st = 0; st < D / 64; st++) {
        const u32x4 k = *(const u32x4 *)(row + (((st * 4 + g) ^ f) * 16));
        const u32x4 k0 = widen8(F16{}, u32x2{k[0], k[1]}), k1 = widen8(F16{}, u32x2{k[2], k[3]});
#pragma unroll
        for (int n = 0; n < NQ; n++) {
          s[n][b] = mfma(F16{}, k0, w.q[n][2 * st], s[n][b]);
          s[n][b] = mfma(F16{}, k1, w.q[n][2 * st + 1], s[n][b]);
        }
      }
    }
  }
  f32x4 kf[2], vf[2];
  if constexpr (BITS == 8) {
#pragma unroll
    for (int b = 0; b < 2; b++) {
      kf[b] = *(const f32x4 *)(ks + b * 16 + 4 * g);
      vf[b] = *(const f32x4 *)(vs + b * 16 + 4 * g);
    }
  }
#pragma unroll
  for (int n = 0; n < NQ; n++) {
    const int32_t gap = w.pos[n] - base - 4 * (int32_t)g;
    const uint32_t mine = there >> (4 * g);
    float z[8];
#pragma unroll
    for (int r = 0; r < 8; r++) {
      z[r] = s[n][r / 4][r % 4];
      if constexpr (BITS == 8) z[r] *= kf[r / 4][r % 4];
    }
    if constexpr (MASKED) {
#pragma unroll
      for (int r = 0; r < 8; r++)
        if (!(sees(gap - few_key(r), window) && (mine >> few_key(r) & 1))) z[r] = -__builtin_huge_valf();
    }
    float top = z[0];
#pragma unroll
    for (int r = 1; r < 8; r++) top = __builtin_fmaxf(top, z[r]);
    top = most_of_four(top) * w.mul[n];
    float f[8];
    if constexpr (BITS == 8) {
      // a scale that is no number belongs to the queries that see its key alone
#pragma unroll
      for (int r = 0; r < 8; r++)
        f[r] = !MASKED || (sees(gap - few_key(r), window) && (mine >> few_key(r) & 1)) ? vf[r / 4][r % 4] : 0.f;
    }
    if constexpr (lifts(T::kRange, BITS)) {
      float largest = 0.f;
#pragma unroll
      for (int r = 0; r < 8; r++) largest = __builtin_fmaxf(largest, __builtin_fabsf(f[r]));
      w.lift[n] = value_lift(most_of_four(largest), w.lift[n]);
      w.z[n] = __builtin_fmaxf(top, w.z[n]);
      top = w.z[n] - w.lift[n];
    }
    top = __builtin_fmaxf(top, w.m[n]);
    const float ref = top == -__builtin_huge_valf() ? 0.f : top;
    if (__ballot(top > w.m[n])) {
      const float back = exp2_of(w.m[n] - ref);
      w.l[n] *= back;
#pragma unroll
      for (int d = 0; d < D / 16; d++) w.o[n][d] *= back;
      w.m[n] = top;
    }
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 8; r++) {
      z[r] = exp2_of(__builtin_fmaf(z[r], w.mul[n], -ref));
      sum += z[r];
    }
    w.l[n] += sum;
    if constexpr (BITS == 8) {
#pragma unroll
      for (int r = 0; r < 8; r++) z[r] *= f[r];
    }
#pragma unroll
    for (int i = 0; i < 4; i++) p[n][i] = pair(T{}, z[2 * i], z[2 * i + 1]);
  }
}
// Their values in LDS, times p.
template <class T, int BITS, int D, int NQ, bool MASKED>
__device__ __forceinline__ void gather_few(Few<T, BITS, D, NQ> &w, const u32x4 (&p)[NQ], const uint8_t *lv, int32_t base, uint32_t there,
                                           int32_t window) {
  typedef FewRows<BITS, D> R;
  const uint32_t lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  auto value = [&](int d) -> u32x4 {  // 32 keys in the order of p, 16 of D
    if constexpr (BITS == 16) {
      const uint32_t r = 4 * g + l16 / 4;
      const uint8_t *lo = lv + r * R::kBytes + (((d * 2 + ((l16 >> 1) & 1)) ^ R::value_swap(r)) * 16) + (l16 & 1) * 8;
      const uint8_t *hi = lv + (r + 16) * R::kBytes + (((d * 2 + ((l16 >> 1) & 1)) ^ R::value_swap(r + 16)) * 16) + (l16 & 1) * 8;
      const u32x2 a = read_turned(lo), b = read_turned(hi);
      return u32x4{a[0], a[1], b[0], b[1]};
    } else {
      const uint32_t slot = l16 / 2, r = 16 * (slot / 4) + 4 * g + slot % 4;
      const uint8_t *at = lv + r * R::kBytes + ((d ^ R::value_swap(r)) * 16) + (l16 & 1) * 8;
      return widen8(T{}, __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                             (__attribute__((address_space(3))) i32x2 *)(__attribute__((address_space(3))) void *)at)));
    }
  };
  bool odd = false;  // as in gather
  if constexpr (BITS == 16 && MASKED) {
    uint32_t most = 0;
#pragma unroll
    for (int d = 0; d < D / 16; d++) {
      most = most_bits(value(d), most);
      __builtin_amdgcn_sched_barrier(0);
    }
    odd = __ballot(joined(most) > finite_bits(T{})) != 0;
  }
#pragma unroll
  for (int d = 0; d < D / 16; d++) {
    u32x4 v = value(d);
    if (odd) v = finite_part(T{}, v);
#pragma unroll
    for (int n = 0; n < NQ; n++) w.o[n][d] = mfma(T{}, v, p[n], w.o[n][d]);
  }
  if (odd) {
#pragma unroll 1
    for (uint32_t e = 0; e < 32; e++) {
      const uint32_t group = e >> 3, word = (e & 7) >> 1, at = 16 * ((e & 7) / 4) + 4 * group + (e & 3);
      const uint32_t bits = g == group ? ((e & 1) ? 0xFFFF0000u : 0xFFFFu) : 0u;
      const u32x4 only = {word == 0 ? bits : 0u, word == 1 ? bits : 0u, word == 2 ? bits : 0u, word == 3 ? bits : 0u};
#pragma unroll
      for (int d = 0; d < D / 16; d++) {
        const u32x4 v = value(d), rest = (v ^ finite_part(T{}, v)) & only;
#pragma unroll
        for (int n = 0; n < NQ; n++) {
          const bool seen = sees(w.pos[n] - base - (int32_t)at, window) && (there >> at & 1);
          const f32x4 t = mfma(T{}, rest, p[n] & only, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int r = 0; r < 4; r++) w.o[n][d][r] += seen ? t[r] : 0.f;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

constexpr uint32_t kListed = 512;  // sequences
constexpr int kFewCost = 12;
// Sums of the lanes up to each: within rows of 16, then rows before, then halves.
__device__ __forceinline__ uint32_t sums_of_wave(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 15, 15, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 15, 15, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 15, 15, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 15, 15, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 10, 15, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 12, 15, false);
  return v;
}
// a / b, mostly of small numbers.
__device__ __forceinline__ int64_t ratio(int64_t a, uint32_t b) { return a >> 32 ? a / b : (int64_t)((uint32_t)a / b); }

template <class T, int BITS, int D, int NQ, int W>
__global__ __launch_bounds__(64 * W, BITS == 8 && D < 256 ? 2 : 1) void attend_few(const Pages c, const Sequences b, const Attend a) {
  typedef FewRows<BITS, D> R;
  constexpr int kTile = 32 * R::kBytes, kLoads = kTile / 1024, kRowsPer = 32 / kLoads, kRows = 16 * NQ;
  extern __shared__ __align__(1024) uint8_t lds[];  // [W][2][keys, values], then joined
  __shared__ float scales[W][2][64], ms[W][kRows], ls[W][kRows];
  __shared__ int64_t before[kListed + 1];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t *buf = lds + wave * (4 * kTile);
  // The work is the tiles of all sequences, head by head, in one row: each workgroup has an
  // equal run of it, which ends in one sequence and goes on in the next, so parts are
  // as long as they can be and all workgroups end together.  A head's keys count for kFewCost
  // tiles more than they are, what beginning and ending them takes; they are split where
  // a run ends.  (More than kListed sequences are not split: a piece for each of their heads.)
  const bool listed = a.few_splits > 1;
  auto tiles_of = [&](uint32_t s) -> uint32_t {
    const Span sp = span_of(b, s);
    const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
    if (rows == 0 || (!a.alone && rows > a.cap)) return 0;
    const uint32_t count = rows < a.cap ? rows : a.cap;
    const Cuts k = cuts_of(c, b, sp.first + sp.ahead, sp.first + (int32_t)((count - 1) / a.group) + sp.ahead, sp.length, a.window, kFewShift, 1, 1);
    return (k.end > k.begin ? (uint32_t)(k.end - k.begin) : 1) + kFewCost;  // (rows that see nothing are cleared)
  };
  int64_t run = 1, end = (int64_t)b.count * c.heads;  // of places
  if (listed) {
    // places 1 .. count: tiles up to and with a sequence's
    int64_t so_far = 0;
    for (uint32_t s0 = 0; s0 < b.count; s0 += 64) {
      if (wave != 0) break;
      // (64 times 2^25 tiles of a sequence fit)
      const uint32_t n = sums_of_wave(s0 + lane < b.count ? tiles_of(s0 + lane) : 0);
      if (s0 + lane < b.count) before[s0 + lane + 1] = so_far + n;
      so_far += (uint32_t)__builtin_amdgcn_readlane(n, 63);
    }
    if (threadIdx.x == 0) before[0] = 0;
    __syncthreads();
    end = before[b.count] * c.heads;
    run = ratio(end + gridDim.x - 1, gridDim.x);
    run = run < kFewLeast ? kFewLeast : run;
  }
  if (blockIdx.x < c.heads) {
    // rows of no sequence
    const int32_t begin = span_of(b, 0).first, end = span_of(b, b.count - 1).last;
    const uint32_t per = a.group * (D / 8), head = blockIdx.x;
    const uint64_t all = ((uint64_t)begin + (b.tokens - end)) * per;
    for (uint64_t i = threadIdx.x; i < all; i += 64 * W) {
      const uint64_t t = i / per < (uint64_t)begin ? i / per : i / per - begin + end, e = i % per;
      ((u32x4 *)(a.out + (t * a.heads + head * a.group) * D))[e] = u32x4{0, 0, 0, 0};
      if (a.lse && e < a.group) a.lse[t * a.heads + head * a.group + e] = -__builtin_huge_valf();
    }
  }
  const int64_t last_place = listed ? (blockIdx.x + 1) * run < end ? (blockIdx.x + 1) * run : end : end;
  for (int64_t place = blockIdx.x * run, taken = 0; place < last_place; place += listed ? taken : gridDim.x) {
    uint32_t s, head, tile = 0, all_tiles = 0;
    if (listed) {
      s = same(starts_up_to(before, b.count + 1, ratio(place, c.heads)) - 1);
      const uint32_t places = same((uint32_t)(before[s + 1] - before[s]));
      const int64_t in = place - before[s] * c.heads;
      head = same((uint32_t)ratio(in, places));
      tile = same((uint32_t)(in - (int64_t)head * places));
      all_tiles = places - kFewCost;
      taken = places - tile < last_place - place ? places - tile : last_place - place;
      if (tile >= all_tiles) continue;
    } else {
      s = same((uint32_t)(place / c.heads));
      head = same((uint32_t)(place % c.heads));
    }
    const Span sp = span_of(b, s);
    const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
    if (rows == 0 || (!a.alone && rows > a.cap)) continue;
    // whether this is all of the head's keys; its parts lie in workgroups' order
    const bool direct = !listed || (tile == 0 && taken >= all_tiles);
    const uint64_t slot = blockIdx.x + (uint64_t)s * c.heads + head;
    if (listed && tile == 0 && threadIdx.x == 0) {
      // (of those after the first, runs of `run` tiles each)
      a.few_parts[((uint64_t)s * c.heads + head) * 2] = direct ? 1 : (uint32_t)((all_tiles - taken + run - 1) / run) + 1;
      a.few_parts[((uint64_t)s * c.heads + head) * 2 + 1] = (uint32_t)slot;
    }
    const int32_t *table = b.tables + s * b.stride;
    for (uint32_t r0 = 0; r0 < rows; r0 += r0 ? kRows : a.cap) {
      if (r0 && tile) break;  // rows behind the capacity are not split
      const uint32_t most = r0 ? kRows : a.cap, count = rows - r0 < most ? rows - r0 : most;
      const int32_t first = sp.first + (int32_t)(r0 / a.group), last = sp.first + (int32_t)((r0 + count - 1) / a.group);
      const Cuts k = cuts_of(c, b, first + sp.ahead, last + sp.ahead, sp.length, a.window, kFewShift, 1, 1);
      const int32_t t0 = k.begin + (r0 ? 0 : (int32_t)tile), t1 = listed && !r0 && t0 + taken < k.end ? t0 + (int32_t)taken : k.end;
      // Pages (16 keys lie in one) come a tile ahead, by scalar loads; all other loads go to
      // LDS, so that the counts waited for below are those of the rows in flight.  A tile's
      // keys are asked for as soon as those of two tiles before have been multiplied, its
      // values likewise: up to two tiles are in flight with two buffers.
      constexpr int kWait = kLoads + (BITS == 8);  // loads of a tile's keys and scales
      struct Table { int32_t of[2]; } page = {}, page_then = {};
      uint32_t there = 0, next = 0, then = 0;  // the keys that exist: of tile t, t + W, t + 2 W
      const auto *entries = (const __attribute__((address_space(4))) int32_t *)table;
      auto look = [&](int32_t t) {
        if (t >= t1) return;
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const int32_t pos = t * 32 + 16 * j;
          page.of[j] = entries[(uint32_t)(pos < k.stop ? pos : k.stop - 1) >> c.shift];
        }
      };
      auto known = [&](int32_t t) {
        const uint32_t all = ((uint32_t)page.of[0] < c.pages ? 0xFFFFu : 0u) | ((uint32_t)page.of[1] < c.pages ? 0xFFFF0000u : 0u);
        const int32_t left = k.stop - t * 32;
        return left < 32 ? all & ((1u << left) - 1) : all;
      };
      const uint32_t in_load = lane / R::kChunks, chunk = lane % R::kChunks;
      const uint32_t head_bytes = (uint32_t)R::kBytes << c.shift, page_bytes = head_bytes * c.heads, row_mask = (1u << c.shift) - 1;
      const uint32_t at_lds = lds_address(buf);
      auto bring = [&](const uint8_t *pool, int32_t t, const Table &pages, uint32_t all, bool values, uint32_t dst) {
        const uint8_t *mine = pool + (uint64_t)head * head_bytes;
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
          const uint32_t row = i * kRowsPer + in_load, swap = values ? R::value_swap(row) : R::key_swap(row);
          const uint32_t off = in_load * R::kBytes + (chunk ^ swap) * 16;
          if (all == 0xFFFFFFFFu && kRowsPer <= 16) {  // (rows of a load lie in one page)
            ask(mine + ((uint64_t)(uint32_t)pages.of[i * kRowsPer / 16] * page_bytes + (((uint32_t)(t * 32) + i * kRowsPer) & row_mask) * R::kBytes),
                off, dst + i * 1024);
          } else {
            const uint8_t *src = mine + ((uint64_t)(uint32_t)(row < 16 ? pages.of[0] : pages.of[1]) * page_bytes +
                                         (((uint32_t)(t * 32) + row) & row_mask) * R::kBytes + (chunk ^ swap) * 16);
            ask(all >> row & 1 ? src : (const uint8_t *)&g_zero16, dst + i * 1024);
          }
        }
      };
      auto request_keys = [&](int32_t t) -> uint32_t {  // and scales
        if (t >= t1) return 0;
        const uint32_t all = known(t), odd = ((t - t0) / W) & 1;
        bring(c.k, t, page, all, false, at_lds + odd * (2 * kTile));
        if constexpr (BITS == 8) {
          const uint32_t row = lane & 31;
          const uint64_t at = (((uint64_t)(uint32_t)(row < 16 ? page.of[0] : page.of[1]) * c.heads + head) << c.shift) + (((uint32_t)(t * 32) + row) & row_mask);
          ask_word(all >> row & 1 ? (const uint8_t *)((lane < 32 ? c.k_scales : c.v_scales) + at) : (const uint8_t *)&g_zero16,
                   lds_address(scales[wave][odd]));
        }
        page_then = page;
        look(t + W);
        return all;
      };
      auto request_values = [&](int32_t t, uint32_t all) {
        if (t < t1) bring(c.v, t, page_then, all, true, at_lds + (((t - t0) / W) & 1) * (2 * kTile) + kTile);
      };
      const int32_t mine0 = t0 + (int32_t)wave;
      look(mine0);
      Few<T, BITS, D, NQ> w;
      there = request_keys(mine0);
      request_values(mine0, there);
#pragma unroll
      for (int n = 0; n < NQ; n++) {
        const uint32_t r = n * 16 + (lane & 15), mine = r0 + (r < count ? r : count - 1);
        const int32_t token = sp.first + (int32_t)(mine / a.group);
        w.init(n, a.q + token * a.q_token + (head * a.group + mine % a.group) * a.q_head, token + sp.ahead, a.c);
      }
      next = request_keys(mine0 + W);
      request_values(mine0 + W, next);
      for (int32_t t = mine0; t < t1; t += W) {
        const uint32_t odd = ((t - t0) / W) & 1;
        const bool whole = there == 0xFFFFFFFFu && t * 32 + 31 <= first + sp.ahead && last + sp.ahead - t * 32 < a.window;
        const uint8_t *p = buf + odd * (2 * kTile);
        u32x4 weights[NQ];
        // behind the keys of t: its values, and all of t + W
        if (t + W < t1) wait_but<kLoads + kWait + kLoads>();
        else wait_but<kLoads>();
        if (whole) {
          weigh_few<T, BITS, D, NQ, false>(w, weights, p, scales[wave][odd], scales[wave][odd] + 32, t * 32, there, a.window);
        } else {
          weigh_few<T, BITS, D, NQ, true>(w, weights, p, scales[wave][odd], scales[wave][odd] + 32, t * 32, there, a.window);
        }
        wait_reads();  // their place is asked for again
        then = request_keys(t + 2 * W);
        // behind the values of t: all of t + W, the keys of t + 2 W
        if (t + 2 * W < t1) wait_but<kWait + kLoads + kWait>();
        else if (t + W < t1) wait_but<kWait + kLoads>();
        else wait_but<0>();
        if (whole) {
          gather_few<T, BITS, D, NQ, false>(w, weights, p + kTile, t * 32, there, a.window);
        } else {
          gather_few<T, BITS, D, NQ, true>(w, weights, p + kTile, t * 32, there, a.window);
        }
        wait_reads();
        request_values(t + 2 * W, then);
        there = next;
        next = then;
      }
      // the waves' sums: [W][16 NQ][D] in place of the tiles, 16-byte chunks exchanged
      __syncthreads();
      float *part = (float *)lds;
#pragma unroll
      for (int n = 0; n < NQ; n++) {
        const uint32_t r = n * 16 + (lane & 15);
        const float sum = sum_of_four(w.l[n]);
        if (r < count) {
#pragma unroll
          for (int d = 0; d < D / 16; d++) {
            const uint32_t chunk = d * 4 + (lane >> 4);
            *(f32x4 *)(part + (wave * kRows + r) * D + ((chunk ^ (lane & 7)) * 4)) = w.o[n][d];
          }
          ms[wave][r] = w.m[n];
          ls[wave][r] = sum;
        }
      }
      __syncthreads();
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
          v += *(const f32x4 *)(part + (q * kRows + r) * D + ((chunk ^ (r & 7)) * 4)) * f;
          l += ls[q][r] * f;
        }
        const uint32_t row = r0 + r;
        const uint64_t to = (uint64_t)(sp.first + row / a.group) * a.heads + head * a.group + row % a.group;
        if (direct || r0) {
          store4(a.out + to * D + chunk * 4, T{}, l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : v * (1.f / l));
          if (a.lse && chunk == 0) a.lse[to] = lse_of(m, l);
        } else {
          const uint64_t at = slot * a.cap + row;
          *(f32x4 *)(a.few_o + at * D + chunk * 4) = v;
          if (chunk == 0) *(f32x2 *)(a.few_ml + at * 2) = f32x2{m, l};
        }
      }
      __syncthreads();
    }
  }
}

// The parts of a row of few, a workgroup (block of blocks) to a row (sequence, key head, row): D / 4 lanes
// hold it, and 1024 / D groups of them take the parts in turn, so that all are read at
// once (2000 positions for a token in 16 parts: 3 us against 10 with one after the other).
template <class T, int D>
__device__ __forceinline__ void join_few(const Pages &c, const Sequences &b, const Attend &a, uint32_t block,
                                         uint32_t blocks) {
  constexpr uint32_t kLanes = D / 4, kGroups = 256 / kLanes;
  __shared__ f32x4 vs[256];
  __shared__ float ms[kGroups], ls[kGroups];
  const uint32_t chunk = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const uint64_t all = (uint64_t)b.count * c.heads * a.cap;
  for (uint64_t row = block; row < all; row += blocks) {
    const uint32_t r = (uint32_t)(row % a.cap), head = (uint32_t)(row / a.cap % c.heads), s = (uint32_t)(row / a.cap / c.heads);
    const Span sp = span_of(b, s);
    const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
    if (r >= rows || (!a.alone && rows > a.cap)) continue;
    const uint32_t *which = a.few_parts + ((uint64_t)s * c.heads + head) * 2;
    const int32_t parts = (int32_t)which[0];
    if (parts <= 1) continue;
    const uint64_t first = (uint64_t)which[1] * a.cap + r;  // the parts' rows lie cap apart
    float m = -__builtin_huge_valf();
#pragma unroll 4
    for (int32_t p = group; p < parts; p += kGroups) m = __builtin_fmaxf(m, a.few_ml[(first + (uint64_t)p * a.cap) * 2]);
    float ref = m == -__builtin_huge_valf() ? 0.f : m, l = 0.f;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int32_t p = group; p < parts; p += kGroups) {
      const f32x2 t = *(const f32x2 *)(a.few_ml + (first + (uint64_t)p * a.cap) * 2);
      const float f = exp2_of(t[0] - ref);
      v += *(const f32x4 *)(a.few_o + (first + (uint64_t)p * a.cap) * D + chunk * 4) * f;
      l += t[1] * f;
    }
    vs[threadIdx.x] = v;
    if (chunk == 0) {
      ms[group] = m;
      ls[group] = l;
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (uint32_t q = 1; q < kGroups; q++) m = __builtin_fmaxf(m, ms[q]);
      ref = m == -__builtin_huge_valf() ? 0.f : m;
      v = f32x4{0.f, 0.f, 0.f, 0.f};
      l = 0.f;
#pragma unroll
      for (uint32_t q = 0; q < kGroups; q++) {
        const float f = exp2_of(ms[q] - ref);
        v += vs[q * kLanes + chunk] * f;
        l += ls[q] * f;
      }
      const uint64_t to = (uint64_t)(sp.first + r / a.group) * a.heads + head * a.group + r % a.group;
      store4(a.out + to * D + chunk * 4, T{}, l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : v * (1.f / l));
      if (a.lse && chunk == 0) a.lse[to] = lse_of(m, l);
    }
    __syncthreads();
  }
}

// Tile i of ROWS rows lies in sequence s, whose tiles begin at starts[s] * group / ROWS
// (rounded down) + s: no two sequences' overlap, and what lies between them is empty.
template <uint32_t ROWS>
__device__ __forceinline__ int64_t first_tile(const Sequences &b, uint32_t s, uint32_t group) {
  const int32_t at = b.starts[s];
  return (int64_t)((uint64_t)(at < 0 ? 0 : at) * group / ROWS) + s;
}
template <uint32_t ROWS>
__device__ __forceinline__ uint32_t tile_owner(const Sequences &b, uint32_t group, int64_t tile) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0, n = b.count;  // as starts_up_to
  while (n) {
    const uint32_t step = (n + 63) / 64;
    const bool in = lane * step < n && first_tile<ROWS>(b, lo + lane * step, group) <= tile;
    const uint32_t k = __popcll(__ballot(in));
    if (k == 0) break;
    const uint32_t before = lo + n;
    lo = lo + (k - 1) * step + 1;
    n = lo + step - 1 < before ? step - 1 : before - lo;
  }
  return lo ? lo - 1 : b.count;
}

// Tiles of keys in LDS.  With three a step of 16 bits meets once: the tile that is asked for is none
// that is read; two leave room for the scales of 8 bits beside two workgroups' tiles.
constexpr uint32_t key_buffers(int bits) { return bits == 16 ? 3 : 2; }
template <class T, int BITS, int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attend_tile(const Pages c, const Sequences b, const Attend a) {
  typedef Rows<D> R;
  typedef typename KeyType<T, BITS>::type K;
  constexpr int kTile = 64 * R::kBytes, kLoads = kTile / 1024 / NW, kRowsPer = 1024 / R::kBytes;
  constexpr uint32_t kRows = 32 * NW;
  constexpr int kRaw = D / 16 <= NW ? 1 : D / 16 / NW;  // 16 bytes of codes a thread
  constexpr uint32_t kKeys = key_buffers(BITS);
  extern __shared__ __align__(1024) uint8_t lds[];  // keys [kKeys], values [2]
  __shared__ float scales[3][128];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t units = (uint64_t)a.tiles * c.heads * a.tile_splits;
  for (uint64_t id = blockIdx.x; id < units; id += gridDim.x) {
    // the last tiles of a prompt see the most keys: they go first
    const uint32_t head = (uint32_t)(id % c.heads), z = (uint32_t)(id / c.heads % a.tile_splits);
    const int64_t tile = (int64_t)a.tiles - 1 - (int64_t)(id / c.heads / a.tile_splits);
    const uint32_t s = tile_owner<kRows>(b, a.group, tile);
    if (s >= b.count) continue;
    const Span sp = span_of(b, s);
    const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
    const int64_t r0 = (tile - first_tile<kRows>(b, s, a.group)) * kRows;
    if (rows <= a.cap || r0 < 0 || r0 >= (int64_t)rows) continue;  // (before: starts that fall)
    const uint32_t count = rows - (uint32_t)r0 < kRows ? rows - (uint32_t)r0 : kRows;
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
    w.init(a.q + token * a.q_token + (head * a.group + mine % a.group) * a.q_head, token + sp.ahead, a.c);
    // Keys come ahead of values, and pages (16 keys lie in one) a tile ahead of keys, by
    // scalar loads: a wait for those is no wait for rows in flight.
    struct Table { int32_t of[4]; } page = {}, page_before = {};
    uint64_t before = 0, there[4] = {0, 0, 0, 0};  // the keys that exist: of page_before's tile; of t, t + 1, ..
    const auto *entries = (const __attribute__((address_space(4))) int32_t *)table;
    const bool one = c.shift >= 6;  // page of a tile
    auto look = [&](int32_t t) {
      if (t >= t1) return;
      if (one) {
        page.of[0] = entries[(uint32_t)(t * 64) >> c.shift];
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const int32_t pos = t * 64 + 16 * j;
          page.of[j] = entries[(uint32_t)(pos < k.stop ? pos : k.stop - 1) >> c.shift];
        }
      }
    };
    auto known = [&](int32_t t) {
      uint64_t all = (uint32_t)page.of[0] < c.pages ? ~0ull : 0;
      if (!one) {
        all &= 0xFFFF;
#pragma unroll
        for (int j = 1; j < 4; j++)
          if ((uint32_t)page.of[j] < c.pages) all |= 0xFFFFull << (16 * j);
      }
      const int32_t left = k.stop - t * 64;
      return left < 64 ? all & ((1ull << left) - 1) : all;
    };
    // this head's part of a page, and where it begins
    const uint32_t head_bytes = (uint32_t)R::kBytes << c.shift, page_bytes = head_bytes * c.heads, row_mask = (1u << c.shift) - 1;
    auto page_of = [&](const Table &t, uint32_t j) { return (uint32_t)(one || j == 0 ? t.of[0] : j == 1 ? t.of[1] : j == 2 ? t.of[2] : t.of[3]); };
    u32x4 raw_k[kRaw], raw_v[kRaw];
    float scale = 0.f;
    // rows of a load lie in one page; the exchange is the same in all of a wave's loads
    const uint32_t in_load = lane / R::kChunks, chunk = lane % R::kChunks;
    static_assert(kLoads >= 1 && NW * kRowsPer % (R::kKeyPlaces * R::kKeyPer) == 0 &&
                      NW * kRowsPer % (R::kUnits * R::kPer) == 0,
                  "the exchange is the same in all of a wave's loads");
    auto bring = [&](const uint8_t *pool, int32_t t, const Table &pages, uint64_t all, uint32_t swap, uint32_t dst) {
      const uint32_t off = in_load * R::kBytes + (chunk ^ swap) * 16;
      const uint8_t *mine = pool + (uint64_t)head * head_bytes;
      if (one && all == ~0ull) {
        const uint8_t *src = mine + ((uint64_t)(uint32_t)pages.of[0] * page_bytes + (((uint32_t)(t * 64) & row_mask) + wave * kRowsPer) * R::kBytes);
#pragma unroll
        for (int i = 0; i < kLoads; i++) ask(src + i * NW * 1024, off, dst + (i * NW + wave) * 1024);
        return;
      }
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const uint32_t r = (i * NW + wave) * kRowsPer;
        const uint32_t pg = page_of(pages, NW * kRowsPer <= 16 ? i * NW * kRowsPer / 16 : r / 16);
        const uint8_t *src = mine + ((uint64_t)pg * page_bytes + (((uint32_t)(t * 64) + r) & row_mask) * R::kBytes);
        if (all == ~0ull) {
          ask(src, off, dst + (i * NW + wave) * 1024);
        } else {
          ask(all >> (r + in_load) & 1 ? src + off : (const uint8_t *)&g_zero16, dst + (i * NW + wave) * 1024);
        }
      }
    };
    auto fetch = [&](const uint8_t *pool, int32_t t, const Table &pages, uint64_t all, u32x4 (&raw)[kRaw]) {
#pragma unroll
      for (int i = 0; i < kRaw; i++) {
        const uint32_t at16 = i * 64 * NW + threadIdx.x, row = at16 / (D / 16) & 63;
        const uint64_t r = pool_row(c, page_of(pages, row / 16), head, (uint32_t)(t * 64) + row);
        raw[i] = u32x4{0, 0, 0, 0};
        if ((all >> row & 1) && at16 < 64 * (D / 16)) raw[i] = *(const u32x4 *)(pool + r * D + (at16 % (D / 16)) * 16);
      }
    };
    const uint32_t mine_row = wave * kRowsPer + in_load;
    // keys of tile t (and scales); returns those that exist
    auto request_keys = [&](int32_t t, u32x4 (&raw)[kRaw]) -> uint64_t {
      if (t >= t1) return 0;
      const uint64_t all = known(t);
      if constexpr (BITS == 16) {
        bring(c.k, t, page, all, R::key_swap(mine_row), lds_address(lds) + (uint32_t)(t - t0) % kKeys * kTile);
      } else {
        fetch(c.k, t, page, all, raw);
        scale = 0.f;
        if (wave < 2 && (all >> lane & 1))
          scale = (wave ? c.v_scales : c.k_scales)[pool_row(c, page_of(page, lane / 16), head, (uint32_t)(t * 64) + lane)];
      }
      page_before = page;
      before = all;
      look(t + 1);
      return all;
    };
    // values of tile t, whose keys were asked for last
    auto request_values = [&](int32_t t, u32x4 (&raw)[kRaw]) {
      if (t >= t1) return;
      if constexpr (BITS == 16) {
        bring(c.v, t, page_before, before, R::value_swap(mine_row), lds_address(lds) + (kKeys + ((t - t0) & 1)) * kTile);
      } else {
        fetch(c.v, t, page_before, before, raw);
      }
    };
    // codes of 8 bits become 16-bit values on their way to LDS, once for all waves
    auto spread = [&](int32_t t, const u32x4 (&raw)[kRaw], float f, bool values) {
      if (t >= t1) return;
      uint8_t *dst = lds + ((values ? kKeys : 0) + ((t - t0) & 1)) * kTile;
#pragma unroll
      for (int i = 0; i < kRaw; i++) {
        const uint32_t at16 = i * 64 * NW + threadIdx.x, row = at16 / (D / 16), chunk = at16 % (D / 16) * 2;
        if (at16 >= 64 * (D / 16)) break;
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const u32x2 codes = {raw[i][2 * e], raw[i][2 * e + 1]};
          const uint32_t to = row * R::kBytes + (((chunk + e) ^ (values ? R::value_swap(row) : R::key_swap(row))) * 16);
          *(u32x4 *)(dst + to) = values ? widen8(T{}, codes) : widen8(K{}, codes);
        }
      }
      if (!values && wave < 2) scales[(t - t0) % 3][wave * 64 + lane] = wave ? f : f * a.c;
    };
    f32x16 s0, s1;  // settled scores of the first, second 32 keys of a tile
    if (t0 < t1) {
      look(t0);
      there[0] = request_keys(t0, raw_k);
      if constexpr (BITS == 16) {
        request_values(t0, raw_v);
        there[1] = request_keys(t0 + 1, raw_k);
        wait_but<0>();
      } else {
        // (all loads of the first two tiles at once)
        u32x4 raw_k1[kRaw], raw_v0[kRaw];
        const float scale0 = scale;
        request_values(t0, raw_v0);
        there[1] = request_keys(t0 + 1, raw_k1);
        const float scale1 = scale;
        request_values(t0 + 1, raw_v);
        spread(t0, raw_k, scale0, false);
        spread(t0, raw_v0, 0.f, true);
        there[2] = request_keys(t0 + 2, raw_k);
        spread(t0 + 1, raw_k1, scale1, false);
      }
      __syncthreads();
      s0 = scores(w, lds_address(lds));
      const Seen seen(w, t0 * 64, (uint32_t)there[0], a.window);
      refer(w, settle<T, BITS, D, true>(w, s0, scales[0], scales[0] + 64, seen));
    }
    // Tile t, whose s0 is settled; leaves that of tile t + 1.  Each half has the scores of
    // the next 32 keys beside the exponentials of these, on either unit of the SIMD.
    auto step = [&](int32_t t, auto masked) {
      constexpr bool M = decltype(masked)::value;
      const uint32_t at = (uint32_t)(t - t0), base = lds_address(lds);
      const bool more = !M || t + 1 < t1;
      const float *now = scales[at % 3], *then = scales[(at + 1) % 3];
      const uint32_t lk = base + at % kKeys * kTile, next = base + (at + 1) % kKeys * kTile, lv = base + (kKeys + (at & 1)) * kTile;
      const Seen seen0(w, t * 64, (uint32_t)there[0], a.window), seen1(w, t * 64 + 32, (uint32_t)(there[0] >> 32), a.window),
          seen2(w, t * 64 + 64, (uint32_t)there[1], a.window);
      u32x4 p[2];
      // values of t are there (16 bits: and keys of t + 1), those of t - 1 read by all
      if constexpr (BITS == 16) {
        wait_but<0>();
        meet();
        request_values(t + 1, raw_v);
        there[2] = request_keys(t + 2, raw_k);
      } else {
        __syncthreads();
        spread(t + 1, raw_v, 0.f, true);
        request_values(t + 2, raw_v);
      }
      if constexpr (M) {
        s1 = scores(w, lk + 32 * R::kBytes);
        weigh<T, BITS, D, M>(w, s0, p, now + 64, seen0);
        gather<T, BITS, D, M>(w, p, lv, t * 64, (uint32_t)there[0], a.window);
        refer(w, settle<T, BITS, D, M>(w, s1, now + 32, now + 96, seen1));
      } else {
        refer(w, half_step(w, s0, s1, lk + 32 * R::kBytes, lv, now + 64, now + 32, now + 96));
      }
      if constexpr (BITS == 8) {
        // keys of t + 1 are there, those of t read by all
        __syncthreads();
        spread(t + 2, raw_k, scale, false);
        there[3] = request_keys(t + 3, raw_k);
      }
      if constexpr (M) {
        if (more) s0 = scores(w, next);
        weigh<T, BITS, D, M>(w, s1, p, now + 96, seen1);
        gather<T, BITS, D, M>(w, p, lv + 32 * R::kBytes, t * 64 + 32, (uint32_t)(there[0] >> 32), a.window);
        if (more) refer(w, settle<T, BITS, D, M>(w, s0, then, then + 64, seen2));
      } else {
        refer(w, half_step(w, s1, s0, next, lv + 32 * R::kBytes, now + 96, then, then + 64));
      }
      there[0] = there[1];
      there[1] = there[2];
      there[2] = there[3];
    };
    // tiles of which every row of this wave sees every key (from h0 on, before h1), like the next
    // one's, go by themselves
    const int32_t h0 = wlast < a.window ? 0 : ((wlast - a.window) >> 6) + 1, h1 = wfirst + 1 < t1 * 64 ? (wfirst + 1) >> 6 : t1;
    for (int32_t t = t0; t < t1; t++) {
      for (; t >= h0 && t + 1 < h1 && (there[0] & there[1]) == ~0ull; t++) step(t, std::false_type{});
      step(t, std::true_type{});
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

// The parts of a row of tiles (token, head) added up, D / 4 lanes to a row.
template <class T, int D>
__device__ __forceinline__ void join_tiles(const Pages &c, const Sequences &b, const Attend &a, uint32_t block,
                                           uint32_t blocks) {
  constexpr uint32_t kLanes = D / 4;
  const uint32_t chunk = threadIdx.x % kLanes;
  // a wave's rows go together: the search below is the whole wave's
  const uint64_t rows_all = (uint64_t)b.tokens * a.heads, all = rows_all * kLanes;
  for (uint64_t i = (uint64_t)block * 256 + threadIdx.x; i - (threadIdx.x & 63) < all; i += (uint64_t)blocks * 256) {
    const bool in = i < all;
    const uint64_t row = (in ? i : all - 1) / kLanes;
    const int32_t t = (int32_t)(row / a.heads);
    const int32_t t0 = __builtin_amdgcn_readfirstlane(t);
    const uint32_t up_to = starts_up_to(b.starts, b.count + 1, t0);  // 0: before the first
    uint32_t owner = up_to ? up_to - 1 : 0;
    Span sp = {0, 0, 0, 0};
    if (owner < b.count) {
      sp = span_of(b, owner);
      // a wave holds at most 8 rows: walk on to this one's sequence
      while (t >= sp.last && owner + 1 < b.count) sp = span_of(b, ++owner);
    }
    const uint32_t rows = (uint32_t)(sp.last - sp.first) * a.group;
    int32_t parts = 0;
    if (in && t >= sp.first && t < sp.last && rows > a.cap) {
      const uint32_t r = (uint32_t)(t - sp.first) * a.group + (uint32_t)(row % a.heads) % a.group, r0 = r & ~(a.tile_rows - 1);
      const uint32_t count = rows - r0 < a.tile_rows ? rows - r0 : a.tile_rows;
      parts = cuts_of(c, b, sp.first + (int32_t)(r0 / a.group) + sp.ahead, sp.first + (int32_t)((r0 + count - 1) / a.group) + sp.ahead,
                      sp.length, a.window, kTileShift, a.tile_splits, kTileLeast).count;
    }
    if (parts <= 1) continue;
    float m = -__builtin_huge_valf();
#pragma unroll 4
    for (int32_t p = 0; p < parts; p++) m = __builtin_fmaxf(m, a.tile_ml[(p * rows_all + row) * 2]);
    const float ref = m == -__builtin_huge_valf() ? 0.f : m;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll 4
    for (int32_t p = 0; p < parts; p++) {
      const f32x2 ml = *(const f32x2 *)(a.tile_ml + (p * rows_all + row) * 2);
      const float f = exp2_of(ml[0] - ref);
      v += *(const f32x4 *)(a.tile_o + (p * rows_all + row) * D + chunk * 4) * f;
      l += ml[1] * f;
    }
    store4(a.out + row * D + chunk * 4, T{}, l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : v * (1.f / l));
    if (a.lse && chunk == 0) a.lse[row] = lse_of(m, l);
  }
}

// All that splits leave, in one launch: the first few_blocks workgroups join rows of few, the
// others those of tiles (19 sequences of both, FP16 in 8 bits: 43.6 us, two launches 46.8).
template <class T, int D>
__global__ __launch_bounds__(256) void join(const Pages c, const Sequences b, const Attend a, uint32_t few_blocks) {
  if (blockIdx.x < few_blocks) {
    join_few<T, D>(c, b, a, blockIdx.x, few_blocks);
  } else {
    join_tiles<T, D>(c, b, a, blockIdx.x - few_blocks, gridDim.x - few_blocks);
  }
}

// ------------------------------------------------------------------- host
// What a call launches, by what the host knows: rows and table widths, not lengths.
struct Plan {
  Attend a;
  bool tile;
  uint64_t few_o, few_ml, few_parts, tile_o, tile_ml, all;  // workspace offsets
};
constexpr uint64_t kMostParts = 256u << 20;  // bytes of partial sums of tiles
constexpr uint32_t kMostResident = 2048;     // workgroups of attend_few

Plan plan_of(const df_cache *cache, const df_cache_batch *batch, uint64_t tokens, uint32_t heads, int64_t window) {
  Plan p = {};
  Attend &a = p.a;
  const uint64_t kv = cache->kv_heads, seqs = batch->seqs, dim = cache->head_dim;
  a.heads = heads;
  a.group = heads / cache->kv_heads;
  a.window = window <= 0 || window > INT32_MAX ? INT32_MAX : (int32_t)window;
  const uint64_t hint = batch->max_new && batch->max_new < tokens ? batch->max_new : tokens;
  // heads of 256: two blocks of 16 rows do not fit a wave's registers
  const uint64_t rows = dim == 256 ? 16 : 32, fit = rows / a.group;
  p.tile = hint * a.group > rows;
  a.alone = !p.tile;
  a.cap = (uint32_t)((hint < fit ? hint : fit) * a.group);
  a.few_splits = a.tile_splits = 1;
  // the most keys that a sequence's rows may see
  const uint64_t held = (uint64_t)batch->width * cache->page_size;
  const uint64_t seen = held < (uint64_t)a.window + hint ? held : (uint64_t)a.window + hint;
  // few rows are split where there is a table of their sequences, and keys for two parts
  if (a.cap && seqs <= kListed && (seen + 31) / 32 + 1 > kFewLeast) a.few_splits = 2;
  if (p.tile) {
    // 256 rows to a tile where those fill the chip: half of the reads of keys and values
    const uint64_t all = tokens * a.group;
    a.tile_rows = (dim == 64 || dim == 128) && (all + 255) / 256 * kv >= 256 ? 256 : 128;
    a.tiles = (uint32_t)(all / a.tile_rows + seqs);
    const uint64_t units = (all + a.tile_rows - 1) / a.tile_rows * kv, most = (seen + 63) / 64 + 1;
    uint64_t n = units >= 512 ? 1 : 512 / units;
    if (n > most / kTileLeast) n = most / kTileLeast;
    const uint64_t part = tokens * heads * (dim + 2) * 4;
    if (n * part > kMostParts) n = kMostParts / part;
    if (n > 16) n = 16;
    a.tile_splits = n < 1 ? 1 : (uint32_t)n;
  }
  uint64_t at = 0;
  if (a.few_splits > 1) {
    // every run's end makes a part more
    const uint64_t rows = (kMostResident + seqs * kv) * a.cap;
    p.few_o = at;
    at += up(rows * dim * 4, 256);
    p.few_ml = at;
    at += up(rows * 8, 256);
    p.few_parts = at;
    at += up(seqs * kv * 8, 256);
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

constexpr uint32_t kDeclared = 8192;  // LDS that the kernels declare beside what a launch gives, at most
uint32_t grid_of(uint64_t units) { return (uint32_t)(units < (1u << 20) ? units : 1u << 20); }

// Workgroups of a kernel that the current device holds at once (asked once a kernel and device), 256 to
// kMostResident.
uint32_t resident(const void *fn, int threads, uint32_t lds) {
  static std::mutex mu;
  static std::map<std::pair<int, const void *>, uint32_t> known;
  int dev = 0, cus = 0, per = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  try {
    std::lock_guard<std::mutex> lk(mu);
    uint32_t &n = known[{dev, fn}];
    if (!n) {
      if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) cus = 256;
      if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, fn, threads, lds) != hipSuccess || per < 1) per = 1;
      const uint32_t held = (uint32_t)cus * (uint32_t)per;
      n = held < 256 ? 256 : held < kMostResident ? held : kMostResident;
    }
    return n;
  } catch (...) {  // nothing throws across the C entries
    return 256;
  }
}

template <class T, int BITS, int D, int NQ>
hipError_t few_rows(const Plan &p, const Pages &c, const Sequences &b, hipStream_t s) {
  constexpr int W = BITS == 16 && D == 256 ? 2 : 4;
  constexpr uint32_t lds = W * 4 * 32 * FewRows<BITS, D>::kBytes;
  static_assert(lds >= W * 16 * NQ * D * 4, "the waves' sums lie in the tiles' place");
  const hipError_t e = allow_lds((const void *)attend_few<T, BITS, D, NQ, W>, lds, kDeclared);
  if (e != hipSuccess) return e;
  // as many workgroups as the chip holds
  hipLaunchKernelGGL((attend_few<T, BITS, D, NQ, W>), dim3(resident((const void *)attend_few<T, BITS, D, NQ, W>, 64 * W, lds)), dim3(64 * W), lds,
                     s, c, b, p.a);
  return hipGetLastError();
}
template <class T, int BITS, int D, int NW>
hipError_t tiles(const Plan &p, const Pages &c, const Sequences &b, hipStream_t s) {
  constexpr uint32_t lds = (key_buffers(BITS) + 2) * 64 * Rows<D>::kBytes;
  const hipError_t e = allow_lds((const void *)attend_tile<T, BITS, D, NW>, lds, BITS == 8 ? kDeclared : 0);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attend_tile<T, BITS, D, NW>), dim3(grid_of((uint64_t)p.a.tiles * c.heads * p.a.tile_splits)), dim3(64 * NW), lds, s,
                     c, b, p.a);
  return hipGetLastError();
}
template <class T, int BITS, int D>
hipError_t attend(const Plan &p, const Pages &c, const Sequences &b, hipStream_t s) {
  // attend_few goes always: it clears the rows of no sequence
  hipError_t few;
  if constexpr (D == 256) {
    few = few_rows<T, BITS, D, 1>(p, c, b, s);
  } else {
    few = p.a.cap <= 16 ? few_rows<T, BITS, D, 1>(p, c, b, s) : few_rows<T, BITS, D, 2>(p, c, b, s);
  }
  if (few != hipSuccess) return few;
  if (p.tile) {
    hipError_t st;
    if constexpr (D == 64 || D == 128) {
      st = p.a.tile_rows == 256 ? tiles<T, BITS, D, 8>(p, c, b, s) : tiles<T, BITS, D, 4>(p, c, b, s);
    } else {
      st = tiles<T, BITS, D, 4>(p, c, b, s);
    }
    if (st != hipSuccess) return st;
  }
  const uint32_t few_blocks = p.a.few_splits > 1 ? grid_of((uint64_t)b.count * c.heads * p.a.cap) : 0;
  const uint32_t tile_blocks = p.a.tile_splits > 1 ? grid_of(((uint64_t)b.tokens * p.a.heads * (D / 4) + 255) / 256) : 0;
  if (few_blocks + tile_blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((join<T, D>), dim3(few_blocks + tile_blocks), dim3(256), 0, s, c, b, p.a, few_blocks);
  return hipGetLastError();
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
  a.few_parts = (uint32_t *)(ws + p.few_parts);
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
