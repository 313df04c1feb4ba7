// Products with uint4 weights and group scales (gfx950).
//
//   y[m, n]  = sum_k x[m, k] s[n, g] (q[n, k] - z[n, g]),   g = k / group
//   dx[m, k] = sum_n dy[m, n] s[n, g] (q[n, k] - z[n, g])
//
// The weights are the packed nibbles that a uint4 container decodes to: the
// element n * cols + k, two per byte, the even one in the low nibble.
//
// Few rows: u4_tokens (up to 4) and u4_tile (few_rows) feed the matrix cores
// with the integers themselves, and the scale multiplies a group's FP32 sum.
// More rows: the weights are expanded to 16 bits in the caller's workspace and
// the tiled product of dfh_gemm.h takes them.
#include <hip/hip_runtime.h>

#include "dfh.h"
#include "dfh_gemm.h"

namespace {

using namespace dfh;

struct U4 {
  const uint8_t *packed, *zeros;  // zeros null: 8 everywhere
  const void *scales;
  int scale_type;
  uint32_t n, k;
  uint32_t group32;  // group / 32; 0: one group per row
  uint32_t magic;    // floor(2^31 / group32) + 1, or 0
  uint32_t groups;   // per row
  uint32_t once;     // more nibbles than the last-level cache holds: read past it
  uint64_t sstride, zstride;
};

// Group of the 32 elements at 32 * b: floor(b / d) for groups of 32 d elements.
// 2 b (floor(2^31 / d) + 1) / 2^32 = b / d + e with 0 < e <= b / 2^31, so the
// floor is exact while b d < 2^31; cols <= 2^20 keeps both at most 2^15.
__device__ __forceinline__ uint32_t group_of(const U4 &w, uint32_t b) { return __umulhi(b << 1, w.magic); }

__device__ __forceinline__ float scale_at(const U4 &w, uint32_t n, uint32_t g) {
  const uint64_t i = n * w.sstride + g;
  if (w.scale_type == DF_TYPE_F32) return ((const float *)w.scales)[i];
  const uint16_t b = ((const uint16_t *)w.scales)[i];
  return w.scale_type == DF_TYPE_BF16 ? from_bits(BF16{}, b) : from_bits(F16{}, b);
}
// A raw scale of the type that a kernel was made for.
__device__ __forceinline__ float scale_of(const U4 &, float s) { return s; }
__device__ __forceinline__ float scale_of(const U4 &w, uint16_t b) {
  return w.scale_type == DF_TYPE_BF16 ? from_bits(BF16{}, b) : from_bits(F16{}, b);
}
__device__ __forceinline__ float zero_at(const U4 &w, uint32_t n, uint32_t g) {
  return w.zeros ? (float)w.zeros[n * w.zstride + g] : 8.f;
}

// Eight nibbles -> eight 16-bit floats bias + q: a nibble lands in the mantissa
// of a constant where its lowest bit counts one (BF16 16, the top four bits; FP16
// 1024, the low four), a shift and an and-or for the elements i and i + 4.
// widen_pairs leaves them so, in the order 0,4 1,5 2,6 3,7 (8 operations for 8
// weights, FP16 7), for an x whose elements are exchanged likewise; widen pairs
// neighbours with four byte permutes more.
// FP16 then takes 1024 + z off each pair with one packed addition, exactly;
// there is no such addition for BF16, whose bias (and zero point) come off the
// group's sum instead.  16 is the smallest bias that leaves q four bits: what is
// taken off is x (16 + z), so a sum of x (q - z) is as exact as FP32 sums of terms
// a few times larger (with 128, one operation less, about 17 times).
template <class T>
struct Bias;
template <>
struct Bias<BF16> {
  static constexpr uint32_t bits = 0x41804180u;
  static constexpr int shift = 3;
  static constexpr float value = 16.f;
  static constexpr bool in_sum = true;
};
template <>
struct Bias<F16> {
  static constexpr uint32_t bits = 0x64006400u;
  static constexpr int shift = 0;
  static constexpr float value = 1024.f;
  static constexpr bool in_sum = false;
};
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
// (w & mask) | bits in one instruction (truth table 0xEA); left to itself the
// compiler makes two, each with a literal.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  return __builtin_amdgcn_bitop3_b32(w, mask, bits, 0xEA);
}
// off: the pair of -(1024 + z), FP16 only
template <class T>
__device__ __forceinline__ uint32_t unbias(uint32_t v, uint32_t off) {
  if constexpr (Bias<T>::in_sum) return v;
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, v) + __builtin_bit_cast(f16x2, off));
}
template <class T>
__device__ __forceinline__ u32x4 widen_pairs(uint32_t w, uint32_t off) {
  constexpr int s = Bias<T>::shift;
  constexpr uint32_t m = 0x000F000Fu << s, b = Bias<T>::bits;
  return u32x4{unbias<T>(and_or(w << s, m, b), off), unbias<T>(and_or(w >> (4 - s), m, b), off),
               unbias<T>(and_or(w >> (8 - s), m, b), off), unbias<T>(and_or(w >> (12 - s), m, b), off)};
}
template <class T>
__device__ __forceinline__ u32x4 widen(uint32_t w, uint32_t off) {
  const u32x4 p = widen_pairs<T>(w, off);
  return u32x4{__builtin_amdgcn_perm(p[1], p[0], 0x05040100u), __builtin_amdgcn_perm(p[3], p[2], 0x05040100u),
               __builtin_amdgcn_perm(p[1], p[0], 0x07060302u), __builtin_amdgcn_perm(p[3], p[2], 0x07060302u)};
}
// Eight 16-bit values in order into widen_pairs' order.
__device__ __forceinline__ u32x4 pair_up(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
               __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

// One output from the definition, in order; taken where BF16's fast sum is not
// finite (an infinite or very large x: the bias would turn inf * w into NaN).
// 192 x 14336 x 4096, which takes 57 us: 247 us where x is all NaN, 31 ms where
// every row ends in an infinity (43 ms with a wave to an output): no fast path is
// made for such rows.
template <class T>
__device__ float dot_plain(const U4 &w, const uint16_t *xr, uint32_t n) {
  float acc = 0.f;
  const uint8_t *row = w.packed + (uint64_t)n * (w.k / 2);
  for (uint32_t b = 0; b * 32 < w.k; b++) {
    const uint32_t g = group_of(w, b);
    const float s = scale_at(w, n, g), z = zero_at(w, n, g);
    const uint32_t hi = (b + 1) * 32 < w.k ? (b + 1) * 32 : w.k;
    for (uint32_t k = b * 32; k < hi; k++) {
      const uint32_t q = (row[k / 2] >> (4 * (k & 1))) & 15u;
      acc += from_bits(T{}, xr[k]) * (((float)q - z) * s);
    }
    if (acc != acc) break;  // a NaN stays one: a row of them costs one block of 32
  }
  return acc;
}

// A byte 8 where a matrix has no zero points, read like any other.
__device__ const uint32_t g_eights = 0x08080808u;
// Says that zero points lie in global memory: a choice between the caller's and
// g_eights hides it, and flat loads wait for LDS as well (14336 x 4096 for a token:
// 11.4 us against 10.5).
typedef const __attribute__((address_space(1))) uint8_t *GlobalBytes;

// A wave's 16 rows of the weights (row n0 + lane % 16) as the operands below want
// them.  SUB, the groups that 128 elements hold (1, 2, 4), fixes how scales and zero points are read: a stage's 4 SUB (blocks of 128)
// in a row where the group size is 128 / SUB, one by one otherwise (SUB = 4: any
// multiple of 32; 0: a multiple of 128, or one group a row).  Raw values are
// kept and converted at their use: a conversion at the load would wait for it.
template <int BLOCKS, int SUB, class S>
struct Scales {
  static constexpr int G = SUB ? SUB : 1, N = BLOCKS * G;
  const S *ps;
  GlobalBytes pz;
  S raw[N];
  uint32_t zero[(N + 3) / 4];  // four a word
  __device__ __forceinline__ void rows(const U4 &w, uint32_t n0, uint32_t lr) {
    const uint32_t n = n0 + lr, nn = n < w.n ? n : w.n - 1;
    ps = (const S *)w.scales + nn * w.sstride;
    pz = (GlobalBytes)(w.zeros ? w.zeros + nn * w.zstride : (const uint8_t *)&g_eights);
  }
  // those of the blocks at element 32 * b32 on
  __device__ __forceinline__ void request(const U4 &w, uint32_t b32) {
    const uint32_t zon = w.zeros ? 1 : 0;
    const uint32_t g0 = b32 / 4 * G;
    if (SUB && w.group32 * SUB == 4 && g0 + N <= w.groups) {
      __builtin_memcpy(&raw, ps + g0, sizeof raw);
      if (zon) {
        if constexpr (N % 4 == 0) {
          __builtin_memcpy(&zero, (const uint8_t *)(pz + g0), N);
        } else {
          uint16_t h;
          if constexpr (N == 2) __builtin_memcpy(&h, (const uint8_t *)(pz + g0), 2);
          if constexpr (N == 1) h = pz[g0];
          zero[0] = h;
        }
      } else {
#pragma unroll
        for (int g = 0; g < (N + 3) / 4; g++) zero[g] = 0x08080808u;
      }
    } else {
#pragma unroll
      for (int g = 0; g < N; g++) {
        uint32_t gi = group_of(w, b32 + g * (4 / G));
        gi = gi < w.groups ? gi : w.groups - 1;
        raw[g] = ps[gi];
        const uint32_t zb = pz[gi * zon];
        zero[g / 4] = (g & 3 ? zero[g / 4] : 0) | zb << (8 * (g & 3));
      }
    }
  }
  __device__ __forceinline__ float scale(const U4 &w, int g) const { return scale_of(w, raw[g]); }
  __device__ __forceinline__ float zero_point(int g) const {
    return (float)((zero[g / 4] >> (8 * (g & 3))) & 255u);
  }
};

// The four dwords of 16 bytes that the lane groups hold (group kg: elements
// 32 kg .. + 31 of a block), exchanged so that dword d of group kg holds
// elements 32 d + 8 kg .. + 7: a 4 x 4 transposition over the groups.
__device__ __forceinline__ u32x4 by_step(u32x4 q) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(q[0], q[2], false, false));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(q[1], q[3], false, false));
  const u32x2 c = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false));
  const u32x2 d = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false));
  return u32x4{c[0], c[1], d[0], d[1]};
}

template <class T>
__device__ __forceinline__ uint32_t minus_pair(float v) {
  return (uint32_t)to_bits(T{}, -v) * 0x10001u;
}

// acc += s (T - (bias + z) S), or s T where the operand had the bias taken off.
template <class T>
__device__ __forceinline__ float scaled(float acc, float s, float z, float t, float sx) {
  return __builtin_fmaf(s, Bias<T>::in_sum ? __builtin_fmaf(-(Bias<T>::value + z), sx, t) : t, acc);
}

// The last k % 32 elements of the rows, one matrix step from guarded dwords:
// adds to acc[i][0 .. J).  px: this lane's rows of x.
template <class T, int J, int MT, class Acc>
__device__ __forceinline__ void row_ends(const U4 &w, uint32_t n0, const uint16_t *const (&px)[MT], Acc &acc) {
  const uint32_t lane = threadIdx.x & 63, lr = lane & 15, kg = lane >> 4;
  const uint32_t k32 = w.k & ~31u, k = k32 + kg * 8;
  const uint32_t one = (uint32_t)to_bits(T{}, 1.f) * 0x10001u;
  const uint32_t g = group_of(w, k32 / 32);
  const uint32_t n = n0 + lr, nn = n < w.n ? n : w.n - 1;
  uint32_t q = 0;
  if (k < w.k) q = *(const uint32_t *)(w.packed + ((uint64_t)nn * w.k + k) / 2);
  const float s = scale_at(w, nn, g), z = zero_at(w, nn, g);
  const u32x4 f = widen<T>(q, minus_pair<T>(Bias<T>::value + z));
#pragma unroll
  for (int i = 0; i < MT; i++) {
    u32x4 xp = {0, 0, 0, 0};
    if (k < w.k) xp = *(const u32x4 *)(px[i] + k);
    const f32x4 sx = mfma(T{}, xp, u32x4{one, one, one, one}, f32x4{0.f, 0.f, 0.f, 0.f});
    const f32x4 t = mfma(T{}, xp, f, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int r = 0; r < J; r++) acc[i][r] = scaled<T>(acc[i][r], s, z, t[r], sx[r]);
  }
}

// y for up to four rows (tokens).  A workgroup makes 16 columns; each wave
// has a part of the summed index, in stages of 512 elements, and the waves add
// up through LDS.  Matrix operand A is x, B the weights (16 columns n): lane l
// holds 16 bytes of weight row l % 16.  BF16: T = sum x (bias + q) and
// S = sum x (operand B all ones) give a group's part as s (T - (bias + z) S),
// in FP32; FP16: T = sum x (q - z) and s T.  A result's row is 4 (l / 16) + r:
// row m of x is put at 4 m (the rows between hold copies), so the scales cost
// one multiplication a lane, not four.
//
// The loads go to LDS: an operand wants 16 rows side by side, of which a
// register load would fetch 64 bytes each, while here a load takes 256
// contiguous bytes of 4 rows (and x's 512 elements of a row), and what is in
// flight needs no registers.  A wave's two buffers are its own, so the waves
// do not meet before the sum; a stage is requested while the one before is
// used.  LDS rows hold their 16-byte chunks at position chunk ^ row, exchanged
// in the source address.
template <class T, int W, int SUB, class S>
__global__ __launch_bounds__(64 * W) void u4_tokens(const U4 w, const uint16_t *x, uint64_t xs, uint32_t m,
                                                    uint16_t *y) {
  extern __shared__ __align__(1024) uint8_t lds[];
  typedef Scales<4, SUB, S> Sc;
  constexpr int G = Sc::G;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lr = lane & 15, kg = lane >> 4;
  const uint32_t n0 = blockIdx.x * 16;
  const uint32_t k32 = w.k & ~31u;
  const uint32_t stages = (k32 + 511) / 512, per = (stages + W - 1) / W;
  const uint32_t s0 = wave * per, s1 = s0 + per < stages ? s0 + per : stages;
  const uint32_t bytes = 4096 + m * 1024;  // a buffer
  const uint32_t step = per > 1 ? bytes : 0;    // one buffer is enough for one stage
  uint8_t *buf = lds + wave * (bytes + step);
  const uint32_t one = (uint32_t)to_bits(T{}, 1.f) * 0x10001u;
  const u32x4 ones = {one, one, one, one};
  const uint32_t xr = lr >> 2 < m ? lr >> 2 : m - 1;  // the row of x in this lane's operand row
  Sc next, now;
  next.rows(w, n0, lr);
  // this lane's 16 bytes of four weight rows a load
  const uint8_t *src[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t r = i * 4 + (lane >> 4), n = n0 + r;
    src[i] = w.packed + (uint64_t)(n < w.n ? n : w.n - 1) * (w.k / 2) + ((lane & 15) ^ r) * 16;
  }
  auto request = [&](uint32_t st, uint8_t *dst) {
    const bool whole = st * 512 + 512 <= k32;  // uniform
    const uint8_t *p[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      p[i] = src[i] + st * 256;
      if (!whole && st * 512 + ((lane & 15) ^ (i * 4 + (lane >> 4))) * 32 >= k32) p[i] = (const uint8_t *)&g_zero16;
    }
    if (w.once) {  // uniform
#pragma unroll
      for (int i = 0; i < 4; i++) to_lds<true>(p[i], dst + i * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) to_lds(p[i], dst + i * 1024);
    }
    for (uint32_t r = 0; r < m; r++) {
      const uint32_t k = st * 512 + (lane ^ r) * 8;
      to_lds(k < k32 ? (const void *)(x + r * xs + k) : (const void *)&g_zero16, dst + 4096 + r * 1024);
    }
    next.request(w, st * 16);
  };
  float acc[1][1] = {};
  if (s0 < s1) request(s0, buf);
  if (k32 < w.k && wave == W - 1) {
    const uint16_t *px[1] = {x + xr * xs};
    row_ends<T, 1, 1>(w, n0, px, acc);
  }
  for (uint32_t st = s0; st < s1; st++) {
    uint8_t *p = buf + ((st - s0) & 1) * step;
    // this stage has landed, and the last one's reads of the buffer that the next
    // one goes to have returned
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    now = next;
    if (st + 1 < s1) request(st + 1, buf + ((st + 1 - s0) & 1) * step);
    // x into widen_pairs' order where it lies: once a stage, 16 bytes a lane
    for (uint32_t r = 0; r < m; r++) {
      u32x4 *c = (u32x4 *)(p + 4096 + r * 1024) + lane;
      *c = pair_up(*c);
    }
    asm volatile("" ::: "memory");
    const uint8_t *px = p + 4096 + xr * 1024;
#pragma unroll
    for (int b = 0; b < 4; b++) {
      if (st * 512 + b * 128 >= k32) break;  // uniform
      u32x4 xp[4];
      f32x4 sx[G] = {};
#pragma unroll
      for (int d = 0; d < 4; d++) {
        const uint32_t c = b * 16 + (SUB > 1 ? d * 4 + kg : kg * 4 + d);
        xp[d] = *(const u32x4 *)(px + (c ^ xr) * 16);
        if constexpr (Bias<T>::in_sum) sx[d * G / 4] = mfma(T{}, xp[d], ones, sx[d * G / 4]);
      }
      u32x4 q = *(const u32x4 *)(p + lr * 256 + (((b * 4 + kg) ^ lr) * 16));
      if (SUB > 1) q = by_step(q);
      f32x4 t[G] = {};
#pragma unroll
      for (int d = 0; d < 4; d++)
        t[d * G / 4] = mfma(T{}, xp[d],
                            widen_pairs<T>(q[d], minus_pair<T>(Bias<T>::value + now.zero_point(b * G + d * G / 4))),
                            t[d * G / 4]);
#pragma unroll
      for (int g = 0; g < G; g++)
        acc[0][0] = scaled<T>(acc[0][0], now.scale(w, b * G + g), now.zero_point(b * G + g), t[g][0], sx[g][0]);
    }
  }
  // every wave has its last buffer behind it; the sums take its place
  __syncthreads();
  float *part = (float *)lds;  // [W][64]
  part[wave * 64 + lane] = acc[0][0];
  __syncthreads();
  if (wave == 0) {
    const uint32_t mm = lane / 16, n = n0 + (lane & 15);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < W; q++) v += part[q * 64 + lane];
    if (mm < m && n < w.n) {
      if (Bias<T>::in_sum && !(__builtin_fabsf(v) < __builtin_huge_valf())) v = dot_plain<T>(w, x + mm * xs, n);
      y[(uint64_t)mm * w.n + n] = to_bits(T{}, v);
    }
  }
}

// y for a tile of 16 MT rows of x and 64 weight rows, for row counts between
// tokens and prompts.  Eight waves: wave w takes weight rows 16 (w % 4) .. and
// the block w / 4 of a stage's two blocks of 128 elements; all share the stage's
// x in LDS.  Arithmetic as in u4_tokens, all four result rows of a lane used.
// blockIdx.y: split of the summed index; a split's sums go to its FP32 plane
// (one split: straight to y).
template <class T, int MT, int SUB, class S>
__global__ __launch_bounds__(512) void u4_tile(const U4 w, const uint16_t *x, uint64_t xs, uint32_t m, uint32_t mt,
                                               uint32_t per, uint16_t *y, float *planes, uint32_t ld) {
  extern __shared__ __align__(1024) uint8_t lds[];
  typedef Scales<1, SUB, S> Sc;
  constexpr int G = Sc::G, BN = 64, BM = 16 * MT;
  constexpr uint32_t kBuf = BN * 128 + BM * 512;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lr = lane & 15, kg = lane >> 4, wn = wave & 3, wk = wave >> 2;
  const uint32_t m0 = blockIdx.x % mt * BM, nb = blockIdx.x / mt * BN, n0 = nb + wn * 16;
  const uint32_t rows = m - m0 < BM ? m - m0 : BM;
  const uint32_t k32 = w.k & ~31u, stages = (k32 + 255) / 256;
  const uint32_t s0 = blockIdx.y * per, s1 = s0 + per < stages ? s0 + per : stages;
  const uint32_t one = (uint32_t)to_bits(T{}, 1.f) * 0x10001u;
  const u32x4 ones = {one, one, one, one};
  Sc next, now;
  next.rows(w, n0, lr);
  // 8 weight rows of 128 bytes a load
  const uint32_t wr = wave * 8 + lane / 8, wrow = nb + wr < w.n ? nb + wr : w.n - 1;
  const uint8_t *wsrc = w.packed + (uint64_t)wrow * (w.k / 2) + ((lane & 7) ^ swz(wr)) * 16;
  const uint16_t *xsrc[MT];  // 2 rows of x a load
#pragma unroll
  for (int i = 0; i < MT; i++) {
    const uint32_t r = (i * 8 + wave) * 2 + lane / 32;
    xsrc[i] = x + (uint64_t)(m0 + (r < rows ? r : rows - 1)) * xs + ((lane & 31) ^ (r & 15)) * 8;
  }
  auto request = [&](uint32_t st, uint8_t *dst) {
    const bool whole = st * 256 + 256 <= k32;  // uniform
    const uint8_t *q = wsrc + st * 128;
    if (!whole && st * 256 + ((lane & 7) ^ swz(wr)) * 32 >= k32) q = (const uint8_t *)&g_zero16;
    to_lds(q, dst + wave * 1024);
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const uint32_t pair = i * 8 + wave;
      if (pair * 2 >= rows) continue;  // uniform
      const uint16_t *p = xsrc[i] + st * 256;
      if (!whole && st * 256 + ((lane & 31) ^ ((pair * 2 + lane / 32) & 15)) * 8 >= k32) p = (const uint16_t *)&g_zero16;
      to_lds(p, dst + BN * 128 + pair * 1024);
    }
    next.request(w, st * 8 + wk * 4);
  };
  f32x4 acc[MT] = {};
  if (s0 < s1) request(s0, lds);
  if (k32 < w.k && blockIdx.y == 0 && wk == 1) {
    const uint16_t *px[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) px[i] = x + (uint64_t)(m0 + (i * 16 + lr < rows ? i * 16 + lr : rows - 1)) * xs;
    row_ends<T, 4, MT>(w, n0, px, acc);
  }
  for (uint32_t st = s0; st < s1; st++) {
    const uint8_t *p = lds + ((st - s0) & 1) * kBuf;
    wait_but<0>();
    __syncthreads();
    now = next;
    if (st + 1 < s1) request(st + 1, lds + ((st + 1 - s0) & 1) * kBuf);
    if (st * 256 + wk * 128 < k32) {
      const uint8_t *px = p + BN * 128 + lr * 512, *pw = p + (wn * 16 + lr) * 128 + (((wk * 4 + kg) ^ swz(lr)) * 16);
      u32x4 q = *(const u32x4 *)pw;
      f32x4 t[G][MT] = {}, sx[G][MT] = {};
      if (SUB > 1) q = by_step(q);
#pragma unroll
      for (int d = 0; d < 4; d++) {
        constexpr int step = 4 / G;
        const uint32_t c = wk * 16 + (SUB > 1 ? d * 4 + kg : kg * 4 + d);
        u32x4 xp[MT];
#pragma unroll
        for (int i = 0; i < MT; i++) {
          xp[i] = *(const u32x4 *)(px + i * 8192 + ((c ^ lr) * 16));
          if constexpr (Bias<T>::in_sum) sx[d / step][i] = mfma(T{}, xp[i], ones, sx[d / step][i]);
        }
        const u32x4 f = widen<T>(q[d], minus_pair<T>(Bias<T>::value + now.zero_point(d / step)));
#pragma unroll
        for (int i = 0; i < MT; i++) t[d / step][i] = mfma(T{}, xp[i], f, t[d / step][i]);
      }
#pragma unroll
      for (int g = 0; g < G; g++) {
        const float s = now.scale(w, g), z = now.zero_point(g);
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
          for (int r = 0; r < 4; r++) acc[i][r] = scaled<T>(acc[i][r], s, z, t[g][i][r], sx[g][i][r]);
      }
    }
  }
  // the second block's waves hand their sums to the first block's
  __syncthreads();
  f32x4 *part = (f32x4 *)lds;
  if (wk == 1)
#pragma unroll
    for (int i = 0; i < MT; i++) part[(i * 4 + wn) * 64 + lane] = acc[i];
  __syncthreads();
  if (wk == 1) return;
  const uint32_t n = n0 + lr;
#pragma unroll
  for (int i = 0; i < MT; i++) {
    const f32x4 v = acc[i] + part[(i * 4 + wn) * 64 + lane];
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const uint32_t row = m0 + i * 16 + kg * 4 + r;
      if (row >= m || n >= w.n) continue;
      if (planes) {
        planes[((uint64_t)blockIdx.y * m + row) * ld + n] = v[r];
      } else {
        float o = v[r];
        if (Bias<T>::in_sum && !(__builtin_fabsf(o) < __builtin_huge_valf())) o = dot_plain<T>(w, x + (uint64_t)row * xs, n);
        y[(uint64_t)row * w.n + n] = to_bits(T{}, o);
      }
    }
  }
}

// The planes of u4_tile's splits added up.
template <class T>
__global__ __launch_bounds__(256) void join_tiles(const U4 w, const uint16_t *x, uint64_t xs, const float *planes,
                                                  uint32_t splits, uint32_t m, uint32_t ld, uint16_t *y) {
  const uint32_t row = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= w.n) return;
  const f32x4 v = add_planes(planes + (uint64_t)row * ld + n, (uint64_t)m * ld, splits);
#pragma unroll
  for (int e = 0; e < 4; e++) {
    if (n + e >= w.n) break;
    float o = v[e];
    if (Bias<T>::in_sum && !(__builtin_fabsf(o) < __builtin_huge_valf())) o = dot_plain<T>(w, x + row * xs, n + e);
    y[(uint64_t)row * w.n + n + e] = to_bits(T{}, o);
  }
}

// FP16 keeps neither small nor large weights, so its copies are lifted: a power
// of two per row (for the gradient, which sums over the rows, one for the matrix)
// brings the largest scale to 2^6 .. 2^7, with any q - z within FP16, and comes off
// the FP32 sums.  A weight then keeps FP16's 11 bits, or 2^-31 of the largest scale
// where that is more.  BF16 has FP32's range and needs none.
struct Lift {
  const float *peaks;  // gradient: the matrix's largest scale in 256 parts
  float *back;         // what comes off: one a row; gradient: one, and a 1
};
template <class S>
__device__ __forceinline__ float size_at(const U4 &w, const S *p) {
  const float v = __builtin_fabsf(scale_of(w, *p));
  return v < __builtin_huge_valf() ? v : 0.f;  // where not finite, all results are as they are
}
// The largest finite scale of the matrix in 256 parts.
template <class S>
__global__ __launch_bounds__(256) void scale_peaks(const U4 w, float *peaks) {
  const uint64_t all = w.sstride ? (uint64_t)w.n * w.groups : w.groups;
  float v = 0.f;
#pragma unroll 4
  for (uint64_t i = blockIdx.x * 256 + threadIdx.x; i < all; i += 65536) {
    uint64_t at = i;
    if (w.sstride != w.groups) at = i / w.groups * w.sstride + i % w.groups;
    v = __builtin_fmaxf(v, size_at(w, (const S *)w.scales + at));
  }
  v = most_of_256(v);
  if (threadIdx.x == 0) peaks[blockIdx.x] = v;
}

// The weights as 16-bit floats, [n, k]: what the matrix instructions of a long product
// take.  Each is rounded once from FP32 (relative 2^-8 / 2^-11 at most, but for what is
// said above); the sums over them are FP32.
// A workgroup takes 1024 chunks of 8 weights of a row, four a thread, all loaded
// (scales unconverted) before the first is used.
template <class T, class S>
__global__ __launch_bounds__(256) void u4_expand(const U4 w, uint16_t *out, const Lift lift) {
  const uint32_t n = blockIdx.x, chunks = w.k / 8, c0 = blockIdx.y * 1024 + threadIdx.x;
  const uint64_t row = (uint64_t)n * chunks;
  const S *ps = (const S *)w.scales + n * w.sstride;
  const uint8_t *pz = w.zeros ? w.zeros + n * w.zstride : (const uint8_t *)&g_eights;
  const uint32_t zon = w.zeros ? 1 : 0;
  float most = 0.f;
  if constexpr (!Bias<T>::in_sum) {
    // by every wave for itself: the workgroup does not meet
    const uint32_t lane = threadIdx.x & 63;
    if (lift.peaks) {
#pragma unroll
      for (int i = 0; i < 4; i++) most = __builtin_fmaxf(most, lift.peaks[lane + i * 64]);
    } else {
      for (uint32_t g = lane; g < w.groups; g += 64) most = __builtin_fmaxf(most, size_at(w, ps + g));
    }
  }
  uint32_t q[4];
  S s[4];
  uint8_t z[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t c = c0 + i * 256 < chunks ? c0 + i * 256 : chunks - 1, g = group_of(w, c / 4);
    q[i] = ((const uint32_t *)w.packed)[row + c];
    s[i] = ps[g];
    z[i] = pz[g * zon];
  }
  float up = 1.f;
  if constexpr (!Bias<T>::in_sum) {
    const int bits = lift_bits(most_of_wave(most), 6);
    up = power_of_two(bits);
    if (threadIdx.x == 0 && blockIdx.y == 0) {
      if (!lift.peaks) {
        lift.back[n] = power_of_two(-bits);
      } else if (n == 0) {
        lift.back[0] = power_of_two(-bits);
        lift.back[1] = 1.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t c = c0 + i * 256;
    if (c >= chunks) break;
    const float f = scale_of(w, s[i]) * up, o = (float)z[i];
    u32x4 v;
#pragma unroll
    for (int d = 0; d < 4; d++)
      v[d] = pack2(T{}, ((float)((q[i] >> (8 * d)) & 15u) - o) * f, ((float)((q[i] >> (8 * d + 4)) & 15u) - o) * f);
    ((u32x4 *)out)[row + c] = v;
  }
}
// The copy and the lift's part of a workspace, in bytes.
uint64_t copy_bytes(uint64_t n, uint64_t k) { return up(n * k * 2, 256); }
uint64_t lift_bytes(uint64_t n, bool gradient) { return gradient ? 1280 : up(n * 4, 256); }
// Expands into a workspace; what comes off the sums: back, null where nothing does.
template <class T>
const float *expand(const U4 &w, uint8_t *ws, bool gradient, hipStream_t s) {
  Lift lift = {nullptr, nullptr};
  if (!Bias<T>::in_sum) {
    float *f = (float *)(ws + copy_bytes(w.n, w.k));
    lift.back = f;
    if (gradient) {
      lift.peaks = f + 64;
      hipLaunchKernelGGL((w.scale_type == DF_TYPE_F32 ? scale_peaks<float> : scale_peaks<uint16_t>), dim3(256), dim3(256),
                         0, s, w, f + 64);
    }
  }
  auto *fn = w.scale_type == DF_TYPE_F32 ? u4_expand<T, float> : u4_expand<T, uint16_t>;
  hipLaunchKernelGGL(fn, dim3(w.n, (w.k + 8191) / 8192), dim3(256), 0, s, w, (uint16_t *)ws, lift);
  return lift.back;
}

// Sum of FP32 planes [splits][m][ld] -> 16-bit [m, n], times back[n] (EACH) or *back,
// where there is one.
template <class T, bool EACH>
__global__ __launch_bounds__(256) void join_planes(const float *p, uint32_t splits, uint32_t m, uint32_t n,
                                                   uint32_t ld, const float *back, uint16_t *out) {
  const uint32_t row = blockIdx.x;
  float all = 1.f;
  if constexpr (!Bias<T>::in_sum && !EACH) all = *back;
  for (uint32_t c = threadIdx.x * 4; c < n; c += 1024) {
    f32x4 f = {all, all, all, all};
    if constexpr (!Bias<T>::in_sum && EACH) {
#pragma unroll
      for (int e = 0; e < 4; e++) f[e] = back[c + e < n ? c + e : n - 1];
    }
    f32x4 v = add_planes(p + (uint64_t)row * ld + c, (uint64_t)m * ld, splits);
    if constexpr (!Bias<T>::in_sum) v *= f;
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (c + e < n) out[(uint64_t)row * n + c + e] = to_bits(T{}, v[e]);
  }
}

// Rows of n elements into rows of np (n rounded up to 8), zeros past n.  At most
// 2^20 workgroups, so that 2^24 rows stay under a launch's 2^32 threads.
__global__ __launch_bounds__(256) void pad_rows(const uint16_t *src, uint64_t ss, uint32_t m, uint32_t n, uint32_t np,
                                                uint16_t *dst) {
  for (uint64_t r = blockIdx.x; r < m; r += gridDim.x)
    for (uint32_t c = threadIdx.x; c < np; c += 256) dst[r * np + c] = c < n ? src[r * ss + c] : (uint16_t)0;
}

// Rows that u4_tile takes rather than an expansion: the expansion costs a fixed
// time per weight (0.45 us a million), the tile kernel a time per weight and 64
// rows (0.3 us a million once the chip is full, less before).  Tile against
// expansion, us, BF16 (FP16): 200 x 4096 x 4096 28 : 34 (24 : 36), 384 rows of it 38 :
// 40 (33 : 42), 512 41 : 42 (34 : 44); 192 x 14336 x 4096 57 : 82 (54 : 92), 256 rows
// of it 71 : 79 (62 : 87), where the rule does not follow yet; 333 x 2047 x 1416 13 : 23.
bool few_rows(uint64_t m, uint64_t n, uint64_t k) {
  return m <= 192 || (m <= 384 && n * k <= 1u << 24) || (m <= 512 && n * k <= 1u << 22);
}
bool type_ok(df_type t) { return t == DF_TYPE_BF16 || t == DF_TYPE_F16; }

df_status matrix_of(const df_u4_matrix *m, U4 *w) {
  if (!m || !m->packed || !m->scales || ((uintptr_t)m->packed & 3)) return DF_ERR_ARG;
  if (m->rows == 0 || m->rows > (1u << 21) || m->cols == 0 || m->cols > (1u << 20) || m->cols % 8) return DF_ERR_ARG;
  if (m->scale_type != DF_TYPE_BF16 && m->scale_type != DF_TYPE_F16 && m->scale_type != DF_TYPE_F32)
    return DF_ERR_ARG;
  if ((uintptr_t)m->scales & (m->scale_type == DF_TYPE_F32 ? 3 : 1)) return DF_ERR_ARG;
  if (m->group_size == 0 || (m->group_size < m->cols && m->group_size % 32)) return DF_ERR_ARG;
  w->packed = m->packed;
  w->zeros = m->zeros;
  w->scales = m->scales;
  w->scale_type = (int)m->scale_type;
  w->n = (uint32_t)m->rows;
  w->k = (uint32_t)m->cols;
  w->sstride = m->scale_stride;
  w->zstride = m->zero_stride;
  w->group32 = (uint32_t)(m->group_size < m->cols ? m->group_size / 32 : 0);
  w->magic = w->group32 ? (1u << 31) / w->group32 + 1 : 0;
  // 53248 x 16384 (436 MB): 107 us with plain loads, 101 non-temporal; 1024 x 4096
  // (2 MB, found in the cache by the next token): 4.4 against 4.7
  w->once = m->rows * m->cols / 2 >= (256u << 20);
  w->groups = w->group32 ? (uint32_t)((m->cols + m->group_size - 1) / m->group_size) : 1;
  return DF_OK;
}

// y or dx from 16-bit operands, times back; planes: cut_for's splits.
template <class T, bool GRAD>
df_status many_rows(const Gemm &g, uint16_t *out, const float *back, float *planes, hipStream_t s) {
  constexpr bool kColumns = !GRAD && !Bias<T>::in_sum;  // a factor for every column
  const Cut c = cut_for(g.m, g.n, g.k, true);
  if (c.splits <= 1) {
    const EpiStore<kColumns> e = {out,    g.n, GRAD ? back : nullptr, GRAD && back ? back + 1 : nullptr, 1.f,
                                  kColumns ? back : nullptr};
    return product<T, false, GRAD>(g, e, c.shape, 1, s) == hipSuccess ? DF_OK : DF_ERR_HIP;
  }
  const uint32_t ld = (uint32_t)up(g.n, 4);
  if (product<T, false, GRAD>(g, EpiPlane{planes, ld, (uint64_t)g.m * ld, false}, c.shape, c.splits, s) != hipSuccess) return DF_ERR_HIP;
  hipLaunchKernelGGL((join_planes<T, !GRAD>), dim3(g.m), dim3(256), 0, s, (const float *)planes, c.splits, g.m, g.n, ld,
                     back, out);
  return hipGetLastError() == hipSuccess ? DF_OK : DF_ERR_HIP;
}

int sub_of(const U4 &w) { return w.group32 == 4 ? 1 : w.group32 == 2 ? 2 : w.group32 % 4 == 0 ? 0 : 4; }

template <class T, int W, class S>
hipError_t tokens_of(const U4 &w, const uint16_t *x, uint64_t xs, uint32_t m, uint16_t *y, hipStream_t s) {
  const int sub = sub_of(w);
  auto *fn = sub == 0   ? u4_tokens<T, W, 0, S>
             : sub == 1 ? u4_tokens<T, W, 1, S>
             : sub == 2 ? u4_tokens<T, W, 2, S>
                        : u4_tokens<T, W, 4, S>;
  const uint32_t buffers = (w.k / 32 * 32 + 511) / 512 > W ? 2 : 1;
  const uint32_t lds = W * buffers * (4096 + m * 1024);
  const hipError_t e = allow_lds((const void *)fn, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3((w.n + 15) / 16), dim3(64 * W), lds, s, w, x, xs, m, y);
  return hipGetLastError();
}
template <class T, int W>
hipError_t tokens_launch(const U4 &w, const uint16_t *x, uint64_t xs, uint32_t m, uint16_t *y, hipStream_t s) {
  return w.scale_type == DF_TYPE_F32 ? tokens_of<T, W, float>(w, x, xs, m, y, s)
                                     : tokens_of<T, W, uint16_t>(w, x, xs, m, y, s);
}

// How u4_tile cuts a product: splits of the summed index so that up to two
// workgroups come to a CU, of four stages of 256 elements at least (16 x 14336 x
// 4096, 224 tiles: one split 17.8 us, two 15.8, three 16.8, eight 18.2; 23 x 4096 x
// 14336, 64 tiles: one 50, four 18.5, eight 17.7).  A third and fourth buffer a
// workgroup measured the same.
struct TilePlan {
  uint32_t mtile, mt, splits, per, ld;
};
TilePlan few_plan(uint32_t m, uint32_t n, uint32_t k) {
  TilePlan p;
  p.mtile = m <= 16 ? 1 : m <= 32 ? 2 : 4;
  p.mt = (m + 16 * p.mtile - 1) / (16 * p.mtile);
  const uint32_t tiles = p.mt * ((n + 63) / 64), stages = (k / 32 * 32 + 255) / 256;
  uint32_t want = tiles >= 512 ? 1 : 512 / tiles;
  const uint32_t most = stages / 4 < 1 ? 1 : stages / 4;
  want = want < most ? want : most;
  p.per = (stages + want - 1) / want;
  if (p.per == 0) p.per = 1;
  p.splits = stages ? (stages + p.per - 1) / p.per : 1;
  p.ld = (uint32_t)up(n, 4);
  return p;
}

template <class T, int MT, class S>
hipError_t tile_of(const U4 &w, const uint16_t *x, uint64_t xs, uint32_t m, uint16_t *y, float *planes,
                   const TilePlan &p, hipStream_t s) {
  const int sub = sub_of(w);
  auto *fn = sub == 0   ? u4_tile<T, MT, 0, S>
             : sub == 1 ? u4_tile<T, MT, 1, S>
             : sub == 2 ? u4_tile<T, MT, 2, S>
                        : u4_tile<T, MT, 4, S>;
  constexpr uint32_t lds = 2 * (64 * 128 + 16 * MT * 512);
  hipError_t e = allow_lds((const void *)fn, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(p.mt * ((w.n + 63) / 64), p.splits), dim3(512), lds, s, w, x, xs, m, p.mt,
                     p.per, y, p.splits > 1 ? planes : (float *)nullptr, p.ld);
  e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL((join_tiles<T>), dim3((w.n + 1023) / 1024, m), dim3(256), 0, s, w, x, xs, (const float *)planes,
                     p.splits, m, p.ld, y);
  return hipGetLastError();
}
template <class T, int MT>
hipError_t tile_launch(const U4 &w, const uint16_t *x, uint64_t xs, uint32_t m, uint16_t *y, float *planes,
                       const TilePlan &p, hipStream_t s) {
  return w.scale_type == DF_TYPE_F32 ? tile_of<T, MT, float>(w, x, xs, m, y, planes, p, s)
                                     : tile_of<T, MT, uint16_t>(w, x, xs, m, y, planes, p, s);
}

constexpr uint32_t kTokens = 4;

template <class T>
df_status linear(const U4 &w, const uint16_t *x, uint32_t m, uint64_t xs, uint16_t *y, uint8_t *ws, hipStream_t s) {
  hipError_t e;
  if (m <= kTokens) {
    // waves a workgroup: 4 where the columns alone fill the chip (14336 x 4096:
    // 10.5 us, with 8 11.8), 16 where they give one workgroup a CU or less and the
    // rows are long (4096 x 14336: 10.5 us, with 8 12.0), else 8 (4096 x 4096: 5.3
    // us, with 4 6.0); 16 have LDS for one row of x
    e = w.n >= 8192                     ? tokens_launch<T, 4>(w, x, xs, m, y, s)
        : m == 1 && w.n <= 4096 && w.k > 8192 ? tokens_launch<T, 16>(w, x, xs, m, y, s)
                                        : tokens_launch<T, 8>(w, x, xs, m, y, s);
  } else if (few_rows(m, w.n, w.k)) {
    const TilePlan p = few_plan(m, w.n, w.k);
    e = p.mtile == 1   ? tile_launch<T, 1>(w, x, xs, m, y, (float *)ws, p, s)
        : p.mtile == 2 ? tile_launch<T, 2>(w, x, xs, m, y, (float *)ws, p, s)
                       : tile_launch<T, 4>(w, x, xs, m, y, (float *)ws, p, s);
  } else {
    const float *back = expand<T>(w, ws, false, s);
    Gemm g = {x, (const uint16_t *)ws, xs, w.k, m, w.n, w.k, 0, 0, 0, 0};
    return many_rows<T, false>(g, y, back, (float *)(ws + copy_bytes(w.n, w.k) + lift_bytes(w.n, false)), s);
  }
  return e == hipSuccess ? DF_OK : DF_ERR_HIP;
}

template <class T>
df_status linear_grad(const U4 &w, const uint16_t *dy, uint32_t m, uint64_t ds, uint16_t *dx, uint8_t *ws,
                      hipStream_t s) {
  const float *back = expand<T>(w, ws, true, s);
  uint8_t *next = ws + copy_bytes(w.n, w.k) + lift_bytes(w.n, true);
  const uint32_t np = (uint32_t)up(w.n, 8);
  if (np != w.n) {  // the summed index in whole 16-byte chunks
    hipLaunchKernelGGL(pad_rows, dim3(m < 1u << 20 ? m : 1u << 20), dim3(256), 0, s, dy, ds, m, w.n, np, (uint16_t *)next);
    dy = (const uint16_t *)next;
    ds = np;
    next += up((uint64_t)m * np * 2, 256);
  }
  Gemm g = {dy, (const uint16_t *)ws, ds, w.k, m, w.k, w.n, 0, 0, 0, 0};
  return many_rows<T, true>(g, dx, back, (float *)next, s);
}

uint64_t plane_bytes(uint64_t m, uint64_t n, uint64_t k) {
  const Cut c = cut_for(m, n, k, true);
  return c.splits > 1 ? 4ull * c.splits * m * up(n, 4) : 0;
}

}  // namespace

extern "C" {

uint64_t df_linear_u4_workspace_bytes(const df_u4_matrix *w, uint64_t rows) {
  U4 u;
  if (matrix_of(w, &u) != DF_OK || rows <= kTokens || rows > (1u << 24)) return 0;
  if (few_rows(rows, u.n, u.k)) {
    const TilePlan p = few_plan((uint32_t)rows, u.n, u.k);
    return p.splits > 1 ? 4ull * p.splits * rows * p.ld : 0;
  }
  return copy_bytes(w->rows, w->cols) + lift_bytes(w->rows, false) + plane_bytes(rows, w->rows, w->cols);
}

uint64_t df_linear_u4_grad_workspace_bytes(const df_u4_matrix *w, uint64_t rows) {
  U4 u;
  if (matrix_of(w, &u) != DF_OK || rows == 0 || rows > (1u << 24)) return 0;
  const uint64_t np = up(w->rows, 8);
  return copy_bytes(w->rows, w->cols) + lift_bytes(w->rows, true) + (np != w->rows ? up(rows * np * 2, 256) : 0) +
         plane_bytes(rows, w->cols, w->rows);
}

df_status df_linear_u4(const df_u4_matrix *w, df_type type, const void *x, uint64_t rows, uint64_t x_stride, void *y,
                       void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
  U4 u;
  const df_status st = matrix_of(w, &u);
  if (st != DF_OK) return st;
  if (!type_ok(type) || rows > (1u << 24)) return DF_ERR_ARG;
  if (rows == 0) return DF_OK;
  if (!x || !y || ((uintptr_t)x & 15) || ((uintptr_t)y & 15) || x_stride < u.k || x_stride % 8 ||
      x_stride > (1u << 21))
    return DF_ERR_ARG;
  const uint64_t need = df_linear_u4_workspace_bytes(w, rows);
  if (need && (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need)) return DF_ERR_ARG;
  if (type == DF_TYPE_BF16)
    return linear<BF16>(u, (const uint16_t *)x, (uint32_t)rows, x_stride, (uint16_t *)y, (uint8_t *)workspace, stream);
  return linear<F16>(u, (const uint16_t *)x, (uint32_t)rows, x_stride, (uint16_t *)y, (uint8_t *)workspace, stream);
}

df_status df_linear_u4_grad(const df_u4_matrix *w, df_type type, const void *dy, uint64_t rows, uint64_t dy_stride,
                            void *dx, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
  U4 u;
  const df_status st = matrix_of(w, &u);
  if (st != DF_OK) return st;
  if (!type_ok(type) || rows > (1u << 24)) return DF_ERR_ARG;
  if (rows == 0) return DF_OK;
  if (!dy || !dx || ((uintptr_t)dx & 15) || dy_stride < u.n || dy_stride > (1u << 21)) return DF_ERR_ARG;
  if (u.n % 8 ? ((uintptr_t)dy & 1) : (((uintptr_t)dy & 15) || dy_stride % 8)) return DF_ERR_ARG;
  const uint64_t need = df_linear_u4_grad_workspace_bytes(w, rows);
  if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need) return DF_ERR_ARG;
  if (type == DF_TYPE_BF16)
    return linear_grad<BF16>(u, (const uint16_t *)dy, (uint32_t)rows, dy_stride, (uint16_t *)dx, (uint8_t *)workspace,
                             stream);
  return linear_grad<F16>(u, (const uint16_t *)dy, (uint32_t)rows, dy_stride, (uint16_t *)dx, (uint8_t *)workspace,
                          stream);
}

}  // extern "C"
