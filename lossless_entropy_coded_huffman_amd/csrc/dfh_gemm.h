// Tiled products on the matrix cores for gfx950, shared by the uint4 linear
// operators and the vocabulary losses.
//
//   C[m, n] = sum_k A[m, k] B[n, k]
//
// in BF16 or FP16 with FP32 sums.  Either operand may be stored with the summed
// index contiguous ([rows, k]) or across ([k, rows]), so every direction of a
// product reads its operands as they lie.
//
// gemm: one workgroup makes a BM x BN tile.  Each step takes 64 summed elements
// of BM + BN rows from global memory straight into LDS (16 bytes a lane, no
// registers in between) into one of two buffers, while the waves run
// v_mfma_f32_16x16x32 from the other (the step loop is described at the kernel).  An operand of 16 rows wants 8 summed
// elements of one row in a lane: 16 bytes in a [rows, k] tile, and two
// transposing reads (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 elements and
// get a column of 4 each) in a [k, rows] tile.  The 16-byte chunks of an LDS row
// are stored at chunk ^ f(row), so that what one read touches lies in different
// banks; a load writes LDS linearly, so the exchange is in its source address.
#ifndef DFH_GEMM_H
#define DFH_GEMM_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <map>
#include <mutex>
#include <utility>

namespace dfh {
// Unnamed: every source that includes this has kernels of its own, so that two
// code objects never register a kernel under one host symbol.
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct BF16 {
  static constexpr bool kRange = true;  // FP32's
};
struct F16 {
  static constexpr bool kRange = false;
};

__device__ __forceinline__ f32x4 mfma(BF16, u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}
__device__ __forceinline__ f32x4 mfma(F16, u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                0);
}

// FP32 -> 16 bits, round to nearest even (one instruction each on gfx950).
__device__ __forceinline__ uint16_t to_bits(BF16, float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint16_t to_bits(F16, float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ __forceinline__ float from_bits(BF16, uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float from_bits(F16, uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
template <class T>
__device__ __forceinline__ uint32_t pack2(T t, float lo, float hi) {
  return (uint32_t)to_bits(t, lo) | ((uint32_t)to_bits(t, hi) << 16);
}

// FP16 operands made here are lifted into its range by a power of two that the
// FP32 sums lose again: the one that brings their largest size to 2^to .. 2^(to + 1).
__device__ __forceinline__ int lift_bits(float largest, int to) {
  if (largest == 0.f) return 0;
  const int f = to - ((int)(__float_as_uint(largest) >> 23) - 127);
  return f < -112 ? -112 : f > 112 ? 112 : f;
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The largest v of a wave, and of a workgroup of 256; v is not negative.  Lanes
// exchange through registers: neighbours, pairs, the halves of 8 and of 16 mirrored,
// then 16 and 32 lanes swapped (by __shfl_xor, through LDS, 400 x 14336 x 4096 in FP16
// took 95 us, 93 so).
__device__ __forceinline__ float most_of_wave(float v) {
  v = __builtin_fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0xB1, 15, 15, false)));
  v = __builtin_fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x4E, 15, 15, false)));
  v = __builtin_fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x141, 15, 15, false)));
  v = __builtin_fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x140, 15, 15, false)));
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  v = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float most_of_256(float v) {
  __shared__ float top[4];
  v = most_of_wave(v);
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = v;
  __syncthreads();
  return __builtin_fmaxf(__builtin_fmaxf(top[0], top[1]), __builtin_fmaxf(top[2], top[3]));
}

// Wait until all but the N youngest loads of this wave (to LDS too) have landed:
// vmcnt(N), N < 64.
template <int N>
__device__ __forceinline__ void wait_but() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
  asm volatile("" ::: "memory");
}
// A barrier without the waits of __syncthreads; nothing that reads or writes
// memory is moved across it.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Wait until this wave's LDS reads have returned: lgkmcnt(0).
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// 16 bytes a lane from src to dst + 16 lane.  ONCE: non-temporal.
template <bool ONCE = false>
__device__ __forceinline__ void to_lds(const void *src, uint8_t *dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                   (__attribute__((address_space(3))) void *)dst, 16, 0, ONCE ? 2 : 0);
}
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_turned(const uint8_t *p) {
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4 *)(__attribute__((address_space(3))) void *)p);
  return __builtin_bit_cast(u32x2, v);
}

// What a lane past the end of the summed index loads instead.
__device__ const u32x4 g_zero16 = {0, 0, 0, 0};

struct Gemm {
  const uint16_t *a, *b;      // A [m, k] or [k, m], B [n, k] or [k, n]
  uint64_t lda, ldb;          // row strides in elements, multiples of 8
  uint32_t m, n, k;           // [rows, k]: k a multiple of 8; [k, rows]: rows padded to 8
  uint32_t mt, nt;            // tiles
  uint32_t kb_per_split;      // 64-element steps per split of the summed index
  uint32_t first;             // tile of the launch's first workgroup
};

constexpr int kBK = 64;

// Chunk exchange of an LDS row of 64 summed elements (128 bytes): 16 rows read
// at one chunk fall into 16 different places of two rows' span.
__device__ __forceinline__ uint32_t swz(uint32_t row) { return (row >> 1) & 7u; }
// Chunk exchange of an LDS row of R elements at summed index k: a transposing
// read takes 32 bytes (two chunks, so the low bit stays) of rows 8 i + 0..3.
template <int R>
__device__ __forceinline__ uint32_t swz_across(uint32_t k) {
  return R == 32 ? (k >> 2) & 2u : R == 64 ? (k & 2u) | ((k >> 1) & 4u) : ((k & 3u) << 1) | (k & 8u);
}

// Tile of a workgroup.  Workgroups go to the eight XCDs in turn, so XCD id % 8 gets
// a contiguous run of tiles (m fastest), whose B panels its L2 then holds once:
// floor(tiles / 8) of them, and one more in the first tiles % 8 XCDs.
__device__ __forceinline__ uint32_t xcd_tile(uint32_t id, uint32_t tiles) {
  const uint32_t per = tiles / 8, rem = tiles % 8, x = id % 8, l = id / 8;
  return x * per + (x < rem ? x : rem) + l;
}

// One operand of a workgroup's tile: R rows from r0 on.  ACROSS: stored [k, rows].
template <class T, int R, int kWaves, bool ACROSS>
struct Operand {
  static constexpr int kLoads = R / 8 / kWaves;      // of 1 KiB, per wave and step
  static constexpr int kPer = ACROSS ? 512 / R : 8;  // LDS rows a load fills
  const uint8_t *base;
  uint64_t step;  // bytes from one 64-element step to the next
  uint32_t off[kLoads];

  __device__ __forceinline__ void init(const uint16_t *p, uint64_t ld, uint32_t r0, uint32_t total, uint32_t wave,
                                       uint32_t lane) {
    const uint32_t last = total - 1 - r0;  // rows past the end read the last ones, their results are dropped
    base = (const uint8_t *)(ACROSS ? p + r0 : p + r0 * ld);
    step = ACROSS ? ld * (2 * kBK) : 2 * kBK;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      if (ACROSS) {
        const uint32_t k = (i * kWaves + wave) * kPer + lane / (R / 8), c = (lane % (R / 8)) ^ swz_across<R>(k);
        off[i] = k * (uint32_t)ld * 2 + (c < last / 8 ? c : last / 8) * 16;
      } else {
        const uint32_t r = (i * kWaves + wave) * 8 + lane / 8;
        off[i] = (r < last ? r : last) * (uint32_t)ld * 2 + ((lane & 7) ^ swz(r)) * 16;
      }
    }
  }
  // left: summed elements from this step on
  __device__ __forceinline__ void load(uint32_t kb, uint32_t left, uint8_t *dst, uint32_t wave, uint32_t lane) const {
    const uint8_t *src = base + kb * step;
    if (left >= kBK) {
#pragma unroll
      for (int i = 0; i < kLoads; i++) to_lds(src + off[i], dst + (i * kWaves + wave) * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const uint32_t row = (i * kWaves + wave) * kPer;
        const uint32_t k = ACROSS ? row + lane / (R / 8) : ((lane & 7) ^ swz(row + lane / 8)) * 8;
        to_lds(k < left ? src + off[i] : (const uint8_t *)&g_zero16, dst + (i * kWaves + wave) * 1024);
      }
    }
  }
};

// A wave's fragments of an operand: COUNT times 16 rows from LDS row r on.
template <class T, int R, int COUNT, bool ACROSS>
struct Fragments {
  uint32_t at[ACROSS ? COUNT : 2];
  __device__ __forceinline__ void init(uint32_t r, uint32_t lane) {
    const uint32_t lr = lane & 15, kg = lane >> 4;
    if constexpr (ACROSS) {
      const uint32_t k = kg * 8 + lr / 4, f = swz_across<R>(k);
#pragma unroll
      for (int i = 0; i < COUNT; i++)
        at[i] = k * (R * 2) + (((r / 8 + 2 * i) ^ f) + ((lr >> 1) & 1)) * 16 + (lr & 1) * 8;
    } else {
      at[0] = (r + lr) * 128 + (kg ^ swz(lr)) * 16;
      at[1] = (r + lr) * 128 + ((4 + kg) ^ swz(lr)) * 16;
    }
  }
  // fragment i of the step's first or second 32 elements
  __device__ __forceinline__ u32x4 get(const uint8_t *p, int ks, int i) const {
    if constexpr (ACROSS) {
      // rows k .. k + 3 and k + 4 .. k + 7 of this lane's 8; f(k + 4) = f(k), f(k + 32) = f(k)
      const u32x2 lo = read_turned(p + at[i] + ks * (R * 64)), hi = read_turned(p + at[i] + ks * (R * 64) + R * 8);
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
      return *(const u32x4 *)(p + at[ks] + i * 2048);
    }
  }
};

// The step loop keeps the two waves that share a SIMD in opposite phases: half
// of the waves run one barrier late, so one's fragment reads and load requests
// lie under the other's matrix instructions (which go first, s_setprio).  A step
// has two phases, the upper and the lower half of a wave's rows against all its
// columns; each is: read the phase's fragments, request loads, wait for the
// reads, barrier, multiply, barrier.  Requested are, in the first phase of step
// kb, A of step kb + 1 (A of step kb - 1 was last read in the phase before) and,
// in the second, B of step kb + 2 (B of step kb was last read in the first); then
// the wave waits for all but the latter, so step kb + 1 is whole in LDS.  An
// early wave's phase begins after the barrier by which the late waves' reads of
// the phase before have returned, and the other way round, so no request
// overwrites what is still read.
// 2048 x 128256 x 4096: 1614 us (1333 TFLOP/s) against 1787 us with both halves
// in step and one barrier a step; 2048 x 4096 x 14336 in two splits 175 against
// 211 us; with B stored across 218 against 288 us (16384 long).  Four phases a
// step (a quarter of the tile each) 1708 us; 32-element steps in four or five
// buffers 1910 to 2000 us; four waves of 128 x 128 each 2300 us.
template <class T, int BM, int BN, int WM, int WN, bool KA, bool KB, class Epi>
__global__ __launch_bounds__(64 * WM * WN) void gemm(const Gemm g, const Epi epi) {
  constexpr int kWaves = WM * WN;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16, MH = MT / 2;
  constexpr uint32_t kBuf = (BM + BN) * 128;
  typedef Operand<T, BM, kWaves, KA> OA;
  typedef Operand<T, BN, kWaves, KB> OB;
  extern __shared__ __align__(1024) uint8_t lds[];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = xcd_tile(g.first + blockIdx.x, g.mt * g.nt);
  const uint32_t bm = tile % g.mt, bn = tile / g.mt;
  const uint32_t m0 = bm * BM, n0 = bn * BN;
  const uint32_t nkb = (g.k + kBK - 1) / kBK;
  const uint32_t kb0 = blockIdx.y * g.kb_per_split;
  const uint32_t kb1 = kb0 + g.kb_per_split < nkb ? kb0 + g.kb_per_split : nkb;

  OA oa;
  OB ob;
  oa.init(g.a, g.lda, m0, g.m, wave, lane);
  ob.init(g.b, g.ldb, n0, g.n, wave, lane);
  auto buffer = [&](uint32_t kb) { return lds + ((kb - kb0) & 1) * kBuf; };
  auto load_a = [&](uint32_t kb) { oa.load(kb, g.k - kb * kBK, buffer(kb), wave, lane); };
  auto load_b = [&](uint32_t kb) { ob.load(kb, g.k - kb * kBK, buffer(kb) + BM * 128, wave, lane); };
  const uint32_t wm = wave % WM, wn = wave / WM;
  Fragments<T, BM, MT, KA> la;
  Fragments<T, BN, NT, KB> lb;
  la.init(wm * (BM / WM), lane);
  lb.init(wn * (BN / WN), lane);
  f32x4 acc[NT][MT] = {};
  u32x4 fa[2][MH], fb[2][NT];  // by 32 elements of the step
  auto fetch_a = [&](const uint8_t *p, int h) {
#pragma unroll
    for (int ks = 0; ks < 2; ks++)
#pragma unroll
      for (int i = 0; i < MH; i++) fa[ks][i] = la.get(p, ks, h * MH + i);
  };
  auto multiply = [&](int h) {
    wait_reads();
    meet();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int ks = 0; ks < 2; ks++)
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < MH; i++)
          acc[j][h * MH + i] = mfma(T{}, fb[ks][j], fa[ks][i], acc[j][h * MH + i]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    meet();
  };
  if (kb0 < kb1) {
    load_a(kb0);
    load_b(kb0);
    if (kb0 + 1 < kb1) {
      load_a(kb0 + 1);
      load_b(kb0 + 1);
      wait_but<OA::kLoads + OB::kLoads>();
    } else {
      wait_but<0>();
    }
    meet();
    const bool late = wave >= kWaves / 2;
    if (late) meet();
    for (uint32_t kb = kb0; kb < kb1; kb++) {
      const uint8_t *p = buffer(kb);
      fetch_a(p, 0);
#pragma unroll
      for (int ks = 0; ks < 2; ks++)
#pragma unroll
        for (int j = 0; j < NT; j++) fb[ks][j] = lb.get(p + BM * 128, ks, j);
      if (kb > kb0 && kb + 1 < kb1) load_a(kb + 1);
      multiply(0);
      fetch_a(p, 1);
      if (kb + 2 < kb1) {
        load_b(kb + 2);
        wait_but<OB::kLoads>();
      } else {
        wait_but<0>();
      }
      multiply(1);
    }
    if (!late) meet();
  }
  // lane: rows m = .. + i*16 + lane % 16, columns n = .. + j*16 + lane / 16 * 4 + 0..3
  epi.template operator()<T, NT, MT>(acc, m0 + wm * (BM / WM) + (lane & 15), n0 + wn * (BN / WN) + (lane >> 4) * 4, g.m,
                                     g.n, bn * WN + wn, blockIdx.y);
}

// ----------------------------------------------------------------- epilogues
// A lane has 4 consecutive columns of a 16-column block (8 bytes in 16 bits).  Two
// neighbouring blocks' words exchanged between lane groups 2 i and 2 i + 1 give
// each lane 8 consecutive columns of one block: block j (even group) or j + 1
// (odd group), columns 8 (group / 2) .. + 7.  Half as many stores, of 16 bytes.
__device__ __forceinline__ u32x4 pair_blocks(u32x2 a, u32x2 b) {
  const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false));
  const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false));
  return u32x4{lo[0], hi[0], lo[1], hi[1]};
}
// Eight 16-bit columns from `col` on into a row of n that starts at p.
__device__ __forceinline__ void store8(uint16_t *p, uint32_t col, uint32_t n, bool aligned, u32x4 v) {
  if (aligned && col + 8 <= n) {
    *(u32x4 *)(p + col) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (col + e < n) p[col + e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
  }
}

// 16-bit output (base 16-byte aligned), times *scale (null: 1) * *scale2 * mul,
// and column n times columns[n] where COLUMNS.
template <bool COLUMNS = false>
struct EpiStore {
  uint16_t *c;
  uint64_t ldc;
  const float *scale, *scale2;
  float mul;
  const float *columns;
  template <class T, int NT, int MT>
  __device__ __forceinline__ void operator()(f32x4 (&acc)[NT][MT], uint32_t mb, uint32_t nb, uint32_t m, uint32_t n,
                                             uint32_t, uint32_t) const {
    static_assert(NT % 2 == 0, "blocks in pairs");
    const float s = (scale ? *scale * *scale2 : 1.f) * mul;
    const bool aligned = (ldc & 7) == 0;
    const uint32_t kg = (threadIdx.x >> 4) & 3, first = nb - 4 * kg + (kg & 1) * 16 + (kg >> 1) * 8;
    f32x4 f[NT];
    if constexpr (COLUMNS) {
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) f[j][e] = nb + j * 16 + e < n ? columns[nb + j * 16 + e] * s : 0.f;
    }
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const uint32_t row = mb + i * 16;
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        f32x4 v, w;
        if constexpr (COLUMNS) {
          v = acc[j][i] * f[j];
          w = acc[j + 1][i] * f[j + 1];
        } else {
          v = acc[j][i] * s;
          w = acc[j + 1][i] * s;
        }
        const u32x4 o = pair_blocks(u32x2{pack2(T{}, v[0], v[1]), pack2(T{}, v[2], v[3])},
                                    u32x2{pack2(T{}, w[0], w[1]), pack2(T{}, w[2], w[3])});
        if (row < m) store8(c + (uint64_t)row * ldc, first + j * 16, n, aligned, o);
      }
    }
  }
};

// FP32 partial planes [split][..][ld], `stride` elements each, stored or added
// to; ld is n rounded up to a multiple of 4.
struct EpiPlane {
  float *c;
  uint32_t ld;
  uint64_t stride;
  bool add;
  EpiPlane from_row(uint32_t r) const { return EpiPlane{c + (uint64_t)r * ld, ld, stride, add}; }
  template <class T, int NT, int MT>
  __device__ __forceinline__ void operator()(f32x4 (&acc)[NT][MT], uint32_t mb, uint32_t nb, uint32_t m, uint32_t n,
                                             uint32_t, uint32_t split) const {
    float *plane = c + split * stride;
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const uint32_t row = mb + i * 16;
      if (row >= m) continue;
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const uint32_t col = nb + j * 16;
        if (col >= n) continue;
        f32x4 *p = (f32x4 *)(plane + (uint64_t)row * ld + col);
        *p = add ? *p + acc[j][i] : acc[j][i];
      }
    }
  }
};

// Four columns of `count` planes added up, eight loads in flight.
__device__ __forceinline__ f32x4 add_planes(const float *p, uint64_t stride, uint32_t count) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  uint32_t s = 0;
  for (; s + 8 <= count; s += 8) {
    f32x4 t[8];
#pragma unroll
    for (int i = 0; i < 8; i++) t[i] = *(const f32x4 *)(p + (s + i) * stride);
#pragma unroll
    for (int i = 0; i < 8; i++) v += t[i];
  }
  for (; s < count; s++) v += *(const f32x4 *)(p + s * stride);
  return v;
}

// ------------------------------------------------------------------- launch
// Raises a kernel's LDS limit where a launch needs more than 64 KiB, once per
// kernel and device: to all that a CU has, less what the kernel declares itself.
[[maybe_unused]] hipError_t allow_lds(const void *fn, uint32_t bytes, uint32_t declared = 0) {
  if (bytes + declared <= 65536) return hipSuccess;
  static std::mutex mu;
  static std::map<std::pair<int, const void *>, bool> raised;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  try {
    std::lock_guard<std::mutex> lk(mu);
    bool &have = raised[{dev, fn}];
    if (!have) {
      e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024 - declared);
      have = e == hipSuccess;
    }
  } catch (...) {  // nothing throws across the C entries
    e = hipErrorOutOfMemory;
  }
  return e;
}

template <class T, int BM, int BN, int WM, int WN, bool KA, bool KB, class Epi>
hipError_t gemm_launch(Gemm g, const Epi &epi, uint32_t splits, hipStream_t stream) {
  constexpr uint32_t lds = 2 * (BM + BN) * 128;
  g.mt = (g.m + BM - 1) / BM;
  g.nt = (g.n + BN - 1) / BN;
  const uint32_t nkb = (g.k + kBK - 1) / kBK;
  g.kb_per_split = (nkb + splits - 1) / splits;
  const hipError_t e = allow_lds((const void *)gemm<T, BM, BN, WM, WN, KA, KB, Epi>, lds);
  if (e != hipSuccess) return e;
  // a launch holds fewer than 2^32 threads: 2^21 rows of 2^18 columns are 2^23 tiles
  const uint32_t tiles = g.mt * g.nt, most = 1u << 22;
  for (g.first = 0; g.first < tiles; g.first += most) {
    const uint32_t count = tiles - g.first < most ? tiles - g.first : most;
    hipLaunchKernelGGL((gemm<T, BM, BN, WM, WN, KA, KB, Epi>), dim3(count, splits), dim3(64 * WM * WN), lds, stream, g,
                       epi);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  return hipSuccess;
}

// The tiles a product is cut into.
struct Shape {
  uint32_t bm, bn, waves_n, slots;  // slots: workgroups that the chip holds at once
  double step;                      // us a step of 64 summed elements takes with all slots busy
};
constexpr Shape kShapes[5] = {{256, 256, 4, 256, 1.7}, {128, 128, 2, 512, 1.2}, {64, 64, 2, 1024, 1.2},
                              {64, 128, 4, 768, 1.3}, {32, 128, 4, 1024, 1.2}};
template <class T, bool KA, bool KB, class Epi>
hipError_t product(const Gemm &g, const Epi &e, uint32_t shape, uint32_t splits, hipStream_t s) {
  switch (shape) {
    case 0: return gemm_launch<T, 256, 256, 2, 4, KA, KB>(g, e, splits, s);
    case 1: return gemm_launch<T, 128, 128, 2, 2, KA, KB>(g, e, splits, s);
    case 2: return gemm_launch<T, 64, 64, 2, 2, KA, KB>(g, e, splits, s);
    case 3: return gemm_launch<T, 64, 128, 1, 4, KA, KB>(g, e, splits, s);
    default: return gemm_launch<T, 32, 128, 1, 4, KA, KB>(g, e, splits, s);
  }
}

uint64_t up(uint64_t v, uint64_t to) { return (v + to - 1) / to * to; }

// Shape and splits of the summed index for a product, by what its workgroups
// take: rounds of `slots` of them, each its steps plus 4 us to start and end, and
// 4 us plus the planes' traffic at 4 TB/s to join splits; B is read at 5 TB/s at
// most.  A split keeps at least eight steps.  Few rows take a flat tile: they are
// bound by reading B, which 128 rows a workgroup ask for in longer runs and with
// less of A beside it.
struct Cut {
  uint32_t shape, splits;
  double us;
};
Cut cut_for(uint64_t m, uint64_t n, uint64_t k, bool may_split) {
  const uint64_t steps = up(k, kBK) / kBK;
  Cut best = {2, 1, 1e30};
  const int from = m <= 32 ? 4 : m <= 64 ? 3 : 0, to = m <= 32 ? 4 : m <= 64 ? 3 : 2;
  for (int i = from; i <= to; i++) {
    const Shape &sh = kShapes[i];
    const uint64_t tiles = up(m, sh.bm) / sh.bm * (up(n, sh.bn) / sh.bn);
    // one split, powers of two, and as many as fill one round or two
    const uint32_t full = (uint32_t)(sh.slots / tiles), twice = (uint32_t)(2 * sh.slots / tiles);
    for (uint32_t q = 0; q < 8; q++) {
      const uint32_t s = q < 6 ? 1u << q : q == 6 ? full : twice;
      if (s < 1 || s > 32 || (s > 1 && (!may_split || steps / s < 8))) continue;
      double t = (double)up(tiles * s, sh.slots) / sh.slots * ((double)((steps + s - 1) / s) * sh.step + 4.0);
      const double read = 2.0 * (double)n * (double)k / 5e6 + 4.0;
      if (t < read) t = read;
      if (s > 1) t += 4.0 + 8e-6 * (double)(m * n * s) / 4.0;
      if (t < best.us) best = Cut{(uint32_t)i, s, t};
    }
  }
  return best;
}

// The same for a product whose rows may go in two launches: whole tiles of 256
// rows, and up to 64 rows behind them in flat tiles, where that takes less (517
// x 32003 x 2056: a third row of tiles for 5 rows costs a second round, 111 us
// against 57 + 25).  rest.us is 0 where there is one launch.
struct RowCut {
  uint32_t rows;  // in the first launch
  Cut main, rest;
};
[[maybe_unused]] RowCut rows_for(uint64_t m, uint64_t n, uint64_t k, bool may_split) {
  RowCut c = {(uint32_t)m, cut_for(m, n, k, may_split), {0, 0, 0.0}};
  const uint32_t r = (uint32_t)(m % 256);
  if (m > 256 && r && r <= 64) {
    const Cut a = cut_for(m - r, n, k, may_split), b = cut_for(r, n, k, may_split);
    if (a.us + b.us < c.main.us) c = RowCut{(uint32_t)m - r, a, b};
  }
  return c;
}
template <class T, bool KB, class Epi>
hipError_t product_rows(const Gemm &g, const Epi &e, const RowCut &c, hipStream_t s) {
  Gemm f = g;
  f.m = c.rows;
  const hipError_t st = product<T, false, KB>(f, e, c.main.shape, c.main.splits, s);
  if (st != hipSuccess || c.rest.us == 0.0) return st;
  f.m = g.m - c.rows;
  f.a = g.a + (uint64_t)c.rows * g.lda;
  return product<T, false, KB>(f, e.from_row(c.rows), c.rest.shape, c.rest.splits, s);
}

}  // namespace
}  // namespace dfh

#endif
