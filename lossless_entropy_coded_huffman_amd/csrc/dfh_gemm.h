// Tiled products on the matrix cores for gfx950, shared by the uint4 linear
// operators and the vocabulary losses.
//
//   C[m, n] = sum_k A[m, k] B[n, k]
//
// Both operands are row major with the summed index contiguous, in BF16 or
// FP16; sums are FP32.  Products that sum over another index get a transposed
// copy of the operand (made in the caller's workspace), so one kernel serves
// every direction.
//
// gemm_nt: one workgroup makes a BM x BN tile.  Each step takes 64 summed
// elements (128 bytes) of BM + BN rows from global memory straight into LDS
// (16 bytes a lane, no registers in between) into one of two buffers, while
// the waves run v_mfma_f32_16x16x32 from the other.  A row's eight 16-byte
// chunks are stored at position chunk ^ swz(row): the load writes LDS linearly,
// so the exchange is made in the source address, and the 16 rows that a
// fragment read touches at one chunk fall into different banks.
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

struct BF16 {};
struct F16 {};

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

// Wait until every load of this wave (to LDS too) has landed: vmcnt(0).
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// What a lane past the end of the summed index loads instead.
__device__ const u32x4 g_zero16 = {0, 0, 0, 0};

struct Gemm {
  const uint16_t *a, *b;      // A [m, k], B [n, k]
  uint64_t lda, ldb;          // row strides in elements, multiples of 8
  uint32_t m, n, k;           // k a multiple of 8
  uint32_t mt, nt;            // tiles
  uint32_t kb_per_split;      // 64-element steps per split of the summed index
};

constexpr int kBK = 64;

// Chunk exchange of an LDS row.
__device__ __forceinline__ uint32_t swz(uint32_t row) { return (row >> 1) & 7u; }

// Tile of a workgroup.  Workgroups go to the eight XCDs in turn, so workgroup
// id works on tile (id % 8) * ceil(tiles / 8) + id / 8: an XCD gets a contiguous
// run of tiles (m fastest), whose B panels its L2 then holds once.
__device__ __forceinline__ uint32_t xcd_tile(uint32_t id, uint32_t tiles) {
  const uint32_t per = tiles / 8, rem = tiles % 8, x = id % 8, l = id / 8;
  return x * per + (x < rem ? x : rem) + l;
}

template <class T, int BM, int BN, int WM, int WN, class Epi>
__global__ __launch_bounds__(64 * WM * WN) void gemm_nt(const Gemm g, const Epi epi) {
  constexpr int kWaves = WM * WN;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int kRows = BM + BN;
  constexpr int kLoads = kRows / 8 / kWaves, kLoadsA = BM / 8 / kWaves;
  static_assert(kRows % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "whole loads per wave");
  extern __shared__ __align__(1024) uint8_t lds[];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = xcd_tile(blockIdx.x, g.mt * g.nt);
  const uint32_t bm = tile % g.mt, bn = tile / g.mt;
  const uint32_t m0 = bm * BM, n0 = bn * BN;
  const uint32_t nkb = (g.k + kBK - 1) / kBK;
  const uint32_t kb0 = blockIdx.y * g.kb_per_split;
  const uint32_t kb1 = kb0 + g.kb_per_split < nkb ? kb0 + g.kb_per_split : nkb;

  // source of this lane's chunks: the tile's first row (uniform) plus a 32-bit
  // byte offset; rows past the end read the last row (their results are dropped)
  const uint8_t *pa = (const uint8_t *)(g.a + (uint64_t)m0 * g.lda);
  const uint8_t *pb = (const uint8_t *)(g.b + (uint64_t)n0 * g.ldb);
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; i++) {
    const bool isa = i < kLoadsA;
    const uint32_t r = ((isa ? i : i - kLoadsA) * kWaves + wave) * 8 + lane / 8;
    const uint32_t last = isa ? g.m - 1 - m0 : g.n - 1 - n0;
    const uint32_t rr = r < last ? r : last;
    off[i] = rr * (uint32_t)(isa ? g.lda : g.ldb) * 2 + ((lane & 7) ^ swz(r)) * 16;
  }
  auto load = [&](uint32_t kb, uint32_t buf) {
    uint8_t *dst = lds + buf * (kRows * 128);
    const uint64_t kbyte = (uint64_t)kb * (kBK * 2);
    const uint32_t left = g.k - kb * kBK;  // summed elements from here on
    if (left >= kBK) {
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const uint8_t *src = (i < kLoadsA ? pa : pb) + kbyte + off[i];
        const uint32_t row = i < kLoadsA ? (i * kWaves + wave) * 8 : BM + ((i - kLoadsA) * kWaves + wave) * 8;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                         (__attribute__((address_space(3))) void *)(dst + row * 128), 16, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; i++) {
        const uint32_t row = i < kLoadsA ? (i * kWaves + wave) * 8 : BM + ((i - kLoadsA) * kWaves + wave) * 8;
        const uint32_t rl = row - (i < kLoadsA ? 0 : BM) + lane / 8;
        const uint32_t c = (lane & 7) ^ swz(rl);
        const uint8_t *src = (i < kLoadsA ? pa : pb) + kbyte + off[i];
        src = c * 8 < left ? src : (const uint8_t *)&g_zero16;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                         (__attribute__((address_space(3))) void *)(dst + row * 128), 16, 0, 0);
      }
    }
  };

  const uint32_t wm = wave % WM, wn = wave / WM;
  const uint32_t lr = lane & 15, kg = lane >> 4;
  // byte offset of this lane's fragment chunks (first and second 32 elements)
  const uint32_t c0 = (kg ^ swz(lr)) * 16, c1 = ((4 + kg) ^ swz(lr)) * 16;
  const uint32_t ra = (wm * (BM / WM) + lr) * 128, rb = (BM + wn * (BN / WN) + lr) * 128;
  f32x4 acc[NT][MT] = {};
  if (kb0 < kb1) load(kb0, 0);
  wait_loads();
  __syncthreads();
  for (uint32_t kb = kb0; kb < kb1; kb++) {
    const uint32_t buf = (kb - kb0) & 1;
    if (kb + 1 < kb1) load(kb + 1, buf ^ 1);
    const uint8_t *p = lds + buf * (kRows * 128);
#pragma unroll
    for (int ks = 0; ks < 2; ks++) {
      const uint32_t c = ks ? c1 : c0;
      u32x4 fa[MT], fb[NT];
#pragma unroll
      for (int i = 0; i < MT; i++) fa[i] = *(const u32x4 *)(p + ra + i * 2048 + c);
#pragma unroll
      for (int j = 0; j < NT; j++) fb[j] = *(const u32x4 *)(p + rb + j * 2048 + c);
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < MT; i++) acc[j][i] = mfma(T{}, fb[j], fa[i], acc[j][i]);
    }
    wait_loads();  // this wave's part of the next buffer is in LDS
    __syncthreads();
  }
  // lane: rows m = .. + i*16 + lr, columns n = .. + j*16 + kg*4 + 0..3
  epi.template operator()<T, NT, MT>(acc, m0 + wm * (BM / WM) + lr, n0 + wn * (BN / WN) + kg * 4, g.m, g.n,
                                     bn * WN + wn, blockIdx.y);
}

// ----------------------------------------------------------------- epilogues
// 16-bit output, times *scale * mul.
struct EpiStore {
  uint16_t *c;
  uint64_t ldc;
  const float *scale;  // null: 1
  float mul;
  template <class T, int NT, int MT>
  __device__ __forceinline__ void operator()(f32x4 (&acc)[NT][MT], uint32_t mb, uint32_t nb, uint32_t m, uint32_t n,
                                             uint32_t, uint32_t) const {
    const float s = (scale ? *scale : 1.f) * mul;
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const uint32_t row = mb + i * 16;
      if (row >= m) continue;
      uint16_t *p = c + (uint64_t)row * ldc;
      const bool al = ((ldc & 3) == 0);
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const uint32_t col = nb + j * 16;
        const f32x4 v = acc[j][i] * s;
        if (al && col + 4 <= n) {
          *(u32x2 *)(p + col) = u32x2{pack2(T{}, v[0], v[1]), pack2(T{}, v[2], v[3])};
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (col + e < n) p[col + e] = to_bits(T{}, v[e]);
        }
      }
    }
  }
};

// FP32 partial planes [split][m][ld], stored or added to; ld is n rounded up
// to a multiple of 4.
struct EpiPlane {
  float *c;
  uint32_t ld;
  bool add;
  template <class T, int NT, int MT>
  __device__ __forceinline__ void operator()(f32x4 (&acc)[NT][MT], uint32_t mb, uint32_t nb, uint32_t m, uint32_t n,
                                             uint32_t, uint32_t split) const {
    float *plane = c + (uint64_t)split * m * ld;
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

// ------------------------------------------------------------------- launch
// Raises a kernel's LDS limit where a launch needs more than 64 KiB, once per
// kernel and device.
hipError_t allow_lds(const void *fn, uint32_t bytes) {
  if (bytes <= 65536) return hipSuccess;
  static std::mutex mu;
  static std::map<std::pair<int, const void *>, bool> raised;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  try {
    std::lock_guard<std::mutex> lk(mu);
    bool &have = raised[{dev, fn}];
    if (!have) {
      e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
      have = e == hipSuccess;
    }
  } catch (...) {  // nothing throws across the C entries
    e = hipErrorOutOfMemory;
  }
  return e;
}

template <class T, int BM, int BN, int WM, int WN, class Epi>
hipError_t gemm_launch(Gemm g, const Epi &epi, uint32_t splits, hipStream_t stream) {
  constexpr uint32_t lds = 2 * (BM + BN) * 128;
  g.mt = (g.m + BM - 1) / BM;
  g.nt = (g.n + BN - 1) / BN;
  const uint32_t nkb = (g.k + kBK - 1) / kBK;
  g.kb_per_split = (nkb + splits - 1) / splits;
  const hipError_t e = allow_lds((const void *)gemm_nt<T, BM, BN, WM, WN, Epi>, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gemm_nt<T, BM, BN, WM, WN, Epi>), dim3(g.mt * g.nt, splits), dim3(64 * WM * WN), lds, stream, g,
                     epi);
  return hipGetLastError();
}

}  // namespace
}  // namespace dfh

#endif
