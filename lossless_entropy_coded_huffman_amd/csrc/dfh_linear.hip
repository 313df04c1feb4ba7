// Products with uint4 weights and group scales (gfx950).
//
//   y[m, n]  = sum_k x[m, k] s[n, g] (q[n, k] - z[n, g]),   g = k / group
//   dx[m, k] = sum_n dy[m, n] s[n, g] (q[n, k] - z[n, g])
//
// The weights are the packed nibbles that a uint4 container decodes to: the
// element n * cols + k, two per byte, the even one in the low nibble.
//
// Few rows (up to 64): u4_rows reads the nibbles once and feeds the matrix
// cores with the integers themselves; the scale multiplies a group's FP32 sum.
// More rows: the weights are expanded to 16 bits in the caller's workspace and
// gemm_nt does the product.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

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
__device__ __forceinline__ float zero_at(const U4 &w, uint32_t n, uint32_t g) {
  return w.zeros ? (float)w.zeros[n * w.zstride + g] : 8.f;
}

// Eight nibbles -> eight 16-bit floats bias + q, in the order of elements
// 0,4 1,5 2,6 3,7: the nibble lands in the low mantissa bits of a constant
// whose unit in the last place is one (BF16 128, FP16 1024), so a pair costs
// one shift and one and-or.  FP16 then takes 1024 + z off each pair with one
// packed addition, exactly; there is no such addition for BF16, whose bias
// (and zero point) come off the group's sum instead.
template <class T>
struct Bias;
template <>
struct Bias<BF16> {
  static constexpr uint32_t bits = 0x43004300u;
  static constexpr float value = 128.f;
  static constexpr bool in_sum = true;
};
template <>
struct Bias<F16> {
  static constexpr uint32_t bits = 0x64006400u;
  static constexpr float value = 1024.f;
  static constexpr bool in_sum = false;
};
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
// off: the pair of -(1024 + z), FP16 only
template <class T>
__device__ __forceinline__ u32x4 widen(uint32_t w, uint32_t off) {
  constexpr uint32_t m = 0x000F000Fu, b = Bias<T>::bits;
  u32x4 v = {(w & m) | b, ((w >> 4) & m) | b, ((w >> 8) & m) | b, ((w >> 12) & m) | b};
  if constexpr (!Bias<T>::in_sum) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t e = v[i];
      v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, e) + __builtin_bit_cast(f16x2, off));
    }
  }
  return v;
}
// Eight consecutive 16-bit values into the same order.
__device__ __forceinline__ u32x4 pair_up(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
               __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

// One output from the definition, in order; taken where BF16's fast sum is not
// finite (an infinite or very large x: the bias would turn inf * w into NaN).
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
  }
  return acc;
}

// y for up to 16 MT rows.  A workgroup makes 16 NT columns; its waves share
// the summed index (blocks of 128 go to them in turn) and add up through LDS.
// Matrix operand A is x (16 rows), B the weights (16 columns n): lane l loads
// 16 bytes of weight row l % 16, elements 32 (l / 16) .. + 31 of the block, and
// two exchange steps between the lane groups give every 32-element step of the
// block to one matrix instruction, so a scale may change every 32 elements.
// BF16: T = sum x (bias + q) and S = sum x (B operand all ones) give a group's
// part as s (T - (bias + z) S), in FP32; FP16: T = sum x (q - z) and s T.
template <class T, int MT, int NT, int W, int U, bool kSub, bool kWide>
__global__ __launch_bounds__(64 * W) void u4_rows(const U4 w, const uint16_t *x, uint64_t xs, uint32_t m,
                                                  uint16_t *y) {
  __shared__ f32x4 part[W][NT * MT][64];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lr = lane & 15, kg = lane >> 4;
  const uint32_t n0 = blockIdx.x * (16 * NT);
  const uint32_t nkb = (w.k + 127) / 128;
  constexpr int G = kSub ? 4 : 1;
  const uint32_t one = (uint32_t)to_bits(T{}, 1.f) * 0x10001u;
  const u32x4 ones = {one, one, one, one};
  const uint8_t *prow[NT];
  uint32_t nn[NT];
#pragma unroll
  for (int j = 0; j < NT; j++) {
    const uint32_t n = n0 + j * 16 + lr;
    nn[j] = n < w.n ? n : w.n - 1;
    prow[j] = w.packed + (uint64_t)nn[j] * (w.k / 2) + kg * 16;
  }
  const uint16_t *px[MT];
#pragma unroll
  for (int i = 0; i < MT; i++) px[i] = x + (uint64_t)(i * 16 + lr) * xs + kg * 8;

  f32x4 acc[NT][MT] = {};
  for (uint32_t kb = wave; kb < nkb; kb += W * U) {
    u32x4 qw[U][NT], xv[U][MT][4];
    float sc[U][NT][G], ze[U][NT][G];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t b = kb + u * W;
      const uint32_t k0 = b * 128;
#pragma unroll
      for (int j = 0; j < NT; j++) {
        qw[u][j] = u32x4{0, 0, 0, 0};
        if (kWide) {
          if (k0 + kg * 32 < w.k) qw[u][j] = __builtin_nontemporal_load((const u32x4 *)(prow[j] + (uint64_t)b * 64));
        } else {
#pragma unroll
          for (int d = 0; d < 4; d++)
            if (k0 + kg * 32 + d * 8 < w.k) qw[u][j][d] = *(const uint32_t *)(prow[j] + (uint64_t)b * 64 + d * 4);
        }
#pragma unroll
        for (int g = 0; g < G; g++) {
          sc[u][j][g] = 0.f;
          ze[u][j][g] = 0.f;
          if (k0 + g * 32 < w.k) {
            const uint32_t gi = group_of(w, b * 4 + g);
            sc[u][j][g] = scale_at(w, nn[j], gi);
            ze[u][j][g] = zero_at(w, nn[j], gi);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < MT; i++)
#pragma unroll
        for (int d = 0; d < 4; d++) {
          xv[u][i][d] = u32x4{0, 0, 0, 0};
          if (i * 16 + lr < m && k0 + d * 32 + kg * 8 < w.k) xv[u][i][d] = *(const u32x4 *)(px[i] + k0 + d * 32);
        }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (kb + u * W >= nkb) break;  // uniform
      u32x4 xp[MT][4];
      f32x4 sx[MT][G] = {};
#pragma unroll
      for (int i = 0; i < MT; i++)
#pragma unroll
        for (int d = 0; d < 4; d++) {
          xp[i][d] = pair_up(xv[u][i][d]);
          if constexpr (Bias<T>::in_sum) sx[i][kSub ? d : 0] = mfma(T{}, xp[i][d], ones, sx[i][kSub ? d : 0]);
        }
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const u32x4 q = qw[u][j];
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(q[0], q[2], false, false));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(q[1], q[3], false, false));
        const u32x2 c = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false));
        const u32x2 e = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false));
        const uint32_t step[4] = {c[0], c[1], e[0], e[1]};
        f32x4 t[MT][G] = {};
#pragma unroll
        for (int d = 0; d < 4; d++) {
          uint32_t off = 0;
          if constexpr (!Bias<T>::in_sum) off = to_bits(T{}, -(Bias<T>::value + ze[u][j][kSub ? d : 0])) * 0x10001u;
          const u32x4 f = widen<T>(step[d], off);
#pragma unroll
          for (int i = 0; i < MT; i++) t[i][kSub ? d : 0] = mfma(T{}, xp[i][d], f, t[i][kSub ? d : 0]);
        }
#pragma unroll
        for (int g = 0; g < G; g++) {
          const float s = sc[u][j][g], z = Bias<T>::value + ze[u][j][g];
#pragma unroll
          for (int i = 0; i < MT; i++)
#pragma unroll
            for (int e4 = 0; e4 < 4; e4++)
              acc[j][i][e4] = __builtin_fmaf(
                  s, Bias<T>::in_sum ? __builtin_fmaf(-z, sx[i][g][e4], t[i][g][e4]) : t[i][g][e4], acc[j][i][e4]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; j++)
#pragma unroll
    for (int i = 0; i < MT; i++) part[wave][j * MT + i][lane] = acc[j][i];
  __syncthreads();
  for (uint32_t t = threadIdx.x; t < NT * MT * 256; t += 64 * W) {
    const uint32_t tile = t / 256, row = (t / 16) & 15, col = t & 15;  // row of x, column n
    const uint32_t src = (row / 4) * 16 + col;                         // the lane that holds it
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < W; q++) v += ((const float *)&part[q][tile][src])[row & 3];
    const uint32_t mm = (tile % MT) * 16 + row, n = n0 + (tile / MT) * 16 + col;
    if (mm < m && n < w.n) {
      if (Bias<T>::in_sum && !(__builtin_fabsf(v) < __builtin_huge_valf())) v = dot_plain<T>(w, x + (uint64_t)mm * xs, n);
      y[(uint64_t)mm * w.n + n] = to_bits(T{}, v);
    }
  }
}

// The weights as 16-bit floats, [n, k].  Each is rounded once from FP32
// (relative 2^-8 / 2^-11 at most); the sums over them are FP32.
template <class T>
__global__ __launch_bounds__(256) void u4_expand(const U4 w, uint16_t *out) {
  const uint32_t n = blockIdx.x;
  for (uint32_t c = threadIdx.x; c < w.k / 8; c += 256) {
    const uint64_t at = (uint64_t)n * (w.k / 8) + c;
    const uint32_t q = ((const uint32_t *)w.packed)[at];
    const uint32_t g = group_of(w, c / 4);
    const float s = scale_at(w, n, g), z = zero_at(w, n, g);
    u32x4 o;
#pragma unroll
    for (int d = 0; d < 4; d++)
      o[d] = pack2(T{}, ((float)((q >> (8 * d)) & 15u) - z) * s, ((float)((q >> (8 * d + 4)) & 15u) - z) * s);
    ((u32x4 *)out)[at] = o;
  }
}

// The same, transposed: [k, np] with np = n rounded up to 8 (zeros past n).
// 64 x 64 tiles through LDS, whose rows are padded by two elements so that the
// column writes spread over the banks.
template <class T>
__global__ __launch_bounds__(256) void u4_expand_t(const U4 w, uint16_t *out, uint32_t np) {
  __shared__ uint16_t tile[64][72];  // [k][n]
  const uint32_t n0 = blockIdx.x * 64, k0 = blockIdx.y * 64;
  for (uint32_t t = threadIdx.x; t < 512; t += 256) {
    const uint32_t r = t / 8, c = t % 8, n = n0 + r, k = k0 + c * 8;
    uint32_t q = 0;
    float s = 0.f, z = 0.f;
    if (n < w.n && k < w.k) {
      q = *(const uint32_t *)(w.packed + ((uint64_t)n * w.k + k) / 2);
      const uint32_t g = group_of(w, k / 32);
      s = scale_at(w, n, g);
      z = zero_at(w, n, g);
    }
#pragma unroll
    for (int d = 0; d < 8; d++) tile[c * 8 + d][r] = to_bits(T{}, ((float)((q >> (4 * d)) & 15u) - z) * s);
  }
  __syncthreads();
  for (uint32_t t = threadIdx.x; t < 512; t += 256) {
    const uint32_t kk = t / 8, c = t % 8, k = k0 + kk, n = n0 + c * 8;
    if (k < w.k && n < np) *(u32x4 *)(out + (uint64_t)k * np + n) = *(const u32x4 *)&tile[kk][c * 8];
  }
}

// Sum of FP32 planes [splits][m][ld] -> 16-bit [m, n].
template <class T>
__global__ __launch_bounds__(256) void join_planes(const float *p, uint32_t splits, uint32_t m, uint32_t n,
                                                   uint32_t ld, uint16_t *out) {
  const uint32_t row = blockIdx.x;
  for (uint32_t c = threadIdx.x * 4; c < n; c += 1024) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t s = 0; s < splits; s++) v += *(const f32x4 *)(p + ((uint64_t)s * m + row) * ld + c);
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (c + e < n) out[(uint64_t)row * n + c + e] = to_bits(T{}, v[e]);
  }
}

// Rows of n elements into rows of np (n rounded up to 8), zeros past n.
__global__ __launch_bounds__(256) void pad_rows(const uint16_t *src, uint64_t ss, uint32_t n, uint32_t np,
                                                uint16_t *dst) {
  const uint64_t r = blockIdx.x;
  for (uint32_t c = threadIdx.x; c < np; c += 256) dst[r * np + c] = c < n ? src[r * ss + c] : (uint16_t)0;
}

constexpr uint32_t kFewRows = 64;

uint64_t up(uint64_t v, uint64_t to) { return (v + to - 1) / to * to; }

// Splits of the summed index for an output of m x n: enough workgroups of
// 64 x 64 tiles for two per CU, with four 64-element steps each at least.
uint32_t splits_for(uint32_t m, uint32_t n, uint32_t k) {
  const uint64_t tiles = up(m, 64) / 64 * (up(n, 64) / 64);
  if (tiles >= 256) return 1;
  const uint64_t most = up(k, 256) / 256;
  const uint64_t want = (512 + tiles - 1) / tiles;
  return (uint32_t)(want < most ? want : most < 1 ? 1 : most);
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
  return DF_OK;
}

template <class T, class Epi>
hipError_t product(const Gemm &g, const Epi &e, uint32_t splits, hipStream_t s) {
  if (splits > 1) return gemm_launch<T, 64, 64, 2, 2>(g, e, splits, s);
  if ((uint64_t)(up(g.m, 256) / 256) * (up(g.n, 256) / 256) >= 192) return gemm_launch<T, 256, 256, 2, 4>(g, e, 1, s);
  if ((uint64_t)(up(g.m, 128) / 128) * (up(g.n, 128) / 128) >= 192) return gemm_launch<T, 128, 128, 2, 2>(g, e, 1, s);
  return gemm_launch<T, 64, 64, 2, 2>(g, e, 1, s);
}

template <class T>
df_status many_rows(const Gemm &g, uint16_t *out, float *planes, hipStream_t s) {
  const uint32_t splits = splits_for(g.m, g.n, g.k);
  if (splits <= 1)
    return product<T>(g, EpiStore{out, g.n, nullptr, 1.f}, 1, s) == hipSuccess ? DF_OK : DF_ERR_HIP;
  const uint32_t ld = (uint32_t)up(g.n, 4);
  if (product<T>(g, EpiPlane{planes, ld, false}, splits, s) != hipSuccess) return DF_ERR_HIP;
  hipLaunchKernelGGL((join_planes<T>), dim3(g.m), dim3(256), 0, s, (const float *)planes, splits, g.m, g.n, ld, out);
  return hipGetLastError() == hipSuccess ? DF_OK : DF_ERR_HIP;
}

template <class T, int MT, int NT, int W, int U>
hipError_t rows_launch(const U4 &w, const uint16_t *x, uint64_t xs, uint32_t m, uint16_t *y, hipStream_t s) {
  const bool sub = w.group32 % 4 != 0, wide = w.k % 32 == 0 && ((uintptr_t)w.packed & 15) == 0;
  auto *fn = sub ? (wide ? u4_rows<T, MT, NT, W, U, true, true> : u4_rows<T, MT, NT, W, U, true, false>)
                 : (wide ? u4_rows<T, MT, NT, W, U, false, true> : u4_rows<T, MT, NT, W, U, false, false>);
  hipLaunchKernelGGL(fn, dim3((w.n + 16 * NT - 1) / (16 * NT)), dim3(64 * W), 0, s, w, x, xs, m, y);
  return hipGetLastError();
}

template <class T>
df_status linear(const U4 &w, const uint16_t *x, uint32_t m, uint64_t xs, uint16_t *y, uint8_t *ws, hipStream_t s) {
  hipError_t e;
  if (m <= 16) {
    e = rows_launch<T, 1, 1, 8, 4>(w, x, xs, m, y, s);
  } else if (m <= 32) {
    e = rows_launch<T, 2, 2, 8, 2>(w, x, xs, m, y, s);
  } else if (m <= kFewRows) {
    e = rows_launch<T, 4, 2, 4, 1>(w, x, xs, m, y, s);
  } else {
    hipLaunchKernelGGL((u4_expand<T>), dim3(w.n), dim3(256), 0, s, w, (uint16_t *)ws);
    Gemm g = {x, (const uint16_t *)ws, xs, w.k, m, w.n, w.k, 0, 0, 0};
    return many_rows<T>(g, y, (float *)(ws + up((uint64_t)w.n * w.k * 2, 256)), s);
  }
  return e == hipSuccess ? DF_OK : DF_ERR_HIP;
}

template <class T>
df_status linear_grad(const U4 &w, const uint16_t *dy, uint32_t m, uint64_t ds, uint16_t *dx, uint8_t *ws,
                      hipStream_t s) {
  const uint32_t np = (uint32_t)up(w.n, 8);
  hipLaunchKernelGGL((u4_expand_t<T>), dim3((np + 63) / 64, (w.k + 63) / 64), dim3(256), 0, s, w, (uint16_t *)ws, np);
  uint8_t *next = ws + up((uint64_t)np * w.k * 2, 256);
  if (np != w.n) {  // the summed index in whole 16-byte chunks
    hipLaunchKernelGGL(pad_rows, dim3(m), dim3(256), 0, s, dy, ds, w.n, np, (uint16_t *)next);
    dy = (const uint16_t *)next;
    ds = np;
    next += up((uint64_t)m * np * 2, 256);
  }
  Gemm g = {dy, (const uint16_t *)ws, ds, np, m, w.k, np, 0, 0, 0};
  return many_rows<T>(g, dx, (float *)next, s);
}

uint64_t plane_bytes(uint32_t m, uint32_t n, uint32_t k) {
  const uint32_t splits = splits_for(m, n, k);
  return splits > 1 ? 4ull * splits * m * up(n, 4) : 0;
}

}  // namespace

extern "C" {

uint64_t df_linear_u4_workspace_bytes(const df_u4_matrix *w, uint64_t rows) {
  if (!w || rows <= kFewRows || rows > (1u << 24)) return 0;
  return up(w->rows * w->cols * 2, 256) + plane_bytes((uint32_t)rows, (uint32_t)w->rows, (uint32_t)w->cols);
}

uint64_t df_linear_u4_grad_workspace_bytes(const df_u4_matrix *w, uint64_t rows) {
  if (!w || rows == 0 || rows > (1u << 24)) return 0;
  const uint64_t np = up(w->rows, 8);
  return up(np * w->cols * 2, 256) + (np != w->rows ? up(rows * np * 2, 256) : 0) + plane_bytes((uint32_t)rows, (uint32_t)w->cols, (uint32_t)np);
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
