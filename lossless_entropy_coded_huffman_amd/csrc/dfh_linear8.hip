// Products in 8-bit integers (gfx950).
//
//   y[m, n] = xs[m] s[n] sum_k xq[m, k] (q[n, k] - z[n])
//
// The weights are the codes that a uint8 container decodes to, with a scale and a
// zero point for each of their rows; the rows of x are quantised with a scale for
// each (dfh_quant.h).  The matrix cores multiply signed bytes, so they are given
// q - 128, and (128 - z) times the sum of xq is added: all in 32-bit integers, which
// hold every sum of up to 65536 terms (127 * 255 * 65536 < 2^31), so the only
// roundings are x's to its codes and y's.
//
// Few rows: u8_tokens.  More: the rows are quantised into the workspace and the
// tiled product of dfh_gemm.h takes 128 bytes of a row a step where it takes 64
// 16-bit elements, so tiles, loads and LDS are the same.
#include <hip/hip_runtime.h>

#include "dfh.h"
#include "dfh_gemm.h"
#include "dfh_quant.h"

namespace dfh {
namespace {
// Bytes: operand a the weights' codes (any byte), b those of x (signed).  Sums are
// 32-bit integers in the places of the floats.
struct I8 {};
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f32x4 mfma(I8, u32x4 a, u32x4 b, f32x4 c) {
  a ^= 0x80808080u;
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                                         __builtin_bit_cast(i32x4, b),
                                                                         __builtin_bit_cast(i32x4, c), 0, 0, 0));
}
}  // namespace
}  // namespace dfh

namespace {

using namespace dfh;

struct U8 {
  const uint8_t *codes, *zeros;  // zeros null: 128 everywhere
  const void *scales;
  int scale_type;
  uint32_t n, k;
  uint32_t once;  // more bytes than the last-level cache holds: read past it
  uint64_t sstride, zstride;
};
__device__ __forceinline__ float scale_at(const U8 &w, uint32_t n) {
  const uint64_t i = n * w.sstride;
  if (w.scale_type == DF_TYPE_F32) return ((const float *)w.scales)[i];
  const uint16_t b = ((const uint16_t *)w.scales)[i];
  return w.scale_type == DF_TYPE_BF16 ? from_bits(BF16{}, b) : from_bits(F16{}, b);
}
// What the sum of a row's codes counts.
__device__ __forceinline__ int offset_at(const U8 &w, uint32_t n) {
  return w.zeros ? 128 - (int)w.zeros[n * w.zstride] : 0;
}
// A sum as an output: the weight's scale first, so that the product is the size of a
// sum of weights before x's scale, of any size, comes to it.
__device__ __forceinline__ float scaled(int sum, float s, float xs) { return (float)sum * s * xs; }

__device__ __forceinline__ int sum_of_codes(u32x4 c, int sum) {
#pragma unroll
  for (int i = 0; i < 4; i++) sum = __builtin_amdgcn_sdot4((int)c[i], 0x01010101, sum, false);
  return sum;
}
__device__ __forceinline__ uint32_t most_of_wave_bits(uint32_t v) {
  return __float_as_uint(most_of_wave(__uint_as_float(v)));  // magnitudes: their floats are ordered alike
}
__device__ __forceinline__ int sum_of_wave(int v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Rows of x -> codes, scales and (where wanted) sums of codes.  THREADS to a row, of a workgroup's
// BLOCK; the row's first 4 chunks a thread stay in registers between the two passes.
template <class T, int THREADS, int BLOCK>
__global__ __launch_bounds__(BLOCK) void quantise(const uint16_t *x, uint64_t xs, uint32_t m, uint32_t k, uint8_t *codes,
                                                uint64_t cs, float *scales, int *sums) {
  constexpr int kRows = BLOCK / THREADS, kKeep = 4, kWaves = THREADS / 64;
  __shared__ uint32_t tops[BLOCK / 64];
  __shared__ int totals[BLOCK / 64];
  const uint32_t t = threadIdx.x % THREADS, chunks = k / 8;
  for (uint64_t row = (uint64_t)blockIdx.x * kRows + threadIdx.x / THREADS; row < m; row += (uint64_t)gridDim.x * kRows) {
    const u32x4 *src = (const u32x4 *)(x + row * xs);
    u32x4 keep[kKeep];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kKeep; i++) {
      const uint32_t c = t + i * THREADS;
      keep[i] = c < chunks ? src[c] : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < kKeep; i++) top = most_bits(keep[i], top);
    for (uint32_t c = t + kKeep * THREADS; c < chunks; c += THREADS) top = most_bits(src[c], top);
    top = most_of_wave_bits(joined(top));
    if (THREADS > 64) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWaves; i++) top = top > tops[i] ? top : tops[i];
    }
    Quantiser q;
    q.init(T{}, top);
    u32x2 *dst = (u32x2 *)(codes + row * cs);
    int sum = 0;
    auto put = [&](uint32_t c, u32x4 v) {
      const u32x2 o = q.codes(T{}, v);
      dst[c] = o;
      sum = __builtin_amdgcn_sdot4((int)o[0], 0x01010101, sum, false);
      sum = __builtin_amdgcn_sdot4((int)o[1], 0x01010101, sum, false);
    };
#pragma unroll
    for (int i = 0; i < kKeep; i++)
      if (t + i * THREADS < chunks) put(t + i * THREADS, keep[i]);
    for (uint32_t c = t + kKeep * THREADS; c < chunks; c += THREADS) put(c, src[c]);
    if (sums) {
      sum = sum_of_wave(sum);
      if (THREADS > 64) {
        if ((threadIdx.x & 63) == 0) totals[threadIdx.x >> 6] = sum;
        __syncthreads();
        sum = 0;
#pragma unroll
        for (int i = 0; i < kWaves; i++) sum += totals[i];
      }
      if (t == 0) sums[row] = sum;
    }
    if (t == 0) scales[row] = q.scale;
  }
}

// Sums of rows of codes, a wave to a row.
__global__ __launch_bounds__(256) void code_sums(const uint8_t *codes, uint64_t cs, uint32_t m, uint32_t k, int *sums) {
  const uint32_t lane = threadIdx.x & 63;
  for (uint64_t row = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < m; row += (uint64_t)gridDim.x * 4) {
    const u32x4 *src = (const u32x4 *)(codes + row * cs);
    int sum = 0;
    for (uint32_t c = lane; c < k / 16; c += 64) sum = sum_of_codes(src[c], sum);
    sum = sum_of_wave(sum);
    if (lane == 0) sums[row] = sum;
  }
}

// Where the rows of x come from: 16-bit floats, or codes with scales.
struct Rows {
  const void *x;
  uint64_t stride;
  const float *scales;  // null: floats
};

// 16 bytes a lane of a weight row, past the caches where it is read once.
template <bool ONCE>
__device__ __forceinline__ u32x4 read16(const uint8_t *p) {
  typedef const __attribute__((address_space(1))) u32x4 *Global;
  return ONCE ? __builtin_nontemporal_load((Global)p) : *(Global)p;
}

// y for up to four rows (tokens).  A workgroup quantises the rows of x into LDS
// (every workgroup for itself: no launch before), then each of its waves takes R
// weight rows at a time, 1 KiB of each a load, and multiplies bytes four at a time
// (v_dot4); W waves share a row's summed index where there are few rows (KSPLIT).
// The first rows' loads are asked for before x is quantised.
template <class T, int M, int R, int KSPLIT, bool ONCE>
__global__ __launch_bounds__(256) void u8_tokens(const U8 w, const Rows xr, uint16_t *y) {
  extern __shared__ __align__(16) uint8_t lds[];  // [M][kp] codes
  __shared__ float scales[M];
  __shared__ int sums[M], parts[4][M][R];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr uint32_t kGroups = 4 / KSPLIT;  // of waves, with weight rows of their own
  const uint32_t group = wave / KSPLIT, part = wave % KSPLIT;
  const uint32_t steps = (w.k + 1023) / 1024, per = (steps + KSPLIT - 1) / KSPLIT;
  const uint32_t s0 = part * per, s1 = s0 + per < steps ? s0 + per : steps;
  const uint32_t kp = steps * 1024;  // zeros behind k
  const uint32_t blocks = (w.n + R - 1) / R, stride = gridDim.x * kGroups;
  u32x4 next[R];
  const uint8_t *row[R];
  auto rows_of = [&](uint32_t b) {
#pragma unroll
    for (int r = 0; r < R; r++) {
      const uint32_t n = b * R + r;
      row[r] = w.codes + (uint64_t)(n < w.n ? n : w.n - 1) * w.k;
    }
  };
  auto request = [&](uint32_t st) {
    const uint32_t at = st * 1024 + lane * 16, k = at < w.k ? at : 0;  // x's code is 0 there
#pragma unroll
    for (int r = 0; r < R; r++) next[r] = read16<ONCE>(row[r] + k);
  };
  uint32_t b = blockIdx.x * kGroups + group;
  rows_of(b < blocks ? b : blocks - 1);
  if (s0 < s1) request(s0);
  // x's rows
  if (xr.scales) {
#pragma unroll
    for (int m = 0; m < M; m++) {
      const u32x4 *src = (const u32x4 *)((const uint8_t *)xr.x + m * xr.stride);
      for (uint32_t c = threadIdx.x; c < kp / 16; c += 256)
        ((u32x4 *)(lds + m * kp))[c] = c < w.k / 16 ? src[c] : u32x4{0, 0, 0, 0};
      if (threadIdx.x == 0) scales[m] = xr.scales[m];
    }
  } else {
    __shared__ uint32_t tops[4][M];
#pragma unroll
    for (int m = 0; m < M; m++) {
      const u32x4 *src = (const u32x4 *)((const uint16_t *)xr.x + m * xr.stride);
      uint32_t top = 0;
      for (uint32_t c = threadIdx.x; c < w.k / 8; c += 256) top = most_bits(src[c], top);
      top = most_of_wave_bits(joined(top));
      if (lane == 0) tops[wave][m] = top;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; m++) {
      const u32x4 *src = (const u32x4 *)((const uint16_t *)xr.x + m * xr.stride);
      uint32_t top = tops[0][m];
#pragma unroll
      for (int i = 1; i < 4; i++) top = top > tops[i][m] ? top : tops[i][m];
      Quantiser q;
      q.init(T{}, top);
      for (uint32_t c = threadIdx.x; c < kp / 8; c += 256)
        ((u32x2 *)(lds + m * kp))[c] = c < w.k / 8 ? q.codes(T{}, src[c]) : u32x2{0, 0};
      if (threadIdx.x == 0) scales[m] = q.scale;
    }
  }
  __syncthreads();
  if (w.zeros && wave < M) {
    int sum = 0;
    for (uint32_t c = lane; c < kp / 16; c += 64) sum = sum_of_codes(((const u32x4 *)(lds + wave * kp))[c], sum);
    sum = sum_of_wave(sum);
    if (lane == 0) sums[wave] = sum;
  }
  __syncthreads();
  const uint32_t rounds = (blocks + stride - 1) / stride;  // the same for every wave: they meet
  for (uint32_t round = 0; round < rounds; round++, b += stride) {
    int acc[M][R] = {};
    for (uint32_t st = s0; st < s1; st++) {
      u32x4 now[R];
#pragma unroll
      for (int r = 0; r < R; r++) now[r] = next[r];
      if (st + 1 < s1) {
        request(st + 1);
      } else if (round + 1 < rounds) {
        rows_of(b + stride < blocks ? b + stride : blocks - 1);
        request(s0);
      }
#pragma unroll
      for (int m = 0; m < M; m++) {
        const u32x4 c = *(const u32x4 *)(lds + m * kp + st * 1024 + lane * 16);
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
          for (int i = 0; i < 4; i++)
            acc[m][r] = __builtin_amdgcn_sdot4((int)(now[r][i] ^ 0x80808080u), (int)c[i], acc[m][r], false);
      }
    }
#pragma unroll
    for (int m = 0; m < M; m++)
#pragma unroll
      for (int r = 0; r < R; r++) acc[m][r] = sum_of_wave(acc[m][r]);
    if (KSPLIT > 1) {
      if (round) __syncthreads();  // the last round's are read
      if (lane == 0)
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
          for (int r = 0; r < R; r++) parts[wave][m][r] = acc[m][r];
      __syncthreads();
    }
    if (part == 0 && lane < M * R) {
      const uint32_t m = lane / R, r = lane % R, n = b * R + r;
      int sum = 0;
      if (KSPLIT > 1) {
#pragma unroll
        for (int p = 0; p < KSPLIT; p++) sum += parts[group * KSPLIT + p][m][r];
      } else {
#pragma unroll
        for (int mm = 0; mm < M; mm++)
#pragma unroll
          for (int rr = 0; rr < R; rr++)
            if (lane == (uint32_t)(mm * R + rr)) sum = acc[mm][rr];
      }
      if (b < blocks && n < w.n) {
        if (w.zeros) sum += offset_at(w, n) * sums[m];
        y[(uint64_t)m * w.n + n] = to_bits(T{}, scaled(sum, scale_at(w, n), scales[m]));
      }
    }
  }
}

// Integer sums -> y.  T: the output's type.
template <class T>
struct EpiU8 {
  U8 w;
  const float *xs;
  const int *sums;  // of x's codes, where there are zero points
  uint16_t *y;
  template <class, int NT, int MT>
  __device__ __forceinline__ void operator()(f32x4 (&acc)[NT][MT], uint32_t mb, uint32_t nb, uint32_t m, uint32_t n,
                                             uint32_t, uint32_t) const {
    static_assert(NT % 2 == 0, "blocks in pairs");
    const bool aligned = (n & 7) == 0;
    const uint32_t kg = (threadIdx.x >> 4) & 3, first = nb - 4 * kg + (kg & 1) * 16 + (kg >> 1) * 8;
    float s[NT][4];
    int off[NT][4];
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const uint32_t c = nb + j * 16 + e, cc = c < n ? c : n - 1;
        s[j][e] = scale_at(w, cc);
        off[j][e] = offset_at(w, cc);
      }
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const uint32_t row = mb + i * 16, rr = row < m ? row : m - 1;
      const float f = xs[rr];
      const int sum = w.zeros ? sums[rr] : 0;
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        float v[2][4];
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int e = 0; e < 4; e++)
            v[h][e] = scaled(__builtin_bit_cast(i32x4, acc[j + h][i])[e] + off[j + h][e] * sum, s[j + h][e], f);
        const u32x4 o = pair_blocks(u32x2{pack2(T{}, v[0][0], v[0][1]), pack2(T{}, v[0][2], v[0][3])},
                                    u32x2{pack2(T{}, v[1][0], v[1][1]), pack2(T{}, v[1][2], v[1][3])});
        if (row < m) store8(y + (uint64_t)row * n, first + j * 16, n, aligned, o);
      }
    }
  }
};

// Planes of integer sums [splits][m][ld] -> y.
template <class T>
__global__ __launch_bounds__(256) void join_u8(const U8 w, const float *planes, uint32_t splits, uint32_t m, uint32_t ld,
                                               const float *xs, const int *sums, uint16_t *y) {
  const uint32_t n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= w.n) return;
  for (uint32_t row = blockIdx.y; row < m; row += gridDim.y) {
    const int *p = (const int *)planes + (uint64_t)row * ld + n;
    i32x4 v = {0, 0, 0, 0};
    uint32_t s = 0;
    for (; s + 4 <= splits; s += 4) {
      i32x4 t[4];
#pragma unroll
      for (int i = 0; i < 4; i++) t[i] = *(const i32x4 *)(p + (uint64_t)(s + i) * m * ld);
#pragma unroll
      for (int i = 0; i < 4; i++) v += t[i];
    }
    for (; s < splits; s++) v += *(const i32x4 *)(p + (uint64_t)s * m * ld);
    const float f = xs[row];
    const int sum = w.zeros ? sums[row] : 0;
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (n + e < w.n)
        y[(uint64_t)row * w.n + n + e] = to_bits(T{}, scaled(v[e] + offset_at(w, n + e) * sum, scale_at(w, n + e), f));
  }
}

bool type_ok(df_type t) { return t == DF_TYPE_BF16 || t == DF_TYPE_F16; }

df_status matrix_of(const df_u8_matrix *m, U8 *w) {
  if (!m || !m->codes || !m->scales || ((uintptr_t)m->codes & 15)) return DF_ERR_ARG;
  if (m->rows == 0 || m->rows > (1u << 21) || m->cols == 0 || m->cols > 65536 || m->cols % 16) return DF_ERR_ARG;
  if (m->scale_type != DF_TYPE_BF16 && m->scale_type != DF_TYPE_F16 && m->scale_type != DF_TYPE_F32)
    return DF_ERR_ARG;
  if ((uintptr_t)m->scales & (m->scale_type == DF_TYPE_F32 ? 3 : 1)) return DF_ERR_ARG;
  w->codes = m->codes;
  w->zeros = m->zeros;
  w->scales = m->scales;
  w->scale_type = (int)m->scale_type;
  w->n = (uint32_t)m->rows;
  w->k = (uint32_t)m->cols;
  w->sstride = m->scale_stride;
  w->zstride = m->zero_stride;
  w->once = m->rows * m->cols >= (256u << 20);
  return DF_OK;
}

// Rows that u8_tokens takes: their codes have to fit in 60 KiB of LDS.
bool tokens(uint64_t m, uint64_t k) { return m <= 4 && m * up(k, 1024) <= 61440; }

// Tiles and splits of a product: cut_for's, but for few steps (k up to 2048, which cut_for would
// split) where 64 x 64 tiles without splits are up to 4 to a CU: their sums need no second launch
// (128 x 4096 x 1424 14.5 us against 19.4, 333 x 2047 x 1424 16.1 against 22.6; with more steps it
// turns, 333 x 2047 x 4096 29.5 against 24.5, and with more tiles, 768 x 6144 x 2048 32.2
// against 28.8).
Cut cut_of(uint64_t m, uint64_t n, uint64_t k) {
  if (m > 64 && k <= 2048 && up(m, 64) / 64 * (up(n, 64) / 64) <= 1024) return Cut{2, 1, 0.0};
  return cut_for(m, n, k / 2, true);
}

// The workspace of a product of more rows.
struct Space {
  uint64_t codes, scales, sums, planes, all;  // offsets
};
Space space_of(uint64_t m, uint64_t n, uint64_t k, bool floats) {
  Space s;
  s.codes = 0;
  s.scales = floats ? up(m * k, 256) : 0;
  s.sums = s.scales + (floats ? up(m * 4, 256) : 0);
  s.planes = s.sums + up(m * 4, 256);
  const Cut c = cut_of(m, n, k);
  s.all = s.planes + (c.splits > 1 ? 4ull * c.splits * m * up(n, 4) : 0);
  return s;
}

template <class T>
hipError_t quantise_rows(const uint16_t *x, uint64_t xs, uint32_t m, uint32_t k, uint8_t *codes, float *scales, int *sums,
                         hipStream_t s) {
  // a wave to a short row, and 16 to one that the registers of 4 do not hold: all its loads are
  // in flight at once (23 x 14336 3.9 us, 4 waves 4.7; 1024 x 14336 10.2 and 10.3; shorter rows
  // wait for one another instead, 2048 x 4096 11.8 us against 7.1)
  const bool wide = k > 8192;
  const uint32_t per = k <= 2048 ? 4 : 1, blocks = (m + per - 1) / per;
  hipLaunchKernelGGL((wide ? quantise<T, 1024, 1024> : k <= 2048 ? quantise<T, 64, 256> : quantise<T, 256, 256>),
                     dim3(blocks < 1u << 20 ? blocks : 1u << 20), dim3(wide ? 1024 : 256), 0, s, x, xs, m, k, codes,
                     (uint64_t)k, scales, sums);
  return hipGetLastError();
}

template <class T, int M, int R, int KSPLIT>
hipError_t tokens_of(const U8 &w, const Rows &x, uint16_t *y, hipStream_t s) {
  auto *fn = w.once ? u8_tokens<T, M, R, KSPLIT, true> : u8_tokens<T, M, R, KSPLIT, false>;
  const uint32_t lds = M * (uint32_t)up(w.k, 1024);
  const uint32_t blocks = (uint32_t)up(w.n, R * (4 / KSPLIT)) / (R * (4 / KSPLIT));
  const uint32_t most = lds <= 16384 ? 2048 : lds <= 32768 ? 1024 : 512;  // resident at once
  hipLaunchKernelGGL(fn, dim3(blocks < most ? blocks : most), dim3(256), lds, s, w, x, y);
  return hipGetLastError();
}
template <class T, int M>
hipError_t tokens_for(const U8 &w, const Rows &x, uint16_t *y, hipStream_t s) {
  return w.n >= 8192 ? tokens_of<T, M, 4, 1>(w, x, y, s) : tokens_of<T, M, 4, 4>(w, x, y, s);
}

template <class T>
df_status linear(const U8 &w, Rows x, uint32_t m, uint16_t *y, uint8_t *ws, hipStream_t s) {
  if (tokens(m, w.k)) {
    const hipError_t e = m == 1   ? tokens_for<T, 1>(w, x, y, s)
                         : m == 2 ? tokens_for<T, 2>(w, x, y, s)
                         : m == 3 ? tokens_for<T, 3>(w, x, y, s)
                                  : tokens_for<T, 4>(w, x, y, s);
    return e == hipSuccess ? DF_OK : DF_ERR_HIP;
  }
  const Space sp = space_of(m, w.n, w.k, !x.scales);
  int *sums = (int *)(ws + sp.sums);
  const uint8_t *codes = (const uint8_t *)x.x;
  const float *scales = x.scales;
  uint64_t stride = x.stride;
  if (!x.scales) {
    if (quantise_rows<T>((const uint16_t *)x.x, x.stride, m, w.k, ws, (float *)(ws + sp.scales), w.zeros ? sums : nullptr,
                         s) != hipSuccess)
      return DF_ERR_HIP;
    codes = ws;
    scales = (const float *)(ws + sp.scales);
    stride = w.k;
  } else if (w.zeros) {
    const uint32_t blocks = (m + 3) / 4;
    hipLaunchKernelGGL(code_sums, dim3(blocks < 1u << 20 ? blocks : 1u << 20), dim3(256), 0, s, codes, stride, m, w.k, sums);
    if (hipGetLastError() != hipSuccess) return DF_ERR_HIP;
  }
  const Gemm g = {(const uint16_t *)codes, (const uint16_t *)w.codes, stride / 2, w.k / 2, m, w.n, w.k / 2, 0, 0, 0, 0};
  const Cut c = cut_of(m, w.n, w.k);
  if (c.splits <= 1)
    return product<I8, false, false>(g, EpiU8<T>{w, scales, sums, y}, c.shape, 1, s) == hipSuccess ? DF_OK : DF_ERR_HIP;
  const uint32_t ld = (uint32_t)up(w.n, 4);
  float *planes = (float *)(ws + sp.planes);
  if (product<I8, false, false>(g, EpiPlane{planes, ld, (uint64_t)m * ld, false}, c.shape, c.splits, s) != hipSuccess)
    return DF_ERR_HIP;
  hipLaunchKernelGGL((join_u8<T>), dim3((w.n + 1023) / 1024, m < 32768 ? m : 32768), dim3(256), 0, s, w,
                     (const float *)planes, c.splits, m, ld, scales, (const int *)sums, y);
  return hipGetLastError() == hipSuccess ? DF_OK : DF_ERR_HIP;
}

df_status linear_of(const df_u8_matrix *w, df_type type, const Rows &x, uint64_t rows, void *y, void *workspace,
                    uint64_t workspace_bytes, hipStream_t stream) {
  U8 u;
  const df_status st = matrix_of(w, &u);
  if (st != DF_OK) return st;
  if (!type_ok(type) || rows > (1u << 24)) return DF_ERR_ARG;
  if (rows == 0) return DF_OK;
  const uint64_t unit = x.scales ? 16 : 8;  // elements of 16 bytes
  if (!x.x || !y || ((uintptr_t)x.x & 15) || ((uintptr_t)y & 15) || ((uintptr_t)x.scales & 3) || x.stride < u.k ||
      x.stride % unit || x.stride > (1u << 21))
    return DF_ERR_ARG;
  const uint64_t need = tokens(rows, u.k) ? 0 : space_of(rows, u.n, u.k, !x.scales).all;
  if (need && (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need)) return DF_ERR_ARG;
  return type == DF_TYPE_BF16 ? linear<BF16>(u, x, (uint32_t)rows, (uint16_t *)y, (uint8_t *)workspace, stream)
                              : linear<F16>(u, x, (uint32_t)rows, (uint16_t *)y, (uint8_t *)workspace, stream);
}

}  // namespace

extern "C" {

df_status df_quantize_rows(df_type type, const void *x, uint64_t rows, uint64_t cols, uint64_t x_stride, int8_t *codes,
                           float *scales, hipStream_t stream) {
  if (!type_ok(type) || rows > (1u << 24) || cols == 0 || cols > 65536 || cols % 16) return DF_ERR_ARG;
  if (rows == 0) return DF_OK;
  if (!x || !codes || !scales || ((uintptr_t)x & 15) || ((uintptr_t)codes & 15) || ((uintptr_t)scales & 3) ||
      x_stride < cols || x_stride % 8 || x_stride > (1u << 21))
    return DF_ERR_ARG;
  const hipError_t e = type == DF_TYPE_BF16
                           ? quantise_rows<BF16>((const uint16_t *)x, x_stride, (uint32_t)rows, (uint32_t)cols,
                                                 (uint8_t *)codes, scales, nullptr, stream)
                           : quantise_rows<F16>((const uint16_t *)x, x_stride, (uint32_t)rows, (uint32_t)cols,
                                                (uint8_t *)codes, scales, nullptr, stream);
  return e == hipSuccess ? DF_OK : DF_ERR_HIP;
}

uint64_t df_linear_u8_workspace_bytes(const df_u8_matrix *w, uint64_t rows, int codes) {
  U8 u;
  if (matrix_of(w, &u) != DF_OK || rows == 0 || rows > (1u << 24) || tokens(rows, u.k)) return 0;
  return space_of(rows, u.n, u.k, !codes).all;
}

df_status df_linear_u8(const df_u8_matrix *w, df_type type, const void *x, uint64_t rows, uint64_t x_stride, void *y,
                       void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
  return linear_of(w, type, Rows{x, x_stride, nullptr}, rows, y, workspace, workspace_bytes, stream);
}

df_status df_linear_u8_codes(const df_u8_matrix *w, df_type type, const int8_t *codes, const float *scales, uint64_t rows,
                             uint64_t stride, void *y, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
  if (rows && !scales) return DF_ERR_ARG;
  return linear_of(w, type, Rows{codes, stride, scales}, rows, y, workspace, workspace_bytes, stream);
}

}  // extern "C"
