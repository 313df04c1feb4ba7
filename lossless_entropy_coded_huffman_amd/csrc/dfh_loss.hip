// Losses over a large vocabulary without keeping the logits (gfx950).
//
//   z = x head^T,  lse[m] = log sum_v exp(z[m, v] / T)
//   cross entropy: loss = lse - z[label];  distillation: T^2 sum_j t_j (log t_j - z_j / T + lse)
//   dz[m, v] = T g[m] (exp(z / T - lse) - t[m, v]),  dx = dz head,  dhead = dz^T x
//
// with t the row's sparse target (a label is one entry with t = 1, T = 1).
//
// Forward: one pass of gemm whose epilogue reduces each wave's columns to a
// maximum and a sum of exponentials per row; a second kernel joins them.  The
// logits that the targets name have the bits of the ones under the sum, so no
// probability exceeds one and a row that is sure of its label has loss and
// gradient zero: the epilogue writes a label's, and a teacher's entries are
// multiplied again in the same order.  Backward:
// for a piece of the vocabulary that fits the workspace the logits are made
// again, dz goes out in 16 bits, the target entries are put right, and two
// more products take it.  Exponents are in base 2: c = log2(e) / T.
#include <hip/hip_runtime.h>

#include "dfh.h"
#include "dfh_gemm.h"

namespace {

using namespace dfh;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr uint32_t kMaxTop = 1024;

struct Targets {
  const int64_t *labels;  // top == 0
  int64_t ignore;
  const int64_t *index;
  const void *teacher;
  uint64_t istride, tstride;
  int teacher_type;
  uint32_t top, vocab;
  float temp;
};

// What a row keeps: its state, the base-2 log-sum and the target logits.
enum : uint32_t { kNoLoss = 0, kLoss = 1, kBadLabel = 2 };
struct Saved {
  float *share;  // [1]: 1 / the rows that a mean is over, 1 for a sum
  float *lse2;
  uint32_t *state;
  float *picked;  // [rows, max(top, 1)]
};

__device__ __forceinline__ float exp2_(float v) { return __builtin_amdgcn_exp2f(v); }

__device__ __forceinline__ float teacher_at(const Targets &t, uint32_t m, uint32_t j) {
  const uint64_t i = m * t.tstride + j;
  if (t.teacher_type == DF_TYPE_F32) return ((const float *)t.teacher)[i];
  const uint16_t b = ((const uint16_t *)t.teacher)[i];
  return t.teacher_type == DF_TYPE_BF16 ? from_bits(BF16{}, b) : from_bits(F16{}, b);
}
// Vocabulary entry of a row's target j, or -1.
__device__ __forceinline__ int32_t target_of(const Targets &t, uint32_t m, uint32_t j) {
  const int64_t i = t.top ? t.index[m * t.istride + j] : t.labels[m];
  if (!t.top && i == t.ignore) return -1;
  return i >= 0 && i < (int64_t)t.vocab ? (int32_t)i : -1;
}

// ------------------------------------------------------------------ epilogues
// Per row, over this wave's columns: max of z2 = c z and sum of 2^(z2 - max).
// Where there are labels, the one wave whose columns hold a row's writes its z.
struct EpiStats {
  float2 *parts;  // [part][rows]
  uint32_t rows;
  float c;
  const int64_t *labels;
  float *picked;
  EpiStats from_row(uint32_t r) const {
    return EpiStats{parts + r, rows, c, labels ? labels + r : labels, picked + r};
  }
  template <class T, int NT, int MT>
  __device__ __forceinline__ void operator()(f32x4 (&acc)[NT][MT], uint32_t mb, uint32_t nb, uint32_t m, uint32_t n,
                                             uint32_t part, uint32_t) const {
#pragma clang fp contract(off)  // c z is rounded wherever it is made
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const uint32_t row = mb + i * 16;
      if (labels && row < m) {
        const int64_t l = labels[row];
        const uint32_t at = (uint32_t)l - nb;
        if (l >= 0 && l < (int64_t)n && at < NT * 16 && (at & 15) < 4) {
#pragma unroll
          for (int j = 0; j < NT; j++)
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (at == j * 16 + e) picked[row] = acc[j][i][e];
        }
      }
      float mx = -__builtin_huge_valf();
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float v = nb + j * 16 + e < n ? acc[j][i][e] * c : -__builtin_huge_valf();
          acc[j][i][e] = v;
          mx = __builtin_fmaxf(mx, v);
        }
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16));
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32));
      const float ref = mx == -__builtin_huge_valf() ? 0.f : mx;
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) s += exp2_(acc[j][i][e] - ref);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if ((threadIdx.x & 48) == 0 && row < m) parts[(uint64_t)part * rows + row] = float2{mx, s};
    }
  }
};

// dz / (T g) without the target's part, times `mul`: 2^(c z - lse2), rounded to the
// operands' 16 bits, which the products that take it need (an FP32 dz would double
// the traffic and fit no matrix instruction at their rate); zero in rows without a
// loss and in the columns that pad a row to ldz.
// FP16 takes mul = 2^15: probabilities of a large vocabulary lie where FP16
// has few bits or none; the products' epilogues take the factor out again.
struct EpiDz {
  uint16_t *dz;
  uint32_t ldz;
  const float *lse2;
  const uint32_t *state;
  float c, mul;
  EpiDz from_row(uint32_t r) const { return EpiDz{dz + (uint64_t)r * ldz, ldz, lse2 + r, state + r, c, mul}; }
  template <class T, int NT, int MT>
  __device__ __forceinline__ void operator()(f32x4 (&acc)[NT][MT], uint32_t mb, uint32_t nb, uint32_t m, uint32_t n,
                                             uint32_t, uint32_t) const {
#pragma clang fp contract(off)  // as in EpiStats, or p could exceed 1
    static_assert(NT % 2 == 0, "blocks in pairs");
    const uint32_t kg = (threadIdx.x >> 4) & 3, first = nb - 4 * kg + (kg & 1) * 16 + (kg >> 1) * 8;
#pragma unroll
    for (int i = 0; i < MT; i++) {
      const uint32_t row = mb + i * 16, r = row < m ? row : m - 1;
      const bool live = state[r] == kLoss;
      const float l = lse2[r];
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        u32x2 o[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t col = nb + (j + h) * 16;
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; e++) p[e] = live && col + e < n ? exp2_(acc[j + h][i][e] * c - l) * mul : 0.f;
          o[h] = u32x2{pack2(T{}, p[0], p[1]), pack2(T{}, p[2], p[3])};
        }
        const u32x4 v = pair_blocks(o[0], o[1]);
        const uint32_t col = first + j * 16;
        if (row < m && col < ldz) *(u32x4 *)(dz + (uint64_t)row * ldz + col) = v;
      }
    }
  }
};

// ------------------------------------------------------------------- kernels
struct Head {
  const uint16_t *x, *head;
  uint64_t xs, hs;
  uint32_t k;
};
// x[m] . head[v] for sixteen entries a wave, entry lane % 16 (0 for v < 0; m a row
// of x all the same): the diagonal of a matrix product that sums as gemm does, 32
// elements a step in order, so the bits are the ones that its epilogue sees.  Returned
// in the lane whose lane / 16 is a quarter of its entry.
template <class T>
__device__ __forceinline__ float dots_16(const Head &h, uint32_t m, int32_t v) {
  const uint32_t lane = threadIdx.x & 63, off = (lane >> 4) * 8;
  const uint16_t *px = h.x + m * h.xs + off, *ph = h.head + (uint64_t)(v < 0 ? 0 : v) * h.hs + off;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = 8;  // steps in flight
  for (uint32_t k = 0; k < h.k; k += 32 * kAhead) {
    u32x4 a[kAhead], b[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; q++) {
      const uint32_t at = k + q * 32;
      a[q] = b[q] = u32x4{0, 0, 0, 0};
      if (at + off < h.k) {
        if (v >= 0) a[q] = *(const u32x4 *)(ph + at);
        b[q] = *(const u32x4 *)(px + at);
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; q++) acc = mfma(T{}, a[q], b[q], acc);
  }
  const uint32_t e = lane & 3;
  return e == 0 ? acc[0] : e == 1 ? acc[1] : e == 2 ? acc[2] : acc[3];
}

// picked[m, j] = x[m] . head[target j], sixteen entries a wave (0 without a target),
// at most 2^20 workgroups at once: a launch holds fewer than 2^32 threads.
template <class T>
__global__ __launch_bounds__(64) void pick_logits(const Targets t, uint32_t rows, const Head h, float *picked) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t all = (uint64_t)rows * t.top;
  for (uint64_t first = (uint64_t)blockIdx.x * 16; first < all; first += (uint64_t)gridDim.x * 16) {
    const uint64_t e = first + (lane & 15);
    const uint32_t m = (uint32_t)((e < all ? e : first) / t.top), j = (uint32_t)(e % t.top);
    const float z = dots_16<T>(h, m, e < all ? target_of(t, m, j) : -1);
    if (e < all && (lane & 15) / 4 == lane / 16) picked[e] = z;
  }
}

// Parts of a row: `main` in the first `rows` rows, `rest` in those behind them.
struct Parts {
  uint32_t rows, main, rest;
  uint32_t most() const { return main > rest ? main : rest; }
};

// Joins a row's parts and makes its loss.  R rows a workgroup of 256; thread t
// takes parts t / R, t / R + 256 / R, ... (four loads in flight) and targets
// likewise of row t % R.  R = 8 reads 64 bytes of a part at once; few rows take
// R = 1, so that 256 threads share a row's parts (7 rows of 4008 parts: 8 us).
// PICK (with R = 1, where a row has few teacher entries): the four waves make the
// picked logits themselves.
template <class T, int R, bool PICK>
__global__ __launch_bounds__(256) void finish_rows(const Targets t, uint32_t rows, const float2 *parts, Parts np,
                                                   const Head h, Saved sv, float *loss) {
#pragma clang fp contract(off)  // as in EpiStats
  constexpr uint32_t S = 256 / R;
  __shared__ float sa[S][R];
  const uint32_t r = threadIdx.x % R, sl = threadIdx.x / R, m = blockIdx.x * R + r;
  const bool in = m < rows;
  if (PICK) {  // written here, read below after several barriers
    const uint32_t lane = threadIdx.x & 63;
    for (uint32_t first = (threadIdx.x >> 6) * 16; first < t.top; first += 64) {
      const uint32_t j = first + (lane & 15);
      const float z = dots_16<T>(h, m, j < t.top ? target_of(t, m, j) : -1);
      if (j < t.top && (lane & 15) / 4 == lane / 16) sv.picked[(uint64_t)m * t.top + j] = z;
    }
  }
  // over a row's S threads, in a fixed order
  auto join = [&](float v, auto op) {
    sa[sl][r] = v;
    __syncthreads();
#pragma unroll
    for (uint32_t h = S / 2; h; h >>= 1) {
      if (sl < h) sa[sl][r] = op(sa[sl][r], sa[sl + h][r]);
      __syncthreads();
    }
    v = sa[0][r];
    __syncthreads();
    return v;
  };
  auto most = [](float a, float b) { return __builtin_fmaxf(a, b); };
  auto add = [](float a, float b) { return a + b; };
  const float none = -__builtin_huge_valf();
  float mx = none, s = 0.f;
  const uint32_t mine = m < np.rows ? np.main : np.rest;
  for (uint32_t p = sl; in && p < mine; p += 4 * S) {
    float2 v[4];
    float top = mx;
#pragma unroll
    for (uint32_t q = 0; q < 4; q++) {
      v[q] = float2{none, 0.f};
      if (p + q * S < mine) v[q] = parts[(uint64_t)(p + q * S) * rows + m];
    }
#pragma unroll
    for (int q = 0; q < 4; q++) top = most(top, v[q].x);
    const float ref = top == none ? 0.f : top;
    s *= exp2_(mx - ref);
#pragma unroll
    for (int q = 0; q < 4; q++) s += v[q].y * exp2_(v[q].x - ref);
    mx = top;
  }
  const float all = join(mx, most), ref = all == none ? 0.f : all;
  s = join(s * exp2_(mx - ref), add);
  const float over = __builtin_amdgcn_logf(s), lse2 = ref + over;  // base 2
  const float c = kLog2e / t.temp;
  const uint32_t per = t.top ? t.top : 1;
  // the target's softmax over its entries
  float tm = none, any = 0.f;
  for (uint32_t j = sl; in && j < per; j += S)
    if (target_of(t, m, j) >= 0) {
      any = 1.f;
      if (t.top) tm = most(tm, teacher_at(t, m, j) / t.temp);
    }
  any = join(any, most);
  tm = t.top ? join(tm, most) : 0.f;
  const float tref = tm == none ? 0.f : tm;
  float ts = 0.f;
  for (uint32_t j = sl; in && t.top && j < per; j += S)
    if (target_of(t, m, j) >= 0) ts += expf(teacher_at(t, m, j) / t.temp - tref);
  ts = t.top ? join(ts, add) : 1.f;
  const float lts = logf(ts);
  float l = 0.f;
  for (uint32_t j = sl; in && j < per; j += S)
    if (target_of(t, m, j) >= 0) {
      // -log q; 2^(c z - ref) is one of the terms of s
      const float nlq = ((ref - sv.picked[(uint64_t)m * per + j] * c) + over) * kLn2;
      if (!t.top) {
        l = nlq;
      } else {
        const float d = teacher_at(t, m, j) / t.temp - tref, w = expf(d) / ts;
        if (!(w == 0.f)) l += w * ((d - lts) + nlq);
      }
    }
  l = join(l, add) * (t.top ? t.temp * t.temp : 1.f);
  if (in && sl == 0) {
    // a row of entries that all hold -inf has nothing to learn from either
    uint32_t st = any > 0.f && !(t.top && ts == 0.f) ? kLoss : kNoLoss;
    if (!t.top && st == kNoLoss && t.labels[m] != t.ignore) st = kBadLabel;
    sv.lse2[m] = lse2;
    sv.state[m] = st;
    loss[m] = st == kLoss ? l : st == kBadLabel ? __builtin_nanf("") : 0.f;
  }
}

// One workgroup: sum (mean: over the rows that have a loss) of the rows.
__global__ __launch_bounds__(1024) void reduce_rows(const float *rows_loss, const uint32_t *state, uint32_t rows,
                                                    bool mean, float *out, float *share) {
  __shared__ double ss[16];
  __shared__ uint32_t sc[16];
  double s = 0.0;
  uint32_t c = 0;
  for (uint32_t m = threadIdx.x; m < rows; m += 1024) {
    s += rows_loss[m];
    c += state[m] != kNoLoss;
  }
  for (int o = 32; o; o >>= 1) {
    s += __shfl_xor(s, o);
    c += __shfl_xor(c, o);
  }
  if ((threadIdx.x & 63) == 0) {
    ss[threadIdx.x >> 6] = s;
    sc[threadIdx.x >> 6] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    c = 0;
    for (int q = 0; q < 16; q++) {
      s += ss[q];
      c += sc[q];
    }
    *out = (float)(mean ? (c ? s / c : 0.0) : s);
    *share = mean && c ? 1.f / (float)c : 1.f;
  }
}

// Rows with gradients of their own (DF_REDUCE_NONE): peak = max |grad| of the rows
// that have a loss, and gn[m] = grad[m] / peak, which weigh_rows puts on x.  (A
// sum or mean has one gradient, which the products' epilogues take: no row
// factor, no rounding.)
__global__ __launch_bounds__(1024) void row_factors(const uint32_t *state, uint32_t rows, const float *grad, float *gn,
                                                    float *peak) {
  __shared__ float sm[16];
  float mx = 0.f;
  for (uint32_t m = threadIdx.x; m < rows; m += 1024)
    if (state[m] == kLoss) mx = __builtin_fmaxf(mx, __builtin_fabsf(grad[m]));
  for (int o = 32; o; o >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, o));
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = mx;
  __syncthreads();
  mx = 0.f;
  for (int q = 0; q < 16; q++) mx = __builtin_fmaxf(mx, sm[q]);
  const float pk = mx > 0.f ? mx : 1.f;
  for (uint32_t m = threadIdx.x; m < rows; m += 1024) gn[m] = state[m] == kLoss ? grad[m] / pk : 0.f;
  if (threadIdx.x == 0) {
    peak[0] = pk;
    peak[1] = 1.f;
  }
}

// dz at the target entries of vocabulary [v0, v0 + nv): (p - t) * mul with p
// from the picked logit.  Entries of one row that name the same element each
// write the same value, p minus the sum of their t.  One wave per row.
template <class T>
__global__ __launch_bounds__(64) void fix_targets(const Targets t, const Saved sv, uint32_t v0, uint32_t nv, float c,
                                                  float mul, uint16_t *dz, uint32_t ldz) {
#pragma clang fp contract(off)  // as in EpiStats
  __shared__ int32_t ids[kMaxTop];
  __shared__ float ws[kMaxTop];
  const uint32_t m = blockIdx.x, lane = threadIdx.x, per = t.top ? t.top : 1;
  if (sv.state[m] != kLoss) return;
  float mx = -__builtin_huge_valf();
  for (uint32_t j = lane; j < per; j += 64) {
    const int32_t v = target_of(t, m, j);
    const float a = t.top ? teacher_at(t, m, j) / t.temp : 0.f;
    ids[j] = v;
    ws[j] = a;
    if (v >= 0) mx = __builtin_fmaxf(mx, a);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, o));
  float s = 0.f;
  for (uint32_t j = lane; j < per; j += 64) {
    ws[j] = ids[j] >= 0 ? expf(ws[j] - mx) : 0.f;
    s += ws[j];
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  __syncthreads();
  const float l = sv.lse2[m];
  for (uint32_t j = lane; j < per; j += 64) {
    const int32_t v = ids[j];
    if (v < 0 || (uint32_t)v < v0 || (uint32_t)v >= v0 + nv) continue;
    float w = 0.f;
    for (uint32_t q = 0; q < per; q++) w += ids[q] == v ? ws[q] : 0.f;
    const float p = exp2_(sv.picked[(uint64_t)m * per + j] * c - l);
    dz[(uint64_t)m * ldz + (v - v0)] = to_bits(T{}, (p - w / s) * mul);
  }
}

// FP16: the largest finite |gn[m] x[m, c]| in 256 parts.
__global__ __launch_bounds__(256) void weighed_peaks(const uint16_t *x, uint64_t xs, uint32_t rows, uint32_t k,
                                                     const float *gn, float *peaks) {
  float most = 0.f;
  for (uint32_t m = blockIdx.x; m < rows; m += 256) {
    const float f = __builtin_fabsf(gn[m]);
    if (!(f > 0.f)) continue;  // uniform; whatever x holds there
    for (uint32_t c = threadIdx.x; c < k / 8; c += 256) {
      const u32x4 v = *(const u32x4 *)(x + m * xs + c * 8);
#pragma unroll
      for (int d = 0; d < 4; d++) {
        const float a = __builtin_fabsf(from_bits(F16{}, (uint16_t)v[d])), b = __builtin_fabsf(from_bits(F16{}, (uint16_t)(v[d] >> 16)));
        most = __builtin_fmaxf(most, a < __builtin_huge_valf() ? a * f : 0.f);
        most = __builtin_fmaxf(most, b < __builtin_huge_valf() ? b * f : 0.f);
      }
    }
  }
  most = most_of_256(most);
  if (threadIdx.x == 0) peaks[blockIdx.x] = most;
}

// out[c, m] = gn[m] x[m, c] (gn null: x), zeros in rows without a loss (whatever x holds
// there) and in the columns that pad a row to mp: what dhead's sum over the rows
// takes for x, so dz needs no row factor; turned, so that only dz is read across
// there.  64 x 64 tiles through LDS, padded rows spread the column writes.
// With row factors a product is rounded once more, to 2^-8 of itself (BF16) or, lifted
// by the power of two that *back takes off, to 2^-11 or 2^-39 of the largest (FP16):
// the price of 16-bit operands, which dhead rows of small factors pay alike.
template <class T>
__global__ __launch_bounds__(256) void weigh_rows(const uint16_t *x, uint64_t xs, uint32_t rows, uint32_t k,
                                                  const uint32_t *state, const float *gn, const float *peaks,
                                                  float *back, uint16_t *out, uint32_t mp) {
  __shared__ uint16_t tile[64][72];  // [c][m]
  float lift = 1.f;
  if (peaks) {
    const int bits = lift_bits(most_of_256(peaks[threadIdx.x]), 14);
    lift = power_of_two(bits);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *back = power_of_two(-bits);
  }
  const uint32_t m0 = blockIdx.x * 64, c0 = blockIdx.y * 64;
#pragma unroll
  for (uint32_t t = threadIdx.x; t < 512; t += 256) {
    const uint32_t r = t / 8, c = t % 8, m = m0 + r;
    u32x4 v = {0, 0, 0, 0};
    if (m < rows && c0 + c * 8 < k && state[m] == kLoss) {
      v = *(const u32x4 *)(x + m * xs + c0 + c * 8);
      const float f = gn ? gn[m] * lift : 1.f;
#pragma unroll
      for (int d = 0; gn && d < 4; d++)
        v[d] = pack2(T{}, from_bits(T{}, (uint16_t)v[d]) * f, from_bits(T{}, (uint16_t)(v[d] >> 16)) * f);
    }
#pragma unroll
    for (int d = 0; d < 4; d++) {
      tile[c * 8 + 2 * d][r] = (uint16_t)v[d];
      tile[c * 8 + 2 * d + 1][r] = (uint16_t)(v[d] >> 16);
    }
  }
  __syncthreads();
#pragma unroll
  for (uint32_t t = threadIdx.x; t < 512; t += 256) {
    const uint32_t c = t / 8, m = m0 + t % 8 * 8;
    if (c0 + c < k && m < mp) *(u32x4 *)(out + (uint64_t)(c0 + c) * mp + m) = *(const u32x4 *)&tile[c][t % 8 * 8];
  }
}

// dx[m] = mul * grad * share * (sum of the planes), zero in rows without a loss.
template <class T>
__global__ __launch_bounds__(256) void finish_dx(const float *planes, Parts parts, uint32_t rows, uint32_t k,
                                                 const uint32_t *state, const float *grad, const float *share, float mul,
                                                 uint16_t *dx) {
  const uint32_t m = blockIdx.x;
  const bool live = state[m] == kLoss;
  const float f = (share ? grad[0] * *share : grad[m]) * mul;
  const uint32_t splits = m < parts.rows ? parts.main : parts.rest;
  for (uint32_t c = threadIdx.x * 4; c < k; c += 1024) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (live) v = add_planes(planes + (uint64_t)m * k + c, (uint64_t)rows * k, splits) * f;
    *(u32x2 *)(dx + (uint64_t)m * k + c) = u32x2{pack2(T{}, v[0], v[1]), pack2(T{}, v[2], v[3])};
  }
}

__global__ __launch_bounds__(256) void fill_words(uint32_t *p, uint64_t n) {
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256) p[i] = 0;
}

// ---------------------------------------------------------------- host side
Parts parts_of(const RowCut &c, uint64_t n) {
  auto of = [&](const Cut &q) {
    const Shape &sh = kShapes[q.shape];
    return (uint32_t)(up(n, sh.bn) / sh.bn) * sh.waves_n;
  };
  return Parts{c.rows, of(c.main), c.rest.us == 0.0 ? 0 : of(c.rest)};
}
uint64_t parts_bytes(const df_loss *d) {
  return up(8ull * parts_of(rows_for(d->rows, d->vocab, d->hidden, false), d->vocab).most() * d->rows, 256);
}

df_status check(const df_loss *d) {
  if (!d || (d->type != DF_TYPE_BF16 && d->type != DF_TYPE_F16)) return DF_ERR_ARG;
  if (d->reduce != DF_REDUCE_NONE && d->reduce != DF_REDUCE_SUM && d->reduce != DF_REDUCE_MEAN) return DF_ERR_ARG;
  if (d->rows > (1u << 21) || d->vocab == 0 || d->vocab > (1u << 21) || d->hidden == 0 || d->hidden % 8 ||
      d->hidden > (1u << 17))
    return DF_ERR_ARG;
  if (d->x_stride < d->hidden || d->x_stride % 8 || d->x_stride > (1u << 21) || d->head_stride < d->hidden ||
      d->head_stride % 8 || d->head_stride > (1u << 21))
    return DF_ERR_ARG;
  if (d->rows && (!d->x || ((uintptr_t)d->x & 15))) return DF_ERR_ARG;
  if (!d->head || ((uintptr_t)d->head & 15)) return DF_ERR_ARG;
  if (d->top > kMaxTop || !(d->temperature >= 1e-3f) || !(d->temperature <= 1e3f)) return DF_ERR_ARG;
  if (d->top == 0) {
    if (d->temperature != 1.f || (d->rows && (!d->labels || ((uintptr_t)d->labels & 7)))) return DF_ERR_ARG;
  } else {
    if (d->teacher_type != DF_TYPE_BF16 && d->teacher_type != DF_TYPE_F16 && d->teacher_type != DF_TYPE_F32)
      return DF_ERR_ARG;
    if (d->rows && (!d->index || ((uintptr_t)d->index & 7) || !d->teacher ||
                    ((uintptr_t)d->teacher & (d->teacher_type == DF_TYPE_F32 ? 3 : 1))))
      return DF_ERR_ARG;
  }
  return DF_OK;
}
Targets targets_of(const df_loss *d) {
  return Targets{d->labels,       d->ignore_index,        d->index,         d->teacher,          d->index_stride,
                 d->teacher_stride, (int)d->teacher_type, d->top,           (uint32_t)d->vocab,  d->temperature};
}
uint32_t per_row(const df_loss *d) { return d->top ? d->top : 1; }
Saved saved_of(const df_loss *d, void *p) {
  float *f = (float *)p;
  return Saved{f, f + 4, (uint32_t *)(f + 4 + d->rows), f + 4 + 2 * d->rows};
}
#define DFH_TRY(e) \
  do {             \
    if ((e) != hipSuccess) return DF_ERR_HIP; \
  } while (0)

template <class T>
df_status loss_rows(const df_loss *d, float *loss, const Saved &sv, uint8_t *ws, hipStream_t s) {
  const uint32_t rows = (uint32_t)d->rows, vocab = (uint32_t)d->vocab, k = (uint32_t)d->hidden;
  const Targets t = targets_of(d);
  const uint16_t *x = (const uint16_t *)d->x, *head = (const uint16_t *)d->head;
  const Head h = {x, head, d->x_stride, d->head_stride, k};
  // few rows with few entries: 96 rows of 16 x 1024, one launch less of 4.5 us; 64
  // x 4096 in four waves would take longer than the launch
  const bool pick = d->top && rows <= 256 && (uint64_t)d->top * k <= 32768;
  if (d->top && !pick) {
    const uint64_t groups = ((uint64_t)rows * d->top + 15) / 16;
    hipLaunchKernelGGL((pick_logits<T>), dim3((uint32_t)(groups < 1u << 20 ? groups : 1u << 20)), dim3(64), 0, s, t, rows, h, sv.picked);
    DFH_TRY(hipGetLastError());
  }
  float2 *parts = (float2 *)ws;
  const RowCut cut = rows_for(rows, vocab, k, false);
  const Parts np = parts_of(cut, vocab);
  const Gemm g = {x, head, d->x_stride, d->head_stride, rows, vocab, k, 0, 0, 0, 0};
  DFH_TRY((product_rows<T, false>(g, EpiStats{parts, rows, kLog2e / d->temperature, d->top ? nullptr : d->labels, sv.picked}, cut, s)));
  float *per = d->reduce == DF_REDUCE_NONE ? loss : (float *)(ws + parts_bytes(d));
  auto *fn = pick ? finish_rows<T, 1, true> : rows <= 256 ? finish_rows<T, 1, false> : finish_rows<T, 8, false>;
  hipLaunchKernelGGL(fn, dim3(rows <= 256 ? rows : (rows + 7) / 8), dim3(256), 0, s, t, rows, (const float2 *)parts, np,
                     h, sv, per);
  DFH_TRY(hipGetLastError());
  return DF_OK;
}

// How a gradient pass is cut: `nv` vocabulary entries a piece (a multiple of
// 256), so that the piece's dz stays within the last-level cache (256 MB; half of
// it, beside the head's rows); dx is cut into `splits` parts of a piece's sum,
// whose planes take the pieces one after the other.
struct Plan {
  uint32_t nv;
  RowCut dx;
  uint64_t dz, xm, planes, fac, total;
  Parts splits() const { return Parts{dx.rows, dx.main.splits, dx.rest.splits}; }
};
Plan plan_of(const df_loss *d, bool want_dx, bool want_dhead) {
  Plan p;
  const uint64_t rows = d->rows, k = d->hidden, v8 = up(d->vocab, 8);
  uint64_t nv = (128ull << 20) / (2 * rows) / 256 * 256;
  if (nv < 2048) nv = 2048;
  if (nv > v8) nv = v8;
  p.nv = (uint32_t)nv;
  p.dx = rows_for(rows, k, nv, true);
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  p.fac = take(4 * (2 + 256 + rows));
  p.dz = take(2 * rows * nv);
  p.xm = take(want_dhead ? 2 * up(rows, 8) * k : 0);
  p.planes = take(want_dx ? 4ull * p.splits().most() * rows * k : 0);
  p.total = at;
  return p;
}

template <class T>
df_status loss_grad(const df_loss *d, const Saved &sv, const float *grad, uint16_t *dx, uint16_t *dhead, uint8_t *ws,
                    float mul, hipStream_t s) {
  const Plan p = plan_of(d, dx != nullptr, dhead != nullptr);
  const uint32_t rows = (uint32_t)d->rows, vocab = (uint32_t)d->vocab, k = (uint32_t)d->hidden;
  const uint32_t mp = (uint32_t)up(rows, 8);
  const Targets t = targets_of(d);
  const uint16_t *x = (const uint16_t *)d->x, *head = (const uint16_t *)d->head;
  const float c = kLog2e / d->temperature;
  float *peak = (float *)(ws + p.fac), *peaks = peak + 2, *gn = peaks + 256;
  uint16_t *dz = (uint16_t *)(ws + p.dz), *xm = (uint16_t *)(ws + p.xm);
  float *planes = (float *)(ws + p.planes);
  const bool own = d->reduce == DF_REDUCE_NONE;  // every row has its own gradient
  if (own && dhead)
    hipLaunchKernelGGL(row_factors, dim3(1), dim3(1024), 0, s, (const uint32_t *)sv.state, rows, grad, gn, peak);
  const bool lifted = own && d->type == DF_TYPE_F16;
  if (lifted && dhead)
    hipLaunchKernelGGL(weighed_peaks, dim3(256), dim3(256), 0, s, x, d->x_stride, rows, k, (const float *)gn, peaks);
  if (dhead)
    hipLaunchKernelGGL((weigh_rows<T>), dim3((mp + 63) / 64, (k + 63) / 64), dim3(256), 0, s, x, d->x_stride, rows, k,
                       (const uint32_t *)sv.state, own ? (const float *)gn : (const float *)nullptr,
                       lifted ? (const float *)peaks : (const float *)nullptr, peak + 1, xm, mp);
  DFH_TRY(hipGetLastError());
  for (uint32_t v0 = 0; v0 < vocab; v0 += p.nv) {
    const uint32_t nv = vocab - v0 < p.nv ? vocab - v0 : p.nv, ldz = (uint32_t)up(nv, 8);
    const uint16_t *hp = head + (uint64_t)v0 * d->head_stride;
    const Gemm gz = {x, hp, d->x_stride, d->head_stride, rows, nv, k, 0, 0, 0, 0};
    DFH_TRY((product_rows<T, false>(gz, EpiDz{dz, ldz, sv.lse2, sv.state, c, mul}, rows_for(rows, nv, k, false), s)));
    hipLaunchKernelGGL((fix_targets<T>), dim3(rows), dim3(64), 0, s, t, sv, v0, nv, c, mul, dz, ldz);
    DFH_TRY(hipGetLastError());
    if (dhead) {
      const Gemm gw = {dz, xm, ldz, mp, nv, k, rows, 0, 0, 0, 0};
      DFH_TRY((product<T, true, false>(gw, EpiStore<>{dhead + (uint64_t)v0 * k, k, own ? peak : grad, own ? peak + 1 : sv.share, d->temperature / mul, nullptr},
                                      cut_for(nv, k, rows, false).shape, 1, s)));
    }
    if (dx) {
      const Gemm gx = {dz, hp, ldz, d->head_stride, rows, k, nv, 0, 0, 0, 0};
      DFH_TRY((product_rows<T, true>(gx, EpiPlane{planes, k, (uint64_t)rows * k, v0 != 0}, p.dx, s)));
    }
  }
  if (dx) {
    hipLaunchKernelGGL((finish_dx<T>), dim3(rows), dim3(256), 0, s, (const float *)planes, p.splits(), rows, k,
                       (const uint32_t *)sv.state, grad, own ? (const float *)nullptr : (const float *)sv.share,
                       d->temperature / mul, dx);
    DFH_TRY(hipGetLastError());
  }
  return DF_OK;
}

}  // namespace

extern "C" {

uint64_t df_loss_saved_bytes(const df_loss *d) {
  return check(d) == DF_OK ? 16 + 4 * d->rows * (2 + per_row(d)) : 0;
}

uint64_t df_loss_workspace_bytes(const df_loss *d) {
  if (check(d) != DF_OK || d->rows == 0) return 0;
  return parts_bytes(d) + up(4 * d->rows, 256);
}

uint64_t df_loss_grad_workspace_bytes(const df_loss *d, int want_dhead) {
  if (check(d) != DF_OK || d->rows == 0) return 0;
  return plan_of(d, true, want_dhead != 0).total;
}

df_status df_vocab_loss(const df_loss *d, float *loss, void *saved, void *workspace, uint64_t workspace_bytes,
                        hipStream_t stream) {
  df_status st = check(d);
  if (st != DF_OK) return st;
  if (d->rows == 0) {
    if (d->reduce == DF_REDUCE_NONE) return DF_OK;
    if (!loss) return DF_ERR_ARG;
    hipLaunchKernelGGL(fill_words, dim3(1), dim3(256), 0, stream, (uint32_t *)loss, (uint64_t)1);
    return hipGetLastError() == hipSuccess ? DF_OK : DF_ERR_HIP;
  }
  if (!loss || !saved || ((uintptr_t)saved & 3) || ((uintptr_t)loss & 3) || !workspace ||
      ((uintptr_t)workspace & 255) || workspace_bytes < df_loss_workspace_bytes(d))
    return DF_ERR_ARG;
  const Saved sv = saved_of(d, saved);
  uint8_t *ws = (uint8_t *)workspace;
  st = d->type == DF_TYPE_BF16 ? loss_rows<BF16>(d, loss, sv, ws, stream) : loss_rows<F16>(d, loss, sv, ws, stream);
  if (st != DF_OK || d->reduce == DF_REDUCE_NONE) return st;
  const float *per = (const float *)(ws + parts_bytes(d));
  hipLaunchKernelGGL(reduce_rows, dim3(1), dim3(1024), 0, stream, per, (const uint32_t *)sv.state, (uint32_t)d->rows,
                     d->reduce == DF_REDUCE_MEAN, loss, sv.share);
  return hipGetLastError() == hipSuccess ? DF_OK : DF_ERR_HIP;
}

df_status df_vocab_loss_grad(const df_loss *d, const void *saved, const float *grad_loss, void *dx, void *dhead,
                             void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
  const df_status st = check(d);
  if (st != DF_OK) return st;
  if ((!dx && !dhead && d->rows) || ((uintptr_t)dx & 15) || ((uintptr_t)dhead & 15)) return DF_ERR_ARG;
  if (d->rows == 0) {
    if (!dhead) return DF_OK;
    hipLaunchKernelGGL(fill_words, dim3(2048), dim3(256), 0, stream, (uint32_t *)dhead, d->vocab * d->hidden / 2);
    return hipGetLastError() == hipSuccess ? DF_OK : DF_ERR_HIP;
  }
  if (!saved || ((uintptr_t)saved & 3) || !grad_loss || ((uintptr_t)grad_loss & 3) || !workspace ||
      ((uintptr_t)workspace & 255) || workspace_bytes < plan_of(d, dx != nullptr, dhead != nullptr).total)
    return DF_ERR_ARG;
  const Saved sv = saved_of(d, const_cast<void *>(saved));
  if (d->type == DF_TYPE_BF16)
    return loss_grad<BF16>(d, sv, grad_loss, (uint16_t *)dx, (uint16_t *)dhead, (uint8_t *)workspace, 1.f, stream);
  return loss_grad<F16>(d, sv, grad_loss, (uint16_t *)dx, (uint16_t *)dhead, (uint8_t *)workspace, 32768.f, stream);
}

}  // extern "C"
