// Keys and values of new tokens into the pages of a cache, and back (gfx950).
//
// In 16 bits a head's vector is copied; in 8 it becomes codes with one scale (rows of
// dfh_quant.h), and reads back as code * scale, rounded once to 16 bits.
//
// Both ways are bound by memory: D / 8 lanes take a vector, 16 bytes each, so a wave
// has several vectors of one or two tokens in flight; keys and values go in one
// launch.  A workgroup finds the sequence of its first token with one wave-wide
// search and walks on from there.
#include <hip/hip_runtime.h>

#include "dfh.h"
#include "dfh_gemm.h"
#include "dfh_pages.h"
#include "dfh_quant.h"

namespace {

using namespace dfh;

// New vectors: [tokens, heads, D], unit stride in D, other strides in elements.
struct Vectors {
  uint16_t *k, *v;
  uint64_t k_token, k_head, v_token, v_head;
};

// The largest bits among the LANES (4, 8, 16 or 32) lanes of a vector.
template <int LANES>
__device__ __forceinline__ uint32_t most_of_lanes(uint32_t v) {
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) {
    const uint32_t o = __shfl_xor(v, d);
    v = v > o ? v : o;
  }
  return v;
}

// Vector i of a call: head i % heads of token i / heads, keys first, then values.
// A wave walks over all vectors; LANES lanes take one.
template <class T, int D, int BITS, bool WRITE>
__global__ __launch_bounds__(256) void move(const Pages c, const Sequences b, const Vectors n) {
  constexpr int LANES = D / 8, PER = 64 / LANES;
  const uint32_t lane = threadIdx.x & 63, at = lane % LANES;
  const uint64_t all = (uint64_t)b.tokens * c.heads;
  const uint64_t wave = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6), waves = (uint64_t)gridDim.x * 4;
  // a run of vectors a wave, so that its tokens are neighbours
  const uint64_t groups = (all + PER - 1) / PER, per = (groups + waves - 1) / waves;
  const uint64_t g0 = wave * per, g1 = g0 + per < groups ? g0 + per : groups;
  if (g0 >= g1) return;
  const int32_t first = b.count ? b.starts[0] : 0;
  uint32_t s = sequence_of(b, (int32_t)(g0 * PER / c.heads));
  Span p = {0, 0, 0, 0};
  if (s < b.count) p = span_of(b, s);
  for (uint64_t g = g0; g < g1; g++) {
    const uint64_t i = g * PER + lane / LANES;
    const bool there = i < all;
    const int32_t t = there ? (int32_t)(i / c.heads) : 0;
    const uint32_t head = there ? (uint32_t)(i % c.heads) : 0;
    // the sequence of the group's first token; lanes of later ones look for their own
    const int32_t t0 = (int32_t)(g * PER / c.heads);
    if (t0 >= p.last || t0 < p.first) {
      s = sequence_of(b, t0);
      if (s < b.count) p = span_of(b, s);
    }
    uint32_t mine = s;
    Span q = p;
    if (there && t >= p.last) {
      if (mine == b.count && t0 < first) mine = 0;  // a group that begins before the first sequence
      // starts are in order: walk on (a group holds at most 16 tokens)
      while (mine < b.count) {
        q = span_of(b, mine);
        if (t < q.last) break;
        mine++;
      }
    }
    int64_t token = -1;
    if (there && mine < b.count && t >= q.first && t < q.last) token = token_at(c, b, mine, t + q.ahead);
    if (WRITE && token < 0) continue;
    const uint64_t row = token < 0 ? 0 : row_of(c, token, head);
    uint16_t *const vec[2] = {n.k + t * n.k_token + head * n.k_head + at * 8, n.v + t * n.v_token + head * n.v_head + at * 8};
    uint8_t *const page[2] = {c.k + row * (D * BITS / 8) + at * BITS, c.v + row * (D * BITS / 8) + at * BITS};
    float *const scale[2] = {c.k_scales + row, c.v_scales + row};
    // both are read before either is written, the order that the compiler keeps (write_prompts below)
    if constexpr (WRITE) {
      u32x4 x[2];
#pragma unroll
      for (int kv = 0; kv < 2; kv++) x[kv] = *(const u32x4 *)vec[kv];
#pragma unroll
      for (int kv = 0; kv < 2; kv++) {
        if constexpr (BITS == 16) {
          *(u32x4 *)page[kv] = x[kv];
        } else {
          Quantiser z;
          z.init(T{}, most_of_lanes<LANES>(joined(most_bits(x[kv], 0))));
          *(u32x2 *)page[kv] = z.codes(T{}, x[kv]);
          if (at == 0) *scale[kv] = z.scale;
        }
      }
    } else if (there) {
      u32x4 x[2] = {};
      if (token >= 0) {
        if constexpr (BITS == 16) {
#pragma unroll
          for (int kv = 0; kv < 2; kv++) x[kv] = *(const u32x4 *)page[kv];
        } else {
          u32x2 o[2];
          float f[2];
#pragma unroll
          for (int kv = 0; kv < 2; kv++) {
            o[kv] = *(const u32x2 *)page[kv];
            f[kv] = *scale[kv];
          }
#pragma unroll
          for (int kv = 0; kv < 2; kv++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const uint32_t w = o[kv][e / 2] >> (16 * (e & 1));
              x[kv][e] = pack2(T{}, (float)(int8_t)w * f[kv], (float)(int8_t)(w >> 8) * f[kv]);
            }
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; kv++) *(u32x4 *)vec[kv] = x[kv];
    }
  }
}

template <class T, int BITS, bool WRITE>
auto kernel_of(uint32_t dim) {
  return dim == 32    ? move<T, 32, BITS, WRITE>
         : dim == 64  ? move<T, 64, BITS, WRITE>
         : dim == 128 ? move<T, 128, BITS, WRITE>
                      : move<T, 256, BITS, WRITE>;
}
template <bool WRITE>
df_status moved(const df_cache *cache, const df_cache_batch *batch, const Vectors &n, uint64_t tokens, hipStream_t s) {
  const Pages c = pages_of(cache);
  const Sequences b = sequences_of(batch, tokens);
  auto *fn = cache->type == DF_TYPE_BF16
                 ? (cache->bits == 8 ? kernel_of<BF16, 8, WRITE>(c.dim) : kernel_of<BF16, 16, WRITE>(c.dim))
                 : (cache->bits == 8 ? kernel_of<F16, 8, WRITE>(c.dim) : kernel_of<F16, 16, WRITE>(c.dim));
  const uint64_t groups = (tokens * c.heads * c.dim / 8 + 63) / 64, blocks = (groups + 3) / 4;
  hipLaunchKernelGGL(fn, dim3((uint32_t)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s, c, b, n);
  return hipGetLastError() == hipSuccess ? DF_OK : DF_ERR_HIP;
}

bool strides_ok(uint64_t token, uint64_t head) {
  return token % 8 == 0 && head % 8 == 0 && token <= (1u << 30) && head <= (1u << 30);
}

}  // namespace

extern "C" {

df_status df_cache_write(const df_cache *cache, const df_cache_batch *batch, const void *k, uint64_t k_token_stride,
                         uint64_t k_head_stride, const void *v, uint64_t v_token_stride, uint64_t v_head_stride,
                         uint64_t tokens, hipStream_t stream) {
  if (!cache_ok(cache) || !batch_ok(batch, tokens)) return DF_ERR_ARG;
  if (tokens == 0 || batch->seqs == 0) return DF_OK;
  if (!k || !v || (((uintptr_t)k | (uintptr_t)v) & 15) || !strides_ok(k_token_stride, k_head_stride) ||
      !strides_ok(v_token_stride, v_head_stride))
    return DF_ERR_ARG;
  return moved<true>(cache, batch, Vectors{(uint16_t *)k, (uint16_t *)v, k_token_stride, k_head_stride, v_token_stride, v_head_stride},
                     tokens, stream);
}

df_status df_cache_read(const df_cache *cache, const df_cache_batch *batch, void *k, void *v, uint64_t tokens,
                        hipStream_t stream) {
  if (!cache_ok(cache) || !batch_ok(batch, tokens)) return DF_ERR_ARG;
  if (tokens == 0) return DF_OK;
  if (!k || !v || (((uintptr_t)k | (uintptr_t)v) & 15)) return DF_ERR_ARG;
  const uint64_t head = cache->head_dim, token = head * cache->kv_heads;
  return moved<false>(cache, batch, Vectors{(uint16_t *)k, (uint16_t *)v, token, head, token, head}, tokens, stream);
}

}  // extern "C"
