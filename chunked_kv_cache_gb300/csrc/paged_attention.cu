// paged_attention.cu -- attention of one new token per sequence over the paged
// token cache, and the attention weight that each cached token draws.
//
//   x_h(t) = scale * q_h . k(t),  o_h = sum_t e^(x_h(t) - lse_h) v(t),
//   lse_h = ln sum_t e^x_h(t),    mass(t) <- decay * mass(t) + sum_h e^(x_h(t) - lse_h).
//
// The simplest form: one warp per sequence and query head walks the tokens, its
// lanes across the head dimension; a second launch forms each token's weight from
// the log-sum-exps, one warp per token.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sr_device.cuh"
#include "sr_kernels.h"
#include "sr_paged.h"

namespace sr {

namespace {

__device__ __forceinline__ int32_t live_len(const PagedView& c, int32_t seq) {
  return min(max(c.seq_len[seq], 0), c.cap);
}

template <int D>
__device__ __forceinline__ void load_row(const PagedView& c, const void* pages, int64_t row, int head, float (&x)[D / 32],
                                         int lane) {
  const int64_t at = (row * c.n_kv + head) * D;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    if (c.page_type == SR_PAGE_BF16)
      x[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(pages)[at + lane + 32 * i]);
    else
      x[i] = static_cast<float>(static_cast<const __nv_fp8_e4m3*>(pages)[at + lane + 32 * i]);
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}

template <int D>
__global__ void __launch_bounds__(128) paged_attn_simple(const __grid_constant__ PagedAttnParams p) {
  grid_dep_wait();
  const PagedView& c = p.c;
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) / 32, lane = threadIdx.x % 32;
  if (warp >= p.b.n * c.n_heads) return;
  const int i = warp / c.n_heads, h = warp % c.n_heads, kv = h / c.group;
  const int32_t seq = p.b.id[i];
  const int32_t len = live_len(c, seq);
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  const float ks = c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[kv])) : 1.f;
  const float vs = c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[c.n_kv + kv])) : 1.f;
  float q[D / 32], o[D / 32] = {};
  for (int k = 0; k < D / 32; ++k)
    q[k] = __bfloat162float(p.q[(static_cast<int64_t>(i) * c.n_heads + h) * D + lane + 32 * k]);
  float m = -INFINITY, l = 0.f;
  for (int32_t t = 0; t < len; ++t) {
    const int64_t row = paged_row(table, t, c.page_tokens, c.n_pages);
    if (row < 0) {
      if (lane == 0) atomicCAS(c.err_word, 0, SR_DEVERR_BAD_PAGE);
      continue;
    }
    float k[D / 32], v[D / 32];
    load_row<D>(c, c.k_pages, row, kv, k, lane);
    load_row<D>(c, c.v_pages, row, kv, v, lane);
    float s = 0.f;
    for (int j = 0; j < D / 32; ++j) s = fmaf(q[j], k[j], s);
    s = warp_sum(s) * ks * c.scale_log2;
    const float m1 = fmaxf(m, s);
    const float f = exp2f(m - m1), w = exp2f(s - m1);
    l = l * f + w;
    for (int j = 0; j < D / 32; ++j) o[j] = o[j] * f + w * v[j];
    m = m1;
  }
  const float inv = l > 0.f ? vs / l : (l == 0.f ? 0.f : l);
  const int64_t out = static_cast<int64_t>(i) * c.n_heads + h;
  for (int j = 0; j < D / 32; ++j) p.o[out * D + lane + 32 * j] = __float2bfloat16(o[j] * inv);
  const float lse = m == -INFINITY ? m : (m + log2f(l)) * 0.69314718055994531f;
  if (lane == 0) {
    if (p.lse) p.lse[out] = lse;
    p.ws_lse[out] = lse;
  }
}

template <int D>
__global__ void __launch_bounds__(128) paged_mass_simple(const __grid_constant__ PagedAttnParams p) {
  grid_dep_wait();
  const PagedView& c = p.c;
  const int lane = threadIdx.x % 32;
  const int i = blockIdx.x % p.b.n;
  const int32_t seq = p.b.id[i];
  const int32_t len = live_len(c, seq);
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  for (int32_t t = (blockIdx.x / p.b.n) * 4 + threadIdx.x / 32; t < len; t += gridDim.x / p.b.n * 4) {
    const int64_t row = paged_row(table, t, c.page_tokens, c.n_pages);
    if (row < 0) continue;
    float w = 0.f;
    for (int kv = 0; kv < c.n_kv; ++kv) {
      const float ks = c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[kv])) : 1.f;
      float k[D / 32];
      load_row<D>(c, c.k_pages, row, kv, k, lane);
      for (int g = 0; g < c.group; ++g) {
        const int64_t out = static_cast<int64_t>(i) * c.n_heads + kv * c.group + g;
        float s = 0.f;
        for (int j = 0; j < D / 32; ++j) s = fmaf(__bfloat162float(p.q[out * D + lane + 32 * j]), k[j], s);
        w += exp2f(warp_sum(s) * ks * c.scale_log2 - p.ws_lse[out] * 1.4426950408889634f);
      }
    }
    if (lane == 0) {
      float* m = c.token_mass + static_cast<int64_t>(seq) * c.cap + t;
      *m = fmaf(p.mass_decay, *m, w);
    }
  }
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnParams& p, cudaStream_t st) {
  const unsigned grid = (p.b.n * p.c.n_heads + 3) / 4;
  auto k = p.c.head_dim == 128 ? paged_attn_simple<128> : paged_attn_simple<64>;
  cudaError_t e = launch_dependent(k, grid, 128, 0, st, p);
  if (e != cudaSuccess || p.mass_decay < 0.f) return e;
  auto m = p.c.head_dim == 128 ? paged_mass_simple<128> : paged_mass_simple<64>;
  return launch_dependent(m, static_cast<unsigned>(p.b.n) * 64, 128, 0, st, p);
}

}  // namespace sr
