// paged_prompt.cu -- attention of several new tokens per sequence over the paged token cache.
//
// The plainest form: a warp per query row and head walks the tokens that the row sees, its lanes share the head's
// dims, softmax statistics run along.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sr_device.cuh"
#include "sr_kernels.h"
#include "sr_paged.h"

namespace sr {

namespace {

constexpr int kThreads = 128;

// D / 32 neighbouring values of a token, in 32 bits and without 2^e
template <int D, int TYPE>
__device__ __forceinline__ void load_token(float (&x)[D / 32], const void* pages, const PagedView& c, int32_t page, int32_t slot,
                                           int head, int kv_heads, int lane) {
  constexpr int N = D / 32;
  if constexpr (TYPE == SR_PAGE_INT4) {
    const uint8_t* rec = static_cast<const uint8_t*>(pages) + record_at(page, slot, head, kv_heads, c.page_tokens, D);
    const int dim = lane * N;
    const uint32_t u = *reinterpret_cast<const uint16_t*>(rec + (dim / 32) * 256 + (slot & 15) * 16 + (dim % 32) / 4 * 2);
    const uint32_t codes = (u >> 1 | u << 15) & 0xFFFFu;
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(rec[8 * D + (slot & 15) * (D / 16) + dim / 16] << 7)));
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (static_cast<int>(codes >> (4 * (dim % 4 + i)) & 15u) - 8) * s;
  } else {
    const int64_t at = ((static_cast<int64_t>(page) * c.page_tokens + slot) * kv_heads + head) * D + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (TYPE == SR_PAGE_BF16)
        x[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(pages)[at + i]);
      else
        x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(pages)[at + i], __NV_E4M3)));
    }
  }
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads) paged_prompt_kernel(const __grid_constant__ PromptParams p) {
  constexpr int N = D / 32;
  grid_dep_wait();
  grid_dep_launch_dependents();
  const PagedView& c = p.c;
  const int lane = threadIdx.x % 32;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  const int32_t row = static_cast<int32_t>(task / c.n_heads), h = static_cast<int32_t>(task % c.n_heads);
  if (row >= p.row0[p.n]) return;
  int i = 0;
  while (p.row0[i + 1] <= row) ++i;
  const int32_t count = p.row0[i + 1] - p.row0[i], seq = p.id[i];
  const int32_t len = min(max(c.seq_len[seq], 0), c.cap);
  const int32_t sees = p.causal ? max(len - count + (row - p.row0[i]) + 1, 0) : len;
  const int head = h / (c.n_heads / p.kv_heads);
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  const int64_t at = (static_cast<int64_t>(row) * c.n_heads + h) * D + lane * N;
  float q[N], o[N], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    q[k] = __bfloat162float(p.q[at + k]);
    o[k] = 0.f;
  }
  const float scale = fmaxf(c.scale_log2 * (c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[head])) : 1.f), 0x1p-126f);
  const float vscale = c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[p.kv_heads + head])) : 1.f;
  for (int32_t t = 0; t < sees; ++t) {
    const int32_t pg = page_of_group(t >> 4, c.magic), page = table[pg], slot = t - pg * c.page_tokens;
    if (page < 0 || page >= c.n_pages) {
      if (lane == 0) atomicCAS(c.err_word, 0, SR_DEVERR_BAD_PAGE);
      continue;
    }
    float k[N], v[N], x = 0.f;
    load_token<D, TYPE>(k, c.k_pages, c, page, slot, head, p.kv_heads, lane);
    load_token<D, TYPE>(v, c.v_pages, c, page, slot, head, p.kv_heads, lane);
#pragma unroll
    for (int y = 0; y < N; ++y) x = fmaf(q[y], k[y], x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    x *= scale;
    const float m = fmaxf(top, x);
    const float f = top == -INFINITY ? 0.f : ex2_approx(top - m), w = m == -INFINITY ? (x == x ? 0.f : x) : ex2_approx(x - m);
    top = m;
    sum = fmaf(sum, f, w);
#pragma unroll
    for (int y = 0; y < N; ++y) o[y] = fmaf(w, v[y], o[y] * f);
  }
  const float inv = sum == 0.f ? 0.f : vscale / sum;
#pragma unroll
  for (int y = 0; y < N; ++y) p.o[at + y] = __float2bfloat16(sum == 0.f ? 0.f : o[y] * inv);
  if (lane == 0 && p.lse)
    p.lse[static_cast<int64_t>(row) * c.n_heads + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

template <int D, int TYPE>
cudaError_t launch(const PromptParams& p, cudaStream_t st) {
  const int64_t tasks = static_cast<int64_t>(p.row0[p.n]) * p.c.n_heads;
  return launch_dependent(paged_prompt_kernel<D, TYPE>, static_cast<unsigned>((tasks + kThreads / 32 - 1) / (kThreads / 32)),
                          kThreads, 0, st, p);
}

template <int D>
cudaError_t launch(const PromptParams& p, cudaStream_t st) {
  if (p.c.page_type == SR_PAGE_BF16) return launch<D, SR_PAGE_BF16>(p, st);
  if (p.c.page_type == SR_PAGE_INT4) return launch<D, SR_PAGE_INT4>(p, st);
  return launch<D, SR_PAGE_E4M3>(p, st);
}

}  // namespace

cudaError_t launch_paged_prompt(const PromptParams& p, cudaStream_t st) {
  return p.c.head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace sr
