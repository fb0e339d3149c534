// sr_paged_device.cuh -- decoding of the paged cache's pages of fewer than 16 bits, shared by the kernels that read
// them. Internal to libsr.so.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "sr_paged.h"

namespace sr {

// two e4m3 values (the low 16 bits) as fp16, exactly
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t x) {
  uint32_t y;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(static_cast<uint16_t>(x)));
  return y;
}

// ---- 4-bit codes as fp16. A mask puts a code c into the fraction of 16 (16 + c / 32) or of 1 (1 + c / 32); one fused
// product and sum with its scale s then leaves (c - 8) / 32 * s, exactly: at most 7 significant bits, never below fp16's
// smallest number. Four pairs of one word in 9 instructions, scale and all.
__device__ __forceinline__ uint32_t half2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// (x & mask) | bits in one instruction: both constants from registers, since it has room for one of its own
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}
struct DecodeMasks {
  uint32_t lo, hi, in16, in1;
};
__device__ __forceinline__ DecodeMasks decode_masks() {
  DecodeMasks m;
  asm volatile("mov.u32 %0, 0x001E001E; mov.u32 %1, 0x01E001E0; mov.u32 %2, 0x4C004C00; mov.u32 %3, 0x3C003C00;"
               : "=r"(m.lo), "=r"(m.hi), "=r"(m.in16), "=r"(m.in1));
  return m;
}
// What a decoding needs of a pair of scales.
struct ScalePair {
  uint32_t s, off16, off1;
};
__device__ __forceinline__ ScalePair scale_pair(uint32_t s) {
  return {s, half2_mul(s, 0xCC10CC10u), half2_mul(s, 0xBD00BD00u)};     // -16.25 s, -1.25 s
}
// y[i]: the i-th value of the word's low unit and of its high one.
__device__ __forceinline__ void decode_word(uint32_t (&y)[4], uint32_t w, const ScalePair& s, const DecodeMasks& m) {
  const uint32_t z = __byte_perm(w, 0, 0x2301);
  y[0] = half2_fma(and_or(w, m.lo, m.in16), s.s, s.off16);
  y[1] = half2_fma(and_or(w, m.hi, m.in1), s.s, s.off1);
  y[2] = half2_fma(and_or(z, m.lo, m.in16), s.s, s.off16);
  y[3] = half2_fma(and_or(z, m.hi, m.in1), s.s, s.off1);
}
constexpr float kDecoded = 32.f;      // a value is so many times what decode_word leaves


// Value `dim` of token t (16-bit floats of the pages' type, fp16 for those of fewer bits), as the tiles would hold it.
template <int D, int TYPE>
__device__ __forceinline__ float page_value(const PagedView& c, int32_t kv_heads, const void* pages, int32_t seq, int32_t t, int head, int dim) {
  const int32_t pg = page_of_group(t >> 4, c.magic), slot = t - pg * c.page_tokens;
  const int32_t page = __ldg(c.table + static_cast<int64_t>(seq) * c.max_pages + pg);
  if (page < 0 || page >= c.n_pages) return 0.f;
  if constexpr (TYPE == SR_PAGE_INT4) {
    const uint8_t* rec = static_cast<const uint8_t*>(pages) + record_at(page, slot, head, kv_heads, c.page_tokens, D);
    const uint32_t u = *reinterpret_cast<const uint16_t*>(rec + (dim / 32) * 256 + (slot & 15) * 16 + (dim % 32) / 4 * 2);
    const int code = static_cast<int>(((u >> 1 | u << 15) & 0xFFFFu) >> (4 * (dim % 4)) & 15u);
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(rec[8 * D + (slot & 15) * (D / 16) + dim / 16] << 7)));
    return static_cast<float>(code - 8) * s / kDecoded;
  } else {
    const int64_t at = ((static_cast<int64_t>(page) * c.page_tokens + slot) * kv_heads + head) * D + dim;
    if constexpr (TYPE == SR_PAGE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(pages)[at]);
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(pages)[at], __NV_E4M3)));
  }
}

}  // namespace sr
