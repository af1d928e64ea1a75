// Shared by the kernels of the cache held in 4 bits (include/paged_q4.h): its arrays, and the numbers
// that codes stand for.
#pragma once

#include <cuda_fp16.h>

#include "../../include/paged_q4.h"
#include "paged_tc.cuh"

namespace rglru {

// Codes and scales of keys and values; strides in bytes.
struct Q4Cache {
  const uint8_t* kc;
  const uint8_t* ks;
  const uint8_t* vc;
  const uint8_t* vs;
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  int64_t ks_page, ks_token, ks_head, vs_page, vs_token, vs_head;
  int split;  // heads of the attention's work division a key/value head
};

// The eight values of a word of codes, as four pairs of f16.
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two neighbouring scales as a pair of f16.
__device__ __forceinline__ uint32_t q4_scales(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t q4_mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}

// Attention over the cache in 4 bits (paged_attn_q4.cu), `rows` a request in the mean.
cudaError_t launch_paged_attn_q4(PagedArgs a, const Q4Cache& c, bool f32, int rows, cudaStream_t s);
size_t paged_attn_q4_ws_bytes(const paged_shape* s, int rows);

}  // namespace rglru
