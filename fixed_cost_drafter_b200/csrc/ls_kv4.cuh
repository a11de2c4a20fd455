// The 4-bit KV cache's layout and element format (struct ls_paged_kv4): e2m1 codes with one
// e4m3 scale per 16 elements of a row. A code's value has 2 significant bits and a scale 4, so
// their product has at most 6 and lies in [2^-10, 2688]: bf16 and fp16 hold it exactly.
#pragma once
#include <cuda_fp16.h>

#include "ls_common.cuh"

namespace ls {

constexpr int kKv4Group = 16;

// Bytes of one KV head's part of a page: codes and scales of page_size keys and values.
__host__ __device__ inline int kv4_block_bytes(int page_size, int D) { return page_size * (D + D / 8); }

// Where a slot's row lies in its (page, head) block, and the block's sections.
struct Kv4Row {
  unsigned char *k_codes, *v_codes, *k_scales, *v_scales;
};
__device__ inline Kv4Row kv4_row(unsigned char* block, int page_size, int D, int off) {
  Kv4Row r;
  r.k_codes = block + off * (D / 2);
  r.v_codes = block + (page_size + off) * (D / 2);
  unsigned char* sc = block + page_size * D;
  r.k_scales = sc + off * (D / kKv4Group);
  r.v_scales = sc + (page_size + off) * (D / kKv4Group);
  return r;
}

// Eight e2m1 codes as fp16 values, the low half of each byte first.
__device__ inline void e2m1x8_to_half2(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two e4m3 scales (16 bits) as fp16 values.
__device__ inline uint32_t e4m3x2_to_half2(uint16_t s) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(s));
  return h;
}
__device__ inline float e4m3_to_f32(uint32_t byte) {
  const uint32_t h = e4m3x2_to_half2(uint16_t(byte));
  return __half2float(__ushort_as_half(uint16_t(h & 0xffffu)));
}
__device__ inline uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ inline float2 half2_to_f2(uint32_t h) {
  return make_float2(__half2float(__ushort_as_half(uint16_t(h & 0xffffu))), __half2float(__ushort_as_half(uint16_t(h >> 16))));
}

}  // namespace ls
