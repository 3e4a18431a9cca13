// kv4.cuh -- the 4-bit cache's format (include/affinity.h) on the device.
//
// A code's eight magnitudes and a scale's bytes have conversions of their own (two codes of a byte, or two scales,
// to a pair of fp16 numbers: 64 or more pairs a clock and SM), and code * scale is exact in fp16: six significant
// bits between 2^-10 and 2688.  So a pair of elements costs a conversion and a product, and fp16 is what the
// attention's products take.  (Building bf16 pairs from the bits, with shifts and masks, ran at a quarter of that.)
#pragma once

#include "step.cuh"

#include <cstdint>

namespace aff {

// 32 elements, 16 bytes of codes and two scales, are a chunk.
__host__ __device__ __forceinline__ constexpr int kv4_chunks(int d) { return (d + 31) / 32; }

struct Kv4Pool {              // by value in the kernels' parameters
  const uint8_t *k, *v;
  int64_t page_stride, group_stride;
  int32_t n;                  // chunks of a token's row
  int32_t scales;             // where a page's scales begin: 16 n page_size
};

inline Kv4Pool kv4_pool(const aff_kv4_cache* c) {
  const int n = kv4_chunks(c->d_head);
  return {static_cast<const uint8_t*>(c->k), static_cast<const uint8_t*>(c->v), c->page_stride, c->group_stride, n,
          16 * n * c->page_size};
}

#ifdef __CUDACC__
// The scale byte of a token's block from the page's start.
__device__ __forceinline__ int kv4_scale_at(const Kv4Pool& p, int token, int block) {
  return p.scales + ((token >> 2) * 2 * p.n + block) * 4 + (token & 3);
}

// Eight codes to four pairs of fp16 numbers, (0, 1) .. (6, 7).
__device__ __forceinline__ void kv4_decode(uint32_t w, uint32_t (&h)[4]) {
  asm("{.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two scales (the low 16 bits) to a pair of fp16 numbers.
__device__ __forceinline__ uint32_t kv4_scale_pair(uint32_t two) {
  uint32_t r;
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Which of four scale bytes are NaN (0x7F; the sign is not looked at): their top bits.
__device__ __forceinline__ uint32_t kv4_nan_scales(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
#endif

}  // namespace aff
