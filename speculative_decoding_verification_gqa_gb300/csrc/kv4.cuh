// kv4.cuh -- the 4-bit cache format: a row (position, KV head) of d elements is d E2M1 codes
// (two to a byte, the even element in the low nibble) and d / 16 E4M3 scales, one for each
// 16 consecutive elements; an element stands for head scale x block scale x e2m1(code). The
// product of a code and its block scale has at most 6 significant bits and lies in [2^-10,
// 2688] (or is 0), so f16 holds it exactly.
#pragma once

#include <cuda_fp16.h>

#include "internal.cuh"

namespace sv {
namespace {

// Eight E2M1 codes (low nibble first) -> four f16 pairs, exact. (The conversion of a byte's two
// codes takes about 3 clocks of a warp and scheduler; placing the bits by shifts and masks took
// 5.7.)
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two E4M3 codes in the low 16 bits -> an f16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
  uint32_t h;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n"
      : "=r"(h)
      : "r"(c));
  return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t lo_twice(uint32_t h) { return __byte_perm(h, 0, 0x1010); }
__device__ __forceinline__ uint32_t hi_twice(uint32_t h) { return __byte_perm(h, 0, 0x3232); }

}  // namespace
}  // namespace sv
