// widen.cuh -- 8-bit codes to fp16, exactly.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "decode.h"

namespace nmk {

__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Two codes in the low 16 bits -> two fp16, exactly (e4m3, NaN included).
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// Four codes of a word -> two words of two fp16.  int8: the byte with its sign
// bit flipped under 0x64 is the fp16 1024 + 128 + code.
template <int TYPE>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (TYPE == kCacheE4m3) {
    lo = e4m3x2_to_half2(w);
    hi = e4m3x2_to_half2(w >> 16);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = byte_perm(u, 0x64646464u, 0x4140), b = byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off);
    __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  }
}

// Halves of w that are infinite or NaN: bit 0, bit 1.
__device__ __forceinline__ uint32_t bad_halves(uint32_t w) {
  return ((w & 0x7C00u) == 0x7C00u ? 1u : 0u) | ((w & 0x7C000000u) == 0x7C000000u ? 2u : 0u);
}

}  // namespace nmk
