// The 4-bit cache row: 576 e2m1 codes (two a byte, the even dim in the low
// nibble: 288 bytes) and 36 e4m3 scales, one per group of 16 dims.  A value is
// code times scale: e2m1 has two significant bits and e4m3 four, so the product
// has at most six and lies in [2^-10, 2688]: exact in f16, bf16 and fp32.
// A page of ps rows is a block of ps * 324 bytes: the codes of its rows, then
// their scales (so that both are read by contiguous, 16-byte aligned copies).
#pragma once

#include <stdint.h>

namespace mla {

constexpr int kFp4Group = 16;
constexpr int kFp4CodeBytes = 288;   // codes of a row
constexpr int kFp4ScaleBytes = 36;   // scales of a row
constexpr int kFp4RowBytes = kFp4CodeBytes + kFp4ScaleBytes;

namespace ptx {

// Eight e2m1 codes (low nibble of the low byte first) -> four pairs of f16.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Eight fp32 values -> eight e2m1 codes (nearest, ties to even, saturating to +-6).
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* v) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

}  // namespace ptx
}  // namespace mla
