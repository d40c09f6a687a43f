// The 4-bit cache format: its layout, and conversions to and from it.
//
// A cached feature is c s u: c a 4-bit float (e2m1: 0, .5, 1, 1.5, 2, 3, 4, 6 and
// their negatives), s the 8-bit float (e4m3) of its group of 16 features, u a power
// of two of the whole cache.  c s has at most six significant bits, so it is exact in
// fp16 (its range, 2^-10 to 2,688, fits too) and in bf16, and no product of the
// attention starts from a rounded key or value.
//
// A page of one KV head is cut into tiles of 16 tokens of 9 D bytes, so that every
// run of tiles is one contiguous, 16-byte aligned copy with its scales.  In a tile,
// group j has a strip of 128 bytes: eight places of two tokens, 8 bytes of codes
// each, the even feature in the low half of a byte; behind the strips each group has
// its 16 scales.  Tokens 2 p and 2 p + 1 are in place p ^ (j * 128 / D) of strip j: a
// strip spans all banks of the shared memory, and both products read it with 16-byte
// loads, keys by token and four groups at once, values by group and four tokens;
// the exclusive or keeps each quarter of a warp on eight different places.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace cpattn {

constexpr int kFp4Tile = 16;        // tokens of a tile
constexpr float kFp4Top = 6.f;      // largest code value
constexpr float kFp4MinScale = 0.001953125f;  // smallest e4m3, 2^-9
constexpr float kFp4MaxScale = 448.f;

template <int D>
struct Fp4 {
  static constexpr int kGroups = D / 16;
  static constexpr int kTileBytes = 9 * D;
  static constexpr int kScales = 8 * D;  // offset of the scales
  // Offset of the 16 bytes of tokens 2 p and 2 p + 1 of group j.
  static __device__ __forceinline__ int place(int j, int p) {
    return j * 128 + ((p ^ (j * (128 / D))) << 4);
  }
};

// Eight codes to four pairs of fp16, in the order of the features.
__device__ __forceinline__ void fp4x8_to_f16(uint32_t w, uint32_t* o) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Two scales (the low 16 bits) to fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t s) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}\n"
      : "=r"(r)
      : "r"(s));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t v, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}\n"
      : "=f"(lo), "=f"(hi)
      : "r"(v));
}

// The scale byte nearest to x >= 0 (halves to the even one), and its value.
__device__ __forceinline__ uint32_t to_e4m3(float x, float& value) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  float none;
  f16x2_to_f32(e4m3x2_to_f16(r), value, none);
  return r & 0xffu;
}

// Four values to codes, the first in the low half of the first byte; halves to
// the even code, values beyond the range to 6.
__device__ __forceinline__ uint32_t to_fp4x4(float a, float b, float c, float d) {
  uint16_t r;
  asm("{\n\t.reg .b8 x, y;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 y, %4, %3;\n\t"
      "mov.b16 %0, {x, y};\n\t}\n"
      : "=h"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

}  // namespace cpattn
