// quant_block.cuh — block-scaled quantisation of f32 values shared by the 4-bit cast and the norm:
// E2M1 conversion, block scales and where they lie.
//
// Formats ("FP8 混合精度训练工程实践" §九, Blackwell microscaling, in its 8- and 4-bit forms):
//   MXFP8   E4M3 / E5M2 codes, one E8M0 scale 2^X per 32 values, X = floor(log2 amax) - emax
//   MXFP4   E2M1 codes (emax 2), one E8M0 scale per 32 values
//   NVFP4   E2M1 codes, one E4M3 scale s per 16 values under a per-tensor f32 scale g:
//           s = e4m3((amax * g) / 6), code = e2m1(x * (g / s)); s = 0 makes every code of the block +-0
// Every f32 operation is rounded separately (no fused multiply-add), so a code is a function of the
// value, the block maximum and g alone.
#pragma once

#include "ptx.cuh"

namespace fp8t {
namespace blk {

enum : int { kNone = 0, kFP8 = 1, kMXFP8 = 2, kMXFP4 = 3, kNVFP4 = 4 };   // fp8t_quant

// Eight f32 -> eight E2M1 codes, round to nearest even, saturating at +-6; value 0 in the low nibble.
// (E2M1 has no NaN: a NaN value becomes a finite code, its block's scale carries the NaN.)
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Shared exponent of a block from the bit pattern of its largest f32 magnitude; NaN is the caller's.
__device__ __forceinline__ int e8m0_exponent(uint32_t m, int emax) {
  if (m == 0) return -127;
  if (m >= 0x7F800000u) return 127;
  const int e = static_cast<int>(m >> 23);
  const int fl = e ? e - 127 : (31 - __clz(m)) - 149;         // floor(log2) of normal / subnormal
  return max(-127, min(127, fl - emax));
}
// 2^-X (2^-127 is the subnormal 0x00400000).
__device__ __forceinline__ float pow2_neg(int X) {
  return X == 127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(127 - X) << 23);
}

// E8M0 block: the scale byte and the factor the block's values are multiplied by. A NaN in the block
// gives the byte 0xFF and unit scale.
__device__ __forceinline__ uint8_t e8m0_scale(uint32_t amax_bits, int emax, float& factor) {
  if (amax_bits > 0x7F800000u) {
    factor = 1.0f;
    return 0xFF;
  }
  const int X = e8m0_exponent(amax_bits, emax);
  factor = pow2_neg(X);
  return static_cast<uint8_t>(X + 127);
}

// NVFP4 block: E4M3 scale byte and factor g / s. A NaN (block maximum or g) gives the byte 0x7F.
__device__ __forceinline__ uint8_t nvfp4_scale(uint32_t amax_bits, float g, float& factor) {
  const float t = __fdiv_rn(__fmul_rn(__uint_as_float(amax_bits), g), 6.0f);
  if (t != t) {
    factor = 1.0f;
    return 0x7F;
  }
  const uint32_t c = cvt_fp8x2<0>(t, 0.0f) & 0xFFu;            // t >= 0: codes 0 .. 0x7E
  // decode: the E4M3 exponent and mantissa are f32's with another bias; subnormals are multiples of 2^-9
  const float s = c < 8u ? static_cast<float>(c) * 0.001953125f : __uint_as_float((c << 20) + (120u << 23));
  factor = c ? __fdiv_rn(g, s) : 0.0f;
  return static_cast<uint8_t>(c);
}

// Scale bytes are kept in 512-byte atoms of 128 rows x 4 scales: byte (i % 32) * 16 + (i / 32) * 4 + j.
// Offset of row r's 32-bit word (four consecutive scales) number w when a row block holds `words` atoms.
__host__ __device__ __forceinline__ int64_t atom_word(int64_t r, int64_t w, int64_t words) {
  return ((r >> 7) * words + w) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}
// Atoms along K of one row block: MXFP8 one per 128 values as K is; the 4-bit formats pad K to a
// multiple of 256 (one k-block of the 4-bit GEMM), so 2 (MXFP4) or 4 (NVFP4) per 256 values.
__host__ __device__ __forceinline__ int64_t atoms_per_row(int64_t K, int kind) {
  return kind == kMXFP8 ? (K + 127) / 128 : (K + 255) / 256 * (kind == kMXFP4 ? 2 : 4);
}

}  // namespace blk
}  // namespace fp8t
