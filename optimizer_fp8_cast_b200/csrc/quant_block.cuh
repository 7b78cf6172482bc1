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

// Pairs of f32 in a 64-bit register; each half is rounded as the scalar operation would be.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float lo(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
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

// E8M0 block: the scale byte X + 127 of the largest f32 magnitude's bit pattern, and the factor 2^-X that the
// block's values are multiplied by. With e the pattern's exponent field, floor(log2 amax) is e - 127 for a normal
// amax, so the byte is e - emax, clamped at 0 (X = -127); a subnormal or zero amax (e = 0) clamps there too.
// An infinity gives 254 (X = 127; 2^-127 is the subnormal 0x00400000), a NaN 0xFF and unit scale.
__device__ __forceinline__ uint8_t e8m0_scale(uint32_t amax_bits, int emax, float& factor) {
  uint32_t byte = static_cast<uint32_t>(max(static_cast<int>(amax_bits >> 23) - emax, 0));
  uint32_t f = (254u - byte) << 23;
  if (amax_bits >= 0x7F800000u) {
    byte = amax_bits > 0x7F800000u ? 255u : 254u;
    f = amax_bits > 0x7F800000u ? 0x3F800000u : 0x00400000u;
  }
  factor = __uint_as_float(f);
  return static_cast<uint8_t>(byte);
}

// E4M3 code (0 .. 0x7E) of (amax * g) / 6, or 0x7F for a NaN.
// The division is replaced by a multiplication where that cannot change the code. Let t = amax * g and
// p = rn(t * rn(1/6)), v = rn(t / 6); they are at most one f32 apart. The codes differ only if a
// rounding border (a middle of two E4M3 values, an f32 of at most five significant bits) lies on one of the
// two. v is a border only for t = 6 * border exactly (t's neighbours are 2/3 of a step of v away or more),
// and then p is the same number: rn(1/6) is 1/6 * (1 + 2^-25), and border * (1 + 2^-25) rounds back to the
// border. So whenever p is not a number of at most five significant bits, its code is v's.
__device__ __forceinline__ uint32_t nvfp4_scale_code(uint32_t amax_bits, float g) {
  const float t = __fmul_rn(__uint_as_float(amax_bits), g);
  float p = __fmul_rn(t, 0.16666667163372040f);
  if ((__float_as_uint(p) & 0x7FFFFu) == 0) p = __fdiv_rn(t, 6.0f);
  return p > 0.0f ? cvt_fp8x2<0>(p, 0.0f) & 0xFFu : p != p ? 0x7Fu : 0u;      // a g below 0 counts as 0
}
// g / s of a scale code (1 for the NaN code, 0 for s = 0). The E4M3 exponent and mantissa are f32's with
// another bias; subnormals are multiples of 2^-9.
__device__ __forceinline__ float nvfp4_factor(uint32_t c, float g) {
  const float s = c < 8u ? static_cast<float>(c) * 0.001953125f : __uint_as_float((c << 20) + (120u << 23));
  return c == 0x7Fu ? 1.0f : c ? __fdiv_rn(g, s) : 0.0f;
}
// NVFP4 block: E4M3 scale byte and factor g / s. A NaN (block maximum or g) gives the byte 0x7F.
__device__ __forceinline__ uint8_t nvfp4_scale(uint32_t amax_bits, float g, float& factor) {
  const uint32_t c = nvfp4_scale_code(amax_bits, g);
  factor = nvfp4_factor(c, g);
  return static_cast<uint8_t>(c);
}

// The CTA's largest f32 magnitude pattern into *amax_bits, a NaN as the canonical one; every thread calls. One
// atomic per CTA: one per warp, all to the same address, took 0.9 us for 2368 warps. `tops`: a word per warp.
__device__ __forceinline__ void cta_amax(unsigned int* amax_bits, uint32_t top, uint32_t* tops) {
  const int lane = threadIdx.x & 31;
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  top = __reduce_max_sync(0xffffffffu, lane < static_cast<int>(blockDim.x >> 5) ? tops[lane] : 0u);
  if (lane == 0 && top) atomicMax(amax_bits, top > 0x7F800000u ? 0x7FC00000u : top);
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
