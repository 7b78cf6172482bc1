// gated.cuh — the gated feed-forward block in FP8: both projections, the activation and the product in one kernel, and
// the gradient of all that in the product that brings it.
//
// Forward. W holds the gate's and the up projection's weights side by side (N columns each):
//   [G | U] = (A . W) * sa * sb,  h = act(G) * U,  act(g) = g * sigmoid(w(g))
//   w = g (SiLU) or 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU in its tanh form: (1 + tanh(z)) / 2 = sigmoid(2z))
// One accumulator of a pair tile holds 128 columns of G and the same 128 of U: the even CTA's half of B is 128 gate rows, the
// odd CTA's the up rows of the same columns, so every lane has g and u of an element at the same time and h never
// leaves the registers before it is rounded. h is formed from the f32 accumulators; G and U are rounded to BF16 only
// where they are kept for the gradient.
// Backward. dH = (dY . Wd^T) * sa * sb stays in the accumulator (256 columns); with s = sigmoid(w(g))
//   dG = dH * u * (s + g s (1 - s) w'(g)),  dU = dH * g s
// written as [dG | dU] side by side under one scale, so that dX = [dG | dU] . W^T and dW = X^T . [dG | dU] are one
// product each.
#pragma once

#include "gemm_pair.cuh"

namespace fp8t {
namespace gated {

using namespace pair;

enum : int { kSilu = 1, kGelu = 2 };                       // fp8t_act

struct alignas(64) Params {
  CUtensorMap a, b;                // A in 128-row boxes (or [K][M]), B
  CUtensorMap o0, o1;              // 16-bit outputs: G and U (forward), dG and dU (backward)
  CUtensorMap h;                   // forward: h as BF16
  CUtensorMap q0, q1;              // codes: h (forward), dG and dU (backward)
  const float* sa;
  const float* sb;
  const uint16_t* gu;              // backward: [M][2N] BF16
  const float* scale;              // of the codes
  unsigned int* amax_bits;
  float* scale_inv;
  int32_t M, N;
  int32_t tiles_m, tiles_n, total_tiles, num_kb;
  int32_t a_mn, b_mn;
  uint32_t idesc;
  int32_t act, fmt;                // fmt of the codes
  int32_t keep, has_h, has_q;      // which outputs are written
  int32_t tile_start;              // 0
  __device__ __forceinline__ const Params& problem(int) const { return *this; }
};

// sigmoid(w(g)) and w'(g).
template <int ACT>
__device__ __forceinline__ float gate(float g, float* dw = nullptr) {
  float w = g;
  if constexpr (ACT == kGelu) {
    const float g2 = g * g;
    w = 1.5957691216057308f * g * fmaf(0.044715f, g2, 1.0f);
    if (dw) *dw = 1.5957691216057308f * fmaf(0.134145f, g2, 1.0f);
  } else if (dw) {
    *dw = 1.0f;
  }
  return __fdividef(1.0f, 1.0f + __expf(-w));              // exp overflows to infinity where sigmoid is 0
}

// Runs of `kRun` row tiles share their column tiles, so that the weights a wave of tiles reads are read by several rows
// of A while they are in L2.
constexpr int kRun = 8;
__device__ __forceinline__ void place_in_runs(int tiles_m, int tiles_n, int local, int& mt, int& nt) {
  const int run = local / (kRun * tiles_n), in = local - run * kRun * tiles_n;
  const int rows = min(kRun, tiles_m - run * kRun);
  nt = in / rows;
  mt = run * kRun + in - nt * rows;
}

__device__ __forceinline__ void note(uint32_t& top, float v, bool valid) {
  if (valid) top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);
}
// Codes of 32 values of a row under `scale`.
__device__ __forceinline__ void codes32(const float (&v)[32], float scale, int fmt, uint32_t (&q)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = __fmul_rn(v[4 * j], scale), b = __fmul_rn(v[4 * j + 1], scale);
    const float c = __fmul_rn(v[4 * j + 2], scale), d = __fmul_rn(v[4 * j + 3], scale);
    q[j] = fmt == 0 ? cvt_fp8x2<0>(a, b) | cvt_fp8x2<0>(c, d) << 16 : cvt_fp8x2<1>(a, b) | cvt_fp8x2<1>(c, d) << 16;
  }
}
__device__ __forceinline__ void pack16(const float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
}

struct Scalars {
  float alpha, scale;
};
struct Base {
  using Params = gated::Params;
  using Scalars = gated::Scalars;
  static constexpr bool kF16 = false, kAmax = true;
  static __device__ __forceinline__ void place(const Params& P, int local, int& mt, int& nt) {
    place_in_runs(P.tiles_m, P.tiles_n, local, mt, nt);
  }
  static __device__ __forceinline__ Scalars scalars(const Params& g) {
    return {__fmul_rn(ld_dep(g.sa), ld_dep(g.sb)), g.scale ? ld_dep(g.scale) : 1.0f};
  }
  // A CTA whose waits expired has not seen all of its tiles: its amax is a NaN, so that the next scale stays as it is.
  static __device__ __forceinline__ void finish(const Params& g, uint32_t top, bool aborted) {
    if (aborted) top = 0x7FC00000u;
    if (g.amax_bits && top) atomicMax(g.amax_bits, top > 0x7F800000u ? 0x7FC00000u : top);
    if (g.scale_inv && blockIdx.x == 0) *g.scale_inv = __fdiv_rn(1.0f, ld_dep(g.scale));
  }
};

template <int ACT>
struct Forward : Base {
  static __device__ __forceinline__ int b_row(const Params& P, int nt, int rank) { return nt * 128 + rank * P.N; }
  template <class Release>
  static __device__ __forceinline__ void epilogue(const Params& g, const Params&, const Scalars& k, Out& o, int, int nt,
                                                  int row0, int half, uint32_t t_base, Release&& release) {
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      const int c = half * 64 + s * 32, n = nt * 128 + c;
      uint32_t rg[32], ru[32];
      __syncwarp();                                        // one lane stored the chunk before
      tmem_ld_32x32b_x32(t_base + c, rg);
      tmem_ld_32x32b_x32(t_base + 128 + c, ru);
      tmem_ld_wait();
      tmem_reg_fence(rg);
      tmem_reg_fence(ru);
      if (s == 1) release();
      if (n >= g.N || row0 >= g.M) continue;               // chunk entirely outside the matrix
      float gv[32], uv[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        gv[j] = __fmul_rn(__uint_as_float(rg[j]), k.alpha);
        uv[j] = __fmul_rn(__uint_as_float(ru[j]), k.alpha);
      }
      if (g.keep) {
        uint32_t w[16];
        pack16(gv, w);
        store16(o, &g.o0, w, n, row0);
        pack16(uv, w);
        store16(o, &g.o1, w, n, row0);
      }
      // rows past M and columns past N (whose gate is a column of the up projection) stay out of amax: an infinite weight
      // makes NaN of their zeros. N is a multiple of 16
      const bool in = row0 + o.lane < g.M, all = in && n + 16 < g.N;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        gv[j] = gv[j] * gate<ACT>(gv[j]) * uv[j];
        note(o.amax, gv[j], j < 16 ? in : all);
      }
      if (g.has_h) {
        uint32_t w[16];
        pack16(gv, w);
        store16(o, &g.h, w, n, row0);
      }
      if (g.has_q) {
        uint32_t q[8];
        codes32(gv, k.scale, g.fmt, q);
        store8(o, &g.q0, q, n, row0);
      }
    }
  }
};

// 32 BF16 values of a row (four 16-byte loads where they lie within it).
__device__ __forceinline__ void load32(const uint16_t* p, int left, bool row, float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (row && 8 * c < left) x = ld_dep(reinterpret_cast<const uint4*>(p + 8 * c));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * c + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * c + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

template <int ACT>
struct Backward : Base {
  static __device__ __forceinline__ int b_row(const Params&, int nt, int rank) { return nt * kBN + rank * kHalf; }
  template <class Release>
  static __device__ __forceinline__ void epilogue(const Params& g, const Params&, const Scalars& k, Out& o, int, int nt,
                                                  int row0, int half, uint32_t t_base, Release&& release) {
    const int row = row0 + o.lane;
    const bool in = row < g.M;
    const uint16_t* line = g.gu + static_cast<int64_t>(row) * 2 * g.N;
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
      const int c = half * 128 + s * 32, n = nt * kBN + c;
      float gv[32], uv[32];
      load32(line + n, g.N - n, in, gv);
      load32(line + g.N + n, g.N - n, in, uv);
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(t_base + c, r);
      tmem_ld_wait();
      tmem_reg_fence(r);
      if (s == 3) release();
      if (n >= g.N || row0 >= g.M) continue;
      const bool all = in && n + 16 < g.N;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float dh = __fmul_rn(__uint_as_float(r[j]), k.alpha);
        float dw;
        const float sg = gate<ACT>(gv[j], &dw);
        const float rest = sg * (1.0f - sg);
        // where sigmoid is 0 or 1 its slope is 0 whatever g and w'(g) are (they may be infinite)
        const float slope = rest == 0.0f ? 0.0f : gv[j] * rest * dw;
        const float du = dh * (gv[j] * sg);
        gv[j] = dh * uv[j] * (sg + slope);
        uv[j] = du;
        note(o.amax, gv[j], j < 16 ? in : all);
        note(o.amax, uv[j], j < 16 ? in : all);
      }
      if (g.keep) {
        uint32_t w[16];
        pack16(gv, w);
        store16(o, &g.o0, w, n, row0);
        pack16(uv, w);
        store16(o, &g.o1, w, n, row0);
      }
      if (g.has_q) {
        uint32_t q[8];
        codes32(gv, k.scale, g.fmt, q);
        store8(o, &g.q0, q, n, row0);
        codes32(uv, k.scale, g.fmt, q);
        store8(o, &g.q1, q, n, row0);
      }
    }
  }
};

}  // namespace gated
}  // namespace fp8t
