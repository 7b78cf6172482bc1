// gated.cuh — the gated feed-forward block in FP8: both projections, the activation and the product in one kernel, and
// the gradient of all that in the product that brings it.
//
// Forward. W holds the gate's and the up projection's weights side by side (N columns each):
//   [G | U] = (A . W) * sa * sb,  h = act(G) * U,  act(g) = g * sigmoid(w(g))
//   w = g (SiLU) or 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU in its tanh form: (1 + tanh(z)) / 2 = sigmoid(2z))
// One accumulator of a pair tile holds 128 columns of G and the same 128 of U (96 or 64 of each in narrower tiles): the even CTA's half of B is
// gate rows, the odd CTA's the up rows of the same columns, so every lane has g and u of an element at the same time and h never
// leaves the registers before it is rounded. h is formed from the f32 accumulators; G and U are rounded to BF16 only
// where they are kept for the gradient.
// Backward. dH = (dY . Wd^T) * sa * sb stays in the accumulator (256 columns); with s = sigmoid(w(g))
//   dG = dH * u * (s + g s (1 - s) w'(g)),  dU = dH * g s
// written as [dG | dU] side by side under one scale, so that dX = [dG | dU] . W^T and dW = X^T . [dG | dU] are one
// product each.
#pragma once

#include "gemm_pair.cuh"
#include "quant_block.cuh"

namespace fp8t {
namespace gated {

using namespace pair;

enum : int { kSilu = 1, kGelu = 2 };                       // fp8t_act

struct alignas(64) Params {
  CUtensorMap a, b;                // A in boxes of a_rows, B
  CUtensorMap o0, o1;              // 16-bit outputs: G and U (forward), dG and dU (backward)
  CUtensorMap g, u;                // backward: the kept G and U
  CUtensorMap h;                   // forward: h as BF16
  CUtensorMap q0, q1;              // codes: h (forward), dG and dU (backward)
  const float* sa;
  const float* sb;
  const float* scale;              // of the codes
  unsigned int* amax_bits;
  float* scale_inv;
  int32_t M, N;
  int32_t tiles_m, tiles_n, total_tiles, num_kb;
  int32_t a_rows;                  // rows of A's box: 128, or fewer where M is
  int32_t half_n;                  // rows of B of a CTA: a tile has as many outputs (forward) or twice as many (backward)
  int32_t b_mn;                    // 1: B is stored MN-major
  uint32_t idesc;
  int32_t act, fmt;                // fmt of the codes
  int32_t keep, has_h, has_q;      // which outputs are written
};

// Pairs of values: each half is rounded as the scalar operation would be, at half the instructions.
using blk::f32x2;
__device__ __forceinline__ f32x2 both(float v) { return blk::pair(v, v); }
__device__ __forceinline__ float ex2(float x) {            // 2^x, to 2 ulp; infinity and 0 where it leaves the range
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {            // 1 / x, to 1 ulp; 0 for infinity
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;
// Sigmoid of w(g), 0 where it is below 2^-126 (g under -87.3 for SiLU, -10.0 for GELU), and w'(g) where the operator needs it (1 for SiLU). g^2 is held to 10^12, far past where the sigmoid is 0 or
// 1 in f32, so that w' stays finite.
template <int ACT>
__device__ __forceinline__ f32x2 gate(f32x2 g, f32x2& dw) {
  using namespace blk;
  f32x2 x;                                                 // -w log2(e)
  if constexpr (ACT == kGelu) {
    f32x2 g2 = mul2(g, g);
    g2 = blk::pair(fminf(lo(g2), 1e12f), fminf(hi(g2), 1e12f));
    x = mul2(mul2(g, both(-1.5957691216057308f * kLog2e)), fma2(g2, both(0.044715f), both(1.0f)));
    dw = mul2(fma2(g2, both(0.134145f), both(1.0f)), both(1.5957691216057308f));
  } else {
    x = mul2(g, both(-kLog2e));
  }
  const f32x2 d = add2(blk::pair(ex2(lo(x)), ex2(hi(x))), both(1.0f));
  return blk::pair(rcp(lo(d)), rcp(hi(d)));
}
template <int ACT>
__device__ __forceinline__ float gate(float g) {
  f32x2 dw;
  return blk::lo(gate<ACT>(both(g), dw));
}

// max(|a|, |b|, |c|), NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The largest magnitude of a row's 32 values. Rows past M and columns past N stay out of it: an infinite weight makes NaN of
// their zeros. N is a multiple of 16.
__device__ __forceinline__ void note(Out& o, const f32x2 (&v)[16], bool row, bool whole) {
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a = max_abs(a, blk::lo(v[j]), blk::hi(v[j]));
    b = max_abs(b, blk::lo(v[8 + j]), blk::hi(v[8 + j]));
  }
  if (row) o.amax = max(o.amax, max(__float_as_uint(a), whole ? __float_as_uint(b) : 0u) & 0x7FFFFFFFu);
}
// Codes of 32 values of a row under `scale`.
__device__ __forceinline__ void codes32(const f32x2 (&v)[16], f32x2 scale, int fmt, uint32_t (&q)[8]) {
  using namespace blk;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const f32x2 a = mul2(v[2 * j], scale), b = mul2(v[2 * j + 1], scale);
    q[j] = fmt == 0 ? cvt_fp8x2<0>(lo(a), hi(a)) | cvt_fp8x2<0>(lo(b), hi(b)) << 16
                    : cvt_fp8x2<1>(lo(a), hi(a)) | cvt_fp8x2<1>(lo(b), hi(b)) << 16;
  }
}
__device__ __forceinline__ void pack16(const f32x2 (&v)[16], uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(blk::lo(v[j]), blk::hi(v[j]));
}
// 32 accumulator columns times alpha.
__device__ __forceinline__ void scaled(const uint32_t (&r)[32], f32x2 alpha, f32x2 (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = blk::mul2(blk::pair(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), alpha);
}

struct Scalars {
  f32x2 alpha, scale;
};
struct Base {
  using Params = gated::Params;
  using Scalars = gated::Scalars;
  static constexpr bool kF16 = false, kAmax = true, kPhased = false;
  static __device__ __forceinline__ int phases(const Params&) { return 1; }
  static __device__ __forceinline__ int tiles(const Params& g, int) { return g.total_tiles; }
  static __device__ __forceinline__ bool reads(int) { return false; }
  static __device__ __forceinline__ Grid grid(const Params&) { return {}; }
  // b_step: rows of B from one column tile to the next; b_other: from the even CTA's to the odd CTA's
  static __device__ __forceinline__ Work work_of(const Params& g, int tile, int rank, int b_step, int b_other) {
    Work w;
    place_in_runs(g.tiles_m, g.tiles_n, tile, w.mt, w.nt);
    w.a = &g.a;
    w.b = &g.b;
    w.a_row = w.mt * kBM + rank * kHalf;
    w.b_row = w.nt * b_step + rank * b_other;
    w.half_n = g.half_n;
    w.a_bytes = g.a_rows * kBK;
    w.num_kb = g.num_kb;
    w.a_mn = 0;
    w.b_mn = g.b_mn;
    w.idesc = g.idesc;
    w.which = 0;
    return w;
  }
  static __device__ __forceinline__ Scalars scalars(const Params& g) {
    return {both(__fmul_rn(ld_dep(g.sa), ld_dep(g.sb))), both(g.scale ? ld_dep(g.scale) : 1.0f)};
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
  static constexpr int kLoads = 0;
  static __device__ __forceinline__ void prefetch(const Params&, const Work&, int, Out&, int, int) {}
  static __device__ __forceinline__ Work work(const Params& g, int, int tile, int rank) { return work_of(g, tile, rank, g.half_n, g.N); }
  template <class Release, class Ahead>
  static __device__ __forceinline__ bool epilogue(const Params& g, const Work& w, int, const Scalars& k, Out& o, int row0, int half,
                                                  uint32_t t_base, Release&& release, Ahead&&) {
#pragma unroll 1
    for (int c = half * 32; c < w.half_n; c += 64) {
      const int n = w.nt * w.half_n + c;
      uint32_t rg[32], ru[32];
      __syncwarp();                                        // one lane stored the chunk before
      tmem_ld_32x32b_x32(t_base + c, rg);
      tmem_ld_32x32b_x32(t_base + w.half_n + c, ru);
      tmem_ld_wait();
      tmem_reg_fence(rg);
      tmem_reg_fence(ru);
      if (c + 64 >= w.half_n) release();
      if (n >= g.N || row0 >= g.M) continue;               // chunk entirely outside the matrix
      f32x2 gv[16], uv[16];
      scaled(rg, k.alpha, gv);
      scaled(ru, k.alpha, uv);
      if (g.keep) {
        uint32_t v[16];
        pack16(gv, v);
        store16(o, &g.o0, v, n, row0);
        pack16(uv, v);
        store16(o, &g.o1, v, n, row0);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        f32x2 dw;
        gv[j] = blk::mul2(blk::mul2(gv[j], gate<ACT>(gv[j], dw)), uv[j]);
      }
      note(o, gv, row0 + o.lane < g.M, n + 16 < g.N);
      if (g.has_h) {
        uint32_t v[16];
        pack16(gv, v);
        store16(o, &g.h, v, n, row0);
      }
      if (g.has_q) {
        uint32_t q[8];
        codes32(gv, k.scale, g.fmt, q);
        store8(o, &g.q0, q, n, row0);
      }
    }
    return true;
  }
};

__device__ __forceinline__ f32x2 pair_of(uint32_t w) { return blk::pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

template <int ACT>
struct Backward : Base {
  static constexpr int kLoads = 2;
  static __device__ __forceinline__ void fetch_at(const Params& g, Out& o, int row0, int n) {
    const CUtensorMap* const maps[2] = {&g.g, &g.u};
    const int x[2] = {n, n};
    fetch(o, maps, x, row0);
  }
  static __device__ __forceinline__ void prefetch(const Params& g, const Work& w, int, Out& o, int row0, int half) {
    fetch_at(g, o, row0, (2 * w.nt + half) * w.half_n);
  }
  static __device__ __forceinline__ Work work(const Params& g, int, int tile, int rank) { return work_of(g, tile, rank, 2 * g.half_n, g.half_n); }
  template <class Release, class Ahead>
  static __device__ __forceinline__ bool epilogue(const Params& g, const Work& w, int, const Scalars& k, Out& o, int row0, int half,
                                                  uint32_t t_base, Release&& release, Ahead&& ahead) {
    const bool in = row0 + o.lane < g.M;
    const int steps = w.half_n / 32;
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      const int c = half * w.half_n + s * 32, n = 2 * w.half_n * w.nt + c;
      uint4 gw[4], uw[4];
      if (!fetched(o)) return false;
      chunk_row(o, 0, gw);
      chunk_row(o, 1, uw);
      if (s + 1 < steps) fetch_at(g, o, row0, n + 32);
      else ahead();
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(t_base + c, r);
      tmem_ld_wait();
      tmem_reg_fence(r);
      if (s + 1 == steps) release();
      if (n >= g.N || row0 >= g.M) continue;
      f32x2 gv[16], uv[16], dh[16];
      scaled(r, k.alpha, dh);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        gv[j] = pair_of((&gw[j >> 2].x)[j & 3]);
        uv[j] = pair_of((&uw[j >> 2].x)[j & 3]);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        using namespace blk;
        f32x2 dw;
        const f32x2 sg = gate<ACT>(gv[j], dw), gs = mul2(gv[j], sg);
        // g s (1 - s) w': where the sigmoid is 0 or 1 the product is 0 before the finite w' comes in
        f32x2 slope = mul2(gs, fma2(sg, both(-1.0f), both(1.0f)));
        if constexpr (ACT == kGelu) slope = mul2(slope, dw);
        gv[j] = mul2(mul2(dh[j], uv[j]), add2(sg, slope));
        uv[j] = mul2(dh[j], gs);
      }
      note(o, gv, in, n + 16 < g.N);
      note(o, uv, in, n + 16 < g.N);
      if (g.keep) {
        uint32_t v[16];
        pack16(gv, v);
        store16(o, &g.o0, v, n, row0);
        pack16(uv, v);
        store16(o, &g.o1, v, n, row0);
      }
      if (g.has_q) {
        uint32_t q[8];
        codes32(gv, k.scale, g.fmt, q);
        store8(o, &g.q0, q, n, row0);
        codes32(uv, k.scale, g.fmt, q);
        store8(o, &g.q1, q, n, row0);
      }
    }
    return true;
  }
};

}  // namespace gated
}  // namespace fp8t
