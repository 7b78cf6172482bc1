// rmsnorm.cuh — root-mean-square norm in front of a quantised Linear, forward and backward.
//
// Forward, per row of C values (every f32 operation rounded separately):
//   h = bf16(x + residual)        the new residual stream (h = x without a residual)
//   rstd = 1 / sqrt(sum(h^2) / C + eps)
//   y = (h * rstd) * gamma
// and y leaves as BF16 and / or as the codes the following GEMM reads: per-tensor FP8 (f32(y) * scale,
// amax, inverse scale, as the cast of X under delayed scaling), MXFP8, MXFP4 or NVFP4 (row-wise blocks).
// h is rounded to BF16 before it is normed because that is the value the residual stream and the
// backward pass see; y is not rounded to BF16 on the way to its codes (one rounding, f32 to code).
// Statistics are f32.
//
// What bounds it: HBM, 2 B (x) + 2 B (residual) read and 2 B (h) + code bytes written per element; a
// row is read once and held in registers (four 16-byte vectors per thread at most) between the sum of
// squares and the quantisation.
//
// Backward, with xh = h * rstd and g = dy * gamma:
//   dh = rstd * (g - xh * (sum(g * xh) / C)) (+ dres, the gradient that reaches h directly)
//   dgamma = sum over rows of dy * xh
// reads 2 + 2 (+ 2) B and writes 2 B per element. A thread owns the same columns for every row of its
// CTA, so dgamma is summed in registers (f32), one partial row per CTA is left in the workspace, and a
// second kernel adds the partials in index order: the result does not depend on scheduling.
#pragma once

#include "ptx.cuh"
#include "quant_block.cuh"

namespace fp8t {
namespace norm {

constexpr int kMaxThreads = 512;         // per row (128 registers each)
constexpr int kMaxCols = 16384;          // 512 threads x 4 vectors of 8
constexpr int kRowsPerCta = 4;           // warp-per-row form: warps (rows) per CTA
constexpr int kMaxWarpCols = 1024;       // widest row a warp takes (4 vectors of 8 per lane)

struct Fwd {
  const uint4* x;
  const uint4* res;                      // may be null
  const uint4* gamma;
  uint4* h;                              // may be null
  float* rstd;                           // may be null
  uint4* y;                              // may be null
  uint8_t* q;
  uint8_t* sf;
  const float* scale;                    // FP8 / NVFP4
  unsigned int* amax_bits;               // FP8 / NVFP4 (may be null there)
  float* scale_inv;                      // may be null
  int64_t rows;
  int32_t cols, fmt;
  float eps;
};

struct Bwd {
  const uint4* dy;
  const uint4* h;
  const uint4* gamma;
  const float* rstd;
  const uint4* dres;                     // may be null
  uint4* dh;
  float* partials;                       // [gridDim.x][cols]; null: no dgamma
  int64_t rows;
  int32_t cols;
};

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = lo_f32(v.x); f[1] = hi_f32(v.x); f[2] = lo_f32(v.y); f[3] = hi_f32(v.y);
  f[4] = lo_f32(v.z); f[5] = hi_f32(v.z); f[6] = lo_f32(v.w); f[7] = hi_f32(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// Sum over the threads that share a row: the warp, or the CTA (the same value in every thread). The
// CTA form alternates between two shared rows so that one barrier per row is enough.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float (*sh)[32], int parity) {
  v = warp_sum(v);
  if (WARP_ROW) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sh[parity][warp] = v;
  __syncthreads();
  const int n = blockDim.x >> 5;
  return warp_sum(lane < n ? sh[parity][lane] : 0.0f);
}

// VPT: vectors of 8 per thread; WARP_ROW: a warp per row, else the CTA; Q: how y is quantised (blk::k*).
template <int VPT, bool WARP_ROW, int Q>
__global__ void __launch_bounds__(WARP_ROW ? 32 * kRowsPerCta : kMaxThreads) k_rmsnorm_cast(const Fwd p) {
  __shared__ float sh[2][32];
  const int lane = threadIdx.x & 31;
  const int tid = WARP_ROW ? lane : threadIdx.x;
  const int nthr = WARP_ROW ? 32 : blockDim.x;
  const int nvec = p.cols >> 3;
  const int64_t row_step = WARP_ROW ? static_cast<int64_t>(gridDim.x) * kRowsPerCta : gridDim.x;
  int64_t row = WARP_ROW ? static_cast<int64_t>(blockIdx.x) * kRowsPerCta + (threadIdx.x >> 5) : blockIdx.x;

  uint4 gam[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nthr + tid;
    gam[i] = v < nvec ? __ldg(p.gamma + v) : make_uint4(0u, 0u, 0u, 0u);
  }
  const float scale = Q == blk::kFP8 || Q == blk::kNVFP4 ? __ldg(p.scale) : 1.0f;
  const int emax = Q == blk::kMXFP4 ? 2 : (p.fmt == 0 ? 8 : 15);
  const float inv_c = __fdiv_rn(1.0f, static_cast<float>(p.cols));
  uint32_t amax = 0;

  for (int it = 0; row < p.rows; row += row_step, ++it) {
    const int64_t base = row * nvec;
    uint4 hv[VPT];
    float ss = 0.0f;
    {
      uint4 rv[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nthr + tid;
        hv[i] = v < nvec ? ld_stream_u4(p.x + base + v) : make_uint4(0u, 0u, 0u, 0u);
        if (p.res) rv[i] = v < nvec ? ld_stream_u4(p.res + base + v) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float a[8];
        unpack8(hv[i], a);
        if (p.res) {
          float b[8];
          unpack8(rv[i], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] = __fadd_rn(a[j], b[j]);
          hv[i] = pack8(a);
          unpack8(hv[i], a);
          const int v = i * nthr + tid;
          if (p.h && v < nvec) p.h[base + v] = hv[i];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __fmaf_rn(a[j], a[j], ss);
      }
    }
    ss = row_sum<WARP_ROW>(ss, sh, it & 1);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(ss, inv_c), p.eps)));
    if (p.rstd && tid == 0) p.rstd[row] = rstd;

#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      const bool in = v < nvec;
      float y[8], gm[8];
      unpack8(hv[i], y);
      unpack8(gam[i], gm);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(__fmul_rn(y[j], rstd), gm[j]);
      if (p.y && in) p.y[base + v] = pack8(y);
      if (Q == blk::kNone) continue;
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
      if (!in) m = 0;                    // 0 * NaN of a vector past the row's end
      float f = scale;
      if (Q == blk::kFP8) {
        amax = max(amax, m);
      } else {
        // lanes that share a block: 4 x 8 values (2 x 8 for NVFP4)
        if (Q == blk::kNVFP4) amax = max(amax, m);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        if (Q != blk::kNVFP4) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        uint32_t word = Q == blk::kNVFP4 ? blk::nvfp4_scale(m, scale, f) : blk::e8m0_scale(m, emax, f);
        // the four scales of one atom word to the first lane of the 16 (8) that share it
        constexpr int kStep = Q == blk::kNVFP4 ? 2 : 4;
        if (!in) word = 0;
        word |= __shfl_down_sync(0xffffffffu, word, kStep) << 8;
        word |= __shfl_down_sync(0xffffffffu, word, 2 * kStep) << 16;
        if (in && (lane & (4 * kStep - 1)) == 0)
          *reinterpret_cast<uint32_t*>(
              p.sf + blk::atom_word(row, v / (4 * kStep), blk::atoms_per_row(p.cols, Q))) = word;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(y[j], f);
      if (!in) continue;
      if (Q == blk::kMXFP4 || Q == blk::kNVFP4) {
        reinterpret_cast<uint32_t*>(p.q)[base + v] = blk::cvt_e2m1x8(y);
      } else {
        uint2 c;
        if (p.fmt == 0)
          c = make_uint2(cvt_fp8x2<0>(y[0], y[1]) | cvt_fp8x2<0>(y[2], y[3]) << 16,
                         cvt_fp8x2<0>(y[4], y[5]) | cvt_fp8x2<0>(y[6], y[7]) << 16);
        else
          c = make_uint2(cvt_fp8x2<1>(y[0], y[1]) | cvt_fp8x2<1>(y[2], y[3]) << 16,
                         cvt_fp8x2<1>(y[4], y[5]) | cvt_fp8x2<1>(y[6], y[7]) << 16);
        reinterpret_cast<uint2*>(p.q)[base + v] = c;
      }
    }
    if (Q == blk::kMXFP4 || Q == blk::kNVFP4) {        // K padded to 256: the atom words past the row
      constexpr int kPer = Q == blk::kMXFP4 ? 128 : 64;
      const int used = (p.cols + kPer - 1) / kPer, words = static_cast<int>(blk::atoms_per_row(p.cols, Q));
      if (tid < words - used)
        *reinterpret_cast<uint32_t*>(p.sf + blk::atom_word(row, used + tid, words)) = 0u;
    }
  }
  if (Q == blk::kFP8 || Q == blk::kNVFP4) {
    if (p.amax_bits) {
      amax = __reduce_max_sync(0xffffffffu, amax);
      if (amax > 0x7F800000u) amax = 0x7FC00000u;      // canonical NaN
      if (lane == 0 && amax) atomicMax(p.amax_bits, amax);
    }
    if (p.scale_inv && blockIdx.x == 0 && threadIdx.x == 0) *p.scale_inv = __fdiv_rn(1.0f, scale);
  }
}

template <int VPT, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 32 * kRowsPerCta : kMaxThreads) k_rmsnorm_backward(const Bwd p) {
  __shared__ float sh[2][32];
  __shared__ float part[WARP_ROW ? kRowsPerCta - 1 : 1][WARP_ROW ? VPT * 256 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARP_ROW ? lane : threadIdx.x;
  const int nthr = WARP_ROW ? 32 : blockDim.x;
  const int nvec = p.cols >> 3;
  const int64_t row_step = WARP_ROW ? static_cast<int64_t>(gridDim.x) * kRowsPerCta : gridDim.x;
  int64_t row = WARP_ROW ? static_cast<int64_t>(blockIdx.x) * kRowsPerCta + warp : blockIdx.x;

  uint4 gam[VPT];
  float acc[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nthr + tid;
    gam[i] = v < nvec ? __ldg(p.gamma + v) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  }
  const float inv_c = __fdiv_rn(1.0f, static_cast<float>(p.cols));

  for (int it = 0; row < p.rows; row += row_step, ++it) {
    const int64_t base = row * nvec;
    const float rstd = __ldg(p.rstd + row);
    uint4 dv[VPT], hv[VPT], rv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      const bool in = v < nvec;
      dv[i] = in ? ld_stream_u4(p.dy + base + v) : make_uint4(0u, 0u, 0u, 0u);
      hv[i] = in ? ld_stream_u4(p.h + base + v) : make_uint4(0u, 0u, 0u, 0u);
      if (p.dres) rv[i] = in ? ld_stream_u4(p.dres + base + v) : make_uint4(0u, 0u, 0u, 0u);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float d[8], h[8], gm[8];
      unpack8(dv[i], d);
      unpack8(hv[i], h);
      unpack8(gam[i], gm);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = i * nthr + tid < nvec ? __fmul_rn(h[j], rstd) : 0.0f;
        acc[i][j] = __fmaf_rn(d[j], xh, acc[i][j]);
        s = __fmaf_rn(__fmul_rn(d[j], gm[j]), xh, s);
      }
    }
    s = __fmul_rn(row_sum<WARP_ROW>(s, sh, it & 1), inv_c);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float d[8], h[8], gm[8], r[8];
      unpack8(dv[i], d);
      unpack8(hv[i], h);
      unpack8(gam[i], gm);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        d[j] = __fmul_rn(rstd, __fsub_rn(__fmul_rn(d[j], gm[j]), __fmul_rn(__fmul_rn(h[j], rstd), s)));
      if (p.dres) {
        unpack8(rv[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = __fadd_rn(d[j], r[j]);
      }
      const int v = i * nthr + tid;
      if (v < nvec) p.dh[base + v] = pack8(d);
    }
  }
  if (!p.partials) return;
  if (WARP_ROW) {                        // the CTA's warps in order, then one partial row
    if (warp > 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) part[warp - 1][(i * 8 + j) * 32 + lane] = acc[i][j];
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        for (int w = 0; w < kRowsPerCta - 1; ++w) acc[i][j] = __fadd_rn(acc[i][j], part[w][(i * 8 + j) * 32 + lane]);
  }
  float4* out = reinterpret_cast<float4*>(p.partials + static_cast<int64_t>(blockIdx.x) * p.cols);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nthr + tid;
    if (v >= nvec) continue;
    out[2 * v] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    out[2 * v + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
  }
}

// dgamma: 32 columns per CTA, 16 warps take every 16th partial row, then one sum over the warps.
constexpr int kReduceWarps = 16;
__global__ void __launch_bounds__(32 * kReduceWarps)
    k_rmsnorm_dgamma(const float* __restrict__ partials, int n, int cols, float* __restrict__ out_f32,
                     uint16_t* __restrict__ out_bf16) {
  __shared__ float sh[kReduceWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.0f;
  if (c < cols)
    for (int i = warp; i < n; i += kReduceWarps) a = __fadd_rn(a, __ldcg(partials + static_cast<int64_t>(i) * cols + c));
  sh[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
  for (int w = 1; w < kReduceWarps; ++w) a = __fadd_rn(a, sh[w][lane]);
  if (out_f32) out_f32[c] = a;
  if (out_bf16) out_bf16[c] = static_cast<uint16_t>(pack2(a, a));
}

}  // namespace norm
}  // namespace fp8t
