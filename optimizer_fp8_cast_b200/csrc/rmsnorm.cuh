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
// What bounds it: HBM, 2 B (x) + 2 B (residual) read and 2 B (h) + code bytes written per element. A row is
// read once and held in registers (four 16-byte vectors per thread at most) between the sum of squares and
// the quantisation. Scalar arithmetic, 20 instructions per element, kept the loads waiting (45 us for 8192 x 4096 to
// FP8, half of the issue slots used by 16 warps per SM), so it runs on pairs (f32x2 add, multiply, FMA: two elements
// per instruction, each rounded as the scalar one) and amax is a three-input maximum. A thread's loads of a row
// come at once and then none until the next row, so one thread asks for the next row's bytes with a bulk
// prefetch into L2: 47.2 -> 41.1 us (5.7 TB/s); two or three rows ahead gave 43.4 and 45.0.
//
// Backward, with xh = h * rstd and g = dy * gamma:
//   dh = rstd * (g - xh * (sum(g * xh) / C)) (+ dres, the gradient that reaches h directly)
//   dgamma = sum over rows of dy * xh
// reads 2 + 2 (+ 2) B and writes 2 B per element. One CTA per SM holds several row groups (a group: the
// threads that share a row, with a barrier of its own); a thread owns the same columns for every row of its
// group, so dgamma is summed in registers (f32), over the CTA's groups in shared memory, and one
// partial row per CTA goes to the workspace; a second kernel adds the partials. Both orders are fixed: the
// result does not depend on scheduling. With the same prefetch, 8192 x 4096 with dres 58.7 -> 48.5 us. Of rows
// wider than 8192 columns gamma is re-read for every row (from L1) and dres once the row's sum is known, since three or
// four vectors of all inputs per thread spill: 8192 x 8192 on two vectors 92 us (on four 143), 4096 x 16384 121 (147; of
// more than 12288 columns, four vectors, 40 bytes of a thread still spill). Means are the sum times rn(1 / C).
#pragma once

#include "ptx.cuh"
#include "quant_block.cuh"

namespace fp8t {
namespace norm {

constexpr int kMaxThreads = 512;         // per row
constexpr int kMaxCols = 16384;          // 512 threads x 4 vectors of 8
constexpr int kRowsPerCta = 4;           // forward, warp-per-row form: warps (rows) per CTA
constexpr int kMaxWarpCols = 1024;       // widest row a warp takes (4 vectors of 8 per lane)
constexpr int kBwdThreads = 512;         // backward: threads per CTA at most (128 registers each)
constexpr int kBwdCtas = 148;            // backward: CTAs at most, one per SM

// dgamma of a CTA's groups beyond the first: at most 512 threads x 4 vectors x 8 columns
constexpr int kBwdMaxSmem = kBwdThreads * 4 * 8 * 4;

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
  int32_t group;                         // threads per row, a multiple of 32
};

using blk::f32x2;
using blk::pair;
using blk::lo;
using blk::hi;
using blk::add2;
using blk::mul2;
using blk::fma2;
// max(|a|, |b|, |c|), NaN if one is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ f32x2 unpack2(uint32_t w) {        // two BF16, the first in the low half
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack2(f32x2 v) { return pack2(lo(v), hi(v)); }
__device__ __forceinline__ void unpack8(const uint4& v, f32x2 (&f)[4]) {
  f[0] = unpack2(v.x); f[1] = unpack2(v.y); f[2] = unpack2(v.z); f[3] = unpack2(v.w);
}
__device__ __forceinline__ uint4 pack8(const f32x2 (&f)[4]) {
  return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
__device__ __forceinline__ uint4 load_or_zero(const uint4* p, bool in) {
  return in ? ld_stream_u4(p) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// Sum over the threads of a row group (warps first .. first + n - 1 of the CTA, barrier id `bar`), the same
// value in every thread. Shared rows alternate by parity, so one barrier per row is enough.
__device__ __forceinline__ float group_sum(float v, float (*sh)[32], int parity, int first, int n, int bar) {
  v = warp_sum(v);
  if (n == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) sh[parity][threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(n * 32) : "memory");
  return warp_sum(lane < n ? sh[parity][first + lane] : 0.0f);
}

// Eight values -> eight FP8 codes.
template <int FMT>
__device__ __forceinline__ uint2 codes8(const f32x2 (&y)[4]) {
  return make_uint2(cvt_fp8x2<FMT>(lo(y[0]), hi(y[0])) | cvt_fp8x2<FMT>(lo(y[1]), hi(y[1])) << 16,
                    cvt_fp8x2<FMT>(lo(y[2]), hi(y[2])) | cvt_fp8x2<FMT>(lo(y[3]), hi(y[3])) << 16);
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

  pdl_trigger();
  pdl_wait();
  uint4 gam[VPT];
  bool in[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    in[i] = i * nthr + tid < nvec;
    gam[i] = in[i] ? ld_dep(p.gamma + i * nthr + tid) : make_uint4(0u, 0u, 0u, 0u);
  }
  const float scale = Q == blk::kFP8 || Q == blk::kNVFP4 ? ld_dep(p.scale) : 1.0f;
  const int emax = Q == blk::kMXFP4 ? 2 : (p.fmt == 0 ? 8 : 15);
  const float inv_c = __fdiv_rn(1.0f, static_cast<float>(p.cols));
  float amax = 0.0f;

  for (int it = 0; row < p.rows; row += row_step, ++it) {
    const int64_t base = row * nvec + tid;
    f32x2 h[VPT][4];
    float ss = 0.0f;
    if (tid == 0 && row + row_step < p.rows) {           // the row after this one into L2
      const int64_t next = (row + row_step) * nvec;
      l2_prefetch(p.x + next, nvec * 16);
      if (p.res) l2_prefetch(p.res + next, nvec * 16);
    }
    {
      uint4 xv[VPT], rv[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        xv[i] = load_or_zero(p.x + base + i * nthr, in[i]);
        if (p.res) rv[i] = load_or_zero(p.res + base + i * nthr, in[i]);
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        unpack8(xv[i], h[i]);
        if (p.res) {
          f32x2 r[4];
          unpack8(rv[i], r);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[i][j] = add2(h[i][j], r[j]);
          const uint4 hv = pack8(h[i]);
          unpack8(hv, h[i]);
          if (p.h && in[i]) p.h[base + i * nthr] = hv;
        }
        f32x2 s = mul2(h[i][0], h[i][0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) s = fma2(h[i][j], h[i][j], s);
        ss = __fadd_rn(ss, __fadd_rn(lo(s), hi(s)));
      }
    }
    ss = WARP_ROW ? warp_sum(ss) : group_sum(ss, sh, it & 1, 0, nthr >> 5, 0);
    const float rstd = __frsqrt_rn(__fadd_rn(__fmul_rn(ss, inv_c), p.eps));
    const f32x2 rstd2 = pair(rstd, rstd);
    if (p.rstd && tid == 0) p.rstd[row] = rstd;

#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      f32x2 y[4], gm[4];
      unpack8(gam[i], gm);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul2(mul2(h[i][j], rstd2), gm[j]);
      if (p.y && in[i]) p.y[base + i * nthr] = pack8(y);
      if (Q == blk::kNone) continue;
      float m = Q == blk::kFP8 ? amax : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max3_abs(m, lo(y[j]), hi(y[j]));
      float f = scale;
      if (Q == blk::kFP8) {
        if (in[i]) amax = m;             // a vector past the row's end may hold 0 * NaN
      } else {
        uint32_t mb = in[i] ? __float_as_uint(m) : 0u;
        if (Q == blk::kNVFP4) amax = __uint_as_float(max(__float_as_uint(amax), mb));
        // lanes that share a block: 4 x 8 values (2 x 8 for NVFP4)
        mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
        if (Q != blk::kNVFP4) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
        uint32_t word = Q == blk::kNVFP4 ? blk::nvfp4_scale(mb, scale, f) : blk::e8m0_scale(mb, emax, f);
        // the four scales of one atom word to the first lane of the 16 (8) that share it
        constexpr int kStep = Q == blk::kNVFP4 ? 2 : 4;
        if (!in[i]) word = 0;
        word |= __shfl_down_sync(0xffffffffu, word, kStep) << 8;
        word |= __shfl_down_sync(0xffffffffu, word, 2 * kStep) << 16;
        if (in[i] && (lane & (4 * kStep - 1)) == 0)
          *reinterpret_cast<uint32_t*>(p.sf + blk::atom_word(row, (i * nthr + tid) / (4 * kStep),
                                                             blk::atoms_per_row(p.cols, Q))) = word;
      }
      const f32x2 f2 = pair(f, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], f2);
      if (!in[i]) continue;
      if (Q == blk::kMXFP4 || Q == blk::kNVFP4) {
        const float v[8] = {lo(y[0]), hi(y[0]), lo(y[1]), hi(y[1]), lo(y[2]), hi(y[2]), lo(y[3]), hi(y[3])};
        reinterpret_cast<uint32_t*>(p.q)[base + i * nthr] = blk::cvt_e2m1x8(v);
      } else {
        reinterpret_cast<uint2*>(p.q)[base + i * nthr] = p.fmt == 0 ? codes8<0>(y) : codes8<1>(y);
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
      __shared__ uint32_t tops[kMaxThreads / 32];
      blk::cta_amax(p.amax_bits, __float_as_uint(amax), tops);
    }
    if (p.scale_inv && blockIdx.x == 0 && threadIdx.x == 0) *p.scale_inv = __fdiv_rn(1.0f, scale);
  }
}

// A CTA: row groups of p.group threads; group g takes rows blockIdx.x * groups + g, then every
// gridDim.x * groups-th. Dynamic shared memory: (groups - 1) x cols floats.
template <int VPT>
__global__ void __launch_bounds__(kBwdThreads, 1) k_rmsnorm_backward(const Bwd p) {
  extern __shared__ float part[];
  __shared__ float sh[2][32];
  const int nthr = p.group, groups = blockDim.x / nthr, g = threadIdx.x / nthr, tid = threadIdx.x - g * nthr;
  const int nvec = p.cols >> 3;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * groups;

  pdl_trigger();
  pdl_wait();
  constexpr bool kHold = VPT < 3;          // gamma and dres in registers (three vectors would spill, four do all the same)
  uint4 gam[kHold ? VPT : 1];
  f32x2 acc[VPT][4];
  bool in[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    in[i] = i * nthr + tid < nvec;
    if (kHold) gam[i] = in[i] ? ld_dep(p.gamma + i * nthr + tid) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
  }
  auto gamma = [&](int i) {
    return kHold ? gam[i] : in[i] ? ld_dep(p.gamma + i * nthr + tid) : make_uint4(0u, 0u, 0u, 0u);
  };
  const float inv_c = __fdiv_rn(1.0f, static_cast<float>(p.cols));

  int it = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g; row < p.rows; row += row_step, ++it) {
    const int64_t base = row * nvec + tid;
    const float rstd = ld_dep(p.rstd + row);
    const f32x2 rstd2 = pair(rstd, rstd);
    uint4 dv[VPT], hv[VPT], rv[kHold ? VPT : 1];
    if (tid == 0 && row + row_step < p.rows) {           // the row after this one into L2
      const int64_t next = (row + row_step) * nvec;
      l2_prefetch(p.dy + next, nvec * 16);
      l2_prefetch(p.h + next, nvec * 16);
      if (p.dres) l2_prefetch(p.dres + next, nvec * 16);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      dv[i] = load_or_zero(p.dy + base + i * nthr, in[i]);
      hv[i] = load_or_zero(p.h + base + i * nthr, in[i]);
    }
    if (kHold && p.dres) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) rv[i] = load_or_zero(p.dres + base + i * nthr, in[i]);
    }
    f32x2 s2 = 0ull;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      f32x2 d[4], h[4], gm[4];
      unpack8(dv[i], d);
      unpack8(hv[i], h);
      unpack8(gamma(i), gm);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 xh = mul2(h[j], rstd2);
        if (in[i]) acc[i][j] = fma2(d[j], xh, acc[i][j]);     // past the row's end: 0 * an infinite rstd
        if (in[i]) s2 = fma2(mul2(d[j], gm[j]), xh, s2);
      }
    }
    const float s = __fmul_rn(group_sum(__fadd_rn(lo(s2), hi(s2)), sh, it & 1, g * (nthr >> 5), nthr >> 5, g + 1), inv_c);
    const f32x2 ms2 = pair(-s, -s);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      f32x2 d[4], h[4], gm[4];
      unpack8(dv[i], d);
      unpack8(hv[i], h);
      unpack8(gamma(i), gm);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = mul2(rstd2, fma2(mul2(h[j], rstd2), ms2, mul2(d[j], gm[j])));
      if (p.dres) {
        unpack8(kHold ? rv[i] : load_or_zero(p.dres + base + i * nthr, in[i]), h);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = add2(d[j], h[j]);
      }
      if (in[i]) p.dh[base + i * nthr] = pack8(d);
    }
  }
  if (!p.partials) return;
  // the CTA's groups in order, then one partial row
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (g > 0 && in[i]) {
      float4* to = reinterpret_cast<float4*>(part + static_cast<int64_t>(g - 1) * p.cols + (i * nthr + tid) * 8);
      to[0] = make_float4(lo(acc[i][0]), hi(acc[i][0]), lo(acc[i][1]), hi(acc[i][1]));
      to[1] = make_float4(lo(acc[i][2]), hi(acc[i][2]), lo(acc[i][3]), hi(acc[i][3]));
    }
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (!in[i]) continue;
    const int c = (i * nthr + tid) * 8;
    float a[8] = {lo(acc[i][0]), hi(acc[i][0]), lo(acc[i][1]), hi(acc[i][1]),
                  lo(acc[i][2]), hi(acc[i][2]), lo(acc[i][3]), hi(acc[i][3])};
    for (int o = 0; o < groups - 1; ++o) {
      const float4* f = reinterpret_cast<const float4*>(part + static_cast<int64_t>(o) * p.cols + c);
      const float4 u = f[0], v = f[1];
      a[0] = __fadd_rn(a[0], u.x); a[1] = __fadd_rn(a[1], u.y); a[2] = __fadd_rn(a[2], u.z); a[3] = __fadd_rn(a[3], u.w);
      a[4] = __fadd_rn(a[4], v.x); a[5] = __fadd_rn(a[5], v.y); a[6] = __fadd_rn(a[6], v.z); a[7] = __fadd_rn(a[7], v.w);
    }
    float4* out = reinterpret_cast<float4*>(p.partials + static_cast<int64_t>(blockIdx.x) * p.cols + c);
    out[0] = make_float4(a[0], a[1], a[2], a[3]);
    out[1] = make_float4(a[4], a[5], a[6], a[7]);
  }
}

// dgamma: 32 columns per CTA; warp w adds partial rows w, w + 16, .. (at most ten, all loads in flight at
// once), then one sum over the warps in order.
constexpr int kReduceWarps = 16;
constexpr int kReduceLoads = (kBwdCtas + kReduceWarps - 1) / kReduceWarps;
__global__ void __launch_bounds__(32 * kReduceWarps)
    k_rmsnorm_dgamma(const float* partials, int n, int cols, float* out_f32, uint16_t* out_bf16) {
  __shared__ float sh[kReduceWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  pdl_trigger();
  pdl_wait();
  float v[kReduceLoads];
#pragma unroll
  for (int i = 0; i < kReduceLoads; ++i) {
    const int r = warp + i * kReduceWarps;
    v[i] = c < cols && r < n ? __ldcg(partials + static_cast<int64_t>(r) * cols + c) : 0.0f;
  }
  float a = v[0];
#pragma unroll
  for (int i = 1; i < kReduceLoads; ++i) a = __fadd_rn(a, v[i]);
  sh[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
#pragma unroll
  for (int w = 1; w < kReduceWarps; ++w) a = __fadd_rn(a, sh[w][lane]);
  if (out_f32) out_f32[c] = a;
  if (out_bf16) out_bf16[c] = static_cast<uint16_t>(pack2(a, a));
}

}  // namespace norm
}  // namespace fp8t
