// muon.cuh — orthogonalising a matrix by Newton-Schulz products, and the Muon step that is built on it.
//
//   m <- beta m + g / S,   u = g / S + beta m (Nesterov) or m,   X0 = u / |u|_F
//   five (or `steps`) times:   A = X X^T,   B = a I + b A + c A A,   X <- B X       (X^T X and X B for a tall X)
//   p <- p (1 - lr wd) - lr r sqrt(max(rows, cols)) X,   w = bf16(p)
// with (a, b, c) = (3.4445, -4.775, 2.0315): the polynomial a s + b s^3 + c s^5 drives every singular value s of X0
// (all at most 1) towards the band [0.68, 1.21].
//
// The products are FP16 with FP32 accumulation, on the pair tiles of gemm_pair.cuh. X, A and B are held in FP16 under a
// factor of 2^10: FP16 has 11 significant bits where BF16 has 8, at the same rate, and the factor keeps what FP16 has less
// of, range, out of the way. |X|_2 <= 1.21 and |B|_2 <= 3.5 bound every entry by 2^10 * 3.5; an entry below 2^-24 of the
// largest it may have (2^-14 * 2^-10, where FP16 turns subnormal) loses relative precision but its error stays below
// 2^-35, against a root mean square of X0's entries of 1 / sqrt(rows cols) (2^-12.7 for 4096 x 11008).
// Each rounding is one of 2^-12 of an entry, not correlated between entries, and the polynomial's slope is at most 3.45.
// a I stands in B, so X <- B X needs no third operand; its rounding is 2^-12 of a row of X again.
// A and B are symmetric: only the tiles on and above the diagonal are computed, and a tile off it is stored twice, once
// transposed. With s = min(rows, cols), l = max: s^2 l + s^3 + 2 s^2 l operations a step.
// |u|_F is summed in FP64. A call whose any |u|_F is not finite changes no m, p or w (as AdamW skips on a non-finite norm);
// where a product's wait expired p and w stay as they are (a result of muon_orthogonalize becomes NaN).
#pragma once

#include <cuda_fp16.h>

#include "gemm_pair.cuh"

namespace fp8t {
namespace muon {

using namespace pair;

constexpr float kFactor = 1024.0f;                         // of X, A and B

// ------------------------------------------------------------------ the products
struct alignas(64) Matmul {
  CUtensorMap a, b, d;             // operands in 128-byte boxes, D in 32 x 32 ones
  const uint16_t* c;               // FP16 [M][ldc] added with factor beta, or NULL
  float alpha, beta, diagonal;     // D = alpha acc + beta c + diagonal I
  int32_t M, N, num_kb, ldc;
  int32_t tiles_n, symmetric, tile_start;
  int32_t a_mn, b_mn;
  uint32_t idesc;
};
constexpr int kMaxMatrices = 24;
// Up to NP products; a launch's parameters are copied at every launch, and most calls have few matrices.
template <int NP>
struct alignas(64) Group {
  Matmul p[NP];
  int32_t n, total_tiles;
  int32_t* expired;                // set by a CTA whose waits expired
  __device__ __forceinline__ const Matmul& problem(int tile) const {
    int k = 0;
    while (k + 1 < n && p[k + 1].tile_start <= tile) ++k;
    return p[k];
  }
};

template <int NP>
struct Product {
  using Params = Group<NP>;
  struct Scalars {};
  static constexpr bool kF16 = true, kAmax = false;
  static __device__ __forceinline__ Scalars scalars(const Params&) { return {}; }
  static __device__ __forceinline__ void finish(const Params& g, uint32_t, bool aborted) {
    if (aborted) atomicExch(g.expired, 1);
  }
  static __device__ __forceinline__ int b_row(const Matmul&, int nt, int rank) { return nt * kBN + rank * kHalf; }
  static __device__ __forceinline__ void place(const Matmul& P, int local, int& mt, int& nt) {
    if (!P.symmetric) {
      mt = local / P.tiles_n;
      nt = local - mt * P.tiles_n;
      return;
    }
    mt = 0;                                                // rows of the upper triangle: tiles_n, tiles_n - 1, ...
    while (local >= P.tiles_n - mt) local -= P.tiles_n - mt++;
    nt = mt + local;
  }
  template <class Release>
  static __device__ __forceinline__ void epilogue(const Params&, const Matmul& P, const Scalars&, Out& o, int mt, int nt,
                                                  int row0, int half, uint32_t t_base, Release&& release) {
    const int row = row0 + o.lane;
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
      const int c = half * 128 + s * 32, n = nt * kBN + c;
      uint4 cv[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        cv[p] = make_uint4(0, 0, 0, 0);
        if (P.c && row < P.M && n + 8 * p < P.N)            // ldc is a multiple of 8, at least N
          cv[p] = ld_dep(reinterpret_cast<const uint4*>(P.c + static_cast<int64_t>(row) * P.ldc + n + 8 * p));
      }
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(t_base + c, r);
      tmem_ld_wait();
      tmem_reg_fence(r);
      if (s == 3) release();
      if (n >= P.N || row0 >= P.M) continue;
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t h = (&cv[j >> 2].x)[j & 3];
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        float lo = __fmul_rn(__uint_as_float(r[2 * j]), P.alpha), hi = __fmul_rn(__uint_as_float(r[2 * j + 1]), P.alpha);
        lo = fmaf(P.beta, f.x, lo);
        hi = fmaf(P.beta, f.y, hi);
        if (row == n + 2 * j) lo += P.diagonal;
        if (row == n + 2 * j + 1) hi += P.diagonal;
        w[j] = pack_f16x2(lo, hi);
      }
      store16(o, &P.d, w, n, row0);
      if (P.symmetric && mt != nt) store16_transposed(o, &P.d, w, row0, n);
    }
  }
};

// ------------------------------------------------------------------ the passes over the elements
enum : int { kMuon = 0, kOrthBf16 = 1, kOrthF32 = 2 };
struct Tensor {
  float* p;
  float* m;
  const void* g;                   // BF16 gradient, or the matrix to orthogonalise (BF16 or f32)
  uint16_t* w;                     // BF16 weight, or the result
  uint16_t* x;                     // FP16 [rows][pitch], after the last step the orthogonal factor
  int64_t numel;
  int32_t cols, pitch;
  int32_t chunk_start;             // of this table
  float rate;                      // lr r sqrt(max(rows, cols))
};
// 1 / |u|_F as two factors, so that neither overflows: x = (u * s1) * s2 is u / |u|_F * 2^10. ok: |u|_F is finite.
struct Norm {
  float s1, s2;
  int32_t ok, pad;
};
constexpr int kMaxTensors = kMaxMatrices;
struct Table {
  Tensor t[kMaxTensors];
  int32_t n, chunks;
  int32_t first;                   // number of the table's first tensor in the call, and the call's tensors
  int32_t all;
  float beta, inv_scale, keep;     // keep: 1 - lr wd
  int32_t nesterov;
  double* partials;                // one a chunk, of this table
  Norm* norms;                     // one a tensor, of the call
  int32_t* expired;                // a product of this table gave up waiting: its X is not to be used
  int32_t* skipped;
};
constexpr int kPassThreads = 256, kVec = 8, kChunk = kPassThreads * kVec * 4;   // elements of a CTA's chunk

__device__ __forceinline__ int find_tensor(const Table& t, int chunk) {
  int k = 0;
  while (k + 1 < t.n && t.t[k + 1].chunk_start <= chunk) ++k;
  return k;
}
__device__ __forceinline__ void bf16x8(uint4 x, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void f32x8(const float* p, float (&v)[8]) {
  const uint4 a = ld_dep(reinterpret_cast<const uint4*>(p)), b = ld_dep(reinterpret_cast<const uint4*>(p + 4));
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
}
__device__ __forceinline__ void put_f32x8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// Up to eight elements from e on (n of them; the rest zeros): the gradient or matrix, and the momentum.
template <int MODE>
__device__ __forceinline__ void load_g(const Tensor& T, int64_t e, int n, float (&v)[8]) {
  if (n == 8) {
    if constexpr (MODE == kOrthF32) f32x8(static_cast<const float*>(T.g) + e, v);
    else bf16x8(ld_dep(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(T.g) + e)), v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (j < n) {
      if constexpr (MODE == kOrthF32) v[j] = ld_dep(static_cast<const float*>(T.g) + e + j);
      else v[j] = __uint_as_float(static_cast<uint32_t>(ld_dep(static_cast<const uint16_t*>(T.g) + e + j)) << 16);
    }
  }
}
__device__ __forceinline__ void load_f32(const float* p, int64_t e, int n, float (&v)[8]) {
  if (n == 8) return f32x8(p + e, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < n ? ld_dep(p + e + j) : 0.0f;
}
// u and the new momentum of eight elements.
template <int MODE>
__device__ __forceinline__ void update(const Table& t, const Tensor& T, int64_t e, int n, float (&u)[8], float (&m)[8]) {
  load_g<MODE>(T, e, n, u);
  if constexpr (MODE == kMuon) {
    load_f32(T.m, e, n, m);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float g = __fmul_rn(u[j], t.inv_scale);
      m[j] = __fadd_rn(__fmul_rn(m[j], t.beta), g);
      u[j] = t.nesterov ? __fadd_rn(__fmul_rn(m[j], t.beta), g) : m[j];
    }
  }
}

// One partial sum of u^2 a chunk, in a fixed order.
template <int MODE>
__global__ void __launch_bounds__(kPassThreads) k_muon_sumsq(const __grid_constant__ Table t) {
  __shared__ double part[kPassThreads / 32];
  pdl_enter();
  const int chunk = blockIdx.x, k = find_tensor(t, chunk);
  const Tensor& T = t.t[k];
  const int64_t base = static_cast<int64_t>(chunk - T.chunk_start) * kChunk;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kChunk / (kPassThreads * kVec); ++i) {
    const int64_t e = base + (i * kPassThreads + threadIdx.x) * kVec;
    const int n = static_cast<int>(min(static_cast<int64_t>(8), T.numel - e));
    if (n <= 0) continue;
    float u[8], m[8];
    update<MODE>(t, T, e, n, u, m);
    // two f32 squares would overflow where their sum in FP64 does not
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __fma_rn(static_cast<double>(u[j]), static_cast<double>(u[j]), sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum = __dadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kPassThreads / 32; ++w) sum = __dadd_rn(sum, part[w]);
    t.partials[chunk] = sum;
  }
}

// A CTA a tensor: its chunks' sums in a fixed order, and the factors.
__global__ void __launch_bounds__(kPassThreads) k_muon_norms(const __grid_constant__ Table t) {
  __shared__ double part[kPassThreads];
  pdl_enter();
  const int k = blockIdx.x;
  const int c0 = t.t[k].chunk_start, c1 = k + 1 < t.n ? t.t[k + 1].chunk_start : t.chunks;
  double sum = 0.0;
  for (int c = c0 + threadIdx.x; c < c1; c += kPassThreads) sum = __dadd_rn(sum, ld_dep(t.partials + c));
  part[threadIdx.x] = sum;
  __syncthreads();
  for (int o = kPassThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) part[threadIdx.x] = __dadd_rn(part[threadIdx.x], part[threadIdx.x + o]);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    sum = part[0];
    Norm r = {0.0f, 0.0f, 1, 0};
    if (!isfinite(sum)) {
      r.ok = 0;
      r.s1 = r.s2 = __int_as_float(0x7FC00000);
    } else if (sum > 0.0) {                                // |u| = f 2^e, f in [0.5, 1); a zero matrix stays zero
      int e;
      const double f = frexp(sqrt(sum), &e);
      r.s1 = ldexpf(1.0f, -(e / 2));
      r.s2 = static_cast<float>(ldexp(static_cast<double>(kFactor) / f, -(e - e / 2)));
    }
    t.norms[t.first + k] = r;
  }
}

// Whether every tensor of the call has a finite norm; all threads call.
__device__ __forceinline__ bool all_finite(const Table& t) {
  int bad = 0;
  for (int i = threadIdx.x; i < t.all; i += kPassThreads) {
    const uint4 v = ld_dep(reinterpret_cast<const uint4*>(t.norms + i));
    bad |= v.z == 0;
  }
  return __syncthreads_or(bad) == 0;
}

// m <- its new value; X0 = u / |u| in FP16 under 2^10.
template <int MODE>
__global__ void __launch_bounds__(kPassThreads) k_muon_scale(const __grid_constant__ Table t) {
  pdl_enter();
  if (blockIdx.x == 0 && threadIdx.x == 0) *t.expired = 0;
  if (MODE == kMuon) {
    const bool go = all_finite(t);
    if (blockIdx.x == 0 && threadIdx.x == 0 && t.skipped) *t.skipped = go ? 0 : 1;
    if (!go) return;
  }
  const int chunk = blockIdx.x, k = find_tensor(t, chunk);
  const Tensor& T = t.t[k];
  const uint4 nv = ld_dep(reinterpret_cast<const uint4*>(t.norms + t.first + k));
  const float s1 = __uint_as_float(nv.x), s2 = __uint_as_float(nv.y);
  const int64_t base = static_cast<int64_t>(chunk - T.chunk_start) * kChunk;
#pragma unroll
  for (int i = 0; i < kChunk / (kPassThreads * kVec); ++i) {
    const int64_t e = base + (i * kPassThreads + threadIdx.x) * kVec;
    const int n = static_cast<int>(min(static_cast<int64_t>(8), T.numel - e));
    if (n <= 0) continue;
    float u[8], m[8];
    update<MODE>(t, T, e, n, u, m);
    if constexpr (MODE == kMuon) {
      if (n == 8) put_f32x8(T.m + e, m);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) T.m[e + j] = m[j];
    }
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = pack_f16x2(__fmul_rn(__fmul_rn(u[2 * j], s1), s2), __fmul_rn(__fmul_rn(u[2 * j + 1], s1), s2));
    if (T.pitch == T.cols) {                               // a multiple of 8: numel is one too
      *reinterpret_cast<uint4*>(T.x + e) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
      int64_t r = e / T.cols;
      int c = static_cast<int>(e - r * T.cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) T.x[r * T.pitch + c] = static_cast<uint16_t>(h[j >> 1] >> (16 * (j & 1)));
        if (++c == T.cols) c = 0, ++r;
      }
    }
  }
}

// The orthogonal factor into the weights (kMuon), or out as BF16.
template <int MODE>
__global__ void __launch_bounds__(kPassThreads) k_muon_apply(const __grid_constant__ Table t) {
  pdl_enter();
  const bool expired = ld_dep(t.expired) != 0;
  if (MODE == kMuon && !all_finite(t)) return;
  if (MODE == kMuon && expired) {                          // m is new, p and w stay
    if (blockIdx.x == 0 && threadIdx.x == 0 && t.skipped) *t.skipped = 1;
    return;
  }
  const int chunk = blockIdx.x, k = find_tensor(t, chunk);
  const Tensor& T = t.t[k];
  const int64_t base = static_cast<int64_t>(chunk - T.chunk_start) * kChunk;
#pragma unroll
  for (int i = 0; i < kChunk / (kPassThreads * kVec); ++i) {
    const int64_t e = base + (i * kPassThreads + threadIdx.x) * kVec;
    const int n = static_cast<int>(min(static_cast<int64_t>(8), T.numel - e));
    if (n <= 0) continue;
    float x[8];
    if (T.pitch == T.cols) {
      const uint4 h = ld_dep(reinterpret_cast<const uint4*>(T.x + e));
      const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
    } else {
      int64_t r = e / T.cols;
      int c = static_cast<int>(e - r * T.cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = 0.0f;
        if (j < n) x[j] = __half2float(__ushort_as_half(ld_dep(T.x + r * T.pitch + c)));
        if (++c == T.cols) c = 0, ++r;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = MODE != kMuon && expired ? __int_as_float(0x7FC00000) : x[j] * (1.0f / kFactor);
    if constexpr (MODE == kMuon) {
      float p[8];
      load_f32(T.p, e, n, p);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __fsub_rn(__fmul_rn(p[j], t.keep), __fmul_rn(T.rate, x[j]));
      if (n == 8) put_f32x8(T.p + e, x);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) T.p[e + j] = x[j];
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    if (n == 8) {
      *reinterpret_cast<uint4*>(T.w + e) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) T.w[e + j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

}  // namespace muon
}  // namespace fp8t
