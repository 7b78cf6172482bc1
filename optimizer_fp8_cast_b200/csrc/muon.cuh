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
// What that costs. A rounding is off by at most 2^-11 of an entry (2^-12.2 in root mean square), not correlated between entries. A step
// moves an error by the polynomial's slope: by 3.4445 in directions that are still small, by less than 1.6 (up to 4.2 at
// 1.21) in those that have arrived. So where most of them soon arrive the result is off by 1.0e-3 to 1.4e-3 of the factor's norm
// (matrices of noise, spectra that fall as k^-0.5; BF16 intermediates: about 8 times that), and where few do, the noise
// of X0's rounding, 2^-12.2 of its norm times 3.4445^5 = 485, decides: about 0.1 in norm beside a factor of norm sqrt(r) with r
// directions that have arrived. Measured over 256 x 256 to 2600 x 2400, relative to the factor: spectra k^-1 2e-3 to 4e-3, k^-1.5
// 1.0e-2 to 1.2e-2, k^-2 2.0e-2, k^-3 3.7e-2. (The rounding of a BF16 input does eight times that: k^-2 0.15.)
// a I stands in B, so X <- B X needs no third operand; its rounding is at most 2^-11.8 of a row of X, alike in every row.
// A and B are symmetric: only the tiles on and above the diagonal are computed, and a tile off it is stored twice, once
// transposed. With s = min(rows, cols), l = max: s^2 l + s^3 + 2 s^2 l operations a step.
// |u|_F is summed in FP64. A call whose any |u|_F is not finite changes no m, p or w (as AdamW skips on a non-finite norm);
// where a product's wait expired p and w stay as they are (a result of muon_orthogonalize becomes NaN).
#pragma once

#include <cuda_fp16.h>

#include "gemm_pair.cuh"
#include "quant_block.cuh"

namespace fp8t {
namespace muon {

using namespace pair;

constexpr float kFactor = 1024.0f;                         // of X, A and B

// ------------------------------------------------------------------ the products
// All of a table's steps are one launch: three phases a step (A, B, X) behind barriers of the grid. A launch of each phase
// took 9.5 us for a 256 x 256 matrix, of which the products are one (set-up 0.8 us, first loads 1.4, stores 0.9, launch 2).
struct alignas(64) Matrix {
  CUtensorMap x[2], s[2];          // operands in boxes of 64 rows x 64 values: X (two copies), A and B
  CUtensorMap xd[2], sd[2];        // the same as outputs, in boxes of 32 x 32
  int32_t rows, cols;
  int32_t sym_start, x_start;      // first tile in the phases of A and B, and of X
};
constexpr int kMaxMatrices = 24;
// Up to NP matrices: a launch's parameters are copied at every launch, and most calls have few matrices.
template <int NP>
struct alignas(64) Group {
  Matrix m[NP];
  int32_t n, steps;
  int32_t sym_tiles, x_tiles;      // of the phases
  int32_t tile_n;                  // columns of a tile: 256, or 128
  int32_t whole;                   // 1: every tile of A and B is computed, none mirrored
  Grid grid;
};

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;

template <int NP>
struct Steps {
  using Params = Group<NP>;
  struct Scalars {};
  static constexpr bool kF16 = true, kAmax = false, kPhased = true;
  static constexpr int kLoads = 1;
  static __device__ __forceinline__ Scalars scalars(const Params&) { return {}; }
  static __device__ __forceinline__ Grid grid(const Params& g) { return g.grid; }
  static __device__ __forceinline__ int phases(const Params& g) { return 3 * g.steps; }
  static __device__ __forceinline__ int tiles(const Params& g, int ph) { return ph % 3 == 2 ? g.x_tiles : g.sym_tiles; }
  static __device__ __forceinline__ bool reads(int ph) { return ph % 3 == 1; }      // B's epilogue reads A
  static __device__ __forceinline__ void finish(const Params& g, uint32_t, bool aborted) {
    if (aborted) atomicExch(g.grid.expired, 1);
  }
  static __device__ __forceinline__ Work work(const Params& g, int ph, int tile, int rank) {
    const int phase = ph % 3, cur = (ph / 3) & 1;          // X is copy `cur`, the step's result the other
    int k = 0;
    if (phase == 2) {
      while (k + 1 < g.n && g.m[k + 1].x_start <= tile) ++k;
    } else {
      while (k + 1 < g.n && g.m[k + 1].sym_start <= tile) ++k;
    }
    const Matrix& m = g.m[k];
    const bool wide = m.cols >= m.rows;
    const int side = wide ? m.rows : m.cols, lengthwise = wide ? m.cols : m.rows;
    Work w;
    w.which = k;
    w.a_mn = w.b_mn = 0;
    int inner = side;
    if (phase == 2) {                                      // wide: B X; tall: X B
      place_in_runs((m.rows + kBM - 1) / kBM, (m.cols + g.tile_n - 1) / g.tile_n, tile - m.x_start, w.mt, w.nt);
      w.a = wide ? &m.s[1] : &m.x[cur];
      w.b = wide ? &m.x[cur] : &m.s[1];
      w.b_mn = wide ? 1 : 0;
    } else {
      int local = tile - m.sym_start, n = (side + g.tile_n - 1) / g.tile_n;
      w.mt = 0;
      if (g.whole) {
        w.mt = local / n;
        w.nt = local - w.mt * n;
      } else {                                             // the tiles on and above the diagonal: rows of n, n - 1, ...
        while (local >= n) local -= n--, ++w.mt;
        w.nt = w.mt + local;
      }
      w.a = w.b = phase == 0 ? &m.x[cur] : &m.s[0];
      if (phase == 0) {                                    // wide: rows of X; tall: its columns
        inner = lengthwise;
        w.a_mn = w.b_mn = wide ? 0 : 1;
      }
    }
    w.a_row = w.mt * kBM + rank * kHalf;
    w.half_n = g.tile_n / 2;
    w.b_row = w.nt * g.tile_n + rank * w.half_n;
    w.a_bytes = kABytes;
    w.num_kb = (inner + 63) / 64;
    w.idesc = make_idesc_f16(w.a_mn, w.b_mn, g.tile_n);
    return w;
  }
  static __device__ __forceinline__ void fetch_at(const Params& g, const Work& w, Out& o, int row0, int n) {
    const CUtensorMap* const maps[1] = {&g.m[w.which].sd[0]};
    const int x[1] = {n};
    fetch(o, maps, x, row0);
  }
  static __device__ __forceinline__ void prefetch(const Params& g, const Work& w, int ph, Out& o, int row0, int half) {
    if (reads(ph)) fetch_at(g, w, o, row0, 2 * w.half_n * w.nt + half * w.half_n);
  }
  // 32 columns of the accumulator, times alpha: with READ also kB times A's values and a I.
  template <bool READ, class Release, class Ahead>
  static __device__ __forceinline__ bool chunks(const Params& g, const Work& w, const CUtensorMap* d, Out& o, int row0, int half,
                                                int M, int N, bool mirrored, float alpha, uint32_t t_base, Release&& release,
                                                Ahead&& ahead) {
    using namespace blk;
    const int steps = w.half_n / 32;
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      const int c = half * w.half_n + s * 32, n = 2 * w.half_n * w.nt + c;
      uint4 av[4];
      if constexpr (READ) {
        if (!fetched(o)) return false;
        chunk_row(o, 0, av);
        if (s + 1 < steps) fetch_at(g, w, o, row0, n + 32);
        else ahead();
      }
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(t_base + c, r);
      tmem_ld_wait();
      tmem_reg_fence(r);
      if (s + 1 == steps) release();
      if (n >= N || row0 >= M) continue;
      const f32x2 al = blk::pair(alpha, alpha), be = blk::pair(kB, kB);
      f32x2 v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        v[j] = mul2(blk::pair(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), al);
        if constexpr (READ) {
          const uint32_t h = (&av[j >> 2].x)[j & 3];
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          v[j] = fma2(be, blk::pair(f.x, f.y), v[j]);
        }
      }
      uint32_t q[16];
      if (READ && row0 == n) {                             // the diagonal runs through this chunk
#pragma unroll
        for (int j = 0; j < 16; ++j)
          q[j] = pack_f16x2(lo(v[j]) + (o.lane == 2 * j ? kA * kFactor : 0.0f), hi(v[j]) + (o.lane == 2 * j + 1 ? kA * kFactor : 0.0f));
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) q[j] = pack_f16x2(lo(v[j]), hi(v[j]));
      }
      store16(o, d, q, n, row0);
      if (mirrored) store16_transposed(o, d, q, row0, n);
    }
    return true;
  }
  template <class Release, class Ahead>
  static __device__ __forceinline__ bool epilogue(const Params& g, const Work& w, int ph, const Scalars&, Out& o, int row0, int half,
                                                  uint32_t t_base, Release&& release, Ahead&& ahead) {
    const Matrix& m = g.m[w.which];
    const int phase = ph % 3, side = min(m.rows, m.cols);
    const bool mirrored = phase < 2 && !g.whole && w.mt != w.nt;
    if (phase == 1) return chunks<true>(g, w, &m.sd[1], o, row0, half, side, side, mirrored, kC / kFactor, t_base, release, ahead);
    const bool sym = phase == 0;
    return chunks<false>(g, w, sym ? &m.sd[0] : &m.xd[((ph / 3) & 1) ^ 1], o, row0, half, sym ? side : m.rows, sym ? side : m.cols,
                         mirrored, 1.0f / kFactor, t_base, release, ahead);
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
  Grid grid;                       // of the products; expired: one gave up waiting, and X is not to be used
  int32_t* gave_up;                // kMuon: some table's products have
  int32_t* skipped;
  int32_t last;                    // 1: the call's last table
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
// Up to eight elements of a row from e on (`left` of them), 16 bytes aligned or not.
template <int MODE>
__device__ __forceinline__ void load_row(const void* g, int64_t e, int left, bool aligned, float (&v)[8]) {
  const float* f = static_cast<const float*>(g) + e;
  const uint16_t* b = static_cast<const uint16_t*>(g) + e;
  if (aligned && left > 0) {
    if constexpr (MODE == kOrthF32) f32x8(f, v);
    else bf16x8(ld_dep(reinterpret_cast<const uint4*>(b)), v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (j < left) {
      if constexpr (MODE == kOrthF32) v[j] = ld_dep(f + j);
      else v[j] = __uint_as_float(static_cast<uint32_t>(ld_dep(b + j)) << 16);
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

// The factors from the sum of u^2.
__device__ __forceinline__ Norm norm_of(double sum) {
  Norm r = {0.0f, 0.0f, 1, 0};
  if (!isfinite(sum)) {
    r.ok = 0;
    r.s1 = r.s2 = __int_as_float(0x7FC00000);
  } else if (sum > 0.0) {                                  // |u| = f 2^e, f in [0.5, 1); a zero matrix stays zero
    int e;
    const double f = frexp(sqrt(sum), &e);
    r.s1 = ldexpf(1.0f, -(e / 2));
    r.s2 = static_cast<float>(ldexp(static_cast<double>(kFactor) / f, -(e - e / 2)));
  }
  return r;
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
  if (threadIdx.x == 0) t.norms[t.first + k] = norm_of(part[0]);
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
  if (blockIdx.x == 0 && threadIdx.x == 0) *t.grid.counter = 0, *t.grid.expired = 0;
  if (MODE == kMuon) {
    // skipped until the last table's weights are written: a call that fails between the launches has not made the step
    if (blockIdx.x == 0 && threadIdx.x == 0 && t.first == 0) {
      *t.gave_up = 0;
      if (t.skipped) *t.skipped = 1;
    }
    if (!all_finite(t)) return;
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
  const bool expired = ld_dep(t.grid.expired) != 0;
  if (MODE == kMuon) {
    if (!all_finite(t)) return;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      if (expired) *t.gave_up = 1;
      else if (t.last && t.skipped && ld_dep(t.gave_up) == 0) *t.skipped = 0;
    }
    if (expired) return;                                   // m is new, p and w stay
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

// ------------------------------------------------------------------ small matrices
// Up to 256 x 256: one CTA pair keeps a matrix in shared memory over all steps. The phases of the grid-wide form have little to do
// there (6.4 us each, of which the MMAs are one: barrier, first loads, stores); here the epilogue writes the next phase's
// operand where the tensor cores read it (256 x 256: fifteen launches 142 us a call, grid-wide 97, here 40.2; 1.9 us a phase, of
// which the tensor cores compute 1.1).
// CTA r holds (FP16, 128-byte swizzle, zeros past the matrix):
//   xk   rows 128r .. of X, K-major: four blocks of 64 columns
//   xm   columns 128r .. of X, all rows, MN-major: four blocks of 64 rows, each two boxes of 64 columns
//   s    rows 128r .. of A, then of B, K-major
// wide: A = xk xk^T, X <- s xm;  tall: A = xm^T xm, X <- xk s.
// A phase computes the columns 64h .. and 128 + 64h .. (64 each) for h = 0, then h = 1: a CTA's own rows or columns hold the 64 that
// it brings as the second operand, and the first half's epilogue runs beside the second's MMAs (50.8 -> 47.9 us). For that a wide
// matrix's results go elsewhere than its operands: B takes xk's place and the next X that of s, and they change names every step;
// the next phase's MMAs start with the half that is there (47.7 -> 45.8). A tall one waits for both halves.
// A's epilogue leaves (b A + a I) / c in a second accumulator, to which A^2 is added, so that B's only scales (55.5 -> 50.6, with
// A read back from s before).
// X's epilogue writes xk. Its lines lie in xm of the CTA that has their columns just as they do here: an otherwise idle warp
// brings them there, the other CTA's by asynchronous copies (46.0 -> 40.1; the epilogue's own stores of them took 0.7 us a half,
// and all of them by that warp's stores 5 us a step).
constexpr int kSmallSide = 256, kSmallBlock = 16384, kSmallOperand = 4 * kSmallBlock;
constexpr int kSmallN = 128;                              // columns of half a phase
constexpr int kSmallTmem = 512;                           // two accumulators
constexpr int kSmallThreads = 64 + 32 * 16;               // 16 epilogue warps: a TMEM lane quarter and 32 columns of a half each
constexpr int kSmallSmemBytes = 3 * kSmallOperand + 1024 + 512;
struct alignas(64) SmallMatrix {
  CUtensorMap x;                   // kMuon: boxes of 64 rows x 64 values of X0
  const void* g;                   // otherwise: the matrix, rows of cols
  uint16_t* out;                   // kMuon: X in FP16, rows of pitch; otherwise the result
  int32_t rows, cols, pitch, pad;
};
struct alignas(64) SmallGroup {
  SmallMatrix m[kMaxMatrices];     // a CTA pair each
  int32_t steps;
  int32_t* expired;
};
struct SmallSmem {
  double sums[32];                 // of u^2: the cluster's warps
  uint64_t loaded;                 // X has landed
  uint64_t acc_full[2];            // both CTAs: the MMAs of half a phase's columns have completed
  uint64_t ready[2];               // even CTA: the epilogue warps of both have stored that half's results
  uint64_t lines[2];               // this CTA's epilogue warps have stored that half of X
  uint64_t sent;                   // the other CTA's lines of xm have come
  uint64_t columns;                // even CTA: xm is there in both
  uint64_t mma_done;
  uint32_t tmem_base;
  int given_up;                    // a wait expired
};
static_assert(sizeof(SmallSmem) <= 512, "");

// kMuon: X0 comes from the workspace and X goes back there. Otherwise the kernel is the whole call: norm, X0, steps and result, 8 us of
// it where the four passes around the steps took 13.
template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kSmallThreads, 1) k_muon_small(const __grid_constant__ SmallGroup g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* xk = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *xm = xk + kSmallOperand, *sq = xm + kSmallOperand;
  SmallSmem* S = reinterpret_cast<SmallSmem*>(sq + kSmallOperand);
  volatile int* given_up = &S->given_up;
  const SmallMatrix& M = g.m[blockIdx.x >> 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool wide = M.cols >= M.rows;
  const int side = wide ? M.rows : M.cols, lengthwise = wide ? M.cols : M.rows;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&S->loaded), 1);
    mbar_init(smem_u32(&S->acc_full[0]), 1);
    mbar_init(smem_u32(&S->acc_full[1]), 1);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&S->lines[i]), 16);
    mbar_init(smem_u32(&S->sent), 1);
    mbar_init(smem_u32(&S->columns), 2);
    mbar_init(smem_u32(&S->ready[0]), 32);
    mbar_init(smem_u32(&S->ready[1]), 32);
    mbar_init(smem_u32(&S->mma_done), 1);
    *given_up = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&S->tmem_base), kSmallTmem);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  const uint64_t limit = wait_limit_ns();
  const int expire = expire_mode();
  const bool expire_main = expire == kExpireAll, expire_epi = expire == kExpireAll || expire == kExpireGemmEpilogue;
  pdl_enter();
  // Both CTAs give up: who waits for one that has done so waits in vain, and all meet behind the steps.
  auto give_up = [&] {
    if (lane == 0) {
      record_error(kErrTimeout);
      for (uint32_t r = 0; r < 2; ++r)
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&S->given_up), r)), "r"(1) : "memory");
    }
    __syncwarp();
  };
  if constexpr (MODE != kMuon) {
    // a warp takes every 16th of the CTA's rows, a lane eight columns
    const int part = warp - 2, n = lane * 8;
    float v[8][8];
    if (warp >= 2) {
      // A thread's 64 squares in f32 where they are in its range: sixteen roundings of a partial sum and two of the partials', so
      // a sum is off by at most 18 * 2^-24, less than 2^-19, of which the norm has half and X0 is rounded to 2^-11; FP64
      // throughout took 1 us more.
      float part4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int all = static_cast<int>(rank) * kHalf + i * 16 + part;
        load_row<MODE>(M.g, static_cast<int64_t>(all) * M.cols + n, all < M.rows ? M.cols - n : 0, M.cols % 8 == 0, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) part4[j & 3] = __fmaf_rn(v[i][j], v[i][j], part4[j & 3]);
      }
      const float squares = __fadd_rn(__fadd_rn(part4[0], part4[1]), __fadd_rn(part4[2], part4[3]));
      double sum = static_cast<double>(squares);
      if (!(squares >= 0x1p-60f && squares <= 0x1p100f)) {
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = __fma_rn(static_cast<double>(v[i][j]), static_cast<double>(v[i][j]), sum);
      }
      __syncwarp();
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum = __dadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      if (lane < 2)
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&S->sums[rank * 16 + part]), lane)), "d"(sum) : "memory");
      __syncwarp();
    }
    cluster_sync();
    if (warp >= 2) {
      double sum = S->sums[lane];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum = __dadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      const Norm norm = norm_of(sum);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = i * 16 + part;
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = __fmul_rn(__fmul_rn(v[i][2 * j], norm.s1), norm.s2), x1 = __fmul_rn(__fmul_rn(v[i][2 * j + 1], norm.s1), norm.s2);
          h[j] = pack_f16x2(x0, x1);                       // zeros past the matrix, or all of it NaN
        }
        const int at = ((lane & 7) ^ (row & 7)) * 16;
        *reinterpret_cast<uint4*>(xk + (n >> 6) * kSmallBlock + row * 128 + at) = make_uint4(h[0], h[1], h[2], h[3]);
        const int all = static_cast<int>(rank) * kHalf + row;
        const uint32_t to = smem_u32(xm + (all >> 6) * kSmallBlock + ((n & 127) >> 6) * 8192 + (all & 63) * 128 + at);
        st_cluster_v4(mapa_shared(to, n >> 7), h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async_all();
    }
  } else if (warp == 0) {
    if (elect_one()) {
      mbar_arrive_expect_tx(smem_u32(&S->loaded), 2 * kSmallOperand);
      const int at = static_cast<int>(rank) * kHalf;
      for (int b = 0; b < 4; ++b)
        for (int i = 0; i < 2; ++i) {
          const uint32_t to = smem_u32(xk + b * kSmallBlock + i * 8192);
          tma_load_2d(to, &M.x, b * 64, at + i * 64, smem_u32(&S->loaded));
          tma_load_2d(to + kSmallOperand, &M.x, at + i * 64, b * 64, smem_u32(&S->loaded));
        }
    }
    __syncwarp();
    if (!warp_wait(smem_u32(&S->loaded), 0, limit, expire_main)) give_up();
  }
  cluster_sync();                                          // X is there in both CTAs
  const int phases = *given_up ? 0 : 3 * g.steps;
  if (warp == 0) {
    // ---------------- X's columns: lines of xk lie in xm of the CTA that has them as they do here
    bool there = true;
    for (int step = 0; 3 * (step + 1) < phases && there; ++step) {
      const uint8_t* x = wide && !(step & 1) ? sq : xk;    // the step's result
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(&S->sent), kSmallOperand / 2);
      for (int h = 0; h < 2 && there; ++h) {
        there = warp_wait(smem_u32(&S->lines[h]), step & 1, limit, expire_epi);
        if (!there) break;
        for (int i = 0; i < 2; ++i) {                      // 64 rows x 64 columns: the other CTA's, and this one's
          const int at = (static_cast<int>(rank) * 2 + i) * kSmallBlock + h * 8192;
          const uint8_t* from = x + h * kSmallBlock + i * 8192;
          if (lane == 0)
            bulk_copy_cluster(mapa_shared(smem_u32(xm + at), rank ^ 1), smem_u32(from + (rank ^ 1) * 2 * kSmallBlock), 8192,
                              mapa_shared(smem_u32(&S->sent), rank ^ 1));
          const uint4* own = reinterpret_cast<const uint4*>(from + rank * 2 * kSmallBlock) + lane;
          uint4* to = reinterpret_cast<uint4*>(xm + at) + lane;
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = own[(j + k) * 32];
#pragma unroll
            for (int k = 0; k < 8; ++k) to[(j + k) * 32] = v[k];
          }
        }
      }
      if (there) there = warp_wait(smem_u32(&S->sent), step & 1, limit, expire_epi);
      if (!there) {
        give_up();
        break;
      }
      fence_proxy_async_all();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&S->columns), 0));
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issuer
    for (int ph = 0; ph < phases; ++ph) {
      const int phase = ph % 3;
      const bool swapped = wide && ((ph / 3) & 1);
      const uint32_t k0 = smem_u32(swapped ? sq : xk), m0 = smem_u32(xm), s0 = smem_u32(swapped ? xk : sq);
      const bool a_mn = phase == 0 && !wide, b_mn = phase == 0 ? !wide : phase == 2 && wide;
      const uint32_t a0 = phase == 0 ? (wide ? k0 : m0) : phase == 1 ? s0 : k0;
      const uint32_t b0 = phase == 0 ? (wide ? k0 : m0) : phase == 1 || !wide ? s0 : m0;
      const uint32_t idesc = make_idesc_f16(a_mn, b_mn, kSmallN);
      const int blocks = ((phase == 0 ? lengthwise : side) + 63) / 64;
      auto multiply = [&](int h, int b) {
        if (b >= blocks) return;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = a0 + b * kSmallBlock, c = b0 + b * kSmallBlock + h * 8192;
          tc_mma_f16_pair(tmem + (phase == 1 ? kSmallSide : 0) + h * kSmallN,
                          a_mn ? make_sw128_desc_mn16(a + k * 2048) : make_sw128_desc(a + k * 32),
                          b_mn ? make_sw128_desc_mn16(c + k * 2048) : make_sw128_desc(c + k * 32), idesc,
                          (b | k) != 0 || phase == 1 ? 1u : 0u);
        }
      };
      bool there = ph == 0 || warp_wait(smem_u32(&S->ready[0]), (ph - 1) & 1, limit, expire_main);
      // xm has come: a tall matrix's phase 0 reads it, a wide one's phase 1 lets its lines in xk be written over
      if (there && ph >= 3 && phase == (wide ? 1 : 0)) there = warp_wait(smem_u32(&S->columns), (ph / 3 - 1) & 1, limit, expire_main);
      if (there && ph > 0 && !wide) there = warp_wait(smem_u32(&S->ready[1]), (ph - 1) & 1, limit, expire_main);
      tc_fence_after();
      if (there && elect_one()) {
        multiply(0, 0);
        multiply(0, 2);
      }
      __syncwarp();
      if (there && ph > 0 && wide) there = warp_wait(smem_u32(&S->ready[1]), (ph - 1) & 1, limit, expire_main);
      if (!there) {
        give_up();
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        multiply(0, 1);
        multiply(0, 3);
        tc_commit_pair_mc(smem_u32(&S->acc_full[0]), 0x3);
        for (int b = 0; b < 4; ++b) multiply(1, b);
        tc_commit_pair_mc(smem_u32(&S->acc_full[1]), 0x3);
      }
      __syncwarp();
    }
  } else if (warp >= 2) {
    // ---------------- epilogue: what becomes the next phase's operand
    using namespace blk;
    const int quad = warp & 3, part = (warp - 2) >> 2, row = quad * 32 + lane;         // of this CTA's 128
    bool there = true;
    for (int ph = 0; ph < phases && there; ++ph) {
      const int phase = ph % 3;
      const bool swapped = wide && ((ph / 3) & 1);
      uint8_t *kx = swapped ? sq : xk, *ks = swapped ? xk : sq;
      const float alpha = (phase == 1 ? kC : 1.0f) / kFactor;
      const f32x2 al = blk::pair(alpha, alpha);
      const bool last = ph + 1 == 3 * g.steps;
      uint8_t* to = phase == 0 || (wide && phase == 2) ? ks : wide || phase == 2 ? kx : ks;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // a tall matrix's phases 1 and 2 write where the second half's MMAs read
        if (there) there = warp_wait(smem_u32(&S->acc_full[h]), ph & 1, limit, expire_epi);
        if (there && h == 0 && !wide && phase > 0) there = warp_wait(smem_u32(&S->acc_full[1]), ph & 1, limit, expire_epi);
        if (!there) {
          give_up();
          break;
        }
        tc_fence_after();
        const int n = (part >> 1) * 128 + h * 64 + (part & 1) * 32;                  // the columns' place in the matrix
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + h * kSmallN + part * 32;
        uint8_t* line = to + (n >> 6) * kSmallBlock + row * 128;                     // K-major place of (row, n ..)
        const int piece = (n >> 3) & 7;
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(acc + (phase == 1 ? kSmallSide : 0), r);
        tmem_ld_wait();
        tmem_reg_fence(r);
        uint4 q[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint4* place = reinterpret_cast<uint4*>(line + ((piece + p) ^ (row & 7)) * 16);
          uint32_t out[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = 8 * p + 2 * j;
            const f32x2 v = mul2(blk::pair(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), al);
            out[j] = pack_f16x2(lo(v), hi(v));
          }
          q[p] = make_uint4(out[0], out[1], out[2], out[3]);
          *place = q[p];
        }
        if (phase == 0) {                                // where c A^2 is to be added up: b A + a I
          // A as it was rounded, which is the A of A^2: what its rounding does to b A and to c A^2 then cancels for the most part
          // where A is near I (b + 2c = -0.7; with the A before its rounding the factor's error was up to twice as large)
#pragma unroll
          for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t h = (&q[p].x)[j];
              const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h));
              r[8 * p + 2 * j] = __float_as_uint(a.x * (kFactor * kB / kC));
              r[8 * p + 2 * j + 1] = __float_as_uint(a.y * (kFactor * kB / kC));
            }
          if (static_cast<int>(rank) * kHalf + quad * 32 == n) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              r[c] = __float_as_uint(__uint_as_float(r[c]) + (c == lane ? kA / kC * (kFactor * kFactor) : 0.0f));
          }
          tmem_st_32x32b_x32(acc + kSmallSide, r);
          tmem_st_wait();
        }
        tc_fence_before();
        fence_proxy_async_all();                           // for the tensor cores of both CTAs
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(mapa_shared(smem_u32(&S->ready[h]), 0));
          if (phase == 2 && !last) mbar_arrive(smem_u32(&S->lines[h]));
        }
      }
    }
  }
  __syncwarp();
  cluster_sync();
  const bool alive = *given_up == 0;
  if (warp >= 2) {
    // ---------------- the result, a warp a row
    const uint8_t* x = wide && (g.steps & 1) ? sq : xk;
    const int pitch = MODE == kMuon ? M.pitch : M.cols, n = lane * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = i * 16 + warp - 2, all = static_cast<int>(rank) * kHalf + row;
      if (all >= M.rows || n >= M.cols) continue;
      uint16_t* o = M.out + static_cast<int64_t>(all) * pitch + n;
      const uint4 q = *reinterpret_cast<const uint4*>(x + (n >> 6) * kSmallBlock + row * 128 + ((lane & 7) ^ (row & 7)) * 16);
      if constexpr (MODE == kMuon) {
        *reinterpret_cast<uint4*>(o) = q;                  // within the pitch, a multiple of 8
      } else {
        const uint32_t f[4] = {q.x, q.y, q.z, q.w};
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
          w[j] = alive ? pack_bf16x2(v.x * (1.0f / kFactor), v.y * (1.0f / kFactor)) : 0x7FC07FC0u;
        }
        if (M.cols % 8 == 0) {
          *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (n + j < M.cols) o[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
        }
      }
    }
  }
  if (!alive) {
    if (warp == 1 && rank == 0) {                          // MMAs may be in flight
      if (elect_one()) tc_commit_pair(smem_u32(&S->mma_done));
      __syncwarp();
      mbar_wait(smem_u32(&S->mma_done), 0, kDrainLimitNs);
    }
    if (threadIdx.x == 0) {
      if (MODE == kMuon) atomicExch(g.expired, 1);
      const uint64_t t0 = globaltimer_ns();                // loads and copies too
      while (globaltimer_ns() - t0 < kSettleNs) {
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_arrive();               // neither CTA leaves while the other may still write to it or the MMAs read it; a release would
  cluster_wait();                 // wait for the result's stores
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kSmallTmem);
}

}  // namespace muon
}  // namespace fp8t
