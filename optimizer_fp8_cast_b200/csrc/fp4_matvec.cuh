// fp4_matvec.cuh — 4-bit weights times one to eight rows of BF16 activations, optionally with the gate of a feed-forward
// block: y = x . W^T, or y = act(x . Wg^T) * (x . Wu^T) with Wg and Wu the two halves of W's rows.
//
// W is what fp4_cast_multi writes: E2M1 codes [N][K/2] and scale atoms (E8M0 per 32 values, or E4M3 per 16 under a tensor
// scale whose inverse is the call's factor). The weights' bytes bound it: half a byte and a 32nd or 16th for each, once.
// So x stays BF16 (quantising it would save nothing), and the arithmetic has to be short next to the loads:
//   - a weight under its scale is a BF16 number exactly (2 significant bits times a power of two, or times 4 bits). A
//     code's three magnitude bits, put where BF16 has its low exponent bits and its first mantissa bit, are the value times
//     2^-126, subnormals included; one BF16 multiplication by the scale times 2^124 (E4M3: 2^117), both to stay in range, makes
//     two weights. Two shifts, two logic operations and one multiplication for two weights.
//   - products and sums are mma.sync m16n8k16: 16 rows of W, 8 tokens, FP32 accumulators. An FMA per weight and token
//     would cost as much as the decoding for one token and eight times that for eight. A tcgen05 tile would need the decoded
//     weights in shared memory and a 128-row tile's set-up, and would still be bound by the bytes.
// A lane holds 32 consecutive codes (16 bytes) of row g and of row g + 8, lanes 4g .. 4g + 3 the 128 values of a chunk; which of
// the lane's own values goes into which k of an MMA is free as long as x is taken in the same order: the code
// pairs (i, i + 4) of a word. The gated form takes the up row of the same output for row g + 8, so a lane has both.
// A CTA takes 16 rows (8 gated outputs), its warps the chunks of K in turn, all of a warp's loads of a round in flight; the
// warps' sums are added in shared memory in warp order.
#pragma once

#include <cuda_fp16.h>

#include "gated.cuh"

namespace fp8t {
namespace mv {

struct Params {
  const uint16_t* x;               // BF16 [rows][K]
  const uint8_t* q;                // codes
  const uint8_t* sf;               // scale atoms
  const float* factor;             // 1 / tensor scale, or NULL
  uint16_t* y;                     // BF16 [rows][N]
  int32_t rows, N, K;              // N: outputs
  int32_t words;                   // scale words of a row (atoms of a row block)
  int32_t act;                     // 0: W has N rows; else 2N
};
constexpr int kMaxRows = 8;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Codes i and i + 4 of a word as BF16 values times 2^-126.
template <int I>
__device__ __forceinline__ uint32_t raw_pair(uint32_t w) {
  const uint32_t mag = I <= 1 ? w << (6 - 4 * I) : w >> (4 * I - 6);
  const uint32_t sign = w << (12 - 4 * I);
  return (mag & 0x01C001C0u) | (sign & 0x80008000u);
}
// What multiplies the raw pairs of the lane's 32 codes. E8M0 code c: 2^(c - 127 + 124) as the BF16 exponent field c + 124, so
// that a weight is kept at a quarter (6 * 2^127 would not fit; 0.5 * 2^-127 * 2^-2 still does, as a subnormal), and above
// what that field holds a second power of two (blocks of values of 2^4 and more).
__device__ __forceinline__ uint32_t e8m0_factor(uint32_t c, uint32_t& more) {
  more = c > 130u ? (c - 3u) << 7 : 0x3F80u;
  uint32_t f = min(c + 124u, 254u) << 7;
  if (c == 255u) f = 0x7FC0u, more = 0x3F80u;
  more |= more << 16;
  return f | f << 16;
}
// E4M3 scales (two bytes) times 2^117, each in both halves of a word.
__device__ __forceinline__ void e4m3_factors(uint32_t c, uint32_t& f0, uint32_t& f1) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(c));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const float up = __int_as_float((117 + 127) << 23);
  f0 = __byte_perm(__float_as_uint(f.x * up), 0, 0x3232);
  f1 = __byte_perm(__float_as_uint(f.y * up), 0, 0x3232);
}

// A row's 32 codes and their scale bytes, as loaded.
struct Piece {
  uint4 q;
  uint32_t s;
};
template <bool NV>
__device__ __forceinline__ Piece load_piece(const Params& p, int row, bool in, int k, int t, int chunk) {
  Piece r = {make_uint4(0, 0, 0, 0), 0u};
  if (in) {
    r.q = ld_dep(reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(row) * (p.K / 2) + k / 2));
    if constexpr (NV) {
      const uint8_t* at = p.sf + blk::atom_word(row, 2 * chunk + (t >> 1), p.words) + (t & 1) * 2;
      r.s = ld_dep(reinterpret_cast<const uint16_t*>(at));
    } else {
      uint16_t both;                                       // the byte's pair: 16 bits are loaded as aligned
      const uint8_t* at = p.sf + blk::atom_word(row, chunk, p.words) + (t & 2);
      both = ld_dep(reinterpret_cast<const uint16_t*>(at));
      r.s = (both >> ((t & 1) * 8)) & 0xFFu;
    }
  }
  return r;
}
// 8 codes of a row: four BF16 pairs.
__device__ __forceinline__ void decode(uint32_t w, uint32_t f, uint32_t (&v)[4]) {
  v[0] = mul_bf16x2(raw_pair<0>(w), f);
  v[1] = mul_bf16x2(raw_pair<1>(w), f);
  v[2] = mul_bf16x2(raw_pair<2>(w), f);
  v[3] = mul_bf16x2(raw_pair<3>(w), f);
}

// One chunk of 16 rows: 8 MMAs.
template <bool NV>
__device__ __forceinline__ void chunk_mma(float (&acc)[4], const Piece& a, const Piece& b, const uint32_t (&x)[16]) {
  uint32_t fa[2], fb[2], ma = 0x3F803F80u, mb = 0x3F803F80u;
  if constexpr (NV) {
    e4m3_factors(a.s, fa[0], fa[1]);
    e4m3_factors(b.s, fb[0], fb[1]);
  } else {
    fa[0] = fa[1] = e8m0_factor(a.s, ma);
    fb[0] = fb[1] = e8m0_factor(b.s, mb);
  }
  const uint32_t qa[4] = {a.q.x, a.q.y, a.q.z, a.q.w}, qb[4] = {b.q.x, b.q.y, b.q.z, b.q.w};
  const bool large = !NV && __any_sync(0xffffffffu, ma != 0x3F803F80u || mb != 0x3F803F80u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t va[4], vb[4];
    decode(qa[i], fa[i >> 1], va);
    decode(qb[i], fb[i >> 1], vb);
    if (large) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        va[j] = mul_bf16x2(va[j], ma);
        vb[j] = mul_bf16x2(vb[j], mb);
      }
    }
    mma_bf16(acc, va[0], vb[0], va[1], vb[1], x[4 * i], x[4 * i + 1]);
    mma_bf16(acc, va[2], vb[2], va[3], vb[3], x[4 * i + 2], x[4 * i + 3]);
  }
}

// R: groups of 16 rows of a CTA, which share the loads of x; U: chunks in flight; W: most warps.
template <bool NV, int R, int U, int W>
__global__ void __launch_bounds__(32 * W) k_fp4_matvec(const __grid_constant__ Params p) {
  __shared__ float part[W][R][4][33];                      // [warp][group][accumulator][lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int per = p.act ? 8 : 16;                          // outputs of a group
  const int chunks = (p.K + 127) / 128;
  float acc[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.0f;
  pdl_enter();
  for (int c0 = warp; c0 < chunks; c0 += U * warps) {
    Piece a[U][R], b[U][R];
    uint4 xv[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * warps, k = c * 128 + t * 32;
      const bool in = k < p.K;                             // K is a multiple of 32
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int n = (blockIdx.x * R + r) * per + g, second = p.act ? p.N + n : n + 8;
        a[u][r] = load_piece<NV>(p, n, in && n < p.N, k, t, c);
        b[u][r] = load_piece<NV>(p, second, in && (p.act ? n : n + 8) < p.N, k, t, c);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xv[u][i] = make_uint4(0, 0, 0, 0);
        if (in && g < p.rows) xv[u][i] = ld_dep(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(g) * p.K + k) + i);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u * warps >= chunks) break;                 // the same for the warp
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {                        // values (0, 4), (1, 5), (2, 6), (3, 7)
        const uint4 v = xv[u][i];
        x[4 * i] = __byte_perm(v.x, v.z, 0x5410);
        x[4 * i + 1] = __byte_perm(v.x, v.z, 0x7632);
        x[4 * i + 2] = __byte_perm(v.y, v.w, 0x5410);
        x[4 * i + 3] = __byte_perm(v.y, v.w, 0x7632);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) chunk_mma<NV>(acc[r], a[u][r], b[u][r], x);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][r][j][lane] = acc[r][j];
  __syncthreads();
  // accumulator j of lane 4g + t: row g (j < 2) or its second row, token 2t + (j & 1)
  const float factor = (p.factor ? ld_dep(p.factor) : 1.0f) * (NV ? 512.0f : 4.0f);
  for (int i = threadIdx.x; i < R * per * kMaxRows; i += blockDim.x) {
    const int token = i / (R * per), o = i - token * R * per, r = o / per, row = o - r * per;
    const int n = (blockIdx.x * R + r) * per + row;
    if (token >= p.rows || n >= p.N) continue;
    const int l = (row & 7) * 4 + (token >> 1), j = (token & 1) + (row >> 3) * 2;
    float v = 0.0f, w = 0.0f;
    for (int s = 0; s < warps; ++s) {
      v += part[s][r][j][l];
      if (p.act) w += part[s][r][j + 2][l];
    }
    v *= factor;
    if (p.act) v = v * (p.act == gated::kSilu ? gated::gate<gated::kSilu>(v) : gated::gate<gated::kGelu>(v)) * (w * factor);
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    p.y[static_cast<int64_t>(token) * p.N + n] = h;
  }
}

}  // namespace mv
}  // namespace fp8t
