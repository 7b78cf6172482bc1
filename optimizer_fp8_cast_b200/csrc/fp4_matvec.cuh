// fp4_matvec.cuh — 4-bit weights times one to eight rows of BF16 activations, optionally with the gate of a feed-forward
// block: y = x . W^T, or y = act(x . Wg^T) * (x . Wu^T) with Wg and Wu the two halves of W's rows.
//
// W is what fp4_cast_multi writes: E2M1 codes [N][K/2] and scale atoms (E8M0 per 32 values, or E4M3 per 16 under a tensor
// scale whose inverse is the call's factor). The weights' bytes bound it: half a byte and a 32nd or 16th for each, once.
// So x stays BF16 (quantising it would save nothing), and the arithmetic has to be short next to the loads:
//   - a weight under its scale is a BF16 number exactly (2 significant bits times a power of two, or times 4 bits). A
//     code's three magnitude bits, put where BF16 has its low exponent bits and its first mantissa bit, are the value times
//     2^-126, subnormals included; one BF16 multiplication by the scale times 2^124 (E4M3: 2^117), both to stay in range, makes
//     two weights.
//   - products and sums are mma.sync m16n8k16: 16 rows of W, 8 tokens, FP32 accumulators. An FMA per weight and token
//     would cost as much as the decoding for one token and eight times that for eight. A tcgen05 tile would need the decoded
//     weights in shared memory and a 128-row tile's set-up, and would still be bound by the bytes.
// A lane holds 32 consecutive codes (16 bytes) of row g and of row g + 8, lanes 4g .. 4g + 3 the 128 values of a chunk; which of
// the lane's own values goes into which k of an MMA is free as long as x is taken in the same order: the code
// pairs (i, i + 4) of a word. The gated form takes the up row of the same output for row g + 8, so a lane has both.
// A group is 16 rows (8 gated outputs); the warps of a CTA take its chunks of K in turn, and their sums are added in shared
// memory in warp order.
// What bounds it: for few weights the launch and one trip to memory (1 x 4096 x 4096 4.6 us, 1.4 of them its bytes). For many
// (4 x 4096 x 2 x 11008 NVFP4 18.2 us, 7.8 its bytes) no unit is full: by the profiler's counters 3.5 instructions a weight and lane take
// 58% of the issue slots, the logic pipe 57% and DRAM 30%; 1.3 of a scheduler's 4.9 warps are ready in a cycle, and a third of
// a warp's time is spent on loads that its chunk has just issued, for nothing is loaded ahead of a chunk's arithmetic here. With
// one CTA of 16 warps and loads ahead (8 x 11008 x 4096) the slots are at 58% too, 3.9 warps a scheduler, 128 CTAs for 148 SMs. Measured and not kept: a persistent form with three chunks of a warp in
// flight and x in shared memory in the order of the MMAs (21.9 us, and 8 x 11008 x 4096 17.5: filling 176 KB of x is in
// nobody's shadow).
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
// Codes I and I + 4 of a word (I = 0 or 1) as BF16 values times 2^-126. The two nibbles times 2^6 + 2^12 (I = 1: 2^2 + 2^8) put the
// magnitude at bits 6 to 8 and the sign at bit 15; the two copies of a nibble do not meet, and what else there is of them is
// masked away. The multiplication leaves the two logic operations to the pipe that is short here: shifts run on
// the same half-rate pipe as logic does.
template <int I>
__device__ __forceinline__ uint32_t raw_pair(uint32_t w) {
  return (w & (0x000F000Fu << (4 * I))) * (I == 0 ? 0x1040u : 0x104u) & 0x81C081C0u;
}
// What multiplies the raw pairs of the lane's 32 codes. E8M0 code c: 2^(c - 127 + 124) as the BF16 exponent field c + 124, so
// that a weight is kept at a quarter (6 * 2^127 would not fit; 0.5 * 2^-127 * 2^-2 still does, as a subnormal). Above c = 130
// (blocks of values of 2^4 and more) the field is full and a second power of two is needed; 255 is NaN.
constexpr uint32_t kOneE8m0 = 130;
__device__ __forceinline__ uint32_t e8m0_factor(uint32_t c) { return c * 0x00800080u + 0x3E003E00u; }
__device__ __forceinline__ uint32_t e8m0_large(uint32_t c, uint32_t& more) {
  more = c > kOneE8m0 ? (c - 3u) << 7 : 0x3F80u;
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

// A row's 32 codes of a chunk and their scales: E4M3 two bytes, E8M0 the pair of bytes that holds the lane's (16 bits are
// loaded as aligned).
struct Piece {
  uint4 q;
  uint32_t s;
};

// 8 codes of a row: four BF16 pairs.
__device__ __forceinline__ void decode(uint32_t w, uint32_t f, uint32_t (&v)[4]) {
  v[0] = mul_bf16x2(raw_pair<0>(w), f);
  v[1] = mul_bf16x2(raw_pair<1>(w), f);
  v[2] = mul_bf16x2(raw_pair<0>(w >> 8), f);
  v[3] = mul_bf16x2(raw_pair<1>(w >> 8), f);
}

// One chunk of 16 rows: 8 MMAs.
template <bool NV>
__device__ __forceinline__ void chunk_mma(float (&acc)[4], const Piece& a, const Piece& b, const uint4 (&xv)[4], int t) {
  uint32_t fa[2], fb[2], ma = 0x3F803F80u, mb = 0x3F803F80u;
  bool large = false;
  if constexpr (NV) {
    e4m3_factors(a.s, fa[0], fa[1]);
    e4m3_factors(b.s, fb[0], fb[1]);
  } else {
    const uint32_t ca = (a.s >> ((t & 1) * 8)) & 0xFFu, cb = (b.s >> ((t & 1) * 8)) & 0xFFu;
    fa[0] = fa[1] = e8m0_factor(ca);
    fb[0] = fb[1] = e8m0_factor(cb);
    large = __any_sync(0xffffffffu, max(ca, cb) > kOneE8m0);
    if (large) {
      fa[0] = fa[1] = e8m0_large(ca, ma);
      fb[0] = fb[1] = e8m0_large(cb, mb);
    }
  }
  const uint32_t qa[4] = {a.q.x, a.q.y, a.q.z, a.q.w}, qb[4] = {b.q.x, b.q.y, b.q.z, b.q.w};
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
    mma_bf16(acc, va[0], vb[0], va[1], vb[1], xv[i].x, xv[i].y);
    mma_bf16(acc, va[2], vb[2], va[3], vb[3], xv[i].z, xv[i].w);
  }
}

// Eight consecutive values of x in the order of the code pairs: (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint4 in_pairs(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632));
}

// W: most warps; B: CTAs that an SM is to hold; AHEAD: the next chunk is loaded before a chunk's arithmetic. A warp takes two
// groups, which share its x (one: 4 x 4096 x 2 x 11008 21.2 us for 18.2, 8 x 11008 x 4096 12.1 for 11.0).
constexpr int kGroups = 2;
template <bool NV, int W, int B, bool AHEAD>
__global__ void __launch_bounds__(32 * W, B) k_fp4_matvec(const __grid_constant__ Params p) {
  constexpr int R = kGroups;
  __shared__ float part[W][R][4][33];                      // [warp][group][accumulator][lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int per = p.act ? 8 : 16, n0 = blockIdx.x * per * R;   // outputs of a group; this CTA's first
  const int chunks = (p.K + 127) / 128;
  // Rows past N and tokens past the last are loaded as the last one: what they give is not stored.
  const uint8_t *q[R][2], *s[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int n = min(n0 + r * per + g, p.N - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = h == 0 ? n : p.act ? p.N + n : min(n + 8, p.N - 1);
      q[r][h] = p.q + row * (p.K / 2) + warp * 64 + t * 16;
      s[r][h] = p.sf + blk::atom_word(row, NV ? 2 * warp : warp, p.words) + (NV ? (t >> 1) * 512 + (t & 1) * 2 : t & 2);
    }
  }
  const uint16_t* x = p.x + static_cast<int64_t>(min(g, p.rows - 1)) * p.K + warp * 128 + t * 32;
  const int q_step = 64 * warps;
  const int64_t s_step = (NV ? 1024 : 512) * static_cast<int64_t>(warps);
  float acc[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.0f;
  pdl_enter();
  Piece w[R][2];
  uint4 xv[4];
  auto load = [&](int c) {                                 // the next chunk, c; a warp's pointers move on
    if (c * 128 + t * 32 < p.K) {                          // K is a multiple of 32
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[r][h].q = ld_dep(reinterpret_cast<const uint4*>(q[r][h]));
          w[r][h].s = ld_dep(reinterpret_cast<const uint16_t*>(s[r][h]));
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[i] = ld_dep(reinterpret_cast<const uint4*>(x) + i);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) w[r][0] = w[r][1] = {make_uint4(0, 0, 0, 0), 0u};
      xv[0] = xv[1] = xv[2] = xv[3] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        q[r][h] += q_step;
        s[r][h] += s_step;
      }
    x += 128 * warps;
  };
  if (AHEAD && warp < chunks) load(warp);
  for (int c = warp; c < chunks; c += warps) {
    if (!AHEAD) load(c);
    Piece now[R][2];
    uint4 xn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xn[i] = in_pairs(xv[i]);
#pragma unroll
    for (int r = 0; r < R; ++r) now[r][0] = w[r][0], now[r][1] = w[r][1];
    if (AHEAD && c + warps < chunks) load(c + warps);
    __syncwarp();                                          // the MMA's and the vote's lanes together
#pragma unroll
    for (int r = 0; r < R; ++r) chunk_mma<NV>(acc[r], now[r][0], now[r][1], xn, t);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][r][j][lane] = acc[r][j];
  __syncthreads();
  // accumulator j of lane 4g + t: row g (j < 2) or its second row, token 2t + (j & 1)
  const float factor = (p.factor ? ld_dep(p.factor) : 1.0f) * (NV ? 512.0f : 4.0f);
  for (int i = threadIdx.x; i < R * per * p.rows; i += blockDim.x) {
    const int token = i / (R * per), o = i - token * R * per, r = o / per, row = o - r * per, n = n0 + o;
    if (n >= p.N) continue;
    const int l = (row & 7) * 4 + (token >> 1), j = (token & 1) + (row >> 3) * 2;
    float v = 0.0f, w = 0.0f;
    for (int k = 0; k < warps; ++k) {
      v += part[k][r][j][l];
      if (p.act) w += part[k][r][j + 2][l];
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
