// gated_rows.cuh — the gated feed-forward product of gated.cuh for few rows (tokens): h = act(G) * U, [G | U] = (A . W) * sa * sb.
//
// The weights' bytes bound it, once each, and a pair tile (256 rows for one token) leaves a third of the SMs with a tile more than
// the others and streams each tile through one SM pair: 1 x 4096 -> 2 x 11008 30 us, 13.8 of them the bytes. Here the tensor
// cores are used as mma.sync m16n8k32 on FP8: 16 rows of W, 8 gate and the 8 up rows of the same outputs, so that a lane has both;
// 8 tokens; FP32 accumulators. A warp's lanes load the weights straight into the operand's registers; which of a lane's own k
// goes into which place of the MMA is free as long as A is taken in the same order:
//   W as [2N][K]  a lane holds 16 consecutive k of a row, lanes 4g .. 4g + 3 a chunk of 64: two MMAs of two words each
//   W as [K][2N]  a lane holds 4 consecutive outputs of four rows of k: a 4 x 4 byte transpose (8 byte permutations for 16
//                 weights) makes the words of four k, and the MMA's row g is output 4g + j of the j-th MMA
// The warps of a CTA take the chunks of K in turn, the next ones' loads on their way during a chunk's arithmetic, and add up in shared
// memory in warp order. More than eight tokens: a CTA for each eight, which finds the weights in L2; that pays while they are few.
#pragma once

#include "gated.cuh"

namespace fp8t {
namespace gated {

struct RowParams {
  const uint8_t* a;                // [M][K]
  const uint8_t* w;                // [2N][K], or [K][2N]
  uint16_t* gu;                    // [M][2N], or NULL
  uint16_t* h;                     // [M][N], or NULL
  uint8_t* q;                      // [M][N], or NULL
  const float* sa;
  const float* sb;
  const float* scale;
  unsigned int* amax_bits;
  float* scale_inv;
  int32_t M, N, K, act, fmt;
};
constexpr int kRowWarps = 8, kRowTokens = 8;

template <int WF, int AF>
__device__ __forceinline__ void mma_fp8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
#define FP8T_MMA(W, A)                                                                                                         \
  asm("mma.sync.aligned.m16n8k32.row.col.f32." W "." A ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};" \
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                                        \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (WF == 0 && AF == 0) FP8T_MMA("e4m3", "e4m3");
  else if constexpr (WF == 0) FP8T_MMA("e4m3", "e5m2");
  else if constexpr (AF == 0) FP8T_MMA("e5m2", "e4m3");
  else FP8T_MMA("e5m2", "e5m2");
#undef FP8T_MMA
}

// 1 / scale, by one thread of the grid: also where a wait expired, as the pair tiles do (the scale is not the call's result).
__device__ __forceinline__ void store_scale_inv(const RowParams& p) {
  if (p.scale_inv && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.scale_inv = __fdiv_rn(1.0f, ld_dep(p.scale));
}

// The sums of a CTA's warps for output o (of `outs`) and token, and what becomes of them. part: [warp][outs / 8][4][32 + 1] floats, of
// accumulator j of lane 4g + t: gate (j < 2) or up of the output in place g of group `o / 8`, token 2t + (j & 1); place and group as
// `at` gives them.
template <class At>
__device__ __forceinline__ void finish_rows(const RowParams& p, const float* part, int warps, int outs, int n0, int token0, At&& at) {
  const float alpha = __fmul_rn(ld_dep(p.sa), ld_dep(p.sb)), scale = p.scale ? ld_dep(p.scale) : 1.0f;
  const int tokens = min(kRowTokens, p.M - token0), per_warp = outs / 8 * 4 * 33;
  float top = 0.0f;
  for (int i = threadIdx.x; i < outs * tokens; i += blockDim.x) {
    const int token = i / outs, o = i - token * outs, n = n0 + o;
    if (n >= p.N) continue;
    int place, group;
    at(o, place, group);
    const float* s = part + (group * 4 + (token & 1)) * 33 + place * 4 + (token >> 1);
    float g = 0.0f, u = 0.0f;
    for (int w = 0; w < warps; ++w, s += per_warp) {
      g += s[0];
      u += s[2 * 33];
    }
    g = __fmul_rn(g, alpha);
    u = __fmul_rn(u, alpha);
    const int64_t row = token0 + token;
    if (p.gu) {
      const uint32_t both = pack_bf16x2(g, u);
      p.gu[row * 2 * p.N + n] = static_cast<uint16_t>(both);
      p.gu[row * 2 * p.N + p.N + n] = static_cast<uint16_t>(both >> 16);
    }
    const float h = g * (p.act == kSilu ? gate<kSilu>(g) : gate<kGelu>(g)) * u;
    top = max_abs(top, h, h);
    if (p.h) p.h[row * p.N + n] = static_cast<uint16_t>(pack_bf16x2(h, h));
    if (p.q) {
      const float v = __fmul_rn(h, scale);
      p.q[row * p.N + n] = static_cast<uint8_t>(p.fmt == 0 ? cvt_fp8x2<0>(v, v) : cvt_fp8x2<1>(v, v));
    }
  }
  if (p.amax_bits) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7FFFFFFFu);
    if ((threadIdx.x & 31) == 0 && most) atomicMax(p.amax_bits, most > 0x7F800000u ? 0x7FC00000u : most);
  }
  store_scale_inv(p);
}

// W [2N][K]: a CTA takes 16 outputs, a warp all of them for its chunks of 64 k, whose loads are D chunks ahead. Three CTAs on an SM
// for D = 1, two for D = 2 (32 outputs and two CTAs, whose 344 do not all fit at once, 23.2 us for 1 x 4096 -> 2 x 11008).
template <int WF, int AF, int D>
__global__ void __launch_bounds__(32 * kRowWarps, D == 1 ? 3 : 2) k_gated_rows(const __grid_constant__ RowParams p) {
  constexpr int R = 2;
  __shared__ float part[kRowWarps][R][4][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 8 * R, token0 = blockIdx.y * kRowTokens;
  const int chunks = (p.K + 63) / 64;
  // outputs past N and tokens past M are loaded as the last one: what they give is not stored
  const uint8_t* w[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t n = min(n0 + 8 * r + g, p.N - 1);
    w[r][0] = p.w + n * p.K + warp * 64 + t * 16;
    w[r][1] = w[r][0] + static_cast<int64_t>(p.N) * p.K;
  }
  const uint8_t* a = p.a + static_cast<int64_t>(min(token0 + g, p.M - 1)) * p.K + warp * 64 + t * 16;
  float acc[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.0f;
  pdl_enter();
  uint4 wv[D][R][2], av[D];
  auto load = [&](int d, int c) {
    const bool in = c * 64 + t * 16 < p.K;                 // K is a multiple of 16
    av[d] = in ? ld_dep(reinterpret_cast<const uint4*>(a)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wv[d][r][h] = in ? ld_dep(reinterpret_cast<const uint4*>(w[r][h])) : make_uint4(0, 0, 0, 0);
        w[r][h] += 64 * warps;
      }
    a += 64 * warps;
  };
  auto multiply = [&](const uint4 (&v)[R][2], const uint4& x) {
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mma_fp8<WF, AF>(acc[r], v[r][0].x, v[r][1].x, v[r][0].y, v[r][1].y, x.x, x.y);
      mma_fp8<WF, AF>(acc[r], v[r][0].z, v[r][1].z, v[r][0].w, v[r][1].w, x.z, x.w);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, warp + d * warps);
  for (int c = warp; c < chunks; c += D * warps) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      uint4 now[R][2];
      const uint4 x = av[d];
#pragma unroll
      for (int r = 0; r < R; ++r) now[r][0] = wv[d][r][0], now[r][1] = wv[d][r][1];
      if (D > 1 || c + warps < chunks) load(d, c + (D + d) * warps);                   // zeros past K
      multiply(now, x);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][r][j][lane] = acc[r][j];
  __syncthreads();
  finish_rows(p, &part[0][0][0][0], warps, 8 * R, n0, token0, [](int o, int& place, int& group) {
    place = o & 7;
    group = o >> 3;
  });
}

// Four words whose bytes are four outputs of a k each -> four words whose bytes are the four k of an output each.
__device__ __forceinline__ void transpose4(const uint32_t (&v)[4], uint32_t (&o)[4]) {
  const uint32_t a = __byte_perm(v[0], v[1], 0x5140), b = __byte_perm(v[2], v[3], 0x5140);   // outputs 0 and 1
  const uint32_t c = __byte_perm(v[0], v[1], 0x7362), d = __byte_perm(v[2], v[3], 0x7362);   // 2 and 3
  o[0] = __byte_perm(a, b, 0x5410);
  o[1] = __byte_perm(a, b, 0x7632);
  o[2] = __byte_perm(c, d, 0x5410);
  o[3] = __byte_perm(c, d, 0x7632);
}

// W [K][2N]: a CTA takes 32 G outputs, a warp all of them for its chunks of 32 k. Each warp keeps `ring` chunks on their way into
// shared memory (two boxes of 32 k x 32 G outputs, with 128 of them in the 128-byte swizzle, against bank conflicts) and waits for
// them alone; 144 to 192 KB of an SM are in flight. A's words come kAhead chunks ahead, in registers: one chunk ahead their latency
// was the chunk's time (8 x 4096 -> 2 x 11008 21.7 -> 19.8 us, 1 x 11008 -> 2 x 4096 28.2 -> 26.2; since slots are filled behind their
// reads 21.0 and 27.7).
constexpr int kMaxRing = 9, kAhead = 4;
constexpr int row_smem_bytes(int groups, int ring, int warps) { return warps * ring * 2 * 32 * 32 * groups + 1024; }
struct alignas(64) RowMnParams {
  CUtensorMap w;
  RowParams p;
  int32_t ring;                    // 2 .. kMaxRing
};
template <int WF, int AF, int G>
__global__ void __launch_bounds__(32 * kRowWarps, 1) k_gated_rows_mn(const __grid_constant__ RowMnParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t landed[kRowWarps][kMaxRing], taken[kRowWarps];
  __shared__ int given_up;
  const RowParams& p = P.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  constexpr int kOuts = 32 * G, kBytes = 2 * 32 * kOuts;
  const int n0 = blockIdx.x * kOuts, token0 = blockIdx.y * kRowTokens;
  const int chunks = (p.K + 31) / 32;
  if (lane < P.ring) mbar_init(smem_u32(&landed[warp][lane]), 1);
  if (lane == 0) mbar_init(smem_u32(&taken[warp]), 1);
  fence_mbar_init();
  if (threadIdx.x == 0) given_up = 0;
  __syncthreads();
  const uint64_t limit = wait_limit_ns();
  const bool expire = expire_mode() == kExpireAll;
  pdl_enter();
  uint8_t* mine = ring + warp * P.ring * kBytes;
  // boxes past K or 2N read zeros there; gate columns past N are the up projection's: what they give is not stored
  auto fetch = [&](int c, int s) {
    if (lane == 0 && c < chunks) {
      const uint32_t bar = smem_u32(&landed[warp][s]), dst = smem_u32(mine + s * kBytes);
      mbar_arrive_expect_tx(bar, kBytes);
      tma_load_2d(dst, &P.w, n0, c * 32, bar);
      tma_load_2d(dst + kBytes / 2, &P.w, p.N + n0, c * 32, bar);
    }
  };
  for (int s = 0; s < P.ring; ++s) fetch(warp + s * warps, s);
  // A slot that the lanes have issued their loads of: a __syncwarp alone does not keep the copy behind them (pair::fetch), so lane 0
  // sees an arrival first that it has queued behind them (a round trip: 1 x 11008 -> 2 x 4096 27.7 us, 26.1 without it; seen a
  // chunk's arithmetic later instead, the slot stays empty for that long, 28.6).
  uint32_t refills = 0;
  auto refill = [&](int c, int s) {
    __syncwarp();
    if (c >= chunks) return;
    if (lane == 0) {
      mbar_arrive(smem_u32(&taken[warp]));
      mbar_wait(smem_u32(&taken[warp]), refills & 1, limit);
    }
    ++refills;
    fetch(c, s);
  };
  // tokens past M are loaded as the last one; K is a multiple of 16
  const uint8_t* a = p.a + static_cast<int64_t>(min(token0 + g, p.M - 1)) * p.K + 4 * t;
  auto x_of = [&](int c, int h) {
    const int k = c * 32 + 16 * h;
    return k < p.K ? ld_dep(reinterpret_cast<const uint32_t*>(a + k)) : 0u;
  };
  // a lane's k are 4t .. of each 16, read in the order i ^ t, so that the four t of a word lie in different rows of banks
  int at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * t + (i ^ t);
    at[i] = row * kOuts + (G == 4 ? ((g >> 2) ^ (row & 7)) * 16 + (g & 3) * 4 : 4 * g);
  }
  const int order = t == 0 ? 0x3210 : t == 1 ? 0x2301 : t == 2 ? 0x1032 : 0x0123;
  float acc[4 * G][4];
#pragma unroll
  for (int j = 0; j < 4 * G; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
  uint32_t next[kAhead][2];
  auto load_x = [&](int c) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h) next[d][h] = x_of(c + d * warps, h);
  };
  load_x(warp);
  int s = 0, parity = 0;
  bool there = true;
  for (int c0 = warp; c0 < chunks && there; c0 += kAhead * warps) {
    uint32_t x[kAhead][2];
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h) x[d][h] = __byte_perm(next[d][h], 0, order);
    load_x(c0 + kAhead * warps);
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      const int c = c0 + d * warps;
      if (c >= chunks || !there) break;
      there = warp_wait(smem_u32(&landed[warp][s]), parity, limit, expire);
      if (!there) {
        if (lane == 0) record_error(kErrTimeout);
        given_up = 1;
        break;
      }
      const uint8_t* slot = mine + s * kBytes;
#pragma unroll
      for (int q = 0; q < G; ++q) {                        // outputs 32q + 4g ..
        uint32_t v[2][2][4], m[2][2][4];                   // [half of the chunk][gate, up][k]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[h][u][i] = *reinterpret_cast<const uint32_t*>(slot + (at[i] ^ (G == 4 ? q * 32 : 0)) + h * 16 * kOuts + u * (kBytes / 2) + (G == 4 ? 0 : q * 32));
        if (q + 1 == G) refill(c + P.ring * warps, s);
        __syncwarp();                                      // the MMA's lanes together
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int u = 0; u < 2; ++u) transpose4(v[h][u], m[h][u]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_fp8<WF, AF>(acc[4 * q + j], m[0][0][j], m[0][1][j], m[1][0][j], m[1][1][j], x[d][0], x[d][1]);
      }
      if (++s == P.ring) s = 0, parity ^= 1;
    }
  }
  __syncthreads();
  if (given_up) {                                          // loads may still be in flight
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kSettleNs) {
    }
    if (threadIdx.x == 0 && p.amax_bits) atomicMax(p.amax_bits, 0x7FC00000u);
    store_scale_inv(p);
    return;
  }
  float* part = reinterpret_cast<float*>(ring);            // [warp][4 G][4][33]: 2112 G bytes a warp, of ring 2048 G and more
#pragma unroll
  for (int j = 0; j < 4 * G; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) part[((warp * 4 * G + j) * 4 + k) * 33 + lane] = acc[j][k];
  __syncthreads();
  finish_rows(p, part, warps, kOuts, n0, token0, [](int o, int& place, int& group) {
    place = (o & 31) >> 2;
    group = (o >> 5) * 4 + (o & 3);
  });
}

}  // namespace gated
}  // namespace fp8t
