// fp4_cast.cuh — BF16 -> 4-bit block-scaled quantisation (MXFP4, NVFP4), row-wise and column-wise.
//
// The arithmetic is in quant_block.cuh. The 4-bit tensor-core instruction reads both operands K-major
// only, so the column-wise copy (blocks down a column) is written transposed: its row c holds the codes
// of x's column c. Codes are two to a byte, the first in the low nibble; scales in 512-byte atoms, K
// padded to a multiple of 256 with zero scales (zero codes under them come from the GEMM's TMA fill).
//
// Row-wise copies alone (k_fp4_cast_rows): a thread takes 32 consecutive values (two 32-byte loads), so a scale
// is one thread's own work and no lanes exchange anything.
//
// With column-wise copies (k_fp4_cast): each 128 x 128 tile of x arrives as two TMA boxes of 128 rows x 64
// columns (128-byte swizzle) in a double buffer; rows and columns past the matrix read as zeros, which
// quantise to zero codes and the scales of an all-zero block, so the atoms of a ragged edge are complete.
// Every warp does an eighth of both copies:
//   column-wise: two adjacent columns of 32 rows per thread (one 4-byte shared load per row, a warp covers the
//     64 columns of a box row: no bank conflicts), 16 bytes of codes for each of the two transposed rows, staged
//     in shared memory (64-byte swizzle) and stored by one TMA box per tile (straight 16-byte stores, each half
//     a sector, cost 3.5 of 28 us on 8192 x 4096);
//   row-wise: a quarter-warp per block of 8 consecutive rows, 16 bytes of codes per block.
// NVFP4's amax is kept per thread from tile to tile and leaves the CTA by one atomic per tensor: one per warp and
// tile, all to one address, made 16384 x 11008 both ways 237 instead of 114 us.
// Bound: HBM, 2 B read + 0.5 B per copy written (+ 1/32 B MXFP4, 1/16 B NVFP4 of scales) per element. With both
// copies every element is quantised twice (BF16 pairs compared as pairs, multiplied as f32x2 pairs) and latency comes
// first: the 16 warps per SM that 127 registers leave use half of the issue slots and half of DRAM, stalled by turns on
// shared memory, dependencies and a tile's two barriers: 8192 x 4096 both ways 21 us (MXFP4) and 26 (NVFP4), row-wise 14.6 and 16.1
// (tiles with one copy: 16.2 and 18.8), 16384 x 11008 both ways 92 and 114, inputs and outputs of three calls in turn.
#pragma once

#include "ptx.cuh"
#include <cuda_bf16.h>

#include "quant_block.cuh"

namespace fp8t {
namespace fp4 {

constexpr int kTile = 128;
constexpr int kCastThreads = 256;
constexpr int kCastTensors = 8;
constexpr int kHalfBytes = kTile * 64 * 2;                 // one 128-row x 64-column BF16 box
constexpr int kXBytes = 2 * kHalfBytes;
constexpr int kAtomBytes = 2 * 512;                        // atoms of a tile and orientation (NVFP4: 2)
constexpr int kStageBytes = kTile * kTile / 2;             // column-wise codes of a tile: 128 rows of 64 bytes
constexpr int kCastSmemBytes = 2 * kXBytes + kStageBytes + 2 * kAtomBytes + 64 + 1024 /*alignment*/;

struct alignas(64) CastTensor {
  CUtensorMap x_map;               // BF16 [rows][cols], 64 x 128 boxes, 128-byte swizzle
  CUtensorMap qc_map;              // q_col as bytes [cols][rows / 2], 64 x 128 boxes, 64-byte swizzle
  const void* x;
  uint8_t* q_row;                  // [rows][cols / 2] (may be null)
  uint8_t* sf_row;                 // atoms [rows / 128][K = cols]
  uint8_t* q_col;                  // [cols][rows / 2] (may be null)
  uint8_t* sf_col;                 // atoms [cols / 128][K = rows]
  const float* scale;              // NVFP4
  unsigned int* amax_bits;         // NVFP4, may be null
  float* scale_inv;                // NVFP4, may be null
  int32_t rows, cols;
  int32_t tiles_c, tile_start;     // tiles: below 2^26 for rows * cols < 2^40
  int32_t kind;
};

struct alignas(64) CastGroup {
  CastTensor t[kCastTensors];
  int32_t n;
  int32_t total_tiles;
};

// Byte offset of BF16 element (row, col) in a tile as the two swizzled TMA boxes lay it out.
__device__ __forceinline__ uint32_t xoff(int row, int col) {
  return (col >> 6) * kHalfBytes + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}

__device__ __forceinline__ int cast_tensor_of(const CastGroup& g, int tile) {
  int ti = 0;
  while (ti + 1 < g.n && g.t[ti + 1].tile_start <= tile) ++ti;
  return ti;
}

// One thread: the loads of a tile, and its tensor, row tile and column tile for the CTA.
__device__ __forceinline__ void issue_cast_tile(const CastGroup& g, int tile, uint32_t dst, uint32_t bar, int4& at) {
  const int ti = cast_tensor_of(g, tile);
  const CastTensor& T = g.t[ti];
  const int local = tile - T.tile_start, rt = local / T.tiles_c, ct = local - rt * T.tiles_c;
  const int r0 = rt * kTile, c0 = ct * kTile;
  at = make_int4(ti, rt, ct, 0);
  mbar_arrive_expect_tx(bar, kXBytes);               // out-of-range parts are zero-filled
  tma_load_2d(dst, &T.x_map, c0, r0, bar);
  tma_load_2d(dst + kHalfBytes, &T.x_map, c0 + 64, r0, bar);
}

// Larger magnitudes of two BF16 pairs, NaN if one is.
__device__ __forceinline__ uint32_t max_abs2(uint32_t acc, uint32_t v) {
  const __nv_bfloat162 r = __hmax2_nan(reinterpret_cast<const __nv_bfloat162&>(acc),
                                       __habs2(reinterpret_cast<const __nv_bfloat162&>(v)));
  return reinterpret_cast<const uint32_t&>(r);
}
// The two BF16 of a word times a pair of factors.
__device__ __forceinline__ void scale2(uint32_t w, blk::f32x2 f, float& lo, float& hi) {
  const blk::f32x2 v = blk::mul2(blk::pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)), f);
  lo = blk::lo(v);
  hi = blk::hi(v);
}

// Scale byte and factor of a block whose largest BF16 magnitude pattern is m. NVFP4: `factors` holds g / s
// for every scale code (a table in shared memory: a division per block took as long as its 16 codes).
template <bool NV>
__device__ __forceinline__ uint8_t block_scale(uint32_t m, float g, const float* factors, float& f) {
  if (!NV) return blk::e8m0_scale(m << 16, 2, f);
  const uint32_t c = blk::nvfp4_scale_code(m << 16, g);
  f = factors[c];
  return static_cast<uint8_t>(c);
}
// The table, by the first 128 threads.
__device__ __forceinline__ void fill_factors(float* factors, float g) {
  if (threadIdx.x < 128) factors[threadIdx.x] = blk::nvfp4_factor(threadIdx.x, g);
}

// Atom words of a row of K values, K padded to 256: 2 (MXFP4) or 4 (NVFP4) per 256. K goes up to 2^31 - 1, so the sum is
// unsigned.
__device__ __forceinline__ int atom_words(int K, int scales_per_32) {
  return static_cast<int>(((static_cast<uint32_t>(K) + 255u) >> 8) * 2u * scales_per_32);
}

// Position of scale j (0..7) of row r in a tile's one or two atoms.
__device__ __forceinline__ uint32_t atom_off(int r, int j) {
  return (j >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (j & 3);
}

// Two adjacent columns x 32 rows: 16 bytes of codes each, and their scales.
template <bool NV>
__device__ __forceinline__ void col_block(const uint8_t* xs, int rb, int col, float g, const float* factors,
                                          uint4 (&out)[2], uint8_t* atom) {
  constexpr int kB = NV ? 16 : 32, kN = 32 / kB;
  uint32_t code[2][4];
#pragma unroll
  for (int b = 0; b < kN; ++b) {
    uint32_t w[kB], m = 0;
#pragma unroll
    for (int r = 0; r < kB; ++r) w[r] = *reinterpret_cast<const uint32_t*>(xs + xoff(32 * rb + b * kB + r, col));
#pragma unroll
    for (int r = 0; r < kB; ++r) m = max_abs2(m, w[r]);
    float f0, f1;
    atom[atom_off(col, kN * rb + b)] = block_scale<NV>(m & 0xFFFFu, g, factors, f0);
    atom[atom_off(col + 1, kN * rb + b)] = block_scale<NV>(m >> 16, g, factors, f1);
    const blk::f32x2 f = blk::pair(f0, f1);
#pragma unroll
    for (int o = 0; o < kB / 8; ++o) {
      float a[8], c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) scale2(w[o * 8 + j], f, a[j], c[j]);
      code[0][b * (kB / 8) + o] = blk::cvt_e2m1x8(a);
      code[1][b * (kB / 8) + o] = blk::cvt_e2m1x8(c);
    }
  }
  out[0] = make_uint4(code[0][0], code[0][1], code[0][2], code[0][3]);
  out[1] = make_uint4(code[1][0], code[1][1], code[1][2], code[1][3]);
}

__device__ __forceinline__ uint32_t max_abs8(const uint4& v) {
  return max_abs2(max_abs2(max_abs2(max_abs2(0u, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint32_t code8(const uint4& v, float f) {
  const blk::f32x2 f2 = blk::pair(f, f);
  float a[8];
  scale2(v.x, f2, a[0], a[1]);
  scale2(v.y, f2, a[2], a[3]);
  scale2(v.z, f2, a[4], a[5]);
  scale2(v.w, f2, a[6], a[7]);
  return blk::cvt_e2m1x8(a);
}

// 32 consecutive values of a row: 16 bytes of codes, their scales; returns the largest magnitude pattern.
template <bool NV>
__device__ __forceinline__ uint32_t row_block(const uint8_t* xs, int row, int b32, float g, const float* factors,
                                              uint4& out, uint8_t* atom) {
  constexpr int kN = NV ? 2 : 1, kV = 4 / kN;            // blocks, and vectors of 8 per block
  uint4 w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const uint4*>(xs + xoff(row, 32 * b32 + 8 * k));
  uint32_t code[4], top = 0;
#pragma unroll
  for (int b = 0; b < kN; ++b) {
    uint32_t m2 = 0;
#pragma unroll
    for (int k = 0; k < kV; ++k) m2 = max_abs2(m2, max_abs8(w[b * kV + k]));
    const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    top = max(top, m);
    float f;
    atom[atom_off(row, kN * b32 + b)] = block_scale<NV>(m, g, factors, f);
#pragma unroll
    for (int k = 0; k < kV; ++k) code[b * kV + k] = code8(w[b * kV + k], f);
  }
  out = make_uint4(code[0], code[1], code[2], code[3]);
  return top;
}

__global__ void __launch_bounds__(kCastThreads, 2) k_fp4_cast(const __grid_constant__ CastGroup g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* xbuf = smem;                                             // [2][2 boxes][128][128 B]
  uint8_t* stage = smem + 2 * kXBytes;                              // [128 columns][64 B], swizzled
  uint8_t* atom_r = stage + kStageBytes;
  uint8_t* atom_c = atom_r + kAtomBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(atom_c + kAtomBytes);
  __shared__ int s_abort;
  __shared__ float factors[128];             // NVFP4: g / s of the current tensor
  __shared__ int4 where[2];                  // per buffer: tensor, row tile, column tile
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stride = static_cast<int>(gridDim.x);
  __shared__ uint32_t tops[kCastThreads / 32];
  int cur = -1;                              // tensor of the factors
  uint32_t top = 0;                          // its largest magnitude pattern in this thread's tiles
  uint32_t pending = 0, pending_ph = 0;      // thread 0: loads not yet consumed, their phases

  pdl_trigger();
  if (tid == 0) {
    mbar_init(smem_u32(&full[0]), 1);
    mbar_init(smem_u32(&full[1]), 1);
    fence_mbar_init();
    s_abort = 0;
  }
  pdl_wait();
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      const int tile = static_cast<int>(blockIdx.x) + b * stride;
      if (tile < g.total_tiles) {
        issue_cast_tile(g, tile, smem_u32(xbuf + b * kXBytes), smem_u32(&full[b]), where[b]);
        pending |= 1u << b;
      }
    }
  }
  __syncthreads();
  const uint64_t limit = wait_limit_ns();
  const bool expire = expire_mode() == kExpireAll;

  for (int i = 0, tile = static_cast<int>(blockIdx.x); tile < g.total_tiles; ++i, tile += stride) {
    const int buf = i & 1;
    if (tid == 0) {
      if (!mbar_wait(smem_u32(&full[buf]), static_cast<uint32_t>((i >> 1) & 1), limit, expire)) {
        record_error(kErrTimeout);
        s_abort = 1;
      } else {
        pending &= ~(1u << buf);
      }
      bulk_wait_group_read<0>();              // the previous tile's staged codes are stored
    }
    __syncthreads();                          // tile landed; the previous tile's atoms written
    if (s_abort) break;
    const int4 at = where[buf];
    const CastTensor& T = g.t[at.x];
    const int rt = at.y, ct = at.z, r0 = rt * kTile, c0 = ct * kTile, rows = T.rows, cols = T.cols;
    const bool nv = T.kind == blk::kNVFP4;
    const float gs = nv ? ld_dep(T.scale) : 1.0f;
    if (at.x != cur) {                        // the same in every thread; the factors of the last are read
      if (cur >= 0 && g.t[cur].amax_bits) blk::cta_amax(g.t[cur].amax_bits, top << 16, tops);
      cur = at.x;
      top = 0;
      if (nv) {
        fill_factors(factors, gs);
        __syncthreads();
      }
    }
    const uint8_t* xs = xbuf + buf * kXBytes;

    if (T.q_col) {
      // column-wise: rows 32 * (warp % 4) .. + 31, columns 2 * lane (+1) of box warp / 4
      const int rb = warp & 3, col = 64 * (warp >> 2) + 2 * lane;
      uint4 out[2];
      // a block past the matrix has zero values; under g = 0 its scale is 0 also where gs is not finite
      const float ge = r0 + 32 * rb < rows && c0 + col < cols ? gs : 0.0f;
      if (nv) col_block<true>(xs, rb, col, ge, factors, out, atom_c);
      else    col_block<false>(xs, rb, col, gs, factors, out, atom_c);
      uint8_t* s = stage + col * 64 + ((rb ^ (lane & 3)) << 4);      // (col >> 1) & 3 = lane & 3, also for col + 1
      *reinterpret_cast<uint4*>(s) = out[0];
      *reinterpret_cast<uint4*>(s + 64) = out[1];
      fence_proxy_async_smem();                                      // visible to the TMA store
    }
    if (T.q_row || T.amax_bits) {
      const int b = lane >> 3;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 64 * u + 8 * warp + (lane & 7);
        uint4 out;
        const bool in = r0 + row < rows && c0 + 32 * b < cols;  // cols is a multiple of 32
        const uint32_t m = nv ? row_block<true>(xs, row, b, in ? gs : 0.0f, factors, out, atom_r)
                              : row_block<false>(xs, row, b, gs, factors, out, atom_r);
        top = max(top, m);
        if (T.q_row && in)
          *reinterpret_cast<uint4*>(T.q_row + static_cast<int64_t>(r0 + row) * (cols >> 1) + ((c0 + 32 * b) >> 1)) = out;
      }
    }
    __syncthreads();                          // input tile consumed; the atoms complete
    if (tid == 0) {                           // refill the buffer just consumed
      if (T.q_col) {                          // clipped at the matrix edges
        tma_store_2d(&T.qc_map, smem_u32(stage), r0 >> 1, c0);
        bulk_commit_group();
      }
      if (T.scale_inv && rt == 0 && ct == 0) *T.scale_inv = __fdiv_rn(1.0f, gs);
      const int next = tile + 2 * stride;
      if (next < g.total_tiles) {
        issue_cast_tile(g, next, smem_u32(xbuf + buf * kXBytes), smem_u32(&full[buf]), where[buf]);
        pending |= 1u << buf;
        pending_ph = (pending_ph & ~(1u << buf)) | (static_cast<uint32_t>(((i + 2) >> 1) & 1) << buf);
      }
    }
    // a tile's atoms: one (MXFP4) or two (NVFP4); the last tile along K also writes the zero atoms that
    // pad K to a multiple of 256
    const int per = nv ? 2 : 1;
    if (T.q_row && tid < 128) {
      const int words = atom_words(cols, per);
      uint4* dst = reinterpret_cast<uint4*>(T.sf_row + (static_cast<int64_t>(rt) * words + ct * per) * 512);
      if (tid < 32 * per) dst[tid] = reinterpret_cast<const uint4*>(atom_r)[tid];
      else if (ct == T.tiles_c - 1 && ct * per + tid / 32 < words) dst[tid] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (T.q_col && tid >= 128) {
      const int t = tid - 128;
      const int words = atom_words(rows, per);
      uint4* dst = reinterpret_cast<uint4*>(T.sf_col + (static_cast<int64_t>(ct) * words + rt * per) * 512);
      if (t < 32 * per) dst[t] = reinterpret_cast<const uint4*>(atom_c)[t];
      else if (rows - r0 <= kTile && rt * per + t / 32 < words) dst[t] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (cur >= 0 && g.t[cur].amax_bits) blk::cta_amax(g.t[cur].amax_bits, top << 16, tops);
  if (tid == 0) {
    // loads still in flight after an abort must land before shared memory is released
    for (int b = 0; b < 2; ++b)
      if (pending & (1u << b)) mbar_wait(smem_u32(&full[b]), (pending_ph >> b) & 1u, kDrainLimitNs);
    bulk_wait_group<0>();                     // stores complete before the CTA exits
  }
}

// Row-wise copies alone: blocks of 32 values numbered through the matrix, a thread each.
template <bool NV>
__device__ __forceinline__ void cast_rows(const CastTensor& T, float* factors, uint32_t* tops) {
  constexpr int kN = NV ? 2 : 1, kV = 4 / kN;              // scales per 32 values, and vectors of 8 per scale
  const uint32_t per_row = static_cast<uint32_t>(T.cols) >> 5;
  const int words = atom_words(T.cols, kN);
  const int64_t n = static_cast<int64_t>(T.rows) * per_row, stride = static_cast<int64_t>(gridDim.x) * kCastThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kCastThreads + threadIdx.x;
  const float g = NV ? ld_dep(T.scale) : 1.0f;
  if (NV) {
    __syncthreads();                                       // the previous tensor's factors are read
    fill_factors(factors, g);
    __syncthreads();
  }
  const uint8_t* x = static_cast<const uint8_t*>(T.x);
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 31) == 0;   // 16-byte alignment is all a caller owes
  uint8_t* sf = T.sf_row;
  uint32_t top = 0;
  // (row, block) of this thread, and what a stride adds to them
  uint32_t row = static_cast<uint32_t>(first / per_row), b = static_cast<uint32_t>(first - static_cast<int64_t>(row) * per_row);
  const uint32_t drow = static_cast<uint32_t>(stride / per_row), db = static_cast<uint32_t>(stride - static_cast<int64_t>(drow) * per_row);
#pragma unroll 2
  for (int64_t i = first; i < n; i += stride) {
    uint4 w[4];
    if (wide) {
      ld_stream_32(x + i * 64, w[0], w[1]);
      ld_stream_32(x + i * 64 + 32, w[2], w[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = ld_stream_u4(x + i * 64 + 16 * k);
    }
    uint32_t code[4], scales = 0;
#pragma unroll
    for (int s = 0; s < kN; ++s) {
      uint32_t m2 = 0;
#pragma unroll
      for (int k = 0; k < kV; ++k) m2 = max_abs2(m2, max_abs8(w[s * kV + k]));
      const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
      top = max(top, m);
      float f;
      scales |= static_cast<uint32_t>(block_scale<NV>(m, g, factors, f)) << (8 * s);
#pragma unroll
      for (int k = 0; k < kV; ++k) code[s * kV + k] = code8(w[s * kV + k], f);
    }
    *reinterpret_cast<uint4*>(T.q_row + i * 16) = make_uint4(code[0], code[1], code[2], code[3]);
    // byte kN * b of the row's atom words
    uint8_t* at = sf + blk::atom_word(row, (kN * b) >> 2, words) + ((kN * b) & 3);
    if (NV) *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(scales);
    else    *at = static_cast<uint8_t>(scales);
    row += drow;
    b += db;
    if (b >= per_row) {
      b -= per_row;
      ++row;
    }
  }
  if (NV) {
    // one atomic per CTA, by its last warp (no barrier: one here made the loop above spill, 0.15 us of 2.2)
    if (T.amax_bits) {
      top = __reduce_max_sync(0xffffffffu, top);
      if ((threadIdx.x & 31) == 0) {
        atomicMax(&tops[0], top);
        __threadfence_block();
        if (atomicAdd(&tops[1], 1u) == kCastThreads / 32 - 1) {
          __threadfence_block();
          top = atomicExch(&tops[0], 0u);
          tops[1] = 0;
          if (top) atomicMax(T.amax_bits, top > 0x7F80u ? 0x7FC00000u : top << 16);
        }
      }
    }
    if (T.scale_inv && first == 0) *T.scale_inv = __fdiv_rn(1.0f, g);
  }
  // zero scales: K's padding of each row, and the rows that fill up the last atoms
  const int pad = words * 4 - kN * static_cast<int>(per_row);
#pragma unroll 1
  for (int64_t i = first; i < static_cast<int64_t>(T.rows) * pad; i += stride) {
    const int64_t r = i / pad;
    const int j = kN * static_cast<int>(per_row) + static_cast<int>(i - r * pad);
    sf[blk::atom_word(r, j >> 2, words) + (j & 3)] = 0;
  }
  const uint32_t fill = (128u - (static_cast<uint32_t>(T.rows) & 127u)) & 127u;
#pragma unroll 1
  for (int64_t i = first; i < static_cast<int64_t>(fill) * words; i += stride)
    *reinterpret_cast<uint32_t*>(sf + blk::atom_word(T.rows + i / words, i % words, words)) = 0u;
}

__global__ void __launch_bounds__(kCastThreads, 4) k_fp4_cast_rows(const __grid_constant__ CastGroup g) {
  __shared__ float factors[128];
  __shared__ uint32_t tops[2];               // NVFP4: the CTA's largest magnitude, and how many warps have added theirs
  if (threadIdx.x < 2) tops[threadIdx.x] = 0;
  pdl_trigger();
  pdl_wait();
  for (int t = 0; t < g.n; ++t) {
    if (g.t[t].kind == blk::kNVFP4) cast_rows<true>(g.t[t], factors, tops);
    else                            cast_rows<false>(g.t[t], factors, tops);
  }
}

}  // namespace fp4
}  // namespace fp8t
