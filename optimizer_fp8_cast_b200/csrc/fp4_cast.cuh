// fp4_cast.cuh — BF16 -> 4-bit block-scaled quantisation (MXFP4, NVFP4), row-wise and column-wise.
//
// The arithmetic is in quant_block.cuh. The 4-bit tensor-core instruction reads both operands K-major
// only, so the column-wise copy (blocks down a column) is written transposed: its row c holds the codes
// of x's column c. Codes are two to a byte, the first in the low nibble; scales in 512-byte atoms, K
// padded to a multiple of 256 with zero scales (zero codes under them come from the GEMM's TMA fill).
//
// Each 128 x 128 tile of x arrives as two TMA boxes of 128 rows x 64 columns (128-byte swizzle) in a
// double buffer; rows and columns past the matrix read as zeros, which quantise to zero codes and the
// scales of an all-zero block, so the atoms of a ragged edge are complete.
//   warps 0-3: column-wise blocks. A thread takes two adjacent columns of 32 rows (one 4-byte shared
//     load per row, a warp covers the 64 columns of a box row: no bank conflicts) and stores 16 bytes of
//     codes to each of the two transposed rows.
//   warps 4-7: row-wise blocks, a quarter-warp per block of 8 consecutive rows, 16 bytes per block.
// Bound: HBM, 2 B read + 0.5 B per copy written (+ 1/32 B MXFP4, 1/16 B NVFP4 of scales) per element.
#pragma once

#include "ptx.cuh"
#include "quant_block.cuh"

namespace fp8t {
namespace fp4 {

constexpr int kTile = 128;
constexpr int kCastThreads = 256;
constexpr int kCastTensors = 8;
constexpr int kHalfBytes = kTile * 64 * 2;                 // one 128-row x 64-column BF16 box
constexpr int kXBytes = 2 * kHalfBytes;
constexpr int kAtomBytes = 2 * 512;                        // atoms of a tile and orientation (NVFP4: 2)
constexpr int kCastSmemBytes = 2 * kXBytes + 2 * kAtomBytes + 64 + 1024 /*alignment*/;

struct alignas(64) CastTensor {
  CUtensorMap x_map;               // BF16 [rows][cols], 64 x 128 boxes, 128-byte swizzle
  uint8_t* q_row;                  // [rows][cols / 2] (may be null)
  uint8_t* sf_row;                 // atoms [rows / 128][K = cols]
  uint8_t* q_col;                  // [cols][rows / 2] (may be null)
  uint8_t* sf_col;                 // atoms [cols / 128][K = rows]
  const float* scale;              // NVFP4
  unsigned int* amax_bits;         // NVFP4, may be null
  float* scale_inv;                // NVFP4, may be null
  int64_t rows, cols, tiles_c, tile_start;
  int32_t kind;
};

struct alignas(64) CastGroup {
  CastTensor t[kCastTensors];
  int32_t n;
  int64_t total_tiles;
};

// Byte offset of BF16 element (row, col) in a tile as the two swizzled TMA boxes lay it out.
__device__ __forceinline__ uint32_t xoff(int row, int col) {
  return (col >> 6) * kHalfBytes + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
}

__device__ __forceinline__ int cast_tensor_of(const CastGroup& g, int64_t tile) {
  int ti = 0;
  while (ti + 1 < g.n && g.t[ti + 1].tile_start <= tile) ++ti;
  return ti;
}

__device__ __forceinline__ void issue_cast_tile(const CastGroup& g, int64_t tile, uint32_t dst, uint32_t bar) {
  const CastTensor& T = g.t[cast_tensor_of(g, tile)];
  const int64_t local = tile - T.tile_start;
  const int32_t r0 = static_cast<int32_t>((local / T.tiles_c) * kTile);
  const int32_t c0 = static_cast<int32_t>((local % T.tiles_c) * kTile);
  mbar_arrive_expect_tx(bar, kXBytes);               // out-of-range parts are zero-filled
  tma_load_2d(dst, &T.x_map, c0, r0, bar);
  tma_load_2d(dst + kHalfBytes, &T.x_map, c0 + 64, r0, bar);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Scale byte and factor of a block whose largest BF16 magnitude pattern is m.
template <bool NV>
__device__ __forceinline__ uint8_t block_scale(uint32_t m, float g, float& f) {
  return NV ? blk::nvfp4_scale(m << 16, g, f) : blk::e8m0_scale(m << 16, 2, f);
}

// Position of scale j (0..7) of row r in a tile's one or two atoms.
__device__ __forceinline__ uint32_t atom_off(int r, int j) {
  return (j >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (j & 3);
}

// Two adjacent columns x 32 rows: 16 bytes of codes each, and their scales.
template <bool NV>
__device__ __forceinline__ void col_block(const uint8_t* xs, int rb, int col, float g, uint4 (&out)[2],
                                          uint8_t* atom) {
  constexpr int kB = NV ? 16 : 32, kN = 32 / kB;
  uint32_t w[32];
#pragma unroll
  for (int r = 0; r < 32; ++r) w[r] = *reinterpret_cast<const uint32_t*>(xs + xoff(32 * rb + r, col));
  uint32_t code[2][4];
#pragma unroll
  for (int b = 0; b < kN; ++b) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < kB; ++r) m = __vmaxu2(m, w[b * kB + r] & 0x7FFF7FFFu);
    float f0, f1;
    atom[atom_off(col, kN * rb + b)] = block_scale<NV>(m & 0xFFFFu, g, f0);
    atom[atom_off(col + 1, kN * rb + b)] = block_scale<NV>(m >> 16, g, f1);
#pragma unroll
    for (int o = 0; o < kB / 8; ++o) {
      float lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t v = w[b * kB + o * 8 + j];
        lo[j] = __fmul_rn(bf16_lo(v), f0);
        hi[j] = __fmul_rn(bf16_hi(v), f1);
      }
      code[0][b * (kB / 8) + o] = blk::cvt_e2m1x8(lo);
      code[1][b * (kB / 8) + o] = blk::cvt_e2m1x8(hi);
    }
  }
  out[0] = make_uint4(code[0][0], code[0][1], code[0][2], code[0][3]);
  out[1] = make_uint4(code[1][0], code[1][1], code[1][2], code[1][3]);
}

// 32 consecutive values of a row: 16 bytes of codes, their scales; returns the largest magnitude pattern.
template <bool NV>
__device__ __forceinline__ uint32_t row_block(const uint8_t* xs, int row, int b32, float g, uint4& out,
                                              uint8_t* atom) {
  constexpr int kB = NV ? 16 : 32, kN = 32 / kB;
  uint4 w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const uint4*>(xs + xoff(row, 32 * b32 + 8 * k));
  uint32_t code[4], top = 0;
#pragma unroll
  for (int b = 0; b < kN; ++b) {
    uint32_t m2 = 0;
#pragma unroll
    for (int k = 0; k < kB / 8; ++k) {
      const uint4& v = w[b * (kB / 8) + k];
      m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
    }
    const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    top = max(top, m);
    float f;
    atom[atom_off(row, kN * b32 + b)] = block_scale<NV>(m, g, f);
#pragma unroll
    for (int k = 0; k < kB / 8; ++k) {
      const uint4& v = w[b * (kB / 8) + k];
      float a[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                    bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = __fmul_rn(a[j], f);
      code[b * (kB / 8) + k] = blk::cvt_e2m1x8(a);
    }
  }
  out = make_uint4(code[0], code[1], code[2], code[3]);
  return top;
}

__global__ void __launch_bounds__(kCastThreads, 2) k_fp4_cast(const __grid_constant__ CastGroup g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* xbuf = smem;                                             // [2][2 boxes][128][128 B]
  uint8_t* atom_r = smem + 2 * kXBytes;
  uint8_t* atom_c = atom_r + kAtomBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(atom_c + kAtomBytes);
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t stride = gridDim.x;
  uint32_t pending = 0, pending_ph = 0;      // thread 0: loads not yet consumed, their phases

  if (tid == 0) {
    mbar_init(smem_u32(&full[0]), 1);
    mbar_init(smem_u32(&full[1]), 1);
    fence_mbar_init();
    s_abort = 0;
    for (int b = 0; b < 2; ++b) {
      const int64_t tile = blockIdx.x + b * stride;
      if (tile < g.total_tiles) {
        issue_cast_tile(g, tile, smem_u32(xbuf + b * kXBytes), smem_u32(&full[b]));
        pending |= 1u << b;
      }
    }
  }
  __syncthreads();
  const uint64_t limit = wait_limit_ns();
  const bool expire = expire_mode() == kExpireAll;

  for (int64_t i = 0;; ++i) {
    const int64_t tile = blockIdx.x + i * stride;
    if (tile >= g.total_tiles) break;
    const int buf = static_cast<int>(i & 1);
    if (tid == 0) {
      if (!mbar_wait(smem_u32(&full[buf]), static_cast<uint32_t>((i >> 1) & 1), limit, expire)) {
        record_error(kErrTimeout);
        s_abort = 1;
      } else {
        pending &= ~(1u << buf);
      }
    }
    __syncthreads();                          // tile landed; the previous tile's atoms written
    if (s_abort) break;
    const CastTensor& T = g.t[cast_tensor_of(g, tile)];
    const int64_t local = tile - T.tile_start;
    const int64_t rt = local / T.tiles_c, ct = local % T.tiles_c;
    const int64_t r0 = rt * kTile, c0 = ct * kTile;
    const uint8_t* xs = xbuf + buf * kXBytes;
    const bool nv = T.kind == blk::kNVFP4;
    const float gs = nv ? __ldg(T.scale) : 1.0f;

    if (warp < 4) {
      // column-wise: warp w takes rows 32w .. 32w+31, columns 2 * lane (+1) of each box
      if (T.q_col) {
#pragma unroll 1
        for (int box = 0; box < 2; ++box) {
          const int col = 64 * box + 2 * lane;
          uint4 out[2];
          if (nv) col_block<true>(xs, warp, col, gs, out, atom_c);
          else    col_block<false>(xs, warp, col, gs, out, atom_c);
          if (r0 + 32 * warp < T.rows) {      // rows is a multiple of 32: whole blocks
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (c0 + col + c < T.cols)
                *reinterpret_cast<uint4*>(T.q_col + (c0 + col + c) * (T.rows / 2) + (r0 + 32 * warp) / 2) = out[c];
          }
        }
      }
    } else {
      const int wr = warp - 4, b = lane >> 3;
      uint32_t top = 0;
      if (T.q_row || T.amax_bits) {
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          const int row = 32 * u + 8 * wr + (lane & 7);
          uint4 out;
          const uint32_t m = nv ? row_block<true>(xs, row, b, gs, out, atom_r)
                                : row_block<false>(xs, row, b, gs, out, atom_r);
          top = max(top, m);
          if (T.q_row && r0 + row < T.rows && c0 + 32 * b < T.cols)   // cols is a multiple of 32
            *reinterpret_cast<uint4*>(T.q_row + (r0 + row) * (T.cols / 2) + (c0 + 32 * b) / 2) = out;
        }
        if (T.amax_bits) {
          top = __reduce_max_sync(0xffffffffu, top);
          if (top > 0x7F80u) top = 0x7FC0u;   // canonical NaN
          if (lane == 0 && top) atomicMax(T.amax_bits, top << 16);
        }
      }
    }
    __syncthreads();                          // input tile consumed; the atoms complete
    if (tid == 0) {                           // refill the buffer just consumed
      if (T.scale_inv && local == 0) *T.scale_inv = __fdiv_rn(1.0f, gs);
      const int64_t next = tile + 2 * stride;
      if (next < g.total_tiles) {
        issue_cast_tile(g, next, smem_u32(xbuf + buf * kXBytes), smem_u32(&full[buf]));
        pending |= 1u << buf;
        pending_ph = (pending_ph & ~(1u << buf)) | (static_cast<uint32_t>(((i + 2) >> 1) & 1) << buf);
      }
    }
    // a tile's atoms: one (MXFP4) or two (NVFP4); the last tile along K also writes the zero atoms that
    // pad K to a multiple of 256
    const int per = nv ? 2 : 1;
    if (T.q_row && tid < 128) {
      const int64_t words = blk::atoms_per_row(T.cols, T.kind);
      uint4* dst = reinterpret_cast<uint4*>(T.sf_row + (rt * words + ct * per) * 512);
      if (tid < 32 * per) dst[tid] = reinterpret_cast<const uint4*>(atom_r)[tid];
      else if (ct == T.tiles_c - 1 && ct * per + tid / 32 < words) dst[tid] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (T.q_col && tid >= 128) {
      const int t = tid - 128;
      const int64_t words = blk::atoms_per_row(T.rows, T.kind);
      uint4* dst = reinterpret_cast<uint4*>(T.sf_col + (ct * words + rt * per) * 512);
      if (t < 32 * per) dst[t] = reinterpret_cast<const uint4*>(atom_c)[t];
      else if (r0 + kTile >= T.rows && rt * per + t / 32 < words) dst[t] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (tid == 0) {
    // loads still in flight after an abort must land before shared memory is released
    for (int b = 0; b < 2; ++b)
      if (pending & (1u << b)) mbar_wait(smem_u32(&full[b]), (pending_ph >> b) & 1u, kDrainLimitNs);
  }
}

}  // namespace fp4
}  // namespace fp8t
