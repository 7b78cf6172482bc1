// gemm_fp4.cuh — block-scaled GEMM of 4-bit operands (MXFP4, NVFP4) on the 5th-generation tensor cores.
//
//   D[M x N] = bf16((sum_k a_ik sa_i(k) b_jk sb_j(k)) * a_scale_inv * b_scale_inv)
//
// tcgen05.mma kind::mxf4 (E8M0 scale per 32 values) and kind::mxf4nvf4 (E4M3 scale per 16), FP32
// accumulation, K = 64 values (32 bytes) per MMA: the operand bytes, shared-memory layout and cycles
// of an 8-bit MMA of K = 32, at twice its values. Both operands are K-major (the 4-bit kinds read no
// other order), two values per byte.
//
// Large problems (k_fp4_gemm): the 256 x 384 pair tile of the MXFP8 kernel, for the same reason (operand
// bytes per MMA cycle, and TMEM room for the scales). A k-block is 256 values (128 bytes per row). Per
// k-block every 128 rows of A or B bring 2 (MXFP4) or 4 (NVFP4) scale atoms, stored next to each other
// ([MN / 128][K / 256]), which arrive as one TMA box of 1 or 2 KB and are copied to 16 TMEM columns per
// atom step along K: A 4, B 12. Rows of a ragged edge read zero codes (TMA fill), so M and N need not
// be multiples of the tile; K's padding has zero codes and zero scales.
// TMEM: accumulator 0..383, scales from 384 (32 or 64 columns).
// Warp roles, barriers, bounded waits and the register-held epilogue are those of the MXFP8 kernel.
#pragma once

#include "gemm_mx_wide.cuh"

namespace fp8t {
namespace gemm {

constexpr int kStages4 = 4;
constexpr uint32_t kSfCol4 = 384;
template <bool NV>
constexpr int kStageBytes4 = kABytes + kB0BytesX + kB1BytesX + 4 * (NV ? 4 : 2) * 512;
constexpr int kEpiBytes4 = kEpiWarpsX * 2 * kEpiChunkBytes;
template <bool NV>
constexpr int kSmemBytes4 = kStages4 * kStageBytes4<NV> + kEpiBytes4 + 1024 + 256;
static_assert(kStageBytes4<false> % 1024 == 0 && kStageBytes4<true> % 1024 == 0, "stages stay 1024-byte aligned");
static_assert(kSmemBytes4<true> <= 232448, "shared memory of an SM");
static_assert(kSfCol4 + 64 <= static_cast<uint32_t>(kTmemCols), "TMEM columns");

// Block-scaled instruction descriptor of the 4-bit kinds: E2M1 operands, K-major, scale type (bit 23:
// 1 E8M0, 0 E4M3), scale-factor ids of A and B.
template <bool NV>
__device__ __forceinline__ uint32_t make_idesc_fp4(int m, int n, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (NV ? 0u : 1u << 23) |
         (static_cast<uint32_t>(m >> 4) << 24) | (sf_id << 29);
}

template <bool NV>
__device__ __forceinline__ void tc_mma_fp4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                                uint32_t accumulate) {
  if constexpr (NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

template <bool NV>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsX, 1)
    k_fp4_gemm(const __grid_constant__ Group g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  // stage s: [A 128 x 128 B][B0 128 x 128 B][B1 64 x 128 B][scale atoms of A, B 0..127, 128..255, 256..383]
  constexpr int kAtoms = NV ? 4 : 2, kSf = kAtoms * 512, kSfRows = NV ? 2 : 1;
  uint8_t* sStage = smem;
  uint8_t* sEpi = smem + kStages4 * kStageBytes4<NV>;
  SmemX* S = reinterpret_cast<SmemX*>(sEpi + kEpiBytes4);
  volatile int* abort_flag = &S->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int my_tiles = tiles_of(g, cluster, n_clusters);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages4; ++s) {
      mbar_init(smem_u32(&S->full[s]), 1);
      mbar_init(smem_u32(&S->empty[s]), 1);
    }
    mbar_init(smem_u32(&S->acc_full), 1);
    mbar_init(smem_u32(&S->acc_empty), 2 * kEpiWarpsX);
    mbar_init(smem_u32(&S->mma_done), 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int p = 0; p < g.n && p < 8; ++p) {
      tma_prefetch_desc(&g.p[p].a);
      tma_prefetch_desc(&g.p[p].b);
      tma_prefetch_desc(&g.p[p].b64);
      tma_prefetch_desc(&g.p[p].d);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&S->tmem_base), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  const uint64_t limit = wait_limit_ns();
  const int expire = expire_mode();
  const bool expire_main = expire == kExpireAll;
  const bool expire_epi = expire == kExpireAll || expire == kExpireGemmEpilogue;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs)
      uint32_t it = 0, issued = 0;
      for (int i = 0; i < my_tiles && !*abort_flag; ++i) {
        const int tile = tile_at(g, cluster, n_clusters, i);
        const Problem& P = g.p[find_problem(g, tile)];
        int mt, nt;
        bool has1;
        mxw_tile(P, tile - P.tile_start, mt, nt, has1);
        const int m0 = mt * kBM + static_cast<int>(rank) * kHalf;
        const int nb0 = nt * kBNx + static_cast<int>(rank) * kHalf;           // MMA 0 rows
        const int nb1 = nt * kBNx + 256 + static_cast<int>(rank) * (kHalf / 2); // MMA 1 rows
        const int ra = 2 * mt + static_cast<int>(rank), rb = 3 * nt;          // atom rows
        const int num_kb = P.kb128;                                           // k-blocks of 256 values
        const uint32_t tx = 2u * (kABytes + kB0BytesX + 3 * kSf + (has1 ? kB1BytesX + kSf : 0));
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const uint32_t s = it % kStages4, ph = (it / kStages4) & 1;
          if (*abort_flag) break;
          if (!mbar_wait(smem_u32(&S->empty[s]), ph ^ 1, limit, expire_main)) {
            *abort_flag = 1;
            record_error(kErrTimeout);
            break;
          }
          const uint32_t full_leader = mapa_shared(smem_u32(&S->full[s]), 0);
          if (leader) mbar_arrive_expect_tx(smem_u32(&S->full[s]), tx);
          const uint32_t base = smem_u32(sStage + s * kStageBytes4<NV>);
          const uint32_t a_dst = base, b0_dst = base + kABytes, b1_dst = b0_dst + kB0BytesX;
          const uint32_t sf_dst = b1_dst + kB1BytesX;
          tma_load_2d_pair(a_dst, &P.a, kb * kBK, m0, full_leader);
          tma_load_2d_pair(b0_dst, &P.b, kb * kBK, nb0, full_leader);
          tma_load_2d_pair(sf_dst, &P.sfa, 0, (ra * num_kb + kb) * kSfRows, full_leader);
          tma_load_2d_pair(sf_dst + kSf, &P.sfb, 0, (rb * num_kb + kb) * kSfRows, full_leader);
          tma_load_2d_pair(sf_dst + 2 * kSf, &P.sfb, 0, ((rb + 1) * num_kb + kb) * kSfRows, full_leader);
          if (has1) {
            tma_load_2d_pair(b1_dst, &P.b64, kb * kBK, nb1, full_leader);
            tma_load_2d_pair(sf_dst + 3 * kSf, &P.sfb, 0, ((rb + 2) * num_kb + kb) * kSfRows, full_leader);
          }
          ++issued;
        }
      }
      if (leader) {
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t i = issued > kStages4 ? issued - kStages4 : 0; i < issued; ++i) {
          const uint64_t spent = globaltimer_ns() - t0;
          if (spent >= kPairDrainNs) break;
          mbar_wait(smem_u32(&S->full[i % kStages4]), (i / kStages4) & 1, kPairDrainNs - spent);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------- MMA issuer (even CTA): per k-step an N = 256 and an N = 128 MMA
      uint32_t it = 0, local = 0;
      for (int i = 0; i < my_tiles && !*abort_flag; ++i, ++local) {
        const int tile = tile_at(g, cluster, n_clusters, i);
        const Problem& P = g.p[find_problem(g, tile)];
        int mt, nt;
        bool has1;
        mxw_tile(P, tile - P.tile_start, mt, nt, has1);
        const int num_kb = P.kb128;
        if (!mbar_wait(smem_u32(&S->acc_empty), (local & 1) ^ 1, limit, expire_main)) {
          *abort_flag = 1;
          record_error(kErrTimeout);
          break;
        }
        tc_fence_after();
        bool ok = true;
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const uint32_t s = it % kStages4, ph = (it / kStages4) & 1;
          if (*abort_flag || !mbar_wait(smem_u32(&S->full[s]), ph, limit, expire_main)) {
            if (!*abort_flag) record_error(kErrTimeout);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t base = smem_u32(sStage + s * kStageBytes4<NV>);
          const uint32_t a_base = base, b0_base = base + kABytes, b1_base = b0_base + kB0BytesX;
          const uint32_t sf = b1_base + kB1BytesX;
#pragma unroll
          for (int a = 0; a < kAtoms; ++a) {     // 16 scale columns per atom along K: A, B 0, B 1, B 2
            const uint32_t sc = tmem + kSfCol4 + a * 16, at = sf + a * 512;
            tc_cp_32x128b_warpx4_pair(sc, make_sf_desc(at));
            tc_cp_32x128b_warpx4_pair(sc + 4, make_sf_desc(at + kSf));
            tc_cp_32x128b_warpx4_pair(sc + 8, make_sf_desc(at + 2 * kSf));
            if (has1) tc_cp_32x128b_warpx4_pair(sc + 12, make_sf_desc(at + 3 * kSf));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // MXFP4: two scales per 64 values, so an atom serves two MMAs (scale ids 0 and 2); NVFP4: one
            const uint32_t sc = tmem + kSfCol4 + (NV ? k : k >> 1) * 16, id = NV ? 0 : (k & 1) * 2;
            const uint64_t adesc = make_sw128_desc(a_base + k * kUmmaK);
            const uint32_t acc = (kb | k) != 0 ? 1u : 0u;
            tc_mma_fp4_pair<NV>(tmem, adesc, make_sw128_desc(b0_base + k * kUmmaK),
                                make_idesc_fp4<NV>(kBM, 256, id), sc | id << 30, (sc + 4) | id << 30, acc);
            if (has1)
              tc_mma_fp4_pair<NV>(tmem + 256, adesc, make_sw128_desc(b1_base + k * kUmmaK),
                                  make_idesc_fp4<NV>(kBM, 128, id), sc | id << 30, (sc + 12) | id << 30, acc);
          }
          tc_commit_pair_mc(smem_u32(&S->empty[s]), 0x3);
        }
        if (!ok) break;
        tc_commit_pair_mc(smem_u32(&S->acc_full), 0x3);
      }
      tc_commit_pair(smem_u32(&S->mma_done));
      mbar_wait(smem_u32(&S->mma_done), 0, kDrainLimitNs);
    }
  } else {
    // ---------------- epilogue warps 2..9 (both CTAs): TMEM lane quarter warp % 4, column half
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* my_buf = sEpi + (warp - 2) * 2 * kEpiChunkBytes;
    uint32_t local = 0, chunk_count = 0;
    for (int i = 0; i < my_tiles; ++i, ++local) {
      const int tile = tile_at(g, cluster, n_clusters, i);
      if (*abort_flag) break;
      if (!mbar_wait(smem_u32(&S->acc_full), local & 1, limit, expire_epi)) {
        *abort_flag = 1;
        record_error(kErrTimeout);
        break;
      }
      tc_fence_after();
      const Problem& P = g.p[find_problem(g, tile)];
      const float alpha = P.sa ? __fmul_rn(__ldg(P.sa), P.sb ? __ldg(P.sb) : 1.0f) : (P.sb ? __ldg(P.sb) : 1.0f);
      const int M = P.M, N = P.N, local_tile = tile - P.tile_start;
      const int row0 = (local_tile / P.tiles_n) * kBM + static_cast<int>(rank) * kHalf + quad * 32;
      const int n0 = (local_tile % P.tiles_n) * kBNx + half * kAccColsX;
      const uint32_t t_base = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * kAccColsX;
      uint32_t w[kAccColsX / 32][16];
#pragma unroll
      for (int c = 0; c < kAccColsX / 32; ++c) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_base + c * 32, r);
        tmem_ld_wait();
        tmem_reg_fence(r);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          w[c][j] = pack_bf16x2(__fmul_rn(__uint_as_float(r[2 * j]), alpha), __fmul_rn(__uint_as_float(r[2 * j + 1]), alpha));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&S->acc_empty), 0));
#pragma unroll
      for (int c = 0; c < kAccColsX / 32; ++c) {
        if (n0 + c * 32 >= N || row0 >= M) continue;       // chunk entirely outside the matrix
        uint8_t* buf = my_buf + (chunk_count & 1) * kEpiChunkBytes;
        ++chunk_count;
        if (lane == 0) bulk_wait_group_read<1>();
        __syncwarp();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int pp = p ^ ((lane >> 1) & 3);
          *reinterpret_cast<uint4*>(buf + lane * 64 + pp * 16) =
              make_uint4(w[c][4 * p], w[c][4 * p + 1], w[c][4 * p + 2], w[c][4 * p + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&P.d, smem_u32(buf), n0 + c * 32, row0);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kSettleNs) {
    }
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

}  // namespace gemm
}  // namespace fp8t
