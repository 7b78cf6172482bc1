// gemm_fp4.cuh — block-scaled GEMM of 4-bit operands (MXFP4, NVFP4) on the 5th-generation tensor cores.
//
//   D[M x N] = bf16((sum_k a_ik sa_i(k) b_jk sb_j(k)) * a_scale_inv * b_scale_inv)
//
// tcgen05.mma kind::mxf4 (E8M0 scale per 32 values) and kind::mxf4nvf4 (E4M3 scale per 16), FP32
// accumulation, K = 64 values (32 bytes) per MMA: the operand bytes, shared-memory layout and cycles
// of an 8-bit MMA of K = 32, at twice its values. Both operands are K-major (the 4-bit kinds read no
// other order), two values per byte. A k-block is 256 values (128 bytes per row, four MMAs).
//
// Large problems (k_fp4_gemm): a cluster of two CTAs computes a tile of 256 rows by 256 or 384 columns, each CTA
// holding 128 rows of A and 128 (192) of B. Per k-block every 128 rows of A or B bring 2 (MXFP4) or 4
// (NVFP4) scale atoms, stored next to each other ([MN / 128][K / 256]), which arrive as one TMA box of 1 or
// 2 KB; each CTA takes its own A rows' and all of the tile's B rows'. The MMA warp copies an atom step (A 4,
// B 8 or 12 TMEM columns) right before the MMAs that use it.
//
// What bounds it. An MMA (256 x 256 x 64) takes 128 cycles, a k-block of a 256-column tile 512; a scale copy
// takes the copy path 44-71 cycles but runs beside earlier MMAs, so MXFP4's copies are hidden (519 cycles
// per k-block measured with operands resident, 777 for 384 columns) and NVFP4's set the pace (717, 1139).
// Two things make that so:
//   - the issuing warp stays converged and one elected lane issues. Issued from a lane that left its warp, a
//     copy after an mbarrier wait did not overlap the MMAs before it: 1034 against 773 cycles for 8
//     copies and 8 MMAs per k-block;
//   - copies are spread between the MMAs in the order of use.
// Beyond that, L2 is the bound: 12 TB/s through it in a profile of 16384 x 11008 x 4096 (operands, their way from DRAM and
// D), of it 10 to 11 of operands that the SMs take in (35 KB per SM and k-block of a 256-column tile, 44 KB of a
// 384-column one with half as much work again).
//   256 columns: two accumulators let the epilogue of a tile run beside the next tile's MMAs. Two of 256 columns
//     and the scales (24 or 48) do not fit the 512 TMEM columns, so they overlap by kOv columns: accumulator 0
//     at 0..255, accumulator 1 at 256 - kOv, scales after it. The epilogue reads the shared columns first and
//     releases them through a barrier of their own.
//   384 columns (an N = 256 and an N = 128 MMA per step): one accumulator at 0..383, scales after it; the
//     epilogue pulls it into registers, releases it, then stores. The next tile's MMAs wait for that
//     (about 1.5 us), but the tile needs a sixth fewer operand bytes per MMA.
// 16384 x 11008 x 4096: 288 us (MXFP4) and 308 us (NVFP4) on 256 columns, 278 and 280 on 384; in a loop long
// enough to reach the power cap 402 against 370 us with the cast (NVFP4). 1000 x 4096 x 4096 has 64 tiles of
// 256 columns for 74 pairs, but 44 of 384, each half as long again: the host picks by rounds of tiles.
// Rows of a ragged edge read zero codes (TMA fill), so M and N need not be multiples of the tile; K's
// padding has zero codes and zero scales.
// Warp roles (320 threads): warp 0 TMA producer; warp 1 MMA issuer (even CTA), TMEM allocation; warps 2-9
// epilogue, a TMEM lane quarter and a 128-column half each. Waits are bounded as in the other kernels.
#pragma once

#include "gemm_tcgen05.cuh"

namespace fp8t {
namespace gemm {

constexpr int kBN4w = 384;                                        // the wide tile
template <bool WIDE>
constexpr int kStages4 = WIDE ? 4 : 5;
template <bool NV>
constexpr int kSfBytes4 = (NV ? 4 : 2) * 512;                     // scales of 128 rows x 256 values
constexpr int kB1Bytes4 = (kHalf / 2) * kBK;                      // wide: 64 more rows of B per CTA
template <bool NV, bool WIDE>
constexpr int kStageBytes4 = kABytes + kBBytes + 3 * kSfBytes4<NV> + (WIDE ? kB1Bytes4 + kSfBytes4<NV> : 0);
template <bool NV>
constexpr uint32_t kOv4 = NV ? 64 : 32;                           // columns the accumulators share
template <bool NV>
constexpr uint32_t kAcc1Col4 = 256 - kOv4<NV>;
template <bool NV, bool WIDE>
constexpr uint32_t kSfCol4 = WIDE ? kBN4w : 512 - kOv4<NV>;
constexpr int kEpiWarps4 = 8;
constexpr int kThreads4 = 64 + 32 * kEpiWarps4;
constexpr int kEpiBytes4 = kEpiWarps4 * 2 * kEpiChunkBytes;
template <bool NV, bool WIDE>
constexpr int kSmemBytes4 = kStages4<WIDE> * kStageBytes4<NV, WIDE> + kEpiBytes4 + 1024 + 256;
static_assert(kStageBytes4<false, false> % 1024 == 0 && kStageBytes4<true, false> % 1024 == 0 &&
              kStageBytes4<false, true> % 1024 == 0 && kStageBytes4<true, true> % 1024 == 0, "stages stay 1024-byte aligned");
static_assert(kSmemBytes4<true, false> <= 232448 && kSmemBytes4<true, true> <= 232448, "shared memory of an SM");
static_assert(kSfCol4<false, false> + 2 * 12 <= 512 && kSfCol4<true, false> + 4 * 12 <= 512 &&
              kSfCol4<true, true> + 4 * 16 <= 512, "TMEM columns");

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

// One GEMM of a grouped launch; tiles are numbered problem by problem.
struct alignas(64) Problem4 {
  CUtensorMap a, b, d;             // codes [M][K/2], [N][K/2] in 128-row boxes; D [M][N] in 32 x 32 ones
  CUtensorMap b64;                 // wide tiles: B in 64-row boxes
  CUtensorMap sfa, sfb;            // scales in rows of 256 words
  const float* sa;
  const float* sb;
  int32_t M, N, num_kb, tiles_n, tile_start;
};
// Up to NP problems; TABLE: with the host's tile list per cluster (as in the 8-bit GEMMs). A launch's
// parameters are copied at every launch: the table and 24 problems are 26 KB, and a call of one to four
// problems without a list takes 3 KB.
template <int NP, bool TABLE>
struct alignas(64) Group4 {
  static constexpr int kProblems = NP;
  Problem4 p[NP];
  int32_t n, total_tiles;
  __device__ __forceinline__ int tiles_of(int c, int clusters) const {
    return total_tiles > c ? (total_tiles - c + clusters - 1) / clusters : 0;
  }
  __device__ __forceinline__ int tile_at(int c, int clusters, int i) const { return c + i * clusters; }
  __device__ __forceinline__ const Problem4& problem(int tile) const {
    int k = 0;
    while (k + 1 < n && p[k + 1].tile_start <= tile) ++k;
    return p[k];
  }
};
template <int NP>
struct alignas(64) Group4<NP, true> : Group4<NP, false> {
  uint16_t start[kMaxClusters + 1];
  uint16_t order[kMaxSchedTiles];    // cluster c runs order[start[c] .. start[c + 1])
  __device__ __forceinline__ int tiles_of(int c, int) const { return start[c + 1] - start[c]; }
  __device__ __forceinline__ int tile_at(int c, int, int i) const { return order[start[c] + i]; }
};
using SmallGroup4 = Group4<4, false>;
using LargeGroup4 = Group4<kMaxProblems, false>;
using ListGroup4 = Group4<kMaxProblems, true>;

// One lane of a converged warp, the same on every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// A wait by a whole warp: every lane waits, and all agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit, bool expired = false) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit, expired));
}
__device__ __forceinline__ bool warp_aborted(const volatile int* flag) {
  return __any_sync(0xffffffffu, *flag != 0);
}

struct Smem4 {
  uint64_t full[5];             // even CTA: both CTAs' loads of a stage have landed
  uint64_t empty[5];            // both CTAs: the pair MMA has consumed a stage
  uint64_t acc_full[2];         // both CTAs: an accumulator holds a finished tile (wide: only the first)
  uint64_t acc_empty[2];        // even CTA: every epilogue warp of both CTAs has read an accumulator
  uint64_t acc_shared_free;     // even CTA: the warps that read the shared columns have
  uint64_t mma_done;            // even CTA: every issued MMA has completed
  uint32_t tmem_base;
  int abort;
};

// A packed 32 x 32 chunk (a row per lane) into the warp's swizzled staging buffer and out by TMA.
__device__ __forceinline__ void store_chunk4(const CUtensorMap* map, uint8_t* my_buf, uint32_t& chunk_count,
                                             const uint32_t (&w)[16], int lane, int n, int row0) {
  uint8_t* buf = my_buf + (chunk_count & 1) * kEpiChunkBytes;
  ++chunk_count;
  if (lane == 0) bulk_wait_group_read<1>();                // the store that last used buf has read it
  __syncwarp();
  // row `lane` of the chunk: four 16-byte pieces, 64-byte swizzle, matching the store's map
#pragma unroll
  for (int p = 0; p < 4; ++p)
    *reinterpret_cast<uint4*>(buf + lane * 64 + (p ^ ((lane >> 1) & 3)) * 16) =
        make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, smem_u32(buf), n, row0);
    bulk_commit_group();
  }
}
// 32 accumulator columns of this lane, scaled and packed as BF16.
__device__ __forceinline__ void pack_chunk4(const uint32_t (&r)[32], float alpha, uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j)
    w[j] = pack_bf16x2(__fmul_rn(__uint_as_float(r[2 * j]), alpha), __fmul_rn(__uint_as_float(r[2 * j + 1]), alpha));
}

template <bool NV, bool WIDE, class G>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads4, 1)
    k_fp4_gemm(const __grid_constant__ G g) {
  constexpr int kSf = kSfBytes4<NV>, kSfRows = NV ? 2 : 1;
  constexpr int kStages = kStages4<WIDE>, kStage = kStageBytes4<NV, WIDE>, kTileN = WIDE ? kBN4w : kBN;
  constexpr int kB = kBBytes + (WIDE ? kB1Bytes4 : 0), kStep = WIDE ? 16 : 12;   // B bytes; scale columns per step
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // stage s: [A 128 x 128 B][B 128 x 128 B][wide: B 64 x 128 B][scales of A | B rows 0.. | 128.. | 256..]
  uint8_t* sEpi = smem + kStages * kStage;
  Smem4* S = reinterpret_cast<Smem4*>(sEpi + kEpiBytes4);
  volatile int* abort_flag = &S->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int my_tiles = g.tiles_of(cluster, n_clusters);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&S->full[s]), 1);
      mbar_init(smem_u32(&S->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&S->acc_full[a]), 1);
      mbar_init(smem_u32(&S->acc_empty[a]), 2 * kEpiWarps4);
    }
    mbar_init(smem_u32(&S->acc_shared_free), kEpiWarps4);   // half of the warps of each CTA
    mbar_init(smem_u32(&S->mma_done), 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int p = 0; p < g.n && p < 8; ++p) {
      tma_prefetch_desc(&g.p[p].a);
      tma_prefetch_desc(&g.p[p].b);
      tma_prefetch_desc(&g.p[p].d);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&S->tmem_base), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();                 // barriers initialised and TMEM allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  const uint64_t limit = wait_limit_ns();
  const int expire = expire_mode();
  const bool expire_main = expire == kExpireAll;
  const bool expire_epi = expire == kExpireAll || expire == kExpireGemmEpilogue;
  pdl_trigger();
  pdl_wait();

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs)
    const bool one = elect_one();
    uint32_t it = 0, issued = 0;
    for (int i = 0; i < my_tiles && !warp_aborted(abort_flag); ++i) {
      const int tile = g.tile_at(cluster, n_clusters, i);
      const Problem4& P = g.problem(tile);
      const int local = tile - P.tile_start, mt = local / P.tiles_n, nt = local % P.tiles_n;
      const int m0 = mt * kBM + static_cast<int>(rank) * kHalf;
      const int n0 = nt * kTileN + static_cast<int>(rank) * kHalf;
      const int n1 = nt * kTileN + 256 + static_cast<int>(rank) * (kHalf / 2);
      const bool second = WIDE && nt * kTileN + 256 < P.N;                  // the N = 128 MMA has columns
      const uint32_t tx = 2u * (kStage - (WIDE && !second ? kB1Bytes4 + kSf : 0));
      const int ra = 2 * mt + static_cast<int>(rank), rb = (kTileN / 128) * nt;   // 128-row blocks of the scales
      const int num_kb = P.num_kb;                                           // k-blocks of 256 values
      for (int kb = 0; kb < num_kb; ++kb, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1;
        if (warp_aborted(abort_flag)) break;
        if (!warp_wait(smem_u32(&S->empty[s]), ph ^ 1, limit, expire_main)) {
          *abort_flag = 1;
          if (one) record_error(kErrTimeout);
          break;
        }
        if (one) {
          const uint32_t full_leader = mapa_shared(smem_u32(&S->full[s]), 0);
          if (leader) mbar_arrive_expect_tx(smem_u32(&S->full[s]), tx);
          const uint32_t a_dst = smem_u32(smem + s * kStage), b_dst = a_dst + kABytes;
          const uint32_t sf_dst = b_dst + kB;
          tma_load_2d_pair(a_dst, &P.a, kb * kBK, m0, full_leader);
          tma_load_2d_pair(b_dst, &P.b, kb * kBK, n0, full_leader);
          tma_load_2d_pair(sf_dst, &P.sfa, 0, (ra * num_kb + kb) * kSfRows, full_leader);
          tma_load_2d_pair(sf_dst + kSf, &P.sfb, 0, (rb * num_kb + kb) * kSfRows, full_leader);
          tma_load_2d_pair(sf_dst + 2 * kSf, &P.sfb, 0, ((rb + 1) * num_kb + kb) * kSfRows, full_leader);
          if (second) {
            tma_load_2d_pair(b_dst + kBBytes, &P.b64, kb * kBK, n1, full_leader);
            tma_load_2d_pair(sf_dst + 3 * kSf, &P.sfb, 0, ((rb + 2) * num_kb + kb) * kSfRows, full_leader);
          }
        }
        ++issued;
      }
    }
    // the even CTA can see its own stages land: wait for the last ones it armed (one shared budget; after
    // an abort a stage may miss the peer's bytes, and the settle delay below covers loads in flight)
    if (leader) {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
        const uint64_t spent = globaltimer_ns() - t0;
        if (spent >= kPairDrainNs) break;
        mbar_wait(smem_u32(&S->full[i % kStages]), (i / kStages) & 1, kPairDrainNs - spent);
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer (even CTA)
      const bool one = elect_one();
      uint32_t it = 0;
      for (int i = 0; i < my_tiles && !warp_aborted(abort_flag); ++i) {
        const int tile = g.tile_at(cluster, n_clusters, i);
        const Problem4& P = g.problem(tile);
        const int num_kb = P.num_kb;
        const bool second = WIDE && (tile - P.tile_start) % P.tiles_n * kTileN + 256 < P.N;
        const uint32_t acc = WIDE ? 0 : i & 1, aph = WIDE ? i & 1 : (i >> 1) & 1;
        // this accumulator read by the epilogue of two tiles ago (wide: of the last); the columns it shares with
        // the other one by the previous tile's
        if (!warp_wait(smem_u32(&S->acc_empty[acc]), aph ^ 1, limit, expire_main) ||
            (!WIDE && i > 0 && !warp_wait(smem_u32(&S->acc_shared_free), (i - 1) & 1, limit, expire_main))) {
          *abort_flag = 1;
          if (one) record_error(kErrTimeout);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + acc * kAcc1Col4<NV>;
        bool ok = true;
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1;
          if (!warp_wait(smem_u32(&S->full[s]), ph, limit, expire_main) || warp_aborted(abort_flag)) {
            if (one && !*abort_flag) record_error(kErrTimeout);
            *abort_flag = 1;
            ok = false;
            break;
          }
          if (one) {
            const uint32_t a_base = smem_u32(smem + s * kStage), b_base = a_base + kABytes;
            const uint32_t sf = b_base + kB;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // MXFP4: two scales per 64 values, so an atom step serves two MMAs (scale ids 0 and 2)
              const int a = NV ? k : k >> 1;
              const uint32_t sc = tmem + kSfCol4<NV, WIDE> + a * kStep, id = NV ? 0 : (k & 1) * 2;
              if (NV || (k & 1) == 0) {
                tc_cp_32x128b_warpx4_pair(sc, make_sf_desc(sf + a * 512));
                tc_cp_32x128b_warpx4_pair(sc + 4, make_sf_desc(sf + kSf + a * 512));
                tc_cp_32x128b_warpx4_pair(sc + 8, make_sf_desc(sf + 2 * kSf + a * 512));
                if (second) tc_cp_32x128b_warpx4_pair(sc + 12, make_sf_desc(sf + 3 * kSf + a * 512));
              }
              tc_mma_fp4_pair<NV>(d_tmem, make_sw128_desc(a_base + k * kUmmaK), make_sw128_desc(b_base + k * kUmmaK),
                                  make_idesc_fp4<NV>(kBM, kBN, id), sc | id << 30, (sc + 4) | id << 30,
                                  (kb | k) != 0 ? 1u : 0u);
              if (second)
                tc_mma_fp4_pair<NV>(d_tmem + 256, make_sw128_desc(a_base + k * kUmmaK),
                                    make_sw128_desc(b_base + kBBytes + k * kUmmaK), make_idesc_fp4<NV>(kBM, 128, id),
                                    sc | id << 30, (sc + 12) | id << 30, (kb | k) != 0 ? 1u : 0u);
            }
            tc_commit_pair_mc(smem_u32(&S->empty[s]), 0x3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (one) tc_commit_pair_mc(smem_u32(&S->acc_full[acc]), 0x3);
        __syncwarp();
      }
      // every MMA issued here must complete before either CTA frees TMEM or shared memory
      if (one) tc_commit_pair(smem_u32(&S->mma_done));
      __syncwarp();
      mbar_wait(smem_u32(&S->mma_done), 0, kDrainLimitNs);
    }
  } else {
    // ---------------- epilogue warps 2..9 (both CTAs): TMEM lane quarter warp % 4, column half
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* my_buf = sEpi + (warp - 2) * 2 * kEpiChunkBytes;
    uint32_t chunk_count = 0;
    [[maybe_unused]] constexpr int kShared = static_cast<int>(kOv4<NV>) / 32;    // chunks the accumulators share
    for (int i = 0; i < my_tiles; ++i) {
      const int tile = g.tile_at(cluster, n_clusters, i);
      const uint32_t acc = WIDE ? 0 : i & 1, aph = WIDE ? i & 1 : (i >> 1) & 1;
      if (warp_aborted(abort_flag)) break;
      if (!warp_wait(smem_u32(&S->acc_full[acc]), aph, limit, expire_epi)) {
        *abort_flag = 1;
        if (lane == 0) record_error(kErrTimeout);
        break;
      }
      tc_fence_after();
      const Problem4& P = g.problem(tile);
      const float alpha = __fmul_rn(P.sa ? ld_dep(P.sa) : 1.0f, P.sb ? ld_dep(P.sb) : 1.0f);
      const int M = P.M, N = P.N, local = tile - P.tile_start;
      const int row0 = (local / P.tiles_n) * kBM + static_cast<int>(rank) * kHalf + quad * 32;
      const int n0 = (local % P.tiles_n) * kTileN;
      const uint32_t t_base = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * kAcc1Col4<NV>;
      if constexpr (WIDE) {
        // this half's 192 columns into registers, then the accumulator is free
        uint32_t w[kBN4w / 64][16];
#pragma unroll
        for (int s = 0; s < kBN4w / 64; ++s) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(t_base + (half * (kBN4w / 64) + s) * 32, r);
          tmem_ld_wait();
          tmem_reg_fence(r);
          pack_chunk4(r, alpha, w[s]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&S->acc_empty[0]), 0));
#pragma unroll
        for (int s = 0; s < kBN4w / 64; ++s) {
          const int n = n0 + (half * (kBN4w / 64) + s) * 32;
          if (n < N && row0 < M) store_chunk4(&P.d, my_buf, chunk_count, w[s], lane, n, row0);
        }
      } else {
        // the shared columns come first: accumulator 0's last chunks (half 1, walking down), accumulator
        // 1's first (half 0, walking up)
#pragma unroll 1
        for (int step = 0; step < 4; ++step) {
          const int c = half * 4 + (acc == 0 ? 3 - step : step);
          uint32_t r[32];
          __syncwarp();                                    // one lane stored the chunk before
          tmem_ld_32x32b_x32(t_base + c * 32, r);
          tmem_ld_wait();
          tmem_reg_fence(r);
          if (step == kShared - 1 && half == (acc == 0 ? 1 : 0)) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&S->acc_shared_free), 0));
          }
          if (step == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&S->acc_empty[acc]), 0));
          }
          if (n0 + c * 32 >= N || row0 >= M) continue;     // chunk entirely outside the matrix
          uint32_t w[16];
          pack_chunk4(r, alpha, w);
          store_chunk4(&P.d, my_buf, chunk_count, w, lane, n0 + c * 32, row0);
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();                   // every store complete before exit
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {                   // loads of either CTA may still be in flight
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kSettleNs) {
    }
  }
  tc_fence_before();
  cluster_sync();                 // neither CTA leaves while the pair MMA may still read it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// ---------------------------------------------------------------- few rows: K split over a cluster
// A product of at most 128 rows (tokens) leaves most SMs idle under 256 x 256 tiles (a 4096-wide layer: 16
// tiles for 74 pairs), and its time is that of streaming B (the weights). Here the weights are the 128-row
// operand of a one-CTA MMA and the BT tokens the other, so a tile is 128 rows of B by all rows of A, and
// the S CTAs of a cluster each take a contiguous part of K. Every CTA leaves its FP32
// partial tile in the shared memory of the CTAs that own its tokens (groups of four: group j belongs to rank
// j mod S, 16 bytes of a weight row at a time); after a cluster barrier each owner adds the S partials in rank
// order, scales, rounds and stores its tokens' rows of D, 128 columns of a row at a time (a warp per group of tokens, four
// columns per lane: 128 x 4096 x 4096 9.7 -> 9.1 us against two columns per lane of 64, and 7.8 since the next kernel
// is let in behind the set-up). No workspace, and the order of additions is fixed. For many tokens the exchange counts:
// remote stores leave an SM at about 15 bytes per cycle, 1.7 us of these (measured with all of them kept in the CTA).
// TMEM: accumulator (weight rows x tokens) in columns 0..BT-1, then the scales.
constexpr int kSplitThreads = 128;
constexpr int kMaxSplitProblems = 4;
constexpr int64_t kMaxSplitRows = 128;
// The most slots that `groups` of four tokens take over 1 .. 8 owners: S * ceil(groups / S).
constexpr int split_slots(int groups) {
  int most = 0;
  for (int s = 1; s <= 8; ++s) most = s * ((groups + s - 1) / s) > most ? s * ((groups + s - 1) / s) : most;
  return most;
}
template <bool NV, int BT>
struct SplitShape {
  static constexpr int kSf = (NV ? 4 : 2) * 512;                 // scale bytes per 128 rows and k-block
  static constexpr int kStage = kABytes + BT * kBK + 2 * kSf;
  static constexpr int kStages = BT <= 16 ? 4 : 3;                // two CTAs per SM
  static constexpr int kSfCols = 8;                               // TMEM columns per atom step along K
  static constexpr int kTmem = BT <= 32 ? 64 : 2 * BT;
  // partials: beside the stages while two CTAs still fit an SM, so that a CTA may receive them while it
  // computes; else over the stages, behind one more cluster barrier
  static constexpr bool kApart = BT <= 32;
  static constexpr int kRedBytes = split_slots(BT / 4) * 128 * 16;
  static constexpr int kRed = kApart ? kRedBytes : 0;
  static constexpr int kSmem = kStages * kStage + kRed + 1024 + 256;
  static_assert(BT + (NV ? 4 : 2) * kSfCols <= kTmem, "TMEM columns");
  static_assert(kApart || kRedBytes <= kStages * kStage, "the partial tiles fit the stage buffers");
  static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs per SM");
  static_assert(kStage % 1024 == 0, "stages stay 1024-byte aligned");
};

struct alignas(64) SplitProblem {
  CUtensorMap w, t;                      // B [N][K/2] in 128-row boxes, A [M][K/2] in BT-row boxes
  CUtensorMap sfw, sft;                  // their scales
  const float* sa;
  const float* sb;
  uint16_t* D;
  int32_t M, N, num_kb, tile_start;
};
struct alignas(64) SplitGroup {
  SplitProblem p[kMaxSplitProblems];
  int32_t n;
};

template <bool NV>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  if constexpr (NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

template <bool NV, int BT>
__global__ void __launch_bounds__(kSplitThreads) k_fp4_gemm_split(const __grid_constant__ SplitGroup g) {
  using Sh = SplitShape<NV, BT>;
  constexpr int kSf = Sh::kSf, kSfRows = NV ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  struct Bars {
    uint64_t full[Sh::kStages], empty[Sh::kStages], done;
    uint32_t tmem_base;
    int abort;
  };
  Bars* S = reinterpret_cast<Bars*>(smem + Sh::kStages * Sh::kStage + Sh::kRed);
  volatile int* abort_flag = &S->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), ways = static_cast<int>(cluster_nctarank());
  const int tile = blockIdx.x / ways;
  int pi = 0;
  while (pi + 1 < g.n && g.p[pi + 1].tile_start <= tile) ++pi;
  const SplitProblem& P = g.p[pi];
  const int n0 = (tile - P.tile_start) * 128;
  // this CTA's k-blocks; a problem with fewer than the cluster's CTAs leaves some of them none
  const int kb0 = static_cast<int>(static_cast<int64_t>(P.num_kb) * rank / ways);
  const int kb1 = static_cast<int>(static_cast<int64_t>(P.num_kb) * (rank + 1) / ways);

  const uint64_t limit = wait_limit_ns();
  const int expire = expire_mode();
  const bool expire_main = expire == kExpireAll;
  auto load = [&](int kb, uint32_t s) {        // one lane: a k-block into stage s
    const uint32_t bar = smem_u32(&S->full[s]), w = smem_u32(smem + s * Sh::kStage);
    const uint32_t t = w + kABytes, sf = t + BT * kBK;
    mbar_arrive_expect_tx(bar, Sh::kStage);
    tma_load_2d(w, &P.w, kb * kBK, n0, bar);
    tma_load_2d(t, &P.t, kb * kBK, 0, bar);
    tma_load_2d(sf, &P.sfw, 0, ((n0 >> 7) * P.num_kb + kb) * kSfRows, bar);
    tma_load_2d(sf + kSf, &P.sft, 0, kb * kSfRows, bar);
  };

  if (ways > 1 && Sh::kApart) cluster_arrive();          // "running": waited for before the first remote store
  if (threadIdx.x == 0) {
    for (int s = 0; s < Sh::kStages; ++s) {
      mbar_init(smem_u32(&S->full[s]), 1);
      mbar_init(smem_u32(&S->empty[s]), 1);
    }
    mbar_init(smem_u32(&S->done), 1);
    *abort_flag = 0;
    fence_mbar_init();
    pdl_wait();
    // the first loads need nothing but these barriers: they start before the CTA's other set-up
    for (int kb = kb0; kb < kb1 && kb < kb0 + Sh::kStages; ++kb) load(kb, kb - kb0);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&S->tmem_base), Sh::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  // Only now may the next kernel start: one that took this SM's tensor memory first would hold it until this grid has
  // ended, and this CTA would wait for it. By every thread: 128 x 4096 x 4096 7.8 us, by the allocating warp alone 9.2.
  pdl_trigger();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  pdl_wait();

  if (warp == 0) {
    const bool one = elect_one();
    for (int kb = kb0 + Sh::kStages; kb < kb1; ++kb) {
      const uint32_t it = kb - kb0, s = it % Sh::kStages, ph = (it / Sh::kStages) & 1;
      if (!warp_wait(smem_u32(&S->empty[s]), ph ^ 1, limit, expire_main) || warp_aborted(abort_flag)) {
        if (one && !*abort_flag) record_error(kErrTimeout);
        *abort_flag = 1;
        break;
      }
      if (one) load(kb, s);
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    uint32_t issued = 0;
    {
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        const uint32_t s = issued % Sh::kStages, ph = (issued / Sh::kStages) & 1;
        if (!warp_wait(smem_u32(&S->full[s]), ph, limit, expire_main) || warp_aborted(abort_flag)) {
          if (one && !*abort_flag) record_error(kErrTimeout);
          *abort_flag = 1;
          break;
        }
        if (one) {
          const uint32_t w = smem_u32(smem + s * Sh::kStage), t = w + kABytes, sf = t + BT * kBK;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int a = NV ? k : k >> 1;
            const uint32_t sc = tmem + BT + a * Sh::kSfCols, id = NV ? 0 : (k & 1) * 2;
            if (NV || (k & 1) == 0) {
              tc_cp_32x128b_warpx4(sc, make_sf_desc(sf + a * 512));
              tc_cp_32x128b_warpx4(sc + 4, make_sf_desc(sf + kSf + a * 512));
            }
            tc_mma_fp4<NV>(tmem, make_sw128_desc(w + k * kUmmaK), make_sw128_desc(t + k * kUmmaK),
                           make_idesc_fp4<NV>(128, BT, id), sc | id << 30, (sc + 4) | id << 30,
                           (kb > kb0 || k) ? 1u : 0u);
          }
          tc_commit(smem_u32(&S->empty[s]));
        }
        __syncwarp();
      }
      if (one) tc_commit(smem_u32(&S->done));
      __syncwarp();
      // after an abort: loads in flight must land before shared memory is reused or released
      if (*abort_flag) {
        const uint64_t t1 = globaltimer_ns();
        while (globaltimer_ns() - t1 < kSettleNs) {
        }
      }
    }
  }
  __syncwarp();
  if (!warp_wait(smem_u32(&S->done), 0, limit, expire != kExpireNone)) {
    if (lane == 0) record_error(kErrTimeout);
    *abort_flag = 1;
    warp_wait(smem_u32(&S->done), 0, kDrainLimitNs);       // MMAs in flight, whatever the limit was
  }
  __syncwarp();                                            // TMEM loads follow
  tc_fence_after();
  const int per = (BT / 4 + ways - 1) / ways;   // slots: groups of four tokens per owner
  uint32_t red;                                 // [ways][per][128] x 4 f32
  if (Sh::kApart) {
    red = smem_u32(smem + Sh::kStages * Sh::kStage);
    if (ways > 1) cluster_wait();            // every CTA of the cluster runs
  } else {
    red = smem_u32(smem);
    __syncthreads();                         // the MMAs that read the stage buffers are done, in this CTA
    if (ways > 1) cluster_sync();            // and in every CTA that receives partials
  }
  // a weight row's place in its 128, such that eight lanes that read every fourth row (the sum below) meet all banks
  auto place = [](int row) { return row ^ ((row >> 3) & 3); };
  int owner = 0, slot = 0;                      // of the group: j mod ways, j / ways
#pragma unroll 1
  for (int c = 0; c < BT && c < P.M; c += 16) {
    uint32_t r[16];
    tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, r);
    tmem_ld_wait();
    tmem_reg_fence(r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c + 4 * j >= P.M) break;
      if (kb1 == kb0) r[4 * j] = r[4 * j + 1] = r[4 * j + 2] = r[4 * j + 3] = 0u;
      const uint32_t to = red + ((rank * per + slot) * 128 + place(threadIdx.x)) * 16;
      st_cluster_v4(mapa_shared(to, owner), r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
      if (++owner == ways) {
        owner = 0;
        ++slot;
      }
    }
  }
  tc_fence_before();
  if (ways > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, Sh::kTmem);
  if (*abort_flag) return;                   // D is incomplete; the error word says so
  const float alpha = __fmul_rn(P.sa ? ld_dep(P.sa) : 1.0f, P.sb ? ld_dep(P.sb) : 1.0f);
  const float4* part = reinterpret_cast<const float4*>(smem + (red - smem_u32(smem)));
  const int n = n0 + 4 * lane;                 // four weight rows: adjacent columns of D; a group of tokens per warp
  if (n >= P.N) return;                        // N is a multiple of 8
  const int M = P.M, N = P.N;
  uint16_t* D = P.D + n;
  for (int s = warp; (s * ways + rank) * 4 < M; s += kSplitThreads / 32) {
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = part[s * 128 + place(4 * lane + i)];
#pragma unroll 1
    for (int w = 1; w < ways; ++w) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 u = part[(w * per + s) * 128 + place(4 * lane + i)];
        x[i].x = __fadd_rn(x[i].x, u.x); x[i].y = __fadd_rn(x[i].y, u.y);
        x[i].z = __fadd_rn(x[i].z, u.z); x[i].w = __fadd_rn(x[i].w, u.w);
      }
    }
    const int m = (s * ways + rank) * 4;
    auto store = [&](int k, float a, float b, float c, float d) {
      if (m + k < M)
        *reinterpret_cast<uint2*>(D + static_cast<int64_t>(m + k) * N) =
            make_uint2(pack_bf16x2(__fmul_rn(a, alpha), __fmul_rn(b, alpha)), pack_bf16x2(__fmul_rn(c, alpha), __fmul_rn(d, alpha)));
    };
    store(0, x[0].x, x[1].x, x[2].x, x[3].x);
    store(1, x[0].y, x[1].y, x[2].y, x[3].y);
    store(2, x[0].z, x[1].z, x[2].z, x[3].z);
    store(3, x[0].w, x[1].w, x[2].w, x[3].w);
  }
}

}  // namespace gemm
}  // namespace fp8t
