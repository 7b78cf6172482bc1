// gemm_pair.cuh — the pair-tile product that the gated feed-forward and the Newton-Schulz kernels share: operands by
// TMA, tcgen05.mma on a CTA pair, two accumulators, and an epilogue that the operator supplies.
//
// A cluster of two CTAs computes a tile of 256 rows by 256 accumulator columns of A . B^T, K a 128-byte k-block at a time
// (128 FP8 or 64 FP16 values): CTA r holds 128 rows of A and 128 rows of B, 32 KB a stage, six stages. The tile's two
// 256-column accumulators fill tensor memory, so the epilogue of a tile runs beside the next tile's MMAs; it may
// therefore do arithmetic and read other tensors as long as it is shorter than the MMAs of one tile (512 cycles a
// k-block, 16 thousand for K = 4096 in FP8).
// Operands are K-major ([rows][K]) or MN-major ([K][rows]). The 128-byte swizzle holds 128 FP8 but only 64 FP16 values in
// a row, so an MN-major FP16 operand of 128 rows is two boxes of 64 x 64, 8 KB apart (the descriptor's leading byte offset).
//
// An operator Op supplies
//   Params                     grid constants; problem(tile) finds the product that a tile belongs to
//   kF16                       operand type
//   place(P, local, mt, nt)    row and column tile of a problem's tile number
//   b_row(P, nt, rank)         first row of B that a CTA holds
//   epilogue(...)              what becomes of the accumulators, by eight warps: a TMEM lane quarter and a column half each
//   finish(...)                called by a thread of every CTA at its end, with whether a wait of it expired
// Warp roles (320 threads), waits and their limits are those of the 4-bit tile kernel.
#pragma once

#include "gemm_fp4.cuh"

namespace fp8t {
namespace pair {

using namespace gemm;

constexpr int kPairStages = 6;
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int kPairEpiBytes = kPairEpiWarps * 2 * kEpiChunkBytes;
constexpr int kPairSmemBytes = kPairStages * kStageBytes + kPairEpiBytes + 1024 + 256;
static_assert(kPairSmemBytes <= 232448, "shared memory of an SM");

struct PairSmem {
  uint64_t full[kPairStages];     // even CTA: both CTAs' loads of a stage have landed
  uint64_t empty[kPairStages];    // both CTAs: the pair MMA has consumed a stage
  uint64_t acc_full[2];           // both CTAs: an accumulator holds a finished tile
  uint64_t acc_empty[2];          // even CTA: every epilogue warp of both CTAs has read an accumulator
  uint64_t mma_done;              // even CTA: every issued MMA has completed
  uint32_t tmem_base;
  uint32_t amax;                  // largest magnitude pattern that this CTA's epilogue has seen
  int abort;
};
static_assert(sizeof(PairSmem) <= 256, "barriers");

// MN-major FP16: 64 values per 128-byte swizzle row, 8 K-rows (1024 B) per atom, the next 64 values 8 KB on.
__device__ __forceinline__ uint64_t make_sw128_desc_mn16(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);        // start address
  d |= static_cast<uint64_t>(8192 >> 4) << 16;               // leading byte offset: along M or N
  d |= static_cast<uint64_t>(1024 >> 4) << 32;               // stride byte offset: along K
  d |= static_cast<uint64_t>(1) << 46;                       // descriptor version (sm_100)
  d |= static_cast<uint64_t>(2) << 61;                       // 128-byte swizzle
  return d;
}
// FP32 accumulator, FP16 operands, M = 256 (pair), N = 256.
__host__ __device__ constexpr uint32_t make_idesc_f16(int a_mn, int b_mn) { return make_idesc(0, 0, a_mn, b_mn); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What an epilogue warp holds between chunks.
struct Out {
  uint8_t* buf;                   // its two 2 KB staging buffers
  uint32_t count;                 // chunks staged so far
  uint32_t amax;                  // this lane's largest magnitude pattern
  int lane;
};
// A buffer whose last store has been read.
__device__ __forceinline__ uint8_t* next_buffer(Out& o) {
  uint8_t* b = o.buf + (o.count & 1) * kEpiChunkBytes;
  ++o.count;
  if (o.lane == 0) bulk_wait_group_read<1>();
  __syncwarp();
  return b;
}
__device__ __forceinline__ void send(Out& o, const CUtensorMap* map, const uint8_t* b, int x, int y) {
  fence_proxy_async_smem();
  __syncwarp();
  if (o.lane == 0) {
    tma_store_2d(map, smem_u32(b), x, y);
    bulk_commit_group();
  }
}
// 32 x 32 16-bit values, a row per lane, to (row y, column x): 64-byte swizzle.
__device__ __forceinline__ void store16(Out& o, const CUtensorMap* map, const uint32_t (&w)[16], int x, int y) {
  uint8_t* b = next_buffer(o);
#pragma unroll
  for (int p = 0; p < 4; ++p)
    *reinterpret_cast<uint4*>(b + o.lane * 64 + (p ^ ((o.lane >> 1) & 3)) * 16) =
        make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
  send(o, map, b, x, y);
}
// The same chunk transposed: the lane's values become a column. For each j the warp writes the 64 bytes of one row.
__device__ __forceinline__ void store16_transposed(Out& o, const CUtensorMap* map, const uint32_t (&w)[16], int x, int y) {
  uint8_t* b = next_buffer(o);
#pragma unroll
  for (int j = 0; j < 32; ++j)
    *reinterpret_cast<uint16_t*>(b + j * 64 + (((o.lane >> 3) ^ ((j >> 1) & 3)) * 16) + (o.lane & 7) * 2) =
        static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
  send(o, map, b, x, y);
}
// 32 x 32 bytes: 32-byte swizzle.
__device__ __forceinline__ void store8(Out& o, const CUtensorMap* map, const uint32_t (&w)[8], int x, int y) {
  uint8_t* b = next_buffer(o);
#pragma unroll
  for (int p = 0; p < 2; ++p)
    *reinterpret_cast<uint4*>(b + o.lane * 32 + (p ^ ((o.lane >> 2) & 1)) * 16) =
        make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
  send(o, map, b, x, y);
}

template <class Op>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_pair_gemm(const __grid_constant__ typename Op::Params g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sEpi = smem + kPairStages * kStageBytes;          // stage s: [A 128 x 128 B][B 128 x 128 B]
  PairSmem* S = reinterpret_cast<PairSmem*>(sEpi + kPairEpiBytes);
  volatile int* abort_flag = &S->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int total = g.total_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(smem_u32(&S->full[s]), 1);
      mbar_init(smem_u32(&S->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&S->acc_full[a]), 1);
      mbar_init(smem_u32(&S->acc_empty[a]), 2 * kPairEpiWarps);
    }
    mbar_init(smem_u32(&S->mma_done), 1);
    *abort_flag = 0;
    S->amax = 0;
    fence_mbar_init();
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
  pdl_enter();

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs)
    const bool one = elect_one();
    constexpr int kElems = Op::kF16 ? 64 : 128;              // K values of a k-block
    uint32_t it = 0, issued = 0;
    for (int tile = cluster; tile < total && !warp_aborted(abort_flag); tile += n_clusters) {
      const auto& P = g.problem(tile);
      int mt, nt;
      Op::place(P, tile - P.tile_start, mt, nt);
      const int m0 = mt * kBM + static_cast<int>(rank) * kHalf, n0 = Op::b_row(P, nt, static_cast<int>(rank));
      const int num_kb = P.num_kb;
      for (int kb = 0; kb < num_kb; ++kb, ++it) {
        const uint32_t s = it % kPairStages, ph = (it / kPairStages) & 1;
        if (warp_aborted(abort_flag)) break;
        if (!warp_wait(smem_u32(&S->empty[s]), ph ^ 1, limit, expire_main)) {
          *abort_flag = 1;
          if (one) record_error(kErrTimeout);
          break;
        }
        if (one) {
          const uint32_t full_leader = mapa_shared(smem_u32(&S->full[s]), 0);
          if (leader) mbar_arrive_expect_tx(smem_u32(&S->full[s]), kPairTxBytes);
          const uint32_t a_dst = smem_u32(smem + s * kStageBytes), b_dst = a_dst + kABytes;
          if (!P.a_mn) {
            tma_load_2d_pair(a_dst, &P.a, kb * kElems, m0, full_leader);
          } else {
            tma_load_2d_pair(a_dst, &P.a, m0, kb * kElems, full_leader);
            if (Op::kF16) tma_load_2d_pair(a_dst + 8192, &P.a, m0 + 64, kb * kElems, full_leader);
          }
          if (!P.b_mn) {
            tma_load_2d_pair(b_dst, &P.b, kb * kElems, n0, full_leader);
          } else {
            tma_load_2d_pair(b_dst, &P.b, n0, kb * kElems, full_leader);
            if (Op::kF16) tma_load_2d_pair(b_dst + 8192, &P.b, n0 + 64, kb * kElems, full_leader);
          }
        }
        ++issued;
      }
    }
    // the even CTA can see its own stages land: wait for the last ones it armed (one shared budget; after
    // an abort a stage may miss the peer's bytes, and the settle delay below covers loads in flight)
    if (leader) {
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = issued > kPairStages ? issued - kPairStages : 0; i < issued; ++i) {
        const uint64_t spent = globaltimer_ns() - t0;
        if (spent >= kPairDrainNs) break;
        mbar_wait(smem_u32(&S->full[i % kPairStages]), (i / kPairStages) & 1, kPairDrainNs - spent);
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer (even CTA)
      const bool one = elect_one();
      uint32_t it = 0, i = 0;
      for (int tile = cluster; tile < total && !warp_aborted(abort_flag); tile += n_clusters, ++i) {
        const auto& P = g.problem(tile);
        const int num_kb = P.num_kb;
        const uint32_t idesc = P.idesc;
        const bool a_mn = P.a_mn != 0, b_mn = P.b_mn != 0;
        const uint32_t acc = i & 1, aph = (i >> 1) & 1;
        if (!warp_wait(smem_u32(&S->acc_empty[acc]), aph ^ 1, limit, expire_main)) {
          *abort_flag = 1;
          if (one) record_error(kErrTimeout);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + acc * kAccCols;
        bool ok = true;
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const uint32_t s = it % kPairStages, ph = (it / kPairStages) & 1;
          if (!warp_wait(smem_u32(&S->full[s]), ph, limit, expire_main) || warp_aborted(abort_flag)) {
            if (one && !*abort_flag) record_error(kErrTimeout);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          if (one) {
            const uint32_t a_base = smem_u32(smem + s * kStageBytes), b_base = a_base + kABytes;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t more = (kb | k) != 0 ? 1u : 0u;
              if constexpr (Op::kF16)
                tc_mma_f16_pair(d_tmem, a_mn ? make_sw128_desc_mn16(a_base + k * 2048) : make_sw128_desc(a_base + k * 32),
                                b_mn ? make_sw128_desc_mn16(b_base + k * 2048) : make_sw128_desc(b_base + k * 32), idesc, more);
              else
                tc_mma_f8_pair(d_tmem, a_mn ? make_sw128_desc_mn(a_base + k * 4096) : make_sw128_desc(a_base + k * 32),
                               b_mn ? make_sw128_desc_mn(b_base + k * 4096) : make_sw128_desc(b_base + k * 32), idesc, more);
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
    Out o{sEpi + (warp - 2) * 2 * kEpiChunkBytes, 0u, 0u, lane};
    const typename Op::Scalars k = Op::scalars(g);
    uint32_t i = 0;
    for (int tile = cluster; tile < total; tile += n_clusters, ++i) {
      const uint32_t acc = i & 1, aph = (i >> 1) & 1;
      const auto& P = g.problem(tile);
      int mt, nt;
      Op::place(P, tile - P.tile_start, mt, nt);
      if (warp_aborted(abort_flag)) break;
      if (!warp_wait(smem_u32(&S->acc_full[acc]), aph, limit, expire_epi)) {
        *abort_flag = 1;
        if (lane == 0) record_error(kErrTimeout);
        break;
      }
      tc_fence_after();
      const int row0 = mt * kBM + static_cast<int>(rank) * kHalf + quad * 32;
      const uint32_t t_base = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * kAccCols;
      Op::epilogue(g, P, k, o, mt, nt, row0, half, t_base, [&] {          // called once, behind the last TMEM load
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&S->acc_empty[acc]), 0));
      });
    }
    if (lane == 0) bulk_wait_group<0>();                   // every store complete before exit
    __syncwarp();
    if constexpr (Op::kAmax) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, o.amax);
      if (lane == 0 && top) atomicMax(&S->amax, top);
    }
  }
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0) Op::finish(g, S->amax, *abort_flag != 0);
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

}  // namespace pair
}  // namespace fp8t
