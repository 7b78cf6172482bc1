// gemm_pair.cuh — the pair-tile product that the gated feed-forward and the Newton-Schulz kernels share: operands by
// TMA, tcgen05.mma on a CTA pair, two accumulators, and an epilogue that the operator supplies.
//
// A cluster of two CTAs computes a tile of 256 rows by 256 accumulator columns of A . B^T, K a 128-byte k-block at a time
// (128 FP8 or 64 FP16 values): CTA r holds 128 rows of A and 128 rows of B, 32 KB a stage, six stages. The tile's two
// 256-column accumulators fill tensor memory, so the epilogue of a tile runs beside the next tile's MMAs; it may
// therefore do arithmetic and read other tensors as long as it is shorter than the MMAs of one tile (512 cycles a
// k-block, 16 thousand for K = 4096 in FP8). What it reads comes by TMA too, a 32 x 32 chunk ahead, into a buffer of each warp:
// a lane's own loads of its row's 64 bytes fetched every line twice (fp8_gated_gemm_backward 16384 x 4096 x 11008 731 us).
// Operands are K-major ([rows][K]) or MN-major ([K][rows]). The 128-byte swizzle holds 128 FP8 but only 64 FP16 values in
// a row, so an MN-major FP16 operand of 128 rows is two boxes of 64 x 64, 8 KB apart (the descriptor's leading byte offset).
//
// A launch may run several phases, each a set of products that read what the phase before has stored, behind a barrier of the
// whole grid (then launched cooperatively, so that all its CTAs are resident).
//
// An operator Op supplies
//   Params                     grid constants
//   kF16, kPhased, kLoads      operand type; whether there are phases; chunks that its epilogue reads at a time
//   phases(g), tiles(g, ph)    phases, and the tiles of one
//   work(g, ph, tile, rank)    a tile's operands and place (Work)
//   epilogue(...)              what becomes of the accumulators, by eight warps: a TMEM lane quarter and a column half each
//   prefetch(...)              the fetching of a tile's first chunks
//   finish(...)                called by a thread of every CTA at its end, with whether a wait of it expired
// Warp roles (320 threads), waits and their limits are those of the 4-bit tile kernel.
#pragma once

#include "gemm_fp4.cuh"

namespace fp8t {
namespace pair {

using namespace gemm;

constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int kPairMaxStages = 6;
// An operator that reads chunks (Op::kLoads of them at a time, 2 KB each and warp) has a stage less.
template <class Op>
constexpr int kPairStages = Op::kLoads > 0 ? 5 : 6;
template <class Op>
constexpr int kPairEpiBytes = kPairEpiWarps * (2 + Op::kLoads) * kEpiChunkBytes;
template <class Op>
constexpr int kPairSmemBytes = kPairStages<Op> * kStageBytes + kPairEpiBytes<Op> + 1024 + 512;

struct PairSmem {
  uint64_t full[kPairMaxStages];  // even CTA: both CTAs' loads of a stage have landed
  uint64_t empty[kPairMaxStages]; // both CTAs: the pair MMA has consumed a stage
  uint64_t acc_full[2];           // both CTAs: an accumulator holds a finished tile
  uint64_t acc_empty[2];          // even CTA: every epilogue warp of both CTAs has read an accumulator
  uint64_t mma_done;              // even CTA: every issued MMA has completed
  uint64_t loaded[kPairEpiWarps]; // an epilogue warp's chunks have landed
  uint64_t taken[kPairEpiWarps];  // its loads of them have left the queue to shared memory
  uint32_t tmem_base;
  uint32_t amax;                  // largest magnitude pattern that this CTA's epilogue has seen
  uint32_t warps_done;            // phases that its epilogue warps have ended, summed
  int abort;
};
static_assert(sizeof(PairSmem) <= 512, "barriers");

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
// FP32 accumulator, FP16 operands, M = 256 (pair), N = 256 or n.
__host__ __device__ constexpr uint32_t make_idesc_f16(int a_mn, int b_mn, int n = kBN) {
  return make_idesc(0, 0, a_mn, b_mn) - (static_cast<uint32_t>((kBN - n) >> 3) << 17);
}

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
  uint8_t* in;                    // where its chunks are loaded to, and their barriers
  uint32_t loaded, phase;
  uint32_t taken, taken_phase;
  uint64_t limit;
};
// The warp's next chunks: `maps` at column x, row y (whatever lies outside the matrix reads as zeros). The lanes have issued
// their loads of what was there, but a warp's barrier does not wait for them to be carried out: behind a __syncwarp alone the copy
// came first for about one chunk in a million, where the tensor cores keep shared memory busy. So each lane orders its loads
// before the async proxy, and lane 0 sees an arrival that it has queued behind them.
template <int N>
__device__ __forceinline__ void fetch(Out& o, const CUtensorMap* const (&maps)[N], const int (&x)[N], int y) {
  fence_proxy_async_smem();
  __syncwarp();
  if (o.lane == 0) {
    mbar_arrive(o.taken);
    mbar_wait(o.taken, o.taken_phase, o.limit);
    mbar_arrive_expect_tx(o.loaded, N * kEpiChunkBytes);
#pragma unroll
    for (int i = 0; i < N; ++i) tma_load_2d(smem_u32(o.in + i * kEpiChunkBytes), maps[i], x[i], y, o.loaded);
  }
  o.taken_phase ^= 1;
}
// Waits for them; false if the wait expired.
__device__ __forceinline__ bool fetched(Out& o) {
  const bool ok = warp_wait(o.loaded, o.phase, o.limit);
  o.phase ^= 1;
  return ok;
}
// The lane's row of chunk i: 32 16-bit values.
__device__ __forceinline__ void chunk_row(const Out& o, int i, uint4 (&v)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
    v[p] = *reinterpret_cast<const uint4*>(o.in + i * kEpiChunkBytes + o.lane * 64 + (p ^ ((o.lane >> 1) & 3)) * 16);
}
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

// A tile of a product. FP8 boxes are as many rows as a CTA holds, FP16 boxes 64 (one or two of them), of 128 bytes.
struct Work {
  const CUtensorMap *a, *b;
  int a_row, b_row;                // first row of A and of B that this CTA holds
  int mt, nt;                      // row and column tile
  int half_n;                      // rows of B that each CTA holds: 128; 64 or, of FP8, 96 for narrower tiles (not of MN-major FP8)
  int a_bytes;                     // of A's boxes of a k-block
  int num_kb;
  int a_mn, b_mn;                  // 1: operand stored MN-major
  uint32_t idesc;
  int which;                       // the operator's own
};

// Tiles in runs of kRun row tiles, column by column: the 74 tiles that run at a time then read 8 row panels of A and 9 column
// panels of B where row by row they read 2 and all of B's (X = B X of 4096 x 11008: a third of the bytes from memory).
constexpr int kRun = 8;
__device__ __forceinline__ void place_in_runs(int tiles_m, int tiles_n, int local, int& mt, int& nt) {
  const int run = local / (kRun * tiles_n), in = local - run * kRun * tiles_n;
  const int rows = min(kRun, tiles_m - run * kRun);
  nt = in / rows;
  mt = run * kRun + in - nt * rows;
}

// ------------------------------------------------------------------ a barrier of the whole grid
// counter counts the CTAs that have ended a phase, expired is set by one that gave up; both zero at the launch.
struct Grid {
  unsigned int* counter;
  int32_t* expired;
};
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ unsigned int ld_acquire(const unsigned int* p) {
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// By each epilogue warp at a phase's end; lane 0 stored by TMA. What the warp stored is there for other CTAs' TMA loads, and the
// last of the CTA's warps counts the CTA. No warp waits for another here: one may have given up.
__device__ __forceinline__ void grid_arrive(const Grid& g, unsigned int* warps_done, int lane) {
  if (lane == 0) {
    bulk_wait_group<0>();
    fence_proxy_async_all();
    // every warp releases, so that the last one's arrival carries the others' stores
    unsigned int before;
    asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(before) : "r"(smem_u32(warps_done)) : "memory");
    if (before % kPairEpiWarps == kPairEpiWarps - 1)
      asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(g.counter) : "memory");
  }
  __syncwarp();
}
// By a whole warp: until `target` CTAs have arrived; false if that took too long or a CTA gave up.
__device__ __forceinline__ bool grid_wait(const Grid& g, unsigned int target, uint64_t limit, bool expire, int lane) {
  bool ok = true;
  if (lane == 0) {
    const uint64_t t0 = globaltimer_ns();
    while (ok && (expire || ld_acquire(g.counter) < target)) {
      // the clock and the other word only now and then: each is a round trip that would delay the next look at the counter
      int looks = 0;
      while (looks < 16 && (expire || ld_acquire(g.counter) < target)) ++looks;
      if (looks == 16 && (*reinterpret_cast<volatile int32_t*>(g.expired) != 0 || globaltimer_ns() - t0 > limit)) ok = false;
    }
    fence_proxy_async_all();
  }
  return __all_sync(0xffffffffu, ok);
}

template <class Op>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_pair_gemm(const __grid_constant__ typename Op::Params g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int kStages = kPairStages<Op>;
  static_assert(kPairSmemBytes<Op> <= 232448, "shared memory of an SM");
  uint8_t* sEpi = smem + kStages * kStageBytes;              // stage s: [A 128 x 128 B][B 128 x 128 B]
  PairSmem* S = reinterpret_cast<PairSmem*>(sEpi + kPairEpiBytes<Op>);
  volatile int* abort_flag = &S->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int phases = Op::phases(g);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&S->full[s]), 1);
      mbar_init(smem_u32(&S->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&S->acc_full[a]), 1);
      mbar_init(smem_u32(&S->acc_empty[a]), 2 * kPairEpiWarps);
    }
    mbar_init(smem_u32(&S->mma_done), 1);
    for (int w = 0; w < kPairEpiWarps; ++w) {
      mbar_init(smem_u32(&S->loaded[w]), 1);
      mbar_init(smem_u32(&S->taken[w]), 1);
    }
    *abort_flag = 0;
    S->amax = 0;
    S->warps_done = 0;
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
    for (int ph = 0; ph < phases && !warp_aborted(abort_flag); ++ph) {
      if (Op::kPhased && ph > 0 && !grid_wait(Op::grid(g), ph * gridDim.x, limit, expire_main, lane)) {
        *abort_flag = 1;
        if (one) record_error(kErrTimeout);
        break;
      }
      const int total = Op::tiles(g, ph);
      for (int tile = cluster; tile < total && !warp_aborted(abort_flag); tile += n_clusters) {
        const Work w = Op::work(g, ph, tile, static_cast<int>(rank));
        for (int kb = 0; kb < w.num_kb; ++kb, ++it) {
          const uint32_t s = it % kStages, ph_s = (it / kStages) & 1;
          if (warp_aborted(abort_flag)) break;
          if (!warp_wait(smem_u32(&S->empty[s]), ph_s ^ 1, limit, expire_main)) {
            *abort_flag = 1;
            if (one) record_error(kErrTimeout);
            break;
          }
          if (one) {
            const uint32_t full_leader = mapa_shared(smem_u32(&S->full[s]), 0);
            const bool second = Op::kF16 && w.half_n > 64;   // B's second box of 64
            if (leader) mbar_arrive_expect_tx(smem_u32(&S->full[s]), 2 * (w.a_bytes + w.half_n * kBK));
            const uint32_t a_dst = smem_u32(smem + s * kStageBytes), b_dst = a_dst + kABytes;
            const int k0 = kb * kElems;
            tma_load_2d_pair(a_dst, w.a, w.a_mn ? w.a_row : k0, w.a_mn ? k0 : w.a_row, full_leader);
            if (Op::kF16)
              tma_load_2d_pair(a_dst + 8192, w.a, w.a_mn ? w.a_row + 64 : k0, w.a_mn ? k0 : w.a_row + 64, full_leader);
            tma_load_2d_pair(b_dst, w.b, w.b_mn ? w.b_row : k0, w.b_mn ? k0 : w.b_row, full_leader);
            if (second)
              tma_load_2d_pair(b_dst + 8192, w.b, w.b_mn ? w.b_row + 64 : k0, w.b_mn ? k0 : w.b_row + 64, full_leader);
          }
          ++issued;
        }
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
      uint32_t it = 0, i = 0;
      bool ok = true;
      for (int ph = 0; ph < phases && ok; ++ph) {
        const int total = Op::tiles(g, ph);
        for (int tile = cluster; tile < total && ok; tile += n_clusters, ++i) {
          const Work w = Op::work(g, ph, tile, 0);
          const bool a_mn = w.a_mn != 0, b_mn = w.b_mn != 0;
          const uint32_t acc = i & 1, aph = (i >> 1) & 1;
          if (warp_aborted(abort_flag) || !warp_wait(smem_u32(&S->acc_empty[acc]), aph ^ 1, limit, expire_main)) {
            if (one && !*abort_flag) record_error(kErrTimeout);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem + acc * kAccCols;
          for (int kb = 0; kb < w.num_kb; ++kb, ++it) {
            const uint32_t s = it % kStages, ph_s = (it / kStages) & 1;
            // behind a barrier of the grid the first stage may take as long as the slowest CTA
            if (!warp_wait(smem_u32(&S->full[s]), ph_s, Op::kPhased ? 2 * limit : limit, expire_main) || warp_aborted(abort_flag)) {
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
                                  b_mn ? make_sw128_desc_mn16(b_base + k * 2048) : make_sw128_desc(b_base + k * 32), w.idesc, more);
                else
                  tc_mma_f8_pair(d_tmem, a_mn ? make_sw128_desc_mn(a_base + k * 4096) : make_sw128_desc(a_base + k * 32),
                                 b_mn ? make_sw128_desc_mn(b_base + k * 4096) : make_sw128_desc(b_base + k * 32), w.idesc, more);
              }
              tc_commit_pair_mc(smem_u32(&S->empty[s]), 0x3);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (one) tc_commit_pair_mc(smem_u32(&S->acc_full[acc]), 0x3);
          __syncwarp();
        }
      }
      // every MMA issued here must complete before either CTA frees TMEM or shared memory
      if (one) tc_commit_pair(smem_u32(&S->mma_done));
      __syncwarp();
      mbar_wait(smem_u32(&S->mma_done), 0, kDrainLimitNs);
    }
  } else {
    // ---------------- epilogue warps 2..9 (both CTAs): TMEM lane quarter warp % 4, column half
    const int quad = warp & 3, half = (warp - 2) >> 2;
    Out o{sEpi + (warp - 2) * 2 * kEpiChunkBytes, 0u, 0u, lane,
          sEpi + (2 * kPairEpiWarps + (warp - 2) * Op::kLoads) * kEpiChunkBytes, smem_u32(&S->loaded[warp - 2]), 0u,
          smem_u32(&S->taken[warp - 2]), 0u, limit};
    const typename Op::Scalars k = Op::scalars(g);
    uint32_t i = 0;
    bool ok = true;
    for (int ph = 0; ph < phases && ok; ++ph) {
      const int total = Op::tiles(g, ph);
      // the warp's first chunks of a tile, fetched ahead
      auto ahead = [&](int tile) {
        if (Op::kLoads == 0 || tile >= total) return;
        const Work w = Op::work(g, ph, tile, static_cast<int>(rank));
        Op::prefetch(g, w, ph, o, w.mt * kBM + static_cast<int>(rank) * kHalf + quad * 32, half);
      };
      // before it reads what the last phase stored; and a CTA without tiles, so that it does not arrive ahead of the others
      if (Op::kPhased && ph > 0 && (Op::reads(ph) || cluster >= total) &&
          !grid_wait(Op::grid(g), ph * gridDim.x, limit, expire_epi, lane)) {
        *abort_flag = 1;
        if (lane == 0) record_error(kErrTimeout);
        break;
      }
      ahead(cluster);
      for (int tile = cluster; tile < total; tile += n_clusters, ++i) {
        const uint32_t acc = i & 1, aph = (i >> 1) & 1;
        const Work w = Op::work(g, ph, tile, static_cast<int>(rank));
        if (warp_aborted(abort_flag) ||
            !warp_wait(smem_u32(&S->acc_full[acc]), aph, Op::kPhased ? 3 * limit : limit, expire_epi)) {
          if (lane == 0 && !*abort_flag) record_error(kErrTimeout);
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const int row0 = w.mt * kBM + static_cast<int>(rank) * kHalf + quad * 32;
        const uint32_t t_base = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * kAccCols;
        ok = Op::epilogue(g, w, ph, k, o, row0, half, t_base, [&] {   // called once, behind the last TMEM load
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_tmem(mapa_shared(smem_u32(&S->acc_empty[acc]), 0));
        }, [&] { ahead(tile + n_clusters); });             // called once, when the last chunk has been read
        if (!ok) {
          *abort_flag = 1;
          if (lane == 0) record_error(kErrTimeout);
          break;
        }
      }
      if (Op::kPhased && ph + 1 < phases) {
        if (!ok || warp_aborted(abort_flag)) break;        // a CTA that gave up does not arrive
        grid_arrive(Op::grid(g), &S->warps_done, lane);
      }
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
