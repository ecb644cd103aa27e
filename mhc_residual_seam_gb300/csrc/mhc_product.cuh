// Matrix products with a fused epilogue on the tensor cores, for the gated
// projections and their gradient: D[M, N] = sum_k A[m, k] B[n, k], 16-bit
// operands, fp32 accumulators in tensor memory.
//
// One persistent CTA (or pair of CTAs) per SM: a producer thread fetches 64-deep
// tiles of A and B by TMA into a ring of stages, a second thread issues
// tcgen05.mma on them, eight warps turn finished accumulators into outputs while
// the next tile's products run (two accumulators).  A pair works on one tile of
// 256 rows: each CTA holds its 128 rows of A and half of B, so that an SM fetches
// 32 KB a step where a CTA by itself fetches 48.
//
// Either operand may lie with its reduction index k adjacent ("K-major", a row per
// m or n) or with m or n adjacent (a row per k): then a tile is fetched as blocks of
// 64 columns and the MMA reads it transposed.  One launch may do two products, so
// that the second's tiles fill the SMs that the first leaves.
//
// What lies outside the matrices is fetched as zeros, so no size needs padding.
// Every wait is bounded; one that runs out sets bit 1 of the workspace's status
// word and the kernel gives up (mhc_check_status).
#pragma once

#include <type_traits>

#include "mhc_ops.cuh"
#include "mhc_sm100.cuh"

namespace mhc {

// mhc_stream.cu
bool encode(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle sw);

constexpr int kBM = 128, kBK = 64;  // rows of A per CTA, depth of a stage
constexpr int kProductThreads = 384;  // producer, MMA, allocation, an idle warp; eight epilogue warps
constexpr uint64_t kProductLimitNs = 2000000000ull;

// ------------------------------------------------------------ PTX, pairs --
template <int CG>
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1) tmem_dealloc(taddr, ncols);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
template <int CG>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1) {
    tc_mma_bf16(d, a, b, idesc, accumulate);  // (the instruction descriptor names the type)
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// Arrives on `bar` of every CTA of the group when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  if constexpr (CG == 1) {
    tc_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  }
}
// A tile into this CTA's shared memory; its bytes complete on `bar`, a barrier of
// this CTA or (CG = 2, an address from mapa) of the pair's first.
template <int CG>
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
// 16 columns of this warp's 32 lanes; take16 comes before any use.
__device__ __forceinline__ void issue16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void take16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Shared-memory descriptor of a tile in the 128-byte swizzle layout.  K-major: rows of
// 128 bytes (64 k), 8-row groups 1024 bytes apart.  Otherwise blocks of 64 columns (128
// bytes) by 64 k: 8-k groups 1024 bytes apart, blocks 8192.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, bool mn) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(mn ? 8192 >> 4 : 1) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
template <typename E>
__host__ __device__ constexpr uint32_t product_idesc(int M, int N, bool amn, bool bmn) {
  const uint32_t type = sizeof(E) == 2 && !std::is_same<E, __half>::value ? 1u : 0u;  // bf16 or f16
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)amn << 15) | ((uint32_t)bmn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// ----------------------------------------------------------------- kernel --
// One product: D in tiles of (128 CG) x BN, `kblocks` stages each; `amn`: A lies with m
// adjacent.
struct Problem {
  CUtensorMap a, b;
  int num_m, num_n, kblocks;
  bool amn;
};
// The products of one launch.  Tiles are handed out in order, so the ones with more
// stages come first.
template <int N>
struct Work {
  Problem p[N];
  int tiles[N];  // of this and the products before it
  unsigned* status;
};

template <int CG_, int BN_, bool BMN_>
struct Tile {
  static constexpr int CG = CG_, BN = BN_;  // CTAs of a group, columns of its tile
  static constexpr bool BMN = BMN_;         // B lies with n adjacent
  static constexpr int kRowsB = BN / CG;    // rows of B per CTA
  static constexpr int kA = kBM * 128, kB = kRowsB * 128, kStage = kA + kB;
  static constexpr int kStages = (200 * 1024) / kStage < 8 ? (200 * 1024) / kStage : 8;
  static constexpr int kCols = 2 * BN <= 256 ? 256 : 512;  // two accumulators
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024 + 256;
  static constexpr int kBoxB = BMN ? 64 : BN / 2;  // rows of a TMA box of B: a half of the columns may lie elsewhere than the other
};

// Tile number -> (m, n): eight rows of tiles at a time, so that the tiles in flight
// share rows of A and of B in L2.
__device__ __forceinline__ void tile_place(int t, int num_m, int num_n, int& m, int& n) {
  constexpr int kGroup = 8;
  const int per = kGroup * num_n, g = t / per, r = t - g * per;
  const int rows = min(kGroup, num_m - g * kGroup);
  n = r / rows;
  m = g * kGroup + r - n * rows;
}

// Epi: `row_b(n_tile, j)` is the row of B for column j of the tile; `store(tmem, row,
// n_tile, product, part)` makes a lane's row of outputs, every other 16 columns (part 0 or 1).
template <typename E, typename S, int NP, typename Epi>
__global__ void __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ Work<NP> w, const __grid_constant__ Epi epi) {
  constexpr int CG = S::CG, kStages = S::kStages;
  extern __shared__ char raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  char* aligned = raw + (base - smem_u32(raw));
  uint64_t* full = reinterpret_cast<uint64_t*>(aligned + (size_t)kStages * S::kStage);
  uint64_t *empty = full + kStages, *tfull = empty + kStages, *tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, 8 * CG);
    }
    mbar_fence_init();
  }
  if (warp == 2) pair_tmem_alloc<CG>(tmem_slot, S::kCols);
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int groups = gridDim.x / CG, group = blockIdx.x / CG;
  const int tiles = w.tiles[NP - 1];
  auto product_of = [&](int t) { return NP == 2 && t >= w.tiles[0] ? NP - 1 : 0; };
  bool ok = true;

  if (warp == 0) {  // ------------------------------------------- producer
    if (lane == 0) {
      int st = 0, used = 0;
      uint32_t ph = 1;
      for (int t = group; t < tiles && ok; t += groups) {
        const int which = product_of(t);
        const Problem& p = w.p[which];
        int m, n;
        tile_place(which ? t - w.tiles[0] : t, p.num_m, p.num_n, m, n);
        const int row = (m * CG + (int)rank) * kBM;
        for (int k = 0; k < p.kblocks; ++k) {
          ok = mbar_wait_cluster(empty + st, ph, kProductLimitNs);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(full + st, CG * S::kStage);
          const uint32_t bar = CG == 2 ? mapa_shared(smem_u32(full + st), 0) : smem_u32(full + st);
          const uint32_t a = base + st * S::kStage, b = a + S::kA;
          if (p.amn) {
            pair_load<CG>(a, &p.a, bar, row, k * kBK);
            pair_load<CG>(a + 8192, &p.a, bar, row + 64, k * kBK);
          } else {
            pair_load<CG>(a, &p.a, bar, k * kBK, row);
          }
#pragma unroll
          for (int j = 0; j < S::kRowsB; j += S::kBoxB) {
            const int rb = epi.row_b(n, (int)rank * S::kRowsB + j);
            if (S::BMN) pair_load<CG>(b + j * 128, &p.b, bar, rb, k * kBK);
            else pair_load<CG>(b + j * 128, &p.b, bar, k * kBK, rb);
          }
          if (used < kStages) ++used;
          if (++st == kStages) st = 0, ph ^= 1;
        }
      }
      // the MMAs' last arrivals on this CTA's barriers come before it ends
      for (; used > 0 && ok; --used) {
        st = st == 0 ? (ph ^= 1, kStages - 1) : st - 1;
        ok = mbar_wait_cluster(empty + st, ph ^ 1, kProductLimitNs);
      }
    }
  } else if (warp == 1) {  // ------------------------------------------ MMA
    if (lane == 0 && rank == 0) {
      int st = 0, b = 0;
      uint32_t ph = 0, pb = 1;
      for (int t = group; t < tiles && ok; t += groups) {
        ok = mbar_wait_cluster(tempty + b, pb, kProductLimitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + b * S::BN;
        const Problem& p = w.p[product_of(t)];
        const bool amn = p.amn;
        const int kblocks = p.kblocks;
        const uint32_t idesc = product_idesc<E>(kBM * CG, S::BN, amn, S::BMN);
        // 16 of a stage's 64 k: 32 bytes along a K-major row, else two 8-k groups
        const uint32_t step_a = (amn ? 2048 : 32) >> 4, step_b = (S::BMN ? 2048 : 32) >> 4;
        for (int k = 0; k < kblocks; ++k) {
          ok = mbar_wait_cluster(full + st, ph, kProductLimitNs);
          if (!ok) break;
          tc_fence_after();
          const uint64_t da = tile_desc(base + st * S::kStage, amn), db = tile_desc(base + st * S::kStage + S::kA, S::BMN);
#pragma unroll
          for (int q = 0; q < 4; ++q) pair_mma<CG>(d, da + q * step_a, db + q * step_b, idesc, k | q);
          pair_commit<CG>(empty + st);
          if (++st == kStages) st = 0, ph ^= 1;
        }
        if (ok) pair_commit<CG>(tfull + b);
        if ((b ^= 1) == 0) pb ^= 1;
      }
    }
  } else if (warp >= 4) {  // ------------------------------------ epilogue
    int b = 0;
    uint32_t pb = 0;
    for (int t = group; t < tiles && ok; t += groups) {
      ok = __all_sync(0xffffffffu, mbar_wait_cluster(tfull + b, pb, kProductLimitNs));
      if (!ok) break;
      tc_fence_after();
      const int which = product_of(t);
      int m, n;
      tile_place(which ? t - w.tiles[0] : t, w.p[which].num_m, w.p[which].num_n, m, n);
      epi.store(tmem + b * S::BN + ((uint32_t)(warp & 3) << 21), ((int64_t)m * CG + rank) * kBM + (warp & 3) * 32 + lane, n,
                which, (warp - 4) >> 2);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2) mbar_arrive_remote(mapa_shared(smem_u32(tempty + b), 0));
        else mbar_arrive(tempty + b);
      }
      if ((b ^= 1) == 0) pb ^= 1;
    }
  }
  if (!ok) {  // gave up: report, and let copies and MMAs in flight end before anything is freed
    atomicOr(w.status, 2u);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 20000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == 2) pair_tmem_dealloc<CG>(tmem, S::kCols);
}

// ------------------------------------------------------------------- host --
template <typename E>
inline bool encode_2d(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(rows == 1 ? cols : ld) * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  return encode(m, std::is_same<E, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p,
                dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// D [M, num_n tiles] of reduction length K.  A K-major operand is [rows, K], the other
// kind [K, rows]; their row strides are ld_*.
template <typename E, typename S>
inline bool problem(Problem* p, int64_t M, int64_t num_n, int64_t K, const void* a, bool amn, int64_t ld_a, const void* b,
                    int64_t rows_b, int64_t ld_b) {
  p->num_m = (int)((M + kBM * S::CG - 1) / (kBM * S::CG));
  p->num_n = (int)num_n;
  p->kblocks = (int)((K + kBK - 1) / kBK);
  p->amn = amn;
  return encode_2d<E>(&p->a, a, amn ? K : M, amn ? M : K, ld_a, amn ? 64 : kBM) &&
         encode_2d<E>(&p->b, b, S::BMN ? K : rows_b, S::BMN ? rows_b : K, ld_b, S::kBoxB);
}

template <typename E, typename S, int NP, typename Epi>
inline cudaError_t product_launch(Work<NP>& w, const Epi& epi, cudaStream_t s) {
  static SmemGrant grant;
  auto k = product_kernel<E, S, NP, Epi>;
  cudaError_t e = allow_smem(grant, (const void*)k, S::kSmem);
  if (e != cudaSuccess) return e;
  int sms = 0;
  e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  int64_t tiles = 0;
  for (int i = 0; i < NP; ++i) {
    tiles += (int64_t)w.p[i].num_m * w.p[i].num_n;
    if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
    w.tiles[i] = (int)tiles;
  }
  const int64_t groups = tiles < sms / S::CG ? tiles : sms / S::CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * S::CG));
  cfg.blockDim = dim3(kProductThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = S::CG;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k, w, epi);
  if (e != cudaSuccess) cudaGetLastError();  // it is this call's, not the next one's
  return e;
}

}  // namespace mhc
