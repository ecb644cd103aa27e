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
// The tiles that do not fill a last round over the SMs are cut along k into equal runs
// of stages instead, one per group, done first: a run that ends inside a tile leaves fp32
// sums in the workspace, and the group that comes last to a tile adds them up in the
// runs' order and finishes it, while its next tile's products run.  Nothing waits for
// another group, and the sums do not depend on which comes last.
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
constexpr int kEpilogueThreads = 256, kProductThreads = 128 + kEpilogueThreads;  // producer, MMA, allocation, an idle warp; eight epilogue warps
constexpr uint64_t kProductLimitNs = 2000000000ull;

// ------------------------------------------------------------ PTX, pairs --
// Before the first TMA read of what the kernel before this one wrote.
__device__ __forceinline__ void wait_for_inputs() {
  pdl_wait();
  asm volatile("fence.proxy.async;" ::: "memory");
}
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
// The products of one launch: `whole` tiles of each are done as they are, the `rest` in
// `runs` runs.
template <int N>
struct Work {
  Problem p[N];
  int whole[N], rest[N];
  int runs, units;  // units: stages of all the rest
  unsigned *status, *counters;
  float* parts;
};

// A stretch of stages k0 .. k0 + nk of one tile.
struct Stretch {
  int which, m, n, k0, nk;
  int tile, begin;  // of the rest: its number, and its first unit
  bool all;         // the whole tile
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

// The stretches of one group, in order; each role of the kernel goes through them.
template <int N>
struct Walk {
  const Work<N>& w;
  int at, end;  // units of this group's run that are left
  int t, step;  // next whole tile
  __device__ __forceinline__ Walk(const Work<N>& work, int group, int groups) : w(work), at(0), end(0), t(group), step(groups) {
    if (group < w.runs) {
      at = (int)((int64_t)group * w.units / w.runs);
      end = (int)((int64_t)(group + 1) * w.units / w.runs);
    }
  }
  __device__ __forceinline__ bool next(Stretch& s) {
    int index;
    if (at < end) {
      const int units0 = w.rest[0] * w.p[0].kblocks;
      s.which = N == 2 && at >= units0 ? N - 1 : 0;
      const int before = s.which ? units0 : 0, kb = w.p[s.which].kblocks, i = (at - before) / kb;
      s.begin = before + i * kb;
      s.k0 = at - s.begin;
      s.nk = min(kb - s.k0, end - at);
      s.tile = (s.which ? w.rest[0] : 0) + i;
      index = w.whole[s.which] + i;
      at += s.nk;
    } else {
      index = t;
      s.which = 0;
      if (N == 2 && t >= w.whole[0]) s.which = N - 1, index -= w.whole[0];
      if (index >= w.whole[s.which]) return false;
      s.k0 = 0;
      s.nk = w.p[s.which].kblocks;
      t += step;
    }
    s.all = s.nk == w.p[s.which].kblocks;
    tile_place(index, w.p[s.which].num_m, w.p[s.which].num_n, s.m, s.n);
    return true;
  }
  // The run that has unit u.
  __device__ __forceinline__ int run_of(int u) const { return (int)(((int64_t)(u + 1) * w.runs - 1) / w.units); }
};

// Where an epilogue finds 16 columns of its lane's row: in tensor memory, or as the sum of
// a cut tile's parts.  A part lies as four columns of a row together, rows adjacent.
struct FromTmem {
  uint32_t at;
  __device__ __forceinline__ void get(int c, float* v) const {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    __syncwarp();
    issue16(at + c, r);
    take16(r);
  }
  __device__ __forceinline__ void get2(int c, float* v, int d, float* u) const {
    uint32_t *r = reinterpret_cast<uint32_t*>(v), *q = reinterpret_cast<uint32_t*>(u);
    __syncwarp();
    issue16(at + c, r);
    issue16(at + d, q);
    take16(r);
    take16(q);
  }
};
struct FromParts {
  const float* first;  // run r0's part, this lane's row
  const float* next;   // run r0 + 1's: the tile is its first, as for the runs after it
  size_t stride;       // from a run to the one after the next
  int more;            // runs after r0 + 1
  __device__ __forceinline__ static void read(float4* x, const float* p, int c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __ldcg(reinterpret_cast<const float4*>(p + (size_t)(c + 4 * e) * kBM));
  }
  __device__ __forceinline__ static void add(float* v, const float4* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * e] += x[e].x, v[4 * e + 1] += x[e].y, v[4 * e + 2] += x[e].z, v[4 * e + 3] += x[e].w;
  }
  // (all that is fetched here is fetched before any of it is added: the time is the loads' latency)
  __device__ __forceinline__ void get(int c, float* v) const {
    float4 x[4], y[4], z[4];
    read(x, first, c);
    read(y, next, c);
    if (more > 0) read(z, next + stride, c);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
    add(v, x);
    add(v, y);
    if (more > 0) add(v, z);
    for (int i = 2; i <= more; ++i) {
      read(x, next + i * stride, c);
      add(v, x);
    }
  }
  __device__ __forceinline__ void get2(int c, float* v, int d, float* u) const {
    float4 x[4], y[4], p[4], q[4];
    read(x, first, c);
    read(p, first, d);
    read(y, next, c);
    read(q, next, d);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = u[e] = 0.f;
    add(v, x);
    add(u, p);
    add(v, y);
    add(u, q);
    for (int i = 1; i <= more; i += 2) {
      const float *a = next + i * stride, *b = a + stride;
      read(x, a, c);
      read(p, a, d);
      if (i < more) {
        read(y, b, c);
        read(q, b, d);
      }
      add(v, x);
      add(u, p);
      if (i < more) {
        add(v, y);
        add(u, q);
      }
    }
  }
};

// Barrier 1 over THREADS threads; whether `x` holds in all of them.
template <int THREADS>
__device__ __forceinline__ bool all_of(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(THREADS)
      : "memory");
  return r != 0;
}

// Epi: `row_b(n_tile, j)` is the row of B for column j of the tile; `store(source,
// row, n_tile, product, half)` makes a lane's row of outputs, every other 16 columns.
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
  volatile uint32_t* last = tmem_slot + 1;
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
  pdl_launch();  // the next kernel's CTAs may take the place of those that end early

  const int groups = gridDim.x / CG, group = blockIdx.x / CG;
  Walk<NP> walk(w, group, groups);
  Stretch s;
  bool ok = true;

  if (warp == 0) {  // ------------------------------------------- producer
    if (lane == 0) {
      wait_for_inputs();
      int st = 0, used = 0;
      uint32_t ph = 1;
      while (ok && walk.next(s)) {
        const Problem& p = w.p[s.which];
        const int row = (s.m * CG + (int)rank) * kBM;
        for (int k = s.k0; k < s.k0 + s.nk; ++k) {
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
            const int rb = epi.row_b(s.n, (int)rank * S::kRowsB + j);
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
      pdl_wait();  // (no wait with a limit begins before the kernel before this one has ended)
      int st = 0, b = 0;
      uint32_t ph = 0, pb = 1;
      while (ok && walk.next(s)) {
        ok = mbar_wait_cluster(tempty + b, pb, kProductLimitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + b * S::BN;
        const bool amn = w.p[s.which].amn;
        const uint32_t idesc = product_idesc<E>(kBM * CG, S::BN, amn, S::BMN);
        // 16 of a stage's 64 k: 32 bytes along a K-major row, else two 8-k groups
        const uint32_t step_a = (amn ? 2048 : 32) >> 4, step_b = (S::BMN ? 2048 : 32) >> 4;
        for (int k = 0; k < s.nk; ++k) {
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
    pdl_wait();
    const int half = (warp - 4) >> 2, in_tile = (warp & 3) * 32 + lane;
    constexpr size_t kPart = (size_t)kBM * S::BN;
    while (walk.next(s)) {
      ok = all_of<kEpilogueThreads>(mbar_wait_cluster(tfull + b, pb, kProductLimitNs));  // the warps go on, or give up, together
      if (!ok) break;
      tc_fence_after();
      const FromTmem tile = {tmem + b * S::BN + ((uint32_t)(warp & 3) << 21)};
      const int64_t row = ((int64_t)s.m * CG + rank) * kBM + in_tile;
      if (s.all) {
        epi.store(tile, row, s.n, s.which, half);
      } else {
        const bool is_first = s.begin <= (int)((int64_t)group * w.units / w.runs);
        float* mine = w.parts + ((size_t)(group * 2 + !is_first) * CG + rank) * kPart + in_tile * 4;
        for (int c = half * 16; c < S::BN; c += 32) {
          float v[16];
          tile.get(c, v);
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            __stcg(reinterpret_cast<float4*>(mine + (size_t)(c + e) * kBM), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
        }
      }
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2) mbar_arrive_remote(mapa_shared(smem_u32(tempty + b), 0));
        else mbar_arrive(tempty + b);
      }
      if ((b ^= 1) == 0) pb ^= 1;
      if (!s.all) {
        const int r0 = walk.run_of(s.begin), r1 = walk.run_of(s.begin + w.p[s.which].kblocks - 1);
        unsigned* counter = w.counters + s.tile * CG + rank;
        __threadfence();
        named_bar_sync(1, kEpilogueThreads);
        if (threadIdx.x == 128) *last = atomicAdd(counter, 1u) == (unsigned)(r1 - r0);
        named_bar_sync(1, kEpilogueThreads);
        if (*last) {
          __threadfence();
          const bool whole_run = s.begin <= (int)((int64_t)r0 * w.units / w.runs);  // run r0 begins in the tile
          const float* at = w.parts + rank * kPart + in_tile * 4;
          const FromParts sum = {at + (size_t)(r0 * 2 + !whole_run) * CG * kPart, at + (size_t)(r0 + 1) * 2 * CG * kPart,
                                 2 * CG * kPart, r1 - r0 - 1};
          epi.store(sum, row, s.n, s.which, half);
          if (threadIdx.x == 128) *counter = 0;
        }
        named_bar_sync(1, kEpilogueThreads);  // (*last is read before the next tile's is written)
      }
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

// Workspace of the products: the status word, counters of cut tiles, two parts per group.
constexpr int kMostSms = 152;
constexpr size_t kProductCounters = 256, kProductParts = kProductCounters + 32768;
constexpr size_t kProductBytes = kProductParts + (size_t)kMostSms * 2 * kBM * 256 * 4;

// How the tiles of one or two products (n[i] tiles of kb[i] stages) are done by `groups`
// groups: whole rounds, and the rest of each cut into runs where that takes fewer stages (a
// tile of fewer than kShort is mostly its end, and is not cut).  A tile has eight parts at
// most, four where large tiles come after it: its last group reads them one after another.
// What a cut costs, in stages: a few (its sums' way through L2); and, as far as no whole tiles
// after it hide that, five and three for each part where each run is a part of one tile,
// thirty where runs end anywhere, both twice for the large tiles.
struct ProductPlan {
  int64_t whole[2], rest[2], units, runs;
  int64_t stages;  // of the group that has the most
};
inline ProductPlan product_plan(int products, const int64_t* n, const int64_t* kb, int groups) {
  constexpr int kLeast = 4, kShort = 16, kEnd = 8;
  const int large = groups <= kMostSms / 2 ? 2 : 1;
  ProductPlan p = {};
  int64_t tiles = 0, longest = 0, last = 0, rounds = 0, all = 0;
  for (int i = 0; i < products; ++i) {
    all += n[i];
    if (kb[i] < kShort) {
      p.whole[i] = n[i];
      rounds += (n[i] + groups - 1) / groups * (kb[i] > kEnd ? kb[i] : kEnd);
      continue;
    }
    p.whole[i] = n[i] / groups * groups;
    p.rest[i] = n[i] - p.whole[i];
    rounds += n[i] / groups * kb[i];
    p.units += p.rest[i] * kb[i];
    tiles += p.rest[i];
    if (p.rest[i] && kb[i] > longest) longest = kb[i];
    last = kb[i];
  }
  p.stages = rounds;
  if (p.units == 0) return p;
  const int kParts = rounds && large == 2 ? 4 : 8;
  // as whole tiles: the longest come first, a second round where there are more than groups
  const int64_t uncut = all <= groups ? longest - rounds : tiles > groups ? longest + last : longest;
  auto cost = [&](int64_t each, int64_t join) { return each + 6 + (join > rounds ? join - rounds : 0); };
  int64_t cut = uncut + 1;
  if (p.units <= 0x3fffffff) {
    const bool alone = p.units == tiles * longest;  // tiles of one length
    int64_t parts = groups / tiles < kParts ? groups / tiles : kParts;
    if (parts > longest / kLeast) parts = longest / kLeast;
    if (alone && parts >= 2) {
      p.runs = tiles * parts;
      cut = cost((longest + parts - 1) / parts, (5 + 3 * parts) * large);
    } else {
      p.runs = (p.units + kLeast - 1) / kLeast;
      if (p.runs > kParts * p.units / longest) p.runs = kParts * p.units / longest;
      if (p.runs > groups) p.runs = groups;
      if (p.runs < 1) p.runs = 1;
      cut = cost((p.units + p.runs - 1) / p.runs, 30 * large);
    }
  }
  if (cut >= uncut) {
    for (int i = 0; i < products; ++i) p.whole[i] += p.rest[i], p.rest[i] = 0;
    p.units = p.runs = 0;
    cut = uncut;
  }
  p.stages = rounds + cut;
  return p;
}

// Whether tiles of 128 x 128 (a CTA each) take less time than tiles of 256 x 256 (a pair):
// stages times a stage's time, in hundredths of the large tile's 0.3 us, and what the start and
// the last tile's end cost beside them.  T = 8192, H = 5120, F = 10240 takes the gated projections
// 855 us in large tiles and 1273 in small ones; T = 300, H = 512, F = 1368 9.4 and 7.2.
template <typename Tiles>
inline bool product_small(const Tiles& tiles, int products) {
  int64_t n[2], kb[2], large, small;
  for (int i = 0; i < products; ++i) tiles(i, 256, 256, n + i, kb + i);
  large = product_plan(products, n, kb, kMostSms / 2).stages * 100 + 1300;
  for (int i = 0; i < products; ++i) tiles(i, 128, 128, n + i, kb + i);
  small = product_plan(products, n, kb, kMostSms).stages * 74 + 600;
  return small < large;
}

template <typename E, typename S, int NP, typename Epi>
inline cudaError_t product_launch(Work<NP>& w, void* ws, const Epi& epi, cudaStream_t s) {
  static SmemGrant grant;
  auto k = product_kernel<E, S, NP, Epi>;
  cudaError_t e = allow_smem(grant, (const void*)k, S::kSmem);
  if (e != cudaSuccess) return e;
  int sms = 0;
  e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int most = (sms < kMostSms ? sms : kMostSms) / S::CG;
  int64_t n[2], kb[2], tiles = 0;
  for (int i = 0; i < NP; ++i) {
    n[i] = (int64_t)w.p[i].num_m * w.p[i].num_n, kb[i] = w.p[i].kblocks;
    tiles += n[i];
    if (n[i] > 0x3fffffff) return cudaErrorInvalidValue;
  }
  const ProductPlan plan = product_plan(NP, n, kb, most);
  for (int i = 0; i < NP; ++i) w.whole[i] = (int)plan.whole[i], w.rest[i] = (int)plan.rest[i];
  w.units = (int)plan.units, w.runs = (int)plan.runs;
  const int64_t groups = plan.runs == 0 ? (tiles < most ? tiles : most) : (plan.whole[0] + plan.whole[NP - 1] == 0 ? plan.runs : most);
  w.status = static_cast<unsigned*>(ws);
  w.counters = reinterpret_cast<unsigned*>(static_cast<char*>(ws) + kProductCounters);
  w.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kProductParts);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * S::CG));
  cfg.blockDim = dim3(kProductThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = S::CG;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, k, w, epi);
  if (e != cudaSuccess) cudaGetLastError();  // it is this call's, not the next one's
  return e;
}

}  // namespace mhc
