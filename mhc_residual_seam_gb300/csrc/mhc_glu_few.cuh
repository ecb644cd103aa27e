// The gated projections of a few tokens: bound by reading the weights once.
//
// The weights are the product's rows (128 features of the gate and the same 128 of the
// other projection: two accumulators) and the tokens its 16 columns, so they cost 2 KB of
// shared memory a step, not a tile of 128 rows.  The steps (128 features x 64 columns of
// H, 32 KB of weights) of all tiles are cut into one equal run per SM: a run that ends inside
// a tile leaves fp32 sums in the workspace, and the CTA that comes last to a tile adds them
// up in the runs' order and finishes it.  No CTA waits for another one, and the sums do not
// depend on who comes last.
//
// H = 5120, F = 10240: T = 4 38.4 us against 57.4 in tiles of tokens, T = 16 38.6 against
// 41.0 (210 MB of weights are 30.9 at the copy's rate; the steps run at 7 TB/s, the rest is
// the start, 2.3 us to the first step, and the SMs' uneven ends, 3.6).  With more columns
// this form lost from 32 tokens on (T = 64 45.3 against 41.2): the parts grow with them.
#pragma once

#include "mhc_glu.cuh"
#include "mhc_product.cuh"

namespace mhc {

constexpr int kFewTokens = 16;   // most tokens of this form, columns of an accumulator
constexpr int kFewRuns = 152;    // most runs

struct FewPlan {
  int tiles, kblocks, runs;  // feature tiles, steps per tile, runs
};
inline FewPlan few_plan(int H, int F) {
  FewPlan p;
  p.tiles = (F + kBM - 1) / kBM;
  p.kblocks = (H + kBK - 1) / kBK;
  const int64_t total = (int64_t)p.tiles * p.kblocks;
  // at least four steps a run: shorter ones cost more in sums than they save
  int64_t runs = (total + 3) / 4;
  p.runs = (int)(runs < kFewRuns ? runs : kFewRuns);
  return p;
}
// Workspace: status word, a counter per tile (the same place whatever the sizes, so that
// calls of different sizes may share it), two parts per run.
constexpr size_t kFewCounters = kProductCounters, kFewParts = kProductParts;
static_assert(kFewParts - kFewCounters >= (size_t)((1 << 20) / kBM) * 4, "a counter per tile of the largest F");
constexpr size_t kFewPart = (size_t)2 * kFewTokens * kBM;  // floats of a part
constexpr int kFewStage = 2 * kBM * 128 + kFewTokens * 128, kFewStages = 5;
constexpr size_t kFewSmem = (size_t)kFewStages * kFewStage + 1024 + 256;
inline size_t few_bytes(const FewPlan& p) { return kFewParts + (size_t)p.runs * 2 * kFewPart * 4; }

template <typename E>
struct FewArgs {
  CUtensorMap w, x;
  const E* add;
  E *gu, *h;
  int64_t F, ld_add, ld_h;
  unsigned* status;
  unsigned* counters;
  float* parts;
  int T, act, tiles, kblocks;
};

constexpr int kFewEpilogue = 256;  // epilogue threads: two warps per 32 features, eight tokens each
constexpr int kFewAhead = 8;       // steps whose weights are fetched into L2 ahead of the kernel before
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1)
               : "memory");
}
template <typename E>
__global__ void __launch_bounds__(128 + kFewEpilogue, 1) glu_few_kernel(const __grid_constant__ FewArgs<E> p) {
  extern __shared__ char raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  char* aligned = raw + (base - smem_u32(raw));
  constexpr int stage_bytes = kFewStage, stages = kFewStages;
  uint64_t* full = reinterpret_cast<uint64_t*>(aligned + (size_t)stages * stage_bytes);
  uint64_t *empty = full + stages, *tfull = empty + stages, *tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile uint32_t* last = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t stride = 32, tcols = 4 * stride;  // two accumulators, twice, at multiples of 32 columns

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, kFewEpilogue / 32);
    }
    mbar_fence_init();
  }
  if (warp == 2) pair_tmem_alloc<1>(tmem_slot, tcols);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch();  // the next kernel's CTAs may take the place of those that end early

  const int64_t total = (int64_t)p.tiles * p.kblocks, runs = gridDim.x;
  const int64_t begin = blockIdx.x * total / runs, end = (blockIdx.x + 1) * total / runs;
  bool ok = true;

  if (warp == 0) {  // ------------------------------------------- producer
    if (lane == 0) {
      int st = 0, used = 0, tile = (int)(begin / p.kblocks), k = (int)(begin - (int64_t)tile * p.kblocks);
      uint32_t ph = 1;
      prefetch_tmap(&p.w);
      prefetch_tmap(&p.x);
      // While the kernel before this one ends, the first weights come as far as L2 (which also sees
      // what that kernel may still write there).
      for (int i = 0, t = tile, kk = k; i < kFewAhead && begin + i < end; ++i) {
        prefetch_tile(&p.w, kk * kBK, t * kBM);
        prefetch_tile(&p.w, kk * kBK, (int)p.F + t * kBM);
        if (++kk == p.kblocks) kk = 0, ++t;
      }
      wait_for_inputs();
      for (int64_t i = begin; i < end; ++i) {
        ok = mbar_wait(empty + st, ph, kProductLimitNs);
        if (!ok) break;
        mbar_arrive_expect_tx(full + st, stage_bytes);
        const uint32_t at = base + st * stage_bytes, bar = smem_u32(full + st);
        pair_load<1>(at, &p.w, bar, k * kBK, tile * kBM);
        pair_load<1>(at + kBM * 128, &p.w, bar, k * kBK, (int)p.F + tile * kBM);
        pair_load<1>(at + 2 * kBM * 128, &p.x, bar, k * kBK, 0);
        if (used < stages) ++used;
        if (++st == stages) st = 0, ph ^= 1;
        if (++k == p.kblocks) k = 0, ++tile;
      }
      for (; used > 0 && ok; --used) {  // the MMAs' last arrivals come before the CTA ends
        st = st == 0 ? (ph ^= 1, stages - 1) : st - 1;
        ok = mbar_wait(empty + st, ph ^ 1, kProductLimitNs);
      }
    }
  } else if (warp == 1) {  // ------------------------------------------ MMA
    if (lane == 0) {
      pdl_wait();  // (no wait with a limit begins before the kernel before this one has ended)
      const uint32_t idesc = product_idesc<E>(kBM, kFewTokens, false, false);
      int st = 0, b = 0, k = (int)(begin % p.kblocks);
      uint32_t ph = 0, pb = 1;
      for (int64_t i = begin; i < end && ok;) {
        const int n = (int)min((int64_t)(p.kblocks - k), end - i);  // steps of this run in the tile
        ok = mbar_wait(tempty + b, pb, kProductLimitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dg = tmem + b * 2 * stride, du = dg + stride;
        for (int j = 0; j < n; ++j) {
          ok = mbar_wait(full + st, ph, kProductLimitNs);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = base + st * stage_bytes;
          const uint64_t g = tile_desc(at, false), u = tile_desc(at + kBM * 128, false), x = tile_desc(at + 2 * kBM * 128, false);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            pair_mma<1>(dg, g + 2 * q, x + 2 * q, idesc, j | q);
            pair_mma<1>(du, u + 2 * q, x + 2 * q, idesc, j | q);
          }
          pair_commit<1>(empty + st);
          if (++st == stages) st = 0, ph ^= 1;
        }
        if (ok) pair_commit<1>(tfull + b);
        if ((b ^= 1) == 0) pb ^= 1;
        i += n;
        k = 0;
      }
    }
  } else if (warp >= 4) {  // ------------------------------------ epilogue
    pdl_wait();
    const int feature = (warp & 3) * 32 + lane;
    const int c = (warp - 4) >> 2 << 3;  // this warp's first token
    int b = 0, tile = (int)(begin / p.kblocks), k = (int)(begin - (int64_t)tile * p.kblocks);
    uint32_t pb = 0;
    // eight tokens of this lane's feature (what is added is fetched for all of them before it is used)
    auto finish = [&](float* g, float* u) {
      const int64_t f = (int64_t)tile * kBM + feature;
      const int n = min(8, p.T - c);
      if (f >= p.F || n <= 0) return;
      if (p.add) {
        E a[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t t = min(c + i, p.T - 1);
          a[i] = p.add[t * p.ld_add + f];
          v[i] = p.add[t * p.ld_add + p.F + f];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += (float)a[i], u[i] += (float)v[i];
      }
      if (p.gu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          E* o = p.gu + (int64_t)(c + i) * 2 * p.F + f;
          if (i < n) o[0] = (E)g[i], o[p.F] = (E)u[i];
        }
      }
      activate_product<8>(g, u, p.act);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p.h[(c + i) * p.ld_h + f] = (E)g[i];
    };
    // a part lies as four columns of a feature together, features adjacent: 16 bytes a lane
    const size_t at_g = (size_t)c * kBM + feature * 4, at_u = at_g + (size_t)kFewTokens * kBM;
    auto read8 = [&](float4* v, const float* part) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[e] = __ldcg(reinterpret_cast<const float4*>(part + at_g + (size_t)4 * e * kBM));
        v[2 + e] = __ldcg(reinterpret_cast<const float4*>(part + at_u + (size_t)4 * e * kBM));
      }
    };
    auto add8 = [&](float* g, float* u, const float4* v) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        g[4 * e] += v[e].x, g[4 * e + 1] += v[e].y, g[4 * e + 2] += v[e].z, g[4 * e + 3] += v[e].w;
        u[4 * e] += v[2 + e].x, u[4 * e + 1] += v[2 + e].y, u[4 * e + 2] += v[2 + e].z, u[4 * e + 3] += v[2 + e].w;
      }
    };
    for (int64_t i = begin; i < end && ok; ++tile) {
      const int n = (int)min((int64_t)(p.kblocks - k), end - i);
      const bool whole = n == p.kblocks;
      ok = all_of<kFewEpilogue>(mbar_wait(tfull + b, pb, kProductLimitNs));  // the warps go on, or give up, together
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + b * 2 * stride + ((uint32_t)(warp & 3) << 21);
      uint32_t gr[8], ur[8];
      __syncwarp();
      tc_ld_x8_issue(d + c, gr);
      tc_ld_x8_issue(d + stride + c, ur);
      tc_wait_ld_x8(gr);
      tc_wait_ld_x8(ur);
      if (whole) {
        finish(reinterpret_cast<float*>(gr), reinterpret_cast<float*>(ur));
      } else {
        float* mine = p.parts + ((size_t)blockIdx.x * 2 + (i != begin)) * kFewPart;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          __stcg(reinterpret_cast<uint4*>(mine + at_g + (size_t)e * kBM), make_uint4(gr[e], gr[e + 1], gr[e + 2], gr[e + 3]));
          __stcg(reinterpret_cast<uint4*>(mine + at_u + (size_t)e * kBM), make_uint4(ur[e], ur[e + 1], ur[e + 2], ur[e + 3]));
        }
      }
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty + b);
      if ((b ^= 1) == 0) pb ^= 1;
      if (!whole) {
        // the runs that share this tile: those of its first and of its last step, and all between
        const int64_t u0 = (int64_t)tile * p.kblocks, u1 = u0 + p.kblocks - 1;
        const int r0 = (int)(((u0 + 1) * runs - 1) / total), r1 = (int)(((u1 + 1) * runs - 1) / total);
        __threadfence();
        named_bar_sync(1, kFewEpilogue);
        if (threadIdx.x == 128) *last = atomicAdd(p.counters + tile, 1u) == (unsigned)(r1 - r0);
        named_bar_sync(1, kFewEpilogue);
        if (*last) {
          __threadfence();
          auto part_of = [&](int r) {
            const bool first = r * total / runs / p.kblocks == tile;  // the tile is the first of run r
            return p.parts + ((size_t)r * 2 + !first) * kFewPart;
          };
          // (a tile that is not whole has two runs at least, and seldom more than three: fetched together)
          float4 x[4], y[4], z[4];
          read8(x, part_of(r0));
          read8(y, part_of(r0 + 1));
          if (r1 > r0 + 1) read8(z, part_of(r0 + 2));
          float g[8], u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.f;
          add8(g, u, x);
          add8(g, u, y);
          if (r1 > r0 + 1) add8(g, u, z);
          for (int r = r0 + 3; r <= r1; ++r) {
            read8(x, part_of(r));
            add8(g, u, x);
          }
          finish(g, u);
          if (threadIdx.x == 128) p.counters[tile] = 0;
        }
        named_bar_sync(1, kFewEpilogue);  // (*last is read before the next tile's is written)
      }
      i += n;
      k = 0;
    }
  }
  if (!ok) {  // gave up: report, and let copies and MMAs in flight end before anything is freed
    atomicOr(p.status, 2u);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 20000000ull) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) pair_tmem_dealloc<1>(tmem, tcols);
}

template <typename E>
inline cudaError_t glu_few_launch(const void* x, int64_t ld_x, const void* w, const void* add, int64_t ld_add, int act, int64_t T,
                                  int H, int F, void* gu, void* h, int64_t ld_h, void* ws, cudaStream_t s) {
  const FewPlan plan = few_plan(H, F);
  FewArgs<E> p;
  if (!encode_2d<E>(&p.w, w, 2 * (int64_t)F, H, H, kBM) || !encode_2d<E>(&p.x, x, T, H, ld_x, kFewTokens)) return cudaErrorInvalidValue;
  p.add = static_cast<const E*>(add);
  p.gu = static_cast<E*>(gu);
  p.h = static_cast<E*>(h);
  p.F = F, p.ld_add = ld_add, p.ld_h = ld_h, p.T = (int)T, p.act = act;
  p.tiles = plan.tiles, p.kblocks = plan.kblocks;
  p.status = static_cast<unsigned*>(ws);
  p.counters = reinterpret_cast<unsigned*>(static_cast<char*>(ws) + kFewCounters);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kFewParts);
  static SmemGrant grant;
  const cudaError_t e = allow_smem(grant, (const void*)glu_few_kernel<E>, kFewSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(glu_few_kernel<E>, dim3((unsigned)plan.runs), dim3(128 + kFewEpilogue), kFewSmem, s, p);
}

}  // namespace mhc
