// mhc_lora: low-rank adapters of many requests beside a shared projection.
//
//   v[t,:] = A_a x[t],  out[t,:] = base[t,:] + s_a B_a v[t],  a = index[t]
//
// The work is bound by memory (x and base read once, out written once, an adapter's
// weights once per unit).  A unit is up to 64 tokens of one adapter.
//   plan    (more than 64 tokens) sorts runs of 1024 tokens by adapter and cuts them into
//           units, so that tokens in any order share their adapter's weights
//   shrink  v of a unit: a cluster of CTAs shares H, its sums meet in shared memory
//   expand  B v, the scale and base: 32 columns a warp at a time on mma.sync, or, for
//           larger ranks of many tokens, 128 columns a CTA on tcgen05 (lora_wide_kernel)
// With up to 64 tokens each CTA finds its unit by itself.
//
// On mma.sync the order of a product's reduction index and of its columns is free, so
// each thread's fragment is taken from adjacent elements, in pieces of 8 and 16 bytes.

#include <type_traits>

#include "mhc_product.cuh"

namespace mhc {

constexpr int kTok = 64;     // most tokens of a unit
constexpr int kRun = 1024;   // tokens sorted together
constexpr int kMostParts = 8;
constexpr int kExpandCtas = 5;  // per SM, about

struct Unit {
  int adapter;  // -1: tokens without one
  int first;    // in the sorted order
  int count;
  int pad;
};
struct LoraPlan {
  const int* order;   // sorted order -> token; NULL: units are found in the kernel
  const Unit* units;  // kRun per run of tokens
  const int* made;    // units of a run
  int runs;
};

__device__ __forceinline__ int adapter_of(const int* index, int64_t t, int64_t T, int n) {
  if (t >= T) return -2;
  const int i = index[t];
  return i >= 0 && i < n ? i : -1;
}

// ---------------------------------------------------------------- the plan --
// A thread per token: bitonic sort of (adapter, place) words, stable because the place is
// part of them; then the first token of each 64 of an adapter starts a unit.
__global__ void __launch_bounds__(kRun) lora_plan_kernel(const int* index, int64_t T, int n, int* __restrict__ order,
                                                         Unit* __restrict__ units, int* __restrict__ made) {
  __shared__ uint32_t word[2][kRun];
  __shared__ int starts[kRun + 1], last[32], found[32];
  pdl_wait_for(index);
  pdl_launch();
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * kRun;
  const int m = (int)min((int64_t)kRun, T - t0);
  const int id = adapter_of(index, t0 + i, T, n);
  uint32_t key = id == -2 ? 0xffffffffu : ((uint32_t)(id < 0 ? n : id) << 10) | i;
  int side = 0;  // two copies in turn: one barrier an exchange
#pragma unroll
  for (int k = 2; k <= kRun; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      uint32_t other;
      if (j >= 32) {
        word[side][i] = key;
        __syncthreads();
        other = word[side][i ^ j];
        side ^= 1;
      } else {
        other = __shfl_xor_sync(0xffffffffu, key, j);
      }
      const bool low = (i & j) == 0, up = (i & k) == 0;
      key = low == up ? min(key, other) : max(key, other);
    }
  word[side][i] = key;
  __syncthreads();
  const bool live = i < m;
  const int a = (int)(key >> 10);
  // where this adapter's tokens begin: the last start at or before this place
  int begin = live && (i == 0 || (int)(word[side][max(i - 1, 0)] >> 10) != a) ? i : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, begin, d);
    if (lane >= d) begin = max(begin, o);
  }
  if (lane == 31) last[warp] = begin;
  __syncthreads();
  int earlier = lane < warp ? last[lane] : 0;
#pragma unroll
  for (int d = 16; d; d >>= 1) earlier = max(earlier, __shfl_xor_sync(0xffffffffu, earlier, d));
  begin = max(begin, earlier);
  const bool starts_unit = live && (i - begin) % kTok == 0;
  const unsigned b = __ballot_sync(0xffffffffu, starts_unit);
  if (lane == 0) found[warp] = __popc(b);
  __syncthreads();
  const int theirs = found[lane];
  int before = lane < warp ? theirs : 0, total = theirs;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    total += __shfl_xor_sync(0xffffffffu, total, d);
  }
  const int u = before + __popc(b & ((1u << lane) - 1));
  if (starts_unit) starts[u] = i;
  if (i == 0) starts[total] = m, made[blockIdx.x] = total;
  __syncthreads();
  if (live) order[t0 + i] = (int)t0 + (int)(key & (kRun - 1));
  if (starts_unit) units[t0 + u] = {a == n ? -1 : a, (int)t0 + i, starts[u + 1] - i, 0};
}

// ------------------------------------------------------------ finding units --
// With up to 64 tokens: their different adapters in order of appearance, and the tokens of
// one of them.  Made by warp 0, which holds the adapters in two registers a lane (-2: past
// the last token).
struct TileTokens {
  int firsts[kTok], rows[kTok];
  int distinct, count;
};
__device__ __forceinline__ void find_adapters(TileTokens& tile, int id0, int id1, int lane) {
  const unsigned all = 0xffffffffu, below = (1u << lane) - 1;
  // (every lane takes part in every exchange: none of them stands behind a condition)
  const unsigned same0 = __match_any_sync(all, id0) & below, same1 = __match_any_sync(all, id1) & below;
  bool seen = false;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int other = __shfl_sync(all, id0, j);
    seen |= other == id1;
  }
  const bool f0 = id0 != -2 && same0 == 0, f1 = id1 != -2 && same1 == 0 && !seen;
  const unsigned b0 = __ballot_sync(all, f0), b1 = __ballot_sync(all, f1);
  if (f0) tile.firsts[__popc(b0 & below)] = id0;
  if (f1) tile.firsts[__popc(b0) + __popc(b1 & below)] = id1;
  if (lane == 0) tile.distinct = __popc(b0) + __popc(b1);
  __syncwarp();
}
__device__ __forceinline__ void find_tokens(TileTokens& tile, int id, int id0, int id1, int lane) {
  const unsigned all = 0xffffffffu, below = (1u << lane) - 1;
  const unsigned b0 = __ballot_sync(all, id0 == id), b1 = __ballot_sync(all, id1 == id);
  if (id0 == id) tile.rows[__popc(b0 & below)] = lane;
  if (id1 == id) tile.rows[__popc(b0) + __popc(b1 & below)] = lane + 32;
  if (lane == 0) tile.count = __popc(b0) + __popc(b1);
}
// The units of this CTA, every gridDim.x-th, one after another: `next` is called by all
// threads and leaves the tokens in tile.rows (a barrier before the rows are used, and one
// before the next call, are part of it).
struct Units {
  TileTokens& tile;
  const LoraPlan& plan;
  int id0, id1;
  int64_t at, before;  // the next unit; units of the runs before `run`
  int run, made;
  __device__ __forceinline__ Units(TileTokens& t, const LoraPlan& p, const int* index, int64_t T, int n)
      : tile(t), plan(p), id0(0), id1(0), at(blockIdx.x), before(0), run(0), made(0) {
    const int lane = threadIdx.x & 31;
    if (plan.order) {
      made = plan.made[0];
    } else {
      id0 = adapter_of(index, lane, T, n), id1 = adapter_of(index, lane + 32, T, n);
      if (threadIdx.x < 32) find_adapters(tile, id0, id1, lane);
    }
  }
  __device__ __forceinline__ bool next(int& adapter, int& count) {
    __syncthreads();
    if (plan.order) {
      while (at >= before + made) {
        if (++run >= plan.runs) return false;
        before += made;
        made = plan.made[run];
      }
      const Unit unit = plan.units[(int64_t)run * kRun + (at - before)];
      if (threadIdx.x < unit.count) tile.rows[threadIdx.x] = plan.order[unit.first + threadIdx.x];
      adapter = unit.adapter, count = unit.count;
      __syncthreads();
    } else {
      if (at >= tile.distinct) return false;
      adapter = tile.firsts[at];
      if (threadIdx.x < 32) find_tokens(tile, adapter, id0, id1, threadIdx.x);
      __syncthreads();
      count = tile.count;
    }
    at += gridDim.x;
    return true;
  }
};

// ---------------------------------------------------------------- products --
// 16 bytes from `src`, or zeros (then `any` stands in for the address).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void* src, const void* any, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(take ? src : any), "r"(take ? 16 : 0) : "memory");
}
template <typename E>
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<E, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory of a shrink CTA: a ring of stages (64 columns of 64 tokens and of 8 NT of the
// rank), and the sums [64, R rounded up to 16, plus 4], twice: in the ring's place where one
// pass makes the whole rank.
constexpr int kShrinkStages = 4;
template <int NT>
__host__ __device__ constexpr int stage_bytes() {
  return (kTok + NT * 8) * 128;
}
__host__ __device__ constexpr int sums_stride(int R) { return (R + 15) / 16 * 16 + 4; }
template <int NT>
__host__ __device__ constexpr size_t shrink_smem(int R) {
  const size_t sums = (size_t)kTok * sums_stride(R) * 4, ring = kShrinkStages * stage_bytes<NT>();
  return R > NT * 8 ? ring + sums : ring > 2 * sums ? ring : 2 * sums;
}

// acc = the sums of a warp's 16 MG tokens over columns [k0, k1).  All warps fetch a stage
// (cp.async, whole lines of 128 bytes), some stages ahead; a warp takes one half of a stage's
// columns.  16-byte pieces of odd rows lie four further, so that the eight lanes that read
// together meet no bank twice.  T = 8192, H = 5120: rank 16 23 us, rank 64 40, bound by the
// time that a stage takes to come (1.7 to 2.3 us) and the few that fit an SM.
template <typename E, int NT, int MG>
__device__ __forceinline__ void shrink_sums(float (&acc)[MG][NT][4], const E* x, int64_t ld_x, const int* rows, int count, const E* a,
                                            int left, int H, int k0, int k1, uint32_t ring, int m, int half, bool busy) {
  const int lane = threadIdx.x & 31, q = lane & 3, g = lane >> 2;
  // the pieces that this thread fetches: rows tid / 8 + 16 j, columns 8 (tid % 8)
  const int row = threadIdx.x >> 3, c = threadIdx.x & 7;
  const uint32_t put = (row * 8 + (c ^ ((row & 1) << 2))) * 16;
  const E* px[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) px[j] = x + (int64_t)rows[row + 16 * j < count ? row + 16 * j : 0] * ld_x + c * 8;
  const E* pa = a + (int64_t)row * H + c * 8;
  const int64_t row16 = (int64_t)16 * H;
  auto fetch = [&](int slot, int k) {
    const uint32_t at = ring + slot * stage_bytes<NT>() + put;
    const bool in = k + c * 8 < k1;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (16 * j < count) cp_async16_or_zero(at + j * 2048, px[j] + k, x, in);
#pragma unroll
    for (int j = 0; j < (NT + 1) / 2; ++j)
      if (row + 16 * j < NT * 8 && row + 16 * j < left) cp_async16_or_zero(at + kTok * 128 + j * 2048, pa + j * row16 + k, x, in);
  };
  int ahead = k0, filled = 0, slot = 0;
#pragma unroll
  for (int i = 0; i < kShrinkStages - 1; ++i, ahead += 64) {
    if (ahead < k1) fetch(i, ahead);
    cp_async_commit();
  }
  filled = kShrinkStages - 1;
  const uint32_t lane_at = g * 128 + (((half & 1) * 4 + q) ^ ((g & 1) << 2)) * 16;
  for (int k = k0; k < k1; k += 64) {
    cp_async_wait<kShrinkStages - 2>();
    __syncthreads();  // the stage is here, and the one before it has been read by all
    if (ahead < k1) fetch(filled, ahead);
    cp_async_commit();
    ahead += 64;
    if (++filled == kShrinkStages) filled = 0;
    if (busy) {
      const uint32_t at = ring + slot * stage_bytes<NT>() + lane_at;
      uint4 b[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) b[i] = lds16(at + kTok * 128 + i * 1024);
#pragma unroll
      for (int j = 0; j < MG; ++j) {
        const uint4 u = lds16(at + (m * MG + j) * 2048), w = lds16(at + (m * MG + j) * 2048 + 1024);
#pragma unroll
        for (int i = 0; i < NT; ++i) mma16816<E>(acc[j][i], u.x, w.x, u.y, w.y, b[i].x, b[i].y);
#pragma unroll
        for (int i = 0; i < NT; ++i) mma16816<E>(acc[j][i], u.z, w.z, u.w, w.w, b[i].z, b[i].w);
      }
    }
    if (++slot == kShrinkStages) slot = 0;
  }
  cp_async_wait<0>();
  __syncthreads();  // (the sums may take the ring's place)
}

__device__ __forceinline__ float4 lds_cluster(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// A unit's sums, [token][rank] fp32 at `at` in each CTA of the cluster (and, with `apart`, the
// other half's behind them), into v and the factors.
template <typename E>
__device__ __forceinline__ void join_rows(uint32_t at, bool apart, int stride, float s, const int* rows, int count, int R, int warp,
                                          uint4* vq, float* factor) {
  const int lane = threadIdx.x & 31, chunks = (R + 15) / 16, parts = gridDim.z, part = blockIdx.z;
  // this CTA's share of the rows, eight lanes a row, four of the rank a lane and step
  for (int r0 = part * 16; r0 < count; r0 += parts * 16) {
    const int row = r0 + warp * 4 + (lane >> 3), l = lane & 7;
    float4 z[8];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 32 + l * 4;
      z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < count && r < R)
        for (int p = 0; p < parts; ++p) {
          const uint32_t from = mapa_shared(at + (row * stride + r) * 4, p);
          const float4 y = lds_cluster(from);
          z[i] = make_float4(z[i].x + y.x, z[i].y + y.y, z[i].z + y.z, z[i].w + y.w);
          if (apart) {
            const float4 w = lds_cluster(from + kTok * stride * 4);
            z[i] = make_float4(z[i].x + w.x, z[i].y + w.y, z[i].z + w.z, z[i].w + w.w);
          }
        }
      for (float y : {z[i].x, z[i].y, z[i].z, z[i].w})
        if (fabsf(y) <= 3e38f) most = fmaxf(most, fabsf(y));
    }
#pragma unroll
    for (int d = 4; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    // 2^e of the largest, from its exponent bits; rows of zeros and of subnormals stay as they are
    const uint32_t e = __float_as_uint(most) >> 23;
    const bool plain = e < 16 || e > 238;
    const float down = plain ? 1.f : __uint_as_float((254 - e) << 23), up = plain ? 1.f : __uint_as_float(e << 23);
    if (row < count) {
      const int64_t t = rows[row];
      if (l == 0) factor[t] = s * up;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * 32 + l * 4;
        if (r >= chunks * 16) break;
        const float2 w[2] = {{z[i].x * down, z[i].y * down}, {z[i].z * down, z[i].w * down}};
        uint32_t big[2], rest[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          big[p] = word_of(w[p].x, w[p].y, E());
          const float2 f = pair_of(big[p], E());
          // (an infinite value has no rest)
          rest[p] = word_of(fabsf(f.x) <= 3e38f ? w[p].x - f.x : 0.f, fabsf(f.y) <= 3e38f ? w[p].y - f.y : 0.f, E());
        }
        vq[t * chunks * 4 + r / 4] = make_uint4(big[0], big[1], rest[0], rest[1]);
      }
    }
  }
}

// v of the units, as the second product takes it.  The CTAs of a cluster (blockIdx.z) share
// the columns of H; eight NT of the rank at a time.  The sums are joined in a fixed order.
//
// v is fp32 and B has 16 bits: each v is kept as two 16-bit values (its rounding and the
// rounding of the rest, 16 or 22 bits together), and both are multiplied.  A row is first
// brought to about 1 by a power of two, so that fp16 neither overflows nor loses the rest to
// subnormals; `factor` takes it back, with the adapter's scale.  Layout [token][16 of the
// rank][4 adjacent of them: four roundings, four rests].
template <typename E, int NT>
__global__ void __launch_bounds__(128, NT == 16 ? 2 : NT == 8 ? 3 : 4) lora_shrink_kernel(const E* x, int64_t ld_x, const E* a,
                                                          const int* index, const float* scale,
                                                          const LoraPlan plan, int64_t T, int H, int R, int n, int slice,
                                                          uint4* __restrict__ vq, float* __restrict__ factor) {
  extern __shared__ __align__(16) char smem[];
  __shared__ TileTokens tile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, g = lane >> 2;
  const int stride = sums_stride(R);
  float* sums = reinterpret_cast<float*>(R <= NT * 8 ? smem : smem + kShrinkStages * stage_bytes<NT>());
  const int k0 = blockIdx.z * slice, k1 = min(H, k0 + slice);
  pdl_wait_for(x, a, index, scale);
  pdl_launch();
  Units units(tile, plan, index, T, n);
  int id, count;
  while (units.next(id, count)) {
    if (id < 0) continue;
    // two warps take the tokens (16 or 32 each, one warp where there are 16 at most), twice for
    // the halves of a stage's columns
    const int groups = count <= 16 ? 1 : 2, m = warp % groups, half = warp / groups;
    const bool apart = R <= NT * 8;  // room for the sums of both halves
    for (int r0 = 0; r0 < R; r0 += NT * 8) {
      auto go = [&](auto tokens) {
        constexpr int MG = decltype(tokens)::value;
        const bool busy = half < 2 && m * 16 * MG < count;
        float acc[MG][NT][4];
#pragma unroll
        for (int j = 0; j < MG; ++j)
#pragma unroll
          for (int i = 0; i < NT; ++i) acc[j][i][0] = acc[j][i][1] = acc[j][i][2] = acc[j][i][3] = 0.f;
        shrink_sums<E, NT, MG>(acc, x, ld_x, tile.rows, count, a + ((int64_t)id * R + r0) * H, R - r0, H, k0, k1, smem_of(smem), m, half,
                               busy);
        for (int p = 0; p < 2; ++p) {  // the first half's sums, then the second's
          if (busy && half == p) {
#pragma unroll
            for (int j = 0; j < MG; ++j) {
              float* mine = sums + (apart ? p * kTok * stride : 0) + ((m * MG + j) * 16 + g) * stride + r0 + 2 * q;
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                if (r0 + i * 8 + 2 * q >= R) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float2* o = reinterpret_cast<float2*>(mine + 8 * h * stride + i * 8);
                  float2 z = make_float2(acc[j][i][2 * h], acc[j][i][2 * h + 1]);
                  if (!apart && p) z = make_float2(o->x + z.x, o->y + z.y);
                  *o = z;
                }
              }
            }
          }
          if (!apart) __syncthreads();
        }
      };
      if (count <= 32) go(std::integral_constant<int, 1>());
      else go(std::integral_constant<int, 2>());
    }
    __syncwarp();
    cluster_sync_all();
    join_rows<E>(smem_of(sums), apart, stride, scale ? scale[id] : 1.f, tile.rows, count, R, warp, vq, factor);
    __syncwarp();
    cluster_sync_all();  // (the sums are read before the next unit's, or the CTA's end)
  }
}

// 32 columns from c0 of a unit's rows, by one warp.  `frag` holds v as the products take
// it, [16 tokens][16 of the rank][lane]: four registers of roundings, four of rests.
// lane_w points at the lane's first weights; column of fragment column 2 p + e of product
// i: 8 p + 2 i + e, so a thread's eight results of a row are adjacent.
//
// With all 32 columns and a rank of at most 16 CH little is tested but the stores, and rows past
// the unit's last stand in as its first.  The warp keeps the weights of its columns in
// registers for all the tokens and fetches a group's base while the one before it is
// multiplied.
template <typename E, int CH, bool BASE>
__device__ __forceinline__ void expand_full(const uint4* frag, const float* factor, const E* lane_w, int R, const E* base, int64_t ld_b,
                                            E* out, int64_t ld_o, const int* rows, int count, int col, int lane) {
  const int g = lane >> 2, chunks = (R + 15) / 16, left = R - (lane & 3) * 4;
  uint2 w[CH][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < CH; ++c)
      w[c][i] = c * 16 < left ? *reinterpret_cast<const uint2*>(lane_w + 2 * i * R + c * 16) : make_uint2(0, 0);
  const int groups = (count + 15) / 16;
  base += col;
  out += col;
  Raw8<E> old[2][2];
  auto fetch = [&](Raw8<E>* o, int m) {
    if constexpr (BASE) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = m * 16 + g + 8 * h;
        o[h] = ld8_stream(base + rows[row < count ? row : 0] * ld_b);
      }
    }
  };
  auto group = [&](const Raw8<E>* o, int m) {
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    const uint4* f = frag + (m * chunks * 32 + lane) * 2;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (c >= chunks) break;
      const uint4 big = f[c * 64], rest = f[c * 64 + 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) mma16816<E>(acc[i], big.x, big.y, big.z, big.w, w[c][i].x, w[c][i].y);
#pragma unroll
      for (int i = 0; i < 4; ++i) mma16816<E>(acc[i], rest.x, rest.y, rest.z, rest.w, w[c][i].x, w[c][i].y);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = m * 16 + g + 8 * h;
      const float2 k = splat(factor[row]);
      Vec8 y = zero8();
      if constexpr (BASE) y = unpack(o[h]);
#pragma unroll
      for (int e = 0; e < 4; ++e) y.p[e] = __ffma2_rn(k, make_float2(acc[e][2 * h], acc[e][2 * h + 1]), y.p[e]);
      if (row < count) st8_stream(out + rows[row] * ld_o, pack<E>(y));
    }
  };
  fetch(old[0], 0);
  for (int m = 0; m < groups; m += 2) {
    if (m + 1 < groups) fetch(old[1], m + 1);
    group(old[0], m);
    if (m + 1 < groups) {
      if (m + 2 < groups) fetch(old[0], m + 2);
      group(old[1], m + 1);
    }
  }
}
// The same with every test, for what is left.
template <typename E>
__device__ __forceinline__ void expand_any(const uint4* frag, const float* factor, const E* lane_w, int id, int N, int R, const E* base,
                                           int64_t ld_b, E* out, int64_t ld_o, const int* rows, int count, int c0, int lane) {
  const int chunks = (R + 15) / 16, g = lane >> 2, q = lane & 3, col = c0 + q * 8;
  for (int m = 0; m * 16 < count; ++m) {
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    for (int c = 0; id >= 0 && c < chunks; ++c) {
      const uint4* f = frag + ((m * chunks + c) * 32 + lane) * 2;
      const uint4 big = f[0], rest = f[1];
      uint2 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = make_uint2(0, 0);
        if (c0 + (g >> 1) * 8 + 2 * i + (g & 1) < N && c * 16 + q * 4 < R)
          w[i] = *reinterpret_cast<const uint2*>(lane_w + 2 * i * R + c * 16);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mma16816<E>(acc[i], big.x, big.y, big.z, big.w, w[i].x, w[i].y);
        mma16816<E>(acc[i], rest.x, rest.y, rest.z, rest.w, w[i].x, w[i].y);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = m * 16 + g + 8 * h;
      if (row >= count || col >= N) continue;
      const int64_t t = rows[row];
      Vec8 o = zero8();
      if (base) o = unpack(ld8_stream(base + t * ld_b + col));
      if (id >= 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o.p[e] = __ffma2_rn(splat(factor[row]), make_float2(acc[e][2 * h], acc[e][2 * h + 1]), o.p[e]);
      }
      st8_stream(out + t * ld_o + col, pack<E>(o));
    }
  }
}

// out = base + B v for the units, 32 columns a warp at a time.
template <typename E, int CH, bool BASE>
__global__ void __launch_bounds__(128, CH == 8 ? 4 : 5) lora_expand_kernel(const uint4* vq, const float* factor, const E* b,
                                                             const int* index, const LoraPlan plan, int64_t T, int N,
                                                             int R, int n, const E* base, int64_t ld_b, E* out, int64_t ld_o) {
  extern __shared__ uint4 frag[];
  __shared__ TileTokens tile;
  __shared__ float factors[kTok];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, g = lane >> 2, chunks = (R + 15) / 16;
  pdl_wait_for(vq, factor, b, index, base);
  Units units(tile, plan, index, T, n);
  int id, count;
  while (units.next(id, count)) {
    if (id < 0 && base == out) continue;
    if (id >= 0) {
      for (int i = threadIdx.x; i < (count + 15) / 16 * chunks * 32; i += 128) {
        const int c = (i >> 5) % chunks, ra = (i >> 5) / chunks * 16 + g, rb = ra + 8;
        const uint4 u = vq[((int64_t)tile.rows[ra < count ? ra : 0] * chunks + c) * 4 + q];
        const uint4 v = vq[((int64_t)tile.rows[rb < count ? rb : 0] * chunks + c) * 4 + q];
        frag[i * 2] = make_uint4(u.x, v.x, u.y, v.y);
        frag[i * 2 + 1] = make_uint4(u.z, v.z, u.w, v.w);
      }
      if (threadIdx.x < kTok) factors[threadIdx.x] = factor[tile.rows[threadIdx.x < count ? threadIdx.x : 0]];
      __syncthreads();
    }
    const E* bw = b + (int64_t)max(id, 0) * N * R;
    for (int c0 = (blockIdx.z * 4 + warp) * 32; c0 < N; c0 += gridDim.z * 128) {
      const E* lane_w = bw + ((int64_t)c0 + (g >> 1) * 8 + (g & 1)) * R + q * 4;
      if (id >= 0 && c0 + 32 <= N && R <= CH * 16)
        expand_full<E, CH, BASE>(frag, factors, lane_w, R, base, ld_b, out, ld_o, tile.rows, count, c0 + q * 8, lane);
      else
        expand_any<E>(frag, factors, lane_w, id, N, R, base, ld_b, out, ld_o, tile.rows, count, c0, lane);
    }
  }
}

// The same for many tokens and larger ranks, where the form above is bound by shared memory
// and L1 (the weights and v pass through them for every product): tcgen05.mma with the output
// columns as its rows (128, an adapter's weights by TMA) and the unit's tokens as its
// columns, D in tensor memory.  A ninth warp's first thread fetches weights and issues the
// products of a tile while the eight others bring the last one from tensor memory through
// shared memory into rows, where base and out are read and written 256 bytes at a time; a
// tile's base is fetched before its products are waited for.  The weights have one place, filled
// again when the products that read it have ended: a second one would cost an SM its third CTA
// (T = 8192, H = N = 5120, both launches: rank 64 91 us with one place, 97 with two).
constexpr int kWideEpilogue = 256, kWideThreads = kWideEpilogue + 32, kWidePitch = 132;
struct WideShape {
  int blocks;     // of 64 of the rank
  size_t v, weights, rows, bars, bytes;  // offsets from an aligned start
};
__host__ __device__ inline WideShape wide_shape(int R) {
  WideShape w;
  w.blocks = (R + 63) / 64;
  w.v = 0;  // [blocks][roundings, rests][64 tokens][128 bytes]
  w.weights = (size_t)w.blocks * 2 * kTok * 128;
  w.rows = w.weights + (size_t)w.blocks * 128 * 128;
  w.bars = w.rows + (size_t)kTok * kWidePitch * 4;
  w.bytes = w.bars + 128 + 1024;
  return w;
}

template <typename E, bool BASE>
__global__ void __launch_bounds__(kWideThreads, 3) lora_wide_kernel(const __grid_constant__ CUtensorMap map, const uint4* vq,
                                                                const float* factor, const int* index,
                                                                const LoraPlan plan, int64_t T, int N, int R, int n, const E* base,
                                                                int64_t ld_b, E* out, int64_t ld_o, unsigned* status) {
  extern __shared__ char raw[];
  __shared__ TileTokens tile;
  __shared__ float factors[kTok];
  const WideShape shape = wide_shape(R);
  const uint32_t start = (smem_u32(raw) + 1023u) & ~1023u;
  char* aligned = raw + (start - smem_u32(raw));
  float* staged = reinterpret_cast<float*>(aligned + shape.rows);
  uint64_t* full = reinterpret_cast<uint64_t*>(aligned + shape.bars);
  uint64_t *empty = full + 1, *tfull = empty + 1, *tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = (R + 15) / 16;
  if (threadIdx.x == 0) {
    mbar_init(full, 1), mbar_init(empty, 1);
    for (int i = 0; i < 2; ++i) mbar_init(tfull + i, 1), mbar_init(tempty + i, kWideEpilogue / 32);
    mbar_fence_init();
  }
  if (warp == kWideEpilogue / 32) pair_tmem_alloc<1>(tmem_slot, 2 * kTok);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_inputs();
  pdl_wait_for(vq, factor, index, base);
  Units units(tile, plan, index, T, n);
  int id, count, buf = 0;  // (accumulators and the parities go on across units)
  uint32_t ph = 0, pb = 0;
  bool ok = true;
  while (units.next(id, count)) {
    if (id < 0) {  // no adapter: out = base
      if (base != out)
        for (int64_t i = (int64_t)blockIdx.z * kWideThreads + threadIdx.x; i < (int64_t)count * (N / 8); i += (int64_t)gridDim.z * kWideThreads) {
          const int64_t t = tile.rows[i / (N / 8)];
          const int c = (int)(i % (N / 8)) * 8;
          Raw8<E> z = pack<E>(zero8());
          if (BASE) z = ld8_stream(base + t * ld_b + c);
          st8_stream(out + t * ld_o + c, z);
        }
      continue;
    }
    // v into shared memory as rows of 64 of the rank, 16-byte pieces swizzled by the row
    for (int i = threadIdx.x; i < count * chunks * 4; i += kWideThreads) {
      const int row = i / (chunks * 4), p = i - row * chunks * 4;  // p: four of the rank
      const uint4 x = vq[(int64_t)tile.rows[row] * chunks * 4 + p];
      const int block = p >> 4, piece = (p & 15) >> 1;
      char* at = aligned + (size_t)block * 2 * kTok * 128 + row * 128 + ((piece ^ (row & 7)) << 4) + (p & 1) * 8;
      *reinterpret_cast<uint2*>(at) = make_uint2(x.x, x.y);
      *reinterpret_cast<uint2*>(at + kTok * 128) = make_uint2(x.z, x.w);
    }
    if (threadIdx.x < kTok) factors[threadIdx.x] = factor[tile.rows[threadIdx.x < count ? threadIdx.x : 0]];
    fence_proxy_async_smem();
    __syncthreads();
    const int first = blockIdx.z, step = gridDim.z, tiles = (N + 127) / 128;
    if (warp == kWideEpilogue / 32) {
      if (lane == 0) {
        const uint32_t bytes = shape.blocks * 128 * 128;
        constexpr uint32_t idesc = product_idesc<E>(128, kTok, false, false);
        auto fetch = [&](int t) {
          ok = mbar_wait(empty, ph ^ 1, kProductLimitNs);
          if (!ok) return;
          mbar_arrive_expect_tx(full, bytes);
          for (int k = 0; k < shape.blocks; ++k)
            pair_load<1>(start + (uint32_t)shape.weights + k * 128 * 128, &map, smem_u32(full), k * 64, id * N + t * 128);
        };
        fetch(first);
        for (int t = first; t < tiles && ok; t += step) {
          ok = mbar_wait(tempty + buf, pb ^ 1, kProductLimitNs) && mbar_wait(full, ph, kProductLimitNs);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = start + (uint32_t)shape.weights, v = start;
          for (int c = 0; c < chunks; ++c) {
            const uint32_t k = (c & 3) * 32, block = c >> 2;
            const uint64_t da = tile_desc(a + block * 128 * 128 + k, false);
            pair_mma<1>(tmem + buf * kTok, da, tile_desc(v + block * 2 * kTok * 128 + k, false), idesc, c);
            pair_mma<1>(tmem + buf * kTok, da, tile_desc(v + block * 2 * kTok * 128 + kTok * 128 + k, false), idesc, 1);
          }
          pair_commit<1>(empty);
          pair_commit<1>(tfull + buf);
          ph ^= 1;
          if ((buf ^= 1) == 0) pb ^= 1;
          if (t + step < tiles) fetch(t + step);
        }
        // the MMAs that read this unit's v have ended before the next one's takes its place
        if (ok) ok = mbar_wait(empty, ph ^ 1, kProductLimitNs);
      }
    } else {
      constexpr int kRows = kTok / (kWideEpilogue / 32);  // rows a warp reads and writes
      const int r0 = warp * kRows;
      uint2 old[kRows];
      auto fetch = [&](uint2* o, int t) {
        if constexpr (BASE) {
          const int col = t * 128 + lane * 4;
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            if (col < N && r0 + i < count) o[i] = __ldcs(reinterpret_cast<const uint2*>(base + (int64_t)tile.rows[r0 + i] * ld_b + col));
        }
      };
      for (int t = first; t < tiles; t += step) {
        fetch(old, t);
        ok = all_of<kWideEpilogue>(mbar_wait(tfull + buf, pb, kProductLimitNs));  // (also: all have read the last tile's rows)
        if (!ok) break;
        tc_fence_after();
        for (int c = (warp >> 2) * 16; c < count; c += kWideEpilogue / 8) {  // (a warp reads the lanes of its quarter)
          uint32_t d[16];
          __syncwarp();
          issue16(tmem + buf * kTok + c + ((uint32_t)(warp & 3) << 21), d);
          take16(d);
#pragma unroll
          for (int e = 0; e < 16; ++e) staged[(c + e) * kWidePitch + (warp & 3) * 32 + lane] = __uint_as_float(d[e]);
        }
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty + buf);
        if ((buf ^= 1) == 0) pb ^= 1;
        named_bar_sync(1, kWideEpilogue);
        const int col = t * 128 + lane * 4;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int row = r0 + i;
          if (row >= count || col >= N) continue;
          const float4 d = *reinterpret_cast<const float4*>(staged + row * kWidePitch + lane * 4);
          const float f = factors[row];
          float2 lo = make_float2(0.f, 0.f), hi = lo;
          if constexpr (BASE) lo = pair_of(old[i].x, E()), hi = pair_of(old[i].y, E());
          const uint2 o = make_uint2(word_of(fmaf(f, d.x, lo.x), fmaf(f, d.y, lo.y), E()), word_of(fmaf(f, d.z, hi.x), fmaf(f, d.w, hi.y), E()));
          __stcs(reinterpret_cast<uint2*>(out + (int64_t)tile.rows[row] * ld_o + col), o);
        }
      }
    }
    // all give up together
    if (!__syncthreads_and(ok)) {
      if (threadIdx.x == 0) atomicOr(status, 2u);
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 20000000ull) __nanosleep(1000);
      break;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWideEpilogue / 32) pair_tmem_dealloc<1>(tmem, 2 * kTok);
}

// ------------------------------------------------------------------- host --
// Workspace: the status word, the place of the products' counters (which outlive this call where both
// work in one buffer), v, factors, and the plan (order, units, units made per run), each from a multiple
// of 256 bytes.
static_assert(kProductParts % 256 == 0, "");
struct LoraSpace {
  size_t v, factor, order, units, made, bytes;
};
static LoraSpace lora_space(int64_t T, int R) {
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t chunks = (R + 15) / 16, t = (size_t)T;
  LoraSpace s;
  s.v = kProductParts;
  s.factor = s.v + up(t * chunks * 64);
  s.order = s.factor + up(t * 4);
  s.units = s.order + up(t * 4);
  s.made = s.units + up(t * sizeof(Unit));
  s.bytes = s.made + up((t + kRun - 1) / kRun * 4);
  return s;
}

template <typename... Params, typename... Args>
static cudaError_t launch_cluster_z(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = grid.z;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  if (e != cudaSuccess) cudaGetLastError();  // it is this call's, not the next one's
  return e;
}

template <typename E, int NT>
static cudaError_t shrink_launch(dim3 grid, const void* x, int64_t ld_x, const void* a, const int* index, const float* scale,
                                 const LoraPlan& plan, int64_t T, int H, int R, int n, int slice, void* vq, float* factor,
                                 cudaStream_t s) {
  static SmemGrant grant;
  const size_t smem = shrink_smem<NT>(R);
  cudaError_t e = allow_smem(grant, (const void*)lora_shrink_kernel<E, NT>, smem);
  if (e != cudaSuccess) return e;
  return launch_cluster_z(lora_shrink_kernel<E, NT>, grid, dim3(128), smem, s, static_cast<const E*>(x), ld_x, static_cast<const E*>(a),
                          index, scale, plan, T, H, R, n, slice, static_cast<uint4*>(vq), factor);
}

template <typename E>
static cudaError_t lora_launch(const void* x, int64_t ld_x, const void* a, const void* b, const int* index, const float* scale,
                               int64_t T, int H, int N, int R, int n, const void* base, int64_t ld_b, void* out, int64_t ld_o,
                               void* ws, cudaStream_t s) {
  const LoraSpace space = lora_space(T, R);
  char* w = static_cast<char*>(ws);
  float* factor = reinterpret_cast<float*>(w + space.factor);
  LoraPlan plan = {};
  int64_t most, busy;  // units at most, and about how many there are
  cudaError_t e;
  if (T <= kTok) {
    most = busy = T < n + 1 ? T : n + 1;
  } else {
    int* order = reinterpret_cast<int*>(w + space.order);
    Unit* table = reinterpret_cast<Unit*>(w + space.units);
    int* made = reinterpret_cast<int*>(w + space.made);
    const int64_t runs = (T + kRun - 1) / kRun, tokens = T < kRun ? T : kRun;
    most = tokens / kTok + (n + 1 < tokens ? n + 1 : tokens);  // of a run: its tokens by 64, and one more for each adapter
    most = runs * (most < tokens ? most : tokens);
    busy = T / kTok + runs * (n < 4 ? n : 4);
    plan = {order, table, made, (int)runs};
    e = launch_pdl(lora_plan_kernel, dim3((unsigned)runs), dim3(kRun), 0, s, index, T, n, order, table, made);
    if (e != cudaSuccess) return e;
  }
  // parts of H: enough CTAs for a few tokens, at least 128 columns each
  // (more than these gain nothing: two an SM, five for small ranks)
  const int resident = R <= 32 ? 5 * 152 : 334;
  int parts = 1;
  while (parts < kMostParts && busy * parts * 2 <= resident && H / (2 * parts) >= 128) parts *= 2;
  const int slice = ((H + parts - 1) / parts + 63) / 64 * 64;
  const int64_t across = most < (1 << 20) ? most : 1 << 20;  // (those past the last unit end at once)
  const dim3 grid((unsigned)across, 1, parts);
  e = R <= 8    ? shrink_launch<E, 1>(grid, x, ld_x, a, index, scale, plan, T, H, R, n, slice, w + space.v, factor, s)
      : R <= 16 ? shrink_launch<E, 2>(grid, x, ld_x, a, index, scale, plan, T, H, R, n, slice, w + space.v, factor, s)
      : R <= 32 ? shrink_launch<E, 4>(grid, x, ld_x, a, index, scale, plan, T, H, R, n, slice, w + space.v, factor, s)
      : R <= 64 ? shrink_launch<E, 8>(grid, x, ld_x, a, index, scale, plan, T, H, R, n, slice, w + space.v, factor, s)
                : shrink_launch<E, 16>(grid, x, ld_x, a, index, scale, plan, T, H, R, n, slice, w + space.v, factor, s);
  if (e != cudaSuccess) return e;
  // (T = 8192, H = N = 5120, both launches: rank 64 91 against 105 us, rank 128 109 against 182, rank 24 103 against 81)
  // (without adapters there are no weights to lay a tensor map over)
  if (plan.order && R >= 48 && n > 0 && (int64_t)n * N < 0x7fffffff) {
    CUtensorMap map;
    if (!encode_2d<E>(&map, b, (int64_t)n * N, R, R, 128)) return cudaErrorInvalidValue;
    const size_t smem = wide_shape(R).bytes;
    auto kernel = base ? lora_wide_kernel<E, true> : lora_wide_kernel<E, false>;
    static SmemGrant grants[2];
    e = allow_smem(grants[base != nullptr], (const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    // As many CTAs as an SM's 228 KB have room for: three up to rank 64, two up to 128, then one.  (Both
    // launches with one and with two for rank 256: T = 8192, H = N = 5120, 24 prompts 253 and 260 us; T = 1003,
    // H = 2048, N = 10000 73 and 80; 64 adapters in any order, whose units are many as it is, 895 and 870.)
    const int64_t room = (228 << 10) / (smem + 2048);
    int64_t wide = (room * 152 + busy - 1) / busy;
    if (wide > (N + 127) / 128) wide = (N + 127) / 128;
    return launch_pdl(kernel, dim3((unsigned)across, 1, (unsigned)wide), dim3(kWideThreads), smem, s, map,
                      reinterpret_cast<const uint4*>(w + space.v), factor, index, plan, T, N, R, n, static_cast<const E*>(base), ld_b,
                      static_cast<E*>(out), ld_o, static_cast<unsigned*>(ws));
  }
  const int64_t blocks = (N + 127) / 128;
  int64_t wide = (kExpandCtas * 152 + busy - 1) / busy;
  if (wide > blocks) wide = blocks;
  const int64_t each = (blocks + wide - 1) / wide;  // column blocks of a CTA: as even as they can be
  wide = (blocks + each - 1) / each;
  const int which = (R <= 16 ? 0 : R <= 32 ? 1 : R <= 64 ? 2 : 3) + (base ? 4 : 0);
  const decltype(&lora_expand_kernel<E, 1, true>) kernels[] = {
      lora_expand_kernel<E, 1, false>, lora_expand_kernel<E, 2, false>, lora_expand_kernel<E, 4, false>, lora_expand_kernel<E, 8, false>,
      lora_expand_kernel<E, 1, true>,  lora_expand_kernel<E, 2, true>,  lora_expand_kernel<E, 4, true>,  lora_expand_kernel<E, 8, true>};
  static SmemGrant grants[8];
  const size_t smem = (size_t)(kTok / 16) * ((R + 15) / 16) * 1024;
  e = allow_smem(grants[which], (const void*)kernels[which], smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernels[which], dim3((unsigned)across, 1, (unsigned)wide), dim3(128), smem, s, reinterpret_cast<const uint4*>(w + space.v), factor,
                    static_cast<const E*>(b), index, plan, T, N, R, n, static_cast<const E*>(base), ld_b, static_cast<E*>(out), ld_o);
}

}  // namespace mhc

extern "C" size_t mhc_lora_workspace_bytes(int64_t T, int R) { return T > 0 && R > 0 ? mhc::lora_space(T, R).bytes : 0; }

extern "C" int mhc_lora(const void* x, int64_t ld_x, const void* a, const void* b, const int32_t* index, const float* scale,
                        int64_t T, int H, int N, int R, int n, mhc_dtype dtype, const void* base, int64_t ld_base, void* out,
                        int64_t ld_out, void* workspace, size_t ws_bytes, void* stream) {
  using namespace mhc;
  if (dtype != MHC_DT_BF16 && dtype != MHC_DT_F16) return ops_fail(MHC_ERR_CONFIG, "dtype must be bf16 or fp16");
  if (T < 0 || T > (1 << 30) || H <= 0 || H % 8 != 0 || H > (1 << 20) || N <= 0 || N % 8 != 0 || N > (1 << 20) || R <= 0 ||
      R % 8 != 0 || R > 256 || n < 0 || n > (1 << 20))
    return ops_fail(MHC_ERR_SHAPE, "need 0 <= T <= 2^30, H and N (at most 2^20) and R (at most 256) positive multiples of 8, 0 <= n <= 2^20");
  if (ld_x < H || ld_x % 8 != 0 || ld_out < N || ld_out % 8 != 0 || (base && (ld_base < N || ld_base % 8 != 0)))
    return ops_fail(MHC_ERR_SHAPE, "row strides must be multiples of 8, at least the row");
  if (T == 0) return MHC_OK;
  if (!x || !index || !out || (n && (!a || !b))) return ops_fail(MHC_ERR_NULL, "x, a, b, index and out are required");
  for (const void* p : {x, a, b, base, (const void*)out, (const void*)workspace})
    if (!ops_aligned(p, 16)) return ops_fail(MHC_ERR_ALIGN, "matrices and the workspace must be 16-byte aligned");
  if (!ops_aligned(index, 4) || !ops_aligned(scale, 4)) return ops_fail(MHC_ERR_ALIGN, "index and scale must be aligned to their elements");
  if (!workspace || ws_bytes < mhc_lora_workspace_bytes(T, R))
    return ops_fail(MHC_ERR_WORKSPACE, "workspace NULL or smaller than mhc_lora_workspace_bytes()");
  const Rows o = {out, T, N, ld_out, 2}, ws = {workspace, 1, (int64_t)ws_bytes, (int64_t)ws_bytes, 1};
  const Rows in[] = {{x, T, H, ld_x, 2}, {a, n, (int64_t)R * H, (int64_t)R * H, 2}, {b, n, (int64_t)N * R, (int64_t)N * R, 2},
                     {index, 1, T, T, 4}, {scale, 1, n, n, 4}};
  for (const Rows& r : in)
    if (rows_overlap(o, r) || rows_overlap(ws, r)) return ops_fail(MHC_ERR_ALIAS, "out or the workspace overlaps an input");
  const Rows bs = {base, T, N, ld_base, 2};
  if ((rows_overlap(o, bs) && !(out == base && ld_out == ld_base)) || rows_overlap(ws, bs) || rows_overlap(ws, o))
    return ops_fail(MHC_ERR_ALIAS, "out overlaps base (other than base exactly), or the workspace one of them");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MHC_DT_BF16
          ? lora_launch<__nv_bfloat16>(x, ld_x, a, b, index, scale, T, H, N, R, n, base, ld_base, out, ld_out, workspace, s)
          : lora_launch<__half>(x, ld_x, a, b, index, scale, T, H, N, R, n, base, ld_base, out, ld_out, workspace, s);
  return ops_cuda(e, "lora launch");
}
