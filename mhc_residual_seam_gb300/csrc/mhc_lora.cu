// mhc_lora: low-rank adapters of many requests beside a shared projection.
//
//   v[t,:] = A_a x[t],  out[t,:] = base[t,:] + s_a B_a v[t],  a = index[t]
//
// Two launches: the first makes v (split over H, so that a few tokens fill the GPU),
// the second sums the parts and applies B.  Both work on tiles of 64 tokens: a CTA
// finds the different adapters of its tile and takes the tokens of one adapter after
// another as the rows of tensor-core products (mma.sync m16n8k16: the work is bound by
// memory, x and out are read and written once, and an adapter's weights once per tile
// that names it).  Operands go from memory to registers in 16-byte pieces: the order of
// a product's reduction index and of its columns is free, so each thread's fragment is
// taken from adjacent elements.

#include <type_traits>

#include "mhc_ops.cuh"

namespace mhc {

constexpr int kTok = 64;  // tokens of a tile

// The different adapters of a tile in order of appearance (-1: tokens without one), and
// the tokens of one of them.  Made by warp 0.
struct TileTokens {
  int firsts[kTok], rows[kTok];
  int distinct, count;
};

// Warp 0 holds the tile's adapters in two registers a lane (-2: past the last token).
__device__ __forceinline__ int adapter_of(const int* index, int64_t t, int64_t T, int n) {
  if (t >= T) return -2;
  const int i = index[t];
  return i >= 0 && i < n ? i : -1;
}
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

// v[part, t, r] = sum over the part's columns of x[t, h] A[r, h], eight NT of the rank at
// a time.  The four warps share a group of up to 64 tokens by 16 tokens and, where there
// are fewer groups of 16, by columns; their sums are joined in a fixed order.
template <typename E, int NT>
__global__ void __launch_bounds__(128) lora_shrink_kernel(const E* __restrict__ x, int64_t ld_x, const E* __restrict__ a,
                                                          const int* __restrict__ index, int64_t T, int H, int R, int n,
                                                          int slice, float* __restrict__ v) {
  __shared__ TileTokens tile;
  __shared__ float sums[4][16][NT * 8 + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, g = lane >> 2;
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int id0 = adapter_of(index, t0 + lane, T, n), id1 = adapter_of(index, t0 + lane + 32, T, n);
  if (warp == 0) find_adapters(tile, id0, id1, lane);
  __syncthreads();
  pdl_launch();
  const int distinct = tile.distinct;
  const int k0 = blockIdx.z * slice, k1 = min(H, k0 + slice);
  v += (int64_t)blockIdx.z * T * R;
  for (int j = blockIdx.y; j < distinct; j += gridDim.y) {
    const int id = tile.firsts[j];
    if (id < 0) continue;
    if (warp == 0) find_tokens(tile, id, id0, id1, lane);
    __syncthreads();
    const int count = tile.count;
    const int groups = count <= 16 ? 1 : count <= 32 ? 2 : 4, parts = 4 / groups;
    const int m = warp % groups, part = warp / groups;
    const int ra = m * 16 + g, rb = ra + 8;
    const E* xa = ra < count ? x + (t0 + tile.rows[ra]) * ld_x + q * 8 : nullptr;
    const E* xb = rb < count ? x + (t0 + tile.rows[rb]) * ld_x + q * 8 : nullptr;
    for (int r0 = 0; r0 < R; r0 += NT * 8) {
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
      const E* ar = a + ((int64_t)id * R + r0 + g) * H + q * 8;
      if (m * 16 < count) {
        const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll 2
        for (int k = k0 + part * 32; k < k1; k += parts * 32) {
          const bool in = k + q * 8 < k1;
          const uint4 u = in && xa ? *reinterpret_cast<const uint4*>(xa + k) : none;
          const uint4 w = in && xb ? *reinterpret_cast<const uint4*>(xb + k) : none;
          uint4 b[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i)
            b[i] = in && r0 + i * 8 + g < R ? *reinterpret_cast<const uint4*>(ar + (int64_t)i * 8 * H + k) : none;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma16816<E>(acc[i], u.x, w.x, u.y, w.y, b[i].x, b[i].y);
            mma16816<E>(acc[i], u.z, w.z, u.w, w.w, b[i].z, b[i].w);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        *reinterpret_cast<float2*>(&sums[warp][g][i * 8 + 2 * q]) = make_float2(acc[i][0], acc[i][1]);
        *reinterpret_cast<float2*>(&sums[warp][g + 8][i * 8 + 2 * q]) = make_float2(acc[i][2], acc[i][3]);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < count * NT * 8; i += 128) {
        const int row = i / (NT * 8), c = i % (NT * 8);
        if (r0 + c >= R) continue;
        float s = sums[row >> 4][row & 15][c];
        for (int p = 1; p < parts; ++p) s += sums[(row >> 4) + p * groups][row & 15][c];
        v[(t0 + tile.rows[row]) * R + r0 + c] = s;
      }
      __syncthreads();
    }
  }
}

// out = base + s B v for the tokens of a tile, 64 columns a warp at a time.
//
// v is fp32 and B has 16 bits: each v is cut into two 16-bit values (its rounding and
// the rounding of the rest, 16 or 22 bits together), and both are multiplied.  A row is
// first brought to about 1 by a power of two, so that fp16 neither overflows nor loses
// the rest to subnormals.
template <typename E>
__global__ void __launch_bounds__(128) lora_expand_kernel(const float* __restrict__ v, int parts, const E* __restrict__ b,
                                                          const int* __restrict__ index, const float* __restrict__ scale,
                                                          int64_t T, int N, int R, int n, const E* base, int64_t ld_b, E* out,
                                                          int64_t ld_o) {
  extern __shared__ char raw[];
  __shared__ TileTokens tile;
  __shared__ float factor[kTok];
  const int chunks = (R + 15) / 16, width = chunks * 16 + 4;
  // fragments of v, [16 tokens][chunk of 16][lane]: four registers of the rounding, four of the rest
  uint4* frag = reinterpret_cast<uint4*>(raw);
  float* vs = reinterpret_cast<float*>(raw + (size_t)(kTok / 16) * chunks * 1024);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, g = lane >> 2;
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int id0 = adapter_of(index, t0 + lane, T, n), id1 = adapter_of(index, t0 + lane + 32, T, n);
  if (warp == 0) find_adapters(tile, id0, id1, lane);
  __syncthreads();
  pdl_wait();
  const int distinct = tile.distinct;
  for (int j = blockIdx.y; j < distinct; j += gridDim.y) {
    const int id = tile.firsts[j];
    if (id < 0 && base == out) continue;
    if (warp == 0) find_tokens(tile, id, id0, id1, lane);
    __syncthreads();
    const int count = tile.count, groups = (count + 15) / 16;
    if (id >= 0) {
      const float s = scale ? scale[id] : 1.f;
      for (int row = warp; row < groups * 16; row += 4) {  // a warp per row: the parts' sum, and the row's exponent
        float most = 0.f;
        for (int r = lane; r < chunks * 16; r += 32) {
          float z = 0.f;
          if (row < count && r < R) {
            const float* p = v + (t0 + tile.rows[row]) * R + r;
            for (int i = 0; i < parts; ++i) z += p[(int64_t)i * T * R];
          }
          vs[row * width + r] = z;
          if (fabsf(z) <= 3e38f) most = fmaxf(most, fabsf(z));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        // 2^e of the largest, from its exponent bits; rows of zeros and of subnormals as they are
        const uint32_t e = __float_as_uint(most) >> 23;
        const bool plain = e < 16 || e > 238;
        const float down = plain ? 1.f : __uint_as_float((254 - e) << 23), up = plain ? 1.f : __uint_as_float(e << 23);
        for (int r = lane; r < chunks * 16; r += 32) vs[row * width + r] *= down;
        if (lane == 0) factor[row] = s * up;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < groups * chunks * 32; i += 128) {
        const int ln = i & 31, c = (i >> 5) % chunks, m = (i >> 5) / chunks;
        const float4 lo = *reinterpret_cast<const float4*>(vs + (m * 16 + (ln >> 2)) * width + c * 16 + (ln & 3) * 4);
        const float4 hi = *reinterpret_cast<const float4*>(vs + (m * 16 + 8 + (ln >> 2)) * width + c * 16 + (ln & 3) * 4);
        const float2 w[4] = {{lo.x, lo.y}, {hi.x, hi.y}, {lo.z, lo.w}, {hi.z, hi.w}};
        uint32_t big[4], rest[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          big[p] = word_of(w[p].x, w[p].y, E());
          const float2 f = pair_of(big[p], E());
          // (an infinite row has no rest)
          rest[p] = word_of(fabsf(f.x) <= 3e38f ? w[p].x - f.x : 0.f, fabsf(f.y) <= 3e38f ? w[p].y - f.y : 0.f, E());
        }
        frag[i * 2] = make_uint4(big[0], big[1], big[2], big[3]);
        frag[i * 2 + 1] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
      }
      __syncthreads();
    }
    // column of fragment column 2 p + e of product i: 16 p + 2 i + e, so a thread's 16 results of a row are adjacent
    const E* bw = b + (int64_t)max(id, 0) * N * R;
    for (int c0 = (blockIdx.z * 4 + warp) * 64; c0 < N; c0 += gridDim.z * 256) {
      for (int m = 0; m < groups; ++m) {
        float acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        if (id >= 0) {
          for (int c = 0; c < chunks; ++c) {
            const uint4 big = frag[((m * chunks + c) * 32 + lane) * 2], rest = frag[((m * chunks + c) * 32 + lane) * 2 + 1];
            const int r = c * 16 + q * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int col = c0 + (g >> 1) * 16 + 2 * i + (g & 1);
              uint2 w = make_uint2(0, 0);
              if (col < N && r < R) w = *reinterpret_cast<const uint2*>(bw + (int64_t)col * R + r);
              mma16816<E>(acc[i], big.x, big.y, big.z, big.w, w.x, w.y);
              mma16816<E>(acc[i], rest.x, rest.y, rest.z, rest.w, w.x, w.y);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = m * 16 + g + 8 * h;
          if (row >= count) continue;
          const int64_t t = t0 + tile.rows[row];
          const float f = id >= 0 ? factor[row] : 0.f;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int col = c0 + q * 16 + p * 8;
            if (col >= N) break;
            Vec8 o = zero8();
            if (base) o = unpack(ld8_stream(base + t * ld_b + col));
            if (id >= 0) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o.p[e].x = fmaf(f, acc[p * 4 + e][2 * h], o.p[e].x);
                o.p[e].y = fmaf(f, acc[p * 4 + e][2 * h + 1], o.p[e].y);
              }
            }
            st8_stream(out + t * ld_o + col, pack<E>(o));
          }
        }
      }
    }
    __syncthreads();
  }
}

// Parts of H for the first launch: enough CTAs for a few tokens, at least 128 columns each.
constexpr int kMostParts = 16, kWantCtas = 4 * 152;
static int lora_parts(int64_t T, int H) {
  const int64_t tiles = (T + kTok - 1) / kTok, want = (kWantCtas + tiles - 1) / tiles;
  int most = (H + 127) / 128;
  if (most > kMostParts) most = kMostParts;
  return (int)(want < most ? want : most);
}
// CTAs that share a tile's adapters: many where there are few tiles.
static int lora_sharers(int64_t T, int n) {
  const int64_t tiles = (T + kTok - 1) / kTok;
  int64_t most = n + 1 < kTok ? n + 1 : kTok;
  if (T < most) most = T;
  const int64_t want = (152 + tiles - 1) / tiles;
  return (int)(want < most ? want : most);
}

template <typename E>
static cudaError_t lora_launch(const void* x, int64_t ld_x, const void* a, const void* b, const int* index, const float* scale,
                               int64_t T, int H, int N, int R, int n, const void* base, int64_t ld_b, void* out, int64_t ld_o,
                               void* ws, cudaStream_t s) {
  const unsigned tiles = (unsigned)((T + kTok - 1) / kTok), share = (unsigned)lora_sharers(T, n);
  int parts = lora_parts(T, H);
  const int slice = ((H + parts - 1) / parts + 31) / 32 * 32;
  parts = (H + slice - 1) / slice;
  auto k = R <= 8 ? lora_shrink_kernel<E, 1> : R <= 16 ? lora_shrink_kernel<E, 2> : R <= 32 ? lora_shrink_kernel<E, 4> : lora_shrink_kernel<E, 8>;
  float* v = static_cast<float*>(ws);
  k<<<dim3(tiles, share, parts), 128, 0, s>>>(static_cast<const E*>(x), ld_x, static_cast<const E*>(a), index, T, H, R, n, slice, v);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int chunks = (R + 15) / 16;
  const size_t smem = (size_t)(kTok / 16) * chunks * 1024 + (size_t)kTok * (chunks * 16 + 4) * 4;
  static SmemGrant grant;
  e = allow_smem(grant, (const void*)lora_expand_kernel<E>, smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (N + 255) / 256;
  int64_t wide = (8 * 152 + (int64_t)tiles * share - 1) / ((int64_t)tiles * share);
  if (wide > blocks) wide = blocks;
  return launch_pdl(lora_expand_kernel<E>, dim3(tiles, share, (unsigned)wide), dim3(128), smem, s, v, parts, static_cast<const E*>(b), index,
                    scale, T, N, R, n, static_cast<const E*>(base), ld_b, static_cast<E*>(out), ld_o);
}

}  // namespace mhc

extern "C" size_t mhc_lora_workspace_bytes(int64_t T, int R) {
  using namespace mhc;
  if (T <= 0 || R <= 0) return 0;
  // parts * T at most: parts is at most kMostParts, and below kWantCtas / tiles + 1
  const int64_t few = kMostParts * T, many = (int64_t)kWantCtas * kTok + T;
  return (size_t)(few < many ? few : many) * R * 4;
}

extern "C" int mhc_lora(const void* x, int64_t ld_x, const void* a, const void* b, const int32_t* index, const float* scale,
                        int64_t T, int H, int N, int R, int n, mhc_dtype dtype, const void* base, int64_t ld_base, void* out,
                        int64_t ld_out, void* workspace, size_t ws_bytes, void* stream) {
  using namespace mhc;
  if (dtype != MHC_DT_BF16 && dtype != MHC_DT_F16) return ops_fail(MHC_ERR_CONFIG, "dtype must be bf16 or fp16");
  if (T < 0 || T > (1 << 30) || H <= 0 || H % 8 != 0 || H > (1 << 20) || N <= 0 || N % 8 != 0 || N > (1 << 20) || R <= 0 ||
      R % 8 != 0 || R > 256 || n < 0)
    return ops_fail(MHC_ERR_SHAPE, "need 0 <= T <= 2^30, H and N (at most 2^20) and R (at most 256) positive multiples of 8, n >= 0");
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
