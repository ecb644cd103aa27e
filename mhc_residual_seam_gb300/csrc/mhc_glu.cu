// mhc_glu: the gated projections of a feed-forward block in one kernel.

#include "mhc_glu.cuh"
#include "mhc_glu_few.cuh"
#include "mhc_product.cuh"

namespace mhc {

// One tile's accumulator holds the gate's columns in its first half and the other
// projection's in its second, for the same BN / 2 features, so a lane finds g and u of
// one token and feature in its own row.
template <typename E, int BN>
struct GluEpilogue {
  const E* add;
  E *gu, *h;
  int64_t T, F, ld_add, ld_h;
  int act;

  __device__ __forceinline__ int row_b(int n, int j) const {
    constexpr int half = BN / 2;
    return n * half + (j < half ? j : (int)F + j - half);
  }
  template <typename Source>
  __device__ __forceinline__ void store(const Source& from, int64_t row, int n, int, int part) const {
    constexpr int half = BN / 2;
#pragma unroll 1
    for (int c = part * 16; c < half; c += 32) {
      float a[16], b[16];
      from.get2(c, a, half + c, b);
      if (row >= T) continue;
      const int64_t f = (int64_t)n * half + c;
      const int pieces = (int)min((int64_t)2, (F - f) / 8);  // eight features each: F is a multiple of eight
      if (pieces <= 0) continue;
      if (add) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (p >= pieces) break;
          const Vec8 x = unpack(ld8(add + row * ld_add + f + 8 * p)), y = unpack(ld8(add + row * ld_add + F + f + 8 * p));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[8 * p + 2 * e] += x.p[e].x, a[8 * p + 2 * e + 1] += x.p[e].y;
            b[8 * p + 2 * e] += y.p[e].x, b[8 * p + 2 * e + 1] += y.p[e].y;
          }
        }
      }
      if (gu) {
        put16(gu + row * 2 * F + f, a, pieces);
        put16(gu + row * 2 * F + F + f, b, pieces);
      }
      activate_product<16>(a, b, act);
      put16(h + row * ld_h + f, a, pieces);
    }
  }
  __device__ __forceinline__ static void put16(E* out, const float* v, int pieces) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (p >= pieces) break;
      Vec8 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o.p[e] = make_float2(v[8 * p + 2 * e], v[8 * p + 2 * e + 1]);
      st8(out + 8 * p, pack<E>(o));
    }
  }
};

template <typename E, typename S>
static cudaError_t glu_tiles(const void* x, int64_t ld_x, const void* w, const void* add, int64_t ld_add, int act, int64_t T,
                             int H, int F, void* gu, void* h, int64_t ld_h, void* ws, cudaStream_t s) {
  Work<1> p;
  if (!problem<E, S>(&p.p[0], T, (F + S::BN / 2 - 1) / (S::BN / 2), H, x, false, ld_x, w, 2 * (int64_t)F, H))
    return cudaErrorInvalidValue;
  const GluEpilogue<E, S::BN> epi = {static_cast<const E*>(add), static_cast<E*>(gu), static_cast<E*>(h), T, F, ld_add, ld_h, act};
  return product_launch<E, S, 1>(p, ws, epi, s);
}

template <typename E>
static cudaError_t glu_launch(const void* x, int64_t ld_x, const void* w, const void* add, int64_t ld_add, int act, int64_t T,
                              int H, int F, void* gu, void* h, int64_t ld_h, void* ws, cudaStream_t s) {
  if (T <= kFewTokens) return glu_few_launch<E>(x, ld_x, w, add, ld_add, act, T, H, F, gu, h, ld_h, ws, s);
  const int64_t kb = (H + kBK - 1) / kBK;
  if (product_small(
          [&](int, int rows, int columns, int64_t* n, int64_t* k) {
            *n = ((T + rows - 1) / rows) * ((F + columns / 2 - 1) / (columns / 2)), *k = kb;
          },
          1))
    return glu_tiles<E, Tile<1, 128, false>>(x, ld_x, w, add, ld_add, act, T, H, F, gu, h, ld_h, ws, s);
  return glu_tiles<E, Tile<2, 256, false>>(x, ld_x, w, add, ld_add, act, T, H, F, gu, h, ld_h, ws, s);
}

}  // namespace mhc

extern "C" size_t mhc_glu_workspace_bytes(int64_t T, int H, int F) {
  using namespace mhc;
  if (T <= 0 || H <= 0 || F <= 0) return 0;
  const size_t few = few_bytes(few_plan(H, F));
  return few > kProductBytes ? few : kProductBytes;
}

extern "C" int mhc_glu(const void* x, int64_t ld_x, const void* w, const void* add, int64_t ld_add, int act, int64_t T, int H,
                       int F, mhc_dtype dtype, void* gu, void* h, int64_t ld_h, void* workspace, size_t ws_bytes, void* stream) {
  using namespace mhc;
  if (dtype != MHC_DT_BF16 && dtype != MHC_DT_F16) return ops_fail(MHC_ERR_CONFIG, "dtype must be bf16 or fp16");
  if (!act_ok(act)) return ops_fail(MHC_ERR_CONFIG, "unknown activation");
  if (T < 0 || T > (1 << 30) || H <= 0 || H % 8 != 0 || H > (1 << 20) || F <= 0 || F % 8 != 0 || F > (1 << 20))
    return ops_fail(MHC_ERR_SHAPE, "need 0 <= T <= 2^30, H and F positive multiples of 8, at most 2^20");
  if (ld_x < H || ld_x % 8 != 0 || ld_x > (1ll << 36) || ld_h < F || ld_h % 8 != 0 ||
      (add && ((ld_add != 0 && ld_add < 2 * (int64_t)F) || ld_add % 8 != 0)))
    return ops_fail(MHC_ERR_SHAPE, "row strides must be multiples of 8, at least the row (ld_add may be 0)");
  if (T == 0) return MHC_OK;
  if (!x || !w || !h) return ops_fail(MHC_ERR_NULL, "x, w and h are required");
  if (!ops_aligned(x, 16) || !ops_aligned(w, 16) || !ops_aligned(add, 16) || !ops_aligned(gu, 16) || !ops_aligned(h, 16) ||
      !ops_aligned(workspace, 16))
    return ops_fail(MHC_ERR_ALIGN, "matrices and the workspace must be 16-byte aligned");
  if (!workspace || ws_bytes < mhc_glu_workspace_bytes(T, H, F))
    return ops_fail(MHC_ERR_WORKSPACE, "workspace NULL or smaller than mhc_glu_workspace_bytes()");
  const Rows in[] = {{x, T, H, ld_x, 2}, {w, 2 * (int64_t)F, H, H, 2}, {add, ld_add ? T : 1, 2 * (int64_t)F, ld_add ? ld_add : 2 * (int64_t)F, 2}};
  const Rows out[] = {{h, T, F, ld_h, 2}, {gu, T, 2 * (int64_t)F, 2 * (int64_t)F, 2}, {workspace, 1, (int64_t)ws_bytes, (int64_t)ws_bytes, 1}};
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in)
      if (rows_overlap(out[i], r)) return ops_fail(MHC_ERR_ALIAS, "an output or the workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (rows_overlap(out[i], out[j])) return ops_fail(MHC_ERR_ALIAS, "the outputs and the workspace overlap");
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MHC_DT_BF16
          ? glu_launch<__nv_bfloat16>(x, ld_x, w, add, ld_add, act, T, H, F, gu, h, ld_h, workspace, s)
          : glu_launch<__half>(x, ld_x, w, add, ld_add, act, T, H, F, gu, h, ld_h, workspace, s);
  return ops_cuda(e, "glu launch");
}
