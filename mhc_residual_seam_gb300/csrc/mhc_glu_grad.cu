// mhc_glu_grad: the gradient of the gated projections.

#include "mhc_glu.cuh"
#include "mhc_product.cuh"

namespace mhc {

// dg = dh u act'(g), du = dh act(g), from the kept pre-activations, into [T, 2F].  Bound
// by HBM: three rows of F read, two written.  Work item = (token, 8 features).
// dgu is rounded once, to its type: the tensor cores take 16-bit operands, and the products of
// a second 16-bit value for what the rounding leaves would cost as much again.  dx and dw
// (also in fp32) are the exact products of the rounded values in fp32 sums: 2.3e-3 of the
// 2-norm from the unrounded ones in bf16, 2.9e-4 in fp16, with the outputs' own rounding.
template <typename E, int ACT>
__global__ void __launch_bounds__(256) glu_act_grad_kernel(const E* dh, const E* gu, int64_t n,
                                                           int segs, E* __restrict__ dgu) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  const int64_t F = (int64_t)segs * 8;
  pdl_wait_for(dh, gu);
  pdl_launch();
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
    const int64_t t = i / segs;
    const int64_t at = i * 8 + t * F;  // 2 F t + f
    const Vec8 d = unpack(ld8_stream(dh + i * 8)), g = unpack(ld8_stream(gu + at)), u = unpack(ld8_stream(gu + at + F));
    Vec8 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = activate_grad<ACT>(g.p[e].x), y = activate_grad<ACT>(g.p[e].y);
      a.p[e] = make_float2(d.p[e].x * u.p[e].x * x.y, d.p[e].y * u.p[e].y * y.y);
      b.p[e] = make_float2(d.p[e].x * x.x, d.p[e].y * y.x);
    }
    st8(dgu + at, pack<E>(a));
    st8(dgu + at + F, pack<E>(b));
  }
}

// Rows of dx (product 0) and of dw (product 1, of E or fp32, perhaps added to).
template <typename E, int BN>
struct GradEpilogue {
  E* dx;
  void* dw;
  int64_t T, F2, H;
  bool dw32, accumulate;
  bool swapped;  // product 0 is dw's

  __device__ __forceinline__ int row_b(int n, int j) const { return n * BN + j; }
  template <typename O>
  __device__ __forceinline__ void put(O* out, const float* v, bool add) const {
    Vec8 a;
#pragma unroll
    for (int e = 0; e < 4; ++e) a.p[e] = make_float2(v[2 * e], v[2 * e + 1]);
    if (add) {
      const Vec8 o = unpack(ld8(out));
#pragma unroll
      for (int e = 0; e < 4; ++e) a.p[e] = make_float2(a.p[e].x + o.p[e].x, a.p[e].y + o.p[e].y);
    }
    st8(out, pack<O>(a));
  }
  template <typename Source>
  __device__ __forceinline__ void store(const Source& from, int64_t row, int n, int which, int part) const {
    const bool is_w = (which != 0) != swapped;
#pragma unroll 1
    for (int c = part * 16; c < BN; c += 32) {
      float v[16];
      from.get(c, v);
      if (row >= (is_w ? F2 : T)) continue;
#pragma unroll
      for (int p = 0; p < 16; p += 8) {  // eight columns: H is a multiple of eight
        const int64_t col = (int64_t)n * BN + c + p;
        if (col >= H) break;
        const int64_t at = row * H + col;
        if (!is_w) put(dx + at, v + p, false);
        else if (dw32) put(static_cast<float*>(dw) + at, v + p, accumulate);
        else put(static_cast<E*>(dw) + at, v + p, accumulate);
      }
    }
  }
};

// dx = dgu w: the reduction runs over w's rows.  dw = dgu^T x: over the tokens.
template <typename E, typename S>
static cudaError_t grad_products(const void* x, int64_t ld_x, const void* w, int64_t T, int H, int64_t F2, const void* dgu, void* dx,
                                 void* dw, bool dw32, bool accumulate, bool w_first, void* ws, cudaStream_t s) {
  const int64_t cols = (H + S::BN - 1) / S::BN;
  const GradEpilogue<E, S::BN> epi = {static_cast<E*>(dx), dw, T, F2, H, dw32, accumulate, w_first};
  auto make = [&](Problem* p, bool is_w) {
    return is_w ? problem<E, S>(p, F2, cols, T, dgu, true, F2, x, H, ld_x) : problem<E, S>(p, T, cols, F2, dgu, false, F2, w, H, H);
  };
  if (dx && dw) {
    Work<2> p;
    if (!make(&p.p[0], w_first) || !make(&p.p[1], !w_first)) return cudaErrorInvalidValue;
    return product_launch<E, S, 2>(p, ws, epi, s);
  }
  Work<1> p;
  if (!make(&p.p[0], w_first)) return cudaErrorInvalidValue;
  return product_launch<E, S, 1>(p, ws, epi, s);
}

template <typename E>
static cudaError_t glu_grad_launch(const void* dh, const void* gu, const void* x, int64_t ld_x, const void* w, int act, int64_t T,
                                   int H, int F, void* dgu, void* dx, void* dw, bool dw32, bool accumulate, void* ws,
                                   cudaStream_t s) {
  const int segs = F / 8;
  const int64_t n = T * segs;
  int64_t blocks = (n + 255) / 256;
  if (blocks > 0x7fffffff) blocks = 0x7fffffff;
  auto k = act == MHC_ACT_SILU   ? glu_act_grad_kernel<E, MHC_ACT_SILU>
           : act == MHC_ACT_GELU ? glu_act_grad_kernel<E, MHC_ACT_GELU>
           : act == MHC_ACT_RELU ? glu_act_grad_kernel<E, MHC_ACT_RELU>
                                 : glu_act_grad_kernel<E, MHC_ACT_GELU_TANH>;
  const cudaError_t e = launch_pdl(k, dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const E*>(dh), static_cast<const E*>(gu), n,
                                   segs, static_cast<E*>(dgu));
  if (e != cudaSuccess || (!dx && !dw)) return e;
  const int64_t F2 = 2 * (int64_t)F;
  const bool both = dx && dw, w_first = both ? T > F2 : dx == nullptr;  // the product of more stages comes first
  if (product_small(
          [&](int i, int rows, int columns, int64_t* n, int64_t* k) {
            const bool is_w = (i == 0) == w_first;
            *n = (((is_w ? F2 : T) + rows - 1) / rows) * ((H + columns - 1) / columns);
            *k = ((is_w ? T : F2) + kBK - 1) / kBK;
          },
          both ? 2 : 1))
    return grad_products<E, Tile<1, 128, true>>(x, ld_x, w, T, H, F2, dgu, dx, dw, dw32, accumulate, w_first, ws, s);
  return grad_products<E, Tile<2, 256, true>>(x, ld_x, w, T, H, F2, dgu, dx, dw, dw32, accumulate, w_first, ws, s);
}

}  // namespace mhc

extern "C" int mhc_glu_grad(const void* dh, const void* gu, const void* x, int64_t ld_x, const void* w, int act, int64_t T, int H,
                            int F, mhc_dtype dtype, void* dgu, void* dx, void* dw, mhc_dtype dw_dtype, int accumulate,
                            void* workspace, size_t ws_bytes, void* stream) {
  using namespace mhc;
  if (dtype != MHC_DT_BF16 && dtype != MHC_DT_F16) return ops_fail(MHC_ERR_CONFIG, "dtype must be bf16 or fp16");
  if (dw && dw_dtype != MHC_DT_F32 && dw_dtype != dtype) return ops_fail(MHC_ERR_CONFIG, "dw_dtype must be fp32 or dtype");
  if (!act_ok(act)) return ops_fail(MHC_ERR_CONFIG, "unknown activation");
  if (T < 0 || T > (1 << 30) || H <= 0 || H % 8 != 0 || H > (1 << 20) || F <= 0 || F % 8 != 0 || F > (1 << 20))
    return ops_fail(MHC_ERR_SHAPE, "need 0 <= T <= 2^30, H and F positive multiples of 8, at most 2^20");
  if (ld_x < H || ld_x % 8 != 0 || ld_x > (1ll << 36)) return ops_fail(MHC_ERR_SHAPE, "ld_x must be a multiple of 8, at least H");
  const int64_t F2 = 2 * (int64_t)F;
  const size_t wb = dw_dtype == MHC_DT_F32 ? 4 : 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!ops_aligned(dw, 16)) return ops_fail(MHC_ERR_ALIGN, "matrices and the workspace must be 16-byte aligned");
  if (T == 0) {
    if (!dw || accumulate) return MHC_OK;
    return ops_cuda(cudaMemsetAsync(dw, 0, (size_t)F2 * H * wb, s), "clearing dw");
  }
  if (!dh || !gu || !dgu || (dx && !w) || (dw && !x)) return ops_fail(MHC_ERR_NULL, "dh, gu and dgu are required, w for dx, x for dw");
  for (const void* p : {dh, gu, x, w, (const void*)dgu, (const void*)dx, (const void*)workspace})
    if (!ops_aligned(p, 16)) return ops_fail(MHC_ERR_ALIGN, "matrices and the workspace must be 16-byte aligned");
  if (!workspace || ws_bytes < mhc_glu_workspace_bytes(T, H, F))
    return ops_fail(MHC_ERR_WORKSPACE, "workspace NULL or smaller than mhc_glu_workspace_bytes()");
  const size_t tf = (size_t)T * F * 2;
  const Rows in[] = {{x, T, H, ld_x, 2}, {w, F2, H, H, 2}, {dh, T, F, F, 2}, {gu, T, F2, F2, 2}};
  const struct { const void* p; size_t n; } out[] = {{dgu, 2 * tf}, {dx, (size_t)T * H * 2}, {dw, (size_t)F2 * H * wb}, {workspace, ws_bytes}};
  for (int i = 0; i < 4; ++i) {
    for (const Rows& r : in)
      if (rows_overlap({out[i].p, 1, (int64_t)out[i].n, (int64_t)out[i].n, 1}, r))
        return ops_fail(MHC_ERR_ALIAS, "an output or the workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (bytes_overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return ops_fail(MHC_ERR_ALIAS, "the outputs and the workspace overlap");
  }
  const bool dw32 = dw_dtype == MHC_DT_F32;
  const cudaError_t e = dtype == MHC_DT_BF16 ? glu_grad_launch<__nv_bfloat16>(dh, gu, x, ld_x, w, act, T, H, F, dgu, dx, dw, dw32,
                                                                              accumulate != 0, workspace, s)
                                             : glu_grad_launch<__half>(dh, gu, x, ld_x, w, act, T, H, F, dgu, dx, dw, dw32,
                                                                       accumulate != 0, workspace, s);
  return ops_cuda(e, "glu gradient launch");
}
