// mhc_dropout: dropout before a residual add, with a mask that is never stored.

#include "mhc_ops.cuh"

namespace mhc {

// Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): a 128-bit counter under a 64-bit key to
// four 32-bit words.  A round is (a, b, c, d) -> (hi(c M1) ^ b ^ k0, lo(c M1),
// hi(a M0) ^ d ^ k1, lo(a M0)); the key then moves on by (W0, W1).
struct Philox {
  uint32_t k0[10], k1[10];
  __device__ __forceinline__ explicit Philox(uint64_t key) {
    k0[0] = (uint32_t)key;
    k1[0] = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 1; r < 10; ++r) {
      k0[r] = k0[r - 1] + 0x9E3779B9u;
      k1[r] = k1[r - 1] + 0xBB67AE85u;
    }
  }
  __device__ __forceinline__ uint4 operator()(uint64_t lo, uint64_t hi) const {
    uint32_t a = (uint32_t)lo, b = (uint32_t)(lo >> 32), c = (uint32_t)hi, d = (uint32_t)(hi >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
      a = (uint32_t)(q >> 32) ^ b ^ k0[r];
      b = (uint32_t)q;
      c = (uint32_t)(p >> 32) ^ d ^ k1[r];
      d = (uint32_t)p;
    }
    return make_uint4(a, b, c, d);
  }
};

// out = r + (word >= threshold ? scale * y : 0), one rounding.  The word of element
// i = t H + h is word i % 4 of Philox(counter i / 4 and the call's number), so it
// depends on neither strides nor launch shape, and the gradient's call makes the
// same ones.  Work item = 8 adjacent columns = two counters.
template <typename T, bool RES, bool DENSE>
__global__ void __launch_bounds__(256) dropout_kernel(const T* y, int64_t ld_y, const T* r, int64_t ld_r,
                                                      const uint64_t* __restrict__ seed, uint32_t threshold, bool any,
                                                      float scale, int64_t n, int segs, T* out, int64_t ld_o) {
  const Philox draw(seed[0]);
  const uint64_t call = seed[1];
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
    int64_t t = 0, c = i * 8;
    if constexpr (!DENSE) {
      t = i / segs;
      c = (i - t * segs) * 8;
    }
    const Vec8 v = unpack(ld8_stream(y + t * ld_y + c));
    Vec8 x = zero8();
    if constexpr (RES) x = unpack(ld8_stream(r + t * ld_r + c));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 w = draw(2 * (uint64_t)i + h, call);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float2 &o = x.p[2 * h + e], a = v.p[2 * h + e];
        // (a dropped NaN or infinity leaves no trace)
        o.x = any && u[2 * e] >= threshold ? fmaf(a.x, scale, o.x) : o.x;
        o.y = any && u[2 * e + 1] >= threshold ? fmaf(a.y, scale, o.y) : o.y;
      }
    }
    st8_stream(out + t * ld_o + c, pack<T>(x));
  }
}

template <typename T, bool RES>
static cudaError_t dropout_launch(const void* y, int64_t ld_y, const void* r, int64_t ld_r, const void* seed, uint32_t threshold,
                                  bool any, float scale, int64_t T_, int H, void* out, int64_t ld_o, cudaStream_t s) {
  const int segs = H / 8;
  const int64_t n = T_ * segs;
  const bool dense = T_ == 1 || (ld_y == H && ld_o == H && (!RES || ld_r == H));
  int64_t blocks = (n + 255) / 256;
  if (blocks > 0x7fffffff) blocks = 0x7fffffff;
  auto k = dense ? dropout_kernel<T, RES, true> : dropout_kernel<T, RES, false>;
  k<<<(unsigned)blocks, 256, 0, s>>>(static_cast<const T*>(y), ld_y, static_cast<const T*>(r), ld_r,
                                     static_cast<const uint64_t*>(seed), threshold, any, scale, n, segs, static_cast<T*>(out), ld_o);
  return cudaGetLastError();
}

}  // namespace mhc

extern "C" int mhc_dropout(const void* y, int64_t ld_y, const void* r, int64_t ld_r, double p, const uint64_t* seed, int64_t T,
                           int H, mhc_dtype dtype, void* out, int64_t ld_out, void* stream) {
  using namespace mhc;
  if (!dtype_ok(dtype)) return ops_fail(MHC_ERR_CONFIG, "unknown dtype");
  if (!(p >= 0.0 && p <= 1.0)) return ops_fail(MHC_ERR_CONFIG, "p must be in [0, 1]");
  if (T < 0 || T > 0x7fffffff || H <= 0 || H % 8 != 0)
    return ops_fail(MHC_ERR_SHAPE, "need 0 <= T < 2^31 and H a positive multiple of 8");
  if (ld_y < H || ld_y % 8 != 0 || ld_out < H || ld_out % 8 != 0 || (r && (ld_r < H || ld_r % 8 != 0)))
    return ops_fail(MHC_ERR_SHAPE, "row strides must be multiples of 8, at least H");
  if (T == 0) return MHC_OK;
  if (!y || !out || !seed) return ops_fail(MHC_ERR_NULL, "y, out and seed are required");
  if (!ops_aligned(y, 16) || !ops_aligned(r, 16) || !ops_aligned(out, 16) || !ops_aligned(seed, 8))
    return ops_fail(MHC_ERR_ALIGN, "y, r and out must be 16-byte aligned, seed 8-byte");
  const size_t b = dtype_bytes(dtype);
  const Rows o = {out, T, H, ld_out, b};
  // in place on y or r: each element is read by the thread that writes it
  if ((rows_overlap(o, {y, T, H, ld_y, b}) && !(out == y && ld_out == ld_y)) ||
      (rows_overlap(o, {r, T, H, ld_r, b}) && !(out == r && ld_out == ld_r)) || rows_overlap(o, {seed, 1, 2, 2, 8}))
    return ops_fail(MHC_ERR_ALIAS, "out overlaps an input (other than y or r exactly)");
  const double cut = floor(p * 4294967296.0 + 0.5);
  const bool any = cut < 4294967296.0;  // p = 1 keeps nothing
  const uint32_t threshold = any ? (uint32_t)cut : 0;
  const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
  cudaError_t e = cudaSuccess;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  MHC_BY_DTYPE(dtype, E, {
    e = r ? dropout_launch<E, true>(y, ld_y, r, ld_r, seed, threshold, any, scale, T, H, out, ld_out, s)
          : dropout_launch<E, false>(y, ld_y, r, ld_r, seed, threshold, any, scale, T, H, out, ld_out, s);
  });
  return ops_cuda(e, "dropout launch");
}
