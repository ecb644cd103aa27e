// mhc_dropout: dropout before a residual add, with a mask that is never stored.

#include "mhc_ops.cuh"

namespace mhc {

// Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): a 128-bit counter under a 64-bit key to
// four 32-bit words.  A round is (a, b, c, d) -> (hi(c M1) ^ b ^ k0, lo(c M1),
// hi(a M0) ^ d ^ k1, lo(a M0)); the key then moves on by (W0, W1).
//
// Only the counter's lowest word differs between the calls of one object (the
// upper ones are the call's number and a word that a CTA's span of counters
// shares), so one product of the first round and one of the second are made
// once.  The 18 wide products that are left bound the kernel beside memory.
constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u, kW0 = 0x9E3779B9u, kW1 = 0xBB67AE85u;
__device__ __forceinline__ uint32_t wide(uint32_t x, uint32_t m, uint32_t& lo) {
  const uint64_t p = (uint64_t)x * m;
  lo = (uint32_t)p;
  return (uint32_t)(p >> 32);
}
struct Philox {
  uint32_t k0[10], k1[10];  // [0] unused; k1[1] and k0[1] hold what rounds 0 and 1 have in common
  uint32_t c0, d1;
  // `upper` is the second word of the counter, `call` its upper half.
  __device__ __forceinline__ Philox(uint64_t key, uint32_t upper, uint64_t call) {
    const uint32_t key0 = (uint32_t)key, key1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 1; r < 10; ++r) {
      k0[r] = key0 + r * kW0;
      k1[r] = key1 + r * kW1;
    }
    uint32_t lq, lp;
    const uint32_t hq = wide((uint32_t)call, kM1, lq);  // round 0: c is the call's lower word
    c0 = (uint32_t)(call >> 32) ^ key1;
    const uint32_t hp = wide(hq ^ upper ^ key0, kM0, lp);  // round 1: a is the same for every counter
    k0[1] ^= lq;
    k1[1] ^= hp;
    d1 = lp;
    // registers, not sums made again at each use
#pragma unroll
    for (int r = 1; r < 10; ++r) {
      asm volatile("" : "+r"(k0[r]));
      asm volatile("" : "+r"(k1[r]));
    }
  }
  __device__ __forceinline__ uint4 operator()(uint32_t lowest) const {
    uint32_t a, b, c, d, l;
    c = wide(lowest, kM0, d) ^ c0;  // round 0
    a = wide(c, kM1, b) ^ k0[1];    // round 1
    c = d ^ k1[1];
    d = d1;
#pragma unroll
    for (int r = 2; r < 10; ++r) {
      const uint32_t hp = wide(a, kM0, l);
      a = wide(c, kM1, c) ^ b ^ k0[r];
      b = c;
      c = hp ^ d ^ k1[r];
      d = l;
    }
    return make_uint4(a, b, c, d);
  }
};

// out = r + (word >= threshold ? scale * y : 0), one rounding.  The word of element
// i = t H + h is word i % 4 of Philox(counter i / 4 and the call's number), so it
// depends on neither strides nor launch shape, and the gradient's call makes the
// same ones.  Work item = 8 adjacent columns = two counters.
// A thread loads the items of its next step before it draws the present one's numbers,
// so memory and the generator overlap.  T = 16384, H = 5120, bf16: with a residual
// 76.5 us (97 % of the copy; 92 with one item a thread and no loop), without one 66.5
// (86), bound by the multiplier's pipe (72 % busy: 36 wide products an item at 4 cycles a
// warp are 41 us) and by dispatch beside it; its warps wait for loads 6 % of their time.
// Two items a step for many rows (with one 86 and 76 us), one where that would leave
// CTAs without work, and for fp32, whose items are twice as large.
constexpr int kCtas = 4, kSteps = 4;

template <typename T, int PER>
struct Items {
  Raw8<T> v[PER], x[PER];
};

template <typename T, bool RES, bool DENSE, int PER>
__global__ void __launch_bounds__(256, kCtas) dropout_kernel(const T* y, int64_t ld_y, const T* r, int64_t ld_r,
                                                      const uint64_t* seed, uint32_t threshold, bool any,
                                                      float scale, int64_t n, int segs, T* out, int64_t ld_o) {
  pdl_wait_for(y, r, seed);
  pdl_launch();
  const uint64_t key = seed[0], call = seed[1];
  auto place = [&](int64_t i, int64_t ld) -> int64_t {
    if constexpr (DENSE) return i * 8;
    const int64_t t = i / segs;
    return t * ld + (i - t * segs) * 8;
  };
  auto load = [&](Items<T, PER>& it, int64_t first) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t i = first + k * 256;
      if (i >= n) break;
      it.v[k] = ld8_stream(y + place(i, ld_y));
      if constexpr (RES) it.x[k] = ld8_stream(r + place(i, ld_r));
    }
  };
  const int64_t stride = (int64_t)gridDim.x * 256 * PER;
  int64_t first = (int64_t)blockIdx.x * 256 * PER + threadIdx.x;
  Items<T, PER> now, next;
  load(now, first);
  // the CTA's 512 PER counters of one step share their upper word: PER is a power of two
  static_assert((PER & (PER - 1)) == 0, "");
  uint32_t upper = (uint32_t)((uint64_t)first * 2 >> 32);
  Philox draw(key, upper, call);
  for (; first < n; first += stride) {
    load(next, first + stride);
    if (upper != (uint32_t)((uint64_t)first * 2 >> 32)) {
      upper = (uint32_t)((uint64_t)first * 2 >> 32);
      draw = Philox(key, upper, call);
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t i = first + k * 256;
      if (i >= n) break;
      const Vec8 a = unpack(now.v[k]);
      Vec8 o = zero8();
      if constexpr (RES) o = unpack(now.x[k]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 w = draw(2 * (uint32_t)i + h);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 &q = o.p[2 * h + e], f = a.p[2 * h + e];
          // (a dropped NaN or infinity leaves no trace)
          q.x = any && u[2 * e] >= threshold ? fmaf(f.x, scale, q.x) : q.x;
          q.y = any && u[2 * e + 1] >= threshold ? fmaf(f.y, scale, q.y) : q.y;
        }
      }
      st8_stream(out + place(i, ld_o), pack<T>(o));
    }
    now = next;
  }
}

template <typename T, bool RES>
static cudaError_t dropout_launch(const void* y, int64_t ld_y, const void* r, int64_t ld_r, const void* seed, uint32_t threshold,
                                  bool any, float scale, int64_t T_, int H, void* out, int64_t ld_o, cudaStream_t s) {
  const int segs = H / 8;
  const int64_t n = T_ * segs;
  const bool dense = T_ == 1 || (ld_y == H && ld_o == H && (!RES || ld_r == H));
  constexpr int kPer = sizeof(T) == 4 ? 1 : 2;
  const bool many = n >= 152 * kCtas * 256 * kPer;
  int64_t blocks = (n + 256 * (many ? kPer : 1) - 1) / (256 * (many ? kPer : 1));
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (blocks > (int64_t)sms * kCtas * kSteps) blocks = (int64_t)sms * kCtas * kSteps;
  auto k = many ? dense ? dropout_kernel<T, RES, true, kPer> : dropout_kernel<T, RES, false, kPer>
                : dense ? dropout_kernel<T, RES, true, 1> : dropout_kernel<T, RES, false, 1>;
  return launch_pdl(k, dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const T*>(y), ld_y, static_cast<const T*>(r), ld_r,
                    static_cast<const uint64_t*>(seed), threshold, any, scale, n, segs, static_cast<T*>(out), ld_o);
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
