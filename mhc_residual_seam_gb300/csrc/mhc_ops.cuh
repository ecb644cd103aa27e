// What the operators around the seam (embedding, block norms, routing) share:
// eight-column vectors of the three element types held as fp32 in registers,
// sums over a warp or a block, programmatic dependent launch, and the host
// side's argument checks.
#pragma once

#include <mutex>
#include <string>

#include "mhc_common.cuh"
#include "../../include/mhc_seam.h"

namespace mhc {

void set_last_error(const std::string& msg);  // mhc_api.cu: the text mhc_last_error_string() returns

// ------------------------------------------------- eight columns of a row --
// A thread works on eight adjacent columns whatever the type: one 16-byte
// access for the 16-bit types, two for fp32.  Sums and products are fp32;
// store8 rounds once, to nearest even.
struct Vec8 {
  float v[8];
};

template <typename T>
struct Raw8 {  // eight columns as they lie in memory
  uint4 q[sizeof(T) / 2];
};

__device__ __forceinline__ float2 pair_of(uint32_t u, __nv_bfloat16) { return bf16pair(u); }
__device__ __forceinline__ float2 pair_of(uint32_t u, __half) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
__device__ __forceinline__ uint32_t word_of(float a, float b, __nv_bfloat16) { return pack_bf16x2(a, b); }
__device__ __forceinline__ uint32_t word_of(float a, float b, __half) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ Vec8 unpack(const Raw8<T>& r) {
  Vec8 o;
  if constexpr (sizeof(T) == 4) {
    o.v[0] = __uint_as_float(r.q[0].x); o.v[1] = __uint_as_float(r.q[0].y);
    o.v[2] = __uint_as_float(r.q[0].z); o.v[3] = __uint_as_float(r.q[0].w);
    o.v[4] = __uint_as_float(r.q[1].x); o.v[5] = __uint_as_float(r.q[1].y);
    o.v[6] = __uint_as_float(r.q[1].z); o.v[7] = __uint_as_float(r.q[1].w);
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = pair_of(w[i], T());
      o.v[2 * i] = p.x;
      o.v[2 * i + 1] = p.y;
    }
  }
  return o;
}

template <typename T>
__device__ __forceinline__ Raw8<T> pack(const Vec8& x) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
    r.q[0] = make_uint4(__float_as_uint(x.v[0]), __float_as_uint(x.v[1]), __float_as_uint(x.v[2]), __float_as_uint(x.v[3]));
    r.q[1] = make_uint4(__float_as_uint(x.v[4]), __float_as_uint(x.v[5]), __float_as_uint(x.v[6]), __float_as_uint(x.v[7]));
  } else {
    r.q[0] = make_uint4(word_of(x.v[0], x.v[1], T()), word_of(x.v[2], x.v[3], T()), word_of(x.v[4], x.v[5], T()),
                        word_of(x.v[6], x.v[7], T()));
  }
  return r;
}

template <typename T>
__device__ __forceinline__ Raw8<T> ld8(const T* p) {  // read through the cache (reused)
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = *(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ Raw8<T> ld8_stream(const T* p) {  // read once
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ void st8(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) *(reinterpret_cast<uint4*>(p) + i) = r.q[i];
}
template <typename T>
__device__ __forceinline__ void st8_stream(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) __stcs(reinterpret_cast<uint4*>(p) + i, r.q[i]);
}

// ------------------------------------------------------------------ sums --
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// ------------------------------------------- programmatic dependent launch --
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------ host --
inline int ops_fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}
inline int ops_cuda(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MHC_OK;
  set_last_error(std::string(what) + ": " + cudaGetErrorString(e));
  return MHC_ERR_CUDA;
}

inline bool ops_aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t dtype_bytes(int t) { return t == MHC_DT_F32 ? 4 : 2; }
inline bool dtype_ok(int t) { return t == MHC_DT_BF16 || t == MHC_DT_F16 || t == MHC_DT_F32; }

// A [rows, width] matrix of `ld` elements from row to row.
struct Rows {
  const void* p;
  int64_t rows, width, ld;
  size_t size;  // bytes per element
};

// Whether two matrices share a byte.  Matrices with the same row stride may
// interleave (two streams of one [T,4,H] tensor); others are compared as whole
// ranges.
inline bool rows_overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t ea = pa + ((size_t)(a.rows - 1) * a.ld + a.width) * a.size;
  const uintptr_t eb = pb + ((size_t)(b.rows - 1) * b.ld + b.width) * b.size;
  if (ea <= pb || eb <= pa) return false;
  const size_t sa = (size_t)a.ld * a.size, sb = (size_t)b.ld * b.size;
  if (sa != sb || a.rows == 1 || b.rows == 1) return true;
  const size_t d = pb >= pa ? (pb - pa) % sa : (sa - (pa - pb) % sa) % sa;  // b's row start within a's row
  return d < a.width * a.size || d + b.width * b.size > sa;
}

// SM count of the current device, asked for once per device.
inline cudaError_t sm_count(int* out) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!known[dev]) {
    e = cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
  }
  *out = known[dev];
  return cudaSuccess;
}

// Launch that may begin while the kernel before it on the stream ends; the
// kernel calls pdl_wait() before it touches what that kernel wrote.
template <typename... Params, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace mhc

// Calls `F` with the element type that `dtype` names.
#define MHC_BY_DTYPE(dtype, T, ...)                       \
  switch (dtype) {                                        \
    case MHC_DT_BF16: { using T = __nv_bfloat16; __VA_ARGS__; break; } \
    case MHC_DT_F16: { using T = __half; __VA_ARGS__; break; }         \
    default: { using T = float; __VA_ARGS__; break; }     \
  }
