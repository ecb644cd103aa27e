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
  float2 p[4];
};

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ Vec8 zero8() {
  Vec8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = make_float2(0.f, 0.f);
  return o;
}

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
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o.p[2 * i] = make_float2(__uint_as_float(r.q[i].x), __uint_as_float(r.q[i].y));
      o.p[2 * i + 1] = make_float2(__uint_as_float(r.q[i].z), __uint_as_float(r.q[i].w));
    }
  } else {
    o.p[0] = pair_of(r.q[0].x, T());
    o.p[1] = pair_of(r.q[0].y, T());
    o.p[2] = pair_of(r.q[0].z, T());
    o.p[3] = pair_of(r.q[0].w, T());
  }
  return o;
}

template <typename T>
__device__ __forceinline__ Raw8<T> pack(const Vec8& x) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.q[i] = make_uint4(__float_as_uint(x.p[2 * i].x), __float_as_uint(x.p[2 * i].y), __float_as_uint(x.p[2 * i + 1].x),
                          __float_as_uint(x.p[2 * i + 1].y));
  } else {
    r.q[0] = make_uint4(word_of(x.p[0].x, x.p[0].y, T()), word_of(x.p[1].x, x.p[1].y, T()),
                        word_of(x.p[2].x, x.p[2].y, T()), word_of(x.p[3].x, x.p[3].y, T()));
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
// (a 32-byte store of fp32 columns writes whole sectors; the pointer is 32-byte
// aligned where the row is)
__device__ __forceinline__ void st32(float* p, const Raw8<float>& r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.q[0].x), "r"(r.q[0].y), "r"(r.q[0].z),
               "r"(r.q[0].w), "r"(r.q[1].x), "r"(r.q[1].y), "r"(r.q[1].z), "r"(r.q[1].w)
               : "memory");
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

// ------------------------------------------------ rows fetched ahead of use --
// A thread copies the eight columns it will work on into shared memory of its
// own (cp.async), some rows ahead: nobody else reads them, so its own
// wait_group is the only synchronisation.  Shared addresses are 32-bit, global
// ones a row's address plus a 32-bit offset.  The 16-byte halves of fp32 columns
// lie in two planes of `plane` bytes, so a warp's accesses are free of bank
// conflicts.
__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
template <typename T>
__device__ __forceinline__ void fetch8(uint32_t smem, uint32_t plane, const char* src) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) cp_async16(smem + i * plane, src + i * 16);
}
template <typename T>
__device__ __forceinline__ Raw8<T> fetched8(uint32_t smem, uint32_t plane) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = lds16(smem + i * plane);
  return r;
}

// ------------------------------------------------------------------ sums --
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// ------------------------------------------- programmatic dependent launch --
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// pdl_wait() for a kernel that then reads through these pointers: the reads cannot be moved
// above it, whatever the compiler takes them for.
template <typename... P>
__device__ __forceinline__ void pdl_wait_for(P*&... p) {
  pdl_wait();
  (..., [](P*& q) { asm volatile("" : "+l"(q)::"memory"); }(p));
}
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

// Allows a kernel `bytes` of dynamic shared memory, once per kernel and device.
// (An attribute of the function, no stream work: also legal during capture.)
struct SmemGrant {
  std::mutex mu;
  size_t have[64] = {};
};
inline cudaError_t allow_smem(SmemGrant& grant, const void* kernel, size_t bytes) {
  if (bytes <= 40 * 1024) return cudaSuccess;  // with the static part, within the default of 48 KB
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(grant.mu);
  if (grant.have[dev] >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) grant.have[dev] = bytes;
  else cudaGetLastError();  // it is this call's, not the next one's
  return e;
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  if (e != cudaSuccess) cudaGetLastError();  // it is this call's, not the next one's
  return e;
}

}  // namespace mhc

// Calls `F` with the element type that `dtype` names.
#define MHC_BY_DTYPE(dtype, T, ...)                       \
  switch (dtype) {                                        \
    case MHC_DT_BF16: { using T = __nv_bfloat16; __VA_ARGS__; break; } \
    case MHC_DT_F16: { using T = __half; __VA_ARGS__; break; }         \
    default: { using T = float; __VA_ARGS__; break; }     \
  }
