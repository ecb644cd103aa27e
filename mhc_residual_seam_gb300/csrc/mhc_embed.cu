// mhc_embed: rows of an embedding table into the residual streams.

#include "mhc_ops.cuh"

namespace mhc {

// out[t, s, :] = round(scale * table[ids[t] - first, :]) for every stream s; a
// zero row where the id is outside the table.  Bound by HBM: each row is read
// once and written `streams` times.  Work item = (token, 8 columns), in row
// order, so a warp reads and writes 512 adjacent bytes (16-bit types).  One item a
// thread: CTAs start as others end, and an SM that gets through faster takes more
// (T = 16384, H = 5120, four streams: 113 us, 96 % of the copy; with 64 CTAs per SM
// and a loop 117, with 16 127).
template <typename T, typename Id>
__global__ void __launch_bounds__(256) embed_kernel(const Id* __restrict__ ids, const T* __restrict__ table, int64_t ld,
                                                    int64_t V, int64_t first, float scale, int64_t n, int segs, int streams,
                                                    T* __restrict__ out) {
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
    const int64_t t = i / segs;
    const int64_t c = (i - t * segs) * 8;
    const uint64_t row = (uint64_t)(int64_t)ids[t] - (uint64_t)first;  // ids below `first` wrap to above V
    Vec8 x = zero8();
    if (row < (uint64_t)V) {
      x = unpack(ld8(table + (int64_t)row * ld + c));
#pragma unroll
      for (int e = 0; e < 4; ++e) x.p[e] = __fmul2_rn(x.p[e], splat(scale));
    }
    const Raw8<T> r = pack<T>(x);
    T* o = out + t * streams * (int64_t)segs * 8 + c;
    for (int s = 0; s < streams; ++s, o += (int64_t)segs * 8) st8_stream(o, r);
  }
}

template <typename T, typename Id>
static cudaError_t embed_launch(const void* ids, const void* table, int64_t ld, int64_t V, int64_t first, float scale,
                                int64_t T_, int H, int streams, void* out, cudaStream_t s) {
  const int segs = H / 8;
  const int64_t n = T_ * segs;
  int64_t blocks = (n + 255) / 256;
  if (blocks > 0x7fffffff) blocks = 0x7fffffff;
  embed_kernel<T, Id><<<(unsigned)blocks, 256, 0, s>>>(static_cast<const Id*>(ids), static_cast<const T*>(table), ld, V,
                                                       first, scale, n, segs, streams, static_cast<T*>(out));
  return cudaGetLastError();
}

}  // namespace mhc

extern "C" int mhc_embed(const void* ids, int id_bytes, const void* table, int64_t table_ld, int64_t V, int64_t first_id,
                         float scale, int64_t T, int H, int streams, mhc_dtype dtype, void* out, void* stream) {
  using namespace mhc;
  if (!dtype_ok(dtype)) return ops_fail(MHC_ERR_CONFIG, "unknown dtype");
  if (id_bytes != 4 && id_bytes != 8) return ops_fail(MHC_ERR_CONFIG, "id_bytes must be 4 or 8");
  if (T < 0 || V < 0 || H <= 0 || H % 8 != 0 || streams < 1 || streams > 64)
    return ops_fail(MHC_ERR_SHAPE, "need T >= 0, V >= 0, H a positive multiple of 8 and 1 <= streams <= 64");
  if (table_ld < H || table_ld % 8 != 0) return ops_fail(MHC_ERR_SHAPE, "table_ld must be a multiple of 8, at least H");
  if (T == 0) return MHC_OK;
  if (!ids || (!table && V) || !out) return ops_fail(MHC_ERR_NULL, "ids, table and out are required");
  if (!ops_aligned(ids, id_bytes) || !ops_aligned(table, 16) || !ops_aligned(out, 16))
    return ops_fail(MHC_ERR_ALIGN, "table and out must be 16-byte aligned, ids to their size");
  const size_t b = dtype_bytes(dtype);
  const Rows o = {out, T, (int64_t)streams * H, (int64_t)streams * H, b};
  if (rows_overlap(o, {ids, 1, T, T, (size_t)id_bytes}) || rows_overlap(o, {table, V, H, table_ld, b}))
    return ops_fail(MHC_ERR_ALIAS, "out overlaps an input");
  cudaError_t e = cudaSuccess;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  MHC_BY_DTYPE(dtype, E, {
    e = id_bytes == 4 ? embed_launch<E, int32_t>(ids, table, table_ld, V, first_id, scale, T, H, streams, out, s)
                      : embed_launch<E, int64_t>(ids, table, table_ld, V, first_id, scale, T, H, streams, out, s);
  });
  return ops_cuda(e, "embed launch");
}
