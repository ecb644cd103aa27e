// mhc_embed_grad: the gradient of an embedding table from tokens sorted by row.
//
// dtable[v] = scale * sum over the tokens t of row v, in token order, of
// sum_s dout[t, s].  Three steps:
//   1. a stable radix sort of the tokens by row (tokens of no row get the key V,
//      which sorts behind all rows);
//   2. the rows' ends and the sorted tokens are one merged list (a row's end
//      comes behind its tokens); the list is cut into chunks of equal bytes,
//      and each CTA walks one chunk: a token is added to the sum in registers, a
//      row's end writes it (zero where the row has no token);
//   3. a row whose tokens lie in more than one chunk is joined: the chunks'
//      partial sums in chunk order, then the last chunk's tokens.
// No float atomics, so the result does not depend on timing.  Bound by HBM at size:
// T = 16384, V = 131072, H = 5120, four streams, fp32: 558 us for 3.36 GB, 89 % of the
// copy, 541 of them in step 2.

#include "mhc_ops.cuh"

namespace mhc {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kFewTokens = 65536;                            // up to here a tile is kSortThreads tokens, above four times that
constexpr int kDigits = 512;                                 // 9-bit digits at most
constexpr int kColumns = 1024;                               // columns per CTA of the sum
constexpr int kSumThreads = kColumns / 8;

constexpr int kJoinCtas = 1024;  // of the join, over all columns: it takes the rows to join from a list

struct alignas(16) Bounds {  // a chunk's first token and row, and the ones behind its last
  int a0, a1, b0, b1;
};

struct EmbedGradWs {  // byte offsets into the workspace
  size_t key[2], tok[2], hist, places, valid, joins, bounds, carry, total;
  int tiles, chunks, passes, digit_bits;
  bool one;  // one CTA sorts
};
constexpr int kSumRounds = 8;

struct SortArgs {
  const void* ids;
  int64_t first, V, pad;
  bool has_pad;
  int T, bits, shift, tiles;
  uint32_t *key_in, *key_out;
  int *tok_in, *tok_out;
  int *hist_in, *hist_out;  // [tiles][kDigits] of this pass and of the next one
  int passes;
  int* places;              // [tiles][kDigits] of this pass: where a tile's keys of a digit go; null: from the counts
  int* valid;               // [tiles] tokens that have a row
  int* joins;               // how many rows the join has to finish, set to 0 here
};

template <typename Id>
__device__ __forceinline__ uint32_t row_of(const SortArgs& a, int t) {
  const int64_t id = (int64_t) static_cast<const Id*>(a.ids)[t];
  const uint64_t row = (uint64_t)id - (uint64_t)a.first;
  return row < (uint64_t)a.V && !(a.has_pad && id == a.pad) ? (uint32_t)row : (uint32_t)a.V;
}

// Digit counts of each tile for the first pass, the rows of the tokens, and
// zeroed counts for the later passes (which follow the first one's).
template <typename Id, int R>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a) {
  constexpr int kSortTile = kSortThreads * R;
  __shared__ int count[kDigits];
  __shared__ int valid;
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) count[d] = 0;
  if (threadIdx.x == 0) valid = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.joins = 0;
  __syncthreads();
  const int base = (int)blockIdx.x * kSortTile;
  int mine = 0;
  for (int i = threadIdx.x; i < kSortTile && base + i < a.T; i += kSortThreads) {
    const uint32_t k = row_of<Id>(a, base + i);
    a.key_in[base + i] = k;
    mine += k < (uint32_t)a.V;
    atomicAdd(&count[k & ((1u << a.bits) - 1)], 1);
  }
  atomicAdd(&valid, mine);
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) {
    a.hist_in[(int64_t)blockIdx.x * kDigits + d] = count[d];
    for (int p = 1; p < a.passes; ++p) a.hist_in[((int64_t)p * a.tiles + blockIdx.x) * kDigits + d] = 0;
  }
  if (threadIdx.x == 0) a.valid[blockIdx.x] = valid;
}

// The whole sort in one CTA, for up to 1024 * R tokens: keys and tokens stay in
// registers between the passes and change places through shared memory.  One launch
// instead of one per pass and a count.
constexpr int kOneThreads = 1024, kOneWarps = kOneThreads / 32;
constexpr int kOneMost = 4;  // keys per thread at most
static size_t one_smem(int R) { return (size_t)kOneThreads * R * 6 + (size_t)kOneWarps * kDigits * 2; }

template <typename Id, int R>
__global__ void __launch_bounds__(kOneThreads) sort_one_kernel(const SortArgs a) {
  extern __shared__ uint32_t dyn[];
  uint32_t* const keys = dyn;                                                    // [1024 R]
  unsigned short* const toks = reinterpret_cast<unsigned short*>(dyn + kOneThreads * R);  // [1024 R]
  unsigned short* const rank = toks + kOneThreads * R;                           // [kOneWarps][kDigits]
  __shared__ int start[kDigits];
  __shared__ int scan[kDigits / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mask = (1u << a.bits) - 1;
  const int base = warp * 32 * R + lane;  // a warp's keys are in order, 32 at a time
  uint32_t key[R];
  int tok[R];
  int valid = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = base + r * 32;
    tok[r] = i;
    key[r] = i < a.T ? row_of<Id>(a, i) : 0xffffffffu;
    valid += key[r] < (uint32_t)a.V;
  }
  for (int p = 0; p < a.passes; ++p) {
    const int shift = p * a.bits;
    for (int i = threadIdx.x; i < kOneWarps * kDigits / 2; i += kOneThreads) reinterpret_cast<uint32_t*>(rank)[i] = 0;
    __syncthreads();
    int place[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {  // places past T get the digit kDigits: no key
      const uint32_t d = key[r] == 0xffffffffu ? kDigits : (key[r] >> shift) & mask;
      const unsigned peers = __match_any_sync(0xffffffffu, d);
      const unsigned below = peers & ((1u << lane) - 1);
      place[r] = d < kDigits ? rank[warp * kDigits + d] + __popc(below) : 0;
      __syncwarp();
      if (d < kDigits && below == 0) rank[warp * kDigits + d] += (unsigned short)__popc(peers);
      __syncwarp();
    }
    __syncthreads();
    int sum = 0, x = 0;
    if (threadIdx.x < kDigits) {  // the digit's keys in the warps before, and in all
      for (int w = 0; w < kOneWarps; ++w) {
        const int n = rank[w * kDigits + threadIdx.x];
        rank[w * kDigits + threadIdx.x] = (unsigned short)sum;
        sum += n;
      }
      x = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (lane == 31) scan[warp] = x;
    }
    __syncthreads();
    if (threadIdx.x < kDigits) {
      for (int w = 0; w < warp; ++w) x += scan[w];
      start[threadIdx.x] = x - sum;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (key[r] == 0xffffffffu) continue;
      const uint32_t d = (key[r] >> shift) & mask;
      const int at = start[d] + rank[warp * kDigits + d] + place[r];
      keys[at] = key[r];
      toks[at] = (unsigned short)tok[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = base + r * 32;
      if (i < a.T) key[r] = keys[i], tok[r] = toks[i];
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = base + r * 32;
    if (i < a.T) a.key_out[i] = key[r], a.tok_out[i] = tok[r];
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) valid += __shfl_xor_sync(0xffffffffu, valid, d);
  __syncthreads();
  if (lane == 0) start[warp] = valid;
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    for (int w = 0; w < kOneWarps; ++w) n += start[w];
    a.valid[0] = n;
    *a.joins = 0;
  }
}

// Turns the counts of many tiles into places, so that a pass need not read all of
// them: for each digit the keys of smaller digits and of earlier tiles.  First the
// digits' totals and the tiles' sums before (32 digits and 32 slices of tiles per
// CTA); the smaller digits are added by the pass, from `totals`.
__global__ void __launch_bounds__(1024) sort_places_kernel(const int* __restrict__ hist, int tiles, int* __restrict__ places,
                                                           int* __restrict__ totals) {
  __shared__ int sums[32][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t d = blockIdx.x * 32 + lane;
  const int lo = (int)((int64_t)tiles * w / 32), hi = (int)((int64_t)tiles * (w + 1) / 32);
  int sum = 0;
#pragma unroll 8
  for (int b = lo; b < hi; ++b) sum += hist[b * (int64_t)kDigits + d];
  sums[w][lane] = sum;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < w; ++i) before += sums[i][lane];
  if (w == 31) totals[d] = before + sum;
#pragma unroll 8
  for (int b = lo; b < hi; ++b) {
    const int n = hist[b * (int64_t)kDigits + d];
    places[b * (int64_t)kDigits + d] = before;
    before += n;
  }
}

// One pass of the stable sort: a key's place is the keys of smaller digits,
// the same digit in earlier tiles, in earlier warps of the tile, and before it
// in its warp (whose keys are taken in order, 32 at a time).
template <int R>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(const SortArgs a, bool identity, bool last) {
  constexpr int kSortTile = kSortThreads * R, kSortRounds = R;
  __shared__ int start[kDigits];
  __shared__ int scan[kSortWarps];
  __shared__ unsigned short rank[kSortWarps][kDigits];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mask = (1u << a.bits) - 1;
  for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads) (&rank[0][0])[i] = 0;
  pdl_wait();
  // the digit's keys in all tiles and in the tiles before this one
  int before = 0, all = 0;
  if (a.places) {
    before = a.places[(int64_t)blockIdx.x * kDigits + threadIdx.x];
    all = a.places[(int64_t)a.tiles * kDigits + threadIdx.x];
  } else {
    for (int b = 0; b < a.tiles; ++b) {
      const int n = a.hist_in[b * kDigits + threadIdx.x];
      before += b < (int)blockIdx.x ? n : 0;
      all += n;
    }
  }
  int x = all;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) x += scan[w];
  start[threadIdx.x] = x - all + before;
  uint32_t key[kSortRounds];
  int place[kSortRounds];
  const int base = (int)blockIdx.x * kSortTile + warp * 32 * kSortRounds;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int i = base + r * 32 + lane;
    key[r] = i < a.T ? a.key_in[i] : 0xffffffffu;
    const uint32_t d = i < a.T ? (key[r] >> a.shift) & mask : kDigits;  // kDigits: no key
    const unsigned peers = __match_any_sync(0xffffffffu, d);
    const unsigned below = peers & ((1u << lane) - 1);
    place[r] = d < kDigits ? rank[warp][d] + __popc(below) : 0;
    __syncwarp();
    if (d < kDigits && below == 0) rank[warp][d] += (unsigned short)__popc(peers);
    __syncwarp();
  }
  __syncthreads();
  {  // the digit's keys in the warps before
    int sum = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = rank[w][threadIdx.x];
      rank[w][threadIdx.x] = (unsigned short)sum;
      sum += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int i = base + r * 32 + lane;
    if (i >= a.T) continue;
    const uint32_t d = (key[r] >> a.shift) & mask;
    const int at = start[d] + rank[warp][d] + place[r];
    a.key_out[at] = key[r];
    a.tok_out[at] = identity ? i : a.tok_in[i];
    if (!last) atomicAdd(a.hist_out + (int64_t)(at / kSortTile) * kDigits + ((key[r] >> (a.shift + a.bits)) & mask), 1);
  }
}

struct SumArgs {
  const void* dout;
  void* dtable;
  int64_t ld, V;
  int H, streams, tiles, chunks, wt, wr;
  bool accumulate;
  float scale;
  const uint32_t* key;
  const int* tok;
  const int* valid;
  int* joins;  // how many, then the chunks that end a row begun earlier, in any order
  Bounds* bounds;
  float* carry;  // [chunks][2][H]: the sum of the last row's tokens, where it ends later; of the first row's, where
                 // it began earlier
};

// Tokens that have a row: the sum over the sort's tiles.
__device__ __forceinline__ int valid_tokens(const SumArgs& a, int* sh) {
  int n = 0;
  for (int i = threadIdx.x; i < a.tiles; i += blockDim.x) n += a.valid[i];
#pragma unroll
  for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) n += sh[i];
  return n;
}

// Where the merged list is cut so that `target` weight lies before: (token,
// row).  Before token i lie i tokens and key[i] rows' ends.  A warp looks for
// the place, 32 probes at a time.
__device__ __forceinline__ void cut(const SumArgs& a, int n, int64_t target, int* tok, int* row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // the first token that has at least `target` before it
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool less = at < hi && (int64_t)a.wt * at + (int64_t)a.wr * a.key[at] < target;
    const int k = __popc(__ballot_sync(0xffffffffu, less));  // probes 0 .. k-1 lie before
    if (k == 0) {
      hi = lo;
    } else {
      const int last = lo + (k - 1) * step;
      hi = k < 32 && lo + k * step < hi ? lo + k * step : hi;
      lo = last + 1;
    }
  }
  if (lane == 0) {
    const int64_t from = lo ? (int64_t)a.key[lo - 1] : 0, to = lo < n ? (int64_t)a.key[lo] : a.V;
    int64_t r = (target - (int64_t)a.wt * lo + a.wr - 1) / a.wr;
    if (target < (int64_t)a.wt * lo) r = 0;
    *tok = lo;
    *row = (int)(r < from ? from : r > to ? to : r);
  }
}

template <typename O>
__device__ __forceinline__ void store_row(O* o, const Raw8<O>& r, bool wide) {
  if constexpr (sizeof(O) == 4) {
    if (wide) return st32(o, r);
  }
  st8_stream(o, r);
}

template <typename O>
__device__ __forceinline__ void end_row(const SumArgs& a, int64_t row, int64_t c, Vec8 acc, bool wide) {
  O* o = static_cast<O*>(a.dtable) + row * a.ld + c;
#pragma unroll
  for (int e = 0; e < 4; ++e) acc.p[e] = __fmul2_rn(acc.p[e], splat(a.scale));
  if (a.accumulate) {
    const Vec8 old = unpack(ld8(o));
#pragma unroll
    for (int e = 0; e < 4; ++e) acc.p[e] = __fadd2_rn(acc.p[e], old.p[e]);
  }
  store_row(o, pack<O>(acc), wide);
}
__device__ __forceinline__ void add8(Vec8& acc, const Vec8& x) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc.p[e] = __fadd2_rn(acc.p[e], x.p[e]);
}

// Walks one chunk.  The rows of the next GROUP tokens are loaded before the
// present ones are added (GROUP * S loads of 16 or 32 bytes in flight per thread and
// as many being used), whatever rows they belong to.  S: streams, 0 for any number.
constexpr int kWindow = 256;  // tokens of a chunk whose keys are in shared memory at a time
template <typename T, typename O, int S>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumArgs a) {
  constexpr int GROUP = S == 1 ? 4 : S == 2 ? 2 : 1;
  constexpr int LOADS = S ? S : 4;
  __shared__ int sh[kSumThreads / 32];
  __shared__ Bounds sb;
  __shared__ int before;  // the row of the token before the chunk
  __shared__ int wkey[kWindow + 1], wtok[kWindow + 1];
  pdl_wait();
  const int n = valid_tokens(a, sh);
  const int64_t weight = (int64_t)a.wt * n + (int64_t)a.wr * a.V;
  const int chunk = blockIdx.x;
  if (threadIdx.x < 32) {
    cut(a, n, weight * chunk / a.chunks, &sb.a0, &sb.b0);
    __syncwarp();
    if (threadIdx.x == 0) before = sb.a0 ? (int)a.key[sb.a0 - 1] : -1;
  }
  if (threadIdx.x >= 32 ? threadIdx.x < 64 : blockDim.x == 32) {
    if (chunk + 1 < a.chunks) cut(a, n, weight * (chunk + 1) / a.chunks, &sb.a1, &sb.b1);
    else if ((threadIdx.x & 31) == 0) sb.a1 = n, sb.b1 = (int)a.V;
  }
  __syncthreads();
  pdl_launch();
  const Bounds b = sb;
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    a.bounds[chunk] = b;
    if (before == b.b0 && b.b0 < b.b1) a.joins[1 + atomicAdd(a.joins, 1)] = chunk;
  }
  const int64_t c = (int64_t)blockIdx.y * kColumns + threadIdx.x * 8;
  const bool on = c < a.H;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.dtable) | (uintptr_t)(a.ld * sizeof(O))) & 31) == 0;
  float* const carry = a.carry + (int64_t)chunk * 2 * a.H + c;
  const T* const src = static_cast<const T*>(a.dout) + c;
  const int64_t row_elems = (int64_t)a.streams * a.H;
  const Raw8<O> zero = pack<O>(zero8());
  int row = b.b0;
  auto zeros = [&](int to) {  // rows without tokens
    if (!a.accumulate && on)
      for (int r = row; r < to; ++r) store_row(static_cast<O*>(a.dtable) + r * a.ld + c, zero, wide);
    row = to;
  };
  Vec8 acc = zero8();
  auto finish = [&](int k) {  // the tokens of row k end here or in a later chunk
    if (on) {
      if (k >= b.b1) st8(carry, pack<float>(acc));
      else if (k == b.b0 && before == k) st8(carry + a.H, pack<float>(acc));
      else end_row<O>(a, k, c, acc, wide);
    }
    acc = zero8();
    if (k < b.b1) row = k + 1;
  };
  if (before == b.b0 && b.b0 < b.b1 && (b.a0 == b.a1 || (int)a.key[b.a0] != b.b0)) finish(b.b0);  // it has no token here

  for (int w = b.a0; w < b.a1; w += kWindow) {
    const int m = min(kWindow, b.a1 - w);
    __syncthreads();
    for (int i = threadIdx.x; i < m; i += blockDim.x) {
      wkey[i] = (int)a.key[w + i];
      wtok[i] = a.tok[w + i];
    }
    if (threadIdx.x == 0) wkey[m] = w + m < b.a1 ? (int)a.key[w + m] : -1;
    __syncthreads();
    if constexpr (S == 0) {
      for (int i = 0; i < m; ++i) {
        zeros(min(wkey[i], b.b1));
        if (on) {
          const T* p = src + (int64_t)wtok[i] * row_elems;
          for (int s = 0; s < a.streams; s += LOADS) {
            Raw8<T> x[LOADS];
#pragma unroll
            for (int u = 0; u < LOADS; ++u)
              if (s + u < a.streams) x[u] = ld8_stream(p + (int64_t)(s + u) * a.H);
#pragma unroll
            for (int u = 0; u < LOADS; ++u)
              if (s + u < a.streams) add8(acc, unpack(x[u]));
          }
        }
        if (wkey[i + 1] != wkey[i]) finish(wkey[i]);
      }
    } else {
      Raw8<T> cur[GROUP][S], next[GROUP][S];
      auto load = [&](Raw8<T>(&x)[GROUP][S], int i) {
#pragma unroll
        for (int g = 0; g < GROUP; ++g)
          if (i + g < m && on) {
            const T* p = src + (int64_t)wtok[i + g] * row_elems;
#pragma unroll
            for (int s = 0; s < S; ++s) x[g][s] = ld8_stream(p + (int64_t)s * a.H);
          }
      };
      load(cur, 0);
      for (int i = 0; i < m; i += GROUP) {
        load(next, i + GROUP);
#pragma unroll
        for (int g = 0; g < GROUP; ++g) {
          if (i + g < m) {
            const int k = wkey[i + g];
            zeros(min(k, b.b1));
            if (on) {
#pragma unroll
              for (int s = 0; s < S; ++s) add8(acc, unpack(cur[g][s]));
            }
            if (wkey[i + g + 1] != k) finish(k);
          }
        }
#pragma unroll
        for (int g = 0; g < GROUP; ++g)
#pragma unroll
          for (int s = 0; s < S; ++s) cur[g][s] = next[g][s];
      }
    }
  }
  zeros(b.b1);
}

// Rows whose tokens lie in several chunks, by the chunk that holds their end:
// the earlier chunks' sums in chunk order, then its own.  A frequent token has
// hundreds of chunks, so they are taken in kSlices runs, whose sums are added in
// order, and each run's loads eight at a time, whether a chunk has a sum or not
// (empty chunks count as zero).
constexpr int kSlices = 4;
template <typename O>
__global__ void __launch_bounds__(kSumThreads* kSlices) embed_join_kernel(const SumArgs a) {
  __shared__ int first;
  __shared__ float4 part[kSlices - 1][2][kSumThreads];
  pdl_wait();
  const int jobs = a.joins[0];
  const int width = blockDim.x / kSlices, at = threadIdx.x % width, slice = threadIdx.x / width;
  const int64_t c = (int64_t)blockIdx.y * kColumns + at * 8;
  const bool on = c < a.H;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.dtable) | (uintptr_t)(a.ld * sizeof(O))) & 31) == 0;
  for (int job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int chunk = a.joins[1 + job];
    const int row = a.bounds[chunk].b0;
    // the chunk that holds the row's first token: the last one before this that did not begin inside the row
    for (int hi = chunk - 1;; hi -= (int)blockDim.x) {
      __syncthreads();
      if (threadIdx.x == 0) first = -1;
      __syncthreads();
      const int k = hi - (int)threadIdx.x;
      if (k >= 0) {
        const Bounds p = a.bounds[k];
        if (!(p.b0 == row && p.a0 > 0 && (int)a.key[p.a0 - 1] == row)) atomicMax(&first, k);
      }
      __syncthreads();
      if (first >= 0 || hi < (int)blockDim.x) break;
    }
    const int from = max(first, 0), n = chunk - from;
    Vec8 acc = zero8();
    if (on) {
      const int lo = from + (int)((int64_t)n * slice / kSlices), hi = from + (int)((int64_t)n * (slice + 1) / kSlices);
      for (int k = lo; k < hi; k += 8) {
        Raw8<float> x[8];
        bool has[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int q = min(k + u, chunk);  // (the chunk itself has memory too)
          const int2 tokens = *reinterpret_cast<const int2*>(&a.bounds[q].a0);
          has[u] = k + u < hi && tokens.y > tokens.x;  // a chunk with a token: its last is of the row
          x[u] = ld8(a.carry + (int64_t)q * 2 * a.H + c);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (has[u]) add8(acc, unpack(x[u]));
      }
    }
    if (slice) {
      const Raw8<float> mine = pack<float>(acc);
      part[slice - 1][0][at] = *reinterpret_cast<const float4*>(&mine.q[0]);
      part[slice - 1][1][at] = *reinterpret_cast<const float4*>(&mine.q[1]);
    }
    __syncthreads();
    if (slice || !on) continue;
    for (int s = 0; s < kSlices - 1; ++s) {
      Raw8<float> r;
      r.q[0] = *reinterpret_cast<const uint4*>(&part[s][0][at]);
      r.q[1] = *reinterpret_cast<const uint4*>(&part[s][1][at]);
      add8(acc, unpack(r));
    }
    add8(acc, unpack(ld8(a.carry + ((int64_t)chunk * 2 + 1) * a.H + c)));
    end_row<O>(a, row, c, acc, wide);
  }
}

static int bits_of(int64_t v) {
  int b = 0;
  while (v >> b) ++b;
  return b < 1 ? 1 : b;
}

// Workspace and launch plan; a pure function of the sizes.
static EmbedGradWs embed_grad_plan(int64_t T, int64_t V, int H) {
  EmbedGradWs w = {};
  const int bits = bits_of(V);  // keys 0 .. V
  w.passes = (bits + 8) / 9;
  w.digit_bits = (bits + w.passes - 1) / w.passes;
  const int tile = T <= kFewTokens ? kSortThreads : kSortThreads * 4;
  w.tiles = (int)((T + tile - 1) / tile);
  const int cols = (H + kColumns - 1) / kColumns;
  // Chunks: rounds of CTAs, so that an SM that gets through faster takes more (T = 16384,
  // V = 131072, H = 5120: 681 us with 243 chunks, 605 with 487, 568 with 1024, 558 with
  // 1433); at least 16 rows or tokens each; and 7 Mi columns of partial sums (56 MiB) at most,
  // but one chunk an SM (above 48000 columns that is more: 1.2 GB at the widest, 2^20).
  int64_t most = (kSumRounds * 152 * 8 + cols - 1) / cols;
  if (most * H > (int64_t)7 << 20) most = ((int64_t)7 << 20) / H;
  if (most < 152) most = 152;
  int64_t chunks = (T + V + 15) / 16;
  w.chunks = (int)(chunks < 1 ? 1 : chunks > most ? most : chunks);
  w.one = T <= kOneThreads * kOneMost;
  if (w.one) w.tiles = 1;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < 2; ++i) w.key[i] = take((size_t)T * 4), w.tok[i] = take((size_t)T * 4);
  // (the larger tiles of many tokens are fewer at first: the size does not fall there)
  const int room = T > kFewTokens && w.tiles < kFewTokens / kSortThreads ? kFewTokens / kSortThreads : w.tiles;
  w.hist = take((size_t)w.passes * room * kDigits * 4);
  w.places = take(T <= kFewTokens ? 0 : (size_t)(w.tiles + 1) * kDigits * 4);
  w.valid = take((size_t)room * 4);
  w.joins = take((size_t)(w.chunks + 1) * 4);
  w.bounds = take((size_t)w.chunks * sizeof(Bounds));
  w.carry = take((size_t)w.chunks * 2 * H * 4);
  w.total = at;
  return w;
}

template <typename T>
static cudaError_t sum_launch(const SumArgs& a, int grad_dtype, dim3 grid, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const int threads = a.H >= kColumns ? kSumThreads : (a.H / 8 + 31) / 32 * 32;
  auto go = [&](auto o) {
    using O = decltype(o);
    if (a.streams == 1) e = launch_pdl(embed_sum_kernel<T, O, 1>, grid, dim3(threads), 0, s, a);
    else if (a.streams == 2) e = launch_pdl(embed_sum_kernel<T, O, 2>, grid, dim3(threads), 0, s, a);
    else if (a.streams == 4) e = launch_pdl(embed_sum_kernel<T, O, 4>, grid, dim3(threads), 0, s, a);
    else e = launch_pdl(embed_sum_kernel<T, O, 0>, grid, dim3(threads), 0, s, a);
    if (e == cudaSuccess && a.chunks > 1) e = launch_pdl(embed_join_kernel<O>, dim3(a.chunks < kJoinCtas / (int)grid.y ? a.chunks : (kJoinCtas + grid.y - 1) / grid.y, grid.y), dim3(threads * kSlices), 0, s, a);
  };
  if (grad_dtype == MHC_DT_F32) go(float());
  else go(T());
  return e;
}

template <typename Id, int R>
static cudaError_t sort_one_launch(const SortArgs& a, cudaStream_t s) {
  static SmemGrant grant;
  cudaError_t e = allow_smem(grant, (const void*)sort_one_kernel<Id, R>, one_smem(R));
  if (e != cudaSuccess) return e;
  sort_one_kernel<Id, R><<<1, kOneThreads, one_smem(R), s>>>(a);
  return cudaGetLastError();
}
template <typename Id>
static cudaError_t sort_one(const SortArgs& a, cudaStream_t s) {
  return a.T <= kOneThreads ? sort_one_launch<Id, 1>(a, s) : sort_one_launch<Id, kOneMost>(a, s);
}

}  // namespace mhc

extern "C" {

size_t mhc_embed_grad_workspace_bytes(int64_t T, int64_t V, int H) {
  if (T <= 0 || V <= 0 || H <= 0) return 256;
  return mhc::embed_grad_plan(T, V, H).total;
}

int mhc_embed_grad(const void* ids, int id_bytes, const void* dout, mhc_dtype dtype, float scale, int64_t T, int H,
                   int streams, int64_t V, int64_t first_id, const int64_t* padding_id, int accumulate, void* dtable,
                   mhc_dtype grad_dtype, int64_t ld, void* workspace, size_t ws_bytes, void* stream) {
  using namespace mhc;
  if (!dtype_ok(dtype) || !dtype_ok(grad_dtype)) return ops_fail(MHC_ERR_CONFIG, "unknown dtype");
  if (grad_dtype != MHC_DT_F32 && grad_dtype != dtype)
    return ops_fail(MHC_ERR_CONFIG, "the gradient table is fp32 or of the same type as dout");
  if (id_bytes != 4 && id_bytes != 8) return ops_fail(MHC_ERR_CONFIG, "id_bytes must be 4 or 8");
  if (T < 0 || T > 0x40000000 || V < 0 || V > 0x40000000 || H <= 0 || H % 8 != 0 || H > 1 << 20 || streams < 1 ||
      streams > 64)
    return ops_fail(MHC_ERR_SHAPE, "need 0 <= T, V <= 2^30, H a positive multiple of 8 and 1 <= streams <= 64");
  if (ld < H || ld % 8 != 0) return ops_fail(MHC_ERR_SHAPE, "the table's row stride must be a multiple of 8, at least H");
  if (V == 0 || (T == 0 && accumulate)) return MHC_OK;
  if (!dtable || (T && (!ids || !dout))) return ops_fail(MHC_ERR_NULL, "ids, dout and dtable are required");
  if (!ops_aligned(ids, id_bytes) || !ops_aligned(dout, 16) || !ops_aligned(dtable, 16) || !ops_aligned(workspace, 16))
    return ops_fail(MHC_ERR_ALIGN, "dout, dtable and workspace must be 16-byte aligned, ids to their size");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t gb = dtype_bytes(grad_dtype);
  if (T == 0)
    return ops_cuda(cudaMemset2DAsync(dtable, (size_t)ld * gb, 0, (size_t)H * gb, (size_t)V, s), "cudaMemset2DAsync");
  const EmbedGradWs w = embed_grad_plan(T, V, H);
  if (!workspace || ws_bytes < w.total)
    return ops_fail(MHC_ERR_WORKSPACE, "workspace NULL or smaller than mhc_embed_grad_workspace_bytes(T, V, H)");
  const size_t b = dtype_bytes(dtype);
  const Rows in[] = {{ids, 1, T, T, (size_t)id_bytes}, {dout, T, (int64_t)streams * H, (int64_t)streams * H, b}};
  const Rows out[] = {{dtable, V, H, ld, gb}, {workspace, 1, (int64_t)w.total, 1, 1}};
  for (const Rows& o : out)
    for (const Rows& i : in)
      if (rows_overlap(o, i)) return ops_fail(MHC_ERR_ALIAS, "an output overlaps an input");
  if (rows_overlap(out[0], out[1])) return ops_fail(MHC_ERR_ALIAS, "two outputs overlap");

  char* ws = static_cast<char*>(workspace);
  SortArgs a = {};
  a.ids = ids;
  a.first = first_id;
  a.V = V;
  a.has_pad = padding_id != nullptr;
  a.pad = padding_id ? *padding_id : 0;
  a.T = (int)T;
  a.bits = w.digit_bits;
  a.tiles = w.tiles;
  a.passes = w.passes;
  a.valid = reinterpret_cast<int*>(ws + w.valid);
  a.joins = reinterpret_cast<int*>(ws + w.joins);
  int* hist = reinterpret_cast<int*>(ws + w.hist);
  const size_t per_pass = (size_t)w.tiles * kDigits;
  cudaError_t e = cudaSuccess;
  int from = 0;
  if (w.one) {
    a.key_out = reinterpret_cast<uint32_t*>(ws + w.key[0]);
    a.tok_out = reinterpret_cast<int*>(ws + w.tok[0]);
    e = id_bytes == 4 ? sort_one<int32_t>(a, s) : sort_one<int64_t>(a, s);
  }
  for (int p = 0; !w.one && p < w.passes && e == cudaSuccess; ++p, from ^= 1) {
    const bool last = p + 1 == w.passes;
    a.shift = p * w.digit_bits;
    a.key_in = reinterpret_cast<uint32_t*>(ws + w.key[from]);
    a.key_out = reinterpret_cast<uint32_t*>(ws + w.key[from ^ 1]);
    a.tok_in = reinterpret_cast<int*>(ws + w.tok[from]);
    a.tok_out = reinterpret_cast<int*>(ws + w.tok[from ^ 1]);
    a.hist_in = hist + p * per_pass;
    a.hist_out = last ? nullptr : hist + (p + 1) * per_pass;
    const bool few = T <= kFewTokens;
    if (p == 0) {
      if (id_bytes == 4)
        few ? sort_count_kernel<int32_t, 1><<<w.tiles, kSortThreads, 0, s>>>(a)
            : sort_count_kernel<int32_t, 4><<<w.tiles, kSortThreads, 0, s>>>(a);
      else
        few ? sort_count_kernel<int64_t, 1><<<w.tiles, kSortThreads, 0, s>>>(a)
            : sort_count_kernel<int64_t, 4><<<w.tiles, kSortThreads, 0, s>>>(a);
      e = cudaGetLastError();
      if (e != cudaSuccess) break;
    }
    if (few) {
      e = launch_pdl(sort_pass_kernel<1>, dim3(w.tiles), dim3(kSortThreads), 0, s, a, p == 0, last);
    } else {
      a.places = reinterpret_cast<int*>(ws + w.places);
      e = launch_pdl(sort_places_kernel, dim3(kDigits / 32), dim3(1024), 0, s, a.hist_in, w.tiles, a.places,
                     a.places + (size_t)w.tiles * kDigits);
      if (e == cudaSuccess) e = launch_pdl(sort_pass_kernel<4>, dim3(w.tiles), dim3(kSortThreads), 0, s, a, p == 0, last);
    }
  }
  if (e != cudaSuccess) return ops_cuda(e, "embed_grad sort launch");
  SumArgs m = {};
  m.dout = dout;
  m.dtable = dtable;
  m.ld = ld;
  m.V = V;
  m.H = H;
  m.streams = streams;
  m.tiles = w.tiles;
  m.chunks = w.chunks;
  m.wt = (int)(streams * b);
  m.wr = (int)gb;
  m.accumulate = accumulate != 0;
  m.scale = scale;
  m.key = reinterpret_cast<const uint32_t*>(ws + w.key[from]);
  m.tok = reinterpret_cast<const int*>(ws + w.tok[from]);
  m.valid = a.valid;
  m.joins = a.joins;
  m.bounds = reinterpret_cast<Bounds*>(ws + w.bounds);
  m.carry = reinterpret_cast<float*>(ws + w.carry);
  const dim3 grid(w.chunks, (H + kColumns - 1) / kColumns);
  MHC_BY_DTYPE(dtype, E, { e = sum_launch<E>(m, grad_dtype, grid, s); });
  return ops_cuda(e, "embed_grad sum launch");
}

}  // extern "C"
