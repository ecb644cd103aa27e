// mhc_route and its gradient: scores of a token's experts, the choice of the
// best k (in the best groups), their weights and the experts' loads.

#include "mhc_ops.cuh"

namespace mhc {

constexpr int kRouteWarps = 4;
constexpr int kMaxExperts = 1024;
// CTAs per SM of the choice: eight are resident (64 registers a thread), and twice as
// many let an SM that gets through faster take more of them (T = 131072, E = 256: ten
// resident and ten in all took 87 us where these took 81).  Sixteen and 32 experts a lane
// are given the registers of seven and four (sigmoid, bias, k = 8; T = 65536, E = 512: 69 us
// against 84 with as many as they ask for, for 16 bytes of spills; T = 32768, E = 1024: 94 against 124).
constexpr int kRouteResident = 8, kRouteCtas = 16;

template <typename T>
__device__ __forceinline__ float logit_of(const T* p) {
  float l;
  if constexpr (sizeof(T) == 4) l = *p;
  else l = pair_of((uint32_t)*reinterpret_cast<const uint16_t*>(p), T()).x;
  return l == l ? l : -INFINITY;  // a NaN logit is never chosen, as -inf
}

// A lane's EPL logits in 16-byte loads (fewer bytes in one load).
template <typename T, int EPL>
__device__ __forceinline__ void load_logits(const T* p, float* l) {
  constexpr int BYTES = EPL * (int)sizeof(T);
  if constexpr (BYTES >= 16 && sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < EPL / 4; ++i) {
      const float4 q = __ldcs(reinterpret_cast<const float4*>(p) + i);
      l[4 * i] = q.x, l[4 * i + 1] = q.y, l[4 * i + 2] = q.z, l[4 * i + 3] = q.w;
    }
  } else if constexpr (BYTES >= 16) {
#pragma unroll
    for (int i = 0; i < EPL / 8; ++i) {
      const Vec8 q = unpack(ld8_stream(p + 8 * i));
#pragma unroll
      for (int e = 0; e < 4; ++e) l[8 * i + 2 * e] = q.p[e].x, l[8 * i + 2 * e + 1] = q.p[e].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = logit_of(p + i);
  }
}

// exp(l - max) with equal infinities at distance zero.
__device__ __forceinline__ float soft_exp(float l, float m) { return l == -INFINITY ? 0.f : expf(l == m ? 0.f : l - m); }
__device__ __forceinline__ float logistic(float l) { return __frcp_rn(1.0f + expf(-l)); }  // rounded as 1 / (1 + e)
// 1 - logistic(l) = exp(-l) logistic(l): the difference itself has lost half its bits at l = 9 and all at 17
__device__ __forceinline__ float logistic_rest(float l, float v) { return l > 0.f ? expf(-l) * v : 1.0f - v; }

// A key whose unsigned order is the values' order; 0 for what cannot be chosen.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // a -0 (from a bias) counts as +0
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return k ? __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu)) : -INFINITY;
}

struct RouteArgs {
  const void* logits;
  uint32_t ld_bytes, T;  // a row's bytes and the tokens: both below 2^31
  const float* bias;
  int E, groups, top_groups, k;
  int log_slots;  // log2 of the slots kept for a token: k, rounded up to a power of two
  bool sigmoid, renorm;
  bool vector;       // rows are 16-byte aligned and no lane has part of its experts
  bool whole_lanes;  // a group is a power of two of whole lanes
  bool estimate;     // choose from estimated scores first
  float scale;
  int* indices;
  float* weights;
  int* counts;
  unsigned* ticket;  // workspace: CTAs done, then the E loads (all zero between calls)
  unsigned* loads;
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}

// Reductions over a segment of LANES adjacent lanes (one token).
template <int LANES>
__device__ __forceinline__ float seg_max(float x) {
#pragma unroll
  for (int d = LANES / 2; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
template <int LANES>
__device__ __forceinline__ float seg_sum(float x) {
#pragma unroll
  for (int d = LANES / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
template <int LANES>
__device__ __forceinline__ uint32_t seg_max(uint32_t x) {
  if constexpr (LANES == 32) {
    return __reduce_max_sync(0xffffffffu, x);
  } else {
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
  }
}
template <int LANES>
__device__ __forceinline__ int seg_add(int x) {
  if constexpr (LANES == 32) {
    return __reduce_add_sync(0xffffffffu, x);
  } else {
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
  }
}
// The lanes of this thread's segment for which `p` holds, from bit 0.
template <int LANES>
__device__ __forceinline__ unsigned seg_ballot(bool p) {
  const unsigned all = __ballot_sync(0xffffffffu, p);
  if constexpr (LANES == 32) return all;
  else return (all >> (threadIdx.x & 31 & ~(LANES - 1))) & ((1u << LANES) - 1);
}

// --------------------------------------------------- the choice, estimated --
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int LANES>
__device__ __forceinline__ float seg_fmax(float x) {
  if constexpr (LANES == 32) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
  } else {
    return seg_max<LANES>(x);
  }
}

__device__ __forceinline__ void order(float& a, float& b) {  // a >= b
  const float hi = fmaxf(a, b);
  b = fminf(a, b);
  a = hi;
}
__device__ __forceinline__ void sort4(float* v) {
  order(v[0], v[1]), order(v[2], v[3]), order(v[0], v[2]), order(v[1], v[3]), order(v[1], v[2]);
}
// The best of two descending lists of four, descending, into `a`: the larger of
// opposite ends is a bitonic list (Batcher's merge).
__device__ __forceinline__ void merge4(float* a, const float* b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fmaxf(a[i], b[3 - i]);
  order(a[0], a[2]), order(a[1], a[3]), order(a[0], a[1]), order(a[2], a[3]);
}
// Batcher's odd-even merge sort of eight, descending.
__device__ __forceinline__ void sort8(float* v) {
  sort4(v), sort4(v + 4);
  order(v[0], v[4]), order(v[1], v[5]), order(v[2], v[6]), order(v[3], v[7]);
  order(v[2], v[4]), order(v[3], v[5]);
  order(v[1], v[2]), order(v[3], v[4]), order(v[5], v[6]);
}

// LANES lanes work on one token (32 / LANES tokens per warp); lane l of them has
// experts l*EPL .. l*EPL+EPL-1.
//
// The choice is made twice, the second time for few tokens.  First from
// estimated scores (the hardware's exp2 and reciprocal, 4 instructions for a
// sigmoid instead of about 20), with the expert's place in its lane written over the
// lowest log2(EPL) bits: each lane sorts its best few, and a round is one maximum
// over the lanes; the lane that has it writes the slot and moves its list up.
// Slots whose estimates differ by more than the errors of two (`near0`, `near1`) from
// their neighbours, the last of them from the best expert left, are in the order of
// the exact scores.  Where they do not (one token in five hundred of N(0, 1.5) logits
// with a bias), where two groups' sums are too near, or where a lane's list runs out,
// the token is chosen again from the exact scores.
//
// The exact choice has whole order keys; its rounds work on each lane's two best
// with the place in the low bits, and a lane whose two are spent looks for the
// next two.  Keys that differ in those bits only could come in the wrong order;
// they are next to each other in it, so the slots are compared with their
// neighbours by the exact choice, and a token where they disagree (or where the
// k-th and the next agree above the low bits) is done with whole keys, one scan of
// all of them per round.
//
// A warp takes as many tokens in turn as it has lanes for their k slots; checks,
// weights and stores are then one slot per lane.
//
// Bound by instructions: T = 131072, E = 256, 8 of 4 of 8 groups 68 us, 418 a token at
// 72 % of the issue slots; the busiest pipe (ALU: comparisons, maxima, moves) is 57 %
// busy (its floor in HBM is 21 us).
template <typename T, int EPL, int LANES, bool K8>
__global__ void __launch_bounds__(kRouteWarps * 32, EPL <= 8 ? kRouteResident : EPL == 16 ? kRouteResident - 1 : kRouteResident / 2) route_kernel(const RouteArgs a) {
  constexpr uint32_t LOW = EPL - 1;
  const int k = K8 ? 8 : a.k, log_slots = K8 ? 3 : a.log_slots;
  constexpr int TOKENS = 32 / LANES;
  constexpr bool SMEM_GROUPS = LANES == 32;  // groups that do not fall on whole lanes
  __shared__ uint32_t keys[SMEM_GROUPS ? kRouteWarps : 1][SMEM_GROUPS ? EPL * 32 : 1];
  __shared__ int load[EPL * LANES];
  // A warp's batch: 32 slots of 32 >> log_slots tokens.  slot: the expert and its
  // estimate; rest: a token's best estimate left over and how many lanes' experts its
  // slots took; soft: its row's maximum and sum.
  __shared__ int2 slot_[kRouteWarps][32], rest_[kRouteWarps][32];
  __shared__ float2 soft_[kRouteWarps][32];
  const int lane = threadIdx.x & (LANES - 1), warp = threadIdx.x >> 5;
  const int sub = (threadIdx.x & 31) / LANES;
  int2* const slot = slot_[warp];
  int2* const rest = rest_[warp];
  float2* const soft = soft_[warp];
  const int id = threadIdx.x & 31;
  const char* const rows = static_cast<const char*>(a.logits);
  for (int e = threadIdx.x; e < EPL * LANES; e += blockDim.x) load[e] = 0;
  __syncthreads();
  const int per = a.E / a.groups;
  const int group_lanes = per / EPL;  // where groups fall on whole lanes
  const int slots = 1 << log_slots, batch = 32 >> log_slots;
  float bias[EPL];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    bias[i] = a.bias && e < a.E ? a.bias[e] : 0.f;
    finite &= fabsf(bias[i]) < 3e38f;
  }
  const bool estimate = a.estimate && __all_sync(0xffffffffu, finite);
  const bool need_sum = !a.sigmoid && (a.bias || !a.renorm);
  // Estimates nearer than near0 + near1 * estimate may be in the wrong order: twice the
  // error of one.  With a bias (scores at most 1): the score's 5e-7 (sigmoid; softmax: 7e-7 of
  // a score, of two that add up to 1 at most), the sum's rounding and the place.  Without: relative, from exp2's
  // argument (at most 88 away from 0 or from the maximum, which both kinds of softmax scores
  // take off with the same rounding) and the place; 1e-36: scores that exp2 flushes to zero.
  const float place = (LOW + 2) * 2.4e-7f;
  const float near0 = a.bias ? 2e-6f : 1e-36f;
  const float near1 = place + (a.bias ? 0.f : a.sigmoid ? 1.5e-5f : 2.5e-5f);
  float most = 0.f;  // |bias|
#pragma unroll
  for (int i = 0; i < EPL; ++i) most = fmaxf(most, fabsf(bias[i]));
  const float near_group = 2.f * (near0 + near1 * (1.f + warp_max(most)));

  // The lane's logits of the next two passes come through shared memory of its own.
  constexpr int PIECES = EPL * (int)sizeof(T) / 16;  // 16-byte pieces of a lane's logits
  constexpr bool RING = PIECES >= 1 && EPL <= 16;
  __shared__ uint4 ring_[RING ? kRouteWarps : 1][RING ? 2 : 1][RING ? PIECES * 32 : 1];
  const bool ring = RING && a.vector && estimate;
  const uint32_t ring_at = smem_of(&ring_[RING ? warp : 0][0][0]) + (threadIdx.x & 31) * 16;
  const uint32_t stride = gridDim.x * kRouteWarps * batch;
  auto row_of = [&](uint32_t first) {  // a segment without a token repeats the last token's work
    return rows + (uint64_t)(TOKENS == 1 ? first : min(first + sub, a.T - 1)) * a.ld_bytes;
  };
  auto fetch = [&](uint32_t first, int stage) {  // the pass whose first token is `first`
    if constexpr (RING) {
      if (ring && first < a.T) {
        const char* p = row_of(first) + lane * EPL * sizeof(T);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) cp_async16(ring_at + (stage * PIECES + i) * 512, p + i * 16);
      }
      cp_async_commit();
    }
  };
  const uint32_t start = (blockIdx.x * kRouteWarps + warp) * batch;
  // from a token past this batch to the same place of the warp's next batch (batches of
  // one pass: of the one after)
  const uint32_t later = batch > TOKENS ? stride - batch : 2 * (stride - batch);
  fetch(start, 0);
  fetch(TOKENS < batch ? start + TOKENS : start + stride, 1);
  int stage = 0;
  for (uint32_t base = start; base < a.T; base += stride) {
    auto logits = [&](const T* row, float* l) {
      if (a.vector) {
        load_logits<T, EPL>(row + lane * EPL, l);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = lane * EPL + i < a.E ? logit_of(row + lane * EPL + i) : -INFINITY;
      }
    };
    auto softmax = [&](const float* l) {  // the row's maximum, and its sum where a score needs it
      float2 ms = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < EPL; ++i) ms.x = fmaxf(ms.x, l[i]);  // fmaxf passes NaN over
      ms.x = seg_fmax<LANES>(ms.x);
      if (need_sum) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) ms.y += l[i] > -INFINITY ? soft_exp(l[i], ms.x) : 0.f;
        ms.y = seg_sum<LANES>(ms.y);
      }
      return ms;
    };
    const int passes = ((int)min(a.T - base, (uint32_t)batch) + TOKENS - 1) / TOKENS;
    unsigned again = 0;  // passes to choose exactly
    __syncwarp();
    slot[id] = make_int2(-1, __float_as_int(-INFINITY));
    __syncwarp();

    for (int it = 0; estimate && it < passes; ++it) {
      constexpr int KEPT = EPL <= 4 ? EPL : LANES == 8 ? 8 : 4;  // how many of its best a lane keeps sorted
      const int first = (it * TOKENS + sub) << log_slots;
      float v[EPL];
      bool redo = false;
      if (ring) {
        if constexpr (RING) {
          cp_async_wait<1>();
#pragma unroll
          for (int i = 0; i < PIECES; ++i) {
            const uint4 q = lds16(ring_at + (stage * PIECES + i) * 512);
            if constexpr (sizeof(T) == 4) {
              v[4 * i] = __uint_as_float(q.x), v[4 * i + 1] = __uint_as_float(q.y);
              v[4 * i + 2] = __uint_as_float(q.z), v[4 * i + 3] = __uint_as_float(q.w);
            } else {
              Raw8<T> r;
              r.q[0] = q;
              const Vec8 x = unpack(r);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[8 * i + 2 * e] = x.p[e].x, v[8 * i + 2 * e + 1] = x.p[e].y;
            }
          }
          const int on = (it + 2) * TOKENS;  // two passes on: in this batch or in a later one
          fetch(base + on + (on < batch ? 0u : later), stage);
          stage ^= 1;
        }
      } else {
        logits(reinterpret_cast<const T*>(row_of(base + it * TOKENS)), v);
      }
      // logits that are not finite are rare: their sum is not either; masked in a branch
      unsigned dead = 0;
      float odd;
      if constexpr (EPL == 1) {
        odd = v[0];
      } else {
        float2 sum = make_float2(v[0], v[1]);
#pragma unroll
        for (int i = 2; i < EPL; i += 2) sum = __fadd2_rn(sum, make_float2(v[i], v[i + 1]));
        odd = sum.x + sum.y;
      }
      const bool masks = __any_sync(0xffffffffu, !(fabsf(odd) < 3e38f));
      if (masks) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) dead |= (v[i] > -INFINITY ? 0u : 1u) << i;
      }
      if (a.sigmoid) {
        if constexpr (EPL == 1) {
          v[0] = rcp_approx(1.0f + ex2_approx(v[0] * -1.44269504f)) + bias[0];
        } else {
#pragma unroll
          for (int i = 0; i < EPL; i += 2) {  // two experts per instruction where the pipe has it
            float2 s = __fmul2_rn(make_float2(v[i], v[i + 1]), splat(-1.44269504f));
            s = __fadd2_rn(make_float2(ex2_approx(s.x), ex2_approx(s.y)), splat(1.f));
            s = __fadd2_rn(make_float2(rcp_approx(s.x), rcp_approx(s.y)), make_float2(bias[i], bias[i + 1]));
            v[i] = __uint_as_float((__float_as_uint(s.x) & ~LOW) | i);
            v[i + 1] = __uint_as_float((__float_as_uint(s.y) & ~LOW) | (i + 1));
          }
        }
      } else {
        const float2 ms = softmax(v);
        if (lane == 0) soft[it * TOKENS + sub] = ms;
        redo = !(fabsf(ms.x) < 3e38f);
        // the maximum is taken off first, as the exact scores do: a rounding of max * log2 e would scale
        // every score of the row, but not the bias
        const float share = a.bias ? rcp_approx(ms.y) : 1.f;
        if constexpr (EPL == 1) {
          v[0] = fmaf(ex2_approx((v[0] - ms.x) * 1.44269504f), share, bias[0]);
        } else {
#pragma unroll
          for (int i = 0; i < EPL; i += 2) {
            float2 s = __fmul2_rn(__fadd2_rn(make_float2(v[i], v[i + 1]), splat(-ms.x)), splat(1.44269504f));
            s = __ffma2_rn(make_float2(ex2_approx(s.x), ex2_approx(s.y)), splat(share), make_float2(bias[i], bias[i + 1]));
            v[i] = __uint_as_float((__float_as_uint(s.x) & ~LOW) | i);
            v[i + 1] = __uint_as_float((__float_as_uint(s.y) & ~LOW) | (i + 1));
          }
        }
      }
      if (masks) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = (dead >> i) & 1 ? -INFINITY : v[i];
      }
      float b[KEPT];
      if constexpr (KEPT == 8) {
        sort8(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = v[i];
      } else if constexpr (EPL >= 4) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
          sort4(v + i);
          if (i) merge4(v, v + i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = v[i];
      } else {
        if constexpr (EPL == 2) order(v[0], v[1]);
#pragma unroll
        for (int i = 0; i < EPL; ++i) b[i] = v[i];
      }
      if (a.groups > 1) {  // on whole lanes
        float b1 = b[0], b2 = EPL > 1 ? b[KEPT > 1 ? 1 : 0] : -INFINITY;
        for (int d = 1; d < group_lanes; d <<= 1) {
          const float c1 = __shfl_xor_sync(0xffffffffu, b1, d), c2 = __shfl_xor_sync(0xffffffffu, b2, d);
          b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
          b1 = fmaxf(b1, c1);
        }
        const bool two = b2 > -INFINITY;
        const float mine = two ? b1 + b2 : b1;
        float near = near_group;  // (with a bias; else relative to the largest of the sums compared)
        if (!a.bias) near = seg_fmax<LANES>(b1 > -INFINITY ? 2.f * near0 + near1 * (b1 + (two ? b2 : 0.f)) : 0.f);
        // the best groups one by one; then the best one left has to be clearly behind
        float open = mine, last = -INFINITY;
        for (int n = 0; n < a.top_groups; ++n) {
          last = seg_fmax<LANES>(open);
          open = open == last ? -INFINITY : open;
        }
        const float behind = seg_fmax<LANES>(open);
        const bool keep = open == -INFINITY;
        redo |= keep && mine == last && mine - behind <= near;
        const bool kept = keep && mine > -INFINITY;  // equal groups leave the list together: there may be too many
        if constexpr (LANES == 32) redo |= __popc(__ballot_sync(0xffffffffu, kept)) > a.top_groups * group_lanes;
        else redo |= seg_add<LANES>(kept) > a.top_groups * group_lanes;
        if (!keep) {
#pragma unroll
          for (int i = 0; i < KEPT; ++i) b[i] = -INFINITY;
        }
      }
      const bool full = KEPT < EPL && b[KEPT - 1] > -INFINITY;
      int wins = 0;
#pragma unroll(K8 ? 8 : 1)
      for (int j = 0; j < k; ++j) {
        const float top = seg_fmax<LANES>(b[0]);
        const bool win = b[0] == top;  // one lane, or a tie (or no expert left): then wins and slots differ
        if (win) slot[first + j] = make_int2(lane * EPL | (int)(__float_as_uint(top) & LOW), __float_as_int(top));
        wins += win;
#pragma unroll
        for (int i = 0; i + 1 < KEPT; ++i) b[i] = win ? b[i + 1] : b[i];
        b[KEPT - 1] = win ? -INFINITY : b[KEPT - 1];
      }
      const float best = seg_fmax<LANES>(b[0]);
      wins = seg_add<LANES>(wins);
      if (lane == 0) rest[it * TOKENS + sub] = make_int2(__float_as_int(best), wins);
      redo |= full && b[0] == -INFINITY;  // a list has run out
      again |= (unsigned)redo << it;
    }
    __syncwarp();

    // One slot per lane from here: slot `at` of token base + tok.
    const int tok = id >> log_slots, at = id & (slots - 1);
    const bool mine = at < k && base + tok < a.T;
    if (estimate) {
      const int2 r = rest[tok];
      const float v = __int_as_float(slot[id].y);
      const float after = at + 1 < k ? __int_as_float(slot[id + 1 & 31].y) : __int_as_float(r.x);
      const unsigned filled = __ballot_sync(0xffffffffu, mine && v > -INFINITY) >> (id & ~(slots - 1));
      const bool redo = mine && (v - after <= near0 + near1 * fabsf(v) ||  // no slot: NaN, false
                                 __popc(slots == 32 ? filled : filled & ((1u << slots) - 1)) != r.y);
      again |= (unsigned)redo << tok / TOKENS;
      again = __reduce_or_sync(0xffffffffu, again);
    } else {
      again = (2u << (passes - 1)) - 1;
    }

    for (; again; again &= again - 1) {
      const int it = __ffs(again) - 1;
      const T* row = reinterpret_cast<const T*>(row_of(base + it * TOKENS));
      const int first = (it * TOKENS + sub) << log_slots;
      uint32_t key[EPL];
      float m = 0.f, total = 1.f;
      {
        float l[EPL];
        logits(row, l);
        if (a.sigmoid) {
#pragma unroll
          for (int i = 0; i < EPL; ++i) key[i] = l[i] > -INFINITY ? order_key(logistic(l[i]) + bias[i]) : 0u;
        } else {
          const float2 ms = softmax(l);
          m = ms.x, total = ms.y;
          if (lane == 0) soft[it * TOKENS + sub] = ms;
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            const float e = l[i] > -INFINITY ? soft_exp(l[i], m) : 0.f;
            key[i] = l[i] > -INFINITY ? order_key(a.bias ? e / total + bias[i] : e) : 0u;
          }
        }
      }
      if (a.groups > 1) {
        if (!SMEM_GROUPS || a.whole_lanes) {
          uint32_t b1 = 0, b2 = 0;
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            b2 = max(b2, min(b1, key[i]));
            b1 = max(b1, key[i]);
          }
          for (int d = 1; d < group_lanes; d <<= 1) {
            const uint32_t c1 = __shfl_xor_sync(0xffffffffu, b1, d), c2 = __shfl_xor_sync(0xffffffffu, b2, d);
            b2 = max(max(b2, c2), min(b1, c1));
            b1 = max(b1, c1);
          }
          const uint32_t sum = b1 == 0 ? 0u : order_key(order_value(b1) + (b2 ? order_value(b2) : 0.f));
          int rank = 0;
          for (int d = group_lanes; d < LANES; d += group_lanes) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, sum, d);
            rank += other > sum || (other == sum && (lane ^ d) < lane);
          }
          if (rank >= a.top_groups) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = 0;
          }
        } else {
#pragma unroll
          for (int i = 0; i < EPL; ++i) keys[warp][lane * EPL + i] = key[i];
          __syncwarp();
          uint32_t b1 = 0, b2 = 0;
          if (lane < a.groups)
            for (int j = 0; j < per; ++j) {
              const uint32_t q = keys[warp][lane * per + j];
              b2 = max(b2, min(b1, q));
              b1 = max(b1, q);
            }
          __syncwarp();
          const uint32_t sum = b1 == 0 ? 0u : order_key(order_value(b1) + (b2 ? order_value(b2) : 0.f));
          int rank = 0;
          for (int g = 0; g < a.groups; ++g) {
            const uint32_t other = __shfl_sync(0xffffffffu, sum, g);
            rank += other > sum || (other == sum && g < lane);
          }
          const unsigned keep = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.top_groups);
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            if (!((keep >> ((lane * EPL + i) / per & 31)) & 1)) key[i] = 0;
        }
      }

      // the lane's two best keys below `under`
      uint32_t b1, b2;
      auto refill = [&](uint32_t under) {
        b1 = b2 = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          uint32_t p = key[i] ? (key[i] & ~LOW) | (LOW - i) : 0u;
          p = p < under ? p : 0u;
          b2 = max(b2, min(b1, p));
          b1 = max(b1, p);
        }
      };
      refill(0xffffffffu);
      uint32_t held = 0;  // lane j: the key of slot j
      int expert = -1;    // and its expert
      for (int j = 0; j < k; ++j) {
        const uint32_t top = seg_max<LANES>(b1);
        const unsigned have = seg_ballot<LANES>((b1 | LOW) == (top | LOW));
        const int who = __ffs(have) - 1;
        const uint32_t won = __shfl_sync(0xffffffffu, b1, who, LANES);
        if (lane == j && won) {
          held = won;
          expert = who * EPL + (int)(LOW - (won & LOW));
        }
        bool spent = false;
        if (lane == who && won) {
          b1 = b2;
          b2 = 0;
          spent = EPL > 2 && b1 == 0;
        }
        if (EPL > 2 && __any_sync(0xffffffffu, spent)) {
          const uint32_t o1 = b1, o2 = b2;
          refill(won);
          if (!spent) b1 = o1, b2 = o2;
        }
      }
      if constexpr (EPL > 1) {
        const uint32_t next = seg_max<LANES>(b1);  // the best key left
        float pick = -INFINITY;                    // the exact choice of the slot's expert
        if (expert >= 0) {
          const float l = logit_of(row + expert);
          pick = a.sigmoid ? logistic(l) : soft_exp(l, m);
          if (a.bias) pick = (a.sigmoid ? pick : pick / total) + a.bias[expert];
        }
        const uint32_t after = __shfl_down_sync(0xffffffffu, held, 1, LANES);
        const float later = __shfl_down_sync(0xffffffffu, pick, 1, LANES);
        bool unsure = false;
        if (held) {
          if (lane + 1 == k) unsure = (held | LOW) == (next | LOW);
          else if (lane + 1 < k) unsure = after && (held | LOW) == (after | LOW) && pick != later;
        }
        if (__any_sync(0xffffffffu, unsure)) {
          unsigned alive = 0xffffffffu;
          expert = -1;
          for (int j = 0; j < k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) best = max(best, (alive >> i) & 1 ? key[i] : 0u);
            const uint32_t top = seg_max<LANES>(best);
            const int who = __ffs(seg_ballot<LANES>(best == top)) - 1;
            int place = 0;
            if (lane == who) {
#pragma unroll
              for (int i = EPL - 1; i >= 0; --i)
                if (((alive >> i) & 1) && key[i] == top) place = i;
              alive &= ~(1u << place);
            }
            place = __shfl_sync(0xffffffffu, place, who, LANES);
            if (lane == j && top) expert = who * EPL + place;
          }
        }
      }
      if (lane < k) slot[first + lane].x = expert;
    }
    __syncwarp();

    const int e = mine ? slot[id].x : -1;
    float w = 0.f;
    if (e >= 0) {
      const float l = logit_of(reinterpret_cast<const T*>(rows + (uint64_t)(base + tok) * a.ld_bytes) + e);
      if (a.sigmoid) {
        w = logistic(l);
      } else {
        const float2 ms = soft[tok];
        w = soft_exp(l, ms.x);
        if (!a.renorm) w = w / ms.y;
      }
      atomicAdd(&load[e], 1);
    }
    if (a.renorm) {
      float sum = w;
      for (int d = slots >> 1; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      // A bias or the groups can leave the row's maximum far above the chosen logits, whose
      // exponentials then lose bits or are 0: from the chosen ones' own maximum (rare: every
      // token that way took 45.7 us where this takes 43.2, T = 131072, E = 64, k = 6).
      const bool low = !a.sigmoid && sum < 1e-4f;
      if (__any_sync(0xffffffffu, low)) {
        const float l = e >= 0 ? logit_of(reinterpret_cast<const T*>(rows + (uint64_t)(base + tok) * a.ld_bytes) + e) : -INFINITY;
        float m = l;
        for (int d = slots >> 1; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float v = soft_exp(l, m);
        float all = v;
        for (int d = slots >> 1; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
        if (low) w = v, sum = all;
      }
      w = sum > 0.f ? a.scale * w / sum : 0.f;
    } else {
      w *= a.scale;
    }
    if (mine) {
      const uint64_t o = (uint64_t)(base + tok) * k + at;
      a.indices[o] = e;
      a.weights[o] = w;
    }
  }
  if (!a.counts) return;
  // Loads of all CTAs: whole-number atomics, so their order does not matter.
  // The last CTA to come copies them out and leaves the workspace zero.
  __shared__ bool last;
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x)
    if (load[e]) atomicAdd(a.loads + e, (unsigned)load[e]);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atom_add_acq_rel_gpu(a.ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[e] = (int)atomicExch(a.loads + e, 0u);
  if (threadIdx.x == 0) *a.ticket = 0;
}

struct RouteGradArgs {
  const float* dweights;
  const void* logits;
  int64_t ld, T;
  const int* indices;
  int E, k;
  bool sigmoid, renorm;
  float scale;
  void* dlogits;
  int64_t ld_d;
  int log_slots, rows, pad;  // slots per token (log2), tokens per warp, floats of a row in shared memory
  bool vector;               // rows of dlogits are 16-byte pieces
};

template <typename T>
__device__ __forceinline__ void store_one(T* p, float x) {
  if constexpr (sizeof(T) == 4) *p = x;
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)word_of(x, 0.f, T());
}

// A row of gradients from the sums of its slots, through shared memory: `rows` rows
// of `pad` floats per warp, zero but where a slot has added to them.
template <typename T>
__device__ __forceinline__ void store_row(T* d, const float* src, int E, bool vector) {
  const int id = threadIdx.x & 31;
  if (vector) {
    constexpr int N = 16 / (int)sizeof(T);
    for (int i = id * N; i < E; i += 32 * N) {
      if constexpr (sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4*>(d + i), *reinterpret_cast<const float4*>(src + i));
      } else {
        const float4 x = *reinterpret_cast<const float4*>(src + i), y = *reinterpret_cast<const float4*>(src + i + 4);
        __stcs(reinterpret_cast<uint4*>(d + i),
               make_uint4(word_of(x.x, x.y, T()), word_of(x.z, x.w, T()), word_of(y.x, y.y, T()), word_of(y.z, y.w, T())));
      }
    }
  } else {
    for (int i = id; i < E; i += 32) store_one(d + i, src[i]);
  }
}

// A token of mhc_route names an expert once, but a caller's may not: the lanes whose
// slots name the same place (-1: none) ...
__device__ __forceinline__ unsigned same_place(int place) { return __match_any_sync(0xffffffffu, place); }
// ... and their values summed into the lowest of them, in slot order, which alone then stores
// (returns true there): one addend per place and no float atomics, so that the sum's order is fixed.
__device__ __forceinline__ bool join_slots(unsigned same, bool named, float& x) {
  const int id = threadIdx.x & 31;
  const bool first = named && __ffs(same) - 1 == id;
  if (__any_sync(0xffffffffu, named && !first)) {
    float sum = x;
#pragma unroll 1
    for (int j = 1; j < 32; ++j) {
      const float y = __shfl_sync(0xffffffffu, x, j);
      if (first && j > id && (same >> j) & 1) sum += y;
    }
    x = sum;
  }
  return first;
}

// Gradients that only the chosen experts have (sigmoid scores, or softmax
// renormalised over the k): with q = v / sum v and v the score,
//   renorm:  dl = scale q (dw - sum q dw) (1 - v for a sigmoid),   else (sigmoid) dl = scale dw v (1 - v).
// One slot per lane, as many tokens per warp as have room; their rows are put
// together in shared memory, written in 16-byte stores, and the slots' places set
// back to zero.  Bound by the rows written (T = 131072, E = 256, fp32: 134 MB) and
// the chosen logits read (a 64-byte burst of DRAM each: 67 MB): 37 us of the 31 that
// these take at the copy's rate.  Loading the next batch's slots ahead did not change it.
template <typename T>
__global__ void __launch_bounds__(kRouteWarps * 32) route_grad_kernel(const RouteGradArgs a) {
  extern __shared__ float4 dyn[];
  const int id = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* const rows = reinterpret_cast<float*>(dyn) + warp * a.rows * a.pad;
  for (int i = id; i < a.rows * a.pad; i += 32) rows[i] = 0.f;
  const int slots = 1 << a.log_slots, tok = id >> a.log_slots, at = id & (slots - 1);
  const int64_t step = (int64_t)gridDim.x * kRouteWarps * a.rows;
  __syncwarp();
  for (int64_t base = ((int64_t)blockIdx.x * kRouteWarps + warp) * a.rows; base < a.T; base += step) {
    const int64_t t = base + tok;
    int e = -1;
    float dw = 0.f, v = 0.f, l = -INFINITY;
    if (tok < a.rows && t < a.T && at < a.k) {
      e = a.indices[t * a.k + at];
      if (e >= a.E) e = -1;
      if (e >= 0) {
        dw = a.dweights[t * a.k + at];
        l = logit_of(static_cast<const T*>(a.logits) + t * a.ld + e);
      }
    }
    const int place = e >= 0 ? tok * a.pad + e : -1;
    const unsigned same = same_place(place);  // (while the loads are in flight)
    if (a.sigmoid) {
      if (e >= 0) v = logistic(l);
    } else {
      float m = l;
      for (int d = slots >> 1; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      v = soft_exp(l, m);
    }
    float d;
    const float rest = a.sigmoid ? logistic_rest(l, v) : 1.f;
    if (a.renorm) {
      float total = v;
      for (int s = slots >> 1; s; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
      const float q = total > 0.f ? v / total : 0.f;
      float mean = q * dw;
      for (int s = slots >> 1; s; s >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, s);
      d = a.scale * q * (dw - mean) * rest;
    } else {
      d = a.scale * dw * v * rest;
    }
    if (join_slots(same, e >= 0, d)) rows[place] = d;
    __syncwarp();
    const int n = (int)(a.T - base < a.rows ? a.T - base : a.rows);
    T* out = static_cast<T*>(a.dlogits) + base * a.ld_d;
    for (int i = 0; i < n; ++i, out += a.ld_d) store_row(out, rows + i * a.pad, a.E, a.vector);
    __syncwarp();
    if (e >= 0) rows[place] = 0.f;
    __syncwarp();
  }
}

// Softmax without renormalisation, where every logit has a gradient:
//   dl_m = scale p_m (dw_m [m chosen] - sum over the chosen of p dw).
// One warp per token, the row in registers (EPL per lane, a lane's 32 apart).
template <typename T, int EPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_grad_dense_kernel(const RouteGradArgs a) {
  __shared__ float up_[kRouteWarps][EPL * 32];
  const int id = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* const up = up_[warp];
#pragma unroll
  for (int i = 0; i < EPL; ++i) up[i * 32 + id] = 0.f;
  __syncwarp();
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.T; t += (int64_t)gridDim.x * kRouteWarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    int e = id < a.k ? a.indices[t * a.k + id] : -1;
    if (e >= a.E) e = -1;
    const float dw = e >= 0 ? a.dweights[t * a.k + id] : 0.f;
    const unsigned same = same_place(e >= 0 ? e : -1);
    float p[EPL], m = -INFINITY, total = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = i * 32 + id < a.E ? logit_of(row + i * 32 + id) : -INFINITY;
      m = fmaxf(m, p[i]);
    }
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = soft_exp(p[i], m);
      total += p[i];
    }
    total = warp_sum(total);
    const float share = total > 0.f ? 1.f / total : 0.f;
    const float mean = warp_sum(e >= 0 ? soft_exp(logit_of(row + e), m) * share * dw : 0.f);
    float sum = dw;
    if (join_slots(same, e >= 0, sum)) up[e] = sum;
    __syncwarp();
    T* d = static_cast<T*>(a.dlogits) + t * a.ld_d;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i * 32 + id < a.E) store_one(d + i * 32 + id, a.scale * (p[i] * share) * (up[i * 32 + id] - mean));
    __syncwarp();
    if (e >= 0) up[e] = 0.f;
    __syncwarp();
  }
}

// Eight slots of a token (the usual k, and enough tokens for a warp to take four in turn)
// are known when compiling where a lane has eight experts.
template <typename T, int EPL, int LANES>
static void route_go(const RouteArgs& a, unsigned grid, cudaStream_t s) {
  if constexpr (EPL == 8) {
    if (a.k == 8 && a.log_slots == 3) return route_kernel<T, EPL, LANES, true><<<grid, kRouteWarps * 32, 0, s>>>(a);
  }
  route_kernel<T, EPL, LANES, false><<<grid, kRouteWarps * 32, 0, s>>>(a);
}

static int route_checks(int64_t T, int E, int k, int dtype, int score, int64_t ld, float scale) {
  if (!dtype_ok(dtype)) return ops_fail(MHC_ERR_CONFIG, "unknown dtype");
  if (score != MHC_SCORE_SOFTMAX && score != MHC_SCORE_SIGMOID) return ops_fail(MHC_ERR_CONFIG, "unknown score");
  if (T < 0 || E < 1 || E > kMaxExperts) return ops_fail(MHC_ERR_SHAPE, "need T >= 0 and 1 <= E <= 1024");
  if (k < 1 || k > 32 || k > E) return ops_fail(MHC_ERR_SHAPE, "need 1 <= k <= min(E, 32)");
  if (ld < E) return ops_fail(MHC_ERR_SHAPE, "the row stride must be at least E");
  if (T >= ((int64_t)1 << 31) || ld * (int64_t)dtype_bytes(dtype) >= ((int64_t)1 << 31))
    return ops_fail(MHC_ERR_SHAPE, "T and a row's bytes must be below 2^31");
  if (!(scale == scale)) return ops_fail(MHC_ERR_CONFIG, "scale is not a number");
  return MHC_OK;
}

#define MHC_BY_LANES(epl, lanes, ...)                                                              \
  if (lanes == 8) {                                                                                \
    constexpr int L = 8;                                                                           \
    if (epl == 1) { constexpr int N = 1; __VA_ARGS__; }                                            \
    else if (epl == 2) { constexpr int N = 2; __VA_ARGS__; }                                       \
    else if (epl == 4) { constexpr int N = 4; __VA_ARGS__; }                                       \
    else { constexpr int N = 8; __VA_ARGS__; }                                                     \
  } else if (lanes == 16) { constexpr int L = 16, N = 8; __VA_ARGS__; }                            \
  else {                                                                                           \
    constexpr int L = 32;                                                                          \
    if (epl == 1) { constexpr int N = 1; __VA_ARGS__; }                                            \
    else if (epl == 2) { constexpr int N = 2; __VA_ARGS__; }                                       \
    else if (epl == 4) { constexpr int N = 4; __VA_ARGS__; }                                       \
    else if (epl == 8) { constexpr int N = 8; __VA_ARGS__; }                                       \
    else if (epl == 16) { constexpr int N = 16; __VA_ARGS__; }                                     \
    else { constexpr int N = 32; __VA_ARGS__; }                                                    \
  }

#define MHC_BY_EXPERTS(E, ...)                                   \
  if (E <= 32) { constexpr int N = 1; __VA_ARGS__; }             \
  else if (E <= 64) { constexpr int N = 2; __VA_ARGS__; }        \
  else if (E <= 128) { constexpr int N = 4; __VA_ARGS__; }       \
  else if (E <= 256) { constexpr int N = 8; __VA_ARGS__; }       \
  else if (E <= 512) { constexpr int N = 16; __VA_ARGS__; }      \
  else { constexpr int N = 32; __VA_ARGS__; }

}  // namespace mhc

extern "C" {

size_t mhc_route_workspace_bytes(int E) { return E > 0 ? 256 + ((size_t)E * 4 + 255) / 256 * 256 : 0; }

int mhc_route(const void* logits, int64_t ld, mhc_dtype dtype, const float* bias, mhc_score score, int E, int groups,
              int top_groups, int k, int renorm, float scale, int64_t T, int32_t* indices, float* weights,
              int32_t* counts, void* workspace, size_t ws_bytes, void* stream) {
  using namespace mhc;
  int rc = route_checks(T, E, k, dtype, score, ld, scale);
  if (rc != MHC_OK) return rc;
  if (groups < 1 || groups > 32 || E % groups != 0 || top_groups < 1 || top_groups > groups)
    return ops_fail(MHC_ERR_SHAPE, "need 1 <= groups <= 32, E a multiple of groups and 1 <= top_groups <= groups");
  if (k > E / groups * top_groups) return ops_fail(MHC_ERR_SHAPE, "k is more than the experts of top_groups groups");
  if (top_groups == groups) groups = top_groups = 1;  // no group is left out
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!ops_aligned(counts, 4)) return ops_fail(MHC_ERR_ALIGN, "counts is not aligned");
  if (T == 0) return counts ? ops_cuda(cudaMemsetAsync(counts, 0, (size_t)E * 4, s), "cudaMemsetAsync") : MHC_OK;
  if (!logits || !indices || !weights) return ops_fail(MHC_ERR_NULL, "logits, indices and weights are required");
  const size_t b = dtype_bytes(dtype), need = counts ? mhc_route_workspace_bytes(E) : 0;
  if (!ops_aligned(logits, b) || !ops_aligned(bias, 4) || !ops_aligned(indices, 4) || !ops_aligned(weights, 4) ||
      (counts && !ops_aligned(workspace, 16)))
    return ops_fail(MHC_ERR_ALIGN, "a pointer is not aligned to its type");
  if (counts && (!workspace || ws_bytes < need))
    return ops_fail(MHC_ERR_WORKSPACE, "counts needs a workspace of mhc_route_workspace_bytes(E)");
  const Rows in[] = {{logits, T, E, ld, b}, {bias, 1, E, E, 4}};
  const Rows out[] = {{indices, 1, T * k, 1, 4}, {weights, 1, T * k, 1, 4}, {counts, 1, E, E, 4},
                      {counts ? workspace : nullptr, 1, (int64_t)need, 1, 1}};
  for (int o = 0; o < 4; ++o) {
    for (const Rows& i : in)
      if (rows_overlap(out[o], i)) return ops_fail(MHC_ERR_ALIAS, "an output overlaps an input");
    for (int q = o + 1; q < 4; ++q)
      if (rows_overlap(out[o], out[q])) return ops_fail(MHC_ERR_ALIAS, "two outputs overlap");
  }
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return ops_cuda(e, "device query");
  unsigned* ws = static_cast<unsigned*>(workspace);
  // Eight experts a lane where they allow it, so that a warp takes several tokens of a
  // small router; 32 lanes for more slots than lanes and for groups that do not
  // fall on whole lanes.
  int lanes = E <= 64 ? 8 : E <= 128 ? 16 : 32, epl = 1;
  while (epl * lanes < E) epl <<= 1;
  auto whole = [&]() {
    const int per = E / groups, n = per / epl;
    return E == epl * lanes && per % epl == 0 && (n & (n - 1)) == 0;
  };
  if (lanes < 32 && (k > lanes || (groups > 1 && !whole()))) {
    lanes = 32;
    for (epl = 1; epl * lanes < E;) epl <<= 1;
  }
  const bool vector = E == epl * lanes && (epl * b) % 16 == 0 && (ld * b) % 16 == 0 && ops_aligned(logits, 16);
  // Estimates do not help where equal choices are common (16-bit logits without a
  // bias), where groups need the exact path, and where a lane's list of four would
  // run out too often: with n lanes in play, about k^4 / (24 n^3) of the tokens.
  const int64_t n = lanes * top_groups / groups;
  const bool lists = epl <= 4 || lanes == 8 || (int64_t)k * k * k * k <= 2 * n * n * n;
  const bool estimate = (b == 4 || bias) && (groups == 1 || whole()) && lists;
  int log_slots = 0;
  while ((1 << log_slots) < k) ++log_slots;
  // tokens that a warp takes in turn cost latency: only as many as leave two warps per scheduler
  while ((32 >> log_slots) > 32 / lanes && T < (int64_t)sms * 8 * (32 >> log_slots)) ++log_slots;
  const RouteArgs a = {logits, (uint32_t)(ld * b), (uint32_t)T, bias, E, groups, top_groups, k, log_slots, score == MHC_SCORE_SIGMOID, renorm != 0, vector,
                       whole(), estimate, scale, indices, weights, counts, counts ? ws + 16 : nullptr, counts ? ws + 64 : nullptr};
  const int64_t tokens = kRouteWarps * (32 >> log_slots);
  int64_t grid = (T + tokens - 1) / tokens;
  if (grid > (int64_t)sms * kRouteCtas) grid = (int64_t)sms * kRouteCtas;
  MHC_BY_DTYPE(dtype, D, { MHC_BY_LANES(epl, lanes, { route_go<D, N, L>(a, (unsigned)grid, s); }) });
  return ops_cuda(cudaGetLastError(), "route launch");
}

int mhc_route_grad(const float* dweights, const void* logits, int64_t ld, mhc_dtype dtype, const int32_t* indices,
                   mhc_score score, int E, int k, int renorm, float scale, int64_t T, void* dlogits, int64_t ld_d,
                   void* stream) {
  using namespace mhc;
  int rc = route_checks(T, E, k, dtype, score, ld, scale);
  if (rc != MHC_OK) return rc;
  if (ld_d < E) return ops_fail(MHC_ERR_SHAPE, "the row stride must be at least E");
  if (T == 0) return MHC_OK;
  if (!dweights || !logits || !indices || !dlogits)
    return ops_fail(MHC_ERR_NULL, "dweights, logits, indices and dlogits are required");
  const size_t b = dtype_bytes(dtype);
  if (!ops_aligned(logits, b) || !ops_aligned(dlogits, b) || !ops_aligned(dweights, 4) || !ops_aligned(indices, 4))
    return ops_fail(MHC_ERR_ALIGN, "a pointer is not aligned to its type");
  const Rows out = {dlogits, T, E, ld_d, b};
  if (rows_overlap(out, {logits, T, E, ld, b}) || rows_overlap(out, {dweights, 1, T * k, 1, 4}) ||
      rows_overlap(out, {indices, 1, T * k, 1, 4}))
    return ops_fail(MHC_ERR_ALIAS, "dlogits overlaps an input");
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return ops_cuda(e, "device query");
  RouteGradArgs a = {dweights, logits, ld, T, indices, E, k, score == MHC_SCORE_SIGMOID, renorm != 0, scale,
                     dlogits, ld_d, 0, 1, (E + 3) / 4 * 4, false};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t most = (int64_t)sms * 2 * kRouteCtas;
  if (!a.sigmoid && !a.renorm) {
    const int64_t grid = (T + kRouteWarps - 1) / kRouteWarps;
    MHC_BY_DTYPE(dtype, D, {
      MHC_BY_EXPERTS(E, { route_grad_dense_kernel<D, N><<<(unsigned)(grid < most ? grid : most), kRouteWarps * 32, 0, s>>>(a); })
    });
  } else {
    while ((1 << a.log_slots) < k) ++a.log_slots;
    // tokens of a warp: one slot per lane, 8 KB of rows, and enough warps for every scheduler
    a.rows = 32 >> a.log_slots;
    while (a.rows > 1 && (a.rows * a.pad * 4 > 8192 || T < (int64_t)sms * 16 * a.rows)) a.rows >>= 1;
    a.vector = E * b % 16 == 0 && ld_d * b % 16 == 0 && ops_aligned(dlogits, 16);
    const int64_t grid = (T + kRouteWarps * a.rows - 1) / (kRouteWarps * a.rows);
    const size_t smem = (size_t)kRouteWarps * a.rows * a.pad * 4;
    MHC_BY_DTYPE(dtype, D, { route_grad_kernel<D><<<(unsigned)(grid < most ? grid : most), kRouteWarps * 32, smem, s>>>(a); });
  }
  return ops_cuda(cudaGetLastError(), "route_grad launch");
}

}  // extern "C"
