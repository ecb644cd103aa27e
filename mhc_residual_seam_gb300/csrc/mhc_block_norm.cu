// mhc_block_norm and its gradient: the norm after a block, the gate, the
// scaled residual add and the norm before the next block, for one residual
// stream.

#include "mhc_ops.cuh"

namespace mhc {

struct BlockNormArgs {
  const void *y, *r, *gamma_post, *gate, *gamma_pre;
  int64_t ld_y, ld_r, ld_ro, ld_n;
  int gate_mode;
  float scale, eps;
  int64_t T;
  int H;
  void *r_out, *norm;
  float *rstd_post, *rstd_pre;
  int run;  // rows of a CTA
};

struct BlockNormGradArgs {
  const void *dr_out, *dnorm, *y, *r_out, *gamma_post, *gate, *gamma_pre;
  const float *rstd_post, *rstd_pre;
  int gate_mode;
  float scale;
  int64_t T;
  int H;
  void *dy, *dr;
  float *dgamma_post, *dgate, *dgamma_pre;
  float* parts;  // [CTAs][2][H] column sums of each CTA: S and dgamma_pre
  int run;       // rows of a CTA
};

// A team of threads works on one row: a warp (rows of at most 512 columns,
// several teams per CTA) or the whole CTA.  A thread keeps the same VPT groups of
// eight columns for all of its team's rows: two groups, so that what a row costs
// beside its columns (the sums over the team, addresses) is shared by 16 columns.
template <bool WARP>
struct Team {
  int lanes, lane, teams, team;
  __device__ Team() {
    lanes = WARP ? 32 : blockDim.x;
    lane = WARP ? (threadIdx.x & 31) : threadIdx.x;
    teams = WARP ? (blockDim.x >> 5) : 1;
    team = WARP ? (threadIdx.x >> 5) : 0;
  }
};

// The sum over a team; `buf` is the caller's own slot of shared memory for this
// sum (QUADS * 4 warps at most; the places of warps that the CTA lacks hold zero),
// so one barrier per sum is enough.  The warps' sums are added in the same order
// everywhere.
template <bool WARP, int QUADS>
__device__ __forceinline__ float team_sum(float2 v, float4* buf) {
  float x = warp_sum(v.x + v.y);
  if constexpr (!WARP) {
    if ((threadIdx.x & 31) == 0) reinterpret_cast<float*>(buf)[threadIdx.x >> 5] = x;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < QUADS; ++i) {
      const float4 q = buf[i];
      s = __fadd2_rn(s, __fadd2_rn(make_float2(q.x, q.y), make_float2(q.z, q.w)));
    }
    x = s.x + s.y;
  }
  return x;
}

// Eight weights of a row; ones where there is no weight.
template <typename T>
__device__ __forceinline__ Vec8 weight8(const void* w, int g) {
  if (w) return unpack(ld8(static_cast<const T*>(w) + g * 8));
  Vec8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = make_float2(1.f, 1.f);
  return o;
}
template <typename T>
__device__ __forceinline__ float weight1(const void* w, int c) {
  if constexpr (sizeof(T) == 4) return static_cast<const float*>(w)[c];
  else return pair_of((uint32_t)static_cast<const uint16_t*>(w)[c], T()).x;
}
__device__ __forceinline__ Vec8 mul8(const Vec8& a, const Vec8& b) {
  Vec8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = __fmul2_rn(a.p[i], b.p[i]);
  return o;
}

// A CTA of at most kTeamThreads has 96 registers a thread, one of kBigThreads 64.
constexpr int kTeamThreads = 640, kBigThreads = 1024;

// Dynamic shared memory of a CTA: per team, the product of gamma_post and a
// channel gate as fp32 (each thread its own columns), then the fetched rows, then
// per warp and stage four words for the row's scalars.  All addresses are of
// this thread's columns.
template <typename T, int VPT, bool WARP, int STAGES, int MATRICES>
struct TeamMemory {
  uint32_t plane;    // bytes of eight 16-bit columns per group: one plane of a row
  uint32_t matrix;   // bytes of a row of one matrix
  uint32_t weight, ring, scalars;
  uint32_t stage_bytes;
  uint32_t col[VPT], smem[VPT];  // byte offsets of the thread's columns in a row, and in a plane
  bool on[VPT];                  // whether the row has these columns
  __device__ TeamMemory(const Team<WARP>& q, int segs, uint4* dyn) {
    plane = segs * 16;
    matrix = plane * (sizeof(T) / 2);
    stage_bytes = MATRICES * matrix;
    weight = smem_of(dyn) + q.team * plane * 2;
    ring = smem_of(dyn) + q.teams * plane * 2 + q.team * STAGES * stage_bytes;
    scalars = smem_of(dyn) + q.teams * (plane * 2 + STAGES * stage_bytes) + (threadIdx.x >> 5) * STAGES * 16;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int g = q.lane + i * q.lanes;
      on[i] = g < segs;
      col[i] = g * 8 * sizeof(T);
      smem[i] = g * 16;
    }
  }
};

// p = y rho1 gamma_post;  r' = scale r + gate p;  norm = r' rho2 gamma_pre.
// Bound by HBM: y and r are read once, r' and the norm written once; the row
// stays in registers between the two sums of squares.  The norm is formed from
// the fp32 r', so it carries one rounding only.  Each thread fetches its columns
// STAGES rows ahead (one or more: the widest fp32 row fits once), so loads stay in
// flight across the two barriers of a row.  Arithmetic is two columns per
// instruction.  rsqrtf (2 ulp) replaces a square root and a division that every
// thread would repeat.  FULL: every part but a gate is given and each thread has all of
// its columns, known when compiling (no tests per row; T = 16384, H = 5120 bf16: 121 us
// against 125, the gradient 174 against 199).  At that size 102 us, 97 % of the copy.
template <typename T, int VPT, bool WARP, int STAGES, bool FULL>
__global__ void __launch_bounds__(kBigThreads) block_norm_kernel(const BlockNormArgs a) {
  __shared__ float4 buf[2][2][8];
  extern __shared__ uint4 dyn[];
  const Team<WARP> q;
  const int segs = a.H >> 3;
  const float inv = 1.0f / (float)a.H;
  const bool has_y = FULL || a.y, has_r = FULL || a.r, has_post = FULL || a.gamma_post, has_pre = FULL || a.gamma_pre;
  const char* y = static_cast<const char*>(a.y);
  const char* r = static_cast<const char*>(a.r);
  const float* gates = a.gate_mode == MHC_GATE_TOKEN ? static_cast<const float*>(a.gate) : nullptr;
  const int step = q.teams;
  const int64_t first = (int64_t)blockIdx.x * a.run, end = first + a.run < a.T ? first + a.run : a.T;
  const TeamMemory<T, VPT, WARP, STAGES, 2> m(q, segs, dyn);
  auto on = [&](int i) { return FULL || m.on[i]; };
  auto fetch = [&](int64_t t, uint32_t slot, uint32_t scalar) {
    if (t < end) {
      const char* pr = r + t * (a.ld_r * (int)sizeof(T));
      const char* py = y + t * (a.ld_y * (int)sizeof(T));
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (on(i)) {
          if (has_r) fetch8<T>(slot + m.smem[i], m.plane, pr + m.col[i]);
          if (has_y) fetch8<T>(slot + m.matrix + m.smem[i], m.plane, py + m.col[i]);
        }
      if (gates && (threadIdx.x & 31) == 0) cp_async4(scalar, gates + t);
    }
    cp_async_commit();
  };
  int64_t t = first + q.team;
#pragma unroll
  for (int s = 0; s < STAGES; ++s) fetch(t + s * step, m.ring + s * m.stage_bytes, m.scalars + s * 16);
  Raw8<T> wn[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int g = q.lane + i * q.lanes;
    if (on(i)) {
      const Raw8<float> w = pack<float>(
          mul8(weight8<T>(a.gamma_post, g), weight8<T>(a.gate_mode == MHC_GATE_CHANNEL ? a.gate : nullptr, g)));
      sts16(m.weight + m.smem[i], w.q[0]);
      sts16(m.weight + m.plane + m.smem[i], w.q[1]);
      if (has_pre) wn[i] = ld8(static_cast<const T*>(a.gamma_pre) + g * 8);
    }
  }
  if constexpr (!WARP) {
    if (threadIdx.x < 32) buf[threadIdx.x >> 4][(threadIdx.x >> 3) & 1][threadIdx.x & 7] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  }
  int flip = 0;
  uint32_t slot = m.ring, scalar = m.scalars;
  for (; t < end; t += step, flip ^= 1) {
    Vec8 p[VPT], x[VPT];
    cp_async_wait<STAGES - 1>();
    float gt = 1.f;
    if (gates) {
      __syncwarp();
      gt = lds4(scalar);
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!FULL) p[i] = x[i] = zero8();
      if (on(i)) {
        if (has_r) x[i] = unpack(fetched8<T>(slot + m.smem[i], m.plane));
        if (has_y) p[i] = unpack(fetched8<T>(slot + m.matrix + m.smem[i], m.plane));
      }
    }
    fetch(t + STAGES * step, slot, scalar);
    slot += m.stage_bytes;
    scalar += 16;
    if (slot == m.ring + STAGES * m.stage_bytes) slot = m.ring, scalar = m.scalars;
    if (has_y) {
      float k = gt;
      if (has_post) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) ss = __ffma2_rn(p[i].p[e], p[i].p[e], ss);
        const float rho = rsqrtf(fmaf(team_sum<WARP, 8>(ss, buf[flip][0]), inv, a.eps));
        if (q.lane == 0) a.rstd_post[t] = rho;
        k *= rho;
      }
      char* o = static_cast<char*>(a.r_out) + t * (a.ld_ro * (int)sizeof(T));
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (on(i)) {
          const Vec8 wc = unpack(fetched8<float>(m.weight + m.smem[i], m.plane));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[i].p[e] = __ffma2_rn(__fmul2_rn(p[i].p[e], splat(k)), wc.p[e], __fmul2_rn(x[i].p[e], splat(a.scale)));
          st8_stream(reinterpret_cast<T*>(o + m.col[i]), pack<T>(x[i]));
        }
    }
    if (has_pre) {
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = __ffma2_rn(x[i].p[e], x[i].p[e], ss);
      const float rho = rsqrtf(fmaf(team_sum<WARP, 8>(ss, buf[flip][1]), inv, a.eps));
      if (q.lane == 0) a.rstd_pre[t] = rho;
      char* o = static_cast<char*>(a.norm) + t * (a.ld_n * (int)sizeof(T));
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (on(i)) {
          const Vec8 w = unpack(wn[i]);
          Vec8 n;
#pragma unroll
          for (int e = 0; e < 4; ++e) n.p[e] = __fmul2_rn(__fmul2_rn(x[i].p[e], splat(rho)), w.p[e]);
          st8_stream(reinterpret_cast<T*>(o + m.col[i]), pack<T>(n));
        }
    }
  }
  cp_async_wait<0>();
}

// With x = r', c = gamma_pre dnorm and M = sum c x over the row:
//   G = dr_out + rho2 c - x (rho2^3 M / H),  dr = scale G (without y: G),
//   dgamma_pre += rho2 dnorm x
// and with g = rho1 G, w = gamma_post * gate (channel), b = w g, N = sum b y:
//   dy = gate(token) (b - y (rho1^2 N / H)),  dgate(token) = N
//   S += gate(token) g y: dgamma_post = S gate(channel), dgate(channel) = S gamma_post
// (S is one column sum for both; without gamma_post, rho1 = 1 and dy has no second
// term.)  Bound by HBM: four rows read, two written.  A thread keeps the same
// columns over all of its team's rows, so the column sums stay in registers until
// the end; a second kernel adds the CTAs' sums in a fixed order.  Rows and
// their scalars are fetched ahead as in the forward kernel (STAGES 0: fp32 rows
// above 11520 columns, plain loads); FULL as there.  Above 10240 columns 64 registers a
// thread are too few: 250 to 350 bytes of spills.
// T = 16384, H = 5120 bf16: 167 us with the fold, 89 % of the copy.
template <typename T, int VPT, bool WARP, bool BIG, int STAGES, bool FULL>
__global__ void __launch_bounds__(BIG ? kBigThreads : kTeamThreads) block_norm_grad_kernel(const BlockNormGradArgs a) {
  constexpr int QUADS = BIG ? 8 : kTeamThreads / 128;
  __shared__ float4 buf[2][2][8];
  extern __shared__ uint4 dyn[];
  const Team<WARP> q;
  const int segs = a.H >> 3;
  const float inv = 1.0f / (float)a.H;
  const TeamMemory<T, VPT, WARP, STAGES, 4> m(q, segs, dyn);
  const bool has_y = FULL || a.y, has_post = FULL || a.gamma_post, has_pre = FULL || a.gamma_pre, has_dr = FULL || a.dr_out;
  const char* const src[4] = {static_cast<const char*>(a.r_out), static_cast<const char*>(a.dnorm),
                              static_cast<const char*>(a.dr_out), static_cast<const char*>(a.y)};
  const bool has[4] = {has_pre, has_pre, has_dr, has_y};
  const float* gates = a.gate_mode == MHC_GATE_TOKEN ? static_cast<const float*>(a.gate) : nullptr;
  const int row_bytes = a.H * (int)sizeof(T);
  auto on = [&](int i) { return FULL || m.on[i]; };
  const int64_t first = (int64_t)blockIdx.x * a.run, end = first + a.run < a.T ? first + a.run : a.T;
  auto fetch = [&](int64_t t, uint32_t slot, uint32_t scalar) {
    if (t < end) {
      const int64_t row = t * row_bytes;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (has[k]) {
          const char* p = src[k] + row;
#pragma unroll
          for (int i = 0; i < VPT; ++i)
            if (on(i)) fetch8<T>(slot + k * m.matrix + m.smem[i], m.plane, p + m.col[i]);
        }
      if ((threadIdx.x & 31) == 0) {
        if (has_pre) cp_async4(scalar, a.rstd_pre + t);
        if (has_post) cp_async4(scalar + 4, a.rstd_post + t);
        if (gates) cp_async4(scalar + 8, gates + t);
      }
    }
    cp_async_commit();
  };
  const int step = q.teams;
  int64_t t = first + q.team;
#pragma unroll
  for (int s = 0; s < STAGES; ++s) fetch(t + s * step, m.ring + s * m.stage_bytes, m.scalars + s * 16);
  Vec8 s_post[VPT], s_pre[VPT];
  Raw8<T> wn[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int g = q.lane + i * q.lanes;
    s_post[i] = s_pre[i] = zero8();
    if (on(i)) {
      const Raw8<float> w = pack<float>(
          mul8(weight8<T>(a.gamma_post, g), weight8<T>(a.gate_mode == MHC_GATE_CHANNEL ? a.gate : nullptr, g)));
      sts16(m.weight + m.smem[i], w.q[0]);
      sts16(m.weight + m.plane + m.smem[i], w.q[1]);
      if (has_pre) wn[i] = ld8(static_cast<const T*>(a.gamma_pre) + g * 8);
    }
  }
  if constexpr (!WARP) {
    if (threadIdx.x < 32) buf[threadIdx.x >> 4][(threadIdx.x >> 3) & 1][threadIdx.x & 7] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
  }
  int flip = 0;
  uint32_t slot = m.ring, scalar = m.scalars;
  for (; t < end; t += step, flip ^= 1) {
    Vec8 G[VPT], x[VPT];
    const int64_t row = t * row_bytes;
    if constexpr (STAGES > 0) {
      cp_async_wait<(STAGES > 0 ? STAGES - 1 : 0)>();
      __syncwarp();
    }
    float rho2 = 1.f, rho1 = 1.f, gt = 1.f;
    if (has_pre) rho2 = STAGES ? lds4(scalar) : a.rstd_pre[t];
    if (has_post) rho1 = STAGES ? lds4(scalar + 4) : a.rstd_post[t];
    if (gates) gt = STAGES ? lds4(scalar + 8) : gates[t];
    auto take = [&](int k, int i) {
      return unpack(STAGES ? fetched8<T>(slot + k * m.matrix + m.smem[i], m.plane)
                           : ld8_stream(reinterpret_cast<const T*>(src[k] + row + m.col[i])));
    };
    if (has_pre) {
      float2 m2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!FULL) G[i] = x[i] = zero8();
        if (on(i)) {
          x[i] = take(0, i);
          const Vec8 dn = take(1, i), w = unpack(wn[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 dx = __fmul2_rn(dn.p[e], x[i].p[e]);
            s_pre[i].p[e] = __ffma2_rn(dx, splat(rho2), s_pre[i].p[e]);
            G[i].p[e] = __fmul2_rn(w.p[e], dn.p[e]);
            m2 = __ffma2_rn(w.p[e], dx, m2);
          }
        }
      }
      const float k = -rho2 * rho2 * (team_sum<WARP, QUADS>(m2, buf[flip][0]) * inv) * rho2;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const Vec8 d = has_dr && on(i) ? take(2, i) : zero8();
#pragma unroll
        for (int e = 0; e < 4; ++e)
          G[i].p[e] = __ffma2_rn(x[i].p[e], splat(k), __ffma2_rn(G[i].p[e], splat(rho2), d.p[e]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) G[i] = on(i) ? take(2, i) : zero8();
    }
    char* dr = static_cast<char*>(a.dr) + row;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if ((FULL || a.dr) && on(i)) {
        Vec8 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.p[e] = __fmul2_rn(G[i].p[e], splat(a.scale));
        st8_stream(reinterpret_cast<T*>(dr + m.col[i]), pack<T>(o));
      }
    float2 n2 = make_float2(0.f, 0.f);
    if (has_y) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!FULL) x[i] = zero8();
        if (on(i)) {
          x[i] = take(3, i);
          const Vec8 wc = unpack(fetched8<float>(m.weight + m.smem[i], m.plane));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 gr = __fmul2_rn(G[i].p[e], splat(rho1));
            s_post[i].p[e] = __ffma2_rn(__fmul2_rn(gr, splat(gt)), x[i].p[e], s_post[i].p[e]);
            G[i].p[e] = __fmul2_rn(wc.p[e], gr);
            n2 = __ffma2_rn(G[i].p[e], x[i].p[e], n2);
          }
        }
      }
    }
    // the row is in registers: its stage takes the row STAGES further on
    if constexpr (STAGES > 0) {
      __syncwarp();
      fetch(t + STAGES * step, slot, scalar);
      slot += m.stage_bytes;
      scalar += 16;
      if (slot == m.ring + STAGES * m.stage_bytes) slot = m.ring, scalar = m.scalars;
    }
    if (has_y) {
      float k = 0.f;
      if (has_post || gates) {
        const float N = team_sum<WARP, QUADS>(n2, buf[flip][1]);
        if (gates && q.lane == 0) a.dgate[t] = N;
        if (has_post) k = -rho1 * (N * inv) * rho1 * gt;
      }
      char* dy = static_cast<char*>(a.dy) + row;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (on(i)) {
          Vec8 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o.p[e] = __fmul2_rn(G[i].p[e], splat(gt));
            if (has_post) o.p[e] = __ffma2_rn(x[i].p[e], splat(k), o.p[e]);
          }
          st8_stream(reinterpret_cast<T*>(dy + m.col[i]), pack<T>(o));
        }
    }
  }
  if constexpr (STAGES > 0) cp_async_wait<0>();
  pdl_launch();
  const void* channel = a.gate_mode == MHC_GATE_CHANNEL ? a.gate : nullptr;
  const bool want_post = a.dgamma_post || channel, want_pre = a.dgamma_pre;
  // the CTA's column sums: to its row of `parts`, or, where it is the only CTA, to the weights' gradients
  auto finish = [&](int g, const Vec8& post, const Vec8& pre) {
    float* const out = a.parts + (int64_t)blockIdx.x * 2 * a.H + g * 8;
    if (gridDim.x > 1) {
      if (want_post) st8(out, pack<float>(post));
      if (want_pre) st8(out + a.H, pack<float>(pre));
    } else {
      const Vec8 p = mul8(post, weight8<T>(channel, g)), q = mul8(post, weight8<T>(a.gamma_post, g));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = g * 8 + 2 * e;
        if (a.dgamma_post) a.dgamma_post[c] = p.p[e].x, a.dgamma_post[c + 1] = p.p[e].y;
        if (channel) a.dgate[c] = q.p[e].x, a.dgate[c + 1] = q.p[e].y;
        if (want_pre) a.dgamma_pre[c] = pre.p[e].x, a.dgamma_pre[c + 1] = pre.p[e].y;
      }
    }
  };
  if constexpr (!WARP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (on(i)) finish(q.lane + i * q.lanes, s_post[i], s_pre[i]);
  } else {  // the teams' sums in team order, through the shared memory that held their rows
    __syncthreads();
    const uint32_t sums = smem_of(dyn), team_bytes = 4 * m.plane;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (on(i)) {
        const uint32_t at = sums + q.team * team_bytes + m.smem[i];
        const Raw8<float> p = pack<float>(s_post[i]), r = pack<float>(s_pre[i]);
        sts16(at, p.q[0]);
        sts16(at + m.plane, p.q[1]);
        sts16(at + 2 * m.plane, r.q[0]);
        sts16(at + 3 * m.plane, r.q[1]);
      }
    __syncthreads();
    for (int g = threadIdx.x; g < segs; g += blockDim.x) {
      Vec8 post = zero8(), pre = zero8();
      for (int t2 = 0; t2 < q.teams; ++t2) {
        const Vec8 p = unpack(fetched8<float>(sums + t2 * team_bytes + g * 16, m.plane));
        const Vec8 r = unpack(fetched8<float>(sums + t2 * team_bytes + 2 * m.plane + g * 16, m.plane));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          post.p[e] = __fadd2_rn(post.p[e], p.p[e]);
          pre.p[e] = __fadd2_rn(pre.p[e], r.p[e]);
        }
      }
      finish(g, post, pre);
    }
  }
}

// Adds the CTAs' column sums in a fixed order and finishes the weights'
// gradients: 32 * N columns x 32 slices of parts per CTA, N columns a thread (four
// for wide rows, one where that leaves most SMs idle), the slices joined in slice
// order.
template <typename T, int N>
__global__ void __launch_bounds__(1024) block_norm_fold_kernel(const BlockNormGradArgs a, int n) {
  struct alignas(N * 4) Cols {
    float v[N];
  };
  __shared__ Cols sh[32][32];
  pdl_wait();
  const bool post = blockIdx.y == 0;
  const bool channel = a.gate_mode == MHC_GATE_CHANNEL;
  if (post ? !a.dgamma_post && !channel : !a.dgamma_pre) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * N;
  Cols x = {};
  auto add = [&](const Cols& o) {
#pragma unroll
    for (int e = 0; e < N; ++e) x.v[e] += o.v[e];
  };
  if (c < a.H) {
    const float* p = a.parts + (post ? 0 : a.H) + c;
    const int lo = (int)((int64_t)n * w / 32), hi = (int)((int64_t)n * (w + 1) / 32);
#pragma unroll 8
    for (int i = lo; i < hi; ++i) add(*reinterpret_cast<const Cols*>(p + (int64_t)i * 2 * a.H));
  }
  sh[w][lane] = x;
  __syncthreads();
  if (w || c >= a.H) return;
#pragma unroll 8
  for (int i = 1; i < 32; ++i) add(sh[i][lane]);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (!post) {
      a.dgamma_pre[c + e] = x.v[e];
      continue;
    }
    if (a.dgamma_post) a.dgamma_post[c + e] = x.v[e] * (channel ? weight1<T>(a.gate, c + e) : 1.f);
    if (channel) a.dgate[c + e] = x.v[e] * (a.gamma_post ? weight1<T>(a.gamma_post, c + e) : 1.f);
  }
}

// The teams of a row of H columns and how many rows they fetch ahead.
struct TeamPlan {
  bool warp, big;
  int vpt, threads, teams, stages;
  size_t smem;
  int ctas;  // per SM
};

constexpr int kSMs = 152, kFewRows = 4;
constexpr size_t kSmem = 227 * 1024;         // shared memory of an SM
constexpr size_t kCtaSmem = 1024 + 512 + 128;  // what a CTA takes of it beside the dynamic part

// `sm_threads`: threads of an SM that the kernel's registers allow for.
static constexpr TeamPlan team_plan(int H, size_t type_bytes, int matrices, int sm_threads) {
  const int segs = H / 8;
  TeamPlan p = {};
  // (the gradient keeps 64 registers of sums a thread: one warp per CTA instead of four
  // teams with two groups a thread, T = 65536, H = 512 bf16: 77 us against 114)
  p.warp = segs <= (matrices == 4 ? 32 : 64);
  p.vpt = segs <= 32 ? 1 : 2;
  p.threads = p.warp ? 128 : ((segs + 1) / 2 + 31) / 32 * 32;
  p.big = p.threads > kTeamThreads;
  p.teams = p.warp ? 4 : 1;
  const size_t row = (size_t)H * type_bytes * matrices * p.teams, weights = (size_t)H * 4 * p.teams;
  p.ctas = sm_threads / p.threads;
  if (p.ctas < 1) p.ctas = 1;
  if (p.ctas > 16) p.ctas = 16;
  const size_t stage = row + (size_t)(p.threads / 32) * 16;  // with the rows' scalars
  while (p.ctas > 1 && (stage * 2 + weights + kCtaSmem) * p.ctas > kSmem) --p.ctas;
  // two CTAs with one row each in flight rather than one with two: CTAs of a short run
  // have to overlap
  if (p.ctas == 1 && 2 * p.threads <= sm_threads && (stage + weights + kCtaSmem) * 2 <= kSmem) p.ctas = 2;
  const size_t have = kSmem / p.ctas, fixed = weights + kCtaSmem;
  const size_t fit = have > fixed ? (have - fixed) / stage : 0;
  p.stages = fit >= 4 ? 4 : fit >= 2 ? 2 : (int)fit;
  p.smem = weights + stage * p.stages;
  return p;
}

static constexpr TeamPlan norm_plan(int H, size_t b) { return team_plan(H, b, 2, 1024); }
static constexpr TeamPlan grad_plan(int H, size_t b) { return team_plan(H, b, 4, 640); }

// Rows of a CTA.  Forward: runs of four, so that CTAs start as others end and an
// SM that gets through faster takes more of them (T = 16384, H = 5120 bf16: 102 us;
// one run of 36 rows per resident CTA, with the same number of bytes in flight,
// 120; runs of 1, 2 and 9 rows 123, 103 and 105).  Fewer when that leaves SMs idle.
// Gradient: one run per resident CTA, since every run adds a row of column sums
// that has to be written and folded (runs of 54 rows 166 us, 27 rows 172, 16 rows 192).
static int resident_run(int64_t T, const TeamPlan& p) {
  const int64_t slots = (int64_t)kSMs * p.ctas, even = (T + slots - 1) / slots;
  return (int)((even + p.teams - 1) / p.teams * p.teams);
}
static int norm_run(int64_t T, const TeamPlan& p) {
  const int even = resident_run(T, p);
  return even > 4 * p.teams ? 4 * p.teams : even;
}
// A few rows go to one CTA, which needs no fold (T = 4, H = 5120: one launch less).
static int grad_run(int64_t T, const TeamPlan& p) {
  const int few = kFewRows * p.teams;
  return T <= few ? few : resident_run(T, p);
}
static int64_t grad_ctas(int64_t T, const TeamPlan& p) { return (T + grad_run(T, p) - 1) / grad_run(T, p); }
// The most CTAs that T rows or fewer take: one a team's rows, until all are resident.  (A longer
// run halves their number, so grad_ctas itself falls where T grows past a full GPU.)
static int64_t grad_ctas_most(int64_t T, const TeamPlan& p) {
  if (T <= kFewRows * p.teams) return 1;
  const int64_t each = (T + p.teams - 1) / p.teams, slots = (int64_t)kSMs * p.ctas;
  return each < slots ? each : slots;
}

// Whether every thread has all of its columns.
static constexpr bool even_columns(int H, const TeamPlan& p) { return H / 8 == p.vpt * (p.warp ? 32 : p.threads); }

constexpr int kMaxWidth = 16384;

// Whether the plan of some width takes a variant; the others are not compiled.
template <int BYTES, int MATRICES>
static constexpr bool taken(int vpt, bool warp, bool big, int stages, bool full) {
  for (int H = 8; H <= kMaxWidth; H += 8) {
    const TeamPlan p = MATRICES == 2 ? norm_plan(H, BYTES) : grad_plan(H, BYTES);
    if (p.vpt == vpt && p.warp == warp && p.big == big && p.stages == stages && (!full || even_columns(H, p))) return true;
  }
  return false;
}

// Runs its last argument with the plan's variant: groups per thread N, a warp per row W, more
// than kTeamThreads L, rows ahead K, no tests F.
#define MHC_BY_TEAM(plan, full, M, ...)                                                               \
  if (plan.stages == 0) { constexpr int K = 0; constexpr bool F = false; MHC_BY_TEAM_(plan, M, __VA_ARGS__) } \
  else if (full) { constexpr bool F = true; MHC_BY_STAGES(plan, M, __VA_ARGS__) }                     \
  else { constexpr bool F = false; MHC_BY_STAGES(plan, M, __VA_ARGS__) }
#define MHC_BY_STAGES(plan, M, ...)                                                                   \
  if (plan.stages == 4) { constexpr int K = 4; MHC_BY_TEAM_(plan, M, __VA_ARGS__) }                   \
  else if (plan.stages == 2) { constexpr int K = 2; MHC_BY_TEAM_(plan, M, __VA_ARGS__) }              \
  else { constexpr int K = 1; MHC_BY_TEAM_(plan, M, __VA_ARGS__) }
#define MHC_BY_TEAM_(plan, M, ...)                                                                    \
  if (plan.vpt == 1) { MHC_TEAM(1, true, false, M, __VA_ARGS__) }                                     \
  else if (plan.warp) { MHC_TEAM(2, true, false, M, __VA_ARGS__) }                                    \
  else if (!plan.big) { MHC_TEAM(2, false, false, M, __VA_ARGS__) }                                   \
  else { MHC_TEAM(2, false, true, M, __VA_ARGS__) }
#define MHC_TEAM(n, w, l, M, ...)                                                                     \
  constexpr int N = n;                                                                                \
  constexpr bool W = w, L = l;                                                                        \
  if constexpr (taken<(int)sizeof(E), M>(N, W, L, K, F)) { __VA_ARGS__; }

template <typename T, int N, bool W, int K, bool F>
static cudaError_t norm_launch(const BlockNormArgs& a, const TeamPlan& p, cudaStream_t s) {
  static SmemGrant grant;
  cudaError_t e = allow_smem(grant, (const void*)block_norm_kernel<T, N, W, K, F>, p.smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = (a.T + a.run - 1) / a.run;
  block_norm_kernel<T, N, W, K, F><<<(unsigned)grid, p.threads, p.smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int N, bool W, bool L, int K, bool F>
static cudaError_t grad_launch(const BlockNormGradArgs& a, const TeamPlan& p, int64_t grid, cudaStream_t s) {
  static SmemGrant grant;
  cudaError_t e = allow_smem(grant, (const void*)block_norm_grad_kernel<T, N, W, L, K, F>, p.smem);
  if (e != cudaSuccess) return e;
  block_norm_grad_kernel<T, N, W, L, K, F><<<(unsigned)grid, p.threads, p.smem, s>>>(a);
  return cudaGetLastError();
}

static int shape_checks(int64_t T, int H, int dtype, int gate_mode) {
  if (!dtype_ok(dtype)) return ops_fail(MHC_ERR_CONFIG, "unknown dtype");
  if (gate_mode < MHC_GATE_NONE || gate_mode > MHC_GATE_TOKEN) return ops_fail(MHC_ERR_CONFIG, "unknown gate_mode");
  if (T < 0 || T > 0x7fffffff || H <= 0 || H % 8 != 0 || H > kMaxWidth)
    return ops_fail(MHC_ERR_SHAPE, "need 0 <= T < 2^31 and H a positive multiple of 8, at most 16384");
  return MHC_OK;
}

}  // namespace mhc

extern "C" {

int mhc_block_norm(const void* y, int64_t ld_y, const void* r, int64_t ld_r, const void* gamma_post, const void* gate,
                   int gate_mode, const void* gamma_pre, float res_scale, float eps, int64_t T, int H, mhc_dtype dtype,
                   void* r_out, int64_t ld_r_out, void* norm, int64_t ld_norm, float* rstd_post, float* rstd_pre,
                   void* stream) {
  using namespace mhc;
  int rc = shape_checks(T, H, dtype, gate_mode);
  if (rc != MHC_OK) return rc;
  if (!(eps >= 0.f) || eps > 1e30f) return ops_fail(MHC_ERR_CONFIG, "eps must be finite and >= 0");
  if (T == 0) return MHC_OK;
  if (!y) r_out = nullptr;
  if (!gamma_pre) norm = nullptr;
  if ((!r && !y) || (y && !r_out) || (gamma_pre && (!norm || !rstd_pre)) || (gamma_post && !rstd_post))
    return ops_fail(MHC_ERR_NULL, "a required pointer is NULL");
  if ((gate_mode != MHC_GATE_NONE) != (gate != nullptr))
    return ops_fail(MHC_ERR_NULL, "gate must be given exactly when gate_mode is not none");
  if (!y && (gamma_post || gate || !gamma_pre))
    return ops_fail(MHC_ERR_INCOMPLETE_POST, "without y the call is the norm before the first block: gamma_pre only");
  const int64_t lds[] = {y ? ld_y : H, r ? ld_r : H, y ? ld_r_out : H, gamma_pre ? ld_norm : H};
  for (int64_t ld : lds)
    if (ld < H || ld % 8 != 0) return ops_fail(MHC_ERR_SHAPE, "row strides must be multiples of 8, at least H");
  const void* a16[] = {y, r, gamma_post, gate_mode == MHC_GATE_CHANNEL ? gate : nullptr, gamma_pre, r_out, norm};
  for (const void* p : a16)
    if (!ops_aligned(p, 16)) return ops_fail(MHC_ERR_ALIGN, "a pointer that must be 16-byte aligned is not");
  if (!ops_aligned(gate, 4) || !ops_aligned(rstd_post, 4) || !ops_aligned(rstd_pre, 4))
    return ops_fail(MHC_ERR_ALIGN, "a fp32 pointer is not aligned");
  const size_t b = dtype_bytes(dtype);
  const Rows in[] = {{y, T, H, ld_y, b}, {r, T, H, ld_r, b}, {gamma_post, 1, H, H, b},
                     {gate, 1, gate_mode == MHC_GATE_TOKEN ? T : H, H, gate_mode == MHC_GATE_TOKEN ? 4 : b},
                     {gamma_pre, 1, H, H, b}};
  const Rows out[] = {{r_out, T, H, ld_r_out, b}, {norm, T, H, ld_norm, b}, {gamma_post ? rstd_post : nullptr, 1, T, T, 4},
                      {gamma_pre ? rstd_pre : nullptr, 1, T, T, 4}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i)
      if (!(o == 0 && i == 1 && r_out && r_out == r && ld_r_out == ld_r) && rows_overlap(out[o], in[i]))
        return ops_fail(MHC_ERR_ALIAS, "an output overlaps an input");
    for (int q = o + 1; q < 4; ++q)
      if (rows_overlap(out[o], out[q])) return ops_fail(MHC_ERR_ALIAS, "two outputs overlap");
  }
  BlockNormArgs a = {y, r, gamma_post, gate, gamma_pre, ld_y, ld_r, ld_r_out, ld_norm, gate_mode, res_scale, eps,
                           T, H, r_out, norm, rstd_post, rstd_pre, 1};
  const TeamPlan plan = norm_plan(H, b);
  const bool full = y && r && gamma_post && gamma_pre && even_columns(H, plan);
  a.run = norm_run(T, plan);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidConfiguration;  // a plan without a kernel: none
  MHC_BY_DTYPE(dtype, E, { MHC_BY_TEAM(plan, full, 2, { e = norm_launch<E, N, W, K, F>(a, plan, s); }) });
  return ops_cuda(e, "block_norm launch");
}

size_t mhc_block_norm_grad_workspace_bytes(int64_t T, int H) {
  if (T <= 0 || H <= 0) return 0;
  size_t most = 0;  // the plan differs by the type's size
  for (size_t b = 2; b <= 4; b += 2) {
    const mhc::TeamPlan p = mhc::grad_plan(H, b);
    const size_t n = (size_t)mhc::grad_ctas_most(T, p) * 2 * H * sizeof(float);
    if (n > most) most = n;
  }
  return most;
}

int mhc_block_norm_grad(const void* dr_out, const void* dnorm, const void* y, const void* r_out, const void* gamma_post,
                        const void* gate, int gate_mode, const void* gamma_pre, const float* rstd_post,
                        const float* rstd_pre, float res_scale, int64_t T, int H, mhc_dtype dtype, void* dy, void* dr,
                        float* dgamma_post, float* dgate, float* dgamma_pre, void* workspace, size_t ws_bytes,
                        void* stream) {
  using namespace mhc;
  int rc = shape_checks(T, H, dtype, gate_mode);
  if (rc != MHC_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool channel = gate_mode == MHC_GATE_CHANNEL, token = gate_mode == MHC_GATE_TOKEN;
  if ((gamma_post && !dgamma_post) || (gamma_pre && !dgamma_pre) || (gate_mode != MHC_GATE_NONE && !dgate))
    return ops_fail(MHC_ERR_NULL, "a required pointer is NULL");
  if ((gate_mode != MHC_GATE_NONE) != (gate != nullptr) && T > 0)
    return ops_fail(MHC_ERR_NULL, "gate must be given exactly when gate_mode is not none");
  if (!gamma_post) dgamma_post = nullptr;
  if (!gamma_pre) dgamma_pre = nullptr, dnorm = nullptr, r_out = nullptr;
  if (gate_mode == MHC_GATE_NONE) dgate = nullptr;
  if (!ops_aligned(dgamma_post, 4) || !ops_aligned(dgamma_pre, 4) || !ops_aligned(dgate, 4))
    return ops_fail(MHC_ERR_ALIGN, "a fp32 pointer is not aligned");
  if (T == 0) {  // sums over no rows
    float* z[] = {dgamma_post, channel ? dgate : nullptr, dgamma_pre};
    for (float* p : z)
      if (p) {
        rc = ops_cuda(cudaMemsetAsync(p, 0, (size_t)H * 4, s), "cudaMemsetAsync");
        if (rc != MHC_OK) return rc;
      }
    return MHC_OK;
  }
  if ((!dr_out && !gamma_pre) || (!dr && !y) || (y && !dy) || (gamma_pre && (!dnorm || !r_out || !rstd_pre)) ||
      (gamma_post && !rstd_post))
    return ops_fail(MHC_ERR_NULL, "a required pointer is NULL");
  if (!y && (gamma_post || gate || !gamma_pre))
    return ops_fail(MHC_ERR_INCOMPLETE_POST, "without y the call is the norm before the first block: gamma_pre only");
  if (!y) dy = nullptr;
  const void* a16[] = {dr_out, dnorm, y, r_out, gamma_post, channel ? gate : nullptr, gamma_pre, dy, dr, workspace};
  for (const void* p : a16)
    if (!ops_aligned(p, 16)) return ops_fail(MHC_ERR_ALIGN, "a pointer that must be 16-byte aligned is not");
  if (!ops_aligned(gate, 4) || !ops_aligned(rstd_post, 4) || !ops_aligned(rstd_pre, 4))
    return ops_fail(MHC_ERR_ALIGN, "a fp32 pointer is not aligned");
  const size_t need = mhc_block_norm_grad_workspace_bytes(T, H);
  if (!workspace || ws_bytes < need)
    return ops_fail(MHC_ERR_WORKSPACE, "workspace NULL or smaller than mhc_block_norm_grad_workspace_bytes(T, H)");
  const size_t b = dtype_bytes(dtype);
  const Rows in[] = {{dr_out, T, H, H, b}, {dnorm, T, H, H, b}, {y, T, H, H, b}, {r_out, T, H, H, b},
                     {gamma_post, 1, H, H, b}, {gate, 1, token ? T : H, H, token ? 4 : b}, {gamma_pre, 1, H, H, b},
                     {gamma_post ? rstd_post : nullptr, 1, T, T, 4}, {gamma_pre ? rstd_pre : nullptr, 1, T, T, 4}};
  const Rows out[] = {{dy, T, H, H, b}, {dr, T, H, H, b}, {dgamma_post, 1, H, H, 4}, {dgate, 1, token ? T : H, H, 4},
                      {dgamma_pre, 1, H, H, 4}, {workspace, 1, (int64_t)need, 1, 1}};
  for (int o = 0; o < 6; ++o) {
    for (const Rows& i : in)
      if (rows_overlap(out[o], i)) return ops_fail(MHC_ERR_ALIAS, "an output overlaps an input");
    for (int q = o + 1; q < 6; ++q)
      if (rows_overlap(out[o], out[q])) return ops_fail(MHC_ERR_ALIAS, "two outputs overlap");
  }
  // (without y the forward call normed r itself, unscaled)
  BlockNormGradArgs a = {dr_out, dnorm, y, r_out, gamma_post, gate, gamma_pre, rstd_post, rstd_pre, gate_mode,
                               y ? res_scale : 1.f, T, H, dy, dr, dgamma_post, dgate, dgamma_pre, static_cast<float*>(workspace), 1};
  const TeamPlan plan = grad_plan(H, b);
  const bool full = y && dr && dr_out && gamma_post && gamma_pre && even_columns(H, plan);
  a.run = grad_run(T, plan);
  const int64_t grid = grad_ctas(T, plan);
  cudaError_t e = cudaErrorInvalidConfiguration;  // a plan without a kernel: none
  MHC_BY_DTYPE(dtype, E, { MHC_BY_TEAM(plan, full, 4, { e = grad_launch<E, N, W, L, K, F>(a, plan, grid, s); }) });
  if (e == cudaSuccess && grid > 1 && (dgamma_post || dgamma_pre || channel))
    MHC_BY_DTYPE(dtype, E, {
      e = H >= 4096 ? launch_pdl(block_norm_fold_kernel<E, 4>, dim3((H + 127) / 128, 2), dim3(1024), 0, s, a, (int)grid)
                    : launch_pdl(block_norm_fold_kernel<E, 1>, dim3((H + 31) / 32, 2), dim3(1024), 0, s, a, (int)grid);
    });
  return ops_cuda(e, "block_norm_grad launch");
}

}  // extern "C"
