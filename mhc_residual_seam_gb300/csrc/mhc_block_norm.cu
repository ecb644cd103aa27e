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
  float* parts;  // [gridDim.x][3][H] column sums of each CTA: gamma_post, gate, gamma_pre
};

// A team of threads works on one row: a warp (several rows per CTA) or the
// whole CTA.  team_sum adds over the team; `buf` is the caller's own slot of
// shared memory for this sum, so one barrier per sum is enough.
template <bool WARP>
__device__ __forceinline__ float team_sum(float x, float* buf) {
  x = warp_sum(x);
  if constexpr (!WARP) {
    const int w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[w] = x;
    __syncthreads();
    x = 0.f;
    for (int i = 0; i < nw; ++i) x += buf[i];
  }
  return x;
}

// p = y rho1 gamma_post;  r' = scale r + gate p;  norm = r' rho2 gamma_pre.
// Bound by HBM: y and r are read once, r' and the norm written once; the row
// stays in registers between the two sums of squares.  The norm is formed from
// the fp32 r', so it carries one rounding only.
template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 512) block_norm_kernel(const BlockNormArgs a) {
  __shared__ float buf[2][16];
  const int lanes = WARP ? 32 : blockDim.x;
  const int lane = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t t = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && t >= a.T) return;
  const int segs = a.H >> 3;
  const float inv = 1.0f / (float)a.H;
  const T* y = static_cast<const T*>(a.y);
  const T* r = static_cast<const T*>(a.r);

  Vec8 p[VPT], x[VPT];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int g = lane + i * lanes;
    p[i] = {};
    x[i] = {};
    if (g < segs) {
      x[i] = unpack(ld8_stream(r + t * a.ld_r + g * 8));
      if (y) p[i] = unpack(ld8_stream(y + t * a.ld_y + g * 8));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(p[i].v[e], p[i].v[e], ss);
  }
  if (y) {
    float rho = 1.f;
    if (a.gamma_post) {
      ss = team_sum<WARP>(ss, buf[0]);
      rho = 1.0f / sqrtf(fmaf(ss, inv, a.eps));
      if (lane == 0) a.rstd_post[t] = rho;
    }
    const float gt = a.gate_mode == MHC_GATE_TOKEN ? static_cast<const float*>(a.gate)[t] : 1.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int g = lane + i * lanes;
      if (g < segs) {
        Vec8 w, c;
        if (a.gamma_post) w = unpack(ld8(static_cast<const T*>(a.gamma_post) + g * 8));
        if (a.gate_mode == MHC_GATE_CHANNEL) c = unpack(ld8(static_cast<const T*>(a.gate) + g * 8));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float q = p[i].v[e];
          if (a.gamma_post) q = q * rho * w.v[e];
          q *= a.gate_mode == MHC_GATE_CHANNEL ? c.v[e] : gt;
          x[i].v[e] = fmaf(a.scale, x[i].v[e], q);
        }
        st8_stream(static_cast<T*>(a.r_out) + t * a.ld_ro + g * 8, pack<T>(x[i]));
      }
    }
  }
  if (a.gamma_pre) {
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[i].v[e], x[i].v[e], ss);
    ss = team_sum<WARP>(ss, buf[1]);
    const float rho = 1.0f / sqrtf(fmaf(ss, inv, a.eps));
    if (lane == 0) a.rstd_pre[t] = rho;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int g = lane + i * lanes;
      if (g < segs) {
        const Vec8 w = unpack(ld8(static_cast<const T*>(a.gamma_pre) + g * 8));
        Vec8 n;
#pragma unroll
        for (int e = 0; e < 8; ++e) n.v[e] = x[i].v[e] * rho * w.v[e];
        st8_stream(static_cast<T*>(a.norm) + t * a.ld_n + g * 8, pack<T>(n));
      }
    }
  }
}

// With u = r' rho2 and c = gamma_pre dnorm:
//   G = dr_out + rho2 (c - u mean(c u)),  dgamma_pre += dnorm u,  dr = scale G
// and with u = y rho1, dp = gate G, c = gamma_post dp:
//   dy = rho1 (c - u mean(c u)),  dgamma_post += dp u,  dgate += u gamma_post G
// Bound by HBM: four rows read, two written.  A thread keeps the same columns
// over all of its CTA's rows, so the column sums stay in registers until the
// CTA's end; a second kernel adds the CTAs' sums in a fixed order.
template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 512) block_norm_grad_kernel(const BlockNormGradArgs a) {
  __shared__ float buf[2][3][16];
  const int lanes = WARP ? 32 : blockDim.x;
  const int lane = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int teams = WARP ? (blockDim.x >> 5) : 1, team = WARP ? (threadIdx.x >> 5) : 0;
  const int segs = a.H >> 3;
  const float inv = 1.0f / (float)a.H;
  float s_post[VPT][8] = {}, s_gate[VPT][8] = {}, s_pre[VPT][8] = {};
  int flip = 0;
  for (int64_t t = (int64_t)blockIdx.x * teams + team; t < a.T; t += (int64_t)gridDim.x * teams, flip ^= 1) {
    Vec8 G[VPT], u[VPT];
    const int64_t row = t * a.H;
    float m = 0.f;
    if (a.gamma_pre) {
      const float rho = a.rstd_pre[t];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int g = lane + i * lanes;
        G[i] = {};
        u[i] = {};
        if (g < segs) {
          u[i] = unpack(ld8_stream(static_cast<const T*>(a.r_out) + row + g * 8));
          const Vec8 dn = unpack(ld8_stream(static_cast<const T*>(a.dnorm) + row + g * 8));
          const Vec8 w = unpack(ld8(static_cast<const T*>(a.gamma_pre) + g * 8));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            u[i].v[e] *= rho;
            s_pre[i][e] = fmaf(dn.v[e], u[i].v[e], s_pre[i][e]);
            G[i].v[e] = w.v[e] * dn.v[e];
            m = fmaf(G[i].v[e], u[i].v[e], m);
          }
        }
      }
      m = team_sum<WARP>(m, buf[flip][0]) * inv;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) G[i].v[e] = rho * (G[i].v[e] - u[i].v[e] * m);
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) G[i] = {};
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int g = lane + i * lanes;
      if (g < segs) {
        if (a.dr_out) {
          const Vec8 d = unpack(ld8_stream(static_cast<const T*>(a.dr_out) + row + g * 8));
#pragma unroll
          for (int e = 0; e < 8; ++e) G[i].v[e] += d.v[e];
        }
        Vec8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = a.scale * G[i].v[e];
        st8_stream(static_cast<T*>(a.dr) + row + g * 8, pack<T>(o));
      }
    }
    if (!a.y) continue;
    const float rho = a.gamma_post ? a.rstd_post[t] : 1.f;
    const float gt = a.gate_mode == MHC_GATE_TOKEN ? static_cast<const float*>(a.gate)[t] : 1.f;
    float dg = 0.f;
    m = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int g = lane + i * lanes;
      u[i] = {};
      if (g < segs) {
        u[i] = unpack(ld8_stream(static_cast<const T*>(a.y) + row + g * 8));
        Vec8 w, c;
        if (a.gamma_post) w = unpack(ld8(static_cast<const T*>(a.gamma_post) + g * 8));
        if (a.gate_mode == MHC_GATE_CHANNEL) c = unpack(ld8(static_cast<const T*>(a.gate) + g * 8));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[i].v[e] *= rho;
          const float we = a.gamma_post ? w.v[e] : 1.f;
          const float pg = u[i].v[e] * we * G[i].v[e];
          dg += pg;
          s_gate[i][e] += pg;
          const float dp = (a.gate_mode == MHC_GATE_CHANNEL ? c.v[e] : gt) * G[i].v[e];
          s_post[i][e] = fmaf(dp, u[i].v[e], s_post[i][e]);
          G[i].v[e] = dp * we;
          m = fmaf(G[i].v[e], u[i].v[e], m);
        }
      }
    }
    if (a.gate_mode == MHC_GATE_TOKEN) {
      dg = team_sum<WARP>(dg, buf[flip][1]);
      if (lane == 0) a.dgate[t] = dg;
    }
    if (a.gamma_post) m = team_sum<WARP>(m, buf[flip][2]) * inv;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int g = lane + i * lanes;
      if (g < segs) {
        Vec8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = a.gamma_post ? rho * (G[i].v[e] - u[i].v[e] * m) : G[i].v[e];
        st8_stream(static_cast<T*>(a.dy) + row + g * 8, pack<T>(o));
      }
    }
  }
  float* out = a.parts + ((int64_t)blockIdx.x * teams + team) * 3 * a.H;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int g = lane + i * lanes;
    if (g < segs) {
      float* o = out + g * 8;
      if (a.dgamma_post) st8(o, pack<float>(*reinterpret_cast<Vec8*>(s_post[i])));
      if (a.gate_mode == MHC_GATE_CHANNEL) st8(o + a.H, pack<float>(*reinterpret_cast<Vec8*>(s_gate[i])));
      if (a.dgamma_pre) st8(o + 2 * a.H, pack<float>(*reinterpret_cast<Vec8*>(s_pre[i])));
    }
  }
}

// Adds the parts' column sums in part order: 32 columns x 8 slices of parts per
// CTA, the slices joined in slice order.
__global__ void __launch_bounds__(256) block_norm_fold_kernel(const float* __restrict__ parts, int n, int H, float* post,
                                                              float* gate, float* pre) {
  __shared__ float sh[8][33];
  pdl_wait();
  float* out = blockIdx.y == 0 ? post : blockIdx.y == 1 ? gate : pre;
  if (!out) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float x = 0.f;
  if (c < H) {
    const float* p = parts + (int64_t)blockIdx.y * H + c;
    const int lo = (int)((int64_t)n * w / 8), hi = (int)((int64_t)n * (w + 1) / 8);
#pragma unroll 4
    for (int i = lo; i < hi; ++i) x += p[(int64_t)i * 3 * H];
  }
  sh[w][threadIdx.x & 31] = x;
  __syncthreads();
  if (w == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < 8; ++i) x += sh[i][threadIdx.x];
    out[c] = x;
  }
}

// Teams: a warp per row up to 1024 columns, else a CTA per row.
struct TeamPlan {
  bool warp;
  int vpt, threads;
};
static TeamPlan team_plan(int H) {
  const int segs = H / 8;
  TeamPlan p;
  p.warp = segs <= 128;
  if (p.warp) {
    p.threads = 128;
    p.vpt = segs <= 32 ? 1 : segs <= 64 ? 2 : 4;
  } else {
    p.vpt = segs <= 512 ? 1 : segs <= 1024 ? 2 : 4;
    p.threads = ((segs + p.vpt - 1) / p.vpt + 31) / 32 * 32;
  }
  return p;
}

constexpr int kMaxParts = 304;  // column sums kept by the gradient: at most this many teams, two CTAs per SM of 152

static int grad_parts(int64_t T) { return (int)(T < kMaxParts ? T : kMaxParts); }

#define MHC_BY_TEAM(plan, ...)                                                            \
  if (plan.warp) {                                                                        \
    constexpr bool W = true;                                                              \
    if (plan.vpt == 1) { constexpr int N = 1; __VA_ARGS__; }                              \
    else if (plan.vpt == 2) { constexpr int N = 2; __VA_ARGS__; }                         \
    else { constexpr int N = 4; __VA_ARGS__; }                                            \
  } else {                                                                                \
    constexpr bool W = false;                                                             \
    if (plan.vpt == 1) { constexpr int N = 1; __VA_ARGS__; }                              \
    else if (plan.vpt == 2) { constexpr int N = 2; __VA_ARGS__; }                         \
    else { constexpr int N = 4; __VA_ARGS__; }                                            \
  }

constexpr int kMaxWidth = 16384;

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
  if (!r || (y && !r_out) || (gamma_pre && (!norm || !rstd_pre)) || (gamma_post && !rstd_post))
    return ops_fail(MHC_ERR_NULL, "a required pointer is NULL");
  if ((gate_mode != MHC_GATE_NONE) != (gate != nullptr))
    return ops_fail(MHC_ERR_NULL, "gate must be given exactly when gate_mode is not none");
  if (!y && (gamma_post || gate || !gamma_pre))
    return ops_fail(MHC_ERR_INCOMPLETE_POST, "without y the call is the norm before the first block: gamma_pre only");
  const int64_t lds[] = {y ? ld_y : H, ld_r, y ? ld_r_out : H, gamma_pre ? ld_norm : H};
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
      if (!(o == 0 && i == 1 && r_out == r && ld_r_out == ld_r) && rows_overlap(out[o], in[i]))
        return ops_fail(MHC_ERR_ALIAS, "an output overlaps an input");
    for (int q = o + 1; q < 4; ++q)
      if (rows_overlap(out[o], out[q])) return ops_fail(MHC_ERR_ALIAS, "two outputs overlap");
  }
  const BlockNormArgs a = {y, r, gamma_post, gate, gamma_pre, ld_y, ld_r, ld_r_out, ld_norm, gate_mode, res_scale, eps,
                           T, H, r_out, norm, rstd_post, rstd_pre};
  const TeamPlan plan = team_plan(H);
  const unsigned grid = (unsigned)(plan.warp ? (T + 3) / 4 : T);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  MHC_BY_DTYPE(dtype, E, { MHC_BY_TEAM(plan, { block_norm_kernel<E, N, W><<<grid, plan.threads, 0, s>>>(a); }) });
  return ops_cuda(cudaGetLastError(), "block_norm launch");
}

size_t mhc_block_norm_grad_workspace_bytes(int64_t T, int H) {
  if (T <= 0 || H <= 0) return 0;
  return (size_t)mhc::grad_parts(T) * 3 * H * sizeof(float) + 3 * (size_t)H * 4 * sizeof(float);
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
  if ((!dr_out && !gamma_pre) || !dr || (y && !dy) || (gamma_pre && (!dnorm || !r_out || !rstd_pre)) ||
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
  const BlockNormGradArgs a = {dr_out, dnorm, y, r_out, gamma_post, gate, gamma_pre, rstd_post, rstd_pre, gate_mode,
                               res_scale, T, H, dy, dr, dgamma_post, dgate, dgamma_pre, static_cast<float*>(workspace)};
  const TeamPlan plan = team_plan(H);
  int parts = grad_parts(T);
  unsigned grid = (unsigned)parts;
  if (plan.warp) {
    grid = (unsigned)((parts + 3) / 4);
    parts = (int)grid * 4;
  }
  MHC_BY_DTYPE(dtype, E, { MHC_BY_TEAM(plan, { block_norm_grad_kernel<E, N, W><<<grid, plan.threads, 0, s>>>(a); }) });
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && (dgamma_post || dgamma_pre || channel))
    e = launch_pdl(block_norm_fold_kernel, dim3((H + 31) / 32, 3), dim3(256), 0, s, a.parts, parts, H, dgamma_post,
                   channel ? dgate : nullptr, dgamma_pre);
  return ops_cuda(e, "block_norm_grad launch");
}

}  // extern "C"
