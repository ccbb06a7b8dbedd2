// The norms after and before a block, fused with its gate and residual
// scale and the next block's modulation, and their gradient.
//
//   y = res_scale x + gate (N(h) post_gamma)
//   z = (N(y) pre_gamma + pre_beta) (1 + scale) + shift
// with N the identity, (v - mean) r or v r, r = 1 / sqrt(mean square + eps).
// Gradient, with n = N(y), m = N(h) and g the gradient of a norm's output:
//   dN(g; v) = r (g - mean(g) - n mean(g n))       (no mean(g) without mean)
//   t = dy + dN(dz (1 + scale) pre_gamma; y),  dx = res_scale t
//   dh = dN(t gate post_gamma; h)
// and three column sums per condition row carry every reduced gradient:
//   S0 = sum dz, S1 = sum dz n, P = sum t m
//   dshift = S0, dscale = pre_gamma S1 + pre_beta S0, dgate = post_gamma P,
//   dpre_gamma = sum_b (1 + scale_b) S1_b, dpre_beta = sum_b (1 + scale_b) S0_b,
//   dpost_gamma = sum_b gate_b P_b.
//
// Bound by HBM: each row is read and written once and stays in registers
// between the statistics, so a CTA takes whole rows (a thread owns 8 NV
// columns) and R rows at a time, which puts R loads per operand in flight
// and shares one block reduction between R rows. Variances are sums of
// squares of centred values (two reductions), not differences of moments:
// with a mean of 100 standard deviations the latter would lose 4 digits.
// Everything between the loads and the stores is fp32.
#include "backward.h"

namespace moe {
namespace {

constexpr int kMaxWarps = 16;

// Block-wide sums of K <= KM values, the same in every thread. The two
// buffers are used in turn: a thread can be at most one barrier ahead, so
// the buffer it writes is no longer being read.
template <int KM> struct Reducer {
  float *buf;  // [2][kMaxWarps * KM]
  int turn;
};
template <int K, int KM>
__device__ __forceinline__ void block_sum(float (&v)[K], Reducer<KM> &red) {
  static_assert(K <= KM, "");
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *b = red.buf + red.turn * kMaxWarps * KM;
  red.turn ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) b[warp * K + k] = v[k];
  }
  __syncthreads();
  float t = 0.f;
  if (lane < K)
    for (int w = 0; w < nw; ++w) t += b[w * K + lane];
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, t, k);
}

template <typename T>
__device__ __forceinline__ void load_or(const T *p, size_t i, bool live, float fill, float (&f)[8]) {
  if (p && live) {
    load8(p + i, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = fill;
  }
}

// Normalises R rows of fp32 columns in place: v becomes N(v), r its scale.
template <int NV, int R, int KM>
__device__ __forceinline__ void norm_rows(float (&v)[R][NV][8], float (&r)[R], int kind, float eps, int d,
                                          const bool (&col)[NV], Reducer<KM> &red) {
  const float inv_d = 1.0f / (float)d;
  if (kind == MOE_NORM_LAYER) {
    float s[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i] += v[i][q][j];
    }
    block_sum(s, red);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][q][j] = col[q] ? v[i][q][j] - s[i] * inv_d : 0.f;
  }
  float s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    s[i] = 0.f;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i] = fmaf(v[i][q][j], v[i][q][j], s[i]);
  }
  block_sum(s, red);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    r[i] = 1.0f / sqrtf(fmaf(s[i], inv_d, eps));
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][q][j] *= r[i];
  }
}

// g becomes dN(g; v) for n = N(v) with scale r.
template <int NV, int R, int KM>
__device__ __forceinline__ void norm_grad_rows(float (&g)[R][NV][8], const float (&n)[R][NV][8], const float (&r)[R],
                                               int kind, int d, Reducer<KM> &red) {
  const float inv_d = 1.0f / (float)d;
  float s[2 * R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    s[2 * i] = s[2 * i + 1] = 0.f;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[2 * i] += g[i][q][j];
        s[2 * i + 1] = fmaf(g[i][q][j], n[i][q][j], s[2 * i + 1]);
      }
  }
  block_sum(s, red);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float mg = kind == MOE_NORM_LAYER ? s[2 * i] * inv_d : 0.f, mn = s[2 * i + 1] * inv_d;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][q][j] = r[i] * (g[i][q][j] - mg - n[i][q][j] * mn);
  }
}

template <typename T, int NV, int R>
__global__ void __launch_bounds__(512) block_norm_kernel(BlockNormArgs a) {
  __shared__ float red_buf[2 * kMaxWarps * R];
  const T *h = static_cast<const T *>(a.h), *x = static_cast<const T *>(a.x);  // either may be y
  const T *gate = static_cast<const T *>(a.gate), *scale = static_cast<const T *>(a.scale),
          *shift = static_cast<const T *>(a.shift);
  T *y = static_cast<T *>(a.y), *z = static_cast<T *>(a.z);
  Reducer<R> red{red_buf, 0};
  size_t c[NV];
  bool col[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    c[q] = ((size_t)q * blockDim.x + threadIdx.x) * 8;
    col[q] = c[q] < (size_t)a.d;
  }
  for (int64_t s0 = (int64_t)blockIdx.x * R; s0 < a.T; s0 += (int64_t)gridDim.x * R) {
    float u[R][NV][8], xr[R][NV][8], r[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const bool live = col[q] && s0 + i < a.T;
        load_or(h, (size_t)(s0 + i) * a.d + c[q], live, 0.f, u[i][q]);
        load_or(x, (size_t)(s0 + i) * a.d + c[q], live, 0.f, xr[i][q]);
      }
    if (a.post != MOE_NORM_NONE && h) norm_rows(u, r, a.post, a.eps, a.d, col, red);
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      float pg[8];
      load_or(static_cast<const T *>(a.post_gamma), c[q], col[q], 1.f, pg);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool live = col[q] && s0 + i < a.T;
        float gt[8];
        load_or(gate, (size_t)((s0 + i) / a.group) * a.cond_stride + c[q], live, 1.f, gt);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][q][j] = fmaf(a.res_scale, xr[i][q][j], gt[j] * (u[i][q][j] * pg[j]));
        if (y && live) store8(y + (size_t)(s0 + i) * a.d + c[q], u[i][q]);
      }
    }
    if (!z) continue;
    norm_rows(u, r, a.pre, a.eps, a.d, col, red);
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      float pg[8], pb[8];
      load_or(static_cast<const T *>(a.pre_gamma), c[q], col[q], 1.f, pg);
      load_or(static_cast<const T *>(a.pre_beta), c[q], col[q], 0.f, pb);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (!(col[q] && s0 + i < a.T)) continue;
        const size_t at = (size_t)((s0 + i) / a.group) * a.cond_stride + c[q];
        float sc[8], sh[8];
        load_or(scale, at, true, 0.f, sc);
        load_or(shift, at, true, 0.f, sh);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          u[i][q][j] = fmaf(fmaf(u[i][q][j], pg[j], pb[j]), 1.0f + sc[j], sh[j]);
        store8(z + (size_t)(s0 + i) * a.d + c[q], u[i][q]);
      }
    }
  }
}

// The rows are cut into segments of seg_len consecutive tokens of one
// condition row (per_group segments each), a contiguous range of segments to
// a CTA. A segment that is its whole group writes that row's condition
// gradients itself; otherwise its sums go to part [segment][3][d]. The CTA's
// sums for the weights go to wpart [cta][3][d] when they are wanted. A second
// launch adds both up in order.
struct NormBwdPlan {
  int group, per_group, seg_len, grid;
  int64_t groups, segments;
};
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kBwdCtas = 148 * 4;

// `conds`: rows of one group share conditions, so they belong together; else
// the whole input is one group. `rows`: tokens a CTA takes at a time.
NormBwdPlan norm_bwd_plan(int T, int group, bool conds, int rows) {
  NormBwdPlan p;
  p.group = conds && group < T ? group : (T > 0 ? T : 1);
  p.groups = ceil_div(T, p.group);
  const int64_t want = ceil_div(ceil_div(T > 0 ? T : 1, kBwdCtas), rows) * rows;
  p.per_group = (int)ceil_div(p.group, want);
  p.seg_len = (int)(ceil_div(ceil_div(p.group, p.per_group), rows) * rows);
  p.per_group = (int)ceil_div(p.group, p.seg_len);
  p.segments = p.groups * p.per_group;
  p.grid = (int)(p.segments < kBwdCtas ? p.segments : kBwdCtas);
  return p;
}

template <typename T, int NV, int R>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(BlockNormArgs a, NormBwdPlan p, float *part,
                                                             float *wpart) {
  __shared__ float red_buf[2 * kMaxWarps * 2 * R];
  const T *h = static_cast<const T *>(a.h), *y = static_cast<const T *>(a.yin);
  const T *dz = static_cast<const T *>(a.dz), *dy = static_cast<const T *>(a.dy);  // either may be dh or dx
  const T *gate = static_cast<const T *>(a.gate), *scale = static_cast<const T *>(a.scale);
  const T *post_gamma = static_cast<const T *>(a.post_gamma), *pre_gamma = static_cast<const T *>(a.pre_gamma),
          *pre_beta = static_cast<const T *>(a.pre_beta);
  T *dh = static_cast<T *>(a.dh), *dx = static_cast<T *>(a.dx);
  const bool want_h = dh || a.dgate || a.dpost_gamma;
  Reducer<2 * R> red{red_buf, 0};
  size_t c[NV];
  bool col[NV];
  float G1[NV][8], B1[NV][8], GP[NV][8];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    c[q] = ((size_t)q * blockDim.x + threadIdx.x) * 8;
    col[q] = c[q] < (size_t)a.d;
#pragma unroll
    for (int j = 0; j < 8; ++j) G1[q][j] = B1[q][j] = GP[q][j] = 0.f;
  }
  const int64_t g_lo = p.segments * blockIdx.x / p.grid, g_hi = p.segments * (blockIdx.x + 1) / p.grid;
  for (int64_t seg = g_lo; seg < g_hi; ++seg) {
    const int64_t b = seg / p.per_group;
    const int64_t t_lo = b * p.group + (seg - b * p.per_group) * p.seg_len;
    int64_t t_hi = t_lo + p.seg_len;
    if (t_hi > (b + 1) * p.group) t_hi = (b + 1) * p.group;
    if (t_hi > a.T) t_hi = a.T;
    const size_t cond = (size_t)b * a.cond_stride;
    float S0[NV][8], S1[NV][8], P[NV][8], gz[NV][8], gh[NV][8];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      float f[8];
      load_or(scale, cond + c[q], col[q], 0.f, f);
      load_or(pre_gamma, c[q], col[q], 1.f, gz[q]);
#pragma unroll
      for (int j = 0; j < 8; ++j) gz[q][j] *= 1.0f + f[j];
      load_or(gate, cond + c[q], col[q], 1.f, f);
      load_or(post_gamma, c[q], col[q], 1.f, gh[q]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gh[q][j] = col[q] ? gh[q][j] * f[j] : 0.f;  // no column past d enters the post norm's means
        S0[q][j] = S1[q][j] = P[q][j] = 0.f;
      }
    }
    for (int64_t s0 = t_lo; s0 < t_hi; s0 += R) {
      float t[R][NV][8], m[R][NV][8], r[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int q = 0; q < NV; ++q) {
          const bool live = col[q] && s0 + i < t_hi;
          load_or(dy, (size_t)(s0 + i) * a.d + c[q], live, 0.f, t[i][q]);
          load_or(want_h ? h : nullptr, (size_t)(s0 + i) * a.d + c[q], live, 0.f, m[i][q]);
        }
      if (dz) {
        float g[R][NV][8], n[R][NV][8];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int q = 0; q < NV; ++q) {
            const bool live = col[q] && s0 + i < t_hi;
            load_or(y, (size_t)(s0 + i) * a.d + c[q], live, 0.f, n[i][q]);
            load_or(dz, (size_t)(s0 + i) * a.d + c[q], live, 0.f, g[i][q]);
          }
        norm_rows(n, r, a.pre, a.eps, a.d, col, red);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              S0[q][j] += g[i][q][j];
              S1[q][j] = fmaf(g[i][q][j], n[i][q][j], S1[q][j]);
              g[i][q][j] *= gz[q][j];
            }
        norm_grad_rows(g, n, r, a.pre, a.d, red);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) t[i][q][j] += g[i][q][j];
      }
      if (dx) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int q = 0; q < NV; ++q)
            if (col[q] && s0 + i < t_hi) {
              float o[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] = a.res_scale * t[i][q][j];
              store8(dx + (size_t)(s0 + i) * a.d + c[q], o);
            }
      }
      if (!want_h) continue;
      if (a.post != MOE_NORM_NONE) norm_rows(m, r, a.post, a.eps, a.d, col, red);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            P[q][j] = fmaf(t[i][q][j], m[i][q][j], P[q][j]);
            t[i][q][j] *= gh[q][j];
          }
      if (!dh) continue;
      if (a.post != MOE_NORM_NONE) norm_grad_rows(t, m, r, a.post, a.d, red);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int q = 0; q < NV; ++q)
          if (col[q] && s0 + i < t_hi) store8(dh + (size_t)(s0 + i) * a.d + c[q], t[i][q]);
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      if (!col[q]) continue;
      if (wpart) {
        float f[8];
        load_or(scale, cond + c[q], true, 0.f, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          G1[q][j] = fmaf(1.0f + f[j], S1[q][j], G1[q][j]);
          B1[q][j] = fmaf(1.0f + f[j], S0[q][j], B1[q][j]);
        }
        load_or(gate, cond + c[q], true, 1.f, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) GP[q][j] = fmaf(f[j], P[q][j], GP[q][j]);
      }
      if (part) {
        float *o = part + (size_t)seg * 3 * a.d + c[q];
        store8(o, S0[q]);
        store8(o + a.d, S1[q]);
        store8(o + 2 * (size_t)a.d, P[q]);
      } else {
        const size_t at = (size_t)b * a.dcond_stride + c[q];
        float f[8], o[8];
        if (a.dshift) store8(a.dshift + at, S0[q]);
        if (a.dscale) {
          load_or(pre_gamma, c[q], true, 1.f, f);
          load_or(pre_beta, c[q], true, 0.f, o);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = fmaf(f[j], S1[q][j], o[j] * S0[q][j]);
          store8(a.dscale + at, o);
        }
        if (a.dgate) {
          load_or(post_gamma, c[q], true, 1.f, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = f[j] * P[q][j];
          store8(a.dgate + at, o);
        }
      }
    }
  }
  if (!wpart) return;
#pragma unroll
  for (int q = 0; q < NV; ++q)
    if (col[q]) {
      float *o = wpart + (size_t)blockIdx.x * 3 * a.d + c[q];
      store8(o, G1[q]);
      store8(o + a.d, B1[q]);
      store8(o + 2 * (size_t)a.d, GP[q]);
    }
}

// Sums the partial blocks in order: blockIdx.y < groups adds a group's
// segments into its condition gradients, the next one the CTAs' sums into
// the weights' gradients. 32 columns by 8 slices of the list per CTA.
template <typename T>
__global__ void __launch_bounds__(256) block_norm_sum_kernel(BlockNormArgs a, const float *part, const float *wpart,
                                                             int64_t first_task, int64_t groups, int per_group,
                                                             int ctas) {
  __shared__ float sh[3][8][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t task = first_task + blockIdx.y;
  const bool cond = part && task < groups;
  const float *src = cond ? part + (size_t)task * per_group * 3 * a.d : wpart;
  const int n = cond ? per_group : ctas;
  const int col = blockIdx.x * 32 + lane;
  float v[3] = {0.f, 0.f, 0.f};
  if (col < a.d) {
    const int lo = (int)((int64_t)n * slice / 8), hi = (int)((int64_t)n * (slice + 1) / 8);
#pragma unroll 4
    for (int k = lo; k < hi; ++k)
#pragma unroll
      for (int w = 0; w < 3; ++w) v[w] += src[((size_t)k * 3 + w) * a.d + col];
  }
#pragma unroll
  for (int w = 0; w < 3; ++w) sh[w][slice][lane] = v[w];
  __syncthreads();
  if (slice != 0 || col >= a.d) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    v[w] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[w] += sh[w][k][lane];
  }
  if (cond) {
    const size_t at = (size_t)task * a.dcond_stride + col;
    const T *pg = static_cast<const T *>(a.pre_gamma), *pb = static_cast<const T *>(a.pre_beta),
            *po = static_cast<const T *>(a.post_gamma);
    if (a.dshift) a.dshift[at] = v[0];
    if (a.dscale) a.dscale[at] = fmaf(pg ? to_f32(pg[col]) : 1.f, v[1], pb ? to_f32(pb[col]) * v[0] : 0.f);
    if (a.dgate) a.dgate[at] = (po ? to_f32(po[col]) : 1.f) * v[2];
  } else {
    if (a.dpre_gamma) a.dpre_gamma[col] = v[0];
    if (a.dpre_beta) a.dpre_beta[col] = v[1];
    if (a.dpost_gamma) a.dpost_gamma[col] = v[2];
  }
}

// Threads of a CTA whose threads own nv vectors of 8 columns each.
int row_threads(int d, int nv) {
  const int vecs = d / 8;
  return ((vecs + nv - 1) / nv + 31) / 32 * 32;
}
// Up to 4096 columns a thread owns 8 of them (at most 512 threads); wider
// rows take 2 vectors per thread and one row at a time (the backward spills
// there: 12 arrays of 16 columns do not fit 128 registers).
inline bool narrow(int d) { return d <= 4096; }
constexpr int kFwdRows = 2, kBwdRows = 2;

template <typename T>
int run_fwd(const BlockNormArgs &a, cudaStream_t stream) {
  const int64_t sms = num_sms();
  if (!narrow(a.d)) {
    const int64_t grid = a.T < 4 * sms ? a.T : 4 * sms;
    block_norm_kernel<T, 2, 1><<<(unsigned)grid, row_threads(a.d, 2), 0, stream>>>(a);
  } else if (a.T <= 2 * sms) {  // few tokens: a CTA each
    block_norm_kernel<T, 1, 1><<<a.T, row_threads(a.d, 1), 0, stream>>>(a);
  } else {
    const int64_t tiles = (a.T + kFwdRows - 1) / kFwdRows, cap = 16 * sms;
    block_norm_kernel<T, 1, kFwdRows><<<(unsigned)(tiles < cap ? tiles : cap), row_threads(a.d, 1), 0, stream>>>(a);
  }
  return last_launch_status();
}

template <typename T>
int run_bwd(const BlockNormArgs &a, cudaStream_t stream) {
  const bool conds = a.gate || a.scale || a.dgate || a.dscale || a.dshift;
  const int rows = narrow(a.d) && a.group >= kBwdRows ? kBwdRows : 1;
  const NormBwdPlan p = norm_bwd_plan(a.T, a.group, conds, rows);
  const bool cond_out = a.dgate || a.dscale || a.dshift;
  float *part = cond_out && p.per_group > 1 ? a.part : nullptr;
  float *wpart = a.dpre_gamma || a.dpre_beta || a.dpost_gamma
                     ? a.part + (part ? (size_t)p.segments * 3 * a.d : 0) : nullptr;
  if (a.T > 0) {
    if (!narrow(a.d))
      block_norm_bwd_kernel<T, 2, 1><<<p.grid, row_threads(a.d, 2), 0, stream>>>(a, p, part, wpart);
    else if (rows == 1)
      block_norm_bwd_kernel<T, 1, 1><<<p.grid, row_threads(a.d, 1), 0, stream>>>(a, p, part, wpart);
    else
      block_norm_bwd_kernel<T, 1, kBwdRows><<<p.grid, row_threads(a.d, 1), 0, stream>>>(a, p, part, wpart);
  }
  const int64_t first = part ? 0 : p.groups, last = p.groups + (wpart ? 1 : 0);
  for (int64_t t = first; t < last; t += 65535) {
    const unsigned n = (unsigned)(last - t < 65535 ? last - t : 65535);
    block_norm_sum_kernel<T><<<dim3((a.d + 31) / 32, n), 256, 0, stream>>>(a, part, wpart, t, p.groups, p.per_group,
                                                                          a.T > 0 ? p.grid : 0);
  }
  return last_launch_status();
}

}  // namespace

// Partial sums of every way the backward can cut the rows.
size_t block_norm_workspace_bytes(int T, int d, int group) {
  int64_t most = 0;
  for (int rows = 1; rows <= kBwdRows; rows += kBwdRows - 1)
    for (int conds = 0; conds < 2; ++conds) {
      const NormBwdPlan p = norm_bwd_plan(T, group, conds != 0, rows);
      const int64_t n = (p.per_group > 1 ? p.segments : 0) + p.grid;
      if (n > most) most = n;
    }
  return (size_t)most * 3 * d * 4;
}

int launch_block_norm(const BlockNormArgs &a, int dtype, cudaStream_t stream) {
  if (a.T == 0) return MOE_OK;
  return dtype == MOE_BF16 ? run_fwd<__nv_bfloat16>(a, stream) : run_fwd<float>(a, stream);
}

int launch_block_norm_bwd(const BlockNormArgs &a, int dtype, cudaStream_t stream) {
  return dtype == MOE_BF16 ? run_bwd<__nv_bfloat16>(a, stream) : run_bwd<float>(a, stream);
}

}  // namespace moe
