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
// Bound by HBM, and close behind it by instruction issue: each row is read
// and written once and stays in registers between the statistics. A CTA takes
// whole rows, a thread 8 columns of them (16-byte accesses), and several rows
// at a time, whose block reductions share their barriers; the factors and the
// column sums of a thread's columns stay in its registers over all rows of a
// condition row. A warp per row needs no barriers, but a lane then holds 36
// and more columns: too few warps fit an SM to hide their latencies
// (8192 x 1152, LayerNorm: forward 24 us, backward 50-55 us, against 16 and
// 25 + 4.5 here; elementwise kernels over as many bytes take 12.9 and 18.4).
// That is bf16; fp32 rows of the same width have rings twice as large, which
// leave 2 CTAs an SM forward and 1 backward instead of the planned 4 and 3.
// Variances are sums of squares of centred values (two reductions), not
// differences of moments: with a mean of 100 standard deviations the latter
// would lose 4 digits. Everything between the loads and the stores is fp32,
// most of it on packed pairs.
#include "backward.h"
#include "chained.cuh"

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
        load_or(gate, (size_t)((uint32_t)(s0 + i) / (uint32_t)a.group) * a.cond_stride + c[q], live, 1.f, gt);
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
        const size_t at = (size_t)((uint32_t)(s0 + i) / (uint32_t)a.group) * a.cond_stride + c[q];
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
// a CTA.
struct NormPlan {
  int group, per_group, seg_len, grid;
  int64_t groups, segments;
};
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// `conds`: rows of one group share conditions, so they belong together; else
// the whole input is one group. `rows`: tokens a CTA takes at a time, `ctas`:
// those that run at once. With fewer groups than CTAs each group is cut into
// as many segments as still run at once.
NormPlan norm_plan(int T, int group, bool conds, int rows, int ctas) {
  NormPlan p;
  p.group = conds && group < T ? group : (T > 0 ? T : 1);
  p.groups = ceil_div(T, p.group);
  const int64_t cut = p.groups > 0 && p.groups < ctas ? ctas / p.groups : 1;
  p.seg_len = (int)(ceil_div(ceil_div(p.group, cut), rows) * rows);
  p.per_group = (int)ceil_div(p.group, p.seg_len);
  p.segments = p.groups * p.per_group;
  p.grid = (int)(p.segments < ctas ? p.segments : ctas);
  return p;
}
struct Segment {
  int64_t group;
  int lo, hi;  // tokens
};
__device__ __forceinline__ Segment segment_of(const NormPlan &p, int64_t seg, int T) {
  Segment s;
  s.group = seg / p.per_group;
  const int64_t lo = s.group * p.group + (seg - s.group * p.per_group) * p.seg_len;
  int64_t hi = lo + p.seg_len;
  if (hi > (s.group + 1) * p.group) hi = (s.group + 1) * p.group;
  if (hi > T) hi = T;
  s.lo = (int)(lo < T ? lo : T);
  s.hi = (int)hi;
  return s;
}

// ---- many rows of up to 4096 columns: a thread owns 8 of them
//
// 8 fp32 columns as packed pairs.
struct V8 {
  uint64_t v[4];
  __device__ __forceinline__ void fill(float f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_splat(f);
  }
};
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float f2_sum(uint64_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ V8 unpack_v8(const __nv_bfloat16 *p) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // a bf16 is the upper half of its fp32
    r.v[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return r;
}
__device__ __forceinline__ V8 unpack_v8(const float *p) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  V8 r;
  r.v[0] = f2_pack(a.x, a.y);
  r.v[1] = f2_pack(a.z, a.w);
  r.v[2] = f2_pack(b.x, b.y);
  r.v[3] = f2_pack(b.z, b.w);
  return r;
}
// This thread's 8 columns of rows on their way: a ring of DEPTH steps of N
// vectors (rows by operands) in shared memory, filled by cp.async DEPTH - 1
// steps ahead. A thread reads only what it copied, so no barrier is involved.
template <typename T, int N, int DEPTH> struct Fetch {
  T *mine;  // [DEPTH][N][blockDim.x][8], this thread's part
  int slot;
  __device__ __forceinline__ T *at(int step, int k) const {
    return mine + (size_t)(step * N + k) * blockDim.x * 8;
  }
  // Vector k of a step; zeros unless `live`. The memory clobbers here and in
  // wait() keep the reads of the ring on their side of the copies.
  __device__ __forceinline__ void issue(int step, int k, const T *p, bool live) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; i += PER)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       static_cast<uint32_t>(__cvta_generic_to_shared(at(step, k) + i))),
                   "l"(live ? p + i : p), "r"(live ? 16 : 0)
                   : "memory");
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // Until all but the last `later` steps have arrived.
  template <int later> __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(later) : "memory");
  }
  __device__ __forceinline__ void next() { slot = slot == DEPTH - 1 ? 0 : slot + 1; }
  __device__ __forceinline__ int last() const { return slot == 0 ? DEPTH - 1 : slot - 1; }
  __device__ __forceinline__ V8 get(int k) const { return unpack_v8(at(slot, k)); }
};
template <typename T, int N, int DEPTH> size_t fetch_bytes(int threads) {
  return (size_t)DEPTH * N * threads * 8 * sizeof(T);
}
template <typename T>
__device__ __forceinline__ void store_v8(T *p, const V8 &a) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(a.v[i], f[2 * i], f[2 * i + 1]);
  store8(p, f);
}
__device__ __forceinline__ float sum_v8(const V8 &a) {
  return f2_sum(f2_add(f2_add(a.v[0], a.v[1]), f2_add(a.v[2], a.v[3])));
}
__device__ __forceinline__ float dot_v8(const V8 &a, const V8 &b) {
  uint64_t s = f2_mul(a.v[0], b.v[0]), t = f2_mul(a.v[1], b.v[1]);
  s = f2_fma(a.v[2], b.v[2], s);
  t = f2_fma(a.v[3], b.v[3], t);
  return f2_sum(f2_add(s, t));
}
// `f` past the row's end (no thread's columns cross it: d is a multiple of 8).
template <typename T>
__device__ __forceinline__ V8 load_v8_or(const T *p, size_t i, bool live, float f) {
  if (p && live) return unpack_v8(p + i);
  V8 r;
  r.fill(f);
  return r;
}

// Block-wide sums of K = 4 or 8 values, the same in every thread. Halving
// exchanges leave each lane one value to finish (9 shuffles for 8 values
// instead of 40). `buf` holds two buffers used in turn, as above.
constexpr int kVecWarps = 16;
struct VecReducer {
  float *buf;  // [2][kVecWarps][8]
  int turn;
};
template <int K>
__device__ __forceinline__ void block_sum_vec(float (&v)[K], VecReducer &red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float k[K];
#pragma unroll
  for (int i = 0; i < K; ++i) k[i] = v[i];
  int idx = 0;
#pragma unroll
  for (int n = K / 2, o = 16; n >= 1; n /= 2, o /= 2) {
    const bool up = (lane & o) != 0;  // this lane keeps the upper half of the values
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? k[i] : k[i + n], keep = up ? k[i + n] : k[i];
      k[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
    idx = 2 * idx + (up ? 1 : 0);
  }
  constexpr int kRest = 32 / K;  // lanes that share a value
#pragma unroll
  for (int o = kRest / 2; o > 0; o >>= 1) k[0] += __shfl_xor_sync(0xffffffffu, k[0], o);
  float *b = red.buf + red.turn * kVecWarps * 8;
  red.turn ^= 1;
  if ((lane & (kRest - 1)) == 0) b[warp * K + idx] = k[0];
  __syncthreads();
  // Lane l adds up value l mod K over every 32 / K-th warp.
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kVecWarps * K; i += 32)
    if (i + lane < nw * K) t += b[i + lane];
#pragma unroll
  for (int o = K; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = __shfl_sync(0xffffffffu, t, i);
}

// A segment's conditions and weights are folded into three factors per
// column, fg = gate post_gamma, fs = (1 + scale) pre_gamma, fb = (1 + scale)
// pre_beta + shift: y = res_scale x + fg N(h), z = fs N(y) + fb.
constexpr int kFwdRows = 4, kFwdDepth = 2;
// CTAs per SM of the kernels for many rows, with at most MAXT threads (at
// 1152 columns the forward gains from a fourth, 16.8 -> 15.9 us; the backward
// would spill for it).
constexpr int fwd_ctas(int maxt) { return maxt <= 160 ? 4 : maxt <= 256 ? 2 : 1; }
constexpr int bwd_ctas(int maxt) { return maxt <= 160 ? 3 : maxt <= 256 ? 2 : 1; }
template <typename T, int MAXT>
__global__ void __launch_bounds__(MAXT, fwd_ctas(MAXT)) block_norm_vec_kernel(BlockNormArgs a, NormPlan p) {
  constexpr int R = kFwdRows;
  __shared__ __align__(16) float red_buf[2 * kVecWarps * 8];
  extern __shared__ __align__(16) uint8_t ring[];
  VecReducer red{red_buf, 0};
  Fetch<T, 2 * R, kFwdDepth> rows{reinterpret_cast<T *>(ring) + threadIdx.x * 8, 0};
  const T *h = static_cast<const T *>(a.h), *x = static_cast<const T *>(a.x);  // either may be y
  T *y = static_cast<T *>(a.y), *z = static_cast<T *>(a.z);
  const int c = threadIdx.x * 8;
  const bool col = c < a.d;
  const float inv_d = 1.0f / (float)a.d;
  const uint64_t alpha = f2_splat(a.res_scale);
  const int64_t g_lo = p.segments * blockIdx.x / p.grid, g_hi = p.segments * (blockIdx.x + 1) / p.grid;
  // v less its mean, and the rows' scales; columns past d stay 0.
  auto centre = [&](V8 (&v)[R], float (&r)[R], int kind) {
    float s[R];
    if (kind == MOE_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < R; ++i) s[i] = sum_v8(v[i]);
      block_sum_vec(s, red);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint64_t m = f2_splat(col ? -s[i] * inv_d : 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i].v[j] = f2_add(v[i].v[j], m);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = dot_v8(v[i], v[i]);
    block_sum_vec(s, red);
#pragma unroll
    for (int i = 0; i < R; ++i) r[i] = rsqrtf(fmaf(s[i], inv_d, a.eps));
  };
  for (int64_t seg = g_lo; seg < g_hi; ++seg) {
    const Segment sg = segment_of(p, seg, a.T);
    // Rows s0 .. s0 + R - 1 of h and x into a step of the ring.
    auto fetch = [&](int s0, int step) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool live = col && s0 + i < sg.hi;
        const size_t at = (size_t)(s0 + i) * a.d + c;
        rows.issue(step, 2 * i, h ? h + at : x, live && h);
        rows.issue(step, 2 * i + 1, x ? x + at : h, live && x);
      }
      rows.commit();
    };
    rows.template wait<0>();  // the last segment's copies past its end
    rows.slot = 0;
#pragma unroll
    for (int k = 0; k < kFwdDepth - 1; ++k) fetch(sg.lo + k * R, k);
    const size_t cond = (size_t)sg.group * a.cond_stride + c;
    V8 fg = load_v8_or(static_cast<const T *>(a.gate), cond, col, 1.f);
    V8 fs = load_v8_or(static_cast<const T *>(a.scale), cond, col, 0.f);
    V8 fb = load_v8_or(static_cast<const T *>(a.shift), cond, col, 0.f);
    {
      const V8 po = load_v8_or(static_cast<const T *>(a.post_gamma), c, col, 1.f);
      const V8 pg = load_v8_or(static_cast<const T *>(a.pre_gamma), c, col, 1.f);
      const V8 pb = load_v8_or(static_cast<const T *>(a.pre_beta), c, col, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t s1 = f2_add(fs.v[j], f2_splat(1.f));
        fg.v[j] = f2_mul(fg.v[j], po.v[j]);
        fb.v[j] = f2_fma(s1, pb.v[j], fb.v[j]);
        fs.v[j] = f2_mul(s1, pg.v[j]);
      }
    }
    for (int s0 = sg.lo; s0 < sg.hi; s0 += R) {
      fetch(s0 + (kFwdDepth - 1) * R, rows.last());
      rows.template wait<kFwdDepth - 1>();
      V8 u[R];
      float r[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        u[i] = rows.get(2 * i);
        r[i] = 1.f;
      }
      if (h && a.post != MOE_NORM_NONE) centre(u, r, a.post);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint64_t rr = f2_splat(r[i]);
        const V8 xv = rows.get(2 * i + 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t t = f2_mul(f2_mul(u[i].v[j], rr), fg.v[j]);
          u[i].v[j] = f2_fma(alpha, xv.v[j], t);
        }
        if (y && col && s0 + i < sg.hi) store_v8(y + (size_t)(s0 + i) * a.d + c, u[i]);
      }
      rows.next();
      if (!z) continue;
      centre(u, r, a.pre);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (!(col && s0 + i < sg.hi)) continue;
        const uint64_t rr = f2_splat(r[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) u[i].v[j] = f2_fma(f2_mul(u[i].v[j], rr), fs.v[j], fb.v[j]);
        store_v8(z + (size_t)(s0 + i) * a.d + c, u[i]);
      }
    }
  }
}

// The gradient, two rows at a time. With yc = y - mean(y), n = r yc and
// g = dz (1 + scale) pre_gamma:
//   t = dy + r (g - mean(g)) - r^3 mean(g yc) yc
// so that mean(y) and mean(g), then mean(yc^2) and mean(g yc), and the same
// of h, each take one reduction. Sums of a segment as in the other kernels;
// the CTA's sums for the weights are kept in wpart, which only it touches.
constexpr int kBwdRows = 2, kBwdDepth = 3;
template <typename T, bool POST, int MAXT>
__global__ void __launch_bounds__(MAXT, bwd_ctas(MAXT)) block_norm_bwd_vec_kernel(BlockNormArgs a, NormPlan p, float *part,
                                                                 float *wpart) {
  constexpr int R = kBwdRows;
  __shared__ __align__(16) float red_buf[2 * kVecWarps * 8];
  extern __shared__ __align__(16) uint8_t ring[];
  VecReducer red{red_buf, 0};
  chain_next();
  Fetch<T, 4 * R, kBwdDepth> rows{reinterpret_cast<T *>(ring) + threadIdx.x * 8, 0};
  const T *h = static_cast<const T *>(a.h), *y = static_cast<const T *>(a.yin);
  const T *dz = static_cast<const T *>(a.dz), *dy = static_cast<const T *>(a.dy);  // either may be dh or dx
  T *dh = static_cast<T *>(a.dh), *dx = static_cast<T *>(a.dx);
  const bool want_h = dh || a.dgate || a.dpost_gamma;
  const bool pre_mean = a.pre == MOE_NORM_LAYER, post_mean = a.post == MOE_NORM_LAYER;
  const int c = threadIdx.x * 8;
  const bool col = c < a.d;
  const float inv_d = 1.0f / (float)a.d;
  const uint64_t alpha = f2_splat(a.res_scale);
  const int64_t g_lo = p.segments * blockIdx.x / p.grid, g_hi = p.segments * (blockIdx.x + 1) / p.grid;
  for (int64_t seg = g_lo; seg < g_hi; ++seg) {
    const Segment sg = segment_of(p, seg, a.T);
    // Rows s0 .. s0 + R - 1 of y, dz, h and dy into a step of the ring. dh and
    // dx of a row may be its dz or dy, which has been copied by then.
    auto fetch = [&](int s0, int step) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool live = col && s0 + i < sg.hi;
        const size_t at = (size_t)(s0 + i) * a.d + c;
        const T *any = dz ? dz : dy;
        rows.issue(step, 4 * i, dz ? y + at : any, live && dz);
        rows.issue(step, 4 * i + 1, dz ? dz + at : any, live && dz);
        rows.issue(step, 4 * i + 2, want_h && h ? h + at : any, live && want_h && h);
        rows.issue(step, 4 * i + 3, dy ? dy + at : any, live && dy);
      }
      rows.commit();
    };
    rows.template wait<0>();  // the last segment's copies past its end
    rows.slot = 0;
#pragma unroll
    for (int k = 0; k < kBwdDepth - 1; ++k) fetch(sg.lo + k * R, k);
    const size_t cond = (size_t)sg.group * a.cond_stride + c;
    V8 fz = load_v8_or(static_cast<const T *>(a.scale), cond, col, 0.f);
    V8 fh = load_v8_or(static_cast<const T *>(a.gate), cond, col, 1.f);
    V8 S0, S1, P;
    S0.fill(0.f);
    S1.fill(0.f);
    P.fill(0.f);
    {
      // Factors past the row's end are 0: nothing there enters a mean.
      const V8 pg = load_v8_or(static_cast<const T *>(a.pre_gamma), c, col, col ? 1.f : 0.f);
      const V8 po = load_v8_or(static_cast<const T *>(a.post_gamma), c, col, col ? 1.f : 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        fz.v[j] = f2_mul(f2_add(fz.v[j], f2_splat(1.f)), pg.v[j]);
        fh.v[j] = f2_mul(fh.v[j], po.v[j]);
      }
    }
    for (int s0 = sg.lo; s0 < sg.hi; s0 += R) {
      fetch(s0 + (kBwdDepth - 1) * R, rows.last());
      rows.template wait<kBwdDepth - 1>();
      V8 t[R], m[R], n[R], g[R];
      float rh[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        rh[i] = 1.f;
        n[i] = rows.get(4 * i);
        g[i] = rows.get(4 * i + 1);
        if (POST) m[i] = rows.get(4 * i + 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          S0.v[j] = f2_add(S0.v[j], g[i].v[j]);
          g[i].v[j] = f2_mul(g[i].v[j], fz.v[j]);
        }
      }
      constexpr int K = POST ? 8 : 4;
      float s[K], mg[R];
#pragma unroll
      for (int i = 0; i < K; ++i) s[i] = 0.f;
      if (pre_mean || (POST && post_mean)) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          s[i] = sum_v8(n[i]);
          s[R + i] = sum_v8(g[i]);
          if (POST) s[2 * R + i] = sum_v8(m[i]);
        }
        block_sum_vec(s, red);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        mg[i] = pre_mean ? s[R + i] * inv_d : 0.f;
        const uint64_t my = f2_splat(pre_mean && col ? -s[i] * inv_d : 0.f);
        const uint64_t mh = f2_splat(POST && post_mean && col ? -s[POST ? 2 * R + i : 0] * inv_d : 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          n[i].v[j] = f2_add(n[i].v[j], my);
          if (POST) m[i].v[j] = f2_add(m[i].v[j], mh);
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        s[i] = dot_v8(n[i], n[i]);
        s[R + i] = dot_v8(g[i], n[i]);
        if (POST) s[2 * R + i] = dot_v8(m[i], m[i]);
      }
      block_sum_vec(s, red);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool live = col && s0 + i < sg.hi;
        t[i] = rows.get(4 * i + 3);
        if (!POST) m[i] = rows.get(4 * i + 2);
        if (dz) {
          const V8 q = rows.get(4 * i + 1);
          const float r = rsqrtf(fmaf(s[i], inv_d, a.eps));
          const float k = r * (s[R + i] * inv_d) * r;  // mean(g n), times r: n is r yc
          const uint64_t rr = f2_splat(r), c0 = f2_splat(-r * mg[i]), c1 = f2_splat(-k);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            n[i].v[j] = f2_mul(n[i].v[j], rr);  // n
            S1.v[j] = f2_fma(q.v[j], n[i].v[j], S1.v[j]);
            t[i].v[j] = f2_add(t[i].v[j], f2_fma(rr, g[i].v[j], f2_fma(c1, n[i].v[j], c0)));
          }
        }
        if (dx && live) {
          V8 o;
#pragma unroll
          for (int j = 0; j < 4; ++j) o.v[j] = f2_mul(alpha, t[i].v[j]);
          store_v8(dx + (size_t)(s0 + i) * a.d + c, o);
        }
        if (POST) rh[i] = rsqrtf(fmaf(s[POST ? 2 * R + i : 0], inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (POST) m[i].v[j] = f2_mul(m[i].v[j], f2_splat(rh[i]));
          P.v[j] = f2_fma(t[i].v[j], m[i].v[j], P.v[j]);
          t[i].v[j] = f2_mul(t[i].v[j], fh.v[j]);
        }
      }
      rows.next();
      if (!dh) continue;
      if (POST) {
        float w[4];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          w[i] = sum_v8(t[i]);
          w[R + i] = dot_v8(t[i], m[i]);
        }
        block_sum_vec(w, red);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const uint64_t rr = f2_splat(rh[i]), c0 = f2_splat(post_mean ? -rh[i] * (w[i] * inv_d) : 0.f);
          const uint64_t c1 = f2_splat(-rh[i] * (w[R + i] * inv_d));
#pragma unroll
          for (int j = 0; j < 4; ++j) t[i].v[j] = f2_fma(rr, t[i].v[j], f2_fma(c1, m[i].v[j], c0));
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (col && s0 + i < sg.hi) store_v8(dh + (size_t)(s0 + i) * a.d + c, t[i]);
    }
    if (!col) continue;
    if (part) {
      float *o = part + (size_t)seg * 3 * a.d + c;
      store_v8(o, S0);
      store_v8(o + a.d, S1);
      store_v8(o + 2 * (size_t)a.d, P);
    } else {
      const size_t at = (size_t)sg.group * a.dcond_stride + c;
      V8 o;
      if (a.dshift) store_v8(a.dshift + at, S0);
      if (a.dscale) {
        const V8 pg = load_v8_or(static_cast<const T *>(a.pre_gamma), c, true, 1.f);
        const V8 pb = load_v8_or(static_cast<const T *>(a.pre_beta), c, true, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = f2_fma(pg.v[j], S1.v[j], f2_mul(pb.v[j], S0.v[j]));
        store_v8(a.dscale + at, o);
      }
      if (a.dgate) {
        const V8 po = load_v8_or(static_cast<const T *>(a.post_gamma), c, true, 1.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = f2_mul(po.v[j], P.v[j]);
        store_v8(a.dgate + at, o);
      }
    }
    if (wpart) {
      float *o = wpart + (size_t)blockIdx.x * 3 * a.d + c;
      const V8 sc = load_v8_or(static_cast<const T *>(a.scale), cond, true, 0.f);
      const V8 gt = load_v8_or(static_cast<const T *>(a.gate), cond, true, 1.f);
      V8 w0, w1, w2;
      w0.fill(0.f);
      w1.fill(0.f);
      w2.fill(0.f);
      if (seg > g_lo) {
        w0 = unpack_v8(o);
        w1 = unpack_v8(o + a.d);
        w2 = unpack_v8(o + 2 * (size_t)a.d);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t s1 = f2_add(sc.v[j], f2_splat(1.f));
        w0.v[j] = f2_fma(s1, S1.v[j], w0.v[j]);
        w1.v[j] = f2_fma(s1, S0.v[j], w1.v[j]);
        w2.v[j] = f2_fma(gt.v[j], P.v[j], w2.v[j]);
      }
      store_v8(o, w0);
      store_v8(o + a.d, w1);
      store_v8(o + 2 * (size_t)a.d, w2);
    }
  }
}

// ---- gradient of wide rows
//
// A segment that is its whole group writes that row's condition gradients
// itself; otherwise its sums go to part [segment][3][d]. The CTA's sums for
// the weights go to wpart [cta][3][d] when they are wanted. A second launch
// adds both up in order.
template <typename T>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(BlockNormArgs a, NormPlan p, float *part,
                                                             float *wpart) {
  constexpr int NV = 2, R = 1;
  __shared__ float red_buf[2 * kMaxWarps * 2 * R];
  chain_next();
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

// Sums lists of partial blocks [n][3][d] in order, 128 columns by kSlices
// slices of a list per CTA. List blockIdx.y < groups is a group's segments and
// gives its condition gradients; the ones after are kWeightLists parts of the
// CTAs' sums for the weights (hundreds of entries: one CTA per 128 columns
// would take them in at one SM's bandwidth), whose sums go to wsum; a launch
// over wsum (`last`) gives the weights' gradients.
constexpr int kSlices = 16, kWeightLists = 16;
struct NormSums {
  const float *part, *wpart;
  float *wsum;
  int64_t first, groups;  // first: the list of blockIdx.y = 0
  int per_group, ctas, last;
};
template <typename T>
__global__ void __launch_bounds__(32 * kSlices) block_norm_sum_kernel(BlockNormArgs a, NormSums q) {
  __shared__ __align__(16) float sh[3][kSlices][128];
  chain_wait();
  chain_next();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t list = q.first + blockIdx.y;
  const bool cond = list < q.groups;
  const int part = (int)(list - q.groups), c0 = blockIdx.x * 128;
  int n = q.per_group;
  const float *src = q.part + (size_t)list * q.per_group * 3 * a.d;
  if (!cond) {
    const int lo = q.last ? 0 : q.ctas * part / kWeightLists;
    n = q.last ? kWeightLists : q.ctas * (part + 1) / kWeightLists - lo;
    src = (q.last ? q.wsum : q.wpart) + (size_t)lo * 3 * a.d;
  }
  src += c0 + lane * 4;
  float4 v[3];
#pragma unroll
  for (int w = 0; w < 3; ++w) v[w] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c0 + lane * 4 < a.d) {
    const int lo = n * slice / kSlices, hi = n * (slice + 1) / kSlices;
#pragma unroll 4
    for (int k = lo; k < hi; ++k)
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        const float4 f = *reinterpret_cast<const float4 *>(src + ((size_t)k * 3 + w) * a.d);
        v[w].x += f.x;
        v[w].y += f.y;
        v[w].z += f.z;
        v[w].w += f.w;
      }
  }
#pragma unroll
  for (int w = 0; w < 3; ++w) *reinterpret_cast<float4 *>(&sh[w][slice][lane * 4]) = v[w];
  __syncthreads();
  const int col = c0 + threadIdx.x;
  if (threadIdx.x >= 128 || col >= a.d) return;
  float t[3];
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    t[w] = 0.f;
#pragma unroll
    for (int k = 0; k < kSlices; ++k) t[w] += sh[w][k][threadIdx.x];
  }
  if (cond) {
    const size_t at = (size_t)list * a.dcond_stride + col;
    const T *pg = static_cast<const T *>(a.pre_gamma), *pb = static_cast<const T *>(a.pre_beta),
            *po = static_cast<const T *>(a.post_gamma);
    if (a.dshift) a.dshift[at] = t[0];
    if (a.dscale) a.dscale[at] = fmaf(pg ? to_f32(pg[col]) : 1.f, t[1], pb ? to_f32(pb[col]) * t[0] : 0.f);
    if (a.dgate) a.dgate[at] = (po ? to_f32(po[col]) : 1.f) * t[2];
  } else if (!q.last) {
#pragma unroll
    for (int w = 0; w < 3; ++w) q.wsum[((size_t)part * 3 + w) * a.d + col] = t[w];
  } else {
    if (a.dpre_gamma) a.dpre_gamma[col] = t[0];
    if (a.dpre_beta) a.dpre_beta[col] = t[1];
    if (a.dpost_gamma) a.dpost_gamma[col] = t[2];
  }
}

// Threads of a CTA whose threads own nv vectors of 8 columns each.
int row_threads(int d, int nv) {
  const int vecs = d / 8;
  return ((vecs + nv - 1) / nv + 31) / 32 * 32;
}
// Rows of up to 8 KB take a thread per 8 columns (at most 512 threads, and
// rings of at most 196 KB); wider ones 2 vectors per thread and one row at a
// time (the backward spills 512 bytes a thread there: 12 arrays of 16 columns
// do not fit 128 registers).
template <typename T> inline bool narrow(int d) { return d * (int)sizeof(T) <= 8192; }
// The kernels for many rows are built for three bounds on the threads (fp32
// rows of up to 8 KB take at most 256). Their limit on shared memory is set to
// the bound's: one that follows the size of each call could be lowered by
// another host thread between a call's setting it and its launch.
inline int thread_bound(int d) {
  const int t = row_threads(d, 1);
  return t <= 160 ? 160 : t <= 256 ? 256 : 512;
}

template <typename T>
int run_fwd(const BlockNormArgs &a, cudaStream_t stream) {
  const int64_t sms = num_sms();
  if (!narrow<T>(a.d)) {
    const int64_t grid = a.T < 4 * sms ? a.T : 4 * sms;
    block_norm_kernel<T, 2, 1><<<(unsigned)grid, row_threads(a.d, 2), 0, stream>>>(a);
  } else if (a.T <= 2 * sms) {  // few tokens: a CTA each
    block_norm_kernel<T, 1, 1><<<a.T, row_threads(a.d, 1), 0, stream>>>(a);
  } else {
    const NormPlan p = norm_plan(a.T, a.group, a.gate || a.scale || a.shift, kFwdRows,
                                 (int)sms * fwd_ctas(thread_bound(a.d)));
    const int threads = row_threads(a.d, 1), bound = thread_bound(a.d);
    const auto kern = bound == 160                     ? block_norm_vec_kernel<T, 160>
                      : bound == 256 || sizeof(T) == 4 ? block_norm_vec_kernel<T, 256>
                                                       : block_norm_vec_kernel<T, sizeof(T) == 4 ? 256 : 512>;
    const size_t smem = fetch_bytes<T, 2 * kFwdRows, kFwdDepth>(threads);
    const size_t most = fetch_bytes<T, 2 * kFwdRows, kFwdDepth>(bound);
    MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
    kern<<<p.grid, threads, smem, stream>>>(a, p);
  }
  return last_launch_status();
}

// Rows at a time and CTAs at once of the backward. The SMs are counted as the
// B200's 148, not asked for: the plan sizes the workspace, which has to be the
// same on a host without a GPU, and fixes the order of the sums.
template <typename T>
NormPlan bwd_plan(int tokens, int d, int group, bool conds) {
  return narrow<T>(d) ? norm_plan(tokens, group, conds, kBwdRows, 148 * bwd_ctas(thread_bound(d)))
                      : norm_plan(tokens, group, conds, 1, 148);
}

template <typename T, bool POST>
auto bwd_kernel(int bound) {
  return bound == 160                     ? block_norm_bwd_vec_kernel<T, POST, 160>
         : bound == 256 || sizeof(T) == 4 ? block_norm_bwd_vec_kernel<T, POST, 256>
                                          : block_norm_bwd_vec_kernel<T, POST, sizeof(T) == 4 ? 256 : 512>;
}

template <typename T>
int run_bwd(const BlockNormArgs &a, cudaStream_t stream) {
  const bool conds = a.gate || a.scale || a.dgate || a.dscale || a.dshift;
  const NormPlan p = bwd_plan<T>(a.T, a.d, a.group, conds);
  const bool cond_out = a.dgate || a.dscale || a.dshift;
  float *part = cond_out && p.per_group > 1 ? a.part : nullptr;
  float *wpart = a.dpre_gamma || a.dpre_beta || a.dpost_gamma
                     ? a.part + (part ? (size_t)p.segments * 3 * a.d : 0) : nullptr;
  if (a.T > 0) {
    if (!narrow<T>(a.d))
      block_norm_bwd_kernel<T><<<p.grid, row_threads(a.d, 2), 0, stream>>>(a, p, part, wpart);
    else {
      const int threads = row_threads(a.d, 1), bound = thread_bound(a.d);
      const auto kern = a.post == MOE_NORM_NONE ? bwd_kernel<T, false>(bound) : bwd_kernel<T, true>(bound);
      const size_t smem = fetch_bytes<T, 4 * kBwdRows, kBwdDepth>(threads);
      const size_t most = fetch_bytes<T, 4 * kBwdRows, kBwdDepth>(bound);
      MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
      kern<<<p.grid, threads, smem, stream>>>(a, p, part, wpart);
    }
  }
  NormSums q{};
  q.part = part; q.wpart = wpart; q.wsum = wpart + (size_t)p.grid * 3 * a.d;
  q.groups = p.groups; q.per_group = p.per_group; q.ctas = a.T > 0 ? p.grid : 0;
  const unsigned blocks = (a.d + 127) / 128;
  const int64_t end = p.groups + (wpart ? kWeightLists : 0);
  for (q.first = part ? 0 : p.groups; q.first < end; q.first += 65535) {
    const unsigned n = (unsigned)(end - q.first < 65535 ? end - q.first : 65535);
    launch_chained(block_norm_sum_kernel<T>, dim3(blocks, n), 32 * kSlices, 0, stream, a, q);
  }
  if (wpart) {
    q.first = p.groups;
    q.last = 1;
    launch_chained(block_norm_sum_kernel<T>, dim3(blocks, 1), 32 * kSlices, 0, stream, a, q);
  }
  return last_launch_status();
}

}  // namespace

// Partial sums of either way (with or without conditions) the backward can cut the rows.
size_t block_norm_workspace_bytes(int T, int d, int group, int dtype) {
  int64_t most = 0;
  for (int conds = 0; conds < 2; ++conds) {
    const NormPlan p = dtype == MOE_BF16 ? bwd_plan<__nv_bfloat16>(T, d, group, conds != 0)
                                         : bwd_plan<float>(T, d, group, conds != 0);
    const int64_t n = (p.per_group > 1 ? p.segments : 0) + p.grid + kWeightLists;
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
