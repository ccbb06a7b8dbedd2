// Gradients of the token exchange: the combine's (expert-output rows,
// routing weights, constant experts) and the dispatch's (rows back to their
// tokens).
//
// DICE: Staleness-Centric Optimizations for Parallel Diffusion MoE
// Inference, "Conditional Communication": a token's output is the sum of
// its experts' outputs weighted by its routing scores; its gradient
// equation weights the gradient of an expert's output by the same score.
// MMOE: Modernizing Diffusion Transformers with Efficient Expert Design,
// "MoE++ expert layer": identity, zero and constant experts.
//
// Both kernels only move rows, so they are bound by HBM: each lane owns 8
// consecutive features of a 256-feature chunk (16-byte accesses) and a pass
// issues the loads of several chunks before any arithmetic. Dot products and
// sums are fp32 in a fixed order; nothing is accumulated by atomics.
#include "backward.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(h[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

// What the whole warp knows of a mixed constant expert on a token: a0, a1 =
// softmax(Wc x) and <dy, x>, <dy, v>.
struct MixDots {
  float a0, a1, gx, gv;
};
template <typename T>
__device__ __noinline__ MixDots mix_dots(const T *xr, const T *gr, const T *vrow, int d) {
  const int lane = threadIdx.x & 31;
  float z0 = 0.f, z1 = 0.f, gx = 0.f, gv = 0.f;
  for (int c = lane * 8; c < d; c += 256) {
    float x[8], g[8], v[8], w0[8], w1[8];
    load8(xr + c, x);
    load8(gr + c, g);
    load8(vrow + c, v);
    load8(vrow + d + c, w0);
    load8(vrow + 2 * (size_t)d + c, w1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z0 = fmaf(x[i], w0[i], z0);
      z1 = fmaf(x[i], w1[i], z1);
      gx = fmaf(g[i], x[i], gx);
      gv = fmaf(g[i], v[i], gv);
    }
  }
  z0 = warp_sum(z0);
  z1 = warp_sum(z1);
  const float m = fmaxf(z0, z1);
  const float e0 = expf(z0 - m), e1 = expf(z1 - m);
  return {e0 / (e0 + e1), e1 / (e0 + e1), warp_sum(gx), warp_sum(gv)};
}

// Token and expert of assignment `asg`, checked: false (and dw 0) for an
// empty slot or an id out of range.
__device__ __forceinline__ bool assignment_of(const ExchangeBwdArgs &a, int64_t asg, int &s, int &e) {
  const int id = a.sel[asg];
  if (a.routing == MOE_EXPERT_CHOICE) {
    s = id;
    e = (int)((asg / a.C) % a.E);
    if (s < 0 || s >= a.T) {
      set_status(a.dev_status, MOE_DEV_BAD_TOKEN);
      return false;
    }
  } else {
    s = (int)(asg / a.k);
    e = id;
    if (e < 0 || e >= a.E) {
      if (e != -1) set_status(a.dev_status, MOE_DEV_BAD_EXPERT);
      return false;
    }
  }
  return true;
}

// One warp per assignment: the token's gradient row is read again by each
// of its assignments, which sit next to each other under token choice, so
// all but the first read hit L1 or L2. Loads of kPass chunks of both rows
// are in flight together.
constexpr int kPass = 3;
template <typename T>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(ExchangeBwdArgs a, KindTable kinds) {
  const T *__restrict__ dy = static_cast<const T *>(a.dy);
  const T *__restrict__ yp = static_cast<const T *>(a.y_perm);
  const T *__restrict__ x = static_cast<const T *>(a.x);
  const T *__restrict__ cv = static_cast<const T *>(a.const_vecs);
  T *__restrict__ out = static_cast<T *>(a.dy_perm);
  const int lane = threadIdx.x & 31;
  const int64_t nw = (int64_t)gridDim.x * kWarps;
  for (int64_t asg = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); asg < a.n_assign; asg += nw) {
    int s = 0, e = 0;
    const T *src = nullptr;
    T *dst = nullptr;
    bool mix = false;
    if (assignment_of(a, asg, s, e)) {
      const int kind = kinds.kind[e];
      if (kind == MOE_HEAVY) {
        const int row = a.row_of[asg];
        const bool in = row >= 0 && row < a.n_assign;
        if (row >= a.n_assign) set_status(a.dev_status, MOE_DEV_BAD_INDEX);
        if (in) {
          src = yp + (size_t)row * a.d;
          dst = out + (size_t)row * a.d;
        }
      } else if (kind == MOE_IDENTITY) {
        src = x + (size_t)s * a.d;
      } else if (kind == MOE_CONST) {
        src = cv + (size_t)kinds.cidx[e] * (a.const_mix ? 3 : 1) * a.d;
        mix = a.const_mix != 0;
      }
    }
    const T *g = dy + (size_t)s * a.d;
    float dot = 0.f;
    if (mix) {
      const MixDots m = mix_dots(x + (size_t)s * a.d, g, src, a.d);
      dot = m.a0 * m.gx + m.a1 * m.gv;
    } else if (src) {
      const float wgt = dst ? a.w[asg] : 0.f;
      for (int c = lane * 8; c < a.d; c += 256 * kPass) {
        Raw8<T> rg[kPass], rs[kPass];
#pragma unroll
        for (int q = 0; q < kPass; ++q)
          if (c + 256 * q < a.d) {
            rg[q].load(g + c + 256 * q);
            rs[q].load(src + c + 256 * q);
          }
#pragma unroll
        for (int q = 0; q < kPass; ++q)
          if (c + 256 * q < a.d) {
            float fg[8], fs[8];
            rg[q].get(fg);
            rs[q].get(fs);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dot = fmaf(fg[i], fs[i], dot);
              fg[i] *= wgt;
            }
            if (dst) store8(dst + c + 256 * q, fg);
          }
      }
      dot = warp_sum(dot);
    }
    if (lane == 0) a.dw[asg] = dot;
  }
}

// ---- constant experts
//
// dv_c = sum over the assignments of constant expert c of (a1) w dy_s, and
// with const_mix dWc_0 = sum q x_s. CTA (chunk, c, column block) walks its
// chunk of the assignments in batches: the matching ones are listed in
// order, the warps form their coefficients, and then each thread adds the
// listed rows into the 8 columns it owns. Chunks are summed by a second
// launch in chunk order.
__host__ __device__ inline int const_chunks(int64_t n_assign, int n_const) {
  const int64_t want = (n_assign + kThreads - 1) / kThreads;
  const int64_t cap = n_const >= 592 ? 1 : 592 / (n_const > 0 ? n_const : 1);
  return (int)(want < 1 ? 1 : want < cap ? want : cap);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) const_grad_kernel(ExchangeBwdArgs a, KindTable kinds, int chunks) {
  __shared__ int scratch[40];
  __shared__ int list_s[kThreads];
  __shared__ float list_v[kThreads], list_q[kThreads];
  const T *dy = static_cast<const T *>(a.dy);
  const T *x = static_cast<const T *>(a.x);
  const T *cv = static_cast<const T *>(a.const_vecs);
  const int c = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = (blockIdx.z * kThreads + tid) * 8;
  const bool live = col < a.d;
  const int64_t lo = a.n_assign * blockIdx.x / chunks, hi = a.n_assign * (blockIdx.x + 1) / chunks;
  float av[8], aq[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) av[i] = aq[i] = 0.f;
  for (int64_t b = lo; b < hi; b += kThreads) {
    int s = 0, e = 0, hit = 0;
    if (b + tid < hi && assignment_of(a, b + tid, s, e))
      hit = kinds.kind[e] == MOE_CONST && kinds.cidx[e] == c;
    int n = 0;
    const int at = block_exclusive_scan(hit, scratch, &n);
    if (hit) {
      list_s[at] = s;
      list_v[at] = a.w[b + tid];
      list_q[at] = 0.f;
    }
    __syncthreads();
    if (a.const_mix) {
      const T *vrow = cv + (size_t)c * 3 * a.d;
      for (int i = warp; i < n; i += kWarps) {
        const size_t r = (size_t)list_s[i] * a.d;
        const MixDots m = mix_dots(x + r, dy + r, vrow, a.d);
        const float w = list_v[i];
        __syncwarp();
        if (lane == 0) {
          list_v[i] = w * m.a1;
          list_q[i] = m.a0 * m.a1 * (w * m.gx - w * m.gv);
        }
      }
      __syncthreads();
    }
    if (live) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const size_t r = (size_t)list_s[i] * a.d + col;
        float g[8];
        load8(dy + r, g);
        const float v = list_v[i];
#pragma unroll
        for (int j = 0; j < 8; ++j) av[j] = fmaf(v, g[j], av[j]);
        if (a.const_mix) {
          float xv[8];
          load8(x + r, xv);
          const float q = list_q[i];
#pragma unroll
          for (int j = 0; j < 8; ++j) aq[j] = fmaf(q, xv[j], aq[j]);
        }
      }
    }
    __syncthreads();
  }
  if (!live) return;
  const int rows = a.const_mix ? 2 : 1;
  float *p = a.const_part + ((size_t)blockIdx.x * a.n_const + c) * rows * a.d + col;
  store8(p, av);
  if (a.const_mix) store8(p + a.d, aq);
}

// Sum over the chunks: dconst [n_const, d], or [n_const, 3, d] with the
// mixing rows dWc_0 and dWc_1 = -dWc_0.
__global__ void __launch_bounds__(kThreads) const_grad_sum_kernel(const float *part, float *out, int chunks,
                                                                  int n_const, int d, int mix) {
  const int rows = mix ? 2 : 1;
  const int64_t n = (int64_t)n_const * rows * d;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    float t = 0.f;
    for (int k = 0; k < chunks; ++k) t += part[(size_t)k * n + i];
    if (!mix) {
      out[i] = t;
    } else {
      const int64_t r = i / d, col = i - r * d, c = r >> 1;
      float *o = out + (size_t)c * 3 * d + col;
      if (r & 1) {
        o[d] = t;
        o[2 * (size_t)d] = -t;
      } else {
        o[0] = t;
      }
    }
  }
}

// ---- dispatch
//
// One warp per token, or per 256-feature chunk of one when there are too few
// tokens to occupy the GPU. The token's slots are read once, one per lane,
// and turned into a source row and coefficient: 1 on the expert's input
// gradient, q on Wc_0 - Wc_1 (`diff`) for a mixed constant expert; the
// coefficients of dy_s itself are summed over the slots.
template <typename T>
__device__ __forceinline__ void bwd_slots(const ExchangeBwdArgs &a, const KindTable &kinds, bool ec, int s, int j0,
                                          int j1, const T *&src, float &wgt, bool &diff, float &g_coef) {
  const int lane = threadIdx.x & 31;
  src = nullptr;
  wgt = 0.f;
  diff = false;
  float own_g = 0.f;
  const int j = j0 + lane;
  if (j < j1) {
    const int asg = ec ? a.tok_assign[j] : j;
    const bool in = asg >= 0 && asg < a.n_assign;
    const int e = !in ? -1 : ec ? (int)((asg / a.C) % a.E) : a.sel[asg];
    if (!in) set_status(a.dev_status, MOE_DEV_BAD_INDEX);
    if (e >= 0 && e < a.E) {
      const int kind = kinds.kind[e];
      if (kind == MOE_HEAVY) {
        const int row = a.row_of[asg];
        if (row >= 0 && row < a.n_assign) {
          src = static_cast<const T *>(a.dx_perm) + (size_t)row * a.d;
          wgt = 1.f;
        } else if (row >= a.n_assign) {
          set_status(a.dev_status, MOE_DEV_BAD_INDEX);
        }
      } else if (kind == MOE_IDENTITY) {
        own_g = a.w[asg];
      } else if (kind == MOE_CONST && a.const_mix) {
        src = static_cast<const T *>(a.const_vecs) + (size_t)kinds.cidx[e] * 3 * a.d;
        wgt = a.w[asg];
        diff = true;
      }
    }
  }
  for (unsigned mm = __ballot_sync(0xffffffffu, diff); mm; mm &= mm - 1u) {
    const int q = __ffs(mm) - 1;
    const T *vrow = reinterpret_cast<const T *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), q));
    const size_t r = (size_t)s * a.d;
    const MixDots m = mix_dots(static_cast<const T *>(a.x) + r, static_cast<const T *>(a.dy) + r, vrow, a.d);
    if (lane == q) {
      own_g = wgt * m.a0;
      wgt = m.a0 * m.a1 * (wgt * m.gx - wgt * m.gv);
      src += a.d;  // Wc_0
    }
  }
  g_coef += warp_sum(own_g);
}

constexpr int kBatch = 2;
template <typename T>
__global__ void __launch_bounds__(kThreads) dispatch_bwd_kernel(ExchangeBwdArgs a, KindTable kinds) {
  const T *dy = static_cast<const T *>(a.dy);
  const T *add0 = static_cast<const T *>(a.add[0]), *add1 = static_cast<const T *>(a.add[1]),
          *add2 = static_cast<const T *>(a.add[2]);  // may alias dx
  T *dx = static_cast<T *>(a.dx);
  const int lane = threadIdx.x & 31;
  const bool ec = a.routing == MOE_EXPERT_CHOICE;
  const int chunks = (a.d + 255) / 256;
  const int per_item = a.fine ? 1 : chunks, items_per_tok = a.fine ? chunks : 1;
  const int64_t items = (int64_t)a.T * items_per_tok, nw = (int64_t)gridDim.x * kWarps;
  for (int64_t it = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); it < items; it += nw) {
    const int s = (int)(it / items_per_tok);
    const int c_begin = (int)(it - (int64_t)s * items_per_tok) * per_item;
    const int c_end = c_begin + per_item < chunks ? c_begin + per_item : chunks;
    int64_t a0, a1;
    if (ec) {
      a0 = a.tok_ptr[s];
      a1 = a.tok_ptr[s + 1];
      if (a0 < 0 || a1 < a0 || a1 > a.n_assign) {  // a token list out of range: no slots
        if (lane == 0) set_status(a.dev_status, MOE_DEV_BAD_INDEX);
        a0 = a1 = 0;
      }
    } else {
      a0 = (int64_t)s * a.k;
      a1 = a0 + a.k;
    }
    // The slots once per token; past 32 of them the later groups are read
    // again in every pass (g_coef is complete after the first walk).
    const bool one_group = a1 - a0 <= 32;
    const T *m_src = nullptr;
    float m_w = 0.f, g_coef = 0.f;
    bool m_diff = false;
    for (int64_t j0 = a0; j0 < a1; j0 += 32)
      bwd_slots(a, kinds, ec, s, (int)j0, (int)a1, m_src, m_w, m_diff, g_coef);
    const size_t rb = (size_t)s * a.d;
    for (int cb = c_begin; cb < c_end; cb += kPass) {
      int c0[kPass];
      bool live[kPass];
      float acc[kPass][8];
#pragma unroll
      for (int q = 0; q < kPass; ++q) {
        c0[q] = (cb + q) * 256 + lane * 8;
        live[q] = cb + q < c_end && c0[q] < a.d;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[q][i] = 0.f;
        if (!live[q]) continue;
        float t[8];
        if (add0) {
          load8(add0 + rb + c0[q], t);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[q][i] += t[i];
        }
        if (add1) {
          load8(add1 + rb + c0[q], t);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[q][i] += t[i];
        }
        if (add2) {
          load8(add2 + rb + c0[q], t);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[q][i] += t[i];
        }
        if (g_coef != 0.f) {
          load8(dy + rb + c0[q], t);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[q][i] = fmaf(g_coef, t[i], acc[q][i]);
        }
      }
      for (int64_t j0 = a0; j0 < a1; j0 += 32) {
        const T *g_src = m_src;
        float g_w = m_w, unused = 0.f;
        bool g_diff = m_diff;
        if (!one_group) bwd_slots(a, kinds, ec, s, (int)j0, (int)a1, g_src, g_w, g_diff, unused);
        const int nj = (int)(a1 - j0 < 32 ? a1 - j0 : 32);
        for (int jb = 0; jb < nj; jb += kBatch) {
          Raw8<T> raw[kBatch][kPass];
          const T *src[kBatch];
          float wgt[kBatch];
          bool diff[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int j = (jb + u) & 31;
            src[u] = reinterpret_cast<const T *>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(g_src), j));
            wgt[u] = __shfl_sync(0xffffffffu, g_w, j);
            diff[u] = __shfl_sync(0xffffffffu, (int)g_diff, j) != 0;
            if (jb + u >= nj) src[u] = nullptr;
#pragma unroll
            for (int q = 0; q < kPass; ++q)
              if (src[u] && live[q]) raw[u][q].load(src[u] + c0[q]);
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
#pragma unroll
            for (int q = 0; q < kPass; ++q)
              if (src[u] && live[q]) {
                float f[8];
                raw[u][q].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[q][i] = fmaf(wgt[u], f[i], acc[q][i]);
                if (diff[u]) {
                  load8(src[u] + a.d + c0[q], f);
#pragma unroll
                  for (int i = 0; i < 8; ++i) acc[q][i] = fmaf(-wgt[u], f[i], acc[q][i]);
                }
              }
        }
      }
#pragma unroll
      for (int q = 0; q < kPass; ++q)
        if (live[q]) store8(dx + rb + c0[q], acc[q]);
    }
  }
}

template <typename K>
int resident_blocks_of(K kern) {
  int nb = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&nb, kern, kThreads, 0) != cudaSuccess || nb < 1) nb = 1;
  return nb;
}

}  // namespace

size_t const_grad_workspace_bytes(int64_t n_assign, int n_const, int d, int const_mix) {
  if (n_const == 0) return 0;
  return (size_t)const_chunks(n_assign, n_const) * n_const * (const_mix ? 2 : 1) * d * 4;
}

int launch_combine_bwd(const ExchangeBwdArgs &a, const KindTable &kinds, cudaStream_t stream) {
  const bool bf16 = a.dtype == MOE_BF16;
  if (a.n_assign > 0) {
    static const int nb_bf16 = resident_blocks_of(combine_bwd_kernel<__nv_bfloat16>);
    static const int nb_f32 = resident_blocks_of(combine_bwd_kernel<float>);
    int64_t blocks = (a.n_assign + kWarps - 1) / kWarps;
    const int64_t cap = (int64_t)num_sms() * (bf16 ? nb_bf16 : nb_f32);
    if (blocks > cap) blocks = cap;
    if (bf16) combine_bwd_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, stream>>>(a, kinds);
    else combine_bwd_kernel<float><<<(unsigned)blocks, kThreads, 0, stream>>>(a, kinds);
  }
  if (a.dconst && a.n_const > 0) {
    const int chunks = const_chunks(a.n_assign, a.n_const);
    const dim3 grid(chunks, a.n_const, (a.d + kThreads * 8 - 1) / (kThreads * 8));
    if (bf16) const_grad_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a, kinds, chunks);
    else const_grad_kernel<float><<<grid, kThreads, 0, stream>>>(a, kinds, chunks);
    const int64_t n = (int64_t)a.n_const * (a.const_mix ? 2 : 1) * a.d;
    int64_t blocks = (n + kThreads - 1) / kThreads;
    if (blocks > 1184) blocks = 1184;
    const_grad_sum_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a.const_part, a.dconst, chunks, a.n_const, a.d,
                                                                    a.const_mix);
  }
  return last_launch_status();
}

int launch_dispatch_bwd(const ExchangeBwdArgs &a, const KindTable &kinds, cudaStream_t stream) {
  if (a.T == 0) return MOE_OK;
  static const int nb_bf16 = resident_blocks_of(dispatch_bwd_kernel<__nv_bfloat16>);
  static const int nb_f32 = resident_blocks_of(dispatch_bwd_kernel<float>);
  const bool bf16 = a.dtype == MOE_BF16;
  const int64_t cap = (int64_t)num_sms() * (bf16 ? nb_bf16 : nb_f32);
  const int chunks = (a.d + 255) / 256;
  const int64_t passes = (chunks + kPass - 1) / kPass;
  ExchangeBwdArgs ka = a;
  ka.fine = (int64_t)a.T * passes < cap * kWarps ? 1 : 0;  // whole tokens unless that leaves most warps idle
  int64_t blocks = ((int64_t)a.T * (ka.fine ? chunks : 1) + kWarps - 1) / kWarps;
  if (blocks > cap) blocks = cap;
  if (bf16) dispatch_bwd_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, stream>>>(ka, kinds);
  else dispatch_bwd_kernel<float><<<(unsigned)blocks, kThreads, 0, stream>>>(ka, kinds);
  return last_launch_status();
}

}  // namespace moe
