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

// 8 values as loaded (zeros unless `live`), kept apart from their conversion
// so that every load of a pass is issued before the first is waited for.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool live) {
    u = make_uint4(0, 0, 0, 0);
    if (live) u = *reinterpret_cast<const uint4 *>(p);
  }
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
  __device__ __forceinline__ void load(const float *p, bool live) {
    a = b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      a = *reinterpret_cast<const float4 *>(p);
      b = *reinterpret_cast<const float4 *>(p + 4);
    }
  }
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
#pragma unroll 3
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
// all but the first read hit L1 or L2. Loads of kRowPass chunks of both rows
// are in flight together. 16384 rows of 1152 (94 MB): 18 us, with a 14.4 us
// floor.
constexpr int kRowPass = 5;
template <typename T>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(ExchangeBwdArgs a, KindTable kinds) {
  const T *__restrict__ dy = static_cast<const T *>(a.dy);
  const T *__restrict__ yp = static_cast<const T *>(a.y_perm);
  const T *__restrict__ x = static_cast<const T *>(a.x);
  const T *__restrict__ cv = static_cast<const T *>(a.const_vecs);
  T *__restrict__ out = static_cast<T *>(a.dy_perm);
  const int lane = threadIdx.x & 31;
  const int64_t asg = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (asg < a.n_assign) {
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
      if (a.dconst && lane == 0) {
        const float w = a.w[asg];
        a.const_coef[asg] = make_float2(w * m.a1, m.a0 * m.a1 * (w * m.gx - w * m.gv));
      }
    } else if (src) {
      const float wgt = dst ? a.w[asg] : 0.f;
      for (int c = lane * 8; c < a.d; c += 256 * kRowPass) {
        Raw8<T> rg[kRowPass], rs[kRowPass];
#pragma unroll
        for (int q = 0; q < kRowPass; ++q) {
          rg[q].load(g + c + 256 * q, c + 256 * q < a.d);
          rs[q].load(src + c + 256 * q, c + 256 * q < a.d);
        }
#pragma unroll
        for (int q = 0; q < kRowPass; ++q) {
          float fg[8], fs[8];
          rg[q].get(fg);
          rs[q].get(fs);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot = fmaf(fg[i], fs[i], dot);
            fg[i] *= wgt;
          }
          if (dst && c + 256 * q < a.d) store8(dst + c + 256 * q, fg);
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
// with const_mix dWc_0 = sum q x_s; the combine's kernel has left w a1 and q
// of each mixed assignment in const_coef. CTA (chunk, c, column block) lists
// its chunk's matching assignments in order, a batch at a time, and then each
// thread adds the listed rows into the 8 columns it owns. Chunks are summed
// by a second launch in chunk order.
__host__ __device__ inline int const_chunks(int64_t n_assign, int n_const) {
  // 16 assignments or more to a chunk (a chunk also costs its partial sums'
  // traffic), up to four CTAs per SM over the constant experts.
  const int64_t want = (n_assign + 15) / 16, cap = 592 / (n_const > 0 ? n_const : 1);
  return (int)(want < 1 ? 1 : want < cap ? want : cap < 1 ? 1 : cap);
}

template <typename T, bool MIX>
__global__ void __launch_bounds__(kThreads, 4) const_grad_kernel(ExchangeBwdArgs a, KindTable kinds, int chunks) {
  __shared__ int scratch[40];
  __shared__ int list_s[kThreads];
  __shared__ float2 list_c[kThreads];
  const T *dy = static_cast<const T *>(a.dy);
  const T *x = static_cast<const T *>(a.x);
  const int c = blockIdx.y, tid = threadIdx.x;
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
      list_c[at] = MIX ? a.const_coef[b + tid] : make_float2(a.w[b + tid], 0.f);
    }
    __syncthreads();
    if (live) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const size_t r = (size_t)list_s[i] * a.d + col;
        const float2 k = list_c[i];
        float g[8];
        load8(dy + r, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) av[j] = fmaf(k.x, g[j], av[j]);
        if (MIX) {
          load8(x + r, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) aq[j] = fmaf(k.y, g[j], aq[j]);
        }
      }
    }
    __syncthreads();
  }
  if (!live) return;
  float *p = a.const_part + ((size_t)blockIdx.x * a.n_const + c) * (MIX ? 2 : 1) * a.d + col;
  store8(p, av);
  if (MIX) store8(p + a.d, aq);
}

// Sum over the chunks: dconst [n_const, d], or [n_const, 3, d] with the
// mixing rows dWc_0 and dWc_1 = -dWc_0. 64 values by 16 slices of the chunks
// per CTA, the slices added in order.
constexpr int kSumSlices = 16, kSumCols = 64;
__global__ void __launch_bounds__(kSumCols * kSumSlices / 4) const_grad_sum_kernel(const float *part, float *out,
                                                                                  int chunks, int64_t n, int d,
                                                                                  int mix) {
  __shared__ __align__(16) float sh[kSumSlices][kSumCols];
  const int quad = threadIdx.x % (kSumCols / 4), slice = threadIdx.x / (kSumCols / 4);
  const int64_t c0 = (int64_t)blockIdx.x * kSumCols;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c0 + quad * 4 < n) {
    const int lo = chunks * slice / kSumSlices, hi = chunks * (slice + 1) / kSumSlices;
#pragma unroll 8
    for (int k = lo; k < hi; ++k) {
      const float4 f = *reinterpret_cast<const float4 *>(part + (size_t)k * n + c0 + quad * 4);
      v.x += f.x;
      v.y += f.y;
      v.z += f.z;
      v.w += f.w;
    }
  }
  *reinterpret_cast<float4 *>(&sh[slice][quad * 4]) = v;
  __syncthreads();
  const int64_t i = c0 + threadIdx.x;
  if (threadIdx.x >= kSumCols || i >= n) return;
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < kSumSlices; ++k) t += sh[k][threadIdx.x];
  if (!mix) {
    out[i] = t;
  } else {
    const int64_t r = i / d, col = i - r * d;
    float *o = out + (size_t)(r >> 1) * 3 * d + col;
    if (r & 1) {
      o[d] = t;
      o[2 * (size_t)d] = -t;
    } else {
      o[0] = t;
    }
  }
}

// ---- dispatch
//
// A CTA takes a few tokens. First a warp per token walks its slots (token
// list -> row: a chain of dependent loads) and leaves each slot's source in
// shared memory: the row of the expert's input gradient, or for a mixed
// constant expert (MIX; the others' kernel leaves that out) its Wc rows and
// coefficient q, and the sum of the coefficients of dy_s itself. Then the
// warps take the tokens' 256-feature chunks, all of whose sources are known
// and in flight together. 8192 tokens of 2048, expert choice (168 MB): 33 us
// of a 26 us floor; with a warp per token and chunk pair, each walking the
// chain, 48 us.
constexpr int kMaxTok = 8;        // tokens per CTA
constexpr int kMaxSlots = 128;    // slots of a token kept in shared memory (the rest are read where they are used)
constexpr int kBatch = 4;         // slots whose rows are in flight together

struct Slot {
  int row;    // of dx_perm; -1: no source; -2 - c: mixed constant expert c
  float coef; // q of a mixed constant expert
};
// Slot j of the list, without a mixed constant expert's dots; own_g: its
// coefficient of dy_s.
template <bool MIX>
__device__ __forceinline__ Slot slot_of(const ExchangeBwdArgs &a, const KindTable &kinds, bool ec, int j, float &own_g) {
  Slot r{-1, 0.f};
  const int asg = ec ? a.tok_assign[j] : j;
  if (asg < 0 || asg >= a.n_assign) {
    set_status(a.dev_status, MOE_DEV_BAD_INDEX);
    return r;
  }
  const int e = ec ? (int)(((unsigned)asg / (unsigned)a.C) % (unsigned)a.E) : a.sel[asg];
  const int row = a.row_of[asg];
  if (e < 0 || e >= a.E) return r;
  const int kind = kinds.kind[e];
  if (kind == MOE_HEAVY) {
    if (row < a.n_assign) r.row = row < 0 ? -1 : row;
    else set_status(a.dev_status, MOE_DEV_BAD_INDEX);
  } else if (kind == MOE_IDENTITY) {
    own_g += a.w[asg];
  } else if (MIX && kind == MOE_CONST) {
    r.row = -2 - kinds.cidx[e];
    r.coef = a.w[asg];
  }
  return r;
}
// The whole warp: a mixed constant expert's w becomes q; w a0 is returned.
template <typename T>
__device__ __forceinline__ float mix_slot(const ExchangeBwdArgs &a, int s, Slot &r) {
  const size_t at = (size_t)s * a.d;
  const MixDots m = mix_dots(static_cast<const T *>(a.x) + at, static_cast<const T *>(a.dy) + at,
                             static_cast<const T *>(a.const_vecs) + (size_t)(-2 - r.row) * 3 * a.d, a.d);
  const float w = r.coef;
  r.coef = m.a0 * m.a1 * (w * m.gx - w * m.gv);
  return w * m.a0;
}

template <typename T, bool MIX>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) dispatch_bwd_kernel(ExchangeBwdArgs a,
                                                                                        KindTable kinds, int tokens) {
  __shared__ Slot slots[kMaxTok][kMaxSlots];
  __shared__ int s_first[kMaxTok], s_count[kMaxTok];
  __shared__ float s_g[kMaxTok];
  const T *dy = static_cast<const T *>(a.dy), *rows = static_cast<const T *>(a.dx_perm);
  T *dx = static_cast<T *>(a.dx);  // may be any of a.add
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool ec = a.routing == MOE_EXPERT_CHOICE;
  const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0);
  if (warp < nt) {
    const int s = t0 + warp;
    int a0 = s * a.k, n = a.k;
    if (ec) {
      a0 = a.tok_ptr[s];
      n = a.tok_ptr[s + 1] - a0;
      if (a0 < 0 || n < 0 || a0 + (int64_t)n > a.n_assign) {  // a token list out of range: no slots
        if (lane == 0) set_status(a.dev_status, MOE_DEV_BAD_INDEX);
        a0 = n = 0;
      }
    }
    float g = 0.f;
    for (int j0 = 0; j0 < n; j0 += 32) {
      Slot r{-1, 0.f};
      float own = 0.f;
      if (j0 + lane < n) r = slot_of<MIX>(a, kinds, ec, a0 + j0 + lane, own);
      if (MIX) {
        for (unsigned mm = __ballot_sync(0xffffffffu, r.row <= -2); mm; mm &= mm - 1u) {
          const int q = __ffs(mm) - 1;
          Slot m{__shfl_sync(0xffffffffu, r.row, q), __shfl_sync(0xffffffffu, r.coef, q)};
          const float own_q = mix_slot<T>(a, s, m);
          if (lane == q) {
            r = m;
            own += own_q;
          }
        }
      }
      if (j0 + lane < n && j0 + lane < kMaxSlots) slots[warp][j0 + lane] = r;
      g += warp_sum(own);
    }
    if (lane == 0) {
      s_first[warp] = a0;
      s_count[warp] = n;
      s_g[warp] = g;
    }
  }
  __syncthreads();
  const int chunks = (a.d + 255) / 256;
  for (int item = warp; item < nt * chunks; item += kWarps) {
    const int t = item / chunks, c = (item - t * chunks) * 256 + lane * 8, n = s_count[t];
    const bool live = c < a.d;
    const size_t at = (size_t)(t0 + t) * a.d + c;
    Raw8<T> base[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) base[k].load(static_cast<const T *>(a.add[k]) + at, live && a.add[k]);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < n; j0 += kBatch) {
      Slot r[kBatch];
      Raw8<T> raw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        r[u] = Slot{-1, 0.f};
        if (j0 + u < n) {
          if (j0 + u < kMaxSlots) {
            r[u] = slots[t][j0 + u];
          } else {
            float unused = 0.f;
            r[u] = slot_of<MIX>(a, kinds, ec, s_first[t] + j0 + u, unused);
            if (MIX && r[u].row <= -2) mix_slot<T>(a, t0 + t, r[u]);
          }
        }
        const T *src = rows + (size_t)(r[u].row < 0 ? 0 : r[u].row) * a.d;
        if (MIX && r[u].row <= -2)
          src = static_cast<const T *>(a.const_vecs) + ((size_t)(-2 - r[u].row) * 3 + 1) * a.d;
        raw[u].load(src + c, live && r[u].row != -1);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        float f[8];
        raw[u].get(f);
        if (MIX && r[u].row <= -2) {
          float f1[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f1[i] = 0.f;
          if (live) load8(static_cast<const T *>(a.const_vecs) + ((size_t)(-2 - r[u].row) * 3 + 2) * a.d + c, f1);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(r[u].coef, f[i] - f1[i], acc[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += f[i];
        }
      }
    }
    if (!live) continue;
    float f[8], o[8];
    base[0].get(o);
#pragma unroll
    for (int k = 1; k < 3; ++k) {
      base[k].get(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += f[i];
    }
    if (s_g[t] != 0.f) {
      load8(dy + at, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(s_g[t], f[i], o[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] += acc[i];
    store8(dx + at, o);
  }
}

}  // namespace

size_t const_grad_workspace_bytes(int64_t n_assign, int n_const, int d, int const_mix) {
  if (n_const == 0) return 0;
  return (size_t)const_chunks(n_assign, n_const) * n_const * (const_mix ? 2 : 1) * d * 4 +
         (const_mix ? (size_t)n_assign * sizeof(float2) : 0);
}

int launch_combine_bwd(const ExchangeBwdArgs &args, const KindTable &kinds, cudaStream_t stream) {
  ExchangeBwdArgs a = args;
  const bool bf16 = a.dtype == MOE_BF16;
  const int chunks = const_chunks(a.n_assign, a.n_const);
  const int64_t n = (int64_t)a.n_const * (a.const_mix ? 2 : 1) * a.d;
  a.const_coef = reinterpret_cast<float2 *>(a.const_part + (size_t)chunks * n);
  if (a.n_assign > 0) {
    const int64_t blocks = (a.n_assign + kWarps - 1) / kWarps;  // below 2^28: assignments fit 31 bits
    if (bf16) combine_bwd_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, stream>>>(a, kinds);
    else combine_bwd_kernel<float><<<(unsigned)blocks, kThreads, 0, stream>>>(a, kinds);
  }
  if (a.dconst && a.n_const > 0) {
    const dim3 grid(chunks, a.n_const, (a.d + kThreads * 8 - 1) / (kThreads * 8));
    const auto b = a.const_mix ? const_grad_kernel<__nv_bfloat16, true> : const_grad_kernel<__nv_bfloat16, false>;
    const auto f = a.const_mix ? const_grad_kernel<float, true> : const_grad_kernel<float, false>;
    (bf16 ? b : f)<<<grid, kThreads, 0, stream>>>(a, kinds, chunks);
    const_grad_sum_kernel<<<(unsigned)((n + kSumCols - 1) / kSumCols), kSumCols * kSumSlices / 4, 0, stream>>>(
        a.const_part, a.dconst, chunks, n, a.d, a.const_mix);
  }
  return last_launch_status();
}

int launch_dispatch_bwd(const ExchangeBwdArgs &a, const KindTable &kinds, cudaStream_t stream) {
  if (a.T == 0) return MOE_OK;
  // As many tokens per CTA as still leave four CTAs for each SM.
  int tokens = a.T / (4 * num_sms());
  tokens = tokens < 1 ? 1 : tokens > kMaxTok ? kMaxTok : tokens;
  const unsigned blocks = (unsigned)((a.T + tokens - 1) / tokens);
  const bool mix = a.n_const > 0 && a.const_mix;
  const auto b = mix ? dispatch_bwd_kernel<__nv_bfloat16, true> : dispatch_bwd_kernel<__nv_bfloat16, false>;
  const auto f = mix ? dispatch_bwd_kernel<float, true> : dispatch_bwd_kernel<float, false>;
  (a.dtype == MOE_BF16 ? b : f)<<<blocks, kThreads, 0, stream>>>(a, kinds, tokens);
  return last_launch_status();
}

}  // namespace moe
