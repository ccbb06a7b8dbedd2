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
#include "chained.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Volatile: the loads of a pass are issued here, all before the first is
// waited for (the compiler would move a load down to its use, which made one
// round trip to HBM into three in the dispatch).
__device__ __forceinline__ uint4 load16(const void *p) {
  uint4 u;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}
// Zeros unless `live`, without a branch.
__device__ __forceinline__ uint4 load16(const void *p, bool live) {
  uint4 u;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(u.x), "=&r"(u.y), "=&r"(u.z), "=&r"(u.w)
      : "l"(p), "r"((int)live));
  return u;
}
// 8 values as loaded, kept apart from their conversion.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = load16(p); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool live) { u = load16(p, live); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = load16(p);
    b = load16(p + 4);
  }
  __device__ __forceinline__ void load(const float *p, bool live) {
    a = load16(p, live);
    b = load16(p + 4, live);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
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
template <typename T, bool MIX>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(ExchangeBwdArgs a, KindTable kinds) {
  const T *__restrict__ dy = static_cast<const T *>(a.dy);
  const T *__restrict__ yp = static_cast<const T *>(a.y_perm);
  const T *__restrict__ x = static_cast<const T *>(a.x);
  const T *__restrict__ cv = static_cast<const T *>(a.const_vecs);
  T *__restrict__ out = static_cast<T *>(a.dy_perm);
  const int lane = threadIdx.x & 31;
  const int64_t asg = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  chain_next();
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
        src = cv + (size_t)kinds.cidx[e] * (MIX ? 3 : 1) * a.d;
        mix = MIX;
      }
    }
    const T *g = dy + (size_t)s * a.d;
    float dot = 0.f;
    if (MIX && mix) {
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
  // 48 assignments or more to a chunk (a chunk also costs its partial sums'
  // traffic), up to four CTAs per SM over the constant experts.
  const int64_t want = (n_assign + 47) / 48, cap = 592 / (n_const > 0 ? n_const : 1);
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
  chain_wait();
  chain_next();
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
  chain_wait();
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
// One warp per PASS 256-feature chunks of a token. The token's slots are read
// once, one per lane, and turned into a source: the row of the expert's input
// gradient, or for a mixed constant expert (MIX; the others' kernel leaves
// that out) its Wc rows with coefficient q, and the coefficient of dy_s. The
// chain token list -> assignment -> row -> values is four round trips; warps
// enough to hide it stay resident only with few registers, so two chunks and
// BATCH slots at a time (at 62 registers it spills 64 bytes a thread; the mixed
// forms, at 128, up to 96). 8192 tokens of 2048 under expert choice with two
// added gradients (168 MB): 37.8 us in a graph, 0.69 of what an elementwise
// kernel over as many bytes makes of it (26.3). A warp that walks the lists
// ahead of the others took 45 us, four chunks a warp or four tokens in a row
// 43, one chunk and more warps 42.
template <bool MIX> struct Slot {
  int row;    // of dx_perm; -1: no source; -2 - c: mixed constant expert c
  float own;  // coefficient of dy_s: w of an identity, w a0 of a mixed constant expert
  float coef; // q of a mixed constant expert (before its dots: w)
};
template <bool MIX>
__device__ __forceinline__ Slot<MIX> slot_of(const ExchangeBwdArgs &a, const KindTable &kinds, bool ec, int j) {
  Slot<MIX> r{-1, 0.f, 0.f};
  const int asg = ec ? a.tok_assign[j] : j;
  if (asg < 0 || asg >= a.n_assign) {
    set_status(a.dev_status, MOE_DEV_BAD_INDEX);
    return r;
  }
  const int row = a.row_of[asg];
  const int e = ec ? (int)(((unsigned)asg / (unsigned)a.C) % (unsigned)a.E) : a.sel[asg];
  if (e < 0 || e >= a.E) return r;
  const int kind = kinds.kind[e];
  if (kind == MOE_HEAVY) {
    if (row < a.n_assign) r.row = row < 0 ? -1 : row;
    else set_status(a.dev_status, MOE_DEV_BAD_INDEX);
  } else if (kind == MOE_IDENTITY) {
    r.own = a.w[asg];
  } else if (MIX && kind == MOE_CONST) {
    r.row = -2 - kinds.cidx[e];
    r.coef = a.w[asg];
  }
  return r;
}

// 8 fp32 sums as packed pairs.
struct Acc8 {
  uint64_t v[4];
  __device__ __forceinline__ void add(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v[i]) : "l"(f2_pack(f[2 * i], f[2 * i + 1])));
  }
  __device__ __forceinline__ void fma(float w, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_fma(f2_splat(w), f2_pack(f[2 * i], f[2 * i + 1]), v[i]);
  }
};

template <typename T, bool MIX, int PASS, int BATCH, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) dispatch_bwd_kernel(ExchangeBwdArgs a, KindTable kinds) {
  const T *dy = static_cast<const T *>(a.dy), *cv = static_cast<const T *>(a.const_vecs);
  T *dx = static_cast<T *>(a.dx);  // may be any of a.add
  const int lane = threadIdx.x & 31;
  const bool ec = a.routing == MOE_EXPERT_CHOICE;
  const unsigned per_tok = (unsigned)(a.d + 256 * PASS - 1) / (256 * PASS);
  const unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int s = (int)(item / per_tok), c = (int)(item % per_tok) * 256 * PASS + lane * 8;
  if (s >= a.T) return;
  int j_lo = s * a.k, j_hi = j_lo + a.k;
  if (ec) {
    j_lo = a.tok_ptr[s];
    j_hi = a.tok_ptr[s + 1];
    if (j_lo < 0 || j_hi < j_lo || j_hi > a.n_assign) {  // a token list out of range: no slots
      if (lane == 0) set_status(a.dev_status, MOE_DEV_BAD_INDEX);
      j_lo = j_hi = 0;
    }
  }
  // This lane's columns of each chunk; past the row's end it reads others and
  // stores nothing.
  int off[PASS];
#pragma unroll
  for (int q = 0; q < PASS; ++q) off[q] = c + 256 * q < a.d ? c + 256 * q : 0;
  const size_t row0 = (size_t)s * a.d;
  Raw8<T> base[3][PASS];
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (a.add[k]) {
#pragma unroll
      for (int q = 0; q < PASS; ++q) base[k][q].load(static_cast<const T *>(a.add[k]) + row0 + off[q]);
    }
  Acc8 sum[PASS];
#pragma unroll
  for (int q = 0; q < PASS; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[q].v[i] = 0;
  float own = 0.f, f[8];
  for (int j0 = j_lo; j0 < j_hi; j0 += 32) {
    Slot<MIX> mine{-1, 0.f, 0.f};
    if (j0 + lane < j_hi) mine = slot_of<MIX>(a, kinds, ec, j0 + lane);
    if (MIX) {
      for (unsigned mm = __ballot_sync(0xffffffffu, mine.row <= -2); mm; mm &= mm - 1u) {
        const int q = __ffs(mm) - 1, row = __shfl_sync(0xffffffffu, mine.row, q);
        const MixDots m =
            mix_dots(static_cast<const T *>(a.x) + row0, dy + row0, cv + (size_t)(-2 - row) * 3 * a.d, a.d);
        if (lane == q) {
          const float w = mine.coef;
          mine.coef = m.a0 * m.a1 * (w * m.gx - w * m.gv);
          mine.own = w * m.a0;
        }
      }
    }
    if (__any_sync(0xffffffffu, mine.own != 0.f)) own += warp_sum(mine.own);
    // Only slots with a source from here on, in order.
    unsigned left = __ballot_sync(0xffffffffu, mine.row != -1);
    while (left) {
      Raw8<T> raw[BATCH][PASS];
      int row[BATCH];
      float coef[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        row[u] = -1;
        if (left == 0) continue;
        const int q = __ffs(left) - 1;
        left &= left - 1u;
        row[u] = __shfl_sync(0xffffffffu, mine.row, q);
        if (MIX) coef[u] = __shfl_sync(0xffffffffu, mine.coef, q);
        const T *src = MIX && row[u] < 0 ? cv + ((size_t)(-2 - row[u]) * 3 + 1) * a.d
                                         : static_cast<const T *>(a.dx_perm) + (size_t)row[u] * a.d;
#pragma unroll
        for (int i = 0; i < PASS; ++i) raw[u][i].load(src + off[i]);
      }
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        if (row[u] == -1) continue;
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
          raw[u][i].get(f);
          if (MIX && row[u] < 0) {
            sum[i].fma(coef[u], f);
            load8(cv + ((size_t)(-2 - row[u]) * 3 + 2) * a.d + off[i], f);
            sum[i].fma(-coef[u], f);
          } else {
            sum[i].add(f);
          }
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < PASS; ++q) {
    if (c + 256 * q >= a.d) continue;
    if (own != 0.f) {
      load8(dy + row0 + off[q], f);
      sum[q].fma(own, f);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (a.add[k]) {
        base[k][q].get(f);
        sum[q].add(f);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(sum[q].v[i], f[2 * i], f[2 * i + 1]);
    store8(dx + row0 + off[q], f);
  }
}

template <typename T, bool MIX>
int run_dispatch_bwd(const ExchangeBwdArgs &a, const KindTable &kinds, cudaStream_t stream) {
  // Two chunks a warp, unless one still leaves SMs idle.
  const bool few = (int64_t)a.T * ((a.d + 511) / 512) < 16 * (int64_t)num_sms();
  const int64_t items = (int64_t)a.T * (few ? (a.d + 255) / 256 : (a.d + 511) / 512);
  const int64_t blocks = (items + kWarps - 1) / kWarps;
  if (blocks * kWarps > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  constexpr int ctas = sizeof(T) == 2 && !MIX ? 4 : 2;
  if (few) dispatch_bwd_kernel<T, MIX, 1, 8, 2><<<(unsigned)blocks, kThreads, 0, stream>>>(a, kinds);
  else dispatch_bwd_kernel<T, MIX, 2, 2, ctas><<<(unsigned)blocks, kThreads, 0, stream>>>(a, kinds);
  return last_launch_status();
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
    const bool mix = a.n_const > 0 && a.const_mix;
    const auto b = mix ? combine_bwd_kernel<__nv_bfloat16, true> : combine_bwd_kernel<__nv_bfloat16, false>;
    const auto f = mix ? combine_bwd_kernel<float, true> : combine_bwd_kernel<float, false>;
    (bf16 ? b : f)<<<(unsigned)blocks, kThreads, 0, stream>>>(a, kinds);
  }
  if (a.dconst && a.n_const > 0) {
    const dim3 grid(chunks, a.n_const, (a.d + kThreads * 8 - 1) / (kThreads * 8));
    const auto b = a.const_mix ? const_grad_kernel<__nv_bfloat16, true> : const_grad_kernel<__nv_bfloat16, false>;
    const auto f = a.const_mix ? const_grad_kernel<float, true> : const_grad_kernel<float, false>;
    launch_chained(bf16 ? b : f, grid, kThreads, 0, stream, a, kinds, chunks);
    launch_chained(const_grad_sum_kernel, (unsigned)((n + kSumCols - 1) / kSumCols), kSumCols * kSumSlices / 4, 0,
                   stream, a.const_part, a.dconst, chunks, n, a.d, a.const_mix);
  }
  return last_launch_status();
}

int launch_dispatch_bwd(const ExchangeBwdArgs &a, const KindTable &kinds, cudaStream_t stream) {
  if (a.T == 0) return MOE_OK;
  const bool mix = a.n_const > 0 && a.const_mix;
  if (a.dtype == MOE_BF16)
    return mix ? run_dispatch_bwd<__nv_bfloat16, true>(a, kinds, stream)
               : run_dispatch_bwd<__nv_bfloat16, false>(a, kinds, stream);
  return mix ? run_dispatch_bwd<float, true>(a, kinds, stream) : run_dispatch_bwd<float, false>(a, kinds, stream);
}

}  // namespace moe
