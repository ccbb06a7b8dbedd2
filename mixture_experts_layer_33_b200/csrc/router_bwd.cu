// Gradient of the router: routing weights back through the selection and the
// softmax to the logits, the router weights, the bias and x.
//
// EC-DiT: Scaling Diffusion Transformers with Adaptive Expert-Choice
// Routing, section 3: A = softmax(x W_r); a selected expert is weighted by
// its affinity A[s, e]. MMOE, "gate-residual routing": the logits take the
// previous layer's as a scaled term, so the next layer's gradient of that
// term (dz_next) reaches these logits beside the softmax.
//   dA = dprobs + scatter(dw),  dz = A (dA - <A, dA>) + dz_next
//   dx = dz W_r,  dW_r = dz^T x,  dbias = sum_s dz,  dz_prev = scale dz
//
// Two products with one narrow side (E <= 128) each: bound by reading x and
// writing dx once, not by their FLOPs. So after a per-token kernel for dz, a
// CTA owns 128 columns and a range of tokens: per 64-token tile it holds the
// x and W_r columns in shared memory, forms the dx tile (K = E) and adds to
// its dW_r block (K = 64 tokens), which stays in registers until the range
// ends. The token ranges' blocks are summed in order by a last launch.
// bf16 layers multiply on bf16 mma.sync (as the router's forward does: N = E
// is far too narrow for a tcgen05 tile). dz is fp32 and enters as the sum of
// three bf16 terms (8 mantissa bits each, 24 in all), so the products keep
// fp32 accuracy while x and W_r are exact. 8192 x 1152, 19 experts: 24.6 us, 22.6
// in a graph, where an elementwise kernel over as many bytes takes 7.7; launched
// apart and cold 7.4 + 19.7 + 6.0, the middle one with the tensor pipe 43 % and L1
// 64 % busy (three terms, experts padded to 32). The terms one after the other
// along K (4 steps of 16 instead of 6) took 24.6 us in a graph against 23.5 then.
#include "backward.h"
#include "chained.cuh"
#include "mma_sync.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int TT = 64;   // tokens per tile
constexpr int TC = 128;  // columns per CTA (bf16)
constexpr int FC = 64;   // columns per CTA (fp32)

// dz of one token per warp; lane holds experts lane + 32 v.
template <int VPL>
__global__ void __launch_bounds__(kThreads) router_dz_kernel(RouterBwdArgs a) {
  const int lane = threadIdx.x & 31;
  const bool ec = a.routing == MOE_EXPERT_CHOICE;
  const bool renorm = a.renorm && a.routing == MOE_TOKEN_TOPK;
  chain_next();
  for (int64_t s = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); s < a.T; s += (int64_t)gridDim.x * kWarps) {
    float A[VPL], dA[VPL], zn[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane + 32 * v;
      A[v] = e < a.E ? a.probs[s * a.E + e] : 0.f;
      dA[v] = (e < a.E && a.dprobs) ? a.dprobs[s * a.E + e] : 0.f;
      zn[v] = (e < a.E && a.dz_next) ? a.dz_next[s * a.E + e] : 0.f;
    }
    int64_t j0, j1;
    if (ec) {
      j0 = a.tok_ptr[s];
      j1 = a.tok_ptr[s + 1];
      if (j0 < 0 || j1 < j0 || j1 > a.n_assign) {
        if (lane == 0) set_status(a.dev_status, MOE_DEV_BAD_EXPERT);
        j0 = j1 = 0;
      }
    } else {
      j0 = s * a.k;
      j1 = j0 + a.k;
    }
    // Renormalised weights w = A / S: dA = (dw - sum dw w) / S.
    float inner = 0.f, inv = 1.f;
    if (renorm) {
      float S = 0.f;
      for (int64_t j = j0 + lane; j < j1; j += 32) {
        const int e = a.sel[j];
        if (e >= 0 && e < a.E) {
          S += a.probs[s * a.E + e];
          inner = fmaf(a.dw[j], a.w[j], inner);
        }
      }
      S = warp_sum(S);
      inner = warp_sum(inner);
      inv = 1.f / S;
    }
    for (int64_t b = j0; b < j1; b += 32) {
      int e = -1;
      float g = 0.f;
      if (b + lane < j1) {
        int64_t asg = b + lane;
        if (ec) {
          asg = a.tok_assign[asg];
          if (asg >= 0 && asg < a.n_assign) e = (int)((asg / a.C) % a.E);
        } else {
          e = a.sel[asg];
        }
        if (e >= 0 && e < a.E) g = (a.dw[asg] - inner) * inv;
        else if (ec || e != -1) set_status(a.dev_status, MOE_DEV_BAD_EXPERT);
        if (e >= a.E) e = -1;
      }
      const int n = (int)(j1 - b < 32 ? j1 - b : 32);
      for (int j = 0; j < n; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, j);
        const float gj = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          if (ej == lane + 32 * v) dA[v] += gj;
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) dot = fmaf(A[v], dA[v], dot);
    dot = warp_sum(dot);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int e = lane + 32 * v;
      if (e >= a.E) continue;
      float dz = A[v] * (dA[v] - dot);
      if (a.dz_next) dz += zn[v];
      a.dlogits[s * a.E + e] = dz;
      if (a.dz_prev) a.dz_prev[s * a.E + e] = a.zscale * dz;
    }
  }
}

// Four 8x8 blocks, each transposed: fragments of an operand stored K first.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], const void *p) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(s));
}
__device__ __forceinline__ void mma2(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[4], const uint32_t (&b)[4]) {
  mma_bf16_16816(c0, a, {b[0], b[1]});
  mma_bf16_16816(c1, a, {b[2], b[3]});
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// v[n] of lane q becomes v[q] of lane n, among four neighbouring lanes: swaps
// with the lane 1 away, then with the lane 2 away.
__device__ __forceinline__ void transpose4(uint32_t (&v)[4], int q) {
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
    const bool up = q & b;
#pragma unroll
    for (int n = 0; n < 4; ++n)
      if (!(n & b)) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[n] : v[n | b], b);
        if (up) v[n] = got;
        else v[n | b] = got;
      }
  }
}

// MT: E padded to 16 MT experts. Shared memory, bf16, rows padded by 8 to
// spread ldmatrix rows over the banks: two x tiles [TT][TC] (the next one
// is fetched while one is worked on), the W_r columns [16 MT][TC], dz as three
// terms [3][TT][16 MT].
template <int MT> struct RbSmem {
  static constexpr int EP = 16 * MT;
  static constexpr int XP = TC + 8, ZP = EP + 8;
  static constexpr size_t x = 0;  // two tiles
  static constexpr size_t w = x + (size_t)2 * TT * XP * 2;
  static constexpr size_t z = w + (size_t)EP * XP * 2;
  static constexpr size_t total = z + (size_t)3 * TT * ZP * 2;
};

template <int MT>
__global__ void __launch_bounds__(kThreads) router_bwd_bf16_kernel(RouterBwdArgs a, int splits, float *bias_part) {
  using S = RbSmem<MT>;
  constexpr int EP = S::EP, XP = S::XP, ZP = S::ZP;
  extern __shared__ __align__(16) uint8_t sm[];
  __nv_bfloat16 *sx0 = reinterpret_cast<__nv_bfloat16 *>(sm + S::x);
  __nv_bfloat16 *sw = reinterpret_cast<__nv_bfloat16 *>(sm + S::w);
  __nv_bfloat16 *sz = reinterpret_cast<__nv_bfloat16 *>(sm + S::z);
  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x);
  const __nv_bfloat16 *wr = static_cast<const __nv_bfloat16 *>(a.W_r);
  __nv_bfloat16 *dx = static_cast<__nv_bfloat16 *>(a.dx);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c0 = blockIdx.x * TC, split = blockIdx.y;
  const int tiles = (a.T + TT - 1) / TT;
  const int t_lo = (int)((int64_t)tiles * split / splits), t_hi = (int)((int64_t)tiles * (split + 1) / splits);
  const bool want_w = a.dW_r != nullptr, want_x = dx != nullptr;

  if (want_x)
    for (int i = tid; i < EP * (TC / 8); i += kThreads) {
      const int e = i / (TC / 8), c = (i % (TC / 8)) * 8;
      const bool in = e < a.E && c0 + c < a.d;
      cp_async16(sw + e * XP + c, in ? wr + (size_t)e * a.d + c0 + c : wr, in);
    }
  float acc[MT][2][4];  // dW_r: all 16 MT experts x this warp's 16 columns
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
  auto fetch_x = [&](int t) {
    __nv_bfloat16 *o = sx0 + (t & 1) * TT * XP;
    if (want_w && t < t_hi)
      for (int i = tid; i < TT * (TC / 8); i += kThreads) {
        const int r = t * TT + i / (TC / 8), c = (i % (TC / 8)) * 8;
        const bool in = r < a.T && c0 + c < a.d;
        cp_async16(o + (i / (TC / 8)) * XP + c, in ? x + (size_t)r * a.d + c0 + c : x, in);
      }
    cp_async_commit();
  };
  // dz of a tile, read a tile ahead.
  constexpr int ZN = TT * EP / kThreads;
  float zr[ZN];
  auto fetch_z = [&](int t) {
#pragma unroll
    for (int i = 0; i < ZN; ++i) {
      const int r = t * TT + (tid + i * kThreads) / EP, e = (tid + i * kThreads) % EP;
      zr[i] = (t < t_hi && r < a.T && e < a.E) ? a.dlogits[(size_t)r * a.E + e] : 0.f;
    }
  };
  // A thread's zr are all of one expert (EP divides kThreads): column block 0
  // sums them for dbias.
  const bool want_b = a.dbias && blockIdx.x == 0;
  float bias_sum = 0.f;
  fetch_x(t_lo);
  chain_wait();
  chain_next();
  fetch_z(t_lo);
  for (int t = t_lo; t < t_hi; ++t) {
    const int s0 = t * TT;
    __nv_bfloat16 *sx = sx0 + (t & 1) * TT * XP;
    __syncthreads();  // the last tile's dz and the other x tile have been read
    fetch_x(t + 1);
#pragma unroll
    for (int i = 0; i < ZN; ++i) {
      const int r = (tid + i * kThreads) / EP, e = (tid + i * kThreads) % EP;
      const __nv_bfloat16 h = __float2bfloat16_rn(zr[i]);
      const float z1 = zr[i] - __bfloat162float(h);
      const __nv_bfloat16 m = __float2bfloat16_rn(z1);
      sz[r * ZP + e] = h;
      sz[(TT + r) * ZP + e] = m;
      sz[(2 * TT + r) * ZP + e] = __float2bfloat16_rn(z1 - __bfloat162float(m));
      bias_sum += zr[i];
    }
    fetch_z(t + 1);
    cp_async_wait<1>();
    __syncthreads();
    if (want_w) {
      // dW_r[e][c] += sum_r dz[r][e] x[r][c]: A = dz^T (ldmatrix.trans on
      // [token][expert] rows), B = x (ldmatrix.trans on [token][column] rows).
      // A tile's sums are formed on their own and then added in fp32: the
      // tensor cores cut their sums off instead of rounding them, which over
      // 65536 tokens of one sign left dW_r 4e-5 too small in one long chain.
      constexpr int MG = MT < 2 ? MT : 2;  // experts in 16s at a time
      uint32_t b[TT / 16][4];              // columns 16 warp + {0..7, 8..15}, k halves
#pragma unroll
      for (int m0 = 0; m0 < MT; m0 += MG) {
        float t[MG][2][4];
#pragma unroll
        for (int m = 0; m < MG; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) t[m][n][i] = 0.f;
#pragma unroll
        for (int k = 0; k < TT; k += 16) {
          if (m0 == 0) ldmatrix_x4_trans(b[k / 16], sx + (k + (lane & 15)) * XP + warp * 16 + (lane >> 4) * 8);
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int m = 0; m < MG; ++m) {
              uint32_t f[4];
              ldmatrix_x4_trans(f, sz + (p * TT + k + (lane & 7) + ((lane >> 4) << 3)) * ZP + (m0 + m) * 16 +
                                       ((lane >> 3) & 1) * 8);
              mma2(t[m][0], t[m][1], f, b[k / 16]);
            }
        }
#pragma unroll
        for (int m = 0; m < MG; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m0 + m][n][i] += t[m][n][i];
      }
    }
    if (want_x) {
      // dx[r][c] = sum_e dz[r][e] W_r[e][c]: warp (rows 16 (warp & 3), columns 64 (warp >> 2)).
      float o[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
      const int r0 = (warp & 3) * 16, cw = (warp >> 2) * 64;
#pragma unroll
      for (int k = 0; k < EP; k += 16) {
        uint32_t f[3][4];
#pragma unroll
        for (int p = 0; p < 3; ++p)
          ldmatrix_x4(f[p], sz + (p * TT + r0 + (lane & 15)) * ZP + k + (lane >> 4) * 8);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          uint32_t b[4];
          ldmatrix_x4_trans(b, sw + (k + (lane & 15)) * XP + cw + n * 8 + (lane >> 4) * 8);
#pragma unroll
          for (int p = 0; p < 3; ++p) mma2(o[n], o[n + 1], f[p], b);
        }
      }
      // A lane holds two columns of every 8: the four lanes of a row trade
      // them for whole 16-byte pieces, lane q those of block 4 g + q.
      const int q = lane & 3;
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) v[n] = pack_bf16(o[4 * g + n][2 * half], o[4 * g + n][2 * half + 1]);
          transpose4(v, q);
          const int r = s0 + r0 + (lane >> 2) + 8 * half, c = c0 + cw + (4 * g + q) * 8;
          if (r < a.T && c < a.d) *reinterpret_cast<uint4 *>(dx + (size_t)r * a.d + c) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
  }
  if (want_w) {
    float *p = a.part + (size_t)split * a.E * a.d;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int e = m * 16 + (lane >> 2), c = c0 + warp * 16 + n * 8 + (lane & 3) * 2;
        if (c < a.d) {  // d is a multiple of 8, so c + 1 < d too
          if (e < a.E) *reinterpret_cast<float2 *>(p + (size_t)e * a.d + c) = make_float2(acc[m][n][0], acc[m][n][1]);
          if (e + 8 < a.E)
            *reinterpret_cast<float2 *>(p + (size_t)(e + 8) * a.d + c) = make_float2(acc[m][n][2], acc[m][n][3]);
        }
      }
  }
  if (want_b) {
    __shared__ float sb[kThreads];
    sb[tid] = bias_sum;
    __syncthreads();
    if (tid < a.E) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kThreads / EP; ++k) t += sb[k * EP + tid];
      bias_part[(size_t)split * a.E + tid] = t;
    }
  }
}

// The same tiles in fp32 on CUDA cores (fp32 layers are small). A thread owns
// a column and every fourth expert (EPT of them) or row. A tile's sums are
// formed on their own and then added: shorter chains of rounding.
template <int EPT>
__global__ void __launch_bounds__(kThreads) router_bwd_f32_kernel(RouterBwdArgs a, int splits, float *bias_part) {
  extern __shared__ __align__(16) float fm[];
  float *sx = fm;             // [TT][FC]
  float *sw = sx + TT * FC;   // [E][FC]
  float *sz = sw + a.E * FC;  // [TT][E]
  const float *x = static_cast<const float *>(a.x);
  const float *wr = static_cast<const float *>(a.W_r);
  float *dx = static_cast<float *>(a.dx);
  const int tid = threadIdx.x, c0 = blockIdx.x * FC, split = blockIdx.y;
  const int tiles = (a.T + TT - 1) / TT;
  const int t_lo = (int)((int64_t)tiles * split / splits), t_hi = (int)((int64_t)tiles * (split + 1) / splits);
  const int col = tid % FC, lane4 = tid / FC;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  if (dx)
    for (int i = tid; i < a.E * (FC / 4); i += kThreads) {
      const int e = i / (FC / 4), c = c0 + (i % (FC / 4)) * 4;
      *reinterpret_cast<float4 *>(sw + i * 4) =
          c < a.d ? *reinterpret_cast<const float4 *>(wr + (size_t)e * a.d + c) : zero;
    }
  chain_wait();
  chain_next();
  const bool want_b = a.dbias && blockIdx.x == 0;
  float bias_sum[16];  // experts warp + 8 i, in lane 0
#pragma unroll
  for (int i = 0; i < 16; ++i) bias_sum[i] = 0.f;
  float acc[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) acc[i] = 0.f;
  for (int t = t_lo; t < t_hi; ++t) {
    const int s0 = t * TT;
    __syncthreads();
    if (a.dW_r) {
      float4 v[TT * FC / 4 / kThreads];
#pragma unroll
      for (int k = 0; k < TT * FC / 4 / kThreads; ++k) {
        const int i = tid + k * kThreads, r = s0 + i / (FC / 4), c = c0 + (i % (FC / 4)) * 4;
        v[k] = r < a.T && c < a.d ? *reinterpret_cast<const float4 *>(x + (size_t)r * a.d + c) : zero;
      }
#pragma unroll
      for (int k = 0; k < TT * FC / 4 / kThreads; ++k) *reinterpret_cast<float4 *>(sx + (tid + k * kThreads) * 4) = v[k];
    }
    const int live = min(TT, a.T - s0) * a.E;
#pragma unroll 4
    for (int i = tid; i < TT * a.E; i += kThreads) sz[i] = i < live ? a.dlogits[(size_t)s0 * a.E + i] : 0.f;
    __syncthreads();
    if (want_b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = (tid >> 5) + 8 * i;
        if (e < a.E) bias_sum[i] += warp_sum(sz[(tid & 31) * a.E + e] + sz[((tid & 31) + 32) * a.E + e]);
      }
    }
    if (a.dW_r) {
      float v[EPT];
#pragma unroll
      for (int i = 0; i < EPT; ++i) v[i] = 0.f;
#pragma unroll 8
      for (int r = 0; r < TT; ++r) {
        const float xv = sx[r * FC + col];
#pragma unroll
        for (int i = 0; i < EPT; ++i)
          if (lane4 + 4 * i < a.E) v[i] = fmaf(sz[r * a.E + lane4 + 4 * i], xv, v[i]);
      }
#pragma unroll
      for (int i = 0; i < EPT; ++i) acc[i] += v[i];
    }
    if (dx && c0 + col < a.d) {
      float v[TT / 4];
#pragma unroll
      for (int i = 0; i < TT / 4; ++i) v[i] = 0.f;
      for (int e = 0; e < a.E; ++e) {
        const float w = sw[e * FC + col];
#pragma unroll
        for (int i = 0; i < TT / 4; ++i) v[i] = fmaf(sz[(lane4 + 4 * i) * a.E + e], w, v[i]);
      }
#pragma unroll
      for (int i = 0; i < TT / 4; ++i)
        if (s0 + lane4 + 4 * i < a.T) dx[(size_t)(s0 + lane4 + 4 * i) * a.d + c0 + col] = v[i];
    }
  }
  if (a.dW_r && c0 + col < a.d) {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int e = lane4 + 4 * i;
      if (e < a.E) a.part[((size_t)split * a.E + e) * a.d + c0 + col] = acc[i];
    }
  }
  if (want_b && (tid & 31) == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = (tid >> 5) + 8 * i;
      if (e < a.E) bias_part[(size_t)split * a.E + e] = bias_sum[i];
    }
  }
}

// Sums the token ranges in order: dW_r [E, d], and dbias [E] in the last
// block. 64 values by 16 slices of the list per CTA, the slices added in order.
constexpr int kSumSlices = 16, kSumCols = 64, kSumThreads = kSumCols * kSumSlices / 4;
__global__ void __launch_bounds__(kSumThreads) router_bwd_sum_kernel(const float *part, const float *bias_part,
                                                                     float *dW_r, float *dbias, int E, int d,
                                                                     int splits) {
  __shared__ __align__(16) float sh[kSumSlices][kSumCols];
  chain_wait();
  const int64_t nw = dW_r ? (int64_t)E * d : 0, c0 = (int64_t)blockIdx.x * kSumCols;
  if (c0 >= nw) {  // dbias: a thread per expert and slice of the list
    const int width = E <= 32 ? 32 : E <= 64 ? 64 : 128, slices = kSumThreads / width;
    const int e = threadIdx.x % width, slice = threadIdx.x / width;
    float t = 0.f;
    if (e < E)
#pragma unroll 16
      for (int k = splits * slice / slices; k < splits * (slice + 1) / slices; ++k) t += bias_part[(size_t)k * E + e];
    float *o = &sh[0][0];
    o[threadIdx.x] = t;
    __syncthreads();
    if ((int)threadIdx.x >= E) return;
    for (int k = 1; k < slices; ++k) t += o[k * width + threadIdx.x];
    dbias[threadIdx.x] = t;
    return;
  }
  const int quad = threadIdx.x % (kSumCols / 4), slice = threadIdx.x / (kSumCols / 4);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c0 + quad * 4 < nw) {
    const int lo = splits * slice / kSumSlices, hi = splits * (slice + 1) / kSumSlices;
#pragma unroll 4
    for (int k = lo; k < hi; ++k) {
      const float4 f = *reinterpret_cast<const float4 *>(part + (size_t)k * nw + c0 + quad * 4);
      v.x += f.x;
      v.y += f.y;
      v.z += f.z;
      v.w += f.w;
    }
  }
  *reinterpret_cast<float4 *>(&sh[slice][quad * 4]) = v;
  __syncthreads();
  const int64_t i = c0 + threadIdx.x;
  if (threadIdx.x >= kSumCols || i >= nw) return;
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < kSumSlices; ++k) t += sh[k][threadIdx.x];
  dW_r[i] = t;
}

// Token ranges: as many CTAs with the columns as run at once (two per SM), at least one tile
// each, and no more partial dW_r blocks than half the bytes of x. The SMs are counted as the
// B200's 148, not asked for: the ranges size the workspace, which has to be the same on a
// host without a GPU, and fix the order of the sums.
int token_splits(int T, int d, int E, int dtype) {
  const int cols = dtype == MOE_BF16 ? TC : FC, eb = dtype == MOE_BF16 ? 2 : 4;
  const int64_t tiles = (T + TT - 1) / TT, blocks = (d + cols - 1) / cols;
  int64_t n = 2 * 148 / blocks;
  const int64_t cap = (int64_t)T * eb / (8 * (int64_t)E);
  if (n > cap) n = cap;
  if (n > tiles) n = tiles;
  return (int)(n < 1 ? 1 : n);
}

template <int MT>
int run_bf16(const RouterBwdArgs &a, int splits, float *bias_part, cudaStream_t stream) {
  const dim3 grid((a.d + TC - 1) / TC, splits);
  MOE_CUDA_TRY(cudaFuncSetAttribute(router_bwd_bf16_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)RbSmem<MT>::total));
  launch_chained(router_bwd_bf16_kernel<MT>, grid, kThreads, RbSmem<MT>::total, stream, a, splits, bias_part);
  return last_launch_status();
}

}  // namespace

size_t router_bwd_workspace_bytes(int T, int d, int E, int dtype) {
  return (size_t)token_splits(T, d, E, dtype) * ((size_t)E * d + E) * 4;
}

int launch_router_bwd(const RouterBwdArgs &a, cudaStream_t stream) {
  const int splits = token_splits(a.T, a.d, a.E, a.dtype);
  float *bias_part = a.part + (size_t)splits * a.E * a.d;
  if (a.T > 0) {
    int64_t blocks = ((int64_t)a.T + kWarps - 1) / kWarps;
    if (blocks > 8 * (int64_t)num_sms()) blocks = 8 * (int64_t)num_sms();
    const unsigned g = (unsigned)blocks;
    if (a.E <= 32) router_dz_kernel<1><<<g, kThreads, 0, stream>>>(a);
    else if (a.E <= 64) router_dz_kernel<2><<<g, kThreads, 0, stream>>>(a);
    else router_dz_kernel<4><<<g, kThreads, 0, stream>>>(a);
  }
  int st = last_launch_status();
  if (st == MOE_OK && (a.dx || a.dW_r || a.dbias)) {
    if (a.dtype == MOE_BF16) {
      if (a.E <= 16) st = run_bf16<1>(a, splits, bias_part, stream);
      else if (a.E <= 32) st = run_bf16<2>(a, splits, bias_part, stream);
      else if (a.E <= 64) st = run_bf16<4>(a, splits, bias_part, stream);
      else st = run_bf16<8>(a, splits, bias_part, stream);
    } else {
      const auto bytes = [](int E) { return (size_t)(TT * FC + TT * E + E * FC) * 4; };
      const int ept = a.E <= 8 ? 2 : a.E <= 32 ? 8 : 32;
      const auto kern = ept == 2 ? router_bwd_f32_kernel<2> : ept == 8 ? router_bwd_f32_kernel<8> : router_bwd_f32_kernel<32>;
      const size_t smem = bytes(a.E);
      // The limit is the variant's, not the call's: another host thread must not lower it before the launch.
      MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(4 * ept)));
      launch_chained(kern, dim3((a.d + FC - 1) / FC, splits), kThreads, smem, stream, a, splits, bias_part);
      st = last_launch_status();
    }
  }
  if (st != MOE_OK || (!a.dW_r && !a.dbias)) return st;
  const int64_t blocks = (a.dW_r ? ((int64_t)a.E * a.d + kSumCols - 1) / kSumCols : 0) + (a.dbias ? 1 : 0);
  launch_chained(router_bwd_sum_kernel, (unsigned)blocks, kSumThreads, 0, stream, a.part, bias_part, a.dW_r, a.dbias,
                 a.E, a.d, splits);
  return last_launch_status();
}

}  // namespace moe
