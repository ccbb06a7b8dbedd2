// Gradient of the grouped expert MLP in fp32 on CUDA cores, for fp32 layers
// (the tensor cores' fp32-input mode is tf32, which would not meet an fp32
// tolerance).
//
// MMOE: Modernizing Diffusion Transformers with Efficient Expert Design,
// "MoE++ expert layer": heavy experts are standard MLPs. With U = X W1^T,
// H = act(U) per expert:
//   dH = dY W2, dU = dH act'(U), dX = dU W1, dW2 = dY^T H, dW1 = dU^T X.
// One tiled product serves all five: A and B each stored with K or with
// their other dimension contiguous, and either the rows of the output
// (activations) or K (weight gradients) ragged over the row groups.
// Each K tile's products are summed on their own and then added to the
// running sum, which shortens the chains of rounding for long K.
#include "backward.h"
#include "chained.cuh"

namespace moe {
namespace {

constexpr int kBM = 64, kBN = 64, kBK = 16, kThreads = 256;
enum Epi { kStore, kStoreU, kActGrad };

struct Gemm {
  const void *A, *B;
  int64_t lda, ldb, b_group;  // row strides; elements between the groups' B (0: ragged K)
  int M, N, K;                // M (ragged K) or K (ragged M) is per group; the ragged one is unused
  const int32_t *offsets;
  int n_groups;
  int64_t rows;
  void *out;                  // kStore: [.., N]; ragged K: [n_groups][M][N]
  float *U;                   // kStoreU out, kActGrad in: [rows, gated ? 2N : N]
  void *H, *dU;               // kActGrad out
  int gated;
  int32_t *status;
};

// A_T: A is [K][M]; B_T: B is [N][K] (else [K][N]). RAGGED_K: the groups'
// rows are K, else they are the rows of the output.
template <bool A_T, bool B_T, bool RAGGED_K, int EPI>
__global__ void __launch_bounds__(kThreads) mlp_bwd_gemm_kernel(Gemm p) {
  __shared__ float As[kBK][kBM + 4];
  __shared__ float Bs[kBK][kBN + 4];
  __shared__ int s_group;
  __shared__ int64_t s_lo, s_hi;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  if (tid == 0) {
    int g = -1;
    int64_t r0 = 0, r1 = 0, t = blockIdx.y;
    for (int gi = RAGGED_K ? (int)blockIdx.z : 0; gi < p.n_groups; ++gi) {
      int64_t lo = p.offsets ? p.offsets[gi] : 0, hi = p.offsets ? p.offsets[gi + 1] : p.rows;
      check_group_rows(lo, hi, p.rows, p.status);
      const int64_t mt = (hi - lo + kBM - 1) / kBM;
      if (RAGGED_K || t < mt) { g = gi; r0 = RAGGED_K ? lo : lo + t * kBM; r1 = hi; break; }
      t -= mt;
    }
    s_group = g; s_lo = r0; s_hi = r1;
  }
  chain_next();
  chain_wait();
  __syncthreads();
  const int g = s_group;
  if (g < 0) return;
  const int64_t lo = s_lo, hi = s_hi;
  const float *A = static_cast<const float *>(p.A), *B = static_cast<const float *>(p.B) + (RAGGED_K ? 0 : g * p.b_group);
  const int n0 = blockIdx.x * kBN, m0 = RAGGED_K ? blockIdx.y * kBM : 0;
  const int64_t K = RAGGED_K ? hi - lo : p.K;

  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += kBK) {
    for (int i = tid; i < kBM * kBK; i += kThreads) {
      // Consecutive threads read along the contiguous dimension.
      const int ka = A_T ? i / kBM : i % kBK, m = A_T ? i % kBM : i / kBK;
      const int kb = B_T ? i % kBK : i / kBN, n = B_T ? i / kBK : i % kBN;
      float a = 0.f, b = 0.f;
      if (k0 + ka < K) {
        if (RAGGED_K) {
          if (m0 + m < p.M) a = A[(lo + k0 + ka) * p.lda + m0 + m];
        } else if (lo + m < hi) {
          a = A[(lo + m) * p.lda + k0 + ka];
        }
      }
      if (k0 + kb < K && n0 + n < p.N)
        b = B_T ? B[(int64_t)(n0 + n) * p.ldb + k0 + kb] : B[((RAGGED_K ? lo : 0) + k0 + kb) * p.ldb + n0 + n];
      As[ka][m] = a;
      Bs[kb][n] = b;
    }
    __syncthreads();
    float part[4][4] = {};
#pragma unroll
    for (int kk = 0; kk < kBK; ++kk) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = As[kk][ty * 4 + i];
        b[i] = Bs[kk][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(a[i], b[j], part[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += part[i][j];
    __syncthreads();
  }
  float *out = static_cast<float *>(p.out);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = (RAGGED_K ? m0 : lo) + ty * 4 + i;
    if (RAGGED_K ? r >= p.M : r >= hi) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= p.N) continue;
      const float v = acc[i][j];
      if (EPI == kStore) {
        out[((RAGGED_K ? (int64_t)g * p.M : 0) + r) * p.N + n] = v;
      } else if (EPI == kStoreU) {
        p.U[r * p.N + n] = v;
      } else {
        float *H = static_cast<float *>(p.H) + r * p.N + n;
        if (p.gated) {
          const float *u = p.U + r * 2 * p.N + n;
          float *dU = static_cast<float *>(p.dU) + r * 2 * p.N + n;
          const float a = u[0], b = u[p.N], sg = 1.0f / (1.0f + expf(-a));
          *H = a * sg * b;
          dU[0] = v * b * (sg * (1.0f + a * (1.0f - sg)));
          dU[p.N] = v * (a * sg);
        } else {
          const float u = p.U[r * p.N + n], phi = normcdff(u);
          *H = u * phi;
          static_cast<float *>(p.dU)[r * p.N + n] = v * fmaf(u * 0.3989422804f, expf(-0.5f * u * u), phi);
        }
      }
    }
  }
}

inline unsigned tiles(int n) { return (unsigned)(((int64_t)n + kBN - 1) / kBN); }
inline int64_t row_tiles(const MlpBwdProblem &p) {
  return (p.rows + kBM - 1) / kBM + (p.offsets ? p.n_groups : 0);
}

int run(const MlpBwdProblem &p, cudaStream_t stream) {
  const int up = p.gated ? 2 * p.h : p.h;
  const int64_t mt = row_tiles(p);
  Gemm g{};
  g.offsets = p.offsets; g.n_groups = p.n_groups; g.rows = p.rows; g.gated = p.gated; g.status = p.status;
  g.U = static_cast<float *>(p.U); g.H = p.H; g.dU = p.dU;
  bool chained = false;
  auto launch = [&](void (*kern)(Gemm), dim3 grid, const Gemm &q) {
    if (chained) launch_chained(kern, grid, kThreads, 0, stream, q);
    else kern<<<grid, kThreads, 0, stream>>>(q);
    chained = true;
  };
  if (p.rows > 0) {
    Gemm a = g;  // U = X W1^T
    a.A = p.x; a.lda = p.d; a.B = p.W1; a.ldb = p.d; a.b_group = (int64_t)up * p.d; a.N = up; a.K = p.d;
    launch(mlp_bwd_gemm_kernel<false, true, false, kStoreU>, dim3(tiles(up), (unsigned)mt), a);
    Gemm b = g;  // dH = dY W2, then H and dU
    b.A = p.dy; b.lda = p.d; b.B = p.W2; b.ldb = p.h; b.b_group = (int64_t)p.h * p.d; b.N = p.h; b.K = p.d;
    launch(mlp_bwd_gemm_kernel<false, false, false, kActGrad>, dim3(tiles(p.h), (unsigned)mt), b);
    if (p.dx) {
      Gemm c = g;  // dX = dU W1
      c.A = p.dU; c.lda = up; c.B = p.W1; c.ldb = p.d; c.b_group = (int64_t)up * p.d; c.N = p.d; c.K = up;
      c.out = p.dx;
      launch(mlp_bwd_gemm_kernel<false, false, false, kStore>, dim3(tiles(p.d), (unsigned)mt), c);
    }
  }
  if (p.dW2) {
    Gemm w = g;  // dW2 = dY^T H
    w.A = p.dy; w.lda = p.d; w.B = p.H; w.ldb = p.h; w.M = p.d; w.N = p.h; w.out = p.dW2;
    launch(mlp_bwd_gemm_kernel<true, false, true, kStore>, dim3(tiles(p.h), tiles(p.d), p.n_groups), w);
  }
  if (p.dW1) {
    Gemm w = g;  // dW1 = dU^T X
    w.A = p.dU; w.lda = up; w.B = p.x; w.ldb = p.d; w.M = up; w.N = p.d; w.out = p.dW1;
    launch(mlp_bwd_gemm_kernel<true, false, true, kStore>, dim3(tiles(p.d), tiles(up), p.n_groups), w);
  }
  return last_launch_status();
}

}  // namespace

int launch_mlp_bwd_f32(const MlpBwdProblem *p, int n, cudaStream_t stream) {
  for (int i = 0; i < n; ++i)  // grid.y; before either launches
    if (row_tiles(p[i]) > 65535 || tiles(p[i].gated ? 2 * p[i].h : p[i].h) > 65535 || tiles(p[i].d) > 65535)
      return MOE_ERR_UNSUPPORTED;
  int st = MOE_OK;
  for (int i = 0; i < n && st == MOE_OK; ++i) st = run(p[i], stream);
  return st;
}

}  // namespace moe
