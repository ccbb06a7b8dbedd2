// Launch interface of the backward kernels and the block norms, between the
// C ABI (backward_api.cu) and their translation units. Launchers enqueue on
// `stream`, return a moe_status and never synchronise the host.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

// moe_api.cu: the checks and counts every entry point shares.
int check_config(const moe_config *c);
int64_t n_assign_of(const moe_config &c);
int n_const_of(const moe_config &c);
KindTable kind_table(const moe_config &c);

// exchange_bwd.cu
struct ExchangeBwdArgs {
  int routing, T, d, E, k, S, C, dtype, const_mix, n_const;
  int64_t n_assign;
  const int32_t *sel;
  const float *w;
  const int32_t *row_of, *tok_ptr, *tok_assign;
  const void *x, *const_vecs;
  const void *dy;
  // combine
  const void *y_perm;
  void *dy_perm;
  float *dw, *dconst;
  float *const_part;  // workspace of const_grad_workspace_bytes(): chunk sums, then
  float2 *const_coef; // (set by the launcher) w a1 and q of each assignment
  // dispatch
  const void *dx_perm;
  const void *add[3];
  void *dx;
  int32_t *dev_status;
};
size_t const_grad_workspace_bytes(int64_t n_assign, int n_const, int d, int const_mix);
int launch_combine_bwd(const ExchangeBwdArgs &a, const KindTable &kinds, cudaStream_t stream);
int launch_dispatch_bwd(const ExchangeBwdArgs &a, const KindTable &kinds, cudaStream_t stream);

// router_bwd.cu
struct RouterBwdArgs {
  int routing, T, d, E, k, C, dtype, renorm;
  int64_t n_assign;
  float zscale;
  const void *x, *W_r;
  const float *probs, *w, *dw, *dprobs, *dz_next;
  const int32_t *sel, *tok_ptr, *tok_assign;
  float *dlogits, *dz_prev, *dbias, *dW_r;
  void *dx;
  float *part;  // workspace of router_bwd_workspace_bytes()
  int32_t *dev_status;
};
size_t router_bwd_workspace_bytes(int T, int d, int E, int dtype);
int launch_router_bwd(const RouterBwdArgs &a, cudaStream_t stream);

// The grouped MLP's gradient for one set of experts (the routed ones over
// ragged row groups, or the shared one over all tokens).
struct MlpBwdProblem {
  int64_t rows;            // rows of x and dy (an upper bound of the groups' rows)
  int n_groups;
  const int32_t *offsets;  // [n_groups + 1] device row offsets, or NULL: one group of `rows`
  int d, h, gated;
  const void *x, *dy, *W1, *W2;
  void *dx, *dW1, *dW2;    // nullable
  void *H, *dU;            // workspace: [rows, h], [rows, gated ? 2h : h] in the layer dtype
  void *U;                 // workspace of the fp32 path: [rows, gated ? 2h : h] fp32
  int32_t *status;
};
// mlp_bwd_f32.cu: fp32 layers, on CUDA cores, one problem after the other.
int launch_mlp_bwd_f32(const MlpBwdProblem *p, int n, cudaStream_t stream);
// mlp_bwd_sm100.cu: bf16 layers on tcgen05, up to two problems in each launch.
int launch_mlp_bwd_bf16(const MlpBwdProblem *q, int n, int32_t *status, cudaStream_t stream);

// block_norm.cu
struct BlockNormArgs {
  int T, d, group;  // group >= 1: tokens per condition row
  int pre, post;    // moe_norm_kind
  float eps, res_scale;
  const void *h, *x, *post_gamma, *gate, *pre_gamma, *pre_beta, *scale, *shift;
  int64_t cond_stride;
  void *y, *z;
  // backward
  const void *yin, *dz, *dy;
  void *dh, *dx;
  float *dpost_gamma, *dgate, *dpre_gamma, *dpre_beta, *dscale, *dshift;
  int64_t dcond_stride;
  float *part;  // workspace of block_norm_workspace_bytes()
};
constexpr int kNormMaxWidth = 8192;
size_t block_norm_workspace_bytes(int T, int d, int group, int dtype);
int launch_block_norm(const BlockNormArgs &a, int dtype, cudaStream_t stream);
int launch_block_norm_bwd(const BlockNormArgs &a, int dtype, cudaStream_t stream);

}  // namespace moe
