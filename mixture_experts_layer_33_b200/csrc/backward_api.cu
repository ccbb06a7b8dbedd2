// The C ABI of the gradients and the block norms (declared in
// include/moe.h): argument checks, workspace layout, launches.
#include <math.h>

#include "backward.h"

namespace moe {
namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... P>
bool all_aligned16(P... p) {
  return (aligned16(p) && ...);
}

// The kernels count rows and tiles in 32 bits, a tile past the last row too.
constexpr int64_t kMaxRows = 1 << 30;
int check_bwd_config(const moe_config *cfg) {
  const int st = check_config(cfg);
  if (st != MOE_OK) return st;
  const int64_t w1_rows = (int64_t)cfg->n_heavy * cfg->h * (cfg->act == MOE_SWIGLU ? 2 : 1);
  const int64_t shared = (int64_t)cfg->n_shared * cfg->h_shared;
  if (cfg->T > kMaxRows || n_assign_of(*cfg) > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return (cfg->n_heavy > 0 && w1_rows > kMaxRows) || shared > kMaxRows ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Whether two buffers of `bytes` bytes share any.
inline bool overlap(const void *a, const void *b, size_t bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return (p < q ? q - p : p - q) < bytes;
}

// One workspace for the backward entry points, which run one after
// another: each takes it from the start.
struct BwdLayout {
  size_t H, dU, Hs, dUs, U, total;  // grouped MLP (routed, shared); the others use it whole
};
BwdLayout bwd_layout(const moe_config &c) {
  BwdLayout L;
  const size_t eb = c.dtype == MOE_BF16 ? 2 : 4, up = c.act == MOE_SWIGLU ? 2 : 1;
  const size_t r = c.n_heavy > 0 ? (size_t)n_assign_of(c) * c.h : 0;
  const size_t s = (size_t)c.T * c.n_shared * c.h_shared;
  size_t o = kAlign;
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes); return at; };
  L.H = take(r * eb);
  L.dU = take(up * r * eb);
  L.Hs = take(s * eb);
  L.dUs = take(s * eb);
  // The fp32 path keeps U too, of the routed and the shared part in turn.
  L.U = take(c.dtype == MOE_F32 ? (up * r > s ? up * r : s) * 4 : 0);
  const size_t cg = const_grad_workspace_bytes(n_assign_of(c), n_const_of(c), c.d, c.const_mix);
  const size_t rt = router_bwd_workspace_bytes(c.T, c.d, c.E, c.dtype);
  if (o < kAlign + align_up(cg)) o = kAlign + align_up(cg);
  if (o < kAlign + align_up(rt)) o = kAlign + align_up(rt);
  L.total = o;
  return L;
}

int check_bwd_ws(size_t need, void *ws, size_t ws_bytes) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return MOE_ERR_INVALID_ARG;
  return ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}
template <typename T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<uint8_t *>(ws) + off);
}

bool has_kind(const moe_config &c, int kind) {
  for (int e = 0; e < c.E; ++e)
    if (c.expert_kind[e] == kind) return true;
  return false;
}

ExchangeBwdArgs exchange_args(const moe_config &c, const int32_t *sel, const float *w, const int32_t *row_of,
                              const int32_t *tok_ptr, const int32_t *tok_assign, const void *x, const void *const_vecs,
                              const void *dy, int32_t *dev_status) {
  ExchangeBwdArgs a{};
  a.routing = c.routing; a.T = c.T; a.d = c.d; a.E = c.E; a.k = c.k; a.S = c.group_size; a.C = c.capacity;
  a.dtype = c.dtype; a.const_mix = c.const_mix; a.n_const = n_const_of(c); a.n_assign = n_assign_of(c);
  a.sel = sel; a.w = w; a.row_of = row_of; a.tok_ptr = tok_ptr; a.tok_assign = tok_assign;
  a.x = x; a.const_vecs = const_vecs; a.dy = dy; a.dev_status = dev_status;
  return a;
}

int check_norm(const moe_norm_config *c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_BF16 && c->dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (c->T < 0 || c->d < 8 || c->d % 8 != 0 || c->group_size < 0) return MOE_ERR_INVALID_ARG;
  if (c->d > kNormMaxWidth || c->T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  for (int k : {c->pre_kind, c->post_kind})
    if (k != MOE_NORM_NONE && k != MOE_NORM_LAYER && k != MOE_NORM_RMS) return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.f) || !isfinite(c->eps) || !isfinite(c->res_scale)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
inline int norm_group(const moe_norm_config &c) { return c.group_size > 0 ? c.group_size : (c.T > 0 ? c.T : 1); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_backward_workspace_size(const moe_config *cfg, size_t *bytes) {
  const int st = check_bwd_config(cfg);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = bwd_layout(*cfg).total;
  return MOE_OK;
}

int moe_combine_backward(const moe_config *cfg, const void *dy, const void *y_perm, const int32_t *sel, const float *w,
                         const int32_t *row_of, const void *x, const void *const_vecs, void *dy_perm, float *dw,
                         float *dconst, int32_t *dev_status, void *ws, size_t ws_bytes, moe_stream_t stream) {
  int st = check_bwd_config(cfg);
  if (st != MOE_OK) return st;
  const moe_config &c = *cfg;
  const int n_const = n_const_of(c);
  if (n_assign_of(c) > 0) {
    if (!dy || !sel || !w || !row_of || !dw) return MOE_ERR_INVALID_ARG;
    if (c.n_heavy > 0 && (!y_perm || !dy_perm)) return MOE_ERR_INVALID_ARG;
    if ((has_kind(c, MOE_IDENTITY) || (n_const > 0 && c.const_mix)) && !x) return MOE_ERR_INVALID_ARG;
    if (n_const > 0 && !const_vecs) return MOE_ERR_INVALID_ARG;
  }
  if (!all_aligned16(dy, y_perm, x, const_vecs, dy_perm, dconst)) return MOE_ERR_INVALID_ARG;
  if ((st = check_bwd_ws(bwd_layout(c).total, ws, ws_bytes)) != MOE_OK) return st;
  ExchangeBwdArgs a = exchange_args(c, sel, w, row_of, nullptr, nullptr, x, const_vecs, dy, dev_status);
  a.y_perm = y_perm; a.dy_perm = dy_perm; a.dw = dw; a.dconst = n_const > 0 ? dconst : nullptr;
  a.const_part = at<float>(ws, kAlign);
  return launch_combine_bwd(a, kind_table(c), stream);
}

int moe_dispatch_backward(const moe_config *cfg, const void *dx_perm, const void *dy, const int32_t *sel,
                          const float *w, const int32_t *row_of, const int32_t *tok_ptr, const int32_t *tok_assign,
                          const void *x, const void *const_vecs, const void *add0, const void *add1, const void *add2,
                          void *dx, int32_t *dev_status, moe_stream_t stream) {
  const int st = check_bwd_config(cfg);
  if (st != MOE_OK) return st;
  const moe_config &c = *cfg;
  const bool mix = n_const_of(c) > 0 && c.const_mix;
  if (c.T > 0) {
    if (!sel || !w || !row_of || !dx) return MOE_ERR_INVALID_ARG;
    if (c.n_heavy > 0 && !dx_perm) return MOE_ERR_INVALID_ARG;
    if ((has_kind(c, MOE_IDENTITY) || mix) && !dy) return MOE_ERR_INVALID_ARG;
    if (mix && (!x || !const_vecs)) return MOE_ERR_INVALID_ARG;
    // A mixed constant expert's dots take whole rows of dy and x, of which each warp stores a part.
    const size_t row_bytes = (size_t)c.d * (c.dtype == MOE_BF16 ? 2 : 4);
    if (mix && (overlap(dx, dy, c.T * row_bytes) || overlap(dx, x, c.T * row_bytes))) return MOE_ERR_INVALID_ARG;
    if (c.routing == MOE_EXPERT_CHOICE && (!tok_ptr || !tok_assign)) return MOE_ERR_INVALID_ARG;
  }
  if (!all_aligned16(dx_perm, dy, x, const_vecs, add0, add1, add2, dx)) return MOE_ERR_INVALID_ARG;
  ExchangeBwdArgs a = exchange_args(c, sel, w, row_of, tok_ptr, tok_assign, x, const_vecs, dy, dev_status);
  a.dx_perm = dx_perm; a.add[0] = add0; a.add[1] = add1; a.add[2] = add2; a.dx = dx;
  return launch_dispatch_bwd(a, kind_table(c), stream);
}

int moe_router_backward(const moe_config *cfg, const void *x, const void *W_r, const float *probs, const int32_t *sel,
                        const float *w, const float *dw, const int32_t *tok_ptr, const int32_t *tok_assign,
                        const float *dprobs, float *dlogits, float *dz_prev, float *dbias, float *dW_r, void *dx,
                        int32_t *dev_status, void *ws, size_t ws_bytes, moe_stream_t stream) {
  return moe_router_backward_logits(cfg, x, W_r, probs, sel, w, dw, tok_ptr, tok_assign, dprobs, nullptr, dlogits,
                                    dz_prev, dbias, dW_r, dx, dev_status, ws, ws_bytes, stream);
}

int moe_router_backward_logits(const moe_config *cfg, const void *x, const void *W_r, const float *probs,
                               const int32_t *sel, const float *w, const float *dw, const int32_t *tok_ptr,
                               const int32_t *tok_assign, const float *dprobs, const float *dz_next, float *dlogits,
                               float *dz_prev, float *dbias, float *dW_r, void *dx, int32_t *dev_status, void *ws,
                               size_t ws_bytes, moe_stream_t stream) {
  int st = check_bwd_config(cfg);
  if (st != MOE_OK) return st;
  const moe_config &c = *cfg;
  if (c.T > 0) {
    if (!probs || !sel || !dw || !dlogits) return MOE_ERR_INVALID_ARG;
    if (c.renorm && c.routing == MOE_TOKEN_TOPK && !w) return MOE_ERR_INVALID_ARG;
    if (c.routing == MOE_EXPERT_CHOICE && (!tok_ptr || !tok_assign)) return MOE_ERR_INVALID_ARG;
    if (dx && !W_r) return MOE_ERR_INVALID_ARG;
    if (dW_r && !x) return MOE_ERR_INVALID_ARG;
  }
  if (!all_aligned16(x, W_r, dx, dW_r)) return MOE_ERR_INVALID_ARG;
  if ((st = check_bwd_ws(bwd_layout(c).total, ws, ws_bytes)) != MOE_OK) return st;
  RouterBwdArgs a{};
  a.routing = c.routing; a.T = c.T; a.d = c.d; a.E = c.E; a.k = c.k; a.C = c.capacity; a.dtype = c.dtype;
  a.renorm = c.renorm; a.n_assign = n_assign_of(c); a.zscale = c.gate_residual_scale;
  a.x = x; a.W_r = W_r; a.probs = probs; a.w = w; a.dw = dw; a.dprobs = dprobs; a.dz_next = dz_next;
  a.sel = sel; a.tok_ptr = tok_ptr; a.tok_assign = tok_assign;
  a.dlogits = dlogits; a.dz_prev = dz_prev; a.dbias = dbias; a.dW_r = dW_r; a.dx = c.T > 0 ? dx : nullptr;
  a.part = at<float>(ws, kAlign);
  a.dev_status = dev_status;
  return launch_router_bwd(a, stream);
}

int moe_grouped_mlp_backward(const moe_config *cfg, const void *x_perm, const int32_t *offsets, const void *W1,
                             const void *W2, const void *dy_perm, const void *x, const void *Ws1, const void *Ws2,
                             const void *dy_shared, void *dx_perm, void *dW1, void *dW2, void *dx_shared, void *dWs1,
                             void *dWs2, int32_t *dev_status, void *ws, size_t ws_bytes, moe_stream_t stream) {
  int st = check_bwd_config(cfg);
  if (st != MOE_OK) return st;
  const moe_config &c = *cfg;
  const int64_t na = n_assign_of(c), hs = (int64_t)c.n_shared * c.h_shared;
  const bool routed = c.n_heavy > 0 && (dx_perm || dW1 || dW2), shared = hs > 0 && (dx_shared || dWs1 || dWs2);
  if (routed && (!offsets || !W1 || !W2 || (na > 0 && (!x_perm || !dy_perm)))) return MOE_ERR_INVALID_ARG;
  if (shared && (!Ws1 || !Ws2 || (c.T > 0 && (!x || !dy_shared)))) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(x_perm, W1, W2, dy_perm, x, Ws1, Ws2, dy_shared) ||
      !all_aligned16(dx_perm, dW1, dW2, dx_shared, dWs1, dWs2))
    return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(c);
  if ((st = check_bwd_ws(L.total, ws, ws_bytes)) != MOE_OK) return st;
  MlpBwdProblem p[2];
  int n = 0;
  if (routed) {
    MlpBwdProblem &q = p[n++];
    q = MlpBwdProblem{};
    q.rows = na; q.n_groups = c.n_heavy; q.offsets = offsets; q.h = c.h; q.gated = c.act == MOE_SWIGLU;
    q.x = x_perm; q.dy = dy_perm; q.W1 = W1; q.W2 = W2; q.dx = dx_perm; q.dW1 = dW1; q.dW2 = dW2;
  }
  if (shared) {
    MlpBwdProblem &q = p[n++];
    q = MlpBwdProblem{};
    q.rows = c.T; q.n_groups = 1; q.h = (int)hs;
    q.x = x; q.dy = dy_shared; q.W1 = Ws1; q.W2 = Ws2; q.dx = dx_shared; q.dW1 = dWs1; q.dW2 = dWs2;
  }
  for (int i = 0; i < n; ++i) {
    const bool first = i == 0 && routed;
    p[i].d = c.d;
    p[i].status = dev_status;
    p[i].H = at<void>(ws, first ? L.H : L.Hs);
    p[i].dU = at<void>(ws, first ? L.dU : L.dUs);
    p[i].U = at<void>(ws, L.U);
  }
  return c.dtype == MOE_BF16 ? launch_mlp_bwd_bf16(p, n, dev_status, stream) : launch_mlp_bwd_f32(p, n, stream);
}

int moe_block_norm(const moe_norm_config *cfg, const void *h, const void *x, const void *post_gamma, const void *gate,
                   const void *pre_gamma, const void *pre_beta, const void *scale, const void *shift,
                   int64_t cond_stride, void *y, void *z, moe_stream_t stream) {
  const int st = check_norm(cfg);
  if (st != MOE_OK) return st;
  const moe_norm_config &c = *cfg;
  if ((!h && !x && c.T > 0) || (!y && !z)) return MOE_ERR_INVALID_ARG;
  if (!h && (gate || post_gamma) && c.T > 0) return MOE_ERR_INVALID_ARG;
  if (post_gamma && c.post_kind == MOE_NORM_NONE) return MOE_ERR_INVALID_ARG;
  if (c.pre_kind == MOE_NORM_NONE && (z || pre_gamma || pre_beta)) return MOE_ERR_INVALID_ARG;
  if ((gate || scale || shift) && (cond_stride < c.d || cond_stride % 8 != 0)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(h, x, post_gamma, gate, pre_gamma, pre_beta, scale, shift, y, z)) return MOE_ERR_INVALID_ARG;
  BlockNormArgs a{};
  a.T = c.T; a.d = c.d; a.group = norm_group(c); a.pre = c.pre_kind; a.post = c.post_kind;
  a.eps = c.eps; a.res_scale = c.res_scale;
  a.h = h; a.x = x; a.post_gamma = post_gamma; a.gate = gate; a.pre_gamma = pre_gamma; a.pre_beta = pre_beta;
  a.scale = scale; a.shift = shift; a.cond_stride = cond_stride; a.y = y; a.z = z;
  return launch_block_norm(a, c.dtype, stream);
}

int moe_block_norm_workspace_size(const moe_norm_config *cfg, size_t *bytes) {
  const int st = check_norm(cfg);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kAlign + align_up(block_norm_workspace_bytes(cfg->T, cfg->d, norm_group(*cfg), cfg->dtype));
  return MOE_OK;
}

int moe_block_norm_backward(const moe_norm_config *cfg, const void *h, const void *y, const void *post_gamma,
                            const void *gate, const void *pre_gamma, const void *pre_beta, const void *scale,
                            int64_t cond_stride, const void *dz, const void *dy, void *dh, void *dx,
                            float *dpost_gamma, float *dgate, float *dpre_gamma, float *dpre_beta, float *dscale,
                            float *dshift, int64_t dcond_stride, void *ws, size_t ws_bytes, moe_stream_t stream) {
  int st = check_norm(cfg);
  if (st != MOE_OK) return st;
  const moe_norm_config &c = *cfg;
  if (!dz && !dy) return MOE_ERR_INVALID_ARG;
  if (dz && ((!y && c.T > 0) || c.pre_kind == MOE_NORM_NONE)) return MOE_ERR_INVALID_ARG;
  if (!dz && (dscale || dshift || dpre_gamma || dpre_beta)) return MOE_ERR_INVALID_ARG;
  if (!h && c.T > 0 && (dgate || dpost_gamma || (dh && c.post_kind != MOE_NORM_NONE))) return MOE_ERR_INVALID_ARG;
  if ((post_gamma || dpost_gamma) && c.post_kind == MOE_NORM_NONE) return MOE_ERR_INVALID_ARG;
  if (dh && dh == dx) return MOE_ERR_INVALID_ARG;
  if ((gate || scale) && (cond_stride < c.d || cond_stride % 8 != 0)) return MOE_ERR_INVALID_ARG;
  if ((dgate || dscale || dshift) && (dcond_stride < c.d || dcond_stride % 4 != 0)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16(h, y, post_gamma, gate, pre_gamma, pre_beta, scale, dz, dy, dh, dx) ||
      !all_aligned16(dgate, dscale, dshift))
    return MOE_ERR_INVALID_ARG;
  size_t need = 0;
  if ((st = moe_block_norm_workspace_size(cfg, &need)) != MOE_OK) return st;
  if ((st = check_bwd_ws(need, ws, ws_bytes)) != MOE_OK) return st;
  if (c.T == 0 && c.group_size == 0)  // the one condition row that all (no) tokens share
    for (float *o : {dgate, dscale, dshift})
      if (o) MOE_CUDA_TRY(cudaMemsetAsync(o, 0, (size_t)c.d * 4, stream));
  BlockNormArgs a{};
  a.T = c.T; a.d = c.d; a.group = norm_group(c); a.pre = c.pre_kind; a.post = c.post_kind;
  a.eps = c.eps; a.res_scale = c.res_scale;
  a.h = h; a.yin = y; a.post_gamma = post_gamma; a.gate = gate; a.pre_gamma = pre_gamma; a.pre_beta = pre_beta;
  a.scale = scale; a.cond_stride = cond_stride; a.dz = dz; a.dy = dy; a.dh = dh; a.dx = dx;
  a.dpost_gamma = dpost_gamma; a.dgate = dgate; a.dpre_gamma = dpre_gamma; a.dpre_beta = dpre_beta;
  a.dscale = dscale; a.dshift = dshift; a.dcond_stride = dcond_stride; a.part = at<float>(ws, kAlign);
  return launch_block_norm_bwd(a, c.dtype, stream);
}

}  // extern "C"
