"""The gradients' and block norms' entry points check their arguments on the
host: every refusal below happens before any CUDA call (no GPU needed). The
Python binding refuses tensors of the wrong type, size, layout or device."""

import ctypes

import pytest
import torch

OK, BAD, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 1 << 20  # an aligned address, never dereferenced


@pytest.fixture(scope="module")
def m():
    from mixture_experts_layer_33_b200 import build
    build.build()
    from mixture_experts_layer_33_b200 import moe
    return moe


def cfg(m, name="mmoe", **kw):
    from mixture_experts_layer_33_b200 import inputs as gen
    return m.make_config(gen.workload(name, **kw))


def norm(m, **kw):
    return m.make_norm_config(dict(dict(T=64, d=256, dtype="bf16", group_size=16, pre="layer", post="rms"), **kw))


def test_workspace_covers_every_entry_point(m):
    c = cfg(m)
    n = m.backward_workspace_size(c)
    na, T, hs = m.num_assignments(c), c.T, c.n_shared * c.h_shared
    assert n % 256 == 0 and n >= 2 * (na * c.h + T * hs) * 2  # H and dU, routed and shared
    gated = cfg(m, "des_vote")
    assert m.backward_workspace_size(gated) >= 3 * m.num_assignments(gated) * gated.h * 2
    assert m.backward_workspace_size(cfg(m, "mmoe", T=0)) >= 256
    bad = cfg(m)
    bad.d = 12
    with pytest.raises(RuntimeError):
        m.backward_workspace_size(bad)


def combine(m, c, **kw):
    a = dict(dy=FAKE, y_perm=FAKE, sel=FAKE, w=FAKE, row_of=FAKE, x=FAKE, const_vecs=FAKE, dy_perm=FAKE, dw=FAKE,
             dconst=FAKE, status=None, ws=FAKE, ws_bytes=0)
    a.update(kw)
    return m.LIB.moe_combine_backward(ctypes.byref(c), *a.values(), None)


def test_combine_backward_refusals(m):
    c = cfg(m)
    assert combine(m, c) == WORKSPACE
    for n in ("dy", "y_perm", "sel", "w", "row_of", "x", "const_vecs", "dy_perm", "dw"):
        assert combine(m, c, **{n: None}) == BAD, n
    for n in ("dy", "y_perm", "x", "const_vecs", "dy_perm", "dconst"):
        assert combine(m, c, **{n: FAKE + 2}) == BAD, n
    assert combine(m, c, ws=None, ws_bytes=1 << 40) == BAD
    assert combine(m, c, ws=FAKE + 16, ws_bytes=1 << 40) == BAD
    assert m.LIB.moe_combine_backward(None, *[FAKE] * 12, 1 << 40, None) == BAD
    heavy = cfg(m, "ditmoe_xl")  # no lightweight experts: x and const_vecs are not needed
    assert combine(m, heavy, x=None, const_vecs=None) == WORKSPACE


def dispatch(m, c, **kw):
    a = dict(dx_perm=FAKE, dy=FAKE, sel=FAKE, w=FAKE, row_of=FAKE, tok_ptr=None, tok_assign=None, x=FAKE,
             const_vecs=FAKE, add0=None, add1=None, add2=None, dx=FAKE, status=None)
    a.update(kw)
    return m.LIB.moe_dispatch_backward(ctypes.byref(c), *a.values(), None)


def test_dispatch_backward_refusals(m):
    c = cfg(m, "mmoe_constmix")
    for n in ("dx_perm", "dy", "sel", "w", "row_of", "x", "const_vecs", "dx"):
        assert dispatch(m, c, **{n: None}) == BAD, n
    for n in ("dx_perm", "dy", "x", "const_vecs", "add0", "add1", "add2", "dx"):
        assert dispatch(m, c, **{n: FAKE + 8}) == BAD, n
    ec = cfg(m, "ecdit")
    assert dispatch(m, ec, tok_ptr=FAKE) == BAD
    assert dispatch(m, ec, tok_assign=FAKE) == BAD
    assert dispatch(m, cfg(m, "ditmoe_xl", T=0), dx=None, sel=None, w=None, row_of=None) == OK  # nothing to do


def router(m, c, **kw):
    a = dict(x=FAKE, W_r=FAKE, probs=FAKE, sel=FAKE, w=FAKE, dw=FAKE, tok_ptr=None, tok_assign=None, dprobs=None,
             dlogits=FAKE, dz_prev=None, dbias=None, dW_r=FAKE, dx=FAKE, status=None, ws=FAKE, ws_bytes=0)
    a.update(kw)
    return m.LIB.moe_router_backward(ctypes.byref(c), *a.values(), None)


def test_router_backward_refusals(m):
    c = cfg(m)
    assert router(m, c) == WORKSPACE
    for n in ("x", "W_r", "probs", "sel", "dw", "dlogits"):
        assert router(m, c, **{n: None}) == BAD, n
    for n in ("x", "W_r", "dW_r", "dx"):
        assert router(m, c, **{n: FAKE + 4}) == BAD, n
    assert router(m, c, w=None) == WORKSPACE  # the weights are read with renorm only
    c.renorm = 1
    assert router(m, c, w=None) == BAD
    assert router(m, cfg(m, "ecdit"), tok_ptr=FAKE) == BAD
    assert router(m, cfg(m), ws=None, ws_bytes=1 << 40) == BAD


def mlp(m, c, **kw):
    a = dict(x_perm=FAKE, offsets=FAKE, W1=FAKE, W2=FAKE, dy_perm=FAKE, x=FAKE, Ws1=FAKE, Ws2=FAKE, dy_shared=FAKE,
             dx_perm=FAKE, dW1=FAKE, dW2=FAKE, dx_shared=FAKE, dWs1=FAKE, dWs2=FAKE, status=None, ws=FAKE, ws_bytes=0)
    a.update(kw)
    return m.LIB.moe_grouped_mlp_backward(ctypes.byref(c), *a.values(), None)


def test_grouped_mlp_backward_refusals(m):
    c = cfg(m)
    assert mlp(m, c) == WORKSPACE
    for n in ("x_perm", "offsets", "W1", "W2", "dy_perm", "x", "Ws1", "Ws2", "dy_shared"):
        assert mlp(m, c, **{n: None}) == BAD, n
    for n in ("x_perm", "W1", "W2", "dy_perm", "x", "Ws1", "Ws2", "dy_shared", "dx_perm", "dW1", "dW2", "dx_shared",
              "dWs1", "dWs2"):
        assert mlp(m, c, **{n: FAKE + 2}) == BAD, n
    # Nothing of the shared (routed) part asked for: its inputs may be left out.
    assert mlp(m, c, x=None, Ws1=None, Ws2=None, dy_shared=None, dx_shared=None, dWs1=None, dWs2=None) == WORKSPACE
    assert mlp(m, c, x_perm=None, offsets=None, W1=None, W2=None, dy_perm=None, dx_perm=None, dW1=None,
               dW2=None) == WORKSPACE
    assert mlp(m, c, ws=FAKE + 64, ws_bytes=1 << 40) == BAD


def block_norm(m, n, **kw):
    a = dict(h=FAKE, x=FAKE, post_gamma=FAKE, gate=FAKE, pre_gamma=FAKE, pre_beta=FAKE, scale=FAKE, shift=FAKE,
             cond_stride=256, y=FAKE, z=FAKE)
    a.update(kw)
    return m.LIB.moe_block_norm(ctypes.byref(n), *a.values(), None)


@pytest.mark.parametrize("field,value,code", [
    ("T", -1, BAD), ("T", (1 << 30) + 1, UNSUPPORTED), ("d", 12, BAD), ("d", 0, BAD), ("d", 8200, UNSUPPORTED), ("dtype", 5, BAD), ("group_size", -1, BAD),
    ("pre_kind", 3, BAD), ("post_kind", -1, BAD), ("eps", 0.0, BAD), ("eps", -1.0, BAD), ("eps", float("nan"), BAD),
    ("eps", float("inf"), BAD), ("res_scale", float("nan"), BAD)])
def test_norm_config_refusals(m, field, value, code):
    n = norm(m)
    setattr(n, field, value)
    b = ctypes.c_size_t()
    assert m.LIB.moe_block_norm_workspace_size(ctypes.byref(n), ctypes.byref(b)) == code
    assert block_norm(m, n, cond_stride=1 << 20) == code


def test_block_norm_refusals(m):
    n = norm(m)
    assert block_norm(m, n, h=None, x=None) == BAD
    assert block_norm(m, n, y=None, z=None) == BAD
    assert block_norm(m, n, h=None) == BAD  # a gate and a post weight without a block
    for name in ("h", "x", "post_gamma", "gate", "pre_gamma", "pre_beta", "scale", "shift", "y", "z"):
        assert block_norm(m, n, **{name: FAKE + 2}) == BAD, name
    assert block_norm(m, n, cond_stride=248) == BAD
    assert block_norm(m, n, cond_stride=260) == BAD
    assert block_norm(m, norm(m, post="none")) == BAD  # a post weight without a post norm
    assert block_norm(m, norm(m, pre="none")) == BAD   # z without a pre norm
    assert block_norm(m, norm(m, T=0)) == OK           # nothing to do


def norm_bwd(m, n, **kw):
    a = dict(h=FAKE, y=FAKE, post_gamma=FAKE, gate=FAKE, pre_gamma=FAKE, pre_beta=FAKE, scale=FAKE, cond_stride=256,
             dz=FAKE, dy=FAKE, dh=FAKE, dx=FAKE + 4096, dpost_gamma=FAKE, dgate=FAKE, dpre_gamma=FAKE, dpre_beta=FAKE,
             dscale=FAKE, dshift=FAKE, dcond_stride=256, ws=FAKE, ws_bytes=0)
    a.update(kw)
    return m.LIB.moe_block_norm_backward(ctypes.byref(n), *a.values(), None)


def test_block_norm_backward_refusals(m):
    n = norm(m)
    assert norm_bwd(m, n) == WORKSPACE
    assert norm_bwd(m, n, dz=None, dy=None) == BAD
    assert norm_bwd(m, n, y=None) == BAD
    assert norm_bwd(m, n, dz=None) == BAD  # gradients of dz's side without dz
    assert norm_bwd(m, n, h=None) == BAD
    assert norm_bwd(m, n, dx=FAKE) == BAD  # dh and dx in one buffer
    assert norm_bwd(m, n, cond_stride=252) == BAD
    assert norm_bwd(m, n, dcond_stride=255) == BAD
    assert norm_bwd(m, norm(m, post="none")) == BAD
    assert norm_bwd(m, norm(m, pre="none"), dpost_gamma=None) == BAD  # dz without a pre norm
    for name in ("h", "y", "post_gamma", "gate", "pre_gamma", "pre_beta", "scale", "dz", "dy", "dh", "dx", "dgate",
                 "dscale", "dshift"):
        assert norm_bwd(m, n, **{name: FAKE + 2}) == BAD, name
    assert norm_bwd(m, n, ws=None, ws_bytes=1 << 40) == BAD


def test_binding_refuses_wrong_tensors(m, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    p = m._grad_ptr
    assert p(None, "t", torch.float32, 4, 0) is None
    with pytest.raises(TypeError):
        p([1.0], "t", torch.float32, 1, 0)
    for bad in (torch.zeros(4, dtype=torch.float64), torch.zeros(3), torch.zeros(4, 2)[:, 0], torch.zeros(4)):
        with pytest.raises(ValueError):  # type, size, layout, and (the last) a host tensor
            p(bad, "t", torch.float32, 4, 0)
    n = norm(m)
    for bad in (torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.bfloat16),
                torch.zeros(256, 4, dtype=torch.bfloat16).t()):
        with pytest.raises(ValueError):
            m._cond_ptrs(n, (("gate", bad),), torch.bfloat16, 0)
    with pytest.raises(ValueError):
        m.dispatch_backward(cfg(m), None, None, None, None, None, None, None, None, None, None, None, add=[None] * 4)
