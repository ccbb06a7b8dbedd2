"""A training step on no tokens at all: forward_train and backward take what
forward takes, y is empty, and every weight's gradient is zero."""

import pytest
import torch

from mixture_experts_layer_33_b200 import inputs as gen

pytestmark = pytest.mark.gpu

CASES = {
    "topk_shared": ("ditmoe_xl", dict(T=0, d=256, h=320, h_shared=200)),
    "mmoe": ("mmoe", dict(T=0, d=264, h=256, h_shared=136)),
    "constmix": ("mmoe_constmix", dict(T=0, d=128, h=128, h_shared=64)),
    "expert_choice": ("ecdit", dict(T=0, d=256, h=256)),
    "des_vote": ("des_vote", dict(T=0, d=256, h=128)),
    "des_seq": ("des_seq", dict(T=0, d=256, h=128)),
    "f32": ("tiny_fp32", dict(T=0, x_std=1.0)),
}


@pytest.mark.parametrize("name", list(CASES))
def test_step_on_no_tokens(name):
    from mixture_experts_layer_33_b200 import moe as m
    wl, over = CASES[name]
    cfg = gen.workload(wl, **over)
    inp = gen.make_inputs(cfg, "cuda")
    layer = m.MoELayer(cfg, {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")})
    x, zp = inp["x"], inp["z_prev"]
    assert x.shape == (0, cfg["d"])
    assert layer(x, z_prev=zp).shape == x.shape
    y, s = layer.forward_train(x, z_prev=zp)
    layer.bws = m.alloc_backward_workspace(layer.c).fill_(255)
    grads = layer.backward(s, torch.empty_like(x), dlogits=zp)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    assert y.shape == x.shape and grads["x"].shape == x.shape
    for k, w in layer.w.items():
        if w is not None:
            assert grads[k].shape == w.shape and (grads[k] == 0).all(), k
