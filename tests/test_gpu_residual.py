"""The residual of a training step: x itself, by name or as the tensor, has its
gradient in that of x; another tensor's gradient is dy, left to the caller;
none adds nothing."""

import pytest
import torch

from mixture_experts_layer_33_b200 import inputs as gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,over", [("mmoe", dict(T=100, d=264, h=64, h_shared=72)), ("ecdit", dict(T=256, d=64, h=64)),
                                       ("tiny_fp32", dict(T=50, x_std=1.0))])
def test_residual_and_its_gradient(name, over):
    from mixture_experts_layer_33_b200 import moe as m
    cfg = gen.workload(name, **over)
    inp = gen.make_inputs(cfg, "cuda")
    x, zp = inp["x"], inp["z_prev"]
    layer = m.MoELayer(cfg, {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")})
    dy = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(x.dtype)

    def step(residual):
        y, saved = layer.forward_train(x, z_prev=zp, residual=residual)
        return y, layer.backward(saved, dy)["x"]
    y, dx = step("x")
    for other, (y2, dx2) in (("the tensor", step(x)), ("a copy", step(x.clone())), ("none", step(None))):
        assert torch.equal(y2, y) == (other != "none"), other
        assert torch.equal(dx2, dx) == (other == "the tensor"), other
    # Without the residual's part dx is dy less: each of the two is rounded once from its fp32 sum,
    # half a step of |dx| and of |dx - dy|, and the sums take a few fp32 steps.
    off = (dx.double() - step(None)[1].double() - dy.double()).abs()
    half = torch.finfo(x.dtype).eps / 2
    assert (off <= 4 * half * (dx.double().abs() + dy.double().abs())).all()
