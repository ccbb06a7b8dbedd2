"""Training steps of layers without heavy experts, and of layers that carry
weights none of their experts reads: forward, forward_train and backward take
the same weights. Gradients against fp64 differentiation, as in the tests of
the whole step (bf16 3.2e-2, fp32 1e-4 of the largest value); a weight that
nothing reads has gradient zero."""

import pytest
import torch

from mixture_experts_layer_33_b200 import inputs as gen
from test_gpu_train_step import CONST, HEAVY, IDENTITY, TOL, ZERO, close, layer64

pytestmark = pytest.mark.gpu

LIGHT = [IDENTITY, ZERO, CONST]
CASES = {
    "all_light": ("mmoe", dict(T=77, d=264, E=3, kinds=LIGHT, h_shared=72), ()),
    "all_light_no_shared_f32": ("tiny_fp32", dict(T=33, x_std=1.0, E=4, kinds=LIGHT + [CONST]), ()),
    "all_light_mixed": ("mmoe_constmix", dict(T=60, d=520, E=3, kinds=LIGHT, h_shared=64), ()),
    "spare_const_vecs": ("ditmoe_xl", dict(T=50, d=128, h=64, h_shared=64), ("const_vecs",)),
    "spare_shared": ("tiny_fp32", dict(T=33, x_std=1.0), ("Ws1", "Ws2", "const_vecs")),
    "spare_heavy": ("mmoe", dict(T=41, d=64, E=3, kinds=LIGHT, h_shared=72), ("W1", "W2")),
}


@pytest.mark.parametrize("name", list(CASES))
def test_layer_gradients(name):
    from mixture_experts_layer_33_b200 import moe as m
    wl, over, spare = CASES[name]
    cfg = gen.workload(wl, **over)
    inp = gen.make_inputs(cfg, "cuda")
    x, zp = inp["x"], inp["z_prev"]
    weights = {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")}
    if HEAVY not in cfg["kinds"]:
        del weights["W1"], weights["W2"]
    for k in spare:  # of no size that the layer could ask for
        weights[k] = torch.ones(3, 5, cfg["d"], dtype=x.dtype, device="cuda")
    layer = m.MoELayer(cfg, weights)
    y, s = layer.forward_train(x, z_prev=zp)
    close("forward", y, layer(x, z_prev=zp).double().cpu(), 2e-2 if cfg["dtype"] == "bf16" else 1e-4)
    dy = torch.randn(y.shape, generator=torch.Generator(device="cuda").manual_seed(11), device="cuda").to(y.dtype)
    grads = layer.backward(s, dy)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    p = {k: (v.double().cpu().requires_grad_() if v is not None and k not in spare else None)
         for k, v in weights.items()}
    x64 = x.double().cpu().requires_grad_()
    leaves = {"x": x64, **{k: v for k, v in p.items() if v is not None}}
    ref = layer64(cfg, s, x64, zp.double().cpu() if zp is not None else None, p)
    want = dict(zip(leaves, torch.autograd.grad(ref, list(leaves.values()), dy.double().cpu(), allow_unused=True,
                                                materialize_grads=True)))
    assert set(grads) == set(want) | set(spare) | ({"z_prev"} if zp is not None else set())
    for k in want:
        close(k, grads[k], want[k], TOL[cfg["dtype"]])
    for k in spare:
        assert grads[k].shape == weights[k].shape and (grads[k] == 0).all()
        assert grads[k].dtype is (torch.float32 if k == "const_vecs" else x.dtype)
