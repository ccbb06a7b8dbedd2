"""A training step under another default type of torch gives the bytes of the
step under fp32."""

import pytest
import torch

from mixture_experts_layer_33_b200 import inputs as gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float64], ids=str)
@pytest.mark.parametrize("name,over", [("mmoe", dict(T=333, d=264, h=256, h_shared=136)),
                                       ("ecdit", dict(T=512, d=256, h=256)), ("tiny_fp32", dict(T=150, x_std=1.0))])
def test_training_step(name, over, default):
    from mixture_experts_layer_33_b200 import moe as m
    cfg = gen.workload(name, **over)
    inp = gen.make_inputs(cfg, "cuda")
    layer = m.MoELayer(cfg, {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")})

    def step():
        y, saved = layer.forward_train(inp["x"], z_prev=inp["z_prev"])
        return {"y": y, "logits": saved["logits"], "w": saved["w"], **layer.backward(saved, inp["x"])}
    want = step()
    torch.cuda.synchronize()
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        got = step()
        torch.cuda.synchronize()
    finally:
        torch.set_default_dtype(before)
    assert int(layer.status.item()) == 0
    for k in want:
        assert got[k].dtype is want[k].dtype and torch.equal(got[k], want[k]), k
