"""MoELayer.forward_train refuses inputs that do not fit the layer's config
before any work is queued: its buffers have the config's sizes, so a longer
batch, a wider type or too short a z_prev would be written or read past their
ends. Entry points and the device are stand-ins: no GPU."""

import pytest
import torch

ENTRIES = ("router", "select_expert_choice", "core_set_vote", "core_set_union", "dispatch", "grouped_mlp", "combine")


@pytest.fixture(scope="module")
def m():
    from mixture_experts_layer_33_b200 import build
    build.build()
    from mixture_experts_layer_33_b200 import moe
    return moe


@pytest.mark.parametrize("wl", ["mmoe", "tiny_fp32"])
def test_inputs_that_do_not_fit(m, monkeypatch, wl):
    from mixture_experts_layer_33_b200 import inputs as gen
    cfg = gen.workload(wl, T=16, d=64, h=64)
    if cfg.get("n_shared"):
        cfg["h_shared"] = 64
    inp = gen.make_inputs(cfg, "cpu")
    launched = []
    for name in ENTRIES:
        monkeypatch.setattr(m, name, lambda *a, _n=name, **k: launched.append(_n))
    layer = m.MoELayer(cfg, {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")},
                       device="cpu")
    x, T, d, E = inp["x"], 16, 64, cfg["E"]
    other = torch.float32 if x.dtype == torch.bfloat16 else torch.bfloat16

    def t(*shape, dtype=x.dtype):
        return torch.zeros(*shape, dtype=dtype)
    bad = [dict(x=t(T + 1, d)), dict(x=t(T - 1, d)), dict(x=t(2 * T, d // 2)), dict(x=t(T // 2, 2 * d)), dict(x=t(2, 8, d)),
           dict(x=t(T, d, dtype=other)), dict(x=t(d, T).t()), dict(x=t(T, 2 * d)[:, :d]),
           dict(z_prev=t(T - 1, E, dtype=torch.float32)), dict(z_prev=t(T, E, dtype=torch.bfloat16)),
           dict(z_prev=t(E, T, dtype=torch.float32).t()),
           dict(residual=t(T - 1, d)), dict(residual=t(T, d, dtype=other))]
    for kw in bad:
        with pytest.raises(ValueError):
            layer.forward_train(**dict(dict(x=x), **kw))
    with monkeypatch.context() as on_gpu:  # as device tensors, all on device 0, when device 1 is current
        on_gpu.setattr(torch.Tensor, "is_cuda", True)
        on_gpu.setattr(torch.Tensor, "get_device", lambda t: 0)
        on_gpu.setattr(torch.cuda, "current_device", lambda: 1)
        with pytest.raises(ValueError):
            layer.forward_train(x)
    assert not launched
    layer.forward_train(x, z_prev=t(T, E, dtype=torch.float32), residual=t(T, d))
    assert launched
