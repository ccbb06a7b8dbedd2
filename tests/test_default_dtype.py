"""torch's default type does not reach the kernels: under bf16, fp16 or fp64 as
the default every tensor a step hands to an entry point has the type it has
under fp32 (logits, affinities and weights are written as fp32, so a narrower
buffer would be written past its end). Entry points are stand-ins: no GPU."""

import pytest
import torch

ENTRIES = ("router", "select_expert_choice", "core_set_vote", "core_set_union", "dispatch", "grouped_mlp", "combine",
           "combine_backward", "dispatch_backward", "router_backward", "grouped_mlp_backward")


@pytest.fixture(scope="module")
def m():
    from mixture_experts_layer_33_b200 import build
    build.build()
    from mixture_experts_layer_33_b200 import moe
    return moe


def types(step, m, monkeypatch, default):
    """(entry, argument, type and size) of every tensor the step hands over, and of its results."""
    seen = []

    def note(where, v):
        if isinstance(v, torch.Tensor):
            seen.append((*where, v.dtype, tuple(v.shape)))
        elif isinstance(v, (list, tuple)):
            for i, t in enumerate(v):
                note((*where, i), t)
        elif isinstance(v, dict):
            for k, t in v.items():
                note((*where, k), t)
    for name in ENTRIES:
        monkeypatch.setattr(m, name, lambda *a, _n=name, **k: (note((_n,), a), note((_n,), k)))
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        note(("result",), step())
    finally:
        torch.set_default_dtype(before)
    return seen


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float16, torch.float64], ids=str)
@pytest.mark.parametrize("name", ["mmoe_constmix", "ecdit", "des_vote", "des_seq", "tiny_fp32"])
def test_training_step(m, monkeypatch, name, default):
    from mixture_experts_layer_33_b200 import inputs as gen
    cfg = gen.workload(name, d=64, h=64, **({"T": 256} if name == "ecdit" else {"T": 16}))
    if cfg.get("n_shared"):
        cfg["h_shared"] = 64
    inp = gen.make_inputs(cfg, "cpu")
    layer = m.MoELayer(cfg, {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")},
                       device="cpu")

    def step():
        y, saved = layer.forward_train(inp["x"], z_prev=inp["z_prev"])
        return y, saved, layer.backward(saved, inp["x"])
    want = types(step, m, monkeypatch, torch.float32)
    assert ("router", 2, torch.float32, (cfg["T"], cfg["E"])) in want
    assert types(step, m, monkeypatch, default) == want


def test_expert_parallel_route(m, monkeypatch):
    from mixture_experts_layer_33_b200 import expert_parallel as ep
    from mixture_experts_layer_33_b200 import inputs as gen
    cfg = gen.workload("mmoe", T=16, d=64, h=64, h_shared=64)
    inp = gen.make_inputs(cfg, "cpu")
    steps = ep.CudaOps(cfg, ep.ExpertShard(16, 1), 0, inp["W_r"], inp["W1"], inp["W2"], device="cpu")
    want = types(lambda: steps.route(inp["x"]), m, monkeypatch, torch.float32)
    assert types(lambda: steps.route(inp["x"]), m, monkeypatch, torch.bfloat16) == want
