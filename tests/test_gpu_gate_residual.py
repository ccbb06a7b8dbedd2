"""The gate residual through a stack: a layer's logits are the next layer's
z_prev, so the next layer's dz_prev is a gradient on this layer's logits. The
router's gradient with such a term against the formula, and three layers one
after the other against fp64 differentiation of the whole stack.

Bounds of the router: as in its own tests, the term adds its magnitude and one
rounding. Tolerance of the stack: a layer's gradients are within 3.2e-2 (bf16)
or 1e-4 (fp32) of their largest value, as in the tests of one layer; errors of
three layers in a row add up, so three times that. Leaving the term out moves
the earlier layers' router gradients by far more, which is checked."""

import pytest
import torch

from grad_helpers import within
from mixture_experts_layer_33_b200 import inputs as gen
from test_gpu_router_backward import CASES, operands, run, weights
from test_gpu_train_step import close, layer64

pytestmark = pytest.mark.gpu


def _moe():
    from mixture_experts_layer_33_b200 import moe
    return moe


@pytest.mark.parametrize("name", list(CASES))
def test_router_with_a_gradient_on_the_logits(name):
    m, c = _moe(), CASES[name]
    r, o = operands(c)
    T, E = c["T"], c["E"]
    zn = torch.randn(T, E, generator=torch.Generator().manual_seed(17))
    plain = run(c, r, o)
    G = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in {**r, **o}.items()}
    mc = m.make_config(c)

    def call(dz_next, dlogits, **out):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = m.alloc_backward_workspace(mc)
        ws.fill_(255)
        m.router_backward(mc, G["x"], G["W_r"], G["probs"], G["sel"], G["w"], G["dw"], G["tok_ptr"], G["tok_assign"],
                          dlogits, status, ws, dprobs=G["dprobs"], dz_next=dz_next, **out)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return {**out, "dlogits": dlogits}

    def outputs():
        return {"dz_prev": torch.empty(T, E, device="cuda"), "dbias": torch.empty(E, device="cuda"),
                "dW_r": torch.empty(E, c["d"], device="cuda"), "dx": torch.empty_like(G["x"])}
    out = call(zn.cuda(), torch.empty(T, E, device="cuda"), **outputs())
    # Without it: the same bytes as the call that does not know it.
    none = call(None, torch.empty(T, E, device="cuda"), **outputs())
    for k in none:
        assert torch.equal(none[k], plain[k]), k
    # The whole dz is the sum; its magnitude that of the plain one's terms and the new one.
    z = torch.log(o["probs"].double()).requires_grad_()
    A = torch.softmax(z, -1)
    loss = (weights(c, r, A) * o["dw"].double()).sum()
    if c["aux"]:
        loss = loss + (A * o["dprobs"].double()).sum()
    dz = torch.autograd.grad(loss, z)[0] + zn.double()
    A = A.detach()
    dw = o["dw"].double().abs() * (r["eid"] >= 0)
    if c["renorm"]:
        w = r["w"].double().view(T, -1)
        S = A.gather(1, r["eid"].view(T, -1)).sum(-1, keepdim=True)
        dw = ((dw.view(T, -1) + (dw.view(T, -1) * w).sum(-1, keepdim=True)) / S).reshape(-1)
    dA = o["dprobs"].double().abs() if c["aux"] else torch.zeros_like(A)
    dA = dA.index_put((r["tok"], r["eid"].clamp(min=0)), dw, accumulate=True)
    mag = A * (dA + (A * dA).sum(-1, keepdim=True)) + zn.double().abs()
    step = 3 * (E / 32 + 10) + 1
    x, W = o["x"].double(), o["W_r"].double()
    within("dlogits", out["dlogits"], dz, mag, step)
    within("dz_prev", out["dz_prev"], 0.5 * dz, mag, step)
    within("dbias", out["dbias"], dz.sum(0), mag.sum(0), step + T)
    within("dW_r", out["dW_r"], dz.t() @ x, mag.t() @ x.abs(), step + 2 * T)
    within("dx", out["dx"], dz @ W, mag @ W.abs(), step + 2 * E + 4)
    # It may be dlogits' or dz_prev's buffer.
    for key in ("dlogits", "dz_prev"):
        o2 = dict(outputs(), dlogits=torch.empty(T, E, device="cuda"))
        o2[key] = zn.cuda()
        again = call(o2[key], o2.pop("dlogits"), **o2)
        for k in out:
            assert torch.equal(again[k], out[k]), (key, k)


STACKS = {
    "mmoe": ("mmoe", dict(T=200, d=264, h=128, h_shared=72, w_std=0.08)),
    "mmoe_constmix": ("mmoe_constmix", dict(T=150, d=128, h=128, h_shared=64, w_std=0.1)),
    "expert_choice": ("ecdit", dict(T=512, d=128, h=128, w_std=0.1, gate_residual_scale=0.5)),
    "des_vote": ("des_vote", dict(T=48, d=128, h=128, w_std=0.1, gate_residual_scale=0.5)),
    "f32": ("tiny_fp32", dict(T=100, x_std=1.0, w_std=0.15, gate_residual_scale=0.75)),
    "f32_renorm": ("tiny_fp32", dict(T=100, x_std=1.0, w_std=0.15, renorm=1, gate_residual_scale=0.75)),
}


@pytest.mark.parametrize("name", list(STACKS))
def test_three_layers_in_a_row(name):
    m = _moe()
    wl, over = STACKS[name]
    keys = ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")
    layers = []
    for i in range(3):
        cfg = gen.workload(wl, seed=40 + i, **over)
        inp = gen.make_inputs(cfg, "cuda")
        layers.append((cfg, m.MoELayer(cfg, {k: inp[k] for k in keys})))
        if i == 0:
            x, z0 = inp["x"], inp["z_prev"]
    y, z, saved = x, z0, []
    for _, layer in layers:
        y, s = layer.forward_train(y, z_prev=z)
        z = s["logits"]
        saved.append(s)
    dy = torch.randn(y.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(y.dtype)
    grads, d, dz = [None] * 3, dy, None
    for i in (2, 1, 0):
        grads[i] = layers[i][1].backward(saved[i], d, dlogits=dz)
        d, dz = grads[i]["x"], grads[i]["z_prev"]
    torch.cuda.synchronize()
    assert all(int(layer.status.item()) == 0 for _, layer in layers)

    params = [{k: (v.double().cpu().requires_grad_() if v is not None else None) for k, v in layer.w.items()}
              for _, layer in layers]
    x64, z64 = x.double().cpu().requires_grad_(), z0.double().cpu().requires_grad_()

    def stack(cut):
        """The last layer's y; with `cut` the logits pass on without a gradient."""
        y, z = x64, z64
        for (cfg, _), s, p in zip(layers, saved, params):
            zp = z
            z = y @ p["W_r"].t() + cfg["gate_residual_scale"] * zp
            if p.get("logit_bias") is not None:
                z = z + p["logit_bias"]
            y = layer64(cfg, s, y, zp, p)
            z = z.detach() if cut else z
        return y
    names = [(i, k) for i in range(3) for k in params[i] if params[i][k] is not None]
    leaves = [params[i][k] for i, k in names] + [x64, z64]
    want = torch.autograd.grad(stack(False), leaves, dy.double().cpu(), allow_unused=True, materialize_grads=True)
    cut = torch.autograd.grad(stack(True), leaves, dy.double().cpu(), allow_unused=True, materialize_grads=True)
    tol = 3 * (3.2e-2 if layers[0][0]["dtype"] == "bf16" else 1e-4)
    for (i, k), ref in zip(names, want):
        close(f"layer {i} {k}", grads[i][k], ref, tol)
    close("x", grads[0]["x"], want[-2], tol)
    close("z_prev", grads[0]["z_prev"], want[-1], tol)
    # The stack's inputs tell the term apart.
    for key in ((0, "W_r"), (1, "W_r")):
        a, b = want[names.index(key)], cut[names.index(key)]
        assert float((a - b).abs().max()) > 2 * tol * float(a.abs().max()), key
    assert float((want[-1] - cut[-1]).abs().max()) > 2 * tol * float(want[-1].abs().max())
