"""Gradient of the router against fp64 differentiation and differences: token
and expert choice, renormalised weights, a gradient on the affinities, empty
slots, every expert-count variant, odd token counts and widths, both types.

Error bounds: dz passes a dot over E (at most E / 32 + 6 steps) and a few
products of |A| (|dA| + sum A |dA|); with renorm another dot and a division.
dx and dW_r are sums of E and T products whose factors carry dz's error, dz
split in three bf16 terms being exact to 2^-24."""

import pytest
import torch

from grad_helpers import leaf, route, within

pytestmark = pytest.mark.gpu


def case(T, d, E, k=2, dtype="bf16", renorm=0, ec=None, aux=False, empty=0.0):
    c = dict(T=T, d=d, h=16, E=E, k=k, dtype=dtype, act="gelu", routing="token_topk", renorm=renorm, aux=aux,
             empty=empty, gate_residual_scale=0.5)
    if ec:
        c.update(routing="expert_choice", group_size=ec[0], capacity=ec[1], k=0)
    return c


CASES = {
    "top2": case(500, 264, 8),
    "one_token": case(1, 8, 2, k=1),
    "renorm": case(129, 136, 19, k=3, renorm=1, aux=True),
    "renorm_one": case(65, 64, 8, k=1, renorm=1),
    "e33": case(77, 72, 33, k=5, aux=True, empty=0.3),
    "e128": case(200, 520, 128, k=40),
    "f32": case(130, 72, 8, dtype="f32", aux=True),
    "f32_e128": case(70, 136, 128, k=4, dtype="f32", renorm=1),
    "ec": case(256, 200, 16, ec=(64, 8), aux=True),
    "ec_f32": case(128, 64, 40, ec=(64, 40), dtype="f32"),
    "long": case(6000, 128, 8),
}


def _moe():
    from mixture_experts_layer_33_b200 import moe
    return moe


def operands(c, seed=9):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    r = route(c, g, c["empty"])
    o = dict(x=torch.randn(c["T"], c["d"], generator=g).to(dt), W_r=(torch.randn(c["E"], c["d"], generator=g) * 0.2).to(dt),
             dw=torch.randn(r["w"].numel(), generator=g), probs=r["probs"],
             dprobs=torch.randn(c["T"], c["E"], generator=g) if c["aux"] else None)
    return r, o


def run(c, r, o, outs=("dz_prev", "dbias", "dW_r", "dx")):
    m = _moe()
    mc = m.make_config(c)
    G = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in {**r, **o}.items()}
    full = {"dz_prev": torch.empty(c["T"], c["E"], device="cuda"), "dbias": torch.empty(c["E"], device="cuda"),
            "dW_r": torch.empty(c["E"], c["d"], device="cuda"), "dx": torch.empty_like(G["x"])}
    out = {k: full[k] for k in outs}
    dlogits = torch.empty(c["T"], c["E"], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = m.alloc_backward_workspace(mc)
    ws.fill_(255)
    m.router_backward(mc, G["x"], G["W_r"], G["probs"], G["sel"], G["w"], G["dw"], G["tok_ptr"], G["tok_assign"],
                      dlogits, status, ws, dprobs=G["dprobs"], **out)
    torch.cuda.synchronize()
    return {**out, "dlogits": dlogits, "status": int(status.item())}


def weights(c, r, A):
    """The routing weights as functions of the affinities, 0 at empty slots."""
    e = r["eid"].clamp(min=0)
    w = torch.where(r["eid"] >= 0, A[r["tok"], e], 0.0)
    if c["renorm"]:
        w = (w.view(c["T"], -1) / w.view(c["T"], -1).sum(-1, keepdim=True)).reshape(-1)
    return w


@pytest.mark.parametrize("name", list(CASES))
def test_against_fp64(name):
    c = CASES[name]
    r, o = operands(c)
    out = run(c, r, o)
    assert out["status"] == 0
    z = leaf(torch.log(o["probs"].double()))
    A = torch.softmax(z, -1)
    loss = (weights(c, r, A) * o["dw"].double()).sum()
    if c["aux"]:
        loss = loss + (A * o["dprobs"].double()).sum()
    dz = torch.autograd.grad(loss, z)[0]
    # |dA|: dw of the slots (renormalised: (|dw| + sum |dw| w) / S) and dprobs
    A = A.detach()
    dw = o["dw"].double().abs() * (r["eid"] >= 0)
    if c["renorm"]:
        w = r["w"].double().view(c["T"], -1)
        S = A.gather(1, r["eid"].view(c["T"], -1)).sum(-1, keepdim=True)
        dw = ((dw.view(c["T"], -1) + (dw.view(c["T"], -1) * w).sum(-1, keepdim=True)) / S).reshape(-1)
    dA = o["dprobs"].double().abs() if c["aux"] else torch.zeros_like(A)
    dA = dA.index_put((r["tok"], r["eid"].clamp(min=0)), dw, accumulate=True)
    mag = A * (dA + (A * dA).sum(-1, keepdim=True))
    step = 3 * (c["E"] / 32 + 10)
    within("dlogits", out["dlogits"], dz, mag, step)
    within("dz_prev", out["dz_prev"], 0.5 * dz, mag, step)
    within("dbias", out["dbias"], dz.sum(0), mag.sum(0), step + c["T"])
    x, W = o["x"].double(), o["W_r"].double()
    within("dW_r", out["dW_r"], dz.t() @ x, mag.t() @ x.abs(), step + 2 * c["T"])
    within("dx", out["dx"], dz @ W, mag @ W.abs(), step + 2 * c["E"] + 4)


def test_gradient_against_differences():
    c = CASES["f32"]
    r, o = operands(c)
    out = run(c, r, o)
    g = torch.Generator().manual_seed(4)
    x, W = o["x"].double(), o["W_r"].double()
    # Logits whose softmax is the given affinities, moved by x and W_r.
    z0 = torch.log(o["probs"].double()) - x @ W.t()

    def loss(x, W):
        A = torch.softmax(z0 + x @ W.t(), -1)
        return float((weights(c, r, A) * o["dw"].double()).sum() + (A * o["dprobs"].double()).sum())
    h = 1e-5
    for what, base in (("dx", x), ("dW_r", W)):
        v = torch.randn(base.shape, generator=g).double()
        a = (x + h * v, W) if what == "dx" else (x, W + h * v)
        b = (x - h * v, W) if what == "dx" else (x, W - h * v)
        num, got = (loss(*a) - loss(*b)) / (2 * h), out[what].double().cpu()
        assert abs(num - float((got * v).sum())) <= 1e-5 * float((got.abs() * v.abs()).sum()) + 1e-5, what


@pytest.mark.parametrize("name", ["top2", "e33", "f32", "ec"])
def test_left_out_outputs(name):
    c = CASES[name]
    r, o = operands(c)
    full = run(c, r, o)
    for outs in (("dx",), ("dW_r",), ("dbias",), ("dz_prev",), ("dbias", "dx"), ()):
        part = run(c, r, o, outs)
        for k in outs + ("dlogits",):
            assert torch.equal(part[k], full[k]), (outs, k)


def test_bad_ids_are_flagged():
    m = _moe()
    c = CASES["top2"]
    r, o = operands(c)
    good = run(c, r, o)
    r["sel"][10] = 99
    r["sel"][21] = -2
    out = run(c, r, o)
    assert out["status"] & m.DEV_BAD_EXPERT
    tok = r["tok"]
    same = torch.ones(c["T"], dtype=torch.bool)
    same[[int(tok[10]), int(tok[21])]] = False
    assert torch.equal(out["dlogits"].cpu()[same], good["dlogits"].cpu()[same])
    assert torch.isfinite(out["dlogits"]).all()
