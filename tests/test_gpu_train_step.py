"""A training step of the whole layer between two block norms, as a user runs
it: block_norm -> MoELayer.forward_train -> block_norm, and back through
block_norm_backward -> MoELayer.backward -> block_norm_backward, for every
routing. The layer's forward matches moe_forward, its gradients match fp64
differentiation of the same routing, and an fp32 step matches differences.

Tolerances are normwise (max |got - ref| / max |ref|). bf16: each of the
steps in a row (expert outputs, their gradients, H, dU, dx_perm, the router's
dx, the sum) rounds once, at most 2^-8 of its largest terms, and at most 8 of
them follow one another: 8 * 2^-8 = 3.2e-2. fp32: sums over at most 8192
terms and three nested levels, 1e-4 as in the layer's parity tests."""

import numpy as np
import pytest
import torch

from mixture_experts_layer_33_b200 import inputs as gen

pytestmark = pytest.mark.gpu

CASES = {
    "topk_shared": ("ditmoe_xl", dict(T=600, d=256, h=320, h_shared=200)),
    "mmoe": ("mmoe", dict(T=333, d=264, h=256, h_shared=136)),
    "constmix": ("mmoe_constmix", dict(T=200, d=128, h=128, h_shared=64)),
    "expert_choice": ("ecdit", dict(T=512, d=256, h=256)),
    "des_vote": ("des_vote", dict(T=48, d=256, h=128)),
    "des_seq": ("des_seq", dict(T=40, d=256, h=128)),
    "one_token": ("des_vanilla", dict(T=1, d=256, h=128)),
    "f32": ("tiny_fp32", dict(T=150, x_std=1.0)),
    "f32_renorm": ("tiny_fp32", dict(T=64, x_std=1.0, renorm=1)),
}
TOL = {"bf16": 3.2e-2, "f32": 1e-4}
HEAVY, IDENTITY, ZERO, CONST = 0, 1, 2, 3


def _moe():
    from mixture_experts_layer_33_b200 import moe
    return moe


def setup(name):
    m = _moe()
    wl, over = CASES[name]
    cfg = gen.workload(wl, **over)
    inp = gen.make_inputs(cfg, "cuda")
    layer = m.MoELayer(cfg, {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")})
    return m, cfg, inp, layer


def layer64(cfg, s, x, z_prev, p):
    """The layer in fp64 with the routing of `s`, differentiable; the residual is x."""
    T, E, d = cfg["T"], cfg["E"], cfg["d"]
    z = x @ p["W_r"].t()
    if p.get("logit_bias") is not None:
        z = z + p["logit_bias"]
    if z_prev is not None:
        z = z + cfg["gate_residual_scale"] * z_prev
    A = torch.softmax(z, -1)
    sel = s["sel"].long().cpu()
    n = sel.numel()
    if cfg["routing"] == "expert_choice":
        tok, C = sel, cfg["capacity"]
        eid = (torch.arange(n) // C) % E
    else:
        tok, eid = torch.arange(n) // cfg["k"], sel
    w = torch.where(eid >= 0, A[tok, eid.clamp(min=0)], 0.0)
    if cfg.get("renorm"):
        w = (w.view(T, -1) / w.view(T, -1).sum(-1, keepdim=True)).reshape(-1)

    def mlp(v, W1, W2, gated):
        u = v @ W1.t()
        if gated:
            a, b = u.chunk(2, -1)
            return (torch.nn.functional.silu(a) * b) @ W2.t()
        return torch.nn.functional.gelu(u) @ W2.t()
    y = x
    if p.get("Ws1") is not None:
        y = y + mlp(x, p["Ws1"], p["Ws2"], False)
    nc = 0
    for e, kind in enumerate(cfg["kinds"]):
        at = (eid == e).nonzero()[:, 0]
        c, nc = nc, nc + (kind == CONST)
        if at.numel() == 0 or kind == ZERO:
            continue
        v = x[tok[at]]
        if kind == HEAVY:
            out = mlp(v, p["W1"][e], p["W2"][e], cfg["act"] == "swiglu")
        elif kind == IDENTITY:
            out = v
        elif cfg.get("const_mix"):
            a = torch.softmax(v @ p["const_vecs"][c, 1:].t(), -1)
            out = a[:, :1] * v + a[:, 1:] * p["const_vecs"][c, 0]
        else:
            out = p["const_vecs"][c].expand_as(v)
        y = y.index_add(0, tok[at], w[at][:, None] * out)
    return y


def close(what, got, ref, tol):
    got, ref = got.detach().double().cpu(), ref.detach()
    scale = float(ref.abs().max())
    err = float((got - ref).abs().max())
    assert np.isfinite(err) and err <= tol * scale + 1e-30, f"{what}: {err / max(scale, 1e-30):.2e}"


@pytest.mark.parametrize("name", list(CASES))
def test_layer_gradients(name):
    m, cfg, inp, layer = setup(name)
    x, zp = inp["x"], inp["z_prev"]
    y, s = layer.forward_train(x, z_prev=zp)
    close("forward", y, layer(x, z_prev=zp).double().cpu(), 2e-2 if cfg["dtype"] == "bf16" else 1e-4)
    g = torch.Generator(device="cuda").manual_seed(11)
    dy = torch.randn(y.shape, generator=g, device="cuda").to(y.dtype)
    grads = layer.backward(s, dy)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    p = {k: (v.double().cpu().requires_grad_() if v is not None else None) for k, v in layer.w.items()}
    x64 = x.double().cpu().requires_grad_()
    z64 = zp.double().cpu().requires_grad_() if zp is not None else None
    ref = layer64(cfg, s, x64, z64, p)
    leaves = {"x": x64, **({"z_prev": z64} if z64 is not None else {}), **{k: v for k, v in p.items() if v is not None}}
    want = dict(zip(leaves, torch.autograd.grad(ref, list(leaves.values()), dy.double().cpu(), allow_unused=True,
                                                materialize_grads=True)))
    assert set(grads) == set(want)
    for k in want:
        close(k, grads[k], want[k], TOL[cfg["dtype"]])


def test_fp32_layer_against_differences():
    m, cfg, inp, layer = setup("f32")
    x = inp["x"]
    y, s = layer.forward_train(x)
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn(y.shape, generator=g, device="cuda")
    grads = layer.backward(s, dy)
    p = {k: (v.double().cpu() if v is not None else None) for k, v in layer.w.items()}
    base = dict(p, x=x.double().cpu())
    dy64 = dy.double().cpu()

    def loss(q):
        return float((layer64(cfg, s, q["x"], None, q) * dy64).sum())
    for k in ("x", "W_r", "W1", "W2"):
        v = torch.randn(base[k].shape, generator=torch.Generator().manual_seed(5)).double()
        h = 1e-6
        num = (loss(dict(base, **{k: base[k] + h * v})) - loss(dict(base, **{k: base[k] - h * v}))) / (2 * h)
        got = grads[k].double().cpu()
        assert abs(num - float((got * v).sum())) <= 1e-4 * float((got.abs() * v.abs()).sum()) + 1e-5, k


@pytest.mark.parametrize("name", ["mmoe", "expert_choice", "f32"])
def test_block_with_norms(name):
    """z = pre(x) into the layer, its output through the gate into the residual stream and the
    next block's norm, and all the way back: the gradients of x and of the conditions."""
    m, cfg, inp, layer = setup(name)
    T, d, dt = cfg["T"], cfg["d"], inp["x"].dtype
    gs = 50
    B = -(-T // gs)
    g = torch.Generator(device="cuda").manual_seed(21)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)
    cond = rnd(B, 3 * d, std=0.3)
    gate, scale, shift = (cond[:, i * d:(i + 1) * d] for i in range(3))
    enter = m.make_norm_config(dict(T=T, d=d, dtype=cfg["dtype"], group_size=gs, pre="layer"))
    leave = m.make_norm_config(dict(T=T, d=d, dtype=cfg["dtype"], group_size=gs, pre="rms", post="rms"))
    x = rnd(T, d)
    a, y, z = (torch.empty_like(x) for _ in range(3))
    m.block_norm(enter, None, x, z=a, scale=scale, shift=shift)
    h, s = layer.forward_train(a, z_prev=inp["z_prev"], residual=None)
    m.block_norm(leave, h, x, y=y, z=z, gate=gate)
    dy, dz = rnd(T, d), rnd(T, d)
    ws = m.alloc_block_norm_workspace(leave)
    dh, dres, dx = (torch.empty_like(x) for _ in range(3))
    dcond = torch.empty(B, 3 * d, device="cuda")
    dgate, dscale, dshift = (dcond[:, i * d:(i + 1) * d] for i in range(3))
    m.block_norm_backward(leave, h, y, dz, dy, ws, dh=dh, dx=dres, gate=gate, dgate=dgate)
    ga = layer.backward(s, dh)["x"]
    m.block_norm_backward(enter, None, x, ga, dres, ws, dx=dx, scale=scale, dscale=dscale, dshift=dshift)
    torch.cuda.synchronize()
    c64 = [t.double().cpu().requires_grad_() for t in (gate, scale, shift)]
    x64 = x.double().cpu().requires_grad_()
    row = torch.arange(T) // gs
    p = {k: (v.double().cpu() if v is not None else None) for k, v in layer.w.items()}
    zp = inp["z_prev"].double().cpu() if inp["z_prev"] is not None else None
    mu = x64 - x64.mean(-1, keepdim=True)
    a64 = mu / torch.sqrt((mu * mu).mean(-1, keepdim=True) + 1e-6) * (1 + c64[1][row]) + c64[2][row]
    h64 = layer64(cfg, s, a64, zp, p) - a64  # no residual inside

    def rms(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)
    y64 = x64 + c64[0][row] * rms(h64)
    z64 = rms(y64)
    loss = (y64 * dy.double().cpu()).sum() + (z64 * dz.double().cpu()).sum()
    want = torch.autograd.grad(loss, [x64] + c64)
    # Two more norms in the chain, each way: twice the layer's bound.
    tol = 2 * TOL[cfg["dtype"]]
    close("y", y, y64, tol)
    close("z", z, z64, tol)
    for what, got, ref in zip(("dx", "dgate", "dscale", "dshift"), (dx, dgate, dscale, dshift), want):
        close(what, got, ref, tol)


def test_step_is_repeatable_and_captured():
    """The same bits on every run, and from a captured graph of the whole step."""
    m, cfg, inp, layer = setup("mmoe")
    dy = torch.randn_like(inp["x"].float()).to(inp["x"].dtype)

    def step():
        y, s = layer.forward_train(inp["x"], z_prev=inp["z_prev"])
        return {"y": y, **layer.backward(s, dy)}
    first = step()
    torch.cuda.synchronize()
    again = step()
    for k in first:
        assert torch.equal(first[k], again[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for v in held.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], held[k]), k


def test_two_layers_at_once_with_inputs_changing_between_steps():
    """Steps of two layers on two streams, eager and as graphs replayed at once. Each step's
    input is written by the stream itself just before it, nothing waits in between: the bits
    are those of the same steps one at a time."""
    layers = [setup(n) for n in ("mmoe", "constmix")]
    xs, dys, want = [], [], []
    for m, cfg, inp, layer in layers:
        g = torch.Generator(device="cuda").manual_seed(7)
        like = inp["x"]
        xs.append([torch.randn(like.shape, generator=g, device="cuda").to(like.dtype) for _ in range(3)])
        dys.append([torch.randn(like.shape, generator=g, device="cuda").to(like.dtype) for _ in range(3)])
    x_in = [torch.empty_like(x[0]) for x in xs]
    dy_in = [torch.empty_like(d[0]) for d in dys]

    def step(i):
        _, _, inp, layer = layers[i]
        y, s = layer.forward_train(x_in[i], z_prev=inp["z_prev"])
        return {"y": y, **layer.backward(s, dy_in[i])}

    for i in range(2):
        want.append([])
        for k in range(3):
            x_in[i].copy_(xs[i][k])
            dy_in[i].copy_(dys[i][k])
            torch.cuda.synchronize()
            want[i].append({n: t.clone() for n, t in step(i).items()})
            torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    torch.cuda.synchronize()
    for r in range(12):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                x_in[i].copy_(xs[i][r % 3])
                dy_in[i].copy_(dys[i][r % 3])
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        for r, out in enumerate(got[i]):
            for n, t in out.items():
                assert torch.equal(t, want[i][r % 3][n]), ("eager", i, r, n)
    graphs, held = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            held.append(step(i))
    kept = [[], []]
    for r in range(12):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                x_in[i].copy_(xs[i][r % 3])
                dy_in[i].copy_(dys[i][r % 3])
                graphs[i].replay()
                kept[i].append({n: t.clone() for n, t in held[i].items()})
    torch.cuda.synchronize()
    for i in range(2):
        for r, out in enumerate(kept[i]):
            for n, t in out.items():
                assert torch.equal(t, want[i][r % 3][n]), ("graph", i, r, n)
