"""Gradient of the grouped expert MLP against fp64 products of the formulas
and against differences: both activations and types, empty groups, groups of
one row, rows that end inside a 64-row K block and inside a 256-row tile,
widths off the tiles, garbage past the last row, a shared expert, left-out
outputs, another stream and a captured graph.

Error bounds (bf16): H and dU are rounded once (2^-8 of their terms), the
output once more; act'(U) and act(U) are within 4e-6 (1 + |U|) of their
exact values (Abramowitz & Stegun 7.1.26 and the hardware's exponential and
reciprocal) plus the shift of U by its own fp32 sum over d. A sum of K
products on the tensor cores is within 2 K half-steps (2^-24) of the terms'
magnitudes. fp32 layers: K half-steps, act' within 1e-6 (1 + |U|)."""

import math

import pytest
import torch

from grad_helpers import F32, HALF, within

pytestmark = pytest.mark.gpu

CASES = {
    # counts: rows of each expert
    "gelu_small": dict(d=64, h=64, act="gelu", dtype="bf16", counts=[5, 0, 64, 1]),
    "swiglu_small": dict(d=64, h=64, act="swiglu", dtype="bf16", counts=[5, 0, 64, 1]),
    "gelu_tiles": dict(d=264, h=328, act="gelu", dtype="bf16", counts=[257, 3, 130, 0, 511], hs=200),
    "swiglu_tiles": dict(d=136, h=200, act="swiglu", dtype="bf16", counts=[33, 300, 63, 65], hs=72),
    "narrow": dict(d=8, h=8, act="gelu", dtype="bf16", counts=[1, 9]),
    "narrow_swiglu": dict(d=16, h=24, act="swiglu", dtype="bf16", counts=[130, 2], hs=8),
    "wide": dict(d=1152, h=512, act="gelu", dtype="bf16", counts=[700, 100], hs=264),
    "one_row": dict(d=512, h=256, act="swiglu", dtype="bf16", counts=[0, 0, 1, 0]),
    "no_rows": dict(d=64, h=72, act="gelu", dtype="bf16", counts=[0, 0, 0]),
    "many_experts": dict(d=72, h=96, act="gelu", dtype="bf16", counts=[(7 * e) % 11 for e in range(100)]),
    # Many tiles per CTA pair, nearly all of them one tail block: the two CTAs
    # of a pair drift apart by as much as the ring allows.
    "many_tails": dict(d=520, h=776, act="swiglu", dtype="bf16", counts=[1 + e % 9 for e in range(128)]),
    "tails_and_blocks": dict(d=776, h=520, act="gelu", dtype="bf16", counts=[(e * 37) % 150 for e in range(60)]),
    "f32_gelu": dict(d=72, h=136, act="gelu", dtype="f32", counts=[5, 0, 70, 1], hs=40),
    "f32_swiglu": dict(d=40, h=72, act="swiglu", dtype="f32", counts=[17, 64, 0]),
}
SPARE = 11  # assignments past the last heavy row (those of zero-computation experts)


def _moe():
    from mixture_experts_layer_33_b200 import moe
    return moe


def make(c, seed=5):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    E, d, h, hs = len(c["counts"]), c["d"], c["h"], c.get("hs", 0)
    up = 2 * h if c["act"] == "swiglu" else h
    n = sum(c["counts"])
    T = n + SPARE  # top-1: one assignment per token
    off = torch.tensor([0] + torch.tensor(c["counts"]).cumsum(0).tolist(), dtype=torch.int32)

    def t(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dt)
    o = dict(x_perm=t(T, d), dy_perm=t(T, d, std=0.5), W1=t(E, up, d, std=1 / math.sqrt(d)),
             W2=t(E, d, h, std=1 / math.sqrt(h)), x=t(T, d), dy=t(T, d, std=0.5))
    o["x_perm"][n:] = float("nan")
    o["dy_perm"][n:] = float("inf")
    if hs:
        o.update(Ws1=t(hs, d, std=1 / math.sqrt(d)), Ws2=t(d, hs, std=1 / math.sqrt(hs)))
    cfg = dict(T=T, d=d, h=h, E=E, k=1, n_shared=1 if hs else 0, h_shared=hs, dtype=c["dtype"], act=c["act"],
               routing="token_topk")
    return cfg, off, o, dt


def outputs(cfg, o, dt):
    out = {"dx_perm": torch.full_like(o["x_perm"], -3.0), "dW1": torch.full_like(o["W1"], float("nan")),
           "dW2": torch.full_like(o["W2"], float("nan"))}
    if "Ws1" in o:
        out.update(dx_shared=torch.full_like(o["x"], float("nan")), dWs1=torch.full_like(o["Ws1"], float("nan")),
                   dWs2=torch.full_like(o["Ws2"], float("nan")))
    return {k: v.cuda() for k, v in out.items()}


def call(m, c, off, G, out, status, ws, stream=None):
    m.grouped_mlp_backward(c, G["x_perm"], off, G["W1"], G["W2"], G["dy_perm"], G["x"], G.get("Ws1"), G.get("Ws2"),
                           G["dy"], status, ws, stream=stream, **out)


def grads64(x, dy, W1, W2, act):
    """(dx, dW1, dW2) of one expert in fp64 and the magnitudes their errors scale with."""
    x, dy, W1, W2 = (t.double() for t in (x, dy, W1, W2))
    u, dh = x @ W1.t(), dy @ W2
    su = x.abs() @ W1.abs().t()          # magnitude of U's terms
    sh = dy.abs() @ W2.abs()             # ... of dH's
    if act == "swiglu":
        a, b = u.chunk(2, -1)
        sg = torch.sigmoid(a)
        H, f1, f2 = a * sg * b, b * sg * (1 + a * (1 - sg)), a * sg
        dU = torch.cat([dh * f1, dh * f2], -1)
        sua, sub = su.chunk(2, -1)
        # slopes of H, f1, f2 in (a, b) are below 1.1 (1 + |b|) and 1.1
        mH, m1, m2 = (1 + b.abs()) * sua + a.abs() * sub, sub + (1 + b.abs()) * sua, sua
        mU = torch.cat([sh * f1.abs() + dh.abs() * m1, sh * f2.abs() + dh.abs() * m2], -1)
        aU = torch.cat([dh.abs() * (1 + b.abs()), dh.abs() * (1 + a.abs())], -1)
        aH = (1 + a.abs()) * (1 + b.abs())
    else:
        phi = 0.5 * torch.special.erfc(-u * math.sqrt(0.5))
        pdf = torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
        H, f = u * phi, phi + u * pdf
        dU = dh * f
        mH, mU = 1.2 * su, sh * f.abs() + dh.abs() * su   # |GELU'| < 1.13, |GELU''| < 0.8
        aU, aH = dh.abs() * (1 + u.abs()), 1 + u.abs()
    return dict(dx=dU @ W1, dW1=dU.t() @ x, dW2=dy.t() @ H, H=H, dU=dU, mH=mH, mU=mU, aU=aU, aH=aH,
                x=x.abs(), dy=dy.abs(), W1=W1.abs())


def check(what, got, r, d, dtype):
    """One expert's (dx, dW1, dW2) against grads64's."""
    bf = dtype == "bf16"
    rnd = HALF[torch.bfloat16] * 1.01 if bf else F32
    act, per = (4e-6, 2) if bf else (1e-6, 1)
    n, up = r["dU"].shape
    e_H = rnd * r["H"].abs() + act * r["aH"] + per * (d + 8) * F32 * r["mH"]
    e_U = rnd * r["dU"].abs() + act * r["aU"] + per * (d + 8) * F32 * r["mU"]
    dU, H = r["dU"].abs() + e_U, r["H"].abs() + e_H
    if got[0] is not None and n:
        within(what + " dx", got[0], r["dx"], dU @ r["W1"], per * (up + 8), extra=e_U @ r["W1"])
    within(what + " dW1", got[1], r["dW1"], dU.t() @ r["x"], per * (n + 8), extra=e_U.t() @ r["x"])
    within(what + " dW2", got[2], r["dW2"], r["dy"].t() @ H, per * (n + 8), extra=r["dy"].t() @ e_H)


@pytest.mark.parametrize("name", list(CASES))
def test_against_fp64(name):
    m = _moe()
    c = CASES[name]
    cfg, off, o, dt = make(c)
    G = {k: v.cuda() for k, v in o.items()}
    out = outputs(cfg, o, dt)
    mc = m.make_config(cfg)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = m.alloc_backward_workspace(mc)
    ws.fill_(255)  # NaN bits: nothing may be read before it is written
    call(m, mc, off.cuda(), G, out, status, ws)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    n = sum(c["counts"])
    assert (out["dx_perm"][n:] == -3.0).all()
    for e, cnt in enumerate(c["counts"]):
        lo = int(off[e])
        if cnt == 0:
            assert (out["dW1"][e] == 0).all() and (out["dW2"][e] == 0).all(), e
            continue
        r = grads64(o["x_perm"][lo:lo + cnt], o["dy_perm"][lo:lo + cnt], o["W1"][e], o["W2"][e], c["act"])
        check(f"expert {e}", (out["dx_perm"][lo:lo + cnt], out["dW1"][e], out["dW2"][e]), r, c["d"], c["dtype"])
    if c.get("hs"):
        r = grads64(o["x"], o["dy"], o["Ws1"], o["Ws2"], "gelu")
        check("shared", (out["dx_shared"], out["dWs1"], out["dWs2"]), r, c["d"], c["dtype"])


def test_gradient_against_differences():
    """An fp32 layer's gradients against central differences of the fp64 MLP."""
    m = _moe()
    c = CASES["f32_swiglu"]
    cfg, off, o, dt = make(c)
    G = {k: v.cuda() for k, v in o.items()}
    out = outputs(cfg, o, dt)
    mc = m.make_config(cfg)
    call(m, mc, off.cuda(), G, out, None, m.alloc_backward_workspace(mc))
    torch.cuda.synchronize()
    e, lo, cnt, h = 1, int(off[1]), c["counts"][1], c["h"]
    x, dy, W1, W2 = (t.double() for t in (o["x_perm"][lo:lo + cnt], o["dy_perm"][lo:lo + cnt], o["W1"][e], o["W2"][e]))

    def loss(x, W1, W2):
        a, b = (x @ W1.t()).chunk(2, -1)
        return float(((a * torch.sigmoid(a) * b) @ W2.t() * dy).sum())
    g = torch.Generator().manual_seed(2)
    for what, got, args in (("x", out["dx_perm"][lo:lo + cnt], 0), ("W1", out["dW1"][e], 1), ("W2", out["dW2"][e], 2)):
        base = [x, W1, W2]
        v = torch.randn(base[args].shape, generator=g).double()
        step = 1e-5
        hi = list(base); hi[args] = base[args] + step * v
        dn = list(base); dn[args] = base[args] - step * v
        num = (loss(*hi) - loss(*dn)) / (2 * step)
        got = got.double().cpu()
        assert abs(num - float((got * v).sum())) <= 1e-5 * float((got.abs() * v.abs()).sum()) + 1e-5, what


@pytest.mark.parametrize("name", ["gelu_tiles", "swiglu_tiles", "f32_gelu"])
def test_left_out_outputs_leave_the_others_alone(name):
    m = _moe()
    cfg, off, o, dt = make(CASES[name])
    G = {k: v.cuda() for k, v in o.items()}
    off = off.cuda()
    mc = m.make_config(cfg)
    ws = m.alloc_backward_workspace(mc)
    full = outputs(cfg, o, dt)
    call(m, mc, off, G, full, None, ws)
    n = int(off[-1])
    for keep in (["dx_perm"], ["dW1"], ["dW2"], ["dx_shared"], ["dWs1", "dx_perm"], ["dWs2", "dW1"]):
        part = {k: v for k, v in outputs(cfg, o, dt).items() if k in keep}
        call(m, mc, off, G, part, None, ws)
        for k in keep:
            rows = slice(0, n) if k == "dx_perm" else slice(None)
            assert torch.equal(part[k][rows], full[k][rows]), (keep, k)


def test_another_stream_and_a_captured_graph():
    m = _moe()
    cfg, off, o, dt = make(CASES["gelu_tiles"])
    G = {k: v.cuda() for k, v in o.items()}
    off = off.cuda()
    mc = m.make_config(cfg)
    first = outputs(cfg, o, dt)
    call(m, mc, off, G, first, None, m.alloc_backward_workspace(mc))
    torch.cuda.synchronize()
    n = int(off[-1])

    def same(out):
        torch.cuda.synchronize()
        for k, v in out.items():
            rows = slice(0, n) if k == "dx_perm" else slice(None)
            assert torch.equal(v[rows], first[k][rows]), k
    # Two calls at once, on two streams with their own workspaces.
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [outputs(cfg, o, dt) for _ in streams]
    spaces = [m.alloc_backward_workspace(mc) for _ in streams]
    torch.cuda.synchronize()
    for s, out, ws in zip(streams, outs, spaces):
        call(m, mc, off, G, out, None, ws, stream=s)
    for out in outs:
        same(out)
    out = outputs(cfg, o, dt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(m, mc, off, G, out, None, spaces[0])
    for v in out.values():
        v.zero_()
    graph.replay()
    same(out)


@pytest.mark.parametrize("c", [CASES[n] for n in ("gelu_tiles", "swiglu_tiles", "narrow", "no_rows", "many_tails",
                                                  "tails_and_blocks")] + [
    dict(d=256, h=264, act="gelu", dtype="bf16", counts=[1000, 303]),  # dW's K is long, dX has more tiles than likely
    dict(d=256, h=4608, act="gelu", dtype="bf16", counts=[8500, 7500]),  # few long tiles on both sides
], ids=str)
def test_dx_and_dw_do_not_depend_on_being_asked_for_together(c):
    # Which launch a tile runs in changes neither its products nor their order.
    m = _moe()
    cfg, off, o, dt = make(c)
    G, off, mc = {k: v.cuda() for k, v in o.items()}, off.cuda(), m.make_config(cfg)
    ws, status = m.alloc_backward_workspace(mc), torch.zeros(1, dtype=torch.int32, device="cuda")
    both, apart = outputs(cfg, o, dt), outputs(cfg, o, dt)
    call(m, mc, off, G, both, status, ws)
    for side in ([k for k in apart if k.startswith("dx")], [k for k in apart if k.startswith("dW")]):
        call(m, mc, off, G, {k: apart[k] for k in side}, status, ws)
    assert status.item() == 0
    for k in both:
        assert torch.equal(both[k].view(torch.int16), apart[k].view(torch.int16)), k
