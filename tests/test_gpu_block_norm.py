"""The block norms and their gradient against fp64 and differences: every
pair of norm kinds, with and without weights, conditions and operands, one
token to ragged groups, one-token groups, widths from 8 to the limit, both
types, strided conditions, aliased outputs, a mean far from zero, rows of
zeros, another stream and a captured graph.

Error bounds. A row sum is a chain of at most 16 columns per thread, 5
shuffles and 16 warps: 40 half-steps of its terms. So a normalised row is
within 3 * 40 + 10 = 130 half-steps of r (|v| + |mean|) (mean, mean square,
root and product), and a gradient that passes through two norms and the
means of products of two such rows within 1000 half-steps of the same
expression on magnitudes. Sums over tokens add a step per token at most."""

import itertools

import pytest
import torch

from grad_helpers import within

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _moe():
    from mixture_experts_layer_33_b200 import moe
    return moe


def case(T, d, group=0, pre="layer", post="none", dtype="bf16", affine=1, cond=1, alpha=1.0, shift=0.0, h=1, x=1):
    return dict(T=T, d=d, group_size=group, pre=pre, post=post, dtype=dtype, affine=affine, cond=cond, eps=EPS,
                res_scale=alpha, offset=shift, h=h, x=x)


CASES = {f"{pre}_{post}_{dt}": case(70, 264, 16, pre, post, dt, alpha=0.75)
         for pre, post, dt in itertools.product(("layer", "rms"), ("none", "layer", "rms"), ("bf16", "f32"))}
CASES.update({
    "one_token": case(1, 8, pre="rms", post="layer"),
    "plain": case(33, 72, affine=0, cond=0),
    "no_affine": case(300, 136, 77, "layer", "rms", affine=0),
    "no_cond": case(700, 520, 0, "rms", "rms", cond=0),
    "token_groups": case(90, 64, 1, "layer", "rms"),
    "small_groups": case(1001, 200, 3, "rms", "layer", "f32"),
    "group_past_end": case(50, 64, 4096, "layer", "layer"),
    "one_condition": case(1500, 328, 0, "layer", "none"),
    "many_tokens": case(5000, 1152, 256, "layer", "rms"),
    "wide": case(20, 4096, 8, "layer", "rms"),
    "widest": case(9, 8192, 4, "rms", "layer"),
    "widest_f32": case(700, 4104, 300, "layer", "none", "f32"),
    "mean_far": case(60, 1024, 16, "layer", "layer", "f32", shift=300.0),
    "entry": case(64, 256, 16, "layer", "none", h=0),
    "no_residual": case(64, 256, 16, "layer", "rms", x=0),
})


def operands(c, seed=1):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    T, d = c["T"], c["d"]
    B = -(-T // c["group_size"]) if c["group_size"] else 1

    def t(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dt)
    o = {"h": t(T, d) if c["h"] else None, "x": (t(T, d) + c["offset"]).to(dt) if c["x"] else None,
         "y": (t(T, d) + c["offset"]).to(dt), "dz": t(T, d), "dy": t(T, d)}
    if T > 3:
        o["y"][2] = 0  # a row of zeros: n = 0, r = 1 / sqrt(eps)
        if o["h"] is not None:
            o["h"][2] = 0
    cond = t(B, 3 * d + 8, std=0.5)
    for i, n in enumerate(("gate", "scale", "shift")):
        o[n] = cond[:, i * d:(i + 1) * d] if c["cond"] else None
    if not c["h"]:
        o["gate"] = None
    a = c["affine"]
    o["pre_gamma"], o["pre_beta"] = (1 + t(d, std=0.2), t(d, std=0.2)) if a else (None, None)
    o["post_gamma"] = 1 + t(d, std=0.2) if a and c["post"] != "none" and c["h"] else None
    return o, dt, B


def to_gpu(o):
    G = {k: v.cuda() if isinstance(v, torch.Tensor) and v.is_contiguous() else v for k, v in o.items()}
    for n in ("gate", "scale", "shift"):  # keep the rows strided as the projection's chunks are
        if o[n] is not None:
            full = torch.empty(o[n].shape[0], o[n].stride(0) if o[n].shape[0] > 1 else 3 * o[n].shape[1] + 8,
                               dtype=o[n].dtype, device="cuda")
            G[n] = full[:, :o[n].shape[1]]
            G[n].copy_(o[n])
    return G


def rows(c, t):
    if t is None:
        return None
    return t[torch.arange(c["T"]) // c["group_size"]] if c["group_size"] else t.expand(c["T"], -1)


def norm(v, kind):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def norm_mag(v, av, kind):
    """r (|v| + mean |v|): what a normalised row's error scales with, from the row's magnitude av."""
    if kind == "none":
        return av
    m = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    r = 1 / torch.sqrt((m * m).mean(-1, keepdim=True) + EPS)
    return r * (av + av.mean(-1, keepdim=True))


def forward64(c, o):
    f = {k: v.double() if isinstance(v, torch.Tensor) else None for k, v in o.items()}
    one = torch.ones((), dtype=torch.float64)
    pg = f["post_gamma"] if f["post_gamma"] is not None else one
    gt = rows(c, f["gate"]) if f["gate"] is not None else one
    y = torch.zeros(c["T"], c["d"], dtype=torch.float64)
    my = y.clone()
    if f["x"] is not None:
        y, my = y + c["res_scale"] * f["x"], my + c["res_scale"] * f["x"].abs()
    if f["h"] is not None:
        y = y + gt * norm(f["h"], c["post"]) * pg
        my = my + (gt * pg).abs() * norm_mag(f["h"], f["h"].abs(), c["post"])
    ga = f["pre_gamma"] if f["pre_gamma"] is not None else one
    be = f["pre_beta"] if f["pre_beta"] is not None else 0 * one
    sc = 1 + rows(c, f["scale"]) if f["scale"] is not None else one
    sh = rows(c, f["shift"]) if f["shift"] is not None else 0 * one
    z = (norm(y, c["pre"]) * ga + be) * sc + sh
    mz = (norm_mag(y, my, c["pre"]) * ga.abs() + be.abs()) * sc.abs() + sh.abs()
    return y, my, z, mz


@pytest.mark.parametrize("name", list(CASES))
def test_forward_against_fp64(name):
    m = _moe()
    c = CASES[name]
    o, dt, _ = operands(c)
    G = to_gpu(o)
    n = m.make_norm_config(c)
    y, z = (torch.empty(c["T"], c["d"], dtype=dt, device="cuda") for _ in range(2))
    args = dict(post_gamma=G["post_gamma"], gate=G["gate"])
    pre = dict(pre_gamma=G["pre_gamma"], pre_beta=G["pre_beta"], scale=G["scale"], shift=G["shift"])
    m.block_norm(n, G["h"], G["x"], y=y, z=z, **args, **pre)
    ry, my, rz, mz = forward64(c, o)
    within("y", y, ry, my, 140)
    within("z", z, rz, mz, 2 * 140)
    # Either output alone gives the same bytes; y may be x's buffer.
    y2, z2 = torch.empty_like(y), torch.empty_like(z)
    m.block_norm(n, G["h"], G["x"], y=y2, **args)
    m.block_norm(n, G["h"], G["x"], z=z2, **args, **pre)
    assert torch.equal(y2, y) and torch.equal(z2, z)
    if G["x"] is not None:
        buf = G["x"].clone()
        m.block_norm(n, G["h"], buf, y=buf, z=z2, **args, **pre)
        assert torch.equal(buf, y) and torch.equal(z2, z)


def grads64(c, o):
    """Gradients in fp64 (by differentiation at the given y) and magnitudes."""
    f = {k: v.double().contiguous().requires_grad_() if isinstance(v, torch.Tensor) else None for k, v in o.items()}
    one = torch.ones((), dtype=torch.float64)
    ga = f["pre_gamma"] if f["pre_gamma"] is not None else one
    be = f["pre_beta"] if f["pre_beta"] is not None else 0 * one
    sc = 1 + rows(c, f["scale"]) if f["scale"] is not None else one
    dz, dy = o["dz"].double(), o["dy"].double()
    n = norm(f["y"], c["pre"])
    shift = torch.zeros_like(f["scale"]).requires_grad_() if f["scale"] is not None else None
    z = (n * ga + be) * sc + (rows(c, shift) if shift is not None else 0)
    names = [k for k in ("pre_gamma", "pre_beta", "scale") if f[k] is not None]
    got = torch.autograd.grad(z, [f["y"]] + [f[k] for k in names] + ([shift] if shift is not None else []), dz)
    res = {"d" + k: v for k, v in zip(names + ["shift"], got[1:])}
    t = dy + got[0]
    res["dx"] = c["res_scale"] * t
    pg = f["post_gamma"] if f["post_gamma"] is not None else one
    gt = rows(c, f["gate"]) if f["gate"] is not None else one
    mh = None
    if f["h"] is not None:
        u = norm(f["h"], c["post"])
        names = [k for k in ("post_gamma", "gate") if f[k] is not None]
        got = torch.autograd.grad(gt * u * pg, [f["h"]] + [f[k] for k in names], t)
        res["dh"] = got[0]
        res.update({"d" + k: v for k, v in zip(names, got[1:])})
    # Magnitudes.
    d64 = lambda v: v.detach()  # noqa: E731
    y, h = d64(f["y"]), d64(f["h"]) if f["h"] is not None else None

    def grad_mag(g, v, kind):
        if kind == "none":
            return g
        mv = v - v.mean(-1, keepdim=True) if kind == "layer" else v
        r = 1 / torch.sqrt((mv * mv).mean(-1, keepdim=True) + EPS)
        nm = norm_mag(v, v.abs(), kind)
        return r * (g + g.mean(-1, keepdim=True) + nm * (g * nm).mean(-1, keepdim=True))
    sc_, ga_, be_, gt_, pg_ = (d64(v).abs() for v in (sc, ga, be, gt, pg))
    nm = norm_mag(y, y.abs(), c["pre"])
    mt = dy.abs() + grad_mag((dz.abs() * sc_ * ga_), y, c["pre"])
    mag = {"dx": abs(c["res_scale"]) * mt}

    def per_group(t):
        B = -(-c["T"] // c["group_size"]) if c["group_size"] else 1
        idx = torch.arange(c["T"]) // c["group_size"] if c["group_size"] else torch.zeros(c["T"], dtype=torch.long)
        return torch.zeros(B, c["d"], dtype=torch.float64).index_add(0, idx, t.expand(c["T"], -1))
    mag["dshift"], mag["dscale"] = per_group(dz.abs()), per_group(dz.abs() * (nm * ga_ + be_))
    mag["dpre_beta"], mag["dpre_gamma"] = (dz.abs() * sc_).sum(0), (dz.abs() * sc_ * nm).sum(0)
    if h is not None:
        um = norm_mag(h, h.abs(), c["post"])
        mag["dgate"], mag["dpost_gamma"] = per_group(mt * um * pg_), (mt * gt_ * um).sum(0)
        mag["dh"] = grad_mag(mt * gt_ * pg_, h, c["post"])
    return {k: v.detach() for k, v in res.items()}, mag


def run_bwd(c, o, dt, B, alias=False, stream=None):
    m = _moe()
    G = to_gpu(o)
    n = m.make_norm_config(c)
    T, d = c["T"], c["d"]
    out = {"dx": torch.empty(T, d, dtype=dt, device="cuda")}
    if alias:
        out["dx"] = G["dy"]
    if o["h"] is not None:
        out["dh"] = G["dz"] if alias else torch.empty(T, d, dtype=dt, device="cuda")
    cond = torch.full((B, 3 * d + 4), float("nan"), device="cuda")
    for i, k in enumerate(("gate", "scale", "shift")):
        if o[k] is not None:
            out["d" + k] = cond[:, i * d:(i + 1) * d]
    for k in ("pre_gamma", "pre_beta", "post_gamma"):
        if o[k] is not None:
            out["d" + k] = torch.full((d,), float("nan"), device="cuda")
    ws = m.alloc_block_norm_workspace(n)
    ws.fill_(255)

    def go(s=None):
        m.block_norm_backward(n, G["h"], G["y"], G["dz"], G["dy"], ws, post_gamma=G["post_gamma"], gate=G["gate"],
                              pre_gamma=G["pre_gamma"], pre_beta=G["pre_beta"], scale=G["scale"], stream=s, **out)
    go(stream)
    return out, go


@pytest.mark.parametrize("name", list(CASES))
def test_backward_against_fp64(name):
    c = CASES[name]
    o, dt, B = operands(c)
    out, _ = run_bwd(c, o, dt, B)
    ref, mag = grads64(c, o)
    assert set(out) == {k for k in ref if k in out}
    for k, v in out.items():
        tokens = 0 if k in ("dx", "dh") else min(c["T"], 200 + c["T"] // 8)
        within(k, v, ref[k], mag[k], 1000 + tokens)
    again, _ = run_bwd(c, o, dt, B, alias=True)
    for k in out:
        assert torch.equal(again[k], out[k]), k


def test_gradient_against_differences():
    c = CASES["layer_rms_f32"]
    o, dt, B = operands(c)
    # The gradient at the forward's own y.
    y0, _, _, _ = forward64(c, o)
    o["y"] = y0.float()
    out, _ = run_bwd(c, o, dt, B)
    dz, dy = o["dz"].double(), o["dy"].double()
    g = torch.Generator().manual_seed(8)

    def loss(p):
        y, _, z, _ = forward64(c, p)
        return float((y * dy).sum() + (z * dz).sum())
    for k in ("h", "x", "gate", "scale", "shift", "pre_gamma", "pre_beta", "post_gamma"):
        v = torch.randn(o[k].shape, generator=g).double()
        v[2 if k in ("h", "x") else slice(0, 0)] = 0  # not the row of zeros: its curvature is 1 / eps
        h = 1e-6
        hi, lo = dict(o), dict(o)
        hi[k], lo[k] = o[k].double() + h * v, o[k].double() - h * v
        num = (loss(hi) - loss(lo)) / (2 * h)
        got = out["d" + k].double().cpu()
        # fp32 steps of each element; y is rounded to fp32 between the two.
        assert abs(num - float((got * v).sum())) <= 1e-4 * float((got.abs() * v.abs()).sum()) + 1e-4, k


def test_one_sided_gradients():
    """Without dz the step is the residual sum alone; without dy the norm's; sums of both is the whole."""
    m = _moe()
    c = CASES["rms_rms_f32"]
    o, dt, B = operands(c)
    G = to_gpu(o)
    n = m.make_norm_config(c)
    ws = m.alloc_block_norm_workspace(n)
    dx = {k: torch.empty_like(G["y"]) for k in ("z", "y", "both")}
    common = dict(gate=G["gate"], post_gamma=G["post_gamma"], pre_gamma=G["pre_gamma"], scale=G["scale"])
    m.block_norm_backward(n, None, None, None, G["dy"], ws, dx=dx["y"], **common)
    assert torch.equal(dx["y"], c["res_scale"] * G["dy"])
    m.block_norm_backward(n, None, G["y"], G["dz"], None, ws, dx=dx["z"], **common)
    m.block_norm_backward(n, None, G["y"], G["dz"], G["dy"], ws, dx=dx["both"], **common)
    # Each is rounded a few times at the size of its terms.
    bound = 8 * 2.0 ** -24 * (dx["z"].abs() + dx["y"].abs())
    assert ((dx["both"] - (dx["z"] + dx["y"])).abs() <= bound).all()
    dh = torch.empty_like(G["h"])
    m.block_norm_backward(n, G["h"], None, None, G["dy"], ws, dh=dh, **common)
    ref = torch.autograd.grad(rows(c, o["gate"].double()) * norm((hh := o["h"].double().requires_grad_()), "rms")
                              * o["post_gamma"].double(), hh, o["dy"].double())[0]
    fine = torch.arange(c["T"]) != 2
    torch.testing.assert_close(dh.double().cpu()[fine], ref[fine], rtol=1e-4, atol=1e-4)


def test_another_stream_and_a_captured_graph():
    c = CASES["many_tokens"]
    o, dt, B = operands(c)
    out, go = run_bwd(c, o, dt, B)
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in out.items()}
    s = torch.cuda.Stream()
    for run in ("stream", "graph"):
        for v in out.values():
            v.zero_()
        torch.cuda.synchronize()
        if run == "stream":
            go(s)
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                go()
            for v in out.values():
                v.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for k, v in out.items():
            assert torch.equal(v, first[k]), (run, k)
