"""Gradients of the combine and the dispatch against fp64 differentiation of
their definition, and against differences: every expert kind, mixed constant
experts, empty slots and dropped rows, token and expert choice, one token,
more than 32 slots, widths off the 256-feature chunk, bf16 and fp32; rows of
no assignment are left as they were; garbage in rows that nothing refers to;
bad ids flagged; another stream and a captured graph.

Error bounds: a warp's dot product over d values is a chain of d / 32 fused
multiply-adds per lane and 5 additions, so at most d / 32 + 6 half-steps of
the terms' magnitudes, and the mixed constant expert's coefficients pass
through three such sums and a softmax; 8 (d / 32 + 8) covers them. Sums over
tokens add at most one step each."""

import pytest
import torch

from grad_helpers import CONST, HEAVY, IDENTITY, ZERO, leaf, route, sparse_terms, within

pytestmark = pytest.mark.gpu

LIGHT = [IDENTITY, ZERO, CONST]


def case(T, d, E, k=2, dtype="bf16", light=False, mix=0, ec=None, empty=0.0, n_const=1, renorm=0):
    kinds = [HEAVY] * (E - 2 - n_const) + [IDENTITY, ZERO] + [CONST] * n_const if light else [HEAVY] * E
    c = dict(T=T, d=d, h=16, E=E, k=k, dtype=dtype, act="gelu", routing="token_topk", kinds=kinds,
             const_mix=mix, empty=empty, renorm=renorm)
    if ec:
        c.update(routing="expert_choice", group_size=ec[0], capacity=ec[1], k=0)
    return c


CASES = {
    "top2": case(300, 264, 8),
    "one_token": case(1, 8, 4, k=3, light=True),
    "f32": case(65, 72, 8, dtype="f32", light=True),
    "mix": case(130, 328, 9, k=4, light=True, mix=1, n_const=2),
    "mix_f32": case(77, 40, 6, k=3, light=True, mix=1, dtype="f32"),
    "empty_slots": case(100, 1160, 7, k=3, light=True, empty=0.4),
    "all_light": case(50, 64, 3, k=2, light=True),
    "wide_k": case(9, 128, 64, k=40, light=True, mix=1),
    "ec": case(256, 200, 8, ec=(64, 16)),
    "ec_light_mix": case(192, 520, 7, ec=(32, 20), light=True, mix=1),
    "ec_many": case(64, 64, 48, ec=(64, 50)),
    "many_tokens": case(5000, 256, 16, k=2, light=True),
}


def _moe():
    from mixture_experts_layer_33_b200 import moe
    return moe


def operands(c, seed=3):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    T, d = c["T"], c["d"]
    r = route(c, g, c.get("empty", 0.0))
    n = r["w"].numel()
    o = {n_: torch.randn(T, d, generator=g).to(dt) for n_ in ("x", "dy", "add0", "add1")}
    o["y_perm"], o["dx_perm"] = (torch.randn(n, d, generator=g).to(dt) for _ in range(2))
    used = int(r["offsets"][-1])
    o["y_perm"][used:] = float("nan")  # rows of no assignment: any bits
    o["dx_perm"][used:] = float("nan")
    nc = sum(k == CONST for k in c["kinds"])
    o["const_vecs"] = (torch.randn(*((nc, 3, d) if c["const_mix"] else (nc, d)), generator=g) * 0.1).to(dt) if nc else None
    return r, o, dt


def to_gpu(t):
    return None if t is None else t.cuda()


def run(c, r, o, stream=None, into=None):
    m = _moe()
    cfg = m.make_config(c)
    G = {k: to_gpu(v) for k, v in {**r, **o}.items() if isinstance(v, torch.Tensor) or v is None}
    n = r["w"].numel()
    out = into or {"dy_perm": torch.full((n, c["d"]), -7.0, device="cuda", dtype=o["x"].dtype),
                   "dw": torch.empty(n, device="cuda"), "dx": torch.empty_like(G["x"]),
                   "dconst": torch.empty(G["const_vecs"].shape, device="cuda") if G["const_vecs"] is not None else None,
                   "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    ws = m.alloc_backward_workspace(cfg)
    routing = (G["sel"], G["w"], G["row_of"], G["tok_ptr"], G["tok_assign"], G["x"], G["const_vecs"])

    def go(s=None):
        m.combine_backward(cfg, G["dy"], G["y_perm"], *routing, out["dy_perm"], out["dw"], out["status"], ws,
                           dconst=out["dconst"], stream=s)
        m.dispatch_backward(cfg, G["dx_perm"], G["dy"], *routing, out["dx"], out["status"],
                            add=(G["add0"], G["add1"]), stream=s)
    go(stream)
    return out, go


def reference(c, r, o):
    """Gradients of sum(y dy) + sum(x_perm dx_perm) + sum(x (add0 + add1)), by differentiation."""
    x, w, yp = leaf(o["x"]), leaf(r["w"]), leaf(torch.nan_to_num(o["y_perm"]))
    cv = leaf(o["const_vecs"]) if o["const_vecs"] is not None else None
    dy = o["dy"].double()
    row = r["row_of"].long()
    dxp = torch.nan_to_num(o["dx_perm"].double())
    terms = sparse_terms(c, r, x, w, cv, yp)
    loss = (terms * dy[r["tok"]]).sum()
    wanted = [yp, w] + ([cv] if cv is not None else [])
    got = dict(zip(("dy_perm", "dw", "dconst"), torch.autograd.grad(
        loss, wanted, allow_unused=True, materialize_grads=True, retain_graph=True)))
    loss = loss + (x[r["tok"]] * (row >= 0)[:, None] * dxp[row.clamp(min=0)]).sum()
    loss = loss + (x * (o["add0"].double() + o["add1"].double())).sum()
    got["dx"] = torch.autograd.grad(loss, x)[0]
    return got


@pytest.mark.parametrize("name", list(CASES))
def test_against_fp64(name):
    c = CASES[name]
    r, o, dt = operands(c)
    out, _ = run(c, r, o)
    torch.cuda.synchronize()
    assert int(out["status"].item()) == 0
    ref = reference(c, r, o)
    d, T = c["d"], c["T"]
    used = int(r["offsets"][-1])
    row, tok = r["row_of"].long(), r["tok"]
    dy, x = o["dy"].double().abs(), o["x"].double().abs()
    step = 8 * (d / 32 + 8)
    within("dy_perm", out["dy_perm"][:used], ref["dy_perm"][:used], ref["dy_perm"][:used].abs(), 1)
    assert (out["dy_perm"][used:] == -7.0).all()  # left as they were
    # |dw|'s terms: |dy| |E(x)|, the expert's output bounded by its parts.
    e_abs = torch.where((row >= 0)[:, None], torch.nan_to_num(o["y_perm"].double()).abs()[row.clamp(min=0)], x[tok])
    if o["const_vecs"] is not None:
        cv = o["const_vecs"].double().abs()
        e_abs = e_abs + (cv[:, 0] if c["const_mix"] else cv).sum(0)
    mag_w = (dy[tok] * e_abs).sum(-1)
    if c["const_mix"]:  # a0, a1 carry the error of a dot of |x| |Wc|
        z = (x[tok] * o["const_vecs"].double().abs()[:, 1:].sum((0, 1))).sum(-1)
        mag_w = mag_w * (1 + z)
    within("dw", out["dw"], ref["dw"], mag_w, step)
    coef = torch.zeros(T, d, dtype=torch.float64).index_add(0, tok, (r["w"].double().abs()[:, None] * dy[tok]))
    if o["const_vecs"] is not None:
        mag_c = coef.sum(0) * (1 + (float(mag_w.max()) if c["const_mix"] else 0))
        if c["const_mix"]:
            mag_c = mag_c + x.sum(0) * float(mag_w.max())
        within("dconst", out["dconst"], ref["dconst"], mag_c.expand_as(ref["dconst"]), step + T)
    mag_x = coef + o["add0"].double().abs() + o["add1"].double().abs()
    mag_x = mag_x.index_add(0, tok, (row >= 0)[:, None] * torch.nan_to_num(o["dx_perm"].double()).abs()[row.clamp(min=0)])
    if c["const_mix"]:
        wc = o["const_vecs"].double().abs()[:, 1:].sum((0, 1))
        mag_x = mag_x + (mag_w.max() * r["w"].abs().max().double()) * wc * max(1, c["k"])
    within("dx", out["dx"], ref["dx"], mag_x, step)


def test_gradient_against_differences():
    """dw and dx of an fp32 layer against central differences of the fp64 combine."""
    c = CASES["mix_f32"]
    r, o, _ = operands(c)
    out, _ = run(c, r, o)
    torch.cuda.synchronize()
    dy, yp = o["dy"].double(), torch.nan_to_num(o["y_perm"].double())
    cv = o["const_vecs"].double()

    def loss(x, w):
        return float((sparse_terms(c, r, x, w, cv, yp) * dy[r["tok"]]).sum())
    x, w, h = o["x"].double(), r["w"].double(), 1e-5
    g = torch.Generator().manual_seed(1)
    vx, vw = torch.randn(x.shape, generator=g).double(), torch.randn(w.shape, generator=g).double()
    # The x part without the dispatched rows and the added gradients.
    row = r["row_of"].long()
    rest = (o["add0"].double() + o["add1"].double()).index_add(
        0, r["tok"], (row >= 0)[:, None] * torch.nan_to_num(o["dx_perm"].double())[row.clamp(min=0)])
    dx = out["dx"].double().cpu() - rest
    num = (loss(x + h * vx, w) - loss(x - h * vx, w)) / (2 * h)
    got = float((dx * vx).sum())
    # fp32 steps of each element, and the differences' h^2 and 1 / h terms.
    assert abs(num - got) <= 1e-4 * float((dx.abs() * vx.abs()).sum()) + 1e-6
    num = (loss(x, w + h * vw) - loss(x, w - h * vw)) / (2 * h)
    dw = out["dw"].double().cpu()
    assert abs(num - float((dw * vw).sum())) <= 1e-4 * float((dw.abs() * vw.abs()).sum()) + 1e-6


def test_dx_in_place_and_no_adds():
    """dx may be one of the added gradients; without any, dx is the rows alone."""
    m = _moe()
    c = CASES["top2"]
    r, o, dt = operands(c)
    out, _ = run(c, r, o)
    cfg = m.make_config(c)
    G = {k: to_gpu(v) for k, v in {**r, **o}.items() if isinstance(v, torch.Tensor)}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (G["sel"], G["w"], G["row_of"], None, None, None, None)
    buf = G["add0"].clone()
    m.dispatch_backward(cfg, G["dx_perm"], None, *args, buf, st, add=(buf, G["add1"]))
    assert torch.equal(buf, out["dx"])
    bare = torch.empty_like(buf)
    m.dispatch_backward(cfg, G["dx_perm"], None, *args, bare, st)
    ref = G["dx_perm"].float()[G["row_of"].long()].view(c["T"], c["k"], -1).sum(1).to(dt)
    assert torch.equal(bare, ref)


@pytest.mark.parametrize("name", ["top2", "ec", "mix"])
def test_bad_ids_are_flagged_and_add_nothing(name):
    m = _moe()
    c = CASES[name]
    r, o, _ = operands(c)
    ec = c["routing"] == "expert_choice"
    bad = torch.arange(0, r["w"].numel(), 7)
    r["sel"][bad] = torch.where(bad % 2 == 0, 1 << 20, -5).to(torch.int32)
    r["row_of"][bad] = -1
    out, _ = run(c, r, o)
    torch.cuda.synchronize()
    assert int(out["status"].item()) & (m.DEV_BAD_TOKEN if ec else m.DEV_BAD_EXPERT)
    assert (out["dw"].cpu()[bad] == 0).all()
    assert torch.isfinite(out["dx"]).all() and torch.isfinite(out["dw"]).all()


def test_another_stream_and_a_captured_graph():
    """A non-default stream, and a graph captured once and replayed on new inputs in place,
    give the bytes of the eager call."""
    c = CASES["ec_light_mix"]
    r, o, _ = operands(c)
    out, go = run(c, r, o)
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in out.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for v in out.values():
        v.zero_()
    torch.cuda.synchronize()
    go(s)
    torch.cuda.synchronize()
    used = int(r["offsets"][-1])
    for k in ("dw", "dx", "dconst"):
        assert torch.equal(out[k], first[k]), k
    assert torch.equal(out["dy_perm"][:used], first["dy_perm"][:used])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for v in out.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in ("dw", "dx", "dconst"):
        assert torch.equal(out[k], first[k]), k
