"""fp64 references of the layer's gradients, on the CPU, with the magnitudes
that the fp32 error bounds of the GPU tests are derived from.

``within`` checks |got - ref| <= half_step(dtype) |ref| + c 2^-24 mag: one
rounding to the output type (``finfo(t).eps / 2`` relative), and an fp32
evaluation whose rounding errors are at most c half-steps (2^-24) of ``mag``,
the sum of the magnitudes of the terms that are added up."""

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24
HEAVY, IDENTITY, ZERO, CONST = 0, 1, 2, 3


def within(what, got, ref, mag, c, extra=0.0):
    """``extra``: a further absolute bound (a tensor or number)."""
    g = got.detach().double().cpu()
    assert torch.isfinite(ref).all() and torch.isfinite(g).all(), f"{what}: not finite"
    bound = HALF[got.dtype] * ref.abs() + c * F32 * mag + extra + 1e-37
    over = (g - ref).abs() - bound * (1 + HALF[got.dtype])
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, (f"{what}: {float((g - ref).abs().max()):.3e} off at most, "
                        f"{worst:.3e} over the bound")


def route(cfg, gen, empty=0.0):
    """A routing of the config as the layer's steps hand it over (CPU tensors): sel, w, row_of,
    offsets, tok_ptr, tok_assign and per assignment its token, expert and kind."""
    T, E = cfg["T"], cfg["E"]
    kinds = torch.tensor(cfg.get("kinds", [HEAVY] * E))
    probs = torch.softmax(torch.randn(T, E, generator=gen) * 1.5, -1)
    r = {"probs": probs, "kinds": kinds, "tok_ptr": None, "tok_assign": None}
    if cfg["routing"] == "expert_choice":
        S, C = cfg["group_size"], cfg["capacity"]
        G = T // S
        tok = torch.topk(probs.view(G, S, E).transpose(1, 2), C, dim=-1).indices.sort(-1).values
        sel = (tok + (torch.arange(G) * S).view(G, 1, 1)).reshape(-1)
        eid = torch.arange(E).view(1, E, 1).expand(G, E, C).reshape(-1)
        r["tok"], w = sel, probs[sel, eid]
        order = torch.argsort(sel, stable=True)
        r["tok_assign"] = order.to(torch.int32)
        r["tok_ptr"] = torch.searchsorted(sel[order].contiguous(), torch.arange(T + 1)).to(torch.int32)
    else:
        k = cfg["k"]
        sel = torch.topk(probs, k, dim=-1).indices
        w = probs.gather(1, sel)
        if cfg.get("renorm"):
            w = w / w.sum(-1, keepdim=True)
        sel, w, eid = sel.reshape(-1), w.reshape(-1), sel.reshape(-1).clone()
        gone = torch.rand(T * k, generator=gen) < empty
        eid[gone] = -1
        sel = eid
        r["tok"] = torch.arange(T).repeat_interleave(k)
    r["sel"], r["w"], r["eid"] = sel.to(torch.int32), w.float().contiguous(), eid
    kind = torch.where(eid < 0, torch.full_like(eid, ZERO), kinds[eid.clamp(min=0)])
    heavy = kind == HEAVY
    r["kind"], n_heavy = kind, int((kinds == HEAVY).sum())
    key = torch.where(heavy, eid, torch.full_like(eid, E))
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel())
    r["row_of"] = torch.where(heavy, row, torch.full_like(row, -1)).to(torch.int32)
    counts = torch.bincount(key, minlength=E + 1)[:n_heavy]
    r["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return r


def sparse_terms(cfg, r, x, w, cv, yp):
    """The combine's terms per assignment, w_a E_a(x_s), differentiable, fp64."""
    d = x.shape[1]
    n = w.numel()
    kinds = cfg.get("kinds", [HEAVY] * cfg["E"])
    e_out = torch.zeros(n, d, dtype=torch.float64)
    row = r["row_of"].long()
    if yp is not None:
        e_out = e_out + (row >= 0)[:, None] * torch.where((row >= 0)[:, None], yp[row.clamp(min=0)], 0.0)
    e_out = e_out + (r["kind"] == IDENTITY)[:, None] * x[r["tok"]]
    consts = [e for e, k in enumerate(kinds) if k == CONST]
    for i, e in enumerate(consts):
        if cfg.get("const_mix"):
            a = torch.softmax(x @ cv[i, 1:].t(), -1)
            out = a[:, :1] * x + a[:, 1:] * cv[i, 0]
        else:
            out = cv[i].expand_as(x)
        e_out = e_out + (r["eid"] == e)[:, None] * out[r["tok"]]
    return w[:, None] * e_out


def leaf(t):
    return t.double().requires_grad_()
