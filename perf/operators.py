"""The operators that train the MoE layer and wrap it into a block, as timed cases.

Five operators, each with the forms a user of the layer calls:

  combine_bwd   gradient of the combine: expert-output rows, routing weights
                and constant experts
  dispatch_bwd  gradient of the dispatch: expert-input rows back to tokens,
                with the gradients that meet there added
  router_bwd    routing-weight gradient through selection and softmax to the
                logits, the router weights and x
  mlp_bwd       gradient of the grouped expert MLP (and the shared expert)
  norm, norm_bwd  the norms after and before a block fused with its gate,
                residual scale and modulation, and their gradient

With ``own`` false ``run`` computes the plain form: elementary torch
operations in fp32, rounded once at the end. With ``own`` true it makes the
library's calls. ``exact`` computes the same values in fp64 by automatic
differentiation of the forward definition.
"""

import math

import torch

own = False

DEV = "cuda"
HEAVY, IDENTITY, ZERO, CONST = 0, 1, 2, 3
# Expert kinds of a case, by name: "heavy" alone, or the zero-computation
# experts of the MMOE layer (identity, zero, constant) after the heavy ones.
LIGHT = {"heavy": [], "light": [IDENTITY, ZERO, CONST]}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # A training step of a DiT-MoE-XL layer: 32 images x 256 latent tokens, top-2 of 8.
        dict(name="combine_bwd_ditmoe", op="combine_bwd", dtype="bf16", routing="topk", T=8192, d=1152, E=8, k=2,
             group=0, C=0, kinds="heavy", const_mix=0, bias=0.0),
        # An MMOE layer whose lightweight experts take many tokens, mixed constant expert, odd token count.
        dict(name="combine_bwd_mmoe_odd", op="combine_bwd", dtype="bf16", routing="topk", T=4099, d=1152, E=19, k=2,
             group=0, C=0, kinds="light", const_mix=1, bias=0.791),
        # An EC-DiT layer: expert choice, 64 sequences of 128 tokens, tokens with no or many experts.
        dict(name="dispatch_bwd_ecdit", op="dispatch_bwd", dtype="bf16", routing="ec", T=8192, d=2048, E=32, k=0,
             group=128, C=8, kinds="heavy", const_mix=0, bias=0.0, adds=2),
        # A 32-token diffusion-LLM block, top-8 of 64: the smallest call, launch latency.
        dict(name="dispatch_bwd_block32", op="dispatch_bwd", dtype="bf16", routing="topk", T=32, d=2048, E=64, k=8,
             group=0, C=0, kinds="heavy", const_mix=0, bias=0.0, adds=1),
        # The router of an MMOE layer with its gate residual, top-2 of 19.
        dict(name="router_bwd_mmoe", op="router_bwd", dtype="bf16", routing="topk", T=8192, d=1152, E=19, k=2,
             group=0, C=0, kinds="light", const_mix=0, bias=0.0, renorm=0, aux=0, zscale=0.5),
        # A small fp32 layer with renormalised weights and a load-balance gradient on the probabilities.
        dict(name="router_bwd_f32", op="router_bwd", dtype="f32", routing="topk", T=256, d=64, E=8, k=2,
             group=0, C=0, kinds="heavy", const_mix=0, bias=0.0, renorm=1, aux=1, zscale=0.0),
        # The DiT-MoE-XL experts: 8 routed (top-2) and two shared, the heaviest step.
        dict(name="mlp_bwd_ditmoe", op="mlp_bwd", dtype="bf16", act="gelu", T=8192, d=1152, E=8, k=2, h=4608,
             shared=9216),
        # A 32-token block over 64 SwiGLU experts: a few rows each, bound by the weights.
        dict(name="mlp_bwd_block32", op="mlp_bwd", dtype="bf16", act="swiglu", T=32, d=2048, E=64, k=8, h=1024,
             shared=0),
        # Between two DiT blocks: gate and residual of one, LayerNorm and modulation of the next.
        dict(name="norm_between_blocks", op="norm", dtype="bf16", T=8192, d=1152, group=256, pre="layer", post="none",
             affine=0, cond=1, res_scale=1.0),
        # One token of an fp32 stream, RMS norms on both sides of the block.
        dict(name="norm_one_token", op="norm", dtype="f32", T=1, d=2048, group=0, pre="rms", post="rms",
             affine=1, cond=0, res_scale=0.5),
        # The gradient of the step between two DiT blocks.
        dict(name="norm_bwd_between_blocks", op="norm_bwd", dtype="bf16", T=8192, d=1152, group=256, pre="layer",
             post="none", affine=0, cond=1, res_scale=1.0),
        # Norms on both sides with learned weights, a ragged last group, a width off the 64-wide tiles.
        dict(name="norm_bwd_ragged", op="norm_bwd", dtype="bf16", T=3001, d=1160, group=77, pre="layer", post="rms",
             affine=1, cond=1, res_scale=0.75),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["combine_bwd", "dispatch_bwd", "router_bwd", "mlp_bwd", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = 8 * _log(rng, 8, 256)
    if op in ("norm", "norm_bwd"):
        T = _log(rng, 1, 8192 if dtype == "bf16" else 4096)
        return dict(op=op, dtype=dtype, T=T, d=d, group=rng.choice([0, 1, _log(rng, 1, 300), 256]),
                    pre=rng.choice(["layer", "rms"]), post=rng.choice(["none", "layer", "rms"]),
                    affine=rng.randint(0, 1), cond=rng.randint(0, 1), res_scale=rng.choice([1.0, 0.75]))
    if op == "mlp_bwd":
        f32 = dtype == "f32"
        c = dict(op=op, dtype=dtype, act=rng.choice(["gelu", "swiglu"]), T=_log(rng, 1, 300 if f32 else 8192),
                 d=8 * _log(rng, 8, 40 if f32 else 144), E=_log(rng, 1, 32), k=rng.randint(1, 4),
                 h=8 * _log(rng, 8, 60 if f32 else 576), shared=0)
        c["k"] = min(c["k"], c["E"])
        if rng.random() < 0.4:
            c["shared"] = c["h"]
        while work(c)["flops"] > (4e10 if f32 else 1.0e12):
            c["T"] = max(1, c["T"] * 2 // 3)
        return c
    c = dict(op=op, dtype=dtype, routing=rng.choice(["topk", "topk", "ec"]), T=_log(rng, 1, 8192), d=d,
             E=_log(rng, 2, 64), k=0, group=0, C=0, kinds=rng.choice(["heavy", "light"]), const_mix=0, bias=0.0)
    if c["kinds"] == "light":
        c["E"] = max(c["E"], 4)
        c["const_mix"] = rng.randint(0, 1)
        c["bias"] = rng.choice([0.0, 0.791])
    if c["routing"] == "ec":
        c["group"] = min(128, max(8, c["T"] // 4))
        c["T"] = max(1, c["T"] // c["group"]) * c["group"]
        c["C"] = max(1, min(c["group"], 2 * c["group"] // c["E"]))
    else:
        c["k"] = rng.randint(1, min(8, c["E"]))
    while _na(c) * c["d"] * (2 if dtype == "bf16" else 4) > 16384 * 1152 * 2:
        c["d"] = max(8, c["d"] * 2 // 24 * 8)
    if op == "dispatch_bwd":
        c["adds"] = rng.randint(0, 3)
    if op == "router_bwd":
        c.update(renorm=rng.randint(0, 1) if c["routing"] == "topk" else 0, aux=rng.randint(0, 1),
                 zscale=rng.choice([0.0, 0.5]))
    return c


def _na(c):
    return c["T"] // c["group"] * c["E"] * c["C"] if c["routing"] == "ec" else c["T"] * c["k"]


def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _kinds(c):
    light = LIGHT[c["kinds"]]
    return [HEAVY] * (c["E"] - len(light)) + light


# ----------------------------------------------------------------- inputs
def _rand(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * std


def _route(c, g, s):
    """The routing of one layer call, as the router, selection and dispatch hand it over."""
    T, d, E = c["T"], c["d"], c["E"]
    dt = _dt(c)
    kinds = torch.tensor(_kinds(c), device=DEV)
    s["x"] = _rand(g, T, d).to(dt)
    s["W_r"] = _rand(g, E, d, std=1.0 / math.sqrt(d)).to(dt)
    z = s["x"].float() @ s["W_r"].float().t() + c["bias"] * (kinds != HEAVY)
    s["probs"] = torch.softmax(z, -1)
    if c["routing"] == "ec":
        S, C, G = c["group"], c["C"], T // c["group"]
        tok = torch.topk(s["probs"].view(G, S, E).transpose(1, 2), C, dim=-1).indices.sort(-1).values  # [G, E, C]
        sel = (tok + (torch.arange(G, device=DEV) * S).view(G, 1, 1)).reshape(-1)
        eid = torch.arange(E, device=DEV).view(1, E, 1).expand(G, E, C).reshape(-1)
        s["tok"], s["eid"] = sel, eid
        s["w"] = s["probs"][sel, eid]
        order = torch.argsort(sel, stable=True)
        s["tok_assign"] = order.to(torch.int32)
        s["tok_ptr"] = torch.searchsorted(sel[order].contiguous(), torch.arange(T + 1, device=DEV)).to(torch.int32)
        s["sel"] = sel.to(torch.int32)
    else:
        sel = torch.topk(z, c["k"], dim=-1).indices
        w = s["probs"].gather(1, sel)
        if c.get("renorm"):
            w = w / w.sum(-1, keepdim=True)
        s["tok"] = torch.arange(T, device=DEV).repeat_interleave(c["k"])
        s["eid"], s["w"] = sel.reshape(-1), w.reshape(-1).contiguous()
        s["sel"], s["tok_ptr"], s["tok_assign"] = sel.to(torch.int32).contiguous(), None, None
    heavy = kinds[s["eid"]] == HEAVY
    n_heavy = int((kinds == HEAVY).sum())
    key = torch.where(heavy, s["eid"], torch.full_like(s["eid"], E))
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=DEV)
    s["row_of"] = torch.where(heavy, row, torch.full_like(row, -1)).to(torch.int32)
    counts = torch.bincount(key, minlength=E + 1)[:n_heavy]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["kinds"] = kinds
    s["const_vecs"] = None
    if CONST in _kinds(c):
        s["const_vecs"] = _rand(g, 1, 3, d, std=0.02).to(dt) if c["const_mix"] else _rand(g, 1, d, std=0.02).to(dt)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c}
    dt = _dt(c)
    T, d = c["T"], c["d"]
    if c["op"] in ("combine_bwd", "dispatch_bwd", "router_bwd"):
        _route(c, g, s)
        na = _na(c)
        if c["op"] == "combine_bwd":
            s["dy"] = _rand(g, T, d).to(dt)
            s["y_perm"] = _rand(g, na, d, std=0.5).to(dt)
            s["dy_perm"] = torch.zeros(na, d, device=DEV, dtype=dt)  # rows of no expert stay as they are
        elif c["op"] == "dispatch_bwd":
            s["dy"] = _rand(g, T, d).to(dt)
            s["dx_perm"] = _rand(g, na, d, std=0.5).to(dt)
            s["adds"] = [_rand(g, T, d).to(dt) for _ in range(c["adds"])]
        else:
            s["dw"] = _rand(g, na)
            s["dprobs"] = _rand(g, T, c["E"], std=0.1) if c["aux"] else None
    elif c["op"] == "mlp_bwd":
        E, h, k = c["E"], c["h"], c["k"]
        # Top-k of skewed random scores: the uneven expert loads of a trained router.
        score = _rand(g, T, E) + _rand(g, E, std=0.5)
        eid = torch.topk(score, k, dim=-1).indices.reshape(-1)
        counts = torch.bincount(eid, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
        up = 2 * h if c["act"] == "swiglu" else h
        s["x_perm"] = _rand(g, T * k, d).to(dt)
        s["dy_perm"] = _rand(g, T * k, d, std=0.3).to(dt)
        s["W1"] = _rand(g, E, up, d, std=0.02).to(dt)
        s["W2"] = _rand(g, E, d, h, std=0.02).to(dt)
        if c["shared"]:
            s["x"] = _rand(g, T, d).to(dt)
            s["dy"] = _rand(g, T, d).to(dt)
            s["Ws1"] = _rand(g, c["shared"], d, std=0.02).to(dt)
            s["Ws2"] = _rand(g, d, c["shared"], std=0.02).to(dt)
    else:
        B = -(-T // c["group"]) if c["group"] else 1
        # A residual stream: a few channels far larger than the rest, a mean off zero.
        chan = 1.0 + 8.0 * (torch.rand(d, generator=g, device=DEV) < 0.01)
        s["h"] = _rand(g, T, d, std=0.5).to(dt)
        s["x"] = (_rand(g, T, d) * chan + 0.2).to(dt)
        for n in ("gate", "scale", "shift"):
            s[n] = None
        if c["cond"]:  # one projection of the conditioning, cut into its parts
            cond = _rand(g, B, 3 * d, std=0.3).to(dt)
            s["gate"], s["scale"], s["shift"] = cond[:, :d], cond[:, d:2 * d], cond[:, 2 * d:]
        affine = c["affine"]
        s["pre_gamma"] = (1 + _rand(g, d, std=0.1)).to(dt) if affine else None
        s["pre_beta"] = _rand(g, d, std=0.1).to(dt) if affine and c["pre"] == "layer" else None
        s["post_gamma"] = (1 + _rand(g, d, std=0.1)).to(dt) if affine and c["post"] != "none" else None
        if c["op"] == "norm_bwd":
            s["y"] = (_rand(g, T, d) * chan + 0.2).to(dt)
            s["dy"] = _rand(g, T, d).to(dt)
            s["dz"] = _rand(g, T, d).to(dt)
    if own:  # the configuration, workspace and output buffers that a program keeps; nothing of the inputs
        s["kept"] = _kept(c, s)
    return s


# ------------------------------------------------------------ plain forms
def _const_parts(xf, cvf, mix):
    """The constant expert on every token: its output, and a0, a1 when mixed."""
    if not mix:
        return cvf[0].expand_as(xf), None, None
    a = torch.softmax(xf @ cvf[0, 1:].t(), -1)
    return a[:, :1] * xf + a[:, 1:] * cvf[0, 0], a[:, :1], a[:, 1:]


def _plain_combine_bwd(s):
    c, dt = s["case"], _dt(s["case"])
    na, d = _na(c), c["d"]
    dyf, w = s["dy"].float(), s["w"]
    g = dyf[s["tok"]]
    kind = s["kinds"][s["eid"]]
    row = s["row_of"].long()
    heavy = row >= 0
    dot = (g * s["y_perm"].float()[row.clamp(min=0)]).sum(-1)
    dw = torch.where(heavy, dot, torch.zeros_like(dot))
    out = torch.zeros(na + 1, d, device=DEV, dtype=dt)
    out[torch.where(heavy, row, torch.full_like(row, na))] = (w[:, None] * g).to(dt)
    res = {"dy_perm": out[:na], "dw": dw}
    if c["kinds"] == "light":
        xf, cvf = s["x"].float(), s["const_vecs"].float()
        cx, a0, a1 = _const_parts(xf, cvf, c["const_mix"])
        dw = torch.where(kind == IDENTITY, (dyf * xf).sum(-1)[s["tok"]], dw)
        res["dw"] = torch.where(kind == CONST, (dyf * cx).sum(-1)[s["tok"]], dw)
        wc = torch.zeros(c["T"], device=DEV).index_add(0, s["tok"], torch.where(kind == CONST, w, torch.zeros_like(w)))
        gc = wc[:, None] * dyf
        if not c["const_mix"]:
            res["dconst"] = gc.sum(0, keepdim=True)
        else:
            dl = a0 * a1 * ((gc * xf).sum(-1, keepdim=True) - (gc * cvf[0, 0]).sum(-1, keepdim=True))
            dwc = (dl * xf).sum(0)
            res["dconst"] = torch.stack([(a1 * gc).sum(0), dwc, -dwc])[None]
    return res


def _plain_dispatch_bwd(s):
    c, dt = s["case"], _dt(s["case"])
    T, d = c["T"], c["d"]
    row = s["row_of"].long()
    v = torch.where((row >= 0)[:, None], s["dx_perm"].float()[row.clamp(min=0)], torch.zeros((), device=DEV))
    if c["kinds"] == "light":
        dyf = s["dy"].float()
        kind = s["kinds"][s["eid"]]
        g = s["w"][:, None] * dyf[s["tok"]]
        v = torch.where((kind == IDENTITY)[:, None], g, v)
        if c["const_mix"]:
            xf, cvf = s["x"].float(), s["const_vecs"].float()
            _, a0, a1 = _const_parts(xf, cvf, 1)
            a0, a1 = a0[s["tok"]], a1[s["tok"]]
            dl = a0 * a1 * ((g * xf[s["tok"]]).sum(-1, keepdim=True) - (g * cvf[0, 0]).sum(-1, keepdim=True))
            v = torch.where((kind == CONST)[:, None], a0 * g + dl * (cvf[0, 1] - cvf[0, 2]), v)
    if c["routing"] == "ec":
        dx = torch.zeros(T, d, device=DEV).index_add(0, s["tok"], v)
    else:
        dx = v.view(T, c["k"], d).sum(1)
    return {"dx": sum((a.float() for a in s["adds"]), dx).to(dt)}


def _plain_router_bwd(s):
    c, dt = s["case"], _dt(s["case"])
    A, dw = s["probs"], s["dw"]
    dA = torch.zeros_like(A) if s["dprobs"] is None else s["dprobs"]
    if c["renorm"]:
        w, k = s["w"].view(-1, c["k"]), c["k"]
        sums = A.gather(1, s["eid"].view(-1, k)).sum(-1, keepdim=True)
        dw = ((dw.view(-1, k) - (dw.view(-1, k) * w).sum(-1, keepdim=True)) / sums).reshape(-1)
    dA = dA.index_put((s["tok"], s["eid"]), dw, accumulate=True)
    dz = A * (dA - (A * dA).sum(-1, keepdim=True))
    res = {"dlogits": dz, "dbias": dz.sum(0), "dW_r": dz.t() @ s["x"].float(), "dx": (dz @ s["W_r"].float()).to(dt)}
    if c["zscale"]:
        res["dz_prev"] = c["zscale"] * dz
    return res


def _plain_mlp(x, dy, W1, W2, gated):
    """Batched over experts, fp32: [E, M, d] rows (zero past an expert's last) and the weights."""
    u = x @ W1.transpose(1, 2)
    dh = dy @ W2
    if gated:
        h = u.shape[-1] // 2
        a, b = u[..., :h], u[..., h:]
        sg = 1 / (1 + torch.exp(-a))
        act = a * sg * b
        du = torch.cat([dh * b * (sg * (1 + a * (1 - sg))), dh * a * sg], -1)
    else:
        phi = 0.5 * (1 + torch.erf(u * math.sqrt(0.5)))
        act = u * phi
        du = dh * (phi + u * torch.exp(-0.5 * u * u) * (1 / math.sqrt(2 * math.pi)))
    return du @ W1, du.transpose(1, 2) @ x, dy.transpose(1, 2) @ act


def _padded(s, dtype):
    """The ragged row groups as [E, most, d], rows past a group's end zero, and where they go back."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["most"], device=DEV)
    ok = at < off[1:, None]
    n = s["x_perm"].shape[0]
    rows = at.clamp(max=n - 1)
    zero = torch.zeros((), device=DEV, dtype=dtype)
    x = torch.where(ok[..., None], s["x_perm"].to(dtype)[rows], zero)
    dy = torch.where(ok[..., None], s["dy_perm"].to(dtype)[rows], zero)
    return x, dy, torch.where(ok, at, torch.full_like(at, n)).reshape(-1)


def _plain_mlp_bwd(s):
    c, dt = s["case"], _dt(s["case"])
    x, dy, back = _padded(s, torch.float32)
    dx, dW1, dW2 = _plain_mlp(x, dy, s["W1"].float(), s["W2"].float(), c["act"] == "swiglu")
    n, d = s["x_perm"].shape
    out = torch.zeros(n + 1, d, device=DEV, dtype=dt)
    out[back] = dx.reshape(-1, d).to(dt)
    res = {"dx_perm": out[:n], "dW1": dW1.to(dt), "dW2": dW2.to(dt)}
    if c["shared"]:
        dx, dW1, dW2 = _plain_mlp(s["x"].float()[None], s["dy"].float()[None], s["Ws1"].float()[None],
                                  s["Ws2"].float()[None], False)
        res.update(dx_shared=dx[0].to(dt), dWs1=dW1[0].to(dt), dWs2=dW2[0].to(dt))
    return res


NORM_EPS = 1e-6


def _plain_norm(v, kind):
    """The normalised rows and 1 / their scale."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + NORM_EPS)
    return v * r, r


def _plain_norm_bwd(g, hat, r, kind):
    """Gradient of the normalised rows `hat` = norm(v) back to v."""
    t = g - hat * (g * hat).mean(-1, keepdim=True)
    if kind == "layer":
        t = t - g.mean(-1, keepdim=True)
    return r * t


def _rows(c, t):
    """A condition's rows, one per token."""
    if t is None:
        return None
    t = t.float()
    return t.repeat_interleave(c["group"], 0)[: c["T"]] if c["group"] else t


def _f(t):
    return None if t is None else t.float()


def _per_group(c, t):
    """Sum over the tokens that share a condition row: [B, d]."""
    if not c["group"]:
        return t.sum(0, keepdim=True)
    B = -(-c["T"] // c["group"])
    pad = torch.zeros(B * c["group"] - c["T"], c["d"], device=DEV)
    return torch.cat([t, pad]).view(B, c["group"], c["d"]).sum(1)


def _plain_block_norm(s):
    c, dt = s["case"], _dt(s["case"])
    u = s["h"].float()
    if c["post"] != "none":
        u = _plain_norm(u, c["post"])[0]
        if s["post_gamma"] is not None:
            u = u * s["post_gamma"].float()
    if s["gate"] is not None:
        u = u * _rows(c, s["gate"])
    y = c["res_scale"] * s["x"].float() + u
    z = _plain_norm(y, c["pre"])[0]
    if s["pre_gamma"] is not None:
        z = z * s["pre_gamma"].float()
    if s["pre_beta"] is not None:
        z = z + s["pre_beta"].float()
    if s["scale"] is not None:
        z = z * (1 + _rows(c, s["scale"])) + _rows(c, s["shift"])
    return {"y": y.to(dt), "z": z.to(dt)}


def _plain_block_norm_bwd(s):
    c, dt = s["case"], _dt(s["case"])
    res = {}
    hat, r = _plain_norm(s["y"].float(), c["pre"])
    dz = s["dz"].float()
    gam, bet = _f(s["pre_gamma"]), _f(s["pre_beta"])
    if s["scale"] is not None:
        n = hat if gam is None else hat * gam
        n = n if bet is None else n + bet
        res["dscale"], res["dshift"] = _per_group(c, dz * n), _per_group(c, dz)
        dz = dz * (1 + _rows(c, s["scale"]))
    if gam is not None:
        res["dpre_gamma"] = (dz * hat).sum(0)
        dz_in = dz * gam
    else:
        dz_in = dz
    if bet is not None:
        res["dpre_beta"] = dz.sum(0)
    dt_y = s["dy"].float() + _plain_norm_bwd(dz_in, hat, r, c["pre"])
    res["dx"] = (c["res_scale"] * dt_y).to(dt)
    du, hf = dt_y, s["h"].float()
    uh, ur = _plain_norm(hf, c["post"]) if c["post"] != "none" else (hf, None)
    u = uh if s["post_gamma"] is None else uh * s["post_gamma"].float()
    if s["gate"] is not None:
        res["dgate"] = _per_group(c, du * u)
        du = du * _rows(c, s["gate"])
    if s["post_gamma"] is not None:
        res["dpost_gamma"] = (du * uh).sum(0)
        du = du * s["post_gamma"].float()
    if c["post"] != "none":
        du = _plain_norm_bwd(du, uh, ur, c["post"])
    res["dh"] = du.to(dt)
    return res


_PLAIN = dict(combine_bwd=_plain_combine_bwd, dispatch_bwd=_plain_dispatch_bwd, router_bwd=_plain_router_bwd,
              mlp_bwd=_plain_mlp_bwd, norm=_plain_block_norm, norm_bwd=_plain_block_norm_bwd)


# ------------------------------------------------------ the library's calls
def _own_config(c):
    from mixture_experts_layer_33_b200 import moe
    if c["op"] in ("norm", "norm_bwd"):
        return moe.make_norm_config(dict(T=c["T"], d=c["d"], dtype=c["dtype"], group_size=c["group"], pre=c["pre"],
                                         post=c["post"], eps=NORM_EPS, res_scale=c["res_scale"]))
    if c["op"] == "mlp_bwd":
        return moe.make_config(dict(T=c["T"], d=c["d"], h=c["h"], E=c["E"], k=c["k"], dtype=c["dtype"], act=c["act"],
                                    routing="token_topk", n_shared=1 if c["shared"] else 0, h_shared=c["shared"]))
    return moe.make_config(dict(T=c["T"], d=c["d"], h=64, E=c["E"], k=c["k"], dtype=c["dtype"], act="gelu",
                                routing="expert_choice" if c["routing"] == "ec" else "token_topk",
                                group_size=c["group"], capacity=c["C"], kinds=_kinds(c), const_mix=c["const_mix"],
                                renorm=c.get("renorm", 0), gate_residual_scale=c.get("zscale", 0.0)))


def _kept(c, s):
    """What a program sets up once for a shape: configuration, workspace, gradient buffers."""
    from mixture_experts_layer_33_b200 import moe
    cfg = _own_config(c)
    T, d, dt = c["T"], c["d"], _dt(c)
    k = {"moe": moe, "c": cfg, "status": torch.zeros(1, dtype=torch.int32, device=DEV)}

    def f32(*shape):
        return torch.empty(*shape, device=DEV, dtype=torch.float32)

    if c["op"] in ("norm", "norm_bwd"):
        k["ws"] = moe.alloc_block_norm_workspace(cfg) if c["op"] == "norm_bwd" else None
        names = ("y", "z") if c["op"] == "norm" else ("dx", "dh")
        k["out"] = {n: torch.empty(T, d, device=DEV, dtype=dt) for n in names}
        if c["op"] == "norm_bwd":
            B = -(-T // c["group"]) if c["group"] else 1
            if c["cond"]:
                cond = f32(B, 3 * d)
                k["out"].update(dgate=cond[:, :d], dscale=cond[:, d:2 * d], dshift=cond[:, 2 * d:])
            for n in ("pre_gamma", "pre_beta", "post_gamma"):
                if s[n] is not None:
                    k["out"]["d" + n] = f32(d)
        return k
    k["ws"] = moe.alloc_backward_workspace(cfg)
    if c["op"] == "combine_bwd":
        k["out"] = {"dy_perm": s["dy_perm"], "dw": f32(_na(c))}
        if s["const_vecs"] is not None:
            k["out"]["dconst"] = f32(*s["const_vecs"].shape)
    elif c["op"] == "dispatch_bwd":
        k["out"] = {"dx": torch.empty(T, d, device=DEV, dtype=dt)}
    elif c["op"] == "router_bwd":
        k["out"] = {"dlogits": f32(T, c["E"]), "dbias": f32(c["E"]), "dW_r": f32(c["E"], d),
                    "dx": torch.empty(T, d, device=DEV, dtype=dt)}
        if c["zscale"]:
            k["out"]["dz_prev"] = f32(T, c["E"])
    else:
        k["out"] = {"dx_perm": torch.empty_like(s["x_perm"]), "dW1": torch.empty_like(s["W1"]),
                    "dW2": torch.empty_like(s["W2"])}
        if c["shared"]:
            k["out"].update(dx_shared=torch.empty_like(s["x"]), dWs1=torch.empty_like(s["Ws1"]),
                            dWs2=torch.empty_like(s["Ws2"]))
    return k


def _own(s):
    k = s["kept"]
    moe, cfg, ws, out, op = k["moe"], k["c"], k["ws"], k["out"], s["case"]["op"]
    if op == "combine_bwd":
        moe.combine_backward(cfg, s["dy"], s["y_perm"], s["sel"], s["w"], s["row_of"], s["tok_ptr"], s["tok_assign"],
                             s["x"], s["const_vecs"], out["dy_perm"], out["dw"], k["status"], ws,
                             dconst=out.get("dconst"))
    elif op == "dispatch_bwd":
        moe.dispatch_backward(cfg, s["dx_perm"], s["dy"], s["sel"], s["w"], s["row_of"], s["tok_ptr"],
                              s["tok_assign"], s["x"], s["const_vecs"], out["dx"], k["status"], add=s["adds"])
    elif op == "router_bwd":
        moe.router_backward(cfg, s["x"], s["W_r"], s["probs"], s["sel"], s["w"], s["dw"], s["tok_ptr"],
                            s["tok_assign"], out["dlogits"], k["status"], ws, dprobs=s["dprobs"],
                            dz_prev=out.get("dz_prev"), dbias=out["dbias"], dW_r=out["dW_r"], dx=out["dx"])
    elif op == "mlp_bwd":
        moe.grouped_mlp_backward(cfg, s["x_perm"], s["offsets"], s["W1"], s["W2"], s["dy_perm"], s.get("x"),
                                 s.get("Ws1"), s.get("Ws2"), s.get("dy"), k["status"], ws, dx_perm=out["dx_perm"],
                                 dW1=out["dW1"], dW2=out["dW2"], dx_shared=out.get("dx_shared"),
                                 dWs1=out.get("dWs1"), dWs2=out.get("dWs2"))
    elif op == "norm":
        moe.block_norm(cfg, s["h"], s["x"], y=out["y"], z=out["z"], post_gamma=s["post_gamma"], gate=s["gate"],
                       pre_gamma=s["pre_gamma"], pre_beta=s["pre_beta"], scale=s["scale"], shift=s["shift"])
    else:
        moe.block_norm_backward(cfg, s["h"], s["y"], s["dz"], s["dy"], ws, post_gamma=s["post_gamma"],
                                gate=s["gate"], pre_gamma=s["pre_gamma"], pre_beta=s["pre_beta"], scale=s["scale"],
                                **out)
    return out


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    eb = 2 if c["dtype"] == "bf16" else 4
    T, d = c["T"], c["d"]
    act = T * d * eb
    if c["op"] == "norm":
        return {"bytes": 4 * act + (3 * d * (-(-T // c["group"]) if c["group"] else 1) * eb if c["cond"] else 0),
                "flops": 14 * T * d}
    if c["op"] == "norm_bwd":
        B = -(-T // c["group"]) if c["group"] else 1
        return {"bytes": 6 * act + (B * d * (2 * eb + 12) if c["cond"] else 0), "flops": 30 * T * d}
    if c["op"] == "mlp_bwd":
        up = 2 * c["h"] if c["act"] == "swiglu" else c["h"]
        rows = T * c["k"]
        used = min(c["E"], rows)  # experts whose weights are read, at most
        nb = 3 * rows * d * eb + (used + c["E"]) * (up + c["h"]) * d * eb
        # Up projection again, gradient through both layers, both weight gradients.
        fl = 2 * rows * d * (3 * up + 2 * c["h"])
        if c["shared"]:
            nb += 3 * act + 4 * c["shared"] * d * eb
            fl += 2 * T * d * 5 * c["shared"]
        return {"bytes": nb, "flops": fl}
    na = _na(c)
    if c["op"] == "combine_bwd":
        light = 3 / c["E"] if c["kinds"] == "light" else 0
        rows = na * (1 - light)
        return {"bytes": act + 2 * rows * d * eb + (act if light else 0) + na * 16, "flops": 3 * na * d}
    if c["op"] == "dispatch_bwd":
        light = 3 / c["E"] if c["kinds"] == "light" else 0
        return {"bytes": (1 + c["adds"]) * act + na * (1 - light) * d * eb + (act if light else 0) + na * 8,
                "flops": (na + c["adds"] * T) * d}
    tables = (2 + bool(c["aux"]) + bool(c["zscale"])) * T * c["E"] * 4
    return {"bytes": 2 * act + c["E"] * d * (eb + 4) + tables + na * 12, "flops": 4 * T * c["E"] * d}


# ---------------------------------------------- fp64, by differentiation
def _leaf(t):
    return t.double().requires_grad_()


def _exact_sparse(s):
    """combine (and the x terms of the dispatch) from the layer's definition, as a sum over assignments."""
    c = s["case"]
    T, d = c["T"], c["d"]
    tok, kind, row = s["tok"], s["kinds"][s["eid"]], s["row_of"].long()
    x, w = _leaf(s["x"]), _leaf(s["w"])
    cv = _leaf(s["const_vecs"]) if s["const_vecs"] is not None else None
    terms = torch.zeros(tok.numel(), d, device=DEV, dtype=torch.float64)
    if cv is not None:
        if c["const_mix"]:
            e = torch.exp(x @ cv[0, 1:].t())
            con = (e[:, :1] * x + e[:, 1:] * cv[0, 0]) / e.sum(-1, keepdim=True)
        else:
            con = cv[0].expand(T, d)
        terms = terms + (kind == CONST)[:, None] * con[tok] + (kind == IDENTITY)[:, None] * x[tok]
    return tok, row, x, w, cv, terms


def _exact(s):
    c, op = s["case"], s["case"]["op"]
    T, d = c["T"], c["d"]
    f64 = dict(device=DEV, dtype=torch.float64)
    if op == "combine_bwd":
        tok, row, x, w, cv, terms = _exact_sparse(s)
        yp = _leaf(s["y_perm"])
        terms = terms + (row >= 0)[:, None] * yp[row.clamp(min=0)]
        y = torch.zeros(T, d, **f64).index_add(0, tok, w[:, None] * terms)
        wanted = [yp, w] + ([cv] if cv is not None else [])
        got = torch.autograd.grad(y, wanted, s["dy"].double(), allow_unused=True, materialize_grads=True)
        return dict(zip(("dy_perm", "dw", "dconst"), got))
    if op == "dispatch_bwd":
        tok, row, x, w, cv, terms = _exact_sparse(s)
        rows = torch.zeros(row.numel() + 1, d, **f64).index_put((torch.where(row < 0, row.numel(), row),), x[tok])
        loss = (rows[:-1] * s["dx_perm"].double())[: int(s["offsets"][-1])].sum()
        y = torch.zeros(T, d, **f64).index_add(0, tok, w[:, None] * terms)
        loss = loss + (y * s["dy"].double()).sum() + sum((x * a.double()).sum() for a in s["adds"])
        return {"dx": torch.autograd.grad(loss, x)[0]}
    if op == "router_bwd":
        # The logits enter through log A: any z with softmax(z) = A has the same gradient.
        z = torch.log(s["probs"].double().clamp(min=1e-300)).requires_grad_()
        A = torch.softmax(z, -1)
        w = A[s["tok"], s["eid"]]
        if c["renorm"]:
            w = (w.view(T, -1) / w.view(T, -1).sum(-1, keepdim=True)).reshape(-1)
        loss = (w * s["dw"].double()).sum()
        if s["dprobs"] is not None:
            loss = loss + (A * s["dprobs"].double()).sum()
        dz = torch.autograd.grad(loss, z)[0]
        res = {"dlogits": dz, "dbias": dz.sum(0), "dW_r": torch.einsum("te,td->ed", dz, s["x"].double()),
               "dx": torch.einsum("te,ed->td", dz, s["W_r"].double())}
        if c["zscale"]:
            res["dz_prev"] = dz * c["zscale"]
        return res
    if op == "mlp_bwd":
        def mlp(x, dy, W1, W2, gated):
            x, W1, W2 = (t.requires_grad_() for t in (x, W1, W2))
            u = torch.einsum("emd,ehd->emh", x, W1)
            if gated:
                a, b = u.chunk(2, -1)
                hid = torch.nn.functional.silu(a) * b
            else:
                hid = torch.nn.functional.gelu(u)
            return torch.autograd.grad(torch.einsum("emh,edh->emd", hid, W2), (x, W1, W2), dy)
        x, dy, back = _padded(s, torch.float64)
        n = s["x_perm"].shape[0]
        dx, dW1, dW2 = mlp(x, dy, s["W1"].double(), s["W2"].double(), c["act"] == "swiglu")
        out = torch.zeros(n + 1, d, **f64)
        out[back] = dx.reshape(-1, d)
        res = {"dx_perm": out[:n], "dW1": dW1, "dW2": dW2}
        if c["shared"]:
            dx, dW1, dW2 = mlp(*(s[n].double()[None] for n in ("x", "dy", "Ws1", "Ws2")), False)
            res.update(dx_shared=dx[0], dWs1=dW1[0], dWs2=dW2[0])
        return res
    # norm, norm_bwd
    group = torch.arange(T, device=DEV) // c["group"] if c["group"] else torch.zeros(T, device=DEV, dtype=torch.long)
    p = {n: _leaf(s[n]) for n in ("post_gamma", "gate", "pre_gamma", "pre_beta", "scale", "shift") if s[n] is not None}

    def norm(v, kind):
        if kind == "layer":
            return (v - v.mean(-1, keepdim=True)) / torch.sqrt(v.var(-1, keepdim=True, unbiased=False) + NORM_EPS)
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + NORM_EPS)

    def after(h, x):
        u = norm(h, c["post"]) if c["post"] != "none" else h
        u = u * p["post_gamma"] if "post_gamma" in p else u
        u = u * p["gate"][group] if "gate" in p else u
        return c["res_scale"] * x + u

    def before(y):
        z = norm(y, c["pre"])
        z = z * p["pre_gamma"] if "pre_gamma" in p else z
        z = z + p["pre_beta"] if "pre_beta" in p else z
        return z * (1 + p["scale"][group]) + p["shift"][group] if "scale" in p else z

    if op == "norm":
        with torch.no_grad():
            y = after(s["h"].double(), s["x"].double())
            return {"y": y, "z": before(y)}
    # The gradient at the y that the call is given: dz's way to y first, then the sum's way to h and x.
    y, h, x = _leaf(s["y"]), _leaf(s["h"]), _leaf(s["x"])
    names = [n for n in ("pre_gamma", "pre_beta", "scale", "shift") if n in p]
    got = torch.autograd.grad(before(y), [y] + [p[n] for n in names], s["dz"].double())
    res = {"d" + n: v for n, v in zip(names, got[1:])}
    names = [n for n in ("post_gamma", "gate") if n in p]
    back = torch.autograd.grad(after(h, x), [h, x] + [p[n] for n in names], s["dy"].double() + got[0])
    res.update(dh=back[0], dx=back[1], **{"d" + n: v for n, v in zip(names, back[2:])})
    return res


def exact(case, seed):
    return _exact(prepare(case, seed))
