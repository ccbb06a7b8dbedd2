"""Gradient of the block norms on rows whose mean is hundreds of standard
deviations from zero, within bounds that grow with the mean once, as the
kernels' errors do (a product of two such magnitudes lets zeros pass). A CPU
test shows that outputs of zero, a mean left in, and a variance taken as a
difference of moments in fp32 are out of bounds.

Errors, u = 2^-24: a row sum is a chain of at most 40 additions, so a mean is
within 41 u of mean |v|, and a normalised row n within E = 130 u r (|v| + mean
|v|) (mean, mean square, root, product). For dN = r (g - mean g - n mean(g n))
with g off by e:
  err = r (e + mean e + 45 u mean |g| + E |mean(g n)|
           + |n| (45 u mean |g n| + mean(|g| E) + mean(e |n|)))
        + |dN| (60 u + mean(|n| E)) + 8 u r (|g| + |mean g| + |n mean(g n)|),
the second line for the scale r and each operation's own rounding. Sums over
N tokens take N + 60 additions at most (segments, slices, lists)."""

import pytest
import torch

from grad_helpers import F32, HALF, within
from test_gpu_block_norm import EPS, case, grads64, operands, rows, run_bwd

CASES = {
    "narrow": case(60, 1024, 16, "layer", "layer", "f32", shift=300.0),
    "wide": case(40, 4104, 16, "layer", "layer", "f32", shift=300.0),
    "ragged": case(900, 1160, 77, "layer", "rms", "f32", shift=100.0, alpha=0.75),
    "no_post": case(300, 264, 0, "layer", "none", "f32", shift=1000.0),
    "bf16": case(130, 520, 50, "layer", "rms", "bf16", shift=100.0),
}
U = F32


def mean(t):
    return t.mean(-1, keepdim=True)


def norm_error(v, kind):
    """r, n and the error of n."""
    m = v - mean(v) if kind == "layer" else v
    r = 1 / torch.sqrt(mean(m * m) + EPS)
    return r, m * r, 130 * U * r * (v.abs() + mean(v.abs()))


def grad_error(g, e, v, kind):
    """The error of dN(g; v) when g is off by e."""
    r, n, E = norm_error(v, kind)
    mg = mean(g) if kind == "layer" else 0 * mean(g)
    gn = mean(g * n)
    dN = r * (g - mg - n * gn)
    return (r * (e + mean(e) + 45 * U * mean(g.abs()) + E * gn.abs()
                 + n.abs() * (45 * U * mean((g * n).abs()) + mean(g.abs() * E) + mean(e * n.abs())))
            + dN.abs() * (60 * U + mean(n.abs() * E)) + 8 * U * r * (g.abs() + mg.abs() + (n * gn).abs()))


def errors(c, o):
    """Every output's error bound apart from its last rounding."""
    f = {k: v.double() if isinstance(v, torch.Tensor) else None for k, v in o.items()}
    one = torch.ones((), dtype=torch.float64)

    def of(k, default):
        return f[k] if f[k] is not None else default * one
    ga, be, pg = of("pre_gamma", 1), of("pre_beta", 0), of("post_gamma", 1)
    sc = 1 + rows(c, f["scale"]) if f["scale"] is not None else one
    gt = rows(c, f["gate"]) if f["gate"] is not None else one
    T, d = c["T"], c["d"]
    B = -(-T // c["group_size"]) if c["group_size"] else 1
    idx = torch.arange(T) // c["group_size"] if c["group_size"] else torch.zeros(T, dtype=torch.long)

    def group(t):
        return torch.zeros(B, d, dtype=torch.float64).index_add(0, idx, t.expand(T, -1))
    many, each = (T + 60) * U, (min(T, c["group_size"] or T) + 60) * U
    y, dz = f["y"], f["dz"]
    r, n, E = norm_error(y, c["pre"])
    g = dz * sc * ga
    t = f["dy"] + r * (g - (mean(g) if c["pre"] == "layer" else 0) - n * mean(g * n))
    e_t = grad_error(g, 3 * U * g.abs(), y, c["pre"]) + U * t.abs()
    e = {"dx": abs(c["res_scale"]) * (e_t + U * t.abs()),
         "dshift": each * group(dz.abs()),
         "dscale": group(dz.abs() * E * ga.abs()) + (each + 3 * U) * group(dz.abs() * (n.abs() * ga.abs() + be.abs())),
         "dpre_gamma": ((dz * sc).abs() * E).sum(0) + (many + 3 * U) * (dz * sc * n).abs().sum(0),
         "dpre_beta": (many + 3 * U) * (dz * sc).abs().sum(0)}
    u, e_u = f["h"], 0 * f["h"]
    if c["post"] != "none":
        _, u, e_u = norm_error(f["h"], c["post"])
    tg = t * gt * pg
    e_tg = (gt * pg).abs() * e_t + 3 * U * tg.abs()
    e["dh"] = grad_error(tg, e_tg, f["h"], c["post"]) if c["post"] != "none" else e_tg
    e_tu = e_t * u.abs() + t.abs() * e_u
    e["dgate"] = group(e_tu * pg.abs()) + (each + 3 * U) * group((t * u * pg).abs())
    e["dpost_gamma"] = (e_tu * gt.abs()).sum(0) + (many + 3 * U) * (t * u * gt).abs().sum(0)
    return e


def types(c, dt):
    return {k: dt if k in ("dx", "dh") else torch.float32
            for k in ("dx", "dh", "dgate", "dscale", "dshift", "dpre_gamma", "dpre_beta", "dpost_gamma")}


@pytest.mark.parametrize("name", list(CASES))
def test_bounds_tell_mistakes(name):
    c = CASES[name]
    o, dt, _ = operands(c)
    ref, _ = grads64(c, o)
    err, kinds = errors(c, o), types(c, dt)

    def share(k, got):
        g = got.to(kinds[k]).double()
        return float(((g - ref[k]).abs() > HALF[kinds[k]] * ref[k].abs() + err[k] + 1e-37).double().mean())
    for k, v in ref.items():
        within(k, v.to(kinds[k]), v, 0, 0, extra=err[k])
        assert share(k, 0 * v) > 0.8, k
    # y taken with a hundredth of its mean left in; and its variance as a difference of fp32 moments.
    y, dz = o["y"].double(), o["dz"].double()
    sc = 1 + rows(c, o["scale"].double())
    g = dz * sc * o["pre_gamma"].double()

    def dx_of(yc, var):
        r = 1 / torch.sqrt(var + EPS)
        n = yc * r
        return c["res_scale"] * (o["dy"].double() + r * (g - mean(g) - n * mean(g * n)))
    yc = y - mean(y)
    fine = torch.arange(c["T"]) != 2  # not the row of zeros
    torch.testing.assert_close(dx_of(yc, mean(yc * yc))[fine], ref["dx"][fine], rtol=1e-9, atol=1e-9)
    bad = ref["dx"].clone()
    bad[fine] = dx_of(yc + 0.01 * mean(y), mean(yc * yc))[fine]
    assert share("dx", bad) > (0.8 if dt == torch.float32 else 0.2)
    if dt == torch.float32:
        y32 = o["y"].float()
        moments = ((y32 * y32).mean(-1, keepdim=True) - y32.mean(-1, keepdim=True) ** 2).double().clamp(min=0)
        bad[fine] = dx_of(yc, moments)[fine]
        assert share("dx", bad) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_gradients(name):
    c = CASES[name]
    o, dt, B = operands(c)
    out, _ = run_bwd(c, o, dt, B)
    ref, _ = grads64(c, o)
    err = errors(c, o)
    assert set(out) == set(ref)
    for k in out:
        within(k, out[k], ref[k], 0, 0, extra=err[k])
