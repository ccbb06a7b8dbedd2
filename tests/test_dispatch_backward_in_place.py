"""moe_dispatch_backward in place: dx may be one of the added gradients, dy
among them, but not with mixed constant experts, whose dot products take whole
rows of dy and x while other warps store parts of dx. The refusal is a host
check (no GPU needed); the allowed forms give the bytes of the call out of place."""

import ctypes

import pytest
import torch

BAD = 1
FAKE = 1 << 30  # never dereferenced


@pytest.fixture(scope="module")
def m():
    from mixture_experts_layer_33_b200 import build
    build.build()
    from mixture_experts_layer_33_b200 import moe
    return moe


@pytest.mark.parametrize("name", ["mmoe_constmix", "f32"])
def test_dx_over_dy_or_x_is_refused_with_mixed_constant_experts(m, name):
    from mixture_experts_layer_33_b200 import inputs as gen
    wl = gen.workload("mmoe_constmix", T=70, d=520)
    if name == "f32":
        wl["dtype"] = "f32"
    c = m.make_config(wl)
    size = 70 * 520 * (4 if name == "f32" else 2)
    far = {k: FAKE + i * (size + 4096) for i, k in enumerate(
        ("dx_perm", "dy", "sel", "w", "row_of", "tok_ptr", "tok_assign", "x", "const_vecs", "add0", "add1", "add2"))}
    for what in ("dy", "x"):
        for shift in (0, 16, -16, size - 16, 16 - size):
            args = dict(far, add0=far["dy"], dx=far[what] + shift, status=None)
            assert m.LIB.moe_dispatch_backward(ctypes.byref(c), *args.values(), None) == BAD, (what, shift)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_forms_give_the_same_bytes(m, dtype):
    from test_gpu_exchange_backward import case, operands, run, to_gpu
    for mix in (0, 1):
        c = case(700, 1160, 9, k=4, dtype=dtype, light=True, mix=mix, n_const=2)
        r, o, _ = operands(c)
        out, _ = run(c, r, o)  # add = (add0, add1)
        G = {k: to_gpu(v) for k, v in {**r, **o}.items() if isinstance(v, torch.Tensor) or v is None}
        cfg, st = m.make_config(c), torch.zeros(1, dtype=torch.int32, device="cuda")
        routing = (G["sel"], G["w"], G["row_of"], None, None, G["x"], G["const_vecs"])
        for k in ("add0", "add1"):
            buf = dict(add0=G["add0"], add1=G["add1"])
            dx = buf[k] = buf[k].clone()
            m.dispatch_backward(cfg, G["dx_perm"], G["dy"], *routing, dx, st, add=(buf["add0"], buf["add1"]))
            assert torch.equal(dx, out["dx"]), (mix, k)
        want = torch.empty_like(G["dy"])
        m.dispatch_backward(cfg, G["dx_perm"], G["dy"], *routing, want, st, add=(G["dy"], G["add0"]))
        dy = G["dy"].clone()
        if mix:
            for dx, d, x in ((dy, dy, G["x"]), (G["x"], dy, G["x"])):
                with pytest.raises(RuntimeError):
                    m.dispatch_backward(cfg, G["dx_perm"], d, *routing[:5], x, G["const_vecs"], dx, st, add=(d,))
            assert torch.equal(dy, G["dy"])
        else:
            m.dispatch_backward(cfg, G["dx_perm"], dy, *routing, dy, st, add=(dy, G["add0"]))
            assert torch.equal(dy, want)
        assert int(st.item()) == 0
