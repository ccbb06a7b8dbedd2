"""dW_r of the bf16 router gradient over many tokens, where every product of a
sum has one sign: no rounding of a long chain may lean one way.

The kernel multiplies 64-token tiles on the tensor cores (dz as three bf16
terms, 4 steps of 16 tokens each: 12 accumulations, which may each lose 2
half-steps of the partial sum more than an fp32 addition, 4 in all), adds the
tiles' sums in fp32, then the token ranges'. 4096 columns are 32 blocks of
128, for which 9 token ranges run at once: 114 tiles of 65536 tokens a range.
So the sum over the tokens is within 12 * 4 + 114 + 9 + 16 + 1 (dz's split) =
188 half-steps of the sum of magnitudes, here the result itself: 1.12e-5. A
chain of 12 * 114 accumulations that cut off instead of rounding is about
8e-5 off."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [2, 19, 64, 100])
def test_sums_of_one_sign(E):
    from mixture_experts_layer_33_b200 import moe as m
    T, d = 65536, 4096
    g = torch.Generator(device="cuda").manual_seed(E)
    c = m.make_config(dict(T=T, d=d, h=16, E=E, k=1, dtype="bf16", act="gelu", routing="token_topk"))
    x = (torch.rand(T, d, generator=g, device="cuda") + 0.5).bfloat16()
    # One expert takes every token with a positive gradient: its dz is positive, the others' negative.
    probs = torch.softmax(torch.randn(T, E, generator=g, device="cuda"), -1)
    sel = torch.zeros(T, dtype=torch.int32, device="cuda")
    w, dw = probs[:, 0].contiguous(), torch.rand(T, generator=g, device="cuda") + 0.5
    dl, dW = torch.empty(T, E, device="cuda"), torch.empty(E, d, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = m.alloc_backward_workspace(c)
    m.router_backward(c, x, torch.ones(E, d, device="cuda").bfloat16(), probs, sel, w, dw, None, None, dl, status, ws,
                      dW_r=dW)
    assert (dl[:, 0] > 0).all() and (dl[:, 1:] <= 0).all() and int(status.item()) == 0
    ref = sum(dl[b:b + 8192].double().t() @ x[b:b + 8192].double() for b in range(0, T, 8192))
    worst = float(((dW.double() - ref).abs() / ref.abs()).max())
    assert worst <= 188 * 2.0 ** -24, worst
