"""MoELayer's steps with ``stream=``: queued behind a long kernel on that
stream, they return at once, and the caller's stream then allocates and fills
every block it can get. Values are those of the same step on the current
stream, bit for bit: the step's temporaries were not handed out while its
kernels were still to run. Then the other way round: results that the caller
drops while its own stream still reads them are not handed to the next step."""

import pytest
import torch

from mixture_experts_layer_33_b200 import inputs as gen

pytestmark = pytest.mark.gpu

CASES = {
    "mmoe": ("mmoe_constmix", dict(T=200, d=128, h=128, h_shared=64)),
    "expert_choice": ("ecdit", dict(T=512, d=256, h=256)),
    "des_vote": ("des_vote", dict(T=48, d=256, h=128)),
    "des_seq": ("des_seq", dict(T=40, d=256, h=128)),
    "f32": ("tiny_fp32", dict(T=150, x_std=1.0)),
}
PAUSE = 100_000_000  # cycles: about 50 ms


def setup(name):
    from mixture_experts_layer_33_b200 import moe as m
    wl, over = CASES[name]
    cfg = gen.workload(wl, **over)
    inp = gen.make_inputs(cfg, "cuda")
    layer = m.MoELayer(cfg, {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")})
    dy = torch.randn(inp["x"].shape, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    return layer, inp["x"], inp["z_prev"], dy.to(inp["x"].dtype)


def poison(like):
    """Fills blocks of the sizes of `like` (several of each) from the current stream's pool."""
    return [torch.empty_like(t).view(torch.uint8).fill_(255) for t in like for _ in range(4) if t.numel()]


@pytest.mark.parametrize("name", list(CASES))
def test_step_on_a_busy_stream(name):
    layer, x, z_prev, dy = setup(name)
    want = layer(x, z_prev=z_prev)
    y0, s0 = layer.forward_train(x, z_prev=z_prev)
    g0 = layer.backward(s0, dy)
    torch.cuda.synchronize()
    sizes = [t for t in list(s0.values()) + list(g0.values()) + [y0] if isinstance(t, torch.Tensor)]
    side = torch.cuda.Stream()
    busy = 0  # runs that were still queued when the blocks were filled; the first loads kernels, which may wait
    for _ in range(4):
        with torch.cuda.stream(side):
            torch.cuda._sleep(PAUSE)
        y = layer(x, z_prev=z_prev, stream=side)
        filled = poison(sizes)
        yt, s = layer.forward_train(x, z_prev=z_prev, stream=side)
        filled += poison(sizes)
        g = layer.backward(s, dy, stream=side)
        s = {k: v for k, v in s.items() if k in ("logits", "sel")}  # the rest is dropped while it is still read
        filled += poison(sizes)
        busy += not side.query()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(yt, y0)
        assert torch.equal(s["logits"], s0["logits"]) and torch.equal(s["sel"], s0["sel"])
        for n in g0:
            assert torch.equal(g[n], g0[n]), n
        assert all(bool((f == 255).all()) for f in filled)
    assert int(layer.status.item()) == 0
    assert busy, "every step was over before the blocks were filled: nothing was tested"


def test_results_dropped_while_the_caller_reads_them():
    layer, x, _, dy = setup("f32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y0, s0 = layer.forward_train(x)
    g0 = layer.backward(s0, dy)
    torch.cuda.synchronize()
    x2 = torch.randn_like(x)
    torch.cuda.synchronize()
    busy = 0
    for _ in range(4):
        y, s = layer.forward_train(x, stream=side)
        g = layer.backward(s, dy, stream=side)
        torch.cuda.synchronize()
        torch.cuda._sleep(PAUSE)
        kept = {k: v.clone() for k, v in g.items()}  # copies queued behind the pause
        ky = y.clone()
        del y, s, g
        layer.backward(layer.forward_train(x2, stream=side)[1], dy, stream=side)
        busy += not torch.cuda.current_stream().query()
        torch.cuda.synchronize()
        assert torch.equal(ky, y0)
        for k in g0:
            assert torch.equal(kept[k], g0[k]), k
    assert busy


@pytest.mark.parametrize("name", ["mmoe", "expert_choice"])
def test_step_on_a_stream_forked_in_a_capture(name):
    """Captured with stream= a stream forked from the capture's, replayed on new inputs in place."""
    layer, x, z_prev, dy = setup(name)
    x2 = torch.randn_like(x.float()).to(x.dtype)
    x_in = x.clone()

    def step(stream=None):
        y, s = layer.forward_train(x_in, z_prev=z_prev, stream=stream)
        return {"y": y, **layer.backward(s, dy, stream=stream)}
    want = []
    for v in (x, x2):
        x_in.copy_(v)
        want.append({k: t.clone() for k, t in step().items()})
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        held = step(side)
        torch.cuda.current_stream().wait_stream(side)
    for k in range(4):
        x_in.copy_((x, x2)[k % 2])
        graph.replay()
        torch.cuda.synchronize()
        for n, t in held.items():
            assert torch.equal(t, want[k % 2][n]), (k, n)
    assert int(layer.status.item()) == 0
