"""MoELayer's ``stream`` argument, on the host: everything a step allocates is
allocated while ``stream`` is the current stream, so that a block freed when
the step returns can only go to later work of the same stream; what the
caller holds (inputs, results, workspaces) is marked as used by both streams.
The entry points and streams are stand-ins: no GPU is needed."""

import contextlib

import pytest
import torch

ENTRIES = ("router", "select_expert_choice", "core_set_vote", "core_set_union", "dispatch", "grouped_mlp", "combine",
           "forward", "combine_backward", "dispatch_backward", "router_backward", "grouped_mlp_backward")


@pytest.fixture(scope="module")
def m():
    from mixture_experts_layer_33_b200 import build
    build.build()
    from mixture_experts_layer_33_b200 import moe
    return moe


class Stream:
    def __init__(self, name):
        self.name = name


class World:
    """Which stream is current, where each tensor was allocated, and who else it is marked for."""

    def __init__(self, m, monkeypatch):
        self.caller = self.current = Stream("caller")
        self.home, self.marks, self.launches, self.keep = {}, {}, [], []
        for fn in ("empty", "empty_like", "zeros"):
            monkeypatch.setattr(torch, fn, self.noting(getattr(torch, fn)))
        monkeypatch.setattr(torch.cuda, "Stream", Stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current)
        monkeypatch.setattr(torch.cuda, "stream", self.on)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.marks.setdefault(id(t), set()).add(s))
        monkeypatch.setattr(m, "_tensors", lambda *trees: list(flatten(trees)), raising=False)
        for name in ENTRIES:
            monkeypatch.setattr(m, name, lambda *a, stream=None, _n=name, **k: self.launches.append(
                (_n, stream or self.current)))

    def noting(self, fn):
        def made(*a, **k):
            t = fn(*a, **k)
            self.home[id(t)] = self.current
            self.keep.append(t)  # ids stay unique
            return t
        return made

    @contextlib.contextmanager
    def on(self, s):
        before, self.current = self.current, s
        yield
        self.current = before


def flatten(o):
    if isinstance(o, torch.Tensor):
        yield o
    elif isinstance(o, (tuple, list)):
        for v in o:
            yield from flatten(v)
    elif isinstance(o, dict):
        yield from flatten(list(o.values()))


@pytest.mark.parametrize("name", ["mmoe_constmix", "ecdit", "des_vote", "des_seq", "tiny_fp32"])
def test_step_allocates_on_its_stream(m, monkeypatch, name):
    from mixture_experts_layer_33_b200 import inputs as gen
    small = {"ecdit": dict(T=256)}.get(name, dict(T=16))
    cfg = gen.workload(name, d=64, h=64, **small)
    if cfg.get("n_shared"):
        cfg["h_shared"] = 64
    inp = gen.make_inputs(cfg, "cpu")
    world = World(m, monkeypatch)
    layer = m.MoELayer(cfg, {k: inp[k] for k in ("W_r", "W1", "W2", "Ws1", "Ws2", "logit_bias", "const_vecs")},
                       device="cpu")
    x, side = inp["x"], Stream("side")

    def check(step, out, inputs):
        """Since `step` began: all on the side stream; results marked for the caller, inputs for the side."""
        assert world.launches[step[0]:] and all(s is side for _, s in world.launches[step[0]:])
        fresh = world.keep[step[1]:]
        assert fresh
        assert [world.home[id(t)].name for t in fresh] == ["side"] * len(fresh)
        for t in flatten(out):
            assert id(t) not in world.home or world.caller in world.marks.get(id(t), ()), "a result"
        for t in flatten(inputs):
            assert side in world.marks.get(id(t), ()), "an input"

    def now():
        return len(world.launches), len(world.keep)
    at = now()
    y = layer(x, z_prev=inp["z_prev"], stream=side)
    check(at, y, (x, inp["z_prev"], layer.ws, layer.status))
    at = now()
    y, saved = layer.forward_train(x, z_prev=inp["z_prev"], stream=side)
    check(at, (y, saved), (x, inp["z_prev"], layer.ws, layer.status))
    at = now()
    dy, dprobs = torch.ones_like(x), torch.ones(cfg["T"], cfg["E"])
    grads = layer.backward(saved, dy, dprobs=dprobs, stream=side)
    check(at, (grads, layer.bws), (saved, dy, dprobs, layer.status))
    # The workspace stays: a second backward on another stream marks it for that one too.
    other = Stream("other")
    layer.backward(saved, dy, stream=other)
    assert other in world.marks[id(layer.bws)]
    # Without a stream nothing is switched and nothing marked.
    marks = {k: set(v) for k, v in world.marks.items()}
    at = now()
    layer.backward(layer.forward_train(x, z_prev=inp["z_prev"])[1], dy)
    assert all(s is world.caller for _, s in world.launches[at[0]:])
    assert all(world.home[id(t)] is world.caller for t in world.keep[at[1]:])
    assert marks == world.marks
