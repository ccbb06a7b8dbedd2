"""Calls of one kernel with different sizes from two host threads at once, each
with its own stream, buffers and workspace: every call is taken and gives the
bytes of a call made alone. The sizes differ in the shared memory that the
kernel is launched with."""

import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

CALLS = 3000


def _moe():
    from mixture_experts_layer_33_b200 import moe
    return moe


def norm_step(d, dtype):
    m = _moe()
    n = m.make_norm_config(dict(T=320, d=d, dtype=dtype, group_size=0, pre="layer", post="rms"))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(d)
    h, x, dy, dz = (torch.randn(320, d, generator=g, device="cuda").to(dt) for _ in range(4))
    y, z, dh, dx = (torch.empty_like(x) for _ in range(4))
    ws = m.alloc_block_norm_workspace(n)

    def forward(stream=None):
        m.block_norm(n, h, x, y=y, z=z, stream=stream)

    def both(stream=None):
        forward(stream)
        m.block_norm_backward(n, h, y, dz, dy, ws, dh=dh, dx=dx, stream=stream)
    return both, (y, z, dh, dx)


def router_step(E, dtype):
    m = _moe()
    T, d = 70, 64
    c = m.make_config(dict(T=T, d=d, h=16, E=E, k=1, dtype=dtype, act="gelu", routing="token_topk"))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(E)
    x, W = torch.randn(T, d, generator=g, device="cuda").to(dt), torch.randn(E, d, generator=g, device="cuda").to(dt)
    probs = torch.softmax(torch.randn(T, E, generator=g, device="cuda"), -1)
    w, sel = probs.max(-1)
    w, sel, dw = w.contiguous(), sel.to(torch.int32), torch.randn(T, generator=g, device="cuda")
    dl, dW, dx = torch.empty_like(probs), torch.empty(E, d, device="cuda"), torch.empty_like(x)
    st, ws = torch.zeros(1, dtype=torch.int32, device="cuda"), m.alloc_backward_workspace(c)

    def step(stream=None):
        m.router_backward(c, x, W, probs, sel, w, dw, None, None, dl, st, ws, dW_r=dW, dx=dx, stream=stream)
    return step, (dl, dW, dx)


def choice_step(S, C):
    """Expert choice and its dispatch's token lists."""
    m = _moe()
    E, T, d = 4, 2 * S, 64
    c = m.make_config(dict(T=T, d=d, h=16, E=E, k=0, dtype="f32", act="gelu", routing="expert_choice", group_size=S,
                           capacity=C))
    g = torch.Generator(device="cuda").manual_seed(S)
    probs = torch.softmax(torch.randn(T, E, generator=g, device="cuda"), -1)
    x = torch.randn(T, d, generator=g, device="cuda")
    n = m.num_assignments(c)
    sel, perm, row_of, tok_assign = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(4))
    w, offsets = torch.empty(n, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    tok_ptr, x_perm = torch.empty(T + 1, dtype=torch.int32, device="cuda"), torch.empty(n, d, device="cuda")
    st, ws = torch.zeros(1, dtype=torch.int32, device="cuda"), m.alloc_workspace(c)

    def step(stream=None):
        m.select_expert_choice(probs, S, C, sel, w, stream=stream)
        m.dispatch(c, sel, x, x_perm, offsets, perm, row_of, tok_ptr, tok_assign, st, ws, stream=stream)
    return step, (sel, w, offsets, row_of, tok_ptr, tok_assign, x_perm)


PAIRS = {
    "norm_bf16": lambda: (norm_step(64, "bf16"), norm_step(1280, "bf16")),
    "norm_bf16_wide": lambda: (norm_step(2056, "bf16"), norm_step(4096, "bf16")),
    "norm_f32": lambda: (norm_step(64, "f32"), norm_step(1280, "f32")),
    "router_f32": lambda: (router_step(33, "f32"), router_step(128, "f32")),
    "router_bf16": lambda: (router_step(2, "bf16"), router_step(40, "bf16")),
    "expert_choice": lambda: (choice_step(32, 4), choice_step(8192, 16)),
}


class Recorder:
    """In the library's place: notes the calls with their arguments instead of making them."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        fn = getattr(self.lib, name)
        if name == "moe_num_assignments" or name.endswith("_size"):
            return fn
        return lambda *a: self.calls.append((fn, a)) or 0


@pytest.mark.parametrize("name", list(PAIRS))
def test_two_host_threads(name, monkeypatch):
    m = _moe()
    pair = PAIRS[name]()
    want = []
    for step, outs in pair:
        step()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pair]
    # The C calls themselves, so that little but them runs in the threads.
    calls = []
    for (step, _), stream in zip(pair, streams):
        with monkeypatch.context() as noting:
            noting.setattr(m, "LIB", Recorder(m.LIB))
            step(stream)
            calls.append(m.LIB.calls)
    start, errors = threading.Barrier(len(pair)), []

    def work(i):
        try:
            torch.cuda.set_device(0)
            start.wait()
            for k in range(CALLS):
                for fn, args in calls[i]:
                    code = fn(*args)
                    if code:
                        raise RuntimeError(m.status_string(code))
                if k % 100 == 99:
                    streams[i].synchronize()
        except Exception as exc:  # noqa: BLE001
            errors.append((i, k, exc))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(pair))]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)  # the threads take turns between any two steps
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert not errors, errors
    for (_, outs), ref in zip(pair, want):
        for o, r in zip(outs, ref):
            assert torch.equal(o, r)
