"""The gradients count rows and tiles in 32 bits: configs with more than 2^30
tokens, assignments or rows of weights are refused, on the host, before any
pointer is used. No GPU."""

import ctypes

import pytest

UNSUPPORTED = 2
FAKE = 1 << 20


@pytest.fixture(scope="module")
def m():
    from mixture_experts_layer_33_b200 import build
    build.build()
    from mixture_experts_layer_33_b200 import moe
    return moe


def config(m, **kw):
    return m.make_config(dict(dict(T=64, d=8, h=8, E=4, k=1, dtype="bf16", act="gelu", routing="token_topk"), **kw))


LIMIT = 1 << 30
OVER = [dict(T=LIMIT + 1), dict(T=2**31 - 1), dict(T=LIMIT // 2 + 1, k=2), dict(h=LIMIT // 4 + 8),
        dict(h=LIMIT // 8 + 8, act="swiglu"), dict(n_shared=2, h_shared=LIMIT // 2 + 8),
        dict(T=LIMIT // 4 + 16, routing="expert_choice", group_size=16, capacity=16)]
AT = [dict(T=LIMIT), dict(T=LIMIT // 2, k=2), dict(h=LIMIT // 4), dict(h=LIMIT // 8, act="swiglu"),
      dict(n_shared=2, h_shared=LIMIT // 2), dict(T=LIMIT // 4, routing="expert_choice", group_size=16, capacity=16)]


@pytest.mark.parametrize("kw", OVER, ids=str)
def test_beyond_the_limit(m, kw):
    c = config(m, **kw)
    n = ctypes.c_size_t()
    assert m.LIB.moe_backward_workspace_size(ctypes.byref(c), ctypes.byref(n)) == UNSUPPORTED
    calls = dict(moe_combine_backward=11, moe_router_backward=15, moe_router_backward_logits=16,
                 moe_grouped_mlp_backward=16)
    for name, pointers in calls.items():
        code = getattr(m.LIB, name)(ctypes.byref(c), *[FAKE] * pointers, FAKE, 0, None)
        assert code == UNSUPPORTED, name
    assert m.LIB.moe_dispatch_backward(ctypes.byref(c), *[FAKE] * 13, FAKE, None) == UNSUPPORTED


@pytest.mark.parametrize("kw", AT, ids=str)
def test_at_the_limit(m, kw):
    assert m.backward_workspace_size(config(m, **kw)) > 0


WS = 1 << 50  # more than any workspace: the pointers are not used either
LARGE_F32 = {
    "rows": dict(T=65532 * 64, k=1),
    "rows_of_k": dict(T=65532 * 32, k=2),
    # Few routed rows and too many of the shared expert: refused before the routed part is launched.
    "shared_rows": dict(T=65536 * 64, routing="expert_choice", group_size=16384, capacity=1, n_shared=1, h_shared=8),
    "shared_width": dict(T=65536, routing="expert_choice", group_size=16384, capacity=1, n_shared=1,
                         h_shared=65536 * 64),
    "width": dict(h=65536 * 64),
}


@pytest.mark.parametrize("name", list(LARGE_F32))
def test_fp32_mlp_tiles(m, name):
    c = config(m, dtype="f32", **LARGE_F32[name])
    assert m.backward_workspace_size(c) < WS
    code = m.LIB.moe_grouped_mlp_backward(ctypes.byref(c), *[FAKE] * 16, FAKE, WS, None)
    assert code == UNSUPPORTED
