"""ctypes binding of libmoe.so (the C ABI in include/moe.h).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels. PyTorch supplies device memory and the current stream.
Importing this module loads the library and raises ImportError if it has
not been built (``python -m mixture_experts_layer_33_b200.build``); calls
raise RuntimeError with the library's status string when a call fails.
With MOE_DEBUG=1 in the environment it loads the MOE_DEBUG build
(``libmoe_debug.so``, ``build --debug``) instead: the same entry points,
whose kernels also range-check the indices callers hand in.
"""

from __future__ import annotations

import ctypes
import os

import torch

DEBUG_BUILD = os.environ.get("MOE_DEBUG", "0") == "1"
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                         "libmoe_debug.so" if DEBUG_BUILD else "libmoe.so")

MOE_OK = 0
F32, BF16 = 0, 1
TOKEN_TOPK, EXPERT_CHOICE, DES_VOTE, DES_SEQ = 0, 1, 2, 3
GELU_ERF, SWIGLU = 0, 1
HEAVY, IDENTITY, ZERO, CONST = 0, 1, 2, 3
DEV_BAD_EXPERT, DEV_BAD_TOKEN, DEV_TIMEOUT, DEV_OVERFLOW, DEV_BAD_INDEX = 1, 2, 4, 8, 16
BUILD_DEBUG = 1  # moe_build_flags() bit of the MOE_DEBUG build
MAX_EXPERTS = 256
NORM_NONE, NORM_LAYER, NORM_RMS = 0, 1, 2

# Names of every entry point include/moe.h declares.
ENTRY_POINTS = (
    "moe_status_string", "moe_device_check", "moe_num_assignments",
    "moe_workspace_size", "moe_router", "moe_select_topk",
    "moe_select_expert_choice", "moe_core_set_vote", "moe_core_set_union", "moe_dispatch",
    "moe_grouped_mlp", "moe_combine", "moe_forward", "moe_forward_host",
    "moe_dispatch_noalloc", "moe_activation", "moe_test_set_barrier_wait", "moe_build_flags",
    "moe_backward_workspace_size", "moe_combine_backward", "moe_dispatch_backward",
    "moe_router_backward", "moe_router_backward_logits", "moe_grouped_mlp_backward", "moe_block_norm",
    "moe_block_norm_workspace_size", "moe_block_norm_backward",
)
NOALLOC_SCRATCH_BYTES = 256 * 1024  # MOE_NOALLOC_SCRATCH_BYTES


class MoeConfig(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32), ("d", ctypes.c_int32), ("h", ctypes.c_int32),
        ("E", ctypes.c_int32), ("n_heavy", ctypes.c_int32), ("k", ctypes.c_int32),
        ("n_shared", ctypes.c_int32), ("h_shared", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("routing", ctypes.c_int32),
        ("group_size", ctypes.c_int32), ("capacity", ctypes.c_int32), ("M_core", ctypes.c_int32),
        ("gate_residual_scale", ctypes.c_float), ("renorm", ctypes.c_int32),
        ("k_local", ctypes.c_int32), ("const_mix", ctypes.c_int32),
        ("expert_kind", ctypes.c_int32 * MAX_EXPERTS),
    ]


class MoeNormConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d", "dtype", "group_size", "pre_kind", "post_kind")] + [
                    ("eps", ctypes.c_float), ("res_scale", ctypes.c_float)]


class MoeForwardAux(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("logits", "probs", "sel", "w", "votes", "core", "offsets")]


_vp, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_i64 = ctypes.c_int64
_CFG = ctypes.POINTER(MoeConfig)
_NCFG = ctypes.POINTER(MoeNormConfig)
_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [_i32]),
    "moe_device_check": (_i32, [_i32]),
    "moe_num_assignments": (_i32, [_CFG, ctypes.POINTER(ctypes.c_int64)]),
    "moe_workspace_size": (_i32, [_CFG, ctypes.POINTER(_sz)]),
    "moe_router": (_i32, [_vp, _vp, _vp, _vp, _f32, _i32, _i32, _i32, _i32, _vp, _vp, _i32, _i32,
                          _vp, _vp, _vp]),
    "moe_select_topk": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_select_expert_choice": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_core_set_vote": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "moe_core_set_union": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "moe_dispatch": (_i32, [_CFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_dispatch_noalloc": (_i32, [_CFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_activation": (_i32, [_vp, _vp, ctypes.c_int64, _i32, _vp]),
    "moe_test_set_barrier_wait": (_i32, [ctypes.c_uint64, _i32]),
    "moe_build_flags": (_i32, []),
    "moe_grouped_mlp": (_i32, [_CFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                               _vp]),
    "moe_combine": (_i32, [_CFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                           _vp]),
    "moe_forward": (_i32, [_CFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                           ctypes.POINTER(MoeForwardAux), _vp, _vp, _sz, _vp]),
    "moe_backward_workspace_size": (_i32, [_CFG, ctypes.POINTER(_sz)]),
    "moe_combine_backward": (_i32, [_CFG] + [_vp] * 11 + [_vp, _sz, _vp]),
    "moe_dispatch_backward": (_i32, [_CFG] + [_vp] * 13 + [_vp, _vp]),
    "moe_router_backward": (_i32, [_CFG] + [_vp] * 15 + [_vp, _sz, _vp]),
    "moe_router_backward_logits": (_i32, [_CFG] + [_vp] * 16 + [_vp, _sz, _vp]),
    "moe_grouped_mlp_backward": (_i32, [_CFG] + [_vp] * 16 + [_vp, _sz, _vp]),
    "moe_block_norm": (_i32, [_NCFG] + [_vp] * 8 + [_i64, _vp, _vp, _vp]),
    "moe_block_norm_workspace_size": (_i32, [_NCFG, ctypes.POINTER(_sz)]),
    "moe_block_norm_backward": (_i32, [_NCFG] + [_vp] * 7 + [_i64] + [_vp] * 10
                                + [_i64, _vp, _sz, _vp]),
    "moe_forward_host": (_i32, [_CFG, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, _sz, _vp]),
}


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is not built; run `python -m mixture_experts_layer_33_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()
LIB_PATH = _LIB_PATH


def build_flags():
    """MOE_BUILD_* bits of the loaded library (BUILD_DEBUG: the MOE_DEBUG build)."""
    return LIB.moe_build_flags()


def status_string(code):
    return LIB.moe_status_string(int(code)).decode()


def _check(code, what):
    if code != MOE_OK:
        raise RuntimeError(f"{what} failed: {status_string(code)}")


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _dev_ptr(t):
    if t is not None and not t.is_cuda:
        raise ValueError("device tensor expected")
    return _ptr(t)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


# ------------------------------------------------------------------ config
def make_config(cfg) -> MoeConfig:
    """MoeConfig from a workload dict (see ``inputs.WORKLOADS``)."""
    c = MoeConfig()
    kinds = list(cfg.get("kinds", [HEAVY] * cfg["E"]))
    c.T, c.d, c.h, c.E = cfg["T"], cfg["d"], cfg["h"], cfg["E"]
    c.n_heavy = sum(1 for k in kinds if k == HEAVY)
    c.k = cfg.get("k", 0)
    c.n_shared, c.h_shared = cfg.get("n_shared", 0), cfg.get("h_shared", 0)
    c.dtype = BF16 if cfg["dtype"] == "bf16" else F32
    c.act = SWIGLU if cfg["act"] == "swiglu" else GELU_ERF
    c.routing = {"token_topk": TOKEN_TOPK, "expert_choice": EXPERT_CHOICE,
                 "des_vote": DES_VOTE, "des_seq": DES_SEQ}[cfg["routing"]]
    c.group_size = cfg.get("group_size", 0)
    c.capacity = cfg.get("capacity", 0)
    c.M_core = cfg.get("M_core", 0)
    c.gate_residual_scale = float(cfg.get("gate_residual_scale", 0.0))
    c.renorm = int(cfg.get("renorm", 0))
    c.k_local = int(cfg.get("k_local", 0))
    c.const_mix = int(cfg.get("const_mix", 0))
    for e, k in enumerate(kinds):
        c.expert_kind[e] = k
    return c


def num_assignments(c: MoeConfig) -> int:
    n = ctypes.c_int64()
    _check(LIB.moe_num_assignments(ctypes.byref(c), ctypes.byref(n)), "moe_num_assignments")
    return n.value


def workspace_size(c: MoeConfig) -> int:
    n = _sz()
    _check(LIB.moe_workspace_size(ctypes.byref(c), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def alloc_workspace(c: MoeConfig, device="cuda"):
    """A caller-owned workspace of moe_workspace_size() bytes (256-byte aligned)."""
    return torch.empty(workspace_size(c), dtype=torch.uint8, device=device)


def device_check(device=0):
    return LIB.moe_device_check(int(device))


# ------------------------------------------------------------- entry points
def router(x, W_r, logits, probs, bias=None, z_prev=None, z_prev_scale=0.0, k=0, renorm=0,
           idx=None, w=None, stream=None):
    T, d = x.shape
    E = W_r.shape[0]
    dt = BF16 if x.dtype == torch.bfloat16 else F32
    _check(LIB.moe_router(_dev_ptr(x), _dev_ptr(W_r), _dev_ptr(bias), _dev_ptr(z_prev),
                          float(z_prev_scale), T, d, E, dt, _dev_ptr(logits), _dev_ptr(probs),
                          int(k), int(renorm), _dev_ptr(idx), _dev_ptr(w), _stream(stream)),
           "moe_router")


def select_topk(logits, probs, k, idx, w, renorm=0, stream=None):
    T, E = logits.shape
    _check(LIB.moe_select_topk(_dev_ptr(logits), _dev_ptr(probs), T, E, int(k), int(renorm),
                               _dev_ptr(idx), _dev_ptr(w), _stream(stream)), "moe_select_topk")


def select_expert_choice(probs, group_size, C, tok, w, stream=None):
    T, E = probs.shape
    _check(LIB.moe_select_expert_choice(_dev_ptr(probs), T, E, int(group_size), int(C),
                                        _dev_ptr(tok), _dev_ptr(w), _stream(stream)),
           "moe_select_expert_choice")


def core_set_vote(probs, K, M_core, votes, core, idx, w, stream=None):
    N, M = probs.shape
    _check(LIB.moe_core_set_vote(_dev_ptr(probs), N, M, int(K), int(M_core), _dev_ptr(votes),
                                 _dev_ptr(core), _dev_ptr(idx), _dev_ptr(w), _stream(stream)),
           "moe_core_set_vote")


def core_set_union(probs, K, k_local, core, n_core, idx, w, stream=None):
    N, M = probs.shape
    _check(LIB.moe_core_set_union(_dev_ptr(probs), N, M, int(K), int(k_local), _dev_ptr(core),
                                  _dev_ptr(n_core), _dev_ptr(idx), _dev_ptr(w), _stream(stream)),
           "moe_core_set_union")


def dispatch(c: MoeConfig, sel, x, x_perm, offsets, perm, row_of, tok_ptr, tok_assign,
             dev_status, ws, stream=None):
    _check(LIB.moe_dispatch(ctypes.byref(c), _dev_ptr(sel), _dev_ptr(x), _dev_ptr(x_perm),
                            _dev_ptr(offsets), _dev_ptr(perm), _dev_ptr(row_of),
                            _dev_ptr(tok_ptr), _dev_ptr(tok_assign), _dev_ptr(dev_status),
                            _dev_ptr(ws), ws.numel(), _stream(stream)), "moe_dispatch")


def dispatch_noalloc(c: MoeConfig, sel, x, x_perm, offsets, perm, row_of, tok_ptr, tok_assign,
                     dev_status, stream=None):
    """moe_dispatch for callers that cannot allocate device memory.

    Same arguments and outputs as ``dispatch`` minus the workspace: the
    library keeps the histogram scratch in a fixed device array of
    NOALLOC_SCRATCH_BYTES per GPU. Configurations whose scratch would not
    fit (ceil(n_assign/1024) * n_heavy * 4 bytes) are rejected. The first
    call on a device sets up the array's address (make it before any stream
    capture); calls that overlap on the GPU share the array and race.
    """
    code = LIB.moe_dispatch_noalloc(ctypes.byref(c), _dev_ptr(sel), _dev_ptr(x),
                                    _dev_ptr(x_perm), _dev_ptr(offsets), _dev_ptr(perm),
                                    _dev_ptr(row_of), _dev_ptr(tok_ptr), _dev_ptr(tok_assign),
                                    _dev_ptr(dev_status), _stream(stream))
    if code == 2:
        raise RuntimeError(
            "moe_dispatch_noalloc failed: the configuration's dispatch scratch "
            f"(ceil(n_assign/1024) * n_heavy * 4 bytes) exceeds the {NOALLOC_SCRATCH_BYTES}-byte "
            "library-owned array; use dispatch() with a workspace")
    _check(code, "moe_dispatch_noalloc")


def activation(x, y, act=GELU_ERF, stream=None):
    """y = GELU(x) (act=GELU_ERF) or SiLU(x) (act=SWIGLU), fp32 device tensors."""
    _check(LIB.moe_activation(_dev_ptr(x), _dev_ptr(y), x.numel(), int(act), _stream(stream)),
           "moe_activation")


def set_barrier_wait_for_tests(limit_ns=0, extra_arrivals=0):
    """Test hook: the small-block routing kernel's grid-barrier wait limit
    (ns; 0 = the 2 s default) and extra arrivals it waits for (0 = none).
    Process-wide; see moe_test_set_barrier_wait in include/moe.h."""
    _check(LIB.moe_test_set_barrier_wait(int(limit_ns), int(extra_arrivals)),
           "moe_test_set_barrier_wait")


def grouped_mlp(c: MoeConfig, x_perm, offsets, W1, W2, x, Ws1, Ws2, y_perm, y_shared,
                dev_status, ws, stream=None):
    _check(LIB.moe_grouped_mlp(ctypes.byref(c), _dev_ptr(x_perm), _dev_ptr(offsets),
                               _dev_ptr(W1), _dev_ptr(W2), _dev_ptr(x), _dev_ptr(Ws1),
                               _dev_ptr(Ws2), _dev_ptr(y_perm), _dev_ptr(y_shared),
                               _dev_ptr(dev_status), _dev_ptr(ws), ws.numel(), _stream(stream)),
           "moe_grouped_mlp")


def combine(c: MoeConfig, y_perm, y_shared, sel, w, row_of, tok_ptr, tok_assign, x, const_vecs,
            residual, y, dev_status, stream=None):
    _check(LIB.moe_combine(ctypes.byref(c), _dev_ptr(y_perm), _dev_ptr(y_shared), _dev_ptr(sel),
                           _dev_ptr(w), _dev_ptr(row_of), _dev_ptr(tok_ptr),
                           _dev_ptr(tok_assign), _dev_ptr(x), _dev_ptr(const_vecs),
                           _dev_ptr(residual), _dev_ptr(y), _dev_ptr(dev_status),
                           _stream(stream)), "moe_combine")


def forward(c: MoeConfig, x, W_r, W1, W2, y, ws, residual=None, z_prev=None, bias=None,
            Ws1=None, Ws2=None, const_vecs=None, aux=None, dev_status=None, stream=None):
    """The whole layer on device buffers. ``aux`` is a dict of optional
    output tensors (logits, probs, sel, w, votes, core, offsets)."""
    a = None
    if aux:
        a = MoeForwardAux(*[_dev_ptr(aux.get(n)) for n, _ in MoeForwardAux._fields_])
    _check(LIB.moe_forward(ctypes.byref(c), _dev_ptr(x), _dev_ptr(residual), _dev_ptr(z_prev),
                           _dev_ptr(W_r), _dev_ptr(bias), _dev_ptr(W1), _dev_ptr(W2),
                           _dev_ptr(Ws1), _dev_ptr(Ws2), _dev_ptr(const_vecs), _dev_ptr(y),
                           ctypes.byref(a) if a is not None else None, _dev_ptr(dev_status),
                           _dev_ptr(ws), ws.numel(), _stream(stream)), "moe_forward")


def forward_host(c: MoeConfig, x_host, W_r, W1, W2, y_host, ws, residual_host=None,
                 z_prev_host=None, bias=None, Ws1=None, Ws2=None, const_vecs=None,
                 dev_status=None, stream=None):
    """The whole layer with x / residual / z_prev / y in host memory (pin
    them for asynchronous copies); weights stay on the device."""
    for t in (x_host, y_host, residual_host, z_prev_host):
        if t is not None and t.is_cuda:
            raise ValueError("host tensor expected")
    _check(LIB.moe_forward_host(ctypes.byref(c), _ptr(x_host), _ptr(residual_host),
                                _ptr(z_prev_host), _dev_ptr(W_r), _dev_ptr(bias), _dev_ptr(W1),
                                _dev_ptr(W2), _dev_ptr(Ws1), _dev_ptr(Ws2),
                                _dev_ptr(const_vecs), _ptr(y_host), _dev_ptr(dev_status),
                                _dev_ptr(ws), ws.numel(), _stream(stream)), "moe_forward_host")


# ---------------------------------------------------------------- training
def _grad_ptr(t, what, dtype, numel, dev):
    """Device pointer of a tensor argument of the gradients (None stays None): dtype, size,
    contiguity and device are checked, since a short buffer would be written past its end."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if t.dtype is not dtype or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of {numel} elements, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:  # -1: a host tensor
        raise ValueError(f"{what}: expected a tensor on the current CUDA device")
    return t.data_ptr()


def _layer_dtype(c):
    return torch.bfloat16 if c.dtype == BF16 else torch.float32


# The current stream's handle without a Stream object (1 us less per call) where torch has it.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, dev):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _assignments(c):
    """moe_num_assignments of a config that the call itself will check."""
    if c.routing != EXPERT_CHOICE:
        return c.T * c.k
    return c.T // c.group_size * c.E * c.capacity if c.group_size > 0 else 0


def backward_workspace_size(c: MoeConfig) -> int:
    n = _sz()
    _check(LIB.moe_backward_workspace_size(ctypes.byref(c), ctypes.byref(n)),
           "moe_backward_workspace_size")
    return n.value


def alloc_backward_workspace(c: MoeConfig, device="cuda"):
    """A caller-owned workspace for the backward entry points, which may share it as long
    as they do not overlap on the device."""
    return torch.empty(backward_workspace_size(c), dtype=torch.uint8, device=device)


def _n_const(c):
    return sum(1 for e in range(c.n_heavy, c.E) if c.expert_kind[e] == CONST)


def combine_backward(c: MoeConfig, dy, y_perm, sel, w, row_of, tok_ptr, tok_assign, x, const_vecs,
                     dy_perm, dw, dev_status, ws, dconst=None, stream=None):
    """Gradient of ``combine`` (moe_combine_backward in include/moe.h). The token lists are
    accepted for symmetry with ``combine`` and not read."""
    n, dt, f32, i32 = _assignments(c), _layer_dtype(c), torch.float32, torch.int32
    dev = torch.cuda.current_device()
    nc = _n_const(c) * (3 if c.const_mix else 1) * c.d if c.n_heavy < c.E else 0
    _check(LIB.moe_combine_backward(
        ctypes.byref(c), _grad_ptr(dy, "dy", dt, c.T * c.d, dev), _grad_ptr(y_perm, "y_perm", dt, n * c.d, dev),
        _grad_ptr(sel, "sel", i32, n, dev), _grad_ptr(w, "w", f32, n, dev), _grad_ptr(row_of, "row_of", i32, n, dev),
        _grad_ptr(x, "x", dt, c.T * c.d, dev), _grad_ptr(const_vecs, "const_vecs", dt, nc, dev),
        _grad_ptr(dy_perm, "dy_perm", dt, n * c.d, dev), _grad_ptr(dw, "dw", f32, n, dev),
        _grad_ptr(dconst, "dconst", f32, nc, dev), _grad_ptr(dev_status, "dev_status", i32, 1, dev),
        _grad_ptr(ws, "ws", torch.uint8, ws.numel(), dev), ws.numel(), _raw_stream(stream, dev)), "moe_combine_backward")


def dispatch_backward(c: MoeConfig, dx_perm, dy, sel, w, row_of, tok_ptr, tok_assign, x, const_vecs,
                      dx, dev_status, add=(), stream=None):
    """Gradient of ``dispatch``'s row gather and of the combine's x terms, with up to three
    [T, d] gradients ``add`` summed in the same pass (moe_dispatch_backward)."""
    n, dt, f32, i32 = _assignments(c), _layer_dtype(c), torch.float32, torch.int32
    dev = torch.cuda.current_device()
    nc = _n_const(c) * (3 if c.const_mix else 1) * c.d if c.n_heavy < c.E else 0
    if len(add) > 3:
        raise ValueError("add: at most three gradients")
    adds = [_grad_ptr(t, "add", dt, c.T * c.d, dev) for t in add] + [None] * (3 - len(add))
    _check(LIB.moe_dispatch_backward(
        ctypes.byref(c), _grad_ptr(dx_perm, "dx_perm", dt, n * c.d, dev), _grad_ptr(dy, "dy", dt, c.T * c.d, dev),
        _grad_ptr(sel, "sel", i32, n, dev), _grad_ptr(w, "w", f32, n, dev), _grad_ptr(row_of, "row_of", i32, n, dev),
        _grad_ptr(tok_ptr, "tok_ptr", i32, c.T + 1, dev), _grad_ptr(tok_assign, "tok_assign", i32, n, dev),
        _grad_ptr(x, "x", dt, c.T * c.d, dev), _grad_ptr(const_vecs, "const_vecs", dt, nc, dev), *adds,
        _grad_ptr(dx, "dx", dt, c.T * c.d, dev), _grad_ptr(dev_status, "dev_status", i32, 1, dev),
        _raw_stream(stream, dev)), "moe_dispatch_backward")


def router_backward(c: MoeConfig, x, W_r, probs, sel, w, dw, tok_ptr, tok_assign, dlogits,
                    dev_status, ws, dprobs=None, dz_prev=None, dbias=None, dW_r=None, dx=None,
                    stream=None, dz_next=None):
    """Gradient of the routing weights back through selection and softmax to the logits, and
    from there to the router's inputs (moe_router_backward). ``dz_next``: the next layer's
    ``dz_prev``, when it takes these logits as its gate residual (moe_router_backward_logits)."""
    n, dt, f32, i32 = _assignments(c), _layer_dtype(c), torch.float32, torch.int32
    dev = torch.cuda.current_device()
    te = c.T * c.E
    _check(LIB.moe_router_backward_logits(
        ctypes.byref(c), _grad_ptr(x, "x", dt, c.T * c.d, dev), _grad_ptr(W_r, "W_r", dt, c.E * c.d, dev),
        _grad_ptr(probs, "probs", f32, te, dev), _grad_ptr(sel, "sel", i32, n, dev), _grad_ptr(w, "w", f32, n, dev),
        _grad_ptr(dw, "dw", f32, n, dev), _grad_ptr(tok_ptr, "tok_ptr", i32, c.T + 1, dev),
        _grad_ptr(tok_assign, "tok_assign", i32, n, dev), _grad_ptr(dprobs, "dprobs", f32, te, dev),
        _grad_ptr(dz_next, "dz_next", f32, te, dev),
        _grad_ptr(dlogits, "dlogits", f32, te, dev), _grad_ptr(dz_prev, "dz_prev", f32, te, dev),
        _grad_ptr(dbias, "dbias", f32, c.E, dev), _grad_ptr(dW_r, "dW_r", f32, c.E * c.d, dev),
        _grad_ptr(dx, "dx", dt, c.T * c.d, dev), _grad_ptr(dev_status, "dev_status", i32, 1, dev),
        _grad_ptr(ws, "ws", torch.uint8, ws.numel(), dev), ws.numel(), _raw_stream(stream, dev)), "moe_router_backward")


def grouped_mlp_backward(c: MoeConfig, x_perm, offsets, W1, W2, dy_perm, x, Ws1, Ws2, dy_shared,
                         dev_status, ws, dx_perm=None, dW1=None, dW2=None, dx_shared=None,
                         dWs1=None, dWs2=None, stream=None):
    """Gradient of ``grouped_mlp``; any output may be left out (moe_grouped_mlp_backward)."""
    n, dt, i32 = _assignments(c), _layer_dtype(c), torch.int32
    dev = torch.cuda.current_device()
    up, hs = (2 * c.h if c.act == SWIGLU else c.h), c.n_shared * c.h_shared
    n1, n2, ns, td = c.n_heavy * up * c.d, c.n_heavy * c.h * c.d, hs * c.d, c.T * c.d
    _check(LIB.moe_grouped_mlp_backward(
        ctypes.byref(c), _grad_ptr(x_perm, "x_perm", dt, n * c.d, dev),
        _grad_ptr(offsets, "offsets", i32, c.n_heavy + 1, dev), _grad_ptr(W1, "W1", dt, n1, dev),
        _grad_ptr(W2, "W2", dt, n2, dev), _grad_ptr(dy_perm, "dy_perm", dt, n * c.d, dev),
        _grad_ptr(x, "x", dt, td, dev), _grad_ptr(Ws1, "Ws1", dt, ns, dev), _grad_ptr(Ws2, "Ws2", dt, ns, dev),
        _grad_ptr(dy_shared, "dy_shared", dt, td, dev), _grad_ptr(dx_perm, "dx_perm", dt, n * c.d, dev),
        _grad_ptr(dW1, "dW1", dt, n1, dev), _grad_ptr(dW2, "dW2", dt, n2, dev),
        _grad_ptr(dx_shared, "dx_shared", dt, td, dev), _grad_ptr(dWs1, "dWs1", dt, ns, dev),
        _grad_ptr(dWs2, "dWs2", dt, ns, dev), _grad_ptr(dev_status, "dev_status", i32, 1, dev),
        _grad_ptr(ws, "ws", torch.uint8, ws.numel(), dev), ws.numel(), _raw_stream(stream, dev)), "moe_grouped_mlp_backward")


# ------------------------------------------------------------- block norms
def make_norm_config(cfg) -> MoeNormConfig:
    """MoeNormConfig from a dict: T, d, dtype ("bf16" / "f32"), group_size (tokens per condition
    row, 0 for one row), pre and post ("none", "layer", "rms"), eps, res_scale."""
    kinds = {"none": NORM_NONE, "layer": NORM_LAYER, "rms": NORM_RMS}
    return MoeNormConfig(cfg["T"], cfg["d"], BF16 if cfg["dtype"] == "bf16" else F32,
                         cfg.get("group_size", 0), kinds[cfg.get("pre", "layer")],
                         kinds[cfg.get("post", "none")], float(cfg.get("eps", 1e-6)),
                         float(cfg.get("res_scale", 1.0)))


def _cond_ptrs(n: MoeNormConfig, named, dtype, dev):
    """Pointers and the common row stride of condition tensors [rows, d]: chunks of one
    projection, so rows may be further apart than d."""
    rows = -(-n.T // n.group_size) if n.group_size else 1
    stride, ptrs = n.d, []
    for what, t in named:
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype != dtype or tuple(t.shape) != (rows, n.d) or t.stride(1) != 1:
            raise ValueError(f"{what}: expected {dtype} rows [{rows}, {n.d}], got {t.dtype} "
                             f"{tuple(t.shape)} with strides {t.stride()}")
        if t.get_device() != dev:
            raise ValueError(f"{what}: expected a tensor on the current CUDA device")
        if rows > 1:
            if any(p is not None for p in ptrs) and t.stride(0) != stride:
                raise ValueError("condition tensors must have the same row stride")
            stride = t.stride(0)
        ptrs.append(t.data_ptr())
    return ptrs, stride


def block_norm(n: MoeNormConfig, h, x, y=None, z=None, post_gamma=None, gate=None, pre_gamma=None,
               pre_beta=None, scale=None, shift=None, stream=None):
    """y = res_scale x + gate N_post(h) post_gamma; z = (N_pre(y) pre_gamma + pre_beta)(1 + scale)
    + shift (moe_block_norm): the end of one block and the start of the next in one pass."""
    dt, dev = _layer_dtype(n), torch.cuda.current_device()
    td = n.T * n.d
    (gp, scp, shp), stride = _cond_ptrs(n, (("gate", gate), ("scale", scale), ("shift", shift)), dt, dev)
    _check(LIB.moe_block_norm(
        ctypes.byref(n), _grad_ptr(h, "h", dt, td, dev), _grad_ptr(x, "x", dt, td, dev),
        _grad_ptr(post_gamma, "post_gamma", dt, n.d, dev), gp, _grad_ptr(pre_gamma, "pre_gamma", dt, n.d, dev),
        _grad_ptr(pre_beta, "pre_beta", dt, n.d, dev), scp, shp, stride, _grad_ptr(y, "y", dt, td, dev),
        _grad_ptr(z, "z", dt, td, dev), _raw_stream(stream, dev)), "moe_block_norm")


def block_norm_workspace_size(n: MoeNormConfig) -> int:
    b = _sz()
    _check(LIB.moe_block_norm_workspace_size(ctypes.byref(n), ctypes.byref(b)),
           "moe_block_norm_workspace_size")
    return b.value


def alloc_block_norm_workspace(n: MoeNormConfig, device="cuda"):
    return torch.empty(block_norm_workspace_size(n), dtype=torch.uint8, device=device)


def block_norm_backward(n: MoeNormConfig, h, y, dz, dy, ws, dh=None, dx=None, post_gamma=None,
                        gate=None, pre_gamma=None, pre_beta=None, scale=None, dpost_gamma=None,
                        dgate=None, dpre_gamma=None, dpre_beta=None, dscale=None, dshift=None,
                        stream=None):
    """Gradient of ``block_norm`` from dz and dy (moe_block_norm_backward)."""
    dt, f32, dev = _layer_dtype(n), torch.float32, torch.cuda.current_device()
    td = n.T * n.d
    (gp, scp), stride = _cond_ptrs(n, (("gate", gate), ("scale", scale)), dt, dev)
    (dgp, dscp, dshp), dstride = _cond_ptrs(
        n, (("dgate", dgate), ("dscale", dscale), ("dshift", dshift)), f32, dev)
    _check(LIB.moe_block_norm_backward(
        ctypes.byref(n), _grad_ptr(h, "h", dt, td, dev), _grad_ptr(y, "y", dt, td, dev),
        _grad_ptr(post_gamma, "post_gamma", dt, n.d, dev), gp, _grad_ptr(pre_gamma, "pre_gamma", dt, n.d, dev),
        _grad_ptr(pre_beta, "pre_beta", dt, n.d, dev), scp, stride, _grad_ptr(dz, "dz", dt, td, dev),
        _grad_ptr(dy, "dy", dt, td, dev), _grad_ptr(dh, "dh", dt, td, dev), _grad_ptr(dx, "dx", dt, td, dev),
        _grad_ptr(dpost_gamma, "dpost_gamma", f32, n.d, dev), dgp,
        _grad_ptr(dpre_gamma, "dpre_gamma", f32, n.d, dev), _grad_ptr(dpre_beta, "dpre_beta", f32, n.d, dev),
        dscp, dshp, dstride, _grad_ptr(ws, "ws", torch.uint8, ws.numel(), dev), ws.numel(), _raw_stream(stream, dev)), "moe_block_norm_backward")


def _tensors(*trees):
    """The device tensors in nested tuples and dicts."""
    for t in trees:
        if isinstance(t, torch.Tensor):
            if t.is_cuda:
                yield t
        elif isinstance(t, (tuple, list)):
            yield from _tensors(*t)
        elif isinstance(t, dict):
            yield from _tensors(*t.values())


def _run_on(stream, step, inputs):
    """``step()`` on ``stream`` (None: the current stream, as it is). What the step allocates
    belongs to ``stream``, so a block it frees goes to later work of that stream only, while its
    kernels may still be queued; ``inputs`` and the results, which the caller holds and frees, are
    marked as used by both streams."""
    if stream is None:
        return step()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    caller = torch.cuda.current_stream()
    for t in _tensors(inputs):
        t.record_stream(stream)
    with torch.cuda.stream(stream):
        out = step()
    for t in _tensors(out):
        t.record_stream(caller)
    return out


class MoELayer:
    """A configured layer: weights and a workspace resident on one device.

    ``layer(x, z_prev=None)`` returns y; ``residual`` defaults to x.
    ``layer.forward_train(x)`` runs the same layer step by step and keeps what
    ``layer.backward`` needs to turn dy into the gradients of x, the weights
    and the gate residual.

    All three take a ``stream``: the work runs there, after what that stream
    already holds, and the results are ready in its order. A layer's calls
    share its workspaces, so they must not overlap on the device.
    """

    def __init__(self, cfg, weights, device="cuda"):
        self.cfg = cfg
        self.c = make_config(cfg)
        self.w = weights
        self.ws = alloc_workspace(self.c, device)
        self.bws = None  # the backward's workspace, made on first use
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def __call__(self, x, z_prev=None, residual="x", aux=None, stream=None):
        return _run_on(stream, lambda: self._forward(x, z_prev, residual, aux),
                       (x, z_prev, residual, aux, self.ws, self.status))

    def _forward(self, x, z_prev, residual, aux):
        y = torch.empty_like(x)
        res = x if isinstance(residual, str) else residual
        w = self.w
        forward(self.c, x, w["W_r"], w.get("W1"), w.get("W2"), y, self.ws, residual=res, z_prev=z_prev,
                bias=w.get("logit_bias"), Ws1=w.get("Ws1"), Ws2=w.get("Ws2"),
                const_vecs=w.get("const_vecs"), aux=aux, dev_status=self.status)
        return y

    def forward_train(self, x, z_prev=None, residual="x", stream=None):
        """The layer through its stage entry points: (y, saved), ``saved`` holding the routing,
        the dispatched rows and the expert outputs for ``backward``. ``residual`` is "x" or x
        itself (the layer adds x), None, or another [T, d] tensor. ``saved`` keeps x, not a copy."""
        return _run_on(stream, lambda: self._forward_train(x, z_prev, residual),
                       (x, z_prev, residual, self.ws, self.status))

    def _forward_train(self, x, z_prev, residual):
        c, w, dev, i32 = self.c, self.w, x.device, torch.int32
        # The step's buffers have the config's sizes: a longer batch would be written past their ends.
        dt, at = _layer_dtype(c), torch.cuda.current_device() if x.is_cuda else -1
        if tuple(x.shape) != (c.T, c.d):
            raise ValueError(f"x: expected [{c.T}, {c.d}], got {tuple(x.shape)}")
        _grad_ptr(x, "x", dt, c.T * c.d, at)
        _grad_ptr(z_prev, "z_prev", torch.float32, c.T * c.E, at)
        if not isinstance(residual, str):
            _grad_ptr(residual, "residual", dt, c.T * c.d, at)
        n, T, E = num_assignments(c), c.T, c.E
        ec = c.routing == EXPERT_CHOICE

        def ints(*shape):
            return torch.empty(*shape, dtype=i32, device=dev)

        def floats(*shape):  # fp32 whatever torch's default type is: the kernels write 4 bytes
            return torch.empty(*shape, dtype=torch.float32, device=dev)

        s = {"x": x, "residual": "x" if residual is x else residual,
             "logits": floats(T, E), "probs": floats(T, E),
             "sel": ints(n), "w": floats(n), "offsets": ints(c.n_heavy + 1),
             "row_of": ints(n), "tok_ptr": ints(T + 1) if ec else None,
             "tok_assign": ints(n) if ec else None,
             "x_perm": torch.empty(n, c.d, dtype=x.dtype, device=dev),
             "y_perm": torch.empty(n, c.d, dtype=x.dtype, device=dev)}
        if T == 0:  # no rows to route; the weights' gradients are zero
            s["offsets"].zero_()
            return torch.empty_like(x), s
        topk = c.routing == TOKEN_TOPK
        router(x, w["W_r"], s["logits"], s["probs"], bias=w.get("logit_bias"), z_prev=z_prev,
               z_prev_scale=c.gate_residual_scale, k=c.k if topk else 0, renorm=c.renorm if topk else 0,
               idx=s["sel"] if topk else None, w=s["w"] if topk else None)
        if ec:
            select_expert_choice(s["probs"], c.group_size, c.capacity, s["sel"], s["w"])
        elif c.routing == DES_VOTE:
            votes = torch.empty(E, dtype=torch.int64, device=dev)
            core_set_vote(s["probs"], c.k, c.M_core, votes, ints(c.M_core), s["sel"], s["w"])
        elif c.routing == DES_SEQ:
            core_set_union(s["probs"], c.k, c.k_local, ints(E), ints(1), s["sel"], s["w"])
        dispatch(c, s["sel"], x, s["x_perm"], s["offsets"], ints(n), s["row_of"], s["tok_ptr"],
                 s["tok_assign"], self.status, self.ws)
        y_shared = torch.empty_like(x) if c.n_shared else None
        grouped_mlp(c, s["x_perm"], s["offsets"], w.get("W1"), w.get("W2"), x, w.get("Ws1"), w.get("Ws2"),
                    s["y_perm"], y_shared, self.status, self.ws)
        y = torch.empty_like(x)
        combine(c, s["y_perm"], y_shared, s["sel"], s["w"], s["row_of"], s["tok_ptr"],
                s["tok_assign"], x, w.get("const_vecs"), x if isinstance(residual, str) else residual,
                y, self.status)
        return y, s

    def backward(self, saved, dy, dprobs=None, stream=None, dlogits=None):
        """Gradients from dy, the gradient of ``forward_train``'s y, and from gradients that reach
        the affinities (``dprobs``) or the logits (``dlogits``: the z_prev gradient of a next layer
        whose gate residual is ``saved["logits"]``) directly: a dict of x, W_r, logit_bias, W1, W2,
        Ws1, Ws2, const_vecs and z_prev (those the layer has; zero for a weight that none of its experts
        reads). A residual other than x has gradient dy."""
        if self.bws is None:
            self.bws = _run_on(stream, lambda: alloc_backward_workspace(self.c, dy.device), ())
        return _run_on(stream, lambda: self._backward(saved, dy, dprobs, dlogits),
                       (saved, dy, dprobs, dlogits, self.bws, self.status))

    def _backward(self, saved, dy, dprobs, dlogits):
        c, w, s, dev = self.c, self.w, saved, dy.device
        n, x = num_assignments(c), saved["x"]

        def floats(*shape):
            return torch.empty(*shape, dtype=torch.float32, device=dev)

        # Weights that none of the layer's experts reads have gradient zero and go no further.
        used = {"W1": c.n_heavy > 0, "W2": c.n_heavy > 0, "Ws1": c.n_shared > 0, "Ws2": c.n_shared > 0,
                "const_vecs": _n_const(c) > 0}
        W = {k: w.get(k) if on else None for k, on in used.items()}
        cv = W["const_vecs"]
        routing = (s["sel"], s["w"], s["row_of"], s["tok_ptr"], s["tok_assign"], x, cv)
        dy_perm, dw = torch.empty_like(s["y_perm"]), floats(n)
        g = {"W_r": floats(c.E, c.d), "x": torch.empty_like(x)}
        for k, on in used.items():
            if w.get(k) is not None:
                new = torch.empty_like if on else torch.zeros_like
                g[k] = new(w[k], dtype=torch.float32 if k == "const_vecs" else w[k].dtype)
        if w.get("logit_bias") is not None:
            g["logit_bias"] = floats(c.E)
        if c.gate_residual_scale:
            g["z_prev"] = floats(c.T, c.E)
        out = {k: g.get(k) if on else None for k, on in used.items()}
        combine_backward(c, dy, s["y_perm"], *routing, dy_perm, dw, self.status, self.bws,
                         dconst=out["const_vecs"])
        dx_perm = torch.empty_like(s["x_perm"])
        dx_shared = torch.empty_like(x) if c.n_shared else None
        grouped_mlp_backward(c, s["x_perm"], s["offsets"], W["W1"], W["W2"], dy_perm, x, W["Ws1"], W["Ws2"], dy,
                             self.status, self.bws, dx_perm=dx_perm, dW1=out["W1"], dW2=out["W2"],
                             dx_shared=dx_shared, dWs1=out["Ws1"], dWs2=out["Ws2"])
        dx_router = torch.empty_like(x)
        router_backward(c, x, w["W_r"], s["probs"], s["sel"], s["w"], dw, s["tok_ptr"], s["tok_assign"],
                        torch.empty_like(s["probs"]), self.status, self.bws, dprobs=dprobs,
                        dz_prev=g.get("z_prev"), dbias=g.get("logit_bias"), dW_r=g["W_r"], dx=dx_router,
                        dz_next=dlogits)
        add = [dx_router] + ([dx_shared] if c.n_shared else [])
        if isinstance(s["residual"], str):
            add.append(dy)
        dispatch_backward(c, dx_perm, dy, *routing, g["x"], self.status, add=add)
        return g
