"""ctypes binding of libmoe.so (C ABI in include/moe.h).

Argument marshalling only: each function checks the tensors it is given
(device, dtype, shape, contiguity), passes their device pointers and the
current CUDA stream to the function of the same name in libmoe.so, and raises
MoEError on a non-zero status.  Every step of the block runs in the library's
CUDA kernels; there is no CPU path, and a missing library raises at load time.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4
MOE_ERR_DEVICE_TIMEOUT = -5
MOE_ERR_SCRATCH_LIMIT = -6
MOE_ERR_NONFINITE = -7

SCORE_FNS = {"softmax": 0, "sigmoid": 1, "sqrt_softplus": 2}

WS_REGIONS = {"logits": 0, "counts": 1, "offsets": 2, "perm": 3, "row_w": 4, "inv": 5,
              "h": 6, "h_shared": 7, "y": 8, "y_shared": 9, "x_stage": 10,
              "work_counts": 11, "work_gate_up": 12, "work_down": 13}

EXPORTED = ["moe_version", "moe_status_string", "moe_workspace_bytes", "moe_forward",
            "moe_forward_host", "moe_route", "moe_permute", "moe_expert_gate_up", "moe_expert_down",
            "moe_combine", "moe_workspace_region", "moe_device_status", "moe_debug_wait_timeout",
            "moe_route_noalloc", "moe_experts_forward", "moe_rmsnorm", "moe_forward_prenorm",
            "moe_forward_fp8", "moe_expert_gate_up_fp8", "moe_expert_down_fp8", "moe_permute_fp8",
            "moe_sort_tokens", "moe_dispatch", "moe_dispatch_backward", "moe_undispatch", "moe_undispatch_backward",
            "moe_quantize_fp4", "moe_dequantize_fp4", "moe_dispatch_fp4", "moe_matmul_fp4", "moe_swiglu_fp4"]

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
DISPATCH_WORKSPACE_BYTES = 256


class MoEError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("d_ff_shared", ctypes.c_int32)]


class MoeFp8Weight(ctypes.Structure):
    """moe_fp8_weight: E4M3 codes [G, rows, K] and UE8M0 block scales [G, K/32, rows]."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class MoeFp4Tensor(ctypes.Structure):
    """moe_fp4_tensor: E2M1 codes [G, rows, K/2] and UE8M0 block scales [G, ceil(K/128), rows, 4]."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_FAST_CALLS = ["sort_tokens", "dispatch", "dispatch_backward", "undispatch", "undispatch_backward", "quantize_fp4",
               "dequantize_fp4", "dispatch_fp4", "matmul_fp4", "swiglu_fp4"]   # csrc/fastcall.cpp's order

_lib = None
_fastcall = None


def load():
    """Load libmoe.so (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmoe.so not found at {LIB_PATH}: build it with "
                           "`python -m mixture_experts_ffn_16_b200.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    SH = ctypes.POINTER(MoeShape)
    lib.moe_version.restype = I
    lib.moe_version.argtypes = []
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_status_string.argtypes = [I]
    lib.moe_workspace_bytes.restype = SZ
    lib.moe_workspace_bytes.argtypes = [SH]
    fwd = [SH, P, P, P, P, P, P, P, P, P, P, I, I, ctypes.c_float, P, P, P, P, SZ, P]
    lib.moe_forward.restype = I
    lib.moe_forward.argtypes = fwd
    lib.moe_forward_host.restype = I
    lib.moe_forward_host.argtypes = fwd
    lib.moe_forward_prenorm.restype = I
    lib.moe_forward_prenorm.argtypes = [SH, P, P, ctypes.c_float] + fwd[2:]
    F8 = ctypes.POINTER(MoeFp8Weight)
    lib.moe_forward_fp8.restype = I
    lib.moe_forward_fp8.argtypes = [SH, P, P, P, F8, F8, F8, F8, F8, F8] + fwd[10:]
    lib.moe_permute_fp8.restype = I
    lib.moe_permute_fp8.argtypes = [SH, P, P, P, SZ, P]
    lib.moe_expert_gate_up_fp8.restype = I
    lib.moe_expert_gate_up_fp8.argtypes = [SH, P, F8, F8, F8, F8, P, SZ, P]
    lib.moe_expert_down_fp8.restype = I
    lib.moe_expert_down_fp8.argtypes = [SH, F8, F8, P, SZ, P]
    lib.moe_rmsnorm.restype = I
    lib.moe_rmsnorm.argtypes = [SH, P, P, ctypes.c_float, P, P]
    lib.moe_route.restype = I
    lib.moe_route.argtypes = [SH, P, P, P, I, I, ctypes.c_float, P, P, P, SZ, P]
    lib.moe_permute.restype = I
    lib.moe_permute.argtypes = [SH, P, P, P, SZ, P]
    lib.moe_expert_gate_up.restype = I
    lib.moe_expert_gate_up.argtypes = [SH, P, P, P, P, P, P, SZ, P]
    lib.moe_expert_down.restype = I
    lib.moe_expert_down.argtypes = [SH, P, P, P, SZ, P]
    lib.moe_combine.restype = I
    lib.moe_combine.argtypes = [SH, P, P, P, P, SZ, P]
    lib.moe_experts_forward.restype = I
    lib.moe_experts_forward.argtypes = [SH, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
    lib.moe_workspace_region.restype = I
    lib.moe_workspace_region.argtypes = [SH, I, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
    lib.moe_device_status.restype = I
    lib.moe_device_status.argtypes = [P, P]
    lib.moe_debug_wait_timeout.restype = I
    lib.moe_debug_wait_timeout.argtypes = [P, SZ, ctypes.c_uint64, P]
    lib.moe_route_noalloc.restype = I
    lib.moe_route_noalloc.argtypes = [SH, P, P, P, I, I, ctypes.c_float, P, P, P]
    F4 = ctypes.POINTER(MoeFp4Tensor)
    for name, args in (("sort_tokens", [I, I, I, P, P, P, P, SZ, P]),
                       ("dispatch", [I, I, I, I, P, P, P, P]),
                       ("dispatch_backward", [I, I, I, I, P, P, P, P]),
                       ("undispatch", [I, I, I, I, P, P, P, P, P]),
                       ("undispatch_backward", [I, I, I, I, P, P, P, P, P, P, P]),
                       ("quantize_fp4", [I, I, I, I, P, F4, P]),
                       ("dequantize_fp4", [I, I, I, I, F4, P, P]),
                       ("dispatch_fp4", [I, I, I, I, P, P, F4, P]),
                       ("matmul_fp4", [I, I, I, I, F4, P, F4, I, P, P, SZ, P]),
                       ("swiglu_fp4", [I, I, I, I, F4, P, F4, F4, F4, P, SZ, P])):
        fn = getattr(lib, "moe_" + name)
        fn.restype = I
        fn.argtypes = args
    _lib = lib
    return lib


class _NoFast:
    """In place of the native part where it has not been built for this torch and Python: makes no call."""

    def __getattr__(self, name):
        return lambda *args: None


def _fast():
    """The native part of the binding (csrc/fastcall.cpp), given the library's addresses once."""
    global _fastcall
    if _fastcall is None:
        lib = load()
        loader = importlib.machinery.ExtensionFileLoader(__package__ + "._fastcall", _build.fastcall_path())
        try:
            native = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
            loader.exec_module(native)
        except ImportError as e:
            warnings.warn(f"token-dispatch and MXFP4 calls go through ctypes, 3 us of host time more each, until "
                          f"`python -m {__package__}.build` has built their native part: {e}")
            _fastcall = _NoFast()
            return _fastcall
        native.bind(tuple(ctypes.cast(getattr(lib, "moe_" + n), ctypes.c_void_p).value for n in _FAST_CALLS))
        _fastcall = native
    return _fastcall


def _done(status, where):
    """Whether the native part made the call (None: it did not)."""
    if status is None:
        return False
    _check(status, where)
    return True


def status_string(status):
    try:
        return load().moe_status_string(int(status)).decode()
    except Exception:  # noqa: BLE001 - message formatting only
        return "status"


def make_shape(T, d_model, E, k, d_ff, n_shared=0, d_ff_shared=0):
    return MoeShape(int(T), int(d_model), int(E), int(k), int(d_ff), int(n_shared), int(d_ff_shared))


def shape_of(cfg):
    """moe_shape of a MoEConfig (inputs.MoEConfig)."""
    return make_shape(cfg.T, cfg.d, cfg.E, cfg.k, cfg.f, cfg.S, cfg.fs)


def moe_workspace_bytes(shape) -> int:
    return int(load().moe_workspace_bytes(ctypes.byref(shape)))


def moe_workspace_region(shape, region):
    """(offset, bytes) of a named workspace region (see WS_REGIONS)."""
    off, nb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    r = WS_REGIONS[region] if isinstance(region, str) else int(region)
    st = load().moe_workspace_region(ctypes.byref(shape), r, ctypes.byref(off), ctypes.byref(nb))
    if st != MOE_OK:
        raise MoEError(st, "moe_workspace_region")
    return off.value, nb.value


def alloc_workspace(shape, device=None):
    """A device byte tensor large enough for `shape` (256-byte aligned by torch's allocator)."""
    n = moe_workspace_bytes(shape)
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    assert ws.data_ptr() % 256 == 0
    return ws


def _stream(stream):
    if stream is None:
        # the current stream's handle without a Stream object around it (0.1 us against 3.3 us)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _p(t, dtype=None, shape=None, name="", host=False):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if host != (t.device.type == "cpu"):
        raise ValueError(f"{name}: expected a {'host' if host else 'CUDA'} tensor, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.is_neg():                   # the memory holds the negated values
        raise ValueError(f"{name}: a view that negates another tensor (take its resolve_neg())")
    return ctypes.c_void_p(t.data_ptr())


def _check(st, where):
    if st != MOE_OK:
        raise MoEError(st, where)


def _score(score_fn):
    return SCORE_FNS[score_fn] if isinstance(score_fn, str) else int(score_fn)


def _weights(shape, W_gate, W_up, W_down, W_shared_gate, W_shared_up, W_shared_down):
    E, f, d, S, fs = shape.E, shape.d_ff, shape.d_model, shape.n_shared, shape.d_ff_shared
    bf = torch.bfloat16
    return [_p(W_gate, bf, (E, f, d), "W_gate"), _p(W_up, bf, (E, f, d), "W_up"),
            _p(W_down, bf, (E, d, f), "W_down"),
            _p(W_shared_gate, bf, (S, fs, d), "W_shared_gate") if S else None,
            _p(W_shared_up, bf, (S, fs, d), "W_shared_up") if S else None,
            _p(W_shared_down, bf, (S, d, fs), "W_shared_down") if S else None]


def _f8(w, G, rows, K, name):
    """(codes, scales) tensors -> a MoeFp8Weight (None when w is None)."""
    if w is None:
        return None
    codes, scales = w
    return MoeFp8Weight(_p(codes, torch.uint8, (G, rows, K), name + ".codes"),
                        _p(scales, torch.uint8, (G, K // 32, rows), name + ".scales"))


def _f8_weights(shape, W_gate, W_up, W_down, W_shared_gate, W_shared_up, W_shared_down):
    E, f, d, S, fs = shape.E, shape.d_ff, shape.d_model, shape.n_shared, shape.d_ff_shared
    ws = [_f8(W_gate, E, f, d, "W_gate"), _f8(W_up, E, f, d, "W_up"), _f8(W_down, E, d, f, "W_down"),
          _f8(W_shared_gate, S, fs, d, "W_shared_gate") if S else None,
          _f8(W_shared_up, S, fs, d, "W_shared_up") if S else None,
          _f8(W_shared_down, S, d, fs, "W_shared_down") if S else None]
    return [None if w is None else ctypes.pointer(w) for w in ws]


def _gate_vec(shape, W_shared_gate_vec):
    if W_shared_gate_vec is None:
        return None
    return _p(W_shared_gate_vec, torch.bfloat16, (shape.n_shared, shape.d_model), "W_shared_gate_vec")


def moe_forward(shape, x, W_router, expert_bias, W_gate, W_up, W_down, W_shared_gate, W_shared_up,
                W_shared_down, score_fn, norm_topk, route_scale, out, topk_idx, topk_w, workspace,
                stream=None, W_shared_gate_vec=None):
    T, d, E, k = shape.T, shape.d_model, shape.E, shape.k
    bf = torch.bfloat16
    st = load().moe_forward(
        ctypes.byref(shape), _p(x, bf, (T, d), "x"), _p(W_router, bf, (E, d), "W_router"),
        _p(expert_bias, torch.float32, (E,), "expert_bias"),
        *_weights(shape, W_gate, W_up, W_down, W_shared_gate, W_shared_up, W_shared_down),
        _gate_vec(shape, W_shared_gate_vec), _score(score_fn), int(bool(norm_topk)), float(route_scale),
        _p(out, bf, (T, d), "out"), _p(topk_idx, torch.int32, (T, k), "topk_idx"),
        _p(topk_w, torch.float32, (T, k), "topk_w"),
        _p(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "moe_forward")


def moe_forward_prenorm(shape, x, norm_gain, norm_eps, W_router, expert_bias, W_gate, W_up, W_down,
                        W_shared_gate, W_shared_up, W_shared_down, score_fn, norm_topk, route_scale, out,
                        topk_idx, topk_w, workspace, stream=None, W_shared_gate_vec=None):
    """moe_forward behind the pre-norm RMSNorm (zero-centred gains): x is the raw
    residual stream; the normalised rows are left in the workspace region "x_stage"."""
    T, d, E, k = shape.T, shape.d_model, shape.E, shape.k
    bf = torch.bfloat16
    st = load().moe_forward_prenorm(
        ctypes.byref(shape), _p(x, bf, (T, d), "x"), _p(norm_gain, bf, (d,), "norm_gain"), float(norm_eps),
        _p(W_router, bf, (E, d), "W_router"), _p(expert_bias, torch.float32, (E,), "expert_bias"),
        *_weights(shape, W_gate, W_up, W_down, W_shared_gate, W_shared_up, W_shared_down),
        _gate_vec(shape, W_shared_gate_vec), _score(score_fn), int(bool(norm_topk)), float(route_scale),
        _p(out, bf, (T, d), "out"), _p(topk_idx, torch.int32, (T, k), "topk_idx"),
        _p(topk_w, torch.float32, (T, k), "topk_w"),
        _p(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "moe_forward_prenorm")


def moe_forward_fp8(shape, x, W_router, expert_bias, W_gate, W_up, W_down, W_shared_gate, W_shared_up,
                    W_shared_down, score_fn, norm_topk, route_scale, out, topk_idx, topk_w, workspace,
                    stream=None, W_shared_gate_vec=None):
    """moe_forward with block-scaled FP8 expert weights: each W_* is a
    (codes uint8 [G, rows, K], scales uint8 [G, K/32, rows]) pair, or None for
    the shared ones when n_shared == 0."""
    T, d, E, k = shape.T, shape.d_model, shape.E, shape.k
    bf = torch.bfloat16
    st = load().moe_forward_fp8(
        ctypes.byref(shape), _p(x, bf, (T, d), "x"), _p(W_router, bf, (E, d), "W_router"),
        _p(expert_bias, torch.float32, (E,), "expert_bias"),
        *_f8_weights(shape, W_gate, W_up, W_down, W_shared_gate, W_shared_up, W_shared_down),
        _gate_vec(shape, W_shared_gate_vec), _score(score_fn), int(bool(norm_topk)), float(route_scale),
        _p(out, bf, (T, d), "out"), _p(topk_idx, torch.int32, (T, k), "topk_idx"),
        _p(topk_w, torch.float32, (T, k), "topk_w"),
        _p(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "moe_forward_fp8")


def moe_permute_fp8(shape, topk_idx, topk_w, workspace, stream=None):
    """The permute for the FP8 expert steps (their work lists differ from the bf16 ones)."""
    T, k = shape.T, shape.k
    st = load().moe_permute_fp8(ctypes.byref(shape), _p(topk_idx, torch.int32, (T, k), "topk_idx"),
                                _p(topk_w, torch.float32, (T, k), "topk_w"),
                                _p(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "moe_permute_fp8")


def moe_expert_gate_up_fp8(shape, x, W_gate, W_up, W_shared_gate, W_shared_up, workspace, stream=None):
    w = _f8_weights(shape, W_gate, W_up, None, W_shared_gate, W_shared_up, None)
    st = load().moe_expert_gate_up_fp8(ctypes.byref(shape), _p(x, torch.bfloat16, (shape.T, shape.d_model), "x"),
                                       w[0], w[1], w[3], w[4], _p(workspace, torch.uint8, None, "workspace"),
                                       workspace.numel(), _stream(stream))
    _check(st, "moe_expert_gate_up_fp8")


def moe_expert_down_fp8(shape, W_down, W_shared_down, workspace, stream=None):
    w = _f8_weights(shape, None, None, W_down, None, None, W_shared_down)
    st = load().moe_expert_down_fp8(ctypes.byref(shape), w[2], w[5], _p(workspace, torch.uint8, None, "workspace"),
                                    workspace.numel(), _stream(stream))
    _check(st, "moe_expert_down_fp8")


def moe_rmsnorm(shape, x, norm_gain, eps, x_norm, stream=None):
    """x_norm = bf16(x / sqrt(mean(x^2) + eps) * (1 + norm_gain)), computed in double."""
    T, d = shape.T, shape.d_model
    bf = torch.bfloat16
    st = load().moe_rmsnorm(ctypes.byref(shape), _p(x, bf, (T, d), "x"), _p(norm_gain, bf, (d,), "norm_gain"),
                            float(eps), _p(x_norm, bf, (T, d), "x_norm"), _stream(stream))
    _check(st, "moe_rmsnorm")


def moe_forward_host(shape, x_host, W_router, expert_bias, W_gate, W_up, W_down, W_shared_gate,
                     W_shared_up, W_shared_down, score_fn, norm_topk, route_scale, out_host,
                     topk_idx_host, topk_w_host, workspace, stream=None, W_shared_gate_vec=None):
    T, d, E, k = shape.T, shape.d_model, shape.E, shape.k
    bf = torch.bfloat16
    st = load().moe_forward_host(
        ctypes.byref(shape), _p(x_host, bf, (T, d), "x_host", host=True),
        _p(W_router, bf, (E, d), "W_router"), _p(expert_bias, torch.float32, (E,), "expert_bias"),
        *_weights(shape, W_gate, W_up, W_down, W_shared_gate, W_shared_up, W_shared_down),
        _gate_vec(shape, W_shared_gate_vec), _score(score_fn), int(bool(norm_topk)), float(route_scale),
        _p(out_host, bf, (T, d), "out_host", host=True),
        _p(topk_idx_host, torch.int32, (T, k), "topk_idx_host", host=True),
        _p(topk_w_host, torch.float32, (T, k), "topk_w_host", host=True),
        _p(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "moe_forward_host")


def moe_route(shape, x, W_router, expert_bias, score_fn, norm_topk, route_scale, topk_idx, topk_w,
              workspace, stream=None):
    T, d, E, k = shape.T, shape.d_model, shape.E, shape.k
    bf = torch.bfloat16
    st = load().moe_route(
        ctypes.byref(shape), _p(x, bf, (T, d), "x"), _p(W_router, bf, (E, d), "W_router"),
        _p(expert_bias, torch.float32, (E,), "expert_bias"), _score(score_fn), int(bool(norm_topk)),
        float(route_scale), _p(topk_idx, torch.int32, (T, k), "topk_idx"),
        _p(topk_w, torch.float32, (T, k), "topk_w"), _p(workspace, torch.uint8, None, "workspace"),
        workspace.numel(), _stream(stream))
    _check(st, "moe_route")


def moe_route_noalloc(shape, x, W_router, expert_bias, score_fn, norm_topk, route_scale, topk_idx, topk_w,
                      stream=None):
    """moe_route without a workspace, for callers that cannot allocate device
    memory (the library's built-in 16 MiB scratch holds the logits; T * E must
    not exceed 4,194,304).  Calls that overlap on the GPU race."""
    T, d, E, k = shape.T, shape.d_model, shape.E, shape.k
    bf = torch.bfloat16
    st = load().moe_route_noalloc(
        ctypes.byref(shape), _p(x, bf, (T, d), "x"), _p(W_router, bf, (E, d), "W_router"),
        _p(expert_bias, torch.float32, (E,), "expert_bias"), _score(score_fn), int(bool(norm_topk)),
        float(route_scale), _p(topk_idx, torch.int32, (T, k), "topk_idx"),
        _p(topk_w, torch.float32, (T, k), "topk_w"), _stream(stream))
    _check(st, "moe_route_noalloc")


def moe_permute(shape, topk_idx, topk_w, workspace, stream=None):
    T, k = shape.T, shape.k
    st = load().moe_permute(ctypes.byref(shape), _p(topk_idx, torch.int32, (T, k), "topk_idx"),
                            _p(topk_w, torch.float32, (T, k), "topk_w"),
                            _p(workspace, torch.uint8, None, "workspace"), workspace.numel(),
                            _stream(stream))
    _check(st, "moe_permute")


def moe_expert_gate_up(shape, x, W_gate, W_up, W_shared_gate, W_shared_up, workspace, stream=None):
    T, d, E, f, S, fs = shape.T, shape.d_model, shape.E, shape.d_ff, shape.n_shared, shape.d_ff_shared
    bf = torch.bfloat16
    st = load().moe_expert_gate_up(
        ctypes.byref(shape), _p(x, bf, (T, d), "x"), _p(W_gate, bf, (E, f, d), "W_gate"),
        _p(W_up, bf, (E, f, d), "W_up"),
        _p(W_shared_gate, bf, (S, fs, d), "W_shared_gate") if S else None,
        _p(W_shared_up, bf, (S, fs, d), "W_shared_up") if S else None,
        _p(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "moe_expert_gate_up")


def moe_expert_down(shape, W_down, W_shared_down, workspace, stream=None):
    d, E, f, S, fs = shape.d_model, shape.E, shape.d_ff, shape.n_shared, shape.d_ff_shared
    bf = torch.bfloat16
    st = load().moe_expert_down(
        ctypes.byref(shape), _p(W_down, bf, (E, d, f), "W_down"),
        _p(W_shared_down, bf, (S, d, fs), "W_shared_down") if S else None,
        _p(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "moe_expert_down")


def moe_combine(shape, out, workspace, stream=None, x=None, W_shared_gate_vec=None):
    T, d = shape.T, shape.d_model
    st = load().moe_combine(ctypes.byref(shape), _p(x, torch.bfloat16, (T, d), "x"),
                            _gate_vec(shape, W_shared_gate_vec), _p(out, torch.bfloat16, (T, d), "out"),
                            _p(workspace, torch.uint8, None, "workspace"), workspace.numel(),
                            _stream(stream))
    _check(st, "moe_combine")


def moe_experts_forward(shape, x, topk_idx, topk_w, W_gate, W_up, W_down, W_shared_gate, W_shared_up,
                        W_shared_down, out, workspace, stream=None, W_shared_gate_vec=None):
    """Steps a3..a7 on a caller-supplied routing (external-indices mode)."""
    T, d, k = shape.T, shape.d_model, shape.k
    bf = torch.bfloat16
    st = load().moe_experts_forward(
        ctypes.byref(shape), _p(x, bf, (T, d), "x"), _p(topk_idx, torch.int32, (T, k), "topk_idx"),
        _p(topk_w, torch.float32, (T, k), "topk_w"),
        *_weights(shape, W_gate, W_up, W_down, W_shared_gate, W_shared_up, W_shared_down),
        _gate_vec(shape, W_shared_gate_vec), _p(out, bf, (T, d), "out"),
        _p(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "moe_experts_forward")


def moe_device_status(workspace, stream=None) -> int:
    """Synchronises the stream and returns the workspace's device status code."""
    return int(load().moe_device_status(_p(workspace, torch.uint8, None, "workspace"), _stream(stream)))


def moe_debug_wait_timeout(workspace, timeout_ns, stream=None):
    st = load().moe_debug_wait_timeout(_p(workspace, torch.uint8, None, "workspace"), workspace.numel(),
                                       int(timeout_ns), _stream(stream))
    _check(st, "moe_debug_wait_timeout")


# ---- Token dispatch and MXFP4 experts ----
# A call is made by the native part of the binding where every argument is what
# it should be and no stream is given; else here, which says what is wrong.
# Sizes come from the tensors.  An MXFP4 tensor is a (codes uint8 [G, rows, K/2],
# scales uint8 [G, ceil(K/128), rows, 4]) pair; fp4_empty allocates one.  Scales
# kept row by row, [G, rows, K/32] with K a multiple of 128, become that by
# s.view(G, rows, K // 128, 4).transpose(1, 2).contiguous().

def alloc_dispatch_workspace(device=None):
    """The workspace of moe_sort_tokens and the MXFP4 products, its error word cleared."""
    return torch.zeros(DISPATCH_WORKSPACE_BYTES, dtype=torch.uint8, device=device or "cuda")


def fp4_empty(G, rows, K, device=None):
    """An uninitialised MXFP4 tensor of G x rows x K values."""
    u8 = dict(dtype=torch.uint8, device=device or "cuda")
    return torch.empty((G, rows, K // 2), **u8), torch.empty((G, (K + 127) // 128, rows, 4), **u8)


def _dims(t, n, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    s = t.shape
    if len(s) != n:
        raise ValueError(f"{name}: expected {n} dimensions, got shape {tuple(s)}")
    return s


def _dtype(t, name):
    dt = DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
    return dt


def _dev(t):
    """The device of a call whose first tensor is t: it has to be the current one, where the library launches."""
    dev = t.get_device()
    if dev >= 0 and dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _t(t, dtype, shape, name, dev):
    """Address of a contiguous tensor of this type and shape (None: any) on device `dev`."""
    if (type(t) is torch.Tensor and t.dtype is dtype and (shape is None or t.shape == shape) and t.is_contiguous()
            and not t.is_neg() and t.get_device() == dev >= 0):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    _p(t, dtype, shape, name)
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, other tensors on cuda:{dev}")
    return t.data_ptr()


def _on(stream, dev):
    """The stream's handle; None: the current stream of device `dev`, without a Stream object around it."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _fp4_dims(q, name):
    if not isinstance(q, (tuple, list)) or len(q) != 2:
        raise TypeError(f"{name}: expected a (codes, scales) pair")
    G, rows, half = _dims(q[0], 3, name)
    return G, rows, 2 * half


def _f4(q, G, rows, K, name, dev):
    """moe_fp4_tensor of a (codes, scales) pair of G x rows x K values on device `dev` (the call passes its address)."""
    _fp4_dims(q, name)
    c, s = q
    u8 = torch.uint8
    if (type(s) is torch.Tensor and c.dtype is u8 and s.dtype is u8 and c.shape == (G, rows, K // 2)
            and s.shape == (G, (K + 127) // 128, rows, 4) and c.is_contiguous() and s.is_contiguous()
            and not (c.is_neg() or s.is_neg()) and c.get_device() == s.get_device() == dev >= 0):
        return MoeFp4Tensor(c.data_ptr(), s.data_ptr())
    return MoeFp4Tensor(_t(c, u8, (G, rows, K // 2), name + ".codes", dev),
                        _t(s, u8, (G, (K + 127) // 128, rows, 4), name + ".scales", dev))


def moe_sort_tokens(topk_idx, offsets, slot_row, workspace, stream=None):
    """Rows of the (token, slot) pairs in expert order: offsets [E+1], slot_row [T, k] (-1: no expert)."""
    if stream is None and _done(_fast().sort_tokens(topk_idx, offsets, slot_row, workspace), "moe_sort_tokens"):
        return
    T, k = _dims(topk_idx, 2, "topk_idx")
    E = _dims(offsets, 1, "offsets")[0] - 1
    dev, i32 = _dev(topk_idx), torch.int32
    _check(load().moe_sort_tokens(T, k, E, _t(topk_idx, i32, None, "topk_idx", dev),
                                  _t(offsets, i32, None, "offsets", dev), _t(slot_row, i32, (T, k), "slot_row", dev),
                                  _t(workspace, torch.uint8, None, "workspace", dev), workspace.numel(),
                                  _on(stream, dev)), "moe_sort_tokens")


def moe_dispatch(x, slot_row, x_sorted, stream=None):
    """x_sorted[slot_row[t, j]] = x[t]."""
    if stream is None and _done(_fast().dispatch(x, slot_row, x_sorted), "moe_dispatch"):
        return
    (T, d), k = _dims(x, 2, "x"), _dims(slot_row, 2, "slot_row")[1]
    dev, dt = _dev(x), _dtype(x, "x")
    _check(load().moe_dispatch(T, k, d, dt, _t(x, x.dtype, None, "x", dev),
                               _t(slot_row, torch.int32, (T, k), "slot_row", dev),
                               _t(x_sorted, x.dtype, (T * k, d), "x_sorted", dev), _on(stream, dev)), "moe_dispatch")


def moe_dispatch_backward(dx_sorted, slot_row, dx, stream=None):
    """dx[t] = sum_j dx_sorted[slot_row[t, j]]."""
    if stream is None and _done(_fast().dispatch_backward(dx_sorted, slot_row, dx), "moe_dispatch_backward"):
        return
    (T, d), k = _dims(dx, 2, "dx"), _dims(slot_row, 2, "slot_row")[1]
    dev, dt = _dev(dx), _dtype(dx, "dx")
    _check(load().moe_dispatch_backward(T, k, d, dt, _t(dx_sorted, dx.dtype, (T * k, d), "dx_sorted", dev),
                                        _t(slot_row, torch.int32, (T, k), "slot_row", dev),
                                        _t(dx, dx.dtype, None, "dx", dev), _on(stream, dev)), "moe_dispatch_backward")


def moe_undispatch(y, slot_row, topk_w, out, stream=None):
    """out[t] = sum_j topk_w[t, j] y[slot_row[t, j]]."""
    if stream is None and _done(_fast().undispatch(y, slot_row, topk_w, out), "moe_undispatch"):
        return
    (T, d), k = _dims(out, 2, "out"), _dims(slot_row, 2, "slot_row")[1]
    dev, dt = _dev(out), _dtype(out, "out")
    _check(load().moe_undispatch(T, k, d, dt, _t(y, out.dtype, (T * k, d), "y", dev),
                                 _t(slot_row, torch.int32, (T, k), "slot_row", dev),
                                 _t(topk_w, torch.float32, (T, k), "topk_w", dev), _t(out, out.dtype, None, "out", dev),
                                 _on(stream, dev)), "moe_undispatch")


def moe_undispatch_backward(dout, y, slot_row, topk_w, dy, dw, stream=None):
    """dy[slot_row[t, j]] = topk_w[t, j] dout[t]; dw[t, j] = <dout[t], y[slot_row[t, j]]>."""
    if stream is None and _done(_fast().undispatch_backward(dout, y, slot_row, topk_w, dy, dw), "moe_undispatch_backward"):
        return
    (T, d), k = _dims(dout, 2, "dout"), _dims(slot_row, 2, "slot_row")[1]
    dev, dt, f32 = _dev(dout), _dtype(dout, "dout"), torch.float32
    _check(load().moe_undispatch_backward(T, k, d, dt, _t(dout, dout.dtype, None, "dout", dev),
                                          _t(y, dout.dtype, (T * k, d), "y", dev),
                                          _t(slot_row, torch.int32, (T, k), "slot_row", dev),
                                          _t(topk_w, f32, (T, k), "topk_w", dev),
                                          _t(dy, dout.dtype, (T * k, d), "dy", dev), _t(dw, f32, (T, k), "dw", dev),
                                          _on(stream, dev)), "moe_undispatch_backward")


def moe_quantize_fp4(x, codes, scales, stream=None):
    """x [G, rows, K] (bf16, fp16 or fp32) to MXFP4."""
    if stream is None and _done(_fast().quantize_fp4(x, codes, scales), "moe_quantize_fp4"):
        return
    G, rows, K = _dims(x, 3, "x")
    dev, dt = _dev(x), _dtype(x, "x")
    _check(load().moe_quantize_fp4(G, rows, K, dt, _t(x, x.dtype, None, "x", dev),
                                   _f4((codes, scales), G, rows, K, "q", dev), _on(stream, dev)), "moe_quantize_fp4")


def moe_dequantize_fp4(codes, scales, x, stream=None):
    """MXFP4 back to x [G, rows, K] (bf16, fp16 or fp32)."""
    if stream is None and _done(_fast().dequantize_fp4(codes, scales, x), "moe_dequantize_fp4"):
        return
    G, rows, K = _dims(x, 3, "x")
    dev, dt = _dev(x), _dtype(x, "x")
    _check(load().moe_dequantize_fp4(G, rows, K, dt, _f4((codes, scales), G, rows, K, "q", dev),
                                     _t(x, x.dtype, None, "x", dev), _on(stream, dev)), "moe_dequantize_fp4")


def moe_dispatch_fp4(x, slot_row, x_sorted, stream=None):
    """moe_dispatch of x's MXFP4 form: x_sorted is an MXFP4 tensor (G = 1) of T * k rows."""
    if stream is None and _done(_fast().dispatch_fp4(x, slot_row, x_sorted), "moe_dispatch_fp4"):
        return
    (T, d), k = _dims(x, 2, "x"), _dims(slot_row, 2, "slot_row")[1]
    dev, dt = _dev(x), _dtype(x, "x")
    q = _f4(x_sorted, 1, T * k, d, "x_sorted", dev)
    _check(load().moe_dispatch_fp4(T, k, d, dt, _t(x, x.dtype, None, "x", dev),
                                   _t(slot_row, torch.int32, (T, k), "slot_row", dev), q, _on(stream, dev)),
           "moe_dispatch_fp4")


def moe_matmul_fp4(a, offsets, W, out, workspace, stream=None):
    """out[r] = a[r] W[e]^T for the rows offsets[e] <= r < offsets[e+1] of every expert e."""
    if stream is None and _done(_fast().matmul_fp4(a, offsets, W, out, workspace), "moe_matmul_fp4"):
        return
    (_, rows, K), (E, N, _) = _fp4_dims(a, "a"), _fp4_dims(W, "W")
    _dims(out, 2, "out")
    dev, dt = _dev(out), _dtype(out, "out")
    _check(load().moe_matmul_fp4(rows, E, N, K, _f4(a, 1, rows, K, "a", dev),
                                 _t(offsets, torch.int32, (E + 1,), "offsets", dev), _f4(W, E, N, K, "W", dev), dt,
                                 _t(out, out.dtype, (rows, N), "out", dev),
                                 _t(workspace, torch.uint8, None, "workspace", dev), workspace.numel(),
                                 _on(stream, dev)), "moe_matmul_fp4")


def moe_swiglu_fp4(a, offsets, W_gate, W_up, h, workspace, stream=None):
    """h[r] = SiLU(a[r] W_gate[e]^T) * (a[r] W_up[e]^T), as MXFP4 (G = 1)."""
    if stream is None and _done(_fast().swiglu_fp4(a, offsets, W_gate, W_up, h, workspace), "moe_swiglu_fp4"):
        return
    (_, rows, K), (E, f, _) = _fp4_dims(a, "a"), _fp4_dims(W_gate, "W_gate")
    dev = _dev(a[0])
    _check(load().moe_swiglu_fp4(rows, E, f, K, _f4(a, 1, rows, K, "a", dev),
                                 _t(offsets, torch.int32, (E + 1,), "offsets", dev),
                                 _f4(W_gate, E, f, K, "W_gate", dev), _f4(W_up, E, f, K, "W_up", dev),
                                 _f4(h, 1, rows, f, "h", dev), _t(workspace, torch.uint8, None, "workspace", dev),
                                 workspace.numel(), _on(stream, dev)), "moe_swiglu_fp4")


def workspace_view(workspace, shape, region, dtype, dims):
    """A typed view of one workspace region (tests and debugging)."""
    off, nbytes = moe_workspace_region(shape, region)
    itemsize = torch.empty((), dtype=dtype).element_size()
    n = 1
    for x in dims:
        n *= int(x)
    assert n * itemsize <= nbytes, (region, dims, nbytes)
    return workspace[off:off + n * itemsize].view(dtype).view(*dims)


class MoELayer:
    """Convenience holder: weights + workspace for one shape; __call__ runs moe_forward."""

    def __init__(self, cfg, tensors, device="cuda"):
        self.cfg = cfg
        self.shape = shape_of(cfg)
        self.t = tensors
        self.workspace = alloc_workspace(self.shape, device)
        T, d, k = cfg.T, cfg.d, cfg.k
        self.out = torch.empty((T, d), dtype=torch.bfloat16, device=device)
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=device)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=device)
        if cfg.fp8 and cfg.prenorm:
            raise ValueError("MoELayer: the FP8 and pre-norm forms are separate entry points")

    def __call__(self, x=None, stream=None):
        t, c = self.t, self.cfg
        if c.fp8:
            moe_forward_fp8(self.shape, t["x"] if x is None else x, t["W_router"], t["expert_bias"],
                            t["W_gate_f8"], t["W_up_f8"], t["W_down_f8"], t["W_shared_gate_f8"],
                            t["W_shared_up_f8"], t["W_shared_down_f8"], c.score_fn, c.norm_topk, c.route_scale,
                            self.out, self.topk_idx, self.topk_w, self.workspace, stream,
                            W_shared_gate_vec=t.get("W_shared_gate_vec"))
            return self.out, self.topk_idx, self.topk_w
        if c.prenorm:
            moe_forward_prenorm(self.shape, t["x"] if x is None else x, t["norm_gain"], c.norm_eps, t["W_router"],
                                t["expert_bias"], t["W_gate"], t["W_up"], t["W_down"], t["W_shared_gate"],
                                t["W_shared_up"], t["W_shared_down"], c.score_fn, c.norm_topk, c.route_scale,
                                self.out, self.topk_idx, self.topk_w, self.workspace, stream,
                                W_shared_gate_vec=t.get("W_shared_gate_vec"))
            return self.out, self.topk_idx, self.topk_w
        moe_forward(self.shape, t["x"] if x is None else x, t["W_router"], t["expert_bias"],
                    t["W_gate"], t["W_up"], t["W_down"], t["W_shared_gate"], t["W_shared_up"],
                    t["W_shared_down"], c.score_fn, c.norm_topk, c.route_scale, self.out,
                    self.topk_idx, self.topk_w, self.workspace, stream,
                    W_shared_gate_vec=t.get("W_shared_gate_vec"))
        return self.out, self.topk_idx, self.topk_w

    def steps(self, stream=None, events=None):
        """The same pass as __call__, one step at a time; when `events` (6 CUDA
        events) is given, records them around the steps on `stream`."""
        t, c, s = self.t, self.cfg, self.shape
        st = stream
        rec = (lambda i: events[i].record(st)) if events is not None else (lambda i: None)
        rec(0)
        x = t["x"]
        if c.prenorm:
            x = workspace_view(self.workspace, s, "x_stage", torch.bfloat16, (c.T, c.d))
            moe_rmsnorm(s, t["x"], t["norm_gain"], c.norm_eps, x, st)
        moe_route(s, x, t["W_router"], t["expert_bias"], c.score_fn, c.norm_topk, c.route_scale,
                  self.topk_idx, self.topk_w, self.workspace, st)
        rec(1)
        (moe_permute_fp8 if c.fp8 else moe_permute)(s, self.topk_idx, self.topk_w, self.workspace, st)
        rec(2)
        if c.fp8:
            moe_expert_gate_up_fp8(s, x, t["W_gate_f8"], t["W_up_f8"], t["W_shared_gate_f8"],
                                   t["W_shared_up_f8"], self.workspace, st)
        else:
            moe_expert_gate_up(s, x, t["W_gate"], t["W_up"], t["W_shared_gate"], t["W_shared_up"],
                               self.workspace, st)
        rec(3)
        if c.fp8:
            moe_expert_down_fp8(s, t["W_down_f8"], t["W_shared_down_f8"], self.workspace, st)
        else:
            moe_expert_down(s, t["W_down"], t["W_shared_down"], self.workspace, st)
        rec(4)
        moe_combine(s, self.out, self.workspace, st, x=x, W_shared_gate_vec=t.get("W_shared_gate_vec"))
        rec(5)
        return self.out, self.topk_idx, self.topk_w
