"""ctypes binding of libzb (``include/zb.h``): same names, argument marshalling only.

Tensors are passed as ``torch.Tensor`` (their ``data_ptr()`` is handed to the
library) or as plain integer device addresses.  Every compute step runs in the
library's CUDA kernels; nothing here computes.  A missing library raises: there
is no fallback.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

c_void_p = ctypes.c_void_p
c_int32 = ctypes.c_int32
c_size_t = ctypes.c_size_t
c_int64 = ctypes.c_int64
c_float = ctypes.c_float
c_double = ctypes.c_double

ZB_OK = 0
STATUS_NAMES = {
    0: "ZB_OK", -1: "ZB_ERR_ARG", -2: "ZB_ERR_SHAPE", -3: "ZB_ERR_ORDER", -4: "ZB_ERR_STASH_FULL",
    -5: "ZB_ERR_NO_MB", -6: "ZB_ERR_CUDA", -7: "ZB_ERR_DEVICE_TIMEOUT", -8: "ZB_ERR_CAPACITY",
    -9: "ZB_ERR_DEVICE", -10: "ZB_ERR_WORKSPACE",
}
SCHED = {"1f1b": 0, "zbh1": 1, "gpipe": 2, "zb2p": 3}
LAYER_KINDS = {"linear": 0, "mlp": 1, "transformer": 2}


class ZBError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{where}: {self.name}")


class zb_op(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_uint8), ("pad", ctypes.c_uint8 * 3), ("mb", c_int32)]


class zb_stage_config(ctypes.Structure):
    _fields_ = [("kind", c_int32), ("n_layers", c_int32), ("hidden", c_int32), ("ffn", c_int32),
                ("n_heads", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32), ("eps", c_float),
                ("max_tokens", c_int32), ("max_inflight", c_int32), ("attention", c_int32), ("seq_len", c_int32)]


class zb_kernel_stats(ctypes.Structure):
    _fields_ = [("launches", c_int32), ("pad", c_int32), ("ms", ctypes.c_double), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double)]


class zb_rotary_config(ctypes.Structure):
    _fields_ = [("scaling", c_int32), ("rotary_dim", c_int32), ("base", c_double), ("factor", c_double),
                ("context", c_double), ("low", c_double), ("high", c_double)]


class zb_attention_options(ctypes.Structure):
    _fields_ = [("rotary_dim", c_int32), ("rotary_pairs", c_int32), ("turns", c_void_p), ("magnitude", c_float),
                ("cap", c_float), ("slopes", c_void_p)]


class zb_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", c_void_p), ("master", c_void_p), ("grad", c_void_p), ("m", c_void_p), ("v", c_void_p),
                ("m_scale", c_void_p), ("v_scale", c_void_p), ("count", c_int64), ("weight_decay", c_float),
                ("param_dtype", c_int32), ("grad_dtype", c_int32), ("reserved", c_int32)]


class zb_adamw_config(ctypes.Structure):
    _fields_ = [("lr", c_double), ("beta1", c_double), ("beta2", c_double), ("eps", c_double),
                ("state_bits", c_int32), ("stochastic", c_int32), ("seed", ctypes.c_uint32), ("reserved", c_int32)]


class zb_checkpoint(ctypes.Structure):
    _fields_ = [("codes", c_void_p), ("scales", c_void_p)]


class zb_residual_norm(ctypes.Structure):
    _fields_ = [("post_norm", c_int32), ("pre_norm", c_int32), ("gate_kind", c_int32), ("reserved", c_int32),
                ("post_gamma", c_void_p), ("post_beta", c_void_p), ("pre_gamma", c_void_p), ("pre_beta", c_void_p),
                ("gate", c_void_p), ("residual_scale", c_float), ("branch_scale", c_float), ("post_eps", c_float),
                ("pre_eps", c_float)]


ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "relu2": 5}
NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
GATE_KINDS = {"none": 0, "channel": 1, "token": 2}
ROTARY_PAIRS = {"half": 0, "interleaved": 1}
ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}
KERNEL_CLASSES = ["gemm_forward", "gemm_backward_input", "gemm_backward_weight", "row_backward_input",
                  "row_backward_weight", "row_forward", "attn_forward", "attn_backward", "stash_copy"]
ATTENTION_KINDS = {"standin": 0, "causal": 1, "document": 2}


class zb_layer_params(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("w_qkv", "dw_qkv", "w_o", "dw_o", "w_gu", "dw_gu", "w_down",
                                        "dw_down", "gamma1", "dgamma1", "gamma2", "dgamma2", "w", "dw")]


_SIGS = {
    "zb_status_string": (ctypes.c_char_p, [c_int32]),
    "zb_version": (c_int32, []),
    "zb_schedule": (c_int32, [c_int32, c_int32, c_int32, c_int32, ctypes.POINTER(zb_op), c_int32,
                              ctypes.POINTER(c_int32)]),
    "zb_schedule_bubble": (c_int32, [c_int32, c_int32, c_int32, ctypes.POINTER(c_int32),
                                     ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
    "zb_schedule_window_idle": (c_int32, [c_int32, c_int32, c_int32, ctypes.POINTER(ctypes.c_int64),
                                          ctypes.POINTER(ctypes.c_double)]),
    "zb_schedule_search": (c_int32, [c_int32] * 7 + [ctypes.POINTER(zb_op), c_int32, ctypes.POINTER(c_int32),
                                     ctypes.POINTER(c_int32), ctypes.POINTER(ctypes.c_int64)]),
    "zb_op_linear_forward": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32,
                                       c_void_p]),
    "zb_op_backward_input": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p]),
    "zb_op_backward_input_swiglu": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                              c_int32, c_void_p]),
    "zb_op_backward_input_rmsnorm": (c_int32, [c_void_p] * 8 + [c_int32, c_int32, c_int32, c_void_p]),
    "zb_op_backward_input_attention": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32,
                                                 c_int32, c_void_p]),
    "zb_op_backward_weight": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p]),
    "zb_op_backward_weight_group": (c_int32, [c_int32, ctypes.POINTER(c_void_p), ctypes.POINTER(c_void_p),
                                              ctypes.POINTER(c_void_p), c_int32, ctypes.POINTER(c_int32),
                                              ctypes.POINTER(c_int32), c_void_p]),
    "zb_op_rmsnorm_backward_gamma_scratch_bytes": (c_size_t, [c_int32, c_int32]),
    "zb_op_rmsnorm_backward_gamma": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                               c_void_p, c_size_t, c_void_p]),
    "zb_op_rmsnorm_backward_gamma_noalloc_max_floats": (c_size_t, []),
    "zb_op_rmsnorm_backward_gamma_noalloc": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                                       c_void_p]),
    "zb_op_rmsnorm_forward": (c_int32, [c_void_p, c_void_p, c_float, c_void_p, c_void_p, c_int32, c_int32,
                                        c_void_p]),
    "zb_op_swiglu_forward": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p]),
    "zb_op_attention_forward": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p]),
    "zb_op_attention_stat_stride": (c_int32, [c_int32]),
    "zb_op_attention_causal_forward": (c_int32, [c_void_p, c_void_p, c_void_p] + [c_int32] * 5 + [c_void_p]),
    "zb_op_attention_causal_backward": (c_int32, [c_void_p] * 6 + [c_int32] * 5 + [c_void_p]),
    "zb_op_attention_document_plan_bytes": (c_size_t, [c_int32]),
    "zb_op_attention_document_plan": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_size_t, c_void_p, c_void_p]),
    "zb_op_attention_document_scratch_bytes": (c_size_t, [c_int32, c_int32]),
    "zb_op_attention_document_forward": (c_int32, [c_void_p] * 5 + [c_float] + [c_int32] * 4 + [c_void_p]),
    "zb_op_attention_document_backward": (c_int32, [c_void_p] * 7 + [c_float] + [c_int32] * 4
                                          + [c_void_p, c_size_t, c_void_p]),
    "zb_rotary_frequencies": (c_int32, [ctypes.POINTER(zb_rotary_config), ctypes.POINTER(ctypes.c_uint64),
                                        ctypes.POINTER(c_float)]),
    "zb_op_rotary_forward": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_float] + [c_int32] * 5
                             + [c_void_p]),
    "zb_op_rotary_backward": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_float] + [c_int32] * 5
                              + [c_void_p]),
    "zb_op_checkpoint_pack": (c_int32, [c_void_p, ctypes.POINTER(zb_checkpoint), c_int32, c_int32, c_void_p]),
    "zb_op_checkpoint_unpack": (c_int32, [ctypes.POINTER(zb_checkpoint), c_void_p, c_int32, c_int32, c_void_p]),
    "zb_op_linear_activation_forward": (c_int32, [c_void_p] * 6 + [ctypes.POINTER(zb_checkpoint)] * 2 + [c_int32] * 4
                                        + [c_void_p]),
    "zb_op_backward_input_activation_scratch_bytes": (c_size_t, [c_int32, c_int32]),
    "zb_op_backward_input_activation": (c_int32, [c_void_p] * 3 + [ctypes.POINTER(zb_checkpoint), c_void_p, c_void_p]
                                        + [c_int32] * 4 + [c_void_p, c_size_t, c_void_p]),
    "zb_op_activation_backward": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(zb_checkpoint), c_void_p] + [c_int32] * 3
                                  + [c_void_p]),
    "zb_op_backward_bias_scratch_bytes": (c_size_t, [c_int32, c_int32]),
    "zb_op_backward_bias": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_size_t, c_void_p]),
    "zb_op_backward_weight_checkpoint_scratch_bytes": (c_size_t, [c_int32, c_int32]),
    "zb_op_backward_weight_checkpoint": (c_int32, [c_void_p, ctypes.POINTER(zb_checkpoint), c_void_p] + [c_int32] * 3
                                         + [c_void_p, c_size_t, c_void_p]),
    "zb_op_residual_norm_forward": (c_int32, [ctypes.POINTER(zb_residual_norm)] + [c_void_p] * 4
                                    + [ctypes.POINTER(zb_checkpoint), c_void_p, c_int32, c_int32, c_void_p]),
    "zb_op_residual_norm_backward_input": (c_int32, [ctypes.POINTER(zb_residual_norm)] + [c_void_p] * 9
                                           + [c_int32, c_int32, c_void_p]),
    "zb_op_residual_norm_backward_weight_scratch_bytes": (c_size_t, [c_int32, c_int32]),
    "zb_op_residual_norm_backward_weight": (c_int32, [ctypes.POINTER(zb_residual_norm)] + [c_void_p] * 10
                                            + [c_int32, c_int32, c_void_p, c_size_t, c_void_p]),
    "zb_op_adamw_step": (c_int32, [ctypes.POINTER(zb_adamw_tensor), c_int32, ctypes.POINTER(zb_adamw_config), c_int64,
                                   c_void_p, c_void_p, c_void_p, c_void_p]),
    "zb_op_adamw_unpack": (c_int32, [ctypes.POINTER(zb_adamw_tensor), c_int32, ctypes.POINTER(c_void_p),
                                     ctypes.POINTER(c_void_p), c_void_p]),
    "zb_op_grad_norm_scratch_bytes": (c_size_t, [ctypes.POINTER(zb_adamw_tensor), c_int32]),
    "zb_op_grad_norm": (c_int32, [ctypes.POINTER(zb_adamw_tensor), c_int32, c_float, c_void_p, c_void_p, c_size_t,
                                  c_void_p]),
    "zb_device_status": (c_int32, [c_void_p, c_int32, ctypes.POINTER(c_int32)]),
    "zb_selftest_wait_timeout": (c_int32, [c_int32, c_void_p]),
    "zb_stage_workspace_bytes": (c_size_t, [ctypes.POINTER(zb_stage_config)]),
    "zb_stage_create": (c_int32, [ctypes.POINTER(zb_stage_config), ctypes.POINTER(zb_layer_params), c_void_p,
                                  c_size_t, ctypes.POINTER(c_void_p)]),
    "zb_stage_destroy": (c_int32, [c_void_p]),
    "zb_stage_forward": (c_int32, [c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p]),
    "zb_stage_forward_documents": (c_int32, [c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_void_p,
                                             c_void_p]),
    "zb_stage_set_attention": (c_int32, [c_void_p, ctypes.POINTER(zb_attention_options)]),
    "zb_backward_input": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p]),
    "zb_backward_weight": (c_int32, [c_void_p, c_int32, c_void_p]),
    "zb_wgrad_flush": (c_int32, [c_void_p, c_void_p]),
    "zb_stage_sync": (c_int32, [c_void_p, c_void_p]),
    "zb_stage_stats": (c_int32, [c_void_p, ctypes.POINTER(c_int32), ctypes.POINTER(c_int32),
                                 ctypes.POINTER(c_size_t)]),
    "zb_stage_stash_view": (c_int32, [c_void_p, c_int32, c_int32, c_int32, ctypes.POINTER(c_void_p),
                                      ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                                      ctypes.POINTER(c_int32)]),
    "zb_stage_set_tracing": (c_int32, [c_void_p, c_int32]),
    "zb_stage_read_tracing": (c_int32, [c_void_p, ctypes.POINTER(zb_kernel_stats), c_int32]),
}

_LIB = None


def lib():
    """The loaded libzb (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"{_build.LIB} is missing: build it with __graft_entry__.build()")
        handle = ctypes.CDLL(_build.LIB)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def declared_symbols():
    return list(_SIGS)


def _current_stream():
    """The address of torch's current stream on the current device.  torch.cuda.current_stream() builds an object for
    it, 3 us a call, a third of a small operator's whole call; torch's own generated code reads the address directly."""
    global _current_stream
    import torch

    torch.cuda.current_stream()  # initialises CUDA, or says why it cannot be
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    else:
        _current_stream = lambda: raw(_current_device())  # noqa: E731
    return _current_stream()


def _current_device():
    """The number of torch's current device, without the second look at CUDA's state that torch.cuda.current_device()
    takes."""
    global _current_device
    import torch

    torch.cuda.current_device()  # initialises CUDA, or says why it cannot be
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _current_device()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s):
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status, where):
    if status != ZB_OK:
        raise ZBError(status, where)


# ---------------------------------------------------------------- misc / schedule


def zb_status_string(status):
    return lib().zb_status_string(status).decode()


def zb_version():
    return lib().zb_version()


def zb_schedule(kind, stage, p, m):
    """F/B/W order of one stage: list of ("F" | "B" | "W", mb)."""
    n = c_int32(0)
    buf = (zb_op * (3 * m))()
    _check(lib().zb_schedule(SCHED[kind], stage, p, m, buf, 3 * m, ctypes.byref(n)), "zb_schedule")
    return [(chr(buf[i].kind), buf[i].mb) for i in range(n.value)]


def zb_schedule_raw(kind, stage, p, m, cap):
    """Low-level form: (status, n_out, ops) without raising."""
    n = c_int32(-1)
    buf = (zb_op * max(cap, 1))()
    st = lib().zb_schedule(kind, stage, p, m, buf if cap > 0 else None, cap, ctypes.byref(n))
    return st, n.value, [(chr(buf[i].kind), buf[i].mb) for i in range(min(max(n.value, 0), cap))]


def zb_schedule_search(stage, p, m, mem_limit, t_f, t_b, t_w):
    """(order of `stage`, chosen ceiling, makespan) of the memory-limited search."""
    arr = (zb_op * (3 * m))()
    n = c_int32(0)
    limit = c_int32(0)
    span = ctypes.c_int64(0)
    _check(lib().zb_schedule_search(stage, p, m, mem_limit, t_f, t_b, t_w, arr, 3 * m, ctypes.byref(n),
                                    ctypes.byref(limit), ctypes.byref(span)), "zb_schedule_search")
    return [(chr(arr[i].kind), arr[i].mb) for i in range(n.value)], limit.value, span.value


def zb_schedule_bubble(kind, p, m):
    """(makespan, idle / compute, idle / wall) of the unit-time pipeline model."""
    span = c_int32(0)
    a = ctypes.c_double(0)
    b = ctypes.c_double(0)
    _check(lib().zb_schedule_bubble(SCHED[kind], p, m, ctypes.byref(span), ctypes.byref(a), ctypes.byref(b)),
           "zb_schedule_bubble")
    return span.value, a.value, b.value


def zb_schedule_window_idle(kind, p, m):
    """(idle units, idle / compute) inside each stage's own window, summed over stages."""
    n = ctypes.c_int64(0)
    f = ctypes.c_double(0)
    _check(lib().zb_schedule_window_idle(SCHED[kind], p, m, ctypes.byref(n), ctypes.byref(f)),
           "zb_schedule_window_idle")
    return n.value, f.value


# ---------------------------------------------------------------- per-step ops


def zb_op_linear_forward(x, w, residual, y, tokens, in_features, out_features, stream=None):
    _check(lib().zb_op_linear_forward(_ptr(x), _ptr(w), _ptr(residual), _ptr(y), tokens, in_features,
                                      out_features, _stream(stream)), "zb_op_linear_forward")


def zb_op_backward_input(dy, w, dx, tokens, in_features, out_features, stream=None):
    _check(lib().zb_op_backward_input(_ptr(dy), _ptr(w), _ptr(dx), tokens, in_features, out_features,
                                      _stream(stream)), "zb_op_backward_input")


def zb_op_backward_input_swiglu(dy, w_down, gu, dgu, tokens, hidden, ffn, stream=None):
    _check(lib().zb_op_backward_input_swiglu(_ptr(dy), _ptr(w_down), _ptr(gu), _ptr(dgu), tokens, hidden, ffn,
                                             _stream(stream)), "zb_op_backward_input_swiglu")


def zb_op_backward_input_rmsnorm(dy, w, x, rstd, gamma, dres, dn, dx, tokens, hidden, out_features, stream=None):
    _check(lib().zb_op_backward_input_rmsnorm(_ptr(dy), _ptr(w), _ptr(x), _ptr(rstd), _ptr(gamma), _ptr(dres),
                                              _ptr(dn), _ptr(dx), tokens, hidden, out_features, _stream(stream)),
           "zb_op_backward_input_rmsnorm")


def zb_op_backward_input_attention(dh, w_o, dqkv, tokens, n_heads, n_kv_heads, head_dim, stream=None):
    _check(lib().zb_op_backward_input_attention(_ptr(dh), _ptr(w_o), _ptr(dqkv), tokens, n_heads, n_kv_heads,
                                                head_dim, _stream(stream)), "zb_op_backward_input_attention")


def zb_op_backward_weight(dy, x, dw, tokens, in_features, out_features, stream=None):
    _check(lib().zb_op_backward_weight(_ptr(dy), _ptr(x), _ptr(dw), tokens, in_features, out_features,
                                       _stream(stream)), "zb_op_backward_weight")


def zb_op_backward_weight_group(dys, xs, dws, tokens, in_features, out_features, stream=None):
    n = len(dys)
    ptrs = lambda ts: (c_void_p * n)(*[_ptr(t) for t in ts])  # noqa: E731
    ints = lambda vs: (c_int32 * n)(*vs)  # noqa: E731
    _check(lib().zb_op_backward_weight_group(n, ptrs(dys), ptrs(xs), ptrs(dws), tokens, ints(in_features),
                                             ints(out_features), _stream(stream)), "zb_op_backward_weight_group")


def zb_op_rmsnorm_backward_gamma_scratch_bytes(tokens, hidden):
    return lib().zb_op_rmsnorm_backward_gamma_scratch_bytes(tokens, hidden)


def zb_op_rmsnorm_backward_gamma(dn, x, rstd, dgamma, tokens, hidden, scratch, scratch_bytes, stream=None):
    _check(lib().zb_op_rmsnorm_backward_gamma(_ptr(dn), _ptr(x), _ptr(rstd), _ptr(dgamma), tokens, hidden,
                                              _ptr(scratch), scratch_bytes, _stream(stream)),
           "zb_op_rmsnorm_backward_gamma")


def zb_op_rmsnorm_backward_gamma_noalloc_max_floats():
    return lib().zb_op_rmsnorm_backward_gamma_noalloc_max_floats()


def zb_op_rmsnorm_backward_gamma_noalloc(dn, x, rstd, dgamma, tokens, hidden, stream=None):
    """Gamma-gradient reduction without caller scratch (see include/zb.h for its limits)."""
    _check(lib().zb_op_rmsnorm_backward_gamma_noalloc(_ptr(dn), _ptr(x), _ptr(rstd), _ptr(dgamma), tokens, hidden,
                                                      _stream(stream)), "zb_op_rmsnorm_backward_gamma_noalloc")


def zb_op_rmsnorm_forward(x, gamma, eps, n, rstd, tokens, hidden, stream=None):
    _check(lib().zb_op_rmsnorm_forward(_ptr(x), _ptr(gamma), eps, _ptr(n), _ptr(rstd), tokens, hidden,
                                       _stream(stream)), "zb_op_rmsnorm_forward")


def zb_op_swiglu_forward(gu, s, tokens, ffn, stream=None):
    _check(lib().zb_op_swiglu_forward(_ptr(gu), _ptr(s), tokens, ffn, _stream(stream)), "zb_op_swiglu_forward")


def zb_op_attention_forward(qkv, a, tokens, n_heads, n_kv_heads, head_dim, stream=None):
    _check(lib().zb_op_attention_forward(_ptr(qkv), _ptr(a), tokens, n_heads, n_kv_heads, head_dim,
                                         _stream(stream)), "zb_op_attention_forward")


def zb_op_attention_stat_stride(tokens):
    return lib().zb_op_attention_stat_stride(tokens)


def zb_op_attention_causal_forward(qkv, a, lse, tokens, n_heads, n_kv_heads, head_dim, seq_len=0, stream=None):
    _check(lib().zb_op_attention_causal_forward(_ptr(qkv), _ptr(a), _ptr(lse), tokens, n_heads, n_kv_heads,
                                                head_dim, seq_len, _stream(stream)),
           "zb_op_attention_causal_forward")


def zb_op_attention_causal_backward(qkv, a, da, lse, dvec, dqkv, tokens, n_heads, n_kv_heads, head_dim,
                                    seq_len=0, stream=None):
    _check(lib().zb_op_attention_causal_backward(_ptr(qkv), _ptr(a), _ptr(da), _ptr(lse), _ptr(dvec), _ptr(dqkv),
                                                 tokens, n_heads, n_kv_heads, head_dim, seq_len, _stream(stream)),
           "zb_op_attention_causal_backward")


# ---------------------------------------------------------------- attention inside packed documents


def zb_op_attention_document_plan_bytes(tokens):
    return lib().zb_op_attention_document_plan_bytes(tokens)


def zb_op_attention_document_plan(doc_offsets, prefix_len, n_docs, tokens, plan, plan_bytes, positions=None, stream=None):
    _check(lib().zb_op_attention_document_plan(_ptr(doc_offsets), _ptr(prefix_len), n_docs, tokens, _ptr(plan), plan_bytes,
                                               _ptr(positions), _stream(stream)), "zb_op_attention_document_plan")


def zb_op_attention_document_scratch_bytes(tokens, n_heads):
    return lib().zb_op_attention_document_scratch_bytes(tokens, n_heads)


def zb_op_attention_document_forward(qkv, a, lse, plan, slopes, cap, tokens, n_heads, n_kv_heads, head_dim, stream=None):
    _check(lib().zb_op_attention_document_forward(_ptr(qkv), _ptr(a), _ptr(lse), _ptr(plan), _ptr(slopes), cap, tokens,
                                                  n_heads, n_kv_heads, head_dim, _stream(stream)),
           "zb_op_attention_document_forward")


def zb_op_attention_document_backward(qkv, a, da, lse, dqkv, plan, slopes, cap, tokens, n_heads, n_kv_heads, head_dim,
                                      scratch, scratch_bytes, stream=None):
    _check(lib().zb_op_attention_document_backward(_ptr(qkv), _ptr(a), _ptr(da), _ptr(lse), _ptr(dqkv), _ptr(plan),
                                                   _ptr(slopes), cap, tokens, n_heads, n_kv_heads, head_dim, _ptr(scratch),
                                                   scratch_bytes, _stream(stream)), "zb_op_attention_document_backward")


# ---------------------------------------------------------------- rotary positions


def zb_rotary_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0, high=None):
    """(turns, magnitude): the list of 64-bit fractions of a turn per position, and the factor on rotated values.
    `high` defaults to 32 turns (yarn) or 4 (banded)."""
    if high is None:
        high = 4.0 if scaling == "banded" else 32.0
    cfg = zb_rotary_config(ROTARY_SCALINGS[scaling], rotary_dim, base, factor, context, low, high)
    turns = (ctypes.c_uint64 * max(1, rotary_dim // 2))()
    mag = c_float(0)
    _check(lib().zb_rotary_frequencies(ctypes.byref(cfg), turns, ctypes.byref(mag)), "zb_rotary_frequencies")
    return list(turns), mag.value


def zb_op_rotary_forward(x, y, positions, turns, magnitude, tokens, n_heads, head_dim, rotary_dim, pairs="half", ld_x=None,
                         ld_y=None, stream=None):
    """Strides default to dense rows of n_heads heads."""
    dense = n_heads * head_dim
    _check(lib().zb_op_rotary_forward(_ptr(x), dense if ld_x is None else ld_x, _ptr(y), dense if ld_y is None else ld_y,
                                      _ptr(positions), _ptr(turns), magnitude, tokens, n_heads, head_dim, rotary_dim,
                                      ROTARY_PAIRS[pairs], _stream(stream)), "zb_op_rotary_forward")


def zb_op_rotary_backward(dy, dx, positions, turns, magnitude, tokens, n_heads, head_dim, rotary_dim, pairs="half",
                          ld_x=None, ld_y=None, stream=None):
    """`ld_x` is the stride of dy, the input, and `ld_y` that of dx."""
    dense = n_heads * head_dim
    _check(lib().zb_op_rotary_backward(_ptr(dy), dense if ld_x is None else ld_x, _ptr(dx), dense if ld_y is None else ld_y,
                                       _ptr(positions), _ptr(turns), magnitude, tokens, n_heads, head_dim, rotary_dim,
                                       ROTARY_PAIRS[pairs], _stream(stream)), "zb_op_rotary_backward")


# ---------------------------------------------------------------- biased linears, 8-bit checkpoints


def _packed(p):
    """A checkpoint given as (codes, scales), or None."""
    if p is None:
        return None
    return ctypes.byref(zb_checkpoint(_ptr(p[0]), _ptr(p[1])))


def _size(scratch, scratch_bytes):
    """Bytes of a scratch tensor whose size is not given."""
    if scratch_bytes is not None:
        return scratch_bytes
    return 0 if scratch is None else scratch.numel() * scratch.element_size()


def zb_op_checkpoint_pack(x, packed, tokens, width, stream=None):
    """`packed`: the tuple (codes [tokens, width], scales [tokens, width / 32]) of uint8 tensors, here and below."""
    _check(lib().zb_op_checkpoint_pack(_ptr(x), _packed(packed), tokens, width, _stream(stream)), "zb_op_checkpoint_pack")


def zb_op_checkpoint_unpack(packed, x, tokens, width, stream=None):
    _check(lib().zb_op_checkpoint_unpack(_packed(packed), _ptr(x), tokens, width, _stream(stream)), "zb_op_checkpoint_unpack")


def zb_op_linear_activation_forward(x, w, bias, residual, y, tokens, in_features, out_features, activation="none", z=None,
                                    z_packed=None, y_packed=None, stream=None):
    _check(lib().zb_op_linear_activation_forward(_ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(y), _ptr(z),
                                                 _packed(z_packed), _packed(y_packed), tokens, in_features, out_features,
                                                 ACTIVATIONS[activation], _stream(stream)), "zb_op_linear_activation_forward")


def zb_op_backward_input_activation_scratch_bytes(tokens, in_features):
    return lib().zb_op_backward_input_activation_scratch_bytes(tokens, in_features)


def zb_op_backward_input_activation(dy, w, z, dz, tokens, in_features, out_features, activation, z_packed=None, dbias=None,
                                    scratch=None, scratch_bytes=None, stream=None):
    """scratch is read with dbias only; its size defaults to the tensor's.  With relu, z may be the layer's bf16 output
    (without a residual); z_packed loses the gradient of positive values below half a unit."""
    _check(lib().zb_op_backward_input_activation(_ptr(dy), _ptr(w), _ptr(z), _packed(z_packed), _ptr(dz), _ptr(dbias), tokens,
                                                 in_features, out_features, ACTIVATIONS[activation], _ptr(scratch),
                                                 _size(scratch, scratch_bytes), _stream(stream)),
           "zb_op_backward_input_activation")


def zb_op_activation_backward(dy, z, dz, tokens, width, activation, z_packed=None, stream=None):
    _check(lib().zb_op_activation_backward(_ptr(dy), _ptr(z), _packed(z_packed), _ptr(dz), tokens, width,
                                           ACTIVATIONS[activation], _stream(stream)), "zb_op_activation_backward")


def zb_op_backward_bias_scratch_bytes(tokens, out_features):
    return lib().zb_op_backward_bias_scratch_bytes(tokens, out_features)


def zb_op_backward_bias(dy, dbias, tokens, out_features, scratch, scratch_bytes=None, stream=None):
    _check(lib().zb_op_backward_bias(_ptr(dy), _ptr(dbias), tokens, out_features, _ptr(scratch), _size(scratch, scratch_bytes),
                                     _stream(stream)), "zb_op_backward_bias")


def zb_op_backward_weight_checkpoint_scratch_bytes(tokens, in_features):
    return lib().zb_op_backward_weight_checkpoint_scratch_bytes(tokens, in_features)


def zb_op_backward_weight_checkpoint(dy, x_packed, dw, tokens, in_features, out_features, scratch, scratch_bytes=None,
                                     stream=None):
    _check(lib().zb_op_backward_weight_checkpoint(_ptr(dy), _packed(x_packed), _ptr(dw), tokens, in_features, out_features,
                                                  _ptr(scratch), _size(scratch, scratch_bytes), _stream(stream)),
           "zb_op_backward_weight_checkpoint")


# ---------------------------------------------------------------- norms around a block


def make_residual_norm(post="none", pre="none", gate_kind="none", gate=None, post_gamma=None, post_beta=None, pre_gamma=None,
                       pre_beta=None, residual_scale=1.0, branch_scale=1.0, post_eps=1e-5, pre_eps=1e-5):
    """The options and parameters of the residual_norm calls.  It keeps the tensors alive."""
    op = zb_residual_norm(NORM_KINDS[post], NORM_KINDS[pre], GATE_KINDS[gate_kind], 0, _ptr(post_gamma), _ptr(post_beta),
                          _ptr(pre_gamma), _ptr(pre_beta), _ptr(gate), residual_scale, branch_scale, post_eps, pre_eps)
    op.tensors = (post_gamma, post_beta, pre_gamma, pre_beta, gate)
    return op


def zb_op_residual_norm_forward(op, x, y, h, n, stats, tokens, hidden, n_packed=None, stream=None):
    _check(lib().zb_op_residual_norm_forward(ctypes.byref(op), _ptr(x), _ptr(y), _ptr(h), _ptr(n), _packed(n_packed),
                                             _ptr(stats), tokens, hidden, _stream(stream)), "zb_op_residual_norm_forward")


def zb_op_residual_norm_backward_input(op, dn, dres, h, y, stats, dh, dy, tokens, hidden, dx=None, dgate=None, stream=None):
    _check(lib().zb_op_residual_norm_backward_input(ctypes.byref(op), _ptr(dn), _ptr(dres), _ptr(h), _ptr(y), _ptr(stats),
                                                    _ptr(dh), _ptr(dx), _ptr(dy), _ptr(dgate), tokens, hidden,
                                                    _stream(stream)), "zb_op_residual_norm_backward_input")


def zb_op_residual_norm_backward_weight_scratch_bytes(tokens, hidden):
    return lib().zb_op_residual_norm_backward_weight_scratch_bytes(tokens, hidden)


def zb_op_residual_norm_backward_weight(op, dn, h, dh, y, stats, tokens, hidden, scratch, scratch_bytes=None,
                                        dpost_gamma=None, dpost_beta=None, dpre_gamma=None, dpre_beta=None, dgate=None,
                                        stream=None):
    _check(lib().zb_op_residual_norm_backward_weight(ctypes.byref(op), _ptr(dn), _ptr(h), _ptr(dh), _ptr(y), _ptr(stats),
                                                     _ptr(dpost_gamma), _ptr(dpost_beta), _ptr(dpre_gamma), _ptr(dpre_beta),
                                                     _ptr(dgate), tokens, hidden, _ptr(scratch), _size(scratch, scratch_bytes),
                                                     _stream(stream)), "zb_op_residual_norm_backward_weight")


# ---------------------------------------------------------------- AdamW


def adamw_table(tensors):
    """The C array of a list of dicts: param, grad, m, v, and where they apply master, m_scale, v_scale, weight_decay
    (tensors of one device, whose dtypes and sizes it takes).  The table holds addresses: keep the tensors alive."""
    import torch

    codes = {torch.bfloat16: 0, torch.float32: 1}
    arr = (zb_adamw_tensor * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        param, grad = t["param"], t["grad"]
        if param.dtype not in codes or grad.dtype not in codes:
            raise ZBError(-1, "adamw_table (param and grad are bf16 or float32)")
        n = param.numel()
        sizes = {"master": (torch.float32, n), "grad": (grad.dtype, n)}
        if t["m"].dtype == torch.uint8:
            blocks = (n + 255) // 256
            sizes.update(m=(torch.uint8, n), v=(torch.uint8, n), m_scale=(torch.float32, blocks),
                         v_scale=(torch.float32, blocks))
        else:
            sizes.update(m=(torch.float32, n), v=(torch.float32, n))
        for name, (dtype, count) in sizes.items():
            x = t.get(name)
            if x is None and name == "master":
                continue
            if x is None or x.dtype != dtype or x.numel() != count or not x.is_contiguous() or x.device != param.device:
                raise ZBError(-1, f"adamw_table ({name}: {count} contiguous values of {dtype} on param's device)")
        if not param.is_contiguous() or param.device != tensors[0]["param"].device:
            raise ZBError(-1, "adamw_table (param must be contiguous, and on the first one's device)")
        arr[i] = zb_adamw_tensor(_ptr(param), _ptr(t.get("master")), _ptr(grad), _ptr(t["m"]), _ptr(t["v"]),
                                 _ptr(t.get("m_scale")), _ptr(t.get("v_scale")), n, t.get("weight_decay", 0.0),
                                 codes[param.dtype], codes[grad.dtype], 0)
    return arr


def make_adamw_config(lr, beta1=0.9, beta2=0.95, eps=1e-8, state_bits=32, stochastic=False, seed=0):
    return zb_adamw_config(lr, beta1, beta2, eps, state_bits, 1 if stochastic else 0, seed & 0xFFFFFFFF, 0)


def zb_op_adamw_step(table, n, cfg, step, grad_scale=None, lr_device=None, step_device=None, stream=None):
    _check(lib().zb_op_adamw_step(table, n, ctypes.byref(cfg), step, _ptr(grad_scale), _ptr(lr_device), _ptr(step_device),
                                  _stream(stream)), "zb_op_adamw_step")


def zb_op_adamw_unpack(table, n, ms, vs, stream=None):
    ptrs = lambda ts: (c_void_p * max(1, n))(*[_ptr(t) for t in ts])  # noqa: E731
    _check(lib().zb_op_adamw_unpack(table, n, ptrs(ms), ptrs(vs), _stream(stream)), "zb_op_adamw_unpack")


def zb_op_grad_norm_scratch_bytes(table, n):
    return lib().zb_op_grad_norm_scratch_bytes(table, n)


def zb_op_grad_norm(table, n, max_norm, out, scratch, scratch_bytes, stream=None):
    _check(lib().zb_op_grad_norm(table, n, max_norm, _ptr(out), _ptr(scratch), scratch_bytes, _stream(stream)),
           "zb_op_grad_norm")


def zb_device_status(stream=None, reset=False):
    """(status, code): status is ZB_OK or ZB_ERR_DEVICE_TIMEOUT; never raises on a timeout."""
    code = c_int32(0)
    st = lib().zb_device_status(_stream(stream), 1 if reset else 0, ctypes.byref(code))
    if st not in (ZB_OK, -7):
        raise ZBError(st, "zb_device_status")
    return st, code.value


def zb_selftest_wait_timeout(limit_us, stream=None):
    _check(lib().zb_selftest_wait_timeout(limit_us, _stream(stream)), "zb_selftest_wait_timeout")


# ---------------------------------------------------------------- stage


def make_config(kind, n_layers, hidden, ffn, n_heads=0, n_kv_heads=0, head_dim=0, eps=1e-5, max_tokens=128,
                max_inflight=1, attention="standin", seq_len=0):
    return zb_stage_config(LAYER_KINDS[kind], n_layers, hidden, ffn, n_heads, n_kv_heads, head_dim, eps,
                           max_tokens, max_inflight, ATTENTION_KINDS[attention], seq_len)


def zb_stage_workspace_bytes(cfg):
    return lib().zb_stage_workspace_bytes(ctypes.byref(cfg))


def zb_stage_create(cfg, layers, workspace, workspace_bytes):
    """layers: list of dicts name -> tensor / int pointer (names of zb_layer_params)."""
    arr = (zb_layer_params * len(layers))()
    for i, d in enumerate(layers):
        for k, v in d.items():
            setattr(arr[i], k, _ptr(v))
    handle = c_void_p(0)
    _check(lib().zb_stage_create(ctypes.byref(cfg), arr, _ptr(workspace), workspace_bytes, ctypes.byref(handle)),
           "zb_stage_create")
    return handle.value


def zb_stage_destroy(st):
    _check(lib().zb_stage_destroy(st), "zb_stage_destroy")


def zb_stage_forward(st, mb, x, tokens, y, stream=None):
    _check(lib().zb_stage_forward(st, mb, _ptr(x), tokens, _ptr(y), _stream(stream)), "zb_stage_forward")


def zb_stage_forward_documents(st, mb, x, tokens, doc_offsets, prefix_len, n_docs, y, stream=None):
    _check(lib().zb_stage_forward_documents(st, mb, _ptr(x), tokens, _ptr(doc_offsets), _ptr(prefix_len), n_docs, _ptr(y),
                                            _stream(stream)), "zb_stage_forward_documents")


def zb_stage_set_attention(st, rotary_dim=0, pairs="half", turns=None, magnitude=1.0, cap=0.0, slopes=None):
    opt = zb_attention_options(rotary_dim, ROTARY_PAIRS[pairs], _ptr(turns), magnitude, cap, _ptr(slopes))
    _check(lib().zb_stage_set_attention(st, ctypes.byref(opt)), "zb_stage_set_attention")


def zb_backward_input(st, mb, dy, dx, stream=None):
    _check(lib().zb_backward_input(st, mb, _ptr(dy), _ptr(dx), _stream(stream)), "zb_backward_input")


def zb_backward_weight(st, mb, stream=None):
    _check(lib().zb_backward_weight(st, mb, _stream(stream)), "zb_backward_weight")


def zb_wgrad_flush(st, stream=None):
    _check(lib().zb_wgrad_flush(st, _stream(stream)), "zb_wgrad_flush")


def zb_stage_sync(st, stream=None):
    _check(lib().zb_stage_sync(st, _stream(stream)), "zb_stage_sync")


def zb_stage_stats(st):
    a, b, c = c_int32(0), c_int32(0), c_size_t(0)
    _check(lib().zb_stage_stats(st, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)), "zb_stage_stats")
    return a.value, b.value, c.value


STASH_TENSORS = ["x", "rstd1", "n1", "a", "h", "rstd2", "n2", "gu", "s", "dy", "dn2", "dh", "dqkv", "dn1", "qkv",
                 "lse"]


def zb_stage_stash_view(st, mb, layer, tensor):
    """(device address, rows, cols, element bytes) of one stashed tensor; `tensor` is a name of
    STASH_TENSORS or its index."""
    idx = STASH_TENSORS.index(tensor) if isinstance(tensor, str) else int(tensor)
    ptr, rows, cols, eb = c_void_p(0), ctypes.c_int64(0), ctypes.c_int64(0), c_int32(0)
    _check(lib().zb_stage_stash_view(st, mb, layer, idx, ctypes.byref(ptr), ctypes.byref(rows), ctypes.byref(cols),
                                     ctypes.byref(eb)), "zb_stage_stash_view")
    return ptr.value or 0, rows.value, cols.value, eb.value


def zb_stage_set_tracing(st, enable):
    _check(lib().zb_stage_set_tracing(st, 1 if enable else 0), "zb_stage_set_tracing")


def zb_stage_read_tracing(st, reset=True):
    """dict kernel class -> {"launches", "ms", "flops", "bytes"} of the launches recorded so far."""
    arr = (zb_kernel_stats * len(KERNEL_CLASSES))()
    _check(lib().zb_stage_read_tracing(st, arr, 1 if reset else 0), "zb_stage_read_tracing")
    return {name: {"launches": arr[i].launches, "ms": arr[i].ms, "flops": arr[i].flops, "bytes": arr[i].bytes}
            for i, name in enumerate(KERNEL_CLASSES)}
