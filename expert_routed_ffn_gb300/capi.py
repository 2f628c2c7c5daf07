"""ctypes binding of libmoe.so (include/moe.h): argument marshalling only.

Every step of the block runs in the library's CUDA kernels; this module only
passes device pointers, sizes and the current torch stream.  There is no
fallback: if libmoe.so has not been built (``expert_routed_ffn_gb300.build``),
``load()`` raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "_build", "libmoe.so")
HEADER = os.path.join(ROOT, "include", "moe.h")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_OOM, MOE_ERR_TIMEOUT, \
    MOE_ERR_DEVICE_CHECK = range(7)
STATUS_NAMES = ["MOE_OK", "MOE_ERR_INVALID_ARG", "MOE_ERR_UNSUPPORTED", "MOE_ERR_CUDA",
                "MOE_ERR_OOM", "MOE_ERR_TIMEOUT", "MOE_ERR_DEVICE_CHECK"]
MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 0, 1
MOE_ACT_SILU, MOE_ACT_SWIGLU_OAI = 0, 1
MOE_DTYPE_BF16, MOE_DTYPE_F32 = 0, 1
MOE_NORM_NONE, MOE_NORM_RMS, MOE_NORM_GEMMA = 0, 1, 2
MOE_GATE_NONE, MOE_GATE_TOKEN, MOE_GATE_CHANNEL = 0, 1, 2
MOE_WEIGHTS_BF16, MOE_WEIGHTS_MXFP8, MOE_WEIGHTS_MXFP4 = 0, 1, 2
WEIGHT_FORMATS = {"bf16": MOE_WEIGHTS_BF16, "mxfp8": MOE_WEIGHTS_MXFP8, "mxfp4": MOE_WEIGHTS_MXFP4}
SCALE_KEYS = ("gate_scale", "up_scale", "down_scale", "sh_gate_scale", "sh_up_scale", "sh_down_scale")
MOE_OPT_PATH, MOE_OPT_WAIT_LIMIT_NS, MOE_OPT_STAGE_EVENTS, MOE_OPT_FUSE_EXPERTS, MOE_OPT_PREFETCH = 0, 1, 2, 3, 4
MOE_OPT_TRACE = 5
MOE_OPT_GEMM_PAIR = 6
MOE_OPT_GRAPH = 8
MOE_OPT_PAIR_SWAP = 9
MOE_OPT_COMBINE_OVERLAP = 10
MOE_OPT_STAGED_STORES = 11
MOE_BUF_GEMM_STATS = 6
MOE_BUF_ROUTER_STATS = 7
MOE_BUF_NORMED_X = 8
MOE_BUF_SHARED_HIDDEN = 9
TRACE_FIELDS = 5  # first begin, first ready, last ready, first end, last end
PATH_AUTO, PATH_DECODE, PATH_GROUPED, PATH_SWAPPED = 0, 1, 2, 3
(MOE_BUF_TOPK_IDX, MOE_BUF_TOPK_W, MOE_BUF_EXPERT_OFFS, MOE_BUF_SORTED_TOKEN, MOE_BUF_SLOT,
 MOE_BUF_HIDDEN) = range(6)


class MoeConfig(ctypes.Structure):
    _fields_ = [
        ("hidden_size", ctypes.c_int), ("num_experts", ctypes.c_int),
        ("num_experts_per_tok", ctypes.c_int), ("num_shared_experts", ctypes.c_int),
        ("moe_intermediate_size", ctypes.c_int), ("shared_intermediate_size", ctypes.c_int),
        ("shared_packed", ctypes.c_int), ("score_func", ctypes.c_int), ("route_norm", ctypes.c_int),
        ("route_scale", ctypes.c_float), ("hidden_act", ctypes.c_int), ("act_alpha", ctypes.c_float),
        ("act_limit", ctypes.c_float), ("act_beta", ctypes.c_float), ("act_dtype", ctypes.c_int),
        ("max_tokens", ctypes.c_int), ("mlp_norm", ctypes.c_int), ("rms_norm_eps", ctypes.c_float),
        ("weight_format", ctypes.c_int),
    ]


class MoeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("router_w", "expert_bias", "gate", "up", "down", "sh_gate", "sh_up", "sh_down",
                 "pre_norm_w", "post_norm_w", "gate_scale", "up_scale", "down_scale", "sh_gate_scale",
                 "sh_up_scale", "sh_down_scale")]


class MoeStats(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("kernel_launches", ctypes.c_int),
                ("workspace_bytes", ctypes.c_longlong)]


def header_symbols() -> list:
    """Names of the functions include/moe.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:moe_status|void|const char \*)\s*(moe_\w+)\s*\(", text, re.M)))


_lib = None


def load():
    """Load libmoe.so (must already be built: expert_routed_ffn_gb300.build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmoe.so is not built ({LIB_PATH}); run expert_routed_ffn_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    P, I, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
    L.moe_create.argtypes = [ctypes.POINTER(MoeConfig), ctypes.POINTER(MoeWeights), ctypes.POINTER(P)]
    L.moe_route.argtypes = [P, P, I, P, P, P]
    L.moe_forward.argtypes = [P, P, I, P, P]
    L.moe_forward_host.argtypes = [P, P, I, P, P]
    L.moe_sync_status.argtypes = [P]
    L.moe_destroy.argtypes = [P]
    L.moe_destroy.restype = None
    L.moe_last_error.argtypes = []
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_set_option.argtypes = [P, I, LL]
    L.moe_get_stats.argtypes = [P, ctypes.POINTER(MoeStats)]
    L.moe_inspect.argtypes = [P, I, P, ctypes.c_size_t, P]
    L.moe_get_stage_times.argtypes = [P, ctypes.POINTER(ctypes.c_float), I, ctypes.POINTER(I)]
    L.moe_get_trace.argtypes = [P, ctypes.POINTER(ctypes.c_double), I, ctypes.POINTER(I)]
    L.moe_get_stage_name.argtypes = [P, I]
    L.moe_get_stage_name.restype = ctypes.c_char_p
    L.moe_dispatch_noalloc.argtypes = [P, I, I, I, P, P, P, P, P]
    L.moe_operators_status.argtypes = []
    L.moe_operators_wait_limit.argtypes = [LL]
    L.moe_grouped_forward.argtypes = [P, P, P, I, I, I, I, I, P, P]
    L.moe_grouped_dgrad.argtypes = [P, P, P, I, I, I, I, I, P, P]
    L.moe_grouped_wgrad.argtypes = [P, P, P, I, I, I, I, I, I, P, P]
    SZ, F = ctypes.c_size_t, ctypes.c_float
    L.moe_grouped_gated_forward.argtypes = [P, P, P, P, I, I, I, I, I, F, F, F, P, P, P, P]
    L.moe_grouped_gated_backward.argtypes = [P, P, P, P, P, I, I, I, I, I, F, F, F, P, P, P]
    L.moe_grouped_gated_dgrad.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P]
    L.moe_sandwich_norm.argtypes = [P, P, P, P, P, I, F, F, I, I, I, I, I, P, P, P]
    L.moe_sandwich_norm_workspace.argtypes = [I, I, ctypes.POINTER(SZ)]
    L.moe_sandwich_norm_backward.argtypes = [P, P, P, P, P, P, P, I, F, F, I, I, I, I, I, P, P, P, P, P, P, SZ, P]
    L.moe_orthogonalize_workspace.argtypes = [I, I, I, ctypes.POINTER(SZ)]
    L.moe_orthogonalize.argtypes = [P, I, I, I, I, ctypes.POINTER(F), I, F, F, P, P, SZ, P]
    L.moe_mx_quantize.argtypes = [P, I, I, I, I, I, P, P, P]
    L.moe_mx_dequantize.argtypes = [P, P, I, I, I, I, I, P, P]
    L.moe_mx_grouped_forward.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P]
    L.moe_clip_workspace.argtypes = [I, ctypes.POINTER(SZ)]
    L.moe_clip_grad_norm.argtypes = [P, I, ctypes.c_float, P, P, SZ, P]
    for name in ("moe_create", "moe_route", "moe_forward", "moe_forward_host", "moe_sync_status", "moe_dispatch_noalloc",
                 "moe_set_option", "moe_get_stats", "moe_inspect", "moe_get_stage_times", "moe_get_trace",
                 "moe_operators_status", "moe_operators_wait_limit", "moe_grouped_forward", "moe_grouped_dgrad", "moe_grouped_wgrad", "moe_mx_quantize",
                 "moe_mx_dequantize", "moe_mx_grouped_forward", "moe_clip_workspace", "moe_clip_grad_norm",
                 "moe_grouped_gated_forward", "moe_grouped_gated_backward", "moe_grouped_gated_dgrad",
                 "moe_sandwich_norm", "moe_sandwich_norm_workspace", "moe_sandwich_norm_backward",
                 "moe_orthogonalize_workspace", "moe_orthogonalize"):
        getattr(L, name).restype = I
    _lib = L
    return L


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = load().moe_last_error().decode(errors="replace")
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{where}: {name}: {msg}")


def check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def config_from_shape(shape, max_tokens: int = None) -> MoeConfig:
    """C config from a workloads.MoeShape (the pages' config keys)."""
    return MoeConfig(
        hidden_size=shape.H, num_experts=shape.E, num_experts_per_tok=shape.k,
        num_shared_experts=shape.num_shared_experts, moe_intermediate_size=shape.I,
        shared_intermediate_size=0 if shape.shared_packed else shape.S,
        shared_packed=int(shape.shared_packed),
        score_func={"sigmoid": MOE_SCORE_SIGMOID, "softmax": MOE_SCORE_SOFTMAX}[shape.score_func],
        route_norm=int(shape.route_norm), route_scale=shape.route_scale,
        hidden_act={"silu": MOE_ACT_SILU, "swigluoai": MOE_ACT_SWIGLU_OAI}[shape.hidden_act],
        act_alpha=shape.act_alpha, act_limit=shape.act_limit, act_beta=shape.act_beta,
        act_dtype={"bf16": MOE_DTYPE_BF16, "f32": MOE_DTYPE_F32}[shape.dtype],
        max_tokens=max(1, shape.T if max_tokens is None else max_tokens),
        mlp_norm={"none": MOE_NORM_NONE, "rms": MOE_NORM_RMS, "gemma": MOE_NORM_GEMMA}[shape.mlp_norm],
        rms_norm_eps=shape.rms_norm_eps,
        weight_format=WEIGHT_FORMATS[getattr(shape, "weight_format", "bf16")])


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class MoeBlock:
    """One handle of libmoe.so over borrowed torch CUDA tensors.

    weights: dict with router_w [E,H] fp32, expert_bias [E] fp32 (or None),
    gate/up [E',I,H], down [E',H,I] bf16 and sh_gate/sh_up [S,H], sh_down [H,S]
    bf16 (or None), and pre_norm_w / post_norm_w [H] fp32 with the sandwich
    norms.  MX weight formats: the six expert tensors hold uint8 element codes
    and gate_scale ... sh_down_scale their uint8 E8M0 scales.  The tensors are
    kept referenced for the handle's lifetime.
    """

    def __init__(self, config: MoeConfig, weights: dict):
        import torch
        self._torch = torch
        self.cfg = config
        self._keep = {k: v for k, v in weights.items() if isinstance(v, torch.Tensor)}
        w = MoeWeights(**{k: (None if weights.get(k) is None else weights[k].data_ptr())
                          for k in ("router_w", "expert_bias", "gate", "up", "down", "sh_gate",
                                    "sh_up", "sh_down", "pre_norm_w", "post_norm_w") + SCALE_KEYS})
        h = ctypes.c_void_p()
        check(load().moe_create(ctypes.byref(config), ctypes.byref(w), ctypes.byref(h)), "moe_create")
        self.h = h
        self.x_dtype = torch.float32 if config.act_dtype == MOE_DTYPE_F32 else torch.bfloat16

    def close(self):
        if getattr(self, "h", None):
            load().moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def route(self, X, stream=None):
        T = X.shape[0]
        torch = self._torch
        idx = torch.empty((T, self.cfg.num_experts_per_tok), dtype=torch.int32, device=X.device)
        w = torch.empty((T, self.cfg.num_experts_per_tok), dtype=torch.float32, device=X.device)
        check(load().moe_route(self.h, _ptr(X), T, _ptr(idx), _ptr(w), _stream(stream)), "moe_route")
        return idx, w

    def forward(self, X, Y=None, stream=None):
        if Y is None:
            Y = self._torch.empty_like(X)
        check(load().moe_forward(self.h, _ptr(X), X.shape[0], _ptr(Y), _stream(stream)), "moe_forward")
        return Y

    def forward_host(self, X_host, Y_host, stream=None):
        check(load().moe_forward_host(self.h, _ptr(X_host), X_host.shape[0], _ptr(Y_host),
                                      _stream(stream)), "moe_forward_host")
        return Y_host

    def sync_status(self) -> int:
        return load().moe_sync_status(self.h)

    def set_option(self, option: int, value: int):
        check(load().moe_set_option(self.h, option, int(value)), "moe_set_option")

    def stats(self) -> MoeStats:
        s = MoeStats()
        check(load().moe_get_stats(self.h, ctypes.byref(s)), "moe_get_stats")
        return s

    def stage_times(self) -> list:
        buf = (ctypes.c_float * 8)()
        n = ctypes.c_int()
        check(load().moe_get_stage_times(self.h, buf, 8, ctypes.byref(n)), "moe_get_stage_times")
        return [buf[i] for i in range(n.value)]

    def trace(self) -> list:
        """(name, first_begin, first_ready, last_ready, first_end, last_end) in us per kernel
        of the last forward (MOE_OPT_TRACE on)."""
        buf = (ctypes.c_double * (TRACE_FIELDS * 8))()
        n = ctypes.c_int()
        check(load().moe_get_trace(self.h, buf, 8, ctypes.byref(n)), "moe_get_trace")
        names = self.stage_names()
        return [(names[i],) + tuple(buf[TRACE_FIELDS * i + f] for f in range(TRACE_FIELDS)) for i in range(n.value)]

    def stage_names(self) -> list:
        L = load()
        return [L.moe_get_stage_name(self.h, i).decode() for i in range(self.stats().kernel_launches)]

    def inspect(self, buffer: int, count: int, dtype, stream=None):
        torch = self._torch
        out = torch.empty(count, dtype=dtype, device="cuda")
        nbytes = count * out.element_size()
        check(load().moe_inspect(self.h, buffer, _ptr(out), nbytes, _stream(stream)), "moe_inspect")
        return out


def block_from_inputs(shape, inputs: dict, max_tokens: int = None) -> MoeBlock:
    """MoeBlock over a workloads.make_inputs() dict on the GPU (expert weights
    rounded to bf16 when the workload stores them in fp32)."""
    from .workloads import expert_weights_bf16
    w = dict(router_w=inputs["router_w"], expert_bias=inputs["expert_bias"], **expert_weights_bf16(inputs),
             pre_norm_w=inputs.get("pre_norm_w"), post_norm_w=inputs.get("post_norm_w"),
             **{k: inputs.get(k) for k in SCALE_KEYS})
    blk = MoeBlock(config_from_shape(shape, max_tokens), w)
    return blk


# ------------------------------------------------------------------ operators
# The products of the block one at a time and what surrounds them (include/moe.h,
# "Operators around the stacked expert weights").  Each runs on the device of its
# tensors, on `stream` or that device's current stream, and allocates only outputs it
# was not given.  None of them is recorded by autograd: results never require a gradient,
# whatever the inputs do, and the gradients are operators of their own.  After offsets that
# break the rule, a result allocated here is uninitialised: operators_status() tells.

_torch = _device = _raw_stream = None


def _t():
    """torch, imported with the first operator."""
    global _torch, _device, _raw_stream
    if _torch is None:
        import torch
        load()
        _device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        _torch = torch
    return _torch


def _need(cond, message):
    if not cond:
        raise ValueError(message)


def _fits(*sizes):
    """The library takes sizes as int; ctypes would pass on their lower 32 bits."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"sizes must be below 2^31: {sizes}")


def _dtype_code(dtype):
    if dtype is _torch.bfloat16:
        return MOE_DTYPE_BF16
    if dtype is _torch.float32:
        return MOE_DTYPE_F32
    raise ValueError(f"dtype must be bfloat16 or float32, not {dtype}")


def _tensor(t, name, shape, dtype, index):
    """t is a contiguous CUDA tensor of this shape and type on device `index`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous() and index >= 0:
        return
    _need(index >= 0 and t.get_device() == index, f"{name} must be on the CUDA device of the other tensors")
    _need(t.dtype is dtype, f"{name} must be {dtype}, not {t.dtype}")
    _need(t.shape == shape, f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    _need(t.is_contiguous(), f"{name} must be contiguous")


def _enter(index, stream):
    """(raw stream, undo): makes the tensors' device the current one and `stream` its current
    stream (so that outputs are allocated for it).  undo is None where nothing had to change."""
    if stream is None and _device() == index:
        return _raw_stream(index), None
    _need(index >= 0 and (stream is None or stream.device_index == index), "the stream must be of the tensors' device")
    undo = contextlib.ExitStack()
    undo.enter_context(_torch.cuda.device(index))
    if stream is not None:
        undo.enter_context(_torch.cuda.stream(stream))
    return _torch.cuda.current_stream().cuda_stream, undo


def _leave(undo):
    if undo is not None:
        undo.close()


def operators_status(device=None) -> int:
    """moe_operators_status on `device` (default: the current one): synchronises, returns
    and clears what the operators recorded there."""
    with _t().cuda.device(device):
        return load().moe_operators_status()


def _grouped(name, A, W, offs, out, out_dtype, stream, forward):
    torch = _t()
    _need(W.dim() == 3 and A.dim() == 2, "W must be [E, N, K] and X or dY [rows, ..]")
    E, N, K = W.shape
    cols, red = (N, K) if forward else (K, N)
    rows = A.shape[0]
    _fits(rows, E, N, K)
    index = A.get_device()
    _tensor(A, "X" if forward else "dY", (rows, red), torch.bfloat16, index)
    _tensor(W, "W", (E, N, K), torch.bfloat16, index)
    _tensor(offs, "offs", (E + 1,), torch.int32, index)
    raw, undo = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty((rows, cols), dtype=out_dtype or torch.bfloat16, device=A.device)
        else:
            _tensor(out, "out", (rows, cols), out_dtype or out.dtype, index)
        status = getattr(_lib, name)(A.data_ptr(), W.data_ptr(), offs.data_ptr(), rows, E, N, K, _dtype_code(out.dtype),
                                     out.data_ptr(), raw)
    finally:
        _leave(undo)
    check(status, name)
    return out


def grouped_forward(X, W, offs, out=None, out_dtype=None, stream=None):
    """Y[r] = W[e] X[r] for the rows offs[e] <= r < offs[e + 1] of X [rows, K] bf16; W [E, N, K]
    bf16, offs [E + 1] int32.  Returns out (default: a new [rows, N] tensor of out_dtype, bf16
    by default), whose rows outside [offs[0], offs[E]) are left as they were."""
    return _grouped("moe_grouped_forward", X, W, offs, out, out_dtype, stream, True)


def grouped_dgrad(dY, W, offs, out=None, out_dtype=None, stream=None):
    """The gradient of grouped_forward by its X: dX[r] = W[e]^T dY[r], dY [rows, N] bf16."""
    return _grouped("moe_grouped_dgrad", dY, W, offs, out, out_dtype, stream, False)


def grouped_wgrad(dY, X, offs, out=None, out_dtype=None, accumulate=False, stream=None):
    """The gradient of grouped_forward by its W: dW[e] = sum over e's rows of dY[r] X[r]^T, in
    out (default: a new [E, N, K] tensor, fp32 unless out_dtype says otherwise).  accumulate:
    add to what out holds."""
    torch = _t()
    _need(X.dim() == 2 and dY.dim() == 2, "X must be [rows, K] and dY [rows, N]")
    _need(offs.dim() == 1 and offs.numel() >= 2, "offs must be [E + 1]")
    _need(out is not None or not accumulate, "accumulate needs out")
    (rows, K), N, E = X.shape, dY.shape[1], offs.numel() - 1
    _fits(rows, E, N, K)
    index = X.get_device()
    _tensor(X, "X", (rows, K), torch.bfloat16, index)
    _tensor(dY, "dY", (rows, N), torch.bfloat16, index)
    _tensor(offs, "offs", (E + 1,), torch.int32, index)
    raw, undo = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty((E, N, K), dtype=out_dtype or torch.float32, device=X.device)
        else:
            _tensor(out, "out", (E, N, K), out_dtype or out.dtype, index)
        status = _lib.moe_grouped_wgrad(dY.data_ptr(), X.data_ptr(), offs.data_ptr(), rows, E, N, K,
                                        _dtype_code(out.dtype), int(accumulate), out.data_ptr(), raw)
    finally:
        _leave(undo)
    check(status, "moe_grouped_wgrad")
    return out


def _act_code(act):
    if act == "silu":
        return MOE_ACT_SILU
    _need(act == "swigluoai", f"act must be 'silu' or 'swigluoai', not {act!r}")
    return MOE_ACT_SWIGLU_OAI


def _outputs(given, names, shape, dtype, device):
    """The tensors given, or new ones."""
    if given is None:
        return tuple(_torch.empty(shape, dtype=dtype, device=device) for _ in names)
    given = tuple(given)
    _need(len(given) == len(names), f"need the tensors {', '.join(names)}")
    for t, name in zip(given, names):
        _tensor(t, name, shape, dtype, device.index)
    return given


def grouped_gated_forward(X, Wg, Wu, offs, act="silu", alpha=1.702, limit=7.0, beta=1.0, out=None, save=None, stream=None):
    """H = act(G, U), G[r] = Wg[e] X[r], U[r] = Wu[e] X[r] for the rows of expert e as in
    grouped_forward; X [rows, K], Wg and Wu [E, I, K] bf16.  act: "silu", or "swigluoai" with
    alpha, limit and beta.  Returns H [rows, I] bf16 (`out`, or a new tensor); with save=True, or
    save=(G, U) to write into, (H, G, U) for the backward pass.  Rows outside
    [offs[0], offs[E]) are left as they were."""
    torch = _t()
    _need(Wg.dim() == 3 and X.dim() == 2, "Wg must be [E, I, K] and X [rows, K]")
    (E, I, K), rows, code = Wg.shape, X.shape[0], _act_code(act)
    _fits(rows, E, I, K)
    index, bf = X.get_device(), torch.bfloat16
    _tensor(X, "X", (rows, K), bf, index)
    _tensor(Wg, "Wg", (E, I, K), bf, index)
    _tensor(Wu, "Wu", (E, I, K), bf, index)
    _tensor(offs, "offs", (E + 1,), torch.int32, index)
    keep = save is not None and save is not False
    raw, undo = _enter(index, stream)
    try:
        H, = _outputs(None if out is None else (out,), ("out",), (rows, I), bf, X.device)
        G, U = _outputs(None if save is True else save, ("G", "U"), (rows, I), bf, X.device) if keep else (None, None)
        status = _lib.moe_grouped_gated_forward(
            X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), offs.data_ptr(), rows, E, I, K, code, alpha, limit, beta, H.data_ptr(),
            G.data_ptr() if keep else None, U.data_ptr() if keep else None, raw)
    finally:
        _leave(undo)
    check(status, "moe_grouped_gated_forward")
    return (H, G, U) if keep else H


def grouped_gated_backward(dY, Wd, G, U, offs, act="silu", alpha=1.702, limit=7.0, beta=1.0, out=None, stream=None):
    """The gradients (dG, dU) [rows, I] bf16 of grouped_gated_forward's G and U, from dY [rows, K]
    bf16, the gradient of grouped_forward(H, Wd, offs) with Wd [E, K, I]: dH = dY Wd stays in fp32.
    out=(dG, dU): tensors to write into.  Rows outside [offs[0], offs[E]) are left as they were."""
    torch = _t()
    _need(Wd.dim() == 3 and dY.dim() == 2, "Wd must be [E, K, I] and dY [rows, K]")
    (E, K, I), rows, code = Wd.shape, dY.shape[0], _act_code(act)
    _fits(rows, E, I, K)
    index, bf = dY.get_device(), torch.bfloat16
    _tensor(dY, "dY", (rows, K), bf, index)
    _tensor(Wd, "Wd", (E, K, I), bf, index)
    _tensor(G, "G", (rows, I), bf, index)
    _tensor(U, "U", (rows, I), bf, index)
    _tensor(offs, "offs", (E + 1,), torch.int32, index)
    raw, undo = _enter(index, stream)
    try:
        dG, dU = _outputs(out, ("dG", "dU"), (rows, I), bf, dY.device)
        status = _lib.moe_grouped_gated_backward(
            dY.data_ptr(), Wd.data_ptr(), G.data_ptr(), U.data_ptr(), offs.data_ptr(), rows, E, I, K, code, alpha, limit, beta,
            dG.data_ptr(), dU.data_ptr(), raw)
    finally:
        _leave(undo)
    check(status, "moe_grouped_gated_backward")
    return dG, dU


def grouped_gated_dgrad(dG, dU, Wg, Wu, offs, out=None, out_dtype=None, stream=None):
    """The gradient of grouped_gated_forward by its X: dX[r] = Wg[e]^T dG[r] + Wu[e]^T dU[r], in out
    (default: a new [rows, K] tensor of out_dtype, bf16 by default), whose rows outside
    [offs[0], offs[E]) are left as they were."""
    torch = _t()
    _need(Wg.dim() == 3 and dG.dim() == 2, "Wg must be [E, I, K] and dG [rows, I]")
    (E, I, K), rows = Wg.shape, dG.shape[0]
    _fits(rows, E, I, K)
    index, bf = dG.get_device(), torch.bfloat16
    _tensor(dG, "dG", (rows, I), bf, index)
    _tensor(dU, "dU", (rows, I), bf, index)
    _tensor(Wg, "Wg", (E, I, K), bf, index)
    _tensor(Wu, "Wu", (E, I, K), bf, index)
    _tensor(offs, "offs", (E + 1,), torch.int32, index)
    raw, undo = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty((rows, K), dtype=out_dtype or bf, device=dG.device)
        else:
            _tensor(out, "out", (rows, K), out_dtype or out.dtype, index)
        status = _lib.moe_grouped_gated_dgrad(dG.data_ptr(), dU.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), offs.data_ptr(),
                                              rows, E, I, K, _dtype_code(out.dtype), out.data_ptr(), raw)
    finally:
        _leave(undo)
    check(status, "moe_grouped_gated_dgrad")
    return out


def _address(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=1024)
def _norm_workspace(T, H):
    need = ctypes.c_size_t()
    check(_lib.moe_sandwich_norm_workspace(T, H, ctypes.byref(need)), "moe_sandwich_norm_backward")
    return need.value


def _norm_arguments(X, F, pre_w, post_w, gate, kind):
    """Checks what both directions take: X [T, H], F and the parameters.  Returns X's shape, the
    device's index, the kind's code and the gate's kind."""
    f32, shape = _torch.float32, X.shape
    if len(shape) != 2:
        raise ValueError("X must be [T, H]")
    T, H = shape
    _fits(T, H)
    index = X.get_device()
    _tensor(X, "X", shape, X.dtype, index)
    if F is not None:
        _tensor(F, "F", shape, F.dtype, index)
    if pre_w is not None:
        _tensor(pre_w, "pre_w", (H,), f32, index)
    if post_w is not None:
        _tensor(post_w, "post_w", (H,), f32, index)
    if kind != "rms" and kind != "gemma":
        raise ValueError(f"kind must be 'rms' or 'gemma', not {kind!r}")
    gate_kind = MOE_GATE_NONE
    if gate is not None:
        gate_kind = MOE_GATE_TOKEN if gate.dim() == 2 else MOE_GATE_CHANNEL
        _tensor(gate, "gate", (T, 1) if gate_kind == MOE_GATE_TOKEN else (H,), f32, index)
    return shape, index, MOE_NORM_GEMMA if kind == "gemma" else MOE_NORM_RMS, gate_kind


def sandwich_norm(X, F=None, pre_w=None, post_w=None, gate=None, residual_scale=1.0, eps=1e-5, kind="rms", X_out=None,
                  N_out=None, n_dtype=None, stream=None):
    """X' = residual_scale X + gate * norm(F) post_w and N = norm(X') pre_w, the norms after one block and
    before the next with the residual between them.  X [T, H] (bf16 or fp32) is the residual stream, F
    [T, H] the block's result (of its own type, which N has too); pre_w and post_w [H] fp32, gate [H] or
    [T, 1] fp32.  Returns (X', N): without post_w F is added as it is, without pre_w N is None,
    without F X' is X itself and N = norm(X) pre_w (of n_dtype, by default X's).  kind "gemma": weights
    are 1 + w.  X_out may be X, and N_out may be F.  A gate begins at 16 bytes as every tensor does (gate[1:] does not)."""
    torch = _t()
    shape, index, code, gate_kind = _norm_arguments(X, F, pre_w, post_w, gate, kind)
    of_n = F.dtype if F is not None else n_dtype or (X.dtype if N_out is None else N_out.dtype)
    if n_dtype is not None and n_dtype is not of_n:
        raise ValueError("N has F's type")
    x_code, n_code = _dtype_code(X.dtype), _dtype_code(of_n)
    if X_out is not None and F is None or N_out is not None and pre_w is None:
        raise ValueError("X_out needs F, and N_out needs pre_w")
    raw, undo = _enter(index, stream)
    try:
        if F is not None:
            if X_out is None:
                X_out = torch.empty_like(X)
            else:
                _tensor(X_out, "X_out", shape, X.dtype, index)
        if pre_w is not None:
            if N_out is None:
                N_out = torch.empty_like(F) if F is not None else torch.empty(shape, dtype=of_n, device=X.device)
            else:
                _tensor(N_out, "N_out", shape, of_n, index)
        status = _lib.moe_sandwich_norm(X.data_ptr(), _address(F), _address(pre_w), _address(post_w), _address(gate), gate_kind,
                                        residual_scale, eps, code, *shape, x_code, n_code, _address(X_out), _address(N_out), raw)
    finally:
        _leave(undo)
    check(status, "moe_sandwich_norm")
    return (X if F is None else X_out), N_out


def sandwich_norm_backward(dX, dN, X, F=None, pre_w=None, post_w=None, gate=None, residual_scale=1.0, eps=1e-5, kind="rms",
                           dX_out=None, dF_out=None, stream=None):
    """The gradients of sandwich_norm from those of X' and N (dX may be None for zeros, dN is None without
    pre_w), X being the X' it returned: (of its X, of F, of pre_w, of post_w, of the gate), None where
    there is no such tensor.  dX_out may be dX, and dF_out may be dN."""
    torch = _t()
    shape, index, code, gate_kind = _norm_arguments(X, F, pre_w, post_w, gate, kind)
    of_n = F.dtype if F is not None else X.dtype if dN is None else dN.dtype
    x_code, n_code = _dtype_code(X.dtype), _dtype_code(of_n)
    if (dN is None) != (pre_w is None) or dX is None and pre_w is None or dF_out is not None and F is None:
        raise ValueError("dN goes with pre_w, dX is needed without it, and dF_out needs F")
    if dX is not None:
        _tensor(dX, "dX", shape, X.dtype, index)
    if dN is not None:
        _tensor(dN, "dN", shape, of_n, index)
    need = _norm_workspace(*shape)
    raw, undo = _enter(index, stream)
    try:
        if dX_out is None:
            dX_out = torch.empty_like(X)
        else:
            _tensor(dX_out, "dX_out", shape, X.dtype, index)
        if F is not None:
            if dF_out is None:
                dF_out = torch.empty_like(F)
            else:
                _tensor(dF_out, "dF_out", shape, of_n, index)
        dpre = None if pre_w is None else torch.empty_like(pre_w)
        dpost = None if post_w is None else torch.empty_like(post_w)
        dgate = None if gate is None else torch.empty_like(gate)
        work = torch.empty(need, dtype=torch.uint8, device=X.device)
        status = _lib.moe_sandwich_norm_backward(
            _address(dX), _address(dN), X.data_ptr(), _address(F), _address(pre_w), _address(post_w), _address(gate), gate_kind,
            residual_scale, eps, code, *shape, x_code, n_code, dX_out.data_ptr(), _address(dF_out), _address(dpre),
            _address(dpost), _address(dgate), work.data_ptr(), need, raw)
    finally:
        _leave(undo)
    check(status, "moe_sandwich_norm_backward")
    return dX_out, dF_out, dpre, dpost, dgate


def _mx_format(fmt):
    if fmt == "mxfp4":
        return MOE_WEIGHTS_MXFP4
    _need(fmt == "mxfp8", f"fmt must be 'mxfp8' or 'mxfp4', not {fmt!r}")
    return MOE_WEIGHTS_MXFP8


def _mx_shapes(shape, code, of):
    """(slices, rows, K, the shape of codes (of 1) or values (of 2), that of scales) of a tensor of
    values (of 1) or codes (of 2)."""
    two = code == MOE_WEIGHTS_MXFP4
    if len(shape) == 2:
        rows, K = shape
        last = (K // 2 if two else K) if of == 1 else (2 * K if two else K)
        K = K if of == 1 else last
        _fits(rows, K)
        return 1, rows, K, (rows, last), (K // 32, rows)
    _need(len(shape) == 3, "the tensor must be [rows, K] or [slices, rows, K]")
    slices, rows, K = shape
    last = (K // 2 if two else K) if of == 1 else (2 * K if two else K)
    K = K if of == 1 else last
    _fits(slices, rows, K)
    return slices, rows, K, (slices, rows, last), (slices, K // 32, rows)


def mx_quantize(X, fmt, codes=None, scales=None, stream=None):
    """[rows, K] or [slices, rows, K] bf16 or fp32 -> element codes and block scales (uint8) in
    the layout of the block's MX weights: codes [.., rows, K] (mxfp8) or [.., rows, K / 2]
    (mxfp4), scales [.., K / 32, rows]."""
    torch = _t()
    code = _mx_format(fmt)
    slices, rows, K, of_codes, of_scales = _mx_shapes(X.shape, code, 1)
    index, kind, u8 = X.get_device(), X.dtype, torch.uint8
    dtype = _dtype_code(kind)
    _need(index >= 0 and X.is_contiguous(), "X must be a contiguous CUDA tensor")
    raw, undo = _enter(index, stream)
    try:
        if codes is None:
            codes = torch.empty(of_codes, dtype=u8, device=X.device)
        else:
            _tensor(codes, "codes", of_codes, u8, index)
        if scales is None:
            scales = torch.empty(of_scales, dtype=u8, device=X.device)
        else:
            _tensor(scales, "scales", of_scales, u8, index)
        status = _lib.moe_mx_quantize(X.data_ptr(), dtype, slices, rows, K, code, codes.data_ptr(), scales.data_ptr(), raw)
    finally:
        _leave(undo)
    check(status, "moe_mx_quantize")
    return codes, scales


def mx_dequantize(codes, scales, fmt, dtype=None, out=None, stream=None):
    """The values of mx_quantize's codes and scales as dtype (bf16 by default)."""
    torch = _t()
    code = _mx_format(fmt)
    slices, rows, K, of_values, of_scales = _mx_shapes(codes.shape, code, 2)
    index = codes.get_device()
    _need(index >= 0 and codes.is_contiguous() and codes.dtype is torch.uint8, "codes must be a contiguous uint8 CUDA tensor")
    _tensor(scales, "scales", of_scales, torch.uint8, index)
    raw, undo = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty(of_values, dtype=dtype or torch.bfloat16, device=codes.device)
        else:
            _tensor(out, "out", of_values, dtype or out.dtype, index)
        status = _lib.moe_mx_dequantize(codes.data_ptr(), scales.data_ptr(), code, slices, rows, K, _dtype_code(out.dtype),
                                        out.data_ptr(), raw)
    finally:
        _leave(undo)
    check(status, "moe_mx_dequantize")
    return out


def mx_grouped_forward(Xc, Xs, Wc, Ws, offs, out=None, out_dtype=None, stream=None):
    """grouped_forward on MXFP4 operands: Xc [rows, K / 2], Xs [K / 32, rows], Wc [E, N, K / 2],
    Ws [E, K / 32, N] uint8 as mx_quantize gives them, offs [E + 1] int32.  Returns out (default:
    a new [rows, N] tensor of out_dtype, bf16 by default), whose rows outside
    [offs[0], offs[E]) are left as they were."""
    torch = _t()
    _need(Wc.dim() == 3 and Xc.dim() == 2, "Wc must be [E, N, K / 2] and Xc [rows, K / 2]")
    E, N, half = Wc.shape
    rows, K = Xc.shape[0], 2 * half
    _fits(rows, E, N, K)
    index, u8 = Xc.get_device(), torch.uint8
    _tensor(Xc, "Xc", (rows, half), u8, index)
    _tensor(Xs, "Xs", (K // 32, rows), u8, index)
    _tensor(Wc, "Wc", (E, N, half), u8, index)
    _tensor(Ws, "Ws", (E, K // 32, N), u8, index)
    _tensor(offs, "offs", (E + 1,), torch.int32, index)
    raw, undo = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty((rows, N), dtype=out_dtype or torch.bfloat16, device=Xc.device)
        else:
            _tensor(out, "out", (rows, N), out_dtype or out.dtype, index)
        status = _lib.moe_mx_grouped_forward(Xc.data_ptr(), Xs.data_ptr(), Wc.data_ptr(), Ws.data_ptr(), offs.data_ptr(),
                                             rows, E, N, K, _dtype_code(out.dtype), out.data_ptr(), raw)
    finally:
        _leave(undo)
    check(status, "moe_mx_grouped_forward")
    return out


class MoeGrad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_longlong), ("dtype", ctypes.c_int)]


def clip_grad_norm(grads, max_norm, out=None, stream=None):
    """The norm of all `grads` (one or more contiguous bf16 or fp32 CUDA tensors of one device)
    together, as a 0-dim fp32 tensor, and the gradients times min(1, max_norm / norm): in place,
    or into the tensors `out`.  If a gradient holds an infinity or a NaN the norm says so and the
    gradients are passed on as they are; a finite norm beyond fp32 is reported as an infinity and
    the gradients are clipped by its value.  Results must not overlap other tensors of the lists:
    a gradient that is there twice cannot be clipped in place."""
    torch = _t()
    T = torch.Tensor
    grads = list(grads)
    n = len(grads)
    _need(n > 0, "clip_grad_norm needs at least one gradient")
    index = grads[0].get_device()
    types, counts = [g.dtype for g in grads], list(map(T.numel, grads))
    both, src = grads, list(map(T.data_ptr, grads))
    dst = src
    if out is not None:
        out = list(out)
        _need(len(out) == n, "out must have a tensor for each gradient")
        _need([o.dtype for o in out] == types and list(map(T.numel, out)) == counts,
              "out must have the gradients' types and sizes")
        both, dst = grads + out, list(map(T.data_ptr, out))
    _need(index >= 0 and set(map(T.get_device, both)) == {index}, "the gradients must be on one CUDA device")
    _need(all(map(T.is_contiguous, both)), "the gradients must be contiguous")
    code = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32}
    kinds = set(types)
    _need(kinds <= code.keys(), "the gradients must be bfloat16 or float32")
    flat = [0] * (5 * n)  # an array of moe_grad: grad, out, count, dtype and its padding
    flat[0::5], flat[1::5], flat[2::5] = src, dst, counts
    flat[3::5] = [code[types[0]]] * n if len(kinds) == 1 else map(code.__getitem__, types)
    table = struct.pack("@" + "PPqii" * n, *flat)
    need = ctypes.c_size_t()
    check(_lib.moe_clip_workspace(n, ctypes.byref(need)), "moe_clip_workspace")
    raw, undo = _enter(index, stream)
    try:
        device = grads[0].device
        norm = torch.empty((), dtype=torch.float32, device=device)
        work = torch.empty(need.value, dtype=torch.uint8, device=device)
        status = _lib.moe_clip_grad_norm(table, n, max_norm, norm.data_ptr(), work.data_ptr(), need.value, raw)
    finally:
        _leave(undo)
    check(status, "moe_clip_grad_norm")
    return norm


def orthogonalize(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0, out=None, stream=None):
    """scale times the matrices of G ([N, K] or [E, N, K], bf16 or fp32) with their singular values moved
    towards one by Newton-Schulz products: X = G / (|G| + eps), then `steps` times
    X <- a X + (b A + c A^2) X with A = X X^T.  coefficients: (a, b, c), or one such triple for each step.  Returns
    out (default: a new tensor), bf16 of G's shape; out may be G where G is bf16."""
    torch = _t()
    _need(G.dim() in (2, 3), "G must be [N, K] or [E, N, K]")
    E, N, K = G.shape if G.dim() == 3 else (1, *G.shape)
    _fits(E, N, K)
    index, code = G.get_device(), _dtype_code(G.dtype)
    _need(index >= 0 and G.is_contiguous(), "G must be a contiguous CUDA tensor")
    triples = list(coefficients)
    if triples and not hasattr(triples[0], "__len__"):
        triples = [triples] * steps
    _need(len(triples) == steps and all(len(c) == 3 for c in triples), "coefficients must be (a, b, c), or a triple for each step")
    table = (ctypes.c_float * (3 * steps))(*[v for c in triples for v in c])
    need = ctypes.c_size_t()
    check(_lib.moe_orthogonalize_workspace(E, N, K, ctypes.byref(need)), "moe_orthogonalize")
    raw, undo = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty(G.shape, dtype=torch.bfloat16, device=G.device)
        else:
            _tensor(out, "out", G.shape, torch.bfloat16, index)
        work = torch.empty(need.value, dtype=torch.uint8, device=G.device)
        status = _lib.moe_orthogonalize(G.data_ptr(), code, E, N, K, table, steps, eps, scale, out.data_ptr(), work.data_ptr(),
                                        need.value, raw)
    finally:
        _leave(undo)
    check(status, "moe_orthogonalize")
    return out
