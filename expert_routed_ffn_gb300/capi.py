"""ctypes binding of libmoe.so (include/moe.h): argument marshalling only.

Every step of the block runs in the library's CUDA kernels; this module only
passes device pointers, sizes and the current torch stream.  There is no
fallback: if libmoe.so has not been built (``expert_routed_ffn_gb300.build``),
``load()`` raises.
"""

from __future__ import annotations

import contextlib
import ctypes
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
    SZ = ctypes.c_size_t
    L.moe_mx_quantize.argtypes = [P, I, I, I, I, I, P, P, P]
    L.moe_mx_dequantize.argtypes = [P, P, I, I, I, I, I, P, P]
    L.moe_mx_grouped_forward.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P]
    L.moe_clip_workspace.argtypes = [I, ctypes.POINTER(SZ)]
    L.moe_clip_grad_norm.argtypes = [P, I, ctypes.c_float, P, P, SZ, P]
    for name in ("moe_create", "moe_route", "moe_forward", "moe_forward_host", "moe_sync_status", "moe_dispatch_noalloc",
                 "moe_set_option", "moe_get_stats", "moe_inspect", "moe_get_stage_times", "moe_get_trace",
                 "moe_operators_status", "moe_operators_wait_limit", "moe_grouped_forward", "moe_grouped_dgrad", "moe_grouped_wgrad", "moe_mx_quantize",
                 "moe_mx_dequantize", "moe_mx_grouped_forward", "moe_clip_workspace", "moe_clip_grad_norm"):
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
