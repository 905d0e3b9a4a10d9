"""ctypes binding of libforge (include/forge.h), same names as the C ABI.

This module only marshals arguments: it checks that torch tensors have the
dtype, shape, device and contiguity the C ABI documents, passes their data
pointers and the current CUDA stream, and turns a non-OK status into
ForgeError.  Every step of the computation runs in the library's kernels.
Loading fails loudly if the library has not been built.
"""

import ctypes
import os
import threading

import torch

from . import build as _build

c_int32, c_int64, c_uint64, c_float, c_void_p = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                                                 ctypes.c_float, ctypes.c_void_p)

OPT_KINDS = {"adamw": 0, "nadam": 1, "radam": 2, "lion": 3, "rmsprop": 4, "adagrad": 5,
             "sgd": 6, "sgd_momentum": 7}
W_FP32, W_BF16_SR = 0, 1
STATE_FP32, STATE_INT8_B64, STATE_BF16 = 0, 1, 2
STATE_INT8_B32, STATE_INT8_B128, STATE_INT8_B256 = 3, 4, 5
INT8_STATE_OF_BLOCK = {32: STATE_INT8_B32, 64: STATE_INT8_B64, 128: STATE_INT8_B128,
                       256: STATE_INT8_B256}
G_FP32, G_BF16 = 0, 1
ACT_KINDS = {"silu": 0, "gelu_tanh": 1}
CODE_BLOCK = 128  # elements of a row that share a scale of the E4M3 codes
USES_S1 = {"adamw", "nadam", "radam", "lion", "sgd_momentum"}
USES_S2 = {"adamw", "nadam", "radam", "rmsprop", "adagrad"}

STATUS = {0: "FORGE_OK", 1: "FORGE_ERR_INVALID_ARG", 2: "FORGE_ERR_UNSUPPORTED",
          3: "FORGE_ERR_CUDA", 4: "FORGE_ERR_TIMEOUT", 5: "FORGE_ERR_DEVICE"}


class ForgeLinear(ctypes.Structure):
    _fields_ = [("T", c_int64), ("N", c_int64), ("K", c_int64),
                ("X", c_void_p), ("dY", c_void_p), ("dX", c_void_p)]


class ForgeLinearFp8(ctypes.Structure):
    _fields_ = [("T", c_int64), ("N", c_int64), ("K", c_int64),
                ("Xt", c_void_p), ("dYt", c_void_p), ("x_scale", c_float), ("dy_scale", c_float)]


class ForgeState(ctypes.Structure):
    _fields_ = [("W", c_void_p), ("w_dtype", c_int32), ("s_dtype", c_int32),
                ("s1", c_void_p), ("s2", c_void_p), ("s1_scale", c_void_p), ("s2_scale", c_void_p)]


class ForgeHparams(ctypes.Structure):
    _fields_ = [(n, c_float) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "alpha",
                                       "momentum")]


class ForgeGrouped(ctypes.Structure):
    _fields_ = [("T", c_int64), ("N", c_int64), ("K", c_int64), ("groups", c_int32), ("offsets", c_void_p),
                ("X", c_void_p), ("dY", c_void_p), ("Y", c_void_p), ("dX", c_void_p)]


class ForgeTensor(ctypes.Structure):
    _fields_ = [("n", c_int64), ("grad", c_void_p), ("W", c_void_p), ("s1", c_void_p), ("s2", c_void_p),
                ("s1_scale", c_void_p), ("s2_scale", c_void_p)]


class ForgeRmsnorm(ctypes.Structure):
    _fields_ = [("T", c_int64), ("K", c_int64), ("x", c_void_p), ("residual", c_void_p), ("w", c_void_p),
                ("eps", c_float), ("yt_scale", c_float), ("h", c_void_p), ("rstd", c_void_p),
                ("y", c_void_p), ("yq", c_void_p), ("yq_scale", c_void_p), ("yt", c_void_p),
                ("amax", c_void_p)]


class ForgeRmsnormGrad(ctypes.Structure):
    _fields_ = [("T", c_int64), ("K", c_int64), ("dy", c_void_p), ("h", c_void_p), ("w", c_void_p),
                ("rstd", c_void_p), ("dh", c_void_p), ("dx", c_void_p), ("dw", c_void_p),
                ("workspace", c_void_p)]


class ForgeGated(ctypes.Structure):
    _fields_ = [("T", c_int64), ("F", c_int64), ("K", c_int64), ("act", c_int32), ("X", c_void_p), ("W", c_void_p),
                ("Y", c_void_p), ("gu", c_void_p), ("gu_codes", c_void_p), ("gu_scale", c_void_p)]


class ForgeGatedGrad(ctypes.Structure):
    _fields_ = [("T", c_int64), ("F", c_int64), ("N", c_int64), ("act", c_int32), ("dY", c_void_p), ("Wd", c_void_p),
                ("gu", c_void_p), ("gu_codes", c_void_p), ("gu_scale", c_void_p), ("dGU", c_void_p), ("Y", c_void_p)]


class ForgeLinearE4m3(ctypes.Structure):
    _fields_ = [("T", c_int64), ("N", c_int64), ("K", c_int64), ("Xq", c_void_p), ("x_scale", c_void_p),
                ("Wq", c_void_p), ("w_scale", c_void_p), ("Y", c_void_p)]


HPARAM_DEFAULTS = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, alpha=0.99,
                       momentum=0.0)


class ForgeError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {message}")


_lock = threading.Lock()
_lib = None

_SIGNATURES = {
    "forge_linear_bwd_step": (c_int32, [ctypes.POINTER(ForgeLinear), ctypes.POINTER(ForgeState),
                                        c_int32, ctypes.POINTER(ForgeHparams), c_int64, c_uint64,
                                        c_void_p]),
    "forge_linear_bwd_step_static": (c_int32, [ctypes.POINTER(ForgeLinear), ctypes.POINTER(ForgeState),
                                               c_int32, ctypes.POINTER(ForgeHparams), c_int64, c_uint64,
                                               c_void_p]),
    "forge_linear_bwd_step_shard": (c_int32, [ctypes.POINTER(ForgeLinear), ctypes.POINTER(ForgeState),
                                              c_int32, ctypes.POINTER(ForgeHparams), c_int64, c_uint64,
                                              c_int64, c_void_p]),
    "forge_linear_bwd_step_fp8": (c_int32, [ctypes.POINTER(ForgeLinearFp8), ctypes.POINTER(ForgeState),
                                            c_int32, ctypes.POINTER(ForgeHparams), c_int64, c_uint64,
                                            c_void_p]),
    "forge_linear_dgrad": (c_int32, [ctypes.POINTER(ForgeLinear), c_void_p, c_int32, c_void_p]),
    "forge_unfused_wgrad": (c_int32, [ctypes.POINTER(ForgeLinear), c_void_p, c_void_p]),
    "forge_unfused_opt_step": (c_int32, [c_void_p, ctypes.POINTER(ForgeState), c_int64, c_int64,
                                         c_int32, ctypes.POINTER(ForgeHparams), c_int64, c_uint64,
                                         c_void_p]),
    "forge_quantize_state": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int32,
                                       c_void_p]),
    "forge_dequantize_state": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int32,
                                         c_void_p]),
    "forge_quantize_state_block": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int32,
                                             c_int32, c_void_p]),
    "forge_dequantize_state_block": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_int32,
                                               c_int32, c_void_p]),
    "forge_grouped_linear": (c_int32, [ctypes.POINTER(ForgeGrouped), c_void_p, c_void_p]),
    "forge_grouped_dgrad": (c_int32, [ctypes.POINTER(ForgeGrouped), c_void_p, c_void_p]),
    "forge_grouped_bwd_step": (c_int32, [ctypes.POINTER(ForgeGrouped), ctypes.POINTER(ForgeState), c_int32,
                                         ctypes.POINTER(ForgeHparams), c_int64, c_uint64, c_void_p]),
    "forge_multi_opt_step": (c_int32, [ctypes.POINTER(ForgeTensor), c_int32, c_int32, c_int32, c_int32,
                                       c_int32, ctypes.POINTER(ForgeHparams), c_int64, c_uint64,
                                       c_void_p]),
    "forge_rmsnorm_fwd": (c_int32, [ctypes.POINTER(ForgeRmsnorm), c_void_p]),
    "forge_rmsnorm_bwd": (c_int32, [ctypes.POINTER(ForgeRmsnormGrad), c_void_p]),
    "forge_rmsnorm_bwd_workspace": (c_int64, [c_int64, c_int64]),
    "forge_gated_linear": (c_int32, [ctypes.POINTER(ForgeGated), c_void_p]),
    "forge_gated_dgrad": (c_int32, [ctypes.POINTER(ForgeGatedGrad), c_void_p]),
    "forge_quantize_e4m3": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_int64, c_int64, c_int32, c_void_p]),
    "forge_dequantize_e4m3": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int64, c_int64, c_int32, c_void_p]),
    "forge_linear_e4m3": (c_int32, [ctypes.POINTER(ForgeLinearE4m3), c_void_p]),
    "forge_get_device_status": (c_int32, [c_void_p]),
    "forge_set_wait_limit_ns": (c_int32, [c_uint64]),
    "forge_debug_skip_loads": (c_int32, [c_int32]),
    "forge_set_step_fusion": (None, [c_int32]),
    "forge_status_string": (ctypes.c_char_p, [c_int32]),
    "forge_last_error_message": (ctypes.c_char_p, []),
    "forge_abi_version": (c_int32, []),
}


def library_path() -> str:
    return os.environ.get("FORGE_LIBRARY", _build.lib_path("libforge.so"))


def lib() -> ctypes.CDLL:
    """The loaded libforge.  Raises if it has not been built (no fallback)."""
    global _lib
    L = _lib
    if L is not None:
        return L
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"libforge is not built ({path} missing); run "
                                   "optimizer_tcgen05_dw_gb300.build.build() first")
            L = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
        return _lib


def _check(status: int):
    if status != 0:
        msg = lib().forge_last_error_message().decode(errors="replace")
        raise ForgeError(status, msg)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a torch.cuda.Stream object
# (the call's largest fixed cost otherwise); the public route until CUDA is
# initialised or where these accessors are missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _cur_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_cur_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _need(t, name, dtype, shape):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def hparams(**kw) -> ForgeHparams:
    h = dict(HPARAM_DEFAULTS)
    for k, v in kw.items():
        if k not in h:
            raise KeyError(f"unknown hyper-parameter {k}")
        h[k] = v
    return ForgeHparams(**{k: float(v) for k, v in h.items()})


_hp_cache = {}


def _hparams_of(hp: dict) -> ForgeHparams:
    """hparams(**hp), kept for dicts of plain Python numbers (the library only
    reads the struct during the call, so calls may share it)."""
    try:
        key = tuple(hp.items())
        h = _hp_cache.get(key)
    except TypeError:  # an unhashable value
        return hparams(**hp)
    if h is None:
        h = hparams(**hp)
        if all(type(v) in (float, int) for _, v in key):
            if len(_hp_cache) >= 256:
                _hp_cache.clear()
            _hp_cache[key] = h
    return h


def make_state(W, s1=None, s2=None, s1_scale=None, s2_scale=None) -> ForgeState:
    """A forge_state_t for W (fp32 or bf16) and optional fp32 / INT8 states."""
    N, K = W.shape
    wd = W.dtype
    if wd == torch.float32:
        wdt = W_FP32
    elif wd == torch.bfloat16:
        wdt = W_BF16_SR
    else:
        raise TypeError(f"W must be float32 or bfloat16, got {W.dtype}")
    _need(W, "W", wd, (N, K))
    d1 = None if s1 is None else s1.dtype
    d2 = None if s2 is None else s2.dtype
    if d1 in (None, torch.float32) and d2 in (None, torch.float32):  # fp32 or no states
        if s1 is not None:
            _need(s1, "s1", torch.float32, (N, K))
        if s2 is not None:
            _need(s2, "s2", torch.float32, (N, K))
        return ForgeState(W.data_ptr(), wdt, STATE_FP32, _ptr(s1), _ptr(s2), _ptr(s1_scale),
                          _ptr(s2_scale))
    int8 = d1 in (torch.int8, torch.uint8) or d2 in (torch.int8, torch.uint8)
    bf16 = d1 == torch.bfloat16 or d2 == torch.bfloat16
    if bf16:
        for t, nm in ((s1, "s1"), (s2, "s2")):
            if t is not None:
                _need(t, nm, torch.bfloat16, (N, K))
        return ForgeState(_ptr(W), wdt, STATE_BF16, _ptr(s1), _ptr(s2), None, None)
    sdt = STATE_FP32
    if int8:
        # the block width follows from the scale arrays: [N, K / block]
        sc = s1_scale if s1_scale is not None else s2_scale
        if sc is None or sc.dim() != 2 or sc.shape[1] == 0 or K % sc.shape[1] != 0 \
                or K // sc.shape[1] not in INT8_STATE_OF_BLOCK:
            raise ValueError("INT8 states need [N, K / B] float32 scales with B in 32, 64, 128, 256")
        block = K // sc.shape[1]
        sdt = INT8_STATE_OF_BLOCK[block]
        if s1 is not None:
            _need(s1, "s1", torch.int8, (N, K))
            _need(s1_scale, "s1_scale", torch.float32, (N, K // block))
        if s2 is not None:
            _need(s2, "s2", torch.uint8, (N, K))
            _need(s2_scale, "s2_scale", torch.float32, (N, K // block))
    else:
        for t, nm in ((s1, "s1"), (s2, "s2")):
            if t is not None:
                _need(t, nm, torch.float32, (N, K))
    return ForgeState(_ptr(W), wdt, sdt, _ptr(s1), _ptr(s2), _ptr(s1_scale), _ptr(s2_scale))


def forge_linear_bwd_step(X, dY, W, opt: str, hp: dict, step: int, seed: int, s1=None, s2=None,
                          s1_scale=None, s2_scale=None, dX=None, stream=None):
    """The fused FORGE step on one linear layer (updates W and states in place;
    writes dX from the pre-update W when dX is given)."""
    T, K = X.shape
    N = W.shape[0]
    _need(X, "X", torch.bfloat16, (T, K))
    _need(dY, "dY", torch.bfloat16, (T, N))
    if dX is not None:
        _need(dX, "dX", torch.bfloat16, (T, K))
    st = make_state(W, s1, s2, s1_scale, s2_scale)
    lin = ForgeLinear(T, N, K, _ptr(X), _ptr(dY), _ptr(dX))
    _check(lib().forge_linear_bwd_step(ctypes.byref(lin), ctypes.byref(st), OPT_KINDS[opt],
                                       ctypes.byref(_hparams_of(hp)), int(step),
                                       int(seed) & 0xFFFFFFFFFFFFFFFF, _stream(stream)))


def forge_linear_bwd_step_shard(X, dY, W, opt: str, hp: dict, step: int, seed: int, row_offset: int,
                                s1=None, s2=None, s1_scale=None, s2_scale=None, dX=None, stream=None):
    """The FORGE step on rows [row_offset, row_offset + N) of a larger weight
    matrix (a column-parallel shard): dY holds the shard's N columns of the
    upstream gradient, W and the states the shard's rows; stochastic rounding
    uses the elements' indices in the whole matrix.  dX, if given, receives the
    shard's partial input gradient (the layer's dX is the sum over shards)."""
    T, K = X.shape
    N = W.shape[0]
    _need(X, "X", torch.bfloat16, (T, K))
    _need(dY, "dY", torch.bfloat16, (T, N))
    if dX is not None:
        _need(dX, "dX", torch.bfloat16, (T, K))
    st = make_state(W, s1, s2, s1_scale, s2_scale)
    lin = ForgeLinear(T, N, K, _ptr(X), _ptr(dY), _ptr(dX))
    _check(lib().forge_linear_bwd_step_shard(ctypes.byref(lin), ctypes.byref(st), OPT_KINDS[opt],
                                             ctypes.byref(_hparams_of(hp)), int(step),
                                             int(seed) & 0xFFFFFFFFFFFFFFFF, int(row_offset),
                                             _stream(stream)))


def forge_linear_bwd_step_static(X, dY, W, opt: str, hp: dict, step: int, seed: int, s1=None,
                                 s2=None, s1_scale=None, s2_scale=None, dX=None, stream=None):
    """forge_linear_bwd_step with its one-launch scratch in the library's own
    static device array (no allocation; calls on one device must not overlap)."""
    T, K = X.shape
    N = W.shape[0]
    _need(X, "X", torch.bfloat16, (T, K))
    _need(dY, "dY", torch.bfloat16, (T, N))
    if dX is not None:
        _need(dX, "dX", torch.bfloat16, (T, K))
    st = make_state(W, s1, s2, s1_scale, s2_scale)
    lin = ForgeLinear(T, N, K, _ptr(X), _ptr(dY), _ptr(dX))
    _check(lib().forge_linear_bwd_step_static(ctypes.byref(lin), ctypes.byref(st), OPT_KINDS[opt],
                                              ctypes.byref(_hparams_of(hp)), int(step),
                                              int(seed) & 0xFFFFFFFFFFFFFFFF, _stream(stream)))


def forge_linear_bwd_step_fp8(Xt, dYt, x_scale: float, dy_scale: float, W, opt: str, hp: dict,
                              step: int, seed: int, s1=None, s2=None, s1_scale=None, s2_scale=None,
                              stream=None):
    """The FORGE step from E4M3 operands: Xt [K, T] and dYt [N, T] codes
    (torch.float8_e4m3fn or uint8), token-contiguous, with one scale each;
    updates the bf16 W and the states in place (no dX)."""
    K, T = Xt.shape
    N = W.shape[0]
    for t, name, shape in ((Xt, "Xt", (K, T)), (dYt, "dYt", (N, T))):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise TypeError(f"{name}: expected torch.float8_e4m3fn or uint8 E4M3 codes, got {t.dtype}")
        _need(t, name, t.dtype, shape)
    st = make_state(W, s1, s2, s1_scale, s2_scale)
    lin = ForgeLinearFp8(T, N, K, _ptr(Xt), _ptr(dYt), float(x_scale), float(dy_scale))
    _check(lib().forge_linear_bwd_step_fp8(ctypes.byref(lin), ctypes.byref(st), OPT_KINDS[opt],
                                           ctypes.byref(_hparams_of(hp)), int(step),
                                           int(seed) & 0xFFFFFFFFFFFFFFFF, _stream(stream)))


def forge_linear_dgrad(dY, W, dX, stream=None):
    T, N = dY.shape
    K = W.shape[1]
    _need(dY, "dY", torch.bfloat16, (T, N))
    _need(dX, "dX", torch.bfloat16, (T, K))
    _need(W, "W", W.dtype, (N, K))
    wdt = W_FP32 if W.dtype == torch.float32 else W_BF16_SR
    lin = ForgeLinear(T, N, K, None, _ptr(dY), _ptr(dX))
    _check(lib().forge_linear_dgrad(ctypes.byref(lin), _ptr(W), wdt, _stream(stream)))


def forge_unfused_wgrad(X, dY, dW, stream=None):
    T, K = X.shape
    N = dY.shape[1]
    _need(X, "X", torch.bfloat16, (T, K))
    _need(dY, "dY", torch.bfloat16, (T, N))
    _need(dW, "dW", torch.float32, (N, K))
    lin = ForgeLinear(T, N, K, _ptr(X), _ptr(dY), None)
    _check(lib().forge_unfused_wgrad(ctypes.byref(lin), _ptr(dW), _stream(stream)))


def forge_unfused_opt_step(dW, W, opt: str, hp: dict, step: int, seed: int, s1=None, s2=None,
                           s1_scale=None, s2_scale=None, stream=None):
    N, K = W.shape
    if dW is not None:
        _need(dW, "dW", torch.float32, (N, K))
    st = make_state(W, s1, s2, s1_scale, s2_scale)
    _check(lib().forge_unfused_opt_step(_ptr(dW), ctypes.byref(st), N, K, OPT_KINDS[opt],
                                        ctypes.byref(_hparams_of(hp)), int(step),
                                        int(seed) & 0xFFFFFFFFFFFFFFFF, _stream(stream)))


def forge_quantize_state(x, codes, absmax, is_signed: bool, stream=None, block: int = 64):
    """x fp32 [rows, cols] -> INT8 codes and absmax [rows, cols / block]."""
    rows, cols = x.shape
    _need(x, "x", torch.float32, (rows, cols))
    _need(codes, "codes", torch.int8 if is_signed else torch.uint8, (rows, cols))
    _need(absmax, "absmax", torch.float32, (rows, cols // block))
    _check(lib().forge_quantize_state_block(_ptr(x), _ptr(codes), _ptr(absmax), rows, cols,
                                            1 if is_signed else 0, int(block), _stream(stream)))


def forge_dequantize_state(codes, absmax, x, is_signed: bool, stream=None, block: int = 64):
    rows, cols = x.shape
    _need(x, "x", torch.float32, (rows, cols))
    _need(codes, "codes", torch.int8 if is_signed else torch.uint8, (rows, cols))
    _need(absmax, "absmax", torch.float32, (rows, cols // block))
    _check(lib().forge_dequantize_state_block(_ptr(codes), _ptr(absmax), _ptr(x), rows, cols,
                                              1 if is_signed else 0, int(block), _stream(stream)))


def _experts(W, offsets):
    """(groups, N, K) of W [groups, N, K] bf16, and the offsets' check."""
    if W.dim() != 3:
        raise ValueError(f"W: expected [groups, N, K], got {tuple(W.shape)}")
    E, N, K = W.shape
    _need(W, "W", torch.bfloat16, (E, N, K))
    _need(offsets, "offsets", torch.int32, (E + 1,))
    return E, N, K


def forge_grouped_linear(X, W, offsets, Y, stream=None):
    """Y[t] = W[e] X[t] for the rows offsets[e] .. offsets[e+1]-1 of X [T, K] of
    every expert e: W [groups, N, K], Y [T, N], all bf16; offsets [groups + 1]
    int32 on the device.  Rows of no group become zero."""
    E, N, K = _experts(W, offsets)
    T = X.shape[0]
    _need(X, "X", torch.bfloat16, (T, K))
    _need(Y, "Y", torch.bfloat16, (T, N))
    g = ForgeGrouped(T, N, K, E, offsets.data_ptr(), X.data_ptr(), None, Y.data_ptr(), None)
    _check(lib().forge_grouped_linear(ctypes.byref(g), W.data_ptr(), _stream(stream)))


def forge_grouped_dgrad(dY, W, offsets, dX, stream=None):
    """dX[t] = W[e]^T dY[t], as forge_grouped_linear."""
    E, N, K = _experts(W, offsets)
    T = dY.shape[0]
    _need(dY, "dY", torch.bfloat16, (T, N))
    _need(dX, "dX", torch.bfloat16, (T, K))
    g = ForgeGrouped(T, N, K, E, offsets.data_ptr(), None, dY.data_ptr(), None, dX.data_ptr())
    _check(lib().forge_grouped_dgrad(ctypes.byref(g), W.data_ptr(), _stream(stream)))


def forge_grouped_bwd_step(X, dY, W, offsets, opt: str, hp: dict, step: int, seed: int, s1=None, s2=None,
                           s1_scale=None, s2_scale=None, dX=None, stream=None):
    """The FORGE step on every expert's weight W[e] (bf16, with the states of
    forge_linear_bwd_step in the same [groups, N, K] layout; INT8 scales
    [groups, N, K / B]): W and the states are updated in place, dX, if given,
    comes from the weights before the update."""
    E, N, K = _experts(W, offsets)
    T = X.shape[0]
    _need(X, "X", torch.bfloat16, (T, K))
    _need(dY, "dY", torch.bfloat16, (T, N))
    if dX is not None:
        _need(dX, "dX", torch.bfloat16, (T, K))
    rows = [t if t is None else _flat_rows(t, name, E, N) for t, name in
            ((s1, "s1"), (s2, "s2"), (s1_scale, "s1_scale"), (s2_scale, "s2_scale"))]
    st = make_state(W.view(E * N, K), *rows)
    g = ForgeGrouped(T, N, K, E, offsets.data_ptr(), X.data_ptr(), dY.data_ptr(), None, _ptr(dX))
    _check(lib().forge_grouped_bwd_step(ctypes.byref(g), ctypes.byref(st), OPT_KINDS[opt],
                                        ctypes.byref(_hparams_of(hp)), int(step), int(seed) & 0xFFFFFFFFFFFFFFFF,
                                        _stream(stream)))


def _flat_rows(t, name, E, N):
    if t.dim() != 3 or t.shape[0] != E or t.shape[1] != N:
        raise ValueError(f"{name}: expected [groups, N, ..] = [{E}, {N}, ..], got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.view(E * N, t.shape[2])


class ForgeTensors:
    """The tensor table of forge_multi_opt_step (make_tensors builds it): the C
    array of pointers, and the tensors themselves so that they stay alive."""

    __slots__ = ("table", "count", "w_dtype", "g_dtype", "s_dtype", "kept")


def _one_dtype(tensors, name, allowed):
    """The dtype that the tensors share (None when there are none)."""
    found = {t.dtype for t in tensors if t is not None}
    if len(found) > 1:
        raise TypeError(f"{name}: one dtype a call, got {sorted(map(str, found))}; make one table per dtype")
    if not found:
        return None
    d = found.pop()
    if d not in allowed:
        raise TypeError(f"{name}: expected one of {', '.join(map(str, allowed))}, got {d}")
    return d


def _need_flat(t, name, dtype, n):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def make_tensors(weights, grads, s1=None, s2=None, s1_scale=None, s2_scale=None, block: int = 64) -> ForgeTensors:
    """The table of one forge_multi_opt_step group, built once and used step
    after step: lists of equal length of weights (float32 or bfloat16),
    gradients (float32 or bfloat16; None entries mean a zero gradient) and
    states (float32, bfloat16, or int8 s1 / uint8 s2 codes with float32 absmax
    of ceil(n / block) blocks of the flattened tensor), any shapes and lengths,
    contiguous.  The gradients' values may change between steps, their storage
    may not: the table holds (and keeps alive) the tensors it was built from, and
    a step after one was replaced still reads the old one, so build a table again
    then (or zero gradients in place instead of dropping them)."""
    weights, grads = list(weights), list(grads)
    n = len(weights)

    def listed(v, name):
        v = [None] * n if v is None else list(v)
        if len(v) != n:
            raise ValueError(f"{name}: expected {n} tensors, got {len(v)}")
        return v

    grads, s1, s2 = listed(grads, "grads"), listed(s1, "s1"), listed(s2, "s2")
    s1_scale, s2_scale = listed(s1_scale, "s1_scale"), listed(s2_scale, "s2_scale")
    if any(w is None for w in weights):
        raise ValueError("weights: every entry must be a tensor")
    f32, b16 = torch.float32, torch.bfloat16
    wd = _one_dtype(weights, "weights", (f32, b16)) or f32
    gd = _one_dtype(grads, "grads", (f32, b16)) or f32
    d1 = _one_dtype(s1, "s1", (f32, b16, torch.int8))
    d2 = _one_dtype(s2, "s2", (f32, b16, torch.uint8))
    int8 = d1 == torch.int8 or d2 == torch.uint8
    if d1 is not None and d2 is not None and (d1 == torch.int8) != (d2 == torch.uint8) \
            or not int8 and None not in (d1, d2) and d1 != d2:
        raise TypeError(f"s1 and s2 must be kept alike, got {d1} and {d2}")
    if int8 and block not in INT8_STATE_OF_BLOCK:
        raise ValueError("block must be 32, 64, 128 or 256")
    out = ForgeTensors()
    out.count = n
    out.w_dtype = W_FP32 if wd == f32 else W_BF16_SR
    out.g_dtype = G_FP32 if gd == f32 else G_BF16
    out.s_dtype = (INT8_STATE_OF_BLOCK[block] if int8 else STATE_BF16 if b16 in (d1, d2) else STATE_FP32)
    out.table = (ForgeTensor * max(1, n))()
    for i, (w, g, a, b, sa, sb) in enumerate(zip(weights, grads, s1, s2, s1_scale, s2_scale)):
        e = w.numel()
        _need_flat(w, f"weights[{i}]", wd, e)
        for t, name, d in ((g, "grads", gd), (a, "s1", d1), (b, "s2", d2)):
            if t is not None:
                _need_flat(t, f"{name}[{i}]", d, e)
        if int8:
            for t, sc, name in ((a, sa, "s1_scale"), (b, sb, "s2_scale")):
                if t is not None:
                    if sc is None:
                        raise ValueError(f"{name}[{i}] is required with INT8 states")
                    _need_flat(sc, f"{name}[{i}]", f32, (e + block - 1) // block)
        out.table[i] = ForgeTensor(e, _ptr(g), _ptr(w), _ptr(a), _ptr(b), _ptr(sa) if int8 else None,
                                   _ptr(sb) if int8 else None)
    out.kept = (weights, grads, s1, s2, s1_scale, s2_scale)
    return out


def forge_multi_opt_step(tensors: ForgeTensors, opt: str, hp: dict, step: int, seed: int, stream=None):
    """One optimizer step over every tensor of the table (make_tensors), in
    place; bf16 weights of tensor i round with the seed `seed + i`."""
    _check(lib().forge_multi_opt_step(tensors.table, tensors.count, tensors.w_dtype, tensors.g_dtype,
                                      tensors.s_dtype, OPT_KINDS[opt], ctypes.byref(_hparams_of(hp)),
                                      int(step), int(seed) & 0xFFFFFFFFFFFFFFFF, _stream(stream)))


def _rows(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a [T, K] tensor, got {tuple(t.shape)}")
    return t.shape


def forge_rmsnorm_fwd(x, w, eps: float, residual=None, h=None, rstd=None, y=None, yq=None, yq_scale=None,
                      yt=None, yt_scale: float = 1.0, amax=None, stream=None):
    """Root-mean-square norm of x [T, K] bf16 (+ residual) with weight w [K]
    bf16.  Writes the outputs given: h (the sum, bf16; may be x or residual), rstd [T], y
    [T, K] bf16 (may be x or residual where h is not), yq [T, K] E4M3 with yq_scale [T], yt [K, T] E4M3 of y /
    yt_scale with amax [1]."""
    T, K = shape = _rows(x, "x")
    _need(x, "x", torch.bfloat16, shape)
    _need(w, "w", torch.bfloat16, (K,))
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, shape)
    if h is not None:
        _need(h, "h", torch.bfloat16, shape)
    if rstd is not None:
        _need(rstd, "rstd", torch.float32, (T,))
    if y is not None:
        _need(y, "y", torch.bfloat16, shape)
    if yq is not None:
        _need(yq, "yq", torch.float8_e4m3fn, shape)
        _need(yq_scale, "yq_scale", torch.float32, (T,))
    if yt is not None:
        _need(yt, "yt", torch.float8_e4m3fn, (K, T))
    if amax is not None:
        _need(amax, "amax", torch.float32, (1,))
    p = ForgeRmsnorm(T, K, x.data_ptr(), _ptr(residual), w.data_ptr(), eps, yt_scale, _ptr(h), _ptr(rstd), _ptr(y),
                     _ptr(yq), _ptr(yq_scale), _ptr(yt), _ptr(amax))
    _check(lib().forge_rmsnorm_fwd(ctypes.byref(p), _stream(stream)))


def forge_rmsnorm_bwd_workspace(T: int, K: int) -> int:
    """Floats of workspace that forge_rmsnorm_bwd needs for [T, K]."""
    n = lib().forge_rmsnorm_bwd_workspace(int(T), int(K))
    if n < 0:
        raise ForgeError(1, lib().forge_last_error_message().decode(errors="replace"))
    return int(n)


def forge_rmsnorm_bwd(dy, h, w, rstd, dx, dw, workspace, dh=None, stream=None):
    """Gradient of forge_rmsnorm_fwd: dx [T, K] bf16 (of x and the residual
    alike; dh, the gradient reaching h itself, is added) and dw [K] float32.
    workspace: float32, forge_rmsnorm_bwd_workspace(T, K) elements or more."""
    T, K = shape = _rows(dy, "dy")
    _need(dy, "dy", torch.bfloat16, shape)
    _need(h, "h", torch.bfloat16, shape)
    _need(w, "w", torch.bfloat16, (K,))
    _need(rstd, "rstd", torch.float32, (T,))
    _need(dx, "dx", torch.bfloat16, shape)
    _need(dw, "dw", torch.float32, (K,))
    if dh is not None:
        _need(dh, "dh", torch.bfloat16, shape)
    _need(workspace, "workspace", torch.float32, workspace.shape)
    if workspace.numel() < forge_rmsnorm_bwd_workspace(T, K):
        raise ValueError(f"workspace: need {forge_rmsnorm_bwd_workspace(T, K)} elements, got {workspace.numel()}")
    p = ForgeRmsnormGrad(T, K, dy.data_ptr(), h.data_ptr(), w.data_ptr(), rstd.data_ptr(), _ptr(dh), dx.data_ptr(),
                         dw.data_ptr(), workspace.data_ptr())
    _check(lib().forge_rmsnorm_bwd(ctypes.byref(p), _stream(stream)))


def _here(*tensors):
    """Every tensor given lies on the current device, whose stream the call goes to."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must be on the current device, cuda:{dev}; got one on {t.device}")


def _act(act):
    if act not in ACT_KINDS:
        raise ValueError(f"act: expected one of {', '.join(ACT_KINDS)}, got {act!r}")
    return ACT_KINDS[act]


def _kept(T, F, gu, gu_codes, gu_scale):
    """The checks of what forge_gated_linear keeps for its gradient."""
    if gu is not None and gu_codes is not None:
        raise ValueError("gu and gu_codes: one of them")
    if gu is not None:
        _need(gu, "gu", torch.bfloat16, (T, 2 * F))
    if gu_codes is not None:
        _need(gu_codes, "gu_codes", torch.float8_e4m3fn, (T, 2 * F))
    if gu_codes is not None or gu_scale is not None:
        _need(gu_scale, "gu_scale", torch.float32, (T, 2, (F + CODE_BLOCK - 1) // CODE_BLOCK))


def forge_gated_linear(X, W, Y, act: str = "silu", gu=None, gu_codes=None, gu_scale=None, stream=None):
    """Y = act(X Wg^T) * (X Wu^T): X [T, K], W [2F, K] (the gate's F rows, then
    the up projection's), Y [T, F], all bf16; act "silu" or "gelu_tanh".  For
    forge_gated_dgrad it keeps the two projections side by side in gu [T, 2F]
    bf16, or in gu_codes [T, 2F] (torch.float8_e4m3fn) with gu_scale
    [T, 2, ceil(F / 128)]."""
    T, K = _rows(X, "X")
    F = _rows(W, "W")[0] // 2
    _need(X, "X", torch.bfloat16, (T, K))
    _need(W, "W", torch.bfloat16, (2 * F, K))
    _need(Y, "Y", torch.bfloat16, (T, F))
    _kept(T, F, gu, gu_codes, gu_scale)
    _here(X, W, Y, gu, gu_codes, gu_scale)
    g = ForgeGated(T, F, K, _act(act), X.data_ptr(), W.data_ptr(), Y.data_ptr(), _ptr(gu), _ptr(gu_codes), _ptr(gu_scale))
    _check(lib().forge_gated_linear(ctypes.byref(g), _stream(stream)))


def forge_gated_dgrad(dY, Wd, dGU, act: str = "silu", gu=None, gu_codes=None, gu_scale=None, Y=None, stream=None):
    """The gradient of forge_gated_linear through the down projection Wd [N, F]:
    from dY [T, N] and what was kept (gu, or gu_codes and gu_scale), dGU
    [T, 2F] (the gradients of both projections side by side; may be gu itself)
    and, if given, Y [T, F] formed again.  Then forge_linear_bwd_step(Y, dY, Wd, ..)
    and forge_linear_bwd_step(X, dGU, W, .., dX=dX) step the weights."""
    T, N = _rows(dY, "dY")
    F = _rows(Wd, "Wd")[1]
    _need(dY, "dY", torch.bfloat16, (T, N))
    _need(Wd, "Wd", torch.bfloat16, (N, F))
    _need(dGU, "dGU", torch.bfloat16, (T, 2 * F))
    if gu is None and gu_codes is None:
        raise ValueError("gu or gu_codes is required")
    _kept(T, F, gu, gu_codes, gu_scale)
    if Y is not None:
        _need(Y, "Y", torch.bfloat16, (T, F))
    _here(dY, Wd, dGU, gu, gu_codes, gu_scale, Y)
    g = ForgeGatedGrad(T, F, N, _act(act), dY.data_ptr(), Wd.data_ptr(), _ptr(gu), _ptr(gu_codes), _ptr(gu_scale),
                       dGU.data_ptr(), _ptr(Y))
    _check(lib().forge_gated_dgrad(ctypes.byref(g), _stream(stream)))


def _coded(codes, scale, x, block_rows):
    """(rows, cols, x's dtype code) of x [rows, cols] and its codes and scales."""
    shape = rows, cols = _rows(x, "x")
    if block_rows not in (1, CODE_BLOCK):
        raise ValueError(f"block_rows must be 1 or {CODE_BLOCK}, got {block_rows}")
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"x: expected torch.bfloat16 or torch.float32, got {x.dtype}")
    _need(x, "x", x.dtype, shape)
    _need(codes, "codes", torch.float8_e4m3fn, shape)
    _need(scale, "scale", torch.float32, (rows if block_rows == 1 else (rows + CODE_BLOCK - 1) // CODE_BLOCK,
                                          (cols + CODE_BLOCK - 1) // CODE_BLOCK))
    _here(x, codes, scale)
    return rows, cols, G_FP32 if x.dtype == torch.float32 else G_BF16


def forge_quantize_e4m3(x, codes, scale, block_rows: int = 1, stream=None):
    """x [rows, cols] (bf16 or float32) -> codes (torch.float8_e4m3fn) and a
    float32 scale for each 128 elements of a row (block_rows 1: scale
    [rows, ceil(cols / 128)]) or each 128 x 128 (block_rows 128: scale
    [ceil(rows / 128), ceil(cols / 128)])."""
    rows, cols, dt = _coded(codes, scale, x, block_rows)
    _check(lib().forge_quantize_e4m3(x.data_ptr(), dt, codes.data_ptr(), scale.data_ptr(), rows, cols, int(block_rows),
                                     _stream(stream)))


def forge_dequantize_e4m3(codes, scale, x, block_rows: int = 1, stream=None):
    """The inverse map: x = codes * scale, rounded to x's dtype."""
    rows, cols, dt = _coded(codes, scale, x, block_rows)
    _check(lib().forge_dequantize_e4m3(codes.data_ptr(), scale.data_ptr(), x.data_ptr(), dt, rows, cols, int(block_rows),
                                       _stream(stream)))


def forge_linear_e4m3(Xq, x_scale, Wq, w_scale, Y, stream=None):
    """Y [T, N] bf16 = X W^T from codes Xq [T, K] with x_scale [T, ceil(K / 128)]
    and Wq [N, K] with w_scale [ceil(N / 128), ceil(K / 128)], as
    forge_quantize_e4m3 writes them (block_rows 1 and 128)."""
    T, K = _rows(Xq, "Xq")
    N = _rows(Wq, "Wq")[0]
    blocks = lambda n: (n + CODE_BLOCK - 1) // CODE_BLOCK  # noqa: E731
    _need(Xq, "Xq", torch.float8_e4m3fn, (T, K))
    _need(x_scale, "x_scale", torch.float32, (T, blocks(K)))
    _need(Wq, "Wq", torch.float8_e4m3fn, (N, K))
    _need(w_scale, "w_scale", torch.float32, (blocks(N), blocks(K)))
    _need(Y, "Y", torch.bfloat16, (T, N))
    _here(Xq, x_scale, Wq, w_scale, Y)
    g = ForgeLinearE4m3(T, N, K, Xq.data_ptr(), x_scale.data_ptr(), Wq.data_ptr(), w_scale.data_ptr(), Y.data_ptr())
    _check(lib().forge_linear_e4m3(ctypes.byref(g), _stream(stream)))


def forge_get_device_status(stream=None):
    """Synchronises the stream; raises ForgeError if a kernel reported an error."""
    _check(lib().forge_get_device_status(_stream(stream)))


def forge_set_wait_limit_ns(ns: int):
    _check(lib().forge_set_wait_limit_ns(int(ns)))


def forge_set_step_fusion(enable: bool):
    """Allow (default) or forbid the one-launch dX + FORGE step."""
    lib().forge_set_step_fusion(1 if enable else 0)


def forge_debug_skip_loads(enable: bool):
    _check(lib().forge_debug_skip_loads(1 if enable else 0))


def forge_abi_version() -> int:
    return int(lib().forge_abi_version())
