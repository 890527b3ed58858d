"""Thin Python binding of ``libbitlinear.so`` (argument marshalling only).

Each ``bitlinear_*`` function here has the name, arguments and meaning of the C entry
point declared in ``include/bitlinear.h``; it checks that the torch tensors it is given
are CUDA, contiguous and of the expected dtype and shape, passes their device pointers
and the current CUDA stream, and raises ``BitLinearError`` on a non-zero status.  All
arithmetic happens in the library's CUDA kernels.  There is no fallback: if the library
cannot be loaded, every call raises.

The helpers at the end (``quantize_weights``, ``quantize_act``, ``forward``) only
allocate the output tensors with torch and call the entry points above.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbitlinear.so")

BL_OK = 0
BL_OUT_F32, BL_OUT_BF16, BL_OUT_I32 = 0, 1, 2
(BL_PATH_AUTO, BL_PATH_GEMV, BL_PATH_TC, BL_PATH_TC_1SM, BL_PATH_TC_2SM, BL_PATH_SKINNY, BL_PATH_GEMV_STREAM,
 BL_PATH_GEMV_TMA) = range(8)
BL_ERRBIT_BAD_CODE, BL_ERRBIT_TIMEOUT, BL_ERRBIT_INDEX = 0x1, 0x2, 0x4
BL_XQ_ROWMAJOR, BL_XQ_K16_EVENODD, BL_XQ_K16_STRIDE4 = 0, 1, 2
BL_NORM_RMS, BL_NORM_LAYER = 0, 1

EXPORTED = [
    "bitlinear_workspace_size", "bitlinear_quantize_weights",
    "bitlinear_quantize_weights_with_scale", "bitlinear_pack", "bitlinear_quantize_act",
    "bitlinear_forward", "bitlinear_forward_path", "bitlinear_quantize_act_layout",
    "bitlinear_forward_layout", "bitlinear_norm_quantize_act", "bitlinear_forward_rowscale",
    "bitlinear_tl5_row_bytes", "bitlinear_pack_tl5", "bitlinear_repack_tl5", "bitlinear_forward_tl5",
    "bitlinear_ste_backward_input", "bitlinear_ste_backward_weight", "bitlinear_forward_stall_test",
    "bitlinear_norm_forward", "bitlinear_norm_backward_workspace_size", "bitlinear_norm_backward",
    "bitlinear_fp8_row_bytes", "bitlinear_fp8_quantize_act", "bitlinear_fp8_quantize_weights",
    "bitlinear_fp8_forward", "bitlinear_fp8_backward_input", "bitlinear_fp8_backward_weight",
    "bitlinear_fp8_stall_test", "bitlinear_norm_backward_stall_test",
    "bitlinear_last_cuda_error",
    "bitlinear_status_string",
]


class BitLinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = lib().bitlinear_status_string(status).decode()
        extra = ""
        if name == "BL_ERR_CUDA":
            extra = " (cudaError %d)" % lib().bitlinear_last_cuda_error()
        super().__init__("%s: %s%s" % (where, name, extra))


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libbitlinear.so is not built (run "
                               "`python -m ternary_weight_bit_absmean_b200.build_lib`): %s" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, I64, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
        S = ctypes.c_int
        L.bitlinear_workspace_size.argtypes = [I64, I64]
        L.bitlinear_workspace_size.restype = ctypes.c_size_t
        L.bitlinear_quantize_weights.argtypes = [P, I64, I64, F, P, P, P, ctypes.c_size_t, P]
        L.bitlinear_quantize_weights.restype = S
        L.bitlinear_quantize_weights_with_scale.argtypes = [P, I64, I64, P, P, P]
        L.bitlinear_quantize_weights_with_scale.restype = S
        L.bitlinear_pack.argtypes = [P, I64, I64, P, P, P]
        L.bitlinear_pack.restype = S
        L.bitlinear_quantize_act.argtypes = [P, I64, I64, F, P, P, P]
        L.bitlinear_quantize_act.restype = S
        L.bitlinear_forward.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, P]
        L.bitlinear_forward.restype = S
        L.bitlinear_forward_path.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, S, P]
        L.bitlinear_forward_path.restype = S
        L.bitlinear_quantize_act_layout.argtypes = [P, I64, I64, F, P, P, S, P]
        L.bitlinear_quantize_act_layout.restype = S
        L.bitlinear_forward_layout.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, S, S, P]
        L.bitlinear_forward_layout.restype = S
        L.bitlinear_forward_rowscale.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, S, S, P]
        L.bitlinear_forward_rowscale.restype = S
        L.bitlinear_norm_quantize_act.argtypes = [P, P, I64, I64, S, F, F, P, P, S, P]
        L.bitlinear_norm_quantize_act.restype = S
        L.bitlinear_tl5_row_bytes.argtypes = [I64]
        L.bitlinear_tl5_row_bytes.restype = I64
        L.bitlinear_pack_tl5.argtypes = [P, I64, I64, P, P, P]
        L.bitlinear_pack_tl5.restype = S
        L.bitlinear_repack_tl5.argtypes = [P, I64, I64, P, P]
        L.bitlinear_repack_tl5.restype = S
        L.bitlinear_forward_tl5.argtypes = [P, P, P, P, I64, I64, I64, P, S, P]
        L.bitlinear_forward_tl5.restype = S
        L.bitlinear_ste_backward_input.argtypes = [P, P, P, I64, I64, I64, P, P]
        L.bitlinear_ste_backward_input.restype = S
        L.bitlinear_ste_backward_weight.argtypes = [P, P, P, P, I64, I64, I64, P, P]
        L.bitlinear_ste_backward_weight.restype = S
        L.bitlinear_forward_stall_test.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, S, S, ctypes.c_uint64,
                                                   ctypes.c_int32, P]
        L.bitlinear_forward_stall_test.restype = S
        L.bitlinear_norm_forward.argtypes = [P, S, P, P, I64, I64, S, F, P, S, P]
        L.bitlinear_norm_forward.restype = S
        L.bitlinear_norm_backward_workspace_size.argtypes = [I64, I64]
        L.bitlinear_norm_backward_workspace_size.restype = ctypes.c_size_t
        L.bitlinear_norm_backward.argtypes = [P, S, P, S, P, I64, I64, S, F, P, S, P, P, P, ctypes.c_size_t, P, P]
        L.bitlinear_norm_backward.restype = S
        L.bitlinear_norm_backward_stall_test.argtypes = [P, S, P, S, P, I64, I64, S, F, P, S, P, P, P, ctypes.c_size_t, P,
                                                         ctypes.c_uint64, ctypes.c_int32, P]
        L.bitlinear_norm_backward_stall_test.restype = S
        L.bitlinear_fp8_row_bytes.argtypes = [I64]
        L.bitlinear_fp8_row_bytes.restype = I64
        L.bitlinear_fp8_quantize_act.argtypes = [P, S, I64, I64, F, P, P, P, P, P]
        L.bitlinear_fp8_quantize_act.restype = S
        L.bitlinear_fp8_quantize_weights.argtypes = [P, S, I64, I64, F, P, P, P, P]
        L.bitlinear_fp8_quantize_weights.restype = S
        L.bitlinear_fp8_forward.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, P]
        L.bitlinear_fp8_forward.restype = S
        L.bitlinear_fp8_stall_test.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, ctypes.c_uint64, ctypes.c_int32, P]
        L.bitlinear_fp8_stall_test.restype = S
        L.bitlinear_fp8_backward_input.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, P]
        L.bitlinear_fp8_backward_input.restype = S
        L.bitlinear_fp8_backward_weight.argtypes = [P, P, P, P, I64, I64, I64, P, S, P, P]
        L.bitlinear_fp8_backward_weight.restype = S
        L.bitlinear_last_cuda_error.argtypes = []
        L.bitlinear_last_cuda_error.restype = ctypes.c_int
        L.bitlinear_status_string.argtypes = [ctypes.c_int]
        L.bitlinear_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, dtype, name: str, shape=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _opt(t, name):
    return None if t is None else _dev(t, torch.int32, name, (1,))


def _check(status: int, where: str):
    if status != BL_OK:
        raise BitLinearError(status, where)


def bitlinear_workspace_size(N: int, K: int) -> int:
    return int(lib().bitlinear_workspace_size(N, K))


def bitlinear_quantize_weights(W, eps, gamma_out, packed_out, ws, stream=None):
    N, K = W.shape
    _check(lib().bitlinear_quantize_weights(
        _dev(W, torch.float32, "W"), N, K, float(eps), _dev(gamma_out, torch.float32, "gamma_out", (1,)),
        _dev(packed_out, torch.uint8, "packed_out", (N, K // 4)), _dev(ws, torch.uint8, "ws"),
        ws.numel(), _stream(stream)), "bitlinear_quantize_weights")


def bitlinear_quantize_weights_with_scale(W, gamma, packed_out, stream=None):
    N, K = W.shape
    _check(lib().bitlinear_quantize_weights_with_scale(
        _dev(W, torch.float32, "W"), N, K, _dev(gamma, torch.float32, "gamma", (1,)),
        _dev(packed_out, torch.uint8, "packed_out", (N, K // 4)), _stream(stream)),
        "bitlinear_quantize_weights_with_scale")


def bitlinear_pack(codes, packed_out, err_word=None, stream=None):
    N, K = codes.shape
    _check(lib().bitlinear_pack(
        _dev(codes, torch.int8, "codes"), N, K, _dev(packed_out, torch.uint8, "packed_out", (N, K // 4)),
        _opt(err_word, "err_word"), _stream(stream)), "bitlinear_pack")


def bitlinear_quantize_act(X, eps, xq_out, s_out, stream=None, layout=BL_XQ_ROWMAJOR):
    M, K = X.shape
    args = (_dev(X, torch.bfloat16, "X"), M, K, float(eps), _dev(xq_out, torch.int8, "xq_out", (M, K)),
            _dev(s_out, torch.float32, "s_out", (M,)))
    if layout == BL_XQ_ROWMAJOR:
        _check(lib().bitlinear_quantize_act(*args, _stream(stream)), "bitlinear_quantize_act")
    else:
        _check(lib().bitlinear_quantize_act_layout(*args, int(layout), _stream(stream)),
               "bitlinear_quantize_act_layout")


def bitlinear_norm_quantize_act(X, norm_weight, kind, norm_eps, eps, xq_out, s_out, stream=None,
                                layout=BL_XQ_ROWMAJOR):
    M, K = X.shape
    w = None if norm_weight is None else _dev(norm_weight, torch.float32, "norm_weight", (K,))
    _check(lib().bitlinear_norm_quantize_act(
        _dev(X, torch.bfloat16, "X"), w, M, K, int(kind), float(norm_eps), float(eps),
        _dev(xq_out, torch.int8, "xq_out", (M, K)), _dev(s_out, torch.float32, "s_out", (M,)), int(layout),
        _stream(stream)), "bitlinear_norm_quantize_act")


_OUT_DT = {BL_OUT_F32: torch.float32, BL_OUT_BF16: torch.bfloat16, BL_OUT_I32: torch.int32}


def bitlinear_forward(xq, s, packed, gamma, out, err_word=None, stream=None, path=BL_PATH_AUTO,
                      layout=BL_XQ_ROWMAJOR):
    M, K = xq.shape
    N = packed.shape[0]
    kind = {v: k for k, v in _OUT_DT.items()}.get(out.dtype)
    if kind is None:
        raise TypeError("out must be float32, bfloat16 or int32")
    args = (_dev(xq, torch.int8, "xq"), _dev(s, torch.float32, "s", (M,)),
            _dev(packed, torch.uint8, "packed", (N, K // 4)), _dev(gamma, torch.float32, "gamma", (1,)),
            M, N, K, _dev(out, out.dtype, "out", (M, N)), kind, _opt(err_word, "err_word"))
    if layout != BL_XQ_ROWMAJOR:
        _check(lib().bitlinear_forward_layout(*args, int(layout), int(path), _stream(stream)),
               "bitlinear_forward_layout")
    elif path == BL_PATH_AUTO:
        _check(lib().bitlinear_forward(*args, _stream(stream)), "bitlinear_forward")
    else:
        _check(lib().bitlinear_forward_path(*args, int(path), _stream(stream)), "bitlinear_forward_path")


def bitlinear_forward_stall_test(xq, s, packed, gamma, out, err_word, wait_limit_ns, stall_after_loads,
                                 stream=None, path=BL_PATH_TC_1SM, layout=BL_XQ_ROWMAJOR):
    """The forward with every device wait limited to wait_limit_ns and each block's load
    producer stopped after stall_after_loads loads (a test of the bounded waits)."""
    M, K = xq.shape
    N = packed.shape[0]
    kind = {v: k for k, v in _OUT_DT.items()}.get(out.dtype)
    if kind is None:
        raise TypeError("out must be float32, bfloat16 or int32")
    _check(lib().bitlinear_forward_stall_test(
        _dev(xq, torch.int8, "xq"), _dev(s, torch.float32, "s", (M,)),
        _dev(packed, torch.uint8, "packed", (N, K // 4)), _dev(gamma, torch.float32, "gamma", (1,)),
        M, N, K, _dev(out, out.dtype, "out", (M, N)), kind, _opt(err_word, "err_word"), int(layout), int(path),
        int(wait_limit_ns), int(stall_after_loads), _stream(stream)), "bitlinear_forward_stall_test")


def bitlinear_forward_rowscale(xq, s, packed, gamma_rows, out, err_word=None, stream=None, path=BL_PATH_AUTO,
                               layout=BL_XQ_ROWMAJOR):
    M, K = xq.shape
    N = packed.shape[0]
    kind = {v: k for k, v in _OUT_DT.items()}.get(out.dtype)
    if kind is None:
        raise TypeError("out must be float32, bfloat16 or int32")
    _check(lib().bitlinear_forward_rowscale(
        _dev(xq, torch.int8, "xq"), _dev(s, torch.float32, "s", (M,)),
        _dev(packed, torch.uint8, "packed", (N, K // 4)), _dev(gamma_rows, torch.float32, "gamma_rows", (N,)),
        M, N, K, _dev(out, out.dtype, "out", (M, N)), kind, _opt(err_word, "err_word"), int(layout), int(path),
        _stream(stream)), "bitlinear_forward_rowscale")


def bitlinear_tl5_row_bytes(K):
    return int(lib().bitlinear_tl5_row_bytes(int(K)))


def bitlinear_pack_tl5(codes, tl5_out, err_word=None, stream=None):
    N, K = codes.shape
    _check(lib().bitlinear_pack_tl5(
        _dev(codes, torch.int8, "codes"), N, K, _dev(tl5_out, torch.uint8, "tl5_out", (N, bitlinear_tl5_row_bytes(K))),
        _opt(err_word, "err_word"), _stream(stream)), "bitlinear_pack_tl5")


def bitlinear_repack_tl5(packed, tl5_out, stream=None):
    N, KB = packed.shape
    K = 4 * KB
    _check(lib().bitlinear_repack_tl5(
        _dev(packed, torch.uint8, "packed"), N, K,
        _dev(tl5_out, torch.uint8, "tl5_out", (N, bitlinear_tl5_row_bytes(K))), _stream(stream)),
        "bitlinear_repack_tl5")


def bitlinear_forward_tl5(xq, s, tl5, gamma, out, stream=None):
    M, K = xq.shape
    N = tl5.shape[0]
    kind = {v: k for k, v in _OUT_DT.items()}.get(out.dtype)
    if kind is None:
        raise TypeError("out must be float32, bfloat16 or int32")
    _check(lib().bitlinear_forward_tl5(
        _dev(xq, torch.int8, "xq"), _dev(s, torch.float32, "s", (M,)),
        _dev(tl5, torch.uint8, "tl5", (N, bitlinear_tl5_row_bytes(K))), _dev(gamma, torch.float32, "gamma"),
        M, N, K, _dev(out, out.dtype, "out", (M, N)), kind, _stream(stream)), "bitlinear_forward_tl5")


def bitlinear_ste_backward_input(dY, packed, gamma, dX, stream=None):
    M, N = dY.shape
    K = 4 * packed.shape[1]
    _check(lib().bitlinear_ste_backward_input(
        _dev(dY, torch.float32, "dY"), _dev(packed, torch.uint8, "packed", (N, K // 4)),
        _dev(gamma, torch.float32, "gamma"), M, N, K, _dev(dX, torch.float32, "dX", (M, K)), _stream(stream)),
        "bitlinear_ste_backward_input")


def bitlinear_ste_backward_weight(dY, xq, s, gamma, dW, stream=None):
    M, N = dY.shape
    K = xq.shape[1]
    _check(lib().bitlinear_ste_backward_weight(
        _dev(dY, torch.float32, "dY"), _dev(xq, torch.int8, "xq", (M, K)), _dev(s, torch.float32, "s", (M,)),
        _dev(gamma, torch.float32, "gamma"), M, N, K, _dev(dW, torch.float32, "dW", (N, K)), _stream(stream)),
        "bitlinear_ste_backward_weight")


# The norm and e4m3 calls run on the device of their tensors (all on one), whichever is
# current, and on its current stream or the one given.  A serving loop makes them for single
# tokens, where the host's time counts, so the common case (that device is current, no stream
# given) takes no context manager.

_FLOATS = {torch.float32: BL_OUT_F32, torch.bfloat16: BL_OUT_BF16}
_E4M3 = torch.float8_e4m3fn
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _scope(stream, tensors):
    """A context in which the tensors' device, and `stream` if given, are current."""
    index = None
    for t in tensors:
        if not t.is_cuda:
            raise TypeError("every tensor must be a CUDA tensor")
        if index is None:
            index = t.get_device()
        elif t.get_device() != index:
            raise ValueError("tensors must be on one device, got cuda:%d and cuda:%d" % (index, t.get_device()))
    if index is None:
        raise TypeError("no CUDA tensor given")
    if stream is None:
        return torch.cuda.device(index)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    if stream.device.index != index:
        raise ValueError("the stream is on %s, the tensors on cuda:%d" % (stream.device, index))
    return torch.cuda.stream(stream)


def _scoped(call):
    """Runs `call` in the scope of its tensors: everything passed to it that is one, and the
    keyword argument `stream`, which the call itself then does without."""
    @functools.wraps(call)
    def run(*args, stream=None, **kwargs):
        if stream is None:
            # the common case: every tensor on one device, which is current
            index = None
            for a in (*args, *kwargs.values()) if kwargs else args:
                if isinstance(a, torch.Tensor):
                    i = a.get_device()
                    if index is None:
                        index = i
                    elif i != index:
                        index = -1
                        break
            if index is not None and index >= 0 and index == _device():
                return call(*args, **kwargs)
        with _scope(stream, [a for a in (*args, *kwargs.values()) if isinstance(a, torch.Tensor)]):
            return call(*args, **kwargs)
    return run


def _here(t) -> int:
    """The current stream of the tensor's device."""
    return _raw_stream(t.get_device())


def _ptr(t, dtype, name: str, shape=None) -> int:
    """_dev, with the usual case (nothing to complain about) decided by a few quick tests."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous() and (
            shape is None or t.shape == shape):
        return t.data_ptr()
    return _dev(t, dtype, name, shape)


def _float(t, name: str, shape=None):
    """(pointer, bl_dtype) of an fp32 or bf16 tensor."""
    kind = _FLOATS.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if kind is None:
        raise TypeError("%s must be float32 or bfloat16" % name)
    return _ptr(t, t.dtype, name, shape), kind


def _vec(t, name, K):
    return None if t is None else _ptr(t, torch.float32, name, (K,))


def _matrix(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a matrix" % name)
    return t.shape


def _blocks(n: int) -> int:
    return -(-n // 128)


def _up16(n: int) -> int:
    return -(-n // 16) * 16


@_scoped
def bitlinear_norm_forward(X, norm_weight, norm_bias, kind, norm_eps, out):
    M, K = _matrix(X, "X")
    _check(lib().bitlinear_norm_forward(
        *_float(X, "X"), _vec(norm_weight, "norm_weight", K), _vec(norm_bias, "norm_bias", K), M, K, int(kind),
        float(norm_eps), *_float(out, "out", (M, K)), _here(X)), "bitlinear_norm_forward")


def bitlinear_norm_backward_workspace_size(M: int, K: int) -> int:
    return int(lib().bitlinear_norm_backward_workspace_size(int(M), int(K)))


@_scoped
def bitlinear_norm_backward(dY, X, norm_weight, kind, norm_eps, dX, dweight, dbias, ws, err_word=None):
    M, K = _matrix(X, "X")
    _check(lib().bitlinear_norm_backward(
        *_float(dY, "dY", (M, K)), *_float(X, "X"), _vec(norm_weight, "norm_weight", K), M, K, int(kind),
        float(norm_eps), *_float(dX, "dX", (M, K)), _vec(dweight, "dweight", K), _vec(dbias, "dbias", K),
        None if ws is None else _ptr(ws, torch.uint8, "ws"), 0 if ws is None else ws.numel(),
        _opt(err_word, "err_word"), _here(dY)),
        "bitlinear_norm_backward")


@_scoped
def bitlinear_norm_backward_stall_test(dY, X, norm_weight, kind, norm_eps, dX, dweight, dbias, ws, err_word,
                                       wait_limit_ns, stall_after_loads):
    """The norm's backward with every device wait limited to wait_limit_ns and the loads of each
    block's rows stopped after stall_after_loads of them (a test of the bounded waits)."""
    M, K = _matrix(X, "X")
    _check(lib().bitlinear_norm_backward_stall_test(
        *_float(dY, "dY", (M, K)), *_float(X, "X"), _vec(norm_weight, "norm_weight", K), M, K, int(kind),
        float(norm_eps), *_float(dX, "dX", (M, K)), _vec(dweight, "dweight", K), _vec(dbias, "dbias", K),
        None if ws is None else _ptr(ws, torch.uint8, "ws"), 0 if ws is None else ws.numel(),
        _opt(err_word, "err_word"), int(wait_limit_ns), int(stall_after_loads), _here(dY)),
        "bitlinear_norm_backward_stall_test")


def bitlinear_fp8_row_bytes(K: int) -> int:
    return int(lib().bitlinear_fp8_row_bytes(int(K)))


@_scoped
def bitlinear_fp8_quantize_act(X, eps, xq_out, s_out, xqt_out=None, st_out=None):
    M, K = _matrix(X, "X")
    _check(lib().bitlinear_fp8_quantize_act(
        *_float(X, "X"), M, K, float(eps),
        None if xq_out is None else _ptr(xq_out, _E4M3, "xq_out", (M, _up16(K))),
        None if s_out is None else _ptr(s_out, torch.float32, "s_out", (_blocks(K), M)),
        None if xqt_out is None else _ptr(xqt_out, _E4M3, "xqt_out", (K, _up16(M))),
        None if st_out is None else _ptr(st_out, torch.float32, "st_out", (_blocks(M), K)), _here(X)),
        "bitlinear_fp8_quantize_act")


@_scoped
def bitlinear_fp8_quantize_weights(W, eps, wq_out, s_out, wqt_out=None):
    N, K = _matrix(W, "W")
    _check(lib().bitlinear_fp8_quantize_weights(
        *_float(W, "W"), N, K, float(eps),
        None if wq_out is None else _ptr(wq_out, _E4M3, "wq_out", (N, _up16(K))),
        _ptr(s_out, torch.float32, "s_out", (_blocks(N), _blocks(K))),
        None if wqt_out is None else _ptr(wqt_out, _E4M3, "wqt_out", (K, _up16(N))),
        _here(W)), "bitlinear_fp8_quantize_weights")


def _codes_of(left, right, names, length=None):
    """Rows of two code matrices and the length of the contraction: `length`, or the padded length
    of their rows, which gives the same where the codes behind `length` are zeros, as the
    quantisers leave them."""
    rows_l, n = _matrix(left, names[0])
    rows_r, n_r = _matrix(right, names[1])
    if n != n_r or n % 16 != 0:
        raise ValueError("%s and %s must have rows of the same multiple of 16 codes, got %d and %d"
                         % (*names, n, n_r))
    if length is None:
        return rows_l, rows_r, n
    length = int(length)
    if length < 1 or _up16(length) != n:
        raise ValueError("rows of %d codes do not hold %d and their padding to a multiple of 16" % (n, length))
    return rows_l, rows_r, length


@_scoped
def bitlinear_fp8_forward(xq, sx, wq, sw, out, err_word=None, K=None):
    M, N, K = _codes_of(xq, wq, ("xq", "wq"), K)
    _check(lib().bitlinear_fp8_forward(
        _ptr(xq, _E4M3, "xq"), _ptr(sx, torch.float32, "sx", (_blocks(K), M)), _ptr(wq, _E4M3, "wq"),
        _ptr(sw, torch.float32, "sw", (_blocks(N), _blocks(K))), M, N, K, *_float(out, "out", (M, N)),
        _opt(err_word, "err_word"), _here(xq)), "bitlinear_fp8_forward")


@_scoped
def bitlinear_fp8_stall_test(xq, sx, wq, sw, out, err_word, wait_limit_ns, stall_after_loads):
    """The product with every device wait limited to wait_limit_ns and each block's load
    producer stopped after stall_after_loads loads (a test of the bounded waits)."""
    M, N, K = _codes_of(xq, wq, ("xq", "wq"))
    _check(lib().bitlinear_fp8_stall_test(
        _ptr(xq, _E4M3, "xq"), _ptr(sx, torch.float32, "sx", (_blocks(K), M)), _ptr(wq, _E4M3, "wq"),
        _ptr(sw, torch.float32, "sw", (_blocks(N), _blocks(K))), M, N, K, *_float(out, "out", (M, N)),
        _opt(err_word, "err_word"), int(wait_limit_ns), int(stall_after_loads), _here(xq)),
        "bitlinear_fp8_stall_test")


@_scoped
def bitlinear_fp8_backward_input(dyq, sdy, wqt, sw, dX, err_word=None, N=None):
    M, K, N = _codes_of(dyq, wqt, ("dyq", "wqt"), N)
    _check(lib().bitlinear_fp8_backward_input(
        _ptr(dyq, _E4M3, "dyq"), _ptr(sdy, torch.float32, "sdy", (_blocks(N), M)), _ptr(wqt, _E4M3, "wqt"),
        _ptr(sw, torch.float32, "sw", (_blocks(N), _blocks(K))), M, N, K, *_float(dX, "dX", (M, K)),
        _opt(err_word, "err_word"), _here(dyq)), "bitlinear_fp8_backward_input")


@_scoped
def bitlinear_fp8_backward_weight(dyqt, sdyt, xqt, sxt, dW, err_word=None, M=None):
    N, K, M = _codes_of(dyqt, xqt, ("dyqt", "xqt"), M)
    _check(lib().bitlinear_fp8_backward_weight(
        _ptr(dyqt, _E4M3, "dyqt"), _ptr(sdyt, torch.float32, "sdyt", (_blocks(M), N)), _ptr(xqt, _E4M3, "xqt"),
        _ptr(sxt, torch.float32, "sxt", (_blocks(M), K)), M, N, K, *_float(dW, "dW", (N, K)),
        _opt(err_word, "err_word"), _here(dyqt)), "bitlinear_fp8_backward_weight")


# ----------------------------------------------------------- allocating helpers --

def quantize_weights(W: torch.Tensor, eps: float = 1e-5, stream=None):
    """(gamma [1] fp32, packed [N, K/4] uint8) of an fp32 CUDA weight matrix."""
    N, K = W.shape
    gamma = torch.empty(1, dtype=torch.float32, device=W.device)
    packed = torch.empty(N, K // 4, dtype=torch.uint8, device=W.device)
    ws = torch.empty(max(1, bitlinear_workspace_size(N, K)), dtype=torch.uint8, device=W.device)
    bitlinear_quantize_weights(W, eps, gamma, packed, ws, stream)
    return gamma, packed


def quantize_act(X: torch.Tensor, eps: float = 1e-5, stream=None, layout=BL_XQ_ROWMAJOR):
    """(x_q [M, K] int8, s [M] fp32) of a bf16 CUDA activation matrix."""
    M, K = X.shape
    xq = torch.empty(M, K, dtype=torch.int8, device=X.device)
    s = torch.empty(M, dtype=torch.float32, device=X.device)
    bitlinear_quantize_act(X, eps, xq, s, stream, layout)
    return xq, s


def norm_quantize_act(X: torch.Tensor, norm_weight=None, kind=BL_NORM_RMS, norm_eps: float = 1e-5,
                      eps: float = 1e-5, stream=None, layout=BL_XQ_ROWMAJOR):
    """(x_q [M, K] int8, s [M] fp32) of RMSNorm / LayerNorm(X) for a bf16 CUDA matrix."""
    M, K = X.shape
    xq = torch.empty(M, K, dtype=torch.int8, device=X.device)
    s = torch.empty(M, dtype=torch.float32, device=X.device)
    bitlinear_norm_quantize_act(X, norm_weight, kind, norm_eps, eps, xq, s, stream, layout)
    return xq, s


def forward(xq, s, packed, gamma, out_dtype=torch.float32, stream=None, path=BL_PATH_AUTO, err_word=None,
            layout=BL_XQ_ROWMAJOR):
    """y [M, N] of the BitLinear forward from quantised operands."""
    out = torch.empty(xq.shape[0], packed.shape[0], dtype=out_dtype, device=xq.device)
    bitlinear_forward(xq, s, packed, gamma, out, err_word, stream, path, layout)
    return out


def pack_tl5(codes: torch.Tensor, stream=None):
    """[N, tl5_row_bytes(K)] uint8: int8 codes in the five-per-byte format."""
    N, K = codes.shape
    out = torch.empty(N, bitlinear_tl5_row_bytes(K), dtype=torch.uint8, device=codes.device)
    bitlinear_pack_tl5(codes, out, None, stream)
    return out


def repack_tl5(packed: torch.Tensor, stream=None):
    """[N, tl5_row_bytes(K)] uint8 from the 2-bit format [N, K/4]."""
    N, KB = packed.shape
    out = torch.empty(N, bitlinear_tl5_row_bytes(4 * KB), dtype=torch.uint8, device=packed.device)
    bitlinear_repack_tl5(packed, out, stream)
    return out


def forward_tl5(xq, s, tl5, gamma, out_dtype=torch.float32, stream=None):
    """y [M, N] from row-major x_q and weights in the five-per-byte format."""
    out = torch.empty(xq.shape[0], tl5.shape[0], dtype=out_dtype, device=xq.device)
    bitlinear_forward_tl5(xq, s, tl5, gamma, out, stream)
    return out


def ste_backward(dY, packed, xq, s, gamma, stream=None):
    """(dX [M, K], dW [N, K]) fp32: the straight-through gradients of the forward."""
    M, N = dY.shape
    K = 4 * packed.shape[1]
    dX = torch.empty(M, K, dtype=torch.float32, device=dY.device)
    dW = torch.empty(N, K, dtype=torch.float32, device=dY.device)
    bitlinear_ste_backward_input(dY, packed, gamma, dX, stream)
    bitlinear_ste_backward_weight(dY, xq, s, gamma, dW, stream)
    return dX, dW


# The helpers below take `stream` too (_scoped), and call the entry points' bodies directly:
# their own arguments have been looked at, and what they allocate is on the same device and,
# with a stream, belongs to it.

@_scoped
def norm_forward(X: torch.Tensor, norm_weight=None, norm_bias=None, kind=BL_NORM_RMS, norm_eps: float = 1e-5,
                 out_dtype=None):
    """RMSNorm / LayerNorm(X) [M, K] of an fp32 or bf16 CUDA matrix, as out_dtype (X's by default)."""
    out = X.new_empty(X.shape, dtype=out_dtype or X.dtype)
    bitlinear_norm_forward.__wrapped__(X, norm_weight, norm_bias, kind, norm_eps, out)
    return out


@_scoped
def norm_backward(dY: torch.Tensor, X: torch.Tensor, norm_weight=None, kind=BL_NORM_RMS, norm_eps: float = 1e-5,
                  bias: bool = False, dx_dtype=None, err_word=None):
    """(dX [M, K], dweight [K] fp32, dbias [K] fp32) of norm_forward for the gradient dY at its
    result.  dX is dx_dtype (dY's type by default); dweight is None without a norm_weight,
    dbias unless `bias`."""
    M, K = _matrix(X, "X")
    dX = X.new_empty((M, K), dtype=dx_dtype or dY.dtype)
    dw = X.new_empty(K, dtype=torch.float32) if norm_weight is not None else None
    db = X.new_empty(K, dtype=torch.float32) if bias else None
    n = bitlinear_norm_backward_workspace_size(M, K)
    ws = X.new_empty(n, dtype=torch.uint8) if n else None
    bitlinear_norm_backward.__wrapped__(dY, X, norm_weight, kind, norm_eps, dX, dw, db, ws, err_word)
    return dX, dw, db


@_scoped
def fp8_quantize_act(X: torch.Tensor, eps: float = 1e-5, transposed: bool = False):
    """(xq, sx) of an fp32 or bf16 CUDA matrix: e4m3 codes [M, K rounded up to 16] and one fp32
    scale per 128 elements of a row [ceil(K/128), M].  With `transposed` also (xqt, sxt), the
    codes [K, M rounded up to 16] with one scale per 128 elements of a column."""
    M, K = _matrix(X, "X")
    out = (X.new_empty((M, _up16(K)), dtype=_E4M3), X.new_empty((_blocks(K), M), dtype=torch.float32))
    if transposed:
        out += (X.new_empty((K, _up16(M)), dtype=_E4M3), X.new_empty((_blocks(M), K), dtype=torch.float32))
    bitlinear_fp8_quantize_act.__wrapped__(X, eps, *out)
    return out


@_scoped
def fp8_quantize_weights(W: torch.Tensor, eps: float = 1e-5, transposed: bool = False):
    """(wq, sw) of an fp32 or bf16 CUDA weight matrix: e4m3 codes [N, K rounded up to 16] and one
    fp32 scale per 128 x 128 block.  With `transposed` also wqt, the codes [K, N rounded up to 16]."""
    N, K = _matrix(W, "W")
    out = (W.new_empty((N, _up16(K)), dtype=_E4M3), W.new_empty((_blocks(N), _blocks(K)), dtype=torch.float32))
    if transposed:
        out += (W.new_empty((K, _up16(N)), dtype=_E4M3),)
    bitlinear_fp8_quantize_weights.__wrapped__(W, eps, *out)
    return out


@_scoped
def fp8_forward(xq, sx, wq, sw, out_dtype=torch.float32, err_word=None, K=None):
    """y [M, N] = x w^T from the codes and scales of fp8_quantize_act and fp8_quantize_weights.
    Without K, whole rows of codes are contracted: what pads them to a multiple of 16 must be
    zeros (the quantisers' is).  With K it is not read."""
    out = sx.new_empty((xq.shape[0], wq.shape[0]), dtype=out_dtype)
    bitlinear_fp8_forward.__wrapped__(xq, sx, wq, sw, out, err_word, K)
    return out


@_scoped
def fp8_backward_input(dyq, sdy, wqt, sw, out_dtype=torch.float32, err_word=None, N=None):
    """dX [M, K] = dY w from the gradient's codes and the transposed weight codes.  Without N, what
    pads their rows must be zeros (see fp8_forward)."""
    dX = sdy.new_empty((dyq.shape[0], wqt.shape[0]), dtype=out_dtype)
    bitlinear_fp8_backward_input.__wrapped__(dyq, sdy, wqt, sw, dX, err_word, N)
    return dX


@_scoped
def fp8_backward_weight(dyqt, sdyt, xqt, sxt, out_dtype=torch.float32, err_word=None, M=None):
    """dW [N, K] = dY^T x from the transposed codes of the gradient and the activations.  Without M,
    what pads their rows must be zeros (see fp8_forward)."""
    dW = sdyt.new_empty((dyqt.shape[0], xqt.shape[0]), dtype=out_dtype)
    bitlinear_fp8_backward_weight.__wrapped__(dyqt, sdyt, xqt, sxt, dW, err_word, M)
    return dW
