"""The block-scaled 8-bit floating-point operators: e4m3 numbers with one fp32
scale per block of 128 columns (include/int8mm.h, "Block-scaled 8-bit floating
point").

    W_f8, w_scale = fp8_quantize_weight(W)                  # once, offline
    X_f8, x_scale, H = fp8_rms_norm(X, g, residual=R)       # or fp8_quantize(X)
    GU = fp8_matmul(X_f8, x_scale, W_f8, w_scale)
    A_f8, a_scale = fp8_silu_mul(GU)

Activations and weights are fp16 or bf16; e4m3 tensors are
torch.float8_e4m3fn.  Serving operators: their results carry no gradient.
Each call runs on the device of its first tensor, on that device's current
stream unless `stream` is given; buffers a call allocates are allocated on
its stream, and tensors given to a call with a `stream` may be dropped as soon
as it returns, as with any other call.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _check, load

__all__ = ["FP8_BLOCK", "fp8_kpad", "fp8_pack_weight", "fp8_quantize_weight", "fp8_quantize",
           "fp8_rms_norm", "fp8_silu_mul", "fp8_matmul", "fp8_matmul_config"]

FP8_BLOCK = 128
_E4M3 = torch.float8_e4m3fn
_TYPES = {torch.float16: 0, torch.bfloat16: 1}  # int8mm_type
_HALVES = tuple(_TYPES)


def fp8_kpad(K: int) -> int:
    """K rounded up to the 128-column blocks of the packed e4m3 layout."""
    return (K + 127) // 128 * 128


def _blocks(n: int) -> int:
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


def _tensor(t, name: str, dtypes, shape, device=None):
    """A contiguous GPU tensor of one of `dtypes` and of `shape` (its first
    size None: any), or with `shape` dimensions, on `device` if given."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    have = t.shape
    if (len(have) != shape if isinstance(shape, int) else have != shape and (
            len(have) != len(shape) or shape[0] is not None or have[1:] != shape[1:])):
        want = (None,) * shape if isinstance(shape, int) else shape
        want = tuple("any" if w is None else w for w in want)
        raise ValueError(f"{name} must have shape {want}, got {tuple(have)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call on {device}")
    return t


# The current stream's handle on a device; torch.cuda.current_stream builds an
# object around it first (3 us of a single-token call's 13)
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere(t, stream) -> bool:
    """Whether a call on t's device (and `stream`) has to make them current first."""
    return stream is not None or t.get_device() != _device_now()


@contextlib.contextmanager
def _current(t, stream, *others):
    """t's device and `stream` made current for a call on t and `others`."""
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        yield
    if stream is not None:
        # the allocator gives a tensor's memory away in the order of the stream
        # it was allocated on: not before this one is through with it either
        for u in (t, *others):
            if u is not None:
                u.record_stream(stream)


def _at(t):
    """The address the library takes; None for an absent or empty tensor."""
    return None if t is None else t.data_ptr() or None


def _quantized(out, M, K, device, like=None):
    """The (e4m3 [M, K], scales [ceil(K/128), M]) a quantizer writes: `out`, or
    new (empty_like, where a tensor of that shape is at hand, is the faster call)."""
    if out is None:
        return (torch.empty((M, K), dtype=_E4M3, device=device) if like is None
                else torch.empty_like(like, dtype=_E4M3),
                torch.empty((_blocks(K), M), dtype=torch.float32, device=device))
    q, s = out
    return (_tensor(q, "out[0]", (_E4M3,), (M, K), device),
            _tensor(s, "out[1]", (torch.float32,), (_blocks(K), M), device))


def fp8_pack_weight(Wq: torch.Tensor, stream=None) -> torch.Tensor:
    """e4m3 weights [N,K] row-major (a checkpoint's, with scales [ceil(N/128),
    ceil(K/128)]) -> the packed layout, as an e4m3 tensor [N, fp8_kpad(K)] (an
    opaque buffer)."""
    _tensor(Wq, "Wq", (_E4M3,), 2)
    if _elsewhere(Wq, stream):
        with _current(Wq, stream):
            return fp8_pack_weight(Wq)
    N, K = Wq.shape
    out = torch.empty((N, fp8_kpad(K)), dtype=_E4M3, device=Wq.device)
    _check(load().fp8_pack_weight(_at(Wq), N, K, _at(out), _stream_of(Wq.get_device())))
    return out


def fp8_quantize_weight(W: torch.Tensor, stream=None):
    """W fp16 or bf16 [K,N] -> (W_f8 packed e4m3 [N, fp8_kpad(K)], w_scale fp32
    [ceil(N/128), ceil(K/128)]), one scale per 128 x 128 block."""
    _tensor(W, "W", _HALVES, 2)
    if _elsewhere(W, stream):
        with _current(W, stream):
            return fp8_quantize_weight(W)
    K, N = W.shape
    W_f8 = torch.empty((N, fp8_kpad(K)), dtype=_E4M3, device=W.device)
    w_scale = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=W.device)
    _check(load().fp8_quantize_weight(_at(W), _TYPES[W.dtype], K, N, _at(W_f8), _at(w_scale),
                                      _stream_of(W.get_device())))
    return W_f8, w_scale


def fp8_quantize(X: torch.Tensor, out=None, stream=None):
    """X fp16 or bf16 [M,K] -> (X_f8 e4m3 [M,K], x_scale fp32 [ceil(K/128), M]).
    `out`: such a pair to write into."""
    _tensor(X, "X", _HALVES, 2)
    if _elsewhere(X, stream):
        with _current(X, stream, *(out or ())):
            return fp8_quantize(X, out=out)
    M, K = X.shape
    X_f8, x_scale = _quantized(out, M, K, X.device, X)
    _check(load().fp8_quantize(_at(X), _TYPES[X.dtype], M, K, _at(X_f8), _at(x_scale),
                               _stream_of(X.get_device())))
    return X_f8, x_scale


def fp8_rms_norm(X: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: torch.Tensor | None = None,
                 residual_out: torch.Tensor | None = None, out=None, stream=None):
    """The quantized root-mean-square norm of X [M,K] with weight [K]:
    (X_f8, x_scale), or with `residual` [M,K], whose sum with X (rounded to
    their type) is normed instead, (X_f8, x_scale, H) with H that sum.
    `residual_out` takes H; it may be `residual` itself."""
    _tensor(X, "X", _HALVES, 2)
    if _elsewhere(X, stream):
        with _current(X, stream, weight, residual, residual_out, *(out or ())):
            return fp8_rms_norm(X, weight, eps, residual, residual_out, out)
    M, K = X.shape
    _tensor(weight, "weight", (X.dtype,), (K,), X.device)
    if residual is not None:
        _tensor(residual, "residual", (X.dtype,), (M, K), X.device)
        if residual_out is not None:
            _tensor(residual_out, "residual_out", (X.dtype,), (M, K), X.device)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    X_f8, x_scale = _quantized(out, M, K, X.device, X)
    H = residual_out
    if residual is not None and H is None:
        H = torch.empty_like(X)
    _check(load().fp8_rms_norm(_at(X), _at(residual), _at(weight), _TYPES[X.dtype], M, K,
                               float(eps), _at(H), _at(X_f8), _at(x_scale),
                               _stream_of(X.get_device())))
    return (X_f8, x_scale) if residual is None else (X_f8, x_scale, H)


def fp8_silu_mul(gate_up: torch.Tensor, out=None, stream=None):
    """gate_up fp16 or bf16 [M,2K] (K gates, then K ups) -> the quantized
    silu(gate) * up: (A_f8 e4m3 [M,K], a_scale fp32 [ceil(K/128), M])."""
    _tensor(gate_up, "gate_up", _HALVES, 2)
    if _elsewhere(gate_up, stream):
        with _current(gate_up, stream, *(out or ())):
            return fp8_silu_mul(gate_up, out=out)
    M, K2 = gate_up.shape
    if K2 % 2:
        raise ValueError(f"gate_up must have an even number of columns, got {K2}")
    K = K2 // 2
    A_f8, a_scale = _quantized(out, M, K, gate_up.device)
    _check(load().fp8_silu_mul(_at(gate_up), _TYPES[gate_up.dtype], M, K, _at(A_f8), _at(a_scale),
                               _stream_of(gate_up.get_device())))
    return A_f8, a_scale


def fp8_matmul(X_f8: torch.Tensor, x_scale: torch.Tensor, W_f8: torch.Tensor,
               w_scale: torch.Tensor, bias: torch.Tensor | None = None,
               out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Y [M,N] = the block-scaled product of X_f8 [M,K] (with x_scale
    [ceil(K/128), M]) and the packed W_f8 [N, fp8_kpad(K)] (with w_scale
    [ceil(N/128), ceil(K/128)]), plus `bias` [N].  Y and bias are of
    `out_dtype` (fp16 or bf16; by default that of `out`, else of bias, else bf16)."""
    _tensor(X_f8, "X_f8", (_E4M3,), 2)
    if _elsewhere(X_f8, stream):
        with _current(X_f8, stream, x_scale, W_f8, w_scale, bias, out):
            return fp8_matmul(X_f8, x_scale, W_f8, w_scale, bias, out_dtype, out)
    M, K = X_f8.shape
    dev = X_f8.device
    _tensor(x_scale, "x_scale", (torch.float32,), (_blocks(K), M), dev)
    _tensor(W_f8, "W_f8", (_E4M3,), (None, fp8_kpad(K)), dev)
    N = W_f8.shape[0]
    _tensor(w_scale, "w_scale", (torch.float32,), (_blocks(N), _blocks(K)), dev)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else bias.dtype if bias is not None else torch.bfloat16
    if out_dtype not in _TYPES:
        raise TypeError(f"out_dtype must be {' or '.join(map(str, _TYPES))}, got {out_dtype}")
    if bias is not None:
        _tensor(bias, "bias", (out_dtype,), (N,), dev)
    if out is not None:
        _tensor(out, "out", (out_dtype,), (M, N), dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    _check(load().fp8_matmul(_at(X_f8), _at(x_scale), M, K, _at(W_f8), _at(w_scale), N, _at(bias),
                             _TYPES[out_dtype], _at(out), _stream_of(X_f8.get_device())))
    return out


def fp8_matmul_config(M: int, N: int, K: int):
    """What fp8_matmul launches for these sizes on the current device:
    ("decode", feature blocks of 16 per workgroup, token blocks of 16),
    ("tiled", BM, BN, stages), or ("split", n1, BM, stages): features below n1
    in 256x256 tiles, the rest in a second launch of BM x 128 tiles."""
    cfg = (ctypes.c_int32 * 4)()
    _check(load().fp8_matmul_config(M, N, K, cfg))
    if cfg[0] == 0:
        return ("decode", int(cfg[1]), int(cfg[2]))
    return (("tiled", "split")[cfg[0] - 1], int(cfg[1]), int(cfg[2]), int(cfg[3]))
