"""The mixture-of-experts operators: the router, and the experts' gated
feed-forward for few tokens from block-scaled e4m3 weights (include/int8mm.h,
"Mixture of experts").

    up, up_scale = fp8_quantize_experts(W_up)          # [E,K,2I], once, offline
    down, down_scale = fp8_quantize_experts(W_down)    # [E,I,K]
    Y, H = fp8_sandwich_norm(X, R, post, pre, quantize=False)
    experts, weights = moe_route(Y, W_router, top_k=8)
    Z = fp8_moe(Y, experts, weights, up, up_scale, down, down_scale)

Serving operators: their results carry no gradient.  Devices and streams as in
fp8.py.
"""
from __future__ import annotations

import functools

import torch

from . import _check, load
from .fp8 import (_E4M3, _HALVES, _TYPES, _at, _blocks, _current, _elsewhere, _stream_of, _tensor,
                  fp8_kpad)

__all__ = ["MOE_MAX_EXPERTS", "MOE_MAX_TOP_K", "MOE_MAX_PAIRS", "moe_route", "fp8_moe",
           "fp8_pack_experts", "fp8_quantize_experts"]

MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 1024, 32
MOE_MAX_PAIRS = 8192  # tokens * top_k of one fp8_moe call
_I32, _F32 = (torch.int32,), (torch.float32,)


# a foreign call of 1 us for what a loop asks again and again
@functools.lru_cache(maxsize=256)
def _route_bytes(M, K, E, top_k):
    return load().moe_route_workspace_size(M, K, E, top_k)


@functools.lru_cache(maxsize=256)
def _moe_bytes(M, K, I, E, top_k):
    return load().fp8_moe_workspace_size(M, K, I, E, top_k)


def fp8_pack_experts(Wq: torch.Tensor, stream=None) -> torch.Tensor:
    """e4m3 weights [E,N,K] row-major (a checkpoint's experts, with scales [E,
    ceil(N/128), ceil(K/128)]) -> each expert in the packed layout, as an e4m3
    tensor [E, N, fp8_kpad(K)] (an opaque buffer)."""
    _tensor(Wq, "Wq", (_E4M3,), 3)
    if _elsewhere(Wq, stream):
        with _current(Wq, stream):
            return fp8_pack_experts(Wq)
    E, N, K = Wq.shape
    out = torch.empty((E, N, fp8_kpad(K)), dtype=_E4M3, device=Wq.device)
    on = _stream_of(Wq.get_device())
    for e in range(E):
        _check(load().fp8_pack_weight(_at(Wq[e]), N, K, _at(out[e]), on))
    return out


def fp8_quantize_experts(W: torch.Tensor, stream=None):
    """W fp16 or bf16 [E,K,N] -> (packed e4m3 [E, N, fp8_kpad(K)], scales fp32
    [E, ceil(N/128), ceil(K/128)]), each expert as by fp8_quantize_weight."""
    _tensor(W, "W", _HALVES, 3)
    if _elsewhere(W, stream):
        with _current(W, stream):
            return fp8_quantize_experts(W)
    E, K, N = W.shape
    W_f8 = torch.empty((E, N, fp8_kpad(K)), dtype=_E4M3, device=W.device)
    w_scale = torch.empty((E, _blocks(N), _blocks(K)), dtype=torch.float32, device=W.device)
    on = _stream_of(W.get_device())
    one = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=W.device)
    for e in range(E):
        # an expert's scales need not start at a multiple of 16 bytes
        _check(load().fp8_quantize_weight(_at(W[e]), _TYPES[W.dtype], K, N, _at(W_f8[e]), _at(one),
                                          on))
        w_scale[e] = one
    return W_f8, w_scale


def moe_route(X: torch.Tensor, W: torch.Tensor, top_k: int, normalize: bool = True, out=None,
              stream=None):
    """The experts of each token of X [M,K] by the router W [E,K], both fp16 or
    both bf16: (experts int32 [M, top_k] in descending order of their logits,
    ties to the lower index; weights fp32 [M, top_k], their softmax over all
    experts, divided by its sum over the chosen ones with `normalize`).  `out`:
    such a pair to write into."""
    _tensor(X, "X", _HALVES, 2)
    if _elsewhere(X, stream):
        with _current(X, stream, W, *(out or ())):
            return moe_route(X, W, top_k, normalize, out)
    M, K = X.shape
    dev = X.device
    _tensor(W, "W", (X.dtype,), (None, K), dev)
    E = W.shape[0]
    if not 0 <= top_k <= MOE_MAX_TOP_K:  # not a size to allocate
        raise ValueError(f"top_k must be 1 to {MOE_MAX_TOP_K}, got {top_k}")
    if out is None:
        # sizes by themselves and empty_like: 0.4 us less each than a tuple of sizes
        experts = torch.empty(M, top_k, dtype=torch.int32, device=dev)
        weights = torch.empty_like(experts, dtype=torch.float32)
    else:
        experts = _tensor(out[0], "out[0]", _I32, (M, top_k), dev)
        weights = _tensor(out[1], "out[1]", _F32, (M, top_k), dev)
    size = _route_bytes(M, K, E, top_k)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(load().moe_route(_at(X), _at(W), _TYPES[X.dtype], M, K, E, top_k, bool(normalize),
                            _at(experts), _at(weights), _at(ws), size, _stream_of(X.get_device())))
    return experts, weights


def fp8_moe(X: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, gate_up: torch.Tensor,
            gate_up_scale: torch.Tensor, down: torch.Tensor, down_scale: torch.Tensor,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [M,K] = for each token of X [M,K] (fp16 or bf16) the sum over its places
    j of weights[m,j] * (silu(x . G^T) * (x . U^T)) . D^T with the matrices of
    the expert experts[m,j]; an expert outside 0 .. E-1 contributes nothing.
    gate_up [E, 2I, fp8_kpad(K)] (I gates, then I ups) and down [E, K,
    fp8_kpad(I)] as fp8_pack_experts or fp8_quantize_experts leaves them, with
    their scales [E, ceil(2I/128), ceil(K/128)] and [E, ceil(K/128),
    ceil(I/128)].  At most MOE_MAX_PAIRS pairs of a token and a place."""
    _tensor(X, "X", _HALVES, 2)
    if _elsewhere(X, stream):
        with _current(X, stream, experts, weights, gate_up, gate_up_scale, down, down_scale, out):
            return fp8_moe(X, experts, weights, gate_up, gate_up_scale, down, down_scale, out)
    M, K = X.shape
    dev = X.device
    top_k = _tensor(experts, "experts", _I32, 2, dev).shape[1]
    if experts.shape[0] != M:
        raise ValueError(f"experts has {experts.shape[0]} rows, X {M}")
    _tensor(weights, "weights", _F32, (M, top_k), dev)
    E, I2, columns = _tensor(gate_up, "gate_up", (_E4M3,), 3, dev).shape
    if I2 % 2 or columns != fp8_kpad(K):
        raise ValueError(f"gate_up must have an even number of rows and {fp8_kpad(K)} columns, "
                         f"got {I2} and {columns}")
    I = I2 // 2
    _tensor(gate_up_scale, "gate_up_scale", _F32, (E, _blocks(I2), _blocks(K)), dev)
    _tensor(down, "down", (_E4M3,), (E, K, fp8_kpad(I)), dev)
    _tensor(down_scale, "down_scale", _F32, (E, _blocks(K), _blocks(I)), dev)
    if out is None:
        out = torch.empty_like(X)
    else:
        _tensor(out, "out", (X.dtype,), (M, K), dev)
    size = _moe_bytes(M, K, I, E, top_k)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(load().fp8_moe(_at(X), _TYPES[X.dtype], M, K, _at(experts), _at(weights), top_k,
                          _at(gate_up), _at(gate_up_scale), _at(down), _at(down_scale), I, E,
                          _at(out), _at(ws), size, _stream_of(X.get_device())))
    return out
