"""Torch modules over the C-ABI: an fp16 linear layer whose forward pass is
the LLM.int8() decomposed matmul, and its block-scaled e4m3 counterpart with
the norm that feeds it.

The layer of the brain.gartu.xyz page's practical example ("Exemple
pratique") replaces an nn.Linear (with bias) by an int8 layer with
threshold 6.0 whose forward pass does the mixed-precision decomposition by
itself; this is that layer for this library.  Weights are quantized once,
when the module is built.  All arithmetic runs in the HIP library.
"""
from __future__ import annotations

import torch

from . import (FP8_BLOCK, build_outlier_cache, fp8_matmul, fp8_pack_weight, fp8_quantize,
               fp8_quantize_weight, fp8_rms_norm, mixed_matmul, mixed_matmul_cached,
               quantize_weight, workspace_size)

_HALVES = (torch.float16, torch.bfloat16)


class Int8MixedLinear(torch.nn.Module):
    """y = x . W^T + b for fp16 x [..., in_features] on the GPU.

    Buffers: w_i8 (packed int8 weights), w_absmax (fp32 [out]), the source
    of the outlier rows -- either w_kn (the fp16 weights as [in, out]) or,
    with `outlier_dims` given, cache (the fp16 rows of those static dims
    only; dims outside it fall back to dequantized int8 rows and are
    flagged) -- and bias (fp16 [out] or None).  `threshold` is the outlier
    threshold alpha; `n_cap` bounds the outlier columns per call
    (in_features, always enough, by default).
    """

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None,
                 threshold: float = 6.0, n_cap: int | None = None, outlier_dims=None):
        super().__init__()
        if weight.dim() != 2 or weight.device.type != "cuda":
            raise TypeError("weight must be a 2-D CUDA tensor [out_features, in_features]")
        out_features, in_features = weight.shape
        w_kn = weight.detach().to(torch.float16).t().contiguous()
        w_i8, w_absmax = quantize_weight(w_kn)
        self.register_buffer("w_i8", w_i8)
        self.register_buffer("w_absmax", w_absmax)
        if outlier_dims is None:
            self.register_buffer("w_kn", w_kn)
            self.register_buffer("cache", None)
        else:
            # memory-lean: only the fp16 rows of the static outlier dims stay
            self.register_buffer("w_kn", None)
            self.register_buffer("cache", build_outlier_cache(w_kn, outlier_dims))
            del w_kn
        if bias is not None:
            bias = bias.detach().to(device=weight.device, dtype=torch.float16).contiguous()
        self.register_buffer("bias", bias)
        self.in_features = in_features
        self.out_features = out_features
        self.threshold = float(threshold)
        self.n_cap = in_features if n_cap is None else int(n_cap)

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, threshold: float = 6.0,
                    n_cap: int | None = None, outlier_dims=None) -> "Int8MixedLinear":
        return cls(linear.weight, linear.bias, threshold, n_cap, outlier_dims)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, threshold={self.threshold}, n_cap={self.n_cap}")

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        x2 = x.reshape(-1, self.in_features)
        if x2.dtype != torch.float16 or not x2.is_contiguous():
            x2 = x2.to(torch.float16).contiguous()
        M = x2.shape[0]
        # the caching allocator makes the per-call workspace cheap and
        # keeps concurrent calls on different streams apart
        ws = torch.empty(workspace_size(M, self.in_features, self.out_features, self.n_cap),
                         dtype=torch.uint8, device=x2.device)
        if self.cache is None:
            y = mixed_matmul(x2, self.w_i8, self.w_absmax, self.w_kn, alpha=self.threshold,
                             bias=self.bias, n_cap=self.n_cap, workspace=ws)
        else:
            y = mixed_matmul_cached(x2, self.w_i8, self.w_absmax, self.cache,
                                    alpha=self.threshold, bias=self.bias, n_cap=self.n_cap,
                                    workspace=ws)
        return y.reshape(*x.shape[:-1], self.out_features)


class Fp8RMSNorm(torch.nn.Module):
    """The root-mean-square norm in front of Fp8BlockLinear layers, with the
    residual's addition: forward(x, residual) gives ((e4m3, scales), h) with
    h = x + residual, forward(x) the pair (e4m3, scales) alone.  x [..., K] of
    the weight's type, which half() and bfloat16() change; the pair is 2-D, one
    row per token, and every Fp8BlockLinear that reads this norm takes it as it is.
    """

    def __init__(self, weight: torch.Tensor, eps: float = 1e-6):
        super().__init__()
        if weight.dim() != 1 or weight.device.type != "cuda":
            raise TypeError("weight must be a 1-D CUDA tensor")
        self.register_buffer("weight", weight.detach().clone())
        self.eps = float(eps)

    def _apply(self, fn, recurse=True):
        # half() and bfloat16() change the weight's type; float() and the like,
        # to a type that the operator does not take, only move it
        held = self.weight
        super()._apply(fn, recurse)
        if self.weight.dtype != held.dtype and self.weight.dtype not in _HALVES:
            self.weight = held.to(self.weight.device)
        return self

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        K = self.weight.numel()
        if x.shape[-1] != K:
            raise ValueError(f"expected last dimension {K}, got {x.shape[-1]}")
        x2 = x.reshape(-1, K).contiguous()
        if residual is None:
            return fp8_rms_norm(x2, self.weight, eps=self.eps)
        if residual.shape != x.shape:
            raise ValueError(f"residual {tuple(residual.shape)}, x {tuple(x.shape)}")
        q, s, h = fp8_rms_norm(x2, self.weight, eps=self.eps,
                               residual=residual.reshape(-1, K).contiguous())
        return (q, s), h.reshape(x.shape)


class Fp8BlockLinear(torch.nn.Module):
    """y = x . W^T + b with block-scaled e4m3 weights (quantized once, when the
    module is built) and activations (quantized per call).

    x: fp16 or bf16 [..., in_features], or the pair (e4m3 [M, in_features],
    scales) that Fp8RMSNorm, fp8_quantize or fp8_silu_mul leaves; then y is
    [M, out_features].  y is of the module's 16-bit type, the weight's at
    first; half() and bfloat16() change it, and never the weights.  Buffers: w_f8 (packed), w_scale, bias or None.  For serving: y
    carries no gradient.
    """

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None):
        super().__init__()
        if weight.dim() != 2 or weight.device.type != "cuda":
            raise TypeError("weight must be a 2-D CUDA tensor [out_features, in_features]")
        if weight.dtype not in _HALVES:
            raise TypeError(f"weight must be fp16 or bf16, got {weight.dtype}")
        w_f8, w_scale = fp8_quantize_weight(weight.detach().t().contiguous())
        self._set(w_f8, w_scale, weight.shape[1], weight.dtype, bias)

    def _set(self, w_f8, w_scale, in_features, dtype, bias):
        self.register_buffer("w_f8", w_f8)
        self.register_buffer("w_scale", w_scale)
        if bias is not None:
            if bias.shape != w_f8.shape[:1]:
                raise ValueError(f"bias must have shape {tuple(w_f8.shape[:1])}, got {tuple(bias.shape)}")
            bias = bias.detach().to(device=w_f8.device, dtype=dtype).contiguous()
        self.register_buffer("bias", bias)
        self.in_features, self.out_features = in_features, w_f8.shape[0]
        self.dtype = dtype

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear) -> "Fp8BlockLinear":
        return cls(linear.weight, linear.bias)

    @classmethod
    def from_quantized(cls, weight: torch.Tensor, w_scale: torch.Tensor,
                       bias: torch.Tensor | None = None,
                       dtype: torch.dtype = torch.bfloat16) -> "Fp8BlockLinear":
        """A checkpoint's e4m3 weight [out, in] with its scales
        [ceil(out/128), ceil(in/128)]; y is of `dtype`, fp16 or bf16."""
        if weight.dim() != 2:
            raise TypeError("weight must be a 2-D CUDA tensor [out_features, in_features]")
        if dtype not in _HALVES:
            raise TypeError(f"dtype must be fp16 or bf16, got {dtype}")
        blocks = tuple((n + FP8_BLOCK - 1) // FP8_BLOCK for n in weight.shape)
        if w_scale.shape != blocks:
            raise ValueError(f"w_scale must have shape {blocks}, got {tuple(w_scale.shape)}")
        self = cls.__new__(cls)
        torch.nn.Module.__init__(self)
        w_scale = w_scale.detach().to(device=weight.device, dtype=torch.float32).contiguous()
        self._set(fp8_pack_weight(weight.detach()), w_scale, weight.shape[1], dtype, bias)
        return self

    def _apply(self, fn, recurse=True):
        # half(), to(torch.bfloat16) and the like choose the type of y and bias;
        # the e4m3 numbers and their fp32 scales only follow to another device
        held, bias = {"w_f8": self.w_f8, "w_scale": self.w_scale}, self.bias
        probe = fn(torch.empty(0, dtype=self.dtype, device=self.w_f8.device))
        super()._apply(fn, recurse)
        for name, t in held.items():
            if getattr(self, name).dtype != t.dtype:
                setattr(self, name, t.to(getattr(self, name).device))
        if probe.dtype in _HALVES:
            self.dtype = probe.dtype
        if bias is not None and self.bias.dtype != self.dtype:  # from the bias as it was
            self.bias = bias.to(device=self.bias.device, dtype=self.dtype)
        return self

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, dtype={self.dtype}")

    def forward(self, x) -> torch.Tensor:
        pair = not isinstance(x, torch.Tensor)
        # for pairs too: the packed weight holds in_features only rounded up to
        # 128, so the product takes another width as it comes
        width = (x[0] if pair else x).shape[-1]
        if width != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {width}")
        if pair:
            q, s = x
            return fp8_matmul(q, s, self.w_f8, self.w_scale, bias=self.bias, out_dtype=self.dtype)
        q, s = fp8_quantize(x.reshape(-1, self.in_features).contiguous())
        y = fp8_matmul(q, s, self.w_f8, self.w_scale, bias=self.bias, out_dtype=self.dtype)
        return y.reshape(*x.shape[:-1], self.out_features)


__all__ = ["Int8MixedLinear", "Fp8BlockLinear", "Fp8RMSNorm"]
