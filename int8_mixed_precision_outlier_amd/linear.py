"""Torch modules over the C-ABI: an fp16 linear layer whose forward pass is
the LLM.int8() decomposed matmul, its block-scaled e4m3 counterpart with the
norms that feed it, and a mixture of experts with block-scaled e4m3 weights.

The layer of the brain.gartu.xyz page's practical example ("Exemple
pratique") replaces an nn.Linear (with bias) by an int8 layer with
threshold 6.0 whose forward pass does the mixed-precision decomposition by
itself; this is that layer for this library.  Weights are quantized once,
when the module is built.  All arithmetic runs in the HIP library.
"""
from __future__ import annotations

import torch

from . import (FP8_BLOCK, MOE_MAX_EXPERTS, MOE_MAX_PAIRS, MOE_MAX_TOP_K, build_outlier_cache,
               fp8_matmul, fp8_moe, fp8_pack_experts, fp8_pack_weight, fp8_quantize,
               fp8_quantize_weight, fp8_rms_norm, fp8_sandwich_norm, mixed_matmul,
               mixed_matmul_cached, moe_route, quantize_weight, workspace_size)

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


class Fp8SandwichNorm(torch.nn.Module):
    """The norm after a block, the residual's addition and the norm before the
    next block: forward(x, residual, gate=None) for a block's output x gives
    (y, h) with h = residual_scale * residual + gate * norm(x), the next residual,
    and y = norm(h): with `quantize` the pair (e4m3, scales) that Fp8BlockLinear
    layers take, else a tensor like x, as Fp8MoE takes it.  x [..., K] of the
    weights' type, which half() and bfloat16() change; gate [K], or [G, K] with G
    dividing the tokens, a row for each of G equal parts of them in turn.
    """

    def __init__(self, post_weight: torch.Tensor, pre_weight: torch.Tensor, eps: float = 1e-6,
                 residual_scale: float = 1.0, quantize: bool = True):
        super().__init__()
        for name, w in (("post_weight", post_weight), ("pre_weight", pre_weight)):
            if w.dim() != 1 or w.device.type != "cuda":
                raise TypeError(f"{name} must be a 1-D CUDA tensor")
        if post_weight.shape != pre_weight.shape or post_weight.dtype != pre_weight.dtype:
            raise ValueError("post_weight and pre_weight must have one shape and type")
        self.register_buffer("post_weight", post_weight.detach().clone())
        self.register_buffer("pre_weight", pre_weight.detach().clone())
        self.eps, self.residual_scale = float(eps), float(residual_scale)
        self.quantize = bool(quantize)

    def _apply(self, fn, recurse=True):
        # as Fp8RMSNorm: float() and the like only move the weights
        held = {"post_weight": self.post_weight, "pre_weight": self.pre_weight}
        super()._apply(fn, recurse)
        for name, t in held.items():
            now = getattr(self, name)
            if now.dtype != t.dtype and now.dtype not in _HALVES:
                setattr(self, name, t.to(now.device))
        return self

    def forward(self, x: torch.Tensor, residual: torch.Tensor, gate: torch.Tensor | None = None):
        K = self.post_weight.numel()
        if x.shape[-1] != K:
            raise ValueError(f"expected last dimension {K}, got {x.shape[-1]}")
        if residual.shape != x.shape:
            raise ValueError(f"residual {tuple(residual.shape)}, x {tuple(x.shape)}")
        out = fp8_sandwich_norm(x.reshape(-1, K).contiguous(), residual.reshape(-1, K).contiguous(),
                                self.post_weight, self.pre_weight,
                                gate=None if gate is None else gate.contiguous(),
                                residual_scale=self.residual_scale, eps=self.eps,
                                quantize=self.quantize)
        y = out[:2] if self.quantize else out[0].reshape(x.shape)
        return y, out[-1].reshape(x.shape)


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


class Fp8MoE(torch.nn.Module):
    """A mixture of experts with gated feed-forwards, for few tokens at a time: y
    = sum over a token's top_k experts, by the router, of p_e * D_e (silu(G_e x) *
    U_e x).  x [..., K] fp16 or bf16, y like x.  Built from fp16 or bf16 weights as
    linear layers hold them, router [E, K], gate_up [E, 2I, K] (I gates, then I
    ups) and down [E, K, I], the experts' quantized once, or by from_quantized
    from a checkpoint's e4m3 ones.  `normalize`: a token's weights sum to 1.

    Buffers: router (of x's type; half() and bfloat16() change it), gate_up,
    gate_up_scale, down, down_scale.  For serving: y carries no gradient.  More
    than MOE_MAX_PAIRS places of tokens are run in several calls.
    """

    def __init__(self, router: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, top_k: int,
                 normalize: bool = True):
        super().__init__()
        self._check_shapes(router, gate_up, down)
        for name, w in (("gate_up", gate_up), ("down", down)):
            if w.dtype not in _HALVES:
                raise TypeError(f"{name} must be fp16 or bf16, got {w.dtype}")
        held = []
        for w in (gate_up, down):
            # one expert at a time: a transposed copy of all would double the memory
            parts = [fp8_quantize_weight(w[e].detach().t().contiguous()) for e in range(w.shape[0])]
            held += [torch.stack([q.view(torch.uint8) for q, _ in parts]).view(torch.float8_e4m3fn),
                     torch.stack([s for _, s in parts])]
        self._set(router, *held, top_k, normalize)

    @staticmethod
    def _check_shapes(router, gate_up, down):
        if router.dim() != 2 or gate_up.dim() != 3 or down.dim() != 3:
            raise TypeError("router must be [E, K], gate_up [E, 2I, K] and down [E, K, I]")
        (E, K), I2 = router.shape, gate_up.shape[1]
        if E > MOE_MAX_EXPERTS:
            raise ValueError(f"at most {MOE_MAX_EXPERTS} experts, got {E}")
        if E < 1 or I2 % 2 or gate_up.shape != (E, I2, K) or down.shape != (E, K, I2 // 2):
            raise ValueError(f"router {tuple(router.shape)}, gate_up {tuple(gate_up.shape)} and down "
                             f"{tuple(down.shape)} do not fit as [E, K], [E, 2I, K] and [E, K, I]")
        if router.dtype not in _HALVES:
            raise TypeError(f"router must be fp16 or bf16, got {router.dtype}")
        if any(t.device.type != "cuda" for t in (router, gate_up, down)):
            raise TypeError("router, gate_up and down must be CUDA tensors")

    def _set(self, router, gate_up, gate_up_scale, down, down_scale, top_k, normalize):
        most = min(router.shape[0], MOE_MAX_TOP_K)
        if not 1 <= top_k <= most:
            raise ValueError(f"top_k must be 1 to {most}, got {top_k}")
        self.register_buffer("router", router.detach().clone(memory_format=torch.contiguous_format))
        for name, t in (("gate_up", gate_up), ("gate_up_scale", gate_up_scale), ("down", down),
                        ("down_scale", down_scale)):
            self.register_buffer(name, t)
        self.top_k, self.normalize = int(top_k), bool(normalize)

    @classmethod
    def from_quantized(cls, router: torch.Tensor, gate_up: torch.Tensor, gate_up_scale: torch.Tensor,
                       down: torch.Tensor, down_scale: torch.Tensor, top_k: int,
                       normalize: bool = True) -> "Fp8MoE":
        """A checkpoint's e4m3 experts, gate_up [E, 2I, K] and down [E, K, I], with
        their scales [E, ceil(2I/128), ceil(K/128)] and [E, ceil(K/128), ceil(I/128)]."""
        cls._check_shapes(router, gate_up, down)
        scales = []
        for name, w, s in (("gate_up_scale", gate_up, gate_up_scale), ("down_scale", down, down_scale)):
            blocks = (w.shape[0], *((n + FP8_BLOCK - 1) // FP8_BLOCK for n in w.shape[1:]))
            if s.shape != blocks:
                raise ValueError(f"{name} must have shape {blocks}, got {tuple(s.shape)}")
            scales.append(s.detach().to(device=w.device, dtype=torch.float32).contiguous())
        self = cls.__new__(cls)
        torch.nn.Module.__init__(self)
        self._set(router, fp8_pack_experts(gate_up.detach().contiguous()), scales[0],
                  fp8_pack_experts(down.detach().contiguous()), scales[1], top_k, normalize)
        return self

    def _apply(self, fn, recurse=True):
        # half() and bfloat16() change the router's type, float() and the like only
        # move it; the e4m3 numbers and their fp32 scales only follow to another device
        held = dict(self.named_buffers(recurse=False))
        super()._apply(fn, recurse)
        for name, t in held.items():
            now = getattr(self, name)
            if now.dtype != t.dtype and not (name == "router" and now.dtype in _HALVES):
                setattr(self, name, t.to(now.device))
        return self

    def extra_repr(self) -> str:
        E, K = self.router.shape
        return (f"features={K}, experts={E}, expert_features={self.gate_up.shape[1] // 2}, "
                f"top_k={self.top_k}, normalize={self.normalize}")

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        K = self.router.shape[1]
        if x.shape[-1] != K:
            raise ValueError(f"expected last dimension {K}, got {x.shape[-1]}")
        x2 = x.reshape(-1, K).contiguous()
        y = torch.empty_like(x2)
        most = MOE_MAX_PAIRS // self.top_k
        for m in range(0, max(1, x2.shape[0]), most):
            part = x2[m:m + most]
            experts, weights = moe_route(part, self.router, self.top_k, normalize=self.normalize)
            fp8_moe(part, experts, weights, self.gate_up, self.gate_up_scale, self.down,
                    self.down_scale, out=y[m:m + most])
        return y.reshape(x.shape)


__all__ = ["Int8MixedLinear", "Fp8BlockLinear", "Fp8RMSNorm", "Fp8SandwichNorm", "Fp8MoE"]
