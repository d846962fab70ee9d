"""The mixture-of-experts layer and the sandwich norm's on the GPU: what they
compute, several calls for many tokens, refusals of the entry points."""
import numpy as np
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8
from int8_mixed_precision_outlier_amd.linear import Fp8BlockLinear, Fp8MoE, Fp8SandwichNorm
from oracle import fp8_block as F
from oracle import moe as O
from tests.test_moe_gpu import E4M3, TYPES, f64, near, rows

pytestmark = pytest.mark.gpu


def weights(E, K, I, dtype):
    w = lambda *s: torch.stack([rows(s[1], s[2], dtype, 10 * e + s[1], std=0.05, outliers=1) for e in range(s[0])])  # noqa: E731
    return rows(E, K, dtype, 1, std=0.1, outliers=0), w(E, 2 * I, K), w(E, K, I)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(1,), (2, 3), (40,), (2, 5, 7)])
def test_moe_layer(shape, dtype):
    E, K, I, k = 6, 272, 144, 2
    router, up, down = weights(E, K, I, dtype)
    layer = Fp8MoE(router, up, down, k)
    M = int(np.prod(shape))
    x = rows(M, K, dtype, 3, std=1.0, outliers=2)
    y = layer(x.view(*shape, K))
    assert y.shape == (*shape, K) and y.dtype == dtype and not y.requires_grad
    q = [[F.quantize_weight_blocks(f64(w[e]).T) for e in range(E)] for w in (up, down)]
    uq, us, dq, ds = (np.stack([t[n] for t in w]) for w in q for n in range(2))
    oe, _ = O.route64(f64(x), f64(router), k, True)
    _, p = i8.moe_route(x, router, k)
    sums = ((128 + 3 + 8) * 2.0 ** -23, (256 + 2 + 8) * 2.0 ** -23)
    near(y.view(M, K), *O.moe64(f64(x), oe, p.cpu().numpy(), uq, us, dq, ds, sums), dtype, shape)
    gpu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    again = Fp8MoE.from_quantized(router, gpu(uq).view(E4M3), torch.nn.Parameter(torch.from_numpy(us)),
                                  gpu(dq).view(E4M3), gpu(ds), k)
    assert torch.equal(again(x), y.view(M, K)) and not list(again.parameters())
    again.load_state_dict(layer.state_dict())
    assert torch.equal(again(x), y.view(M, K))
    layer.float()
    assert torch.equal(layer(x), y.view(M, K))
    with pytest.raises(ValueError):
        layer(x[:, :16])
    with pytest.raises(ValueError, match="gate_up_scale"):
        Fp8MoE.from_quantized(router, gpu(uq).view(E4M3), gpu(us)[:, :1, :1], gpu(dq).view(E4M3), gpu(ds), k)


@pytest.mark.parametrize("M,k", [(0, 2), (4096, 2), (4097, 2), (9000, 1), (1500, 6)])
def test_moe_layer_many_tokens(M, k):
    """More places than one call takes: several, with the same results as alone."""
    E, K, I = 6, 144, 48
    layer = Fp8MoE(*weights(E, K, I, torch.bfloat16), k, normalize=False)
    x = rows(M, K, torch.bfloat16, 5, std=1.0, outliers=2)
    y = layer(x)
    assert y.shape == (M, K)
    for m in range(0, M, 700):
        part = layer(x[m:m + 700].clone())
        # other tokens in a call change the order of no sum, only which kernel makes it
        assert float((part.float() - y[m:m + 700].float()).norm()) <= 2.0 ** -9 * float(part.float().norm())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_norm_layer_in_front_of_others(dtype):
    K = 272
    post, pre = rows(1, K, dtype, 1, outliers=0)[0], rows(1, K, dtype, 2, outliers=0)[0]
    x, r, gate = rows(6, K, dtype, 3).view(2, 3, K), rows(6, K, dtype, 4).view(2, 3, K), rows(2, K, dtype, 5)
    norm = Fp8SandwichNorm(post, pre, eps=1e-5, residual_scale=1.5)
    pair, h = norm(x, r, gate)
    want = i8.fp8_sandwich_norm(x.view(6, K), r.view(6, K), post, pre, gate=gate, residual_scale=1.5, eps=1e-5)
    assert h.shape == x.shape and torch.equal(h.view(6, K), want[2])
    linear = Fp8BlockLinear(rows(32, K, dtype, 6))
    assert torch.equal(linear(pair), linear(want[:2]))
    half = Fp8SandwichNorm(post, pre, eps=1e-5, residual_scale=1.5, quantize=False)
    y, h2 = half(x, r, gate)
    assert y.shape == x.shape and torch.equal(h2, h)
    moe = Fp8MoE(*weights(6, K, 144, dtype), 2)
    assert moe(y).shape == x.shape
    half.float()
    assert torch.equal(half(x, r, gate)[0], y)
    strided = torch.empty((2, 3, 2 * K), dtype=dtype, device="cuda")[..., :K].copy_(x)
    assert torch.equal(norm(strided, r, gate)[1], h)


def test_refusals():
    half, bf = torch.float16, torch.bfloat16
    x, w = rows(4, 272, half, 1), rows(1, 272, half, 2)[0]
    norm = lambda **k: i8.fp8_sandwich_norm(**{**dict(X=x, residual=x, post_weight=w, pre_weight=w), **k})  # noqa: E731
    q, s, _ = norm()
    router = rows(6, 272, half, 3)
    e, p = i8.moe_route(x, router, 2)
    up, us = i8.fp8_quantize_experts(rows(3 * 272, 64, half, 4).view(3, 272, 64))
    down, ds = i8.fp8_quantize_experts(rows(3 * 32, 272, half, 5).view(3, 32, 272))
    moe = lambda **k: i8.fp8_moe(**{**dict(X=x, experts=e, weights=p, gate_up=up, gate_up_scale=us, down=down,  # noqa: E731
                                           down_scale=ds), **k})
    moe()
    bad = [
        (TypeError, lambda: norm(X=x.float())), (TypeError, lambda: norm(residual=x.to(bf))),
        (ValueError, lambda: norm(residual=x[:3])), (ValueError, lambda: norm(X=x.t())),
        (TypeError, lambda: norm(post_weight=w.cpu())), (ValueError, lambda: norm(pre_weight=w[:16])),
        (ValueError, lambda: norm(gate=x[:3])), (ValueError, lambda: norm(gate=x[:0])),
        (ValueError, lambda: norm(gate=w[:16])), (ValueError, lambda: norm(gate=x[None])),
        (TypeError, lambda: norm(gate=w.to(bf))), (ValueError, lambda: norm(out=(q[:2], s))),
        (TypeError, lambda: norm(out=x, quantize=False, residual_out=x.float())),
        (TypeError, lambda: norm(out=x.to(bf), quantize=False)),
        (i8.Int8mmError, lambda: norm(eps=0.0)), (i8.Int8mmError, lambda: norm(residual_scale=float("inf"))),
        (i8.Int8mmError, lambda: i8.fp8_sandwich_norm(x[:, :24].contiguous(), x[:, :24].contiguous(), w[:24].clone(), w[:24].clone())),
        (TypeError, lambda: i8.moe_route(x.float(), router, 2)), (TypeError, lambda: i8.moe_route(x, router.to(bf), 2)),
        (ValueError, lambda: i8.moe_route(x, router[:, :16], 2)), (i8.Int8mmError, lambda: i8.moe_route(x, router, 7)),
        (i8.Int8mmError, lambda: i8.moe_route(x, router, 0)), (ValueError, lambda: i8.moe_route(x, router, 2, out=(e[:2], p))),
        (TypeError, lambda: i8.moe_route(x, router, 2, out=(e.long(), p))),
        (TypeError, lambda: moe(experts=e.long())), (ValueError, lambda: moe(experts=e[:3])),
        (ValueError, lambda: moe(experts=e[:, 0])), (ValueError, lambda: moe(weights=p[:, :1])),
        (TypeError, lambda: moe(weights=p.half())), (ValueError, lambda: moe(gate_up=up[:, :63])),
        (ValueError, lambda: moe(gate_up=up[:2].contiguous())), (ValueError, lambda: moe(down=down[:, :256].contiguous())),
        (ValueError, lambda: moe(gate_up_scale=us[:, :, :2].contiguous())), (TypeError, lambda: moe(down_scale=ds.half())),
        (ValueError, lambda: moe(X=x[:, :256].contiguous())), (TypeError, lambda: moe(out=x.to(bf))),
        (ValueError, lambda: moe(out=x[:3])), (ValueError, lambda: moe(experts=e.t().contiguous().t())),
        (TypeError, lambda: i8.fp8_pack_experts(up.view(torch.uint8))), (ValueError, lambda: i8.fp8_pack_experts(up[0])),
        (ValueError, lambda: i8.fp8_quantize_experts(x)),
    ]
    for n, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"refusal {n} did not raise")
    many = torch.zeros((i8.MOE_MAX_PAIRS // 2 + 1, 272), dtype=half, device="cuda")
    with pytest.raises(i8.Int8mmError):
        moe(X=many, experts=torch.zeros((len(many), 2), dtype=torch.int32, device="cuda"),
            weights=torch.zeros((len(many), 2), device="cuda"))


def test_refuses_what_is_no_gate_and_no_size():
    x = rows(4, 272, torch.float16, 1)
    for gate, err in ((2.0, TypeError), (x[0, 0], ValueError), (x[0].cpu(), TypeError)):
        with pytest.raises(err):
            i8.fp8_sandwich_norm(x, x, x[0], x[1], gate=gate)
    for top_k in (-1, i8.MOE_MAX_TOP_K + 1, 1 << 40):
        with pytest.raises(ValueError):
            i8.moe_route(x, x, top_k)
