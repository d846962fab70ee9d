"""The experts' products at the ends of fp32's range, where the sum of a block's
products passes it and the block's scale brings it back; tolerances as derived in
test_moe_gpu.py."""
import numpy as np
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8
from oracle import fp8_block as F
from oracle import moe as O
from tests.test_moe_gpu import KERNELS, TYPES, Case, f64, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,I,E,k", KERNELS)
@pytest.mark.parametrize("power", [100, 118])
def test_large_tokens_small_scales(M, K, I, E, k, power):
    """bf16 tokens near the type's end: a block's numbers times them add up to more
    than fp32 holds, times the block's scale they do not."""
    c = Case(M, K, I, E, k, torch.bfloat16, seed=23)
    c.x = (c.x.float().clamp(-500, 500) * 2.0 ** power).bfloat16()
    assert torch.isfinite(c.x).all()
    c.up_s *= np.float32(2.0 ** -power)
    Y = c.check()
    assert float(Y.float().abs().mean()) > 1e-3


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,I,E,k", KERNELS)
def test_large_gated_products_small_scales(M, K, I, E, k, dtype):
    """The same in the second product: gated products of about 2^120.  Of 400 tokens
    one has a gated product of 2^128.15 by the formula, which fp32 does not hold:
    tokens whose own gated products pass fp32's range are not compared."""
    c = Case(M, K, I, E, k, dtype, seed=25)
    c.up_s *= np.float32(2.0 ** 58)
    c.down_s *= np.float32(2.0 ** -116)
    largest = np.zeros(M)
    for e in range(E):
        m, _ = np.nonzero(c.experts == e)
        if len(m):
            a = F.silu_mul64(f64(c.x)[m] @ O.weight64(c.up[e], c.up_s[e]).T)
            np.maximum.at(largest, m, np.abs(a).max(1))
    held = largest < np.finfo(np.float32).max
    assert held.sum() >= 0.99 * M
    want, tol = c.oracle()
    assert np.all(np.isfinite(want)) and np.abs(want).mean() > 1e-3
    near(i8.fp8_moe(*c.gpu())[torch.from_numpy(held).cuda()], want[held], tol[held], dtype, (M, K, I, E, k))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,I,E,k", KERNELS)
def test_scales_of_every_kind(M, K, I, E, k, dtype):
    """Scales that are negative, zero, subnormal, and past 2^100 with numbers that
    bring them back, next to ordinary ones."""
    c = Case(M, K, I, E, k, dtype, seed=27)
    c.up_s[:, 0] *= np.float32(-1)
    c.up_s[:, -1, -1] = 0.0
    c.down_s[:, 0, 0] = np.float32(2.0 ** -140)
    c.down_s[:, -1] *= np.float32(-1.75)
    c.check()
    c = Case(M, K, I, E, k, dtype, seed=29)
    # the least number, 2^-9, in a block of scale 2^104: 2^95 times tokens of 2^-95
    # and below (fp16 tokens cannot be that small: the scale of their products is)
    if dtype == torch.bfloat16:
        c.x = (c.x.float() * 2.0 ** -100).bfloat16()
        c.up &= 0x81
        c.up_s = (c.up_s * np.float32(2.0 ** 113)).astype(np.float32)
        assert c.up_s.max() > 2.0 ** 101 and np.abs(f64(c.x)).max() < 2.0 ** -90
        c.check()
        assert float(i8.fp8_moe(*c.gpu()).float().abs().max()) > 0


@pytest.mark.parametrize("M,K,I,E,k", KERNELS)
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_scales_that_are_no_numbers(M, K, I, E, k, bad):
    """An infinite or NaN scale makes its expert's tokens infinite or NaN, and no others."""
    c = Case(M, K, I, E, k, torch.bfloat16, seed=31)
    e = int(c.experts[0, 0])
    hit = torch.from_numpy((c.experts == e).any(1)).cuda()
    want = i8.fp8_moe(*c.gpu())
    c.down_s[e] = bad
    Y = i8.fp8_moe(*c.gpu())
    assert not torch.isfinite(Y[hit]).any() and torch.equal(Y[~hit], want[~hit])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,I,E,k", KERNELS)
@pytest.mark.parametrize("sign", [1, -1])
def test_gated_products_between_the_largest_bf16_and_fp32_numbers(M, K, I, E, k, dtype, sign):
    """2^128 (1 - 2^-12)^2: the nearest bf16 number would be infinite."""
    c = Case(M, K, I, E, k, dtype, seed=33)
    c.x[:] = 0
    c.x[:, 0] = 1
    c.up[:] = 0
    c.up[:, :I, 0], c.up[:, I:, 0] = 0x38, 0x38 if sign > 0 else 0xb8  # 1 and 1 or -1
    c.up_s[:] = np.float32(2.0 ** 64 * (1 - 2.0 ** -12))
    c.down_s *= np.float32(2.0 ** -128)
    Y = c.check()
    assert float(Y.float().abs().mean()) > 1e-3


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,k", [(0, 2), (1, 2), (1, 32), (3, 2), (30, 9), (4000, 2)])
def test_no_features_between_the_products(M, k, dtype):
    """I = 0 writes zeros whatever the pairs' weights and experts are."""
    E, K = 64, 400
    e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    x = torch.full((M, K), float("nan"), dtype=dtype, device="cuda")
    experts = torch.arange(M * k, dtype=torch.int32, device="cuda").remainder(E + 2).sub(1).view(M, k)
    out = torch.full_like(x, 7)
    for weight in (1.0, float("nan"), float("inf")):
        w = torch.full((M, k), weight, device="cuda")
        assert i8.fp8_moe(x, experts, w, e8(E, 0, 512), f(E, 0, 4), e8(E, K, 0), f(E, 4, 0), out=out.fill_(7)) is out
        assert bool((out == 0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,I,E,k", KERNELS)
@pytest.mark.parametrize("power", [40, 56, 60])
def test_small_gated_products_large_scales(M, K, I, E, k, dtype, power):
    """Gated products of about 2^(-2 power), whose second bf16 number is below the
    type's normal ones, and a second matrix that brings them back."""
    c = Case(M, K, I, E, k, dtype, seed=35)
    c.up_s *= np.float32(2.0 ** -power)
    c.down_s *= np.float32(2.0 ** (2 * power))
    Y = c.check()
    assert float(Y.float().abs().mean()) > 1e-3
