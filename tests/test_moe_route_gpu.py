"""The router where its sums are at their limits: no columns for the most tokens
and experts, and the matrix instructions' sums against 64 bits."""
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,E,k", [(1 << 18, 1024, 32), (1 << 18, 256, 1), ((1 << 18) - 1, 65, 3), (16384, 1024, 2),
                                   (16383, 1024, 2)])
def test_no_columns_for_many_tokens(M, E, k):
    """More sums than one launch has wavefronts, all of them 0: the first experts,
    with equal weights."""
    z = lambda n: torch.empty((n, 0), dtype=torch.float16, device="cuda")  # noqa: E731
    e, p = i8.moe_route(z(M), z(E), k, normalize=False)
    assert bool((e == torch.arange(k, dtype=torch.int32, device="cuda")).all())
    assert bool(((p * E - 1).abs() <= 64 * 2.0 ** -24).all())
    del e, p
    torch.cuda.empty_cache()


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("M,E,k", [(64, 1, 1), (40000, 1, 1), (40000, 2, 2), (40000, 2, 1)])
def test_products_past_fp32_of_few_experts(M, E, k, normalize):
    """Logits of 2^252 and more are finite in 64 bits: the weights of equal ones are
    equal, that of a single expert is 1."""
    x = torch.full((M, 1024), 1e38, dtype=torch.bfloat16, device="cuda")
    w = torch.full((E, 1024), 1e38, dtype=torch.bfloat16, device="cuda")
    for sign in (1, -1):
        e, p = i8.moe_route(x, w * sign, k, normalize=normalize)
        assert bool((e == torch.arange(k, dtype=torch.int32, device="cuda")).all())
        assert bool((p == 1 / (k if normalize else E)).all())
    x[3, 5] = float("inf")
    e, p = i8.moe_route(x, w, k, normalize=normalize)
    assert bool(p[3].isnan().all()) and bool((p[4:] == 1 / (k if normalize else E)).all())
