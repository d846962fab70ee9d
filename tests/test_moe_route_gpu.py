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
