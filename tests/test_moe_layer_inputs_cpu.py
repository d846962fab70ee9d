"""What the mixture-of-experts layer keeps of the weights that it is given, without a
GPU."""
import pytest
import torch

from int8_mixed_precision_outlier_amd.linear import Fp8MoE

E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("form", ["transposed", "strided", "expanded"])
def test_router_of_any_strides(form, dtype):
    """The router's operator takes contiguous rows; a weight held as [K, E], a part of
    a larger one or one row for all experts is kept as such rows."""
    E, K = 3, 48
    w = torch.arange(E * K, dtype=torch.float32).view(E, K).to(dtype)
    given = {"transposed": lambda: w.t().contiguous().t(), "strided": lambda: torch.cat([w, w], 1)[:, :K],
             "expanded": lambda: w[:1].expand(E, K)}[form]()
    assert not given.is_contiguous()
    layer = Fp8MoE.__new__(Fp8MoE)
    torch.nn.Module.__init__(layer)
    zeros = lambda *s: torch.zeros(s, dtype=torch.uint8).view(E4M3)  # noqa: E731
    layer._set(given, zeros(E, 64, 128), torch.ones(E, 1, 1), zeros(E, K, 128), torch.ones(E, 1, 1), 2, True)
    assert layer.router.is_contiguous() and torch.equal(layer.router, given)
    assert layer.router.data_ptr() != given.data_ptr()
