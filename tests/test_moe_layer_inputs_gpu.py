"""The mixture-of-experts layers on the GPU, for inputs that a caller may hold in
other forms than the usual ones."""
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8
from int8_mixed_precision_outlier_amd.linear import Fp8SandwichNorm
from tests.test_moe_gpu import rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quantize", [True, False])
@pytest.mark.parametrize("G", [0, 1, 4])
def test_no_tokens_with_gates(G, quantize):
    """An empty batch with a row of gates for each of its tokens, or more."""
    K = 272
    x, w = torch.empty((0, K), dtype=torch.bfloat16, device="cuda"), rows(1, K, torch.bfloat16, 2)[0]
    gate = rows(4, K, torch.bfloat16, 3)[:G]
    out = i8.fp8_sandwich_norm(x, x, w, w, gate=gate, quantize=quantize)
    assert out[0].shape == out[-1].shape == (0, K)
    y, h = Fp8SandwichNorm(w, w, quantize=quantize)(x.view(2, 0, K), x.view(2, 0, K), gate)
    assert h.shape == (2, 0, K)
