"""The block-scaled e4m3 layers on the GPU: refusals of operands that the
kernels alone would take, changes of type, lifetimes of given tensors."""
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8
from int8_mixed_precision_outlier_amd.linear import Fp8BlockLinear, Fp8RMSNorm

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def acts(M, K, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((M, K), generator=g, device="cuda").to(dtype)


def test_pair_of_another_width():
    layer = Fp8BlockLinear(acts(32, 272, torch.bfloat16, 1))
    for k in (288, 384):
        with pytest.raises(ValueError, match="272"):
            layer(i8.fp8_quantize(acts(5, k, torch.bfloat16, 2)))
    x = acts(5, 272, torch.bfloat16, 3)
    assert torch.equal(layer(i8.fp8_quantize(x)), layer(x))


def test_from_quantized_scales_from_elsewhere():
    """A checkpoint's scales as a parameter on the host: moved, and no parameter
    of the layer."""
    w = acts(32, 272, torch.float32, 4).to(E4M3)
    ws = torch.rand(1, 3)
    layer = Fp8BlockLinear.from_quantized(w, torch.nn.Parameter(ws))
    x = acts(5, 272, torch.bfloat16, 5)
    assert torch.equal(layer(x), i8.fp8_matmul(*i8.fp8_quantize(x), i8.fp8_pack_weight(w), ws.cuda()))
    assert not list(layer.parameters()) and not layer.w_scale.requires_grad


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_model_after_float(dtype):
    """A norm and the layer behind it give after float() what they gave before."""
    K = 272
    model = torch.nn.ModuleList([Fp8RMSNorm(acts(1, K, dtype, 6)[0]), Fp8BlockLinear(acts(32, K, dtype, 7))])
    x, r = acts(5, K, dtype, 8), acts(5, K, dtype, 9)

    def run():
        pair, h = model[0](x, r)
        return model[1](pair), h
    want = run()
    model.float()
    assert all(torch.equal(a, b) and a.dtype == dtype for a, b in zip(run(), want))
