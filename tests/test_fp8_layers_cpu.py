"""The block-scaled e4m3 layers, what needs no GPU: refusals that come before
any kernel, and changes of type."""
import pytest
import torch

from int8_mixed_precision_outlier_amd.linear import Fp8BlockLinear, Fp8RMSNorm

E4M3 = torch.float8_e4m3fn


def block_linear(K=272, N=32, dtype=torch.bfloat16, bias=None):
    """A layer over buffers on the CPU, as a moved one: it refuses before it computes."""
    layer = Fp8BlockLinear.__new__(Fp8BlockLinear)
    torch.nn.Module.__init__(layer)
    kb = -(-K // 128)
    w = torch.arange(N * kb * 128).remainder(120).to(torch.uint8).view(N, kb * 128).view(E4M3)
    layer._set(w, torch.rand(-(-N // 128), kb), K, dtype, bias)
    return layer


@pytest.mark.parametrize("K,wrong", [(272, (256, 288, 384, 400)), (384, (272, 368)), (16, (32, 128))])
def test_pair_of_another_width(K, wrong):
    """The packed weight keeps K rounded up to 128 only, so a pair of another
    width would pass the product's own checks."""
    layer = block_linear(K)
    for k in wrong:
        q = torch.zeros((5, k)).to(E4M3)
        with pytest.raises(ValueError, match=f"{K}.*{k}"):
            layer((q, torch.ones(-(-k // 128), 5)))
    for k in (K + 16, 7):
        with pytest.raises(ValueError, match=f"{K}.*{k}"):
            layer(torch.zeros((5, k), dtype=torch.bfloat16))


def test_from_quantized_looks_at_its_arguments():
    """Scales, bias and types that no forward could take are refused when the
    layer is built."""
    w = torch.zeros((144, 272)).to(E4M3)  # scales [2, 3]
    make = lambda scale=(2, 3), **k: Fp8BlockLinear.from_quantized(w, torch.ones(scale), **k)  # noqa: E731
    for scale in ((3, 2), (2, 2), (1, 3), (6,), (2, 3, 1), ()):
        with pytest.raises(ValueError, match=r"w_scale.*\(2, 3\)"):
            make(scale)
    for dtype in (torch.float32, E4M3, torch.int8):
        with pytest.raises(TypeError, match="dtype"):
            make(dtype=dtype)
    with pytest.raises(TypeError, match="2-D"):
        Fp8BlockLinear.from_quantized(w[0], torch.ones(2, 3))
    with pytest.raises(TypeError, match="CUDA"):
        make()  # the weight itself: packing is the GPU's


@pytest.mark.parametrize("shape", [(31,), (272,), (32, 1), ()])
def test_bias_of_another_size(shape):
    with pytest.raises(ValueError, match="bias"):
        block_linear(bias=torch.zeros(shape))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_norm_keeps_a_16_bit_type(dtype):
    """float(), double() and to(e4m3) of a model leave the norm a weight that it
    takes, as they leave the linear layers; half() and bfloat16() change it."""
    norm = Fp8RMSNorm.__new__(Fp8RMSNorm)
    torch.nn.Module.__init__(norm)
    w = (torch.arange(64) / 7).to(dtype)
    norm.register_buffer("weight", w.clone())
    outer = torch.nn.Sequential(norm, torch.nn.Linear(4, 4))
    for change in (outer.float, outer.double, lambda: outer.to(E4M3), lambda: outer.to("cpu"), norm.float):
        change()
        assert norm.weight.dtype == dtype and torch.equal(norm.weight, w)
        assert set(norm.state_dict()) == {"weight"}
    assert outer.half()[0].weight.dtype == torch.float16
    assert outer.to(torch.bfloat16)[0].weight.dtype == torch.bfloat16
    assert norm.to("meta").to_empty(device="cpu").weight.dtype == torch.bfloat16


def test_bias_survives_types_of_fewer_bits():
    """to(e4m3) of a model around the layer leaves its bias unrounded."""
    b = torch.linspace(-1, 1, 32).to(torch.bfloat16)
    layer = block_linear(bias=b)
    torch.nn.Sequential(layer).to(E4M3)
    assert layer.dtype == layer.bias.dtype == torch.bfloat16 and torch.equal(layer.bias, b)
    w, ws = layer.w_f8.view(torch.uint8).clone(), layer.w_scale.clone()
    layer.to(torch.float8_e5m2).float()
    assert torch.equal(layer.bias, b) and torch.equal(layer.w_scale, ws)
    assert layer.w_f8.dtype == E4M3 and torch.equal(layer.w_f8.view(torch.uint8), w)
