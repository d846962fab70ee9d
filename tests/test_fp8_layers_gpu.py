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


def test_tensors_given_to_another_stream_may_be_dropped():
    """A call with `stream` reads tensors of the current stream.  While that
    stream is busy, new tensors of the current one get other memory than the
    operands that the caller no longer holds."""
    M = K = N = 4096
    half = torch.bfloat16
    stream = torch.cuda.Stream()
    w = torch.zeros((4 * N, 4 * K), device="cuda", dtype=half)
    busy = [*i8.fp8_quantize(torch.zeros((M, 4 * K), device="cuda", dtype=half)), *i8.fp8_quantize_weight(w)]
    del w
    x, gu, g = acts(M, K, half, 1), acts(M, 2 * K, half, 2), acts(1, K, half, 3)[0]
    q, s = i8.fp8_quantize(x)
    calls = [(i8.fp8_quantize, lambda: (x.clone(),)), (i8.fp8_silu_mul, lambda: (gu.clone(),)),
             (i8.fp8_rms_norm, lambda: (x.clone(), g.clone(), 1e-6, x.clone())),
             (i8.fp8_quantize_weight, lambda: (x.clone(),)), (i8.fp8_pack_weight, lambda: (q.clone(),)),
             (i8.fp8_matmul, lambda: (q.clone(), s.clone(), *i8.fp8_quantize_weight(x)))]
    for call, operands in calls:
        want = call(*operands())
        args = operands()
        torch.cuda.synchronize()
        for _ in range(24):  # about 20 ms
            i8.fp8_matmul(*busy, stream=stream)
        got = call(*args, stream=stream)
        held = [(a.data_ptr(), a.shape, a.dtype) for a in args if isinstance(a, torch.Tensor)]
        del args
        new = [torch.empty(shape, dtype=dtype, device="cuda") for _, shape, dtype in held for _ in range(2)]
        assert not stream.query(), "the stream was to be busy meanwhile"
        assert not {t.data_ptr() for t in new} & {p for p, _, _ in held}, call
        for t in new:
            t.view(torch.uint8).fill_(0x7f)
        torch.cuda.synchronize()
        pairs = zip(got, want) if isinstance(got, tuple) else [(got, want)]
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in pairs), call
