"""The mixture-of-experts layer and the sandwich norm's, what needs no GPU:
refusals that come before any kernel, and changes of type."""
import pytest
import torch

from int8_mixed_precision_outlier_amd.linear import Fp8MoE, Fp8SandwichNorm

E4M3 = torch.float8_e4m3fn


def moe(dtype=torch.bfloat16):
    """A layer over buffers on the CPU, as a moved one: it refuses before it computes."""
    layer = Fp8MoE.__new__(Fp8MoE)
    torch.nn.Module.__init__(layer)
    code = lambda *s: torch.arange(s[0] * s[1] * s[2]).remainder(120).to(torch.uint8).view(s).view(E4M3)  # noqa: E731
    layer._set((torch.arange(3 * 48) / 7).view(3, 48).to(dtype), code(3, 64, 128), torch.rand(3, 1, 1),
               code(3, 48, 128), torch.rand(3, 1, 1), 2, True)
    return layer


def test_last_dimension():
    for k in (16, 64, 128):
        with pytest.raises(ValueError, match=f"48.*{k}"):
            moe()(torch.zeros((5, k), dtype=torch.bfloat16))


def test_shapes_that_do_not_fit():
    r, u, d = torch.zeros((3, 48)).half(), torch.zeros((3, 64, 48)).half(), torch.zeros((3, 48, 32)).half()
    for bad in ((r[:2], u, d), (r, u[:, :63], d), (r, u[:, :, :32], d), (r, u, d[:, :32]), (r, u, d[:2]),
                (r, u, torch.zeros((3, 48, 64)).half()), (r[:0], u[:0], d[:0])):
        with pytest.raises(ValueError, match="router"):
            Fp8MoE(*bad, 2)
    for bad in ((r[0], u, d), (r, u[0], d), (r, u, d[0]), (r.float(), u, d)):
        with pytest.raises(TypeError):
            Fp8MoE(*bad, 2)
    with pytest.raises(TypeError, match="CUDA"):
        Fp8MoE(r, u, d, 2)
    for k in (0, 4, -1):
        with pytest.raises(ValueError, match="top_k"):
            moe()._set(r, u, None, d, None, k, True)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_changes_of_type(dtype):
    """float(), double() and to(e4m3) of a model leave the layer what it computes
    with; half() and bfloat16() change the router's type alone."""
    layer = moe(dtype)
    held = {n: t.clone() for n, t in layer.named_buffers()}
    outer = torch.nn.Sequential(layer, torch.nn.Linear(4, 4))
    for change in (outer.float, outer.double, lambda: outer.to(E4M3), lambda: outer.to("cpu"), layer.float):
        change()
        for n, t in held.items():
            now = getattr(layer, n)
            assert now.dtype == t.dtype and torch.equal(now.contiguous().view(torch.uint8), t.contiguous().view(torch.uint8)), n
    for other in (torch.float16, torch.bfloat16):
        outer.to(other)
        assert layer.router.dtype == other and layer.gate_up.dtype == layer.down.dtype == E4M3
        assert layer.gate_up_scale.dtype == torch.float32
    assert set(layer.state_dict()) == {"router", "gate_up", "gate_up_scale", "down", "down_scale"}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_norm_keeps_a_16_bit_type(dtype):
    norm = Fp8SandwichNorm.__new__(Fp8SandwichNorm)
    torch.nn.Module.__init__(norm)
    w = (torch.arange(64) / 7).to(dtype)
    norm.register_buffer("post_weight", w.clone())
    norm.register_buffer("pre_weight", w.clone() * 2)
    outer = torch.nn.Sequential(norm)
    for change in (outer.float, outer.double, lambda: outer.to(E4M3), norm.float):
        change()
        assert norm.post_weight.dtype == dtype and torch.equal(norm.post_weight, w) and torch.equal(norm.pre_weight, w * 2)
    assert outer.half()[0].post_weight.dtype == torch.float16
    assert outer.to(torch.bfloat16)[0].pre_weight.dtype == torch.bfloat16


def test_norm_refuses():
    w = torch.ones(32).half()
    with pytest.raises(TypeError, match="CUDA"):
        Fp8SandwichNorm(w, w)
    with pytest.raises(TypeError, match="1-D"):
        Fp8SandwichNorm(w[None], w)
    norm = Fp8SandwichNorm.__new__(Fp8SandwichNorm)
    torch.nn.Module.__init__(norm)
    norm.register_buffer("post_weight", w)
    norm.register_buffer("pre_weight", w)
    with pytest.raises(ValueError, match="32"):
        norm(torch.zeros(2, 16).half(), torch.zeros(2, 16).half())
    with pytest.raises(ValueError, match="residual"):
        norm(torch.zeros(2, 32).half(), torch.zeros(1, 32).half())
