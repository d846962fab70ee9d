"""Block-scaled e4m3 operators, what needs no GPU: the oracle against torch's
e4m3 type and brute force, and the refusals of the C-ABI and the binding."""
import ctypes
import os

import numpy as np
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8
from oracle import fp8_block as F

FAKE = ctypes.c_void_p(1 << 20)  # aligned non-null; never dereferenced (checks fail first)
ODD = ctypes.c_void_p((1 << 20) + 8)
EINVAL, EALIGN, OK = i8.STATUS_EINVAL, i8.STATUS_EALIGN, i8.STATUS_OK

needs_lib = pytest.mark.skipif(not os.path.exists(i8.LIB_PATH),
                               reason="libint8mm.so not built (run __graft_entry__.build())")


def test_e4m3_values_are_torch_s():
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(F.e4m3_decode(b), t, equal_nan=True)


def test_e4m3_encode_is_torch_s_rounding():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 2, 20000),
                        F.E4M3_VALUES, -F.E4M3_VALUES,
                        (F.E4M3_VALUES[1:] + F.E4M3_VALUES[:-1]) / 2, [448.00003, 463.9, 0.0]])
    x = x[np.abs(x) < 464].astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(F.e4m3_encode(x), t)


def test_oracle_blocks_by_hand():
    """One row of 144 columns: the first block's scale from its outlier, the
    second's (16 columns) from its own maximum, zeros on the floor."""
    x = np.zeros((2, 144), np.float16)
    x[0, :4] = [100, -1, 0.25, 50]
    x[0, 128:131] = [0.5, -0.25, 0.125]
    q, s = F.quantize_blocks(x)
    assert s.shape == (2, 2)
    assert s[0, 0] == np.float32(100) / np.float32(448) and s[1, 0] == np.float32(0.5) / np.float32(448)
    assert s[0, 1] == s[1, 1] == np.float32(2.0 ** -100) / np.float32(448)
    v = F.e4m3_decode(q)
    assert list(v[0, :4]) == [448, -4.5, 1.125, 224]  # 4.48 -> 4.5, 1.12 -> 1.125
    assert list(v[0, 128:131]) == [448, -224, 112]
    assert not v[1].any() and not v[0, 4:128].any()


def test_oracle_matmul_by_loops():
    rng = np.random.default_rng(2)
    M, K, N = 3, 144, 144
    xq, xs = F.quantize_blocks(rng.standard_normal((M, K)))
    wq, ws = F.quantize_weight_blocks(rng.standard_normal((K, N)))
    y, _, _ = F.matmul64(xq, xs, wq, ws)
    xv, wv = F.e4m3_decode(xq), F.e4m3_decode(wq)
    for m, n in [(0, 0), (2, 143), (1, 127), (1, 128)]:
        want = sum(xv[m, k] * wv[n, k] * float(xs[k // 128, m]) * float(ws[n // 128, k // 128])
                   for k in range(K))
        assert abs(y[m, n] - want) <= 1e-12 * max(1.0, abs(want))


def test_oracle_packed_layout_by_formula():
    rng = np.random.default_rng(3)
    N, K = 48, 272
    wq = rng.integers(0, 255, (N, K)).astype(np.uint8)
    p = F.pack_weight(wq).reshape(-1)
    KB = 3
    for n, k in [(0, 0), (17, 5), (47, 271), (16, 128), (31, 127), (5, 143)]:
        o = ((n // 16) * KB + k // 128) * 2048 + (((k // 16) % 8) * 16 + n % 16) * 16 + k % 16
        assert p[o] == wq[n, k]
    assert p.size == N * 384 and np.count_nonzero(p) == np.count_nonzero(wq)


@needs_lib
def test_packed_size():
    lib = i8.load()
    assert lib.fp8_packed_size(48, 272) == 48 * 384
    assert lib.fp8_packed_size(49152, 12288) == 49152 * 12288
    for N, K in [(40, 128), (48, 120), (-16, 128), (16, -16), (16, 65552), (32784, 65536)]:
        assert lib.fp8_packed_size(N, K) == -1, (N, K)


@needs_lib
def test_quantizers_refuse():
    lib = i8.load()
    for f, wide in ((lib.fp8_quantize, 1), (lib.fp8_silu_mul, 2)):
        call = lambda X=FAKE, type=0, M=4, K=64, q=FAKE, s=FAKE: f(X, type, M, K, q, s, None)  # noqa: E731
        assert call(type=2) == EINVAL and call(type=-1) == EINVAL
        assert call(M=-1) == EINVAL and call(K=-16) == EINVAL and call(K=65552) == EINVAL
        assert call(M=(1 << 31) // (64 * wide) + 1) == EINVAL
        assert call(K=72) == EALIGN
        assert call(X=None) == EINVAL and call(q=None) == EINVAL and call(s=None) == EINVAL
        assert call(X=ODD) == EALIGN and call(q=ODD) == EALIGN and call(s=ODD) == EALIGN
        assert call(M=0) == OK and call(K=0) == OK


@needs_lib
def test_rms_norm_refuses():
    lib = i8.load()

    def call(X=FAKE, R=FAKE, g=FAKE, type=1, M=4, K=64, eps=1e-6, H=FAKE, q=FAKE, s=FAKE):
        return lib.fp8_rms_norm(X, R, g, type, M, K, ctypes.c_float(eps), H, q, s, None)
    assert call(type=7) == EINVAL
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == EINVAL, eps
    assert call(K=72) == EALIGN and call(K=65552) == EINVAL and call(M=-1) == EINVAL
    assert call(M=1 << 26) == EINVAL
    assert call(R=None) == EINVAL and call(H=None) == EINVAL  # H goes with the residual
    for name in ("X", "g", "q", "s"):
        assert call(**{name: None}) == EINVAL, name
    for name in ("X", "R", "g", "H", "q", "s"):
        assert call(**{name: ODD}) == EALIGN, name
    assert call(M=0) == OK and call(K=0) == OK


@needs_lib
def test_weight_functions_refuse():
    lib = i8.load()
    q = lambda W=FAKE, type=0, K=64, N=32, o=FAKE, s=FAKE: lib.fp8_quantize_weight(W, type, K, N, o, s, None)  # noqa: E731
    p = lambda W=FAKE, N=32, K=64, o=FAKE: lib.fp8_pack_weight(W, N, K, o, None)  # noqa: E731
    assert q(type=2) == EINVAL and q(W=None) == EINVAL and q(o=None) == EINVAL and q(s=None) == EINVAL
    assert q(K=72) == EALIGN and q(N=40) == EALIGN and q(W=ODD) == EALIGN and q(o=ODD) == EALIGN
    assert p(W=None) == EINVAL and p(o=None) == EINVAL and p(K=72) == EALIGN and p(N=40) == EALIGN
    assert p(W=ODD) == EALIGN and p(o=ODD) == EALIGN and p(N=-16) == EINVAL
    assert q(N=32784, K=65536) == EINVAL and p(N=32784, K=65536) == EINVAL
    assert q(K=0) == OK and q(N=0) == OK and p(K=0) == OK and p(N=0) == OK


@needs_lib
def test_matmul_refuses():
    lib = i8.load()

    def call(X=FAKE, xs=FAKE, M=4, K=64, W=FAKE, ws=FAKE, N=32, b=None, type=0, Y=FAKE):
        return lib.fp8_matmul(X, xs, M, K, W, ws, N, b, type, Y, None)
    assert call(type=2) == EINVAL
    assert call(M=-1) == EINVAL and call(N=-16) == EINVAL and call(K=-16) == EINVAL
    assert call(K=65552) == EINVAL and call(K=72) == EALIGN and call(N=40) == EALIGN
    assert call(M=1 << 26) == EINVAL and call(M=1 << 25, K=16, N=128) == EINVAL  # M*K, M*N
    assert call(N=32784, K=65536, M=1) == EINVAL
    for name in ("X", "xs", "W", "ws", "Y"):
        assert call(**{name: None}) == EINVAL, name
        assert call(**{name: ODD}) == EALIGN, name
    assert call(b=ODD) == EALIGN
    assert call(M=0) == OK and call(N=0) == OK


@needs_lib
def test_binding_wants_gpu_tensors():
    x = torch.zeros((4, 64), dtype=torch.float16)
    q, s = x.to(torch.float8_e4m3fn), torch.zeros((1, 4))
    for f in (lambda: i8.fp8_quantize(x), lambda: i8.fp8_silu_mul(x), lambda: i8.fp8_rms_norm(x, x[0]),
              lambda: i8.fp8_quantize_weight(x), lambda: i8.fp8_pack_weight(q),
              lambda: i8.fp8_matmul(q, s, q, s)):
        with pytest.raises(TypeError, match="CUDA"):
            f()
    from int8_mixed_precision_outlier_amd.linear import Fp8BlockLinear, Fp8RMSNorm
    with pytest.raises(TypeError):
        Fp8BlockLinear(x)
    with pytest.raises(TypeError):
        Fp8RMSNorm(x[0])


def test_module_type_changes_leave_the_weights():
    """half(), bfloat16(), float() and moves of a module around the layer: the
    e4m3 bytes and fp32 scales stay, bias and y take the 16-bit types."""
    from int8_mixed_precision_outlier_amd.linear import Fp8BlockLinear
    layer = Fp8BlockLinear.__new__(Fp8BlockLinear)
    torch.nn.Module.__init__(layer)
    w = torch.arange(32 * 128).remainder(251).to(torch.uint8).view(32, 128).view(torch.float8_e4m3fn)
    ws = torch.rand(1, 1)
    layer._set(w.clone(), ws.clone(), 128, torch.bfloat16, torch.arange(32.0))
    outer = torch.nn.Sequential(layer, torch.nn.Linear(32, 8))
    for change, dtype in ((lambda: outer.half(), torch.float16), (lambda: outer.to(torch.bfloat16), torch.bfloat16),
                          (lambda: outer.float(), torch.bfloat16), (lambda: outer.to("cpu"), torch.bfloat16),
                          (lambda: layer.half(), torch.float16), (lambda: outer.double(), torch.float16)):
        assert change() in (outer, layer)
        assert layer.dtype == dtype and layer.bias.dtype == dtype
        assert torch.equal(layer.bias.float(), torch.arange(32.0))
        assert layer.w_f8.dtype == w.dtype and torch.equal(layer.w_f8.view(torch.uint8), w.view(torch.uint8))
        assert layer.w_scale.dtype == torch.float32 and torch.equal(layer.w_scale, ws)
        assert set(layer.state_dict()) == {"w_f8", "w_scale", "bias"}
    meta = layer.to("meta")
    assert meta.w_f8.device.type == "meta" and meta.to_empty(device="cpu").w_f8.dtype == w.dtype


@needs_lib
def test_kernel_choice_over_seeded_sizes():
    """The planner on 256 CUs over 4000 seeded sizes: streaming up to 64 tokens
    and only up to 128, with the token blocks the tokens need; only tiles the
    library builds; a split only at a multiple of 256 strictly inside N, in
    whole rounds of 256x256 tiles in front."""
    import torch
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the expected choices are those of 256 CUs")
    rng = np.random.default_rng(77)
    tiles = {(256, 256, 2), (256, 128, 3), (128, 128, 2), (128, 128, 4), (64, 128, 4)}
    seen = set()
    for _ in range(4000):
        M = int(rng.choice([rng.integers(1, 129), rng.integers(129, 6000)]))
        N = int(np.exp(rng.uniform(0, np.log(4000)))) * 16
        c = i8.fp8_matmul_config(M, N, 16)
        seen.add(c[0] if c[0] == "split" else c)
        if M <= 64 or c[0] == "decode":
            T = -(-M // 16)
            assert c[0] == "decode" and M <= 128 and c[1] in (1, 2, 3, 4, 5, 6, 9), (M, N, c)
            assert c[2] == T and (T <= 4 or c[1] in ((1, 2, 3, 4, 5), (1, 3, 4))[T > 7]), (M, N, c)
        elif c[0] == "tiled":
            assert c[1:] in tiles, (M, N, c)
        else:
            assert c[0] == "split" and c[1] % 256 == 0 and 0 < c[1] < N, (M, N, c)
            assert (c[2], 128, c[3]) in tiles, (M, N, c)
            tm = -(-M // 256)
            assert tm * (c[1] // 256) + tm > -(-tm * (c[1] // 256) // 256) * 256, (M, N, c)
    assert {("tiled",) + t for t in tiles} | {"split"} <= seen
    with pytest.raises(i8.Int8mmError):
        i8.fp8_matmul_config(4, 24, 64)
    with pytest.raises(i8.Int8mmError):
        i8.fp8_matmul_config(0, 32, 64)
