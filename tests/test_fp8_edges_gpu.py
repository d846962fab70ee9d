"""Block-scaled e4m3 operators on the GPU at the edges of their ranges, against
the 64-bit oracle (oracle/fp8_block.py)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8
from oracle import fp8_block as F

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]
E4M3 = torch.float8_e4m3fn


def f32(t):
    return t.detach().float().cpu().numpy()


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# Half steps (2^-24) of the gated product: the exponential instruction 2, its
# correction 1, the fma that joins them to 1 + exp(-g) 1, the reciprocal
# instruction 2, the products with gate and up 1 each; a hundredth for the
# second-order terms.  The argument's remainder and log2(e)'s are in the
# correction, the scalings by powers of two are exact.  The division by 448 adds
# one to the scale's.
GATE = 8.01 * 2.0 ** -24


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_silu_mul_far_gates(dtype):
    """Gates whose 1 / (1 + exp(-g)) is no normal fp32 number, and subnormal
    gates, beside ups of the type's largest.  Each block holds one value."""
    top, least = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    gates = [-86.0, -87.0, -87.25, -87.5, -88.0, -88.25, -88.5, least, -least, 5 * least]
    if dtype == torch.float16:
        gates += [-87.3125, -87.375, -88.6875]
    ups = [top, -top, top / 16, 1e30 if dtype == torch.bfloat16 else 1e3]
    GU = torch.tensor([(g, u) for g in gates for u in ups], dtype=torch.float64).to(dtype)
    q, s = i8.fp8_silu_mul(GU[:, :, None].expand(-1, -1, 128).reshape(-1, 256).cuda())
    y = F.silu_mul64(f32(GU))[:, 0]
    s, v = s[0].cpu().numpy().astype(np.float64), F.e4m3_decode(raw(q))
    s64 = np.maximum(np.abs(y), 2.0 ** -100) / 448
    assert np.all(np.abs(s - s64) <= (GATE + 2.0 ** -24) * s64), (GU, s / s64 - 1)
    want = (y / s)[:, None]
    tol = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10) + (2 * GATE + 2.0 ** -22) * np.abs(want)
    assert np.all(np.abs(v - want) <= tol), GU[np.any(np.abs(v - want) > tol, 1)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_silu_mul_gates_past_exp(dtype):
    """exp(-g) past fp32's range: a zero, whatever the finite up."""
    top = torch.finfo(dtype).max
    GU = torch.tensor([(g, u) for g in (-89.0, -100.0, -top) for u in (top, -top, 1.0)], dtype=torch.float64)
    q, _ = i8.fp8_silu_mul(GU.to(dtype)[:, :, None].expand(-1, -1, 128).reshape(-1, 256).cuda())
    assert not np.any(F.e4m3_decode(raw(q)))


def integers(rows, cols, seed):
    """e4m3 codes of the integers -4 .. 4 on the GPU."""
    table = torch.from_numpy(F.e4m3_encode(np.arange(-4, 5))).cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        out[r:r + n] = table[torch.randint(0, 9, (n, cols), generator=g, device="cuda", dtype=torch.int32)]
    return out


@pytest.mark.parametrize("K", [65536, 65520])
@pytest.mark.parametrize("M,N", [(1, 32768), (40, 32768), (32768, 16), (130, 32768)])
def test_matmul_ends_of_the_largest_operands(M, N, K):
    """Operands of up to 2^31 bytes.  The tokens are zero but for the first and
    the last K block, the scales are one, so the product is a sum of 256
    integers at most, exact up to the result's rounding: a last block that is
    not read, or read from elsewhere, shows."""
    x, w = integers(M, K, 1), integers(N, K, 2)
    last = (K - 1) // 128 * 128
    x[:, 128:last] = 0
    ones = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    Y = i8.fp8_matmul(x.view(E4M3), ones(-(-K // 128), M), i8.fp8_pack_weight(w.view(E4M3)),
                      ones(-(-N // 128), -(-K // 128)), out_dtype=torch.float16)
    m = sorted({0, M // 2, max(0, M - 3), max(0, M - 2), M - 1})
    n = [*range(16), *range(N - 16, N)] if N > 32 else list(range(N))
    want = F.e4m3_decode(raw(x[m])) @ F.e4m3_decode(raw(w[n])).T
    assert np.array_equal(Y[m][:, n].cpu().numpy(), want.astype(np.float16))
    assert len(np.unique(want)) > 2
    if M > 1:  # every row has a last block of its own
        assert not torch.equal(Y[-1], Y[-2])


def test_two_streams_overlap():
    """Calls in turn on two streams, enqueued faster than they run, give what
    they give alone."""
    def operands(M, K, N, seed):
        x, w = integers(M, K, seed).view(E4M3), i8.fp8_pack_weight(integers(N, K, seed + 1).view(E4M3))
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
        return x, rnd(K // 128, M), w, rnd(-(-N // 128), K // 128)
    args = [operands(40, 12288, 12288, 1), operands(300, 8192, 8192, 3)]
    gate = [torch.randn((512, 16384), device="cuda").to(torch.bfloat16) for _ in args]
    call = lambda k: (i8.fp8_matmul(*args[k]), *i8.fp8_silu_mul(gate[k]))  # noqa: E731
    alone = [call(k) for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    ends = [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in args]
    got = []
    for r in range(30):
        for k, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                if r == 0:
                    ends[k][0].record()
                got.append((k, call(k)))
                if r == 29:
                    ends[k][1].record()
    torch.cuda.synchronize()
    assert ends[0][0].elapsed_time(ends[1][1]) > 0 and ends[1][0].elapsed_time(ends[0][1]) > 0
    for k, outs in got:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, alone[k]))


CAPTURE = """
import sys
import torch
sys.path.insert(0, {root!r})
import int8_mixed_precision_outlier_amd as i8
M, N, K = {sizes}
assert i8.fp8_matmul_config(M, N, K)[0] == {kind!r}
g = torch.Generator(device="cuda").manual_seed(1)
code = lambda *s: torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
w = i8.fp8_pack_weight(code(N, K))
ws = torch.rand((-(-N // 128), -(-K // 128)), device="cuda") * 1e-3
x, res = (torch.randn((M, K), generator=g, device="cuda").bfloat16() for _ in range(2))
weight = x[0].clone()
def chain():
    q, s, h = i8.fp8_rms_norm(x, weight, residual=res)
    y = i8.fp8_matmul(q, s, w, ws)
    return (q, s, h, y, *i8.fp8_silu_mul(y), *i8.fp8_quantize(h))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = chain()
for k in range(3):
    x.copy_(torch.randn((M, K), generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    want = chain()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, want)), k
print("replays equal")
"""


@pytest.mark.parametrize("sizes,kind", [((5, 4096, 528), "decode"), ((200, 2080, 528), "tiled"),
                                        ((1900, 9600, 272), "split")])
def test_first_calls_of_a_process_inside_a_capture(sizes, kind):
    """A process whose first norm, product, gate and quantizer are captured: no
    module is loaded and no limit raised before the capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE.format(root=root, sizes=sizes, kind=kind)],
                       capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout.strip() == "replays equal", r.stderr[-2000:]


def unpacked(w, N, KB):
    """The packed weight's rows, for blocks of 16 rows at a time: [N, KB * 128]."""
    return w.view(torch.uint8).view(-1, KB, 8, 16, 16).permute(0, 3, 1, 2, 4).reshape(N, KB * 128)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K,N", [(4096, 12288), (5136, 20464), (65536, 32768), (65520, 32752), (16, 1 << 24)])
def test_quantize_weight_large(K, N, dtype):
    """Every scale and number of large weights, bit for bit, 128 features at a
    time for some of them and the last: the quotients are those of 64 bits
    rounded to 32, which is what a 32-bit division gives."""
    KB = -(-K // 128)
    g = torch.Generator(device="cuda").manual_seed(K + N)
    W = torch.empty((K, N), dtype=dtype, device="cuda")
    for k in range(0, K, 4096):
        rows = min(4096, K - k)
        for n in range(0, N, 1 << 20):
            cols = min(1 << 20, N - n)
            W[k:k + rows, n:n + cols] = torch.randn((rows, cols), generator=g, device="cuda") * 0.02
    w, ws = i8.fp8_quantize_weight(W)
    assert w.shape == (N, KB * 128) and ws.shape == (-(-N // 128), KB)
    nbs = sorted({*range(0, ws.shape[0], max(1, ws.shape[0] // 12)), ws.shape[0] - 1})
    for nb in nbs:
        cols = slice(nb * 128, min(N, nb * 128 + 128))
        n = cols.stop - cols.start
        t = torch.zeros((n, KB * 128), device="cuda")
        t[:, :K] = W[:, cols].t().float()
        t = t.view(n, KB, 128)
        a = t.abs().amax((0, 2)).clamp(min=2.0 ** -100).double()
        assert torch.equal(ws[nb], (a / 448).float()), nb
        q = (t * (448 / a).float()[None, :, None]).view(n, KB * 128).to(E4M3)
        assert torch.equal(unpacked(w[cols], n, KB), q.view(torch.uint8)), nb


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_silu_mul_blocks_of_all_magnitudes(dtype):
    """Blocks whose maximum lies at either side of 2^120 and of fp32's range,
    next to ordinary blocks of the same rows: the gated products in 64 bits."""
    rng = np.random.default_rng(8)
    M, K = 37, 640
    big = np.log2(float(torch.finfo(dtype).max))
    gate = rng.uniform(-6, 6, (M, K))
    up = rng.standard_normal((M, K))
    for m in range(M):
        for b in range(5):
            c = b * 128 + int(rng.integers(128))  # one large product per block
            lg, lu = (rng.uniform(0, big - 0.01, 2) if (m + b) % 3 else (1.0, 0.0))
            gate[m, c], up[m, c] = 2.0 ** lg, rng.choice([-1, 1]) * 2.0 ** lu
    GU = torch.from_numpy(np.concatenate([gate, up], 1)).to(dtype)
    q, s = i8.fp8_silu_mul(GU.cuda())
    y = F.silu_mul64(f32(GU))
    s, v = s.cpu().numpy().astype(np.float64), F.e4m3_decode(raw(q))
    a = np.abs(y).reshape(M, 5, 128).max(2).T
    inside, past = a < (1 - 2.0 ** -20) * 2.0 ** 128, a > (1 + 2.0 ** -20) * 2.0 ** 128
    assert np.all(np.abs(s - a / 448)[inside] <= (GATE + 2.0 ** -24) * a[inside] / 448)
    assert np.all(np.isinf(s[past]))
    ok = np.repeat(inside.T, 128, 1)
    want = y / np.repeat(np.where(inside, s, 1.0).T, 128, 1)
    tol = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10) + (2 * GATE + 2.0 ** -22) * np.abs(want)
    assert np.all((np.abs(v - want) <= tol)[ok])
    if dtype == torch.bfloat16:
        assert past.any() and (inside & (a > 2.0 ** 120)).any()


@pytest.mark.parametrize("M,N", [(1, 1 << 24), (128, (1 << 24) - 16), (1 << 27, 16), ((1 << 26) - 5, 32)])
def test_matmul_most_features_and_tokens(M, N):
    """The largest counts of features and of tokens that K = 16 allows: the
    first, middle and last ones, exactly."""
    K = 16
    x, w = integers(M, K, 5), integers(N, K, 6)
    ones = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    Y = i8.fp8_matmul(x.view(E4M3), ones(1, M), i8.fp8_pack_weight(w.view(E4M3)), ones(-(-N // 128), 1),
                      out_dtype=torch.float16)
    for m in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(max(0, M - 300), M)):
        for n in (slice(0, 300), slice(N // 2, N // 2 + 300), slice(max(0, N - 300), N)):
            want = F.e4m3_decode(raw(x[m])) @ F.e4m3_decode(raw(w[n])).T
            assert np.array_equal(Y[m, n].cpu().numpy(), want.astype(np.float16)), (m, n)
    del x, w, Y
    torch.cuda.empty_cache()


def test_capture_on_a_given_stream():
    """Calls captured on the stream that they are given, with temporaries that
    are dropped inside: every replay gives what eager calls give."""
    K, N, M = 528, 272, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, weight = rnd(M, K), i8.fp8_quantize_weight(rnd(K, 2 * N)), rnd(K)

    def chain(stream):
        q, s, h = i8.fp8_rms_norm(x, weight, residual=x, stream=stream)
        gu = i8.fp8_matmul(q, s, *w, stream=stream)
        del q, s
        return h, *i8.fp8_silu_mul(gu, stream=stream)
    stream = torch.cuda.Stream()
    chain(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = chain(stream)
    for k in range(4):
        x.copy_(rnd(M, K))
        graph.replay()
        want = chain(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, want)), k
