"""Mixture-of-experts operators and the sandwich norm on the GPU at the edges:
in a row, in captured graphs, on other streams, on given memory, at the size
limits; tolerances as derived in test_moe_gpu.py."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8
from oracle import fp8_block as F
from oracle import moe as O
from tests.test_moe_gpu import E4M3, TYPES, Case, experts_of, f64, near, norm_bounds, raw, rows

pytestmark = pytest.mark.gpu


def same(a, b):
    return all(torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8)) for u, v in zip(a, b))


class Block:
    """Norm, router, experts, norm, as a decoder layer has them in a row."""

    def __init__(self, M, K, I, E, k, dtype, seed=1):
        self.M, self.K, self.k, self.dtype = M, K, k, dtype
        self.x, self.r = rows(M, K, dtype, seed), rows(M, K, dtype, seed + 1)
        self.post, self.pre = ((1 + 0.1 * rows(1, K, dtype, seed + s, outliers=0)[0].float()).to(dtype) for s in (2, 3))
        self.gate = rows(1, K, dtype, seed + 4, std=1.0, outliers=0)[0]
        self.router = (rows(E, K, dtype, seed + 5, std=1.0, outliers=0).float() / K ** 0.5).to(dtype)
        self.up_q, self.up_s = experts_of(E, 2 * I, K, seed + 6)
        self.down_q, self.down_s = experts_of(E, K, I, seed + 7)
        pack = lambda q: i8.fp8_pack_experts(torch.from_numpy(q).cuda().view(E4M3))  # noqa: E731
        self.w = (pack(self.up_q), torch.from_numpy(self.up_s).cuda(), pack(self.down_q), torch.from_numpy(self.down_s).cuda())

    def run(self, stream=None):
        y, h = i8.fp8_sandwich_norm(self.x, self.r, self.post, self.pre, gate=self.gate, quantize=False, stream=stream)
        e, p = i8.moe_route(y, self.router, self.k, stream=stream)
        z = i8.fp8_moe(y, e, p, *self.w, stream=stream)
        q, s, h2 = i8.fp8_sandwich_norm(z, h, self.post, self.pre, stream=stream)
        return y, h, e, p, z, q, s, h2

    def change(self, seed):
        self.x.copy_(rows(self.M, self.K, self.dtype, seed))
        self.r.copy_(rows(self.M, self.K, self.dtype, seed + 1))


# sizes that take each kernel: pairs alone, columns split, shared tiles, and the
# router's sums in 64 bits and by matrix instructions
BLOCKS = [(1, 528, 272, 16, 4), (3, 528, 272, 64, 4), (13, 528, 272, 16, 4), (45, 528, 272, 16, 4),
          (330, 1040, 144, 120, 6)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,I,E,k", BLOCKS)
def test_block_in_a_row(M, K, I, E, k, dtype):
    """Each stage against 64 bits from what the stage before left."""
    b = Block(M, K, I, E, k, dtype)
    y, h, e, p, z, q, s, h2 = b.run()
    eps = float(np.float32(1e-6))
    post, pre = f64(b.post), f64(b.pre)
    h64, dh, y64, dy = norm_bounds(f64(b.x), f64(b.r), post, pre, f64(b.gate)[None], 1.0, eps)
    near(h, h64, dh, dtype, "H")
    near(y, y64, dy, dtype, "Y")
    oe, op = O.route64(f64(y), f64(b.router), k, True)
    assert np.array_equal(e.cpu().numpy(), oe) and np.allclose(f64(p), op, rtol=2e-4)
    kb = lambda n: -(-n // 128)  # noqa: E731
    sums = ((128 + kb(K) + 8) * 2.0 ** -23, (256 + kb(I) + 8) * 2.0 ** -23)
    near(z, *O.moe64(f64(y), oe, p.cpu().numpy(), b.up_q, b.up_s, b.down_q, b.down_s, sums), dtype, "Z")
    h64, dh, y64, dy = norm_bounds(f64(z), f64(h), post, pre, None, 1.0, eps)
    near(h2, h64, dh, dtype, "H2")
    got = F.e4m3_decode(raw(q)) * F.spread_columns(f64(s), K)
    assert np.linalg.norm(got - y64) <= 2.0 ** -4 * np.linalg.norm(y64)


@pytest.mark.parametrize("M,K,I,E,k", BLOCKS)
def test_graph_replays(M, K, I, E, k):
    """Captured once and replayed with new inputs, whose tokens go to other
    experts, eager work between; two graphs in turn."""
    blocks = [Block(M, K, I, E, k, torch.bfloat16, seed) for seed in (1, 40)]
    graphs = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = b.run()
        graphs.append((graph, out))
    for t in range(4):
        for b, (graph, out) in zip(blocks, graphs):
            b.change(100 + 2 * t)
            graph.replay()
        wants = [b.run() for b in blocks]
        torch.cuda.synchronize()
        for (_, out), want in zip(graphs, wants):
            assert same(out, want), t


CAPTURE = """
import sys
import torch
sys.path.insert(0, {root!r})
import int8_mixed_precision_outlier_amd as i8
M, K, I, E, k = {sizes}
g = torch.Generator(device="cuda").manual_seed(1)
code = lambda *s: i8.fp8_pack_experts(torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn))
scale = lambda *s: torch.rand(s, generator=g, device="cuda") * 1e-3
half = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
b = lambda n: -(-n // 128)
w = (code(E, 2 * I, K), scale(E, b(2 * I), b(K)), code(E, K, I), scale(E, b(K), b(I)))
x, r, post, router = half(M, K), half(M, K), half(K), half(E, K)
def chain():
    y, h = i8.fp8_sandwich_norm(x, r, post, post, quantize=False)
    e, p = i8.moe_route(y, router, k)
    z = i8.fp8_moe(y, e, p, *w)
    return (y, h, e, p, z, *i8.fp8_sandwich_norm(z, h, post, post))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = chain()
for t in range(3):
    x.copy_(half(M, K))
    graph.replay()
    torch.cuda.synchronize()
    want = chain()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, want)), t
print("replays equal")
"""


@pytest.mark.parametrize("sizes", [(1, 528, 272, 16, 4), (13, 528, 272, 16, 4), (330, 1040, 144, 120, 6), (5000, 528, 16, 64, 1)])
def test_first_calls_of_a_process_inside_a_capture(sizes):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURE.format(root=root, sizes=sizes)], capture_output=True, text=True,
                       timeout=100)
    assert r.returncode == 0 and r.stdout.strip() == "replays equal", r.stderr[-2000:]


def test_two_streams_overlap():
    """Calls in turn on two streams, enqueued faster than they run, give what they
    give alone."""
    blocks = [Block(45, 2064, 1040, 24, 4, torch.bfloat16, 1), Block(13, 2064, 2064, 16, 4, torch.float16, 30)]
    alone = [b.run() for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = []
    for _ in range(20):
        for k, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got.append((k, blocks[k].run()))
    torch.cuda.synchronize()
    for k, out in got:
        assert same(out, alone[k])


def test_capture_on_a_given_stream():
    b = Block(13, 528, 272, 16, 4, torch.bfloat16)
    stream = torch.cuda.Stream()
    b.run(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = b.run(stream)
    for t in range(4):
        b.change(50 + 2 * t)
        graph.replay()
        want = b.run()
        torch.cuda.synchronize()
        assert same(out, want), t


def test_tensors_given_to_another_stream_may_be_dropped():
    """A call with `stream` reads tensors of the current stream; while that stream
    is busy, new tensors get other memory than operands that the caller dropped."""
    stream = torch.cuda.Stream()
    big = torch.zeros((4096, 16384), device="cuda", dtype=torch.bfloat16)
    busy = [*i8.fp8_quantize(big), *i8.fp8_quantize_weight(big.t().contiguous())]
    del big
    c = Case(24, 1040, 528, 8, 2, torch.bfloat16)
    x, e, p, *w = c.gpu()
    post, router = rows(1, 1040, torch.bfloat16, 2)[0], rows(8, 1040, torch.bfloat16, 3)
    calls = [(i8.fp8_sandwich_norm, lambda: (x.clone(), x.clone(), post.clone(), post.clone(), post.clone())),
             (i8.moe_route, lambda: (x.clone(), router.clone(), 2)),
             (i8.fp8_moe, lambda: (x.clone(), e.clone(), p.clone(), *(t.clone() for t in w))),
             (i8.fp8_pack_experts, lambda: (torch.from_numpy(c.up).cuda().view(E4M3),)),
             (i8.fp8_quantize_experts, lambda: (rows(48, 1040, torch.bfloat16, 4).view(3, 16, 1040),))]
    for call, operands in calls:
        want = call(*operands())
        args = operands()
        torch.cuda.synchronize()
        for _ in range(24):
            i8.fp8_matmul(*busy, stream=stream)
        got = call(*args, stream=stream)
        held = [(a.data_ptr(), a.shape, a.dtype) for a in args if isinstance(a, torch.Tensor)]
        del args
        new = [torch.empty(shape, dtype=dtype, device="cuda") for _, shape, dtype in held for _ in range(2)]
        assert not stream.query(), "the stream was to be busy meanwhile"
        assert not {t.data_ptr() for t in new} & {q for q, _, _ in held}, call
        for t in new:
            t.view(torch.uint8).fill_(0x7f)
        torch.cuda.synchronize()
        assert same(got if isinstance(got, tuple) else [got], want if isinstance(want, tuple) else [want]), call


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("M,K,I,E,k", [(1, 144, 272, 3, 2), (2, 144, 272, 30, 3), (9, 400, 80, 4, 2), (33, 272, 144, 5, 2),
                                       (300, 144, 48, 70, 6)])
def test_given_memory(M, K, I, E, k):
    """Workspace of any contents; nothing is written in front of, between or behind
    the workspace and the outputs, and inputs stay as they are."""
    c = Case(M, K, I, E, k, torch.float16, seed=4)
    c.experts.reshape(-1)[::3] = -1
    args = c.gpu()
    x, e, p, up, us, down, ds = args
    want = i8.fp8_moe(*args)
    copies = [t.clone() for t in args]
    lib = i8.load()
    size = lib.fp8_moe_workspace_size(M, K, I, E, k)
    for fill in (0x00, 0x7f, 0xff):
        ws = torch.full((size + 512,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((M * K + 64,), 5.0, dtype=torch.float16, device="cuda")
        y = out[32:32 + M * K]
        assert lib.fp8_moe(ptr(x), 0, M, K, ptr(e), ptr(p), k, ptr(up), ptr(us), ptr(down), ptr(ds), I, E, ptr(y),
                           ctypes.c_void_p(ws.data_ptr() + 256), size, None) == 0
        torch.cuda.synchronize()
        assert torch.equal(y.view(M, K), want)
        assert bool((out[:32] == 5).all()) and bool((out[32 + M * K:] == 5).all())
        assert bool((ws[:256] == fill).all()) and bool((ws[256 + size:] == fill).all())
    assert same(args, copies)


@pytest.mark.parametrize("M,K,E,k", [(3, 144, 7, 3), (300, 2064, 70, 5), (4100, 144, 65, 2)])
def test_route_given_memory(M, K, E, k):
    x, w = rows(M, K, torch.bfloat16, 1), rows(E, K, torch.bfloat16, 2)
    want = i8.moe_route(x, w, k)
    lib = i8.load()
    size = lib.moe_route_workspace_size(M, K, E, k)
    for fill in (0x00, 0x7f, 0xff):
        ws = torch.full((size + 512,), fill, dtype=torch.uint8, device="cuda")
        e = torch.full((M * k + 64,), -7, dtype=torch.int32, device="cuda")
        p = torch.full((M * k + 64,), -7.0, device="cuda")
        at = lambda t: ctypes.c_void_p(t.data_ptr() + 4 * 31)  # noqa: E731
        assert lib.moe_route(ptr(x), ptr(w), 1, M, K, E, k, 1, at(e), at(p), ctypes.c_void_p(ws.data_ptr() + 256), size,
                             None) == 0
        torch.cuda.synchronize()
        n = slice(31, 31 + M * k)
        assert torch.equal(e[n].view(M, k), want[0]) and torch.equal(p[n].view(M, k), want[1])
        for t in (e, p):
            assert bool((t[:31] == -7).all()) and bool((t[31 + M * k:] == -7).all())
        assert bool((ws[:256] == fill).all()) and bool((ws[256 + size:] == fill).all())


@pytest.mark.parametrize("M,K", [(1, 144), (17, 1040), (600, 272), (3, 12304)])
def test_sandwich_norm_leaves_memory_behind(M, K):
    x, r = rows(M, K, torch.bfloat16, 1), rows(M, K, torch.bfloat16, 2)
    w, kb = x[0].contiguous(), -(-K // 128)
    q = torch.full((M * K + 512,), 1.0, device="cuda").to(E4M3)
    s = torch.full((kb * M + 64,), 7.0, device="cuda")
    bufs = [torch.full((M * K + 64,), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    H, Y = (b[32:32 + M * K].view(M, K) for b in bufs)
    out = (q[256:256 + M * K].view(M, K), s[32:32 + kb * M].view(kb, M))
    assert same(i8.fp8_sandwich_norm(x, r, w, w, residual_out=H, out=out), i8.fp8_sandwich_norm(x, r, w, w))
    assert same(i8.fp8_sandwich_norm(x, r, w, w, quantize=False, residual_out=H, out=Y),
                i8.fp8_sandwich_norm(x, r, w, w, quantize=False))
    assert bool((q[:256].float() == 1).all()) and bool((q[256 + M * K:].float() == 1).all())
    assert bool((s[:32] == 7).all()) and bool((s[32 + kb * M:] == 7).all())
    for b in bufs:
        assert bool((b[:32] == 9).all()) and bool((b[32 + M * K:] == 9).all())


# ---- size limits -------------------------------------------------------------

def codes(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("M,k", [(1, 3), (20, 3), (200, 3), (300, 4)])
def test_experts_past_four_gigabytes(M, k):
    """600 experts of 8 and 4 MB: byte offsets past 32 bits; tokens at the first, a
    middle and the last experts, through each kernel."""
    E, K, I = 600, 2048, 2048
    up, down = codes(E, 2 * I, K, seed=1).view(E4M3), codes(E, K, I, seed=2).view(E4M3)
    g = torch.Generator(device="cuda").manual_seed(3)
    us, ds = (torch.rand((E, a, b), generator=g, device="cuda") * 2e-4 for a, b in ((32, 16), (16, 16)))
    x = rows(M, K, torch.bfloat16, 4, std=1.0, outliers=0)
    used = [0, 301, E - 1, E - 2]
    experts = torch.tensor(used[:k], dtype=torch.int32, device="cuda").expand(M, k).contiguous()
    weights = torch.rand((M, k), generator=g, device="cuda")
    pu, pd = i8.fp8_pack_experts(up), i8.fp8_pack_experts(down)
    Y = i8.fp8_moe(x, experts, weights, pu, us, pd, ds)
    place = {e: n for n, e in enumerate(used)}
    few = np.vectorize(place.get)(experts.cpu().numpy()).astype(np.int32)
    pick = torch.tensor(used, device="cuda")
    sums = ((128 + 16 + 8) * 2.0 ** -23, (256 + 16 + 8) * 2.0 ** -23)
    m = sorted({0, M // 2, M - 1})
    near(Y[m], *O.moe64(f64(x[m]), few[m], weights.cpu().numpy()[m], raw(up.view(torch.uint8)[pick]),
                        us[pick].cpu().numpy(), raw(down.view(torch.uint8)[pick]), ds[pick].cpu().numpy(), sums),
         torch.bfloat16, (M, k))
    del up, down, pu, pd
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [1, 5, 20])
def test_largest_expert(M):
    """Experts whose first matrix has 2^31 bytes; tokens that are zero but for their
    first and last columns, results of the first and last features."""
    E, K, I = 2, 65536, 16384
    up, down = codes(E, 2 * I, K, seed=5).view(E4M3), codes(E, K, I, seed=6).view(E4M3)
    g = torch.Generator(device="cuda").manual_seed(7)
    us, ds = (torch.rand((E, a, b), generator=g, device="cuda") * 2e-4 for a, b in ((256, 512), (512, 128)))
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    cols = torch.cat([torch.arange(128), torch.arange(K - 128, K)]).cuda()
    x[:, cols] = rows(M, 256, torch.bfloat16, 8, std=1.0, outliers=0)
    experts = torch.tensor([1, 0], dtype=torch.int32, device="cuda").expand(M, 2).contiguous()
    weights = torch.rand((M, 2), generator=g, device="cuda")
    Y = i8.fp8_moe(x, experts, weights, i8.fp8_pack_experts(up), us, i8.fp8_pack_experts(down), ds)
    for first in (0, K - 128):
        f = slice(first, first + 128)
        few = (raw(up.view(torch.uint8)[:, :, cols]), us[:, :, [0, 511]].cpu().numpy(),
               raw(down.view(torch.uint8)[:, f]), ds[:, first // 128:first // 128 + 1].cpu().numpy())
        y, tol = moe_features(f64(x[:, cols]), experts.cpu().numpy(), weights.cpu().numpy(), *few)
        near(Y[:, f], y, tol, torch.bfloat16, (M, first))
    del up, down, us, ds, Y
    torch.cuda.empty_cache()


def moe_features(x, experts, weights, up, us, down, ds):
    """O.moe64 for some features of the result: down [E, features, I].  Columns
    that are left out add nothing, and their blocks' sums of zeros no error."""
    pad = np.zeros((x.shape[0], down.shape[1]))
    n = down.shape[1]
    assert n == 128 and x.shape[1] == 256
    out = [np.zeros_like(pad), np.zeros_like(pad)]
    for e in range(len(up)):
        # as two experts' products with an x of 256 columns
        wu = O.weight64(up[e], us[e])
        gu = x @ wu.T
        err = (128 + 2 + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(wu).T)
        I = gu.shape[1] // 2
        a = F.silu_mul64(gu)
        silu = F.silu_mul64(np.concatenate([gu[:, :I], np.ones((len(x), I))], 1))
        da = 1.1 * err[:, :I] * (np.abs(gu[:, I:]) + err[:, I:]) + np.abs(silu) * err[:, I:]
        da = da + (8 * 2.0 ** -24 + 2.0 ** -17) * (np.abs(a) + da)
        wd = O.weight64(down[e], ds[e])
        for j in range(experts.shape[1]):
            assert (experts[:, j] == experts[0, j]).all()
            if experts[0, j] != e:
                continue
            p = weights[:, j:j + 1].astype(np.float64)
            out[0] += p * (a @ wd.T)
            out[1] += p * (da @ np.abs(wd).T + (256 + 128 + 9) * 2.0 ** -23 * ((np.abs(a) + da) @ np.abs(wd).T))
    return out[0], out[1] + 2 * 2.0 ** -23 * (np.abs(out[0]) + out[1])


@pytest.mark.parametrize("M,k,E", [(4096, 2, 1024), (256, 32, 1024), (8192, 1, 3), (1, 32, 1024), (2, 32, 1024)])
def test_most_pairs_and_experts(M, k, E):
    c = Case(M, 144, 48, E, k, torch.bfloat16, seed=21)
    c.experts[:, 0] = E - 1
    c.check(what=(M, k, E))
    c.experts[:] = 1  # all pairs at one expert
    c.check(what=(M, k, E, "one"))


@pytest.mark.parametrize("M,K,E,k", [(1 << 18, 16, 128, 8), (1 << 18, 16, 1024, 2), ((1 << 18) - 3, 144, 8, 8),
                                     (32768, 65536, 4, 2)])
def test_route_most_tokens(M, K, E, k):
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for m in range(0, M, 4096):
        x[m:m + 4096] = torch.randn((min(4096, M - m), K), generator=g, device="cuda")
    w = (torch.randn((E, K), generator=g, device="cuda") / K ** 0.5).bfloat16()
    e, p = i8.moe_route(x, w, k, normalize=False)
    for m in (slice(0, 64), slice(M // 2, M // 2 + 64), slice(M - 64, M)):
        oe, op = O.route64(f64(x[m]), f64(w), k, False)
        assert np.array_equal(e[m].cpu().numpy(), oe) and np.allclose(f64(p[m]), op, rtol=1e-4)
    assert int(e.min()) >= 0 and int(e.max()) < E
    del x, e, p
    torch.cuda.empty_cache()


@pytest.mark.parametrize("quantize", [True, False])
@pytest.mark.parametrize("M,K", [(4096, 12288), (12000, 4096), (24000, 2048), (90000, 512), (3000, 16384), (1500, 32784),
                                 (1000, 65536)])
def test_sandwich_norm_past_the_cache(M, K, quantize):
    """Rows of more bytes than the last-level cache holds: what a call on a few of
    them gives, bit for bit."""
    x, r = rows(64, K, torch.bfloat16, 1), rows(64, K, torch.bfloat16, 2)
    post, pre, gate = (rows(1, K, torch.bfloat16, s, outliers=0)[0] for s in (3, 4, 5))
    n = -(-M // 64)
    call = lambda a, b: i8.fp8_sandwich_norm(a, b, post, pre, gate=gate, quantize=quantize)  # noqa: E731
    want = call(x, r)
    got = call(x.repeat(n, 1)[:M], r.repeat(n, 1)[:M])
    for a, b, tokens_last in zip(got, want, (False, quantize, False)):
        b = b.repeat(1, n)[:, :M] if tokens_last else b.view(torch.uint8).repeat(n, 1)[:M]
        assert torch.equal(a if tokens_last else a.view(torch.uint8), b)
    del got
    torch.cuda.empty_cache()


def test_sandwich_norm_at_the_size_limit():
    """2^31 elements, and more rows than one launch takes: the last rows."""
    for M, K, G in ((32768, 65536, 2), ((1 << 21) + 6, 16, (1 << 20) + 3)):
        x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
        r = torch.full((M, K), 2.0, dtype=torch.bfloat16, device="cuda")
        x[-3:], r[-3:] = rows(3, K, torch.bfloat16, 1), rows(3, K, torch.bfloat16, 2)
        w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
        gate = torch.full((G, K), 0.5, dtype=torch.bfloat16, device="cuda")
        gate[-1] = 0.25
        y, h = i8.fp8_sandwich_norm(x, r, w, w, gate=gate, quantize=False, residual_out=r if G > 2 else None)
        res = rows(3, K, torch.bfloat16, 2)
        each = M // G
        last = f64(gate)[[(M - 3 + i) // each for i in range(3)]] if K == 16 else np.repeat(f64(gate[-1:]), 3, 0)
        h64, dh, y64, dy = norm_bounds(f64(x[-3:]), f64(res), f64(w), f64(w), last, 1.0, float(np.float32(1e-6)))
        near(h[-3:], h64, dh, torch.bfloat16, "H")
        near(y[-3:], y64, dy, torch.bfloat16, "Y")
        assert bool((h[:each] == 2.5).all()) and bool((y[:-3] == 1).all())
        del x, r, y, h
        torch.cuda.empty_cache()
