"""Mixture-of-experts operators and the sandwich norm on the GPU, through the
public entry points, against the 64-bit oracle (oracle/moe.py).

Tolerances, derived:
  norms    the first norm's factor: a sum of squares is a chain of at most 64
           fma per thread, 6 shuffle steps and 16 wavefront sums of positive
           terms, 86 * 2^-24 relative, halved by the square root, and at most 6
           more half steps for the division, + eps, sqrt, the reciprocal; with
           three products (weight, gate, the factor) |dz| <= 52 * 2^-24 |z|.
           h adds the scaled residual and one fma: |dh| <= |dz| + 2^-24 (|z| +
           2 |alpha r| + |h|).  The second factor is off by what dh, in the
           2-norm, is of h, and by 49 * 2^-24 again; y takes two products.
           H and Y are then off by half a step of their type, e4m3 numbers by
           2^-4 (or 2^-10 below the smallest normal number), scales by the
           largest dy of their block over 448 and two half steps.
  router   the order is exact: logits in tests differ by far more than 64-bit
           sums err, or not at all.  Weights: the difference of two logits,
           rounded to fp32, is off by 2^-24 of itself, and so is its
           exponential by that times |difference|; expf 2 half steps (1 ulp),
           the sum of up to 1024 terms 16 + 6 additions, two divisions, the sum
           over the chosen ones 32: (64 + |l - max|) * 2^-24.  Above 2^25 products
           (tokens x columns x experts) a logit is a 64-bit sum of fp32 sums of 32
           exact products: 31 additions each within 2^-23 of the running
           magnitude, so it is off by b = 32 * 2^-23 sum |x w| at most, and a
           weight by the factor exp(2 b) of the largest b of its token: its own
           exponential's and the sum's.
  experts  a block of 128 columns: 4 instructions of 32 exact products, each of
           whose additions is within 2^-23 of the running magnitude, then one fma
           per block and at most 8 partial sums: (128 + KB + 8) * 2^-23 of the
           sum of magnitudes; twice the additions where the left operand is the
           sum of two numbers.  The gated product and its two bf16 parts as in
           the oracle.  Then half a step of Y's type and half its smallest
           subnormal.
"""
import numpy as np
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8
from oracle import fp8_block as F
from oracle import moe as O

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]
E4M3 = torch.float8_e4m3fn
H = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def rows(M, K, dtype, seed, std=0.5, outliers=7):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * std
    for c in rng.choice(K, min(outliers, K // 16), replace=False):
        x[:, c] *= 60
    return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()


def near(got, want, tol, dtype, what):
    """`got` of a 16-bit type against a value and what it may be off before its rounding."""
    fi = torch.finfo(dtype)
    tol = tol + fi.eps / 2 * (np.abs(want) + tol) + fi.smallest_normal * fi.eps / 2
    off = np.abs(f64(got) - want)
    assert np.all(off <= tol), (what, float(np.max(off - tol)), float(np.max(off)))


# ---- norms -------------------------------------------------------------------

def norm_bounds(x, r, post, pre, gate, alpha, eps):
    h, y, z = O.sandwich64(x, r, post, pre, gate, alpha, eps)
    dh = 52 * H * np.abs(z) + H * (np.abs(z) + 2 * np.abs(alpha * r) + np.abs(h))
    size = lambda v: np.sqrt((v * v).sum(1, keepdims=True))  # noqa: E731
    factor = np.abs(pre) / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    rel = size(dh) / np.maximum(size(h), 1e-300) + 52 * H
    return h, dh, y, (dh * factor + rel * np.abs(y)) * (1 + 1e-4)


NORMS = [(1, 16, 0), (1, 128, 1), (3, 112, 3), (4, 528, 2), (17, 1040, 0), (6, 2064, 6), (12, 4112, 4), (1, 5120, 1),
         (5, 8208, 5), (33, 12288, 1), (2, 16400, 2), (2, 32784, 0), (2, 65536, 1),
         # a row's every count of threads and chunks, many rows too
         (2, 512, 1), (2, 1024, 0), (2, 2048, 2), (2, 4096, 1), (600, 5136, 600), (2, 6144, 0), (520, 12304, 1)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,G", NORMS)
def test_sandwich_norm(M, K, G, dtype):
    x, r = rows(M, K, dtype, K + M), rows(M, K, dtype, K + M + 1)
    post, pre = ((1 + 0.2 * rows(1, K, dtype, s, outliers=0)[0].float()).to(dtype) for s in (2, 3))
    gate = rows(G, K, dtype, 4, std=1.0, outliers=0) if G else None
    if M > 2:
        x[1] = 0  # the block gave nothing: h is the residual alone
        x[2], r[2] = 0, 0  # nothing at all: y = 0, scales on the floor
    alpha, eps = (2.5, 1e-5) if G % 2 else (-0.75, 1e-6)
    a64, e64 = float(np.float32(alpha)), float(np.float32(eps))
    h, dh, y, dy = norm_bounds(f64(x), f64(r), f64(post), f64(pre), None if gate is None else f64(gate), a64, e64)
    args = dict(gate=gate, residual_scale=alpha, eps=eps)
    Y, Hs = i8.fp8_sandwich_norm(x, r, post, pre, quantize=False, **args)
    near(Hs, h, dh, dtype, "H")
    near(Y, y, dy, dtype, "Y")
    q, s, H2 = i8.fp8_sandwich_norm(x, r, post, pre, **args)
    assert torch.equal(H2, Hs)
    kb = -(-K // 128)
    pad = lambda v: np.pad(np.abs(v), ((0, 0), (0, kb * 128 - K))).reshape(M, kb, 128).max(2).T  # noqa: E731
    s64 = np.maximum(pad(y), 2.0 ** -100) / 448
    ds = pad(dy) / 448 + 2 * H * s64
    got = f64(s)
    assert np.all(np.abs(got - s64) <= ds)
    spread = F.spread_columns(got, K)
    v, want = F.e4m3_decode(raw(q)), y / spread
    off = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** -10) + (dy / spread + 2.0 ** -22 * np.abs(want)) * (1 + 2.0 ** -4)
    assert np.all(np.abs(v - want) <= off), float(np.max(np.abs(v - want) - off))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_sandwich_norm_buffers(dtype):
    """H in the residual's or X's buffer, given outputs, the gate's forms, a bad row."""
    M, K = 6, 272
    x, r = rows(M, K, dtype, 1), rows(M, K, dtype, 2)
    post, pre, gate = (rows(1, K, dtype, s, outliers=0)[0] for s in (3, 4, 5))
    want = i8.fp8_sandwich_norm(x, r, post, pre, gate=gate)
    same = lambda a, b: all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))  # noqa: E731
    r2, x2 = r.clone(), x.clone()
    got = i8.fp8_sandwich_norm(x, r2, post, pre, gate=gate[None], residual_out=r2)
    assert got[2].data_ptr() == r2.data_ptr() and same(want, got)
    assert same(want, i8.fp8_sandwich_norm(x2, r, post, pre, gate=gate.expand(M, K).contiguous(), residual_out=x2))
    out = (torch.empty((M, K), dtype=E4M3, device="cuda"), torch.empty((3, M), device="cuda"))
    got = i8.fp8_sandwich_norm(x, r, post, pre, gate=gate.expand(3, K).contiguous(), out=out)
    assert got[0] is out[0] and same(want, got)
    y = torch.empty_like(x)
    plain = i8.fp8_sandwich_norm(x, r, post, pre, gate=gate, quantize=False, out=y)
    assert plain[0] is y and torch.equal(plain[1], want[2])
    # without a gate: as with a gate of ones; the same tensor twice
    assert same(i8.fp8_sandwich_norm(x, x, post, pre),
                i8.fp8_sandwich_norm(x, x, post, pre, gate=torch.ones_like(gate)))
    # a NaN, an infinity in one row each: the other rows stay
    xb = x.clone()
    xb[2, 5], xb[4, 9] = float("nan"), float("inf")
    bad = i8.fp8_sandwich_norm(xb, r, post, pre, gate=gate, quantize=False)
    keep = [0, 1, 3, 5]
    assert torch.equal(bad[0][keep], plain[0][keep]) and torch.equal(bad[1][keep], plain[1][keep])
    assert torch.isnan(bad[0][2]).all() and torch.isnan(bad[1][2]).all()
    assert torch.isnan(bad[1][4, 9])
    for M, K in ((0, 128), (3, 0)):
        e = torch.empty((M, K), dtype=dtype, device="cuda")
        w = torch.empty(K, dtype=dtype, device="cuda")
        q, s, hh = i8.fp8_sandwich_norm(e, e, w, w, gate=w if M else None)
        assert q.shape == (M, K) and hh.shape == (M, K)


# ---- router ------------------------------------------------------------------

ROUTES = [(1, 16, 1, 1), (1, 4096, 128, 8), (3, 144, 2, 2), (5, 272, 61, 6), (64, 528, 64, 8), (65, 1040, 65, 3),
          (7, 5136, 130, 32), (300, 400, 257, 9), (2, 65536, 8, 2), (33, 256, 1000, 32), (700, 1024, 128, 8),
          # matrix instructions: every count of experts per lane, both workgroups, ragged ends
          (300, 2064, 61, 6), (17, 65536, 33, 1), (300, 2064, 257, 9), (100, 1040, 1000, 32), (2500, 272, 120, 8),
          (1031, 144, 250, 1), (4096, 80, 128, 8), (600, 80, 1024, 32)]


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,E,k", ROUTES)
def test_route(M, K, E, k, dtype, normalize):
    x = rows(M, K, dtype, M + K)
    w = (rows(E, K, dtype, E, std=1.0, outliers=0).float() / K ** 0.5).to(dtype)
    if E > 3:
        w[E - 1] = w[1]  # equal logits
    if M > 2:
        x[2] = 0  # all equal: the first experts
    experts, weights = i8.moe_route(x, w, k, normalize=normalize)
    assert experts.dtype == torch.int32 and weights.dtype == torch.float32
    oe, ow = O.route64(f64(x), f64(w), k, normalize)
    logits = f64(x) @ f64(w).T
    if E > 3:
        logits[:, E - 1] = logits[:, 1]
        oe = np.argsort(-logits, 1, kind="stable")[:, :k]
    assert np.array_equal(experts.cpu().numpy(), oe)
    far = logits.max(1, keepdims=True) - np.take_along_axis(logits, oe, 1)
    if normalize:  # the sum's terms are off by theirs
        far = far + far.max(1, keepdims=True)
    rel = (64 + far) * H * 1.01
    if M * E * K > 2 ** 25:
        b = 32 * 2.0 ** -23 * (np.abs(f64(x)) @ np.abs(f64(w)).T).max(1, keepdims=True)
        rel = rel + np.expm1(2 * b * (2 if normalize else 1))
    assert np.all(np.abs(f64(weights) - ow) <= rel * ow + 2.0 ** -149)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M", [1, 200])
def test_route_close_logits(M, dtype):
    """Logits that fp32 sums cannot tell apart: each expert's row is the same but
    for one small entry, so the order is that of the entries."""
    K, E, k = 4096, 96, 12
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(dtype)
    x[:, 7] = 1.0
    w = torch.from_numpy(np.repeat(rng.standard_normal((1, K)), E, 0).astype(np.float32)).to(dtype)
    small = 2.0 ** -24 * (1 + rng.permutation(E) / 128.0) if dtype == torch.bfloat16 else 2.0 ** -24 * (1 + rng.permutation(E))
    w[:, 7] = torch.from_numpy(small).to(dtype)
    experts, _ = i8.moe_route(x.cuda(), w.cuda(), k)
    want = np.argsort(-w[:, 7].double().numpy(), kind="stable")[:k]
    assert len(set(w[:, 7].tolist())) == E
    assert np.array_equal(experts.cpu().numpy(), np.repeat(want[None], M, 0))


@pytest.mark.parametrize("scale", [(100, 40), (-100, -30)], ids=["large", "small"])
@pytest.mark.parametrize("M", [3, 100])
def test_route_outside_fp32(M, scale):
    """Products that fp32 cannot hold, too large or too small: the order is that
    of 64 bits all the same."""
    K, E, k = 1040, 400, 8
    x = (rows(M, K, torch.bfloat16, M, std=1.0, outliers=0).float() * 2.0 ** scale[0]).bfloat16()
    w = (rows(E, K, torch.bfloat16, 2, std=1.0, outliers=0).float() * 2.0 ** scale[1]).bfloat16()
    experts, weights = i8.moe_route(x, w, k, normalize=False)
    oe, ow = O.route64(f64(x), f64(w), k, False)
    assert np.array_equal(experts.cpu().numpy(), oe)
    assert np.allclose(f64(weights), ow, rtol=64 * 2.0 ** -24, atol=2.0 ** -126)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,E", [(6, 144, 70), (40, 4112, 230), (700, 1040, 70)])
def test_route_bad_values(M, K, E, dtype):
    """NaN and infinite logits: experts stay distinct and in range; other rows stay."""
    k = 32
    x, w = rows(M, K, dtype, 1), rows(E, K, dtype, 2, std=0.1)
    we, ww = i8.moe_route(x, w, k)
    x[1, 3] = float("nan")
    x[3, 5] = float("inf")
    for normalize in (False, True):
        e, v = i8.moe_route(x, w, k, normalize=normalize)
        for m in (1, 3):
            assert sorted(set(e[m].tolist())) == sorted(e[m].tolist()) and 0 <= e[m].min() and e[m].max() < E
            assert torch.isnan(v[m]).any()
        assert e[1].tolist() == list(range(k)) and torch.isnan(v[1]).all()
        keep = [0, 2, *range(4, M)]
        assert torch.equal(e[keep], we[keep])
        if normalize:
            assert torch.equal(v[keep], ww[keep])
    # one expert's row: it ranks last, and spoils the weights of every token
    x = rows(M, K, dtype, 1)
    w[4, 0] = float("nan")
    e, v = i8.moe_route(x, w, k)
    assert torch.isnan(v).all() and not (e == 4).any()


def test_route_no_columns_and_no_tokens():
    w = torch.empty((5, 0), dtype=torch.float16, device="cuda")
    e, v = i8.moe_route(torch.empty((3, 0), dtype=torch.float16, device="cuda"), w, 2, normalize=False)
    assert e.tolist() == [[0, 1]] * 3 and torch.allclose(v, torch.full_like(v, 0.2))
    e, v = i8.moe_route(torch.empty((0, 16), dtype=torch.float16, device="cuda"),
                        torch.ones((5, 16), dtype=torch.float16, device="cuda"), 2)
    assert e.shape == v.shape == (0, 2)


# ---- experts -----------------------------------------------------------------

def experts_of(E, N, K, seed):
    """Random e4m3 bytes [E, N, K] of the middle binades and scales over some."""
    rng = np.random.default_rng(seed)
    q = (rng.integers(0, 120, (E, N, K)) | (rng.integers(0, 2, (E, N, K)) << 7)).astype(np.uint8)
    s = (2.0 ** rng.uniform(-1, 1, (E, -(-N // 128), -(-K // 128))) / (60 * K ** 0.5)).astype(np.float32)
    return q, s


class Case:
    def __init__(self, M, K, I, E, k, dtype, seed=0):
        rng = np.random.default_rng(seed + M + K)
        self.dtype, self.E = dtype, E
        self.x = rows(M, K, dtype, seed + 1, std=1.0, outliers=1)
        self.experts = rng.integers(0, E, (M, k)).astype(np.int32)
        self.weights = rng.uniform(0, 1, (M, k)).astype(np.float32)
        self.up, self.up_s = experts_of(E, 2 * I, K, seed + 2)
        self.down, self.down_s = experts_of(E, K, I, seed + 3)
        self.I = I

    def gpu(self):
        pack = lambda q: i8.fp8_pack_experts(torch.from_numpy(q).cuda().view(E4M3))  # noqa: E731
        t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        return (self.x, t(self.experts), t(self.weights), pack(self.up), t(self.up_s), pack(self.down), t(self.down_s))

    def oracle(self):
        K = self.x.shape[1]
        kb = lambda n: -(-n // 128)  # noqa: E731
        sums = ((128 + kb(K) + 8) * 2.0 ** -23, (256 + kb(self.I) + 8) * 2.0 ** -23)
        return O.moe64(f64(self.x), self.experts, self.weights, self.up, self.up_s, self.down, self.down_s, sums)

    def check(self, Y=None, what=None):
        Y = i8.fp8_moe(*self.gpu()) if Y is None else Y
        assert Y.dtype == self.dtype
        near(Y, *self.oracle(), self.dtype, what)
        return Y


SIZES = [(1, 16, 16, 1, 1), (1, 128, 128, 4, 2), (1, 1040, 272, 8, 2), (2, 144, 400, 300, 3), (3, 272, 16, 5, 5),
         (5, 528, 144, 16, 4), (16, 256, 656, 8, 2), (17, 400, 80, 7, 6), (33, 144, 272, 2, 2), (40, 272, 144, 64, 8),
         (64, 128, 128, 1, 1), (65, 144, 32, 2, 1), (130, 400, 144, 3, 2), (200, 144, 144, 40, 6), (600, 272, 48, 9, 4),
         (12, 2064, 1168, 6, 2), (70, 1168, 1040, 5, 2),
         # shared tiles of 1 to 4 blocks of tokens and several passes, first product, second, both
         (100, 144, 1168, 16, 2), (250, 272, 1168, 16, 3), (400, 144, 1168, 16, 3), (60, 2064, 80, 60, 2),
         (300, 1040, 272, 110, 8), (700, 2064, 144, 60, 6), (340, 1040, 272, 120, 16),
         # the columns split, 64 tokens at a time
         (90, 144, 1168, 1, 1), (150, 400, 1040, 2, 2), (33, 1040, 144, 3, 2)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,I,E,k", SIZES)
def test_moe(M, K, I, E, k, dtype):
    """One token to many, fewer pairs than experts and more, fewer columns than a
    block, widths whose up rows begin inside a scale block; experts repeat within
    a token."""
    Case(M, K, I, E, k, dtype).check(what=(M, K, I, E, k))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,E,k", [(1, 9, 4), (20, 6, 3), (90, 70, 2), (7, 50, 6)])
def test_moe_empty_places(M, E, k, dtype):
    """Experts out of range contribute nothing; tokens may be left with none."""
    c = Case(M, 272, 144, E, k, dtype, seed=5)
    bad = np.array([-1, E, E + 7, -(2 ** 31), 2 ** 31 - 1, 1024, -2], np.int64).astype(np.int32)
    flat = c.experts.reshape(-1)
    flat[::2] = bad[np.arange(len(flat[::2])) % len(bad)]
    c.experts[M // 2] = -1
    Y = c.check()
    assert not Y[M // 2].any()
    c.experts[:] = -1
    assert not c.check().any()


@pytest.mark.parametrize("M", [15, 16, 31, 32, 33, 48, 64, 65, 100, 129])
@pytest.mark.parametrize("E,k", [(3, 2), (300, 2)])
def test_moe_one_expert_for_all(M, E, k):
    """All tokens at one expert, twice each, whether slots are pairs or experts."""
    c = Case(M, 144, 144, E, k, torch.bfloat16, seed=9)
    c.experts[:] = 2
    c.check()


@pytest.mark.parametrize("K,I", [(1040, 528), (272, 2064)])
def test_moe_precision(K, I):
    """fp16 results stay at their own rounding, at most 2^-11 of each value: what
    the products add, 2^-17 between them and their fp32 sums, is at most an
    eighth of it."""
    c = Case(24, K, I, 4, 2, torch.float16, seed=3)
    want, _ = c.oracle()
    Y = f64(i8.fp8_moe(*c.gpu()))
    assert np.linalg.norm(Y - want) <= (2.0 ** -11 + 2.0 ** -14) * np.linalg.norm(want)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_moe_bad_values_stay(dtype):
    """NaN and infinities of a token, an expert's weights or a pair's weight reach
    no other token; unused experts and padding may hold anything."""
    c = Case(20, 272, 144, 6, 2, dtype, seed=11)
    c.experts[c.experts == 5] = 4  # expert 5 is not used
    args = c.gpu()
    want = c.check(i8.fp8_moe(*args))
    x, e, w, up, us, down, ds = args
    x = x.clone()
    x[3, 100] = float("nan")
    x[7, 271] = float("inf")
    w = w.clone()
    w[11, 1] = float("nan")
    up, down = up.clone(), down.clone()
    up.view(torch.uint8)[5] = 0x7f
    down.view(torch.uint8)[5] = 0x7f
    ds = ds.clone()
    ds[5] = float("inf")
    Y = i8.fp8_moe(x, e, w, up, us, down, ds)
    bad = [3, 7, 11]
    keep = [m for m in range(20) if m not in bad]
    assert torch.equal(Y[keep], want[keep])
    assert torch.isnan(Y[3]).all() and torch.isnan(Y[11]).all() and not torch.isfinite(Y[7]).any()


# sizes that take each kernel: pairs alone, columns split, shared tiles
KERNELS = [(1, 272, 144, 6, 2), (12, 272, 144, 6, 2), (400, 144, 1168, 16, 3), (340, 1040, 272, 120, 16),
           (150, 400, 1040, 2, 2)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,I,E,k", KERNELS)
def test_moe_bad_weights(M, K, I, E, k, dtype):
    """A NaN among an expert's numbers reaches the tokens of that expert and no
    others: all features from the first matrix, one from the second."""
    c = Case(M, K, I, E, k, dtype, seed=17)
    e = int(c.experts[0, 0])
    hit = torch.from_numpy((c.experts == e).any(1)).cuda()
    want = i8.fp8_moe(*c.gpu())
    up = c.up.copy()
    c.up[e, 2 * I - 1, K - 1] = 0x7f
    Y = i8.fp8_moe(*c.gpu())
    assert torch.isnan(Y[hit]).all() and torch.equal(Y[~hit], want[~hit])
    c.up = up
    c.down[e, K - 1, 0] = 0xff
    Y = i8.fp8_moe(*c.gpu())
    assert torch.isnan(Y[hit, K - 1]).all()
    assert torch.equal(Y[:, :K - 1], want[:, :K - 1]) and torch.equal(Y[~hit], want[~hit])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,I,E,k", KERNELS)
def test_moe_subnormal_activations(M, K, I, E, k, dtype):
    """Activations below the type's normal numbers count as what they are."""
    c = Case(M, K, I, E, k, dtype, seed=19)
    fi = torch.finfo(dtype)
    least, bits = fi.smallest_normal * fi.eps, 10 if dtype == torch.float16 else 7
    n = np.random.default_rng(1).integers(-2 ** bits + 1, 2 ** bits, (M, K))
    c.x = torch.from_numpy(n * least).to(dtype).cuda()
    assert np.array_equal(f64(c.x), n * least)
    c.up_s *= np.float32(2.0 ** -bits / least)
    Y = c.check()
    assert float(Y.float().abs().mean()) > 1e-3


def test_moe_large_products():
    """Gated products past fp16's range, whose weighted sum is within it."""
    c = Case(4, 272, 144, 3, 2, torch.float16, seed=13)
    c.up_s *= 256.0
    c.down_s *= 2.0 ** -16
    c.check()


def test_moe_repeatable_and_out():
    c = Case(64, 528, 272, 16, 4, torch.bfloat16, seed=15)
    args = c.gpu()
    Y = i8.fp8_moe(*args)
    out = torch.full_like(Y, float("nan"))
    for _ in range(5):
        assert i8.fp8_moe(*args, out=out) is out and torch.equal(out, Y)
    # a token's result does not depend on the others'
    one = i8.fp8_moe(c.x[5:6].clone(), args[1][5:6].clone(), args[2][5:6].clone(), *args[3:])
    near(one, f64(Y[5:6]), 2 * c.oracle()[1][5:6], torch.bfloat16, "alone")


def test_moe_empty_sizes():
    z = lambda *s, d=torch.float16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    e8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda").view(E4M3)  # noqa: E731
    i32 = lambda *s: z(*s, d=torch.int32)  # noqa: E731
    f = lambda *s: z(*s, d=torch.float32)  # noqa: E731
    Y = i8.fp8_moe(z(0, 32), i32(0, 2), f(0, 2), e8(3, 32, 128), f(3, 1, 1), e8(3, 32, 128), f(3, 1, 1))
    assert Y.shape == (0, 32)
    Y = i8.fp8_moe(torch.ones_like(z(4, 32)), i32(4, 2), f(4, 2) + 1, e8(3, 0, 128), f(3, 0, 1), e8(3, 32, 0), f(3, 1, 0))
    assert Y.shape == (4, 32) and not Y.any()
    assert i8.fp8_moe(z(4, 0), i32(4, 2), f(4, 2), e8(3, 32, 0), f(3, 1, 0), e8(3, 0, 128), f(3, 0, 1)).shape == (4, 0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_and_pack_experts(dtype):
    W = torch.stack([rows(144, 80, dtype, s, std=0.02, outliers=2) for s in range(3)])
    q, s = i8.fp8_quantize_experts(W)
    for e in range(3):
        qe, se = i8.fp8_quantize_weight(W[e])
        assert torch.equal(q[e].view(torch.uint8), qe.view(torch.uint8)) and torch.equal(s[e], se)
    bytes_ = torch.randint(0, 120, (3, 48, 272), dtype=torch.uint8, device="cuda")
    p = i8.fp8_pack_experts(bytes_.view(E4M3))
    for e in range(3):
        assert np.array_equal(raw(p[e]), F.pack_weight(raw(bytes_[e])))
