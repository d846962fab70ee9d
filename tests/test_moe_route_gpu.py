"""The router where its sums are at their limits: no columns for the most tokens
and experts, and the matrix instructions' sums against 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import int8_mixed_precision_outlier_amd as i8

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.mark.parametrize("M,E,k", [(1 << 18, 1024, 32), (1 << 18, 256, 1), ((1 << 18) - 1, 65, 3), (16384, 1024, 2),
                                   (16383, 1024, 2)])
def test_no_columns_for_many_tokens(M, E, k):
    """More sums than one launch has wavefronts, all of them 0: the first experts,
    with equal weights."""
    z = lambda n: torch.empty((n, 0), dtype=torch.float16, device="cuda")  # noqa: E731
    e, p = i8.moe_route(z(M), z(E), k, normalize=False)
    assert bool((e == torch.arange(k, dtype=torch.int32, device="cuda")).all())
    assert bool(((p * E - 1).abs() <= 64 * 2.0 ** -24).all())
    del e, p
    torch.cuda.empty_cache()


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("M,E,k", [(64, 1, 1), (40000, 1, 1), (40000, 2, 2), (40000, 2, 1)])
def test_products_past_fp32_of_few_experts(M, E, k, normalize):
    """Logits of 2^252 and more are finite in 64 bits: the weights of equal ones are
    equal, that of a single expert is 1."""
    x = torch.full((M, 1024), 1e38, dtype=torch.bfloat16, device="cuda")
    w = torch.full((E, 1024), 1e38, dtype=torch.bfloat16, device="cuda")
    for sign in (1, -1):
        e, p = i8.moe_route(x, w * sign, k, normalize=normalize)
        assert bool((e == torch.arange(k, dtype=torch.int32, device="cuda")).all())
        assert bool((p == 1 / (k if normalize else E)).all())
    x[3, 5] = float("inf")
    e, p = i8.moe_route(x, w, k, normalize=normalize)
    assert bool(p[3].isnan().all()) and bool((p[4:] == 1 / (k if normalize else E)).all())


def tile_sums(x, w):
    """The matrix instructions' logits [M, E] and their bounds, as moe_route leaves
    them in its workspace: 64-bit sums, then (256-byte aligned) the bounds in fp32."""
    (M, K), E = x.shape, w.shape[0]
    assert M * E * K > 2 ** 25
    lib = i8.load()
    size = lib.moe_route_workspace_size(M, K, E, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    e, p = torch.empty(M, dtype=torch.int32, device="cuda"), torch.empty(M, device="cuda")
    at = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert lib.moe_route(at(x), at(w), int(x.dtype == torch.bfloat16), M, K, E, 1, 0, at(e), at(p), at(ws), size, None) == 0
    torch.cuda.synchronize()
    n = M * E * 8
    first = (n + 255) // 256 * 256
    return ws[:n].view(torch.float64).view(M, E), ws[first:first + M * E * 4].view(torch.float32).view(M, E)


def patterns(K, dtype, seed):
    """Pairs of operands [M, K], [E, K] that are hard on a sum of 32 products."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, E = 4096, (1 << 13) // K + 64
    R = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    U = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    yield "normal", R(M, K), R(E, K)
    yield "wide", R(M, K) * 2.0 ** torch.floor(U(M, K) * 22 - 14), R(E, K) * 2.0 ** torch.floor(U(E, K) * 22 - 14)
    # neighbours cancel but for 2^-6 of them
    x, w = R(M, K), R(E, K)
    x[:, 1::2], w[:, 1::2] = x[:, ::2], -w[:, ::2] * (1 + 2.0 ** -6)
    yield "cancelling", x, w
    # one large product in 32, in every place, and the others where alignment to it
    # drops some of their bits or all of them
    where = torch.arange(K, device="cuda") % 32 == torch.arange(M, device="cuda")[:, None] % 32
    for up in range(0, 15, 2):
        for sign in (1.0, -1.0):
            x = torch.where(where, 2.0 ** 14, 1.0)
            w = sign * (1 + U(E, K).mul_(8).floor_().div_(8))
            put = torch.arange(K, device="cuda") % 32 == torch.arange(E, device="cuda")[:, None] % 32
            yield "one large, 2^%d, %g" % (14 + up, sign), x, torch.where(put, 2.0 ** up, w)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("K", [32, 96, 1040])
def test_matrix_instructions_sums_stay_within_their_bound(K, dtype):
    """Each sum of 32 exact products is off by less than 32 * 2^-23 of the sum of
    their magnitudes, as the order's exactness needs, and by less than the bound
    that comes with it (measured: at most 4 * 2^-23)."""
    for name, x, w in patterns(K, dtype, K):
        x, w = x.to(dtype), w.to(dtype)
        assert torch.isfinite(x).all() and torch.isfinite(w).all(), name
        L, bound = tile_sums(x, w)
        x, w = x.double(), w.double()
        off, size = (L - x @ w.t()).abs(), x.abs() @ w.abs().t()
        # the 64-bit sums, here and there: at most K additions of 2^-53 each
        assert bool((off <= (32 * 2.0 ** -23 + 2 * K * 2.0 ** -53) * size).all()), (name, float((off / size).max()) * 2 ** 23)
        assert bool((off <= bound.double()).all()), name


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("seed", [1, 2])
def test_order_of_logits_that_cancel(seed, dtype):
    """Each expert's row is its own: 2048 columns whose products cancel, in other
    instructions than their counterparts, and one column that makes the logit.
    The logits' gaps go from far below what the fp32 sums lose to above the bound;
    the order is that of the one column all the same."""
    M, H, E, k = 600, 1024, 64, 32
    rng = np.random.default_rng(seed)
    half = rng.standard_normal((M, H))
    rows = rng.standard_normal((E, H))
    place = rng.permutation(H)
    x = np.zeros((M, 2 * H + 16))
    w = np.zeros((E, 2 * H + 16))
    x[:, :H], x[:, H:2 * H] = half, half[:, place]
    w[:, :H], w[:, H:2 * H] = rows, -rows[:, place]
    x[:, 2 * H] = 1
    value = 2.0 ** np.repeat(np.linspace(-24, 7, 32).round(), 2)
    value[1::2] *= -1
    w[:, 2 * H] = value[rng.permutation(E)]
    x, w = (torch.from_numpy(a.astype(np.float32)).to(dtype).cuda() for a in (x, w))
    L, bound = tile_sums(x, w)
    exact = w[:, 2 * H].double()
    want = torch.argsort(-exact, stable=True)[:k].to(torch.int32)
    assert (torch.argsort(-L, 1)[:, :k] != want).any(1).float().mean() > 0.5, "the fp32 sums' own order was to be another"
    assert float(exact.max()) > 4 * float(bound.max()), "the largest gaps were to be past the bound"
    e, p = i8.moe_route(x, w, k)
    assert bool((e == want).all())
    # M = 8 takes 64-bit sums throughout
    assert torch.equal(i8.moe_route(x[:8].contiguous(), w, k)[0], e[:8])
