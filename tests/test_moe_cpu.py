"""Mixture-of-experts operators and the sandwich norm without a GPU: the oracle
against element-by-element loops, and the C functions' refusals."""
import ctypes
import math
import os

import numpy as np
import pytest

import int8_mixed_precision_outlier_amd as i8
from oracle import fp8_block as F
from oracle import moe as O

EINVAL, EALIGN, EWS, OK = i8.STATUS_EINVAL, i8.STATUS_EALIGN, i8.STATUS_EWORKSPACE, i8.STATUS_OK
FAKE = 1 << 20  # aligned non-null; never dereferenced (checks fail first)
built = pytest.mark.skipif(not os.path.exists(i8.LIB_PATH),
                           reason="libint8mm.so not built (run __graft_entry__.build())")


# ---- oracle ------------------------------------------------------------------

def test_oracle_sandwich():
    rng = np.random.default_rng(1)
    M, K = 4, 6
    x, r = rng.standard_normal((2, M, K))
    post, pre = rng.standard_normal((2, K))
    gate = rng.standard_normal((2, K))
    h, y, z = O.sandwich64(x, r, post, pre, gate, 0.5, 1e-3)
    for m in range(M):
        rms = math.sqrt(sum(v * v for v in x[m]) / K + 1e-3)
        hm = [0.5 * r[m, k] + gate[m // 2, k] * (x[m, k] / rms * post[k]) for k in range(K)]
        rms2 = math.sqrt(sum(v * v for v in hm) / K + 1e-3)
        assert np.allclose(h[m], hm, rtol=1e-13) and np.allclose(y[m], [hm[k] / rms2 * pre[k] for k in range(K)], rtol=1e-13)


def test_oracle_route():
    x = np.array([[1.0, 2.0], [0.0, 0.0], [np.nan, 1.0]])
    w = np.array([[1.0, 0.0], [0.0, 1.0], [0.0, 1.0], [1.0, 1.0]])
    e, p = O.route64(x, w, 3, False)
    assert e.tolist() == [[3, 1, 2], [0, 1, 2], [0, 1, 2]]
    z = sum(math.exp(v) for v in (1, 2, 2, 3))
    assert np.allclose(p[0], [math.exp(3) / z, math.exp(2) / z, math.exp(2) / z]) and np.allclose(p[1], 0.25)
    assert np.isnan(p[2]).all()
    assert np.allclose(O.route64(x, w, 3, True)[1][:2].sum(1), 1.0)


def test_oracle_moe():
    rng = np.random.default_rng(2)
    M, K, I, E, k = 3, 5, 4, 3, 2
    x = rng.standard_normal((M, K))
    up, down = rng.integers(0, 100, (E, 2 * I, K)).astype(np.uint8), rng.integers(0, 100, (E, K, I)).astype(np.uint8)
    us, ds = rng.uniform(0.1, 0.2, (E, 1, 1)), rng.uniform(0.1, 0.2, (E, 1, 1))
    experts = np.array([[0, 2], [1, 1], [-1, 7]])
    weights = rng.uniform(0, 1, (M, k))
    y, tol = O.moe64(x, experts, weights, up, us, down, ds, (1e-6, 1e-6))
    for m in range(M):
        want = np.zeros(K)
        for j in range(k):
            e = experts[m, j]
            if not 0 <= e < E:
                continue
            gu = [sum(x[m, c] * F.e4m3_decode(up[e, n, c]) * us[e, 0, 0] for c in range(K)) for n in range(2 * I)]
            a = [gu[i] / (1 + math.exp(-gu[i])) * gu[I + i] for i in range(I)]
            for n in range(K):
                want[n] += weights[m, j] * sum(a[i] * F.e4m3_decode(down[e, n, i]) * ds[e, 0, 0] for i in range(I))
        assert np.allclose(y[m], want, rtol=1e-12)
    assert np.all(tol[:2] > 0) and not tol[2].any()


# ---- refusals ----------------------------------------------------------------

def sandwich(**over):
    a = dict(X=FAKE, residual=FAKE, post=FAKE, pre=FAKE, gate=None, gates=0, alpha=1.0, type=0, M=4, K=32, eps=1e-6,
             H=FAKE, Y=None, q=FAKE, s=FAKE)
    a.update(over)
    p = lambda n: a[n] if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    return i8.load().fp8_sandwich_norm(p("X"), p("residual"), p("post"), p("pre"), p("gate"), a["gates"], a["alpha"],
                                       a["type"], a["M"], a["K"], a["eps"], p("H"), p("Y"), p("q"), p("s"), None)


SANDWICH = [(dict(type=2), EINVAL), (dict(type=-1), EINVAL), (dict(M=-1), EINVAL), (dict(K=-16), EINVAL),
            (dict(K=65552), EINVAL), (dict(K=40), EALIGN), (dict(M=1 << 27, K=32), EINVAL), (dict(eps=0.0), EINVAL),
            (dict(eps=math.inf), EINVAL), (dict(eps=math.nan), EINVAL), (dict(alpha=math.nan), EINVAL),
            (dict(alpha=math.inf), EINVAL), (dict(gate=FAKE), EINVAL), (dict(gates=2), EINVAL),
            (dict(gate=FAKE, gates=3), EINVAL), (dict(gate=FAKE, gates=8), EINVAL), (dict(gate=FAKE, gates=-2), EINVAL),
            (dict(X=None), EINVAL), (dict(residual=None), EINVAL), (dict(post=None), EINVAL), (dict(pre=None), EINVAL),
            (dict(H=None), EINVAL), (dict(q=None), EINVAL), (dict(s=None), EINVAL), (dict(q=None, s=None), EINVAL),
            (dict(Y=FAKE), EINVAL), (dict(Y=FAKE, q=None), EINVAL)]
SANDWICH += [(dict([(n, FAKE + 8)]), EALIGN) for n in ("X", "residual", "post", "pre", "H", "q", "s")]
SANDWICH += [(dict(gate=FAKE + 8, gates=2), EALIGN), (dict(Y=FAKE + 8, q=None, s=None), EALIGN),
             (dict(M=0, X=None), OK), (dict(K=0, X=None), OK)]


@built
@pytest.mark.parametrize("over,status", SANDWICH, ids=str)
def test_sandwich_norm_refuses(over, status):
    assert sandwich(**over) == status


def route(**over):
    a = dict(X=FAKE, W=FAKE, type=0, M=4, K=32, E=8, k=2, e=FAKE, w=FAKE, ws=FAKE, size=None)
    a.update(over)
    p = lambda n: a[n] if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    size = i8.load().moe_route_workspace_size(a["M"], a["K"], a["E"], a["k"]) if a["size"] is None else a["size"]
    return i8.load().moe_route(p("X"), p("W"), a["type"], a["M"], a["K"], a["E"], a["k"], 1, p("e"), p("w"), p("ws"), size, None)


ROUTE = [(dict(type=3), EINVAL), (dict(M=-1), EINVAL), (dict(M=(1 << 18) + 1), EINVAL), (dict(M=1 << 40, K=0), EINVAL),
         (dict(K=8), EALIGN), (dict(K=65552), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL), (dict(E=-3), EINVAL),
         (dict(k=0), EINVAL), (dict(k=9), EINVAL), (dict(k=-1), EINVAL), (dict(E=64, k=33), EINVAL),
         (dict(M=1 << 17, K=65536), EINVAL), (dict(X=None), EINVAL), (dict(W=None), EINVAL), (dict(e=None), EINVAL),
         (dict(w=None), EINVAL), (dict(ws=None), EINVAL), (dict(X=FAKE + 8), EALIGN), (dict(W=FAKE + 8), EALIGN),
         (dict(e=FAKE + 2), EALIGN), (dict(w=FAKE + 1), EALIGN), (dict(ws=FAKE + 128), EALIGN), (dict(size=0), EWS),
         (dict(size=-1 + 4 * 8 * 4), EWS), (dict(M=0, X=None, e=None), OK)]


@built
@pytest.mark.parametrize("over,status", ROUTE, ids=str)
def test_route_refuses(over, status):
    assert route(**over) == status


def moe(**over):
    a = dict(X=FAKE, type=1, M=4, K=32, e=FAKE, w=FAKE, k=2, up=FAKE, us=FAKE, down=FAKE, ds=FAKE, I=48, E=8, Y=FAKE,
             ws=FAKE, size=None)
    a.update(over)
    p = lambda n: a[n] if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    size = i8.load().fp8_moe_workspace_size(a["M"], a["K"], a["I"], a["E"], a["k"]) if a["size"] is None else a["size"]
    return i8.load().fp8_moe(p("X"), a["type"], a["M"], a["K"], p("e"), p("w"), a["k"], p("up"), p("us"), p("down"),
                             p("ds"), a["I"], a["E"], p("Y"), p("ws"), size, None)


MOE = [(dict(type=2), EINVAL), (dict(M=-1), EINVAL), (dict(M=4097), EINVAL), (dict(M=8193, k=1), EINVAL),
       (dict(M=1 << 62), EINVAL), (dict(K=24), EALIGN), (dict(I=24), EALIGN), (dict(I=-16), EINVAL), (dict(I=65552), EINVAL),
       (dict(K=65552), EINVAL), (dict(K=65536, I=32768), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL),
       (dict(k=0), EINVAL), (dict(k=33), EINVAL), (dict(size=0), EWS), (dict(size=256), EWS), (dict(ws=FAKE + 64), EALIGN),
       (dict(e=FAKE + 2), EALIGN), (dict(w=FAKE + 2), EALIGN), (dict(M=0, X=None), OK), (dict(K=0, X=None), OK)]
MOE += [(dict([(n, None)]), EINVAL) for n in ("X", "e", "w", "up", "us", "down", "ds", "Y", "ws")]
MOE += [(dict([(n, FAKE + 8)]), EALIGN) for n in ("X", "up", "us", "down", "ds", "Y")]


@built
@pytest.mark.parametrize("over,status", MOE, ids=str)
def test_moe_refuses(over, status):
    assert moe(**over) == status


@built
def test_workspace_sizes():
    lib = i8.load()
    assert lib.moe_route_workspace_size(4, 32, 8, 9) == 0 and lib.moe_route_workspace_size(0, 32, 8, 2) == 0
    assert lib.moe_route_workspace_size(100, 32, 8, 2) >= 100 * 8 * 8
    assert lib.fp8_moe_workspace_size(4, 32, 24, 8, 2) == 0
    for M, K, I, E, k in ((1, 16, 16, 1, 1), (4096, 65536, 128, 1024, 2), (256, 128, 65536, 2, 32)):
        assert lib.fp8_moe_workspace_size(M, K, I, E, k) >= M * k * I * 4
    assert i8.MOE_MAX_PAIRS == 8192


def test_operators_need_gpu_tensors():
    import torch
    x = torch.zeros((2, 32), dtype=torch.float16)
    with pytest.raises(TypeError):
        i8.fp8_sandwich_norm(x, x, x[0], x[0])
    with pytest.raises(TypeError):
        i8.moe_route(x, x, 1)
    with pytest.raises(TypeError):
        i8.fp8_moe(x, x, x, x, x, x, x)
    with pytest.raises(TypeError):
        i8.fp8_pack_experts(x)
    with pytest.raises(TypeError):
        i8.fp8_quantize_experts(x[None])
