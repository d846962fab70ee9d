"""The measured cases of a mixture-of-experts block for serving: the norms
after one block and before the next with the block's gate and the residual's
scale between them, the router, and the experts' gated feed-forward from
block-scaled e4m3 weights for a few tokens.

Hidden sizes are those of the library's own workloads (4096, 5120, 12288) and
odd ones beside them; experts' sizes are generic.  A case's `M` is the number
of tokens, `K` the hidden size, `E` the experts, `top_k` those of a token, `I`
the width of one expert's feed-forward.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
FLOOR = 2.0 ** -100  # least block maximum that a scale is made from
EPS = 1e-5

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token between an attention and its feed-forward, gated by the token's own condition
        dict(name="norm 1x5120", op="norm", M=1, K=5120, dtype="bf16", gates=1, alpha=1.0, quantize=True),
        # a ragged batch of prompts, a width that ends inside a block, no gate, the residual scaled as in deep stacks;
        # what follows is a router and experts, which take 16 bits
        dict(name="norm 333x4112", op="norm", M=333, K=4112, dtype="fp16", gates=0, alpha=2.5, quantize=False),
        # 175B-scale prefill of 4 sequences, one row of gates for each
        dict(name="norm 4096x12288", op="norm", M=4096, K=12288, dtype="bf16", gates=4, alpha=1.0, quantize=True),
        # the router of one new token
        dict(name="route 1x4096 128", op="route", M=1, K=4096, E=128, top_k=8, normalize=True, dtype="bf16"),
        # a short chunk of prompt, every size odd
        dict(name="route 77x5136 61", op="route", M=77, K=5136, E=61, top_k=6, normalize=False, dtype="fp16"),
        # a prefill's router
        dict(name="route 4096x5120 128", op="route", M=4096, K=5120, E=128, top_k=8, normalize=True, dtype="bf16"),
        # the smallest experts' call, latency: one token, two of eight narrow experts
        dict(name="moe 1x1040 8", op="moe", M=1, K=1040, I=272, E=8, top_k=2, padded=0, dtype="fp16"),
        # one new token, eight of many experts
        dict(name="moe 1x4096 128", op="moe", M=1, K=4096, I=1408, E=128, top_k=8, padded=0, dtype="bf16"),
        # two of eight wide experts, a batch of 16 of which 3 places are empty
        dict(name="moe 16x5120 8", op="moe", M=16, K=5120, I=8192, E=8, top_k=2, padded=3, dtype="bf16"),
        # 37 sequences decoded together, every size odd
        dict(name="moe 37x5136 61", op="moe", M=37, K=5136, I=1360, E=61, top_k=6, padded=0, dtype="fp16"),
        # 64 sequences decoded together: nearly every expert has a few tokens
        dict(name="moe 64x4096 128", op="moe", M=64, K=4096, I=1408, E=128, top_k=8, padded=0, dtype="bf16"),
        # a large batch, or a chunk of prompt: about 32 tokens an expert
        dict(name="moe 512x4096 128", op="moe", M=512, K=4096, I=1408, E=128, top_k=8, padded=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "moe", "moe"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "moe":
        M = rng.randint(1, 32) if rng.random() < 0.5 else _log(rng, 33, 512)
        K, I = 16 * _log(rng, 16, 480), 16 * _log(rng, 8, 176)
        E = min(_log(rng, 4, 128), 128 * 4096 * 1408 // (K * I))
        E = max(E, 4)
        top_k = rng.randint(1, min(8, E))
        M = min(M, 512 * 8 * 4096 * 1408 // (top_k * K * I))
        return dict(op=op, M=M, K=K, I=I, E=E, top_k=top_k, padded=rng.choice([0, 0, M // 8]), dtype=dtype)
    # the few-token sizes of serving as often as the long ones
    M = rng.randint(1, 64) if rng.random() < 0.4 else _log(rng, 65, 4096)
    if op == "norm":
        K = 16 * _log(rng, 16, 768)
        gates = rng.choice([0, 1, M])  # none, one row for all tokens, one for each
        return dict(op=op, M=M, K=K, dtype=dtype, gates=gates, alpha=rng.choice([1.0, 0.5, 2.5]), quantize=rng.random() < 0.6)
    E = rng.randint(4, 128)
    return dict(op=op, M=M, K=16 * _log(rng, 16, 320), E=E, top_k=rng.randint(1, min(8, E)), normalize=rng.random() < 0.5, dtype=dtype)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, M, K, dtype):
    """Ordinary columns N(0, 0.5^2) clipped at 5, seven columns of 20 to 130 in three rows of four."""
    x = _randn(g, M, K).mul_(0.5).clamp_(-5.0, 5.0)
    dims = torch.randperm(K, generator=g, device="cuda")[:7]
    mag = torch.rand((M, dims.numel()), generator=g, device="cuda") * 110.0 + 20.0
    sign = torch.where(torch.rand(mag.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    rows = torch.rand((M, 1), generator=g, device="cuda") < 0.75
    x[:, dims] = torch.where(rows, mag * sign, x[:, dims])
    return x.to(dtype)


def _normed(g, M, K, dtype):
    """Rows as a norm leaves them: N(0, 1), seven columns ten times that."""
    x = _randn(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[:7]] *= 10.0
    return x.to(dtype)


def _spread(s, N, K):
    """Scales [E, ceil(N/128), ceil(K/128)] -> one per element, [E, N, K]."""
    return s.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]


def _experts(g, E, N, K):
    """Weights of E experts as a checkpoint holds them, about N(0, 1/K): e4m3 [E, N, K], a scale per 128 x 128 block."""
    q = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        q[e] = _randn(g, N, K).mul_(110.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    spread = torch.rand((E, -(-N // BLOCK), -(-K // BLOCK)), generator=g, device="cuda") * 0.4 + 0.8
    return q, spread * (1.0 / (110.0 * math.sqrt(K)))


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, K, dtype = case["M"], case["K"], _TYPES[case["dtype"]]
    s = dict(case, dtype=dtype)
    if case["op"] == "norm":
        s["x"], s["residual"] = _activations(g, M, K, dtype), _activations(g, M, K, dtype)
        s["post"] = (1.0 + 0.2 * _randn(g, K)).to(dtype)
        s["pre"] = (1.0 + 0.2 * _randn(g, K)).to(dtype)
        s["gate"] = (0.5 + 0.5 * _randn(g, case["gates"], K)).to(dtype) if case["gates"] else None
        return s
    E, k = case["E"], case["top_k"]
    s["x"] = _normed(g, M, K, dtype)
    if case["op"] == "route":
        s["w"] = _randn(g, E, K).mul_(1.5 / math.sqrt(K)).to(dtype)
        return s
    # experts as a router chooses them, some more popular than others
    p = torch.softmax(1.5 * _randn(g, M, E) + 0.5 * _randn(g, E), 1)
    w, e = torch.sort(p, dim=1, descending=True)
    s["weights"] = (w[:, :k] / w[:, :k].sum(1, keepdim=True)).contiguous()
    s["experts"] = e[:, :k].to(torch.int32).contiguous()
    if case["padded"]:
        s["experts"][M - case["padded"]:] = -1  # empty places of the batch
    s["up_q"], s["up_s"] = _experts(g, E, 2 * case["I"], K)
    s["down_q"], s["down_s"] = _experts(g, E, K, case["I"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] == "moe":
        import int8_mixed_precision_outlier_amd as i8
        s["up_q"], s["down_q"] = i8.fp8_pack_experts(s["up_q"]), i8.fp8_pack_experts(s["down_q"])  # laid out once, at load
    return s


def _run_own(s):
    import int8_mixed_precision_outlier_amd as i8
    if s["op"] == "norm":
        return i8.fp8_sandwich_norm(s["x"], s["residual"], s["post"], s["pre"], gate=s["gate"],
                                    residual_scale=s["alpha"], eps=EPS, quantize=s["quantize"])
    if s["op"] == "route":
        return i8.moe_route(s["x"], s["w"], s["top_k"], normalize=s["normalize"])
    return i8.fp8_moe(s["x"], s["experts"], s["weights"], s["up_q"], s["up_s"], s["down_q"], s["down_s"])


def _norm(x, weight):
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * weight.float()


def _blocks_of_rows(y):
    """Plain quantizer of fp32 rows: (e4m3 [M, K], fp32 scales [ceil(K/128), M]).
    The e4m3 tensor holds numbers of its own type; each times its block's scale is the row's value."""
    M, K = y.shape
    kb = -(-K // BLOCK)
    padded = torch.nn.functional.pad(y, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    amax = padded.abs().amax(2).clamp(min=FLOOR)
    q = (padded * (E4M3_MAX / amax)[:, :, None]).view(M, kb * BLOCK)[:, :K]
    return q.to(torch.float8_e4m3fn), (amax / E4M3_MAX).t().contiguous()


def _run_norm(s):
    z = _norm(s["x"].float(), s["post"])
    if s["gate"] is not None:
        z = z.view(s["gates"], -1, s["K"]).mul_(s["gate"].float()[:, None]).view(z.shape)
    h = s["alpha"] * s["residual"].float() + z
    y = _norm(h, s["pre"])
    return (*(_blocks_of_rows(y) if s["quantize"] else (y.to(s["dtype"]),)), h.to(s["dtype"]))


def _run_route(s):
    # in 64 bits: experts' places next to each other decide
    p = torch.softmax(s["x"].double() @ s["w"].double().t(), 1)
    w, e = torch.sort(p, dim=1, descending=True, stable=True)
    w, e = w[:, :s["top_k"]], e[:, :s["top_k"]]
    if s["normalize"]:
        w = w / w.sum(1, keepdim=True)
    return e.to(torch.int32), w.float()


def _run_moe(s):
    M, K, I, E, k = s["M"], s["K"], s["I"], s["E"], s["top_k"]
    live = s["experts"] >= 0
    at = s["experts"].clamp(min=0).long()
    weights = torch.where(live, s["weights"], 0.0)
    if M * k < E:  # the weights of each token's experts, one by one
        at = at.view(-1)
        pick = lambda q, sc: q.view(torch.uint8)[at].view(q.dtype).float().mul_(_spread(sc[at], *q.shape[1:]))  # noqa: E731
        x = s["x"].float().repeat_interleave(k, 0)[:, :, None]
        gate, up = torch.matmul(pick(s["up_q"], s["up_s"]), x).split(I, 1)
        a = gate / (1.0 + torch.exp(-gate)) * up
        y = torch.matmul(pick(s["down_q"], s["down_s"]), a).view(M, k, K)
        return (y * weights[:, :, None]).sum(1).to(s["dtype"])
    # every expert for every token
    whole = lambda q, sc: q.float().mul_(_spread(sc, *q.shape[1:]))  # noqa: E731
    share = torch.zeros((M, E), device="cuda").scatter_add_(1, at, weights)
    gate, up = torch.matmul(whole(s["up_q"], s["up_s"]), s["x"].float().t().contiguous()).split(I, 1)
    a = gate / (1.0 + torch.exp(-gate)) * up * share.t()[:, None, :]
    return torch.matmul(whole(s["down_q"], s["down_s"]), a).sum(0).t().contiguous().to(s["dtype"])


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _run_norm, "route": _run_route, "moe": _run_moe}[s["op"]](s)


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        out = M * K + 4 * M * -(-K // BLOCK) if case["quantize"] else 2 * M * K
        return dict(bytes=6 * M * K + out + 2 * K * (2 + case["gates"]), flops=15 * M * K)
    E, k = case["E"], case["top_k"]
    if case["op"] == "route":
        return dict(bytes=2 * (M + E) * K + 8 * M * k, flops=2 * M * E * K)
    I, live = case["I"], M - case["padded"]
    # the experts that some token has: each expert is missed by a token with about 1 - k/E
    used = min(E, live * k, max(k, E * (1.0 - (1.0 - k / E) ** live)))
    one = 3 * I * K + 4 * (-(-2 * I // BLOCK) * -(-K // BLOCK) + -(-K // BLOCK) * -(-I // BLOCK))
    return dict(bytes=used * one + 4 * M * K + 8 * M * k, flops=6 * live * k * I * K)


def exact(case, seed):
    s = _inputs(case, seed)
    M, K = s["M"], s["K"]
    x = s["x"].double()
    if s["op"] == "norm":
        branch = x / torch.sqrt(x.square().sum(1, keepdim=True) / K + EPS) * s["post"].double()
        if s["gate"] is not None:
            branch = branch * s["gate"].double().repeat_interleave(M // s["gates"], 0)
        h = s["residual"].double() * s["alpha"] + branch
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / K + EPS) * s["pre"].double()
        if not s["quantize"]:
            return y, h
        qs, scales = [], []
        for c in range(0, K, BLOCK):
            part = y[:, c:c + BLOCK]
            scale = part.abs().max(1).values.clamp(min=FLOOR) / E4M3_MAX
            qs.append(part / scale[:, None])
            scales.append(scale)
        return torch.cat(qs, 1), torch.stack(scales), h
    if s["op"] == "route":
        logits = torch.stack([(x * w).sum(1) for w in s["w"].double()], 1)
        e = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :s["top_k"]]
        chosen = torch.exp(torch.gather(logits, 1, e) - logits.max(1, keepdim=True).values)
        among = chosen if s["normalize"] else torch.exp(logits - logits.max(1, keepdim=True).values)
        return e.to(torch.int32), chosen / among.sum(1, keepdim=True)
    y = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        m, j = torch.nonzero(s["experts"] == e, as_tuple=True)
        if not m.numel():
            continue
        up = s["up_q"][e].double() * _spread(s["up_s"][e:e + 1], 2 * s["I"], K)[0].double()
        down = s["down_q"][e].double() * _spread(s["down_s"][e:e + 1], K, s["I"])[0].double()
        gate_up = x[m] @ up.t()
        gate = gate_up[:, :s["I"]]
        out = (gate * torch.sigmoid(gate) * gate_up[:, s["I"]:]) @ down.t()
        y.index_add_(0, m, out * s["weights"][m, j].double()[:, None])
    return y
