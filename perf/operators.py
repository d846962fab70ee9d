"""The measured cases of the block-scaled 8-bit floating-point operators: the
product with one scale per 128-column block, and the operators that make its
left operand (the quantizer, the root-mean-square norm with the residual's
addition, the SiLU-gated product).

Sizes are those of the library's own workloads (hidden sizes 4096, 5120 and
12288, features 20480, 36864 and 49152), and odd ones beside them.  A case's
`M` is the number of tokens, `K` the columns of the 8-bit operand and `N` the
features of the product.
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
        # norm before a projection, one new token of the 175B-scale model
        dict(name="norm 1x12288", op="norm", M=1, K=12288, dtype="bf16", residual=True),
        # a ragged batch of prompts, a width that ends inside a block, first layer (no residual yet)
        dict(name="norm 333x4112", op="norm", M=333, K=4112, dtype="fp16", residual=False),
        # 175B-scale prefill
        dict(name="norm 4096x12288", op="norm", M=4096, K=12288, dtype="bf16", residual=True),
        # an attention's output before its projection: 17 tokens being decoded, and a prefill
        dict(name="quantize 17x4096", op="quantize", M=17, K=4096, dtype="fp16"),
        dict(name="quantize 4096x12288", op="quantize", M=4096, K=12288, dtype="bf16"),
        # gated FFN before its down projection: one token, and a 13B-scale prefill
        dict(name="silu 1x20480", op="silu", M=1, K=20480, dtype="bf16"),
        dict(name="silu 2048x20480", op="silu", M=2048, K=20480, dtype="fp16"),
        # one new token through the smallest layer: latency
        dict(name="matmul 1x4096x4096", op="matmul", M=1, K=4096, N=4096, dtype="fp16", bias=False),
        # 32 tokens through the fused QKV projection: the weight's stream
        dict(name="matmul 32x12288x36864", op="matmul", M=32, K=12288, N=36864, dtype="bf16", bias=True),
        # a short chunk of prompt, every size odd
        dict(name="matmul 77x5136x20464", op="matmul", M=77, K=5136, N=20464, dtype="fp16", bias=True),
        # 13B-scale FFN prefill
        dict(name="matmul 2048x5120x20480", op="matmul", M=2048, K=5120, N=20480, dtype="fp16", bias=False),
        # 175B-scale FFN prefill
        dict(name="matmul 4096x12288x49152", op="matmul", M=4096, K=12288, N=49152, dtype="bf16", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "silu", "matmul", "matmul"])
    # the few-token sizes of serving as often as the long ones
    M = rng.randint(1, 64) if rng.random() < 0.4 else _log(rng, 65, 4096)
    K = 16 * _log(rng, 16, 1280 if op == "silu" else 768)
    dtype = rng.choice(["fp16", "bf16"])
    if op == "norm":
        return dict(op=op, M=M, K=K, dtype=dtype, residual=rng.random() < 0.7)
    if op != "matmul":
        return dict(op=op, M=M, K=K, dtype=dtype)
    return dict(op=op, M=M, K=K, N=16 * _log(rng, 16, 3000), dtype=dtype, bias=rng.random() < 0.5)


def _activations(g, M, K, dtype):
    """Ordinary columns N(0, 0.5^2) clipped at 5, seven columns of 20 to 130 in three rows of four."""
    x = torch.randn((M, K), generator=g, device="cuda").mul_(0.5).clamp_(-5.0, 5.0)
    dims = torch.randperm(K, generator=g, device="cuda")[:7]
    mag = torch.rand((M, dims.numel()), generator=g, device="cuda") * 110.0 + 20.0
    sign = torch.where(torch.rand(mag.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    rows = torch.rand((M, 1), generator=g, device="cuda") < 0.75
    x[:, dims] = torch.where(rows, mag * sign, x[:, dims])
    return x.to(dtype)


def _spread(s, n):
    """One value per 128 along dim 0 -> one per element."""
    return s.repeat_interleave(BLOCK, 0)[:n]


def _blocks_of_rows(y):
    """Plain quantizer of fp32 rows: (e4m3 [M, K], fp32 scales [ceil(K/128), M]).
    The e4m3 tensor holds numbers of its own type; each times its block's scale is the row's value."""
    M, K = y.shape
    kb = -(-K // BLOCK)
    padded = torch.nn.functional.pad(y, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    amax = padded.abs().amax(2).clamp(min=FLOOR)
    q = (padded * (E4M3_MAX / amax)[:, :, None]).view(M, kb * BLOCK)[:, :K]
    return q.to(torch.float8_e4m3fn), (amax / E4M3_MAX).t().contiguous()


def _weight(g, N, K):
    """Random N(0, 0.02^2) weights as a checkpoint holds them: e4m3 [N, K] and a scale per 128 x 128 block."""
    w = torch.randn((N, K), generator=g, device="cuda").mul_(0.02)
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    w = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    scale = w.abs().amax((1, 3)) / E4M3_MAX
    w = w.div_(scale[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * BLOCK, kb * BLOCK)
    return w[:N, :K].contiguous(), scale.contiguous()


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, K, dtype = case["M"], case["K"], _TYPES[case["dtype"]]
    s = dict(op=case["op"], M=M, K=K, dtype=dtype)
    if case["op"] == "norm":
        s["x"] = _activations(g, M, K, dtype)
        s["weight"] = (1.0 + 0.2 * torch.randn((K,), generator=g, device="cuda")).to(dtype)
        s["residual"] = _activations(g, M, K, dtype) if case["residual"] else None
    elif case["op"] == "quantize":
        s["x"] = _activations(g, M, K, dtype)
    elif case["op"] == "silu":
        s["x"] = torch.randn((M, 2 * K), generator=g, device="cuda").mul_(2.0).to(dtype)
    else:
        s["N"] = case["N"]
        s["xq"], s["xs"] = _blocks_of_rows(_activations(g, M, K, dtype).float())
        s["wq"], s["ws"] = _weight(g, case["N"], K)
        s["bias"] = torch.randn((case["N"],), generator=g, device="cuda").to(dtype) if case["bias"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] == "matmul":
        import int8_mixed_precision_outlier_amd as i8
        s["wq"] = i8.fp8_pack_weight(s["wq"])  # laid out once, at load
    return s


def _run_own(s):
    import int8_mixed_precision_outlier_amd as i8
    if s["op"] == "norm":
        return i8.fp8_rms_norm(s["x"], s["weight"], eps=EPS, residual=s["residual"])
    if s["op"] == "quantize":
        return i8.fp8_quantize(s["x"])
    if s["op"] == "silu":
        return i8.fp8_silu_mul(s["x"])
    return i8.fp8_matmul(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"], out_dtype=s["dtype"])


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = (h + s["residual"].float()).to(s["dtype"])
            out = (h,)
            h = h.float()
        else:
            out = ()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
        return _blocks_of_rows(y) + out
    if s["op"] == "quantize":
        return _blocks_of_rows(s["x"].float())
    if s["op"] == "silu":
        gate, up = s["x"].float().split(s["K"], 1)
        return _blocks_of_rows(gate / (1.0 + torch.exp(-gate)) * up)
    K, N = s["K"], s["N"]
    x = s["xq"].float() * _spread(s["xs"], K).t()
    w = s["wq"].float() * _spread(_spread(s["ws"], N).t(), K).t()
    y = x @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["dtype"])


def work(case):
    M, K = case["M"], case["K"]
    scales = 4 * M * -(-K // BLOCK)
    if case["op"] == "norm":
        wide = 3 if case["residual"] else 1  # rows of x, and of the residual in and out
        return dict(bytes=2 * M * K * wide + 2 * K + M * K + scales, flops=8 * M * K)
    if case["op"] == "quantize":
        return dict(bytes=3 * M * K + scales, flops=3 * M * K)
    if case["op"] == "silu":
        return dict(bytes=5 * M * K + scales, flops=8 * M * K)
    N = case["N"]
    b = M * K + scales + N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK) + 2 * M * N + (2 * N if case["bias"] else 0)
    return dict(bytes=b, flops=2 * M * N * K)


def _exact_blocks(y):
    """64-bit quantizer: q before its rounding to e4m3, and the scales."""
    M, K = y.shape
    qs, scales = [], []
    for k in range(0, K, BLOCK):
        part = y[:, k:k + BLOCK]
        scale = part.abs().max(1).values.clamp(min=FLOOR) / E4M3_MAX
        qs.append(part / scale[:, None])
        scales.append(scale)
    return torch.cat(qs, 1), torch.stack(scales)


def exact(case, seed):
    s = _inputs(case, seed)
    M, K = s["M"], s["K"]
    if s["op"] == "norm":
        h = s["x"].double()
        out = ()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["dtype"]).double()  # the sum is exact, then the type's one rounding
            out = (h,)
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / K + EPS) * s["weight"].double()
        return _exact_blocks(y) + out
    if s["op"] == "quantize":
        return _exact_blocks(s["x"].double())
    if s["op"] == "silu":
        gate, up = s["x"][:, :K].double(), s["x"][:, K:].double()
        return _exact_blocks(gate * torch.sigmoid(gate) * up)
    y = torch.zeros((M, s["N"]), dtype=torch.float64, device="cuda")
    for b in range(-(-K // BLOCK)):
        cols = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        part = s["xq"][:, cols].double() @ s["wq"][:, cols].double().t()
        sw = s["ws"][:, b].double().repeat_interleave(BLOCK)[:s["N"]]
        y.addcmul_(part.mul_(s["xs"][b].double()[:, None]), sw[None, :])
    return y if s["bias"] is None else y + s["bias"].double()
