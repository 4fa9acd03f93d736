"""Cases of the operators around the packed linear layer: the layer with bias, activation and residual
in its epilogue, the gated feed-forward projection with its backward pass, and the layer's input gradient.

Weights are packed as the library packs them: codes of 4 bits, 8 per int32 word along K (lowest K index in
the lowest nibble), one BF16 scale and one int32 zero point per group along K, W = (q - z) s.  A gated
weight holds the gate rows, then as many up rows.
"""
import math

import torch

own = False  # set by the tools: false runs the plain forms, true the library's entry points

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")  # in the order of the library's activation codes


def listed():
    return [
        # one new token after attention: the output projection added to the residual stream
        dict(name="linear 1 token residual", op="linear", M=1, K=5120, N=5120, group=128, bias=False, act="none", residual=True),
        # a small serving batch: the feed-forward's second projection added to the residual stream
        dict(name="linear 7 tokens residual", op="linear", M=7, K=28672, N=8192, group=128, bias=False, act="none", residual=True),
        # a larger serving batch: the attention's input projection with its bias, finer groups
        dict(name="linear 33 tokens bias g64", op="linear", M=33, K=8192, N=10240, group=64, bias=True, act="none", residual=False),
        # a prompt through a classic feed-forward's first projection
        dict(name="linear 1000 tokens bias gelu", op="linear", M=1000, K=4096, N=16384, group=128, bias=True, act="gelu", residual=False),
        # a long prompt through the feed-forward's second projection
        dict(name="linear 4096 tokens residual", op="linear", M=4096, K=28672, N=8192, group=128, bias=False, act="none", residual=True),
        # one new token through the gated projections
        dict(name="gated 1 token", op="gated", M=1, K=5120, N=51200, group=128, act="silu", save=False),
        # a serving batch through the gated projections, the finest groups
        dict(name="gated 48 tokens g32", op="gated", M=48, K=5120, N=51200, group=32, act="silu", save=False),
        # training with frozen weights: the forward pass keeps the pre-activations
        dict(name="gated 2048 tokens saved", op="gated", M=2048, K=8192, N=57344, group=128, act="silu", save=True),
        # a short sequence's gradient through the attention's input projection
        dict(name="dx 100 tokens", op="dx", M=100, K=5120, N=7680, group=128),
        # a long sequence's gradient through the attention's input projection
        dict(name="dx 4096 tokens", op="dx", M=4096, K=8192, N=10240, group=128),
        # backward of a gated block of odd width
        dict(name="gated backward 333 tokens odd", op="gated_backward", M=333, K=4096, N=22002, group=64, act="gelu_tanh"),
        # backward of the largest gated block
        dict(name="gated backward 2048 tokens", op="gated_backward", M=2048, K=8192, N=57344, group=128, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "gated", "dx", "gated_backward"))
    K = 128 * _log(rng, 8, 224)
    N = _log(rng, 512, 57344)
    if op.startswith("gated"):
        N = 2 * max(1, N // 2)
    M = _log(rng, 1, 4096) if op in ("linear", "gated") else _log(rng, 8, 4096)
    while M * N * K > 2 ** 39:  # no more work than the largest listed case
        M = max(1, M * 3 // 4)
    case = dict(op=op, M=M, K=K, N=N, group=rng.choice((128, 128, 64, 32)))
    if op == "linear":
        case.update(bias=rng.random() < 0.5, act=rng.choice(ACTS), residual=rng.random() < 0.5)
    if op == "gated":
        case.update(act=rng.choice(("silu", "gelu", "gelu_tanh")), save=rng.random() < 0.5)
    if op == "gated_backward":
        case.update(act=rng.choice(("silu", "gelu", "gelu_tanh")))
    return case


def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    b = N * K / 2 + 6.0 * N * (K // case["group"])  # codes, scales and zero points
    op = case["op"]
    if op == "linear":
        b += 2 * M * K + 2 * M * N + (2 * N if case["bias"] else 0) + (2 * M * N if case["residual"] else 0)
    elif op == "gated":
        b += 2 * M * K + M * N + (2 * M * N if case["save"] else 0)
    elif op == "dx":
        b += 2 * M * N + 2 * M * K
    else:
        b += M * N + 2 * M * N + 2 * M * N + 2 * M * K
    return {"bytes": float(b), "flops": 2.0 * M * N * K}


def _packed(N, K, group, gen):
    """A weight of standard deviation 0.02, quantised group by group and packed."""
    qweight = torch.empty((N, K // 8), dtype=torch.int32, device="cuda")
    scales = torch.empty((N, K // group), dtype=torch.bfloat16, device="cuda")
    zeros = torch.empty((N, K // group), dtype=torch.int32, device="cuda")
    shift = 4 * torch.arange(8, device="cuda", dtype=torch.int64)
    for r in range(0, N, 4096):
        n = min(4096, N - r)
        w = 0.02 * torch.randn((n, K // group, group), device="cuda", generator=gen)
        lo, hi = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
        s = ((hi - lo) / 15).to(torch.bfloat16)
        z = torch.round(-lo / s.float())
        q = (torch.round(w / s.float()) + z).clamp_(0, 15).to(torch.int64).view(n, K // 8, 8)
        qweight[r : r + n] = (q << shift).sum(-1).to(torch.int32)
        scales[r : r + n] = s.squeeze(-1)
        zeros[r : r + n] = z.squeeze(-1).to(torch.int32)
    return qweight, scales, zeros


def _activations(M, K, gen):
    """Unit normal with one channel in a hundred twenty times larger, as a transformer's hidden state."""
    x = torch.randn((M, K), device="cuda", generator=gen)
    x[:, torch.randperm(K, device="cuda", generator=gen)[: max(1, K // 100)]] *= 20
    return x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    st = dict(case)
    st["q"], st["s"], st["z"] = _packed(N, K, case["group"], gen)
    st["bias_t"] = st["residual_t"] = None
    if op in ("linear", "gated"):
        st["X"] = _activations(M, K, gen)
    if op == "linear":
        if case["bias"]:
            st["bias_t"] = normal(N).to(torch.bfloat16)
        if case["residual"]:
            st["residual_t"] = (4 * normal(M, N)).to(torch.bfloat16)
    if op == "dx":  # gradients are small, and some tokens' far smaller than others'
        st["dY"] = (normal(M, N) * 1e-3 * torch.exp2(3 * normal(M, 1))).to(torch.bfloat16)
    if op == "gated_backward":
        st["dH"] = (normal(M, N // 2) * 1e-3 * torch.exp2(3 * normal(M, 1))).to(torch.bfloat16)
        st["GU"] = (2 * normal(M, N)).to(torch.bfloat16)
    if own:  # what a caller of the library keeps: the zeroed workspace and the output buffers
        import weight_only_int4_linear_b200 as w4

        st["lib"], st["code"] = w4, ACTS.index(case.get("act", "none"))
        forward = op in ("linear", "gated")
        size = w4.fused_workspace_bytes(M, N, K, case["group"]) if forward else w4.dx_workspace_bytes(M, N, K, case["group"])
        st["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        if op == "linear":
            st["Y"] = new(M, N)
        elif op == "gated":
            st["H"], st["out_GU"] = new(M, N // 2), new(M, N) if case["save"] else None
        else:
            st["dX"] = new(M, K)
            if op == "gated_backward":
                st["dGU"] = new(M, N)
    return st


def _weight(st):
    """The dequantised weight in 32 bits (each value exact)."""
    N, K = st["N"], st["K"]
    shift = 4 * torch.arange(8, device="cuda", dtype=torch.int32)
    codes = ((st["q"][:, :, None] >> shift) & 15).view(N, -1, st["group"])
    return ((codes - st["z"][:, :, None]).float() * st["s"][:, :, None].float()).view(N, K)


def _act(x, act):
    if act == "relu":
        return x.clamp_min(0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _act_grad(x, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if act == "gelu":
        return 0.5 * torch.special.erfc(-x / math.sqrt(2)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def run(st):
    op, bf = st["op"], torch.bfloat16
    if own:
        w4, w = st["lib"], (st["q"], st["s"], st["z"])
        if op == "linear":
            w4.linear_fused(st["X"], *w, st["Y"], st["ws"], bias=st["bias_t"], act=st["code"], residual=st["residual_t"], group=st["group"])
            return st["Y"]
        if op == "gated":
            w4.gated(st["X"], *w, st["H"], st["ws"], act=st["code"], GU=st["out_GU"], group=st["group"])
            return [st["H"], st["out_GU"]] if st["save"] else [st["H"]]
        if op == "dx":
            w4.linear_dx(st["dY"], *w, st["dX"], st["ws"], group=st["group"])
            return st["dX"]
        w4.gated_backward(st["dH"], st["GU"], *w, st["dGU"], st["dX"], st["ws"], act=st["code"], group=st["group"])
        return [st["dX"], st["dGU"]]
    W, I = _weight(st), st["N"] // 2
    if op == "linear":
        y = st["X"].float() @ W.t()
        if st["bias_t"] is not None:
            y = y + st["bias_t"].float()
        y = _act(y, st["act"])
        if st["residual_t"] is not None:
            y = y + st["residual_t"].float()
        return y.to(bf)
    if op == "gated":
        y = st["X"].float() @ W.t()
        h = (_act(y[:, :I], st["act"]) * y[:, I:]).to(bf)
        return [h, y.to(bf)] if st["save"] else [h]
    if op == "dx":
        return (st["dY"].float() @ W).to(bf)
    g, u, d = st["GU"][:, :I].float(), st["GU"][:, I:].float(), st["dH"].float()
    dgu = torch.cat([d * u * _act_grad(g, st["act"]), d * _act(g, st["act"])], 1)
    return [(dgu @ W).to(bf), dgu.to(bf)]


def exact(case, seed):
    """The operators' definitions in 64 bits, the weight taken some rows at a time."""
    st = prepare(case, seed)
    f8, N, K, I, op = torch.float64, case["N"], case["K"], case["N"] // 2, case["op"]

    def rows(a, b):  # rows a..b of the weight, from the bytes of the packed words (little endian)
        by = st["q"][a:b].contiguous().view(torch.uint8)
        c = torch.stack([by % 16, by // 16], -1).reshape(b - a, K).to(f8)
        g = case["group"]
        return (c - st["z"][a:b].to(f8).repeat_interleave(g, 1)) * st["s"][a:b].to(f8).repeat_interleave(g, 1)

    cuts = [(a, min(a + 4096, N)) for a in range(0, N, 4096)]

    def f(x):
        name = case["act"]
        if name == "relu":
            return torch.where(x > 0, x, torch.zeros_like(x))
        if name == "silu":
            return x * torch.sigmoid(x)
        if name == "gelu":
            return x * torch.special.ndtr(x)
        if name == "gelu_tanh":
            return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x**3))
        return x

    if op in ("linear", "gated"):
        x = st["X"].to(f8)
        y = torch.cat([x @ rows(a, b).T for a, b in cuts], 1)
        if op == "gated":
            h = f(y[:, :I]) * y[:, I:]
            return [h, y] if case["save"] else [h]
        y = f(y + (st["bias_t"].to(f8) if case["bias"] else 0))
        return y + st["residual_t"].to(f8) if case["residual"] else y
    if op == "dx":
        d = st["dY"].to(f8)
        return sum(d[:, a:b] @ rows(a, b) for a, b in cuts)
    g = st["GU"][:, :I].to(f8).requires_grad_(True)
    u = st["GU"][:, I:].to(f8).requires_grad_(True)
    (f(g) * u).backward(st["dH"].to(f8))  # the derivative from the definition, by automatic differentiation
    d = torch.cat([g.grad, u.grad], 1)
    return [sum(d[:, a:b] @ rows(a, b) for a, b in cuts), d]
