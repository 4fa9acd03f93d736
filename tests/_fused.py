"""References in 64 bits and error bounds for the fused operators (epilogue, gated projection, gradients).

Bounds.  u16 = 2^-8 is BF16's largest relative rounding error and 2^-11 FP16's (half a step).  A sum of C products
p_i whose operands carry a relative error r ends within (r + (C / 16) 2^-22) sum |p_i| of the exact one: each
tensor-core step of 16 products adds at most 2^-22 of the running magnitude.  r is
  * GEMM paths: 2^-11, the rounding of the scaled weight to FP16 (tokens are exact except below 2^-29 of their row's
    maximum, an absolute 2^-40 of it);
  * integer GEMVs: none, but each activation may be off by 2^-18 of its group's maximum (the fixed-point step).
Both are charged to every path.  Activations have slopes of at most 1.13 and are computed to 2^-18 of their value."""
from __future__ import annotations

import math

import torch

import weight_only_int4_linear_b200 as w4

U16 = 2.0 ** -8
TINY = 2.0 ** -134  # half a step of BF16's subnormals
SLOPE = 1.13
F8 = torch.float64
ACTS = [w4.ACT_NONE, w4.ACT_RELU, w4.ACT_SILU, w4.ACT_GELU, w4.ACT_GELU_TANH]


def pack(W: torch.Tensor, group: int, symmetric: bool = False):
    N, K = W.shape
    pw = w4.PackedWeight(N, K, device=W.device, group=group)
    status = torch.zeros(1, dtype=torch.int32, device=W.device)
    w4.quantize_pack_g(W, group, pw.qweight, pw.scales, pw.zeros, status, symmetric=symmetric)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return pw


def weight64(pw) -> torch.Tensor:
    codes = torch.stack([(pw.qweight >> (4 * i)) & 15 for i in range(8)], -1).reshape(pw.N, pw.K).to(F8)
    g = pw.group
    return (codes - pw.zeros.to(F8).repeat_interleave(g, 1)) * pw.scales.to(F8).repeat_interleave(g, 1)


def make_weight(N: int, K: int, group: int, seed: int, far: bool = False):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    W = 0.02 * torch.randn((N, K), device="cuda", generator=gen)
    W[: max(1, N // 7)] += 0.05           # zero points spread over the grid and past it
    W *= torch.exp2(torch.randint(-6, 7, (N, 1), device="cuda", generator=gen).float())  # rows of other sizes
    if far:
        W[0] = 20.0 + 0.01 * torch.randn(K, device="cuda", generator=gen)  # zero points beyond 1024
        W[N // 2, :128] -= 30.0
        W[N - 1] = 0.0
    return pack(W, group)


def tokens(M: int, K: int, seed: int, scale: float = 1.0) -> torch.Tensor:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    x = scale * torch.randn((M, K), device="cuda", generator=gen)
    x[:, torch.randperm(K, device="cuda", generator=gen)[: max(1, K // 100)]] *= 20
    return x.to(torch.bfloat16)


def act64(x: torch.Tensor, act: int) -> torch.Tensor:
    if act == w4.ACT_RELU:
        return torch.relu(x)
    if act == w4.ACT_SILU:
        return x * torch.sigmoid(x)
    if act == w4.ACT_GELU:
        return 0.5 * x * torch.special.erfc(-x / math.sqrt(2))
    if act == w4.ACT_GELU_TANH:
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    return x


def grad64(x: torch.Tensor, act: int) -> torch.Tensor:
    if act == w4.ACT_RELU:
        return (x > 0).to(F8)
    if act == w4.ACT_SILU:
        s = torch.sigmoid(x)
        return s * (1 + x * torch.sigmoid(-x))
    if act == w4.ACT_GELU:
        return 0.5 * torch.special.erfc(-x / math.sqrt(2)) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if act == w4.ACT_GELU_TANH:
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (x + 0.044715 * x ** 3))
        return s + x * s * (1 - s) * c * (1 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def product64(X: torch.Tensor, W: torch.Tensor, group: int = 128):
    """X . W^T and the bound of its error before any rounding of the output."""
    K = X.shape[1]
    x, gmax = X.to(F8), X.to(F8).abs().reshape(X.shape[0], K // 128, 128).amax(-1).repeat_interleave(128, 1)
    r = 2.0 ** -11 + (K / 16 + 4) * 2.0 ** -22
    return x @ W.T, r * (x.abs() @ W.abs().T) + 2.0 ** -18 * (gmax @ W.abs().T)


def linear64(X, W, bias, act, residual):
    s, e = product64(X, W)
    if bias is not None:
        s = s + bias.to(F8)
    y = act64(s, act)
    e = SLOPE * e + 2.0 ** -18 * y.abs()
    if residual is not None:
        y = y + residual.to(F8)
    return y, e + 2.0 ** -22 * y.abs() + U16 * (y.abs() + e) + TINY


def gated64(X, W, act):
    s, e = product64(X, W)
    I = W.shape[0] // 2
    g, u, eg, eu = s[:, :I], s[:, I:], e[:, :I], e[:, I:]
    f = act64(g, act)
    ef = SLOPE * eg + 2.0 ** -18 * f.abs()
    h = f * u
    eh = ef * u.abs() + f.abs() * eu + ef * eu
    return h, eh * (1 + U16) + U16 * h.abs() + 2.0 ** -22 * h.abs() + TINY, s, e + U16 * (s.abs() + e) + TINY


def dx64(d, W, inv_s=None, r_d: float = 0.0, size=None):
    """d . W (d in 64 bits, its FP16 operand off by r_d relative) and the bound of the BF16 result.

    A token's operands d_n 2^e_n are scaled so that the largest -- of d, or of the bound `size` that the gated backward
    scales by -- is in [2^14, 2^15); FP16's half step is 2^-25 at least, so each may be off by 2^-39 of it.  2^e_n |W'|
    with |W'| < 2^15 stands for a weight row whose largest value is within 2^5 of that (2^e_n bounds the row by whole
    powers: the exponents of scale and zero point separately): N 2^-34 of the largest |size_n| max_k |W[n][k]| in all."""
    N = W.shape[0]
    top = ((d if size is None else size).abs() * W.abs().amax(1)).amax(1, keepdim=True)
    r = 2.0 ** -11 + r_d + (N / 16 + 4) * 2.0 ** -22
    y, e = d @ W, r * (d.abs() @ W.abs()) + 2.0 ** -34 * N * top
    if inv_s is not None:
        y, e = y * inv_s.to(F8), e * inv_s.to(F8).abs()
    return y, e + 2.0 ** -22 * y.abs() + U16 * (y.abs() + e) + TINY


def grads64(dH, GU, act):
    I = dH.shape[1]
    g, u, d = GU[:, :I].to(F8), GU[:, I:].to(F8), dH.to(F8)
    out = torch.cat([d * u * grad64(g, act), d * act64(g, act)], 1)
    # act' is a sum of terms of magnitude up to about 1.2: computed to 2^-17 absolutely
    e = torch.cat([2.0 ** -17 * (d * u).abs(), 2.0 ** -17 * (d * act64(g, act)).abs()], 1)
    return out, e


def gated_size(dH, GU):
    """What the gated backward scales a token by: |dH| max(2 |U|, |G|) for both halves."""
    I = dH.shape[1]
    b = dH.to(F8).abs() * torch.maximum(2 * GU[:, I:].to(F8).abs(), GU[:, :I].to(F8).abs())
    return torch.cat([b, b], 1)


def check(got: torch.Tensor, want: torch.Tensor, bound: torch.Tensor, what: str = "") -> None:
    g = got.to(F8)
    assert g.shape == want.shape, what
    assert bool(torch.isfinite(g).all()), f"{what}: non-finite outputs"
    over = (g - want).abs() / bound.clamp_min(1e-300)
    worst = float(over.max())
    assert worst <= 1.0, f"{what}: error {worst:.3g} times the bound at {divmod(int(over.argmax()), want.shape[1])}"


def workspace(nbytes: int) -> torch.Tensor:
    assert nbytes > 0 and nbytes % 256 == 0
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


def nans(*shape) -> torch.Tensor:
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
