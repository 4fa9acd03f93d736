"""The fused linear layer, the gated projection, the input gradient and the gated backward pass on the GPU against
their definitions in 64 bits; bounds derived in tests/_fused.py."""
import numpy as np
import pytest
import torch

import oracle
import weight_only_int4_linear_b200 as w4
from tests import _fused as F

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (scale * torch.randn(shape, device="cuda", generator=gen)).to(BF)


def _done():
    torch.cuda.synchronize()
    assert w4.device_fault() == 0


def _linear(X, pw, bias=None, act=0, residual=None, inv_s=None, Y=None, ws=None):
    M, N = X.shape[0], pw.N
    Y = F.nans(M, N) if Y is None else Y
    ws = F.workspace(w4.fused_workspace_bytes(M, N, pw.K, pw.group)) if ws is None else ws
    w4.linear_fused(X, pw.qweight, pw.scales, pw.zeros, Y, ws, bias=bias, act=act, residual=residual, group=pw.group,
                    inv_s=inv_s)
    _done()
    return Y


def _gated(X, pw, act, save, inv_s=None):
    M, I = X.shape[0], pw.N // 2
    H, GU = F.nans(M, I), F.nans(M, pw.N) if save else None
    ws = F.workspace(w4.fused_workspace_bytes(M, pw.N, pw.K, pw.group))
    w4.gated(X, pw.qweight, pw.scales, pw.zeros, H, ws, act=act, GU=GU, group=pw.group, inv_s=inv_s)
    _done()
    return H, GU


def _dx(dY, pw, inv_s=None):
    dX = F.nans(dY.shape[0], pw.K)
    ws = F.workspace(w4.dx_workspace_bytes(dY.shape[0], pw.N, pw.K, pw.group))
    w4.linear_dx(dY, pw.qweight, pw.scales, pw.zeros, dX, ws, group=pw.group, inv_s=inv_s)
    _done()
    return dX


def _backward(dH, GU, pw, act, inv_s=None, in_place=False):
    M = dH.shape[0]
    dGU, dX = GU if in_place else F.nans(M, pw.N), F.nans(M, pw.K)
    ws = F.workspace(w4.dx_workspace_bytes(M, pw.N, pw.K, pw.group))
    w4.gated_backward(dH, GU, pw.qweight, pw.scales, pw.zeros, dGU, dX, ws, act=act, group=pw.group, inv_s=inv_s)
    _done()
    return dGU, dX


# one token and 2-16 tokens (integer GEMVs), every tile width of the GEMM, ragged tokens and rows, a K that is no
# multiple of 1024, contractions of one group, cut and whole tiles
FORWARD = [(1, 257, 1024, 128), (1, 130, 512, 64), (1, 96, 1024, 32), (1, 77, 128, 128), (1, 300, 384, 32),
           (2, 200, 1024, 128), (9, 513, 2048, 128), (16, 129, 1024, 128), (16, 129, 640, 128), (3, 260, 512, 64),
           (17, 257, 1024, 128), (40, 1000, 384, 64), (64, 70, 256, 32), (65, 300, 1024, 128), (128, 513, 640, 128),
           (129, 200, 2048, 64), (300, 1030, 512, 32), (513, 259, 128, 128),
           # rows longer than a block's step and more than 256 groups; two waves of tiles and a rest; most of a wave
           (20, 70, 9216, 32), (200, 130, 9216, 128), (300, 19500, 256, 128), (200, 17900, 128, 128), (90, 19500, 128, 64)]


@pytest.mark.parametrize("M,N,K,G", FORWARD)
def test_linear_fused_against_64_bits(cuda_lib, M, N, K, G):
    pw = F.make_weight(N, K, G, seed=M + N + K, far=True)
    W, X = F.weight64(pw), F.tokens(M, K, M + K)
    bias, res = _rand(N, 3, 2.0), _rand((M, N), 4, 4.0)
    act = F.ACTS[(M + N) % 5]
    for b, a, r in [(None, w4.ACT_NONE, None), (bias, act, res)]:
        want, bound = F.linear64(X, W, b, a, r)
        F.check(_linear(X, pw, b, a, r), want, bound, f"bias={b is not None} act={a}")


@pytest.mark.parametrize("act", F.ACTS)
@pytest.mark.parametrize("M", [1, 5, 33])
def test_every_activation_with_and_without_bias_and_residual(cuda_lib, M, act):
    N, K = 300, 1024
    pw = F.make_weight(N, K, 128, seed=act)
    W, X = F.weight64(pw), F.tokens(M, K, act)
    for b in (None, _rand(N, 5)):
        for r in (None, _rand((M, N), 6)):
            want, bound = F.linear64(X, W, b, act, r)
            F.check(_linear(X, pw, b, act, r), want, bound, f"act={act} bias={b is not None} residual={r is not None}")


@pytest.mark.parametrize("M,N,K,G", [(1, 258, 1024, 128), (1, 514, 512, 32), (1, 2, 1024, 128), (2, 402, 1024, 128),
                                     (13, 770, 2048, 128), (16, 130, 640, 64), (31, 258, 1024, 128), (64, 1026, 384, 32),
                                     (100, 514, 512, 64), (200, 1538, 1024, 128), (260, 34, 128, 128),
                                     (260, 19458, 128, 64), (50, 100, 9216, 32)])
@pytest.mark.parametrize("save", [False, True])
def test_gated_against_64_bits(cuda_lib, M, N, K, G, save):
    pw = F.make_weight(N, K, G, seed=N + K, far=True)
    X = F.tokens(M, K, M)
    act = [w4.ACT_SILU, w4.ACT_GELU, w4.ACT_GELU_TANH, w4.ACT_RELU, w4.ACT_NONE][(M + K // 128) % 5]
    want, bound, gu, gu_bound = F.gated64(X, F.weight64(pw), act)
    H, GU = _gated(X, pw, act, save)
    F.check(H, want, bound, "H")
    if save:
        F.check(GU, gu, gu_bound, "GU")


BACKWARD = [(1, 257, 128, 128), (1, 1000, 1024, 64), (5, 64, 384, 32), (33, 129, 640, 128), (64, 1003, 512, 64),
            (100, 520, 1024, 32), (128, 65, 256, 128), (200, 2050, 384, 128), (300, 96, 1152, 64), (600, 770, 512, 32),
            # several steps per row of the gradients' preparation, its form for many tokens, many tiles, many groups
            (3, 9000, 256, 128), (2, 8195, 128, 64), (601, 5000, 384, 64), (300, 130, 19456, 128), (5, 40, 9216, 32)]


@pytest.mark.parametrize("M,N,K,G", BACKWARD)
def test_linear_dx_against_64_bits(cuda_lib, M, N, K, G):
    pw = F.make_weight(N, K, G, seed=N * 3 + K, far=True)
    dY = _rand((M, N), M, 1e-3)
    dY[M // 2] *= 2.0 ** 40  # tokens of other magnitudes
    dY[0, : N // 2] = 0
    want, bound = F.dx64(dY.to(F.F8), F.weight64(pw))
    F.check(_dx(dY, pw), want, bound)


@pytest.mark.parametrize("M,N,K,G", [(1, 258, 128, 128), (7, 1030, 384, 64), (64, 514, 512, 32), (90, 1536, 640, 128),
                                     (257, 130, 1024, 128), (300, 2064, 256, 32), (2, 18000, 256, 64), (3, 16402, 128, 128)])
@pytest.mark.parametrize("act", F.ACTS)
def test_gated_backward_against_64_bits(cuda_lib, M, N, K, G, act):
    pw = F.make_weight(N, K, G, seed=N + K + 1, far=True)
    dH, GU = _rand((M, N // 2), M + act, 1e-2), _rand((M, N), M + 50, 3.0)
    GU[0, :8] = torch.tensor([-100.0, 100.0, -30.0, 30.0, 0.0, -0.0, -12.0, 12.0], device="cuda", dtype=BF)
    GU[0, 8:16] = torch.tensor([-87.0, -87.5, -88.0, -89.0, 87.5, 89.0, -3e4, 3e4], device="cuda", dtype=BF)
    d, e = F.grads64(dH, GU, act)
    dGU, dX = _backward(dH, GU, pw, act)
    F.check(dGU, d, e + F.U16 * (d.abs() + e) + F.TINY, "dGU")
    W = F.weight64(pw)
    want, bound = F.dx64(d, W, r_d=2.0 ** -11, size=F.gated_size(dH, GU))
    F.check(dX, want, bound + (1 + F.U16) * (e @ W.abs()), "dX")
    keep = GU.clone()
    dGU2, dX2 = _backward(dH, keep, pw, act, in_place=True)  # dGU in GU's place: the same bits
    assert dGU2.data_ptr() == keep.data_ptr()
    assert torch.equal(dGU2, dGU) and torch.equal(dX2, dX)


@pytest.mark.parametrize("M,K,G", [(1, 1024, 128), (1, 512, 64), (6, 1024, 128), (50, 640, 32)])
def test_awq_scales_forward_and_backward(cuda_lib, M, K, G):
    N = 258
    pw = F.make_weight(N, K, G, seed=K + M)
    X = F.tokens(M, K, 9)
    inv = torch.exp2(torch.linspace(-3, 3, K, device="cuda")) * 1.1
    bits = X.view(torch.int16).cpu().numpy().view(np.uint16)
    Xs = torch.from_numpy(oracle.awq_scale_activations(bits, inv.cpu().numpy()).view(np.int16)).cuda().view(BF)
    W = F.weight64(pw)
    want, bound = F.linear64(Xs, W, None, w4.ACT_RELU, None)
    F.check(_linear(X, pw, None, w4.ACT_RELU, None, inv_s=inv), want, bound, "linear_fused")
    want, bound, _, _ = F.gated64(Xs, W, w4.ACT_SILU)
    F.check(_gated(X, pw, w4.ACT_SILU, False, inv_s=inv)[0], want, bound, "gated")
    dY = _rand((M, N), 8)
    want, bound = F.dx64(dY.to(F.F8), W, inv)
    F.check(_dx(dY, pw, inv), want, bound, "linear_dx")


@pytest.mark.parametrize("M", [1, 4, 24, 300])
def test_residual_in_place(cuda_lib, M):
    """Y = act(X W^T) + Y: the same bits as with a residual of its own."""
    N, K = 520, 1024
    pw = F.make_weight(N, K, 128, seed=5)
    X, res = F.tokens(M, K, 1), _rand((M, N), 2, 3.0)
    apart = _linear(X, pw, None, w4.ACT_SILU, res)
    both = res.clone()
    _linear(X, pw, None, w4.ACT_SILU, both, Y=both)
    assert torch.equal(apart, both)


@pytest.mark.parametrize("M", [1, 3, 30, 140])
def test_extreme_magnitudes(cuda_lib, M):
    """Rows and tokens at the ends of BF16's range: nothing leaves the operands' range unless the result does."""
    N, K = 260, 1024
    pw = F.make_weight(N, K, 128, seed=11)
    W = F.weight64(pw)
    X = F.tokens(M, K, 3)
    for scale in (2.0 ** 100, 2.0 ** -100):
        Xs = (X.double() * scale).to(BF)
        want, bound = F.linear64(Xs, W, None, w4.ACT_NONE, None)
        F.check(_linear(Xs, pw), want, bound, f"scale {scale}")
        dY = (_rand((M, N), 7).double() * scale).to(BF)
        want, bound = F.dx64(dY.to(F.F8), W)
        F.check(_dx(dY, pw), want, bound, f"dx scale {scale}")
    Z = torch.zeros((M, K), dtype=BF, device="cuda")
    assert not _linear(Z, pw).any() and not _dx(torch.zeros((M, N), dtype=BF, device="cuda"), pw).any()
    Z[:, 5] = 1.0  # one-hot tokens give BF16 of a weight column (FP16 first: 12 of its 13 bits)
    want, bound = F.linear64(Z, W, None, w4.ACT_NONE, None)
    F.check(_linear(Z, pw), want, bound, "one-hot")


@pytest.mark.parametrize("M", [2, 70])
def test_gated_backward_at_the_ends_of_the_range(cuda_lib, M):
    """Gradients of extreme size, rows of extreme weights (their powers of two are no normal FP32 numbers), and tokens
    whose every gate is shut, whose operand is made from the rounded gradients."""
    N, K = 514, 256
    pw = F.make_weight(N, K, 64, seed=13, far=True)
    pw.scales[3::7] = (pw.scales[3::7].double() * 2.0 ** -112).to(BF)
    W = F.weight64(pw)
    for scale in (2.0 ** 90, 2.0 ** -95, 1.0):
        for act in (w4.ACT_SILU, w4.ACT_GELU, w4.ACT_GELU_TANH):
            dH, GU = (_rand((M, N // 2), 1).double() * scale).to(BF), _rand((M, N), 2, 2.0)
            shut = M // 2
            GU[shut, : N // 2] = -abs(GU[shut, : N // 2]) - (30.0 if act == w4.ACT_SILU else 7.0)
            d, e = F.grads64(dH, GU, act)
            # FP32 holds the shut gates' gradients to a relative 2^-16 (a difference of two small terms, e^x for large
            # x); below 2^-126 to half a step of its subnormals times the factors that follow
            e[shut] = 2.0 ** -14 * (dH[shut].double().abs() * (1 + GU[shut, : N // 2].double().abs()) ** 3
                                    * torch.exp(GU[shut, : N // 2].double())).repeat(2) * torch.cat(
                [GU[shut, N // 2:].double().abs() + 1, torch.ones(N // 2, device="cuda", dtype=F.F8)])
            e = e + 2.0 ** -126
            dGU, dX = _backward(dH, GU, pw, act)
            F.check(dGU, d, e + F.U16 * (d.abs() + e) + F.TINY, f"dGU {scale} {act}")
            want, bound = F.dx64(d, W, r_d=2.0 ** -8, size=F.gated_size(dH, GU))
            F.check(dX, want, bound + (1 + F.U16) * (e @ W.abs()), f"dX {scale} {act}")


@pytest.mark.parametrize("M,N,K,G", [(20, 258, 4096, 128), (100, 514, 3968, 32), (300, 1030, 8192, 64)])
def test_cut_tiles_forward(cuda_lib, M, N, K, G):
    """Few tiles of a long contraction, cut over the clusters and joined: every mode's epilogue after the join."""
    pw = F.make_weight(N, K, G, seed=31, far=True)
    W, X = F.weight64(pw), F.tokens(M, K, 5)
    bias, residual = _rand((N,), 6), _rand((M, N), 7)
    F.check(_linear(X, pw, bias, w4.ACT_GELU, residual), *F.linear64(X, W, bias, w4.ACT_GELU, residual), "linear")
    want, bound, gu, gu_bound = F.gated64(X, W, w4.ACT_SILU)
    H, GU = _gated(X, pw, w4.ACT_SILU, True)
    F.check(GU, gu, gu_bound, "GU")
    F.check(H, want, bound, "H")


@pytest.mark.parametrize("M", [20, 100, 300])
def test_cut_tiles_backward(cuda_lib, M):
    N, K, act = 8194, 384, w4.ACT_SILU
    pw = F.make_weight(N, K, 128, seed=32)
    W, dY = F.weight64(pw), _rand((M, N), 9)
    F.check(_dx(dY, pw), *F.dx64(dY.to(F.F8), W), "dx")
    dH, GU = _rand((M, N // 2), 3), _rand((M, N), 4, 2.0)
    d, e = F.grads64(dH, GU, act)
    dGU, dX = _backward(dH, GU, pw, act)
    F.check(dGU, d, e + F.U16 * (d.abs() + e) + F.TINY, "dGU")
    want, bound = F.dx64(d, W, r_d=2.0 ** -11, size=F.gated_size(dH, GU))
    F.check(dX, want, bound + (1 + F.U16) * (e @ W.abs()), "dX")


@pytest.mark.parametrize("M", [20, 90, 300])
def test_whole_tiles_of_tokens_and_rows_of_every_size(cuda_lib, M):
    """A wave of uncut tiles whose tokens, and whose rows, span FP32's range, beside tiles of ordinary ones."""
    n = 19500  # 77 tiles of rows, more than a wave of the 74 clusters for every tile width
    size = torch.ones(M, 1, dtype=F.F8, device="cuda")
    size[1::5], size[3::5] = 2.0 ** 100, 2.0 ** -100
    pw = F.make_weight(n, 128, 64, seed=21)
    pw.scales[300:800:3] = (pw.scales[300:800:3].double() * 2.0 ** -110).to(BF)
    W = F.weight64(pw)
    X = (F.tokens(M, 128, 4).double() * size).to(BF)
    bias, residual = _rand((n,), 5), _rand((M, n), 6)
    F.check(_linear(X, pw, bias, w4.ACT_RELU, residual), *F.linear64(X, W, bias, w4.ACT_RELU, residual), "linear")
    F.check(_linear(X, pw), *F.linear64(X, W, None, w4.ACT_NONE, None), "plain")
    small = X.clone()
    small[1::5] = F.tokens(M, 128, 4)[1::5]  # a product of two halves of 2^100 is past BF16
    want, bound, gu, gu_bound = F.gated64(small, W, w4.ACT_RELU)
    H, GU = _gated(small, pw, w4.ACT_RELU, True)
    F.check(GU, gu, gu_bound, "GU")
    F.check(H, want, bound, "H")
    pw = F.make_weight(130, 19456, 128, seed=22)
    dY = (_rand((M, 130), 8).double() * size).to(BF)
    F.check(_dx(dY, pw), *F.dx64(dY.to(F.F8), F.weight64(pw)), "dx")


@pytest.mark.parametrize("M,N", [(3, 18000), (3, 18004), (3, 18002), (40, 9000), (310, 512), (310, 516), (310, 514)])
def test_gradient_rows_of_every_alignment_shared_by_blocks(cuda_lib, M, N):
    """Long rows of few tokens (several blocks a token) and short rows of many, in 16-byte, 4-byte and single accesses;
    shut gates, extreme rows of weights and extreme gradients take the other ways through the preparation."""
    K, act = 256, w4.ACT_SILU
    pw = F.make_weight(N, K, 64, seed=41, far=True)
    for tiny in (False, True):  # 2^-112: powers of two that are no normal FP32 numbers
        if tiny:
            pw.scales[3::7] = (pw.scales[3::7].double() * 2.0 ** -112).to(BF)
        W = F.weight64(pw)
        for scale in (1.0, 2.0 ** 90):
            dY = (_rand((M, N), 1).double() * scale).to(BF)
            F.check(_dx(dY, pw), *F.dx64(dY.to(F.F8), W), f"dx {scale} {tiny}")
            dH, GU = dY[:, : N // 2].contiguous(), _rand((M, N), 2, 2.0)
            shut = M // 2
            GU[shut, : N // 2] = -abs(GU[shut, : N // 2]) - 30.0
            d, e = F.grads64(dH, GU, act)
            # a shut gate's gradient to a relative 2^-14 of e^x and its factors, as in the test above
            e[shut] = 2.0 ** -14 * (dH[shut].double().abs() * (1 + GU[shut, : N // 2].double().abs()) ** 3
                                    * torch.exp(GU[shut, : N // 2].double())).repeat(2) * torch.cat(
                [GU[shut, N // 2:].double().abs() + 1, torch.ones(N // 2, device="cuda", dtype=F.F8)])
            e = e + 2.0 ** -126
            dGU, dX = _backward(dH, GU, pw, act)
            F.check(dGU, d, e + F.U16 * (d.abs() + e) + F.TINY, f"dGU {scale} {tiny}")
            want, bound = F.dx64(d, W, r_d=2.0 ** -8, size=F.gated_size(dH, GU))
            F.check(dX, want, bound + (1 + F.U16) * (e @ W.abs()), f"dX {scale} {tiny}")
            dGU2, dX2 = _backward(dH, GU.clone(), pw, act, in_place=True)
            assert torch.equal(dGU2.view(torch.int16), dGU.view(torch.int16))
            assert torch.equal(dX2.view(torch.int16), dX.view(torch.int16))


@pytest.mark.parametrize("N,K,G", [(300, 18560, 32), (520, 9088, 32), (130, 16640, 64)])
def test_few_rows_of_many_groups(cuda_lib, N, K, G):
    """The weights' words of few rows: eight rows a block, rows of more groups than a block holds."""
    pw = F.make_weight(N, K, G, seed=43, far=True)
    W, X, dY = F.weight64(pw), F.tokens(20, K, 2), _rand((20, N), 3)
    F.check(_linear(X, pw), *F.linear64(X, W, None, w4.ACT_NONE, None), "forward")
    F.check(_dx(dY, pw), *F.dx64(dY.to(F.F8), W), "dx")


@pytest.mark.parametrize("act", F.ACTS)
def test_activations_of_every_bf16_value(cuda_lib, act):
    """One-hot tokens against a weight of one give the activation of each finite BF16 value, and a gated backward pass
    with dH = U = 1 its derivative.

    e^-|u| is a power of two whose exponent, at most 142 in size before the result vanishes, carries the relative errors
    of |u| log2 e or x^2 (up to four roundings of 2^-24) and its own rounding of at most 2^-18: in all below 2^-15 of the
    value."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(BF)
    x = x[x.double().isfinite()].reshape(-1, 1)
    M, K = x.shape[0], 128
    pw = w4.PackedWeight(2, K, device=x.device, group=128)
    pw.scales.fill_(1.0)
    pw.zeros.fill_(8)
    pw.qweight.fill_(-2004318072)  # codes 8
    pw.qweight[:, 0] += 1
    X = torch.zeros((M, K), dtype=BF, device="cuda")
    X[:, :1] = x
    want = F.act64(x.double(), act).expand(M, 2)
    e = 2.0 ** -15 * want.abs()
    F.check(_linear(X, pw, act=act), want, e + F.U16 * (want.abs() + e) + F.TINY, "activation")
    one = torch.ones_like(x)
    d, e = F.grads64(one, torch.cat([x, one], 1), act)
    # 1 / (1 + e^-x) and e^x of x down to -88: |x| 2^-24 log2 e and a few roundings more, as above; x act'(x) terms cancel
    # to 2^-17 absolutely (grads64)
    e = e + 2.0 ** -15 * d.abs()
    dGU = F.nans(M, 2)
    ws = F.workspace(w4.dx_workspace_bytes(M, 2, K, 128))
    w4.gated_backward(one, torch.cat([x, one], 1).contiguous(), pw.qweight, pw.scales, pw.zeros, dGU, F.nans(M, K), ws, act=act)
    _done()
    F.check(dGU, d, e + F.U16 * (d.abs() + e) + F.TINY, "gradients")


def test_tiny_weights_both_ways(cuda_lib):
    N, K = 260, 1024
    pw = F.make_weight(N, K, 128, seed=14)
    pw.scales[1::3] = (pw.scales[1::3].double() * 2.0 ** -110).to(BF)
    W = F.weight64(pw)
    for M in (1, 6, 40, 150):
        X = F.tokens(M, K, 2)
        F.check(_linear(X, pw), *F.linear64(X, W, None, w4.ACT_NONE, None), f"forward {M}")
        dY = _rand((M, N), 3)
        dY[:, 0::3] = 0
        dY[:, 2::3] = 0  # only the tiny rows count
        F.check(_dx(dY, pw), *F.dx64(dY.to(F.F8), W), f"dx {M}")


def test_refusals_leave_the_outputs(cuda_lib):
    N, K, M = 130, 1024, 20
    pw = F.make_weight(N, K, 128, seed=3)
    q = (pw.qweight, pw.scales, pw.zeros)
    X, Y, dX = F.tokens(M, K, 1), F.nans(M, N), F.nans(M, K)
    H, GU = F.nans(M, N // 2), F.nans(M, N)
    ws = F.workspace(w4.fused_workspace_bytes(M, N, K))
    short = ws[: 256 * 1024]

    def status(f):
        with pytest.raises(w4.W4A16Error) as e:
            f()
        return e.value.status

    assert status(lambda: w4.linear_fused(X, *q, Y, short)) == w4.ERR_WORKSPACE
    assert status(lambda: w4.gated(X, *q, H, short, GU=GU)) == w4.ERR_WORKSPACE
    assert status(lambda: w4.linear_dx(Y, *q, dX, short)) == w4.ERR_WORKSPACE
    assert status(lambda: w4.gated_backward(H, Y, *q, GU, dX, short)) == w4.ERR_WORKSPACE
    assert status(lambda: w4.linear_fused(X, *q, Y, ws, act=9)) == w4.ERR_ARG
    for bad, err in [(lambda: w4.linear_fused(X, *q, Y[:-1], ws), ValueError),
                     (lambda: w4.linear_fused(X, *q, Y.float(), ws), TypeError),
                     (lambda: w4.linear_fused(X.t().contiguous().t(), *q, Y, ws), ValueError),
                     (lambda: w4.linear_fused(X, *q, Y, None), TypeError),
                     (lambda: w4.linear_fused(X, *q, Y, ws.cpu()), ValueError),
                     (lambda: w4.linear_fused(X, *q, Y, ws, bias=Y[0, :-1]), ValueError),
                     (lambda: w4.linear_fused(X, *q, Y, ws, residual=X), ValueError),
                     (lambda: w4.linear_fused(X, *q, Y, ws, group=64), ValueError),
                     (lambda: w4.linear_fused(X, *q, Y, ws, group=96), ValueError),
                     (lambda: w4.gated(X, *q, Y, ws), ValueError),
                     (lambda: w4.linear_dx(X, *q, dX, ws), ValueError)]:
        with pytest.raises(err):
            bad()
    _done()
    for t in (Y, dX, H, GU):
        assert bool(torch.isnan(t).all())


def test_other_streams_and_raw_handles(cuda_lib):
    N, K, M = 258, 1024, 20
    pw = F.make_weight(N, K, 128, seed=3)
    X, ws = F.tokens(M, K, 1), F.workspace(w4.fused_workspace_bytes(M, N, K))
    ref = _linear(X, pw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [F.nans(M, N) for _ in range(3)]
    w4.linear_fused(X, pw.qweight, pw.scales, pw.zeros, outs[0], ws, stream=s)
    w4.linear_fused(X, pw.qweight, pw.scales, pw.zeros, outs[1], ws, stream=s.cuda_stream)
    with torch.cuda.stream(s):
        w4.linear_fused(X, pw.qweight, pw.scales, pw.zeros, outs[2], ws)
    _done()
    assert all(torch.equal(ref, o) for o in outs)


def test_rows_behind_the_last_token_stay(cuda_lib):
    N, K = 258, 1024
    pw = F.make_weight(N, K, 128, seed=2)
    for M in (1, 5, 20, 70, 200):
        big, hbig, dbig = F.nans(M + 3, N), F.nans(M + 3, N // 2), F.nans(M + 3, K)
        for t in (big, hbig, dbig):
            t.fill_(7.0)
        X, ws = F.tokens(M, K, 1), F.workspace(w4.fused_workspace_bytes(M, N, K))
        w4.linear_fused(X, pw.qweight, pw.scales, pw.zeros, big[:M], ws)
        w4.gated(X, pw.qweight, pw.scales, pw.zeros, hbig[:M], ws)
        w4.linear_dx(_rand((M, N), 3), pw.qweight, pw.scales, pw.zeros, dbig[:M], F.workspace(w4.dx_workspace_bytes(M, N, K)))
        _done()
        for t in (big, hbig, dbig):
            assert bool((t[M:] == 7).all()), M


def test_one_workspace_serves_mixed_calls_and_repeats_bits(cuda_lib):
    """Calls of every path in turn on one workspace: repeated calls give the same bits, the library's other layers
    among them, and the counters end at zero."""
    N, K = 514, 2048
    pw = F.make_weight(N, K, 128, seed=21)
    Ms = [1, 7, 30, 100, 300, 1, 7, 30, 100, 300]
    size = max(max(w4.fused_workspace_bytes(m, N, K), w4.dx_workspace_bytes(m, N, K), w4.workspace_bytes(m, N, K)) for m in Ms)
    ws = F.workspace(size)
    q = (pw.qweight, pw.scales, pw.zeros)
    seen = {}
    for m in Ms:
        X, dY = F.tokens(m, K, m), _rand((m, N), m)
        Y, H, GU, dX, L = F.nans(m, N), F.nans(m, N // 2), F.nans(m, N), F.nans(m, K), F.nans(m, N)
        w4.linear_fused(X, *q, Y, ws, act=w4.ACT_GELU)
        w4.gated(X, *q, H, ws, GU=GU)
        w4.linear(X, *q, L, ws)
        w4.linear_dx(dY, *q, dX, ws)
        dGU, dX2 = F.nans(m, N), F.nans(m, K)
        w4.gated_backward(H, GU, *q, dGU, dX2, ws)
        _done()
        outs = [Y, H, GU, dX, dGU, dX2, L]
        if m in seen:
            assert all(torch.equal(a, b) for a, b in zip(outs, seen[m]))
        seen[m] = outs
    assert not ws[: 256 * 1024].any()


def _block(X, gu, down, res, ws, bufs):
    """A feed-forward block and its backward pass as a training step runs them: H = silu(G) U, Y = H Wd^T + res,
    then dH = dY Wd, dX."""
    H, GU, Y, dH, dGU, dX = bufs
    w4.gated(X, *gu, H, ws, GU=GU)
    w4.linear_fused(H, *down, Y, ws, residual=res)
    w4.linear_dx(Y, *down, dH, ws)  # the loss is |Y|^2 / 2
    w4.gated_backward(dH, GU, *gu, dGU, dX, ws)


@pytest.mark.parametrize("M", [1, 12, 150])
def test_feed_forward_block_together_eager_and_captured(cuda_lib, M):
    K, I = 1024, 1152
    pg, pd = F.make_weight(2 * I, K, 128, seed=31), F.make_weight(K, I, 128, seed=32)
    gu, down = (pg.qweight, pg.scales, pg.zeros), (pd.qweight, pd.scales, pd.zeros)
    X, res = F.tokens(M, K, 4, 0.05), _rand((M, K), 5)
    size = max(w4.fused_workspace_bytes(M, 2 * I, K), w4.fused_workspace_bytes(M, K, I),
               w4.dx_workspace_bytes(M, K, I), w4.dx_workspace_bytes(M, 2 * I, K))
    ws = F.workspace(size)
    new = lambda: (F.nans(M, I), F.nans(M, 2 * I), F.nans(M, K), F.nans(M, I), F.nans(M, 2 * I), F.nans(M, K))  # noqa: E731
    eager, graphed = new(), new()
    _block(X, gu, down, res, ws, eager)
    _done()
    # each step against its definition, from the tensors the step before really handed on
    Wg, Wd = F.weight64(pg), F.weight64(pd)
    H, GU, Y, dH, dGU, dX = eager
    h, hb, s, sb = F.gated64(X, Wg, w4.ACT_SILU)
    F.check(H, h, hb, "H")
    F.check(GU, s, sb, "GU")
    F.check(Y, *F.linear64(H, Wd, None, w4.ACT_NONE, res), "Y")
    F.check(dH, *F.dx64(Y.to(F.F8), Wd), "dH")
    d, e = F.grads64(dH, GU, w4.ACT_SILU)
    want, bound = F.dx64(d, Wg, r_d=2.0 ** -11, size=F.gated_size(dH, GU))
    F.check(dX, want, bound + (1 + F.U16) * (e @ Wg.abs()), "dX")

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            _block(X, gu, down, res, ws, graphed)
    for _ in range(3):
        graph.replay()
    _done()
    assert all(torch.equal(a, b) for a, b in zip(eager, graphed))


def test_two_streams_with_a_workspace_each(cuda_lib):
    N, K, M = 1026, 1024, 40
    pw = F.make_weight(N, K, 128, seed=41)
    q = (pw.qweight, pw.scales, pw.zeros)
    X = [F.tokens(M, K, i) for i in range(2)]
    ref = []
    for i in range(2):
        H, ws = F.nans(M, N // 2), F.workspace(w4.fused_workspace_bytes(M, N, K))
        w4.gated(X[i], *q, H, ws)
        _done()
        ref.append(H)
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [F.workspace(w4.fused_workspace_bytes(M, N, K)) for _ in range(2)]
    outs = [F.nans(M, N // 2) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            w4.gated(X[i], *q, outs[i], wss[i], stream=streams[i])
    _done()
    assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])


def test_gradient_against_differences(cuda_lib):
    """dX of a gated block against central differences of the definition in 64 bits, along random directions."""
    M, N, K = 3, 258, 256
    pw = F.make_weight(N, K, 64, seed=51)
    W = F.weight64(pw)
    X = F.tokens(M, K, 6, 0.3)
    dH = _rand((M, N // 2), 7)
    for act in (w4.ACT_SILU, w4.ACT_GELU, w4.ACT_GELU_TANH):
        _, GU = _gated(X, pw, act, True)
        _, dX = _backward(dH, GU, pw, act)

        def loss(x):
            s = x @ W.T
            return (dH.to(F.F8) * F.act64(s[:, : N // 2], act) * s[:, N // 2:]).sum()

        gen = torch.Generator(device="cuda")
        gen.manual_seed(act)
        for _ in range(4):
            v = torch.randn((M, K), device="cuda", generator=gen, dtype=F.F8)
            h = 1e-5
            diff = float((loss(X.to(F.F8) + h * v) - loss(X.to(F.F8) - h * v)) / (2 * h))
            got = float((dX.to(F.F8) * v).sum())
            # GU and dX are BF16 (2^-8 each, and act' changes with G by at most 0.8 |dG|): errors of independent sign
            # over M K terms, bounded here by their sum of magnitudes times 2^-8 and G's own part of the product
            s = X.to(F.F8) @ W.T
            g, u = s[:, : N // 2], s[:, N // 2:]
            d = torch.cat([(dH.to(F.F8) * u).abs() * (1.13 + 0.8 * g.abs()), dH.to(F.F8).abs() * (F.act64(g, act).abs() + 1.13 * g.abs())], 1)
            bound = 2.0 ** -8 * float((dX.to(F.F8) * v).abs().sum()) + 2.0 ** -8 * float((d * (v.abs() @ W.abs().T)).sum())
            assert abs(got - diff) <= bound, (act, got, diff, bound)
