"""The fused operators at the edges of their inputs: rows and groups of the weight that hold nothing but zeros, sums that
are NaN or past FP32's range."""
import math

import pytest
import torch

import weight_only_int4_linear_b200 as w4
from tests import _fused as F
from tests.test_gpu_fused import BF, _backward, _dx, _gated, _linear, _rand

pytestmark = pytest.mark.gpu


# A zero group or row is stored with a scale that says nothing about its values (the quantiser's is 1): it must not decide
# how the others are scaled.  (dx64 takes a row's size from its largest value; the groups of zeros here lie more than 2^4
# above their row's others and are left out of it, as rows of zeros always are.)
def _sparse_weight(N, K, G, size, seed, symmetric=False):
    """Weights of one size with rows of zeros as the quantiser stores them, rows whose scales are zero, and rows with one
    or several zero groups, the first and the last among them."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    W = size * torch.randn((N, K), device="cuda", generator=gen)
    W[1::5] = 0.0
    W[3::5, :G] = 0.0
    W[4::5, K - G:] = 0.0
    W[4::10, G : 3 * G] = 0.0
    pw = F.pack(W, G, symmetric)
    pw.scales[2::15] = 0.0
    for rows, groups, scale in [(slice(7, None, 35), slice(None), 2.0 ** 20), (slice(9, None, 35), slice(0, 1), 2.0 ** 70)]:
        pw.zeros[rows, groups], pw.scales[rows, groups] = 8, scale  # pruned after packing: codes 8, any scale
        pw.qweight.view(N, K // G, G // 8)[rows, groups] = -2004318072
    return pw


SPARSE = [(3, 258, 256, 64), (40, 520, 1024, 128), (100, 130, 384, 32), (310, 514, 512, 64), (20, 70, 18560, 32)]


@pytest.mark.parametrize("M,N,K,G", SPARSE)
@pytest.mark.parametrize("size", [1e-2, 1e-6, 1e-10])
@pytest.mark.parametrize("symmetric", [False, True])
def test_gradients_beside_rows_and_groups_of_zeros(cuda_lib, M, N, K, G, size, symmetric):
    pw = _sparse_weight(N, K, G, size, N + K, symmetric)
    W = F.weight64(pw)
    dead = (W == 0).all(1)
    assert int(dead.sum()) >= N // 5
    dY = _rand((M, N), 1, 1e-3)
    dY[:, dead] *= 2.0 ** 12  # the largest gradients belong to rows that add nothing
    F.check(_dx(dY, pw), *F.dx64(dY.to(F.F8), W), "dx")
    act = w4.ACT_SILU
    dH, GU = dY[:, : N // 2].contiguous(), _rand((M, N), 2, 2.0)
    d, e = F.grads64(dH, GU, act)
    dGU, dX = _backward(dH, GU, pw, act)
    F.check(dGU, d, e + F.U16 * (d.abs() + e) + F.TINY, "dGU")
    want, bound = F.dx64(d, W, r_d=2.0 ** -11, size=F.gated_size(dH, GU))
    F.check(dX, want, bound + (1 + F.U16) * (e @ W.abs()), "dX")


@pytest.mark.parametrize("M,N,K,G", SPARSE + [(1, 258, 1024, 128), (7, 258, 1024, 128), (1, 258, 512, 32)])
@pytest.mark.parametrize("size", [1e-2, 1e-9, 1e-11])
@pytest.mark.parametrize("symmetric", [False, True])
def test_forward_beside_groups_of_zeros(cuda_lib, M, N, K, G, size, symmetric):
    pw = _sparse_weight(N, K, G, size, N + K, symmetric)
    W, X = F.weight64(pw), F.tokens(M, K, 3)
    F.check(_linear(X, pw), *F.linear64(X, W, None, w4.ACT_NONE, None), "linear")
    want, bound, gu, gu_bound = F.gated64(X, W, w4.ACT_NONE)
    H, GU = _gated(X, pw, w4.ACT_NONE, True)
    F.check(GU, gu, gu_bound, "GU")
    F.check(H, want, bound, "H")


@pytest.mark.parametrize("M", [5, 70])
def test_a_weight_of_zeros_and_one_live_row(cuda_lib, M):
    N, K = 258, 1024
    zero = F.pack(torch.zeros((N, K), device="cuda"), 128)
    dY = _rand((M, N), 1)
    assert not _dx(dY, zero).any() and not _linear(F.tokens(M, K, 2), zero).any()
    W = torch.zeros((N, K), device="cuda")
    W[N - 1, K - 1] = 1e-8  # the last value of the last group
    one = F.pack(W, 128)
    F.check(_dx(dY, one), *F.dx64(dY.to(F.F8), F.weight64(one)), "one value")
    far = F.pack(W + 0.0, 128)
    far.scales[0], far.zeros[0] = 2.0 ** -60, 5000  # beside a row whose zero points are far beyond the codes
    F.check(_dx(dY, far), *F.dx64(dY.to(F.F8), F.weight64(far)), "far zero points")


@pytest.mark.parametrize("act", F.ACTS)
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_not_a_number_reaches_the_output(cuda_lib, M, act):
    """A sum that is NaN stays NaN through every activation, and its neighbours keep their values."""
    N, K = 300, 1024
    pw = F.make_weight(N, K, 128, seed=act)
    X, bias = F.tokens(M, K, act), _rand(N, 5)
    plain = _linear(X, pw, bias, act)
    bias[::7] = math.nan
    Y = _linear(X, pw, bias, act)
    assert torch.equal(Y.isnan(), bias.isnan().expand(M, N))
    assert torch.equal(Y[:, ~bias.isnan()], plain[:, ~bias.isnan()])


@pytest.mark.parametrize("act", F.ACTS)
def test_a_token_that_is_not_a_number_through_the_gate(cuda_lib, act):
    M, N, K = 40, 258, 640  # tokens of the GEMM (the integer GEMVs take finite values only)
    pw = F.make_weight(N, K, 128, seed=act)
    X = F.tokens(M, K, act)
    X[3, 7] = math.nan
    H, GU = _gated(X, pw, act, True)
    assert bool(H[3].isnan().all()) and bool(GU[3].isnan().all())
    X[3, 7] = 0.0
    keep = torch.arange(M, device="cuda") != 3
    again, _ = _gated(X, pw, act, True)
    assert torch.equal(H[keep], again[keep])


@pytest.mark.parametrize("act", F.ACTS)
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_infinite_sums_give_the_limit(cuda_lib, M, act):
    N, K = 300, 1024
    pw = F.make_weight(N, K, 128, seed=act)
    X, bias = F.tokens(M, K, act), _rand(N, 5)
    plain = _linear(X, pw, bias, act)
    bias[100], bias[299] = -math.inf, math.inf
    Y = _linear(X, pw, bias, act)
    assert bool((Y[:, 100] == (-math.inf if act == w4.ACT_NONE else 0.0)).all()), Y[:, 100]
    assert bool((Y[:, 299] == math.inf).all())
    keep = bias.isfinite()
    assert torch.equal(Y[:, keep], plain[:, keep])


@pytest.mark.parametrize("act", F.ACTS[1:])
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_gate_sums_below_the_range(cuda_lib, M, act):
    """Finite inputs whose gate sum is below FP32's range: the gate is shut, H is 0."""
    N, K = 130, 1024
    I = N // 2
    W = 0.02 * torch.rand((N, K), device="cuda") + 0.01
    W[:I] *= 2.0 ** 20
    pw = F.pack(W, 128)
    X = torch.full((M, K), -(2.0 ** 110), dtype=BF, device="cuda")
    H, GU = _gated(X, pw, act, True)
    assert bool((GU[:, :I] == -math.inf).all()) and bool(GU[:, I:].isfinite().all())
    assert bool((H == 0).all()), H


@pytest.mark.parametrize("M,N", [(3, 258), (70, 514), (310, 512), (3, 18000)])
@pytest.mark.parametrize("act", F.ACTS)
def test_gated_gradients_whose_first_product_leaves_the_range(cuda_lib, M, N, act):
    """dH U past FP32's largest number under a gate that brings the gradient back or shuts it, also where the weight's row
    is zero, in the first token; the last token's ends of the range meet a gate of ordinary size."""
    K, I = 256, N // 2
    pw = F.make_weight(N, K, 64, seed=17)
    pw.scales[3] = 0.0
    pw.scales[I + 2] = 0.0
    W = F.weight64(pw)
    dH, GU = _rand((M, I), 1), _rand((M, N), 2, 2.0)
    gates = {w4.ACT_SILU: [-30000.0, -3.0, -60.0, -70.0], w4.ACT_GELU: [-30000.0, -3.0, -10.5, -11.0],
             w4.ACT_GELU_TANH: [-30000.0, -3.0, -8.7, -9.0]}.get(act, [-1.0, -3.0, -8.0, -9.0])
    GU[0, :4] = torch.tensor(gates, device="cuda").to(BF)
    dH[0, :4] = torch.tensor([2.0 ** 60, 2.0 ** 60, 2.0 ** 100, 2.0 ** 100], device="cuda").to(BF)
    GU[0, I : I + 4] = torch.tensor([2.0 ** 100, -(2.0 ** 60), 2.0 ** 100, -(2.0 ** 100)], device="cuda").to(BF)
    if act == w4.ACT_NONE:
        GU[0, I : I + 4] = 2.0 ** 20
    dH[M - 1, I - 1], GU[M - 1, I - 1] = 3e36 if act == w4.ACT_NONE else 3e38, -1.0
    GU[M - 1, N - 1] = 3.3e38 if act == w4.ACT_RELU else 0.5
    d, e = F.grads64(dH, GU, act)
    assert bool((d.abs() < 3e38).all())
    # FP32 holds a shut gate's gradients to a relative 2^-11: differences of two terms of e^x, x off by |x| 2^-22 at most
    for part in (slice(0, 4), slice(I, I + 4)):
        e[0, part] = 2.0 ** -11 * d[0, part].abs()
    if act == w4.ACT_RELU:
        e[M - 1] = 0.0  # the factors are 0 and 1
    dGU, dX = _backward(dH, GU, pw, act)
    F.check(dGU, d, e + F.U16 * (d.abs() + e) + F.TINY, "dGU")
    size = F.gated_size(dH, GU)
    size[[0, M - 1]] = d[[0, M - 1]].abs()  # at the ends of the range a token is scaled by its gradients themselves
    want, bound = F.dx64(d, W, r_d=2.0 ** -11, size=size)
    F.check(dX, want, bound + (1 + F.U16) * (e @ W.abs()), "dX")
    dGU2, dX2 = _backward(dH, GU.clone(), pw, act, in_place=True)
    assert torch.equal(dGU2, dGU) and torch.equal(dX2, dX)


@pytest.mark.parametrize("M,N,K", [(3, 258, 256), (40, 8194, 384), (300, 130, 1024), (20, 130, 19456)])
@pytest.mark.parametrize("up", [False, True])
def test_channel_scales_bring_gradients_back_into_the_range(cuda_lib, M, N, K, up):
    """Sums past FP32's range, or below its smallest number, that the channel's scale brings back."""
    pw = F.make_weight(N, K, 128, seed=19)
    pw.scales.copy_((pw.scales.double() * 2.0 ** (-30 if up else 10)).to(BF))
    W = F.weight64(pw)
    dY = (_rand((M, N), 1).double() * 2.0 ** (-125 if up else 120)).to(BF)
    inv = torch.exp2(torch.linspace(-2, 2, K, device="cuda")) * 2.0 ** (60 if up else -40)
    want, bound = F.dx64(dY.to(F.F8), W, inv)
    assert 1e-30 < float(want.abs().max()) < 1e38
    F.check(_dx(dY, pw, inv), want, bound)


@pytest.mark.parametrize("M,N,K,G", [(1, 258, 512, 64), (6, 1030, 1024, 128), (50, 258, 640, 32), (100, 18002, 256, 128),
                                     (300, 514, 384, 64)])
def test_gated_backward_with_channel_scales(cuda_lib, M, N, K, G):
    pw = F.make_weight(N, K, G, seed=K + M, far=True)
    W, act = F.weight64(pw), F.ACTS[1 + M % 4]
    inv = torch.exp2(torch.linspace(-3, 3, K, device="cuda")) * 1.1
    dH, GU = _rand((M, N // 2), M, 1e-2), _rand((M, N), M + 50, 3.0)
    d, e = F.grads64(dH, GU, act)
    dGU, dX = _backward(dH, GU, pw, act, inv_s=inv)
    F.check(dGU, d, e + F.U16 * (d.abs() + e) + F.TINY, "dGU")
    want, bound = F.dx64(d, W, inv, r_d=2.0 ** -11, size=F.gated_size(dH, GU))
    F.check(dX, want, bound + (1 + F.U16) * (e @ W.abs()) * inv.double(), "dX")
