"""How far the fused operators' outputs are from 64 bits as a whole: no further than BF16 outputs have to be.

Bounds per element add the magnitudes of all errors and leave room that a coarser operand would fit into; norms do not."""
import pytest
import torch

import weight_only_int4_linear_b200 as w4
from tests import _fused as F
from tests.test_gpu_fused import BF, _backward, _dx, _gated, _linear, _rand

pytestmark = pytest.mark.gpu


def _excess(got, want):
    """Distance from `want` over that of `want` rounded to BF16."""
    own = (want.float().to(BF).double() - want).norm()
    return float((got.double() - want).norm() / own)


# Rounding to BF16 is off by 1.65e-3 of the outputs (root mean square; 2^-8 / sqrt 3 of a mantissa of 1, half of it of one
# near 2).  FP16 operands are each off by at most 2^-11 / sqrt 3 = 2.8e-4 of a term, independently, which is the sum's
# error relative to it; the gated product's two sums and the activation's slope of 1.13 make it 4.6e-4 at most, an FP16
# gradient 4e-4 with its weight.  Squared and added, 1.04 times the rounding alone; the integer GEMVs' fixed-point step,
# 2^-18 of a group's largest activation, is less.  Weights rounded to BF16 add 1.4e-3 (1.31 times), and are told apart.
MOST = 1.1


@pytest.mark.parametrize("M,N,K,G", [(1, 51200, 1024, 128), (8, 8192, 1024, 128), (48, 8192, 4096, 64), (100, 4096, 2048, 32),
                                     (300, 4096, 4096, 128)])
def test_errors_are_those_of_the_outputs_own_rounding(cuda_lib, M, N, K, G):
    pw = F.make_weight(N, K, G, seed=K)
    W, X, act = F.weight64(pw), F.tokens(M, K, 5), w4.ACT_SILU
    coarse = W.to(BF).double()

    want = X.double() @ W.T
    assert _excess(_linear(X, pw), want) <= MOST
    assert _excess((X.double() @ coarse.T).float().to(BF), want) > MOST
    H, GU = _gated(X, pw, act, True)
    assert _excess(GU, want) <= MOST
    assert _excess(H, F.act64(want[:, : N // 2], act) * want[:, N // 2 :]) <= MOST

    dY = _rand((M, N), 7)
    want = dY.double() @ W
    assert _excess(_dx(dY, pw), want) <= MOST
    assert _excess((dY.double() @ coarse).float().to(BF), want) > MOST
    dH, GU = _rand((M, N // 2), 8), _rand((M, N), 9, 2.0)
    d, _ = F.grads64(dH, GU, act)
    dGU, dX = _backward(dH, GU, pw, act)
    assert _excess(dGU, d) <= MOST
    assert _excess(dX, d @ W) <= MOST
