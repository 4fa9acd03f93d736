"""Host-side refusals of the fused operators: status codes before any launch, and the binding's own checks (no GPU)."""
import ctypes

import pytest
import torch

import weight_only_int4_linear_b200 as w4
from weight_only_int4_linear_b200 import build as w4build

P = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
U = ctypes.c_void_p(0x10008)  # misaligned
WS = 1 << 40


@pytest.fixture(scope="module")
def lib():
    w4build.build()
    return w4.load()


def linear(lib, X=P, inv=None, M=1, K=1024, G=128, q=P, s=P, z=P, N=16, bias=None, act=0, res=None, Y=P, ws=P, n=WS):
    return lib.w4a16_linear_fused(X, inv, M, K, G, q, s, z, N, bias, act, res, Y, ws, n, None)


def gated(lib, X=P, inv=None, M=1, K=1024, G=128, q=P, s=P, z=P, N=16, act=2, H=P, GU=None, ws=P, n=WS):
    return lib.w4a16_gated(X, inv, M, K, G, q, s, z, N, act, H, GU, ws, n, None)


def dx(lib, dY=P, M=1, N=16, G=128, q=P, s=P, z=P, K=1024, inv=None, dX=P, ws=P, n=WS):
    return lib.w4a16_linear_dx(dY, M, N, G, q, s, z, K, inv, dX, ws, n, None)


def backward(lib, dH=P, GU=P, M=1, N=16, act=2, G=128, q=P, s=P, z=P, K=1024, inv=None, dGU=P, dX=P, ws=P, n=WS):
    return lib.w4a16_gated_backward(dH, GU, M, N, act, G, q, s, z, K, inv, dGU, dX, ws, n, None)


@pytest.mark.parametrize("call,names", [(linear, ["X", "q", "s", "z", "Y"]), (gated, ["X", "q", "s", "z", "H"]),
                                        (dx, ["dY", "q", "s", "z", "dX"]),
                                        (backward, ["dH", "GU", "q", "s", "z", "dGU", "dX"])])
def test_null_and_misaligned_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == w4.ERR_ARG, n
        assert call(lib, **{n: U}) == w4.ERR_ALIGN, n
    assert call(lib, inv=U) == w4.ERR_ALIGN
    if call is linear:
        assert call(lib, bias=U) == w4.ERR_ALIGN and call(lib, res=U) == w4.ERR_ALIGN
    if call is gated:
        assert call(lib, GU=U) == w4.ERR_ALIGN


@pytest.mark.parametrize("call", [linear, gated, dx, backward])
def test_shapes_groups_and_activations(lib, call):
    for bad in (dict(M=0), dict(M=-3), dict(N=0), dict(K=0), dict(G=48), dict(G=0), dict(G=256)):
        assert call(lib, **bad) == w4.ERR_ARG, bad
    for bad in (dict(K=100), dict(K=1088), dict(M=1 << 31), dict(N=1 << 31)):
        assert call(lib, **bad) == w4.ERR_SHAPE, bad
    if call is not dx:
        assert call(lib, act=-1) == w4.ERR_ARG and call(lib, act=5) == w4.ERR_ARG
    if call in (gated, backward):
        assert call(lib, N=17) == w4.ERR_SHAPE
    if not torch.cuda.is_available():
        assert call(lib) == w4.ERR_DEVICE  # well-formed arguments reach the device check


def test_workspace_bytes(lib):
    for f in (lib.w4a16_fused_workspace_bytes, lib.w4a16_dx_workspace_bytes):
        for bad in [(0, 16, 1024, 128), (1, 0, 1024, 128), (1, 16, 100, 128), (1, 16, 1024, 48), (1, 1 << 31, 1024, 128)]:
            assert f(*bad) == 0, bad
        for M in (1, 2, 16, 17, 100, 4096):
            for G in (32, 64, 128):
                b = f(M, 1001, 1152, G)
                assert b > 256 * 1024 and b % 256 == 0


def test_binding_refuses_before_the_library(lib):
    X = torch.zeros((1, 128), dtype=torch.bfloat16)
    q, s, z = torch.zeros((16, 16), dtype=torch.int32), torch.zeros((16, 1), dtype=torch.bfloat16), torch.zeros((16, 1), dtype=torch.int32)
    Y, ws = torch.zeros((1, 16), dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        w4.linear_fused(X, q, s, z, Y, ws)
    with pytest.raises(ValueError, match="two dimensions"):
        w4.linear_fused(X[0], q, s, z, Y, ws)
    with pytest.raises(TypeError, match="torch.Tensor"):
        w4.gated([1.0], q, s, z, Y, ws)
    with pytest.raises(ValueError, match="even number"):
        w4.gated(X, q[:15], s[:15], z[:15], Y, ws)
    with pytest.raises(ValueError, match="two rows"):
        w4.gated_backward(Y, Y, q, s, z, Y, X, ws)
