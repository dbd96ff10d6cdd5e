"""Fused MXFP4 entry points without a GPU: the argument checks of the C ABI (every refusal
comes before a device is touched), workspace sizes, and the Python layer's refusals."""
import ctypes

import pytest
import torch

import dequant_gemv_nf4_amd as nf4

EINVAL, EALIGN, ERANGE = -1, -2, -3
P = ctypes.c_void_p(0x100000)      # fake, 256-byte aligned; never dereferenced on these paths
NULL = ctypes.c_void_p(0)
BIG = 1 << 50
GELU, SWIGLU = 3, 5


def off(n):
    return ctypes.c_void_p(0x100000 + n)


@pytest.fixture(scope="module")
def lib():
    return nf4._lib._load()


def linear(lib, N=64, K=64, M=3, act=0, codes=P, scales=P, X=P, bias=NULL, bias_dtype=0, residual=NULL, Y=P,
           out=0, Z=NULL):
    return lib.nf4_mx_linear(codes, scales, N, K, X, M, bias, bias_dtype, act, residual, Y, out, Z, NULL)


def linear_grad(lib, N=64, K=64, M=3, act=GELU, codes=P, scales=P, dY=P, Z=P, dZ=P, dbias=NULL, dX=P, out=0,
                ws=P, nbytes=BIG):
    return lib.nf4_mx_linear_grad(codes, scales, N, K, dY, Z, act, M, dZ, dbias, dX, out, ws, nbytes, NULL)


def loss(lib, N=64, K=64, M=3, codes=P, scales=P, X=P, targets=P, loss=P, lse=P, dloss=NULL, dX=NULL, out=0,
         ws=P, nbytes=BIG, status=NULL):
    return lib.nf4_mx_cross_entropy(codes, scales, N, K, X, targets, M, loss, lse, dloss, dX, out, ws, nbytes,
                                    status, NULL)


def moe(lib, E=4, H=64, I=64, T=3, topk=2, act=SWIGLU, c1=P, s1=P, c2=P, s2=P, X=P, experts=P, weights=P,
        residual=NULL, out=P, out_dtype=0, ws=P, nbytes=BIG):
    return lib.nf4_moe_mlp(c1, s1, c2, s2, E, H, I, X, experts, weights, T, topk, act, residual, out, out_dtype,
                           ws, nbytes, NULL)


ALL = (linear, linear_grad, loss)
SHAPES = [(0, 32, EINVAL), (-8, 32, EINVAL), (8, 0, EINVAL), (8, 48, EINVAL), (8, -32, EINVAL),
          (8, 32768 + 32, ERANGE), (1 << 31, 32, ERANGE), (1 << 17, 32768, ERANGE), (1 << 62, 1 << 40, ERANGE)]


@pytest.mark.parametrize("N,K,expect", SHAPES)
def test_matrix_shapes(lib, N, K, expect):
    for call in ALL:
        assert call(lib, N=N, K=K) == expect, call.__name__
    assert lib.nf4_mx_linear_grad_workspace_bytes(N, K, 4) == -1
    assert lib.nf4_mx_cross_entropy_workspace_bytes(N, K, 4, 1) == -1
    # the first matrix is [2 I][H], the second [H][I]
    assert moe(lib, H=K, I=N) in (EINVAL, ERANGE)
    assert lib.nf4_moe_mlp_workspace_bytes(4, K, N, SWIGLU, 3, 2) == -1


@pytest.mark.parametrize("M", [0, -1, 1 << 26, 1 << 60])
def test_rows(lib, M):
    for call in ALL:
        assert call(lib, M=M) == ERANGE, call.__name__
    assert lib.nf4_mx_linear_grad_workspace_bytes(64, 64, M) == -1
    assert lib.nf4_mx_cross_entropy_workspace_bytes(64, 64, M, 0) == -1


def test_limits(lib):
    assert linear_grad(lib, M=(1 << 21) + 1) == ERANGE
    assert linear_grad(lib, N=(1 << 23) + 8, K=32) == ERANGE
    assert linear_grad(lib, N=60) == EINVAL
    assert loss(lib, N=(1 << 23) + 1, K=32) == ERANGE
    for act in (5, 6):
        assert linear(lib, N=63, act=act) == EINVAL
    for e, expect in ((0, EINVAL), (-1, EINVAL), (513, ERANGE)):
        assert moe(lib, E=e) == expect
    for k, expect in ((0, EINVAL), (-1, EINVAL), (513, ERANGE), (1 << 60, ERANGE)):
        assert moe(lib, topk=k) == expect
    for t, expect in ((-1, EINVAL), (65, ERANGE), (1 << 60, ERANGE)):
        assert moe(lib, T=t) == expect
    assert moe(lib, H=48) == EINVAL and moe(lib, I=48) == EINVAL
    assert moe(lib, H=32, I=32768 + 32) == ERANGE and moe(lib, H=32768 + 32, I=32) == ERANGE
    assert moe(lib, H=32768, I=32768 * 8) == ERANGE


@pytest.mark.parametrize("value", [-1, 7, 100])
def test_unknown_acts_and_dtypes(lib, value):
    assert linear(lib, act=value) == linear_grad(lib, act=value) == moe(lib, act=value) == EINVAL
    assert linear(lib, out=value) == linear_grad(lib, out=value) == moe(lib, out_dtype=value) == EINVAL
    assert linear(lib, bias=P, bias_dtype=value) == EINVAL
    assert loss(lib, dX=P, dloss=P, out=value) == EINVAL


POINTERS = [(linear, "codes", 16, False), (linear, "scales", 1, False), (linear, "X", 16, False),
            (linear, "Y", 16, False), (linear, "bias", 4, True), (linear, "residual", 16, True),
            (linear, "Z", 16, True),
            (linear_grad, "codes", 16, False), (linear_grad, "scales", 1, False), (linear_grad, "dY", 16, False),
            (linear_grad, "Z", 16, False), (linear_grad, "dZ", 16, False), (linear_grad, "dX", 16, False),
            (linear_grad, "dbias", 4, True), (linear_grad, "ws", 256, True),
            (loss, "codes", 16, False), (loss, "scales", 1, False), (loss, "X", 16, False),
            (loss, "targets", 8, False), (loss, "loss", 4, False), (loss, "lse", 4, False),
            (loss, "status", 4, True), (loss, "ws", 256, True),
            (moe, "c1", 16, False), (moe, "s1", 1, False), (moe, "c2", 16, False), (moe, "s2", 1, False),
            (moe, "X", 16, False), (moe, "experts", 8, False), (moe, "weights", 4, False),
            (moe, "out", 16, False), (moe, "residual", 16, True), (moe, "ws", 256, True)]


@pytest.mark.parametrize("call,name,align,optional", POINTERS)
def test_null_and_misaligned_pointers(lib, call, name, align, optional):
    if not optional:
        assert call(lib, **{name: NULL}) == EINVAL
    while align > 1:
        align //= 2
        assert call(lib, **{name: off(align)}) == EALIGN, align


def test_a_bf16_bias_needs_two_bytes(lib):
    assert linear(lib, bias=off(1), bias_dtype=1) == EALIGN
    assert linear(lib, bias=off(2), bias_dtype=0) == EALIGN
    assert linear(lib, bias=off(2), bias_dtype=1) not in (EALIGN, EINVAL)


def test_gradient_of_the_loss_is_all_or_nothing(lib):
    assert loss(lib, dX=P) == loss(lib, dloss=P) == EINVAL
    assert loss(lib, dX=off(8), dloss=P) == EALIGN and loss(lib, dX=P, dloss=off(2)) == EALIGN


def test_workspaces(lib):
    need = lib.nf4_mx_cross_entropy_workspace_bytes(1000, 64, 10, 0)
    more = lib.nf4_mx_cross_entropy_workspace_bytes(1000, 64, 10, 1)
    assert 0 < need < more
    assert loss(lib, N=1000, M=10, nbytes=need - 1) == ERANGE and loss(lib, N=1000, M=10, ws=NULL) == ERANGE
    assert loss(lib, N=1000, M=10, dX=P, dloss=P, nbytes=more - 1) == ERANGE
    assert loss(lib, N=1000, M=10, nbytes=need) not in (EINVAL, EALIGN)
    few = lib.nf4_mx_linear_grad_workspace_bytes(4096, 4096, 1)
    assert few > 0
    assert linear_grad(lib, N=4096, K=4096, M=1, nbytes=few - 1) == ERANGE
    assert linear_grad(lib, N=4096, K=4096, M=1, ws=NULL) == ERANGE
    for t, k, e in ((1, 2, 8), (64, 2, 8), (64, 512, 512)):
        need = lib.nf4_moe_mlp_workspace_bytes(e, 64, 64, SWIGLU, t, k)
        assert need >= t * min(k, e) * 64 * 2
        assert moe(lib, E=e, T=t, topk=k, nbytes=need - 1) == ERANGE
        assert moe(lib, E=e, T=t, topk=k, ws=NULL) == ERANGE
    assert lib.nf4_moe_mlp_workspace_bytes(8, 64, 64, SWIGLU, 0, 2) == 0


@pytest.mark.parametrize("rows", [1, 100, 4096, 4097, 20000, (1 << 26) - 1])
def test_the_loss_keeps_no_logits(lib, rows):
    """Whatever the rows and the vocabulary, the workspace stays below its stated bound."""
    for n, k in ((128256, 4096), (1 << 23, 32), (100, 32768)):
        assert 0 < lib.nf4_mx_cross_entropy_workspace_bytes(n, k, rows, 0) <= 1 << 28
        some = min(rows, 4096 + 128)
        # few rows: up to 256 parts of up to 32 rows
        parts = 4 * k * max(2 * some, 256 * 32)
        assert lib.nf4_mx_cross_entropy_workspace_bytes(n, k, rows, 1) <= (1 << 28) + parts


def test_workspace_sizes_in_python(lib):
    assert nf4.mx_cross_entropy_workspace_bytes(1000, 64, 10) == \
        lib.nf4_mx_cross_entropy_workspace_bytes(1000, 64, 10, 0)
    assert nf4.moe_mlp_workspace_bytes(8, 64, 64, 0, 2) == 0
    assert nf4.mx_linear_grad_workspace_bytes(4096, 4096, 1) > 0
    for call in (lambda: nf4.mx_cross_entropy_workspace_bytes(10, 48, 1),
                 lambda: nf4.mx_linear_grad_workspace_bytes(12, 64, 1),
                 lambda: nf4.moe_mlp_workspace_bytes(8, 64, 64, 65, 2)):
        with pytest.raises(ValueError, match="invalid"):
            call()
    with pytest.raises(ValueError, match="act is 'tanh'"):
        nf4.moe_mlp_workspace_bytes(8, 64, 64, 1, 2, act="tanh")


def test_python_refuses_host_tensors():
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    X = torch.zeros((3, 64), dtype=torch.bfloat16)
    ids, w = torch.zeros((3, 2), dtype=torch.int64), torch.zeros((3, 2))
    for call in (lambda: nf4.mx_linear(codes, scales, X), lambda: nf4.mx_linear_grad(codes, scales, X),
                 lambda: nf4.mx_cross_entropy(codes, scales, X, ids[:, 0]),
                 lambda: nf4.moe_mlp(codes[None], scales[None], codes[None], scales[None], X, ids, w)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
