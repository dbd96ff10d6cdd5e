"""Calls of the fused MXFP4 operators that their documentation allows and that lie at an edge:
layers of experts that no token goes to, infinite logits; and gradients by differences."""
import pytest
import torch

import dequant_gemv_nf4_amd as nf4
import grad_differences
from mx_reference import values
from test_gpu_fused import ACTS, BF, DEV, F32, inside, loss_reference, matrix, rand, run_moe

pytestmark = pytest.mark.gpu


# 16 columns a workgroup of the second product, 64, 64 by H; shared out over workgroups and not
@pytest.mark.parametrize("t,k,e,h,i", [(1, 1, 1, 64, 96), (4, 2, 8, 4096, 14336), (1, 2, 8, 4128, 64),
                                       (3, 2, 8, 8192, 544), (16, 8, 512, 256, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_moe_without_any_expert(t, k, e, h, i, dtype):
    """Every token gets its residual, or zero."""
    none = torch.full((t, k), -1, device=DEV)
    none[t - 1, k - 1] = e
    for residual in (False, True):
        m1, m2, x, experts, weights, out = run_moe(t, k, e, h, i, experts=none, residual=residual, dtype=dtype, seed=h)
        assert torch.equal(out, rand((t, h), h + 6, dtype) if residual else torch.zeros_like(out))


def head_with(n, k, special, seed):
    """A head whose column k = 0 is zero, but in the rows `special`, where it is 6 2^s, s > 0."""
    codes, scales = matrix(n, k, seed)
    codes[:, 0] &= 0xF0
    codes[special, 0] |= 7
    scales[special, 0] = 129
    return codes, scales


@pytest.mark.parametrize("m,n", [(9, 2000), (40, 50000), (2100, 36000)])
def test_loss_of_logits_of_minus_infinity(m, n):
    """A logit of -infinity (a product beyond fp32) has probability zero: beside finite ones
    the row's lse, loss and gradient are those of the others."""
    k, special = 96, torch.tensor([7, n // 2, n - 1], device=DEV)
    codes, scales = head_with(n, k, special, 1)
    x = rand((m, k), 2)
    low = torch.arange(m, device=DEV) % 3 == 1
    x[:, 0] = torch.where(low, -3e38, 0.0).to(BF)
    targets = torch.arange(m, device=DEV) % 7           # rows that both heads have
    dloss = rand((m,), 3, F32)
    loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, dloss, out_dtype=F32)
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[special] = False
    for rows, keep in ((low, rest), (~low, torch.ones_like(rest))):
        want = loss_reference(codes[keep], scales[keep], x[rows], targets[rows], dloss[rows])
        inside(lse[rows], want[2], want[3], "lse")
        inside(loss[rows], want[0], want[1], "loss")
        inside(dx[rows], want[4], want[5] + 1e-36, "dX")
    # as the target: the loss is infinite, lse and gradient are not
    targets[:] = n - 1
    loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, dloss, out_dtype=F32)
    want = loss_reference(codes[rest], scales[rest], x[low], targets[low] * 0, None)
    inside(lse[low], want[2], want[3], "lse")           # (the target's part is added last: other bits)
    assert bool((loss[low] == float("inf")).all()) and bool(torch.isfinite(loss[~low]).all())
    v = values(codes, scales)
    p = torch.softmax(x[low].double() @ v[rest].t().contiguous(), 1)
    g = dloss[low].double().unsqueeze(1)
    want = (p @ v[rest] - v[n - 1]) * g
    inside(dx[low], want, 2.0 ** -7 * (p @ v[rest].abs() + v[n - 1].abs()) * g.abs(), "dX")


def test_loss_of_nothing_but_infinities():
    n, k = 3000, 64
    codes, scales = head_with(n, k, torch.arange(n, device=DEV), 1)
    x = rand((4, k), 2)
    x[:, 0] = torch.tensor([-3e38, 3e38, 0.0, -3e38], device=DEV).to(BF)
    targets = torch.tensor([3, 3, 3, -1], device=DEV)
    loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, torch.ones(4, device=DEV))
    assert lse[0] == float("-inf") and lse[3] == float("-inf") and not torch.isfinite(lse[1])
    assert not torch.isfinite(loss[:2]).any() and not torch.isfinite(dx[:2]).any()
    assert torch.isfinite(lse[2]) and torch.isfinite(loss[2]) and torch.isfinite(dx[2]).all()
    assert loss[3] == 0 and (dx[3] == 0).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(3, 64, 64), (40, 128, 96), (600, 64, 32)])
def test_gradient_against_differences(act, m, n, k):
    """dZ, dbias and dX against differences of the activation itself; the bounds are shown to
    refuse wrong gradients in test_grad_differences.py."""
    codes, scales = matrix(n, k, m + n)
    v = values(codes, scales)
    x, bias = rand((m, k), m + 1), rand((n,), m + 2, F32, 0.1)
    exact = x.double() @ v.t().contiguous() + bias.double()
    y, z = nf4.mx_linear(codes, scales, x, bias=bias, act=act, out_dtype=F32, keep_z=True)
    dy = rand(y.shape, m + 3)
    dx, dz, db = nf4.mx_linear_grad(codes, scales, dy, z, act, out_dtype=F32, bias_grad=True)
    assert grad_differences.check_dz(act, z, dy, dz) == 0
    assert grad_differences.check_dbias(act, z, dy, db) == 0
    assert grad_differences.check_dx(dz, v, dx) == 0
    assert grad_differences.check_whole(act, exact, dy, v, dx) == 0
