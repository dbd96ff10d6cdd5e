"""Calls of the fused MXFP4 operators that their documentation allows and that lie at an edge:
layers of experts that no token goes to, as many tokens as there may be, infinite logits, values
that have no part, scales at any address; and gradients by differences."""
import pytest
import torch

import dequant_gemv_nf4_amd as nf4
import grad_differences
from mx_reference import values
from test_gpu_fused import (ACTS, BF, DEV, F32, inside, linear_reference, loss_reference, matrix, moe_reference,
                            rand, run_grad, run_linear, run_loss, run_moe)

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


@pytest.mark.parametrize("m,n,k", [(65, 32000, 256), (2, 5001, 96), (2100, 40003, 64)])
def test_losses_with_and_without_gradient(m, n, k):
    """One call with the gradient and one without, which takes the vocabulary in fewer pieces
    (the last size: two and one): both within the reference's bounds."""
    codes, scales = matrix(n, k, 1)
    x = rand((m, k), 2)
    targets = torch.arange(m, device=DEV) * 97 % n
    targets[::9] = -1
    loss, lse, _ = nf4.mx_cross_entropy(codes, scales, x, targets, torch.ones(m, device=DEV))
    alone, lse_alone = nf4.mx_cross_entropy(codes, scales, x, targets)
    want = loss_reference(codes, scales, x, targets, None)
    for a, b in ((loss, lse), (alone, lse_alone)):
        inside(a, want[0], want[1], "loss")
        inside(b, want[2], want[3], "lse")


# few rows an expert with 16 and with 64 columns a workgroup of the second product, with and
# without parts that meet; the most tokens of that form, whose sums take 128 KB of LDS; tiles
FORMS = [(3, 2, 8, 256, 320), (4, 2, 8, 4096, 7168), (5, 1, 4, 4160, 544), (64, 1, 16, 4096, 1536),
         (61, 2, 32, 2080, 2080), (64, 2, 4, 512, 160)]


@pytest.mark.parametrize("t,k,e,h,i", FORMS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_moe_forms_in_place(t, k, e, h, i, dtype):
    """Every form with a residual, which may be the output itself."""
    m1, m2, x, experts, weights, out = run_moe(t, k, e, h, i, residual=True, dtype=dtype, seed=h)
    r = rand((t, h), h + 6, dtype)
    ws = torch.empty(nf4.moe_mlp_workspace_bytes(e, h, i, t, k), dtype=torch.uint8, device=DEV)
    nf4.nf4_moe_mlp(*m1, *m2, x, experts, weights, r, residual=r, workspace=ws)
    assert torch.equal(r, out)


@pytest.mark.parametrize("t,k,e,h,i", FORMS)
def test_moe_values_that_have_no_part(t, k, e, h, i):
    """NaN in the weights of slots without an expert, and in tokens without any slot."""
    m1, m2 = matrix(2 * i, h, 1, lead=(e,)), matrix(h, i, 2, lead=(e,))
    x, weights = rand((t, h), 3), rand((t, k + 1), 4, F32)
    experts = torch.arange(t * (k + 1), device=DEV).reshape(t, k + 1) * 5 % e
    experts[:, k] = -1
    experts[0] = e
    weights[:, k] = float("nan")
    weights[0] = float("inf")
    x[0] = float("nan")
    out = nf4.moe_mlp(*m1, *m2, x, experts, weights)
    want = nf4.moe_mlp(*m1, *m2, torch.where(torch.isnan(x), 0, x).to(BF), experts,
                       torch.where(torch.isfinite(weights), weights, 0))
    assert torch.equal(out, want) and bool(torch.isfinite(out).all()) and bool((out[0] == 0).all())


def test_loss_gradients_of_ignored_rows_have_no_part():
    codes, scales = matrix(3001, 96, 1)
    x = rand((20, 96), 2)
    targets = torch.arange(20, device=DEV) * 31
    targets[::3], targets[1] = -100, 5000
    dloss = rand((20,), 3, F32)
    want = nf4.mx_cross_entropy(codes, scales, x, targets, dloss)
    out = (targets < 0) | (targets >= 3001)
    dloss[out], x[out] = float("nan"), float("inf")
    got = nf4.mx_cross_entropy(codes, scales, x, targets, dloss)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert bool((got[0][out] == 0).all()) and bool((got[2][out] == 0).all())


def shifted(scales, by):
    """The same scale bytes `by` bytes off a multiple of 16."""
    buf = torch.zeros(scales.numel() + 16, dtype=torch.uint8, device=DEV)
    buf[by:by + scales.numel()] = scales.reshape(-1)
    return buf[by:by + scales.numel()].view(scales.shape)


@pytest.mark.parametrize("by", [1, 2, 7])
@pytest.mark.parametrize("m", [1, 4, 20, 100])
def test_scales_and_biases_anywhere(m, by):
    """Scales have no alignment, a bias that of its type: within the bounds at any address."""
    n, k = 1040, 256
    codes, scales = matrix(n, k, 1)
    s = shifted(scales, by)
    x = rand((m, k), 2)
    for dtype in (BF, F32):
        bias = rand((n + 3,), 3, dtype)[3:]
        for act in ("silu", "swiglu"):
            y, z = nf4.mx_linear(codes, s, x, bias=bias, act=act, keep_z=True)
            want = linear_reference(codes, scales, x, bias, act, None, BF)
            inside(y, want[0], want[1], "Y")
            inside(z, want[2], want[3], "Z")
    dy = rand((m, n), 4)
    dx = nf4.mx_linear_grad(codes, s, dy, out_dtype=F32)[0]
    v = values(codes, scales)
    inside(dx, dy.double() @ v, (n + 40) * 2.0 ** -24 * (dy.double().abs() @ v.abs()) + 1e-30, "dX")
    targets = torch.arange(m, device=DEV) * 7
    loss, lse, dx = nf4.mx_cross_entropy(codes, s, x, targets, torch.ones(m, device=DEV), out_dtype=F32)
    want = loss_reference(codes, scales, x, targets, torch.ones(m, device=DEV))
    inside(lse, want[2], want[3], "lse")
    inside(loss, want[0], want[1], "loss")
    inside(dx, want[4], want[5] + 1e-36, "dX")


@pytest.mark.parametrize("by", [1, 2, 7])
@pytest.mark.parametrize("t,k,e,h,i", FORMS)
def test_expert_scales_anywhere(t, k, e, h, i, by):
    m1, m2, x, experts, weights, _ = run_moe(t, k, e, h, i, dtype=F32, seed=by)
    out = nf4.moe_mlp(m1[0], shifted(m1[1], by), m2[0], shifted(m2[1], by), x, experts, weights, out_dtype=F32)
    want, tol = moe_reference(m1, m2, x, experts, weights, "swiglu", None, F32)
    inside(out, want, tol, "experts")


# Sizes of the tiles and plans that the tests of kernels and shapes leave out
MORE_TILES = [(193, 25094, 32), (200, 26006, 128)]
MORE_GRADIENTS = [(70, 504, 1152), (1827, 3912, 32), (33, 29608, 2816), (330, 24, 4128), (1040, 744, 3712)]


@pytest.mark.parametrize("m,n,k", MORE_TILES)
@pytest.mark.parametrize("act,bias", [("geglu", BF), ("silu", F32)])
def test_more_linear_tiles(m, n, k, act, bias):
    run_linear(m, n, k, act, bias=bias, residual=act == "silu", keep=act == "geglu", seed=k + m)


@pytest.mark.parametrize("m,n,k", MORE_TILES)
def test_more_loss_tiles(m, n, k):
    run_loss(m, n, k, True, seed=k, dtype=BF)


@pytest.mark.parametrize("m,n,k", MORE_GRADIENTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_gradients(m, n, k, dtype):
    run_grad(m, n, k, "swiglu" if n % 16 == 0 else "silu", True, dtype, seed=n)
