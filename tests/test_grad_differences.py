"""The gradient check by differences, on the CPU: the right gradient (autograd in float64,
rounded as the operator documents) is inside its bounds, and gradients with a mistake are not."""
import pytest
import torch

import grad_differences as gd
from mx_reference import values

ACTS = (None, "relu", "silu", "gelu", "gelu_tanh", "swiglu", "geglu")
BF = torch.bfloat16


def make(act, m=5, n=64, k=64):
    g = torch.Generator().manual_seed(len(str(act)))
    z = 1.5 * torch.randn((m, n), generator=g, dtype=torch.float64)
    cols = n // 2 if act in gd.GATED else n
    dy = torch.randn((m, cols), generator=g).to(BF)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(120, 124, (n, k // 32), generator=g).to(torch.uint8)
    return z, dy, values(codes, scales)


def gradient(act, z, dy):
    z = z.double().clone().requires_grad_()
    a = z.chunk(2, dim=-1)
    y = gd.forward(act, a[0]) * a[1] if act in gd.GATED else gd.forward(act, z)
    return torch.autograd.grad(y, z, dy.double())[0]


@pytest.mark.parametrize("act", ACTS)
def test_the_right_gradient_is_inside(act):
    exact, dy, v = make(act)
    z = exact.to(BF)
    dz = gradient(act, z, dy)
    rounded = dz.to(BF)
    assert gd.check_dz(act, z, dy, rounded) == 0
    assert gd.check_dbias(act, z, dy, dz.float().sum(0)) == 0
    assert gd.check_dx(rounded, v, (rounded.double() @ v).float()) == 0
    assert gd.check_whole(act, exact, dy, v, (rounded.double() @ v).float()) == 0


def mistakes(act, z, dy):
    """(name, wrong dZ) in float64."""
    dz = gradient(act, z, dy)
    yield "zero", torch.zeros_like(dz)
    yield "sign", -dz
    zd, d = z.double(), dy.double()
    a = zd.chunk(2, dim=-1)[0]
    first = {"silu": torch.sigmoid, "swiglu": torch.sigmoid, "gelu": lambda t: (1 + torch.erf(t / 2 ** 0.5)) / 2,
             "gelu_tanh": lambda t: gd.forward("gelu_tanh", t) / t, "geglu": lambda t: gd.forward("geglu", t) / t}
    if act in gd.GATED:
        b = zd.chunk(2, dim=-1)[1]
        yield "slope without its second term", torch.cat([d * b * first[act](a), d * gd.forward(act, a)], -1)
        yield "slope left out", torch.cat([d * b, d * gd.forward(act, a)], -1)
        yield "gated value left out", torch.cat([dz.chunk(2, dim=-1)[0] / b, d * gd.forward(act, a)], -1)
        yield "halves changed", torch.cat(dz.chunk(2, dim=-1)[::-1], -1)
    elif act is not None:
        yield "slope left out", d.clone()
        if act != "relu":
            yield "slope without its second term", d * first[act](zd)
    if act in ("gelu", "gelu_tanh", "geglu"):
        other = "gelu_tanh" if act == "gelu" else "gelu"
        if act == "geglu":
            yield "the other gelu's slope", torch.cat([d * b * gd.slope(other, a), d * gd.forward(act, a)], -1)
        else:
            yield "the other gelu's slope", d * gd.slope(other, zd)


@pytest.mark.parametrize("act", ACTS)
def test_wrong_gradients_are_outside(act):
    exact, dy, v = make(act, m=40)
    z = exact.to(BF)
    right = gradient(act, z, dy).to(BF)
    for name, wrong in mistakes(act, z, dy):
        assert gd.check_dz(act, z, dy, wrong.to(BF)) > 0, name
        assert gd.check_dbias(act, z, dy, wrong.float().sum(0)) > 0, name
        assert gd.check_dx(right, v, (wrong.to(BF).double() @ v).float()) > 0, name
        if "other gelu" not in name:  # (they differ by 4e-4 of z, less than bf16)
            assert gd.check_whole(act, exact, dy, v, (wrong.to(BF).double() @ v).float()) > 0, name
    missing = v.clone()
    missing[17] = 0
    assert gd.check_dx(right, v, (right.double() @ missing).float()) > 0
    assert gd.check_dbias(act, z, dy, right.double()[:-1].sum(0).float()) > 0
