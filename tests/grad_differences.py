"""The gradient of the fused product by differences of its activation, in 64 bits: what the
activations are is written down here, what their slopes are is not.  Used on the GPU against
the kernels, and on the CPU against wrong gradients, which have to fall outside its bounds.

Bounds, per element: a slope is off by 2^-20, a value of the activation by 2^-20 |z|, their
products by 2^-22 of themselves, dZ by half a step of bf16 more, a sum of m of them by
(m + 8) 2^-24 of its magnitudes; the difference itself by `DIFF`."""
import math

import torch

GATED = ("swiglu", "geglu")
STEP = 1e-5
# h^2 / 6 |f'''| < 2e-11 |f'''|, |f'''| < 2 for all of them, and two roundings of |f| 2^-53 / h
# < 2e-11 |z|, |z| < 16
DIFF = 1e-9


def forward(act, z):
    """f(z) elementwise."""
    if act is None:
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act in ("silu", "swiglu"):
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * (1 + torch.erf(z / math.sqrt(2))) / 2
    return z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))) / 2


def slope(act, z):
    return (forward(act, z + STEP) - forward(act, z - STEP)) / (2 * STEP)


def expected(act, z, dy):
    """(dZ before its rounding, its bound without that) from z and dy, in float64."""
    z, dy = z.double(), dy.double()
    assert float(z.abs().max()) < 16
    if act == "relu":  # no difference over the kink
        assert bool(((z.abs() > STEP) | (z == 0)).all())
    if act in GATED:
        a, b = z.chunk(2, dim=-1)
        dz = torch.cat([dy * b * slope(act, a), dy * forward(act, a)], dim=-1)
        off = torch.cat([(dy * b).abs(), (dy * a).abs()], dim=-1)
    else:
        at = torch.where(z == 0, torch.full_like(z, -1.0), z) if act == "relu" else z
        dz, off = dy * slope(act, at), dy.abs()
    return dz, (2.0 ** -20 + DIFF) * off + 2.0 ** -22 * dz.abs()


def outside(got, want, tol):
    """How many elements are farther from `want` than `tol`."""
    return int((~((got.double() - want).abs() <= tol)).sum())


def check_dz(act, z, dy, dz):
    want, off = expected(act, z, dy)
    return outside(dz, want, off + 2.0 ** -8 * (want.abs() + off))


def check_dbias(act, z, dy, db):
    want, off = expected(act, z, dy)
    m = want.shape[0]
    return outside(db, want.sum(0), off.sum(0) + (m + 8) * 2.0 ** -24 * want.abs().sum(0))


def check_dx(dz, v, dx):
    """dX from the rounded dZ: sums of n products, and of their parts."""
    n = v.shape[0]
    d = dz.double()
    return outside(dx, d @ v, (n + 40) * 2.0 ** -24 * (d.abs() @ v.abs()))


def check_whole(act, z, dy, v, dx):
    """dX through both roundings, of z and of dZ (each half a step of bf16), from the unrounded
    z: |f''| <= 1.13 (largest for gelu_tanh; 0.5 silu, 0.8 gelu), |f'| <= 1.13."""
    want, off = expected(act, z, dy)
    z, dy = z.double(), dy.double()
    if act in GATED:
        a, b = (t.abs() for t in z.chunk(2, dim=-1))
        moved = torch.cat([dy.abs() * 1.13 * b * (a + 1), dy.abs() * 1.13 * a], dim=-1)
    elif act in (None, "relu"):
        moved = torch.zeros_like(want)
    else:
        moved = 1.13 * dy.abs() * z.abs()
    size = off + 2.0 ** -8 * 1.01 * (want.abs() + moved)
    n = v.shape[0]
    return outside(dx, want @ v, size @ v.abs() + (n + 40) * 2.0 ** -24 * ((want.abs() + size) @ v.abs()))
