"""Fused forms of the MXFP4 products on the GPU against 64-bit definitions: the product
with bias, activation and residual and its gradient, the head's cross entropy, and the
expert layer for a few tokens.

Tolerances.  Sums of T products are off by at most (T + 8) 2^-24 of the sum of their
magnitudes; an activation by 2^-20 |z|, its slope by 2^-20, and |f'| <= 1.13; rounding to
bf16 by 2^-8 of the value, to fp32 by 2^-24."""
import math

import pytest
import torch

import dequant_gemv_nf4_amd as nf4
from gpu_guard import alloc, check
from mx_reference import values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
GATED = ("swiglu", "geglu")
ACTS = (None, "relu", "silu", "gelu", "gelu_tanh", "swiglu", "geglu")
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def matrix(n, k, seed, sigma=0.05, lead=()):
    """Random packed bytes: every code, scales around sigma."""
    g = gen(seed)
    codes = torch.randint(0, 256, (*lead, n, k // 2), dtype=torch.uint8, device=DEV, generator=g)
    mid = 127 + round(math.log2(sigma))
    scales = torch.randint(mid - 2, mid + 2, (*lead, n, k // 32), device=DEV, generator=g)
    return codes, scales.to(torch.uint8)


def rand(shape, seed, dtype=BF, scale=1.0):
    return (scale * torch.randn(shape, device=DEV, generator=gen(seed))).to(dtype)


def f64(act, z):
    """(f(z), f'(z)) in float64."""
    if act is None:
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act in ("silu", "swiglu"):
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if act == "gelu":
        c = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(a * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * (1 - s) * a * (1 + 3 * 0.044715 * z * z)


def inside(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                                 f"{float((err / tol).nan_to_num(nan=1e9).max()):.3g} x tolerance")


def linear_reference(codes, scales, x, bias, act, residual, dtype):
    """(y, tolerance, z, tolerance of z)."""
    v = values(codes, scales)
    k = v.shape[1]
    z = x.double() @ v.t().contiguous()
    dz = (k + 8) * 2.0 ** -24 * (x.double().abs() @ v.abs().t().contiguous()) + 1e-30
    if bias is not None:
        z = z + bias.double()
        dz = dz + 2.0 ** -23 * (z.abs() + bias.double().abs())
    if act in GATED:
        a, b = z.chunk(2, dim=-1)
        da, db = dz.chunk(2, dim=-1)
        f = f64(act, a)[0]
        df = 1.13 * da + 2.0 ** -20 * (a.abs() + da)
        y, tol = f * b, df * (b.abs() + db) + f.abs() * db + 2.0 ** -23 * (f * b).abs()
    else:
        y = f64(act, z)[0]
        tol = 1.13 * dz + (0 if act in (None, "relu") else 2.0 ** -20) * (z.abs() + dz)
    if residual is not None:
        y = y + residual.double()
        tol = tol + 2.0 ** -23 * (y.abs() + residual.double().abs())
    half = HALF[dtype]
    return y, tol * (1 + half) + half * y.abs() + 1e-30, z, dz * (1 + HALF[BF]) + HALF[BF] * z.abs()


def run_linear(m, n, k, act, bias=None, residual=False, dtype=BF, keep=False, seed=0, vector=False):
    codes, scales = matrix(n, k, seed + 1)
    cols = n // 2 if act in GATED else n
    x = rand((k,) if vector else (m, k), seed + 2)
    b = None if bias is None else rand((n,), seed + 3, bias)
    lead = () if vector else (m,)
    r = rand((*lead, cols), seed + 4, dtype) if residual else None
    ybuf, y = alloc((*lead, cols), dtype, DEV)
    zbuf, z = alloc((*lead, n), BF, DEV) if keep else (None, None)
    nf4.nf4_mx_linear(codes, scales, x, y, b, act, r, z)
    want, tol, zw, ztol = linear_reference(codes, scales, x, b, act, r, dtype)
    inside(y, want, tol, f"Y {m}x{n}x{k} {act}")
    check(ybuf, "Y")
    if keep:
        inside(z, zw, ztol, "Z")
        check(zbuf, "Z")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 2, 3, 17, 40, 70])
def test_linear_acts(m, act):
    run_linear(m, 272, 160, act, bias=F32, residual=True, keep=True, seed=m)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bias", [None, BF, F32])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_linear_operands(act, bias, dtype):
    for residual in (False, True):
        run_linear(5, 96, 64, act, bias, residual, dtype, keep=residual, seed=7)


# columns that are no multiple of a vector, of a tile, of anything
@pytest.mark.parametrize("n", [1, 2, 3, 17, 30, 66, 129, 250])
@pytest.mark.parametrize("m", [1, 4, 9, 33])
def test_linear_odd_columns(m, n):
    run_linear(m, n, 96, "silu", bias=F32, residual=True, keep=True, seed=n)
    if n % 2 == 0:
        run_linear(m, n, 96, "swiglu", bias=BF, residual=True, dtype=F32, keep=True, seed=n)


# each kernel: one, two, four rows; tiles of 16 x 32 up to 128 x 256; scales at odd strides
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (2, 4096, 2080), (4, 2048, 4096), (8, 4096, 4096),
                                   (16, 10240, 512), (16, 28672, 256), (33, 24576, 256),
                                   (100, 6144, 512), (40, 26624, 288), (300, 13824, 256),
                                   (300, 13824, 96), (520, 14336, 256), (520, 14336, 160),
                                   (700, 13824, 128), (700, 13810, 96), (200, 28672, 128), (200, 28610, 160)])
@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh"])
def test_linear_kernels(m, n, k, act):
    run_linear(m, n, k, act, bias=F32, residual=True, keep=m % 2 == 0, seed=k + m)


def test_linear_vector_and_in_place():
    run_linear(1, 64, 64, "relu", residual=True, vector=True)
    codes, scales = matrix(96, 64, 1)
    x, r = rand((6, 64), 2), rand((6, 96), 3)
    want = nf4.mx_linear(codes, scales, x, act="silu", residual=r)
    nf4.nf4_mx_linear(codes, scales, x, r, act="silu", residual=r)
    assert torch.equal(r, want)


# One size of each tile of the products with epilogues, with whole words of scales and
# (second of each) without, the last columns of a tile left out
TILES = [(600, 20010, 128), (600, 20010, 160), (200, 40006, 128), (200, 40006, 160), (200, 20010, 128),
         (200, 20010, 160), (100, 9000, 128), (100, 9000, 160), (20, 40006, 128), (20, 40006, 160),
         (100, 2050, 128), (100, 2050, 160), (100, 2050, 4096), (100, 2050, 4128), (40, 130, 128),
         (40, 130, 160), (40, 4100, 1024), (40, 4100, 1056), (40, 130, 1024), (40, 130, 1056)]


@pytest.mark.parametrize("m,n,k", TILES)
@pytest.mark.parametrize("act,bias", [("geglu", BF), ("silu", F32)])
def test_linear_tiles(m, n, k, act, bias):
    run_linear(m, n, k, act, bias=bias, residual=act == "silu", keep=act == "geglu", seed=k + m)


def test_linear_is_the_product():
    """Without bias, activation and residual the sums are nf4_mx_gemm's, bit for bit."""
    for m in (1, 3, 20, 300):
        codes, scales = matrix(1024, 512, m)
        x = rand((m, 512), m)
        for dtype in (BF, F32):
            assert torch.equal(nf4.mx_linear(codes, scales, x, out_dtype=dtype),
                               nf4.mx_gemm(codes, scales, x, out_dtype=dtype))


def test_linear_large_values():
    """Activations where exp overflows and where nothing is left of the small side."""
    codes = torch.full((32, 16), 0x22, dtype=torch.uint8, device=DEV)  # every value 1
    scales = torch.full((32, 1), 127, dtype=torch.uint8, device=DEV)
    x = torch.zeros((6, 32), dtype=BF, device=DEV)
    x[:, 0] = torch.tensor([-1e30, -200.0, -20.0, 20.0, 200.0, 1e30], device=DEV).to(BF)
    for act in ACTS[1:5]:
        y = nf4.mx_linear(codes, scales, x, act=act, out_dtype=F32)
        want = f64(act, x[:, :1].double()).__getitem__(0).expand(6, 32)
        inside(y, want, 2.0 ** -20 * x[:, :1].double().abs(), act)
    x[:, 0] = torch.tensor([float("inf"), float("nan"), 1, 2, 3, 4], device=DEV).to(BF)
    for act in ACTS[1:5]:
        y = nf4.mx_linear(codes, scales, x, act=act, out_dtype=F32)
        assert torch.isinf(y[0]).all() and torch.isnan(y[1]).all() and torch.isfinite(y[2:]).all()


def grad_reference(codes, scales, dy, z, act):
    """(dz, tolerance, db, tolerance)."""
    z, dy = z.double(), dy.double()
    if act in GATED:
        a, b = z.chunk(2, dim=-1)
        f, df = f64(act, a)
        dz = torch.cat([dy * b * df, dy * f], dim=-1)
        off = torch.cat([2.0 ** -20 * (dy * b).abs(), 2.0 ** -20 * (dy * a).abs()], dim=-1)
    else:
        dz = dy * f64(act, z)[1]
        off = 2.0 ** -20 * dy.abs()
    off = off + 2.0 ** -22 * dz.abs()
    m = dz.reshape(-1, dz.shape[-1]).shape[0]
    db = dz.reshape(m, -1).sum(0)
    dbtol = off.reshape(m, -1).sum(0) + (m + 8) * 2.0 ** -24 * dz.abs().reshape(m, -1).sum(0)
    return dz, off + HALF[BF] * dz.abs() + 1e-30, db, dbtol + 1e-30


def run_grad(m, n, k, act, bias, dtype=BF, seed=0):
    codes, scales = matrix(n, k, seed + 1)
    cols = n // 2 if act in GATED else n
    z, dy = rand((m, n), seed + 2, scale=2.0), rand((m, cols), seed + 3)
    dxbuf, dx = alloc((m, k), dtype, DEV)
    dzbuf, dz = alloc((m, n), BF, DEV)
    dbbuf, db = alloc((n,), F32, DEV) if bias else (None, None)
    need = nf4.mx_linear_grad_workspace_bytes(n, k, m)
    wsbuf, ws = alloc((need,), torch.uint8, DEV) if need else (None, None)
    nf4.nf4_mx_linear_grad(codes, scales, dy, z, act, dx, dz, db, ws)
    want, tol, dbw, dbtol = grad_reference(codes, scales, dy, z, act)
    inside(dz, want, tol, f"dZ {m}x{n}x{k} {act}")
    if bias:
        inside(db, dbw, dbtol, "dbias")
        check(dbbuf, "dbias")
    v = values(codes, scales)
    mag = (n + 40) * 2.0 ** -24 * (dz.double().abs() @ v.abs())   # 40: the parts' sums
    want = dz.double() @ v
    inside(dx, want, mag * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + 1e-30, "dX")
    for buf in (dxbuf, dzbuf) + ((wsbuf,) if need else ()):
        check(buf, "gradient")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 5, 17, 40, 130])
def test_grad_acts(m, act):
    run_grad(m, 272, 160, act, True, seed=m)


@pytest.mark.parametrize("m,n,k", [(1, 8, 32), (2, 16, 64), (1, 4096, 4096), (20, 8192, 96), (77, 13824, 640),
                                   (64, 1000, 4096), (700, 504, 1056), (2100, 64, 4096), (50, 1032, 32),
                                   (33, 4104, 8192), (300, 8192, 1056), (300, 8192, 1152), (1100, 8200, 2464),
                                   (1100, 8200, 2560), (1000, 8200, 1504), (1200, 2056, 4128), (130, 28672, 256)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_grad_shapes(m, n, k, dtype):
    run_grad(m, n, k, "swiglu" if n % 16 == 0 else "silu", m % 2 == 0, dtype, seed=n)


@pytest.mark.parametrize("act", ACTS)
def test_grad_by_differences(act):
    """The gradient agrees with central differences of the 64-bit forward."""
    m, n, k = 3, 32, 64
    codes, scales = matrix(n, k, 5)
    x, b = rand((m, k), 6), rand((n,), 7, F32)
    y, z = nf4.mx_linear(codes, scales, x, bias=b, act=act, out_dtype=F32, keep_z=True)
    dy = rand(y.shape, 8)
    dx, _, db = nf4.mx_linear_grad(codes, scales, dy, z, act, out_dtype=F32, bias_grad=True)

    def total(x, b):
        v = values(codes, scales)
        z = x @ v.t().contiguous() + b
        if act in GATED:
            p, q = z.chunk(2, dim=-1)
            return float((f64(act, p)[0] * q * dy.double()).sum())
        return float((f64(act, z)[0] * dy.double()).sum())

    h = 1e-5
    x64, b64 = x.double(), b.double()
    # z and dZ are rounded to bf16 in between: 2^-7 of the gradient's terms, whose size the
    # rows' norms bound
    v = values(codes, scales)
    size = float(dy.double().abs().sum(1).max() * (z.double().abs().max() + 1.13) * 1.6)
    for i, j in ((0, 0), (1, 17), (2, 63)):
        if act == "relu" and float((x64[i] @ v.t()).add(b64).abs().min()) < 1e-3:
            continue
        e = torch.zeros_like(x64)
        e[i, j] = h
        want = (total(x64 + e, b64) - total(x64 - e, b64)) / (2 * h)
        assert abs(float(dx[i, j]) - want) <= 2.0 ** -7 * size * float(v[:, j].abs().max()), (act, i, j)
    for j in (0, 15, 31):
        e = torch.zeros_like(b64)
        e[j] = h
        want = (total(x64, b64 + e) - total(x64, b64 - e)) / (2 * h)
        assert abs(float(db[j]) - want) <= 2.0 ** -7 * size * m, (act, j)


@pytest.mark.parametrize("act", [None, "silu", "swiglu"])
@pytest.mark.parametrize("m", [511, 512, 577, 3000])
def test_bias_gradient_of_many_rows(m, act):
    """Rows shared out over workgroups; dbias anywhere that fp32 may lie."""
    n, k = 136, 64
    codes, scales = matrix(n, k, 1)
    dy, z = rand((m, n // 2 if act == "swiglu" else n), 2), rand((m, n), 3)
    buf, ws = alloc((nf4.mx_linear_grad_workspace_bytes(n, k, m),), torch.uint8, DEV)
    db = torch.full((n + 5,), 7.0, device=DEV)
    dx, dz = torch.empty((m, k), device=DEV), torch.empty_like(z)
    nf4.nf4_mx_linear_grad(codes, scales, dy, None if act is None else z, act, dx, dz, db[3:3 + n], ws)
    check(buf, "workspace")
    assert (db[:3] == 7).all() and (db[3 + n:] == 7).all()
    want, tol = grad_reference(codes, scales, dy, z, act)[2:]
    inside(db[3:3 + n], want, tol, f"dbias {m} {act}")


def test_grad_without_activation():
    codes, scales = matrix(64, 96, 1)
    dy = rand((9, 64), 2)
    dx, dz, db = nf4.mx_linear_grad(codes, scales, dy, out_dtype=F32, bias_grad=True)
    assert dz is dy
    off = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    same = nf4.mx_gemm_grouped_grad(codes[None], scales[None], dy, off)
    tol = 72 * 2.0 ** -23 * (dy.double().abs() @ values(codes, scales).abs())
    inside(dx, same.double(), tol, "dX")
    inside(db, dy.double().sum(0), 17 * 2.0 ** -24 * dy.double().abs().sum(0), "dbias")


def test_slopes_at_large_values():
    codes, scales = matrix(32, 32, 1)
    z = torch.tensor([-3e38, -1e20, -88.0, -30.0, -6.0, 0.0, 5.0, 8.0, 30.0, 88.0, 1e20, 3e38],
                     device=DEV).to(BF)
    z = z.repeat(3)[:32].reshape(1, 32).contiguous()
    dy = torch.ones_like(z)
    for act in ACTS[1:5]:
        dz = nf4.mx_linear_grad(codes, scales, dy, z, act)[1]
        want = f64(act, z.double().clamp(-1e4, 1e4))[1]
        inside(dz, want, 2.0 ** -20 + HALF[BF] * want.abs(), act)


# ------------------------------------------------------------ cross entropy ----
def loss_reference(codes, scales, x, targets, dloss):
    """(loss, tolerance, lse, tolerance, dX, tolerance) in float64."""
    v = values(codes, scales)
    n, k = v.shape
    l = x.double() @ v.t().contiguous()
    dl = ((k + 8) * 2.0 ** -24 * (x.double().abs() @ v.abs().t().contiguous())).amax(1)
    lse = torch.logsumexp(l, dim=1)
    top = l.abs().amax(1)
    # exp 2^-20 a 64 of |l|; sums of it in fp32: 16 terms a lane, then strips a thread, threads,
    # pieces, each in turn or as a tree, fewer than 128 steps
    e = 2.0 ** -20 * (1 + top / 64) + 2.0 ** -17
    lsetol = dl + e + 2.0 ** -22 * lse.abs()
    kept = (targets >= 0) & (targets < n)
    at = torch.where(kept, targets, 0).unsqueeze(1)
    lt = l.gather(1, at).squeeze(1)
    loss = torch.where(kept, lse - lt, 0.0)
    losstol = torch.where(kept, lsetol + dl + 2.0 ** -23 * (lse.abs() + lt.abs()), 0.0)
    if dloss is None:
        return loss, losstol, lse, lsetol
    p = torch.exp(l - lse.unsqueeze(1))
    g = torch.where(kept, dloss.double(), 0.0).unsqueeze(1)
    mag = p @ v.abs()
    off = mag * (2.0 ** -8 + 2 * (dl + e).unsqueeze(1) + (n + 40) * 2.0 ** -24)
    row = v[at.squeeze(1)]
    dx = (p @ v - row) * g
    off = (off + 2.0 ** -22 * (mag + row.abs())) * g.abs()
    return loss, losstol, lse, lsetol, dx, off


def run_loss(m, n, k, grad, dtype=BF, seed=0, scale=1.0, sigma=0.05, ignored=True):
    codes, scales = matrix(n, k, seed + 1, sigma)
    x = rand((m, k), seed + 2, scale=scale)
    targets = torch.randint(0, n, (m,), device=DEV, generator=gen(seed + 3))
    if ignored:
        targets[::5] = -100
        targets[3::7] = -1
    dloss = rand((m,), seed + 4, F32) if grad else None
    need = nf4.mx_cross_entropy_workspace_bytes(n, k, m, grad)
    wsbuf, ws = alloc((need,), torch.uint8, DEV)
    lbuf, loss = alloc((m,), F32, DEV)
    ebuf, lse = alloc((m,), F32, DEV)
    dbuf, dx = alloc((m, k), dtype, DEV) if grad else (None, None)
    nf4.nf4_mx_cross_entropy(codes, scales, x, targets, loss, lse, dloss, dx, ws)
    want = loss_reference(codes, scales, x, targets, dloss)
    what = f"{m}x{n}x{k}"
    inside(lse, want[2], want[3], "lse " + what)
    inside(loss, want[0], want[1], "loss " + what)
    if grad:
        tol = want[5] * (1 + HALF[dtype]) + HALF[dtype] * want[4].abs() + 1e-36
        inside(dx, want[4], torch.where((targets < 0).unsqueeze(1), 0.0, tol), "dX " + what)
        check(dbuf, "dX")
    for buf in (wsbuf, lbuf, ebuf):
        check(buf, "cross entropy")


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("n", [1, 2, 8, 17, 100, 257, 1031])
@pytest.mark.parametrize("m", [1, 5, 17, 40, 100])
def test_loss_small(m, n, grad):
    run_loss(m, n, 96, grad, seed=n, dtype=F32 if n % 2 else BF)


@pytest.mark.parametrize("m,n,k", [(1, 32000, 4096), (5, 32000, 512), (16, 128256, 128), (33, 50257, 160),
                                   (70, 50257, 96), (300, 32001, 256), (2100, 40003, 64), (4200, 301, 32),
                                   (4100, 17000, 32), (130, 700, 8192), (700, 13810, 64), (200, 28609, 96),
                                   (300, 13801, 96), (400, 48000, 64)])
@pytest.mark.parametrize("grad", [False, True])
def test_loss_shapes(m, n, k, grad):
    run_loss(m, n, k, grad, seed=k, dtype=BF if m % 2 else F32)


@pytest.mark.parametrize("m,n,k", TILES)
def test_loss_tiles(m, n, k):
    run_loss(m, n, k, True, seed=k, dtype=BF)


@pytest.mark.parametrize("scale", [0.0, 1e-3, 30.0, 1000.0])
def test_loss_ranges(scale):
    """Logits that are all zero, nearly equal, and hundreds or ten thousands apart."""
    run_loss(37, 3000, 128, True, seed=3, scale=scale, dtype=F32)


def test_loss_rising_maximum():
    """Every strip beats the ones before by far, so all but the last count for nothing; and
    the other way round; over several pieces."""
    m, n, k = 2100, 36000, 32
    codes = torch.zeros((n, 16), dtype=torch.uint8, device=DEV)
    codes[:, 0] = 2                                     # value 1 at k = 0
    step = torch.arange(n, device=DEV) * 24 // n        # powers of two 2^0 .. 2^23
    for order in (step, step.flip(0)):
        scales = (110 + order).to(torch.uint8).reshape(n, 1)
        x = torch.zeros((m, k), dtype=BF, device=DEV)
        x[:, 0] = torch.linspace(-64, 64, m, device=DEV).to(BF)
        targets = torch.arange(m, device=DEV) * 17 % n
        dloss = torch.ones(m, device=DEV)
        loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, dloss, out_dtype=F32)
        want = loss_reference(codes, scales, x, targets, dloss)
        inside(lse, want[2], want[3], "lse")
        inside(loss, want[0], want[1], "loss")
        inside(dx, want[4], want[5] + 1e-36, "dX")


def test_loss_of_huge_logits():
    """Logits up to 2^29: finite, and right to what fp32 holds of them; a row that has one
    far above the others is its one-hot gradient."""
    m, n, k = 40, 5000, 32
    codes = torch.zeros((n, 16), dtype=torch.uint8, device=DEV)
    codes[:, 0] = 2                                     # value 1 at k = 0
    codes[:, 8] = 4                                     # value 2 at k = 16
    scales = (127 + torch.arange(n, device=DEV) % 24).to(torch.uint8).reshape(n, 1)
    scales[n - 1] = 127 + 26
    x = torch.zeros((m, k), dtype=BF, device=DEV)
    x[:, 0] = torch.linspace(-8, 8, m, device=DEV).to(BF)
    targets = torch.arange(m, device=DEV) * 131 % n
    targets[m - 1] = n - 1
    loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, torch.ones(m, device=DEV), out_dtype=F32)
    l = x.double() @ values(codes, scales).t().contiguous()
    assert float(l.max()) == 2.0 ** 29 and float(l.min()) == -2.0 ** 29
    want = loss_reference(codes, scales, x, targets, torch.ones(m, device=DEV))
    inside(lse, want[2], want[3], "lse")
    inside(loss, want[0], want[1], "loss")
    v = values(codes, scales)
    top = x[:, 0] > 0.1                                 # the last column is the largest by far
    one = v[n - 1] - v[targets]
    inside(dx[top], one[top], 2.0 ** -8 * (v[n - 1].abs() + v[targets].abs())[top], "dX")
    assert (dx[m - 1] == 0).all() and loss[m - 1] == 0


def test_loss_of_well_predicted_tokens():
    """Targets of probabilities from next to nothing up to 1 - 3e-5: the loss and the gradient
    are as precise as they are small (the target's own value is not rounded)."""
    m, n, k = 24, 5000, 64
    codes, scales = matrix(n, k, 1)
    v = values(codes, scales)
    targets = torch.arange(m, device=DEV) * 200 + 7
    row = v[targets]
    x = (row * (torch.linspace(8, 30, m, device=DEV) / (row * row).sum(1)).unsqueeze(1)).to(BF)
    dloss = torch.ones(m, device=DEV)
    loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, dloss, out_dtype=F32)
    l = x.double() @ v.t().contiguous()
    dl = ((k + 8) * 2.0 ** -24 * (x.double().abs() @ v.abs().t().contiguous())).amax(1)
    others = l.clone()
    others[torch.arange(m), targets] = float("-inf")
    rest = torch.logsumexp(others, 1) - l.gather(1, targets.unsqueeze(1)).squeeze(1)   # log of the ratio
    want = torch.nn.functional.softplus(rest)
    assert float(want.min()) < 1e-4 and int((want < 0.1).sum()) > 5
    # the ratio of two sums of exp, each off by e relative to itself
    e = 2 * dl + 2 * (2.0 ** -20 * (1 + l.abs().amax(1) / 64) + 2.0 ** -17)
    # where the ratio is below 1 it is taken as such, else as a difference of logs
    tol = torch.where(rest < -0.01, e * want + 2.0 ** -22 * want, e + 2.0 ** -21 * lse.double().abs())
    inside(loss, want, tol, "loss")
    p = torch.softmax(others, 1)
    share = torch.sigmoid(rest).unsqueeze(1)                  # 1 - p of the target
    want = share * (p @ v - row)
    size = share * (p @ v.abs() + row.abs())
    inside(dx, want, size * (2.0 ** -8 + (n + 40) * 2.0 ** -24 + 2 * e.unsqueeze(1)), "dX")


def test_loss_not_finite():
    codes, scales = matrix(5000, 64, 1)
    x = rand((8, 64), 2)
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    x[3] = float("nan")
    targets = torch.tensor([1, 2, 3, -1, 4, 5, -7, 6], device=DEV)
    loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, torch.ones(8, device=DEV))
    assert not torch.isfinite(lse[1:4]).any() and not torch.isfinite(loss[1:3]).any()
    assert not torch.isfinite(dx[1:3]).any()
    assert loss[3] == 0 and (dx[3] == 0).all() and (dx[6] == 0).all() and torch.isfinite(lse[6])
    rest = [0, 4, 5, 7]
    alone = nf4.mx_cross_entropy(codes, scales, x[rest].contiguous(), targets[rest], torch.ones(4, device=DEV))
    want = loss_reference(codes, scales, x[rest], targets[rest], torch.ones(4, device=DEV))
    inside(loss[rest], want[0], want[1], "loss")
    inside(alone[0], want[0], want[1], "loss")
    inside(dx[rest], want[4], want[5] * 1.01 + 2.0 ** -8 * want[4].abs(), "dX")


def test_loss_bad_targets():
    codes, scales = matrix(100, 64, 1)
    x = rand((6, 64), 2)
    targets = torch.tensor([0, 99, 100, -1, 1 << 40, -(1 << 40)], device=DEV)
    ones = torch.ones(6, device=DEV)
    with pytest.raises(ValueError, match="flagged targets"):
        nf4.mx_cross_entropy(codes, scales, x, targets, check=True)
    loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, ones)
    assert (loss[2:] == 0).all() and (dx[2:] == 0).all() and (loss[:2] != 0).all()
    nf4.mx_cross_entropy(codes, scales, x, targets.clamp(max=99), ones, check=True)
    status = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    ws = torch.empty(nf4.mx_cross_entropy_workspace_bytes(100, 64, 6), dtype=torch.uint8, device=DEV)
    nf4.nf4_mx_cross_entropy(codes, scales, x, targets, loss, lse, workspace=ws, dev_status=status)
    assert int(status) == nf4.LOSS_BAD_TARGET


def test_loss_by_differences():
    m, n, k = 4, 500, 64
    codes, scales = matrix(n, k, 1)
    x = rand((m, k), 2)
    targets = torch.tensor([3, 499, -100, 250], device=DEV)
    dloss = rand((m,), 3, F32)
    dx = nf4.mx_cross_entropy(codes, scales, x, targets, dloss, out_dtype=F32)[2]
    v = values(codes, scales)

    def total(x):
        l = x @ v.t().contiguous()
        t = targets.clamp(min=0).unsqueeze(1)
        one = torch.logsumexp(l, 1) - l.gather(1, t).squeeze(1)
        return float((torch.where(targets >= 0, one, 0.0) * dloss.double()).sum())

    for i, j in ((0, 0), (1, 63), (2, 5), (3, 31)):
        e = torch.zeros((m, k), dtype=torch.float64, device=DEV)
        e[i, j] = 1e-5
        want = (total(x.double() + e) - total(x.double() - e)) / 2e-5
        # bf16 values: 2^-8 of the mean of |v|; the difference itself: 1e-9
        assert abs(float(dx[i, j]) - want) <= 2.0 ** -7 * float(v[:, j].abs().max() * dloss[i].abs()) + 1e-9


def test_loss_same_bits():
    """Twice the same, and the losses with and without gradient agree within their bounds."""
    codes, scales = matrix(32000, 256, 1)
    x = rand((65, 256), 2)
    targets = torch.randint(0, 32000, (65,), device=DEV)
    a = nf4.mx_cross_entropy(codes, scales, x, targets, torch.ones(65, device=DEV))
    b = nf4.mx_cross_entropy(codes, scales, x, targets, torch.ones(65, device=DEV))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


# -------------------------------------------------- expert layer for few tokens ----
def moe_reference(m1, m2, x, experts, weights, act, residual, dtype):
    """(out, tolerance) in float64."""
    num, t = m1[0].shape[0], x.shape[0]
    out = torch.zeros((t, m2[0].shape[1]), dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    share = torch.zeros((t, num), dtype=torch.float64, device=DEV)
    kept = (experts >= 0) & (experts < num)
    share.scatter_add_(1, torch.where(kept, experts, 0), torch.where(kept, weights.double(), 0.0))
    size = torch.zeros_like(share)
    size.scatter_add_(1, torch.where(kept, experts, 0), torch.where(kept, weights.double().abs(), 0.0))
    used = torch.zeros_like(share, dtype=torch.bool)
    used.scatter_(1, torch.where(kept, experts, 0), kept) if experts.numel() else None
    for e in range(num):
        tok = torch.nonzero((torch.where(kept, experts, -1) == e).any(1)).squeeze(1)
        if not tok.numel():
            continue
        a, atol, _, _ = linear_reference(m1[0][e], m1[1][e], x[tok], None, act, None, F32)
        w, wsize = share[tok, e].unsqueeze(1), size[tok, e].unsqueeze(1)
        a, atol = a * w, atol * w.abs() + 2.0 ** -21 * a.abs() * wsize
        atol = atol + 2.0 ** -8 * (a.abs() + atol)                 # rounded to bf16
        v = values(m2[0][e], m2[1][e])
        out.index_add_(0, tok, a @ v.t().contiguous())
        off = atol + (v.shape[1] + 8) * 2.0 ** -24 * (a.abs() + atol)
        tol.index_add_(0, tok, off @ v.abs().t().contiguous())
    # the sums of a token's experts, and of the waves, in fp32
    tol = tol + (experts.shape[1] + 24) * 2.0 ** -24 * (out.abs() + tol)
    if residual is not None:
        out = out + residual.double()
        tol = tol + 2.0 ** -23 * (out.abs() + residual.double().abs())
    return out, tol * (1 + HALF[dtype]) + HALF[dtype] * out.abs() + 1e-30


def run_moe(t, k, e, h, i, act="swiglu", residual=False, dtype=BF, seed=0, experts=None):
    m1 = matrix(2 * i if act in GATED else i, h, seed + 1, lead=(e,))
    m2 = matrix(h, i, seed + 2, lead=(e,))
    x = rand((t, h), seed + 3)
    if experts is None:
        experts = torch.rand((t, e), device=DEV, generator=gen(seed + 4)).argsort(1)[:, :k].contiguous()
    weights = rand(experts.shape, seed + 5, F32)
    r = rand((t, h), seed + 6, dtype) if residual else None
    obuf, out = alloc((t, h), dtype, DEV)
    need = nf4.moe_mlp_workspace_bytes(e, h, i, t, experts.shape[1], act)
    wbuf, ws = alloc((need,), torch.uint8, DEV)
    nf4.nf4_moe_mlp(*m1, *m2, x, experts, weights, out, act, r, ws)
    want, tol = moe_reference(m1, m2, x, experts, weights, act, r, dtype)
    inside(out, want, tol, f"experts {t}x{k} of {e}, {h} x {i} {act}")
    check(obuf, "out")
    check(wbuf, "workspace")
    return m1, m2, x, experts, weights, out


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,k,e", [(1, 1, 1), (1, 2, 8), (5, 2, 8), (17, 2, 3), (40, 3, 8), (64, 4, 16)])
def test_moe_acts(t, k, e, act):
    run_moe(t, k, e, 96, 64, act, residual=t % 2 == 0, seed=t)


@pytest.mark.parametrize("t,k,e,h,i", [(1, 8, 128, 2048, 768), (19, 8, 128, 256, 96), (64, 2, 128, 512, 160),
                                       (64, 1, 512, 32, 32), (64, 8, 8, 1024, 32), (64, 2, 8, 512, 4096),
                                       (2, 2, 4, 32, 14336), (3, 4, 6, 8192, 32), (33, 2, 16, 544, 1056),
                                       (64, 512, 512, 32, 32), (5, 2, 8, 4640, 544), (1, 1, 4, 8192, 512), (3, 2, 8, 4640, 544), (1, 8, 16, 7168, 96), (16, 16, 16, 160, 224), (1, 1, 2, 4096, 8224),
                                       (48, 40, 64, 64, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_moe_shapes(t, k, e, h, i, dtype):
    run_moe(t, k, e, h, i, residual=dtype == F32, dtype=dtype, seed=h)


@pytest.mark.parametrize("t,e", [(4, 8), (64, 8), (64, 64)])
def test_moe_routing(t, e):
    """All tokens on one expert, a token on one expert twice, slots and tokens without one."""
    one = torch.full((t, 2), e - 1, device=DEV)
    run_moe(t, 2, e, 64, 96, experts=one, seed=1)
    twice = torch.randint(0, e, (t, 1), device=DEV, generator=gen(2)).expand(t, 3).contiguous()
    twice[:, 1] = (twice[:, 1] + 1) % e
    run_moe(t, 3, e, 64, 96, experts=twice, residual=True, seed=2)
    some = torch.randint(-1, e + 1, (t, 4), device=DEV, generator=gen(3))
    some[0], some[t - 1, 1:] = -1, torch.tensor([1 << 40, -(1 << 40), e], device=DEV)
    for residual in (False, True):
        run_moe(t, 4, e, 64, 96, experts=some, residual=residual, seed=3)
    none = torch.full((t, 2), -1, device=DEV)
    out = run_moe(t, 2, e, 64, 96, experts=none, seed=4)[-1]
    assert (out == 0).all()


def test_moe_is_the_layer_of_its_parts():
    """The layer as sort, gather, products, activation and combine give it."""
    t, k, e, h, i = 24, 2, 8, 256, 512
    m1, m2, x, experts, weights, out = run_moe(t, k, e, h, i, dtype=F32)
    offsets, _, place = nf4.moe_sort(experts, e)
    z = nf4.mx_gemm_grouped(*m1, nf4.moe_gather(x, place), offsets)
    gate, up = z.chunk(2, dim=1)
    a = (torch.nn.functional.silu(gate) * up).to(BF)
    y = nf4.moe_combine(nf4.mx_gemm_grouped(*m2, a, offsets), place, weights)
    want, tol = moe_reference(m1, m2, x, experts, weights, "swiglu", None, F32)
    inside(y, want, tol, "parts")
    inside(out, want, tol, "whole")


def test_moe_infinite_expert_stays_with_its_tokens():
    t, k, e, h, i = 6, 2, 8, 64, 64
    for n in (6, 64):
        m1, m2 = matrix(2 * i, h, 1, lead=(e,)), matrix(h, i, 2, lead=(e,))
        m1[1][3, 5, 0] = 255                                   # a NaN row of expert 3
        x = rand((n, h), 3)
        x[2, 7] = float("inf")
        experts = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7], [3, 0], [1, 2]], device=DEV)
        experts = experts.repeat(11, 1)[:n].contiguous()
        x[8:] = x[8:].clamp(-3, 3)
        weights = torch.ones((n, 2), device=DEV)
        out = nf4.moe_mlp(*m1, *m2, x, experts, weights)
        bad = (experts == 3).any(1)
        bad[2] = True
        assert torch.equal(torch.isnan(out).any(1), bad)


def test_moe_no_tokens():
    m1, m2 = matrix(64, 32, 1, lead=(4,)), matrix(32, 32, 2, lead=(4,))
    out = nf4.moe_mlp(*m1, *m2, torch.empty((0, 32), dtype=BF, device=DEV),
                      torch.empty((0, 2), dtype=torch.int64, device=DEV), torch.empty((0, 2), device=DEV))
    assert out.shape == (0, 32)
