"""MXFP4 on the GPU against 64-bit definitions: quantising and unpacking bit for
bit, the products (bf16 rows, packed rows, grouped by expert and the gradient)
within the bound of fp32 sums of exact products, over sizes at which tiles, steps
and blocks end inside; NaN, infinities, extreme scales, streams, graphs."""
import pytest
import torch

import gpu_guard
import mx_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def nf4():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    import dequant_gemv_nf4_amd as m
    m._lib._load()
    return m


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, seed, dtype=F32, sigma=1.0):
    return (sigma * torch.randn(shape, generator=gen(seed), device=DEV)).to(dtype)


def packed(shape, seed, lo=118, hi=132):
    """Random codes and scale bytes of a matrix or a stack of matrices [.., N, K]."""
    *lead, K = shape
    codes = torch.randint(0, 256, (*lead, K // 2), generator=gen(seed), device=DEV,
                          dtype=torch.uint8)
    scales = torch.randint(lo, hi, (*lead, K // 32), generator=gen(seed + 1), device=DEV,
                           dtype=torch.uint8)
    return codes, scales


# ------------------------------------------------------ quantise, unpack ----
def check_pack(nf4, W):
    N, K = W.shape
    cb, codes = gpu_guard.alloc((N, K // 2), torch.uint8, DEV)
    sb, scales = gpu_guard.alloc((N, K // 32), torch.uint8, DEV)
    status = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    nf4.nf4_mx_pack(W, codes, scales, status)
    torch.cuda.synchronize()
    rc, rs, bad = ref.quantise(W.cpu())
    assert torch.equal(scales.cpu(), rs)
    assert torch.equal(codes.cpu(), rc)
    assert int(status) == (nf4.PACK_NONFINITE if bad else 0)
    gpu_guard.check(cb, "codes")
    gpu_guard.check(sb, "scales")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,K", [(1, 32), (3, 96), (17, 4096), (129, 160), (2, 32768), (700, 2080)])
def test_pack_bit_exact(nf4, N, K, dtype):
    check_pack(nf4, normal((N, K), N * 7 + K, dtype, 0.02))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_pack_extremes_and_ties(nf4, dtype):
    """Blocks of zeros and of -0, subnormals, the largest finite values, the
    smallest power of two that still scales, and every rounding tie at 12 scales."""
    rows = [torch.zeros(32), torch.full((32,), -0.0), torch.full((32,), 2.0 ** -133),
            torch.full((32,), 2.0 ** -126), torch.full((32,), 2.0 ** -125),
            torch.full((32,), torch.finfo(dtype).max), torch.linspace(-1, 1, 32) * 2.0 ** -130]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    step = 2.0 ** -7 if dtype == BF else 2.0 ** -23
    around = torch.cat([ties, ties * (1 + step), ties * (1 - step), -ties])
    for e in (-126, -125, -100, -20, -3, -1, 0, 1, 7, 60, 100, 124):
        rows.append(around.double().mul(2.0 ** e).float())
    check_pack(nf4, torch.stack(rows).to(dtype).to(DEV))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_pack_flags_nonfinite_blocks_only(nf4, dtype, value):
    W = normal((5, 192), 3, dtype)
    W[2, 70] = value
    W[4, 191] = value
    check_pack(nf4, W)
    with pytest.raises(ValueError, match="flagged"):
        nf4.mx_pack(W)
    codes, scales = nf4.mx_pack(W, check=False)
    out = nf4.mx_unpack(codes, scales)
    bad = torch.isnan(out)
    assert int(bad.sum()) == 64 and bool(bad[2, 64:96].all()) and bool(bad[4, 160:].all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_unpack_every_code_at_every_scale(nf4, dtype):
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8, device=DEV).reshape(256, 1).repeat(1, 16)
    buf, out = gpu_guard.alloc((256, 512), dtype, DEV)
    nf4.nf4_mx_unpack(codes, scales, out)
    torch.cuda.synchronize()
    want = ref.values(codes, scales)
    got = out.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    # beyond the type's range: infinity
    top = torch.finfo(F32).max
    want = torch.where(want.abs() > top, torch.sign(want) * float("inf"), want)
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    gpu_guard.check(buf)


def test_pack_beyond_32_bit_offsets(nf4):
    """A matrix of more than 2^32 bytes, packed and unpacked: its last rows."""
    N, K, last = 70000, 32768, 3
    W = torch.zeros((N, K), dtype=BF, device=DEV)
    assert W.numel() * 2 > 1 << 32
    W[-last:] = normal((last, K), 5, BF)
    codes, scales = nf4.mx_pack(W)
    rc, rs, _ = ref.quantise(W[-last:].cpu())
    assert torch.equal(codes[-last:].cpu(), rc) and torch.equal(scales[-last:].cpu(), rs)
    assert not bool(codes[:-last].any()) and not bool(scales[:-last].any())
    nf4.nf4_mx_unpack(codes, scales, W)
    assert torch.equal(W[-last:].double(), ref.values(codes[-last:], scales[-last:]))


# ------------------------------------------------------------- products ----
MS = [1, 2, 15, 16, 17, 33, 64, 65, 129, 300]
SHAPES = [(1, 32), (15, 64), (17, 96), (100, 1056), (257, 512), (512, 4128), (2048, 384), (36, 14336)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", MS)
def test_gemm(nf4, M, N, K):
    codes, scales = packed((N, K), 11 * M + N + K)
    X = normal((M, K), M + K, BF)
    want, mag = ref.product(X, ref.values(codes, scales))
    for dtype in (F32, BF):
        buf, Y = gpu_guard.alloc((M, N), dtype, DEV)
        nf4.nf4_mx_gemm(codes, scales, X, Y)
        torch.cuda.synchronize()
        gpu_guard.check(buf)
        ref.close(Y, want, mag, K, f"M={M} N={N} K={K} {dtype}")


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", MS)
def test_gemm_packed(nf4, M, N, K):
    codes, scales = packed((N, K), 13 * M + N + K)
    xcodes, xscales = packed((M, K), 17 * M + N + K)
    want, mag = ref.product(ref.values(xcodes, xscales), ref.values(codes, scales))
    for dtype in (F32, BF):
        buf, Y = gpu_guard.alloc((M, N), dtype, DEV)
        nf4.nf4_mx_gemm_packed(codes, scales, xcodes, xscales, Y)
        torch.cuda.synchronize()
        gpu_guard.check(buf)
        ref.close(Y, want, mag, K, f"M={M} N={N} K={K} {dtype}")


def test_gemm_of_a_vector_and_of_an_unaligned_scale_view(nf4):
    codes, scales = packed((100, 256), 5)
    x = normal((256,), 6, BF)
    assert nf4.mx_gemm(codes, scales, x).shape == (100,)
    flat = torch.empty(scales.numel() + 1, dtype=torch.uint8, device=DEV)
    view = flat[1:].view_as(scales)
    view.copy_(scales)
    for M in (1, 40, 200):
        X = normal((M, 256), M, BF)
        assert torch.equal(nf4.mx_gemm(codes, view, X), nf4.mx_gemm(codes, scales, X))
        xc, xs = nf4.mx_pack(X)
        assert torch.equal(nf4.mx_gemm_packed(codes, view, xc, xs),
                           nf4.mx_gemm_packed(codes, scales, xc, xs))


@pytest.mark.parametrize("M", [3, 40, 150])
def test_nan_and_infinity_stay_in_their_row_and_column(nf4, M):
    N, K = 70, 224
    codes, scales = packed((N, K), 21)
    scales[33, 2] = 255
    X = normal((M, K), 22, BF)
    X[1, 5] = float("nan")
    X[2, 223] = float("inf")
    Y = nf4.mx_gemm(codes, scales, X)
    nan = torch.isnan(Y)
    assert bool(nan[1].all()) and bool(nan[:, 33].all())
    rest = torch.ones(M, dtype=torch.bool, device=DEV)
    rest[1:3] = False
    clean = Y[rest][:, torch.arange(N, device=DEV) != 33]
    assert bool(torch.isfinite(clean).all())
    # an infinite input: +-inf by the weight's sign, NaN at a weight of zero
    v = ref.values(codes, scales)[:, 223]
    row = Y[2].double()
    pos = (v > 0) & ~torch.isnan(ref.values(codes, scales)).any(1)
    assert bool((row[pos] == float("inf")).all())
    xc, xs = nf4.mx_pack(X, check=False)
    P = nf4.mx_gemm_packed(codes, scales, xc, xs)
    assert bool(torch.isnan(P[1:3]).all()) and bool(torch.isnan(P[:, 33]).all())
    assert bool(torch.isfinite(P[rest][:, torch.arange(N, device=DEV) != 33]).all())


@pytest.mark.parametrize("K", [32, 96, 128, 224, 384, 416, 640])
@pytest.mark.parametrize("M", [1, 3, 20, 40, 100, 600])
def test_nan_scale_next_to_a_row_that_ends_inside_a_step(nf4, M, K):
    """Every second weight row NaN from its first block on, and every second row of
    X: the rows between, whose last step ends inside their neighbour, stay clean."""
    N = 512
    codes, scales = packed((N, K), K)
    scales[1::2] = 255
    X = normal((M, K), M, BF)
    X[1::2] = float("nan")
    want, mag = ref.product(X[0::2], ref.values(codes, scales)[0::2])
    Y = nf4.mx_gemm(codes, scales, X)
    ref.close(Y[0::2, 0::2].contiguous(), want, mag, K)
    assert bool(torch.isnan(Y[:, 1::2]).all()) and bool(torch.isnan(Y[1::2]).all())
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    G = nf4.mx_gemm_grouped(codes[None], scales[None], X, off)
    ref.close(G[0::2, 0::2].contiguous(), want, mag, K)
    # the gradient: NaN columns stay apart (the sum runs over the rows)
    codes, scales = packed((64, K), K + 1)
    scales[:, K // 64:] = 255
    dY = normal((M, 64), M, BF)
    dY[1::2] = float("nan")
    v = ref.values(codes, scales)
    clean = K // 64 * 32
    dX = nf4.mx_gemm_grouped_grad(codes[None], scales[None], dY, off)
    want, mag = ref.product(dY[0::2], v[:, :clean].t())
    ref.close(dX[0::2, :clean].contiguous(), want, mag, 64)
    assert bool(torch.isnan(dX[:, clean:]).all())


@pytest.mark.parametrize("M", [2, 40, 150])
def test_extreme_scales(nf4, M):
    """Weights near the smallest scale times large activations, and the reverse:
    no product is flushed."""
    N, K = 40, 128
    for lo, hi, sx in ((0, 3, 2.0 ** 100), (245, 248, 2.0 ** -100)):
        codes, scales = packed((N, K), lo + 1, lo, hi)
        X = normal((M, K), 9, F32).mul(sx).to(BF)
        want, mag = ref.product(X, ref.values(codes, scales))
        ref.close(nf4.mx_gemm(codes, scales, X), want, mag, K)
        off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
        dY = normal((M, N), 10, F32).mul(sx).to(BF)
        v = ref.values(codes, scales)
        want, mag = ref.product(dY, v.t())
        ref.close(nf4.mx_gemm_grouped_grad(codes[None], scales[None], dY, off), want, mag, N)


# -------------------------------------------------------------- grouped ----
def offsets_of(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


COUNTS = [([1], 0), ([0, 0, 0], 5), ([3, 0, 1, 0], 0), ([17, 64, 0, 1, 130], 3),
          ([0] * 70 + [5, 9], 2), ([2] * 130, 0), ([300, 1, 0, 33], 0), ([0, 1000], 17),
          ([128, 256, 64], 0)]


@pytest.mark.parametrize("counts,tail", COUNTS, ids=lambda v: str(v) if isinstance(v, int) else
                         f"{len(v)}x{sum(v)}")
@pytest.mark.parametrize("N,K", [(24, 64), (264, 288), (520, 1120)])
def test_grouped_and_gradient(nf4, counts, tail, N, K):
    E, R = len(counts), sum(counts) + tail
    codes, scales = packed((E, N, K), E + R + N)
    off = offsets_of(counts)
    X, dY = normal((R, K), 31, BF), normal((R, N), 32, BF)
    for dtype in (F32, BF):
        buf, Y = gpu_guard.alloc((R, N), dtype, DEV)
        nf4.nf4_mx_gemm_grouped(codes, scales, X, off, Y)
        buf2, dX = gpu_guard.alloc((R, K), dtype, DEV)
        nf4.nf4_mx_gemm_grouped_grad(codes, scales, dY, off, dX)
        torch.cuda.synchronize()
        gpu_guard.check(buf)
        gpu_guard.check(buf2)
        a = 0
        for e, c in enumerate(counts):
            v = ref.values(codes[e], scales[e])
            want, mag = ref.product(X[a:a + c], v)
            ref.close(Y[a:a + c], want, mag, K, f"expert {e}")
            want, mag = ref.product(dY[a:a + c], v.t())
            ref.close(dX[a:a + c], want, mag, N, f"gradient of expert {e}")
            a += c
        assert not bool(Y[a:].any()) and not bool(dX[a:].any())


@pytest.mark.parametrize("R", [7, 8, 9, 10])
@pytest.mark.parametrize("counts", ["spread", "pairs", "one"])
def test_grouped_around_the_rows_of_one_grid_group(nf4, counts, R):
    """As many row tiles as share an XCD and one more or less: rows of experts of their
    own, in pairs, and all of one expert."""
    E, N, K = 12, 264, 288
    codes, scales = packed((E, N, K), R)
    at = {"spread": list(range(R)), "pairs": [2 + i // 2 for i in range(R)], "one": [5] * R}[counts]
    X = normal((R, K), 41, BF)
    Y = nf4.mx_gemm_grouped(codes, scales, X, offsets_of([at.count(e) for e in range(E)]))
    for i, e in enumerate(at):
        want, mag = ref.product(X[i:i + 1], ref.values(codes[e], scales[e]))
        ref.close(Y[i:i + 1], want, mag, K, f"row {i}")


def test_grouped_without_rows(nf4):
    codes, scales = packed((3, 32, 64), 1)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert nf4.mx_gemm_grouped(codes, scales, torch.empty((0, 64), dtype=BF, device=DEV),
                               off).shape == (0, 32)
    assert nf4.mx_gemm_grouped_grad(codes, scales, torch.empty((0, 32), dtype=BF, device=DEV),
                                    off).shape == (0, 64)


@pytest.mark.parametrize("R", [9, 100])
def test_grouped_holds_bad_offsets_inside_the_arrays(nf4, R):
    """Offsets below 0, past R and descending: nothing outside the outputs is
    written (what is inside is unspecified)."""
    codes, scales = packed((4, 48, 96), 2)
    off = torch.tensor([-7, 3, 1 << 30, 2, R + 50], dtype=torch.int32, device=DEV)
    buf, Y = gpu_guard.alloc((R, 48), F32, DEV)
    nf4.nf4_mx_gemm_grouped(codes, scales, normal((R, 96), 1, BF), off, Y)
    buf2, dX = gpu_guard.alloc((R, 96), F32, DEV)
    nf4.nf4_mx_gemm_grouped_grad(codes, scales, normal((R, 48), 1, BF), off, dX)
    torch.cuda.synchronize()
    gpu_guard.check(buf)
    gpu_guard.check(buf2)


@pytest.mark.parametrize("R", [12, 90, 400])
def test_gradient_is_the_difference_quotient(nf4, R):
    """Small whole numbers: every sum is exact, so the difference of the forward
    product along a direction equals the gradient's inner product exactly."""
    E, N, K = 3, 40, 96
    g = gen(R)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.full((E, N, K // 32), 128, dtype=torch.uint8, device=DEV)  # whole values
    whole = lambda *s: torch.randint(-3, 4, s, generator=g, device=DEV).to(BF)  # noqa: E731
    X, V, dY = whole(R, K), whole(R, K), whole(R, N)
    off = offsets_of([R // 2, 0, R - R // 2])
    dX = nf4.mx_gemm_grouped_grad(codes, scales, dY, off)
    up = nf4.mx_gemm_grouped(codes, scales, X + V, off)
    down = nf4.mx_gemm_grouped(codes, scales, X - V, off)
    lhs = (dY.double() * (up.double() - down.double())).sum() / 2
    rhs = (dX.double() * V.double()).sum()
    assert float(lhs) == float(rhs)


def test_stack_beyond_32_bit_offsets(nf4):
    """The last expert of a stack of more than 4 GiB of codes."""
    E, N, K = 45, 14336, 14336
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    assert codes.numel() > 1 << 32
    c, s = packed((N, K), 77)
    codes[-1], scales[-1] = c, s
    v = ref.values(c, s)
    for R in (5, 70):
        off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        off[-1] = R
        X, dY = normal((R, K), R, BF), normal((R, N), R + 1, BF)
        want, mag = ref.product(X, v)
        ref.close(nf4.mx_gemm_grouped(codes, scales, X, off), want, mag, K)
        want, mag = ref.product(dY, v.t())
        ref.close(nf4.mx_gemm_grouped_grad(codes, scales, dY, off), want, mag, N)


@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_extreme_scales_of_two_packed_matrices(nf4, M):
    """The smallest scales times the largest, either way round, and both in the middle."""
    N, K = 70, 256
    for lo, slo in ((0, 250), (250, 0), (127, 127)):
        codes, scales = packed((N, K), lo + 1, lo, lo + 4)
        xcodes, xscales = packed((M, K), slo + 2, slo, slo + 4)
        want, mag = ref.product(ref.values(xcodes, xscales), ref.values(codes, scales))
        ref.close(nf4.mx_gemm_packed(codes, scales, xcodes, xscales), want, mag, K, f"{lo} {slo}")


@pytest.mark.parametrize("M", [1, 2, 20, 300])
def test_subnormal_rows(nf4, M):
    """Rows of bf16 subnormals times weights that bring them back to ordinary values."""
    N, K = 50, 160
    codes, scales = packed((N, K), 3, 240, 245)
    X = (normal((M, K), 4).sign() * 2.0 ** -130).to(BF)
    assert bool((X != 0).all()) and float(X.float().abs().max()) < 2.0 ** -126
    want, mag = ref.product(X, ref.values(codes, scales))
    ref.close(nf4.mx_gemm(codes, scales, X), want, mag, K)
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    dY = (normal((M, 48), 4).sign() * 2.0 ** -130).to(BF)
    codes, scales = packed((48, K), 3, 240, 245)
    want, mag = ref.product(dY, ref.values(codes, scales).t())
    ref.close(nf4.mx_gemm_grouped_grad(codes[None], scales[None], dY, off), want, mag, 48)


def within(got, want, mag, terms):
    """(terms + 8) (2^-24 of the magnitudes + 2^-149), and half a unit of bf16."""
    tol = (terms + 8) * (2.0 ** -24 * mag + 2.0 ** -149)
    if got.dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + torch.clamp(2.0 ** -8 * want.abs(), min=2.0 ** -134)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3g} x tolerance"


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("size", [-165, -150, -140, -126, -100])
@pytest.mark.parametrize("M", [1, 2, 3, 40, 300])
def test_sums_near_the_smallest_numbers(nf4, M, size, dtype):
    """Products around 2^size: below 2^-126 they are rounded to multiples of 2^-149, and
    neither they nor their sums are flushed."""
    N, K = 264, 160
    half = size // 2
    codes, scales = packed((N, K), size % 97, 126 + half, 129 + half)
    X = normal((M, K), 4).mul(2.0 ** (size - half)).to(BF)
    dY = normal((M, N), 5).mul(2.0 ** (size - half)).to(BF)
    v = ref.values(codes, scales)
    within(nf4.mx_gemm(codes, scales, X, out_dtype=dtype), *ref.product(X, v), K)
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    within(nf4.mx_gemm_grouped(codes[None], scales[None], X, off, out_dtype=dtype),
           *ref.product(X, v), K)
    within(nf4.mx_gemm_grouped_grad(codes[None], scales[None], dY, off, out_dtype=dtype),
           *ref.product(dY, v.t()), N)
    xc, xs = nf4.mx_pack(X)
    within(nf4.mx_gemm_packed(codes, scales, xc, xs, out_dtype=dtype),
           *ref.product(ref.values(xc, xs), v), K)


@pytest.mark.parametrize("M", [1, 2, 3, 40, 300])
def test_scales_beyond_what_packing_writes(nf4, M):
    """s = 253 and 254: values of 2^128 and more are infinite with bf16 rows and finite
    between two packed matrices; up to s = 252 all are finite."""
    N, K = 264, 160
    X = normal((M, K), 4).mul(2.0 ** -20).to(BF)
    X[-1, 66] = 0.0
    dY = normal((M, N), 5).mul(2.0 ** -20).to(BF)
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    xc, xs = nf4.mx_pack(X)
    for s in (252, 253, 254):
        codes, scales = packed((N, K), s, 100, 110)
        codes &= 0x33  # magnitudes up to 1.5
        scales[:] = 240
        scales[5, 2] = s
        codes[5, 33] = 0x67 if s == 252 else 0x06 if s == 253 else 0x04  # 6, 4; 4; 2
        v = ref.values(codes, scales)
        u = ref.values(xc, xs)
        want, mag = ref.product(u, v)
        within(nf4.mx_gemm_packed(codes, scales, xc, xs), want, mag, K)
        big = v.abs() >= 2.0 ** 128
        assert int(big.sum()) == (0 if s == 252 else 1)
        v = torch.where(big, torch.sign(v) * float("inf"), v)
        for Y in (nf4.mx_gemm(codes, scales, X),
                  nf4.mx_gemm_grouped(codes[None], scales[None], X, off)):
            inf = big.any(1)
            want, mag = ref.product(X, v[~inf])
            within(Y[:, ~inf], want, mag, K)
            if s > 252:  # the sign of the one infinite product; NaN where x is zero
                x = X[:, big[5]].reshape(-1).double()
                want = torch.where(x == 0, float("nan"), torch.sign(x) * float("inf"))
                assert torch.equal(Y[:, 5].double().nan_to_num(7.0), want.nan_to_num(7.0))
        dX = nf4.mx_gemm_grouped_grad(codes[None], scales[None], dY, off)
        inf = big.any(0)
        want, mag = ref.product(dY, v[:, ~inf].t())
        within(dX[:, ~inf], want, mag, N)
        if s > 252:
            want = torch.sign(dY[:, 5].double()) * float("inf")
            assert torch.equal(dX[:, inf].reshape(-1).double(), want)


@pytest.mark.parametrize("M", [1, 2, 4, 5, 70, 400])
def test_longest_rows(nf4, M):
    """K = 32768 (sixteen chunks of the row kernel), and a gradient over many rows of
    a narrow matrix."""
    N, K = 37, 32768
    codes, scales = packed((N, K), 1)
    X = normal((M, K), 2, BF)
    want, mag = ref.product(X, ref.values(codes, scales))
    ref.close(nf4.mx_gemm(codes, scales, X), want, mag, K)
    off = torch.tensor([0, M, M, M], dtype=torch.int32, device=DEV)
    three = [t.expand(3, *t.shape).contiguous() for t in (codes, scales)]
    ref.close(nf4.mx_gemm_grouped(*three, X, off), want, mag, K)
    N, K = (1 << 18) + 8, 64
    codes, scales = packed((N, K), 3)
    dY = normal((M, N), 4, BF)
    want, mag = ref.product(dY, ref.values(codes, scales).t())
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    ref.close(nf4.mx_gemm_grouped_grad(codes[None], scales[None], dY, off), want, mag, N)


@pytest.mark.parametrize("nan", [False, True])
@pytest.mark.parametrize("K", [32, 96, 128, 224, 640, 1056])
def test_largest_tiles(nf4, K, nan):
    """Enough rows and columns for the largest tiles, the last of each cut short; with
    `nan`, every second row of either side."""
    M, N = 3000, 4204
    codes, scales = packed((N, K), K)
    X = normal((M, K), K + 1, BF)
    if nan:
        scales[1::2] = 255
        X[1::2] = float("nan")
    xc, xs = nf4.mx_pack(X, check=False)
    u, v = nf4.mx_unpack(xc, xs), ref.values(codes, scales)
    for rows, call in ((X, lambda Y: nf4.nf4_mx_gemm(codes, scales, X, Y)),
                       (u, lambda Y: nf4.nf4_mx_gemm_packed(codes, scales, xc, xs, Y))):
        step = 2 if nan else 1
        want, mag = ref.product(rows[::step], v[::step])
        for dtype in (F32, BF):
            buf, Y = gpu_guard.alloc((M, N), dtype, DEV)
            call(Y)
            torch.cuda.synchronize()
            gpu_guard.check(buf)
            ref.close(Y[::step, ::step].contiguous(), want, mag, K, f"K={K} {dtype}")
            assert not nan or bool(torch.isnan(Y[1::2]).all() and torch.isnan(Y[:, 1::2]).all())


@pytest.mark.parametrize("K", [1024, 2016, 3040])
@pytest.mark.parametrize("N", [8, 72, 264, 1032])
def test_gradient_of_many_rows(nf4, N, K):
    """The tiles of 64 rows, with and without N shared out, N ending inside a stage."""
    counts = [1900, 0, 1100, 37]
    R = sum(counts) + 5
    codes, scales = packed((4, N, K), N + K)
    dY = normal((R, N), N, BF)
    off = offsets_of(counts)
    for dtype in (F32, BF):
        buf, dX = gpu_guard.alloc((R, K), dtype, DEV)
        nf4.nf4_mx_gemm_grouped_grad(codes, scales, dY, off, dX)
        torch.cuda.synchronize()
        gpu_guard.check(buf)
        a = 0
        for e, c in enumerate(counts):
            want, mag = ref.product(dY[a:a + c], ref.values(codes[e], scales[e]).t())
            ref.close(dX[a:a + c], want, mag, N, f"expert {e}")
            a += c
        assert not bool(dX[a:].any())


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("N", [64, 72, 104])
@pytest.mark.parametrize("K,counts", [(96, [3, 0, 5]), (256, [20, 40]), (2016, [450, 450]),
                                      (2048, [900, 0, 900]), (2016, [1300, 1300]),
                                      (2048, [2100, 2100]), (2048, [10] * 60)],
                         ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}x{sum(v)}")
def test_grouped_with_unaligned_scales_between_nan_bytes(nf4, K, counts, N, shift):
    """Scales at any byte, all bytes around them 255 and each expert but the first
    beginning with a NaN row: the tiles of every size, stages that N ends in and K-groups
    whose share is past N keep to the matrix, and NaN to its row and columns."""
    E, R = len(counts), sum(counts)
    codes, aligned = packed((E, N, K), K + N + shift)
    aligned[1:, 0, :2] = 255
    flat = torch.full((256 + aligned.numel() + 8192,), 255, dtype=torch.uint8, device=DEV)
    scales = flat[256 + shift:256 + shift + aligned.numel()].view_as(aligned)
    scales.copy_(aligned)
    off = offsets_of(counts)
    X, dY = normal((R, K), 61, BF), normal((R, N), 62, BF)
    buf, Y = gpu_guard.alloc((R, N), F32, DEV)
    nf4.nf4_mx_gemm_grouped(codes, scales, X, off, Y)
    buf2, dX = gpu_guard.alloc((R, K), F32, DEV)
    nf4.nf4_mx_gemm_grouped_grad(codes, scales, dY, off, dX)
    torch.cuda.synchronize()
    gpu_guard.check(buf)
    gpu_guard.check(buf2)
    a = 0
    for e, c in enumerate(counts):
        v = ref.values(codes[e], scales[e])
        first, cols = (1, 64) if e else (0, 0)  # rows of the matrix and columns that are NaN
        want, mag = ref.product(X[a:a + c], v[first:])
        ref.close(Y[a:a + c, first:], want, mag, K, f"expert {e}")
        want, mag = ref.product(dY[a:a + c], v[:, cols:].t())
        ref.close(dX[a:a + c, cols:], want, mag, N, f"gradient of expert {e}")
        assert bool(torch.isnan(Y[a:a + c, :first]).all())
        assert bool(torch.isnan(dX[a:a + c, :cols]).all())
        a += c


@pytest.mark.parametrize("K", [160, 1152])
@pytest.mark.parametrize("M,N", [(2, 5001), (4, 5001), (10, 5001), (16, 8200), (10, 9001),
                                 (10, 25000), (40, 7001), (17, 14001), (40, 28672), (50, 28675),
                                 (100, 14001), (500, 6300), (300, 20004)])
def test_every_tile_of_the_product(nf4, M, N, K):
    """Rows and columns on each side of the sizes at which another tile is taken."""
    codes, scales = packed((N, K), M + N)
    X = normal((M, K), 3, BF)
    want, mag = ref.product(X, ref.values(codes, scales))
    buf, Y = gpu_guard.alloc((M, N), F32, DEV)
    nf4.nf4_mx_gemm(codes, scales, X, Y)
    torch.cuda.synchronize()
    gpu_guard.check(buf)
    ref.close(Y, want, mag, K)
    ref.close(nf4.mx_gemm(codes, scales, X, out_dtype=BF), want, mag, K)


def test_rows_and_outputs_beyond_32_bit_offsets(nf4):
    """More than 2^32 bytes of X, of Y, of packed rows and of dX: the last rows."""
    last = 9
    N, K, M = 48, 16384, 140000
    codes, scales = packed((N, K), 1)
    v = ref.values(codes, scales)
    X = torch.zeros((M, K), dtype=BF, device=DEV)
    X[-last:] = normal((last, K), 2, BF)
    assert X.numel() * 2 > 1 << 32
    want, mag = ref.product(X[-last:], v)
    Y = nf4.mx_gemm(codes, scales, X)
    ref.close(Y[-last:], want, mag, K)
    assert not bool(Y[:-last].any())
    off = torch.tensor([0, M - last - 3, M - 2], dtype=torch.int32, device=DEV)
    two = [torch.stack([t, t]) for t in (codes, scales)]
    Y = nf4.mx_gemm_grouped(*two, X, off)
    ref.close(Y[M - last:M - 2], want[:-2], mag[:-2], K)
    assert not bool(Y[-2:].any())
    dY = torch.zeros((M, N), dtype=BF, device=DEV)
    dY[-last:] = normal((last, N), 3, BF)
    want, mag = ref.product(dY[-last:], v.t())
    dX = X
    nf4.nf4_mx_gemm_grouped_grad(*two, dY, off, dX)
    ref.close(dX[M - last:M - 2], want[:-2], mag[:-2], N)
    assert not bool(dX[-2:].any())
    del X, dX, dY, Y
    N, K, M = 65536, 64, 40000
    codes, scales = packed((N, K), 5)
    X = normal((M, K), 6, BF)
    Y = torch.empty((M, N), dtype=BF, device=DEV)
    assert Y.numel() * 2 > 1 << 32
    xc, xs = nf4.mx_pack(X)
    for rows, call in ((X, lambda: nf4.nf4_mx_gemm(codes, scales, X, Y)),
                       (nf4.mx_unpack(xc, xs), lambda: nf4.nf4_mx_gemm_packed(codes, scales, xc, xs, Y))):
        Y.fill_(float("nan"))
        call()
        want, mag = ref.product(rows[-last:], ref.values(codes, scales))
        ref.close(Y[-last:], want, mag, K)
        assert not bool(torch.isnan(Y).any())
    del Y
    K, M = 32768, 300000
    codes, scales = packed((48, K), 7)
    xc, xs = packed((M, K), 8)
    assert xc.numel() > 1 << 32
    want, mag = ref.product(ref.values(xc[-last:], xs[-last:]), ref.values(codes, scales))
    ref.close(nf4.mx_gemm_packed(codes, scales, xc, xs)[-last:], want, mag, K)


# ------------------------------------------------------ streams, graphs ----
def test_results_repeat_bit_for_bit(nf4):
    codes, scales = packed((1000, 2048), 3)
    for M in (1, 20, 300):
        X = normal((M, 2048), M, BF)
        xc, xs = nf4.mx_pack(X)
        a, b = nf4.mx_gemm(codes, scales, X), nf4.mx_gemm_packed(codes, scales, xc, xs)
        for _ in range(3):
            assert torch.equal(nf4.mx_gemm(codes, scales, X), a)
            assert torch.equal(nf4.mx_gemm_packed(codes, scales, xc, xs), b)


def test_on_another_stream(nf4):
    codes, scales = packed((500, 1024), 3)
    X = normal((70, 1024), 4, BF)
    want = nf4.mx_gemm(codes, scales, X)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    W = normal((64, 1024), 8)
    got = nf4.mx_gemm(codes, scales, X, stream=side)
    c, s = nf4.mx_pack(W, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    rc, rs, _ = ref.quantise(W.cpu())
    assert torch.equal(c.cpu(), rc) and torch.equal(s.cpu(), rs)


@pytest.mark.parametrize("M", [1, 30, 200])
def test_captured_and_replayed_with_new_inputs(nf4, M):
    N, K = 300, 512
    codes, scales = packed((N, K), 3)
    X = normal((M, K), 4, BF)
    xc = torch.empty((M, K // 2), dtype=torch.uint8, device=DEV)
    xs = torch.empty((M, K // 32), dtype=torch.uint8, device=DEV)
    Y, P = torch.empty((M, N), device=DEV), torch.empty((M, N), device=DEV)
    off = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    G = torch.empty((M, N), device=DEV)

    def step():
        nf4.nf4_mx_gemm(codes, scales, X, Y)
        nf4.nf4_mx_pack(X, xc, xs)
        nf4.nf4_mx_gemm_packed(codes, scales, xc, xs, P)
        nf4.nf4_mx_gemm_grouped(codes[None], scales[None], X, off, G)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        X.copy_(normal((M, K), 50 + i, BF))
        graph.replay()
        torch.cuda.synchronize()
        got = Y.clone(), P.clone(), G.clone()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (Y, P, G)))


def test_arguments_are_refused_by_name(nf4):
    codes, scales = packed((64, 128), 1)
    X = normal((4, 128), 1, BF)
    with pytest.raises(TypeError, match="X has dtype"):
        nf4.mx_gemm(codes, scales, X.float())
    with pytest.raises(ValueError, match="contiguous"):
        nf4.mx_gemm(codes, scales, normal((4, 256), 1, BF)[:, ::2])
    with pytest.raises(ValueError, match="columns"):
        nf4.mx_gemm(codes, scales, normal((4, 96), 1, BF))
    with pytest.raises(ValueError, match="scales"):
        nf4.mx_gemm(codes, scales[:, :3].contiguous(), X)
    with pytest.raises(ValueError, match="GPU"):
        nf4.mx_gemm(codes.cpu(), scales, X)
    with pytest.raises(TypeError):
        nf4.mx_gemm(codes, scales, X, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="K ="):
        xc, xs = nf4.mx_pack(normal((4, 96), 1))
        nf4.mx_gemm_packed(codes, scales, xc, xs)
    with pytest.raises(ValueError, match="needs scales"):
        nf4.mx_pack(normal((4, 80), 1))
    with pytest.raises(ValueError, match="offsets"):
        nf4.mx_gemm_grouped(codes[None], scales[None], X,
                            torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError, match="offsets"):
        nf4.mx_gemm_grouped(codes[None], scales[None], X, torch.zeros(2, device=DEV).long())
    with pytest.raises(nf4.NF4Error):  # N not a multiple of 8
        c, s = packed((1, 60, 64), 1)
        nf4.mx_gemm_grouped_grad(c, s, normal((4, 60), 1, BF),
                                 torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(nf4.NF4Error):  # X not 16-byte aligned
        flat = torch.zeros(4 * 128 + 1, dtype=BF, device=DEV)
        nf4.mx_gemm(codes, scales, flat[1:].view(4, 128))
