"""The fused MXFP4 operators as programs use them: together, on other streams, two at
once, captured and replayed, at the largest sizes, and their refusals."""
import pytest
import torch

import dequant_gemv_nf4_amd as nf4
from test_gpu_fused import (BF, DEV, F32, HALF, gen, inside, linear_reference, loss_reference, matrix,
                            moe_reference, rand)
from mx_reference import values

pytestmark = pytest.mark.gpu


def inputs(seed, m=70, n=4096, k=2048, vocab=40000, experts=8, inner=1024):
    a = dict(up=matrix(2 * inner, k, seed, lead=()), down=matrix(k, inner, seed + 1), head=matrix(vocab, k, seed + 2),
             w1=matrix(2 * inner, k, seed + 3, lead=(experts,)), w2=matrix(k, inner, seed + 4, lead=(experts,)),
             x=rand((m, k), seed + 5), few=rand((9, k), seed + 6), bias=rand((k,), seed + 7, F32))
    a["targets"] = torch.randint(0, vocab, (m,), device=DEV, generator=gen(seed + 8))
    a["dloss"] = rand((m,), seed + 9, F32)
    a["experts"] = torch.rand((9, experts), device=DEV, generator=gen(seed + 10)).argsort(1)[:, :2].contiguous()
    a["weights"] = rand((9, 2), seed + 11, F32).abs()
    a["dy"] = rand((m, inner), seed + 12)
    a["z"] = rand((m, 2 * inner), seed + 13)
    return a


@pytest.fixture(scope="module")
def args():
    a = inputs(1)
    torch.cuda.synchronize()
    return a


CALLS = {
    "linear": lambda a, s: nf4.mx_linear(*a["up"], a["x"], act="swiglu", keep_z=True, stream=s),
    "linear-token": lambda a, s: nf4.mx_linear(*a["head"], a["x"][0], stream=s),
    "linear_grad": lambda a, s: nf4.mx_linear_grad(*a["up"], a["dy"], a["z"], "swiglu", bias_grad=True, stream=s),
    "loss": lambda a, s: nf4.mx_cross_entropy(*a["head"], a["x"], a["targets"], stream=s),
    "loss-grad": lambda a, s: nf4.mx_cross_entropy(*a["head"], a["x"], a["targets"], a["dloss"], stream=s),
    "moe": lambda a, s: nf4.moe_mlp(*a["w1"], *a["w2"], a["few"], a["experts"], a["weights"], stream=s),
    "moe-many": lambda a, s: nf4.moe_mlp(*a["w1"], *a["w2"], a["x"][:64], a["targets"][:64, None] % 8 *
                                         torch.ones((1, 2), dtype=torch.int64, device=DEV), a["dloss"][:64, None] *
                                         torch.ones((1, 2), device=DEV), stream=s),
}


def tensors(out):
    return [t for t in out if t is not None] if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", [n for n in CALLS if n != "moe-many"])
def test_on_another_stream(args, name, raw):
    """The same bits, with work queued on the current stream whose freed blocks the call
    must not take."""
    want = [t.clone() for t in tensors(CALLS[name](args, None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.randn((4096, 4096), device=DEV)
    freed = [torch.empty_like(t) for t in want for _ in range(2)] + [torch.empty(1 << 27, dtype=torch.uint8, device=DEV)]
    for _ in range(20):
        busy = busy @ busy
    for t in freed:
        t.fill_(0)
    del t, freed
    got = tensors(CALLS[name](args, side.cuda_stream if raw else side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()


def test_two_at_once(args):
    """Every operator on two streams side by side, several times, with inputs of its own."""
    other = inputs(100)
    torch.cuda.synchronize()
    want = [[[t.clone() for t in tensors(f(a, None))] for f in CALLS.values()] for a in (args, other)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for i, f in enumerate(CALLS.values()):
            for j, a in enumerate((args, other)):
                with torch.cuda.stream(streams[j]):
                    got.append((j, i, tensors(f(a, None))))
    torch.cuda.synchronize()
    for j, i, out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want[j][i])), (j, i)


@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed(args, name):
    """Every replay against the eager call on the inputs of that time, with eager work and
    synchronizations between the replays; then two graphs of one call replayed at once."""
    a = {k: tuple(t.clone() for t in v) if isinstance(v, tuple) else v.clone() for k, v in args.items()}
    call = CALLS[name]
    call(a, None)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = tensors(call(a, None))
        graphs.append((g, out))
    for i in range(3):
        for k in ("x", "few", "dy", "z"):
            a[k].copy_(rand(a[k].shape, 1000 * i + len(k)))
        a["targets"].copy_(torch.randint(0, 40000, a["targets"].shape, device=DEV, generator=gen(i)))
        if i == 1:
            a["targets"][::3] = -100
        a["experts"].copy_(torch.randint(-1 if i == 1 else 0, 8, a["experts"].shape, device=DEV, generator=gen(i)))
        want = [t.clone() for t in tensors(call(a, None))]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(p, q) for p, q in zip(out, want)), i


def test_a_layer_and_its_loss_together():
    """One training step through the operators: gated layer, residual, head and loss, and
    back, against 64 bits; between the operators the reference takes their rounded values."""
    m, k, inner, vocab = 50, 256, 320, 3001
    up, down, head = matrix(2 * inner, k, 1), matrix(k, inner, 2), matrix(vocab, k, 3)
    x, bias = rand((m, k), 4), rand((k,), 5, F32)
    targets = torch.randint(0, vocab, (m,), device=DEV, generator=gen(6))
    targets[::4] = -100
    dloss = torch.where(targets >= 0, 1.0 / int((targets >= 0).sum()), 0.0).float()
    h, z = nf4.mx_linear(*up, x, act="swiglu", keep_z=True)
    y = nf4.mx_linear(*down, h, bias=bias, residual=x)
    loss, lse, dy = nf4.mx_cross_entropy(*head, y, targets, dloss)
    dh, dz2, dbias = nf4.mx_linear_grad(*down, dy, bias_grad=True)
    dx, dz, _ = nf4.mx_linear_grad(*up, dh, z, "swiglu", out_dtype=F32)
    dx = dx + dy.float()
    want = linear_reference(*up, x, None, "swiglu", None, BF)
    inside(h, want[0], want[1], "h")
    inside(z, want[2], want[3], "z")
    want = linear_reference(*down, h, bias, None, x, BF)
    inside(y, want[0], want[1], "y")
    want = loss_reference(*head, y, targets, dloss)
    inside(loss, want[0], want[1], "loss")
    inside(dy, want[4], want[5] * (1 + HALF[BF]) + HALF[BF] * want[4].abs() + 1e-36, "dy")
    assert dz2 is dy
    v = values(*down)
    inside(dh, dy.double() @ v, (k + 40) * 2.0 ** -23 * (dy.double().abs() @ v.abs())
           + HALF[BF] * (dy.double() @ v).abs() + 1e-36, "dh")
    inside(dbias, dy.double().sum(0), (m + 8) * 2.0 ** -24 * dy.double().abs().sum(0) + 1e-36, "dbias")
    v = values(*up)
    inside(dx, dz.double() @ v + dy.double(), (2 * inner + 40) * 2.0 ** -23 * (dz.double().abs() @ v.abs())
           + 2.0 ** -23 * dy.double().abs() + 1e-36, "dx")


def test_decode_step_together(args):
    """One token: attention output with residual, expert layer with residual, scores of the head."""
    x = args["few"][:1].contiguous()
    y = nf4.mx_linear(*args["down"], rand((1, 1024), 3), residual=x)
    out = nf4.moe_mlp(*args["w1"], *args["w2"], y, args["experts"][:1].contiguous(),
                      args["weights"][:1].contiguous(), residual=y)
    want, tol = moe_reference(args["w1"], args["w2"], y, args["experts"][:1], args["weights"][:1], "swiglu", y, BF)
    inside(out, want, tol, "experts")
    loss, lse = nf4.mx_cross_entropy(*args["head"], out, args["targets"][:1].contiguous())
    logits = nf4.mx_linear(*args["head"], out, out_dtype=F32)
    want = loss_reference(*args["head"], out, args["targets"][:1], None)
    inside(loss, want[0], want[1], "loss")
    inside(torch.logsumexp(logits.double(), 1), want[2], want[3] + 1e-6 * want[2].abs(), "logits")


# ---------------------------------------------------------------- largest sizes ----
def sampled(out, want_rows, rows, what):
    want, tol = want_rows
    inside(out[rows], want, tol, what)


def test_rows_beyond_32_bit_offsets():
    """Outputs, kept values and gradients whose byte offsets pass 2^32."""
    m, n, k = 36000, 65536, 32
    codes, scales = matrix(n, k, 1)
    x, r = rand((m, k), 2), None
    rows = torch.tensor([0, 1, 16383, 16384, 32767, 32768, 35999], device=DEV)
    y, z = nf4.mx_linear(codes, scales, x, act="silu", keep_z=True)
    want = linear_reference(codes, scales, x[rows], None, "silu", r, BF)
    inside(y[rows], want[0], want[1], "Y")
    inside(z[rows], want[2], want[3], "Z")
    dx, dz, db = nf4.mx_linear_grad(codes, scales, y, z, "silu", out_dtype=F32)
    del y
    v = values(codes, scales)
    d = dz[rows].double()
    inside(dx[rows], d @ v, (n + 40) * 2.0 ** -24 * (d.abs() @ v.abs()) + 1e-30, "dX")


def test_the_largest_head():
    m, n, k = 33, 1 << 23, 32
    codes, scales = matrix(n, k, 1)
    x = rand((m, k), 2)
    targets = torch.randint(0, n, (m,), device=DEV, generator=gen(3))
    targets[0], targets[1] = 0, n - 1
    loss, lse, dx = nf4.mx_cross_entropy(codes, scales, x, targets, torch.ones(m, device=DEV), out_dtype=F32)
    v = values(codes, scales)
    l = x.double() @ v.t().contiguous()
    ref = torch.logsumexp(l, 1)
    lt = l.gather(1, targets.unsqueeze(1)).squeeze(1)
    # sums of 2^23 terms: 2^17 strips in turn of 512 or a tree, at most 2^10 steps of fp32
    tol = 2.0 ** -13 + 2.0 ** -22 * ref.abs() + 48 * 2.0 ** -24 * l.abs().amax(1)
    inside(lse, ref, tol, "lse")
    inside(loss, ref - lt, 2 * tol, "loss")
    p = torch.exp(l - ref.unsqueeze(1))
    mag = p @ v.abs()
    want = p @ v - v[targets]
    # the parts' sums run over up to 2^23 / 128 rows each in stages of 64: 2^11 steps and a stage's 64
    inside(dx, want, mag * (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -12) + 2.0 ** -20 * want.abs(), "dX")


@pytest.mark.parametrize("t,k,e,h,i", [(64, 2, 64, 1024, 2048), (64, 4, 8, 512, 2048), (64, 4, 8, 512, 2080),
                                       (2, 2, 4, 8224, 64), (64, 2, 64, 1056, 2080), (20, 4, 8, 4128, 4096),
                                       (1, 2, 3, 96, 32768), (64, 2, 4, 16384, 64)])
def test_more_expert_shapes(t, k, e, h, i):
    from test_gpu_fused import run_moe
    run_moe(t, k, e, h, i, residual=True, seed=i)


# -------------------------------------------------------------------- refusals ----
def test_refusals_name_the_argument(args):
    up, x = args["up"], args["x"]
    inner, k = 1024, 2048
    bad = [
        (ValueError, "act is 'tanh'", lambda: nf4.mx_linear(*up, x, act="tanh")),
        (ValueError, "X has", lambda: nf4.mx_linear(*up, x[:, :64].contiguous())),
        (ValueError, "contiguous", lambda: nf4.mx_linear(*up, x.t())),
        (TypeError, "X has dtype", lambda: nf4.mx_linear(*up, x.float())),
        (ValueError, "bias must be", lambda: nf4.mx_linear(*up, x, bias=args["bias"][:5].contiguous())),
        (ValueError, "residual must be", lambda: nf4.mx_linear(*up, x, act="swiglu", residual=x)),
        (TypeError, "residual has dtype", lambda: nf4.mx_linear(*args["down"], args["dy"], residual=x, out_dtype=F32)),
        (TypeError, "out_dtype", lambda: nf4.mx_linear(*up, x, out_dtype=torch.float16)),
        (ValueError, "is odd", lambda: nf4.mx_linear(up[0][:7], up[1][:7], x, act="geglu")),
        (ValueError, "dY has", lambda: nf4.mx_linear_grad(*up, args["dy"], args["z"], "silu")),
        (ValueError, "Z must be", lambda: nf4.mx_linear_grad(*up, args["dy"], args["dy"], "swiglu")),
        (TypeError, "Z must be", lambda: nf4.mx_linear_grad(*up, args["dy"], None, "swiglu")),
        (nf4.NF4Error, "EINVAL", lambda: nf4.mx_linear_grad(up[0][:12], up[1][:12], args["z"][:, :12].contiguous())),
        (ValueError, "targets must be", lambda: nf4.mx_cross_entropy(*args["head"], x, args["targets"][:3])),
        (TypeError, "targets has dtype", lambda: nf4.mx_cross_entropy(*args["head"], x, args["targets"].int())),
        (ValueError, "dloss must be", lambda: nf4.mx_cross_entropy(*args["head"], x, args["targets"], args["dloss"][:2])),
        # no rows: an empty tensor has a null pointer, as in nf4_mx_gemm
        (nf4.NF4Error, "EINVAL", lambda: nf4.mx_cross_entropy(*args["head"], x[:0], args["targets"][:0])),
        (nf4.NF4Error, "EINVAL", lambda: nf4.mx_linear(*up, x[:0])),
        (ValueError, "up to 64 tokens", lambda: nf4.moe_mlp(*args["w1"], *args["w2"], x, args["experts"], args["weights"])),
        (ValueError, "needs codes2", lambda: nf4.moe_mlp(*args["w1"], *args["w2"], args["few"], args["experts"],
                                                        args["weights"], act="silu")),
        (ValueError, "experts must be", lambda: nf4.moe_mlp(*args["w1"], *args["w2"], args["few"][:4],
                                                           args["experts"], args["weights"])),
        (ValueError, "weights must be", lambda: nf4.moe_mlp(*args["w1"], *args["w2"], args["few"], args["experts"],
                                                           args["weights"][:, :1].contiguous())),
        (TypeError, "weights has dtype", lambda: nf4.moe_mlp(*args["w1"], *args["w2"], args["few"], args["experts"],
                                                            args["weights"].to(BF))),
    ]
    for kind, text, call in bad:
        with pytest.raises(kind, match=text):
            call()


def test_missing_and_short_workspaces(args):
    few, w = args["few"], args["weights"]
    need = nf4.moe_mlp_workspace_bytes(8, 2048, 1024, 9, 2)
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device=DEV)):
        with pytest.raises(nf4.NF4Error, match="ERANGE"):
            nf4.nf4_moe_mlp(*args["w1"], *args["w2"], few, args["experts"], w, torch.empty_like(few), workspace=ws)
    loss = torch.empty(70, device=DEV)
    with pytest.raises(nf4.NF4Error, match="ERANGE"):
        nf4.nf4_mx_cross_entropy(*args["head"], args["x"], args["targets"], loss, loss.clone())
    with pytest.raises(ValueError, match="given together"):
        nf4.nf4_mx_cross_entropy(*args["head"], args["x"], args["targets"], loss, loss.clone(), dloss=args["dloss"])
