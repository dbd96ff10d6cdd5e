"""Calls with `stream=`: the functions that allocate take their outputs' memory from
the stream they run on, so neither work still queued on the current stream nor later
allocations there share it while it is written."""
import pytest
import torch

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


@pytest.fixture(scope="module")
def args(nf4):
    """Inputs whose outputs have sizes of their own, all above the allocator's small blocks."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    E, N, K, R = 2, 4096, 2048, 1024
    W = torch.randn((N, K), generator=g, device=DEV)
    codes, scales = nf4.mx_pack(W)
    X = torch.randn((R, K), generator=g, device=DEV).to(BF)
    xc, xs = nf4.mx_pack(X)
    ids = torch.randint(0, E, (1 << 18, 4), generator=g, device=DEV)
    route = torch.randint(0, E, (R // 2, 2), generator=g, device=DEV)
    offsets, _, place = nf4.moe_sort(route, E)
    w = torch.rand((R // 2, 2), generator=g, device=DEV)
    out = dict(W=W, codes=codes, scales=scales, stack=torch.stack([codes, codes]),
               sstack=torch.stack([scales, scales]), X=X, xc=xc, xs=xs, ids=ids, offsets=offsets,
               place=place, w=w, dY=torch.randn((R, N), generator=g, device=DEV).to(BF))
    out["ncodes"], out["nscales"] = nf4.pack(W)
    out["rows"] = torch.randint(0, N, (2000,), generator=g, device=DEV)
    out["wide"] = torch.stack([out["ncodes"]] * 80).reshape(80 * N, K // 2)
    out["wscales"] = torch.stack([out["nscales"]] * 80).reshape(80 * N, K // 64)
    torch.cuda.synchronize()
    return out


CALLS = {
    "mx_pack": lambda m, a, s: m.mx_pack(a["W"], stream=s, check=False),
    "mx_unpack": lambda m, a, s: m.mx_unpack(a["codes"], a["scales"], stream=s),
    "mx_gemm": lambda m, a, s: m.mx_gemm(a["codes"], a["scales"], a["X"], stream=s),
    "mx_gemm_packed": lambda m, a, s: m.mx_gemm_packed(a["codes"], a["scales"], a["xc"], a["xs"],
                                                       stream=s),
    "mx_gemm_grouped": lambda m, a, s: m.mx_gemm_grouped(a["stack"], a["sstack"], a["X"],
                                                         a["offsets"], stream=s),
    "mx_gemm_grouped_grad": lambda m, a, s: m.mx_gemm_grouped_grad(
        a["stack"], a["sstack"], a["dY"], a["offsets"], stream=s),
    "moe_sort": lambda m, a, s: m.moe_sort(a["ids"], 2, stream=s),
    "moe_gather": lambda m, a, s: m.moe_gather(a["X"][:512], a["place"], stream=s),
    "moe_combine": lambda m, a, s: m.moe_combine(a["X"], a["place"], a["w"], stream=s),
    "moe_combine_grad": lambda m, a, s: m.moe_combine_grad(a["X"][:512], a["X"], a["place"],
                                                           a["w"], stream=s),
    "pack": lambda m, a, s: m.pack(a["W"], stream=s, check=False),
    "unpack": lambda m, a, s: m.unpack(a["ncodes"], a["nscales"], 2048, stream=s),
    "gemv": lambda m, a, s: m.gemv(a["wide"], a["wscales"], a["X"][0], stream=s),
    "gemm-small": lambda m, a, s: m.gemm(a["wide"], a["wscales"], a["X"][:8], stream=s),
    "gemm-prompt": lambda m, a, s: m.gemm(a["ncodes"], a["nscales"], a["X"], stream=s),
    "embed": lambda m, a, s: m.embed(a["ncodes"], a["nscales"], 2048, a["rows"], stream=s),
}


def tensors(out):
    return list(out) if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_outputs_are_the_streams_own(nf4, args, name, raw):
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    want = [t.clone() for t in tensors(CALLS[name](nf4, args, None))]
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed on the current stream with work queued on them
    busy = torch.empty((4096, 4096), device=DEV)
    freed = [torch.empty_like(t) for t in want for _ in range(2)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in freed]
    for _ in range(20):
        busy = busy @ busy
    for t in freed:
        t.fill_(0)
    del t, freed
    got = tensors(CALLS[name](nf4, args, stream))
    for t in got:
        a, b = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
        assert all(b <= lo or hi <= a for lo, hi in spans)
    main.wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # a result that is dropped is not handed out to the current stream
    torch.cuda.synchronize()
    got = tensors(CALLS[name](nf4, args, stream))
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in got]
    del got, t
    for t in [torch.empty_like(t) for t in want for _ in range(2)]:
        a, b = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
        assert all(b <= lo or hi <= a for lo, hi in spans)
    torch.cuda.synchronize()


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", ["mx_pack", "pack"])
def test_packing_reads_its_status_on_the_stream(nf4, args, name, raw):
    """check=True waits for the call's own stream, behind work queued there."""
    side = torch.cuda.Stream()
    W = args["W"].clone()
    W[7, 3] = float("nan")
    busy = torch.randn((4096, 4096), device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy
    with pytest.raises(ValueError, match="flagged"):
        getattr(nf4, name)(W, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()


@pytest.mark.parametrize("null", ["handle", "stream"])
@pytest.mark.parametrize("name", CALLS)
def test_the_default_stream_by_its_null_handle(nf4, args, name, null):
    """Another stream is current: the call runs on the default one, behind work queued
    there, and takes its memory."""
    default, side = torch.cuda.default_stream(), torch.cuda.Stream()
    stream = default if null == "stream" else default.cuda_stream
    assert default.cuda_stream == 0
    want = [t.clone() for t in tensors(CALLS[name](nf4, args, None))]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = tensors(CALLS[name](nf4, args, stream))
    # freed on the default stream, its blocks serve the next such call there
    spans = [t.data_ptr() for t in got]
    side.wait_stream(default)
    with torch.cuda.stream(side):
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    side.synchronize()
    del got
    again = tensors(CALLS[name](nf4, args, None))
    assert sorted(t.data_ptr() for t in again) == sorted(spans)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["mx_pack", "pack", "moe_sort"])
def test_status_on_the_null_handle(nf4, args, name):
    W, ids = args["W"].clone(), args["ids"].clone()
    W[7, 3] = float("nan")
    ids[9, 1] = 5
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        with pytest.raises(ValueError, match="flagged"):
            if name == "moe_sort":
                nf4.moe_sort(ids, 2, stream=0, check=True)
            else:
                getattr(nf4, name)(W, stream=0)


def test_workspace_of_the_null_handle(nf4):
    default = torch.cuda.default_stream()
    kept = nf4.workspace_for(DEV, 1 << 16, default)  # other calls may have used this one
    with torch.cuda.stream(torch.cuda.Stream()):
        assert nf4.workspace_for(DEV, 1 << 16, 0) is kept
        ws = nf4.workspace_for(DEV, kept.numel() + 1, 0)
        assert ws is not kept and nf4.workspace_for(DEV, kept.numel() + 1, default) is ws
    default.synchronize()
    assert not bool(ws.any())


@pytest.mark.parametrize("fork", [False, True], ids=["same", "forked"])
def test_captured_with_a_stream_argument(nf4, args, fork):
    """Calls on the capturing stream by its argument, or on one that forks from it and
    joins again; every replay against the eager call, with eager work in between."""
    X = args["X"].clone()

    def step(s):
        xc, xs = nf4.mx_pack(X, stream=s, check=False)
        rows = nf4.moe_gather(X[:512], args["place"], stream=s)
        return (nf4.mx_gemm(args["codes"], args["scales"], X, stream=s),
                nf4.mx_gemm_packed(args["codes"], args["scales"], xc, xs, stream=s),
                nf4.mx_gemm_grouped(args["stack"], args["sstack"], rows, args["offsets"], stream=s))
    step(None)
    torch.cuda.synchronize()
    main, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        if fork:
            other.wait_stream(main)
        out = step(other if fork else main)
        if fork:
            main.wait_stream(other)
    for i in range(3):
        X.copy_(torch.randn(X.shape, device=DEV).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step(None)))
        torch.cuda.synchronize()
