"""Routing on the GPU against plain definitions: the sort exactly, the row
operators and their gradients within the bounds of fp32 sums; odd widths, slots
without an expert, bad ids, unaligned views, graphs; and a whole expert layer,
forward and backward, as a model runs it."""
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


def normal(shape, seed, dtype=F32):
    return torch.randn(shape, generator=gen(seed), device=DEV).to(dtype)


def ids(T, topk, E, seed, none=0.1):
    """Skewed expert ids with a share of slots that have none."""
    e = (torch.rand((T, topk), generator=gen(seed), device=DEV) ** 2 * E).long().clamp(max=E - 1)
    gone = torch.rand((T, topk), generator=gen(seed + 1), device=DEV) < none
    return torch.where(gone, torch.full_like(e, -1), e)


def check_sort(nf4, experts, E):
    T, topk = experts.shape
    bo, offsets = gpu_guard.alloc(E + 1, torch.int32, DEV)
    br, order = gpu_guard.alloc(T * topk, torch.int32, DEV)
    bp, place = gpu_guard.alloc((T, topk), torch.int32, DEV)
    status = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    nf4.nf4_moe_sort(experts, E, offsets, order, place, status)
    torch.cuda.synchronize()
    o, r, p, bad = ref.sort_slots(experts.cpu(), E)
    assert offsets.tolist() == o
    assert order.tolist() == r
    assert place.reshape(-1).tolist() == p
    assert int(status) == (nf4.MOE_BAD_ID if bad else 0)
    for b in (bo, br, bp):
        gpu_guard.check(b)


@pytest.mark.parametrize("E", [1, 2, 8, 63, 64, 512])
@pytest.mark.parametrize("T,topk", [(1, 1), (1, 8), (5, 2), (63, 1), (64, 1), (65, 3), (1024, 4),
                                    (4095, 1), (2731, 3), (8191, 1), (2048, 4), (8193, 1),
                                    (3000, 7)])
def test_sort(nf4, T, topk, E):
    check_sort(nf4, ids(T, topk, E, T + E), E)


def test_sort_of_many_slots(nf4):
    check_sort(nf4, ids(40000, 5, 100, 3), 100)


@pytest.mark.parametrize("E", [1, 63, 64, 127, 128, 255, 256, 511, 512])
def test_sort_shares_the_chunks_out(nf4, E):
    """Every division of the chunks' counts over the scan's threads, exactly: keys in
    ascending order, equal keys in order of slot."""
    T, topk = 30001, 4
    e = ids(T, topk, E, E)
    e[::701] = E - 1
    offsets, order, place = nf4.moe_sort(e, E)
    key = torch.where(e < 0, torch.full_like(e, E), e).reshape(-1)
    want = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)
    assert offsets.tolist() == [0] + torch.cumsum(counts[:E], 0).tolist()
    kept = int(offsets[-1])
    assert torch.equal(order[:kept].long(), want[:kept])
    assert torch.equal(-order[kept:].long() - 1, want[kept:])
    row = torch.empty_like(want)
    row[want] = torch.arange(want.numel(), device=DEV)
    assert torch.equal(place.reshape(-1).long(), torch.where(key == E, -row - 1, row))


@pytest.mark.parametrize("T", [7, 5000])
def test_sort_one_expert_no_expert_and_bad_ids(nf4, T):
    E = 6
    check_sort(nf4, torch.full((T, 3), 4, dtype=torch.int64, device=DEV), E)
    check_sort(nf4, torch.full((T, 3), -1, dtype=torch.int64, device=DEV), E)
    e = ids(T, 3, E, 5)
    for bad in (E, -2, 1 << 40, -(1 << 62)):
        e[T // 2, 1] = bad
        check_sort(nf4, e, E)


@pytest.mark.parametrize("T", [7, 5000])
@pytest.mark.parametrize("side", [False, True], ids=["current", "side"])
def test_sort_refuses_bad_ids_when_asked(nf4, T, side):
    E = 6
    stream = torch.cuda.Stream() if side else None
    e = ids(T, 3, E, 5)
    good = [t.clone() for t in nf4.moe_sort(e, E)]
    torch.cuda.synchronize()
    for a, b in zip(nf4.moe_sort(e, E, stream=stream, check=True), good):
        assert torch.equal(a, b)
    for bad in (E, -2, 1 << 40, -(1 << 62)):
        e[T // 2, 1] = bad
        torch.cuda.synchronize()
        with pytest.raises(ValueError, match="expert ids"):
            nf4.moe_sort(e, E, stream=stream, check=True)
        offsets, order, place = nf4.moe_sort(e, E)  # not asked: a slot without an expert
        assert int(place[T // 2, 1]) < 0


def test_no_tokens(nf4):
    e = torch.empty((0, 2), dtype=torch.int64, device=DEV)
    offsets, order, place = nf4.moe_sort(e, 4)
    assert offsets.tolist() == [0] * 5 and order.numel() == 0 and place.shape == (0, 2)
    X = torch.empty((0, 16), device=DEV)
    assert nf4.moe_gather(X, place).shape == (0, 16)
    assert nf4.moe_combine(X, place).shape == (0, 16)
    dY, dw = nf4.moe_combine_grad(X, X, place, torch.empty((0, 2), device=DEV))
    assert dY.shape == (0, 16) and dw.shape == (0, 2)


def view(t, shift):
    """A copy of t at an address `shift` elements past an aligned one."""
    flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
    v = flat[shift:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,topk,H", [(1, 1, 1), (1, 8, 4096), (5, 2, 7), (33, 3, 64), (17, 5, 1001),
                                      (200, 4, 2048), (64, 9, 520), (9, 2, 5000), (3, 1, 16384)])
@pytest.mark.parametrize("shift", [0, 1])
def test_rows_and_gradients(nf4, T, topk, H, dtype, shift):
    E = 5
    _, order, place = nf4.moe_sort(ids(T, topk, E, T + H), E)
    p = place.reshape(-1).long()
    on = p >= 0
    row = torch.where(on, p, -p - 1)
    X, dOut = view(normal((T, H), 1, dtype), shift), view(normal((T, H), 2, dtype), shift)
    Y = view(normal((T * topk, H), 3, dtype), shift)
    # a row without an expert is never read
    Y[row[~on]] = float("nan")
    w = normal((T, topk), 4)
    tok = torch.arange(T, device=DEV).repeat_interleave(topk)

    buf, rows = gpu_guard.alloc((T * topk, H), dtype, DEV)
    nf4.nf4_moe_gather(X, place, rows)
    torch.cuda.synchronize()
    want = torch.zeros((T * topk, H), dtype=dtype, device=DEV)
    want[row[on]] = X[tok[on]]
    assert torch.equal(rows, want)
    gpu_guard.check(buf)

    y = torch.where(on.unsqueeze(1), Y.double()[row], 0.0).reshape(T, topk, H)
    for weights in (w, None):
        f = torch.ones_like(w) if weights is None else w
        buf, out = gpu_guard.alloc((T, H), dtype, DEV)
        nf4.nf4_moe_combine(Y, place, weights, out)
        torch.cuda.synchronize()
        gpu_guard.check(buf)
        terms = y * f.double().unsqueeze(2)
        ref.close(out, terms.sum(1), terms.abs().sum(1), topk, "combine")

    buf, dY = gpu_guard.alloc((T * topk, H), dtype, DEV)
    buf2, dw = gpu_guard.alloc((T, topk), F32, DEV)
    nf4.nf4_moe_combine_grad(dOut, Y, place, w, dY, dw)
    torch.cuda.synchronize()
    gpu_guard.check(buf)
    gpu_guard.check(buf2)
    want = torch.zeros((T * topk, H), dtype=torch.float64, device=DEV)
    want[row[on]] = dOut.double()[tok[on]] * w.double().reshape(-1, 1)[on]
    ref.close(dY, want, want.abs(), 1, "dY")
    terms = dOut.double().unsqueeze(1) * y
    ref.close(dw, terms.sum(2), terms.abs().sum(2), H, "dweights")
    assert not bool(dY[row[~on]].any()) and not bool(dw.reshape(-1)[~on].any())


def test_gradients_are_difference_quotients(nf4):
    """combine and gather are linear in each argument: with small whole numbers the
    differences along a direction equal the gradients' inner products exactly."""
    T, topk, H, E = 40, 3, 72, 4
    g = gen(1)
    whole = lambda *s: torch.randint(-4, 5, s, generator=g, device=DEV).float()  # noqa: E731
    _, _, place = nf4.moe_sort(ids(T, topk, E, 7), E)
    Y, dOut, w, v, V = whole(T * topk, H), whole(T, H), whole(T, topk), whole(T, topk), \
        whole(T * topk, H)
    dY, dw = nf4.moe_combine_grad(dOut, Y, place, w)
    f = lambda y, u: (dOut.double() * nf4.moe_combine(y, place, u).double()).sum()  # noqa: E731
    assert float(f(Y, w + v) - f(Y, w - v)) / 2 == float((dw.double() * v.double()).sum())
    assert float(f(Y + V, w) - f(Y - V, w)) / 2 == float((dY.double() * V.double()).sum())
    X, D, dP = whole(T, H), whole(T, H), whole(T * topk, H)
    dX = nf4.moe_combine(dP, place)
    h = lambda x: (dP.double() * nf4.moe_gather(x, place).double()).sum()  # noqa: E731
    assert float(h(X + D) - h(X - D)) / 2 == float((dX.double() * D.double()).sum())


def test_an_expert_twice_in_one_token(nf4):
    T, topk, E, H = 70, 4, 3, 40
    e = torch.tensor([[2, 2, 0, 2]], device=DEV).repeat(T, 1)
    check_sort(nf4, e, E)
    _, _, place = nf4.moe_sort(e, E)
    X = normal((T, H), 1)
    rows = nf4.moe_gather(X, place)
    assert torch.equal(rows[place.long()], X.unsqueeze(1).expand(T, topk, H))
    w = torch.ones((T, topk), device=DEV)
    w[:, 1] = -1.0
    w[:, 2:] = 0.0
    assert not bool(nf4.moe_combine(rows, place, w).any())


def test_most_slots_of_a_token_and_most_experts(nf4):
    T, topk, E, H = 5, 512, 512, 36
    e = torch.stack([torch.randperm(E, generator=gen(t), device=DEV) for t in range(T)])
    e[3] = -1
    check_sort(nf4, e, E)
    _, _, place = nf4.moe_sort(e, E)
    Y, w, dOut = normal((T * topk, H), 1), normal((T, topk), 2), normal((T, H), 3)
    on = place >= 0
    y = torch.where(on.unsqueeze(2), Y.double()[place.clamp(min=0).long()], 0.0)
    terms = y * w.double().unsqueeze(2)
    ref.close(nf4.moe_combine(Y, place, w), terms.sum(1), terms.abs().sum(1), topk, "combine")
    dY, dw = nf4.moe_combine_grad(dOut, Y, place, w)
    terms = dOut.double().unsqueeze(1) * y
    ref.close(dw, terms.sum(2), terms.abs().sum(2), H, "dweights")
    want = dOut.double().unsqueeze(1) * w.double().unsqueeze(2)
    ref.close(dY[place[on].long()], want[on], want[on].abs(), 1, "dY")


def test_rows_beyond_32_bit_offsets(nf4):
    T, topk, H = 70000, 4, 8192
    place = torch.randperm(T * topk, generator=gen(1), device=DEV).int().reshape(T, topk)
    X = normal((T, H), 2, BF)
    rows = nf4.moe_gather(X, place)
    assert rows.numel() * 2 > 1 << 32
    for j in range(topk):
        assert torch.equal(rows[place[-50:, j].long()], X[-50:])
        assert torch.equal(rows[place[:50, j].long()], X[:50])
    top = int(place.reshape(-1).argmax())  # the slot of the last row
    assert torch.equal(rows[-1], X[top // topk])
    w = torch.full((T, topk), 0.25, device=DEV)
    assert torch.equal(nf4.moe_combine(rows, place, w), X)
    dY, dw = nf4.moe_combine_grad(X, rows, place, w)
    assert torch.equal(dY[-1], X[top // topk] * 0.25)
    want = X[-50:].double().square().sum(1, keepdim=True).expand(50, topk)
    ref.close(dw[-50:], want, want, H, "dweights")


def test_place_entries_outside_the_rows_are_skipped(nf4):
    T, topk, H = 6, 2, 64
    place = torch.arange(T * topk, dtype=torch.int32, device=DEV).reshape(T, topk)
    place[1, 0], place[2, 1], place[3, 0] = 1 << 30, -(1 << 30), 2147483647
    place[4, 1] = -2147483648
    bufs = [gpu_guard.alloc((T * topk, H), F32, DEV), gpu_guard.alloc((T, H), F32, DEV),
            gpu_guard.alloc((T * topk, H), F32, DEV), gpu_guard.alloc((T, topk), F32, DEV)]
    X, Y, w = normal((T, H), 1), normal((T * topk, H), 2), normal((T, topk), 3)
    nf4.nf4_moe_gather(X, place, bufs[0][1])
    nf4.nf4_moe_combine(Y, place, w, bufs[1][1])
    nf4.nf4_moe_combine_grad(X, Y, place, w, bufs[2][1], bufs[3][1])
    torch.cuda.synchronize()
    for b, _ in bufs:
        gpu_guard.check(b)
    assert bool(torch.isfinite(bufs[1][1]).all())
    assert float(bufs[3][1][1, 0]) == 0.0 and float(bufs[3][1][4, 1]) == 0.0


def test_arguments_are_refused_by_name(nf4):
    e = ids(4, 2, 3, 1)
    offsets, order, place = nf4.moe_sort(e, 3)
    X, Y = normal((4, 16), 1), normal((8, 16), 2)
    with pytest.raises(TypeError, match="experts"):
        nf4.moe_sort(e.int(), 3)
    with pytest.raises(nf4.NF4Error):
        nf4.moe_sort(e, nf4.MOE_MAX_E + 1)
    with pytest.raises(ValueError, match="X must be"):
        nf4.moe_gather(X[:3], place)
    with pytest.raises(ValueError, match="Y must be"):
        nf4.moe_combine(Y[:7], place)
    with pytest.raises(ValueError, match="weights"):
        nf4.moe_combine(Y, place, normal((4, 3), 1))
    with pytest.raises(TypeError, match="weights"):
        nf4.moe_combine_grad(X, Y, place, None)
    with pytest.raises(TypeError, match="dtype"):
        nf4.moe_combine_grad(X.to(BF), Y, place, normal((4, 2), 1))
    with pytest.raises(TypeError, match="X has dtype"):
        nf4.moe_gather(X.half(), place)


# ------------------------------------------------------- a whole layer ----
class Layer:
    """Router -> experts' gate|up -> silu(gate) * up -> down -> weighted sum, on
    packed frozen matrices, with buffers of its own (so that it can be captured)."""

    def __init__(self, nf4, T, topk, E, H, F, seed):
        self.nf4, self.T, self.topk, self.E, self.H, self.F = nf4, T, topk, E, H, F
        up = 0.05 * normal((E * 2 * F, H), seed)
        down = 0.05 * normal((E * H, F), seed + 1)
        c, s = nf4.mx_pack(up)
        self.up = c.view(E, 2 * F, H // 2), s.view(E, 2 * F, H // 32)
        c, s = nf4.mx_pack(down)
        self.down = c.view(E, H, F // 2), s.view(E, H, F // 32)

    def forward(self, x, experts, w):
        n = self.nf4
        s = {}
        s["offsets"], s["order"], s["place"] = n.moe_sort(experts, self.E)
        s["rows"] = n.moe_gather(x, s["place"])
        s["gu"] = n.mx_gemm_grouped(*self.up, s["rows"], s["offsets"], out_dtype=BF)
        g, u = s["gu"].float().chunk(2, dim=1)
        s["act"] = (torch.nn.functional.silu(g) * u).to(BF)
        s["y"] = n.mx_gemm_grouped(*self.down, s["act"], s["offsets"], out_dtype=BF)
        s["out"] = n.moe_combine(s["y"], s["place"], w)
        return s

    def backward(self, s, w, dout):
        n = self.nf4
        b = {}
        b["dy"], b["dw"] = n.moe_combine_grad(dout, s["y"], s["place"], w)
        b["dact"] = n.mx_gemm_grouped_grad(*self.down, b["dy"], s["offsets"], out_dtype=F32)
        g, u = s["gu"].float().chunk(2, dim=1)
        sg = torch.sigmoid(g)
        b["dgu"] = torch.cat([b["dact"] * u * sg * (1 + g * (1 - sg)), b["dact"] * g * sg],
                             dim=1).to(BF)
        b["drows"] = n.mx_gemm_grouped_grad(*self.up, b["dgu"], s["offsets"], out_dtype=BF)
        b["dx"] = n.moe_combine(b["drows"], s["place"])
        return b


def check_layer(layer, x, experts, w, dout):
    """Every operator of one pass against its definition on the inputs it got."""
    s = layer.forward(x, experts, w)
    b = layer.backward(s, w, dout)
    torch.cuda.synchronize()
    o, r, p, _ = ref.sort_slots(experts.cpu(), layer.E)
    assert s["offsets"].tolist() == o and s["order"].tolist() == r
    for e in range(layer.E):
        lo, hi = o[e], o[e + 1]
        up = ref.values(layer.up[0][e], layer.up[1][e])
        down = ref.values(layer.down[0][e], layer.down[1][e])
        for got, rows, v, terms in ((s["gu"], s["rows"], up, layer.H),
                                    (s["y"], s["act"], down, layer.F),
                                    (b["dact"], b["dy"], down.t(), layer.H),
                                    (b["drows"], b["dgu"], up.t(), 2 * layer.F)):
            want, mag = ref.product(rows[lo:hi], v)
            ref.close(got[lo:hi], want, mag, terms)
    place = torch.tensor(p, device=DEV).reshape(experts.shape)
    on = (place >= 0).unsqueeze(2)
    row = torch.where(place >= 0, place, 0)
    for rows, f, got in ((s["y"], w, s["out"]), (b["drows"], torch.ones_like(w), b["dx"])):
        terms = torch.where(on, rows.double()[row], 0.0) * f.double().unsqueeze(2)
        ref.close(got, terms.sum(1), terms.abs().sum(1), layer.topk)
    return s, b


@pytest.mark.parametrize("T,topk,E", [(1, 2, 8), (6, 2, 8), (70, 3, 5), (400, 2, 4)])
def test_expert_layer_forward_and_backward(nf4, T, topk, E):
    layer = Layer(nf4, T, topk, E, 256, 160, 5)
    check_layer(layer, normal((T, 256), 1, BF), ids(T, topk, E, 2), normal((T, topk), 3).sigmoid(),
                normal((T, 256), 4, BF))


def test_expert_layer_captured_and_replayed_with_new_routing(nf4):
    T, topk, E, H = 37, 2, 6, 256
    layer = Layer(nf4, T, topk, E, H, 96, 5)
    x, w, dout = normal((T, H), 1, BF), normal((T, topk), 3).sigmoid(), normal((T, H), 4, BF)
    experts = ids(T, topk, E, 2)

    def step():
        s = layer.forward(x, experts, w)
        return s, layer.backward(s, w, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s, b = step()
    for i in range(4):
        x.copy_(normal((T, H), 10 + i, BF))
        experts.copy_(ids(T, topk, E, 20 + i, none=0.3 * i))
        graph.replay()
        torch.cuda.synchronize()
        s2, b2 = check_layer(layer, x, experts, w, dout)
        for name in ("place", "out"):
            assert torch.equal(s[name], s2[name])
        for name in ("dx", "dw"):
            assert torch.equal(b[name], b2[name])


def test_two_streams_at_once(nf4):
    """Two layers' passes in flight together: no operator keeps state."""
    layers = [Layer(nf4, 50, 2, 4, 128, 64, 9 + i) for i in range(2)]
    args = [(normal((50, 128), i, BF), ids(50, 2, 4, 30 + i), normal((50, 2), i).sigmoid())
            for i in range(2)]
    want = [layer.forward(*a)["out"].clone() for layer, a in zip(layers, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for st, layer, a in zip(streams, layers, args):
            with torch.cuda.stream(st):
                got.append(layer.forward(*a)["out"])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
