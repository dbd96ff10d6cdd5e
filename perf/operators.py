"""Timed cases of the MXFP4 operators and of the routing of tokens to experts.

Five kinds of case, each one call sequence of a user's program:

quantise  a bf16 or fp32 matrix to MXFP4 (e2m1 codes, one power-of-two scale per
          32 values along K); the pass returns the values the codes stand for.
product   Y = X . dequant(W)^T, X bf16, W packed; Y fp32.
packed    X quantised to MXFP4 in the call, then the product of two packed
          matrices; Y fp32.
route     tokens sorted by expert, their rows gathered, the experts' rows summed
          back with the routing weights; with "train", the gradients too.
experts   each expert's packed matrix times its own rows of the sorted tokens,
          bf16 out; with "train", the gradient of the rows too (the packed
          weights are frozen).

`own` chooses between the plain form (elementary torch operations in fp32) and
this package's operators.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32


# ---------------------------------------------------------------- cases ----
def listed():
    return [
        # one token's hidden state before a product of two packed matrices
        dict(name="quantise-token", kind="quantise", n=1, k=4096, dtype="bf16"),
        # the gate and up matrices of an 8B-sized layer, packed at load time
        dict(name="quantise-gate-up", kind="quantise", n=28672, k=4096, dtype="fp32"),
        # decode: one token through the down projection of an 8B-sized layer
        dict(name="product-token", kind="product", m=1, n=4096, k=14336),
        # a prompt of odd length through gate and up of the same layer
        dict(name="product-prompt", kind="product", m=509, n=28672, k=4096),
        # a short prompt chunk through q, k and v
        dict(name="packed-chunk", kind="packed", m=37, n=6144, k=4096),
        # a long prompt, or several together, through gate and up
        dict(name="packed-prompt", kind="packed", m=4096, n=28672, k=4096),
        # a decode batch: five sequences' tokens, two experts each
        dict(name="route-decode", kind="route", t=5, k=2, e=8, h=4096, dtype="bf16",
             dropped=0, train=False),
        # a training batch of ragged sequences; padded tokens have no expert
        dict(name="route-train", kind="route", t=8191, k=4, e=64, h=2048, dtype="bf16",
             dropped=300, train=True),
        # the same path held in fp32 throughout, two wide experts' worth a token
        dict(name="route-train-fp32", kind="route", t=2048, k=2, e=8, h=4096, dtype="fp32",
             dropped=0, train=True),
        # decode: four tokens, two experts each, through the experts' gate and up
        dict(name="experts-decode", kind="experts", r=8, e=8, n=28672, k=4096, train=False),
        # a fine-tuning step on a short batch over many small experts
        dict(name="experts-train-small", kind="experts", r=1003, e=32, n=2048, k=2048,
             train=True),
        # a fine-tuning step on a long batch, two experts a token
        dict(name="experts-train", kind="experts", r=16382, e=8, n=14336, k=4096, train=True),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantise", "product", "product", "packed", "route", "route", "experts",
                       "experts"])
    if kind == "quantise":
        k = BLOCK * _loguniform(rng, 1, 448)
        n = _loguniform(rng, 1, max(1, min(32768, 100_000_000 // k)))
        return dict(kind=kind, n=n, k=k, dtype=rng.choice(["bf16", "fp32"]))
    if kind in ("product", "packed"):
        k = BLOCK * _loguniform(rng, 4, 448)
        n = _loguniform(rng, 17, min(28672, 110_000_000 // k))
        m = _loguniform(rng, 1, 2048)
        return dict(kind=kind, m=m, n=n, k=k)
    if kind == "route":
        h = _loguniform(rng, 64, 8192)
        e = _loguniform(rng, 2, 256)
        k = rng.randint(1, min(8, e))
        t = _loguniform(rng, 1, max(1, min(16384, 40_000_000 // (h * k))))
        return dict(kind=kind, t=t, k=k, e=e, h=h, dtype=rng.choice(["bf16", "fp32"]),
                    dropped=rng.randint(0, t * k // 8), train=rng.random() < 0.6)
    k = BLOCK * _loguniform(rng, 8, 256)
    n = 8 * _loguniform(rng, 16, 1024)
    e = _loguniform(rng, 1, max(1, min(64, 400_000_000 // (n * k))))
    return dict(kind=kind, r=_loguniform(rng, 1, 8192), e=e, n=n, k=k,
                train=rng.random() < 0.5)


def _counts(r, e):
    """Rows per expert, most popular first: shares fall as 1 / (rank + 2), so a
    small batch leaves experts without a row."""
    share = [1.0 / (i + 2) for i in range(e)]
    total = sum(share)
    counts = [int(r * s / total) for s in share]
    i = 0
    while sum(counts) < r:
        counts[i % e] += 1
        i += 1
    return counts


def work(case):
    kind = case["kind"]
    if kind == "quantise":
        n = case["n"] * case["k"]
        # read, codes and scales out and in again, values out in fp32
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 2 * n * 17 // 32 + 4 * n,
                "flops": 2 * n}
    if kind in ("product", "packed"):
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k * 17 // 32 + 2 * m * k + 4 * m * n, "flops": 2 * m * n * k}
    if kind == "route":
        t, k, h, r = case["t"], case["k"], case["h"], case["t"] * case["k"]
        b = 2 if case["dtype"] == "bf16" else 4
        size = 8 * r + 4 * (2 * r + case["e"] + 1)            # ids, order, place, offsets
        size += b * h * (t + r) + b * h * (r + t) + 4 * r     # gather; combine
        flops = 2 * r * h
        if case["train"]:
            size += b * h * (r + t) + b * h * (t + 2 * r) + 4 * r  # the gradients of both
            flops += 4 * r * h
        return {"bytes": size, "flops": flops}
    r, n, k = case["r"], case["n"], case["k"]
    active = sum(c > 0 for c in _counts(r, case["e"]))
    size = active * n * k * 17 // 32 + 2 * r * (n + k) + 4 * (case["e"] + 1)
    times = 2 if case["train"] else 1
    return {"bytes": times * size, "flops": times * 2 * r * n * k}


# --------------------------------------------------------------- inputs ----
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + salt) & 0x7FFFFFFFFFFFFFFF)
    return g


def _activations(m, k, seed, salt):
    """Hidden states: normal, with a spread of channel sizes as layers have it."""
    g = _gen(seed, salt)
    channel = torch.exp(0.5 * torch.randn(k, generator=g, device=DEV))
    return torch.randn((m, k), generator=g, device=DEV) * channel


def _exponent(amax):
    """Shared exponent of a block: floor(log2 amax) - 2 (6 = 1.5 * 2^2 is the
    largest element), held to what an 8-bit power of two can say."""
    e = torch.frexp(amax).exponent - 3
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    return e.clamp(-127, 127)


def _codes(x):
    """(e2m1 codes, shared exponents) of fp32 [..., K] in blocks of 32."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    e = _exponent(b.abs().amax(-1))
    a = torch.ldexp(b.abs(), -e.unsqueeze(-1))
    # nearest of 0 .5 1 1.5 2 3 4 6, a tie to the even code; 6 is the largest
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5.0))
    c = c + 8 * torch.signbit(b).to(torch.uint8)
    return c.reshape(x.shape), e


def _lut():
    m = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.cat([m, -m])


def _pack(x):
    """Packed bytes (low nibble = even k) and scale bytes of a plain matrix."""
    c, e = _codes(x)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """fp32 values of packed bytes [.., K/2] and scale bytes [.., K/32]."""
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = _lut()[c.to(torch.int32)].reshape(*scales.shape, BLOCK)
    return torch.ldexp(v, scales.to(torch.int32).unsqueeze(-1) - 127).reshape(c.shape)


def _weights(n, k, seed, salt):
    return 0.02 * torch.randn((n, k), generator=_gen(seed, salt), device=DEV)


def prepare(case, seed):
    kind = case["kind"]
    s = dict(case)
    if kind == "quantise":
        x = _activations(case["n"], case["k"], seed, 1)
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else 0.02 * x
    elif kind in ("product", "packed"):
        s["codes"], s["scales"] = _pack(_weights(case["n"], case["k"], seed, 2))
        s["x"] = _activations(case["m"], case["k"], seed, 3).to(torch.bfloat16)
    elif kind == "route":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        t, k, e, h = case["t"], case["k"], case["e"], case["h"]
        g = _gen(seed, 4)
        # a router's scores: some experts are more popular than others
        score = torch.randn((t, e), generator=g, device=DEV) \
            + torch.randn(e, generator=g, device=DEV)
        top = torch.topk(score, k, dim=1)
        s["experts"] = top.indices.contiguous()
        s["weights"] = torch.softmax(top.values, dim=1)
        if case["dropped"]:
            gone = torch.randperm(t * k, generator=g, device=DEV)[:case["dropped"]]
            s["experts"].view(-1)[gone] = -1
        s["x"] = _activations(t, h, seed, 5).to(dt)
        s["y"] = _activations(t * k, h, seed, 6).to(dt)
        if case["train"]:
            s["dout"] = (0.01 * _activations(t, h, seed, 7)).to(dt)
            s["dp"] = (0.01 * _activations(t * k, h, seed, 8)).to(dt)
    else:
        r, e, n, k = case["r"], case["e"], case["n"], case["k"]
        perm = torch.randperm(e, generator=_gen(seed, 9), device=DEV).tolist()
        counts = _counts(r, e)
        bounds = [0]
        for i in range(e):
            bounds.append(bounds[-1] + counts[perm[i]])
        s["bounds"] = bounds
        s["offsets"] = torch.tensor(bounds, dtype=torch.int32, device=DEV)
        s["codes"] = torch.empty((e, n, k // 2), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((e, n, k // BLOCK), dtype=torch.uint8, device=DEV)
        for i in range(e):
            s["codes"][i], s["scales"][i] = _pack(_weights(n, k, seed, 100 + i))
        s["x"] = _activations(r, k, seed, 10).to(torch.bfloat16)
        if case["train"]:
            s["dy"] = (0.01 * _activations(r, n, seed, 11)).to(torch.bfloat16)
    return s


# ------------------------------------------------------------- one pass ----
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import dequant_gemv_nf4_amd as nf4
    kind = s["kind"]
    if kind == "quantise":
        codes, scales = nf4.mx_pack(s["x"], check=False)
        return nf4.mx_unpack(codes, scales)
    if kind == "product":
        return nf4.mx_gemm(s["codes"], s["scales"], s["x"])
    if kind == "packed":
        xcodes, xscales = nf4.mx_pack(s["x"], check=False)
        return nf4.mx_gemm_packed(s["codes"], s["scales"], xcodes, xscales)
    if kind == "route":
        offsets, order, place = nf4.moe_sort(s["experts"], s["e"])
        rows = nf4.moe_gather(s["x"], place)
        out = nf4.moe_combine(s["y"], place, s["weights"])
        if not s["train"]:
            return offsets, order, place, rows, out
        dx = nf4.moe_combine(s["dp"], place)
        dy, dw = nf4.moe_combine_grad(s["dout"], s["y"], place, s["weights"])
        return offsets, order, place, rows, out, dx, dy, dw
    y = nf4.mx_gemm_grouped(s["codes"], s["scales"], s["x"], s["offsets"],
                            out_dtype=torch.bfloat16)
    if not s["train"]:
        return y
    return y, nf4.mx_gemm_grouped_grad(s["codes"], s["scales"], s["dy"], s["offsets"],
                                       out_dtype=torch.bfloat16)


def _sort_plain(experts, e):
    """Rows in order of expert, then of slot (token-major); a slot without an
    expert comes last and is written as ~slot, its place as ~row."""
    flat = experts.reshape(-1)
    key = torch.where(flat < 0, torch.full_like(flat, e), flat)
    slot = torch.sort(key, stable=True).indices
    kept = key[slot] < e
    order = torch.where(kept, slot, -slot - 1).to(torch.int32)
    place = torch.empty_like(order)
    row = torch.arange(flat.numel(), device=flat.device)
    place[slot] = torch.where(kept, row, -row - 1).to(torch.int32)
    bound = torch.arange(e + 1, device=flat.device)
    offsets = (key.unsqueeze(0) < bound.unsqueeze(1)).sum(1).to(torch.int32)
    return offsets, order, place.reshape(experts.shape)


def _take(x, index, keep):
    """Rows index of x in fp32, zero where keep is false."""
    return torch.where(keep.unsqueeze(-1), x[index.clamp(min=0).long()].float(),
                       torch.zeros((), device=x.device))


def _run_plain(s):
    kind = s["kind"]
    if kind == "quantise":
        return _values(*_pack(s["x"].float()))
    if kind == "product":
        return s["x"].float() @ _values(s["codes"], s["scales"]).t()
    if kind == "packed":
        return _values(*_pack(s["x"].float())) @ _values(s["codes"], s["scales"]).t()
    if kind == "route":
        x, y, w, t, k = s["x"], s["y"], s["weights"], s["t"], s["k"]
        offsets, order, place = _sort_plain(s["experts"], s["e"])
        rows = _take(x, torch.div(order, k, rounding_mode="floor"), order >= 0).to(x.dtype)
        picked = _take(y, place.reshape(-1), place.reshape(-1) >= 0).reshape(t, k, -1)
        out = (picked * w.unsqueeze(-1)).sum(1).to(y.dtype)
        if not s["train"]:
            return offsets, order, place, rows, out
        flat = place.reshape(-1)
        dx = _take(s["dp"], flat, flat >= 0).reshape(t, k, -1).sum(1).to(y.dtype)
        dw = (s["dout"].float().unsqueeze(1) * picked).sum(2)
        slot = order.clamp(min=0).long()
        dy = _take(s["dout"], torch.div(order, k, rounding_mode="floor"), order >= 0)
        dy = (dy * w.reshape(-1)[slot].unsqueeze(-1)).to(y.dtype)
        return offsets, order, place, rows, out, dx, dy, dw
    y = torch.empty((s["r"], s["n"]), dtype=torch.bfloat16, device=DEV)
    dx = torch.empty((s["r"], s["k"]), dtype=torch.bfloat16, device=DEV) if s["train"] else None
    for i in range(s["e"]):
        a, b = s["bounds"][i], s["bounds"][i + 1]
        if a == b:
            continue
        v = _values(s["codes"][i], s["scales"][i])
        y[a:b] = (s["x"][a:b].float() @ v.t()).to(torch.bfloat16)
        if s["train"]:
            dx[a:b] = (s["dy"][a:b].float() @ v).to(torch.bfloat16)
    return (y, dx) if s["train"] else y


# ------------------------------------------------- the definition in 64 bits ----
def _levels64(codes, scales):
    """Element values by the format's fields: sign, 2 exponent bits with bias 1,
    1 mantissa bit, subnormal at exponent 0; times 2^(scale byte - 127)."""
    n = codes.shape[:-1]
    c = torch.empty((*n, 2 * codes.shape[-1]), dtype=torch.uint8, device=codes.device)
    c[..., 0::2] = codes % 16
    c[..., 1::2] = codes // 16
    mant, ex, sign = (c % 2).double(), ((c // 2) % 4).double(), (c // 8).double()
    mag = torch.where(ex > 0, (1 + mant / 2) * torch.exp2(ex - 1), mant / 2)
    scale = torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=-1)
    return (1 - 2 * sign) * mag * scale


def _quantised64(x):
    """x rounded to the format: the block's power of two, then the nearest of the
    levels, found by distance, with a tie to the level of even mantissa."""
    b = x.double().reshape(-1, BLOCK)
    top = b.abs().max(dim=1, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    # log2 rounds: put the power of two on the right side of the value
    e = torch.where(torch.exp2(e) > top, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= top, e + 1, e)
    step = torch.exp2(torch.where(top > 0, e - 2, torch.full_like(e, -127)).clamp(-127, 127))
    a = b.abs() / step
    best = torch.zeros_like(a)
    gap = a.clone()
    for i, level in enumerate((0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), start=1):
        d = (a - level).abs()
        better = (d < gap) | ((d == gap) & (i % 2 == 0))
        best = torch.where(better, torch.full_like(a, level), best)
        gap = torch.where(better, d, gap)
    return (torch.sign(b) * best * step).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantise":
        x = s["x"]
        out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        rows = max(1, (1 << 24) // case["k"])
        for i in range(0, case["n"], rows):
            out[i:i + rows] = _quantised64(x[i:i + rows])
        return out
    if kind in ("product", "packed"):
        x = _quantised64(s["x"]) if kind == "packed" else s["x"].double()
        return x @ _levels64(s["codes"], s["scales"]).t().contiguous()
    if kind == "route":
        t, k, e = case["t"], case["k"], case["e"]
        flat = s["experts"].reshape(-1).tolist()
        buckets = [[] for _ in range(e + 1)]
        for i, v in enumerate(flat):
            buckets[v if v >= 0 else e].append(i)
        offsets = [0]
        for lst in buckets[:e]:
            offsets.append(offsets[-1] + len(lst))
        order = [i for lst in buckets[:e] for i in lst] + [~i for i in buckets[e]]
        place = [0] * (t * k)
        for row, i in enumerate(order):
            if i >= 0:
                place[i] = row
            else:
                place[~i] = ~row
        ints = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (offsets, order, place)]
        kept = torch.tensor([i for i in order if i >= 0], dtype=torch.long, device=DEV)
        n = kept.numel()
        tok = kept // k
        w = s["weights"].double().reshape(-1)
        rows = torch.zeros((t * k, case["h"]), dtype=torch.float64, device=DEV)
        rows[:n] = s["x"].double()[tok]
        out = torch.zeros((t, case["h"]), dtype=torch.float64, device=DEV)
        y = s["y"].double()
        out.index_add_(0, tok, y[:n] * w[kept].unsqueeze(1))
        res = [ints[0], ints[1], ints[2].reshape(t, k), rows, out]
        if case["train"]:
            dx = torch.zeros_like(out)
            dx.index_add_(0, tok, s["dp"].double()[:n])
            dy = torch.zeros_like(rows)
            dout = s["dout"].double()
            dy[:n] = dout[tok] * w[kept].unsqueeze(1)
            dw = torch.zeros(t * k, dtype=torch.float64, device=DEV)
            dw[kept] = torch.linalg.vecdot(dout[tok], y[:n])
            res += [dx, dy, dw.reshape(t, k)]
        return tuple(res)
    y = torch.empty((case["r"], case["n"]), dtype=torch.float64, device=DEV)
    dx = torch.empty((case["r"], case["k"]), dtype=torch.float64, device=DEV)
    for i in range(case["e"]):
        a, b = s["bounds"][i], s["bounds"][i + 1]
        if a < b:
            v = _levels64(s["codes"][i], s["scales"][i])
            y[a:b] = s["x"][a:b].double() @ v.t().contiguous()
            if case["train"]:
                dx[a:b] = s["dy"][a:b].double() @ v
    return (y, dx) if case["train"] else y
