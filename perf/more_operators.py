"""Timed cases of the fused forms of the MXFP4 products.

Four kinds of case, each one call of a user's program:

linear  Y = act(X . dequant(W)^T + bias) + residual, X bf16, W packed; act is a plain
        activation or a gated one (the matrix's first half gates its second); with
        "keep", the values in front of the activation too, for the backward pass.
grad    the gradients of that: of the values in front of the activation, of X and of
        the bias, from the gradient of Y and the values kept (the weights are frozen).
loss    softmax cross entropy of X . dequant(W)^T, W a packed head of a large
        vocabulary: losses and log-sum-exps; with "train", the gradient of X too.
moe     a whole expert layer for a few tokens: each token through its experts' gated
        pair of matrices, summed with the routing weights.

`own` chooses between the plain form (elementary torch operations in fp32) and this
package's operators.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
GATED = ("swiglu", "geglu")


# ---------------------------------------------------------------- cases ----
def listed():
    return [
        # decode: one token through gate and up of an 8B-sized layer, gated
        dict(name="linear-token", kind="linear", m=1, n=28672, k=4096, act="swiglu", bias=False,
             residual=False, out="bf16", keep=False),
        # decode: the attention output of one token, added to the residual stream
        dict(name="linear-residual", kind="linear", m=1, n=4096, k=4096, act="none", bias=False,
             residual=True, out="bf16", keep=False),
        # training forward of a prompt of odd length through gate and up
        dict(name="linear-prompt", kind="linear", m=1021, n=28672, k=4096, act="swiglu",
             bias=False, residual=False, out="bf16", keep=True),
        # a prompt chunk through a biased layer with gelu, 13B-sized, held in fp32
        dict(name="linear-bias", kind="linear", m=333, n=13824, k=5120, act="gelu", bias=True,
             residual=False, out="fp32", keep=False),
        # a short training batch back through the same layer
        dict(name="grad-chunk", kind="grad", m=77, n=13824, k=5120, act="gelu", bias=True),
        # a training batch back through gate and up
        dict(name="grad-prompt", kind="grad", m=2048, n=28672, k=4096, act="swiglu", bias=False),
        # scoring the few candidate tokens of a request, 7B-sized head
        dict(name="loss-score", kind="loss", m=5, v=32000, k=4096, ignored=0, train=False),
        # the loss of a held-out text over a large vocabulary
        dict(name="loss-eval", kind="loss", m=1000, v=128256, k=4096, ignored=31, train=False),
        # a fine-tuning step's loss and gradient; the prompt's tokens are ignored
        dict(name="loss-train", kind="loss", m=2047, v=128256, k=4096, ignored=500, train=True),
        # decode: one token, two of eight large experts
        dict(name="moe-token", kind="moe", t=1, k=2, e=8, h=4096, i=14336, act="swiglu"),
        # a decode batch of ragged size over many small experts
        dict(name="moe-batch", kind="moe", t=19, k=8, e=128, h=2048, i=768, act="swiglu"),
        # drafted tokens of several sequences verified together: every expert has rows
        dict(name="moe-verify", kind="moe", t=64, k=2, e=8, h=4096, i=14336, act="swiglu"),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "grad", "loss", "loss", "moe", "moe"])
    if kind in ("linear", "grad"):
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu", "swiglu", "geglu"])
        k = BLOCK * _loguniform(rng, 4, 448)
        n = _loguniform(rng, 17, min(28672, 120_000_000 // k))
        m = _loguniform(rng, 1, 2048)
        bias = rng.random() < 0.5
        if kind == "grad":
            return dict(kind=kind, m=m, n=n + -n % 16, k=k, act=act, bias=bias)
        if act in GATED:
            n += n % 2
        return dict(kind=kind, m=m, n=n, k=k, act=act, bias=bias, residual=rng.random() < 0.5,
                    out=rng.choice(["bf16", "fp32"]), keep=rng.random() < 0.3)
    if kind == "loss":
        k = BLOCK * _loguniform(rng, 4, 256)
        v = _loguniform(rng, 100, min(160_000, 520_000_000 // k))
        m = _loguniform(rng, 1, max(1, min(4096, 1_000_000_000_000 // (v * k), 250_000_000 // v)))
        return dict(kind=kind, m=m, v=v, k=k, ignored=rng.randint(0, m // 4),
                    train=rng.random() < 0.5)
    h = BLOCK * _loguniform(rng, 4, 160)
    i = BLOCK * _loguniform(rng, 4, 448)
    e = _loguniform(rng, 2, max(2, min(128, 400_000_000 // (h * i))))
    return dict(kind=kind, t=_loguniform(rng, 1, 64), k=rng.randint(1, min(8, e)), e=e, h=h, i=i,
                act=rng.choice(["swiglu", "swiglu", "geglu", "silu"]))


def work(case):
    kind = case["kind"]
    if kind == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        cols = n // 2 if case["act"] in GATED else n
        b = 2 if case["out"] == "bf16" else 4
        size = n * k * 17 // 32 + 2 * m * k + b * m * cols
        size += 4 * n * case["bias"] + b * m * cols * case["residual"] + 2 * m * n * case["keep"]
        return {"bytes": size, "flops": 2 * m * n * k}
    if kind == "grad":
        m, n, k = case["m"], case["n"], case["k"]
        cols = n // 2 if case["act"] in GATED else n
        size = n * k * 17 // 32 + 2 * m * k + 2 * m * cols + 4 * m * n + 4 * n * case["bias"]
        return {"bytes": size, "flops": 2 * m * n * k}
    if kind == "loss":
        m, v, k = case["m"], case["v"], case["k"]
        size = v * k * 17 // 32 + 2 * m * k + 8 * m + 8 * m
        if case["train"]:
            size += 4 * m + 2 * m * k
        return {"bytes": size, "flops": (4 if case["train"] else 2) * m * v * k}
    t, k, e, h, i = case["t"], case["k"], case["e"], case["h"], case["i"]
    # experts that at least one of t tokens takes, k of e each
    active = max(k, int(e * (1 - (1 - k / e) ** t)))
    wide = 3 if case["act"] in GATED else 2
    return {"bytes": active * wide * h * i * 17 // 32 + 4 * t * h + 12 * t * k,
            "flops": 2 * t * k * wide * h * i}


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


def _pack(x):
    """MXFP4 codes [.., K/2] (low nibble = even k) and scale bytes [.., K/32] of fp32
    x: per block of 32 the power of two floor(log2 max) - 2, values rounded to the
    nearest of 0 .5 1 1.5 2 3 4 6."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1)
    e = torch.frexp(top).exponent - 3
    e = torch.where(top == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e.unsqueeze(-1))
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5.0))
    c = (c + 8 * torch.signbit(b).to(torch.uint8)).reshape(x.shape)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """fp32 values of packed bytes [.., K/2] and scale bytes [.., K/32]."""
    m = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = torch.cat([m, -m])[c.to(torch.int32)].reshape(*scales.shape, BLOCK)
    return torch.ldexp(v, scales.to(torch.int32).unsqueeze(-1) - 127).reshape(c.shape)


def _weights(n, k, seed, salt):
    return 0.02 * torch.randn((n, k), generator=_gen(seed, salt), device=DEV)


def _experts(e, n, k, seed, salt):
    codes = torch.empty((e, n, k // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((e, n, k // BLOCK), dtype=torch.uint8, device=DEV)
    for i in range(e):
        codes[i], scales[i] = _pack(_weights(n, k, seed, salt + i))
    return codes, scales


def prepare(case, seed):
    kind = case["kind"]
    s = dict(case)
    if kind in ("linear", "grad"):
        m, n, k = case["m"], case["n"], case["k"]
        cols = n // 2 if case["act"] in GATED else n
        s["codes"], s["scales"] = _pack(_weights(n, k, seed, 1))
        if kind == "linear":
            s["x"] = _activations(m, k, seed, 2).to(torch.bfloat16)
            s["dtype"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
            s["b"] = 0.1 * torch.randn(n, generator=_gen(seed, 3), device=DEV) \
                if case["bias"] else None
            s["r"] = _activations(m, cols, seed, 4).to(s["dtype"]) if case["residual"] else None
        else:
            s["z"] = (1.5 * torch.randn((m, n), generator=_gen(seed, 5),
                                        device=DEV)).to(torch.bfloat16)
            s["dy"] = (0.01 * _activations(m, cols, seed, 6)).to(torch.bfloat16)
    elif kind == "loss":
        m, v, k = case["m"], case["v"], case["k"]
        w = _weights(v, k, seed, 7)
        g = _gen(seed, 8)
        targets = torch.randint(0, v, (m,), generator=g, device=DEV)
        x = _activations(m, k, seed, 9)
        # a trained model's states: the target's logit stands out, more for some tokens
        x += 12.0 * torch.rand((m, 1), generator=g, device=DEV) * w[targets]
        s["x"] = x.to(torch.bfloat16)
        s["codes"], s["scales"] = _pack(w)
        if case["ignored"]:
            targets[torch.randperm(m, generator=g, device=DEV)[:case["ignored"]]] = -100
        s["targets"] = targets
        # the mean over the tokens that count
        s["dloss"] = torch.where(targets >= 0, 1.0 / max(1, m - case["ignored"]), 0.0)
    else:
        t, k, e, h, i = case["t"], case["k"], case["e"], case["h"], case["i"]
        up = 2 * i if case["act"] in GATED else i
        s["codes1"], s["scales1"] = _experts(e, up, h, seed, 1000)
        s["codes2"], s["scales2"] = _experts(e, h, i, seed, 3000)
        s["x"] = _activations(t, h, seed, 10).to(torch.bfloat16)
        top = torch.topk(torch.randn((t, e), generator=_gen(seed, 11), device=DEV), k, dim=1)
        s["experts"] = top.indices.contiguous()
        s["weights"] = torch.softmax(top.values, dim=1)
    return s


# ------------------------------------------------------------- one pass ----
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import dequant_gemv_nf4_amd as nf4
    kind = s["kind"]
    act = None if s.get("act") == "none" else s.get("act")
    if kind == "linear":
        return nf4.mx_linear(s["codes"], s["scales"], s["x"], bias=s["b"], act=act,
                             residual=s["r"], out_dtype=s["dtype"], keep_z=s["keep"])
    if kind == "grad":
        dx, dz, db = nf4.mx_linear_grad(s["codes"], s["scales"], s["dy"], s["z"], act=act,
                                        bias_grad=s["bias"])
        return (dx, dz, db) if s["bias"] else (dx, dz)
    if kind == "loss":
        return nf4.mx_cross_entropy(s["codes"], s["scales"], s["x"], s["targets"],
                                    dloss=s["dloss"] if s["train"] else None)
    return nf4.moe_mlp(s["codes1"], s["scales1"], s["codes2"], s["scales2"], s["x"],
                       s["experts"], s["weights"], act=act)


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act in ("silu", "swiglu"):
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act in ("silu", "swiglu"):
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) \
            + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)


def _gate(z, act):
    if act in GATED:
        a, b = z.chunk(2, dim=-1)
        return _act(a, act) * b
    return _act(z, act)


def _run_plain(s):
    kind = s["kind"]
    if kind == "linear":
        z = s["x"].float() @ _values(s["codes"], s["scales"]).t()
        if s["b"] is not None:
            z = z + s["b"]
        y = _gate(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        y = y.to(s["dtype"])
        return (y, z.to(torch.bfloat16)) if s["keep"] else y
    if kind == "grad":
        z, dy = s["z"].float(), s["dy"].float()
        if s["act"] in GATED:
            a, b = z.chunk(2, dim=-1)
            dz = torch.cat([dy * b * _slope(a, s["act"]), dy * _act(a, s["act"])], dim=-1)
        else:
            dz = dy * _slope(z, s["act"])
        dx = (dz @ _values(s["codes"], s["scales"])).to(torch.bfloat16)
        out = (dx, dz.to(torch.bfloat16))
        return out + (dz.sum(0),) if s["bias"] else out
    if kind == "loss":
        v = _values(s["codes"], s["scales"])
        logits = s["x"].float() @ v.t()
        top = logits.amax(1, keepdim=True)
        p = torch.exp(logits - top)
        total = p.sum(1, keepdim=True)
        lse = (top + torch.log(total)).squeeze(1)
        counts = s["targets"] >= 0
        index = s["targets"].clamp(min=0).unsqueeze(1)
        loss = torch.where(counts, lse - logits.gather(1, index).squeeze(1), 0.0)
        if not s["train"]:
            return loss, lse
        p = p / total
        p.scatter_add_(1, index, torch.full_like(total, -1.0))
        dx = (p * torch.where(counts, s["dloss"], 0.0).unsqueeze(1)) @ v
        return loss, lse, dx.to(torch.bfloat16)
    t, k, e = s["t"], s["k"], s["e"]
    flat, x, w = s["experts"].reshape(-1), s["x"].float(), s["weights"]
    if t * k < e:  # the slots' own matrices
        v1 = _values(s["codes1"][flat], s["scales1"][flat])
        z = torch.bmm(v1, x.repeat_interleave(k, dim=0).unsqueeze(2)).squeeze(2)
        a = _gate(z, s["act"]) * w.reshape(-1, 1)
        v2 = _values(s["codes2"][flat], s["scales2"][flat])
        y = torch.bmm(v2, a.unsqueeze(2)).reshape(t, k, -1)
        return y.sum(1).to(torch.bfloat16)
    # every expert's matrices, with the weight 0 where a token does not go
    v1 = _values(s["codes1"], s["scales1"])
    z = (x @ v1.reshape(-1, v1.shape[2]).t()).reshape(t, e, -1)
    share = torch.zeros((t, e), device=DEV).scatter_add_(1, s["experts"], w)
    a = (_gate(z, s["act"]) * share.unsqueeze(2)).transpose(0, 1).contiguous()
    v2 = _values(s["codes2"], s["scales2"])
    return torch.bmm(a, v2.transpose(1, 2).contiguous()).sum(0).to(torch.bfloat16)


# ------------------------------------------------- the definition in 64 bits ----
def _levels64(codes, scales):
    """Element values by the format's fields: sign, 2 exponent bits with bias 1,
    1 mantissa bit, subnormal at exponent 0; times 2^(scale byte - 127)."""
    out = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 25) // max(1, codes.shape[1]))
    for i in range(0, codes.shape[0], step):
        part = codes[i:i + step]
        c = torch.empty((part.shape[0], 2 * part.shape[1]), dtype=torch.uint8, device=DEV)
        c[:, 0::2] = part % 16
        c[:, 1::2] = part // 16
        mant, ex, sign = (c % 2).double(), ((c // 2) % 4).double(), (c // 8).double()
        mag = torch.where(ex > 0, (1 + mant / 2) * torch.exp2(ex - 1), mant / 2)
        power = torch.exp2(scales[i:i + step].double() - 127)
        out[i:i + step] = (1 - 2 * sign) * mag * power.repeat_interleave(BLOCK, dim=1)
    return out


def _f64(name, z):
    """(f(z), f'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
    if name in ("silu", "swiglu"):
        p = 1 / (1 + torch.exp(-z))
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / 2 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
    c = 2 * (2 / math.pi) ** 0.5
    p = 1 / (1 + torch.exp(-c * (z + 0.044715 * z ** 3)))
    return z * p, p + z * p * (1 - p) * c * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "linear":
        v = _levels64(s["codes"], s["scales"])
        z = torch.matmul(v, s["x"].double().t().contiguous()).t().contiguous()
        if case["bias"]:
            z += s["b"].double()
        if case["act"] in GATED:
            half = case["n"] // 2
            y = _f64(case["act"], z[:, :half])[0] * z[:, half:]
        else:
            y = _f64(case["act"], z)[0]
        if case["residual"]:
            y = y + s["r"].double()
        return (y, z) if case["keep"] else y
    if kind == "grad":
        z, dy = s["z"].double(), s["dy"].double()
        dz = torch.empty_like(z)
        if case["act"] in GATED:
            half = case["n"] // 2
            f, df = _f64(case["act"], z[:, :half])
            dz[:, :half] = df * z[:, half:] * dy
            dz[:, half:] = f * dy
        else:
            dz = _f64(case["act"], z)[1] * dy
        dx = dz @ _levels64(s["codes"], s["scales"])
        return (dx, dz, dz.sum(0)) if case["bias"] else (dx, dz)
    if kind == "loss":
        v = _levels64(s["codes"], s["scales"])
        logits = torch.matmul(v, s["x"].double().t().contiguous()).t().contiguous()
        lse = torch.logsumexp(logits, dim=1)
        rows = torch.nonzero(s["targets"] >= 0).squeeze(1)
        at = s["targets"][rows]
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - logits[rows, at]
        if not case["train"]:
            return loss, lse
        d = torch.zeros_like(logits)
        d[rows] = torch.exp(logits[rows] - lse[rows].unsqueeze(1))
        d[rows, at] -= 1.0
        dx = (d * s["dloss"].double().unsqueeze(1)) @ v
        return loss, lse, dx
    out = torch.zeros((case["t"], case["h"]), dtype=torch.float64, device=DEV)
    for e in range(case["e"]):
        tok, slot = torch.nonzero(s["experts"] == e, as_tuple=True)
        if tok.numel() == 0:
            continue
        v1 = _levels64(s["codes1"][e], s["scales1"][e])
        z = s["x"][tok].double() @ v1.t().contiguous()
        if case["act"] in GATED:
            a = _f64(case["act"], z[:, :case["i"]])[0] * z[:, case["i"]:]
        else:
            a = _f64(case["act"], z)[0]
        y = a @ _levels64(s["codes2"][e], s["scales2"][e]).t().contiguous()
        out.index_add_(0, tok, y * s["weights"][tok, slot].double().unsqueeze(1))
    return out
