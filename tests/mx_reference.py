"""Plain 64-bit definitions the MXFP4 and routing tests compare against (torch
float64 on the device of their inputs; shares no code with the library)."""
import torch

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def values(codes, scales):
    """float64 values of packed codes [.., K/2] and scale bytes [.., K/32]."""
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64,
                       device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return lut[c] * s.repeat_interleave(32, dim=-1)


def quantise(w):
    """(codes uint8 [N][K/2], scales uint8 [N][K/32]) of a matrix, in float64."""
    n, k = w.shape
    b = w.double().reshape(n, k // 32, 32)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad.unsqueeze(-1), torch.zeros_like(b), b)
    top = b.abs().amax(-1)
    e = torch.frexp(top).exponent.long() - 1 - 2
    e = torch.where(top == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    a = b.abs() * torch.exp2(-e.double()).unsqueeze(-1)
    code = torch.zeros_like(a, dtype=torch.long)
    for i in range(7):
        mid = (LEVELS[i] + LEVELS[i + 1]) / 2
        # ties to the even code: up when the code above is even
        code += ((a >= mid) if (i + 1) % 2 == 0 else (a > mid)).long()
    code += 8 * torch.signbit(b).long()
    code = torch.where(bad.unsqueeze(-1), torch.zeros_like(code), code).reshape(n, k)
    scales = torch.where(bad, torch.full_like(e, 255), e + 127)
    packed = code[:, 0::2] + 16 * code[:, 1::2]
    return packed.to(torch.uint8), scales.to(torch.uint8), bool(bad.any())


def product(x, v):
    """(x . v^T, |x| . |v|^T) in float64."""
    x = x.double()
    return x @ v.t().contiguous(), x.abs() @ v.abs().t().contiguous()


def close(got, want, mag, terms, what=""):
    """fp32 sums of `terms` products in any order are off by at most
    (terms + 8) 2^-24 of the sum of magnitudes (8: the cross-wave adds and the
    final rounding); a bf16 output adds half a step, 2^-8 of the value."""
    tol = (terms + 8) * 2.0 ** -24 * mag + 1e-30
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    err = (got.double() - want).abs()
    ok = err <= tol
    assert bool(ok.all()), (f"{what}: {int((~ok).sum())} of {ok.numel()} outside, worst "
                            f"{float((err / tol).nan_to_num(nan=float('inf')).max()):.3g} x tolerance")


def sort_slots(experts, num_experts):
    """(offsets, order, place, bad) as lists: a stable sort by expert, slots
    without one last and written as ~."""
    T, k = experts.shape
    flat = experts.reshape(-1).tolist()
    buckets = [[] for _ in range(num_experts + 1)]
    bad = False
    for f, e in enumerate(flat):
        bad |= e != -1 and not 0 <= e < num_experts
        buckets[e if 0 <= e < num_experts else num_experts].append(f)
    offsets = [0]
    for b in buckets[:num_experts]:
        offsets.append(offsets[-1] + len(b))
    order = [f for b in buckets[:num_experts] for f in b] + [~f for f in buckets[num_experts]]
    place = [0] * (T * k)
    for row, f in enumerate(order):
        if f >= 0:
            place[f] = row
        else:
            place[~f] = ~row
    return offsets, order, place, bad
