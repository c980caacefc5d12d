"""Inputs and 64-bit references shared by the tests of the microscaled operators and of the experts' routing (no library
code)."""

import math

import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def pow2(e):
    """2^e in 64 bits for whole e, put together from its bits (torch.ldexp goes through a power in 32 bits)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def strides(cols):
    return (-(-cols // 2) + 15) // 16 * 16, (-(-cols // 32) + 3) // 4 * 4


def make_mx4(gen, rows, cols, low=115, high=130, device="cuda", extra=0):
    """Random codes and scale bytes low..high: (codes, scales), padded, the padding full of what must not be read (codes 0xFF,
    scales NaN).  extra: further padding of the rows, 16 bytes of codes and 4 of scales each."""
    cs, ss = strides(cols)
    cs, ss = cs + 16 * extra, ss + 4 * extra
    codes = torch.randint(0, 256, (rows, cs), generator=gen, device=device, dtype=torch.uint8)
    scales = torch.randint(low, high + 1, (rows, ss), generator=gen, device=device, dtype=torch.uint8)
    codes[:, -(-cols // 2):] = 0xFF
    if cols % 2:
        codes[:, cols // 2] |= 0xF0
    scales[:, -(-cols // 32):] = 255
    return codes, scales


def values(codes, scales, cols):
    """The matrix in 64 bits, from the bits of its codes."""
    k = torch.arange(cols, device=codes.device)
    q = (codes[:, k // 2].int() >> (4 * (k % 2))) & 15
    grid = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
    s = scales[:, k // 32].int()
    unit = torch.where(s == 255, torch.full_like(s, float("nan"), dtype=torch.float64), pow2(s - 127))
    return torch.where(q >= 8, -1.0, 1.0) * grid[(q & 7).long()] * unit


def quantize_f64(x):
    """(exponent bytes [rows, G], codes [rows, cols]) of x, by search: the nearest value, of two the one of even code."""
    rows, cols = x.shape
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    scales = torch.zeros((rows, -(-cols // 32)), dtype=torch.uint8, device=x.device)
    codes = torch.zeros((rows, cols), dtype=torch.uint8, device=x.device)
    for g in range(scales.shape[1]):
        v = x[:, 32 * g:32 * g + 32].double()
        top = v.abs().amax(1)
        bad = ~torch.isfinite(top)
        top = torch.where(bad, torch.ones_like(top), top)
        e = torch.where(top > 0, torch.frexp(top)[1] - 1 - 2, torch.full_like(top, -127, dtype=torch.int32)).clamp(min=-127)
        t = (v.abs() / pow2(e).unsqueeze(1)).clamp(max=6.0)
        d = (t.unsqueeze(2) - grid).abs()
        near = d == d.amin(2, keepdim=True)
        rank = torch.tensor([0, 8, 1, 9, 2, 10, 3, 11], device=x.device)          # even codes first
        c = torch.where(near, rank, 99).argmin(2).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
        scales[:, g] = torch.where(bad, 255, e + 127).to(torch.uint8)
        codes[:, 32 * g:32 * g + 32] = torch.where(bad.unsqueeze(1), torch.zeros_like(c), c)
    return scales, codes


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def product_bound(x, w, K):
    """What fp32 sums of exact products may be off by: 2^-24 of the sum of the absolute terms for each addition, of which a
    sum of K terms has fewer than K, counted twice for what the matrix instruction adds inside."""
    return (x.abs() @ w.abs().t()) * (2 * K * 2.0 ** -24)


def check(got, want, bound, dtype, what=""):
    """got (dtype) against want (64 bits): bound, half a step of the type and its smallest number."""
    tol = bound + want.abs() * half_step(dtype) * (1 + 2.0 ** -8) + bound * half_step(dtype) + torch.finfo(dtype).tiny * half_step(dtype)
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float((err / tol).nan_to_num(1e9).max()):.3g} of the tolerance")


def route_f64(logits, top_k, bias=None, sigmoid=False, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """[(expert, weight, s of every live expert), ...] of every token, from the definition."""
    E = logits.shape[-1]
    b = bias.double().cpu().tolist() if bias is not None else None
    out = []
    for z in logits.double().cpu().reshape(-1, E).tolist():
        live = [i for i in range(E) if z[i] == z[i] and z[i] != -math.inf]
        if sigmoid:
            s = {i: 1 / (1 + math.exp(-z[i])) if z[i] > -700 else 0.0 for i in live}
        else:
            top = max((z[i] for i in live), default=0.0)
            den = math.fsum(math.exp(z[i] - top) for i in live)
            s = {i: math.exp(z[i] - top) / den for i in live}
        rank = dict(s)
        if b:
            live = [i for i in live if b[i] == b[i] and b[i] != -math.inf]
            rank = {i: s[i] + b[i] for i in live}
        if groups > 1:
            per = E // groups
            two = {}
            for i in live:
                two.setdefault(i // per, []).append(rank[i])
            order = sorted(two, key=lambda g: (-sum(sorted(two[g], reverse=True)[:2]), g))
            kept = set(order[:top_groups])
            live = [i for i in live if i // per in kept]
        chosen = sorted(live, key=lambda i: (-(rank[i] if b else z[i]), i))[:top_k]
        # shares by the logarithms of the scores, which do not underflow
        log_s = {i: (-math.log1p(math.exp(-z[i])) if z[i] > -700 else z[i]) if sigmoid else z[i] for i in chosen}
        top = max(log_s.values(), default=0.0)
        total = math.fsum(math.exp(v - top) for v in log_s.values())
        w = [math.exp(log_s[i] - top) / total if renormalize else s[i] for i in chosen]
        out.append(([(i, v * scale) for i, v in zip(chosen, w)], s))
    return out
