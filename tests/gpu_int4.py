"""Inputs and 64-bit references shared by the int4 GEMV and mixture-of-experts tests (no library code)."""

import math

import torch


def make_int4(gen, rows, cols, group, zeros, scale_dtype, device="cuda"):
    """Random codes over the whole range, scales with both signs, zero points over 0..15 with a few far ones:
    (codes [rows, cols], scales [rows, G], zeros [rows, G] or None)."""
    g = -(-cols // group) if group else 1
    q = torch.randint(0, 16, (rows, cols), generator=gen, device=device, dtype=torch.uint8)
    s = (torch.randn((rows, g), generator=gen, device=device) * 0.01).to(scale_dtype)
    z = torch.randint(0, 16, (rows, g), generator=gen, device=device, dtype=torch.uint8) if zeros else None
    if zeros:
        z[::7, ::3] = 255
    return q, s, z


def int4_f64(q, s, z, group):
    """W in 64 bits."""
    cols = q.shape[1]
    gi = torch.arange(cols, device=q.device) // group if group else torch.zeros(cols, dtype=torch.long, device=q.device)
    zz = 8.0 if z is None else z.double()[:, gi]
    return s.double()[:, gi] * (q.double() - zz)


def route_f64(logits, top_k, renormalize):
    """[(expert, weight), ...] of every token, from the definition."""
    out = []
    for row in logits.double().cpu().tolist():
        order = sorted(range(len(row)), key=lambda i: (-row[i], i))
        chosen = [i for i in order[:top_k] if row[i] != -math.inf]
        if not chosen:
            out.append([])
            continue
        top = row[chosen[0]]
        den = math.fsum(math.exp(row[i] - top) for i in (chosen if renormalize else range(len(row))))
        out.append([(i, math.exp(row[i] - top) / den) for i in chosen])
    return out


def moe_f64(x, routes, up_of, down_of):
    """(y, bound) in 64 bits; up_of(e) -> (Wg, Wu) [I, H], down_of(e) -> Wd [H, I], both float64.  bound is the sum
    of the absolute terms of y, taken through both products, that rounding errors are measured against."""
    xd = x.double()
    y = torch.zeros(xd.shape, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(y)
    for t, chosen in enumerate(routes):
        for e, w in chosen:
            wg, wu = up_of(e)
            wd = down_of(e)
            g, u = wg @ xd[t], wu @ xd[t]
            sg = g / (1 + torch.exp(-g))
            y[t] += w * (wd @ (sg * u))
            # |d silu(g)| <= 1.1 |dg|; g, u carry errors relative to the sums of their absolute terms
            ag, au = wg.abs() @ xd[t].abs(), wu.abs() @ xd[t].abs()
            bound[t] += w * (wd.abs() @ (1.1 * ag * u.abs() + sg.abs() * au + (sg * u).abs()))
    return y, bound
