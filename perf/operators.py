"""Cases of the 4-bit serving operators: the decode product with group-scaled
int4 weights and the mixture-of-experts layer for a few tokens, over int4 and NF4
experts.

Each case can run in two forms on the same inputs: plain elementary torch
operations in 32 bits (``own = False``) or the library's calls (``own = True``).
``exact`` gives the results in 64 bits.
"""

import math
import statistics

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# The weights of one decoder layer: q, k, v, o, gate, up, down as [N, K].
_LAYER = [[4096, 4096]] * 4 + [[11008, 4096]] * 2 + [[4096, 11008]]


# ------------------------------------------------------------------ cases
def _gemv(name, shapes, M, group, zeros=True, dtype="bf16", scale_dtype="f16"):
    c = {"op": "gemv_int4", "shapes": ";".join(f"{n}x{k}" for n, k in shapes), "M": M, "group": group,
         "zeros": zeros, "dtype": dtype, "scale_dtype": scale_dtype}
    if name:
        c["name"] = name
    return c


def _moe(name, fmt, T, E, top_k, H, I, group=128, zeros=True, dtype="bf16", scale_dtype="f16", nested=True,
         renormalize=True, logits_dtype="f32", masked=False):
    c = {"op": "moe", "fmt": fmt, "T": T, "E": E, "top_k": top_k, "H": H, "I": I, "group": group, "zeros": zeros,
         "dtype": dtype, "scale_dtype": scale_dtype, "nested": nested, "renormalize": renormalize,
         "logits_dtype": logits_dtype, "masked": masked}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one small projection of a small model: latency of a single call
        _gemv("gemv_1024_m1", [[1024, 1024]], 1, 64),
        # a decoder layer's seven weights for one token, one call
        _gemv("gemv_layer_m1", _LAYER, 1, 128),
        # the widest matrix of a 70B-shaped layer, four sequences decoding together, fp16 activations
        _gemv("gemv_28672_m4", [[28672, 8192]], 4, 128, dtype="f16"),
        # a decoder layer for a full batch of sixteen, symmetric codes in the smallest groups
        _gemv("gemv_layer_m16_g32", _LAYER, 16, 32, zeros=False, scale_dtype="bf16"),
        # odd sizes: no dimension a multiple of anything, one scale per row
        _gemv("gemv_edge_m3", [[3000, 4099]], 3, 0, dtype="f16"),
        # one token through two of eight large experts
        _moe("moe_int4_8x11008_t1", "int4", 1, 8, 2, 4096, 11008),
        # one token through eight of many small experts: the latency end of serving
        _moe("moe_int4_64x1024_t1", "int4", 1, 64, 8, 2048, 1024),
        # sixteen sequences decoding together: most small experts are touched
        _moe("moe_int4_64x1024_t16", "int4", 16, 64, 8, 2048, 1024, zeros=False, scale_dtype="bf16",
             renormalize=False),
        # odd expert sizes in fp16, smallest groups, a router that masks experts and whole tokens
        _moe("moe_int4_edge_t7", "int4", 7, 11, 3, 1001, 777, group=32, dtype="f16", logits_dtype="f16",
             masked=True),
        # experts in the library's own NF4 form with double-quantized scales, one token, small experts
        _moe("moe_nf4_64x1024_t1", "nf4", 1, 64, 8, 2048, 1024, group=64),
        # the same form, large experts, four tokens
        _moe("moe_nf4_8x11008_t4", "nf4", 4, 8, 2, 4096, 11008, group=64),
        # a full batch over small experts with plain fp32 block scales of 128
        _moe("moe_nf4_64x1024_t16", "nf4", 16, 64, 8, 2048, 1024, group=128, nested=False, logits_dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "f16"])
    scale_dtype = rng.choice(["bf16", "f16"])
    zeros = rng.random() < 0.6
    if rng.random() < 0.5:
        group = rng.choice([32, 64, 128, 256, 0])
        shapes = []
        for _ in range(rng.choice([1, 1, 2, 3, 7])):
            n, k = _log_int(rng, 33, 28672), _log_int(rng, 100, 11008)
            if rng.random() < 0.6:
                n, k = max(16, n // 16 * 16), max(128, k // 128 * 128)
            while n * k > 28672 * 8192 // 8:
                n = (n + 1) // 2
            shapes.append([n, k])
        return _gemv(None, shapes, rng.randint(1, 16), group, zeros, dtype, scale_dtype)
    fmt = rng.choice(["int4", "nf4"])
    E = _log_int(rng, 2, 128)
    top_k = rng.randint(1, min(8, E))
    H, I = _log_int(rng, 128, 4096), _log_int(rng, 64, 8192)
    if fmt == "nf4" or rng.random() < 0.5:
        H, I = max(64, H // 64 * 64), max(64, I // 64 * 64)
    while E * H * I > 6 * 4096 * 8192:
        I = max(64, I // 2 // 64 * 64)
        if I == 64:
            E = max(top_k, E // 2)
    group = rng.choice([64, 128, 256]) if fmt == "nf4" else rng.choice([32, 64, 128, 256, 0])
    T = rng.randint(1, 16)
    return _moe(None, fmt, T, E, top_k, H, I, group, zeros, "bf16" if fmt == "nf4" else dtype,
                scale_dtype, rng.random() < 0.5, rng.random() < 0.5, rng.choice(["f32", "bf16", "f16"]),
                T > 1 and rng.random() < 0.3)


def _shapes(case):
    return [[int(v) for v in s.split("x")] for s in case["shapes"].split(";")]


# ------------------------------------------------------------------ inputs
def _randn(gen, shape, sigma, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * sigma).to(dtype)


def _pack(q):
    """codes [N, K] -> bytes [N, stride], first code of a pair in the high nibble, rows padded to 16 bytes"""
    n, k = q.shape
    stride = (-(-k // 2) + 15) // 16 * 16
    p = torch.zeros((n, 2 * stride), dtype=torch.uint8, device=q.device)
    p[:, :k] = q
    return (p[:, 0::2] << 4) | p[:, 1::2]


def _int4_of(w, group, zeros, scale_dtype):
    """round-to-nearest group quantization of w [N, K] (fp32): (codes, scales, zeros or None)"""
    n, k = w.shape
    g = group if group else k
    pad = -(-k // g) * g
    wp = torch.zeros((n, pad), dtype=torch.float32, device=w.device)
    wp[:, :k] = w
    wg = wp.view(n, pad // g, g)
    if zeros:
        lo, hi = wg.amin(2).clamp(max=0.0), wg.amax(2).clamp(min=0.0)
        s = ((hi - lo) / 15).to(scale_dtype)
        z = torch.round(-lo / s.float().clamp(min=1e-20)).clamp(0, 15)
    else:
        s = (wg.abs().amax(2) / 7).to(scale_dtype)
        z = torch.full_like(s, 8.0, dtype=torch.float32)
    q = (torch.round(wg / s.float().clamp(min=1e-20).unsqueeze(2)) + z.unsqueeze(2)).clamp(0, 15)
    q = q.view(n, pad)[:, :k].to(torch.uint8)
    return _pack(q), s.contiguous(), z.to(torch.uint8).contiguous() if zeros else None


def _nf4_levels():
    nd = statistics.NormalDist()
    top = nd.inv_cdf(31 / 32)
    return torch.tensor([nd.inv_cdf((2 * i + 1) / 32) / top for i in range(16)], dtype=torch.float64).float()


def _nf4_of(w, block, levels):
    """(codes, absmax) of the flattened w, nearest level"""
    wb = w.reshape(-1, block)
    a = wb.abs().amax(1)
    t = wb / a.clamp(min=1e-30).unsqueeze(1)
    mid = (levels[1:] + levels[:-1]) / 2
    q = torch.bucketize(t, mid).to(torch.uint8).view(-1)
    return (q[0::2] << 4) | q[1::2], a


def _double_quant(absmax):
    nb = absmax.numel()
    mean = absmax.mean().reshape(1)
    c = torch.zeros(-(-nb // 256) * 256, dtype=torch.float32, device=absmax.device)
    c[:nb] = absmax - mean
    c = c.view(-1, 256)
    s = c.abs().amax(1)
    q8 = torch.round(c / s.clamp(min=1e-30).unsqueeze(1) * 127).to(torch.int8).view(-1)[:nb].contiguous()
    return q8, (s / 127).contiguous(), mean


def _experts_int4(gen, E, rows, cols, case):
    parts = [_int4_of(_randn(gen, (rows, cols), 0.02, torch.float32), case["group"], case["zeros"],
                      _DT[case["scale_dtype"]]) for _ in range(E)]
    return {"codes": torch.cat([p[0] for p in parts]), "scales": torch.cat([p[1] for p in parts]),
            "zeros": torch.cat([p[2] for p in parts]) if case["zeros"] else None,
            "rows": rows * E, "cols": cols}


def _experts_nf4(gen, E, rows, cols, case, levels):
    # rows * cols is a multiple of 64 * 64, so no block crosses from one expert into the next
    parts = [_nf4_of(_randn(gen, (rows, cols), 0.02, torch.bfloat16).float(), case["group"], levels)
             for _ in range(E)]
    codes, absmax = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    w = {"codes": codes, "absmax": absmax, "rows": rows * E, "cols": cols}
    if case["nested"]:
        w["q8"], w["dq_scale"], w["dq_mean"] = _double_quant(absmax)
        w["absmax"] = None
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]
    st = {"case": case}
    if case["op"] == "gemv_int4":
        st["w"], st["x"] = [], []
        for n, k in _shapes(case):
            codes, scales, zeros = _int4_of(_randn(gen, (n, k), 0.02, torch.float32), case["group"], case["zeros"],
                                            _DT[case["scale_dtype"]])
            st["w"].append({"codes": codes, "scales": scales, "zeros": zeros, "rows": n, "cols": k})
            st["x"].append(_randn(gen, (case["M"], k), 1.0, dt))
    else:
        E, H, I = case["E"], case["H"], case["I"]
        if case["fmt"] == "int4":
            st["up"] = _experts_int4(gen, E, 2 * I, H, case)
            st["down"] = _experts_int4(gen, E, H, I, case)
        else:
            st["levels"] = _nf4_levels().cuda()
            st["up"] = _experts_nf4(gen, E, 2 * I, H, case, st["levels"])
            st["down"] = _experts_nf4(gen, E, H, I, case, st["levels"])
        st["x"] = _randn(gen, (case["T"], H), 1.0, dt)
        lg = torch.randn((case["T"], E), generator=gen, device="cuda") * 1.5
        if case["masked"]:
            hide = torch.rand((case["T"], E), generator=gen, device="cuda") < 0.5
            hide[case["T"] // 2] = True                    # a padding token: no expert at all
            lg = lg.masked_fill(hide, float("-inf"))
        st["logits"] = lg.to(_DT[case["logits_dtype"]])
    if own:
        import bit_blockwise_weight_amd as qk
        st["qk"] = qk
        if case["op"] == "gemv_int4":
            st["tasks"] = [(x, qk.qk_int4_state_init(w["rows"], w["cols"], case["group"], w["codes"], w["scales"],
                                                     w["zeros"])) for x, w in zip(st["x"], st["w"])]
        else:
            for name in ("up", "down"):
                w = st[name]
                if case["fmt"] == "int4":
                    st[name + "_state"] = qk.qk_int4_state_init(w["rows"], w["cols"], case["group"], w["codes"],
                                                                w["scales"], w["zeros"])
                else:
                    st[name + "_state"] = qk.qk_state_init(
                        qk.NF4, st["levels"], w["rows"], w["cols"], case["group"], w["codes"], w["absmax"],
                        w.get("q8"), w.get("dq_scale"), w.get("dq_mean"))
    return st


# ------------------------------------------------------------------ plain form
def _plain_int4(w, row0, rows, case):
    cols = w["cols"]
    b = w["codes"][row0:row0 + rows]
    q = torch.stack((b >> 4, b & 15), 2).view(rows, -1)[:, :cols].float()
    g = case["group"] if case["group"] else cols
    s = w["scales"][row0:row0 + rows].float().repeat_interleave(g, 1)[:, :cols]
    if w["zeros"] is None:
        return (q - 8.0) * s
    return (q - w["zeros"][row0:row0 + rows].float().repeat_interleave(g, 1)[:, :cols]) * s


def _plain_nf4(w, row0, rows, case, levels):
    cols = w["cols"]
    e0, n = row0 * cols, rows * cols                        # cols is even: an expert's rows start on a byte
    b = w["codes"][e0 // 2:(e0 + n) // 2]
    lv = levels.to(torch.bfloat16).float()                  # the 4-bit products read the levels in bf16
    v = torch.stack((lv[(b >> 4).int()], lv[(b & 15).int()]), 1).view(-1)
    blk = torch.arange(e0, e0 + n, device=b.device) // case["group"]
    if w["absmax"] is None:
        a = w["q8"].float() * w["dq_scale"].repeat_interleave(256)[:w["q8"].numel()] + w["dq_mean"]
    else:
        a = w["absmax"]
    return (v * a[blk]).view(rows, cols)


def _plain_moe(st):
    case = st["case"]
    E, I, H = case["E"], case["I"], case["H"]
    x = st["x"].float()
    lg = st["logits"].float()
    top, ids = torch.sort(lg, dim=1, descending=True, stable=True)
    top, ids = top[:, :case["top_k"]], ids[:, :case["top_k"]]
    m = top[:, :1]
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(top - m)
    den = p.sum(1, keepdim=True) if case["renormalize"] else torch.exp(lg - m).sum(1, keepdim=True)
    p = torch.where(den > 0, p / den, torch.zeros_like(p))
    y = torch.zeros((x.shape[0], H), dtype=torch.float32, device=x.device)
    for e in range(E):
        we = (p * (ids == e)).sum(1, keepdim=True)
        if case["fmt"] == "int4":
            up, down = _plain_int4(st["up"], e * 2 * I, 2 * I, case), _plain_int4(st["down"], e * H, H, case)
        else:
            up = _plain_nf4(st["up"], e * 2 * I, 2 * I, case, st["levels"])
            down = _plain_nf4(st["down"], e * H, H, case, st["levels"])
        gu = x @ up.t()
        g, u = gu[:, :I], gu[:, I:]
        h = g / (1 + torch.exp(-g)) * u
        y = y + we * (h @ down.t())
    return y.to(st["x"].dtype)


def run(state):
    case = state["case"]
    if own:
        qk = state["qk"]
        if case["op"] == "gemv_int4":
            if len(state["tasks"]) == 1:
                return qk.qk_gemv_int4(*state["tasks"][0])
            return qk.qk_gemv_int4_grouped(state["tasks"])
        call = qk.qk_moe_int4 if case["fmt"] == "int4" else qk.qk_moe_nf4
        return call(state["x"], state["logits"], case["top_k"], state["up_state"], state["down_state"],
                    renormalize=case["renormalize"])
    if case["op"] == "gemv_int4":
        ys = [(x.float() @ _plain_int4(w, 0, w["rows"], case).t()).to(x.dtype)
              for x, w in zip(state["x"], state["w"])]
        return ys[0] if len(ys) == 1 else ys
    return _plain_moe(state)


# ------------------------------------------------------------------ work of one pass
def _int4_bytes(rows, cols, case):
    groups = -(-cols // case["group"]) if case["group"] else 1
    return rows * (-(-cols // 2)) + rows * groups * (3 if case["zeros"] else 2)


def _nf4_bytes(rows, cols, case):
    nb = rows * cols / case["group"]
    return rows * cols / 2 + nb * (1 + 4 / 256 if case["nested"] else 4)


def work(case):
    if case["op"] == "gemv_int4":
        b = f = 0
        for n, k in _shapes(case):
            b += _int4_bytes(n, k, case) + 2 * case["M"] * (n + k)
            f += 2 * case["M"] * n * k
        return {"bytes": b, "flops": f}
    T, E, k, H, I = case["T"], case["E"], case["top_k"], case["H"], case["I"]
    live, avail = T, E
    if case["masked"]:
        live, avail = max(T - 1, 0), max(E // 2, 1)
        k = min(k, avail)
    touched = E * (1 - (1 - k / E) ** live)                 # distinct experts that random routing reaches
    one = _int4_bytes if case["fmt"] == "int4" else _nf4_bytes
    per_expert = one(2 * I, H, case) + one(H, I, case)
    el = 4 if case["logits_dtype"] == "f32" else 2
    return {"bytes": int(touched * per_expert + 4 * T * H + el * T * E), "flops": 2 * live * k * 3 * H * I}


# ------------------------------------------------------------------ 64-bit results
def _exact_w(w, r0, rows, case, levels):
    """rows of a 4-bit weight as float64, from the definition element by element"""
    cols, grp = w["cols"], case["group"]
    dev = w["codes"].device
    r = torch.arange(r0, r0 + rows, device=dev).unsqueeze(1)
    c = torch.arange(cols, device=dev).unsqueeze(0)
    if case["op"] == "gemv_int4" or case["fmt"] == "int4":
        byte = w["codes"].index_select(0, r.view(-1)).index_select(1, (c // 2).view(-1))
        q = torch.where(c % 2 == 0, byte // 16, byte % 16).double()
        gi = (c // grp if grp else torch.zeros_like(c)).view(-1)
        s = w["scales"].index_select(0, r.view(-1)).double().index_select(1, gi)
        z = 8.0 if w["zeros"] is None else w["zeros"].index_select(0, r.view(-1)).double().index_select(1, gi)
        return s * (q - z)
    e = r * cols + c
    byte = w["codes"][e // 2]
    q = torch.where(e % 2 == 0, byte // 16, byte % 16).long()
    del byte
    lv = levels.bfloat16().double()
    blk = e // grp
    del e
    if w["absmax"] is None:
        a = w["q8"].double() * w["dq_scale"].double()[torch.arange(w["q8"].numel(), device=dev) // 256] \
            + w["dq_mean"].double()
    else:
        a = w["absmax"].double()
    return lv[q] * a[blk]


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "gemv_int4":
        ys = []
        for x, w in zip(st["x"], st["w"]):
            step = max(1, (1 << 26) // w["cols"])
            ys.append(torch.cat([x.double() @ _exact_w(w, r, min(step, w["rows"] - r), case, None).t()
                                 for r in range(0, w["rows"], step)], 1))
        return ys[0] if len(ys) == 1 else ys
    H, I, k = case["H"], case["I"], case["top_k"]
    lg = st["logits"].double().cpu().tolist()
    x = st["x"].double()
    y = torch.zeros((case["T"], H), dtype=torch.float64, device=x.device)
    todo = {}
    for t, row in enumerate(lg):
        order = sorted(range(len(row)), key=lambda i: (-row[i], i))
        chosen = [i for i in order[:k] if row[i] != -math.inf]
        if not chosen:
            continue
        top = row[chosen[0]]
        over = chosen if case["renormalize"] else range(len(row))
        den = math.fsum(math.exp(row[i] - top) for i in over)
        for i in chosen:
            todo.setdefault(i, []).append((t, math.exp(row[i] - top) / den))
    for e, users in todo.items():
        up = _exact_w(st["up"], e * 2 * I, 2 * I, case, st.get("levels"))
        rows = torch.tensor([t for t, _ in users], device=x.device)
        p = torch.tensor([v for _, v in users], dtype=torch.float64, device=x.device).unsqueeze(1)
        gu = x[rows] @ up.t()
        del up
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        y[rows] += p * (h @ _exact_w(st["down"], e * H, H, case, st.get("levels")).t())
    return y
