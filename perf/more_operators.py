"""Cases of the microscaled 4-bit operators and of the experts' routing: quantization
of rows into groups of 32 e2m1 values with a power-of-two scale each, the products of
two such matrices and of 16-bit rows with one, the router of a mixture-of-experts
layer with its gradient, and the experts' products over a routing.

Each case can run in two forms on the same inputs: plain elementary torch operations
(``own = False``) or the library's calls (``own = True``).  ``exact`` gives the results
in 64 bits.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ cases
def _named(case, name):
    if name:
        case["name"] = name
    return case


def _quant(name, rows, cols, dtype="bf16", pitch=0):
    return _named({"op": "quantize", "rows": rows, "cols": cols, "dtype": dtype, "pitch": pitch}, name)


def _gemm(name, M, N, K, dtype="bf16"):
    return _named({"op": "gemm", "M": M, "N": N, "K": K, "dtype": dtype}, name)


def _gemv(name, M, N, K, dtype="bf16"):
    return _named({"op": "gemv", "M": M, "N": N, "K": K, "dtype": dtype}, name)


def _route(name, T, E, top_k, score="softmax", bias=False, groups=1, top_groups=1, renormalize=True, scale=1.0,
           dtype="f32", masked=False, train=False):
    return _named({"op": "route", "T": T, "E": E, "top_k": top_k, "score": score, "bias": bias, "groups": groups,
                   "top_groups": top_groups, "renormalize": renormalize, "scale": scale, "dtype": dtype,
                   "masked": masked, "train": train}, name)


def _experts(name, part, T, E, top_k, H, I, dtype="bf16", masked=False):
    return _named({"op": "experts", "part": part, "T": T, "E": E, "top_k": top_k, "H": H, "I": I, "dtype": dtype,
                   "masked": masked}, name)


def listed():
    return [
        # the activations of one token: latency of the step in front of every product
        _quant("quant_token", 1, 4096),
        # the widest weight of a 70B-shaped layer, quantized when a model is loaded
        _quant("quant_weight", 28672, 8192),
        # a square projection of a 4096-wide layer for a prompt of 4096 tokens
        _gemm("gemm_4096", 4096, 4096, 4096),
        # the widest product of a 70B-shaped layer, 2048 tokens
        _gemm("gemm_28672", 2048, 28672, 8192),
        # odd sizes: neither the weight's rows nor its columns are a multiple of anything
        _gemm("gemm_edge", 512, 3000, 4099, "f16"),
        # a small projection for one token, activations left in 16 bits: latency
        _gemv("gemv_1024_m1", 1, 1024, 1024),
        # the widest matrix of a 70B-shaped layer, four sequences decoding together
        _gemv("gemv_28672_m4", 4, 28672, 8192, "f16"),
        # sixteen sequences decoding together over 64 experts
        _route("route_t16", 16, 64, 8),
        # a training step's router: balanced by a bias, experts in groups, forward and backward
        _route("route_train_t8192", 8192, 256, 8, "sigmoid", True, 8, 4, True, 2.5, "f32", True, True),
        # the gate and up products of one token's eight experts
        _experts("up_64x1024_t1", "up", 1, 64, 8, 2048, 1024),
        # the same layer for a prompt
        _experts("up_64x1024_t4096", "up", 4096, 64, 8, 2048, 1024),
        # the down products and their weighted sums for a prompt over few large experts, some tokens routed nowhere
        _experts("down_8x11008_t512", "down", 512, 8, 2, 4096, 11008, masked=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """a size over the logarithm of the range; half of them multiples of 128 where they are large enough"""
    n = _log_int(rng, lo, hi)
    return n // 128 * 128 if n > 256 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "gemv", "gemv", "route", "route", "experts", "experts"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "quantize":
        rows, cols = _log_int(rng, 1, 8192), _size(rng, 32, 16384)
        while rows * cols > 28672 * 8192 // 4:
            rows = (rows + 1) // 2
        return _quant(None, rows, cols, rng.choice(["bf16", "f16", "f32"]),
                      cols + rng.randint(1, 512) if rng.random() < 0.3 else 0)
    if op == "gemm":
        M, N, K = _log_int(rng, 1, 8192), _size(rng, 33, 16384), _size(rng, 100, 11008)
        while M * N * K > 2048 * 28672 * 8192 // 4:
            M = (M + 1) // 2
        return _gemm(None, M, N, K, dtype)
    if op == "gemv":
        N, K = _size(rng, 33, 28672), _size(rng, 100, 11008)
        while N * K > 28672 * 8192 // 2:
            N = (N + 1) // 2
        return _gemv(None, rng.randint(1, 16), N, K, dtype)
    if op == "route":
        E = _log_int(rng, 2, 512)
        groups = rng.choice([1, 1, 2, 4, 8])
        groups = groups if E >= 4 * groups else 1
        E = E // groups * groups
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, E // groups * top_groups))
        return _route(None, _log_int(rng, 1, 8192), E, top_k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5,
                      groups, top_groups, rng.random() < 0.7, rng.choice([1.0, 2.5]),
                      rng.choice(["f32", "bf16", "f16"]), rng.random() < 0.3, rng.random() < 0.5)
    E = _log_int(rng, 2, 128)
    top_k = rng.randint(1, min(8, E))
    H, I = _size(rng, 128, 4096), _size(rng, 64, 8192)
    while E * H * I > 4 * 4096 * 8192:
        I = max(64, I // 2)
        if I == 64:
            E = max(top_k, E // 2)
    T = _log_int(rng, 1, 4096)
    while T * top_k * H * I > 4096 * 8 * 2048 * 1024 or T * E * H * I > 4096 * 64 * 2048 * 1024:
        T = max(1, T // 2)
    return _experts(None, rng.choice(["up", "down"]), T, E, top_k, H, I, dtype, rng.random() < 0.3)


# ------------------------------------------------------------------ inputs
def _randn(gen, shape, sigma=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * sigma


def _pow2(e):
    """2^e in 64 bits for whole e, put together from its bits"""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _acts(gen, rows, cols):
    """activations: normal values, one column in a hundred twenty times larger"""
    gain = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    return _randn(gen, (rows, cols)) * gain


def _strides(cols):
    return (-(-cols // 2) + 15) // 16 * 16, (-(-cols // 32) + 3) // 4 * 4


def _mx4_of(x):
    """(codes, scales) of x [rows, cols] (fp32), rows padded: per group of 32 the scale 2^(floor(log2 max) - 2) as a
    biased exponent, the values divided by it rounded to e2m1 (to even, at most 6), the first of a pair in the low bits"""
    rows, cols = x.shape
    cs, ss = _strides(cols)
    codes = torch.zeros((rows, cs), dtype=torch.uint8, device=x.device)
    scales = torch.zeros((rows, ss), dtype=torch.uint8, device=x.device)
    groups = -(-cols // 32)
    step = max(1, (1 << 25) // (groups * 32))
    for r in range(0, rows, step):
        v = torch.zeros((min(step, rows - r), groups * 32), dtype=torch.float32, device=x.device)
        v[:, :cols] = x[r:r + step]
        e, q = _mx4_plain(v.view(v.shape[0], groups, 32))
        q = q.view(v.shape[0], -1)
        codes[r:r + step, :groups * 16] = q[:, 0::2] | (q[:, 1::2] << 4)
        scales[r:r + step, :groups] = e
    return codes, scales


def _mx4_plain(v):
    """(biased scale exponent [..., G], codes [..., G, 32]) of fp32 groups [..., G, 32]"""
    a = v.abs()
    top = a.amax(-1)
    e = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)               # the exponent bits are floor(log2) + 127
    # a / 2^(e - 127), in two factors that are both ordinary numbers
    half = 127 - e
    t = a * _pow2(half // 2).float().unsqueeze(-1) * _pow2(half - half // 2).float().unsqueeze(-1)
    code = torch.zeros_like(t, dtype=torch.uint8)
    for mid, closed in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                        (5.0, False)):
        code += (t >= mid) if closed else (t > mid)                    # a tie goes to the even code
    code |= (torch.signbit(v)).to(torch.uint8) << 3
    return e.to(torch.uint8), code


def _weights(gen, rows, cols):
    codes, scales = [], []
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        c, s = _mx4_of(_randn(gen, (min(step, rows - r), cols), 0.02))
        codes.append(c)
        scales.append(s)
    return {"codes": torch.cat(codes), "scales": torch.cat(scales), "rows": rows, "cols": cols}


def _acts_mx4(gen, rows, cols):
    codes, scales = _mx4_of(_acts(gen, rows, cols))
    return {"codes": codes, "scales": scales, "rows": rows, "cols": cols}


def _routing(gen, case):
    """ids [T, k] of distinct experts, some more popular than others, and their weights; tokens routed nowhere"""
    T, E, k = case["T"], case["E"], case["top_k"]
    lg = _randn(gen, (T, E), 1.5) + _randn(gen, (E,), 0.5)
    top, ids = torch.sort(lg, dim=1, descending=True, stable=True)
    w, ids = torch.softmax(top[:, :k], 1), ids[:, :k].int()
    if case["masked"]:
        off = torch.rand((T, 1), generator=gen, device="cuda") < 0.1
        w, ids = w.masked_fill(off, 0.0), ids.masked_fill(off, -1)
    return ids.contiguous(), w.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]
    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        rows, cols, pitch = case["rows"], case["cols"], case["pitch"] or case["cols"]
        if rows < 8192:
            x = _acts(gen, rows, pitch).to(dt)
        else:
            x = torch.cat([_randn(gen, (min(4096, rows - r), pitch), 0.02).to(dt) for r in range(0, rows, 4096)])
        st["x"] = x[:, :cols]                                          # rows of a wider matrix where there is a pitch
    elif op == "gemm":
        st["x"] = _acts_mx4(gen, case["M"], case["K"])
        st["w"] = _weights(gen, case["N"], case["K"])
    elif op == "gemv":
        st["x"] = _acts(gen, case["M"], case["K"]).to(dt)
        st["w"] = _weights(gen, case["N"], case["K"])
    elif op == "route":
        T, E, k = case["T"], case["E"], case["top_k"]
        lg = _randn(gen, (T, E), 1.5)
        if case["masked"]:
            hide = torch.rand((T, E), generator=gen, device="cuda") < 0.2
            hide[T // 2] = True                                        # a padding token: no expert at all
            lg = lg.masked_fill(hide, float("-inf"))
        st["logits"] = lg.to(dt)
        st["bias"] = _randn(gen, (E,), 0.1) if case["bias"] else None
        if case["train"]:
            st["dweights"] = _randn(gen, (T, k), 0.01)
    else:
        T, E, k, H, I = (case[n] for n in ("T", "E", "top_k", "H", "I"))
        st["ids"], st["weights"] = _routing(gen, case)
        if case["part"] == "up":
            st["x"] = _acts_mx4(gen, T, H)
            st["w"] = _weights(gen, E * 2 * I, H)
        else:
            st["x"] = _acts_mx4(gen, T * k, I)
            st["w"] = _weights(gen, E * H, I)
    if own:
        import bit_blockwise_weight_amd as qk
        st["qk"] = qk
        for name in ("x", "w"):
            if isinstance(st.get(name), dict):
                m = st[name]
                st[name + "_state"] = qk.qk_mx4_state_init(m["rows"], m["cols"], m["codes"], m["scales"])
        if op == "experts" and case["part"] == "down":
            st["plan"] = qk.qk_moe_plan(st["ids"], case["E"])          # the layer's first product has made it
    return st


# ------------------------------------------------------------------ plain form
def _values(m, row0=0, rows=None):
    """rows of a microscaled matrix in fp32"""
    rows = m["rows"] if rows is None else rows
    cols, groups = m["cols"], -(-m["cols"] // 32)
    b = m["codes"][row0:row0 + rows, :groups * 16]
    q = torch.stack((b & 15, b >> 4), 2).view(rows, groups, 32)
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float32, device=b.device)
    s = _pow2(m["scales"][row0:row0 + rows, :groups].long() - 127).float()
    return (table[q.int()] * s.unsqueeze(2)).view(rows, groups * 32)[:, :cols]


def _plain_quant(state):
    x = state["x"]
    rows, cols = x.shape
    groups = -(-cols // 32)
    v = torch.zeros((rows, groups * 32), dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    e, q = _mx4_plain(v.view(rows, groups, 32))
    table = torch.tensor(_E2M1 + [-t for t in _E2M1], dtype=torch.float32, device=x.device)
    y = table[q.int()] * _pow2(e.long() - 127).float().unsqueeze(2)
    return [y.view(rows, -1)[:, :cols].to(x.dtype), e]


def _plain_route(state):
    case, lg = state["case"], state["logits"].double()                 # 64 bits: which of two close scores is larger
    T, E, k = case["T"], case["E"], case["top_k"]
    dead = lg == float("-inf")
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-lg))
    else:
        m = lg.amax(1, keepdim=True)
        s = torch.exp(lg - torch.where(m == float("-inf"), torch.zeros_like(m), m))
        total = s.sum(1, keepdim=True)
        s = torch.where(total > 0, s / total, torch.zeros_like(s))
    biased = s if state["bias"] is None else s + state["bias"].double()
    key = lg if state["bias"] is None else biased
    key = key.masked_fill(dead, float("-inf"))
    if case["groups"] > 1:
        g = biased.masked_fill(dead, float("-inf")).view(T, case["groups"], -1)
        two = torch.sort(g, dim=2, descending=True)[0][:, :, :2]
        none = two[:, :, 0] == float("-inf")
        gs = two.masked_fill(two == float("-inf"), 0.0).sum(2).masked_fill(none, float("-inf"))
        best = torch.sort(gs, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter(1, best, True)
        key = key.masked_fill(~keep.repeat_interleave(E // case["groups"], 1), float("-inf"))
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    there = top != float("-inf")
    p = torch.where(there, torch.gather(s, 1, ids), torch.zeros_like(top))
    total = p.sum(1, keepdim=True)
    share = torch.where(total > 0, p / total, torch.zeros_like(p))
    w = (share if case["renormalize"] else p) * case["scale"]
    out = [torch.where(there, ids, torch.full_like(ids, -1)).int(), w.float()]
    if case["train"]:
        dw = torch.where(there, state["dweights"].double() * case["scale"], torch.zeros_like(p))
        if case["renormalize"]:
            dp = torch.where(total > 0, (dw - (dw * share).sum(1, keepdim=True)) / total, torch.zeros_like(p))
        else:
            dp = dw
        if case["score"] == "sigmoid":
            dz = torch.zeros_like(s).scatter(1, ids, dp * p * (1 - p) * there)
        else:
            ds = torch.zeros_like(s).scatter(1, ids, dp * there)
            dz = s * (ds - (dp * p).sum(1, keepdim=True))
        out.append(dz.to(state["logits"].dtype))
    return out


def _plain_experts(state):
    case, ids = state["case"], state["ids"]
    T, E, k, H, I = (case[n] for n in ("T", "E", "top_k", "H", "I"))
    x = _values(state["x"])
    if case["part"] == "up":
        out = torch.zeros((T, k, I), dtype=torch.float32, device=x.device)
        for e in range(E):
            gu = x @ _values(state["w"], e * 2 * I, 2 * I).t()
            g, u = gu[:, :I], gu[:, I:]
            h = g / (1 + torch.exp(-g)) * u
            out = torch.where((ids == e).unsqueeze(2), h.unsqueeze(1), out)
        return out.view(T * k, I).to(_DT[case["dtype"]])
    x = x.view(T, k, I)
    y = torch.zeros((T, H), dtype=torch.float32, device=x.device)
    for e in range(E):
        mine = ids == e
        h = (x * mine.unsqueeze(2)).sum(1)
        y = y + (state["weights"] * mine).sum(1, keepdim=True) * (h @ _values(state["w"], e * H, H).t())
    return y.to(_DT[case["dtype"]])


def run(state):
    case = state["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if own:
        qk = state["qk"]
        if op == "quantize":
            x = state["x"]
            codes, scales = qk.qk_mx4_quantize(x)
            y = qk.qk_mx4_dequantize(qk.qk_mx4_state_init(x.shape[0], x.shape[1], codes, scales), x.dtype)
            return [y, scales[:, :-(-x.shape[1] // 32)]]
        if op == "gemm":
            return qk.qk_gemm_mx4(state["x_state"], state["w_state"], dt)
        if op == "gemv":
            return qk.qk_gemv_mx4(state["x"], state["w_state"])
        if op == "route":
            score = qk.SIGMOID if case["score"] == "sigmoid" else qk.SOFTMAX
            ids, w = qk.qk_moe_route(state["logits"], case["top_k"], state["bias"], score, case["groups"],
                                     case["top_groups"], case["renormalize"], case["scale"])
            if not case["train"]:
                return [ids, w]
            return [ids, w, qk.qk_moe_route_backward(state["logits"], ids, state["dweights"], score,
                                                     case["renormalize"], case["scale"])]
        if case["part"] == "up":
            return qk.qk_moe_up_mx4(state["x_state"], state["w_state"], qk.qk_moe_plan(state["ids"], case["E"]), dt)
        return qk.qk_moe_down_mx4(state["x_state"], state["w_state"], state["plan"], state["weights"], dt)
    if op == "quantize":
        return _plain_quant(state)
    if op == "gemm":
        return (_values(state["x"]) @ _values(state["w"]).t()).to(dt)
    if op == "gemv":
        return (state["x"].float() @ _values(state["w"]).t()).to(dt)
    if op == "route":
        return _plain_route(state)
    return _plain_experts(state)


# ------------------------------------------------------------------ work of one pass
def _mx4_bytes(rows, cols):
    return rows * (-(-cols // 2) + -(-cols // 32))


def work(case):
    op, el = case["op"], 4 if case["dtype"] == "f32" else 2
    if op == "quantize":
        n = case["rows"] * case["cols"]
        # read, written in 4 bits, read again, written
        return {"bytes": 2 * el * n + 2 * _mx4_bytes(case["rows"], case["cols"]), "flops": 4 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _mx4_bytes(M, K) + _mx4_bytes(N, K) + el * M * N, "flops": 2 * M * N * K}
    if op == "gemv":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _mx4_bytes(N, K) + el * M * (N + K), "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["top_k"]
    if op == "route":
        b = T * E * el + T * k * 8 + (4 * E if case["bias"] else 0)
        f = T * E * 8
        if case["train"]:
            b += T * k * 4 + T * E * el
            f += T * E * 4
        return {"bytes": b, "flops": f}
    H, I = case["H"], case["I"]
    live = T * 0.9 if case["masked"] else T
    touched = E * (1 - (1 - k / E) ** live)                            # distinct experts that even routing reaches
    if case["part"] == "up":
        return {"bytes": int(touched * _mx4_bytes(2 * I, H) + _mx4_bytes(T, H) + el * T * k * I + 4 * T * k),
                "flops": int(2 * live * k * 2 * H * I)}
    return {"bytes": int(touched * _mx4_bytes(H, I) + _mx4_bytes(T * k, I) + el * T * H + 8 * T * k),
            "flops": int(2 * live * k * H * I)}


# ------------------------------------------------------------------ 64-bit results
def _exact_values(m, r0=0, rows=None):
    """rows of a microscaled matrix as float64, element by element from the bits of its codes"""
    rows = m["rows"] if rows is None else rows
    k = torch.arange(m["cols"], device=m["codes"].device)
    byte = m["codes"][r0:r0 + rows].index_select(1, k // 2)
    q = torch.where(k % 2 == 0, byte % 16, byte // 16).double()
    del byte
    sign = torch.where(q >= 8, -1.0, 1.0)
    q = q % 8
    ex, man = torch.floor(q / 2), q % 2
    mag = torch.where(ex == 0, man * 0.5, (1 + man / 2) * _pow2(ex - 1))
    s = _pow2(m["scales"][r0:r0 + rows].long() - 127)
    return sign * mag * s.index_select(1, k // 32)


def _exact_product(x, w, r0, rows):
    step = max(1, (1 << 26) // w["cols"])
    return torch.cat([x @ _exact_values(w, r, min(step, r0 + rows - r)).t() for r in range(r0, r0 + rows, step)], 1)


def _exact_quant(x):
    rows, cols = x.shape
    y = torch.empty((rows, cols), dtype=torch.float64, device=x.device)
    e = torch.empty((rows, -(-cols // 32)), dtype=torch.int64, device=x.device)
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    whole = cols // 32 * 32
    for r in range(0, rows, 2048):
        for c0, c1 in ((0, whole), (whole, cols)):
            if c0 == c1:
                continue
            v = x[r:r + 2048, c0:c1].double().reshape(min(2048, rows - r), -1, min(32, c1 - c0))
            top = v.abs().amax(2)
            ex = torch.frexp(top)[1] - 1                               # top = f 2^(ex + 1), f in [1/2, 1)
            ex = torch.where(top > 0, (ex - 2).clamp(min=-127), torch.full_like(ex, -127))
            unit = _pow2(ex).unsqueeze(2)
            t = v.abs() / unit
            hi = torch.bucketize(t.clamp(max=6.0), grid).clamp(max=7)  # the first value not under t
            lo = (hi - 1).clamp(min=0)
            up, down = grid[hi] - t.clamp(max=6.0), t.clamp(max=6.0) - grid[lo]
            q = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
            y[r:r + 2048, c0:c1] = (torch.copysign(grid[q], v) * unit).view(v.shape[0], -1)
            e[r:r + 2048, c0 // 32:-(-c1 // 32)] = ex + 127
    return [y, e.to(torch.uint8)]


def _exact_route(st):
    """token by token on the host"""
    case, k = st["case"], st["case"]["top_k"]
    E, groups = case["E"], case["groups"]
    bias = st["bias"].double().cpu().tolist() if st["bias"] is not None else None
    dws = st["dweights"].double().cpu().tolist() if case["train"] else None
    all_ids, all_w, all_dz = [], [], []
    for t, z in enumerate(st["logits"].double().cpu().tolist()):
        live = [i for i in range(E) if z[i] != -math.inf]
        if case["score"] == "sigmoid":
            s = {i: 1 / (1 + math.exp(-z[i])) for i in live}
        else:
            top = max((z[i] for i in live), default=0.0)
            den = math.fsum(math.exp(z[i] - top) for i in live)
            s = {i: math.exp(z[i] - top) / den for i in live}
        ranked = {i: s[i] + bias[i] for i in live} if bias else s
        if groups > 1:
            per = E // groups
            score = {}
            for i in live:
                score.setdefault(i // per, []).append(ranked[i])
            order = sorted(score, key=lambda g: (-sum(sorted(score[g], reverse=True)[:2]), g))
            kept = set(order[:case["top_groups"]])
            live = [i for i in live if i // per in kept]
        by = ranked if bias else z
        chosen = sorted(live, key=lambda i: (-by[i], i))[:k]
        total = math.fsum(s[i] for i in chosen) if case["renormalize"] else 1.0
        w = [s[i] / total * case["scale"] for i in chosen]
        all_ids.append(chosen + [-1] * (k - len(chosen)))
        all_w.append(w + [0.0] * (k - len(chosen)))
        if case["train"]:
            dw = [v * case["scale"] for v in dws[t][:len(chosen)]]
            if case["renormalize"]:
                mean = math.fsum(a * s[i] / total for a, i in zip(dw, chosen))
                dw = [(a - mean) / total for a in dw]
            dz = [0.0] * E
            if case["score"] == "sigmoid":
                for a, i in zip(dw, chosen):
                    dz[i] = a * s[i] * (1 - s[i])
            else:
                mean = math.fsum(a * s[i] for a, i in zip(dw, chosen))
                for i in s:
                    dz[i] = -s[i] * mean
                for a, i in zip(dw, chosen):
                    dz[i] += s[i] * a
            all_dz.append(dz)
    dev = st["logits"].device
    out = [torch.tensor(all_ids, dtype=torch.int32, device=dev), torch.tensor(all_w, dtype=torch.float64, device=dev)]
    if case["train"]:
        out.append(torch.tensor(all_dz, dtype=torch.float64, device=dev))
    return out


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    op = case["op"]
    if op == "quantize":
        return _exact_quant(st["x"])
    if op == "gemm":
        return _exact_product(_exact_values(st["x"]), st["w"], 0, case["N"])
    if op == "gemv":
        return _exact_product(st["x"].double(), st["w"], 0, case["N"])
    if op == "route":
        return _exact_route(st)
    T, k, H, I = (case[n] for n in ("T", "top_k", "H", "I"))
    flat = st["ids"].view(-1)
    x = _exact_values(st["x"])
    if case["part"] == "up":
        out = torch.zeros((T * k, I), dtype=torch.float64, device=x.device)
    else:
        out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        slots = torch.nonzero(flat == e).view(-1)
        if slots.numel() == 0:
            continue
        if case["part"] == "up":
            gu = _exact_product(x[slots // k], st["w"], e * 2 * I, 2 * I)
            out[slots] = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        else:
            w = st["weights"].view(-1)[slots].double().unsqueeze(1)
            out.index_add_(0, slots // k, w * _exact_product(x[slots], st["w"], e * H, H))
    return out
