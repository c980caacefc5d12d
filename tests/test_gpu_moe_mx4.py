"""The experts' products over a routing, microscaled, on the GPU against 64-bit references, and the whole layer as it is used."""

import pytest
import torch

import bit_blockwise_weight_amd as qk
from gpu_mx4 import check, make_mx4, product_bound, values

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ids(g, T, top_k, E, none):
    """Distinct experts per token, a few of them popular; some slots, and whole tokens, without one"""
    z = torch.randn((T, E), generator=g, device="cuda") + 2 * torch.randn(E, generator=g, device="cuda")
    ids = torch.sort(z, dim=1, descending=True)[1][:, :top_k].int()
    if none:
        ids[torch.rand((T, top_k), generator=g, device="cuda") < 0.2] = -1
        ids[T // 2] = -1
        ids[0, 0] = E                                            # outside too
    return ids.contiguous()


def _case(T, top_k, E, H, I, seed, none=True):
    g = _gen(seed)
    c = {"ids": _ids(g, T, top_k, E, none), "x": make_mx4(g, T, H, 118, 126), "up": make_mx4(g, E * 2 * I, H, 112, 120),
         "h": make_mx4(g, T * top_k, I, 118, 126, extra=1), "down": make_mx4(g, E * H, I, 112, 120)}
    c["w"] = torch.rand((T, top_k), generator=g, device="cuda")
    return c


def _up_f64(c, T, top_k, E, H, I):
    want = torch.zeros((T * top_k, I), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    x = values(*c["x"], H)
    flat = c["ids"].view(-1)
    for e in range(E):
        s = torch.nonzero(flat == e).view(-1)
        if s.numel() == 0:
            continue
        w = values(c["up"][0][e * 2 * I:(e + 1) * 2 * I], c["up"][1][e * 2 * I:(e + 1) * 2 * I], H)
        xe = x[s // top_k]
        g, u = xe @ w[:I].t(), xe @ w[I:].t()
        bg, bu = product_bound(xe, w[:I], H), product_bound(xe, w[I:], H)
        sg = torch.nn.functional.silu(g)
        want[s] = sg * u
        # |d silu| <= 1.1 |dg|; silu in fp32: the exponential to 2 steps, a sum, a quotient, a product
        bound[s] = 1.1 * bg * (u.abs() + bu) + sg.abs() * bu + (sg * u).abs() * 8 * 2.0 ** -24
    return want, bound


def _down_f64(c, T, top_k, E, H, I):
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    h = values(*c["h"], I)
    flat, wt = c["ids"].view(-1), c["w"].double().view(-1)
    for e in range(E):
        s = torch.nonzero(flat == e).view(-1)
        if s.numel() == 0:
            continue
        w = values(c["down"][0][e * H:(e + 1) * H], c["down"][1][e * H:(e + 1) * H], I)
        he, ws = h[s], wt[s].unsqueeze(1)
        want.index_add_(0, s // top_k, ws * (he @ w.t()))
        bound.index_add_(0, s // top_k, ws * (product_bound(he, w, I) + (he.abs() @ w.abs().t()) * (top_k + 1) * 2.0 ** -24))
    return want, bound


def _run(c, T, top_k, E, H, I, dtype):
    plan = qk.qk_moe_plan(c["ids"], E)
    buf = torch.full((T * top_k * I + 32,), 77.0, dtype=dtype, device="cuda")
    h = qk.qk_moe_up_mx4(qk.qk_mx4_state_init(T, H, *c["x"]), qk.qk_mx4_state_init(E * 2 * I, H, *c["up"]), plan, dtype,
                         buf[:T * top_k * I].view(T * top_k, I))
    assert bool((buf[T * top_k * I:] == 77.0).all())
    out = torch.full((T * H + 32,), 77.0, dtype=dtype, device="cuda")
    w = c["w"].clone()
    w[(c["ids"] < 0) | (c["ids"] >= E)] = float("nan")           # weights of slots without an expert do not matter
    ws = torch.full((qk.qk_moe_down_mx4_workspace_size(T, top_k, H),), 0xFF, dtype=torch.uint8, device="cuda")
    hs = c["h"][1].clone()
    hs[((c["ids"] < 0) | (c["ids"] >= E)).view(-1)] = 255        # nor what h holds there
    y = qk.qk_moe_down_mx4(qk.qk_mx4_state_init(T * top_k, I, c["h"][0], hs), qk.qk_mx4_state_init(E * H, I, *c["down"]), plan, w,
                           dtype, out[:T * H].view(T, H), ws)
    assert bool((out[T * H:] == 77.0).all())
    return h, y


@pytest.mark.parametrize("T,top_k,E,H,I", [(1, 1, 1, 32, 16), (1, 8, 64, 512, 128), (2, 2, 3, 100, 33), (7, 3, 11, 1001, 77),
                                           (16, 4, 8, 260, 130), (40, 2, 4, 513, 200), (100, 4, 6, 256, 64), (200, 2, 5, 300, 150),
                                           (300, 6, 6, 1000, 129), (1000, 2, 3, 257, 300), (900, 8, 16, 512, 128),
                                           (33, 32, 40, 64, 16), (5, 1, 512, 96, 40)])
def test_experts(T, top_k, E, H, I):
    c = _case(T, top_k, E, H, I, T + E)
    h, y = _run(c, T, top_k, E, H, I, torch.float32)
    flat = c["ids"].view(-1)
    assert float(h[(flat < 0) | (flat >= E)].abs().sum()) == 0.0
    check(h, *_up_f64(c, T, top_k, E, H, I), torch.float32, "up")
    check(y, *_down_f64(c, T, top_k, E, H, I), torch.float32, "down")


@pytest.mark.parametrize("T,top_k,E,H,I", [(1500, 2, 4, 300, 1500), (1500, 2, 4, 3001, 130), (400, 8, 64, 300, 500),
                                           (400, 8, 64, 1100, 90), (2600, 1, 3, 700, 1290)])
def test_more_tiles_than_workgroups(T, top_k, E, H, I):
    """A workgroup makes several tiles, some of them of slots without an expert."""
    c = _case(T, top_k, E, H, I, T + E + H)
    h, y = _run(c, T, top_k, E, H, I, torch.float32)
    flat = c["ids"].view(-1)
    assert float(h[(flat < 0) | (flat >= E)].abs().sum()) == 0.0
    check(h, *_up_f64(c, T, top_k, E, H, I), torch.float32, "up")
    check(y, *_down_f64(c, T, top_k, E, H, I), torch.float32, "down")


@pytest.mark.parametrize("K", [1, 32, 255, 256, 257, 512, 513, 770, 1030, 1290, 1536, 1540, 1800, 2049, 3100])
@pytest.mark.parametrize("T", [60, 300])
def test_experts_lengths(T, K):
    E, top_k = 2, 2
    c = _case(T, top_k, E, K, 72, T + K)
    h, _ = _run(c, T, top_k, E, K, 72, torch.float32)
    check(h, *_up_f64(c, T, top_k, E, K, 72), torch.float32, "up")
    c = _case(T, top_k, E, 72, K, T + K + 1)
    _, y = _run(c, T, top_k, E, 72, K, torch.float32)
    check(y, *_down_f64(c, T, top_k, E, 72, K), torch.float32, "down")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 9, 90, 600])
def test_experts_in_16_bits(dtype, T):
    E, top_k, H, I = 4, 2, 384, 96
    c = _case(T, top_k, E, H, I, T)
    h, y = _run(c, T, top_k, E, H, I, DT[dtype])
    check(h, *_up_f64(c, T, top_k, E, H, I), DT[dtype], "up")
    check(y, *_down_f64(c, T, top_k, E, H, I), DT[dtype], "down")


@pytest.mark.parametrize("T", [3, 50, 400])
def test_all_tokens_on_one_expert_and_none(T):
    E, top_k, H, I = 6, 2, 200, 100
    c = _case(T, top_k, E, H, I, T, none=False)
    c["ids"][:, 0], c["ids"][:, 1] = 5, 5                        # the same expert twice
    h, y = _run(c, T, top_k, E, H, I, torch.float32)
    check(h, *_up_f64(c, T, top_k, E, H, I), torch.float32)
    check(y, *_down_f64(c, T, top_k, E, H, I), torch.float32)
    c["ids"].fill_(-1)
    h, y = _run(c, T, top_k, E, H, I, torch.float32)
    assert float(h.abs().max()) == 0.0 and float(y.abs().max()) == 0.0


def test_a_slot_does_not_depend_on_the_others_values():
    T, top_k, E, H, I = 60, 2, 4, 512, 64
    c = _case(T, top_k, E, H, I, 3, none=False)
    h, y = _run(c, T, top_k, E, H, I, torch.bfloat16)
    c["x"][1][1:] = 255
    c["h"][1][top_k:] = 255
    h2, y2 = _run(c, T, top_k, E, H, I, torch.bfloat16)
    assert torch.equal(h2[:top_k], h[:top_k]) and torch.equal(y2[0], y[0]) and bool(torch.isnan(h2[top_k:]).all())


def _layer_inputs(g, T, E, top_k, H, I, dtype):
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    router = torch.randn((E, H), generator=g, device="cuda").to(dtype) * H ** -0.5
    up = qk.quantize_mx4((torch.randn((E * 2 * I, H), generator=g, device="cuda") * 0.05).to(dtype))
    down = qk.quantize_mx4((torch.randn((E * H, I), generator=g, device="cuda") * 0.05).to(dtype))
    return x, router, up, down


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 24, 500])
def test_layer_as_used(dtype, T):
    """Router, plan, quantization, products: the layer against the same steps in 64 bits from the library's own quantized
    operands."""
    dt = DT[dtype]
    E, top_k, H, I = 16, 4, 512, 160
    g = _gen(T)
    x, router, up, down = _layer_inputs(g, T, E, top_k, H, I, dt)
    logits = (x.float() @ router.float().t())
    bias = torch.randn(E, generator=g, device="cuda") * 0.05
    ids, w = qk.qk_moe_route(logits, top_k, bias, qk.SIGMOID, groups=4, top_groups=2, scale=2.5)
    y = qk.moe_mx4(x, ids, w, up, down)
    xq = qk.quantize_mx4(x)
    c = {"ids": ids, "x": (xq.codes, xq.scales), "up": (up.codes, up.scales), "down": (down.codes, down.scales), "w": w}
    h = qk.qk_moe_up_mx4(xq.state, up.state, qk.qk_moe_plan(ids, E), dt)
    check(h, *_up_f64(c, T, top_k, E, H, I), dt, "up")
    hq = qk.quantize_mx4(h)
    c["h"] = (hq.codes, hq.scales)
    check(y, *_down_f64(c, T, top_k, E, H, I), dt, "down")


def test_layer_captured_and_replayed():
    T, E, top_k, H, I = 30, 8, 2, 256, 96
    g = _gen(50)
    x, router, up, down = _layer_inputs(g, T, E, top_k, H, I, torch.bfloat16)
    rt = router.float().t().contiguous()

    def layer():
        ids, w = qk.qk_moe_route(x.float() @ rt, top_k)
        return qk.moe_mx4(x, ids, w, up, down)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for _ in range(3):
        x.copy_(torch.randn((T, H), generator=g, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer())


def test_two_layers_at_once():
    T, E, top_k, H, I = 64, 8, 2, 512, 128
    g = _gen(51)
    a, b = (_layer_inputs(g, T, E, top_k, H, I, torch.bfloat16) for _ in range(2))
    routes = [qk.qk_moe_route(x.float() @ r.float().t(), top_k) for x, r, _, _ in (a, b)]
    want = [qk.moe_mx4(x, i, w, u, d) for (x, _, u, d), (i, w) in zip((a, b), routes)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(4):
        for n, ((x, _, u, d), (i, w)) in enumerate(zip((a, b), routes)):
            with torch.cuda.stream(streams[n]):
                got[n] = qk.moe_mx4(x, i, w, u, d)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_stack_past_32_bits():
    """Stacked experts of more than 4 GiB of codes; only the last expert's weights are not zero."""
    E, H, I = 330, 4096, 4096
    up = torch.zeros((E * 2 * I, H // 2), dtype=torch.uint8, device="cuda")
    us = torch.full((E * 2 * I, H // 32), 120, dtype=torch.uint8, device="cuda")
    g = _gen(52)
    tc, ts = make_mx4(g, 2 * I, H, 112, 120)
    up[-2 * I:], us[-2 * I:] = tc, ts
    for T in (2, 300):
        x = make_mx4(g, T, H, 118, 126)
        ids = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
        ids[0] = 7
        h = qk.qk_moe_up_mx4(qk.qk_mx4_state_init(T, H, *x), qk.qk_mx4_state_init(E * 2 * I, H, up, us), qk.qk_moe_plan(ids, E))
        assert float(h[0].abs().max()) == 0.0
        c = {"ids": torch.zeros((1, 1), dtype=torch.int32, device="cuda"), "x": (x[0][1:2], x[1][1:2]), "up": (tc, ts)}
        check(h[1:2], *_up_f64(c, 1, 1, 1, H, I), torch.bfloat16)


def test_more_outputs_than_a_launch_has_threads_for():
    T, I, H = (1 << 18) + 1, 32, 1 << 16
    g = _gen(53)
    h, down = make_mx4(g, T, I, 118, 126), make_mx4(g, H, I, 112, 120)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    w = torch.rand((T, 1), generator=g, device="cuda")
    y = qk.qk_moe_down_mx4(qk.qk_mx4_state_init(T, I, *h), qk.qk_mx4_state_init(H, I, *down), qk.qk_moe_plan(ids, 1), w)
    for r in (slice(0, 3), slice((1 << 16) - 2, (1 << 16) + 2), slice(T - 2, T)):
        c = {"ids": ids[r], "h": (h[0][r], h[1][r]), "down": down, "w": w[r]}
        check(y[r], *_down_f64(c, r.stop - r.start, 1, 1, H, I), torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 60, 300])
def test_gates_of_every_size(dtype, T):
    """SwiGLU of gates to the largest numbers and past them: each gate is one weight times 1."""
    I, H = 32, 32
    scales = [253, 252, 251, 254, 250, 134, 131, 129, 128, 127, 124, 100, 20, 1]
    codes = [5, 7, 7, 7, 4, 7, 7, 5, 7, 2, 1, 3, 6, 2]               # 2.55e38 twice, 1.28e38, infinite, 2.1e37, 768, 96, 12, ...
    up = torch.zeros((2 * I, 16), dtype=torch.uint8, device="cuda")
    us = torch.full((2 * I, 4), 127, dtype=torch.uint8, device="cuda")
    for i in range(I):
        up[i, 0] = codes[i // 2 % 14] | 8 * (i % 2)
        us[i, 0] = scales[i // 2 % 14]
        up[I + i, 0], us[I + i, 0] = 2, 124                         # the up product: 1/8
    x = torch.zeros((T, 16), dtype=torch.uint8, device="cuda")
    x[:, 0] = 2
    xs = torch.full((T, 4), 127, dtype=torch.uint8, device="cuda")
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    h = qk.qk_moe_up_mx4(qk.qk_mx4_state_init(T, H, x, xs), qk.qk_mx4_state_init(2 * I, H, up, us), qk.qk_moe_plan(ids, 1), DT[dtype])
    gate = values(up[:I], us[:I], H)[:, 0]
    gate = torch.where(gate.abs() >= 2.0 ** 128, gate.sign() * float("inf"), gate)
    # x / (1 + exp(-x)) but for -inf, which has no value in fp32
    want = torch.nn.functional.silu(gate) * 0.125
    there = gate != float("-inf")
    got, want = h[:, there].double(), want[there].expand(T, -1)
    assert torch.equal(torch.isinf(got), torch.isinf(want)) and not bool(torch.isnan(got).any())
    fin = torch.isfinite(want)
    # silu in fp32: the exponential to 2 steps (none below 2^-126), a sum, a quotient, a product; in 16 bits the exponential's
    # rounded exponent, |g| of it
    size = want.abs() * (8 + (0 if dtype == "f32" else 2 * 96)) * 2.0 ** -24 + 96 * 0.125 * 2.0 ** -126
    check(h[:, there][fin], want[fin], size[fin], DT[dtype])


@pytest.mark.parametrize("T,top_k,E,H,I", [(1, 2, 3, 40, 4099), (20, 2, 4, 130, 3000), (500, 2, 2, 200, 1000), (900, 4, 8, 300, 2050),
                                           (4000, 1, 2, 2100, 600)])
def test_down_of_whole_numbers_is_exact(T, top_k, E, H, I):
    """Sums below 2^24 units: nothing may be lost, however small beside the rest."""
    g = _gen(T + I)
    c = {"ids": _ids(g, T, top_k, E, True), "h": make_mx4(g, T * top_k, I, 127, 128), "down": make_mx4(g, E * H, I, 126, 127)}
    c["w"] = torch.randint(1, 5, (T, top_k), generator=g, device="cuda").float()
    y = qk.qk_moe_down_mx4(qk.qk_mx4_state_init(T * top_k, I, *c["h"]), qk.qk_mx4_state_init(E * H, I, *c["down"]),
                           qk.qk_moe_plan(c["ids"], E), c["w"], torch.float32)
    want, bound = _down_f64(c, T, top_k, E, H, I)
    # multiples of 1/8; the bound holds the sums of absolute values, 2 I 2^-24 of them and more
    assert float(bound.max()) * 2 ** 24 / (2 * I) * 8 < 2 ** 24
    assert torch.equal(y.double(), want)
