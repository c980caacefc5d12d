"""Router of a mixture-of-experts layer, its gradient and the plan, on the GPU against 64-bit references."""

import pytest
import torch

import bit_blockwise_weight_amd as qk
from gpu_mx4 import half_step, route_f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _check(logits, top_k, **kw):
    want = route_f64(logits, top_k, kw.get("bias"), kw.get("score") == qk.SIGMOID, kw.get("groups", 1), kw.get("top_groups", 1),
                     kw.get("renormalize", True), kw.get("scale", 1.0))
    ids, w = qk.qk_moe_route(logits, top_k, **kw)
    gi, gw = ids.cpu().tolist(), w.double().cpu().tolist()
    for t, (chosen, _) in enumerate(want):
        assert gi[t] == [e for e, _ in chosen] + [-1] * (top_k - len(chosen)), t
        for j in range(top_k):
            v = chosen[j][1] if j < len(chosen) else 0.0
            # a score in fp32: the exponential's argument may be off by half a step of the largest logit's size
            assert abs(gw[t][j] - v) <= abs(v) * 2.0 ** -24 * 64 + 1e-44, (t, j, gw[t][j], v)
    return ids, w


@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,top_k", [(1, 1, 1, 1), (2, 1, 1, 2), (7, 1, 1, 3), (64, 1, 1, 8), (65, 1, 1, 4),
                                                       (64, 8, 3, 6), (256, 8, 4, 8), (12, 4, 2, 6), (130, 13, 5, 16),
                                                       (512, 1, 1, 32), (512, 64, 9, 32), (60, 3, 1, 4), (9, 9, 4, 4)])
def test_route(score, renormalize, bias, E, groups, top_groups, top_k):
    g = _gen(E * 131 + top_k)
    z = torch.randn((37, E), generator=g, device="cuda") * 1.5
    b = torch.randn(E, generator=g, device="cuda") * 0.1 if bias else None
    _check(z, top_k, bias=b, score=score, groups=groups, top_groups=top_groups, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
@pytest.mark.parametrize("groups", [1, 4])
def test_ties_go_to_the_lower_index(dtype, score, groups):
    g = _gen(1)
    z = (torch.randint(-3, 4, (200, 32), generator=g, device="cuda").float() * 0.5).to(DT[dtype])
    _check(z, 7, score=score, groups=groups, top_groups=min(groups, 2))
    b = torch.randint(0, 2, (32,), generator=g, device="cuda").float() * 0.25
    _check(z, 7, score=score, bias=b, groups=groups, top_groups=min(groups, 2))
    _check(torch.zeros((3, 32), device="cuda").to(DT[dtype]), 9, score=score, groups=groups, top_groups=min(groups, 3))


@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
def test_close_ranks_are_told_apart(score):
    """Scores that round to the same fp32 number, and to neighbouring ones."""
    g = _gen(2)
    z = 17.0 + torch.randint(0, 9, (64, 40), generator=g, device="cuda").float() * 2.0 ** -19
    _check(z, 12, score=score)
    b = torch.full((40,), 0.125, device="cuda")
    _check(z, 12, score=score, bias=b)
    # ranks s + bias closer than a step of fp32
    z = torch.randn((64, 40), generator=g, device="cuda")
    near = torch.sigmoid(z[0].double()) if score == qk.SIGMOID else torch.softmax(z[0].double(), 0)
    z[1:] = z[0]
    b = (1.0 - near + torch.randn(40, generator=g, device="cuda").double() * 1e-9).float()
    _check(z, 12, score=score, bias=b)
    _check(z, 12, score=score, bias=b, groups=8, top_groups=4)


@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("bias", [False, True])
def test_masks(score, groups, bias):
    g = _gen(3)
    z = torch.randn((60, 32), generator=g, device="cuda")
    z[torch.rand((60, 32), generator=g, device="cuda") < 0.6] = float("-inf")
    z[5] = float("-inf")
    z[6] = float("nan")
    z[7, 1:] = float("-inf")
    z[8, :24] = float("-inf")
    z[9, ::2] = float("nan")
    z[10] = torch.finfo(torch.float32).min                       # the lowest finite value masks nothing
    z[11, 4:] = torch.finfo(torch.float32).min
    b = torch.randn(32, generator=g, device="cuda") * 0.1 if bias else None
    if bias:
        b[3], b[20] = float("-inf"), float("nan")
    for renormalize in (True, False):
        ids, w = _check(z, 6, score=score, bias=b, groups=groups, top_groups=min(groups, 2), renormalize=renormalize)
    assert bool((ids[5] == -1).all()) and bool((ids[6] == -1).all()) and float(w[5:7].abs().max()) == 0.0


def test_infinite_logit_counts_as_the_largest_number():
    z = torch.zeros((2, 8), device="cuda")
    z[0, 5] = float("inf")
    z[1, 2], z[1, 6] = float("inf"), float("inf")
    ids, w = qk.qk_moe_route(z, 2)
    assert ids.tolist() == [[5, 0], [2, 6]] and w.tolist() == [[1.0, 0.0], [0.5, 0.5]]
    ids, w = qk.qk_moe_route(z, 2, score=qk.SIGMOID, renormalize=False)
    assert ids.tolist() == [[5, 0], [2, 6]] and w.tolist() == [[1.0, 0.5], [1.0, 1.0]]


def test_scores_too_small_for_a_number_keep_their_shares():
    z = torch.tensor([[-1000.0, -1001.0, -1003.0, -2000.0], [-60.0, -61.0, -60.5, -100.0]], device="cuda")
    _check(z, 3, score=qk.SIGMOID)
    b = torch.tensor([0.0, 0.0, 0.0, 1.0], device="cuda")
    _check(z, 2, score=qk.SIGMOID, bias=b)
    _check(z, 2, score=qk.SOFTMAX, bias=b)
    z = torch.tensor([[0.0, -500.0, -501.0, -502.0]], device="cuda")
    _check(z, 2, bias=torch.tensor([-5.0, 0.0, 0.0, 0.0], device="cuda"))


def _weights_f64(z, ids, sigmoid, renormalize, scale):
    """The weights as a function of the logits, in 64 bits, for autograd (dead: id -1)."""
    s = torch.sigmoid(z) if sigmoid else torch.softmax(z, 1)
    there = ids >= 0
    p = torch.where(there, s.gather(1, ids.clamp(min=0).long()), torch.zeros((), dtype=z.dtype))
    if renormalize:
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(there, p * scale, torch.zeros((), dtype=z.dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E,top_k", [(1, 1), (5, 2), (64, 8), (100, 7), (256, 8), (512, 32)])
def test_backward(dtype, score, renormalize, E, top_k):
    g = _gen(E + top_k)
    dt = DT[dtype]
    z = (torch.randn((33, E), generator=g, device="cuda") * 1.5).to(dt)
    z[:, ::5] = float("-inf") if E > 40 else z[:, ::5]
    if E > 40:
        z[4] = float("-inf")
    ids, _ = qk.qk_moe_route(z, top_k, score=score, renormalize=renormalize, scale=2.5)
    dw = torch.randn((33, top_k), generator=g, device="cuda")
    zz = z.double().cpu()
    zz = torch.where(zz == float("-inf"), torch.full_like(zz, -1e4), zz).requires_grad_(True)
    _weights_f64(zz, ids.cpu(), score == qk.SIGMOID, renormalize, 2.5).backward(dw.double().cpu())
    dw[ids < 0] = float("nan")                                   # not read
    got = qk.qk_moe_route_backward(z, ids, dw, score, renormalize, 2.5).double().cpu()
    want = zz.grad
    # terms of a token's sums are at most its largest |dweights| * scale each
    size = 2.5 * dw.nan_to_num(0.0).abs().amax(1, keepdim=True).double().cpu()
    tol = want.abs() * half_step(dt) * 1.01 + size * 64 * 2.0 ** -24
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())
    if E > 40:
        assert float(got[4].abs().max()) == 0.0 and float(got[:, ::5].abs().max()) == 0.0
    # the gradient of a renormalized weight's sum is zero: equal dweights
    if renormalize:
        flat = qk.qk_moe_route_backward(z, ids, torch.ones_like(dw), score, True, 2.5)
        assert float(flat.float().abs().max()) <= 2.5 * 64 * 2.0 ** -24


@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_against_differences(score, renormalize):
    g = _gen(21)
    z = torch.randn((6, 20), generator=g, device="cuda")
    ids, _ = qk.qk_moe_route(z, 20, score=score, renormalize=renormalize)        # all experts: no choice changes
    dw = torch.randn((6, 20), generator=g, device="cuda")
    got = qk.qk_moe_route_backward(z, ids, dw, score, renormalize).double()
    h = 2.0 ** -6

    def loss(zz):
        i, w = qk.qk_moe_route(zz, 20, score=score, renormalize=renormalize)
        d = torch.zeros_like(dw).scatter(1, ids.long(), dw)      # of each expert
        return (w.double() * d.gather(1, i.long()).double()).sum(1)

    for e in range(20):
        up, down = z.clone(), z.clone()
        up[:, e] += h
        down[:, e] -= h
        diff = (loss(up) - loss(down)) / ((up - down)[:, e].double())
        # third derivatives of these weights are under 1: h^2 / 6 of the sum of |dw|; the weights are rounded to fp32
        tol = dw.abs().sum(1).double() * (h * h / 6 + 2.0 ** -24 / h * 2)
        assert bool(((got[:, e] - diff).abs() <= tol).all()), e


def test_backward_over_the_logits_themselves_and_wrong_ids():
    g = _gen(22)
    z = torch.randn((50, 70), generator=g, device="cuda")
    ids, _ = qk.qk_moe_route(z, 4, renormalize=False)
    dw = torch.randn((50, 4), generator=g, device="cuda")
    want = qk.qk_moe_route_backward(z, ids, dw, renormalize=False)
    zz = z.clone()
    assert torch.equal(qk.qk_moe_route_backward(zz, ids, dw, renormalize=False, dlogits=zz), want) and torch.equal(zz, want)
    bad = ids.clone()
    bad[:, 2] = torch.tensor([70, -7, 2 ** 30, -2 ** 31, 1000] * 10, dtype=torch.int32, device="cuda")
    a, b = bad.clone(), dw.clone()
    a[:, 2], b[:, 2] = -1, 0
    assert torch.equal(qk.qk_moe_route_backward(z, bad, dw, renormalize=False), qk.qk_moe_route_backward(z, a, b, renormalize=False))


@pytest.mark.parametrize("T", [511, 512, 513, 1023, 1025, 4096, 4097, 8191, 8192, 8193, 16385, 32768, 32769, 49153, 100001])
def test_plan_lengths(T):
    """Slots of a workgroup's runs, whole and with one more or less."""
    g = _gen(T)
    ids = torch.randint(-1, 8, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    p = qk.qk_moe_plan(ids, 7)
    flat = torch.where(ids.view(-1) < 0, torch.full_like(ids.view(-1), 7), ids.view(-1)).long()
    n = torch.bincount(flat, minlength=8)
    assert torch.equal(p.slots.long(), torch.sort(flat, stable=True)[1])
    assert torch.equal(p.first.long(), torch.cumsum(n, 0) - n)


@pytest.mark.parametrize("T,top_k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (40, 4, 512), (700, 3, 17), (5000, 8, 64), (2049, 1, 3)])
def test_plan(T, top_k, E):
    g = _gen(T)
    ids = torch.randint(-1, E + 1, (T, top_k), generator=g, device="cuda", dtype=torch.int32)   # E, -1: no expert
    ids[T // 2] = 0                                              # the same expert more than once
    buf = torch.full((qk.qk_moe_plan_size(T, top_k, E) // 4 + 16,), 77, dtype=torch.int32, device="cuda")
    p = qk.qk_moe_plan(ids, E, buf)
    flat = ids.view(-1).long()
    flat = torch.where((flat < 0) | (flat >= E), torch.full_like(flat, E), flat)
    want = torch.sort(flat, stable=True)[1]
    assert torch.equal(p.slots.long(), want)
    assert torch.equal(p.first.long(), torch.cumsum(torch.bincount(flat, minlength=E + 1), 0) - torch.bincount(flat, minlength=E + 1))
    assert bool((buf[-16:] == 77).all())
    if T > 1000:
        ids.fill_(-1)
        p = qk.qk_moe_plan(ids, E)
        assert int(p.first.abs().max()) == 0 and torch.equal(p.slots.long(), torch.arange(T * top_k, device="cuda"))


def test_route_captured_replayed_and_on_another_stream():
    g = _gen(30)
    z = torch.randn((100, 64), generator=g, device="cuda")
    dw = torch.randn((100, 8), generator=g, device="cuda")
    ids, w = qk.qk_moe_route(z, 8)
    plan = qk.qk_moe_plan(ids, 64)
    dz = qk.qk_moe_route_backward(z, ids, dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk.qk_moe_route(z, 8, ids=ids, weights=w)
        qk.qk_moe_plan(ids, 64, plan.data)
        qk.qk_moe_route_backward(z, ids, dw, dlogits=dz)
    side = torch.cuda.Stream()
    for _ in range(3):
        z.copy_(torch.randn((100, 64), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            i2, w2 = qk.qk_moe_route(z, 8)
            p2 = qk.qk_moe_plan(i2, 64)
            d2 = qk.qk_moe_route_backward(z, i2, dw)
        side.synchronize()
        assert torch.equal(ids, i2) and torch.equal(w, w2) and torch.equal(dz, d2)
        assert torch.equal(plan.slots, p2.slots) and torch.equal(plan.first, p2.first)


def test_many_tokens():
    g = _gen(31)
    z = torch.randn((20000, 8), generator=g, device="cuda").bfloat16()
    ids, w = qk.qk_moe_route(z, 2)
    top, want = torch.sort(z.float(), dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), want[:, :2])
    ref = torch.softmax(top[:, :2].double(), 1)
    assert bool(((w.double() - ref).abs() <= ref * 2.0 ** -24 * 64).all())


def test_most_tokens():
    """2^26 tokens of one expert: more threads than a launch may have."""
    T = 1 << 26
    z = torch.zeros((T, 1), device="cuda")
    z[-1], z[1 << 24], z[(1 << 24) - 1] = float("-inf"), 2.0, -3.0
    ids, w = qk.qk_moe_route(z, 1, score=qk.SIGMOID, renormalize=False)
    want = torch.sigmoid(z.double())
    assert int(ids[-1]) == -1 and int(ids.sum()) == -1
    assert bool(((w.double() - want).abs() <= 4 * 2.0 ** -24).all())
    dz = qk.qk_moe_route_backward(z, ids, torch.ones_like(w), score=qk.SIGMOID, renormalize=False)
    assert bool(((dz.double() - want * (1 - want)).abs() <= 4 * 2.0 ** -24).all())


@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
@pytest.mark.parametrize("size", [32.0, 100.0, 1000.0, 1e30])
@pytest.mark.parametrize("E,groups,top_groups", [(4, 2, 1), (16, 4, 2), (128, 8, 3)])
def test_groups_of_biases_of_opposite_sign(score, size, E, groups, top_groups):
    """The two best ranks of a group cancel: their sum is small, what 32 bits take from each of them is not.  Sums of groups a
    few 2^-18 apart."""
    g = _gen(int(size) % 1009 + E)
    per = E // groups
    z = torch.randn((1500, 1, per), generator=g, device="cuda") * 0.5
    z = (z + torch.randn((1500, groups, per), generator=g, device="cuda") * 2.0 ** -18).reshape(1500, E)
    b = torch.full((E,), -2.0 * size, device="cuda")
    b[::per], b[1::per] = size, -size
    _check(z, 2, score=score, bias=b, groups=groups, top_groups=top_groups)
    if (E, size) == (4, 100.0) and score == qk.SIGMOID:           # sums 1.00000610 and 1.00000457
        ids, _ = qk.qk_moe_route(torch.tensor([[1.22e-5, 1.22e-5, 1.83e-5, 0.0]], device="cuda"), 1, b, score, groups=2)
        assert ids.tolist() == [[0]]


@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
@pytest.mark.parametrize("E,groups,top_groups,top_k", [(8, 2, 2, 8), (8, 4, 2, 4), (64, 8, 3, 20), (12, 4, 3, 9), (16, 16, 5, 5)])
def test_biases_of_the_largest_size(score, E, groups, top_groups, top_k):
    """A bias of the lowest finite value masks nothing: its experts, and groups of them whose sums pass fp32, come last.  The
    largest value ranks first."""
    g = _gen(E + groups)
    z = torch.randn((40, E), generator=g, device="cuda")
    z[5, E // 2:] = float("-inf")
    per, lowest = E // groups, torch.finfo(torch.float32).min
    one = torch.randn(E, generator=g, device="cuda") * 0.1
    one[per:] = lowest                                           # all groups but the first
    every = torch.full((E,), lowest, device="cuda")
    last = torch.randn(E, generator=g, device="cuda") * 0.1
    last[-per:] = -lowest
    mixed = one.clone()
    mixed[::per], mixed[-per:] = -lowest, float("-inf")
    for b in (one, every, -every, last, mixed):
        _check(z, top_k, score=score, bias=b, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("score", [qk.SOFTMAX, qk.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E,top_k", [(5, 5), (64, 8), (300, 8)])
@pytest.mark.parametrize("gap", [4.0, 12.0, 30.0])
def test_backward_where_one_expert_has_nearly_all(score, renormalize, E, top_k, gap):
    """The largest expert's gradient is what the others' small shares leave of its own: it keeps its digits."""
    g = _gen(E + int(gap))
    T = 40
    z = -gap + torch.randint(0, 4, (T, E), generator=g, device="cuda").float() * 0.25
    top = torch.randint(0, E, (T, 1), generator=g, device="cuda")
    z.scatter_(1, top, gap)
    ids, _ = qk.qk_moe_route(z, top_k, score=score, renormalize=renormalize)
    assert torch.equal(ids[:, :1].long(), top)
    # nothing cancels but the largest one's share against the whole: the others' d are on the other side of its own
    dw = -1.0 - torch.rand((T, top_k), generator=g, device="cuda")
    dw[:, 0] = 1.0
    zz = z.double().cpu().requires_grad_(True)
    _weights_f64(zz, ids.cpu(), score == qk.SIGMOID, renormalize, 1.0).backward(dw.double().cpu())
    got = qk.qk_moe_route_backward(z, ids, dw, score, renormalize).double().cpu()
    want = zz.grad
    if not renormalize and score == qk.SOFTMAX:
        # in 64 bits, too, 1 - s cancels: from the others' shares instead
        s = torch.softmax(z.double().cpu(), 1)
        d = torch.zeros_like(s).scatter(1, ids.cpu().long(), dw.double().cpu())
        t = top.cpu()
        others = s.scatter(1, t, 0.0)
        want = s * (d - (s * d).sum(1, keepdim=True))
        want.scatter_(1, t, s.gather(1, t) * (others.sum(1, keepdim=True) - (others * d).sum(1, keepdim=True)))
    elif not renormalize:
        i = ids.cpu().long()
        z8 = z.double().cpu().gather(1, i)
        want = torch.zeros_like(want).scatter(1, i, dw.double().cpu() * torch.sigmoid(z8) * torch.sigmoid(-z8))
    else:
        s = torch.sigmoid(z.double().cpu()) if score == qk.SIGMOID else torch.softmax(z.double().cpu(), 1)
        i = ids.cpu().long()
        c = s.gather(1, i)
        p, d = c / c.sum(1, keepdim=True), dw.double().cpu() - 1.0
        own = p * (d - (p * d).sum(1, keepdim=True)) * (torch.sigmoid(-z.double().cpu()).gather(1, i) if score == qk.SIGMOID else 1.0)
        want = torch.zeros_like(s).scatter(1, i, own)
    # half steps of fp32: an exponential 4, sums of shares 9 + 6, the quotient and the products 6, sums of the chosen 6, the
    # others' sum 9, the last difference 1
    tol = want.abs() * 41 * 2.0 ** -24
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / want.abs().clamp(min=1e-300)).max() * 2 ** 24)
