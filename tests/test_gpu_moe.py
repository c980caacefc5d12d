"""qk_moe_int4 and qk_moe_nf4 against the layer in 64 bits.

Tolerance, derived before the first run.  y is rounded once: finfo.eps / 2 relative to the value.  h is kept as a
bf16 pair: 2^-8 of the first rounding times 2^-8 of the second, 2^-16 relative.  (int4 experts with few tokens
hold x and h to 2^-22 of the largest of 128 values instead, which for values of one size is less than that.)  The two products are fp32 sums:
their errors are 2^-24 * depth of the sums of their absolute terms, scaled for int4 by the excess of the stored codes
(up to 271 + |z| instead of |q - z|; see the GEMV's tests), which here multiplies the absolute weights.  depth of a
product over K: 128 + 2 ceil(K / 128) + 32.
"""

import pytest
import torch

import bit_blockwise_weight_amd as qk
from tests.gpu_common import require_gpu, say
from tests.gpu_int4 import int4_f64, make_int4, moe_f64, route_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Int4Experts:
    def __init__(self, gen, E, rows, cols, group, zeros, scale_dtype):
        self.group, self.rows = group, rows
        self.q, self.s, self.z = make_int4(gen, E * rows, cols, group, zeros, scale_dtype)
        self.w = qk.Int4Weight(self.q, self.s, self.z, group)
        self.state = self.w.state
        self.excess = 271.0 + 255.0

    def f64(self, e):
        r = slice(e * self.rows, (e + 1) * self.rows)
        return int4_f64(self.q[r], self.s[r], None if self.z is None else self.z[r], self.group)

    def step(self, e):                       # |s| of every element
        r = slice(e * self.rows, (e + 1) * self.rows)
        one = torch.ones_like(self.q[r])
        return int4_f64(one, self.s[r], torch.zeros_like(self.s[r], dtype=torch.uint8), self.group).abs()


class Nf4Experts:
    def __init__(self, gen, E, rows, cols, block, kind, nested):
        self.rows, self.cols, self.block = rows, cols, block
        w = (torch.randn((E * rows, cols), generator=gen, device="cuda") * 0.02).to(torch.bfloat16)
        self.qw = qk.quantize(w, block, kind, double_quant=nested)
        self.state = self.qw.state
        lv = torch.tensor(list(self.state.levels), device="cuda").to(torch.bfloat16).double()
        b = self.qw.codes
        codes = torch.stack((b >> 4, b & 15), 1).view(-1).long()
        n = torch.arange(E * rows * cols, device="cuda") // block
        if nested:
            a = self.qw.q8.double() * self.qw.scale.double().repeat_interleave(256)[:self.qw.q8.numel()] \
                + self.qw.mean.double()
        else:
            a = self.qw.absmax.double()
        self.all = (lv[codes] * a[n]).view(E * rows, cols)

    def f64(self, e):
        return self.all[e * self.rows:(e + 1) * self.rows]


def _tolerance(x, routes, up, down, I, H, dtype, ref, bound):
    depth = max(128 + 2 * -(-k // 128) + 32 for k in (I, H))
    if isinstance(up, Int4Experts):
        # the same bound with every weight replaced by |s| times what its stored code may weigh
        _, bound = moe_f64_abs(x, routes, up, down, I)
    return torch.finfo(dtype).eps / 2 * ref.abs() + (2.0 ** -24 * depth + 2.0 ** -16) * bound \
        + torch.finfo(dtype).smallest_normal


def moe_f64_abs(x, routes, up, down, I):
    """The bound of moe_f64 for int4 experts: errors of g, u and y relative to sums over |s| * excess."""
    xd = x.double()
    bound = torch.zeros(xd.shape, dtype=torch.float64, device=x.device)
    for t, chosen in enumerate(routes):
        for e, w in chosen:
            wu, wd = up.f64(e), down.f64(e)
            gu = wu @ xd[t]
            g, u = gu[:I], gu[I:]
            sg = g / (1 + torch.exp(-g))
            agu = up.excess * (up.step(e) @ xd[t].abs())
            bound[t] += w * (wd.abs() @ (1.1 * agu[:I] * u.abs() + sg.abs() * agu[I:])
                             + down.excess * (down.step(e) @ (sg * u).abs()))
    return None, bound


def _check(y, ref, tol, what):
    # a value that rounds past the type's largest is an infinity of its sign
    top = torch.finfo(y.dtype).max
    over = (ref.abs() + tol > top) & (y.double() == ref.sign() * float("inf"))
    err = torch.where(over, torch.zeros_like(ref), (y.double() - ref).abs())
    worst = float((err / tol).max())
    assert worst <= 1.0, f"{what}: error {worst} of the tolerance"
    # The bound above adds worst cases.  In the norm, the last rounding is at most half a step of every value, and the
    # rounding errors of the sums are independent: 2^-24 times the codes' excess (526 / 8) times sqrt(depth) or so, 2^-13.
    rel = float(err.norm() / torch.where(over, torch.zeros_like(ref), ref).norm().clamp(min=1e-300))
    assert rel <= torch.finfo(y.dtype).eps / 2 + 2.0 ** -13, f"{what}: relative error {rel} in the norm"


def _run(seed, T, E, top_k, H, I, make_up, make_down, dtype, renorm, logits_dtype=torch.float32, logits=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    up, down = make_up(gen), make_down(gen)
    x = torch.randn((T, H), generator=gen, device="cuda").to(dtype)
    if logits is None:
        logits = (torch.randn((T, E), generator=gen, device="cuda") * 1.5).to(logits_dtype)
    routes = route_f64(logits, top_k, renorm)
    ref, bound = moe_f64(x, routes, lambda e: (up.f64(e)[:I], up.f64(e)[I:]), down.f64)
    tol = _tolerance(x, routes, up, down, I, H, dtype, ref, bound)
    call = qk.qk_moe_int4 if isinstance(up, Int4Experts) else qk.qk_moe_nf4
    args = (x, logits, top_k, up.state, down.state, renorm)
    _check(call(*args), ref, tol, f"T={T} E={E} top_k={top_k} H={H} I={I}")
    return call, args, up, down


INT4 = [(1, 1, 1, 16, 16), (1, 8, 2, 256, 512), (2, 5, 3, 100, 77), (3, 64, 8, 512, 256), (7, 11, 3, 1001, 777),
        (8, 4, 4, 128, 130), (9, 16, 2, 96, 1), (16, 64, 8, 256, 384), (16, 256, 16, 64, 64), (1, 2, 1, 4100, 1100)]


@pytest.mark.parametrize("group,zeros,dtype,scale_dtype", [
    (32, True, torch.bfloat16, torch.float16), (64, False, torch.float16, torch.float16),
    (128, True, torch.float16, torch.bfloat16), (256, True, torch.bfloat16, torch.bfloat16),
    (0, False, torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("renorm", [True, False])
def test_int4_against_64_bits(group, zeros, dtype, scale_dtype, renorm):
    for i, (T, E, k, H, I) in enumerate(INT4):
        say(f"case: moe_int4 T={T} E={E} top_k={k} H={H} I={I} group={group} zeros={zeros} {dtype} renorm={renorm}")
        _run(i, T, E, k, H, I, lambda g: Int4Experts(g, E, 2 * I, H, group, zeros, scale_dtype),
             lambda g: Int4Experts(g, E, H, I, group, zeros, scale_dtype), dtype, renorm,
             (torch.float32, torch.bfloat16, torch.float16)[i % 3])


NF4 = [(1, 8, 2, 256, 512), (2, 3, 3, 64, 64), (4, 16, 4, 192, 320), (9, 8, 2, 448, 128), (16, 32, 8, 128, 192)]


@pytest.mark.parametrize("block,kind,nested", [(64, qk.NF4, True), (128, qk.NF4, False), (256, qk.FP4, True),
                                               (64, qk.FP4, False), (128, qk.NF4, True)])
def test_nf4_against_64_bits(block, kind, nested):
    for i, (T, E, k, H, I) in enumerate(NF4):
        say(f"case: moe_nf4 T={T} E={E} top_k={k} H={H} I={I} block={block} kind={kind} nested={nested}")
        _run(50 + i, T, E, k, H, I, lambda g: Nf4Experts(g, E, 2 * I, H, block, kind, nested),
             lambda g: Nf4Experts(g, E, H, I, block, kind, nested), torch.bfloat16, i % 2 == 0)


def _int4_small(g, E=6, H=160, I=96):
    return Int4Experts(g, E, 2 * I, H, 32, True, torch.float16), Int4Experts(g, E, H, I, 32, True, torch.float16)


def test_ties_masks_and_empty_tokens():
    inf = float("-inf")
    nan = float("nan")
    say("case: moe_int4 ties, masks, empty tokens")
    lg = torch.tensor([[1.0, 1.0, 1.0, 1.0, 1.0, 1.0],           # all equal: experts 0, 1, 2
                       [inf, inf, inf, inf, inf, inf],           # nothing to choose
                       [inf, 2.0, inf, inf, inf, inf],           # one expert for three places
                       [inf, inf, 0.5, 0.5, inf, -300.0],        # a weight that underflows
                       [3e38, -3e38, 0.0, 3e38, -3e38, 1.0],     # far apart
                       [torch.finfo(torch.float32).min] * 6])    # the type's lowest value is a value
    lg = lg.cuda()
    for renorm in (True, False):
        gen = torch.Generator(device="cuda").manual_seed(5)
        up, down = _int4_small(gen)
        x = torch.randn((6, 160), generator=gen, device="cuda").to(torch.bfloat16)
        routes = route_f64(lg, 3, renorm)
        ref, _ = moe_f64(x, routes, lambda e: (up.f64(e)[:96], up.f64(e)[96:]), down.f64)
        y = qk.qk_moe_int4(x, lg, 3, up.state, down.state, renorm)
        tol = _tolerance(x, routes, up, down, 96, 160, x.dtype, ref, None)
        _check(y, ref, tol, f"renorm={renorm}")
        assert bool((y[1] == 0).all())
        # a NaN logit masks as -inf does, and an empty token's own values do not matter
        l2, x2 = lg.clone(), x.clone()
        l2[2, 3] = nan
        x2[1] = nan
        assert torch.equal(qk.qk_moe_int4(x2, l2, 3, up.state, down.state, renorm), y)


def test_all_tokens_empty_and_poisoned_workspace():
    say("case: moe_int4 nothing chosen anywhere; stale workspaces")
    gen = torch.Generator(device="cuda").manual_seed(6)
    up, down = _int4_small(gen)
    x = torch.randn((16, 160), generator=gen, device="cuda").to(torch.bfloat16)
    lg = torch.randn((16, 6), generator=gen, device="cuda")
    want = qk.qk_moe_int4(x, lg, 2, up.state, down.state)
    n = qk.qk_moe_workspace_size(16, 2, 160, 96)
    for fill in (0xFF, 0x7F, 0x00):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(qk.qk_moe_int4(x, lg, 2, up.state, down.state, workspace=ws[:n]), want)
        assert bool((ws[n:] == fill).all())
        y0 = qk.qk_moe_int4(x, torch.full_like(lg, float("-inf")), 2, up.state, down.state, workspace=ws[:n])
        assert bool((y0 == 0).all())


def test_tokens_do_not_depend_on_each_other():
    say("case: moe tokens alone and together")
    gen = torch.Generator(device="cuda").manual_seed(7)
    up, down = _int4_small(gen)
    x = torch.randn((8, 160), generator=gen, device="cuda").to(torch.bfloat16)
    lg = torch.randn((8, 6), generator=gen, device="cuda")
    y = qk.qk_moe_int4(x, lg, 2, up.state, down.state)
    for t in range(8):
        x2, l2 = x.clone(), torch.full_like(lg, float("-inf"))
        l2[t] = lg[t]
        x2[:t] = float("inf")
        x2[t + 1:] = float("nan")
        assert torch.equal(qk.qk_moe_int4(x2, l2, 2, up.state, down.state)[t], y[t])


def test_in_place_streams_and_graphs():
    say("case: moe in place, side stream, graph")
    gen = torch.Generator(device="cuda").manual_seed(8)
    up = Nf4Experts(gen, 8, 2 * 128, 256, 64, qk.NF4, True)
    down = Nf4Experts(gen, 8, 256, 128, 64, qk.NF4, True)
    x = torch.randn((5, 256), generator=gen, device="cuda").to(torch.bfloat16)
    lg = torch.randn((5, 8), generator=gen, device="cuda")
    want = qk.qk_moe_nf4(x, lg, 2, up.state, down.state)
    xi = x.clone()
    assert qk.qk_moe_nf4(xi, lg, 2, up.state, down.state, y=xi) is xi and torch.equal(xi, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = qk.qk_moe_nf4(x, lg, 2, up.state, down.state)
    side.synchronize()
    assert torch.equal(y2, want)
    xs, ls, y = x.clone(), lg.clone(), torch.empty_like(want)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    ya = torch.empty_like(want)
    with torch.cuda.graph(g1):
        qk.qk_moe_nf4(xs, ls, 2, up.state, down.state, y=y)
    with torch.cuda.graph(g2):
        qk.qk_moe_nf4(xs, ls, 2, up.state, down.state, y=ya)
    for i in range(3):
        xs.copy_(x * (1 + i))
        ls.copy_(lg.roll(i, 1))
        eager = qk.qk_moe_nf4(xs, ls, 2, up.state, down.state)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(ya, eager)


def test_decode_layer_of_both_operators():
    """A decode step's products as they follow each other: int4 projections in one grouped call, their output
    through an int4 expert layer and through an NF4 one; each step against 64 bits on the step's own input."""
    say("case: grouped projections, then both expert layers")
    gen = torch.Generator(device="cuda").manual_seed(9)
    H, E, I, T = 512, 8, 256, 4
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    proj = [Int4Experts(gen, 1, n, H, 128, True, torch.float16) for n in (H, H // 4, E)]
    hidden, _, lg = qk.qk_gemv_int4_grouped([(x, p.state) for p in proj])
    for y, p in zip((hidden, lg), (proj[0], proj[2])):
        ref = x.double() @ p.f64(0).t()
        assert float((y.double() - ref).norm() / ref.norm()) < 2.0 ** -8
    routes = route_f64(lg, 2, True)
    up, down = Int4Experts(gen, E, 2 * I, H, 128, True, torch.float16), Int4Experts(gen, E, H, I, 128, True, torch.float16)
    y1 = qk.qk_moe_int4(hidden, lg, 2, up.state, down.state)
    ref, bound = moe_f64(hidden, routes, lambda e: (up.f64(e)[:I], up.f64(e)[I:]), down.f64)
    _check(y1, ref, _tolerance(hidden, routes, up, down, I, H, torch.bfloat16, ref, bound), "int4 layer")
    un, dn = Nf4Experts(gen, E, 2 * I, H, 64, qk.NF4, True), Nf4Experts(gen, E, H, I, 64, qk.NF4, True)
    y2 = qk.qk_moe_nf4(hidden, lg, 2, un.state, dn.state)
    ref, bound = moe_f64(hidden, routes, lambda e: (un.f64(e)[:I], un.f64(e)[I:]), dn.f64)
    _check(y2, ref, _tolerance(hidden, routes, un, dn, I, H, torch.bfloat16, ref, bound), "NF4 layer")


def test_a_row_of_infinite_block_scales_stays_in_its_outputs():
    """K = 64 * odd: the chunk that holds a row's end reaches into the next row's blocks."""
    say("case: moe_nf4 infinite block scales: of an expert that nobody chooses, of one row of a chosen one")
    gen = torch.Generator(device="cuda").manual_seed(10)
    E, H, I, block = 3, 192, 64, 64
    up, down = (Nf4Experts(gen, E, 2 * I, H, block, qk.NF4, False), Nf4Experts(gen, E, H, I, block, qk.NF4, False))
    x = torch.randn((2, H), generator=gen, device="cuda").to(torch.bfloat16)
    lg = torch.tensor([[1.0, float("-inf"), 0.0]] * 2, device="cuda")         # expert 1 lies between the chosen ones
    want = qk.qk_moe_nf4(x, lg, 2, up.state, down.state)
    assert bool(torch.isfinite(want).all())
    for e, n in ((up, 2 * I * H), (down, H * I)):
        e.qw.absmax[n // block:2 * n // block] = float("inf")                 # the blocks of expert 1 alone
    assert torch.equal(qk.qk_moe_nf4(x, lg, 2, up.state, down.state), want)
    down.qw.absmax[2 * H + 17] = float("inf")                                 # row 17 of expert 2: output 17
    y = qk.qk_moe_nf4(x, lg, 2, up.state, down.state)
    keep = torch.arange(H, device="cuda") != 17
    assert torch.equal(y[:, keep], want[:, keep]) and not bool(torch.isfinite(y[:, 17]).any())


@pytest.mark.parametrize("E", [3, 4, 9])
def test_every_token_at_the_same_expert(E):
    """16 tokens of one expert: as many as a pass takes, or several passes; few and many experts beside it."""
    T, H, I = 16, 200, 136
    lg = torch.zeros((T, E), device="cuda")
    lg[:, 1] = 3.0
    lg[5:, 2] = 1.0
    for k in (1, 2):
        say(f"case: moe 16 tokens of one expert E={E} top_k={k}")
        for group in (32, 128):
            _run(60, T, E, k, H, I, lambda g: Int4Experts(g, E, 2 * I, H, group, True, torch.float16),
                 lambda g: Int4Experts(g, E, H, I, group, True, torch.float16), torch.bfloat16, True, logits=lg)
        _run(61, T, E, k, 192, 128, lambda g: Nf4Experts(g, E, 2 * 128, 192, 64, qk.NF4, True),
             lambda g: Nf4Experts(g, E, 192, 128, 64, qk.NF4, True), torch.bfloat16, True, logits=lg)


@pytest.mark.parametrize("H,I", [(12032, 64), (64, 12032)])
@pytest.mark.parametrize("T,E", [(1, 2), (4, 3), (7, 2), (16, 2), (16, 9)])
def test_long_rows(H, I, T, E):
    """Rows whose activations do not stay on the chip, for each number of tokens that a pass takes."""
    say(f"case: moe long rows H={H} I={I} T={T} E={E}")
    for dtype in (torch.bfloat16, torch.float16):
        _run(62, T, E, 2, H, I, lambda g: Int4Experts(g, E, 2 * I, H, 32, True, torch.bfloat16),
             lambda g: Int4Experts(g, E, H, I, 64, True, torch.bfloat16), dtype, True)
    _run(63, T, E, 2, H, I, lambda g: Nf4Experts(g, E, 2 * I, H, 64, qk.NF4, True),
         lambda g: Nf4Experts(g, E, H, I, 128, qk.NF4, False), torch.bfloat16, True)


def test_two_calls_at_once():
    say("case: moe two streams, a workspace each")
    gen = torch.Generator(device="cuda").manual_seed(11)
    up, down = _int4_small(gen)
    xs = [torch.randn((16, 160), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    lg = torch.randn((16, 6), generator=gen, device="cuda")
    want = [qk.qk_moe_int4(x, lg, 3, up.state, down.state) for x in xs]
    n = qk.qk_moe_workspace_size(16, 3, 160, 96)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                qk.qk_moe_int4(xs[i], lg, 3, up.state, down.state, y=ys[i], workspace=ws[i])
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(y, w)


def test_experts_behind_four_gib():
    """A stack of 8.6 GB of codes whose last expert alone is not zero."""
    E, H, I = 64, 4096, 16384
    say(f"case: moe_int4 E={E} H={H} I={I}")
    gen = torch.Generator(device="cuda").manual_seed(12)

    def last(rows, cols):
        q, s, z = make_int4(gen, rows, cols, 128, True, torch.float16)
        w = qk.Int4Weight(q, s, z, 128)
        codes = torch.zeros((E * rows, cols // 2), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((E * rows, cols // 128), dtype=torch.float16, device="cuda")
        zeros = torch.zeros((E * rows, cols // 128), dtype=torch.uint8, device="cuda")
        codes[-rows:], scales[-rows:], zeros[-rows:] = w.codes, s, z
        return w, (codes, scales, zeros), qk.qk_int4_state_init(E * rows, cols, 128, codes, scales, zeros)

    u1, u_all, up = last(2 * I, H)
    d1, d_all, down = last(H, I)
    x = torch.randn((3, H), generator=gen, device="cuda").to(torch.bfloat16)
    lg = torch.full((3, E), float("-inf"), device="cuda")
    lg[:, E - 1] = 0.5
    lg[1, 7] = 0.5                                           # a zero expert for half of token 1
    y = qk.qk_moe_int4(x, lg, 2, up, down)
    alone = qk.qk_moe_int4(x, torch.zeros((3, 1), device="cuda"), 1, u1.state, d1.state)
    assert torch.equal(y[0], alone[0]) and torch.equal(y[2], alone[2])
    assert float((2 * y[1].double() - alone[1].double()).norm() / alone[1].double().norm()) < 2.0 ** -7
    assert bool((alone != 0).any())


def test_first_call_inside_a_capture():
    """Sizes that nothing ran before, captured without an eager call: the library sets up its kernels on the way."""
    say("case: moe and gemv captured first")
    gen = torch.Generator(device="cuda").manual_seed(13)
    H, I, E, T = 7040, 320, 5, 15
    up, down = (Int4Experts(gen, E, 2 * I, H, 64, False, torch.bfloat16), Int4Experts(gen, E, H, I, 64, False, torch.bfloat16))
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch.float16)
    lg = torch.randn((T, E), generator=gen, device="cuda")
    y, z = torch.empty_like(x), torch.empty((T, 2 * E * I), dtype=x.dtype, device="cuda")
    ws = torch.empty(qk.qk_moe_workspace_size(T, 3, H, I), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qk.qk_moe_int4(x, lg, 3, up.state, down.state, y=y, workspace=ws)
        qk.qk_gemv_int4(x, up.state, z)
    for _ in range(3):
        y.zero_()
        z.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, qk.qk_moe_int4(x, lg, 3, up.state, down.state)) and torch.equal(z, up.w.gemv(x))
