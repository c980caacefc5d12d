"""qk_gemv_int4 and qk_gemv_int4_grouped against the product in 64 bits.

Tolerance, derived before the first run.  y is rounded once to 16 bits: half a step, finfo.eps / 2 relative to
the value.  Before that a dot product of K terms is summed in fp32 in some order; each of its products carries
codes of up to 143 (bf16: 128 + q, the excess taken off after the sum) next to a value of |q - z| that may be 0,
so an absolute error of at most 2^-24 * depth * sum |x| |s| (143 + |z + 128|) arises, where depth bounds the
number of roundings an addend passes.  Every MFMA adds 32 products to an accumulator (taken as 32 roundings), a
chunk makes up to 4 of them, a wave takes ceil(K / 1024) chunks, and 8 waves are added: depth <=
128 + 2 ceil(K / 1024) + 8 + 4.
Up to M = 4 the sums over a chunk are exact integers instead, of activations rounded to 2^-22 of their chunk's
largest: 4 * 2^-24 max |x| for each |s| |q - z|.  Of values that are all of one size (|x| on average a fifth of the
largest, as in random normal rows) that is 20 of the roundings above, and the 128 of the accumulators do not occur.
Rows that are not of one size have a test of their own, which counts the largest value.
"""

import pytest
import torch

import bit_blockwise_weight_amd as qk
from tests.gpu_common import require_gpu, say
from tests.gpu_int4 import int4_f64, make_int4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _case(seed, M, N, K, group, zeros, dtype, scale_dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, s, z = make_int4(gen, N, K, group, zeros, scale_dtype)
    x = torch.randn((M, K), generator=gen, device="cuda").to(dtype)
    w64 = int4_f64(q, s, z, group)
    gi = torch.arange(K, device="cuda") // group if group else torch.zeros(K, dtype=torch.long, device="cuda")
    zz = 8.0 if z is None else z.double()[:, gi]
    absw = s.double().abs()[:, gi] * (143.0 + 128.0 + zz)
    ref = x.double() @ w64.t()
    depth = 128 + 2 * -(-K // 1024) + 12
    tol = torch.finfo(dtype).eps / 2 * ref.abs() + 2.0 ** -24 * depth * (x.double().abs() @ absw.t()) \
        + torch.finfo(dtype).smallest_normal
    return qk.Int4Weight(q, s, z, group), x, ref, tol


def _check(y, ref, tol, what):
    err = (y.double() - ref).abs()
    worst = float((err / tol).max())
    assert worst <= 1.0, f"{what}: error {worst} of the tolerance"


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 17, 31), (2, 33, 257), (3, 64, 1024), (4, 100, 1025), (5, 48, 2048), (7, 31, 999),
          (8, 1024, 1024), (9, 160, 4096), (16, 130, 3000), (16, 3000, 4099), (1, 4096, 4096), (1, 500, 11008)]


@pytest.mark.parametrize("group", [32, 64, 128, 256, 0])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("dtype,scale_dtype", [(torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16),
                                               (torch.bfloat16, torch.bfloat16)])
def test_gemv_against_64_bits(group, zeros, dtype, scale_dtype):
    for i, (M, N, K) in enumerate(SHAPES):
        say(f"case: gemv_int4 M={M} N={N} K={K} group={group} zeros={zeros} {dtype} {scale_dtype}")
        w, x, ref, tol = _case(100 + i, M, N, K, group, zeros, dtype, scale_dtype)
        _check(w.gemv(x), ref, tol, f"M={M} N={N} K={K} group={group}")


@pytest.mark.parametrize("M", range(1, 17))
def test_every_row_count(M):
    say(f"case: gemv_int4 every row count M={M}")
    w, x, ref, tol = _case(M, M, 80, 1500, 64, True, torch.bfloat16, torch.float16)
    _check(w.gemv(x), ref, tol, f"M={M}")


def test_group_of_weights_equals_single_calls_bitwise():
    for dtype in (torch.bfloat16, torch.float16):
        for M in (1, 4, 16):
            say(f"case: gemv_int4 grouped M={M} {dtype}")
            sizes = [(16, 128, 128), (48, 1000, 32), (1000, 1024, 64), (33, 4099, 0), (7, 64, 256), (300, 2048, 32)] * 4
            ws, xs = [], []
            for i, (N, K, group) in enumerate(sizes):
                w, x, _, _ = _case(i, M, N, K, group, i % 2 == 0, dtype, torch.float16)
                ws.append(w)
                xs.append(x)
            ys = qk.qk_gemv_int4_grouped([(x, w.state) for x, w in zip(xs, ws)])
            for i, (w, x, y) in enumerate(zip(ws, xs, ys)):
                assert torch.equal(y, w.gemv(x)), f"task {i}"


def test_unaligned_rows_and_outputs_inside_larger_buffers():
    """x and y at odd 2-byte offsets of larger buffers: the same bits as aligned ones, and no byte beside y changes."""
    for M, N, K in ((3, 50, 1024), (16, 33, 77)):
        say(f"case: gemv_int4 unaligned M={M} N={N} K={K}")
        w, x, ref, tol = _case(7, M, N, K, 64, True, torch.float16, torch.float16)
        want = w.gemv(x)
        for off in (1, 3, 5):
            xb = torch.full((M * K + 64,), float("nan"), dtype=x.dtype, device="cuda")
            xb[off:off + M * K] = x.view(-1)
            yb = torch.full((M * N + 64,), 7.0, dtype=x.dtype, device="cuda")
            y = yb[off:off + M * N].view(M, N)
            w2 = qk.qk_gemv_int4(xb[off:off + M * K].view(M, K), w.state, y)
            assert torch.equal(w2, want)
            assert bool((yb[:off] == 7).all()) and bool((yb[off + M * N:] == 7).all())


def test_padding_of_the_codes_is_ignored():
    say("case: gemv_int4 code padding")
    w, x, ref, tol = _case(8, 2, 40, 999, 128, True, torch.bfloat16, torch.float16)
    want = w.gemv(x)
    wide = torch.full((40, w.codes.shape[1] + 48), 0xA5, dtype=torch.uint8, device="cuda")
    wide[:, :500] = w.codes[:, :500]
    wide[:, 499] = (w.codes[:, 499] & 0xF0) | 0x07           # K is odd: the last low nibble holds no code
    st = qk.qk_int4_state_init(40, 999, 128, wide, w.scales, w.zeros)
    assert torch.equal(qk.qk_gemv_int4(x, st), want)


def test_infinite_activation_reaches_its_outputs_only():
    say("case: gemv_int4 rows do not mix")
    w, x, ref, tol = _case(9, 4, 64, 512, 32, False, torch.bfloat16, torch.float16)
    want = w.gemv(x)
    x2 = x.clone()
    x2[2, 100] = float("inf")
    y = w.gemv(x2)
    for m in (0, 1, 3):
        assert torch.equal(y[m], want[m])
    assert not bool(torch.isfinite(y[2]).any())


def test_graph_replays_and_streams():
    say("case: gemv_int4 graph and side stream")
    w, x, ref, tol = _case(10, 3, 256, 1024, 128, True, torch.bfloat16, torch.float16)
    want = w.gemv(x)
    y = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = w.gemv(x)
    side.synchronize()
    assert torch.equal(y2, want)
    g = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(g):
        w.gemv(xs, y)
    for i in range(3):
        xs.copy_(x * (i + 1))
        eager = w.gemv(xs)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 16])
def test_memory_behind_the_scales_is_not_used(group, M):
    """Scales and zero points that end inside a dword, and at a row that ends inside a chunk, with NaN behind them."""
    for N, K in ((1, 1), (1, 32), (3, 33), (5, 160), (7, 300)):
        say(f"case: gemv_int4 NaN behind the scales M={M} N={N} K={K} group={group}")
        w, x, ref, tol = _case(11, M, N, K, group, True, torch.bfloat16, torch.float16)
        n = w.scales.numel()
        sb = torch.full((n + 64,), float("nan"), dtype=torch.float16, device="cuda")
        zb = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
        sb[:n] = w.scales.reshape(-1)
        zb[:n] = w.zeros.reshape(-1)
        st = qk.qk_int4_state_init(N, K, group, w.codes, sb[:n].view(N, -1), zb[:n].view(N, -1))
        _check(qk.qk_gemv_int4(x, st), ref, tol, f"N={N} K={K} group={group}")


@pytest.mark.parametrize("M", [1, 8])
def test_a_row_of_infinite_scales_stays_in_its_outputs(M):
    """The scales behind a row's last group are the next row's."""
    say(f"case: gemv_int4 infinite scales in one row M={M}")
    for group, K in ((32, 160), (64, 192), (128, 384)):
        w, x, ref, tol = _case(12, M, 40, K, group, True, torch.bfloat16, torch.float16)
        s = w.scales.clone()
        s[17] = float("inf")
        st = qk.qk_int4_state_init(40, K, group, w.codes, s, w.zeros)
        y = qk.qk_gemv_int4(x, st)
        keep = torch.arange(40, device="cuda") != 17
        assert torch.equal(y[:, keep], w.gemv(x)[:, keep])
        assert not bool(torch.isfinite(y[:, 17]).any())


@pytest.mark.parametrize("M", [1, 16])
def test_rows_of_codes_far_apart(M):
    """300 rows, 16 MiB from one to the next: offsets that pass 32 bits, for one group per row and for several."""
    buf = torch.empty((300, 1 << 24), dtype=torch.uint8, device="cuda")
    for K, group in ((64, 0), (1000, 32)):
        say(f"case: gemv_int4 rows 16 MiB apart M={M} K={K}")
        w, x, ref, tol = _case(13, M, 300, K, group, True, torch.bfloat16, torch.float16)
        buf[:, :w.codes.shape[1]] = w.codes
        st = qk.qk_int4_state_init(300, K, group, buf, w.scales, w.zeros)
        _check(qk.qk_gemv_int4(x, st), ref, tol, f"M={M} K={K}")


def test_a_matrix_of_more_than_four_gib():
    """The last rows of 9 GB of codes (2^21 rows of 8192 columns), against the same rows alone."""
    N, K, tail = 1 << 21, 8192, 1000
    for M in (1, 9):
        say(f"case: gemv_int4 2^21 rows M={M}")
        gen = torch.Generator(device="cuda").manual_seed(14)
        q, s, z = make_int4(gen, tail, K, 128, True, torch.float16)
        w = qk.Int4Weight(q, s, z, 128)
        codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((N, K // 128), dtype=torch.float16, device="cuda")
        zeros = torch.zeros((N, K // 128), dtype=torch.uint8, device="cuda")
        codes[-tail:], scales[-tail:], zeros[-tail:] = w.codes, s, z
        x = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
        y = qk.qk_gemv_int4(x, qk.qk_int4_state_init(N, K, 128, codes, scales, zeros))
        assert bool((y[:, :-tail] == 0).all())
        ref = x.double() @ int4_f64(q, s, z, 128).t()
        assert float((y[:, -tail:].double() - ref).norm() / ref.norm()) < 2.0 ** -8
        del codes, scales, zeros, y
        torch.cuda.empty_cache()


@pytest.mark.parametrize("group", [32, 64, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_of_very_different_size(group, dtype):
    """Rows with one value far above its neighbours, very small rows, zeros.  Up to four rows are held in fixed point,
    to 2^-22 of the largest value in each run of 128 inputs; 2^-121 below 2^-100."""
    M, N, K = 4, 96, 1000
    w, x, _, _ = _case(15, M, N, K, group, True, dtype, torch.bfloat16)
    x[0, 77] = 1000.0
    x[1, ::130] *= 500.0
    x[2] *= 2.0 ** -12 if dtype is torch.float16 else 2.0 ** -60
    x[3] = 0
    x[3, 999] = 1.0
    codes = torch.stack((w.codes >> 4, w.codes & 15), 2).view(N, -1)[:, :K]
    w64 = int4_f64(codes, w.scales, w.zeros, group)
    gi = torch.arange(K, device="cuda") // group
    absw = w.scales.double().abs()[:, gi] * (143.0 + 128.0 + w.zeros.double()[:, gi])
    ref = x.double() @ w64.t()
    big = torch.nn.functional.pad(x.double().abs(), (0, 24)).view(M, 8, 128).amax(2).repeat_interleave(128, 1)[:, :K]
    for m in range(1, M + 1):
        say(f"case: gemv_int4 values of different size M={m} group={group} {dtype}")
        tol = torch.finfo(dtype).eps / 2 * ref.abs() + 2.0 ** -24 * 150 * (x.double().abs() @ absw.t()) \
            + 2.0 ** -22 * (big @ w64.abs().t()) + torch.finfo(dtype).smallest_normal
        _check(w.gemv(x[:m].contiguous()), ref[:m], tol[:m], f"M={m}")
    if dtype is torch.bfloat16:
        say("case: gemv_int4 the largest and the smallest numbers")
        x2 = torch.zeros((2, K), dtype=dtype, device="cuda")
        x2[0] = 2.0 ** -120
        x2[1, 5] = torch.finfo(dtype).max
        y = w.gemv(x2)
        assert bool((y[0].double().abs() < 2.0 ** -80).all())
        want = (x2[1, 5].double() * w64[:, 5]).to(dtype)
        same = y[1] == want                                  # infinities of one sign among them
        assert bool((same | ((y[1].double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs())).all())


def test_refusals_on_the_device():
    say("case: gemv_int4 refusals")
    w, x, _, _ = _case(16, 4, 32, 64, 32, True, torch.bfloat16, torch.float16)
    with pytest.raises(ValueError, match="contiguous"):
        w.gemv(x.t().contiguous().t())
    with pytest.raises(ValueError):
        w.gemv(x, torch.empty((4, 31), dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError):
        w.gemv(x, torch.empty((4, 32), dtype=torch.float32, device="cuda"))
    with pytest.raises(RuntimeError, match="1..16"):
        w.gemv(torch.zeros((17, 64), dtype=x.dtype, device="cuda"))
    with pytest.raises(RuntimeError, match="overlaps"):
        qk.qk_gemv_int4_grouped([(x, w.state), (x, w.state)], [y := torch.empty((4, 32), dtype=x.dtype, device="cuda"), y])
