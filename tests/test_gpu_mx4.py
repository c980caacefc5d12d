"""The microscaled 4-bit operators on the GPU against 64-bit references: quantization and its inverse, the product of two
microscaled matrices, the product of 16-bit rows with one."""

import pytest
import torch

import bit_blockwise_weight_amd as qk
from gpu_mx4 import check, half_step, make_mx4, product_bound, quantize_f64, strides, values

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes_of(packed, cols):
    k = torch.arange(cols, device=packed.device)
    return ((packed[:, k // 2].int() >> (4 * (k % 2))) & 15).to(torch.uint8)


def _quantized(x, want_scales, want_codes):
    rows, cols = x.shape
    codes, scales = qk.qk_mx4_quantize(x)
    assert codes.shape == (rows, strides(cols)[0]) and scales.shape == (rows, strides(cols)[1])
    assert torch.equal(scales[:, :want_scales.shape[1]], want_scales)
    got = _codes_of(codes, cols)
    off = torch.nonzero(got != want_codes)[:4].tolist()
    assert not off, [(r, c, float(x[r, c]), int(scales[r, c // 32]), int(got[r, c]), int(want_codes[r, c])) for r, c in off]
    return codes, scales


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (2, 33), (5, 127), (7, 129), (4, 4099), (33, 1000), (257, 96)])
def test_quantize_against_search(dtype, rows, cols):
    g = _gen(rows * 7919 + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda") * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g, device="cuda").float())
    x[torch.rand((rows, cols), generator=g, device="cuda") < 0.05] = 0
    x[rows // 2] = 0
    x = x.to(DT[dtype])
    s, c = quantize_f64(x)
    codes, scales = _quantized(x, s, c)
    # whole groups are written, zero past the row's end
    groups = -(-cols // 32)
    if cols % 2:
        assert int((codes[:, cols // 2] >> 4).max()) == 0
    assert int(codes[:, -(-cols // 2):groups * 16].sum()) == 0 and int(scales[:, groups:].sum()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_borders(dtype):
    """Every border between two values and its neighbours, at several exponents, and both signs."""
    dt = DT[dtype]
    exps = {"bf16": (-120, -7, 0, 9, 120), "f16": (-12, -7, 0, 9, 13), "f32": (-120, -7, 0, 9, 120)}[dtype]
    rows = []
    for e in exps:
        for top in (4.0, 6.0, 7.5):
            mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
            row = [top]
            for m in mids:
                row += [m, m * (1 + torch.finfo(dt).eps), m * (1 - torch.finfo(dt).eps / 2), -m]
            row += [-0.0, 0.0, -top]
            rows.append([v * 2.0 ** e for v in row])
    x = torch.tensor(rows, dtype=torch.float64, device="cuda").to(dt)
    s, c = quantize_f64(x)
    codes, _ = _quantized(x, s, c)
    assert int(_codes_of(codes, 32)[0, 29]) == 8                 # -0 stays -0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_extremes(dtype):
    dt = DT[dtype]
    fi = torch.finfo(dt)
    small = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}[dtype]
    x = torch.zeros((8, 96), dtype=torch.float64, device="cuda")
    x[0, 3], x[0, 40], x[0, 41] = fi.max, -fi.max, fi.tiny
    x[1, 5], x[1, 6], x[1, 70] = small, -3 * small, 5 * small
    x[2, 0], x[2, 64] = fi.tiny, fi.tiny * 3
    x = x.to(dt)
    x[3, 1], x[3, 33] = float("inf"), 1.0
    x[4, 95] = float("-inf")
    x[5, 2], x[5, 3] = float("nan"), 7.0
    x[6] = 1.0
    s, c = quantize_f64(x)
    codes, scales = _quantized(x, s, c)
    assert scales[3, 0] == 255 and scales[3, 1] != 255 and scales[4, 2] == 255 and scales[5, 0] == 255
    y = qk.qk_mx4_dequantize(qk.qk_mx4_state_init(8, 96, codes, scales), torch.float32)
    assert bool(torch.isnan(y[3, :32]).all()) and bool(torch.isnan(y[5, :32]).all()) and not bool(torch.isnan(y[3, 32:]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_quantize_rows_apart_and_unaligned(dtype, off):
    g = _gen(11)
    wide = torch.randn((9, 300), generator=g, device="cuda").to(DT[dtype])
    x = wide[:, off:off + 201]
    s, c = quantize_f64(x)
    _quantized(x, s, c)
    one = wide.view(-1)[off:off + 5 * 96].view(5, 96)
    s, c = quantize_f64(one)
    _quantized(one, s, c)


def test_quantize_writes_nothing_else():
    g = _gen(12)
    x = torch.randn((6, 70), generator=g, device="cuda")
    codes = torch.full((8, 64), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((8, 12), 0xA5, dtype=torch.uint8, device="cuda")
    qk.qk_mx4_quantize(x, codes[:6], scales[:6])
    s, c = quantize_f64(x)
    assert torch.equal(_codes_of(codes[:6], 70), c) and torch.equal(scales[:6, :3], s)
    assert bool((codes[:6, 48:] == 0xA5).all()) and bool((codes[6:] == 0xA5).all())
    assert bool((scales[:6, 4:] == 0xA5).all()) and bool((scales[6:] == 0xA5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 31), (3, 33), (5, 257), (64, 1000), (3, 4099)])
def test_dequantize(dtype, rows, cols):
    dt = DT[dtype]
    codes, scales = make_mx4(_gen(rows + cols), rows, cols, 100, 150, extra=1)
    want = values(codes, scales, cols)
    buf = torch.full((rows * cols + 8,), 77.0, dtype=dt, device="cuda")
    for at in (0, 1):                                             # aligned to elements only
        out = buf[at:at + rows * cols].view(rows, cols)
        got = qk.qk_mx4_dequantize(qk.qk_mx4_state_init(rows, cols, codes, scales), dt, out)
        assert torch.equal(got, want.to(torch.float32).to(dt))
        assert bool((buf[at + rows * cols:] == 77.0).all())


def test_dequantize_every_scale():
    codes = torch.tensor([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] + [0] * 8], dtype=torch.uint8, device="cuda").repeat(256, 1)
    scales = torch.zeros((256, 4), dtype=torch.uint8, device="cuda")
    scales[:, 0] = torch.arange(256, device="cuda")
    want = values(codes, scales, 32)
    for dt in DT.values():
        got = qk.qk_mx4_dequantize(qk.qk_mx4_state_init(256, 32, codes, scales), dt)
        assert torch.equal(torch.nan_to_num(got.double(), nan=-1e300), torch.nan_to_num(want.float().to(dt).double(), nan=-1e300))


def _product(M, N, K, dtype, seed, low=115, high=130, extra=0):
    g = _gen(seed)
    xc, xs = make_mx4(g, M, K, low, high, extra=extra)
    wc, ws = make_mx4(g, N, K, low, high, extra=2 * extra)
    y = torch.full((M * N + 64,), 77.0, dtype=dtype, device="cuda")
    got = qk.qk_gemm_mx4(qk.qk_mx4_state_init(M, K, xc, xs), qk.qk_mx4_state_init(N, K, wc, ws), dtype, y[:M * N].view(M, N))
    assert bool((y[M * N:] == 77.0).all())
    xv, wv = values(xc, xs, K), values(wc, ws, K)
    check(got, xv @ wv.t(), product_bound(xv, wv, K), dtype, f"{M}x{N}x{K}")
    return got


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 128, 130, 257])
@pytest.mark.parametrize("N,K", [(1, 32), (16, 256), (33, 100), (130, 1000), (257, 513)])
def test_gemm_sizes(M, N, K):
    _product(M, N, K, torch.float32, M * 1009 + N + K)


@pytest.mark.parametrize("K", [1, 31, 32, 33, 63, 64, 96, 224, 255, 256, 257, 287, 511, 512, 513, 768, 1023, 1024, 1025, 1281, 3001, 4099])
@pytest.mark.parametrize("M", [3, 40, 200])
def test_gemm_lengths(M, K):
    _product(M, 70, K, torch.bfloat16, M + 31 * K, extra=K % 3)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(512, 3000, 4099), (1000, 5000, 640), (2100, 2100, 300), (4, 28672, 1024), (48, 4096, 2048)])
def test_gemm_large(dtype, M, N, K):
    _product(M, N, K, DT[dtype], M + N + K, 118, 126)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(2304, 4096, 300), (2250, 4001, 530), (1100, 4096, 1300), (1090, 4030, 2049)])
def test_gemm_more_tiles_than_workgroups(dtype, M, N, K):
    _product(M, N, K, DT[dtype], M + N + K, 118, 126)


@pytest.mark.parametrize("M", [5, 30, 300])
def test_gemm_wide_scales(M):
    """Groups of very different size, the least and the largest scales among them."""
    g = _gen(M)
    K, N = 700, 90
    xc, xs = make_mx4(g, M, K, 60, 150)
    wc, ws = make_mx4(g, N, K, 60, 150)
    xs[:, 3], ws[:, 5] = 0, 1
    xs[0, :22], ws[1, :22] = 200, 20
    got = qk.qk_gemm_mx4(qk.qk_mx4_state_init(M, K, xc, xs), qk.qk_mx4_state_init(N, K, wc, ws), torch.float32)
    xv, wv = values(xc, xs, K), values(wc, ws, K)
    check(got, xv @ wv.t(), product_bound(xv, wv, K), torch.float32)


@pytest.mark.parametrize("M", [4, 20, 50, 300])
def test_gemm_nan_scales_stay_in_their_rows(M):
    g = _gen(M)
    N, K = 140, 1050
    xc, xs = make_mx4(g, M, K)
    wc, ws = make_mx4(g, N, K)
    xs[2, 32], ws[7, 0], ws[139, 20] = 255, 255, 255
    got = qk.qk_gemm_mx4(qk.qk_mx4_state_init(M, K, xc, xs), qk.qk_mx4_state_init(N, K, wc, ws), torch.float32)
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[2], bad[:, 7], bad[:, 139] = True, True, True
    assert torch.equal(torch.isnan(got), bad)
    xs[2, 32], ws[7, 0], ws[139, 20] = 120, 120, 120
    xv, wv = values(xc, xs, K), values(wc, ws, K)
    check(got[~bad], (xv @ wv.t())[~bad], product_bound(xv, wv, K)[~bad], torch.float32)


def test_gemm_output_aligned_to_its_elements_only():
    g = _gen(3)
    for M in (3, 200):
        N, K = 133, 320
        xc, xs = make_mx4(g, M, K)
        wc, ws = make_mx4(g, N, K)
        xv, wv = values(xc, xs, K), values(wc, ws, K)
        for dt in DT.values():
            y = torch.full((M * N + 9,), 77.0, dtype=dt, device="cuda")
            got = qk.qk_gemm_mx4(qk.qk_mx4_state_init(M, K, xc, xs), qk.qk_mx4_state_init(N, K, wc, ws), dt, y[1:1 + M * N].view(M, N))
            check(got, xv @ wv.t(), product_bound(xv, wv, K), dt)
            assert float(y[0]) == 77.0 and bool((y[1 + M * N:] == 77.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 13, 16])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 32), (33, 100), (70, 256), (300, 1000), (1024, 1024), (65, 4099), (48, 16384)])
def test_gemv(dtype, M, N, K):
    dt = DT[dtype]
    g = _gen(M * 31 + N + K)
    wc, ws = make_mx4(g, N, K, extra=M % 2)
    x = torch.randn((M, K), generator=g, device="cuda").to(dt)
    y = torch.full((M * N + 64,), 77.0, dtype=dt, device="cuda")
    got = qk.qk_gemv_mx4(x, qk.qk_mx4_state_init(N, K, wc, ws), y[:M * N].view(M, N))
    wv = values(wc, ws, K)
    check(got, x.double() @ wv.t(), product_bound(x.double(), wv, K), dt)
    assert bool((y[M * N:] == 77.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gemv_values_of_different_size(dtype):
    """Nothing is taken from a small term by a large neighbour whose weight is 0, and scales reach over the whole range that
    the type of the result holds."""
    dt = DT[dtype]
    g = _gen(5)
    N, K = 64, 512
    wc, ws = make_mx4(g, N, K, 100, 125)
    x = torch.randn((3, K), generator=g, device="cuda").to(dt)
    x[:, 5] = 3e4
    wc[:, 2] &= 0x0F                                             # the weights that column 5 meets
    ws[3], ws[4, :8], ws[5, 3] = 1, 30, 250
    wc[5, 48:64] = 0
    got = qk.qk_gemv_mx4(x, qk.qk_mx4_state_init(N, K, wc, ws))
    wv = values(wc, ws, K)
    tiny = torch.full((3, N), K * 2.0 ** -126, dtype=torch.float64, device="cuda") * x.double().abs().amax()
    check(got, x.double() @ wv.t(), product_bound(x.double(), wv, K) + tiny, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gemv_bad_values_stay_in_their_rows(dtype):
    dt = DT[dtype]
    g = _gen(6)
    N, K = 100, 1000
    wc, ws = make_mx4(g, N, K)
    x = torch.randn((5, K), generator=g, device="cuda").to(dt)
    x[1, 999], x[3, 0] = float("nan"), float("inf")
    ws[17, 31] = 255
    got = qk.qk_gemv_mx4(x, qk.qk_mx4_state_init(N, K, wc, ws))
    assert not bool(torch.isfinite(got[1]).any()) and not bool(torch.isfinite(got[3]).any()) and bool(torch.isnan(got[:, 17]).all())
    keep = [i for i in range(N) if i != 17]
    assert bool(torch.isfinite(got[[0, 2, 4]][:, keep]).all())


def test_same_bits_every_call_and_on_another_stream():
    g = _gen(8)
    xc, xs = make_mx4(g, 300, 700)
    wc, ws = make_mx4(g, 260, 700)
    X, W = qk.qk_mx4_state_init(300, 700, xc, xs), qk.qk_mx4_state_init(260, 700, wc, ws)
    a = torch.randn((4, 700), generator=g, device="cuda").bfloat16()
    first = qk.qk_gemm_mx4(X, W), qk.qk_gemv_mx4(a, W), qk.qk_mx4_quantize(a)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = qk.qk_gemm_mx4(X, W), qk.qk_gemv_mx4(a, W), qk.qk_mx4_quantize(a)[0]
    side.synchronize()
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_captured_and_replayed():
    g = _gen(9)
    x = torch.randn((20, 500), generator=g, device="cuda").bfloat16()
    w = qk.quantize_mx4(torch.randn((300, 500), generator=g, device="cuda").bfloat16())
    codes, scales = qk.qk_mx4_quantize(x)
    X = qk.qk_mx4_state_init(20, 500, codes, scales)
    y, v = qk.qk_gemm_mx4(X, w.state), qk.qk_gemv_mx4(x[:3], w.state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qk.qk_mx4_quantize(x, codes, scales)
        qk.qk_gemm_mx4(X, w.state, y=y)
        qk.qk_gemv_mx4(x[:3], w.state, v)
    for i in range(3):
        x.copy_(torch.randn((20, 500), generator=g, device="cuda").bfloat16())
        y.zero_()
        v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, qk.qk_gemm_mx4(qk.quantize_mx4(x).state, w.state)), i
        assert torch.equal(v, qk.qk_gemv_mx4(x[:3], w.state)), i


def test_weight_class_runs_as_used():
    g = _gen(10)
    w0 = torch.randn((200, 416), generator=g, device="cuda").bfloat16() * 0.02
    w = qk.quantize_mx4(w0)
    assert w.shape == (200, 416)
    v = w.dequantize(torch.float32)
    # floor(log2 top) - 2: a value is off by half its step or, between 6 and 8 units, by what exceeds 6 (a quarter)
    assert float(((v - w0.float()).abs() / w0.float().abs().view(200, 13, 32).amax(2).repeat_interleave(32, 1)).max()) <= 0.25
    x = torch.randn((37, 416), generator=g, device="cuda").bfloat16()
    xq = qk.quantize_mx4(x).dequantize(torch.float32).double()
    check(w.gemm(x), xq @ v.double().t(), product_bound(xq, v.double(), 416), torch.bfloat16)
    check(w.gemv(x[:7]), x[:7].double() @ v.double().t(), product_bound(x[:7].double(), v.double(), 416), torch.bfloat16)
    assert half_step(torch.bfloat16) == 2.0 ** -8


def test_offsets_past_32_bits():
    """A weight of more than 4 GiB of codes: its last rows."""
    N, K = 540000, 16384
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda")
    g = _gen(13)
    tc, ts = make_mx4(g, 40, K)
    codes[-40:], scales[-40:] = tc, ts
    W = qk.qk_mx4_state_init(N, K, codes, scales)
    wv = values(tc, ts, K)
    x = torch.randn((2, K), generator=g, device="cuda").bfloat16()
    got = qk.qk_gemv_mx4(x, W)
    assert float(got[:, :-40].abs().max()) == 0.0
    check(got[:, -40:], x.double() @ wv.t(), product_bound(x.double(), wv, K), torch.bfloat16)
    for M in (2, 300):
        xc, xs = make_mx4(g, M, K)
        got = qk.qk_gemm_mx4(qk.qk_mx4_state_init(M, K, xc, xs), W)
        xv = values(xc, xs, K)
        assert float(got[:, :-40].abs().max()) == 0.0
        check(got[:, -40:], xv @ wv.t(), product_bound(xv, wv, K), torch.bfloat16)
    del got
    tail = qk.qk_mx4_dequantize(qk.qk_mx4_state_init(N, K, codes, scales))[-40:]
    assert torch.equal(tail, wv.bfloat16())


def test_more_short_rows_than_a_launch_has_threads_for():
    rows = (1 << 29) + 7
    x = torch.ones((rows, 1), dtype=torch.bfloat16, device="cuda")
    at = [0, 1, (1 << 28) - 1, 1 << 28, 1 << 29, rows - 1]
    for i, r in enumerate(at):
        x[r] = -2.0 ** i
    codes, scales = qk.qk_mx4_quantize(x)
    st = qk.qk_mx4_state_init(rows, 1, codes, scales)
    y = qk.qk_mx4_dequantize(st)
    assert torch.equal(y, x)
    del y
    one = qk.quantize_mx4(torch.ones((1, 1), dtype=torch.bfloat16, device="cuda"))
    got = qk.qk_gemm_mx4(one.state, st, torch.bfloat16)             # so many outputs of one row
    assert torch.equal(got.view(-1), x.view(-1))
    del got
    got = qk.qk_gemm_mx4(st, one.state, torch.bfloat16)             # and so many rows
    assert torch.equal(got.view(-1), x.view(-1))


@pytest.mark.parametrize("M", [1, 3, 6, 16])
@pytest.mark.parametrize("N,K", [(64, 512), (33, 100), (300, 1001), (48, 16384), (70000, 300)])
def test_gemv_largest_scales(M, N, K):
    """Weights of the two largest scales pass bf16 (and fp32) by themselves; their products with small activations do not.
    What lies past a row's end, and weights of 0, meet them too."""
    dt = torch.bfloat16
    g = _gen(M + N + K)
    wc, ws = make_mx4(g, N, K, 115, 130)
    groups = -(-K // 32)
    big = torch.rand((N, groups), generator=g, device="cuda") < 0.2
    ws[:, :groups] = torch.where(big, torch.randint(252, 255, (N, groups), generator=g, device="cuda", dtype=torch.uint8), ws[:, :groups])
    ws[::3, groups - 1] = 254                                    # the last group, partial in most
    ws[4], wc[5, :16], ws[5, 0] = 254, 0, 253                    # (row 5: weights of 0)
    ws[5, 1:groups] = 120
    x = (torch.randn((M, K), generator=g, device="cuda") * 2.0 ** -20).to(dt)
    x[:, ::7] = 0
    if M > 1:
        x[1] = 0
    got = qk.qk_gemv_mx4(x, qk.qk_mx4_state_init(N, K, wc, ws))
    wv = values(wc, ws, K)
    bound = product_bound(x.double(), wv, K)
    check(got, x.double() @ wv.t(), bound, dt)
    if M > 1:
        assert float(got[1].abs().max()) == 0.0
    if M > 1:                                                    # a row's bits do not depend on the others
        other = x.clone()
        other[0] = float("nan")
        assert torch.equal(qk.qk_gemv_mx4(other, qk.qk_mx4_state_init(N, K, wc, ws))[1:], got[1:])
    ws[7, 0] = 255                                               # beside a NaN scale, too
    got = qk.qk_gemv_mx4(x, qk.qk_mx4_state_init(N, K, wc, ws))
    keep = torch.arange(N, device="cuda") != 7
    assert bool(torch.isnan(got[:, 7]).all())
    check(got[:, keep], (x.double() @ wv.t())[:, keep], bound[:, keep], dt)


@pytest.mark.parametrize("M", [5, 30, 100, 300])
def test_gemm_largest_scales(M):
    """The two largest scales against small ones: no product of a value and a scale is made by itself."""
    g = _gen(M)
    N, K = 150, 700
    xc, xs = make_mx4(g, M, K, 60, 100)
    wc, ws = make_mx4(g, N, K, 115, 130)
    ws[::3, 4], ws[1::3, 21], ws[2::5, 0] = 254, 253, 252
    got = qk.qk_gemm_mx4(qk.qk_mx4_state_init(M, K, xc, xs), qk.qk_mx4_state_init(N, K, wc, ws), torch.float32)
    xv, wv = values(xc, xs, K), values(wc, ws, K)
    check(got, xv @ wv.t(), product_bound(xv, wv, K), torch.float32)


@pytest.mark.parametrize("M", [1, 16, 30, 100, 130, 700, 2100])
@pytest.mark.parametrize("N,K", [(40, 4099), (300, 1000), (2100, 8192)])
def test_gemm_of_whole_numbers_is_exact(M, N, K):
    """Sums below 2^24 units: nothing may be lost, however small beside the rest."""
    g = _gen(M + N + K)
    xc, xs = make_mx4(g, M, K, 127, 128)
    wc, ws = make_mx4(g, N, K, 126, 127)
    got = qk.qk_gemm_mx4(qk.qk_mx4_state_init(M, K, xc, xs), qk.qk_mx4_state_init(N, K, wc, ws), torch.float32)
    xv, wv = values(xc, xs, K), values(wc, ws, K)
    # values are multiples of 1/2 and 1/4, at most 12 and 6: sums of multiples of 1/8
    assert float((xv.abs() @ wv.abs().t()).max()) * 8 < 2 ** 24
    assert torch.equal(got.double(), xv @ wv.t())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 4, 7, 16])
@pytest.mark.parametrize("N,K", [(40, 4099), (300, 1000), (70000, 300), (48, 16384)])
def test_gemv_of_whole_numbers_is_exact(dtype, M, N, K):
    g = _gen(M + N + K)
    wc, ws = make_mx4(g, N, K, 126, 128)
    x = torch.randint(-8, 9, (M, K), generator=g, device="cuda").to(DT[dtype])
    x[:, ::3] = 0.5
    wv = values(wc, ws, K)
    # multiples of 1/8; sums of absolute values below 2^24 of them
    assert float((x.double().abs() @ wv.abs().t()).max()) * 8 < 2 ** 24
    got = qk.qk_gemv_mx4(x, qk.qk_mx4_state_init(N, K, wc, ws))
    assert torch.equal(got, (x.double() @ wv.t()).float().to(DT[dtype]))
