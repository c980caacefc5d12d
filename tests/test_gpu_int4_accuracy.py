"""How far qk_gemv_int4 is from the product in 64 bits where rounding shows: large activations whose weights are 0,
values of ordinary size in the norm.

Tolerance, derived before the first run.  y is rounded once: half a step, finfo.eps / 2 relative to the value.  Before
that the products are summed in fp32 (a sum in a matrix instruction may cut instead of rounding: a whole step, 2^-23, of
the terms that it has).  A term is |x| |s| |q - z|: one whose code is its zero point is 0 and costs nothing, however
large its activation.  An addend passes at most 4 matrix instructions of 32 products in its chunk of 128, a scale, a
factor, one addition for every 1024 of K at least and 8 waves: depth 128 + ceil(K / 128) + 16.
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


def _tolerance(x, w64, ref, dtype):
    K = x.shape[1]
    terms = x.double().abs() @ w64.abs().t()
    return torch.finfo(dtype).eps / 2 * ref.abs() + 2.0 ** -23 * (128 + -(-K // 128) + 16) * terms \
        + torch.finfo(dtype).smallest_normal


def _norm_bound(dtype, values):
    """A rounding is off by at most half a step, and spread evenly over it: in the norm 1 / sqrt(3) of that, with
    three standard deviations on top: a squared error is v^2 u^2, u even, v (a normal sum times a normal scale) of fourth
    moment 9, which makes 9 * 9 / 5 - 1 the variance of one relative to its mean.  The sums' own rounding, independent
    from term to term, is 2^-23 sqrt(128 + 16) of them and less than 2^-18 of the result."""
    spread = min(1 + 3 * (15.2 / values) ** 0.5 / 2, 3 ** 0.5)
    return torch.finfo(dtype).eps / 2 * 3 ** -0.5 * spread + 2.0 ** -18


def _check(y, ref, tol, what):
    err = (y.double() - ref).abs()
    worst = float((err / tol).max())
    assert worst <= 1.0, f"{what}: error {worst} of the tolerance"
    rel = float(err.norm() / ref.norm())
    bound = _norm_bound(y.dtype, ref.numel())
    assert rel <= bound, f"{what}: relative error {rel} in the norm, {bound} allowed"


@pytest.mark.parametrize("dtype,size", [(torch.float16, 60000.0), (torch.bfloat16, 2.0 ** 15), (torch.bfloat16, 2.0 ** 24)])
@pytest.mark.parametrize("group", [32, 64, 128, 0])
@pytest.mark.parametrize("zeros", [True, False])
def test_large_activation_of_weight_zero(dtype, size, group, zeros):
    """One activation far above the others, whose code is the zero point in every row: it must not cost the others
    any accuracy, at any number of rows."""
    N = 64
    for K in (128, 1000, 4096):
        gen = torch.Generator(device="cuda").manual_seed(K)
        q, s, z = make_int4(gen, N, K, group, zeros, torch.float16)
        if zeros:
            z.clamp_(max=15)
        at = [5, K // 2 + 3] if K > 128 else [77]
        for k in at:
            q[:, k] = 8 if z is None else z[:, k // group if group else 0]
        w64 = int4_f64(q, s, z, group)
        assert bool((w64[:, at] == 0).all())
        w = qk.Int4Weight(q, s, z, group)
        x = torch.randn((16, K), generator=gen, device="cuda").to(dtype)
        x[:, at] = size
        ref = x.double() @ w64.t()
        tol = _tolerance(x, w64, ref, dtype)
        # the large value itself is no term: its own |x| |w| above is 0
        for M in (1, 2, 4, 5, 8, 16):
            say(f"case: gemv_int4 large activation of weight 0 M={M} K={K} group={group} zeros={zeros} {dtype} {size}")
            _check(w.gemv(x[:M].contiguous()), ref[:M], tol[:M], f"M={M} K={K} group={group}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_far_below_the_largest(dtype):
    """Values of 8 bits and 2^25 to 2^28 below one of weight 0 (fp16: of 11 bits, the type's smallest ones): held exactly."""
    N, K = 64, 384
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, s, z = make_int4(gen, N, K, 128, True, torch.float16)
    z.clamp_(max=15)
    at = [0, 200, 383]
    for k in at:
        q[:, k] = z[:, k // 128]
    w64 = int4_f64(q, s, z, 128)
    w = qk.Int4Weight(q, s, z, 128)
    sign = torch.randint(0, 2, (16, K), generator=gen, device="cuda") * 2.0 - 1
    x = (1 + torch.randint(0, 128, (16, K), generator=gen, device="cuda") / 128) * sign
    x = (x * 2.0 ** torch.randint(0, 4, (16, K), generator=gen, device="cuda")).to(dtype)
    if dtype is torch.float16:
        x = x * 2.0 ** -14                                   # 2^-14 and up, to 7 bits below: partly subnormal
        x[:, ::2] *= 2.0 ** -7
    x[:, at] = 2.0 ** 28 if dtype is torch.bfloat16 else 65504.0
    ref = x.double() @ w64.t()
    # (fp16 outputs of this size are subnormal: half of 2^-24 and no more than that)
    tol = _tolerance(x, w64, ref, dtype) - torch.finfo(dtype).smallest_normal + 2.0 ** -25
    for M in (1, 4, 7, 16):
        say(f"case: gemv_int4 values far below the largest M={M} {dtype}")
        err = (w.gemv(x[:M].contiguous()).double() - ref[:M]).abs()
        assert float((err / tol[:M]).max()) <= 1.0, f"M={M}"


def _random(seed, M, N, K, group, zeros, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, s, z = make_int4(gen, N, K, group, zeros, torch.float16)
    if zeros:
        z.clamp_(max=15)
    x = torch.randn((M, K), generator=gen, device="cuda").to(dtype)
    w64 = int4_f64(q, s, z, group)
    ref = x.double() @ w64.t()
    return qk.Int4Weight(q, s, z, group), x, ref, _tolerance(x, w64, ref, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 16])
def test_several_items_per_workgroup(M, group, dtype):
    """More rows than the chip's workgroups take at a time in one item each, in two tiles a wave where that is done:
    sums are kept in turn in each of the places for them, and the next item's codes are on their way."""
    for N, K in ((20011, 1024), (40000, 2048)):
        say(f"case: gemv_int4 several items M={M} N={N} K={K} group={group} {dtype}")
        w, x, ref, tol = _random(20, M, N, K, group, group != 64, dtype)
        _check(w.gemv(x), ref, tol, f"M={M} N={N} K={K} group={group}")


@pytest.mark.parametrize("M,K", [(2, 28032), (4, 14100), (5, 12032), (8, 14080), (16, 12000)])
@pytest.mark.parametrize("group", [32, 128])
def test_several_items_with_streamed_activations(M, K, group):
    """The same where a row's activations do not stay on the chip."""
    for dtype in (torch.bfloat16, torch.float16):
        say(f"case: gemv_int4 several items, streamed activations M={M} K={K} group={group} {dtype}")
        w, x, ref, tol = _random(21, M, 17011, K, group, True, dtype)
        _check(w.gemv(x), ref, tol, f"M={M} K={K} group={group}")


@pytest.mark.parametrize("M", [1, 4, 8])
def test_grouped_equals_single_where_the_launches_differ(M):
    """Weights that alone take one tile a wave, together two; and short rows beside a long one that does not stay."""
    for sizes in ([(4096, 4096, 128)] * 7, [(2048, 1024, 64), (1024, 14100, 64), (3000, 2048, 64), (20000, 1024, 64)],
                  [(2048, 1024, 32), (100, 28032, 32), (4096, 512, 32)]):
        say(f"case: gemv_int4 grouped against single M={M} {sizes[0]} and {len(sizes) - 1} more")
        for dtype in (torch.bfloat16, torch.float16):
            made = [_random(30 + i, M, N, K, group, True, dtype) for i, (N, K, group) in enumerate(sizes)]
            ys = qk.qk_gemv_int4_grouped([(x, w.state) for w, x, _, _ in made])
            for y, (w, x, ref, tol) in zip(ys, made):
                assert torch.equal(y, w.gemv(x))
                _check(y, ref, tol, f"M={M} {dtype}")
