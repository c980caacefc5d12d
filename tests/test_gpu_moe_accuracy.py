"""What the expert layer keeps of the inner values h.

All numbers here are integers that every step of the layer holds exactly as long as it keeps 23 bits or more, so the
output has to be the exact one.  Token t has x[0] = 1, x[1] = 13 and integers of 1..40 elsewhere; every gate row gives
g = 7 * 1 + 2 * 13 = 33, whose silu is 33 (1 / (1 + exp(-33)) is 1 to 2^-47); the up rows 2 i and 2 i + 1 differ by one
at x[0] alone, so h[2 i + 1] = h[2 i] + 33, of about 2^19.4; a row of the down matrix takes -c, +c of two such pairs, so its
sum has terms under 2^24 together, no rounding in fp32, and is 33 (c1 + c2), at most 198: a 16-bit number.  Of 16 bits
an h of 2^19.4 would be off by up to 4.
"""

import pytest
import torch

import bit_blockwise_weight_amd as qk
from tests.gpu_common import require_gpu, say
from tests.gpu_int4 import moe_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _weights(gen, H, I, large):
    """(gate_up [2 I, H], down [H, I]) in -8..7, scales of the gate_up rows [2 I, 1], the down sums c1 + c2 [H]"""
    gate = torch.zeros((I, H), dtype=torch.int64)
    gate[:, 0], gate[:, 1] = 7, 2
    up = torch.randint(1, 8, (I // 2, H), generator=gen).repeat_interleave(2, 0)
    up[:, 0] = torch.tensor([2, 3]).repeat(I // 2)
    scale = torch.ones((2 * I, 1))
    if large:                                  # a pair far above the others, of weight 0 everywhere
        scale[I + 4:I + 6] = 1024.0
    down = torch.zeros((H, I), dtype=torch.int64)
    sums = torch.zeros(H, dtype=torch.int64)
    pairs = [i for i in range(I // 2) if not (large and i == 2)]
    for n in range(H):
        a, b = torch.randperm(len(pairs), generator=gen)[:2].tolist()
        for i in (pairs[a], pairs[b]):
            c = int(torch.randint(1, 4, (1,), generator=gen)) * (1 if n % 2 else -1)
            down[n, 2 * i], down[n, 2 * i + 1] = -c, c
            sums[n] += c
    return torch.cat([gate, up]), down, scale, sums


def _tokens(gen, T, H, dtype):
    x = torch.randint(1, 41, (T, H), generator=gen)
    x[:, 0], x[:, 1] = 1, 13
    return x.to(dtype).cuda()


def _logits(T, E, dtype=torch.float32):
    lg = torch.zeros((T, E))
    lg[:, 1] = 400.0                           # every token at expert 1, whose weight is then 1
    return lg.to(dtype).cuda()


def _stack(w, scale, E):
    """expert 1 of E, the others zero"""
    q = torch.full((E * w.shape[0], w.shape[1]), 8, dtype=torch.uint8)
    q[w.shape[0]:2 * w.shape[0]] = (w + 8).to(torch.uint8)
    s = torch.ones((E * w.shape[0], 1))
    if scale is not None:
        s[w.shape[0]:2 * w.shape[0]] = scale
    return q.cuda(), s.cuda()


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("E", [2, 16])
@pytest.mark.parametrize("H,I", [(256, 128), (256, 2048)])
def test_int4_keeps_the_inner_values(H, I, E, large):
    gen = torch.Generator().manual_seed(1)
    gu, down, scale, sums = _weights(gen, H, I, large)
    (q1, s1), (q2, s2) = _stack(gu, scale, E), _stack(down, None, E)
    for group in (32, 64, 128, 0):
        n1, n2 = -(-H // group) if group else 1, -(-I // group) if group else 1
        w1 = qk.Int4Weight(q1, s1.expand(-1, n1).half(), None, group)
        w2 = qk.Int4Weight(q2, s2.expand(-1, n2).bfloat16(), None, group)
        for T in (1, 2, 3, 4, 8, 16):
            for dtype in (torch.bfloat16, torch.float16):
                say(f"case: moe_int4 inner values T={T} E={E} H={H} I={I} group={group} large={large} {dtype}")
                x = _tokens(gen, T, H, dtype)
                y = qk.qk_moe_int4(x, _logits(T, E), 1, w1.state, w2.state)
                assert torch.equal(y.cpu().long(), (33 * sums).expand(T, H)), f"T={T} group={group}"


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("E", [2, 16])
@pytest.mark.parametrize("H,I", [(256, 128), (256, 2048)])
def test_levels_keep_the_inner_values(H, I, E, large):
    """The same with a level table of its own, -8..7 (with +7 and 2^-3 in the place of two that are not used here)."""
    gen = torch.Generator().manual_seed(2)
    gu, down, scale, sums = _weights(gen, H, I, large)
    (q1, s1), (q2, s2) = _stack(gu, scale, E), _stack(down, None, E)
    levels = torch.arange(-8.0, 8.0)
    levels[0], levels[1] = 2.0 ** -12, 1.0e4
    keep = []

    def state(q, s, block):
        codes = ((q[:, 0::2] << 4) | q[:, 1::2]).view(-1)
        absmax = s.expand(-1, q.shape[1] // block).reshape(-1).contiguous().float()
        keep.append((codes, absmax))
        return qk.qk_state_init(qk.CUSTOM, levels, q.shape[0], q.shape[1], block, codes, absmax)

    for block in (64, 128):
        up, dn = state(q1, s1, block), state(q2, s2, block)
        for T in (1, 2, 3, 4, 8, 16):
            say(f"case: moe_nf4 own levels, inner values T={T} E={E} H={H} I={I} block={block} large={large}")
            x = _tokens(gen, T, H, torch.bfloat16)
            y = qk.qk_moe_nf4(x, _logits(T, E), 1, up, dn)
            assert torch.equal(y.cpu().long(), (33 * sums).expand(T, H)), f"T={T} block={block}"


def test_levels_of_very_different_size():
    """A table whose levels span 2^28, rows that read the small ones alone: each counts as its bf16 copy.  Tolerance: the
    output's rounding, and fp32 sums over at most 4 matrix instructions of 32 products a chunk, a scale, a factor, 4 chunks
    and 8 waves for each product (2^-23 a step, of the terms that it has), of which h itself is 2^-24."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    H, I, block, T = 256, 128, 64, 3
    levels = torch.tensor([1.37 * 2.0 ** (-2 * i) * (-1) ** i for i in range(15)] + [0.0])
    lv = levels.bfloat16().double().cuda()

    def weight(rows, cols):
        q = torch.randint(0, 4, (rows, cols), generator=gen, device="cuda", dtype=torch.uint8)
        q[1::4] += 10                                        # 2^-20 to 2^-26 of the largest, and no other
        q[2::4] = torch.randint(0, 16, (len(q[2::4]), cols), generator=gen, device="cuda", dtype=torch.uint8)
        q[1::4, ::9] = 15
        absmax = torch.rand(rows * cols // block, generator=gen, device="cuda") + 0.5
        codes = ((q[:, 0::2] << 4) | q[:, 1::2]).contiguous().view(-1)
        w = lv[q.long()] * absmax.double().view(rows, -1).repeat_interleave(block, 1)
        return w, qk.qk_state_init(qk.CUSTOM, levels, rows, cols, block, codes, absmax)

    up, up_state = weight(2 * I, H)
    down, down_state = weight(H, I)
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    x[:, ::5] *= 8
    y = qk.qk_moe_nf4(x, torch.zeros((T, 1), device="cuda"), 1, up_state, down_state)
    say("case: moe_nf4 levels of very different size")
    ref, bound = moe_f64(x, [[(0, 1.0)]] * T, lambda e: (up[:I], up[I:]), lambda e: down)
    tol = torch.finfo(x.dtype).eps / 2 * ref.abs() + 2.0 ** -23 * (128 + 4 + 8 + 2) * bound + 2.0 ** -126
    assert float(((y.double() - ref).abs() / tol).max()) <= 1.0
    small = slice(1, H, 4)
    assert float((y.double() - ref)[:, small].norm() / ref[:, small].norm()) <= torch.finfo(x.dtype).eps / 2
