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

