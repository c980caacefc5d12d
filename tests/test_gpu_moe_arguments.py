"""Arguments of the expert layer's binding that are not plain numbers."""

import pytest
import torch

import bit_blockwise_weight_amd as qk
from tests.gpu_common import require_gpu, say
from tests.gpu_int4 import make_int4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_top_k_as_a_tensor_that_changes():
    """The workspace goes by the value of top_k at the call, not by the object."""
    say("case: moe top_k as a host tensor, 1 then 4")
    gen = torch.Generator(device="cuda").manual_seed(1)
    E, H, I, T = 6, 96, 64, 5
    up = qk.Int4Weight(*make_int4(gen, E * 2 * I, H, 32, True, torch.float16), 32)
    down = qk.Int4Weight(*make_int4(gen, E * H, I, 32, True, torch.float16), 32)
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    lg = torch.randn((T, E), generator=gen, device="cuda")
    k = torch.tensor(1)
    for value in (1, 4, 2):
        k.fill_(value)
        assert torch.equal(qk.qk_moe_int4(x, lg, k, up.state, down.state), qk.qk_moe_int4(x, lg, value, up.state, down.state))
