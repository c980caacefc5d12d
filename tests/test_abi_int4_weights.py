"""What the binding refuses of the parts of an int4 weight, on host tensors (no GPU needed: a weight that passes these
checks is refused for not being on a device, which is how a test sees that it passed)."""

import pytest
import torch

import bit_blockwise_weight_amd as qk


def _codes(rows, cols):
    return torch.zeros((rows, (cols // 2 + 15) // 16 * 16), dtype=torch.uint8)


@pytest.mark.parametrize("rows,cols,group", [(6, 128, 32), (64, 96, 32), (5, 300, 128)])
def test_scales_and_zeros_laid_out_by_group_are_refused(rows, cols, group):
    """[G, rows] has as many values as [rows, G], and is how some checkpoints hold them."""
    groups = -(-cols // group)
    assert groups != rows
    scales, zeros = torch.ones((rows, groups), dtype=torch.float16), torch.zeros((rows, groups), dtype=torch.uint8)

    def init(s, z):
        return qk.qk_int4_state_init(rows, cols, group, _codes(rows, cols), s, z)

    with pytest.raises(ValueError, match="scales must be"):
        init(scales.t().contiguous(), zeros)
    with pytest.raises(ValueError, match="zeros must be"):
        init(scales, zeros.t().contiguous())
    for s, z in ((scales, zeros), (scales, None), (scales.view(-1), zeros.view(-1)), (scales.view(1, rows, groups), zeros)):
        with pytest.raises(ValueError, match="HIP device"):
            init(s, z)


def test_one_group_per_row_in_any_shape():
    """The memory is the same."""
    for shape in ((8, 1), (8,), (1, 8)):
        with pytest.raises(ValueError, match="HIP device"):
            qk.qk_int4_state_init(8, 64, 0, _codes(8, 64), torch.ones(shape, dtype=torch.float16))
