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


@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8, torch.int32, torch.int64])
def test_codes_outside_four_bits_are_refused(dtype):
    scales = torch.ones((2, 1), dtype=torch.float16)
    for bad in ((16, -3, -1, 255) if dtype is not torch.int8 else (16, -3, -1, 127)):
        if dtype is torch.uint8 and bad < 0:
            continue
        codes = torch.full((2, 32), 7, dtype=dtype)
        codes[1, 5] = bad
        with pytest.raises(ValueError, match="0..15"):
            qk.Int4Weight(codes, scales, None, 32)
    with pytest.raises(ValueError, match="HIP device"):
        qk.Int4Weight(torch.arange(32).remainder(16).expand(2, 32).to(dtype), scales, None, 32)


@pytest.mark.parametrize("dtype,bad", [(torch.float32, (7.6, -1.0, 256.0, float("nan"), float("inf"))),
                                       (torch.float16, (8.5, -2.0, 300.0)), (torch.int32, (-1, 256)), (torch.int8, (-1,))])
def test_zero_points_that_are_no_bytes_are_refused(dtype, bad):
    codes, scales = torch.zeros((2, 64), dtype=torch.uint8), torch.ones((2, 2), dtype=torch.float16)
    for v in bad:
        zeros = torch.full((2, 2), 8, dtype=dtype)
        zeros[0, 1] = v
        with pytest.raises(ValueError, match="0..255"):
            qk.Int4Weight(codes, scales, zeros, 32)
    with pytest.raises(ValueError, match="HIP device"):
        qk.Int4Weight(codes, scales, torch.full((2, 2), 8, dtype=dtype), 32)
