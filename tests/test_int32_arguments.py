"""The binding refuses numbers that do not fit the library's 32-bit arguments, of
which ctypes would pass the low 32 bits on.  On the CPU: sizes from tensors without
storage, refused before anything is asked of the device."""
import pytest
import torch

from combine_get_dispatch_02_amd import ep

WRAPS = [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63, 2 ** 64 + 2, -2 ** 31 - 1, -2 ** 32 + 1]


def empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("v", WRAPS)
def test_numbers(v):
    l = torch.zeros(4, 8)
    for kw in (dict(num_groups=v), dict(topk_groups=v), dict(group_top=v)):
        with pytest.raises(ValueError, match="ep_route.*32-bit"):
            ep.ep_route(l, 2, **kw)
    with pytest.raises(ValueError, match="ep_route.*32-bit"):
        ep.ep_route(l, v)
    x, off = torch.zeros(4, 128).bfloat16(), torch.zeros(2, dtype=torch.int32)
    w, s = torch.zeros(2, 8, 64, dtype=torch.uint8), torch.zeros(2, 8, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="ep_expert_linear_w4.*32-bit"):
        ep.ep_expert_linear_w4(x, off, w, s, capacity=v)


@pytest.mark.parametrize("v", [2 ** 31, 2 ** 32 + 8])
def test_sizes_of_tensors(v):
    i64, bf16, i32, u8 = torch.int64, torch.bfloat16, torch.int32, torch.uint8
    with pytest.raises(ValueError, match="ep_route.*32-bit"):
        ep.ep_route(empty(1, v), 2)
    with pytest.raises(ValueError, match="ep_route_backward.*32-bit"):
        ep.ep_route_backward(empty(1, v), empty(1, 2, dtype=i64), empty(1, 2))
    with pytest.raises(ValueError, match="ep_route_backward.*32-bit"):
        ep.ep_route_backward(empty(1, 8), empty(1, v, dtype=i64), empty(1, v))
    with pytest.raises(ValueError, match="ep_combine_backward.*32-bit"):
        ep.ep_combine_backward(empty(1, v, dtype=bf16), empty(2, v, dtype=bf16), empty(1, 2, dtype=i32), None)
    with pytest.raises(ValueError, match="ep_combine_backward.*32-bit"):
        ep.ep_combine_backward(empty(1, 8, dtype=bf16), empty(2, 8, dtype=bf16), empty(1, v, dtype=i32), None)
    for x, w in ((empty(1, v, dtype=bf16), empty(2, 8, 64, dtype=u8)), (empty(1, 128, dtype=bf16), empty(v, 8, 64, dtype=u8)),
                 (empty(1, 128, dtype=bf16), empty(2, v, 64, dtype=u8))):
        with pytest.raises(ValueError, match="ep_expert_linear_w4.*32-bit"):
            ep.ep_expert_linear_w4(x, empty(3, dtype=i32), w, empty(2, 8, 4, dtype=u8))


def test_what_fits_is_the_library_s_to_refuse():
    """A number of 32 bits gets as far as the next check."""
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_route(torch.zeros(4, 8), 2 ** 31 - 1, num_groups=-2 ** 31)
