"""ep_expert_linear_i8 in each of the ways the library takes (by rows, inputs, outputs and
items), with the bounds of test_gpu_expert_i8.py."""
import numpy as np
import pytest
import torch

import i8_plan
from combine_get_dispatch_02_amd import ep
from test_gpu_expert_i8 import DEV, check, dev, matrix, rows_of

pytestmark = pytest.mark.gpu


def counted(counts, K, N, silu, capacity=0):
    rows = len(counts) * capacity if capacity else sum(counts)
    return i8_plan.way(rows, len(counts), K, N, silu)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [1024, 1152, 1280, 1408, 2048, 7168, 8320, 65536])
def test_streamed_and_split(K, silu):
    for counts, N in (([1, 0, 16, 3], 40), ([2], 72), ([40, 17], 104)):
        assert counted(counts, K, N, silu) == "streams"
        check(counts, K, N, silu, seed=K)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [1024, 1152, 1536])
def test_streamed_whole(K, silu):
    """Items for more than the waves of every block: 18 experts of one row."""
    N = 1960 if silu else 3912
    assert counted([1] * 18, K, N, silu) == "streams"
    check([1] * 18, K, N, silu, seed=K)


def test_streamed_padded():
    counts = [0, 20, 7, 1, 33]
    assert counted(counts, 1024, 104, False, 33) == "streams"
    check(counts, 1024, 104, False, capacity=33)
    check(counts, 1152, 104, True, capacity=33)


HEIGHTS = [1, 16, 17, 32, 33, 64, 65, 96, 127, 128, 129, 191, 192, 193, 255, 256, 257, 320, 513, 700]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 896])
@pytest.mark.parametrize("rows", HEIGHTS)
def test_tiles_of_every_height(rows, K, silu):
    assert counted([rows, 0, 40], K, 136, silu) == "tiles"
    check([rows, 0, 40], K, 136, silu, seed=rows)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [128, 256, 384, 640, 1024, 1152])
def test_tiles_in_a_row(K, silu):
    """Several items a block, of all heights in turn: loads that run on from one to the
    next, and stores between them."""
    rng = np.random.default_rng(K)
    counts = [HEIGHTS[i] if i < len(HEIGHTS) else int(v) for i, v in enumerate(rng.integers(0, 280, 50))]
    N = 1032 if silu else 2056
    assert counted(counts, K, N, silu) == "tiles"
    check(counts, K, N, silu, seed=K)
    check([256] * 40, K, N, silu, seed=K + 1)


@pytest.mark.parametrize("height", [60, 120, 180, 250])
def test_the_same_item_after_item(height):
    """All blocks the same few codes over and over: every item of one height, three a
    block, K of one stage up; and ten runs give one result."""
    for K in (128, 256, 1280):
        counts = [height] * 48
        y = check(counts, K, 4096, False, seed=K)
        x, xs = rows_of(sum(counts), K, K)
        w, ws = matrix(48, 4096, K, K)
        args = dev(x), dev(xs), dev(np.cumsum([0] + counts).astype(np.int32)), dev(w), dev(ws)
        for _ in range(10):
            assert torch.equal(ep.ep_expert_linear_i8(*args), y)


def test_outputs_up_to_the_limit():
    N, K = 1 << 22, 128
    x, xs = rows_of(70, K, 1)
    w, ws = matrix(1, 8, K, 2)
    big = torch.zeros(1, N, K, dtype=torch.int8, device=DEV)
    big[0, -8:] = dev(w[0])
    scales = torch.ones(1, N, device=DEV)
    scales[0, -8:] = dev(ws[0])
    off = torch.tensor([0, 70], dtype=torch.int32, device=DEV)
    y = ep.ep_expert_linear_i8(dev(x), dev(xs), off, big, scales)
    one = ep.ep_expert_linear_i8(dev(x), dev(xs), off, dev(w), dev(ws))
    assert torch.equal(y[:, -8:], one) and not y[:, :-8].any()
