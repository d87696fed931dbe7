"""ep_expert_linear_w4 in each of the ways the library takes (by rows of an
expert, inputs, outputs and items), with the bounds of test_gpu_expert_w4.py."""
import numpy as np
import pytest
import torch

from combine_get_dispatch_02_amd import ep
from test_gpu_expert_w4 import DEV, check, inputs, weights

pytestmark = pytest.mark.gpu


# Scales through shared memory (K up to 8192), eight at a time (K % 256 == 0), singly.
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [128, 256, 512, 1024, 2560, 7168, 8064, 8192, 8320, 8704, 768, 1280, 640, 1152])
def test_streamed_and_split(K, silu):
    check([1, 0, 16, 3], K, 40, silu, seed=K)
    check([2], K, 72, silu, seed=K)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K,N", [(512, 1000), (1536, 136), (768, 1000), (384, 1000), (256, 1000)])
def test_streamed_whole(K, N, silu):
    """Items for every wave: 90 experts of few rows."""
    rng = np.random.default_rng(K)
    check([int(v) for v in rng.integers(0, 16, 90)], K, N if N < 500 else N // (2 if silu else 1) // 8 * 8, silu, seed=K)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 1024, 1408])
@pytest.mark.parametrize("rows", [17, 32, 33, 64, 65, 96, 97, 128, 129, 200])
def test_tiles_of_every_height(rows, K, silu):
    check([rows, 0, 40], K, 136, silu, seed=rows)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [128, 384, 512, 640, 768, 896, 1152])
@pytest.mark.parametrize("tallest", [64, 128])
def test_tiles_of_every_height_and_depth(tallest, K, silu):
    """36 experts and outputs enough for tiles of `tallest` rows, which are full,
    or end after 1 to 4 times 32 rows; inputs that end 0 to 3 steps into the four
    whose scales are loaded at once."""
    counts = [int(v) for v in np.linspace(13, tallest, 36)]
    check(counts, K, 1288 if silu else 2568, silu, seed=K)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("N", [8, 56, 64, 72, 256, 264, 512, 520, 776])
def test_tiles_of_every_width(N, silu):
    check([70, 20], 256, N, silu, seed=N)


@pytest.mark.parametrize("silu", [False, True])
def test_full_tiles(silu):
    """So many rows and outputs that tiles keep their 128 rows."""
    check([1601, 33, 0, 1570, 128, 2900], 256, 1032 if silu else 2056, silu, seed=1)


@pytest.mark.parametrize("capacity,counts", [(33, [33, 16, 17, 0, 1]), (130, [130, 129, 16, 3, 64, 0]), (17, [17, 16, 0, 2])])
def test_padded_regions_of_both_kinds(capacity, counts):
    for silu in (False, True):
        check(counts, 512, 88, silu, capacity=capacity, seed=capacity)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [256, 640, 1024])
def test_rows_about_the_two_ways(K, silu):
    counts = [12, 13, 0, 11, 16, 14, 12, 17, 1]
    check(counts, K, 72, silu, seed=K)
    check(counts, K, 72, silu, capacity=17, seed=K)
    check([12, 3, 0, 11], K, 72, silu, capacity=12, seed=K)


def test_one_row_the_same_in_every_tile():
    wc, ws = (torch.from_numpy(v).to(DEV) for v in weights(1, 600, 640, 2))
    x = inputs(1, 640, 1).expand(1000, 640).contiguous().to(DEV)
    y = ep.ep_expert_linear_w4(x, torch.tensor([0, 1000], dtype=torch.int32, device=DEV), wc, ws)
    assert torch.equal(y, y[:1].expand_as(y))


def test_skewed_batch_of_thousands():
    """Zipf rows: one expert with most of them, many with one or none."""
    counts = [int(v) for v in 3000 / np.arange(1, 200) ** 1.3]
    check(counts + [0] * 57, 128, 40, True, seed=9)


def test_offsets_out_of_order_share_no_row():
    """Each expert takes what the ones before it have left."""
    x = inputs(50, 256, 3)
    wc, ws = weights(5, 24, 256, 4)
    dev = [torch.from_numpy(v).to(DEV) for v in (wc, ws)]
    for m, spans in (([0, 30, 10, 40, 20, 50], [(0, 30), (0, 0), (30, 10), (0, 0), (40, 10)]),
                     ([-7, 20, 2 ** 31 - 1, 0, 50, 50], [(0, 20), (20, 30), (0, 0), (0, 0), (0, 0)]),
                     ([40, 30, 20, 10, 5, 0], [(0, 0)] * 5),
                     ([5, 5, 60, 60, 3, 2], [(0, 0), (5, 45), (0, 0), (0, 0), (0, 0)])):
        y = torch.full((50, 24), 7.0, dtype=torch.bfloat16, device=DEV)
        ep.ep_expert_linear_w4(x.to(DEV), torch.tensor(m, dtype=torch.int32, device=DEV), *dev, out=y)
        ref = torch.full((50, 24), 7.0, dtype=torch.bfloat16, device=DEV)
        for e, (first, count) in enumerate(spans):
            if count:
                off = torch.zeros(6, dtype=torch.int32, device=DEV)
                off[e + 1:] = count
                ref[first:first + count] = ep.ep_expert_linear_w4(x[first:first + count].to(DEV).contiguous(), off, *dev)
        # One row alone may be split among waves where a batch is not.
        assert torch.allclose(y.float(), ref.float(), rtol=2.0 ** -7, atol=1e-3)


def test_scales_at_any_word():
    """w_scales needs 4-byte alignment only."""
    for K in (512, 1024, 768, 640):
        wc, ws = weights(3, 48, K, 5)
        room = torch.zeros(ws.size + 12, dtype=torch.uint8, device=DEV)
        x, off = inputs(40, K, 1).to(DEV), torch.tensor([0, 3, 30, 40], dtype=torch.int32, device=DEV)
        codes, scales = torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
        ref = ep.ep_expert_linear_w4(x, off, codes, scales, epilogue="silu_mul")
        for shift in (4, 8, 12):
            room[shift:shift + ws.size] = scales.view(-1)
            at = room[shift:shift + ws.size].view(3, 48, K // 32)
            assert torch.equal(ep.ep_expert_linear_w4(x, off, codes, at, epilogue="silu_mul"), ref)
