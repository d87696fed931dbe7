"""ep_expert_linear_w4 on sizes that take its tiles (and whole, unsplit streams past
8192 inputs).  Which way a size takes is asked of the library's own rule, so a test
that no longer gets where it should fails, here and on the CPU.  Bounds as in
test_gpu_expert_w4.py."""
import numpy as np
import pytest
import torch

import plain64
import w4_plan
from combine_get_dispatch_02_amd import ep
from test_gpu_expert_w4 import DEV, check, inputs, weights

gpu = pytest.mark.gpu
HEIGHTS = [17, 32, 33, 64, 65, 96, 97, 128, 129, 200, 0, 13, 1, 255, 50, 80, 12, 112, 40, 31, 63, 95, 127, 100]


def narrow_counts(tile_rows, tail):
    """Whole tiles and a last one of `tail` rows."""
    return {32: [300, 290 + tail], 64: [10240, 256 + tail], 128: [20608 + tail]}[tile_rows]


# (counts, capacity, K's, N, silu, way, rows of a tile)
def sizes():
    ks = (128, 384, 512, 640, 896)
    for silu in (False, True):
        yield "heights", HEIGHTS, 0, ks, 2312 if silu else 4616, silu, "tiles", 128
        yield "heights 64", HEIGHTS, 0, (512, 768, 1408), 1288 if silu else 2568, silu, "tiles", 64
        few = [int(v) for v in np.random.default_rng(1).integers(0, 41, 40)]
        few[:6] = [12, 13, 40, 0, 1, 17]
        yield "padded", few, 40, (384, 896, 1024), 360 if silu else 712, silu, "both", 32
        yield "packed", [v // 2 for v in few[:-1]] + [500], 0, (640, 1024), 776 if silu else 1544, silu, "both", 32
        tall = [130, 129, 12, 13, 64, 0, 97, 33] * 5
        yield "padded tall", tall, 130, (256, 896), 1544 if silu else 3080, silu, "both", 128
        many = [0] * 2048
        for e in range(0, 2048, 97):
            many[e] = e % 89 + 1
        many[2047] = 3000 - sum(many)
        yield "2048 experts", many, 0, (128, 512), 40 if silu else 72, silu, "both", 128


SIZES = list(sizes())
NARROW = [(32, 8), (32, 56), (32, 64), (32, 72), (32, 256), (32, 264), (32, 512), (32, 520), (32, 776), (64, 8), (64, 72),
          (128, 8), (128, 264), (128, 776)]
LONG = [(8320, "single"), (8704, "eight")]
FULL = [340] * 5                                    # 1700 rows, tiles of 32


def rows_of(counts, capacity):
    return len(counts) * capacity if capacity else sum(counts)


def test_sizes_take_the_way_they_are_meant_for():
    for name, counts, capacity, _, N, silu, way, tile_rows in SIZES:
        assert w4_plan.way(rows_of(counts, capacity), capacity, len(counts), N, silu) == (way, tile_rows), name
    for tile_rows, N in NARROW:
        for tail in (20, 60, 90):
            counts = narrow_counts(tile_rows, tail)
            assert w4_plan.way(sum(counts), 0, len(counts), N, False) == ("tiles", tile_rows)
    for K, how in LONG:
        assert w4_plan.scales(K) == how
        assert w4_plan.way(180, 0, 90, 520, False) == w4_plan.way(180, 0, 90, 264, True) == ("streams", 0)
    assert w4_plan.way(1700, 0, 5, 40, False) == w4_plan.way(1700, 0, 5, 40, True) == ("tiles", 32)
    assert w4_plan.way(1700, 340, 5, 1032, False) == ("both", 32)
    assert w4_plan.way(sum(HEIGHTS), 0, 24, 4616, False) == ("tiles", 128)


@gpu
@pytest.mark.parametrize("case", [(*s[:3], K, *s[4:6]) for s in SIZES for K in s[3]],
                         ids=lambda c: f"{c[0]}-{c[3]}-{'silu' if c[5] else 'none'}".replace(" ", "_"))
def test_tiles(case):
    _, counts, capacity, K, N, silu = case
    check(counts, K, N, silu, capacity=capacity, seed=K, extra=0 if capacity else 7)


@gpu
@pytest.mark.parametrize("tile_rows,N", NARROW)
def test_narrow_outputs(tile_rows, N):
    """Waves past the last output, which bring token rows only."""
    for tail, K in ((20, 512), (60, 640), (90, 896)):
        check(narrow_counts(tile_rows, tail), K, N, False, seed=N)


@gpu
@pytest.mark.parametrize("K,how", LONG)
@pytest.mark.parametrize("silu", [False, True])
def test_whole_streams_of_long_rows(K, how, silu):
    """90 experts x 9 columns: more than 1.25 items for each of 512 blocks, so each
    wave takes whole items.  Every fifth expert is compared."""
    E, N = 90, 264 if silu else 520
    counts = [e % 3 + 1 for e in range(E)]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, (wc, ws) = inputs(int(off[-1]), K, 3), weights(E, (2 if silu else 1) * N, K, K)
    y = ep.ep_expert_linear_w4(x.to(DEV), torch.from_numpy(off).to(DEV), torch.from_numpy(wc).to(DEV),
                               torch.from_numpy(ws).to(DEV), epilogue="silu_mul" if silu else "none")
    got, x64 = y.double().cpu().numpy(), x.double().numpy()
    for e in [*range(0, E, 5), E - 1]:
        at = slice(int(off[e]), int(off[e + 1]))
        ref, size = plain64.expert_linear(x64[at], [(0, counts[e])], plain64.decode_w4(wc[e:e + 1], ws[e:e + 1]), silu)
        assert (np.abs(got[at] - ref) <= (K + 8) * 2.0 ** -23 * size + 2.0 ** -8 * 1.01 * np.abs(ref) + 2.0 ** -120).all()


def run(x, rows, codes, scales, silu=False, capacity=0):
    """y of 7s with a row before and after it that must stay 7."""
    n = x.shape[0]
    N = codes.shape[1] // (2 if silu else 1)
    room = torch.full((n + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_linear_w4(x, torch.tensor(rows, dtype=torch.int32, device=DEV), codes, scales, capacity=capacity,
                           epilogue="silu_mul" if silu else "none", out=room[1:n + 1])
    assert (room[0] == 7).all() and (room[n + 1] == 7).all()
    return room[1:n + 1]


@gpu
@pytest.mark.parametrize("silu", [False, True])
def test_nan_and_infinite_rows_stay_in_their_row(silu):
    """Beside others in a tile, as its last row (which rows that are not there
    repeat), and behind the last expert."""
    E, K, N = 5, 640, 40
    x, (wc, ws) = inputs(1700, K, 1), weights(E, (2 if silu else 1) * N, K, 4)
    codes, scales = torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
    off = [0, 340, 641, 1000, 1320, 1690]
    clean = run(x.to(DEV), off, codes, scales, silu)
    bad = {5: float("nan"), 640: float("nan"), 700: float("inf"), 1689: -float("inf")}
    for r, v in bad.items():
        x[r] = v
    x[1690:] = float("nan")
    y = run(x.to(DEV), off, codes, scales, silu)
    keep = torch.ones(1700, dtype=torch.bool, device=DEV)
    keep[list(bad)] = False
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[[5, 640]]).all() and not torch.isfinite(y[[700, 1689]]).any()


@gpu
def test_a_nan_scale_reaches_its_outputs_only():
    wc, ws = weights(5, 40, 640, 3)
    ws[1, 5, 3] = 255
    y = check(FULL, 640, 40, False, wc=wc, ws=ws)
    assert torch.isnan(y[340:680, 5]).all() and int(torch.isnan(y).sum()) == 340


@gpu
def test_offsets_out_of_order_or_range():
    """As the same rows by offsets in order: each expert takes what the ones before
    it have left, of the rows there are."""
    x, (wc, ws) = inputs(1700, 640, 3).to(DEV), weights(5, 40, 640, 4)
    codes, scales = torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
    top, low = 2 ** 31 - 1, -2 ** 31
    for m, same in (([0, 1020, 340, 1360, 680, 1700], [0, 1020, 1020, 1360, 1360, 1700]),
                    ([-7, 680, top, 0, 1700, 1700], [0, 680, 1700, 1700, 1700, 1700]),
                    ([1500, 1000, 700, 400, 200, 0], [0] * 6),
                    ([150, 150, 9000, 9000, 3, 2], [150, 150, 1700, 1700, 1700, 1700]),
                    ([low, top, 0, 40, 40, low], [0, 1700, 1700, 1700, 1700, 1700]),
                    ([0, 400, 800, 1200, 1600, 5000], [0, 400, 800, 1200, 1600, 1700])):
        assert torch.equal(run(x, m, codes, scales), run(x, same, codes, scales)), m
    wc, ws = weights(5, 1032, 640, 4)
    codes, scales = torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
    assert torch.equal(run(x, [-1, 341, top, low, 12], codes, scales, capacity=340),
                       run(x, [0, 340, 340, 0, 12], codes, scales, capacity=340))


@gpu
@pytest.mark.parametrize("K", [512, 640, 896])
def test_scales_at_any_word(K):
    """w_scales needs 4-byte alignment only, also where 16 bytes are loaded at once."""
    for counts, N in ((FULL, 40), (HEIGHTS, 4616)):
        E = len(counts)
        wc, ws = weights(E, N, K, 5)
        off = np.concatenate([[0], np.cumsum(counts)]).tolist()
        x, codes, scales = inputs(off[-1], K, 1).to(DEV), torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
        ref = run(x, off, codes, scales)
        for shift in (4, 8, 12):
            room = torch.full((ws.size + 12,), 255, dtype=torch.uint8, device=DEV)
            room[shift:shift + ws.size] = scales.view(-1)
            assert torch.equal(run(x, off, codes, room[shift:shift + ws.size].view(ws.shape)), ref)


@gpu
def test_captured_tiles_replay_with_other_offsets():
    """The launches are chosen by sizes alone, so a graph takes any offsets."""
    x, (wc, ws) = inputs(1700, 896, 3).to(DEV), weights(5, 40, 896, 4)
    codes, scales = torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
    rows, y = torch.tensor([0, 340, 680, 1020, 1360, 1700], dtype=torch.int32, device=DEV), torch.empty(1700, 40, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ep.ep_expert_linear_w4(x, rows, codes, scales, out=y)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_linear_w4(x, rows, codes, scales, out=y)
    for off in ([0, 1, 14, 14, 1000, 1700], [0, 0, 0, 0, 0, 1700], [0, 95, 97, 1500, 1513, 1514], [3, 3, 3, 3, 3, 3]):
        eager = run(x, off, codes, scales)
        y.fill_(7)
        rows.copy_(torch.tensor(off, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
