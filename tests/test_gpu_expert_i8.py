"""ep_expert_linear_i8 against the 64-bit form of plain64_i8.py, whose bounds (sums are
exact) leave the rounding of the result to bf16, half a step: 2^-8."""
import numpy as np
import pytest
import torch

import plain64_i8 as plain
from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(a):
    return torch.from_numpy(a).to(DEV)


def matrix(E, W, K, seed):
    rng = np.random.default_rng([seed, W, K])
    return rng.integers(-128, 128, (E, W, K), dtype=np.int8), (rng.random((E, W), dtype=np.float32) + 0.5) / (74 * K ** 0.5)


def rows_of(rows, K, seed):
    rng = np.random.default_rng([seed, rows, 1])
    return rng.integers(-128, 128, (rows, K), dtype=np.int8), (rng.random(rows, dtype=np.float32) + 0.5) / 74


def check(counts, K, N, silu, capacity=0, seed=0, extra=0, x=None, xs=None, w=None, ws=None):
    """counts: rows of each expert; extra: rows behind the last expert's."""
    E = len(counts)
    print("[i8]", counts if E < 12 else (E, max(counts)), K, N, silu, capacity, flush=True)
    if capacity:
        spans = [(e * capacity, c) for e, c in enumerate(counts)]
        rows, m = E * capacity, np.array(counts, np.int32)
    else:
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        spans, rows, m = [(int(off[e]), counts[e]) for e in range(E)], int(off[-1]) + extra, off
    if x is None:
        x, xs = rows_of(rows, K, seed)
    if w is None:
        w, ws = matrix(E, (2 if silu else 1) * N, K, seed)
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_linear_i8(dev(x), dev(xs), dev(m), dev(w), dev(ws), capacity=capacity, epilogue="silu_mul" if silu else "none", out=y)
    ref, tol = plain.linear(x, xs, spans, w, ws, silu)
    got = y.double().cpu().numpy()
    none = np.ones(rows, bool)
    for first, count in spans:
        none[first:first + count] = False
    assert (got[none] == 7).all(), "rows of no expert were written"
    got, ref, tol = got[~none], ref[~none], tol[~none]
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    bad = np.abs(got - ref) > tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -130
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    return y


COUNTS = [[1], [0, 1, 0], [1, 0, 2, 16], [17, 15, 33, 0, 1], [64, 65, 5, 130], [300], [3] * 40, [200, 90, 129], [256, 257, 128]]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
def test_packed_rows(counts, silu):
    check(counts, 256, 72, silu, seed=len(counts))
    check(counts, 128, 200, silu, seed=len(counts), extra=5)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K,N", [(128, 8), (128, 16), (384, 64), (640, 24), (512, 136), (1024, 264), (2048, 96), (1152, 520), (7168, 40)])
def test_sizes(K, N, silu):
    check([5, 0, 1, 40], K, N, silu, seed=K)
    check([140, 1], K, N, silu, seed=K)
    check([70, 260], K, N, silu, seed=K)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("capacity,counts", [(1, [1, 0, 1]), (20, [20, 0, 3, 17]), (150, [150, 149, 0, 2]), (7, [7] * 30), (300, [300, 0, 16, 17])])
def test_padded_rows(capacity, counts, silu):
    check(counts, 384, 104, silu, capacity=capacity, seed=capacity)


@pytest.mark.parametrize("counts", [[3], [400]])
def test_largest_sums(counts):
    """Every code -128: sums of 2^14 K, 2^30 at the largest K."""
    K = 1 << 16
    x, w = np.full((counts[0], K), -128, np.int8), np.full((1, 16, K), -128, np.int8)
    w[0, 1] = 127
    y = check(counts, K, 16, False, x=x, xs=np.full(counts[0], 0.5, np.float32), w=w, ws=np.full((1, 16), 2.0 ** -20, np.float32))
    assert (y[:, 0].double() == 2.0 ** 30 * 2.0 ** -21).all()


@pytest.mark.parametrize("rows", [9, 40, 200])
def test_one_code_at_a_time(rows):
    """Inputs that are 1 in one place: the output is the weight there, so that no input
    is met by another's weight."""
    K, N = 256, 64
    rng = np.random.default_rng(3)
    w = rng.integers(-128, 128, (1, N, K), dtype=np.int8)
    for at in range(0, K, rows):
        x = np.zeros((rows, K), np.int8)
        x[np.arange(rows), (at + np.arange(rows)) % K] = 1
        y = ep.ep_expert_linear_i8(dev(x), torch.ones(rows, device=DEV), dev(np.array([0, rows], np.int32)), dev(w),
                                   torch.ones(1, N, device=DEV))
        assert np.array_equal(y.double().cpu().numpy(), w[0].T[(at + np.arange(rows)) % K].astype(np.float64))


@pytest.mark.parametrize("counts", [[3, 4], [40, 170]])
def test_nan_scales_stay_where_they_are(counts):
    x, xs = rows_of(sum(counts), 256, 3)
    w, ws = matrix(2, 48, 256, 3)
    xs[1], xs[2], ws[1, 5] = np.nan, np.inf, np.nan
    y = ep.ep_expert_linear_i8(dev(x), dev(xs), dev(np.cumsum([0] + counts).astype(np.int32)), dev(w), dev(ws)).cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1:3] = True
    want[counts[0]:, 5] = True
    assert torch.equal(bad, want)


def test_bad_maps_stay_inside_the_buffers():
    """Offsets and counts out of range are limited to the rows given."""
    (x, xs), (w, ws) = rows_of(40, 128, 2), matrix(4, 16, 128, 5)
    x, xs, w, ws = dev(x), dev(xs), dev(w), dev(ws)
    room = torch.full((42, 16), 7.0, dtype=torch.bfloat16, device=DEV)
    for m in ([-5, 10, 20, 30, 1000], [0, 50, 60, 70, 80], [-2 ** 31, 2 ** 31 - 1, 0, 40, 40], [0, 0, 0, 0, 0],
              [40, 30, 20, 10, 0]):
        ep.ep_expert_linear_i8(x, xs, torch.tensor(m, dtype=torch.int32, device=DEV), w, ws, out=room[1:41])
        assert (room[0] == 7).all() and (room[41] == 7).all()
    for m in ([-1, 11, 2 ** 31 - 1, -2 ** 31], [10, 10, 10, 10]):
        ep.ep_expert_linear_i8(x, xs, torch.tensor(m, dtype=torch.int32, device=DEV), w, ws, capacity=10, out=room[1:41])
        assert (room[0] == 7).all() and (room[41] == 7).all()
    full = ep.ep_expert_linear_i8(x, xs, torch.tensor([10] * 4, dtype=torch.int32, device=DEV), w, ws, capacity=10)
    over = ep.ep_expert_linear_i8(x, xs, torch.tensor([99] * 4, dtype=torch.int32, device=DEV), w, ws, capacity=10)
    assert torch.equal(full, over)


@pytest.mark.parametrize("K,N", [(512, 64), (1024, 520)])
def test_a_row_s_result_is_the_same_anywhere(K, N):
    """Sums are exact, so neither a row's neighbours nor the way its expert's size takes
    change its result."""
    w, ws = matrix(1, N, K, 6)
    x, xs = rows_of(1, K, 3)
    want = None
    for rows in (1, 13, 17, 40, 70, 200, 300, 600):
        y = ep.ep_expert_linear_i8(dev(np.repeat(x, rows, 0)), dev(np.repeat(xs, rows)), dev(np.array([0, rows], np.int32)), dev(w), dev(ws))
        want = y[:1] if want is None else want
        assert torch.equal(y, want.expand_as(y))


def test_many_experts_and_a_skewed_batch():
    counts = [0] * 2048
    for e in (0, 3, 700, 701, 2047):
        counts[e] = e % 37 + 1
    check(counts, 128, 8, False)
    rng = np.random.default_rng(0)
    check([int(v) for v in 400 / np.arange(1, 65) ** 1.2] + [int(rng.integers(0, 3)) for _ in range(64)], 256, 136, True)


def test_offsets_past_32_bits():
    """Weights (5.4 GB), rows of x and rows of y past 2^32."""
    E, N, K = 330, 2304, 7168
    w = torch.zeros(E, N, K, dtype=torch.int8, device=DEV)
    ws = torch.ones(E, N, device=DEV)
    c, s = matrix(1, N, K, 7)
    w[-1], ws[-1] = dev(c[0]), dev(s[0])
    for n in (6, 300):
        x, xs = rows_of(n, K, 8)
        x, xs = dev(x), dev(xs)
        one = ep.ep_expert_linear_i8(x, xs, torch.tensor([0, n], dtype=torch.int32, device=DEV), w[-1:], ws[-1:])
        rows = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        rows[-1] = n
        assert torch.equal(ep.ep_expert_linear_i8(x, xs, rows, w, ws), one)
    del w, ws
    cap, K, N = 600000, 8192, 8192
    x = torch.empty(2, cap, K, dtype=torch.int8, device=DEV)
    xs = torch.empty(2, cap, device=DEV)
    c, s = matrix(2, N, K, 10)
    c, s = dev(c), dev(s)
    y = torch.empty(2, cap, N, dtype=torch.bfloat16, device=DEV)
    for n in (5, 90):
        a, b = rows_of(n, K, 9)
        x[1, :n], xs[1, :n] = dev(a), dev(b)
        ep.ep_expert_linear_i8(x, xs, torch.tensor([0, n], dtype=torch.int32, device=DEV), c, s, capacity=cap, out=y)
        one = ep.ep_expert_linear_i8(dev(a), dev(b), torch.tensor([0, n], dtype=torch.int32, device=DEV), c[1:].contiguous(), s[1:].contiguous())
        assert torch.equal(y[1, :n], one)


def test_no_rows():
    w, ws = matrix(2, 16, 128, 5)
    e = ep.ep_expert_linear_i8(torch.zeros(0, 128, dtype=torch.int8, device=DEV), torch.zeros(0, device=DEV),
                               torch.zeros(3, dtype=torch.int32, device=DEV), dev(w), dev(ws))
    assert e.shape == (0, 16)
