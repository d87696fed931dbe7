"""ep_expert_linear_w4 against the 64-bit form of plain64.py.

Products of a code, its scale and a bf16 input are exact in fp32.  K of them are
added in some order, each addition off by at most a whole step (2^-23) of the
magnitudes' sum, which bounds the accumulator; silu and the product add a few
steps (8 here), and the result is rounded to bf16, half a step (2^-8).
"""
import numpy as np
import pytest
import torch

import plain64
from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def weights(E, W, K, seed, lo=118, hi=124):
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (E, W, K // 2), dtype=np.uint8),
            rng.integers(lo, hi, (E, W, K // 32), dtype=np.uint8))


def inputs(rows, K, seed):
    rng = np.random.default_rng([seed, 1])
    return torch.from_numpy(rng.standard_normal((rows, K), dtype=np.float32)).bfloat16()


def check(counts, K, N, silu, capacity=0, seed=0, extra=0, x=None, wc=None, ws=None):
    """counts: rows of each expert; extra: rows behind the last expert's."""
    E = len(counts)
    print("[w4]", counts if E < 12 else (E, max(counts)), K, N, silu, capacity, flush=True)
    if capacity:
        spans = [(e * capacity, c) for e, c in enumerate(counts)]
        rows, m = E * capacity, np.array(counts, np.int32)
    else:
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        spans, rows, m = [(int(off[e]), counts[e]) for e in range(E)], int(off[-1]) + extra, off
    if x is None:
        x = inputs(rows, K, seed)
    if wc is None:
        wc, ws = weights(E, (2 if silu else 1) * N, K, seed)
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_linear_w4(x.to(DEV), torch.from_numpy(m).to(DEV), torch.from_numpy(wc).to(DEV),
                           torch.from_numpy(ws).to(DEV), capacity=capacity, epilogue="silu_mul" if silu else "none", out=y)
    ref, size = plain64.expert_linear(x.double().numpy(), spans, plain64.decode_w4(wc, ws), silu)
    got = y.double().cpu().numpy()
    none = np.ones(rows, bool)
    for first, count in spans:
        none[first:first + count] = False
    assert (got[none] == 7).all(), "rows of no expert were written"
    got, ref, size = got[~none], ref[~none], size[~none]
    tol = (K + 8) * 2.0 ** -23 * size + 2.0 ** -8 * 1.01 * np.abs(ref) + 2.0 ** -120
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    return y


COUNTS = [[1], [0, 1, 0], [1, 0, 2, 16], [17, 15, 33, 0, 1], [64, 5, 130], [300], [3] * 40, [200, 90, 129]]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
def test_packed_rows(counts, silu):
    check(counts, 256, 72, silu, seed=len(counts))
    check(counts, 128, 200, silu, seed=len(counts), extra=5)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K,N", [(128, 8), (128, 16), (384, 64), (640, 24), (512, 136), (1024, 264), (2048, 96), (1152, 520)])
def test_sizes(K, N, silu):
    check([5, 0, 1, 40], K, N, silu, seed=K)
    check([140, 1], K, N, silu, seed=K)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("capacity,counts", [(1, [1, 0, 1]), (20, [20, 0, 3, 17]), (150, [150, 149, 0, 2]), (7, [7] * 30)])
def test_padded_rows(capacity, counts, silu):
    check(counts, 384, 104, silu, capacity=capacity, seed=capacity)


def test_every_code_and_scale():
    """Each code at each scale that keeps code * scale in bf16's range, picked
    out by an input that is 1 in one place: the output is the weight itself."""
    K, N = 128, 256
    scales = np.arange(0, 256, dtype=np.uint8)                     # one scale per output
    wc = np.zeros((1, N, K // 2), np.uint8)
    for i in range(K):
        wc[0, :, i // 2] |= np.uint8((i % 16) << (4 * (i % 2)))
    ws = np.repeat(scales[None, :, None], K // 32, axis=2)
    x = torch.eye(K).bfloat16()
    y = ep.ep_expert_linear_w4(x.to(DEV), torch.tensor([0, K], dtype=torch.int32, device=DEV),
                               torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV))
    ref = plain64.decode_w4(wc, ws)[0].T                           # [K, N]
    got = y.double().cpu().numpy()
    # From scale 2^126 on the code 4 is 2^128, past the largest bf16 (and fp32)
    # number, 2^128 - 2^120: it is infinite, and infinity times the inputs that
    # are 0 is NaN.  Up to 2^125 the largest weight is 6 * 2^125 = 1.5 * 2^127.
    assert np.array_equal(got[:, :253], ref[:, :253])
    assert np.isnan(got[:, 255]).all()


def test_a_nan_scale_reaches_its_outputs_only():
    wc, ws = weights(2, 48, 256, 3)
    ws[1, 5, 3] = 255
    y = check([3, 4], 256, 48, False, wc=wc, ws=ws)
    assert torch.isnan(y[3:, 5]).all() and int(torch.isnan(y).sum()) == 4


def test_nan_rows_stay_in_their_row():
    """A NaN or infinite input, in a row of a tile or behind the last row."""
    x = inputs(20, 256, 1)
    x[4] = float("nan")
    x[17:] = float("nan")                                          # rows of no expert
    wc, ws = weights(2, 32, 256, 4)
    y = torch.full((20, 32), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_linear_w4(x.to(DEV), torch.tensor([0, 9, 17], dtype=torch.int32, device=DEV),
                           torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV), out=y)
    assert torch.isnan(y[4]).all() and int(torch.isnan(y).sum()) == 32 and (y[17:] == 7).all()


def test_bad_maps_stay_inside_the_buffers():
    """Offsets and counts out of range are limited to the rows given."""
    x, (wc, ws) = inputs(40, 128, 2).to(DEV), weights(4, 16, 128, 5)
    wc, ws = torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
    room = torch.full((42, 16), 7.0, dtype=torch.bfloat16, device=DEV)
    for m in ([-5, 10, 20, 30, 1000], [0, 50, 60, 70, 80], [-2 ** 31, 2 ** 31 - 1, 0, 40, 40], [0, 0, 0, 0, 0],
              [40, 30, 20, 10, 0]):
        ep.ep_expert_linear_w4(x, torch.tensor(m, dtype=torch.int32, device=DEV), wc, ws, out=room[1:41])
        assert (room[0] == 7).all() and (room[41] == 7).all()
    for m in ([-1, 11, 2 ** 31 - 1, -2 ** 31], [10, 10, 10, 10]):
        ep.ep_expert_linear_w4(x, torch.tensor(m, dtype=torch.int32, device=DEV), wc, ws, capacity=10, out=room[1:41])
        assert (room[0] == 7).all() and (room[41] == 7).all()
    full = ep.ep_expert_linear_w4(x, torch.tensor([10] * 4, dtype=torch.int32, device=DEV), wc, ws, capacity=10)
    over = ep.ep_expert_linear_w4(x, torch.tensor([99] * 4, dtype=torch.int32, device=DEV), wc, ws, capacity=10)
    assert torch.equal(full, over)


def test_the_same_row_anywhere():
    """A row's result does not depend on its neighbours or its place, within one
    launch shape."""
    wc, ws = weights(1, 64, 512, 6)
    wc, ws = torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
    x = inputs(1, 512, 3).expand(200, 512).contiguous().to(DEV)
    y = ep.ep_expert_linear_w4(x, torch.tensor([0, 200], dtype=torch.int32, device=DEV), wc, ws)
    assert torch.equal(y, y[:1].expand_as(y))


def test_many_experts_and_a_skewed_batch():
    counts = [0] * 2048
    for e in (0, 3, 700, 701, 2047):
        counts[e] = e % 37 + 1
    check(counts, 128, 8, False)
    rng = np.random.default_rng(0)
    check([int(v) for v in 400 / np.arange(1, 65) ** 1.2] + [int(rng.integers(0, 3)) for _ in range(64)], 256, 136, True)


def test_offsets_past_32_bits():
    """Weights (4.8 GB of codes), rows of x and rows of y past 2^32."""
    E, N, K = 330, 4096, 7168
    wc = torch.zeros(E, N, K // 2, dtype=torch.uint8, device=DEV)
    ws = torch.full((E, N, K // 32), 120, dtype=torch.uint8, device=DEV)
    c, s = weights(1, N, K, 7)
    wc[-1], ws[-1] = torch.from_numpy(c[0]).to(DEV), torch.from_numpy(s[0]).to(DEV)
    x = inputs(6, K, 8).to(DEV)
    one = ep.ep_expert_linear_w4(x, torch.tensor([0, 6], dtype=torch.int32, device=DEV), wc[-1:], ws[-1:])
    rows = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    rows[-1] = 6
    assert torch.equal(ep.ep_expert_linear_w4(x, rows, wc, ws), one)
    del wc, ws
    cap, K, N = 300000, 8192, 8192
    x = torch.empty(2, cap, K, dtype=torch.bfloat16, device=DEV)
    x[1, :5] = inputs(5, K, 9).to(DEV)
    c, s = weights(2, N, K, 10)
    c, s = torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV)
    y = ep.ep_expert_linear_w4(x, torch.tensor([0, 5], dtype=torch.int32, device=DEV), c, s, capacity=cap)
    one = ep.ep_expert_linear_w4(x[1, :5].contiguous(), torch.tensor([0, 5], dtype=torch.int32, device=DEV), c[1:], s[1:])
    # Both add the same products, perhaps in another order.
    a, b = y[1, :5].double(), one.double()
    size = (x[1, :5].double().abs() @ torch.from_numpy(np.abs(plain64.decode_w4(c[1].cpu().numpy(), s[1].cpu().numpy()))).to(DEV).t())
    assert ((a - b).abs() <= 2 * K * 2.0 ** -23 * size + 2.0 ** -7 * b.abs()).all()


def test_refusals():
    x, (wc, ws) = inputs(4, 128, 2).to(DEV), weights(2, 16, 128, 5)
    wc, ws = torch.from_numpy(wc).to(DEV), torch.from_numpy(ws).to(DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="epilogue must be"):
        ep.ep_expert_linear_w4(x, off, wc, ws, epilogue="relu")
    with pytest.raises(ValueError, match="recv_expert_offset"):
        ep.ep_expert_linear_w4(x, off[:2], wc, ws)
    with pytest.raises(ValueError, match="recv_count"):
        ep.ep_expert_linear_w4(x, off, wc, ws, capacity=2)
    with pytest.raises(ValueError, match="w_scales"):
        ep.ep_expert_linear_w4(x, off, wc, ws[:, :, :3].contiguous())
    with pytest.raises(ValueError, match="even number"):
        ep.ep_expert_linear_w4(x, off, wc[:, :15].contiguous(), ws[:, :15].contiguous(), epilogue="silu_mul")
    with pytest.raises(ep.EPError, match="out_features must be"):
        ep.ep_expert_linear_w4(x, off, wc[:, :12].contiguous(), ws[:, :12].contiguous())
    with pytest.raises(ep.EPError, match="in_features must be"):
        ep.ep_expert_linear_w4(x[:, :64].contiguous(), off, wc[:, :, :32].contiguous(), ws[:, :, :2].contiguous())
    with pytest.raises(ep.EPError, match="num_experts \\* capacity"):
        ep.ep_expert_linear_w4(x, off[:2].contiguous(), wc, ws, capacity=3)
    with pytest.raises(ValueError, match="needs"):
        ep.ep_expert_linear_w4(x, off, wc, ws, out=torch.empty(3, 16, dtype=torch.bfloat16, device=DEV))
    e = ep.ep_expert_linear_w4(x[:0], off * 0, wc, ws)
    assert e.shape == (0, 16)
