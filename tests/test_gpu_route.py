"""ep_route and ep_route_backward against the 64-bit forms of plain64.py.

Experts are compared exactly.  Weights: a unit u is 2^-24, half a step of fp32.
A score's exponent l - top is off by one unit of its size, its exp by 2 units
(one step), the sum of up to 64 terms a lane and 6 joins by at most 70, the
division and the scale by 2: with |l - top| <= span on both sides of the
division, (2 span + 80) u in all.  (The sum over all experts uses the hardware's
2^x, off by 2.5 units of l - top: 2.5 times the softmax's mean of |l - top|, which
is at most ln 2048 = 7.6, so 19 of the 70, of which the sum itself has 38.)
Gradients: the same for each share and
score, a few units for the products, so (4 span + 240) u of the sum of the
terms' magnitudes, then half a step of the logits' type.
"""
import math

import numpy as np
import pytest
import torch

import plain64
from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def make(T, E, dtype, seed, sigma=1.5):
    g = torch.Generator().manual_seed(seed)
    return (sigma * torch.randn(T, E, generator=g)).to(TYPES[dtype])


def span_of(l):
    f = l[np.isfinite(l)]
    return float(f.max() - f.min()) if f.size else 0.0


def check_route(l, k, sigmoid=False, bias=None, groups=1, topk_groups=1, group_top=2, renorm=True, scale=1.0):
    print("[route]", tuple(l.shape), l.dtype, k, sigmoid, bias is not None, groups, topk_groups, group_top, renorm, flush=True)
    got = ep.ep_route(l.to(DEV), k, score="sigmoid" if sigmoid else "softmax",
                      bias=None if bias is None else bias.to(DEV), num_groups=groups, topk_groups=topk_groups,
                      group_top=group_top, renormalize=renorm, scale=scale)
    l64 = l.double().numpy()
    idx, w = plain64.route(l64, k, sigmoid, None if bias is None else bias.numpy(), groups, topk_groups, group_top,
                           renorm, scale)
    np.testing.assert_array_equal(got["topk_idx"].cpu().numpy(), idx)
    gw = got["topk_weights"].cpu().numpy().astype(np.float64)
    span = min(span_of(l64), 200.0)         # past that a softmax term is 0 in both
    # Below the smallest normal number a step is 2^-149: a few of them.
    np.testing.assert_array_less(np.abs(gw - w), (2 * span + 80) * U * np.abs(w) + abs(scale) * 2.0 ** -140)
    return got


def check_backward(l, idx, g, sigmoid, renorm, scale):
    out = ep.ep_route_backward(l.to(DEV), idx.to(DEV), g.to(DEV), score="sigmoid" if sigmoid else "softmax",
                               renormalize=renorm, scale=scale)
    assert out.dtype == l.dtype and out.shape == l.shape
    l64 = l.double().numpy()
    d, size = plain64.route_backward(l64, idx.numpy(), g.numpy(), sigmoid, renorm, scale)
    got = out.double().cpu().numpy()
    span = min(span_of(l64), 200.0)
    info = torch.finfo(l.dtype)
    tol = (4 * span + 240) * U * size + info.eps / 2 * np.abs(d) * 1.01 + info.smallest_normal * info.eps + 2.0 ** -130
    bad = ~(np.abs(got - d) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], d[bad][:5])
    return out


SHAPES = [(1, 1, 1), (1, 256, 8), (3, 5, 5), (17, 60, 4), (64, 64, 6), (33, 100, 7), (70, 160, 16), (129, 256, 8),
          (20, 257, 9), (9, 384, 12), (12, 512, 17), (5, 1000, 33), (3, 2048, 64)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route_shapes(T, E, k, dtype):
    l = make(T, E, dtype, 100 * E + k)
    for sigmoid in (False, True):
        for renorm in (False, True):
            r = check_route(l, k, sigmoid, renorm=renorm, scale=2.5)
            g = torch.randn(T, k, generator=torch.Generator().manual_seed(E))
            check_backward(l, r["topk_idx"].cpu(), g, sigmoid, renorm, 2.5)
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(k))
    for sigmoid in (False, True):
        check_route(l, k, sigmoid, bias=b, renorm=True)
        check_route(l, k, sigmoid, bias=b, renorm=False)


@pytest.mark.parametrize("E,groups,topk_groups,k", [(256, 8, 4, 8), (64, 64, 3, 3), (64, 2, 1, 32), (160, 8, 3, 6),
                                                    (12, 4, 2, 5), (2048, 32, 5, 20), (60, 6, 6, 4), (7, 7, 7, 7)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_groups(E, groups, topk_groups, k, group_top):
    for sigmoid in (False, True):
        for dtype in ("fp32", "bf16"):
            l = make(21, E, dtype, E + k)
            check_route(l, k, sigmoid, groups=groups, topk_groups=topk_groups, group_top=group_top)
            b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(3))
            check_route(l, k, sigmoid, bias=b, groups=groups, topk_groups=topk_groups, group_top=group_top, renorm=False)


def test_route_ties_go_to_the_lowest_index():
    l = torch.zeros(5, 256)
    l[1, 7:] = 1.0
    l[2] = torch.arange(256) % 3
    l[3, ::2] = -0.0                          # equal to 0
    l[4] = torch.round(torch.randn(256, generator=torch.Generator().manual_seed(0)))
    for sigmoid in (False, True):
        for bias in (None, torch.zeros(256), torch.full((256,), 0.25)):
            for groups, tg in ((1, 1), (8, 4)):
                for gt in (1, 2):
                    check_route(l, 8, sigmoid, bias=bias, groups=groups, topk_groups=tg, group_top=gt)
    r = ep.ep_route(l[:1].to(DEV), 8)
    assert r["topk_idx"].tolist() == [list(range(8))]


def special():
    l = make(12, 64, "fp32", 5)
    inf, nan = math.inf, math.nan
    l[0] = -inf                               # a padding token
    l[1, :] = -inf
    l[1, 40] = 0.5                            # one expert left
    l[2, ::2] = -inf
    l[3, :61] = nan                           # masked places hold NaN
    l[4, 10] = inf
    l[5, [3, 9, 50]] = inf
    l[6] = nan
    l[7] = torch.finfo(torch.float32).min     # a mask of the type's lowest value
    l[7, [5, 6]] = 1.0
    l[8] = -150.0                             # sigmoid and shares far below fp32's range
    l[8, 4] = -140.0
    l[9] = 100.0
    l[10] = torch.finfo(torch.float32).max
    l[11, 20:] = -inf
    return l


@pytest.mark.parametrize("k", [1, 6, 64])
def test_route_empty_and_extreme_rows(k):
    l = special()
    b = 0.1 * torch.randn(64, generator=torch.Generator().manual_seed(3))
    b[11] = -math.inf
    b[12] = math.nan
    b[13] = math.inf
    for sigmoid in (False, True):
        for renorm in (False, True):
            for bias in (None, b):
                for groups, tg in ((1, 1), (4, 4)):
                    r = check_route(l, k, sigmoid, bias=bias, groups=groups, topk_groups=tg, renorm=renorm)
                    assert torch.isfinite(r["topk_weights"]).all()
                    assert (r["topk_idx"][0] == -1).all() and (r["topk_weights"][0] == 0).all()
                    if renorm:
                        sums = r["topk_weights"].double().sum(dim=1).cpu()
                        some = (r["topk_idx"] >= 0).any(dim=1).cpu()
                        # k shares of half a step each, and the sum they were divided by.
                        assert ((sums[some] - 1).abs() <= 160 * U).all()
                    g = torch.randn(12, k, generator=torch.Generator().manual_seed(k))
                    d = check_backward(l, r["topk_idx"].cpu(), g, sigmoid, renorm, 1.5)
                    assert torch.isfinite(d).all() and (d[0] == 0).all() and (d[6] == 0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_takes_any_ids(dtype, sigmoid, renorm):
    """Ids of the caller's own: twice the same, empty, out of range."""
    l = make(6, 40, dtype, 1)
    idx = torch.randint(0, 40, (6, 5), generator=torch.Generator().manual_seed(2))
    idx[0] = torch.tensor([3, 3, 3, 3, 3])
    idx[1] = torch.tensor([-1, 7, 7, 9, 40])
    idx[2] = -1
    idx[3, 2] = 2 ** 40
    idx[4, 0] = -2 ** 62
    check_backward(l, idx, torch.randn(6, 5, generator=torch.Generator().manual_seed(4)), sigmoid, renorm, 0.7)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E", [(5, 31), (4483, 31), (9000, 104), (40, 512)])
def test_one_renormalised_choice_has_no_gradient(T, E, sigmoid, dtype):
    """Its weight is the scale whatever the logits: a / a is 1 and g - g is 0, with
    no rounding in between."""
    l = (30 * make(T, E, dtype, 5).float()).to(TYPES[dtype]).to(DEV)
    score = "sigmoid" if sigmoid else "softmax"
    r = ep.ep_route(l, 1, score=score, renormalize=True, scale=2.5)
    assert (r["topk_weights"] == 2.5).all()
    g = torch.randn(T, 1, generator=torch.Generator().manual_seed(6)).to(DEV)
    assert (ep.ep_route_backward(l, r["topk_idx"], g, score=score, renormalize=True, scale=2.5) == 0).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(sigmoid, renorm):
    """Central differences of the 64-bit weights at the chosen ids.  With a step
    h the difference is off by h^2 / 6 times a third derivative (at most 6 times
    the scale for a softmax or a sigmoid, and a few slots add) and 2^-52 / h of
    rounding: h = 1e-4 gives 1e-7."""
    T, E, k, h = 2, 9, 4, 1e-4
    l = make(T, E, "fp32", 11)
    r = ep.ep_route(l.to(DEV), k, score="sigmoid" if sigmoid else "softmax", renormalize=renorm, scale=1.5)
    idx, g = r["topk_idx"].cpu().numpy(), np.random.default_rng(0).standard_normal((T, k)).astype(np.float32)

    def loss(v):
        total = 0.0
        for t in range(T):
            s = plain64.scores(v[t], sigmoid)[idx[t]]
            total += float((g[t] * 1.5 * (s / s.sum() if renorm else s)).sum())
        return total

    d = ep.ep_route_backward(l.to(DEV), r["topk_idx"], torch.from_numpy(g).to(DEV),
                             score="sigmoid" if sigmoid else "softmax", renormalize=renorm, scale=1.5).cpu().numpy()
    v = l.double().numpy()
    for t in range(T):
        for e in range(E):
            a, b = v.copy(), v.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - d[t, e]) <= 1e-6


def test_unaligned_logits_and_outputs_of_the_caller():
    """Logits that start at an odd element, outputs passed in, and a batch that
    ends inside a block: what lies behind the outputs stays."""
    for dtype in TYPES:
        for E in (60, 256):
            l = make(30, E, dtype, 2)
            room = torch.zeros(30 * E + 1, dtype=TYPES[dtype], device=DEV)
            room[1:] = l.to(DEV).view(-1)
            at = room[1:].view(30, E)
            r = ep.ep_route(l.to(DEV), 6, score="sigmoid")
            idx = torch.full((31, 6), 77, dtype=torch.int64, device=DEV)
            w = torch.full((31, 6), 77.0, device=DEV)
            ep.ep_route(at, 6, score="sigmoid", out=dict(topk_idx=idx[:30], topk_weights=w[:30]))
            assert torch.equal(idx[:30], r["topk_idx"]) and torch.equal(w[:30], r["topk_weights"])
            assert (idx[30] == 77).all() and (w[30] == 77).all()
            back = torch.full((30 * E + 2,), 7.0, dtype=TYPES[dtype], device=DEV)
            ep.ep_route_backward(at, idx[:30], w[:30], score="softmax", renormalize=False, out=back[1:-1].view(30, E))
            ref = ep.ep_route_backward(l.to(DEV), idx[:30], w[:30], score="softmax", renormalize=False)
            assert torch.equal(back[1:-1].view(30, E), ref) and back[0] == 7 and back[-1] == 7


def test_no_tokens():
    r = ep.ep_route(torch.empty(0, 16, device=DEV), 3)
    assert r["topk_idx"].shape == (0, 3) and r["topk_weights"].shape == (0, 3)
    d = ep.ep_route_backward(torch.empty(0, 16, device=DEV), r["topk_idx"], r["topk_weights"])
    assert d.shape == (0, 16)


def test_more_than_2_31_logits():
    """1,100,000 tokens of 2048 experts (2.25 G elements): the last tokens equal
    the same tokens in a batch of their own."""
    T, E, k = 1100000, 2048, 4
    l = torch.zeros(T, E, dtype=torch.float16, device=DEV)
    tail = make(40, E, "fp16", 9).to(DEV)
    l[-40:] = tail
    r, ref = ep.ep_route(l, k), ep.ep_route(tail, k)
    assert torch.equal(r["topk_idx"][-40:], ref["topk_idx"])
    assert torch.equal(r["topk_weights"][-40:], ref["topk_weights"])
    assert (r["topk_idx"][:-40] == torch.arange(k, device=DEV)).all()
    g = torch.zeros(T, k, device=DEV)
    g[-40:] = torch.randn(40, k, generator=torch.Generator().manual_seed(0)).to(DEV)
    d = ep.ep_route_backward(l, r["topk_idx"], g, renormalize=False)
    assert torch.equal(d[-40:], ep.ep_route_backward(tail, ref["topk_idx"], g[-40:].contiguous(), renormalize=False))
    assert not d[:-40].any()


def test_binding_refusals_on_the_device():
    l = torch.zeros(4, 8, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        ep.ep_route(torch.zeros(4, 16, device=DEV)[:, ::2], 2)
    with pytest.raises(ValueError, match="score must be"):
        ep.ep_route(l, 2, score="tanh")
    with pytest.raises(ValueError, match="bias must be"):
        ep.ep_route(l, 2, bias=torch.zeros(7, device=DEV))
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_route_backward(l, torch.zeros(4, 2, dtype=torch.int64, device=DEV), torch.zeros(4, 2))
    with pytest.raises(ep.EPError, match="num_topk exceeds"):
        ep.ep_route(l, 9)
    with pytest.raises(ep.EPError, match="num_topk < 1"):
        ep.ep_route(l, 0)
    with pytest.raises(ValueError, match="disagree on num_tokens"):
        ep.ep_route_backward(l, torch.zeros(3, 2, dtype=torch.int64, device=DEV), torch.zeros(3, 2, device=DEV))
    with pytest.raises(ValueError, match="shape of topk_idx"):
        ep.ep_route_backward(l, torch.zeros(4, 2, dtype=torch.int64, device=DEV), torch.zeros(4, 3, device=DEV))
