"""ep_moe_i8 over the range of magnitudes of what is between its products.

Every number is a small integer times a power of two, so that each step of the layer is
exact in fp32 and the results have to be equal to those worked out here:
x = 127 * 2^n in channel 0 and 2^n in channel 1: scale 2^n, codes 127 and 1;
gate = 2^g from g = 7 on, where 1 + exp(-gate) is 1 in fp32, so silu(gate) = gate;
h_i = u_i * 2^s with whole u_i up to 127 in magnitude, one of them 127: scale 2^s, codes
u_i (the quotient 127 h_i / max |h| is u_i to a few 2^-24 of it);
y = (sum of u_i * w_i) * 2^d, a whole number below 2^24 times a power of two.
"""
import numpy as np
import pytest
import torch

from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def layer(H, F, exponents, seed):
    """An expert for each s of `exponents`: max |h| = 127 * 2^s, and down scales that bring
    y back to whole numbers."""
    rng = np.random.default_rng([seed, H, F])
    E = len(exponents)
    u = rng.integers(-126, 127, (E, F))
    u[np.arange(E), rng.integers(0, F, E)] = rng.choice([-127, 127], E)
    up = np.zeros((E, 2 * F, H), np.int8)
    up[:, :F, 1], up[:, F:, 1] = 1, u
    s = np.array(exponents)
    g = np.where(s > 0, 40, 7)
    us = np.empty((E, 2 * F), np.float32)
    us[:, :F], us[:, F:] = np.exp2(g.astype(np.float64))[:, None], np.exp2((s - g).astype(np.float64))[:, None]
    down = rng.integers(-127, 128, (E, H, F)).astype(np.int8)
    return u, [up, us, down, np.exp2(-s.astype(np.float64))[:, None].repeat(H, 1).astype(np.float32)]


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().double().numpy()


def run(x, idx, weights, w):
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    return ep.ep_moe_i8(torch.from_numpy(x).bfloat16().to(DEV), to(idx), to(weights), *[to(a) for a in w]).double().cpu().numpy()


def tokens(T, H):
    x = np.zeros((T, H), np.float32)
    x[:, 0], x[:, 1] = 127, 1
    return x


# 127 * 2^s: from the least that has codes (2^-119 and more) to the last below 2^128, and
# on both sides of 2^126, above which a reciprocal is below the normal numbers.
EXPONENTS = [-125, -124, -100, -67, -60, -30, 0, 1, 30, 54, 60, 100, 118, 119, 120, 121]


@pytest.mark.parametrize("H,F", [(128, 128), (2048, 256), (4224, 128)])
def test_every_size_of_h(H, F):
    u, w = layer(H, F, EXPONENTS, 1)
    E = len(EXPONENTS)
    y = np.einsum("enf,ef->en", w[2].astype(np.int64), u)
    assert np.abs(y).max() < 1 << 24
    # each expert by itself, then pairs of a large and a small one
    got = run(tokens(E, H), np.arange(E)[:, None], np.ones((E, 1), np.float32), w)
    for e, s in enumerate(EXPONENTS):
        assert np.array_equal(got[e], bf16(y[e])), s
    pairs = np.stack([np.arange(E), np.arange(E)[::-1]], axis=1)
    got = run(tokens(E, H), pairs, np.tile(np.array([1, 0.5], np.float32), (E, 1)), w)
    assert np.array_equal(got, bf16(y[pairs[:, 0]] + 0.5 * y[pairs[:, 1]]))


def test_h_below_the_least_has_codes_of_zero():
    u, w = layer(128, 128, [-126, 0], 2)
    got = run(tokens(1, 128), np.array([[0, 1]]), np.ones((1, 2), np.float32), w)
    assert np.array_equal(got[0], bf16(w[2][1].astype(np.int64) @ u[1]))


def test_results_past_the_range_are_infinite():
    """h just fits fp32, y does not."""
    u, w = layer(256, 128, [121], 3)
    w[3][:] = 1
    y = (w[2][0].astype(np.int64) @ u[0]).astype(np.float64) * 2.0 ** 121
    with np.errstate(over="ignore"):
        want = bf16(y)
    assert np.isinf(want).sum() > 200
    assert np.array_equal(run(tokens(1, 256), np.zeros((1, 1), np.int64), np.ones((1, 1), np.float32), w)[0], want)


def test_h_past_the_range_is_nan():
    u, w = layer(256, 128, [122, 3], 4)
    got = run(tokens(3, 256), np.array([[0], [1], [0]]), np.ones((3, 1), np.float32), w)
    assert np.isnan(got[[0, 2]]).all() and np.array_equal(got[1], bf16(w[2][1].astype(np.int64) @ u[1]))
