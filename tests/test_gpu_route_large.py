"""ep_route and ep_route_backward on batches that take 16 lanes a token, checked
token by token on a sample (with the first and the last tokens) against
plain64.py, with the bounds of test_gpu_route.py, and against the same tokens
in small batches of 64 lanes a token."""
import numpy as np
import pytest
import torch

import plain64
from combine_get_dispatch_02_amd import ep
from test_gpu_route import DEV, TYPES, U, make, span_of

pytestmark = pytest.mark.gpu


def sample(T):
    rng = np.random.default_rng(T)
    return np.unique(np.concatenate([np.arange(9), T - 1 - np.arange(9), rng.integers(0, T, 150)]))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E,k", [(2049, 64, 6), (2500, 50, 16), (2051, 128, 8), (3001, 100, 3), (4099, 256, 8),
                                   (4100, 200, 16), (4097, 512, 8), (4099, 300, 5), (4101, 257, 7), (2048, 5, 2)])
def test_sampled_tokens(T, E, k, dtype):
    l = make(T, E, dtype, T + E)
    l[7] = -torch.inf
    l[T - 2, : E // 2] = float("nan")
    ld, at = l.to(DEV), sample(T)
    l64 = l.double().numpy()[at]
    span = min(span_of(l64), 200.0)
    g = torch.Generator().manual_seed(1)
    b = 0.1 * torch.randn(E, generator=g)
    for sigmoid in (False, True):
        for renorm in (False, True):
            for bias in (None, b):
                r = ep.ep_route(ld, k, score="sigmoid" if sigmoid else "softmax", renormalize=renorm, scale=2.0,
                                bias=None if bias is None else bias.to(DEV))
                idx, w = plain64.route(l64, k, sigmoid, None if bias is None else bias.numpy(), 1, 1, 2, renorm, 2.0)
                np.testing.assert_array_equal(r["topk_idx"].cpu().numpy()[at], idx)
                gw = r["topk_weights"].double().cpu().numpy()[at]
                assert (np.abs(gw - w) <= (2 * span + 80) * U * np.abs(w) + 2.0 ** -140).all()
                for t0 in (0, T - 700):
                    part = ep.ep_route(ld[t0:t0 + 700].contiguous(), k, score="sigmoid" if sigmoid else "softmax",
                                       renormalize=renorm, scale=2.0, bias=None if bias is None else bias.to(DEV))
                    assert torch.equal(part["topk_idx"], r["topk_idx"][t0:t0 + 700])


@pytest.mark.parametrize("E,groups,topk_groups,k", [(256, 8, 4, 8), (128, 4, 1, 8), (64, 16, 5, 6), (160, 8, 3, 6), (256, 64, 9, 12),
                                                    (96, 3, 2, 16), (32, 2, 1, 4), (512, 8, 4, 8), (512, 4, 2, 12)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups(E, groups, topk_groups, k, group_top):
    T = 4100
    l = make(T, E, "fp32", E + groups)
    l[5] = torch.round(l[5])                        # ties
    l[6, : E // groups] = -torch.inf                # a group without experts
    at, b = sample(T), 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(2))
    for sigmoid in (False, True):
        for bias in (None, b):
            r = ep.ep_route(l.to(DEV), k, score="sigmoid" if sigmoid else "softmax", num_groups=groups,
                            topk_groups=topk_groups, group_top=group_top, bias=None if bias is None else bias.to(DEV))
            idx, w = plain64.route(l.double().numpy()[at], k, sigmoid, None if bias is None else bias.numpy(), groups,
                                   topk_groups, group_top, True, 1.0)
            np.testing.assert_array_equal(r["topk_idx"].cpu().numpy()[at], idx)
            assert (np.abs(r["topk_weights"].double().cpu().numpy()[at] - w) <= 110 * U * np.abs(w) + 2.0 ** -140).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E,k", [(6145, 64, 6), (6144, 27, 13), (7001, 128, 16), (12289, 256, 8), (12300, 190, 5)])
def test_gradient_of_sampled_tokens(T, E, k, dtype):
    l = make(T, E, dtype, T)
    l[3] = -torch.inf
    gen = torch.Generator().manual_seed(3)
    idx = torch.randint(-1, E, (T, k), generator=gen)           # empty slots, and ids more than once
    g = torch.randn(T, k, generator=gen)
    at, info = sample(T), torch.finfo(TYPES[dtype])
    l64 = l.double().numpy()[at]
    span = min(span_of(l64), 200.0)
    for sigmoid in (False, True):
        for renorm in (False, True):
            out = ep.ep_route_backward(l.to(DEV), idx.to(DEV), g.to(DEV), score="sigmoid" if sigmoid else "softmax",
                                       renormalize=renorm, scale=1.5)
            d, size = plain64.route_backward(l64, idx.numpy()[at], g.numpy()[at], sigmoid, renorm, 1.5)
            got = out.double().cpu().numpy()[at]
            tol = (4 * span + 240) * U * size + info.eps / 2 * np.abs(d) * 1.01 + info.smallest_normal * info.eps + 2.0 ** -130
            assert (np.abs(got - d) <= tol).all()
            part = ep.ep_route_backward(l[-500:].to(DEV), idx[-500:].to(DEV), g[-500:].to(DEV),
                                        score="sigmoid" if sigmoid else "softmax", renormalize=renorm, scale=1.5)
            # Another order of the sums: a few units, and a step where they straddle a rounding.
            assert torch.allclose(part.float(), out[-500:].float(), rtol=2 * info.eps, atol=1e-6)


def test_rows_behind_the_last_token_stay():
    T, E, k = 4098, 256, 8
    l = make(T, E, "fp32", 0).to(DEV)
    idx = torch.full((T + 3, k), 77, dtype=torch.int64, device=DEV)
    w = torch.full((T + 3, k), 77.0, device=DEV)
    ep.ep_route(l, k, out=dict(topk_idx=idx[:T], topk_weights=w[:T]))
    assert (idx[T:] == 77).all() and (w[T:] == 77).all() and (idx[:T] < E).all()
    back = torch.full((13003, 64), 7.0, device=DEV)
    i2 = torch.zeros(13000, 2, dtype=torch.int64, device=DEV)
    ep.ep_route_backward(torch.randn(13000, 64, device=DEV), i2, torch.ones(13000, 2, device=DEV), out=back[:13000])
    assert (back[13000:] == 7).all()
