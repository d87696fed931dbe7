"""ep_route with experts masked through the logits and through the bias.  A bias of
-inf or NaN keeps an expert from being chosen; its score still counts in a softmax
that is not renormalised, as ep_route_backward (which knows no bias) has it.  A
masked logit has no score.  Bounds as in test_gpu_route.py."""
import math

import numpy as np
import pytest
import torch

from combine_get_dispatch_02_amd import ep
from test_gpu_route import DEV, U, check_backward, make, span_of

pytestmark = pytest.mark.gpu


def exact(l, chosen):
    """Softmax over every logit in 64 bits, at the chosen experts."""
    p = torch.softmax(l.double(), dim=1)
    return p.gather(1, chosen.cpu()).numpy()


# 64 lanes a token, and 16.
@pytest.mark.parametrize("T,E", [(33, 60), (40, 256), (2100, 64), (4200, 256)])
@pytest.mark.parametrize("value", [-math.inf, math.nan])
@pytest.mark.parametrize("groups", [1, 4])
def test_bias_masks_the_choice_only(T, E, value, groups):
    # Whole 64ths: different logits give different scores, whatever their sum.
    k, l = 5, torch.round(make(T, E, "fp32", T) * 64) / 64
    masked = torch.rand(E, generator=torch.Generator().manual_seed(E)) < 0.4
    bias = torch.where(masked, value, 0.0)
    tol = (2 * span_of(l.double().numpy()) + 80) * U
    r = ep.ep_route(l.to(DEV), k, bias=bias.to(DEV), num_groups=groups, topk_groups=groups, renormalize=False)
    idx = r["topk_idx"].cpu()
    assert not masked[idx].any()
    ref = exact(l, idx)
    assert (np.abs(r["topk_weights"].double().cpu().numpy() - ref) <= tol * ref).all()
    # The gradient of the same weights: every logit has one, the masked ones too.
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    d = check_backward(l, idx, g, False, False, 1.0)
    assert (d[:, masked.to(DEV)] != 0).any()
    # Masked logits instead: the same choice, of a softmax over the others.
    other = torch.where(masked, value, l)
    m = ep.ep_route(other.to(DEV), k, bias=torch.zeros(E, device=DEV), num_groups=groups, topk_groups=groups, renormalize=False)
    assert torch.equal(m["topk_idx"], r["topk_idx"])
    ref = exact(torch.where(masked, -math.inf, l), idx)
    assert (np.abs(m["topk_weights"].double().cpu().numpy() - ref) <= tol * ref).all()
    d = check_backward(other, idx, g, False, False, 1.0)
    assert (d[:, masked.to(DEV)] == 0).all()
    # Renormalised over the chosen ones there is no difference but of roundings.
    a = ep.ep_route(l.to(DEV), k, bias=bias.to(DEV), num_groups=groups, topk_groups=groups)["topk_weights"].double()
    b = ep.ep_route(other.to(DEV), k, num_groups=groups, topk_groups=groups, group_top=1)["topk_weights"].double()
    assert ((a - b).abs() <= 2 * tol * b).all()
