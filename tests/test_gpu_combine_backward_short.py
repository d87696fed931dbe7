"""ep_combine_backward on short rows (several slots a wave), with the bounds of
test_gpu_combine_backward.py: a lane adds 4 products to each of two sums (3
roundings, for a product of bf16 numbers is exact), joins them (1) and its slot's
lanes (at most 5): 9 of the 11 roundings that the bound allows."""
import pytest

from test_gpu_combine_backward import check, make

import torch

from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,k", [(1, 1), (3, 5), (33, 4), (130, 8), (9, 64)])
@pytest.mark.parametrize("H", [8, 64, 120, 128, 136, 248, 256, 264])
@pytest.mark.parametrize("weighted", [True, False])
def test_short_rows(T, k, H, weighted):
    g, y, row, w = make(T, H, k, T * k + 3, H + T)
    check(g, y, row, w if weighted else None)


@pytest.mark.parametrize("H", [40, 200])
def test_either_gradient_alone(H):
    g, y, row, w = make(20, H, 3, 70, H)
    both = check(g, y, row, w)
    gd, yd, rd, wd = g.to(DEV), y.to(DEV), row.to(DEV), w.to(DEV)
    r = ep.ep_combine_backward(gd, None, rd, wd, 70, out=dict(grad_expert_out=torch.full_like(yd, 7.0)))
    assert torch.equal(r["grad_expert_out"], both["grad_expert_out"])
    r = ep.ep_combine_backward(gd, yd, rd, wd, out=dict(grad_topk_weights=torch.empty_like(wd)))
    assert torch.equal(r["grad_topk_weights"], both["grad_topk_weights"])
