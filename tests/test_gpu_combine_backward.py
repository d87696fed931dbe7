"""ep_combine_backward against the 64-bit form of plain64.py.

dy = bf16(w g): the product rounded to fp32 and then to bf16, half a step each.
dw: a lane adds ceil(H / 512) products to each of eight sums, then 3 joins and
6 across the wave, each off by at most 2^-24 of the sum of the magnitudes.
"""
import numpy as np
import pytest
import torch

import plain64
from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(T, H, k, rows, seed, empty=0.1):
    rng = np.random.default_rng(seed)
    g = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).bfloat16()
    y = torch.from_numpy(rng.standard_normal((rows, H), dtype=np.float32)).bfloat16()
    w = torch.from_numpy(rng.standard_normal((T, k), dtype=np.float32))
    row = np.full(T * k, -1, np.int32)
    n = min(T * k, rows)
    at = rng.permutation(T * k)[:n]
    row[at] = rng.permutation(rows)[:n]
    row[rng.random(T * k) < empty] = -1
    return g, y, torch.from_numpy(row.reshape(T, k)), w


def check(g, y, row, w, **kw):
    print("[combine_backward]", tuple(g.shape), tuple(row.shape), tuple(y.shape), flush=True)
    H = g.shape[1]
    out = dict(grad_expert_out=torch.full(y.shape, 7.0, dtype=torch.bfloat16, device=DEV),
               grad_topk_weights=torch.full(row.shape, 7.0, device=DEV))
    ep.ep_combine_backward(g.to(DEV), y.to(DEV), row.to(DEV), None if w is None else w.to(DEV), out=out, **kw)
    dy, dw, size = plain64.combine_backward(g.double().numpy(), y.double().numpy(), row.numpy(),
                                            None if w is None else w.numpy())
    got = out["grad_expert_out"].double().cpu().numpy()
    none = np.isnan(dy)
    assert (got[none] == 7).all()
    assert (np.abs(got - dy)[~none] <= (2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(dy) + 2.0 ** -130)[~none]).all()
    gw = out["grad_topk_weights"].double().cpu().numpy()
    assert (gw[row.numpy() < 0] == 0).all()
    assert (np.abs(gw - dw) <= (-(-H // 512) + 10) * 2.0 ** -24 * size).all()
    return out


@pytest.mark.parametrize("T,H,k,rows", [(1, 8, 1, 1), (1, 7168, 8, 8), (3, 512, 2, 9), (17, 520, 5, 100), (40, 1000, 6, 200),
                                        (33, 4096, 8, 264), (9, 64, 64, 576), (5, 16, 3, 0), (7, 2056, 1, 5)])
@pytest.mark.parametrize("weighted", [True, False])
def test_shapes(T, H, k, rows, weighted):
    g, y, row, w = make(T, H, k, rows, T + H)
    check(g, y, row, w if weighted else None)


def test_either_gradient_alone_and_rows_out_of_range():
    g, y, row, w = make(12, 264, 4, 50, 3)
    row[0, 0] = 50
    row[1, 1] = 2 ** 31 - 1
    row[2, 2] = -2 ** 31
    both = check(g, y, torch.where(row >= 50, -1, row), w)
    gd, yd, rd, wd = g.to(DEV), y.to(DEV), row.to(DEV), w.to(DEV)
    dy = torch.full_like(yd, 7.0)
    r = ep.ep_combine_backward(gd, None, rd, wd, 50, out=dict(grad_expert_out=dy))
    assert torch.equal(r["grad_expert_out"], both["grad_expert_out"])
    r = ep.ep_combine_backward(gd, yd, rd, wd, out=dict(grad_topk_weights=torch.empty_like(wd)))
    assert torch.equal(r["grad_topk_weights"], both["grad_topk_weights"])
    r = ep.ep_combine_backward(gd, None, rd, wd, 50)
    assert r["grad_topk_weights"] is None
    # Fewer rows than the tensor holds: the others take no part.
    part = torch.full_like(yd, 7.0)
    r = ep.ep_combine_backward(gd, yd, rd, wd, 30, out=dict(grad_expert_out=part, grad_topk_weights=torch.empty_like(wd)))
    assert (part[30:] == 7).all() and torch.equal(part[:30], both["grad_expert_out"][:30])
    assert torch.equal(r["grad_topk_weights"], torch.where((rd >= 0) & (rd < 30), both["grad_topk_weights"], 0.0))


def test_infinities_and_nan_stay_in_their_slot():
    g, y, row, w = make(4, 128, 2, 8, 5, empty=0.0)
    y[row[1, 0]] = float("nan")
    y[row[2, 1], 3] = float("inf")
    w[3, 0] = float("nan")
    r = ep.ep_combine_backward(g.to(DEV), y.to(DEV), row.to(DEV), w.to(DEV))
    dw, dy = r["grad_topk_weights"].cpu(), r["grad_expert_out"].cpu()
    assert torch.isnan(dw[1, 0]) and not torch.isfinite(dw[2, 1])
    ok = torch.ones(4, 2, dtype=torch.bool)
    ok[1, 0] = ok[2, 1] = False
    assert torch.isfinite(dw[ok]).all()
    assert torch.isnan(dy[row[3, 0]]).all() and torch.isfinite(dy[row[3, 1]]).all()


def test_gradient_of_combine_by_differences():
    """combine is linear in y and in w, so a difference over a whole step is
    exact up to the roundings: the loss sum(c * out) of the 64-bit combine."""
    g, y, row, w = make(3, 16, 2, 6, 8, empty=0.0)
    r = ep.ep_combine_backward(g.to(DEV), y.to(DEV), row.to(DEV), w.to(DEV))
    c, y64, w64, rows = g.double().numpy(), y.double().numpy(), w.double().numpy(), row.numpy()

    def loss(yv, wv):
        return sum(float((c[t] * wv[t, j] * yv[rows[t, j]]).sum()) for t in range(3) for j in range(2))

    base = loss(y64, w64)
    for t in range(3):
        for j in range(2):
            v = w64.copy()
            v[t, j] += 1.0
            assert abs(loss(y64, v) - base - float(r["grad_topk_weights"][t, j])) <= 1e-4
            for h in (0, 7, 15):
                v = y64.copy()
                v[rows[t, j], h] += 1.0
                d = loss(v, w64) - base
                assert abs(d - float(r["grad_expert_out"][rows[t, j], h])) <= 2.0 ** -8 * abs(d) + 1e-9


def test_follows_dispatch_with_empty_slots():
    """The maps of the packed and the padded dispatch, slots dropped and empty."""
    T, H, k, E = 50, 256, 4, 16
    gen = torch.Generator().manual_seed(1)
    idx = torch.rand(T, E, generator=gen).argsort(dim=1)[:, :k].contiguous()
    idx[torch.rand(T, k, generator=gen) < 0.2] = -1
    w = torch.rand(T, k, generator=gen)
    x, g = torch.randn(T, H, generator=gen).bfloat16(), torch.randn(T, H, generator=gen).bfloat16()
    d = ep.ep_dispatch(x.to(DEV), idx.to(DEV), w.to(DEV), E, 4)
    n = int(d["recv_expert_offset"][-1])
    check(g, d["recv_x"][:n].cpu(), d["token_row"].cpu(), w)
    l = ep.ep_dispatch_ll(x.to(DEV), idx.to(DEV), w.to(DEV), E, 7)
    y = torch.randn(E * 7, H, generator=gen).bfloat16()
    check(g, y, l["token_slot"].cpu(), w)


def test_offsets_past_32_bits():
    """Rows whose first element lies past 2^32 (9.8 GB of expert outputs)."""
    rows, H, k = 600000, 8192, 2
    g, small, _, w = make(3, H, k, 6, 4)
    y = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
    y[-6:] = small.to(DEV)
    row = (rows - 1 - torch.arange(6, dtype=torch.int32)).view(3, 2)
    dy = torch.empty_like(y)
    dy[-7] = 7.0
    ref = ep.ep_combine_backward(g.to(DEV), small.to(DEV), (row - (rows - 6)).to(DEV).contiguous(), w.to(DEV))
    r = ep.ep_combine_backward(g.to(DEV), y, row.to(DEV), w.to(DEV),
                               out=dict(grad_expert_out=dy, grad_topk_weights=torch.empty(3, 2, device=DEV)))
    assert torch.equal(r["grad_topk_weights"], ref["grad_topk_weights"])
    assert torch.equal(dy[-6:], ref["grad_expert_out"]) and (dy[-7] == 7).all()


def test_no_tokens_and_refusals():
    e = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    r = ep.ep_combine_backward(e, e, torch.empty(0, 2, dtype=torch.int32, device=DEV), None)
    assert r["grad_topk_weights"].shape == (0, 2)
    g, y, row, w = (v.to(DEV) for v in make(4, 16, 2, 8, 0))
    with pytest.raises(ValueError, match="num_rows is needed"):
        ep.ep_combine_backward(g, None, row, w)
    with pytest.raises(ValueError, match="needs expert_out"):
        ep.ep_combine_backward(g, None, row, w, 8, out=dict(grad_topk_weights=torch.empty_like(w)))
    with pytest.raises(ep.EPError, match="both NULL"):
        ep.ep_combine_backward(g, y, row, w, out={})
    with pytest.raises(ValueError, match="num_rows exceeds"):
        ep.ep_combine_backward(g, y, row, w, 9)
    with pytest.raises(ValueError, match="disagree on hidden"):
        ep.ep_combine_backward(g, torch.zeros(8, 24, dtype=torch.bfloat16, device=DEV), row, w)
    with pytest.raises(ValueError, match="needs"):
        ep.ep_combine_backward(g, y, row, w, out=dict(grad_expert_out=y[:7]))
    with pytest.raises(ep.EPError, match="num_rows must be"):
        ep.ep_combine_backward(g, y, row, w, -1)
