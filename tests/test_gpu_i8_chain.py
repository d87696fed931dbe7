"""The layer in 8-bit integers as larger batches run it, as a whole.

Combine: out[t] is the bf16 of an fma chain over the token's slots of w * y, y being what
the down products gave: k roundings of 2^-24 of the sum of |w y|, and half a step of bf16.

The whole against the 64-bit form, in the norm.  h is rounded to bf16 on its way to its
codes, which moves the quotient 127 h / a by up to 2^-8 of it, and by as much for the
rounding of a; so a code moves by one with a probability of 2 * 2^-8 |code| at most, and
the codes' error has at most the square 2^-7 sum |code| beside theirs, sum code^2.
Products with weights of no order keep that ratio.  y and out are rounded to bf16: 2^-8 of
the norm each at most.  Random signs keep the ratio in the mean only, for which a fifth is
added."""
import numpy as np
import pytest
import torch

import plain64_i8 as plain
from test_gpu_moe_i8 import DEV, Layer, chain

pytestmark = pytest.mark.gpu


def spans_of(rows, E, capacity):
    m = rows.cpu().numpy()
    return [(e * capacity, int(m[e])) if capacity else (int(m[e]), int(m[e + 1] - m[e])) for e in range(E)]


@pytest.mark.parametrize("T,k", [(1, 8), (60, 4), (100, 6), (400, 8)])
@pytest.mark.parametrize("padded", [False, True])
def test_combine_and_the_whole(T, k, padded):
    layer = Layer(512, 256, 16)
    x, idx, w = layer.inputs(T, k)
    capacity = T * k if padded else 0
    d, rows, h, q, y, out = chain(layer, x.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV), capacity)
    out = out.double().cpu().numpy()

    # combine, from the y that was measured
    to = d["token_slot" if padded else "token_row"].cpu().numpy()
    assert np.array_equal(to >= 0, (idx >= 0) & (idx < layer.E))
    each = y.double().cpu().numpy().reshape(-1, layer.H)[np.where(to < 0, 0, to)] * np.where(to < 0, 0.0, w)[:, :, None]
    ref, size = each.sum(axis=1), np.abs(each).sum(axis=1)
    tol = k * plain.U * size

    def combines(ref):
        return (np.abs(out - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -130).all(axis=1)
    assert combines(ref).all()
    # The bound sees a slot that is left out, in every token that has one.
    t, last = np.arange(T), k - 1 - np.argmax((to >= 0)[:, ::-1], axis=1)
    some = (to >= 0).any(axis=1)
    assert some.any() and not combines(ref - each[t, last])[some].any()

    # the whole
    codes = np.concatenate([q["x_i8"].cpu().numpy().reshape(-1, layer.F)[a:a + n] for a, n in spans_of(rows, layer.E, capacity)]).astype(np.float64)
    ratio = 1.2 * np.sqrt(2.0 ** -7 * np.abs(codes).sum() / (codes ** 2).sum()) + 2 * 2.0 ** -8

    def whole(idx):
        return plain.moe(x.double().numpy(), idx, w, layer.up, layer.us, layer.down, layer.ds)[0]

    def off(ref):
        return np.linalg.norm(out - ref) / np.linalg.norm(ref)
    assert ratio < 0.03
    full = whole(idx)
    print("[chain]", T, k, padded, "off", off(full), "bound", ratio, flush=True)
    assert off(full) <= ratio
    dropped = idx.copy()
    dropped[t, last] = -1
    assert off(whole(dropped)) > 5 * ratio
