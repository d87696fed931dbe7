"""ep_moe_i8 at the limits that ep.h gives, together: the most experts, slots, inputs and
outputs, where its blocks fill their shared memory.  A few experts lie among the many;
results have to be equal to those of the few alone in small batches, and those are
compared with the 64-bit form."""
import numpy as np
import pytest
import torch

from combine_get_dispatch_02_amd import ep
from test_gpu_moe_i8 import DEV, Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,H,F", [
    (512, 1, 2048, 6144, 128),          # one part of the tokens, 32 outputs a block
    (8, 64, 2048, 8192, 128),
    (64, 8, 2048, 128, 2048),           # many parts
    (8, 64, 2048, 1920, 128),           # each wave of up by itself
    (8, 64, 2048, 65536, 128),          # one slot a tile
    (16, 32, 2, 256, 32768),            # one slot a chunk
    (512, 1, 3, 6272, 32768),
])
def test_limits(T, k, E, H, F):
    print("[moe_i8 limits]", T, k, E, H, F, flush=True)
    small = Layer(H, F, min(E, 4))
    at = np.sort(np.random.default_rng(E).permutation(E)[: small.E])
    at[-1] = E - 1
    big = []
    for one in small.dev:
        all_ = torch.zeros(E, *one.shape[1:], dtype=one.dtype, device=DEV)
        all_[torch.from_numpy(at).to(DEV)] = one
        big.append(all_)
    x, idx, w = small.inputs(T, k)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    got = ep.ep_moe_i8(x.to(DEV), to(np.where(idx < 0, -1, at[idx])), to(w), *big)
    some = max(1, 64 // k)
    for t in range(0, T, some):
        assert torch.equal(got[t:t + some], small.run(x[t:t + some], idx[t:t + some], w[t:t + some]))
    # (few slots: the 64-bit form takes a second for eight of the largest)
    x, idx, w = small.inputs(2, 2, seed=1, empty=0)
    small.check(x, idx, w)
