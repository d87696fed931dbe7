"""The calls of the 8-bit layer in company: saved maps that point outside, captured
products whose rows change between the replays, a workspace that two graphs share,
two threads at once.  Results have to be equal to those of each call alone, which other
tests compare with plain64_i8.py.
"""
import threading

import numpy as np
import pytest
import torch

import i8_plan
import plain64_i8 as plain
from combine_get_dispatch_02_amd import ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def test_saved_maps_that_point_outside():
    rng = np.random.default_rng(1)
    T, k, H, rows = 37, 4, 272, 90
    x = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).bfloat16()
    to = rng.permutation(T * k).reshape(T, k).astype(np.int32)      # from `rows` on: skipped
    to[3, 1], to[5], to[7, 0], to[9, 2] = -1, -2 ** 31, 2 ** 31 - 1, rows
    out = dict(recv_x_i8=torch.full((rows + 2, H), 9, dtype=torch.int8, device=DEV), recv_scales=torch.full((rows + 2,), 9.0, device=DEV))
    ep.ep_dispatch_i8_cached(x.to(DEV), dev(to), rows, out=out)
    codes, scales = plain.cast(x.double().numpy())
    q, s = np.full((rows + 2, H), 9), np.full(rows + 2, 9, np.float32)
    for t in range(T):
        for r in to[t]:
            if 0 <= r < rows:
                q[r], s[r] = codes[t], scales[t]
    assert np.array_equal(out["recv_x_i8"].cpu().numpy(), q) and np.array_equal(out["recv_scales"].cpu().numpy(), s)


@pytest.mark.parametrize("K,N", [(1024, 256), (384, 272)])
def test_captured_products_of_other_rows(K, N):
    """A graph holds the addresses; how many rows each expert has it reads anew."""
    rng = np.random.default_rng([2, K])
    E, rows = 6, 180
    assert i8_plan.way(rows, E, K, N, False) == ("streams" if K == 1024 else "tiles")
    x, xs = rng.integers(-128, 128, (rows, K), dtype=np.int8), rng.random(rows, dtype=np.float32) / 64
    w, ws = rng.integers(-128, 128, (E, N, K), dtype=np.int8), rng.random((E, N), dtype=np.float32) / (64 * K ** 0.5)
    a = [dev(t) for t in (x, xs, np.zeros(E + 1, np.int32), w, ws)]
    y = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    q = dict(x_i8=torch.empty(rows, N, dtype=torch.int8, device=DEV), x_scales=torch.empty(rows, device=DEV))

    def both(out, cast):
        ep.ep_expert_linear_i8(*a, out=out)
        ep.ep_quantize_i8(out, a[2], out=cast)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(y, q)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(y, q)
    for counts in ([30] * 6, [0] * 6, [180, 0, 0, 0, 0, 0], [0, 1, 0, 2, 0, 100], [17, 16, 15, 33, 64, 3]):
        a[2].copy_(dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)))
        n = sum(counts)
        y.fill_(7.0)
        q["x_i8"].fill_(9)
        q["x_scales"].fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        eager, cast = torch.full_like(y, 7.0), dict(x_i8=torch.full_like(q["x_i8"], 9), x_scales=torch.full_like(q["x_scales"], 9.0))
        both(eager, cast)
        assert torch.equal(y, eager) and all(torch.equal(q[name], cast[name]) for name in q)
        assert (y[n:] == 7).all() and (q["x_i8"][n:] == 9).all() and (q["x_scales"][n:] == 9).all()


class Layer:
    def __init__(self, H, F, E, T, k, seed):
        rng = np.random.default_rng(seed)
        self.weights = [dev(a) for a in (rng.integers(-127, 128, (E, 2 * F, H), dtype=np.int8),
                                         (rng.random((E, 2 * F), dtype=np.float32) + 0.5) / (74 * H ** 0.5),
                                         rng.integers(-127, 128, (E, H, F), dtype=np.int8),
                                         (rng.random((E, H), dtype=np.float32) + 0.5) / (74 * F ** 0.5))]
        self.x = torch.from_numpy(rng.standard_normal((T, H), dtype=np.float32)).bfloat16().to(DEV)
        self.idx, self.w = dev(rng.integers(-1, E, (T, k))), dev(rng.random((T, k), dtype=np.float32))
        self.bytes = ep.ep_moe_i8_workspace_bytes(T, k, F)

    def run(self, **kw):
        return ep.ep_moe_i8(self.x, self.idx, self.w, *self.weights, **kw)


# Few and many slots an expert, inputs that waves share and those that they do not.
LAYERS = [(256, 384, 8, 3, 4), (4096, 128, 8, 64, 8), (2048, 256, 60, 20, 6), (1024, 512, 16, 33, 2)]


def test_a_workspace_that_two_graphs_share():
    """One replay after the other, each ends before the next uses the workspace."""
    layers = [Layer(*a, seed) for seed, a in enumerate(LAYERS)]
    room = torch.full((max(la.bytes for la in layers),), 255, dtype=torch.uint8, device=DEV)
    alone = [la.run() for la in layers]
    outs = [torch.zeros_like(la.x) for la in layers]
    torch.cuda.synchronize()
    graphs = []
    for la, out in zip(layers, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            la.run(out=out, workspace=room)
        graphs.append(g)
    for order in ((0, 1, 2, 3), (3, 1, 0, 2), (2, 2, 1, 3, 0)):
        for out in outs:
            out.zero_()
        for n in order:
            graphs[n].replay()
        torch.cuda.synchronize()
        for out, ref in zip(outs, alone):
            assert torch.equal(out, ref)


def test_two_threads_on_streams_of_their_own():
    layers = [Layer(*a, seed) for seed, a in enumerate(LAYERS[:2])]
    alone = [la.run() for la in layers]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[n].append(layers[n].run())
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for n in (0, 1):
        assert len(got[n]) == 20 and all(torch.equal(g, alone[n]) for g in got[n])
