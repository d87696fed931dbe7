"""csrc/w4_plan.h from Python: the header is plain C++, compiled here with g++ behind
a C interface, so that the CPU tests and the GPU tests ask the same code as the
library does."""
import ctypes
import functools
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_get_dispatch_02_amd", "csrc")

SOURCE = r"""
#include "w4_plan.h"
extern "C" void tile_step(int tiles, int buf, int rest, int* out) {
    const ep::TileStep s = ep::tile_step(tiles, buf, rest);
    out[0] = s.weights; out[1] = s.late; out[2] = s.fills; out[3] = s.later; out[4] = s.idle_later;
}
extern "C" void plan(long long num_rows, int capacity, int E, int N, int silu, int* out) {
    const ep::W4Plan p = ep::w4_plan(num_rows, capacity, E, N, silu != 0);
    out[0] = p.stream_most; out[1] = p.tile_above; out[2] = p.tile_rows;
}
extern "C" int scales(int K) { return ep::w4_scales(K); }
"""


@functools.lru_cache(maxsize=None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "w4_plan.cpp"), os.path.join(d, "w4_plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", so])
        return ctypes.CDLL(so)


def tile_step(tiles, buf, rest):
    """(weights, late, fills, later, idle_later)"""
    out = (ctypes.c_int * 5)()
    lib().tile_step(tiles, buf, rest, out)
    return tuple(out)


ALL = 2 ** 31 - 1


def way(num_rows, capacity, E, N, silu):
    """What a call launches: "streams" (for all rows), "both" (streams for experts of
    few rows, tiles for the others) or "tiles", and the rows of a tile (0: none)."""
    out = (ctypes.c_int * 3)()
    lib().plan(ctypes.c_longlong(num_rows), capacity, E, N, int(silu), out)
    most, above, rows = out
    if above == ALL:
        assert most > 0 and rows == 0
        return "streams", 0
    assert most == above
    return ("both" if most else "tiles"), rows


def scales(K):
    return ("single", "eight", "shared")[lib().scales(K)]
