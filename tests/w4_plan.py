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
