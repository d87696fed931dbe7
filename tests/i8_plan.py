"""csrc/i8_plan.h from Python: the header is plain C++, compiled here with g++ behind
a C interface, so that the CPU tests and the GPU tests ask the same code as the
library does."""
import ctypes
import functools
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_get_dispatch_02_amd", "csrc")

SOURCE = r"""
#include "i8_plan.h"
extern "C" void quarter(int q, int* out) {
    const ep::I8Quarter s = ep::i8_quarter(q);
    out[0] = s.from; out[1] = s.to; out[2] = s.later;
}
extern "C" int streams(long long num_rows, int E, int K, int N, int silu) {
    return ep::i8_streams(num_rows, E, K, N, silu != 0);
}
"""


@functools.lru_cache(maxsize=None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "i8_plan.cpp"), os.path.join(d, "i8_plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", so])
        return ctypes.CDLL(so)


def quarter(q):
    """(from, to, later)"""
    out = (ctypes.c_int * 3)()
    lib().quarter(q, out)
    return tuple(out)


def way(num_rows, E, K, N, silu):
    """What a call launches: "streams" or "tiles"."""
    return "streams" if lib().streams(ctypes.c_longlong(num_rows), E, K, N, int(silu)) else "tiles"
