"""Which kernel the 4-bit head takes for a call, and that the GPU tests reach all
of them (no GPU needed: the choice is plain C++)."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "draft_verification_amd", "csrc")
SHIM = """
#include "sv_head_choice.h"
extern "C" int tile(int rows, long long vocab, int fp4, int group) { return sv::head_tile_rows(rows, vocab, fp4 != 0, group); }
extern "C" int once(int tile, long long blocks) { return sv::head_tile_once(tile, blocks); }
"""
FORMATS = [("fp4", 32), ("int4", 32), ("int4", 64), ("int4", 128)]


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    src, lib = str(d / "choice.cpp"), str(d / "choice.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    L.tile.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    L.once.argtypes = [ctypes.c_int, ctypes.c_longlong]

    def kernel(M, V, fmt, group):
        """(rows of the tile or 0, weights read once)"""
        t = L.tile(M, V, fmt == "fp4", group)
        return t, bool(t and L.once(t, -(-M // t)))
    return kernel


def test_the_choice_is_among_the_kernels(choice):
    for fmt, group in FORMATS:
        for V in (1, 63, 64, 1000, 8000, 50257, 129280, 2 ** 20):
            for M in (1, 8, 9, 16, 17, 31, 33, 64, 65, 100, 559, 4352, 100000):
                t, once = choice(M, V, fmt, group)
                assert t in (0, 16, 32, 64) and (t == 0 or M > 8)
                assert once == (t in (16, 32) and M <= t)
            assert choice(8, V, fmt, group)[0] == 0
        # many rows over a large vocabulary read the weights as seldom as they can
        assert choice(559, 129280, fmt, group) == (64, False)


def test_every_kernel_is_reached_by_the_gpu_tests(choice):
    from tests import test_gpu_n_head as N
    from tests import test_gpu_q_edges as Q
    reached = set()
    for M, V, H, fmt, group, dtype in [c[:6] for c in N.CASES] + N.BLOCKS + Q.HEADS:
        reached.add((fmt, group, dtype) + choice(M, V, fmt, group))
    for fmt, group in FORMATS:
        for dtype in ("f32", "bf16"):
            for kernel in ((0, False), (16, True), (16, False), (32, True), (32, False), (64, False)):
                assert (fmt, group, dtype) + kernel in reached
