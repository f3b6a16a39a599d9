"""CPU checks of how positions are dealt to CTAs, and of an accepted path's
parts as the commit kernel's threads look at them (csrc/psi_paging.h)."""
import ctypes as C
import os
import random
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "rejection_sampling_verify_b200", "csrc")

HARNESS = r"""
#include "psi_paging.h"
extern "C" {
void t_deal(int total, int tile, int splits, int least, int *out) {
  const psi::Ranges r = psi::deal(total, tile, splits, least);
  out[0] = r.units;
  out[1] = r.per;
}
int t_prefix(const int *nodes, int len, int M, int first, int step) {
  return psi::path_prefix(nodes, len, M, first, step);
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("deal")
    src, so = d / "h.cpp", d / "h.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    str(src), "-o", str(so)], check=True)
    lib = C.CDLL(str(so))
    lib.t_deal.argtypes = [C.c_int] * 4 + [C.c_void_p]
    lib.t_deal.restype = None
    lib.t_prefix.argtypes = [C.c_void_p] + [C.c_int] * 4
    return lib


def _check(lib, total, tile, splits, least):
    out = (C.c_int * 2)()
    lib.t_deal(total, tile, splits, least, out)
    units, per = out
    case = (total, tile, splits, least, units, per)
    assert 1 <= units <= splits, case
    assert per % tile == 0 and per > 0, case
    # every position once, and a position in every range: a range that wrote
    # nothing would leave the join a result of nobody's
    assert (units - 1) * per < total <= units * per, case
    tiles = -(-total // tile)
    assert units <= max(1, -(-tiles // least)), case
    # as many ranges as are allowed, up to evening them out: none twice another's share
    share = max(-(-tiles // splits), least)
    assert per <= share * tile, case
    # the kernels form starts of ranges, and positions up to one tile past the last, in 32 bits
    assert (units - 1) * per < 2**31 and (tiles + 1) * tile < 2**31, case


def test_every_position_is_dealt_once(lib):
    for tile in (64, 128):
        for total in [*range(1, 5 * tile + 2, 7), *(tile * k + d for k in (1, 2, 31, 255, 256, 257)
                                                   for d in (-1, 0, 1)), 10**6,
                      2**31 - 1 - 512]:
            for splits in (1, 2, 3, 7, 18, 37, 255, 256):
                for least in (1, 2, 3, 8, 100, 10**6):
                    _check(lib, total, tile, splits, least)
    rng = random.Random(4)
    for _ in range(20000):
        _check(lib, rng.randint(1, 10 ** rng.randint(1, 9)), rng.choice((64, 128)),
               rng.randint(1, 256), rng.randint(1, 64))


def test_parts_of_a_path_agree_with_the_whole(lib):
    rng = random.Random(9)
    for _ in range(2000):
        M = rng.randint(1, 255)
        nodes = sorted(rng.sample(range(M), rng.randint(1, M)))
        for _ in range(rng.randint(0, 2)):
            nodes[rng.randrange(len(nodes))] = rng.choice((-1, M, M + 3, rng.randrange(M)))
        n = rng.choice((len(nodes), rng.randint(-1, len(nodes))))
        arr = np.ascontiguousarray(nodes, dtype=np.int32)
        want, last = 0, -1
        while want < n and last < nodes[want] < M:
            last = nodes[want]
            want += 1
        step = rng.choice((1, 2, 3, 256))
        got = min(lib.t_prefix(arr.ctypes.data, n, M, first, step) for first in range(step))
        assert got == want, (nodes, n, M, step)
