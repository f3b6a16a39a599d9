"""CPU checks of the cache kernels' index arithmetic (csrc/psi_paging.h).

The header's functions compile for the host; a small harness built with the
system compiler exposes them, and they are compared with plain Python over
page sizes, lengths at and past the table's end, bad page indices, offsets
beyond 32 bits, and valid and invalid trees and paths."""
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
using namespace psi;
extern "C" {
long long t_slot(const int *row, int max_pages, int num_pages, int page_size, long long ps,
                 long long ss, long long t) {
  Paging g{};
  g.max_pages = max_pages; g.num_pages = num_pages; g.page_size = page_size;
  g.page_stride = ps; g.slot_stride = ss;
  return slot_offset(g, row, t);
}
int t_depth(const int *parents, int r) { return row_depth(parents, r); }
int t_sees(const int *parents, int r, unsigned *bits) { return row_sees(parents, r, bits); }
int t_prefix(const int *nodes, int len, int M) { return path_prefix(nodes, len, M); }
long long t_pages(long long slots, int page_size) { return pages_for(slots, page_size); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("paging")
    src, so = d / "h.cpp", d / "h.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    str(src), "-o", str(so)], check=True)
    lib = C.CDLL(str(so))
    lib.t_slot.restype = lib.t_pages.restype = C.c_longlong
    lib.t_slot.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_longlong, C.c_longlong,
                           C.c_longlong]
    lib.t_pages.argtypes = [C.c_longlong, C.c_int]
    for f in (lib.t_depth, lib.t_sees, lib.t_prefix):
        f.restype = C.c_int
    lib.t_depth.argtypes = [C.c_void_p, C.c_int]
    lib.t_sees.argtypes = [C.c_void_p, C.c_int, C.c_void_p]
    lib.t_prefix.argtypes = [C.c_void_p, C.c_int, C.c_int]
    return lib


def _arr(x):
    return np.ascontiguousarray(x, dtype=np.int32)


@pytest.mark.parametrize("S", [1, 3, 16, 128, 1024])
def test_slot_offsets_stay_inside_the_pool(lib, S):
    P, mp = 7, 5
    row = _arr([6, 0, -1, 7, 3])  # one page not held, one past the pool
    ps, ss = 3_000_000_000, 1_000_000  # offsets pass 32 bits
    for t in [-1, 0, S - 1, S, 2 * S, 3 * S, 4 * S, 5 * S - 1, 5 * S, 5 * S + 1, 2**31, 2**40]:
        got = lib.t_slot(row.ctypes.data, mp, P, S, ps, ss, t)
        page = row[t // S] if 0 <= t < mp * S else -1
        want = int(page) * ps + (t % S) * ss if 0 <= page < P else -1
        assert got == want, (t, got, want)


def _plain_chain(parents, r):
    """Rows on the way to the root, or None."""
    rows = [r]
    while r > 0:
        p = parents[r - 1]
        if p < -1 or p >= r - 1:
            return None
        r = p + 1
        rows.append(r)
    return rows


def test_rows_and_depths_of_trees(lib):
    rng = random.Random(5)
    for R in (1, 2, 31, 32, 33, 64, 65, 255, 256):
        for kind in ("tree", "bad", "chain"):
            parents = [rng.randint(-1, k - 1) for k in range(R - 1)]
            if kind == "bad":
                for _ in range(1 + R // 16):
                    if R > 1:
                        k = rng.randrange(R - 1)
                        parents[k] = rng.choice((k, k + 1, -2, R, 2**31 - 1, -2**31))
            if kind == "chain":
                parents = list(range(-1, R - 2))
            arr = _arr(parents + [0])
            for r in range(R):
                bits = np.zeros(8, dtype=np.uint32)
                ok = lib.t_sees(arr.ctypes.data, r, bits.ctypes.data)
                rows = _plain_chain(parents, r)
                assert ok == (rows is not None)
                assert lib.t_depth(arr.ctypes.data, r) == (-1 if rows is None else len(rows) - 1)
                got = {i for i in range(256) if (bits[i // 32] >> (i % 32)) & 1}
                assert got == set(rows or [])
                if kind == "chain":  # no parents: the same as the chain spelled out
                    b2 = np.zeros(8, dtype=np.uint32)
                    assert lib.t_sees(None, r, b2.ctypes.data)
                    assert np.array_equal(bits, b2) and lib.t_depth(None, r) == r


def test_accepted_paths_are_cut_at_the_first_bad_node(lib):
    cases = [([0, 2, 5], 3, 8, 3), ([0, 2, 5], 2, 8, 2), ([0, 2, 2], 3, 8, 2), ([3, 1], 2, 8, 1),
             ([-1, 1], 2, 8, 0), ([7, 8], 2, 8, 1), ([1], 0, 8, 0), ([1], -3, 8, 0),
             (list(range(8)), 9, 8, 8)]
    for nodes, n, M, want in cases:
        arr = _arr(nodes + [0] * 8)
        assert lib.t_prefix(arr.ctypes.data, n, M) == want, (nodes, n)


def test_pages_for_lengths(lib):
    for S in (1, 16, 1000):
        for n in (-5, 0, 1, S - 1, S, S + 1, 2**31 + 7):
            assert lib.t_pages(n, S) == (0 if n <= 0 else -(-n // S))
