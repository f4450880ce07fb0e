"""The draft tree's steps and the rows of pages as the paged kernels take them (csrc/paging.h), on the host."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import streaming

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def S(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("tree") / "libtree_host.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "causal_attention_sdpa_b200", "csrc"),
                    os.path.join(ROOT, "tests", "tree_host.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def tree(S, parents):
    N = len(parents)
    anc, depth = (ctypes.c_ulonglong * 64)(), (ctypes.c_int * 64)()
    S.tree_all(N, (ctypes.c_int * N)(*parents), anc, depth)
    return list(anc), list(depth)


def check(S, parents):
    anc, depth = tree(S, parents)
    for n in range(64):
        path = streaming.ancestors(parents, n) if n < len(parents) else [n]
        assert anc[n] == sum(1 << x for x in path), (parents, n)
        assert depth[n] == len(path) - 1


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 34, 63, 64])
def test_trees_match_the_walk_up(S, N):
    check(S, list(range(-1, N - 1)))                                # a chain
    check(S, [-1] * N)                                              # no two related
    check(S, [-1] + [0] * (N - 1))                                  # all children of one
    check(S, [max(-1, n - 2) for n in range(N)])                    # two chains
    check(S, [-1 if n % 33 == 0 else n - 1 for n in range(N)])
    r = np.random.default_rng(N)
    for _ in range(50):
        check(S, [int(r.integers(-1, n)) for n in range(N)])
        check(S, [int(r.integers(max(-1, n - 4), n)) for n in range(N)])


@pytest.mark.parametrize("N", [1, 2, 33, 64])
def test_parents_that_are_none_are_the_context(S, N):
    check(S, list(range(N)))                                        # its own
    check(S, [2 ** 31 - 1] * N)
    check(S, [-2 ** 31] * N)
    r = np.random.default_rng(N)
    for _ in range(100):
        check(S, [int(x) for x in r.integers(-70, 70, N)])
        check(S, [int(r.choice([-2 ** 31, -1, n - 1, n, n + 1, 2 ** 31 - 1])) for n in range(N)])


def test_rows_of_pages(S):
    r = np.random.default_rng(3)
    for _ in range(200):
        page, n_pages, Hkv = int(r.integers(1, 200)), int(r.integers(1, 1000)), int(r.integers(1, 20))
        h, e, at = int(r.integers(0, Hkv)), int(r.integers(-3, n_pages + 3)), int(r.integers(0, page))
        want = (e * Hkv + h) * page + at if 0 <= e < n_pages else -1
        assert S.tree_pool_row(e, at, page, n_pages, Hkv, h) == want
    for e in (-2 ** 31, -1, 10, 2 ** 31 - 1):
        assert S.tree_pool_row(e, 0, 16, 10, 4, 1) == -1
    # the last row of the largest pool, 2^31 - 1 rows
    assert S.tree_pool_row(0, 2 ** 31 - 2, 2 ** 31 - 1, 1, 1, 0) == 2 ** 31 - 2
