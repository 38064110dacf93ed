"""The paged cache's entry points at the edge of what they accept, and the division of an attention call with the
constants that its kernels run with, on a host-only build."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from test_attend_host_cpu import L, OK, EUNSUP, ROOT, append, attend, check_division, launches, reset  # noqa: F401


# ---------------------------------------------------------------- large pages
@pytest.mark.timeout(20, method="thread")
@pytest.mark.parametrize("page", [(1 << 30) - 1, 1 << 30, (1 << 30) + 1, (1 << 31) - 1])
def test_pages_of_any_size(L, page):  # noqa: F811
    """Such a page holds more keys than a request may have, but a table without columns reads none of them."""
    assert L.stub_page_of(page, (1 << 24) - 1) == 0 and L.stub_page_of(page, 0) == 0
    assert attend(L, pages=1, page=page, cols=0, ldt=0, table=0) == OK
    assert len(launches(L)) == 1
    assert attend(L, pages=1, page=page) == EUNSUP
    assert append(L, pages=1, page=page) == OK


# ---------------------------------------------------------------- division
KINDS = ["few", "few, 8 bits", "many"]


@pytest.fixture(scope="module")
def constants(tmp_path_factory):
    """(rows of a tile, cost beside the keys, least range, keys of a tile that is not cut, keys of a round, workgroups)"""
    if not shutil.which("g++"):
        pytest.skip("g++ is not available")
    path = str(tmp_path_factory.mktemp("constants") / "libconstants.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                    os.path.join(ROOT, "tests", "attend_constants.cpp"), "-o", path], check=True)
    lib = ctypes.CDLL(path)

    def of(kind):
        to = (ctypes.c_int * 6)()
        lib.attend_constants(KINDS.index(kind), to)
        return list(to)
    return of


def divided(L, constants, kind, rows, lens, kv, each, causal, groups):  # noqa: F811
    tile, fixed, least, whole, step, most = constants(kind)
    return check_division(L, rows, lens, kv, tile // each, causal, min(groups, most), least, whole, step, fixed)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(40))
def test_division_with_the_constants_of_the_kernels(L, constants, kind, seed):  # noqa: F811
    rng = random.Random(1000 + seed)
    jobs = rng.choice([1, 2, 3, 40, 257, 300])
    top_rows = rng.choice([1, 1, 4, 200, 3000]) if jobs < 100 else rng.choice([1, 20])
    rows = [rng.choice([0, 1, rng.randint(0, top_rows)]) for _ in range(jobs)]
    top = rng.choice([1, 64, 191, 193, 700, 5000, 30000])
    lens = [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(jobs)]
    divided(L, constants, kind, rows, lens, rng.choice([1, 2, 8, 12]), rng.choice([1, 3, 4, 16]), rng.random() < 0.6,
            rng.choice([1, 8, 100, 256, 512, 768]))


@pytest.mark.parametrize("kind", KINDS)
def test_ranges_that_end_beside_the_keys(L, constants, kind):  # noqa: F811
    """The least ranges fall into the cost that tiles have beside their keys, whose pieces hold no key."""
    tile, fixed, least, whole, step, most = constants(kind)
    for keys in (0, 1, whole - 1, whole, whole + 1, whole + step, least - fixed % least, 2 * least, 5 * whole):
        for jobs in (1, 2, 7):
            divided(L, constants, kind, [1] * jobs, [max(keys, 0)] * jobs, 1, 1, 1, most)
            divided(L, constants, kind, [tile * 3 + 1] * jobs, [max(keys, 0)] * jobs, 2, 1, 0, most)
