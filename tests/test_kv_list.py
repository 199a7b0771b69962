"""The arithmetic of the streaming attention's list of work (nq_kv_list.h),
compiled for the CPU: every border that a segment passes finds workers that
exist and whose parts were written, also where sequences that share rows make
the list longer than 32 bits count."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "nq_kv_list.h"
extern "C" {
uint32_t add_sat(uint32_t a, uint32_t b) { return nqk::add_sat(a, b); }
uint32_t total(uint32_t sum) { return nqk::list_total(sum); }
uint32_t share(uint32_t t, uint32_t w, uint32_t least) { return nqk::list_share(t, w, least); }
int parts(uint32_t border, uint32_t s, uint32_t t, uint32_t unit, uint32_t units)
{
    return nqk::list_parts(border, s, t, unit, units);
}
}
"""
WORKERS = 512


@pytest.fixture(scope="module")
def lst(tmp_path_factory):
    compiler = shutil.which("g++") or shutil.which("clang++")
    if not compiler:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("list")
    (d / "list.cc").write_text(SOURCE)
    csrc = os.path.join(ROOT, "group_wise_affine_quantize_amd", "csrc")
    subprocess.run([compiler, "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{csrc}", "-o", str(d / "list.so"),
                    str(d / "list.cc")], check=True)
    lib = ctypes.CDLL(str(d / "list.so"))
    for name, n in (("add_sat", 2), ("total", 1), ("share", 3), ("parts", 5)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [ctypes.c_uint32] * n, ctypes.c_int if name == "parts" else ctypes.c_uint32
    return lib


def saturated(lst, works):
    total = 0
    for w in works:
        total = lst.add_sat(total, w)
    return total


# (units of a segment, segments of a sequence) of the sequences of a batch
BATCHES = {
    "one short": [(3, 1)],
    "one long": [(2049, 4)],
    "uneven": [(1, 8), (700, 8), (0, 0), (33, 8), (1029, 8), (2, 3)],
    "a border at a segment's start": [(8, 64)] * 64,
    "near the limit": [(1 << 20, 2000)],
    # sequences that claim the same rows
    "past 31 bits": [(2048, 1 << 17)] * 9,
    "past 32 bits": [(2048, 1 << 19)] * 12,
    "far past 32 bits": [((1 << 20) + 7, 2000)] * 4096,
}


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("least", [1, 8])
def test_every_border_joins_parts_that_workers_wrote(lst, name, least):
    batch = BATCHES[name]
    true = sum(u * n for u, n in batch)
    total = lst.total(saturated(lst, [u * n for u, n in batch]))
    assert total == min(true, 1 << 31)
    share = lst.share(total, WORKERS, least)
    assert share >= least and share * WORKERS >= total
    for border in range(1, WORKERS):
        at = border * share
        if at >= total:
            break
        first = 0           # the segment that holds unit `at`, by whole numbers of any size
        for units, count in batch:
            if at < first + units * count:
                break
            first += units * count
        unit = (at - first) % units
        if unit == 0 or unit > share:
            continue
        begin, end = at - unit, at - unit + units
        got = lst.parts(border, share, total, unit, units)
        if end > total:
            assert got == 0     # its end was cut off: some parts were never written
            continue
        assert got == (end - 1) // share - begin // share + 1
        assert begin // share == border - 1 and 2 <= got <= WORKERS - (border - 1)


def test_sums_stay_at_their_limit(lst):
    top = 2 ** 32 - 1
    for a, b in ((0, 0), (5, 7), (top, 0), (top, 1), (top, top), (1 << 31, 1 << 31), (1 << 31, (1 << 31) - 1)):
        assert lst.add_sat(a, b) == min(a + b, top)
        assert lst.total(a) == min(a, 1 << 31)
