"""How a norm's gradient deals its rows to workgroups (nq_norm_chunks.h),
compiled for the CPU: every row is in one chunk, none mixes the rows of two
gates unless it holds whole ones, no team has much more than its share of a
chunk, and the workspace for one gate over all rows is never the larger."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "nq_norm_chunks.h"
extern "C" {
int teams(int64_t dim) { return nqk::norm_grad_teams(dim); }
void chunks(int64_t rows, int64_t gates, int teams, int64_t *out)
{
    const nqk::Chunks c = nqk::norm_chunks(rows, gates, teams);
    out[0] = c.chunks, out[1] = c.per_gate, out[2] = c.gates, out[3] = c.cuts, out[4] = c.size;
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    compiler = shutil.which("g++") or shutil.which("clang++")
    if not compiler:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("chunks")
    (d / "chunks.cc").write_text(SOURCE)
    csrc = os.path.join(ROOT, "group_wise_affine_quantize_amd", "csrc")
    subprocess.run([compiler, "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{csrc}", "-o", str(d / "chunks.so"),
                    str(d / "chunks.cc")], check=True)
    lib = ctypes.CDLL(str(d / "chunks.so"))
    lib.teams.argtypes, lib.teams.restype = [ctypes.c_int64], ctypes.c_int
    lib.chunks.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]
    lib.chunks.restype = None
    return lib


def chunks(lib, rows, gates, teams):
    out = (ctypes.c_int64 * 5)()
    lib.chunks(rows, gates, teams, out)
    return dict(zip(("chunks", "per_gate", "gates", "cuts", "size"), out))


def runs_of(c, rows, k):
    """First and last row of chunk k, and the rows that stay with one team."""
    if c["gates"]:
        first = k * c["size"]
        return first, min(first + c["size"], rows), c["per_gate"]
    g, part = divmod(k, c["cuts"])
    first = g * c["per_gate"] + part * c["size"]
    last = first + c["size"] if (part + 1) * c["size"] < c["per_gate"] else (g + 1) * c["per_gate"]
    return first, last, 1


SIZES = [(1, 1), (3, 1), (8, 1), (15, 1), (15, 3), (15, 15), (16, 1), (16, 2), (16, 16), (17, 1), (40, 8), (700, 7), (700, 350),
         (1501, 1501), (2000, 500), (2040, 680), (8192, 4), (8190, 1638), (8190, 819), (8000, 800), (9000, 3), (9000, 1125),
         (120000, 600), (120000, 2400), (120000, 6000), (120000, 120000), (131072, 512), (120000, 1), ((1 << 31) - 2, 2)]


@pytest.mark.parametrize("rows,gates", SIZES)
@pytest.mark.parametrize("teams", [1, 2, 4, 8])
def test_rows_are_dealt_evenly(lib, rows, gates, teams):
    c = chunks(lib, rows, gates, teams)
    want = 16 if rows <= 16 else max(4, -(-rows // 512))
    end = 0
    for k in range(c["chunks"]):
        first, last, run = runs_of(c, rows, k)
        assert first == end and first < last <= rows
        end = last
        assert last - first <= want
        if not c["gates"]:      # a part of one gate
            assert first // c["per_gate"] == (last - 1) // c["per_gate"]
        else:
            assert first % c["per_gate"] == 0 and (last - first) % c["per_gate"] == 0
        # rows that the busiest team has one after the other: at most twice an even share of
        # the most that a chunk holds, or as many as there are runs; one workgroup that
        # spares a second launch may have a gate's eight
        most = -(-((last - first) // run) // teams) * run
        assert most <= max(2 * -(-want // teams), int(want ** 0.5), 8 if rows <= 16 and gates > 1 else 0), (k, c)
    assert end == rows


@pytest.mark.parametrize("rows,gates", SIZES)
@pytest.mark.parametrize("teams", [1, 2, 4, 8])
def test_one_gate_takes_no_more_workspace(lib, rows, gates, teams):
    """The workspace is for any gate of these rows; a call without one takes all rows as one gate's."""
    assert chunks(lib, rows, 1, teams)["chunks"] <= chunks(lib, rows, gates, teams)["chunks"]


def test_teams_of_each_width(lib):
    assert [lib.teams(d) for d in (1, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097, 16384)] == [8, 8, 4, 4, 2, 2, 1, 1, 1, 1]
    assert chunks(lib, 0, 7, 8)["chunks"] == 0
