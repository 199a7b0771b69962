"""The lists of work of attention behind shared prefixes (nq_kv_list.h), compiled
for the CPU: what the join takes for the parts of a segment are the places that
workers wrote, in the order of the units, wherever runs of slots begin and end;
and shares go by what sequences hold."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "nq_kv_list.h"
extern "C" {
uint32_t total(uint32_t sum) { return nqk::list_total(sum); }
uint32_t share(uint32_t t, uint32_t w, uint32_t least) { return nqk::list_share(t, w, least); }
uint32_t least(uint32_t longest) { return nqk::list_least(longest); }
int streams_all(int64_t batch, int64_t rows, int64_t group) { return nqk::list_streams_all(batch, rows, group); }
uint32_t place(uint32_t worker, uint32_t first) { return nqk::list_place(worker, first != 0); }
void units(uint32_t slot0, uint32_t slots, uint32_t extra, uint32_t *out)
{
    const nqk::ListUnits u = nqk::list_units(slot0, slots, extra);
    out[0] = u.first, out[1] = u.count;
}
void segment(uint64_t off, uint32_t slots, uint32_t extra, uint32_t share, uint32_t total, uint32_t *out)
{
    const nqk::ListParts p = nqk::list_segment(off, slots, extra, share, total);
    out[0] = p.first, out[1] = (uint32_t)p.count;
}
}
"""


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
    u32, pair = ctypes.c_uint32, ctypes.POINTER(ctypes.c_uint32)
    for name, args in (("total", [u32]), ("share", [u32] * 3), ("least", [u32]), ("place", [u32] * 2)):
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, u32
    lib.streams_all.argtypes, lib.streams_all.restype = [ctypes.c_int64] * 3, ctypes.c_int
    lib.units.argtypes, lib.units.restype = [u32] * 3 + [pair], None
    lib.segment.argtypes, lib.segment.restype = [ctypes.c_uint64] + [u32] * 4 + [pair], None
    return lib


def two(fn, *args):
    out = (ctypes.c_uint32 * 2)()
    fn(*args, out)
    return out[0], out[1]


def walk(lst, segments, extra, share, total, workers):
    """What each worker leaves: whole segments, and parts (segment, first unit, units) by place."""
    begins, at = [], 0
    for units in segments:
        begins.append(at)
        at += extra + units
    whole, places = set(), {}
    seg = 0
    for worker in range(workers):
        at, end = worker * share, min(total, (worker + 1) * share)
        while at < end:
            while at >= begins[seg] + extra + segments[seg]:
                seg += 1
            span, slot0 = extra + segments[seg], at - begins[seg]
            slots = min(span - slot0, end - at)
            first, count = two(lst.units, slot0, slots, extra)
            assert count <= slots and first + count <= segments[seg]
            if count == segments[seg]:
                whole.add(seg)
            elif count:
                place = lst.place(worker, first == 0)
                assert place not in places and place < 2 * workers
                places[place] = (seg, first, count)
            at += slots
    return begins, whole, places


def check(lst, segments, extra, workers, least=None):
    total = lst.total(sum(extra + u for u in segments))
    share = lst.share(total, workers, lst.least(max(segments)) if least is None else least)
    assert share * workers >= total
    begins, whole, places = walk(lst, segments, extra, share, total, workers)
    for seg, units in enumerate(segments):
        first, count = two(lst.segment, begins[seg], extra + units, extra, share, total)
        assert (count == 1) == (seg in whole), (seg, count)
        if count == 1:
            continue
        got = [places.pop(lst.place(first + i, i == 0)) for i in range(count)]
        at = 0
        for s, unit, n in got:
            assert s == seg and unit == at
            at += n
        assert at == units
    assert not places       # and nothing that was left is not taken


@pytest.mark.parametrize("extra", [0, 1, 2, 4])
@pytest.mark.parametrize("workers", [256, 512])
def test_parts_are_what_workers_left(lst, extra, workers):
    rng = random.Random(extra * 1000 + workers)
    for case in range(36):
        kind = case % 6
        n = rng.choice([1, 2, 7, 60, 700, 2000])
        if kind == 0:
            segments = [rng.randint(1, 3) for _ in range(n)]
        elif kind == 1:
            segments = [rng.choice([1, 1, 1, 2, 300]) for _ in range(n)]
        elif kind == 2:
            segments = [rng.randint(1, 4000)] * min(n, 60)
        elif kind == 3:
            segments = [8 * rng.randint(1, 9) for _ in range(n)]
        elif kind == 4:
            segments = sorted(int(2 ** rng.uniform(0, 13)) for _ in range(min(n, 200)))
        else:
            segments = [1] * n + [rng.randint(1, 20000)] + [1] * n
        check(lst, segments, extra, workers)
        # any least, and so shares below, at and above what a segment is charged
        for least in (1, 3, 4, 6, 64):
            check(lst, segments, extra, workers, least)


def test_segments_past_the_end_are_not_done(lst):
    top = 1 << 31
    assert lst.total(top + 5) == top
    for off in (top - 99, top - 1, top, top + 7, (1 << 32) + 3, 1 << 40):
        assert two(lst.segment, off, 100, 4, 1 << 22, top) == (0, 0)
    first, count = two(lst.segment, top - 100, 100, 4, 1 << 22, top)
    assert (first, count) == (511, 1)


def test_shares_go_by_the_longest_segment(lst):
    """A worker takes no more than a 64th of the longest segment where the list is short, and all workers have
    work as soon as there is a unit for each."""
    assert [lst.least(n) for n in (1, 63, 64, 127, 128, 640, 1 << 25)] == [1, 1, 1, 1, 2, 10, 1 << 19]
    for tokens, heads, workers in ((4096, 8, 256), (4096, 8, 512), (16384, 8, 512), (700, 4, 512), (1 << 20, 1, 512)):
        units = -(-tokens // 64)
        total = heads * units
        share = lst.share(total, workers, lst.least(units))
        busy = -(-total // share)
        assert busy >= min(workers, total, 64 * heads) // 2


@pytest.mark.parametrize("batch,rows,group,all_streamed", [
    (4, 20, 4, True), (64, 256, 4, True), (40, 120, 4, True), (64, 63 + 256, 4, True), (256, 255 + 512, 4, True),
    (257, 256 + 3500, 4, False), (121, 120 + 300, 16, False), (1000, 999 + 5000, 8, False),     # a long chunk among single tokens
    (4, 200, 4, False), (1, 1, 4, False), (1, 4000, 4, False)])
def test_a_long_chunk_among_single_tokens_is_not_streamed(lst, batch, rows, group, all_streamed):
    assert bool(lst.streams_all(batch, rows, group)) == all_streamed
