// The arithmetic of the streaming attention kernel's list of work (see
// nq_kv_attn.h), apart from any GPU: also compiled for the CPU, to be tested.
//
// The host picks units so that the list of sequences that share no rows stays
// below 2^31.  What row_start holds is only known on the device, and sequences
// that overlap can make the list longer than 32 bits count.  So sums saturate,
// the list is cut at kListMax, and a segment that passes the cut is not joined:
// its rows, which other sequences have too, keep what those give them.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define NQ_LIST_FN __host__ __device__ __forceinline__
#else
#define NQ_LIST_FN inline
#endif

namespace nqk {

constexpr uint32_t kListMax = 1u << 31;

NQ_LIST_FN uint32_t add_sat(uint32_t a, uint32_t b)
{
    const uint32_t s = a + b;
    return s < a ? ~0u : s;
}

// Units of the list, from the saturated sum of all sequences'.
NQ_LIST_FN uint32_t list_total(uint32_t sum) { return sum < kListMax ? sum : kListMax; }

// Units per worker, `least` or more.
NQ_LIST_FN uint32_t list_share(uint32_t total, uint32_t workers, uint32_t least)
{
    const uint32_t share = (total + workers - 1) / workers;
    return share < least ? least : share;
}

// Workers border and on have a segment of `units` units of which worker border - 1
// has the first `unit`, the last ones before the border between the two: how
// many workers that is in all.  0 where the segment passes the list's end.
NQ_LIST_FN int list_parts(uint32_t border, uint32_t share, uint32_t total, uint32_t unit, uint32_t units)
{
    const uint32_t end = border * share - unit + units;     // past its last unit
    return end > total ? 0 : (int)((end - 1) / share - border + 2);
}

// Behind shared prefixes a list has slots: before each segment's units `extra` more,
// which stand for what a segment costs besides its own.  A worker's run of
// slots begins and ends anywhere in them.

// The units among slots slot0 .. slot0 + slots - 1 of a segment.
struct ListUnits {
    uint32_t first, count;
};
NQ_LIST_FN ListUnits list_units(uint32_t slot0, uint32_t slots, uint32_t extra)
{
    const uint32_t first = slot0 < extra ? 0u : slot0 - extra, end = slot0 + slots;
    return {first, end < extra ? 0u : end - extra - first};
}

// Slots that a worker takes at least, by the units of the list's longest segment: what
// a segment is cut into is joined in any case (4 sequences of 4 heads behind 700
// tokens: 15 us at 1, 28 at 4), but no more than about 64 parts (3 sequences of 4
// heads over one behind 5k and 21k tokens: 44 us with 331 parts, 32 with 83).
NQ_LIST_FN uint32_t list_least(uint32_t longest) { return longest < 128 ? 1u : longest / 64; }

// Where worker `worker` leaves a part of a segment that it has not whole: each has
// room for the last part of one segment and the first of another.
NQ_LIST_FN uint32_t list_place(uint32_t worker, bool first) { return 2 * worker + (first ? 1 : 0); }

// The parts of the segment of `slots` slots behind slot `off` of the list: the worker
// that has its first unit, and how many have some.  None where it passes the list's end.
struct ListParts {
    uint32_t first;
    int count;
};
NQ_LIST_FN ListParts list_segment(uint64_t off, uint32_t slots, uint32_t extra, uint32_t share, uint32_t total)
{
    if (off + slots > total) return {0, 0};
    const uint32_t first = ((uint32_t)off + extra) / share, last = (uint32_t)(off + slots - 1) / share;
    return {first, (int)(last - first) + 1};
}

// Whether all sequences of a batch are streamed behind shared prefixes, as against
// long ones through the tile kernel, in a launch that most often finds none: up to 64 query
// columns in the mean, and no sequence of more than 4096 among others of a row at
// least.  32 heads over 8, all streamed and not: 4 sequences of 5 rows 38 and 62 us, 64 of
// 4 118 and 120, 63 single tokens and a chunk of 256 rows at 4000 tokens 152 and 230,
// 255 and one of 512 200 and 205, of 1024 315 and 302, of 3500 1193 and 708.
NQ_LIST_FN bool list_streams_all(int64_t batch, int64_t rows, int64_t group)
{
    return batch > 1 && (rows + batch - 1) / batch * group <= 64 && (rows - (batch - 1)) * group <= 4096;
}

}  // namespace nqk
