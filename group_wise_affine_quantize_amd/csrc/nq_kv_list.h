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

}  // namespace nqk
