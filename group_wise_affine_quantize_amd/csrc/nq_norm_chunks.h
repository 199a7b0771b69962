// How the rows of a norm's gradient are dealt to workgroups and their teams of
// waves, apart from any GPU: also compiled for the CPU, to be tested.
//
// A gate's rows are not mixed with another's in one sum, so a workgroup's rows, a
// chunk, are
//   whole gates, each gate's run of rows one team's, which writes its gradient; or
//   all of one gate's rows or a part of them, which the teams take by turns.
// Where gates have fewer rows than a chunk, the first keeps more rows in one sum of
// the other parameters, the second keeps teams at work: it is taken where a chunk
// would hold fewer runs than there are teams to take them.  120000 rows of 512 (eight
// teams) in bf16 with gates of 200 rows, one run to a chunk: 752 us in runs, 201 by
// turns; of 50 rows, four runs: 262 and 173; 8000 rows of 2048 (two teams), gates of
// 10, one run: 78 and 61; but 16000 rows of 512, gates of 8, four runs: 40 and 46.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace nqk {

struct Chunks {
    int64_t chunks;     // workgroups
    int64_t per_gate;   // rows that share a gate
    int64_t gates;      // gates of a chunk (0: the chunk is a part of one)
    int64_t cuts;       // chunks of a gate
    int64_t size;       // rows of a chunk
};

// Teams of a workgroup: eight waves of 512 columns' work each, but one team at
// least (past 4096 columns of 16 waves).
inline int norm_grad_teams(int64_t dim)
{
    int waves = 1;
    while (waves < 8 && dim > 512 * waves) waves *= 2;
    return 8 / waves;
}

inline Chunks norm_chunks(int64_t rows, int64_t gates, int teams)
{
    // two workgroups per compute unit to 4096 columns (8192 rows of 2048: 54 us with
    // one of twice the waves; past that they have 16 waves, of which one fits, and
    // come in two rounds); at least 4 rows each (1501 rows of 1407: 24 us, 26.5 with
    // 8); and up to 16 rows in one, which spares the second launch: to 2048 columns as
    // fast or faster (a call for 16 rows of 512 in bf16 13.7 us, 17.7 cut up; of 2048
    // 17.5 both), past that slower (of 4096 34 and 18, of 16384 120 and 34)
    constexpr int64_t kMost = 512, kLeast = 4, kAlone = 16;
    Chunks c{};
    if (rows == 0) return c;
    const int64_t want = rows <= kAlone ? kAlone : std::max<int64_t>(kLeast, (rows + kMost - 1) / kMost);
    c.per_gate = rows / gates;
    const int64_t runs = want / c.per_gate;
    if (c.per_gate < want && (runs >= std::min<int64_t>(teams, c.per_gate) || (rows <= kAlone && gates > 1))) {
        c.gates = runs;
        c.cuts = 1;
        c.size = c.gates * c.per_gate;
        c.chunks = (gates + c.gates - 1) / c.gates;
    } else {
        c.cuts = (c.per_gate + want - 1) / want;
        c.size = (c.per_gate + c.cuts - 1) / c.cuts;
        c.cuts = (c.per_gate + c.size - 1) / c.size;
        c.chunks = gates * c.cuts;
    }
    return c;
}

}  // namespace nqk
