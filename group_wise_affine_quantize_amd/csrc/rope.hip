// Rotary positions with one or several axes (contract in include/nq.h).
//
// Mathematics.  Pair i of a head, (a, b), becomes
//   scale * (a cos t - b sin t),  scale * (b cos t + a sin t),
//   t = freq[i] * position[axis[i]],
// a rotation: its gradient is the rotation by -t with the same scale.
//
// The angle is taken in 64 bits: at position 10^6 and frequency 1, 32 bits of it
// would be off by 0.03.  It is counted in quarter turns, q = t * 2 / pi; the
// nearest whole number leaves |q| <= 1/2, where the series of sine and cosine
// to the terms x^13 and x^14 are within 2^-45.  One thread takes one pair of one row;
// all of the row's heads use it, out of LDS.  A thread keeps to the same columns of
// the heads it takes, so that it divides by sizes only once.
//
// What bounds it: reading and writing the heads once.  8192 rows of 40 heads of
// 128 in bf16 (168 MB): 34 us in pairs, 4.9 TB/s; 40 in halves, whose swap and
// turns out of LDS are twice as many; 16 rows of 40 heads: 5.5 us, the way from
// an axis to its position to an angle.
#include <algorithm>

#include "nq_kv.h"
#include "nq_layer.h"
#include "nq_tiles.h"
#include "nq_vec.h"

namespace nqk {

namespace {

constexpr int kThreads = 256;
constexpr int kTurns = 1024;        // pairs of all of a workgroup's rows

// cos and sin of t, t in 64 bits.
__device__ __forceinline__ float2 cos_sin(double t)
{
    const double q = t * 0.63661977236758134308;    // quarter turns
    const double n = rint(q);
    const double x = (q - n) * 1.57079632679489661923, s = x * x;
    const double sn = x * fma(s, fma(s, fma(s, fma(s, fma(s, fma(s, 1.0 / 6227020800.0, -1.0 / 39916800.0),
                                                          1.0 / 362880.0), -1.0 / 5040.0), 1.0 / 120.0), -1.0 / 6.0), 1.0);
    const double cs = fma(s, fma(s, fma(s, fma(s, fma(s, fma(s, fma(s, -1.0 / 87178291200.0, 1.0 / 479001600.0),
                                                             -1.0 / 3628800.0), 1.0 / 40320.0), -1.0 / 720.0),
                                        1.0 / 24.0), -0.5), 1.0);
    const int turn = (int)(n - 4.0 * floor(n * 0.25));      // 0 .. 3
    const float a = (float)(turn & 1 ? sn : cs), b = (float)(turn & 1 ? cs : sn);
    return make_float2(turn == 1 || turn == 2 ? -a : a, turn >= 2 ? -b : b);
}

// How a thread comes by the two elements of a pair.
enum {
    kNeighbours,    // the layout of pairs: both lie in its piece of E columns
    kSwap,          // halves: its piece is of one half, a lane of its wave has the other
    kBoth,          // halves: it takes a piece of each
};
// Writing whole heads in neighbouring lanes is what kSwap is for: the memory
// moved twice the bytes of kBoth's stores, of which each covers half of every
// head (8192 rows of 40 heads of 128 in bf16, 168 MB: 57 us, WRITE_SIZE 168 MB for
// 84).  kBoth is left for single elements and for heads of more than 64 pieces.

// Where a thread is among the pieces of a workgroup's rows: `lanes` threads
// take the pieces of one head, and heads follow each other over the rows.
struct Walk {
    int row, head, j;
    __device__ __forceinline__ void carry(int heads)
    {
        while (head >= heads) head -= heads, ++row;
    }
};

// A workgroup takes `rows_each` rows.  Its first loads are on their way while
// the angles are computed, kAhead of them to a thread.
template <typename T, int E, int HOW, bool AL>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeLaunch a, int64_t row0, int rows_each)
{
    constexpr int kAhead = 4;
    constexpr int P = HOW != kNeighbours ? E : E == 1 ? 1 : E / 2;      // pairs that a piece has a part in
    constexpr bool TWO = HOW == kBoth || E == 1;                        // two accesses to a piece
    __shared__ __align__(16) float2 turn[kTurns];
    const int half = a.rotary >> 1, tid = (int)threadIdx.x, lane = tid & 63;
    const int64_t first = row0 + (int64_t)blockIdx.x * rows_each;
    const int rows = a.rows - first < rows_each ? (int)(a.rows - first) : rows_each;
    const T *x = static_cast<const T *>(a.x) + first * a.ldx;
    T *out = static_cast<T *>(a.out) + first * a.ldo;
    // pieces of a head: those that turn, then those that are copied
    const int half_pieces = half / P, turning = HOW == kSwap ? 2 * half_pieces : half_pieces;
    const int per = turning + (a.x == a.out ? 0 : (a.head_dim - a.rotary) / E);
    // heads that are taken at once; with kSwap no head lies in two waves
    const int lanes = per < kThreads ? per : kThreads, in_wave = 64 / lanes;
    const int side = HOW == kSwap ? kThreads / 64 * in_wave : kThreads / lanes;
    const int at0 = HOW == kSwap ? lane : tid, h0 = at0 / lanes;
    const bool idle = HOW == kSwap ? h0 >= in_wave : h0 >= side;
    const int start = at0 - h0 * lanes;
    Walk w{0, HOW == kSwap ? (tid >> 6) * in_wave + h0 : h0, start};
    w.carry(a.heads);
    if (idle) w.row = rows;
    auto advance = [&](Walk &v) {
        v.j += lanes;
        if (v.j >= per) v.j = start, v.head += side, v.carry(a.heads);
    };
    // the columns of a piece (and of its second access)
    auto column = [&](int j) {
        if (j >= turning) return a.rotary + (j - turning) * E;
        return HOW == kNeighbours && E == 1 ? 2 * j : j * E;
    };
    const int second = HOW == kNeighbours ? 1 : half;
    struct Piece {
        Raw<T, E> a, b;
    };
    auto load = [&](const Walk &v, Piece &p) {
        if (v.row >= rows) return;
        const T *at = x + v.row * a.ldx + (int64_t)v.head * a.head_dim + column(v.j);
        p.a = load_raw<T, E, AL>(at);
        if (TWO && v.j < turning) p.b = load_raw<T, E, AL>(at + second);
    };
    // The turns of a piece lie apart by the number of pieces, two of them in 16
    // bytes, so that neighbouring lanes read neighbouring 16 bytes.
    auto turn_at = [&](int row, int piece, int i) -> float2 * {
        if constexpr (P == 1) return turn + row * half + piece;
        else return turn + row * half + 2 * ((i >> 1) * half_pieces + piece) + (i & 1);
    };
    const bool power = (half_pieces & (half_pieces - 1)) == 0 && lanes % (2 * half_pieces) == 0;
    auto finish = [&](const Walk &v, const Piece &p) {
        Raw<T, E> other = p.a;
        const bool upper = HOW == kSwap && v.j >= half_pieces;
        if constexpr (HOW == kSwap) {
            // for all lanes: a head's lanes are all here or all past the rows
            const int from = v.j < turning ? (upper ? lane - half_pieces : lane + half_pieces) : lane;
#pragma unroll
            for (int i = 0; i < Raw<T, E>::words; ++i) {
                const float mine = __uint_as_float(p.a.w[i]);
                other.w[i] = __float_as_uint(power && half_pieces == 8    ? xor_lane<8>(mine, lane)
                                             : power && half_pieces == 16 ? xor_lane<16>(mine, lane)
                                             : power && half_pieces == 4  ? xor_lane<4>(mine, lane)
                                                                          : __shfl(mine, from));
            }
        }
        if (v.row >= rows) return;
        T *at = out + v.row * a.ldo + (int64_t)v.head * a.head_dim + column(v.j);
        if (v.j >= turning) {
            store_raw<T, E, AL>(at, p.a);
            return;
        }
        const int piece = upper ? v.j - half_pieces : v.j;
        float u[E], z[E], r[E], q[E];
        unpack<T, E>(p.a, u);
        if constexpr (HOW == kNeighbours && E > 1) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 t = *turn_at(v.row, piece, i);
                r[2 * i] = fmaf(u[2 * i], t.x, -(u[2 * i + 1] * t.y));
                r[2 * i + 1] = fmaf(u[2 * i + 1], t.x, u[2 * i] * t.y);
            }
        } else if constexpr (HOW == kSwap) {
            unpack<T, E>(other, z);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float2 t = *turn_at(v.row, piece, i);
                const float s = z[i] * t.y;
                r[i] = fmaf(u[i], t.x, upper ? s : -s);
            }
        } else {
            unpack<T, E>(p.b, z);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float2 t = *turn_at(v.row, piece, i);
                r[i] = fmaf(u[i], t.x, -(z[i] * t.y));
                q[i] = fmaf(z[i], t.x, u[i] * t.y);
            }
            store_run<T, E, AL>(at + second, q);
        }
        store_run<T, E, AL>(at, r);
    };
    Walk ahead[kAhead];
    Piece p[kAhead];
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ahead[i] = w, load(w, p[i]), advance(w);
    };
    fetch();
    for (int i = tid; i < rows * half; i += kThreads) {
        const int r = i / half, k = i - r * half, ax = a.axis ? a.axis[k] : 0;
        const double pos = (unsigned)ax < (unsigned)a.axes ? (double)a.positions[(int64_t)ax * a.ldp + first + r] : 0.0;
        const float2 t = cos_sin(pos * a.freq[k]);
        *turn_at(r, k / P, k % P) = make_float2(t.x * a.cos_scale, t.y * a.sin_scale);
    }
    lds_barrier();
    // a wave stays until its last lane is done (it swaps with the others)
    while (__any(ahead[0].row < rows)) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) finish(ahead[i], p[i]);
        fetch();
    }
}

template <typename T, int E> hipError_t rope_go(const RopeLaunch &a, bool aligned, hipStream_t stream)
{
    const int half = a.rotary / 2, whole = a.head_dim / E;
    const int how = a.pairs ? kNeighbours : E > 1 && whole <= 64 ? kSwap : kBoth;
    const int per = how == kBoth || E == 1 ? half / E + (a.head_dim - a.rotary) / E : whole;
    // rows of a workgroup: about four pieces to a thread, but no fewer than 512 workgroups
    int64_t each = std::max<int64_t>(1, std::min<int64_t>(4 * kThreads / ((int64_t)a.heads * per), kTurns / half));
    each = std::max<int64_t>(1, std::min<int64_t>(each, a.rows / 512));
    const int64_t most = most_workgroups(kThreads) * each;
    for (int64_t row0 = 0; row0 < a.rows; row0 += most) {
        const unsigned groups = (unsigned)((std::min<int64_t>(most, a.rows - row0) + each - 1) / each);
        auto go = [&](auto kernel) { kernel<<<groups, kThreads, 0, stream>>>(a, row0, (int)each); };
        if (how == kNeighbours) aligned ? go(rope_kernel<T, E, kNeighbours, true>) : go(rope_kernel<T, E, kNeighbours, false>);
        else if (how == kBoth) aligned ? go(rope_kernel<T, E, kBoth, true>) : go(rope_kernel<T, E, kBoth, false>);
        else if constexpr (E > 1) aligned ? go(rope_kernel<T, E, kSwap, true>) : go(rope_kernel<T, E, kSwap, false>);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// The widest pieces that a head and its halves are made of.
template <typename T> hipError_t rope_width(const RopeLaunch &a, hipStream_t stream)
{
    constexpr int E = 16 / (int)sizeof(T);
    const int fit = a.head_dim | a.rotary | (a.pairs ? 0 : a.rotary / 2);
    const bool aligned = ((uintptr_t)a.x | (uintptr_t)a.out) % 16 == 0 && a.ldx % E == 0 && a.ldo % E == 0;
    if (fit % E == 0) return rope_go<T, E>(a, aligned, stream);
    if (E > 4 && fit % 4 == 0) return rope_go<T, 4>(a, aligned, stream);
    if (fit % 2 == 0) return rope_go<T, 2>(a, aligned, stream);
    return rope_go<T, 1>(a, aligned, stream);
}

}  // namespace

hipError_t launch_rope(const RopeLaunch &a, hipStream_t stream)
{
    return a.x_dt == 0 ? rope_width<float>(a, stream) : rope_width<bf16_bits>(a, stream);
}

}  // namespace nqk
