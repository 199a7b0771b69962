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
// What bounds it: reading and writing the heads once.
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

// A piece of a head: E columns of both halves, E neighbouring columns that
// are whole pairs, or E columns that are only copied.
template <typename T, int E> struct Piece {
    Raw<T, E> a, b;     // b: of the second half, or a pair's second element
};

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
template <typename T, int E, bool PAIRS, bool AL>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeLaunch a, int64_t row0, int rows_each)
{
    constexpr int kAhead = 4, P = E == 1 ? 1 : PAIRS ? E / 2 : E;   // pairs of a piece
    __shared__ float2 turn[kTurns];
    const int half = a.rotary >> 1, tid = (int)threadIdx.x;
    const int64_t first = row0 + (int64_t)blockIdx.x * rows_each;
    const int rows = a.rows - first < rows_each ? (int)(a.rows - first) : rows_each;
    const T *x = static_cast<const T *>(a.x) + first * a.ldx;
    T *out = static_cast<T *>(a.out) + first * a.ldo;
    // pieces of a head: those that turn, then those that are copied
    const int turning = half / P, per = turning + (a.x == a.out ? 0 : (a.head_dim - a.rotary) / E);
    const int lanes = per < kThreads ? per : kThreads, side = kThreads / lanes, mine = tid / lanes;
    Walk w{0, mine, tid - mine * lanes};
    w.carry(a.heads);
    if (mine >= side) w.row = rows;     // no place for another head
    const int start = w.j;
    auto advance = [&](Walk &v) {
        v.j += lanes;
        if (v.j >= per) v.j = start, v.head += side, v.carry(a.heads);
    };
    auto load = [&](const Walk &v, Piece<T, E> &p) {
        if (v.row >= rows) return;
        const T *at = x + v.row * a.ldx + (int64_t)v.head * a.head_dim;
        if (v.j >= turning) p.a = load_raw<T, E, AL>(at + a.rotary + (v.j - turning) * E);
        else if (PAIRS && E > 1) p.a = load_raw<T, E, AL>(at + v.j * E);
        else if (PAIRS) p.a = load_raw<T, E, AL>(at + 2 * v.j), p.b = load_raw<T, E, AL>(at + 2 * v.j + 1);
        else p.a = load_raw<T, E, AL>(at + v.j * E), p.b = load_raw<T, E, AL>(at + half + v.j * E);
    };
    auto finish = [&](const Walk &v, const Piece<T, E> &p) {
        if (v.row >= rows) return;
        T *at = out + v.row * a.ldo + (int64_t)v.head * a.head_dim;
        const float2 *t = turn + v.row * half + v.j * P;
        if (v.j >= turning) store_raw<T, E, AL>(at + a.rotary + (v.j - turning) * E, p.a);
        else if constexpr (PAIRS && E > 1) {
            float u[E], r[E];
            unpack<T, E>(p.a, u);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                r[2 * e] = fmaf(u[2 * e], t[e].x, -(u[2 * e + 1] * t[e].y));
                r[2 * e + 1] = fmaf(u[2 * e + 1], t[e].x, u[2 * e] * t[e].y);
            }
            store_run<T, E, AL>(at + v.j * E, r);
        } else {
            float u[E], z[E], r[E], q[E];
            unpack<T, E>(p.a, u), unpack<T, E>(p.b, z);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                r[e] = fmaf(u[e], t[e].x, -(z[e] * t[e].y));
                q[e] = fmaf(z[e], t[e].x, u[e] * t[e].y);
            }
            store_run<T, E, AL>(at + (PAIRS ? 2 * v.j : v.j * E), r);
            store_run<T, E, AL>(at + (PAIRS ? 2 * v.j + 1 : half + v.j * E), q);
        }
    };
    Walk ahead[kAhead];
    Piece<T, E> p[kAhead];
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ahead[i] = w, load(w, p[i]), advance(w);
    };
    fetch();
    for (int i = tid; i < rows * half; i += kThreads) {
        const int r = i / half, k = i - r * half, ax = a.axis ? a.axis[k] : 0;
        const double pos = (unsigned)ax < (unsigned)a.axes ? (double)a.positions[(int64_t)ax * a.ldp + first + r] : 0.0;
        const float2 t = cos_sin(pos * a.freq[k]);
        turn[i] = make_float2(t.x * a.cos_scale, t.y * a.sin_scale);
    }
    lds_barrier();
    while (ahead[0].row < rows) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) finish(ahead[i], p[i]);
        fetch();
    }
}

template <typename T, int E> hipError_t rope_go(const RopeLaunch &a, bool aligned, hipStream_t stream)
{
    const int half = a.rotary / 2, per = a.pairs && E > 1 ? a.head_dim / E : half / E + (a.head_dim - a.rotary) / E;
    // rows of a workgroup: about four pieces to a thread, but no fewer than 512 workgroups
    int64_t each = std::max<int64_t>(1, std::min<int64_t>(4 * kThreads / ((int64_t)a.heads * per), kTurns / half));
    each = std::max<int64_t>(1, std::min<int64_t>(each, a.rows / 512));
    const int64_t most = most_workgroups(kThreads) * each;
    for (int64_t row0 = 0; row0 < a.rows; row0 += most) {
        const unsigned groups = (unsigned)((std::min<int64_t>(most, a.rows - row0) + each - 1) / each);
        auto go = [&](auto kernel) { kernel<<<groups, kThreads, 0, stream>>>(a, row0, (int)each); };
        if (a.pairs) aligned ? go(rope_kernel<T, E, true, true>) : go(rope_kernel<T, E, true, false>);
        else aligned ? go(rope_kernel<T, E, false, true>) : go(rope_kernel<T, E, false, false>);
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
