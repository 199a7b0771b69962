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
// all of the row's heads use it, out of LDS.
//
// What bounds it: reading and writing the heads once.
#include <algorithm>

#include "nq_kv.h"
#include "nq_layer.h"
#include "nq_vec.h"

namespace nqk {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;      // head_dim up to 1024

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

// A workgroup takes one row, of which each thread takes the same columns of
// every few heads.  E: elements of an access (1: pairs of single elements).
template <typename T, int E> __global__ __launch_bounds__(kThreads) void rope_kernel(RopeLaunch a, int64_t row0)
{
    __shared__ float2 turn[kMaxPairs];
    const int64_t row = row0 + blockIdx.x;
    const int half = a.rotary >> 1, tid = (int)threadIdx.x;
    for (int i = tid; i < half; i += kThreads) {
        const int ax = a.axis ? a.axis[i] : 0;
        const double p = (unsigned)ax < (unsigned)a.axes ? (double)a.positions[(int64_t)ax * a.ldp + row] : 0.0;
        const float2 t = cos_sin(p * a.freq[i]);
        turn[i] = make_float2(t.x * a.cos_scale, t.y * a.sin_scale);
    }
    __syncthreads();
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    T *out = static_cast<T *>(a.out) + row * a.ldo;
    // pieces of a head: those that turn, then those that are copied
    constexpr int P = E == 1 ? 1 : E / 2;       // pairs of a piece of neighbouring pairs
    const int turning = a.pairs ? half / P : half / E;
    const int behind = a.x == a.out ? 0 : (a.head_dim - a.rotary) / E;
    const int per = turning + behind;
    const int count = a.heads * per;
    for (int item = tid + (int)blockIdx.y * kThreads; item < count; item += kThreads * (int)gridDim.y) {
        const int head = (int)((unsigned)item / (unsigned)per), j = item - head * per;
        const int64_t at = (int64_t)head * a.head_dim;
        if (j >= turning) {
            const int64_t c = at + a.rotary + (j - turning) * E;
            store_raw<T, E>(out + c, load_raw<T, E>(x + c));
        } else if (!a.pairs) {
            float u[E], v[E], p[E], q[E];
            load_run<T, E>(x + at + j * E, u);
            load_run<T, E>(x + at + half + j * E, v);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float2 t = turn[j * E + e];
                p[e] = fmaf(u[e], t.x, -(v[e] * t.y));
                q[e] = fmaf(v[e], t.x, u[e] * t.y);
            }
            store_run<T, E>(out + at + j * E, p);
            store_run<T, E>(out + at + half + j * E, q);
        } else {
            constexpr int W = 2 * P;
            float u[W], p[W];
            if constexpr (E == 1) u[0] = Elt<T>::load(x, at + 2 * j), u[1] = Elt<T>::load(x, at + 2 * j + 1);
            else load_run<T, W>(x + at + j * W, u);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 t = turn[j * P + e];
                p[2 * e] = fmaf(u[2 * e], t.x, -(u[2 * e + 1] * t.y));
                p[2 * e + 1] = fmaf(u[2 * e + 1], t.x, u[2 * e] * t.y);
            }
            if constexpr (E == 1) Elt<T>::store(out, at + 2 * j, p[0]), Elt<T>::store(out, at + 2 * j + 1, p[1]);
            else store_run<T, W>(out + at + j * W, p);
        }
    }
}

template <typename T> hipError_t rope_go(const RopeLaunch &a, hipStream_t stream)
{
    constexpr int E = 16 / (int)sizeof(T);
    const int half = a.rotary / 2;
    const bool wide = (((uintptr_t)a.x | (uintptr_t)a.out) & 15) == 0 && a.ldx % E == 0 && a.ldo % E == 0 &&
                      a.head_dim % E == 0 && a.rotary % E == 0 && (a.pairs || half % E == 0);
    const int64_t most = most_workgroups(kThreads);
    for (int64_t row0 = 0; row0 < a.rows; row0 += most) {
        const unsigned rows = (unsigned)std::min<int64_t>(most, a.rows - row0);
        if (wide) rope_kernel<T, E><<<rows, kThreads, 0, stream>>>(a, row0);
        else rope_kernel<T, 1><<<rows, kThreads, 0, stream>>>(a, row0);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_rope(const RopeLaunch &a, hipStream_t stream)
{
    return a.x_dt == 0 ? rope_go<float>(a, stream) : rope_go<bf16_bits>(a, stream);
}

}  // namespace nqk
