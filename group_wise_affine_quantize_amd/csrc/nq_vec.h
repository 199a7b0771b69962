// Runs of E neighbouring elements as fp32, moved by the widest accesses that
// their size has.  AL: runs start at multiples of 16 bytes (or of their size);
// without it they only have to be aligned to their elements, which the memory
// takes as one access all the same (unaligned access is this target's mode), at
// the price of a second line now and then: 1501 rows of 1407 fp32 numbers 11.4 us
// instead of 13.8 with an access for each element.
#pragma once

#include <type_traits>

#include "nq_device.h"

namespace nqk {

typedef uint32_t words4 __attribute__((ext_vector_type(4)));
typedef uint32_t words2 __attribute__((ext_vector_type(2)));
typedef words4 loose4 __attribute__((aligned(2)));
typedef words2 loose2 __attribute__((aligned(2)));
typedef uint32_t loose1 __attribute__((aligned(2)));

// E elements as they lie in memory.
template <typename T, int E> struct Raw {
    static constexpr int bytes = E * (int)sizeof(T), words = bytes < 4 ? 1 : bytes / 4;
    uint32_t w[words];
};

// ONCE: an access of 16 bytes that is not kept in the caches (where runs are
// aligned: others share lines with their neighbours, 25 -> 30 us for a gradient
// of 1501 rows of 1407).
template <typename T, int E, bool AL = true, bool ONCE = false> __device__ __forceinline__ Raw<T, E> load_raw(const T *p)
{
    using W4 = std::conditional_t<AL, words4, loose4>;
    using W2 = std::conditional_t<AL, words2, loose2>;
    using W1 = std::conditional_t<AL, uint32_t, loose1>;
    Raw<T, E> r;
    if constexpr (Raw<T, E>::bytes % 16 == 0) {
#pragma unroll
        for (int i = 0; i < Raw<T, E>::words / 4; ++i) {
            words4 v;
            if constexpr (ONCE && AL) v = __builtin_nontemporal_load(reinterpret_cast<const W4 *>(p) + i);
            else v = reinterpret_cast<const W4 *>(p)[i];
            r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
        }
    } else if constexpr (Raw<T, E>::bytes == 8) {
        const words2 v = *reinterpret_cast<const W2 *>(p);
        r.w[0] = v.x, r.w[1] = v.y;
    } else if constexpr (Raw<T, E>::bytes == 4) r.w[0] = *reinterpret_cast<const W1 *>(p);
    else r.w[0] = *reinterpret_cast<const uint16_t *>(p);
    return r;
}

template <typename T, int E, bool AL = true, bool ONCE = false> __device__ __forceinline__ void store_raw(T *p, const Raw<T, E> &r)
{
    using W4 = std::conditional_t<AL, words4, loose4>;
    using W2 = std::conditional_t<AL, words2, loose2>;
    using W1 = std::conditional_t<AL, uint32_t, loose1>;
    if constexpr (Raw<T, E>::bytes % 16 == 0) {
#pragma unroll
        for (int i = 0; i < Raw<T, E>::words / 4; ++i) {
            const W4 v = words4{r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
            if constexpr (ONCE && AL) __builtin_nontemporal_store(v, reinterpret_cast<W4 *>(p) + i);
            else reinterpret_cast<W4 *>(p)[i] = v;
        }
    } else if constexpr (Raw<T, E>::bytes == 8) *reinterpret_cast<W2 *>(p) = words2{r.w[0], r.w[1]};
    else if constexpr (Raw<T, E>::bytes == 4) *reinterpret_cast<W1 *>(p) = r.w[0];
    else *reinterpret_cast<uint16_t *>(p) = (uint16_t)r.w[0];
}

template <typename T, int E> __device__ __forceinline__ Raw<T, E> raw_zero()
{
    Raw<T, E> r;
#pragma unroll
    for (int i = 0; i < Raw<T, E>::words; ++i) r.w[i] = 0u;
    return r;
}

template <typename T, int E> __device__ __forceinline__ void unpack(const Raw<T, E> &r, float *v)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = __uint_as_float(r.w[i]);
    } else if constexpr (E == 1) v[0] = __uint_as_float(r.w[0] << 16);
    else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            v[2 * i] = __uint_as_float(r.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
        }
    }
}

// Rounded to nearest, ties to even; a NaN stays one.
template <typename T, int E> __device__ __forceinline__ Raw<T, E> pack(const float *v)
{
    Raw<T, E> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < E; ++i) r.w[i] = __float_as_uint(v[i]);
    } else if constexpr (E == 1) r.w[0] = f32_to_bf16(v[0]);
    else {
        typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const bf2 b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
            r.w[i] = __builtin_bit_cast(uint32_t, b);
        }
    }
    return r;
}

template <typename T, int E, bool AL = true> __device__ __forceinline__ void store_run(T *p, const float *v)
{
    store_raw<T, E, AL>(p, pack<T, E>(v));
}

// Columns c .. c + E - 1 of a row of `dim`; what lies behind the row reads as
// zeros and is not written.  With AL, dim is a multiple of E.
template <typename T, int E, bool AL, bool ONCE = false> __device__ __forceinline__ Raw<T, E> load_cols(const T *row, int64_t c, int64_t dim)
{
    if (c + E <= dim) return load_raw<T, E, AL, ONCE>(row + c);
    Raw<T, E> r = raw_zero<T, E>();
    if constexpr (!AL && E > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (c + e < dim) {
                if constexpr (sizeof(T) == 4) r.w[e] = reinterpret_cast<const uint32_t *>(row)[c + e];
                else r.w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[c + e] << (16 * (e & 1));
            }
    }
    return r;
}
template <typename T, int E, bool AL, bool ONCE = false>
__device__ __forceinline__ void store_cols(T *row, int64_t c, int64_t dim, const Raw<T, E> &r)
{
    if (c + E <= dim) store_raw<T, E, AL, ONCE>(row + c, r);
    else if constexpr (!AL && E > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (c + e < dim) {
                if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t *>(row)[c + e] = r.w[e];
                else reinterpret_cast<uint16_t *>(row)[c + e] = (uint16_t)(r.w[e / 2] >> (16 * (e & 1)));
            }
    }
}

// The sum over the first LANES lanes' group of each lane (LANES a power of two).
template <int LANES> __device__ __forceinline__ float lane_sum(float v, int lane)
{
    if constexpr (LANES > 1) v += xor_lane<1>(v, lane);
    if constexpr (LANES > 2) v += xor_lane<2>(v, lane);
    if constexpr (LANES > 4) v += xor_lane<4>(v, lane);
    if constexpr (LANES > 8) v += xor_lane<8>(v, lane);
    if constexpr (LANES > 16) v += xor_lane<16>(v, lane);
    if constexpr (LANES > 32) v += xor_lane<32>(v, lane);
    return v;
}

}  // namespace nqk
