// Device helpers of the key/value cache kernels: the geometry of a call's
// sequences and the 8-bit encodings.
#pragma once

#include "nq_device.h"
#include "nq_kv.h"
#include "nq_kv_list.h"

namespace nqk {

// Smallest non-zero scale of a block: below it, values become zero codes and
// the reciprocals taken of scales stay finite and normal.
constexpr float kKvMinScale = 0x1p-100f;
// Growth past which a held block's older codes all round to zero.
constexpr float kKvGrowLimit = 0x1p20f;

template <int FMT> struct KvFmt;
template <> struct KvFmt<KV_INT8> {
    static constexpr float qmax = 127.0f;
    static constexpr uint32_t zero4 = 0x80808080u;   // four zero codes
};
template <> struct KvFmt<KV_FP8> {
    static constexpr float qmax = 448.0f;
    static constexpr uint32_t zero4 = 0u;
};

// What a code stands for, in units of the block's scale: code - 128, or the
// E4M3 number (bias 7; S.1111.111 is NaN).
template <int FMT> __device__ __forceinline__ float kv_value(uint32_t code)
{
    if constexpr (FMT == KV_INT8) return (float)(int)code - 128.0f;
    else {
        const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)code, 1.0f, false);
        return p[0];
    }
}

// Four codes of one word -> four fp32 values.
template <int FMT> __device__ __forceinline__ void kv_values4(uint32_t w, float *v)
{
    if constexpr (FMT == KV_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int)((w >> (8 * i)) & 255u) - 128.0f;
    } else {
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w, 1.0f, false);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w, 1.0f, true);
        v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
    }
}

// Four fp32 values in units of the scale -> four codes: nearest, ties to
// even, clamped to +-qmax.
template <int FMT> __device__ __forceinline__ uint32_t kv_codes4(const float *v)
{
    constexpr float q = KvFmt<FMT>::qmax;
    if constexpr (FMT == KV_INT8) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float r = fminf(fmaxf(rintf(v[i]), -q), q);
            w |= (uint32_t)((int)r + 128) << (8 * i);
        }
        return w;
    } else {
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(v[i], -q), q);
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
        return (uint32_t)w;
    }
}

template <int FMT> __device__ __forceinline__ uint8_t kv_code(float v)
{
    const float t[4] = {v, 0.0f, 0.0f, 0.0f};
    return (uint8_t)(kv_codes4<FMT>(t) & 255u);
}

// The larger magnitude, an infinity or a NaN above every number.
__device__ __forceinline__ float larger(float top, float v)
{
    const uint32_t a = __float_as_uint(top), b = __float_as_uint(v) & 0x7fffffffu;
    return __uint_as_float(a > b ? a : b);
}

// One sequence of a call, every value clamped: rows r0 .. r0 + n of the call
// are its tokens first .. len (first may be negative: such rows have no
// token).
struct KvSeq {
    int64_t r0, n, len, first;
};

__device__ __forceinline__ KvSeq kv_seq(const KvSeqs &s, int b)
{
    KvSeq q;
    int64_t a = s.row_start[b], e = s.row_start[b + 1];
    a = a < 0 ? 0 : (a > s.rows ? s.rows : a);
    e = e < a ? a : (e > s.rows ? s.rows : e);
    const int64_t len = s.lengths[b];
    q.r0 = a;
    q.n = e - a;
    q.len = len < 0 ? 0 : len;
    q.first = q.len - q.n;
    return q;
}

// The id of block j of sequence b, or -1 where the table or the cache has no
// such block.
__device__ __forceinline__ int64_t kv_block(const KvSeqs &s, int64_t blocks, int b, int64_t j)
{
    if (j < 0 || j >= s.max_blocks) return -1;
    const int64_t id = s.table[(int64_t)b * s.ldt + j];
    return id < 0 || id >= blocks ? -1 : id;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// The same over 32 bits, by lane shifts inside rows of 16 and row broadcasts.
__device__ __forceinline__ uint32_t wave_scan32(uint32_t v)
{
    auto add = [&](int o) { v += (uint32_t)o; };
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true));    // row_shr:1
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true));
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true));
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true));
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row 0 -> 1, 2 -> 3
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // rows 0, 1 -> 2, 3
    return v;
}

// The same, of sums that stay at 2^32 - 1 when they pass it.
__device__ __forceinline__ uint32_t wave_scan32_sat(uint32_t v)
{
    auto add = [&](int o) { v = add_sat(v, (uint32_t)o); };
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true));
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true));
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true));
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true));
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));
    return v;
}

// Finds, for a wave, which sequence holds item `item` when sequence b has
// count(b) items, and the item's number in it; -1 when there is none.  Lanes
// look at 64 sequences at a time.
template <typename Count>
__device__ __forceinline__ int kv_locate(int batch, int64_t item, Count count, int64_t *inside)
{
    const int lane = (int)(threadIdx.x & 63u);
    int64_t base = 0;
    for (int b0 = 0; b0 < batch; b0 += 64) {
        const int b = b0 + lane;
        const int64_t c = b < batch ? count(b) : 0;
        const int64_t upto = wave_scan(c, lane);
        const uint64_t hit = __ballot(base + upto > item);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            *inside = item - base - __shfl(upto - c, l);
            return b0 + l;
        }
        base += __shfl(upto, 63);
    }
    return -1;
}

}  // namespace nqk
