// What the attention kernels over the 8-bit cache share (kv_attention.hip,
// kv_prefill.hip): the geometry of a call, code conversion and fp16 operands.
// The mathematics is at the head of kv_attention.hip.
#pragma once

#include "nq_kv_device.h"

namespace nqk {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;        // tokens per tile
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kPScale = 14.0f;  // log2 of the largest weight
// Value scales with which L can share O's reference: 2^-48 .. 2^16 (see the head
// of kv_attention.hip).  One comparison of their bits, taken from the lower
// end, finds zeros too.
constexpr uint32_t kNearScales = ((uint32_t)(48 + 16) << 23) + 1;
__device__ __forceinline__ uint32_t scale_place(float s) { return __float_as_uint(s) - ((127u - 48u) << 23); }

constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_log2(float x) { return __builtin_amdgcn_logf(x); }

// Eight codes (two words) -> eight fp16 values, exactly.
template <int FMT> __device__ __forceinline__ half8_t codes_to_half(uint32_t w0, uint32_t w1)
{
    uint32_t p[4];
    if constexpr (FMT == KV_INT8) {
        // 0x6400 | c is fp16 1024 + c; less 1152 it is c - 128
        p[0] = __builtin_amdgcn_perm(0x64646464u, w0, 0x04010400u);
        p[1] = __builtin_amdgcn_perm(0x64646464u, w0, 0x04030402u);
        p[2] = __builtin_amdgcn_perm(0x64646464u, w1, 0x04010400u);
        p[3] = __builtin_amdgcn_perm(0x64646464u, w1, 0x04030402u);
        const half2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const half2_t h = __builtin_bit_cast(half2_t, p[i]) - off;
            p[i] = __builtin_bit_cast(uint32_t, h);
        }
    } else {
        p[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w0, 1.0f, false));
        p[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w0, 1.0f, true));
        p[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w1, 1.0f, false));
        p[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w1, 1.0f, true));
    }
    const uint4_t v = {p[0], p[1], p[2], p[3]};
    return __builtin_bit_cast(half8_t, v);
}

// Parts of fp32 numbers in fp16: one for bf16 queries, two for fp32 ones.
template <typename T> struct Parts { static constexpr int n = 2; };
template <> struct Parts<bf16_bits> { static constexpr int n = 1; };

template <int NP> __device__ __forceinline__ void split_half(const float *v, half8_t *h)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const _Float16 a = (_Float16)v[i];
        h[0][i] = a;
        if constexpr (NP == 2) h[1][i] = (_Float16)(v[i] - (float)a);
    }
}

__device__ __forceinline__ float4_t mfma(half8_t a, half8_t b, float4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

struct AttnArgs {
    KvAttnLaunch a;
    float *part_o;      // [workers * 2][columns][D]
    float4 *part_s;     // [workers * 2][columns] of R, L, U
    int workers;        // workgroups of the streaming kernel
    int group;          // query heads per key/value head
    int unit_shift;     // log2 of the tiles of a unit of work
    bool splits;        // whether a segment can have more than one unit
    int few;            // sequences of at most `few` query columns per head are the
                        // streaming kernel's, the others the tile kernel's
    int tile_splits;    // parts that the tile kernel cuts a segment's tokens into
    unsigned tile_bound;    // tile kernel: column tiles at most, over all sequences
};

// The streaming kernel's work is a flat list of units (runs of 64-token
// tiles): for each sequence with rows, for each key/value head and each tile
// of `cols` query rows (a row is a token and one of the head's queries) -- a
// segment -- the units of the tokens that the sequence's rows can see.  Every
// worker takes an equal run of the list, whatever the lengths.
struct StreamSeq {
    int r0, n, first, len;  // rows of the call, tokens (see KvSeq)
    int lo, hi;             // tokens that some row sees (hi <= lo: none)
    int t0, nt;             // first tile, tiles (at least one)
    uint32_t ct;            // column tiles
    uint32_t units;         // per segment
    uint32_t work;          // units of all segments
};

__device__ __forceinline__ StreamSeq stream_seq(const AttnArgs &A, int b, int cols)
{
    const KvAttnLaunch &a = A.a;
    const KvSeq q = kv_seq(a.s, b);
    StreamSeq s;
    s.r0 = (int)q.r0, s.n = (int)q.n, s.first = (int)q.first, s.len = (int)q.len;
    const int cap = (int)(a.s.max_blocks << a.c.block_shift);
    s.hi = s.len < cap ? s.len : cap;
    s.lo = 0;
    if (a.window > 0) {
        const int64_t lo = q.first - a.window + 1;
        s.lo = lo < 0 ? 0 : (int)lo;
    }
    s.t0 = s.lo >> 6;
    s.nt = s.hi > s.lo ? ((s.hi + 63) >> 6) - s.t0 : 1;
    s.ct = s.n * A.group <= A.few ? (uint32_t)(s.n * A.group + cols - 1) / (uint32_t)cols : 0u;
    s.units = (uint32_t)(s.nt + (1 << A.unit_shift) - 1) >> A.unit_shift;
    s.work = s.ct * s.units * (uint32_t)a.c.kv_heads;
    return s;
}

// Where a query column stands: its row of the call, head, and the tokens that
// it sees, [lo, hi).
struct Column {
    int row;            // -1: no such column
    int head;
    int lo, hi;
};

__device__ __forceinline__ Column column(const AttnArgs &A, const StreamSeq &s, int idx, int kv_head)
{
    const KvAttnLaunch &a = A.a;
    Column c;
    c.row = -1, c.head = 0, c.lo = 0, c.hi = 0;
    if (idx < s.n * A.group) {
        const int i = (int)((uint32_t)idx / (uint32_t)A.group);
        c.row = s.r0 + i;
        c.head = kv_head * A.group + (idx - i * A.group);
        const int pos = s.first + i;
        c.hi = a.causal && pos < s.hi ? pos + 1 : s.hi;
        if (a.window > 0) {
            const int64_t lo = (int64_t)pos - a.window + 1;
            c.lo = lo < 0 ? 0 : (int)lo;
        }
    }
    return c;
}

// Eight neighbouring elements, from the 16-byte words that hold them.
template <typename T> __device__ __forceinline__ void unpack_f32x8(const uint4 *w, float *v);
template <> __device__ __forceinline__ void unpack_f32x8<float>(const uint4 *w, float *v)
{
    const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
}
template <> __device__ __forceinline__ void unpack_f32x8<bf16_bits>(const uint4 *w, float *v)
{
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
template <typename T> __device__ __forceinline__ void load_f32x8(const T *p, float *v)
{
    uint4 w[8 * sizeof(T) / 16];
#pragma unroll
    for (int i = 0; i < (int)(8 * sizeof(T) / 16); ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
    unpack_f32x8<T>(w, v);
}

template <typename T> __device__ __forceinline__ void store_f32x4(T *p, const float *v);
template <> __device__ __forceinline__ void store_f32x4<float>(float *p, const float *v)
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <> __device__ __forceinline__ void store_f32x4<bf16_bits>(bf16_bits *p, const float *v)
{
    // the hardware's conversion: nearest, ties to even, NaN stays one
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 a = {(__bf16)v[0], (__bf16)v[1]}, b = {(__bf16)v[2], (__bf16)v[3]};
    uint2 w;
    w.x = __builtin_bit_cast(uint32_t, a);
    w.y = __builtin_bit_cast(uint32_t, b);
    *reinterpret_cast<uint2 *>(p) = w;
}

// A row's power of two: f * 2^k has its largest element in [2^14, 2^15).
// Returns 2^k; *back is 2^-k.  A row that holds an infinity or a NaN gets a
// NaN, and with it every score that a token gives it.
__device__ __forceinline__ float row_scale(float largest, float *back)
{
    int e = (int)(__float_as_uint(largest) >> 23) & 255;   // biased exponent
    if (e == 255) return *back = __builtin_nanf("");
    e = e < 27 ? 27 : e;                                    // both powers stay normal
    *back = __uint_as_float((uint32_t)(e - 14) << 23);
    return __uint_as_float((uint32_t)(254 + 14 - e) << 23);
}

__device__ __forceinline__ float group_max(float v, int lane)   // over the four lanes of a column
{
    v = fmaxf(v, xor_lane<16>(v, lane));
    return fmaxf(v, xor_lane<32>(v, lane));
}
__device__ __forceinline__ float group_sum(float v, int lane)
{
    v += xor_lane<16>(v, lane);
    return v + xor_lane<32>(v, lane);
}

__device__ __forceinline__ float wave_max(float v, int lane)
{
    v = fmaxf(v, xor_lane<1>(v, lane));
    v = fmaxf(v, xor_lane<2>(v, lane));
    v = fmaxf(v, xor_lane<4>(v, lane));
    v = fmaxf(v, xor_lane<8>(v, lane));
    return group_max(v, lane);
}

// 2^(a - b), where a is at most b and -infinity stands for nothing: 0 then.
__device__ __forceinline__ float exp2_below(float a, float b) { return a == kNegInf ? 0.0f : fast_exp2(a - b); }

// Adds `count` tokens with scores z (base 2, -infinity where hidden) to l, the
// sum of 2^z over 2^u; u moves to their maximum when that is larger.
template <typename Score>
__device__ __forceinline__ void add_weights(int count, Score z, float &l, float &u)
{
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < count; ++i) top = fmaxf(top, z(i));
    const float at = top == kNegInf ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < count; ++i) sum += fast_exp2(z(i) - at);
    const float next = fmaxf(u, top);
    l = fmaf(l, exp2_below(u, next), sum * (top == kNegInf ? 1.0f : fast_exp2(top - next)));
    u = next;
}

// O / L, with O over 2^m and L over 2^u: returns O's factor, zero where no
// token was seen.  Where the references differ, half of 2^(m - u) goes into
// the `count` numbers o here: the whole of it can pass fp32 by itself.
__device__ __forceinline__ float out_factor(float l, float m, float u, int count, float *o)
{
    float f = l == 0.0f ? 0.0f : 1.0f / l;      // a NaN stays one
    if (__any(m != u)) {
        const float half = l == 0.0f ? 0.0f : fast_exp2(0.5f * (m - u));
#pragma unroll
        for (int i = 0; i < count; ++i) o[i] *= half;
        f *= half;
    }
    return f;
}

// log of the sum of weights l over 2^u: -infinity for none, NaN for a NaN.
__device__ __forceinline__ float log_sum(float l, float u) { return l == 0.0f ? kNegInf : (u + fast_log2(l)) * kLn2; }

// The tile kernel (kv_prefill.hip).
int prefill_columns(const KvAttnLaunch &a);     // query columns per workgroup
hipError_t launch_kv_prefill(const AttnArgs &A, hipStream_t stream);

}  // namespace nqk
