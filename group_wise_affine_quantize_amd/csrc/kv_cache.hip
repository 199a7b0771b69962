// The 8-bit key/value cache: quantising new tokens into their blocks, and
// reading tokens back (contract in include/nq.h).
//
// Mathematics.  A block of B tokens of one head has one scale s; a value is
// s * c, c the code.  For the tokens that a call writes into a block, a = max
// |x| over them: a block whose first token they hold takes s = a / qmax; a
// block with older tokens keeps s while a <= qmax * s, else takes s * 2^j with
// the smallest j that holds a, and its older codes are rounded to the new
// scale.  Growing by powers of two bounds an old code's total error by one
// step of the last scale (each rounding adds half a step, and the steps at
// least double), where growing to a / qmax each time would let it drift.
//
// Both are bound by memory: a token of a head is read once and written once.
// One workgroup takes one block of one head, keys or values (the two have
// their own scales), so the scale is a workgroup's reduction and no two
// workgroups share a byte.
#include "nq_kv_device.h"

namespace nqk {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_max(float a, float *shared)
{
    const int lane = (int)(threadIdx.x & 63u);
    a = fmaxf(a, xor_lane<1>(a, lane));
    a = fmaxf(a, xor_lane<2>(a, lane));
    a = fmaxf(a, xor_lane<4>(a, lane));
    a = fmaxf(a, xor_lane<8>(a, lane));
    a = fmaxf(a, xor_lane<16>(a, lane));
    a = fmaxf(a, xor_lane<32>(a, lane));
    if (lane == 0) shared[threadIdx.x >> 6] = a;
    __syncthreads();
    return fmaxf(fmaxf(shared[0], shared[1]), fmaxf(shared[2], shared[3]));
}

// 2^-j and the grown scale for a held block; *shrink multiplies older codes.
template <int FMT> __device__ __forceinline__ float grown_scale(float s, float a, float fresh, float *shrink)
{
    *shrink = 1.0f;
    const float reach = s * KvFmt<FMT>::qmax;
    if (!(a > reach)) return s;
    const float ratio = a / reach;
    *shrink = 0.0f;
    if (s == 0.0f || ratio > kKvGrowLimit) return fresh;
    // smallest j with ratio <= 2^j, from the bits of ratio (1 < ratio <= 2^20)
    const uint32_t u = __float_as_uint(ratio);
    const int j = (int)(u >> 23) - 127 + ((u & 0x7fffffu) ? 1 : 0);
    *shrink = __uint_as_float((uint32_t)(127 - j) << 23);
    return s * __uint_as_float((uint32_t)(127 + j) << 23);
}

// Two neighbouring elements as fp32.
template <typename T> __device__ __forceinline__ float2 load2(const T *p);
template <> __device__ __forceinline__ float2 load2<float>(const float *p)
{
    return *reinterpret_cast<const float2 *>(p);
}
template <> __device__ __forceinline__ float2 load2<bf16_bits>(const bf16_bits *p)
{
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// Four neighbouring elements as fp32.
template <typename T> __device__ __forceinline__ float4 load4(const T *p);
template <> __device__ __forceinline__ float4 load4<float>(const float *p)
{
    return *reinterpret_cast<const float4 *>(p);
}
template <> __device__ __forceinline__ float4 load4<bf16_bits>(const bf16_bits *p)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
template <typename T> __device__ __forceinline__ void store4(T *p, const float *v);
template <> __device__ __forceinline__ void store4<float>(float *p, const float *v)
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <> __device__ __forceinline__ void store4<bf16_bits>(bf16_bits *p, const float *v)
{
    uint2 w;
    w.x = f32_to_bf16(v[0]) | f32_to_bf16(v[1]) << 16;
    w.y = f32_to_bf16(v[2]) | f32_to_bf16(v[3]) << 16;
    *reinterpret_cast<uint2 *>(p) = w;
}
template <typename T> __device__ __forceinline__ void store2(T *p, float a, float b);
template <> __device__ __forceinline__ void store2<float>(float *p, float a, float b)
{
    *reinterpret_cast<float2 *>(p) = make_float2(a, b);
}
template <> __device__ __forceinline__ void store2<bf16_bits>(bf16_bits *p, float a, float b)
{
    *reinterpret_cast<uint32_t *>(p) = f32_to_bf16(a) | f32_to_bf16(b) << 16;
}

// One block of one head that a call's rows touch.
struct Item {
    int64_t id;      // the block, or -1
    int64_t row;     // the call's row of the block's slot 0 (may lie before the sequence's rows)
    int lo, hi;      // slots lo .. hi - 1 hold the call's rows
};

__device__ __forceinline__ bool find_item(const KvSeqs &s, const KvCache &c, int64_t item, Item *out)
{
    int64_t j;
    const int sh = c.block_shift;
    const int b = kv_locate(s.batch, item, [&](int i) -> int64_t {
        const KvSeq q = kv_seq(s, i);
        return q.n > 0 ? ((q.len - 1) >> sh) - (q.first >> sh) + 1 : 0;
    }, &j);
    if (b < 0) return false;
    // a sequence with more rows than tokens starts in blocks below 0, which
    // no table has
    const KvSeq q = kv_seq(s, b);
    const int64_t blk = (q.first >> sh) + j, t0 = blk * ((int64_t)1 << sh);
    out->id = kv_block(s, c.blocks, b, blk);
    out->row = q.r0 + t0 - q.first;
    out->lo = (int)(q.first > t0 ? q.first - t0 : 0);
    out->hi = (int)(q.len - t0 < ((int64_t)1 << sh) ? q.len - t0 : ((int64_t)1 << sh));
    return true;
}

template <int FMT, typename T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendLaunch a)
{
    __shared__ float red[4];
    Item it;
    if (!find_item(a.s, a.c, blockIdx.x, &it) || it.id < 0) return;
    const int D = a.c.head_dim, sh = a.c.block_shift, B = 1 << sh, tid = (int)threadIdx.x;
    const int64_t head = blockIdx.y, slab = it.id * a.c.kv_heads + head;
    const bool is_v = blockIdx.z != 0;
    const int64_t ld = is_v ? a.ldv : a.ldk;
    const T *x = static_cast<const T *>(is_v ? a.v : a.k) + it.row * ld + head * D;
    uint8_t *codes = (is_v ? a.c.v_codes : a.c.k_codes) + slab * ((int64_t)D << sh);
    float *scale = (is_v ? a.c.v_scales : a.c.k_scales) + slab;
    const int count = it.hi - it.lo, quads = D >> 2;

    float m = 0.0f;
    for (int i = tid; i < count * quads; i += kThreads) {
        const int t = i / quads, d = (i - t * quads) * 4;
        const float4 v = load4<T>(x + (int64_t)(it.lo + t) * ld + d);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
    }
    const float held = it.lo > 0 ? *scale : 0.0f;   // read before thread 0 stores it below
    m = block_max(m, red);
    const float fresh = m > 0.0f ? fmaxf(m / KvFmt<FMT>::qmax, kKvMinScale) : 0.0f;
    float shrink = 1.0f;
    const float s = it.lo > 0 ? grown_scale<FMT>(held, m, fresh, &shrink) : fresh;
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    if (tid == 0) *scale = s;

    if (!is_v) {
        if (shrink != 1.0f)
            for (int i = tid; i < it.lo * quads; i += kThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(codes) + i;
                float v[4];
                kv_values4<FMT>(*w, v);
                for (int e = 0; e < 4; ++e) v[e] *= shrink;
                *w = kv_codes4<FMT>(v);
            }
        for (int i = tid; i < count * quads; i += kThreads) {
            const int t = it.lo + i / quads, d = (i % quads) * 4;
            const float4 f = load4<T>(x + (int64_t)t * ld + d);
            const float v[4] = {f.x * inv, f.y * inv, f.z * inv, f.w * inv};
            *reinterpret_cast<uint32_t *>(codes + (int64_t)t * D + d) = kv_codes4<FMT>(v);
        }
    } else {
        if (shrink != 1.0f)
            for (int i = tid; i < D * it.lo; i += kThreads) {
                uint8_t *p = codes + ((int64_t)(i / it.lo) << sh) + i % it.lo;
                *p = kv_code<FMT>(kv_value<FMT>(*p) * shrink);
            }
        // a thread transposes 2 columns of 16 slots: loads run along the
        // columns, stores along the slots
        const int pairs = D >> 1;
        for (int i = tid; i < pairs * (B >> 4); i += kThreads) {
            const int d = (i % pairs) * 2, t0 = (i / pairs) * 16;
            if (t0 + 16 <= it.lo || t0 >= it.hi) continue;
            float f[2][16];
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                float2 g = make_float2(0.0f, 0.0f);
                if (t0 + t >= it.lo && t0 + t < it.hi) g = load2<T>(x + (int64_t)(t0 + t) * ld + d);
                f[0][t] = g.x * inv, f[1][t] = g.y * inv;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = kv_codes4<FMT>(f[e] + 4 * q);
                uint8_t *p = codes + ((int64_t)(d + e) << sh) + t0;
                if (t0 >= it.lo && t0 + 16 <= it.hi) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
                else {
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (t0 + t >= it.lo && t0 + t < it.hi) p[t] = (uint8_t)(w[t >> 2] >> (8 * (t & 3)));
                }
            }
        }
    }
}

template <int FMT, typename T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadLaunch a)
{
    Item it;
    if (!find_item(a.s, a.c, blockIdx.x, &it)) return;
    const int D = a.c.head_dim, sh = a.c.block_shift, B = 1 << sh, tid = (int)threadIdx.x;
    const int64_t head = blockIdx.y, ld = (int64_t)a.c.kv_heads * D;
    const bool is_v = blockIdx.z != 0, absent = it.id < 0;
    const int64_t slab = (absent ? 0 : it.id) * a.c.kv_heads + head;
    T *y = static_cast<T *>(is_v ? a.v : a.k) + it.row * ld + head * D;
    const uint8_t *codes = (is_v ? a.c.v_codes : a.c.k_codes) + slab * ((int64_t)D << sh);
    const float s = absent ? 0.0f : (is_v ? a.c.v_scales : a.c.k_scales)[slab];
    const int count = it.hi - it.lo, quads = D >> 2;
    if (!is_v || absent) {
        for (int i = tid; i < count * quads; i += kThreads) {
            const int t = it.lo + i / quads, d = (i % quads) * 4;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (!absent) kv_values4<FMT>(*reinterpret_cast<const uint32_t *>(codes + (int64_t)t * D + d), v);
            for (int e = 0; e < 4; ++e) v[e] *= s;
            store4<T>(y + (int64_t)t * ld + d, v);
        }
    } else {
        const int pairs = D >> 1;
        for (int i = tid; i < pairs * (B >> 4); i += kThreads) {
            const int d = (i % pairs) * 2, t0 = (i / pairs) * 16;
            if (t0 + 16 <= it.lo || t0 >= it.hi) continue;
            float f[2][16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint4 w = *reinterpret_cast<const uint4 *>(codes + ((int64_t)(d + e) << sh) + t0);
                kv_values4<FMT>(w.x, f[e]);
                kv_values4<FMT>(w.y, f[e] + 4);
                kv_values4<FMT>(w.z, f[e] + 8);
                kv_values4<FMT>(w.w, f[e] + 12);
            }
#pragma unroll
            for (int t = 0; t < 16; ++t)
                if (t0 + t >= it.lo && t0 + t < it.hi)
                    store2<T>(y + (int64_t)(t0 + t) * ld + d, f[0][t] * s, f[1][t] * s);
        }
    }
}

// Blocks that a call's rows can touch: each holds a row, and a sequence of n
// rows touches at most n / B + 2.
int64_t max_items(const KvSeqs &s, const KvCache &c)
{
    const int64_t some = (s.rows >> c.block_shift) + 2 * (int64_t)s.batch;
    return s.rows < some ? s.rows : some;
}

}  // namespace

hipError_t launch_kv_append(const KvAppendLaunch &a, hipStream_t stream)
{
    const dim3 grid((unsigned)max_items(a.s, a.c), (unsigned)a.c.kv_heads, 2);
    if (a.format == KV_INT8) {
        if (a.x_dt == 0) kv_append_kernel<KV_INT8, float><<<grid, kThreads, 0, stream>>>(a);
        else kv_append_kernel<KV_INT8, bf16_bits><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (a.x_dt == 0) kv_append_kernel<KV_FP8, float><<<grid, kThreads, 0, stream>>>(a);
        else kv_append_kernel<KV_FP8, bf16_bits><<<grid, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadLaunch &a, hipStream_t stream)
{
    const dim3 grid((unsigned)max_items(a.s, a.c), (unsigned)a.c.kv_heads, 2);
    if (a.format == KV_INT8) {
        if (a.out_dt == 0) kv_read_kernel<KV_INT8, float><<<grid, kThreads, 0, stream>>>(a);
        else kv_read_kernel<KV_INT8, bf16_bits><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (a.out_dt == 0) kv_read_kernel<KV_FP8, float><<<grid, kThreads, 0, stream>>>(a);
        else kv_read_kernel<KV_FP8, bf16_bits><<<grid, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace nqk
