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
// least double), where growing to a / qmax each time would let it drift.  An
// a that is no finite number makes s a NaN, and with it all of the block.
//
// Both are bound by memory: a token of a head is read and written once (by the
// write its row is read twice, for the scale and for the codes, the second
// time from the cache: 77 MB fetched for 59).  14.3k tokens of 8 heads of 128,
// bf16 to E4M3: 88 MB in 24 to 28 us; 107k tokens of int8 back to bf16: 657 MB
// in 150 us, 4.4 TB/s; 16 single tokens 5.6 us, one dependent load after
// another.
//
// One workgroup takes one block of one head, keys or values (the two have
// their own scales), so the scale is a workgroup's reduction and no two
// workgroups share a byte.
#include <type_traits>

#include "nq_kv_device.h"

namespace nqk {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_max(float a, float *shared)
{
    const int lane = (int)(threadIdx.x & 63u);
    a = larger(a, xor_lane<1>(a, lane));
    a = larger(a, xor_lane<2>(a, lane));
    a = larger(a, xor_lane<4>(a, lane));
    a = larger(a, xor_lane<8>(a, lane));
    a = larger(a, xor_lane<16>(a, lane));
    a = larger(a, xor_lane<32>(a, lane));
    if (lane == 0) shared[threadIdx.x >> 6] = a;
    __syncthreads();
    return larger(larger(shared[0], shared[1]), larger(shared[2], shared[3]));
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
// The hardware's bf16 conversion: nearest, ties to even, NaN stays one.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
template <typename T> __device__ __forceinline__ void store4(T *p, const float *v);
template <> __device__ __forceinline__ void store4<float>(float *p, const float *v)
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <> __device__ __forceinline__ void store4<bf16_bits>(bf16_bits *p, const float *v)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float *v);
template <> __device__ __forceinline__ void store8<float>(float *p, const float *v)
{
    store4<float>(p, v);
    store4<float>(p + 4, v + 4);
}
template <> __device__ __forceinline__ void store8<bf16_bits>(bf16_bits *p, const float *v)
{
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
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

// Keys: a thread takes 8 columns of a slot.  Values: kCols columns of kSlots
// neighbouring slots, which it transposes in registers, so that rows are read
// along their columns and codes written along the slots.
constexpr int kCols = 4, kSlots = 8;

template <int D, int FMT, typename T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendLaunch a)
{
    __shared__ float red[4];
    Item it;
    if (!find_item(a.s, a.c, a.item0 + blockIdx.x, &it) || it.id < 0) return;
    const int sh = a.c.block_shift, tid = (int)threadIdx.x;
    const int64_t head = blockIdx.y, slab = it.id * a.c.kv_heads + head;
    const bool is_v = blockIdx.z != 0;
    const int64_t ld = is_v ? a.ldv : a.ldk;
    const T *x = static_cast<const T *>(is_v ? a.v : a.k) + it.row * ld + head * D;
    uint8_t *codes = (is_v ? a.c.v_codes : a.c.k_codes) + slab * ((int64_t)D << sh);
    float *scale = (is_v ? a.c.v_scales : a.c.k_scales) + slab;
    const int count = it.hi - it.lo;

    float m = 0.0f;
#pragma unroll 4
    for (int i = tid; i < count * (D / 8); i += kThreads) {
        const int t = i / (D / 8), d = (i % (D / 8)) * 8;
        const T *p = x + (int64_t)(it.lo + t) * ld + d;
        const float4 v = load4<T>(p), w = load4<T>(p + 4);
        const float all[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
        for (int e = 0; e < 8; ++e) m = larger(m, all[e]);
    }
    const float held = it.lo > 0 ? *scale : 0.0f;   // read before thread 0 stores it below
    m = block_max(m, red);
    const float fresh = m > 0.0f ? fmaxf(m / KvFmt<FMT>::qmax, kKvMinScale) : 0.0f;
    float shrink = 1.0f;
    float s = it.lo > 0 ? grown_scale<FMT>(held, m, fresh, &shrink) : fresh;     // a held NaN stays
    if (!(m < __builtin_inff())) s = __builtin_nanf(""), shrink = 1.0f;
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    if (tid == 0) *scale = s;

    if (!is_v) {
        if (shrink != 1.0f)
            for (int i = tid; i < it.lo * (D / 4); i += kThreads) {
                uint32_t *w = reinterpret_cast<uint32_t *>(codes) + i;
                float v[4];
                kv_values4<FMT>(*w, v);
                for (int e = 0; e < 4; ++e) v[e] *= shrink;
                *w = kv_codes4<FMT>(v);
            }
#pragma unroll 4
        for (int i = tid; i < count * (D / 8); i += kThreads) {
            const int t = it.lo + i / (D / 8), d = (i % (D / 8)) * 8;
            const T *p = x + (int64_t)t * ld + d;
            const float4 f = load4<T>(p), h = load4<T>(p + 4);
            const float v[8] = {f.x * inv, f.y * inv, f.z * inv, f.w * inv, h.x * inv, h.y * inv, h.z * inv, h.w * inv};
            *reinterpret_cast<uint2 *>(codes + (int64_t)t * D + d) = make_uint2(kv_codes4<FMT>(v), kv_codes4<FMT>(v + 4));
        }
        return;
    }
    if (shrink != 1.0f)
        for (int i = tid; i < D * it.lo; i += kThreads) {
            uint8_t *p = codes + ((int64_t)(i / it.lo) << sh) + i % it.lo;
            *p = kv_code<FMT>(kv_value<FMT>(*p) * shrink);
        }
    const int first = it.lo & ~(kSlots - 1), runs = (it.hi - first + kSlots - 1) / kSlots;
    for (int i = tid; i < (D / kCols) * runs; i += kThreads) {
        const int d = (i % (D / kCols)) * kCols, t0 = first + (i / (D / kCols)) * kSlots;
        float f[kCols][kSlots];
#pragma unroll
        for (int t = 0; t < kSlots; ++t) {
            float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (t0 + t >= it.lo && t0 + t < it.hi) g = load4<T>(x + (int64_t)(t0 + t) * ld + d);
            f[0][t] = g.x * inv, f[1][t] = g.y * inv, f[2][t] = g.z * inv, f[3][t] = g.w * inv;
        }
        const bool full = t0 >= it.lo && t0 + kSlots <= it.hi;
#pragma unroll
        for (int e = 0; e < kCols; ++e) {
            const uint32_t w[2] = {kv_codes4<FMT>(f[e]), kv_codes4<FMT>(f[e] + 4)};
            uint8_t *p = codes + ((int64_t)(d + e) << sh) + t0;
            if (full) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
            else {
#pragma unroll
                for (int t = 0; t < kSlots; ++t)
                    if (t0 + t >= it.lo && t0 + t < it.hi) p[t] = (uint8_t)(w[t >> 2] >> (8 * (t & 3)));
            }
        }
    }
}

template <int D, int FMT, typename T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadLaunch a)
{
    Item it;
    if (!find_item(a.s, a.c, a.item0 + blockIdx.x, &it)) return;
    const int sh = a.c.block_shift, tid = (int)threadIdx.x;
    const int64_t head = blockIdx.y, ld = (int64_t)a.c.kv_heads * D;
    const bool is_v = blockIdx.z != 0, absent = it.id < 0;
    const int64_t slab = (absent ? 0 : it.id) * a.c.kv_heads + head;
    T *y = static_cast<T *>(is_v ? a.v : a.k) + it.row * ld + head * D;
    const uint8_t *codes = (is_v ? a.c.v_codes : a.c.k_codes) + slab * ((int64_t)D << sh);
    const float s = absent ? 0.0f : (is_v ? a.c.v_scales : a.c.k_scales)[slab];
    const int count = it.hi - it.lo;
    if (!is_v || absent) {
#pragma unroll 4
        for (int i = tid; i < count * (D / 8); i += kThreads) {
            const int t = it.lo + i / (D / 8), d = (i % (D / 8)) * 8;
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (!absent) {
                const uint2 w = *reinterpret_cast<const uint2 *>(codes + (int64_t)t * D + d);
                kv_values4<FMT>(w.x, v);
                kv_values4<FMT>(w.y, v + 4);
            }
            for (int e = 0; e < 8; ++e) v[e] *= s;
            store8<T>(y + (int64_t)t * ld + d, v);
        }
        return;
    }
    const int first = it.lo & ~(kSlots - 1), runs = (it.hi - first + kSlots - 1) / kSlots;
    for (int i = tid; i < (D / kCols) * runs; i += kThreads) {
        const int d = (i % (D / kCols)) * kCols, t0 = first + (i / (D / kCols)) * kSlots;
        float f[kCols][kSlots];
#pragma unroll
        for (int e = 0; e < kCols; ++e) {
            const uint2 w = *reinterpret_cast<const uint2 *>(codes + ((int64_t)(d + e) << sh) + t0);
            kv_values4<FMT>(w.x, f[e]);
            kv_values4<FMT>(w.y, f[e] + 4);
        }
#pragma unroll
        for (int t = 0; t < kSlots; ++t) {
            const float v[4] = {f[0][t] * s, f[1][t] * s, f[2][t] * s, f[3][t] * s};
            if (t0 + t >= it.lo && t0 + t < it.hi) store4<T>(y + (int64_t)(t0 + t) * ld + d, v);
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

// Calls go(item0, grid) for all blocks, as many at a time as a launch may have.
template <typename Go> hipError_t by_items(const KvSeqs &s, const KvCache &c, Go go)
{
    const int64_t items = max_items(s, c), most = most_workgroups(kThreads);
    for (int64_t at = 0; at < items; at += most) {
        go(at, dim3((unsigned)(items - at < most ? items - at : most), (unsigned)c.kv_heads, 2));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename Go> void by_head_dim(int head_dim, Go go)
{
    switch (head_dim) {
    case 64: go(std::integral_constant<int, 64>()); break;
    case 128: go(std::integral_constant<int, 128>()); break;
    case 192: go(std::integral_constant<int, 192>()); break;
    default: go(std::integral_constant<int, 256>()); break;
    }
}

}  // namespace

hipError_t launch_kv_append(const KvAppendLaunch &call, hipStream_t stream)
{
    KvAppendLaunch a = call;
    return by_items(a.s, a.c, [&](int64_t item0, dim3 grid) {
        a.item0 = item0;
        by_head_dim(a.c.head_dim, [&](auto dim) {
            constexpr int D = decltype(dim)::value;
            if (a.format == KV_INT8) {
                if (a.x_dt == 0) kv_append_kernel<D, KV_INT8, float><<<grid, kThreads, 0, stream>>>(a);
                else kv_append_kernel<D, KV_INT8, bf16_bits><<<grid, kThreads, 0, stream>>>(a);
            } else {
                if (a.x_dt == 0) kv_append_kernel<D, KV_FP8, float><<<grid, kThreads, 0, stream>>>(a);
                else kv_append_kernel<D, KV_FP8, bf16_bits><<<grid, kThreads, 0, stream>>>(a);
            }
        });
    });
}

hipError_t launch_kv_read(const KvReadLaunch &call, hipStream_t stream)
{
    KvReadLaunch a = call;
    return by_items(a.s, a.c, [&](int64_t item0, dim3 grid) {
        a.item0 = item0;
        by_head_dim(a.c.head_dim, [&](auto dim) {
            constexpr int D = decltype(dim)::value;
            if (a.format == KV_INT8) {
                if (a.out_dt == 0) kv_read_kernel<D, KV_INT8, float><<<grid, kThreads, 0, stream>>>(a);
                else kv_read_kernel<D, KV_INT8, bf16_bits><<<grid, kThreads, 0, stream>>>(a);
            } else {
                if (a.out_dt == 0) kv_read_kernel<D, KV_FP8, float><<<grid, kThreads, 0, stream>>>(a);
                else kv_read_kernel<D, KV_FP8, bf16_bits><<<grid, kThreads, 0, stream>>>(a);
            }
        });
    });
}

}  // namespace nqk
