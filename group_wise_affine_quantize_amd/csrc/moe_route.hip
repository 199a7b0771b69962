// Routing tokens to experts, and the gradient of the chosen weights (contract
// in include/nq.h).
//
// Mathematics.  p = softmax(x) or sigmoid(x) of a token's logits x; key = p +
// bias, or x itself without a bias (p has x's order, and x tells apart what
// rounding makes equal in p).  A group's score is the sum of its one or two
// largest keys; the experts of the best groups stay, and the top_k largest
// keys of these are chosen, the lowest index first among equals.  Weights are
// the chosen p, divided by their sum when renormalised, times `scale`.
//
// Gradient, with w_k = scale * p_k (/ S, S = sum of the chosen p):
//   d_k = scale * dw_k, renormalised (d_k - sum_i d_i p_i / S) / S,
//   sigmoid: dx = d_k p_k (1 - p_k) at the chosen experts, 0 elsewhere,
//   softmax: dx_j = p_j (d_j - sum_k d_k p_k), d_j = 0 where not chosen
//   (renormalised, the sum is zero).
//
// A token's logits lie in the registers of LPT = 16 or 64 lanes, so that a
// wave routes four tokens of up to 256 experts at once and the rounds of the
// choice need no memory.
#include "nq_kv_device.h"

namespace nqk {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroups = 64;
constexpr float kNegInf = -__builtin_inff();

// Order-preserving map to unsigned; 0 is below every number's image.
__device__ __forceinline__ uint32_t ordered(float f)
{
    f = f == f ? f + 0.0f : kNegInf;    // NaN sorts as -inf, -0 as 0
    const uint32_t u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int LPT> __device__ __forceinline__ float token_max(float v, int lane)
{
    v = fmaxf(v, xor_lane<1>(v, lane));
    v = fmaxf(v, xor_lane<2>(v, lane));
    v = fmaxf(v, xor_lane<4>(v, lane));
    v = fmaxf(v, xor_lane<8>(v, lane));
    if constexpr (LPT == 64) {
        v = fmaxf(v, xor_lane<16>(v, lane));
        v = fmaxf(v, xor_lane<32>(v, lane));
    }
    return v;
}

template <int LPT> __device__ __forceinline__ float token_sum(float v, int lane)
{
    v += xor_lane<1>(v, lane);
    v += xor_lane<2>(v, lane);
    v += xor_lane<4>(v, lane);
    v += xor_lane<8>(v, lane);
    if constexpr (LPT == 64) {
        v += xor_lane<16>(v, lane);
        v += xor_lane<32>(v, lane);
    }
    return v;
}

template <int LPT> __device__ __forceinline__ uint32_t token_umax(uint32_t v, int lane)
{
    auto step = [&](float o) { const uint32_t u = __float_as_uint(o); v = u > v ? u : v; };
    step(xor_lane<1>(__uint_as_float(v), lane));
    step(xor_lane<2>(__uint_as_float(v), lane));
    step(xor_lane<4>(__uint_as_float(v), lane));
    step(xor_lane<8>(__uint_as_float(v), lane));
    if constexpr (LPT == 64) {
        step(xor_lane<16>(__uint_as_float(v), lane));
        step(xor_lane<32>(__uint_as_float(v), lane));
    }
    return v;
}

// EPL neighbouring logits as fp32, -inf past `experts`.
template <typename T, int EPL>
__device__ __forceinline__ void load_logits(const T *row, int e0, int experts, bool wide, float *x)
{
    if (wide && e0 + EPL <= experts) {
        constexpr int per = 16 / (int)sizeof(T) < EPL ? 16 / (int)sizeof(T) : EPL;
        typedef T vec __attribute__((ext_vector_type(per)));
#pragma unroll
        for (int i = 0; i < EPL; i += per) {
            const vec v = *reinterpret_cast<const vec *>(row + e0 + i);
#pragma unroll
            for (int j = 0; j < per; ++j) {
                const T t = v[j];
                x[i + j] = Elt<T>::load(&t, 0);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) x[j] = e0 + j < experts ? Elt<T>::load(row, e0 + j) : kNegInf;
    }
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// p of a token's logits; for softmax *top and *inv are the maximum and the
// reciprocal-free divisor that any single logit's p can be taken with.
template <int LPT, int EPL>
__device__ __forceinline__ void scores(int kind, const float *x, int lane, float *p, float *top, float *sum)
{
    if (kind == MOE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) p[j] = sigmoid(x[j]);
        *top = 0.0f, *sum = 1.0f;
        return;
    }
    float m = kNegInf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, x[j]);
    m = token_max<LPT>(m, lane);
    const float ref = m == kNegInf ? 0.0f : m;      // no finite logit: every p is 0
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        p[j] = expf(x[j] - ref);
        s += p[j];
    }
    s = token_sum<LPT>(s, lane);
    if (m == kNegInf) s = 1.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) p[j] /= s;
    *top = ref, *sum = s;
}

template <typename T, int LPT, int EPL>
__global__ __launch_bounds__(kThreads) void moe_route_kernel(MoeRouteLaunch a, int wide)
{
    constexpr int TOK = kThreads / LPT;
    __shared__ float sh_key[TOK][LPT * EPL];
    __shared__ uint32_t sh_group[TOK][kMaxGroups];
    __shared__ uint8_t sh_kept[TOK][kMaxGroups];
    const MoeRoute r = a.r;
    const int lane = (int)(threadIdx.x & 63u), tl = (int)threadIdx.x % LPT, slot = (int)threadIdx.x / LPT;
    const int64_t token = (int64_t)blockIdx.x * TOK + slot;
    const bool live = token < a.tokens;
    const T *row = static_cast<const T *>(a.logits) + (live ? token : a.tokens - 1) * a.ldl;
    const int e0 = tl * EPL;

    float x[EPL], p[EPL], top, sum;
    load_logits<T, EPL>(row, e0, r.experts, wide != 0, x);
    scores<LPT, EPL>(r.score, x, lane, p, &top, &sum);
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const float k = a.bias ? (e0 + j < r.experts ? p[j] + a.bias[e0 + j] : 0.0f) : x[j];
        key[j] = e0 + j < r.experts ? ordered(k) : 0u;
        if (r.groups > 1) sh_key[slot][e0 + j] = !a.bias && r.group_best == 2 ? p[j] : k;
    }
    if (r.groups > 1) {
        const int size = r.experts / r.groups;
        __syncthreads();
        for (int g = tl; g < r.groups; g += LPT) {
            float b1 = kNegInf, b2 = kNegInf;
            for (int i = 0; i < size; ++i) {
                const float v = sh_key[slot][g * size + i];
                b2 = fmaxf(b2, fminf(b1, v));
                b1 = fmaxf(b1, v);
            }
            sh_group[slot][g] = ordered(r.group_best == 2 ? b1 + b2 : b1);
        }
        __syncthreads();
        for (int g = tl; g < r.groups; g += LPT) {
            const uint32_t mine = sh_group[slot][g];
            int rank = 0;
            for (int i = 0; i < r.groups; ++i) {
                const uint32_t o = sh_group[slot][i];
                rank += o > mine || (o == mine && i < g);
            }
            sh_kept[slot][g] = rank < r.top_groups;
        }
        __syncthreads();
        int g = e0 / size, left = size - (e0 - g * size);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (left == 0) ++g, left = size;
            if (g < r.groups && !sh_kept[slot][g]) key[j] = 0u;
            --left;
        }
    }

    float mine[2] = {0.0f, 0.0f}, total = 0.0f;
    for (int k = 0; k < r.top_k; ++k) {
        uint32_t best = 0u;
        int bj = 0;
        float bp = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const bool more = key[j] > best;
            best = more ? key[j] : best;
            bj = more ? j : bj;
            bp = more ? p[j] : bp;
        }
        const uint32_t most = token_umax<LPT>(best, lane);
        uint64_t hit = __ballot(best == most);
        if constexpr (LPT == 16) hit = (hit >> (lane & 48)) & 0xffffu;
        const int winner = __ffsll((unsigned long long)hit) - 1;
        const float w = __shfl(bp, (lane & ~(LPT - 1)) + winner);
        total += w;
        if (tl == winner) {
            if (live) a.ids[token * r.top_k + k] = (uint32_t)(e0 + bj);
#pragma unroll
            for (int j = 0; j < EPL; ++j) key[j] = j == bj ? 0u : key[j];
        }
        if (tl == k % LPT) mine[k / LPT] = w;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = tl + i * LPT;
        if (live && k < r.top_k) {
            float w = mine[i];
            if (r.renormalise) w = total > 0.0f ? w / total : 0.0f;
            a.weights[token * r.top_k + k] = w * r.scale;
        }
    }
}

template <typename T, int LPT, int EPL>
__global__ __launch_bounds__(kThreads) void moe_grad_kernel(MoeGradLaunch a, int wide)
{
    constexpr int TOK = kThreads / LPT;
    __shared__ float sh_d[TOK][LPT * EPL];
    const MoeRoute r = a.r;
    const int lane = (int)(threadIdx.x & 63u), tl = (int)threadIdx.x % LPT, slot = (int)threadIdx.x / LPT;
    const int64_t token = (int64_t)blockIdx.x * TOK + slot;
    const bool live = token < a.tokens;
    const int64_t t = live ? token : a.tokens - 1;
    const T *row = static_cast<const T *>(a.logits) + t * a.ldl;
    const int e0 = tl * EPL;

    float x[EPL], p[EPL], top = 0.0f, sum = 1.0f;
    load_logits<T, EPL>(row, e0, r.experts, wide != 0, x);
    const bool soft = r.score == MOE_SOFTMAX;
    if (soft) scores<LPT, EPL>(r.score, x, lane, p, &top, &sum);
#pragma unroll
    for (int j = 0; j < EPL; ++j) sh_d[slot][e0 + j] = 0.0f;

    uint32_t id[2];
    float pk[2], qk[2], d[2], total = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = tl + i * LPT;
        id[i] = k < r.top_k ? a.ids[t * r.top_k + k] : ~0u;
        pk[i] = 0.0f, qk[i] = 0.0f, d[i] = 0.0f;
        if (id[i] < (uint32_t)r.experts) {
            const float v = Elt<T>::load(row, id[i]);
            pk[i] = soft ? expf(v - top) / sum : sigmoid(v);
            qk[i] = sigmoid(-v);                          // 1 - p of a sigmoid, without cancellation
            d[i] = a.dweights[t * r.top_k + k] * r.scale;
        }
        total += pk[i];
        dot += d[i] * pk[i];
    }
    total = token_sum<LPT>(total, lane);
    dot = token_sum<LPT>(dot, lane);
    if (r.renormalise) {
#pragma unroll
        for (int i = 0; i < 2; ++i) d[i] = total > 0.0f ? (d[i] - dot / total) / total : 0.0f;
        dot = 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (id[i] < (uint32_t)r.experts) sh_d[slot][id[i]] = soft ? d[i] : d[i] * pk[i] * qk[i];
    __syncthreads();
    T *out = static_cast<T *>(a.dlogits) + t * r.experts;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const float v = sh_d[slot][e0 + j];
        if (live && e0 + j < r.experts) Elt<T>::store(out, e0 + j, soft ? p[j] * (v - dot) : v);
    }
}

// Whether the rows of logits can be loaded 16 bytes (or a lane's share, if
// that is less) at a time.
bool wide_rows(const void *p, int64_t ld, int bytes)
{
    return ((uintptr_t)p & 15u) == 0 && (ld * bytes) % 16 == 0;
}

template <typename L> unsigned grid_of(const L &a, int lpt)
{
    const int64_t per = kThreads / lpt;
    return (unsigned)((a.tokens + per - 1) / per);
}

template <typename T, int LPT, int EPL> void go(const MoeRouteLaunch &a, int wide, hipStream_t s)
{
    moe_route_kernel<T, LPT, EPL><<<grid_of(a, LPT), kThreads, 0, s>>>(a, wide);
}
template <typename T, int LPT, int EPL> void go(const MoeGradLaunch &a, int wide, hipStream_t s)
{
    moe_grad_kernel<T, LPT, EPL><<<grid_of(a, LPT), kThreads, 0, s>>>(a, wide);
}

template <typename T, typename L> hipError_t by_experts(const L &a, hipStream_t s)
{
    const int wide = wide_rows(a.logits, a.ldl, (int)sizeof(T));
    const int e = a.r.experts;
    if (e <= 64) go<T, 16, 4>(a, wide, s);
    else if (e <= 128) go<T, 16, 8>(a, wide, s);
    else if (e <= 256) go<T, 16, 16>(a, wide, s);
    else if (e <= 512) go<T, 64, 8>(a, wide, s);
    else go<T, 64, 16>(a, wide, s);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const MoeRouteLaunch &a, hipStream_t s)
{
    return a.x_dt == 0 ? by_experts<float>(a, s) : by_experts<bf16_bits>(a, s);
}

hipError_t launch_moe_route_grad(const MoeGradLaunch &a, hipStream_t s)
{
    return a.x_dt == 0 ? by_experts<float>(a, s) : by_experts<bf16_bits>(a, s);
}

}  // namespace nqk
