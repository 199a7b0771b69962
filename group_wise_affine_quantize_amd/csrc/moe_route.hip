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
// A token's logits lie in the registers of LPT = 16 or 64 lanes, EPL
// neighbouring ones in each, so that a wave routes four tokens of up to 256
// experts at once.  Bound by the vector unit: 16384 tokens of 256 experts in
// fp32 (top 8 of 4 of 8 groups, sigmoid and bias, 17.8 MB) take 13.5 us, of
// which the logits' bytes would need 3.5.
//
// The choice of up to kShort experts: every expert is one 64-bit number, its
// ordered key above its falling index, so that numbers are distinct and the
// largest is the one to choose, ties included.  As the bits of a denormal
// double they order under v_max_f64 / v_min_f64: a compare-exchange is two
// instructions.  Each lane sorts its own and keeps the best eight; lists of
// two lanes merge by max(a[i], b[7 - i]) -- a bitonic sequence of the best
// eight -- and three rounds of exchanges, and after log2(LPT) merges every
// lane holds the token's eight in order.  More than kShort are chosen one by one,
// a maximum over the token's lanes each.
#include "nq_kv_device.h"

namespace nqk {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroups = 64;
constexpr int kShort = 8;       // experts per token up to which the choice is by sorting
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

// A NaN logit counts as -inf.
__device__ __forceinline__ float numbered(float x) { return fmaxf(x, kNegInf); }

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
                x[i + j] = numbered(Elt<T>::load(&t, 0));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float t = Elt<T>::load(row, e0 + j < experts ? e0 + j : experts - 1);
            x[j] = e0 + j < experts ? numbered(t) : kNegInf;
        }
    }
}

// e^x to about 1.5 ulp: x log2(e) in two parts, the low one to first order.
__device__ __forceinline__ float exp_of(float x)
{
    constexpr float L = 1.44269502162933349609f, Llo = 1.92596299112661746887e-8f;   // log2(e)
    x = fminf(fmaxf(x, -150.0f), 88.0f);    // 0 from below on; no infinities, whose differences are none
    const float t = x * L, r = fmaf(x, Llo, fmaf(x, L, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e * r, 0.693147180559945309417f, e);
}

__device__ __forceinline__ float sigmoid(float x)
{
    const float d = 1.0f + exp_of(-x);
    const float y = __builtin_amdgcn_rcpf(d);
    return x < -87.0f ? 0.0f : fmaf(fmaf(-d, y, 1.0f), y, y);   // below fp32's normal numbers: 0
}

// p of a token's logits; *top and *sum are a softmax's maximum and divisor,
// from which any single logit's p can be taken.
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
        p[j] = exp_of(x[j] - ref);
        s += p[j];
    }
    s = token_sum<LPT>(s, lane);
    if (m == kNegInf) s = 1.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) p[j] /= s;
    *top = ref, *sum = s;
}

// ---- the choice by sorting
__device__ __forceinline__ double wide_key(uint32_t key, int e)
{
    const uint64_t v = (uint64_t)key << 10 | (uint64_t)(1023 - e);
    return __longlong_as_double((long long)(key ? v : 0));
}
__device__ __forceinline__ void exchange(double &hi, double &lo)
{
    const double a = hi, b = lo;
    hi = __builtin_fmax(a, b), lo = __builtin_fmin(a, b);
}
// Eight numbers that fall and then rise (or any rotation of that) into falling order.
__device__ __forceinline__ void sort_bitonic8(double *v)
{
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) exchange(v[i], v[i + d]);
}
__device__ __forceinline__ void sort8(double *v)      // Batcher's odd-even merge sort, 19 exchanges
{
    exchange(v[0], v[1]), exchange(v[2], v[3]), exchange(v[4], v[5]), exchange(v[6], v[7]);
    exchange(v[0], v[2]), exchange(v[1], v[3]), exchange(v[4], v[6]), exchange(v[5], v[7]);
    exchange(v[1], v[2]), exchange(v[5], v[6]);
    exchange(v[0], v[4]), exchange(v[1], v[5]), exchange(v[2], v[6]), exchange(v[3], v[7]);
    exchange(v[2], v[4]), exchange(v[3], v[5]);
    exchange(v[1], v[2]), exchange(v[3], v[4]), exchange(v[5], v[6]);
}
// A lane's number from the row of 16 turned by TURN lanes.
template <int TURN> __device__ __forceinline__ uint64_t turned(uint64_t v)
{
    constexpr int row_ror = 0x120 + TURN;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)v, row_ror, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(v >> 32), row_ror, 0xF, 0xF, true);
    return (uint64_t)hi << 32 | lo;
}
// v[0 .. 7] and the same of another lane (o) -> the best eight of both.
__device__ __forceinline__ void merge8(double *v, const double *o)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_fmax(v[i], o[i]);
    sort_bitonic8(v);
}
// With the lane TURN places back in the row: turns by 1, 2, 4 and 8 in turn
// give every lane the best of all 16, each counted once.
template <int TURN> __device__ __forceinline__ void merge_turned(double *v)
{
    double o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = __longlong_as_double((long long)turned<TURN>((uint64_t)__double_as_longlong(v[7 - i])));
    merge8(v, o);
}
template <int OFF> __device__ __forceinline__ void merge_rows(double *v, int lane)      // OFF = 16, 32
{
    double o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t u = (uint64_t)__double_as_longlong(v[7 - i]);
        const uint32_t lo = __float_as_uint(xor_lane<OFF>(__uint_as_float((uint32_t)u), lane));
        const uint32_t hi = __float_as_uint(xor_lane<OFF>(__uint_as_float((uint32_t)(u >> 32)), lane));
        o[i] = __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
    }
    merge8(v, o);
}

// Lanes among the 15 others of a row of 16 whose number is larger.
template <int TURN> __device__ __forceinline__ int better_lanes(uint64_t mine)
{
    if constexpr (TURN == 16) return 0;
    else {
        return (turned<TURN>(mine) > mine) + better_lanes<TURN + 1>(mine);
    }
}

// A token's groups when each is a power of two of lanes (LPT = 16): the best
// one or two values of a lane and of its group's lanes, then the group's rank
// among the others by turning the 16 lanes past each other.  Returns whether
// the lane's group stays.
template <int EPL>
__device__ __forceinline__ bool group_stays(const MoeRoute &r, const float *v, int lanes_per_group, int tl, int lane)
{
    float b1 = kNegInf, b2 = kNegInf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        b2 = fmaxf(b2, fminf(b1, v[j]));
        b1 = fmaxf(b1, v[j]);
    }
    auto join = [&](float o1, float o2) {
        b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
        b1 = fmaxf(b1, o1);
    };
    if (lanes_per_group > 1) join(xor_lane<1>(b1, lane), xor_lane<1>(b2, lane));
    if (lanes_per_group > 2) join(xor_lane<2>(b1, lane), xor_lane<2>(b2, lane));
    if (lanes_per_group > 4) join(xor_lane<4>(b1, lane), xor_lane<4>(b2, lane));
    if (lanes_per_group > 8) join(xor_lane<8>(b1, lane), xor_lane<8>(b2, lane));
    const int group = tl / lanes_per_group;
    const uint32_t score = group < r.groups ? ordered(r.group_best == 2 ? b1 + b2 : b1) : 0u;
    const uint64_t mine = (uint64_t)score << 32 | (uint32_t)(63 - group);
    return better_lanes<1>(mine) < r.top_groups * lanes_per_group;
}

template <typename T, int LPT, int EPL, bool SORT>
__global__ __launch_bounds__(kThreads) void moe_route_kernel(MoeRouteLaunch a, int wide, int lanes_per_group)
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

    float x[EPL], p[EPL], top = 0.0f, sum = 1.0f;
    load_logits<T, EPL>(row, e0, r.experts, wide != 0, x);
    const bool summed = r.groups > 1 && r.group_best == 2;
    // a sigmoid's scores are wanted for every expert only where keys are made of them
    if (r.score == MOE_SOFTMAX || a.bias || summed || !SORT) scores<LPT, EPL>(r.score, x, lane, p, &top, &sum);
    float bias[EPL];
    if (a.bias)
#pragma unroll
        for (int j = 0; j < EPL; ++j) bias[j] = a.bias[e0 + j < r.experts ? e0 + j : r.experts - 1];
    uint32_t key[EPL];
    float v[EPL];           // what a group's score is made of
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const bool is = e0 + j < r.experts;
        const float k = a.bias ? p[j] + bias[j] : x[j];
        key[j] = is ? ordered(k) : 0u;
        // a NaN here would count its group's best twice: fminf(best, NaN) is the best
        v[j] = is ? numbered(!a.bias && summed ? p[j] : k) : kNegInf;
    }
    if (LPT == 16 && lanes_per_group > 0) {
        if (!group_stays<EPL>(r, v, lanes_per_group, tl, lane))
#pragma unroll
            for (int j = 0; j < EPL; ++j) key[j] = 0u;
    } else if (r.groups > 1) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) sh_key[slot][e0 + j] = v[j];
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

    if constexpr (SORT) {
        double best[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) best[j] = wide_key(key[j], e0 + j);
        sort8(best);
        if constexpr (EPL == 16) {
            sort8(best + 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) best[i] = __builtin_fmax(best[i], best[15 - i]);
            sort_bitonic8(best);
        }
        merge_turned<1>(best);
        merge_turned<2>(best);
        merge_turned<4>(best);
        merge_turned<8>(best);
        if constexpr (LPT == 64) {
            merge_rows<16>(best, lane);
            merge_rows<32>(best, lane);
        }
        uint32_t low = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) low = tl == i ? (uint32_t)__double_as_longlong(best[i]) : low;
        const int found = 1023 - (int)(low & 1023u), id = found < r.experts ? found : r.experts - 1;
        const bool mine = tl < r.top_k;
        float w = 0.0f;
        if (mine) {             // its logit again: it is in the cache
            const float x1 = numbered(Elt<T>::load(row, id));
            w = r.score == MOE_SIGMOID ? sigmoid(x1) : exp_of(x1 - top) / sum;
        }
        const float total = token_sum<LPT>(w, lane);
        if (live && mine) {
            if (r.renormalise) w = total > 0.0f ? w / total : 0.0f;
            a.ids[token * r.top_k + tl] = (uint32_t)id;
            a.weights[token * r.top_k + tl] = w * r.scale;
        }
        return;
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
            const float v = numbered(Elt<T>::load(row, id[i]));
            pk[i] = soft ? exp_of(v - top) / sum : sigmoid(v);
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
    // lanes of a group, where that is a power of two of 16 lanes; 0: through LDS
    int lanes = 0;
    const int size = a.r.experts / a.r.groups;
    if (LPT == 16 && a.r.groups > 1 && size % EPL == 0) {
        lanes = size / EPL;
        if (lanes & (lanes - 1) || lanes > 16) lanes = 0;
    }
    // Lists of eight are worth their merges where a lane has that many experts
    // (16384 tokens of 256 experts, top 8 of 4 of 8 groups: 13.5 us sorted, 25 one by one; 32768 of 64, top 6:
    // 10.1 and 9.3).
    constexpr bool sorts = EPL >= 8;
    if (sorts && a.r.top_k <= kShort) moe_route_kernel<T, LPT, EPL, sorts><<<grid_of(a, LPT), kThreads, 0, s>>>(a, wide, lanes);
    else moe_route_kernel<T, LPT, EPL, false><<<grid_of(a, LPT), kThreads, 0, s>>>(a, wide, lanes);
}
template <typename T, int LPT, int EPL> void go(const MoeGradLaunch &a, int wide, hipStream_t s)
{
    moe_grad_kernel<T, LPT, EPL><<<grid_of(a, LPT), kThreads, 0, s>>>(a, wide);
}

// The launch's tokens from `t` on.
template <typename T> MoeRouteLaunch from_token(MoeRouteLaunch a, int64_t t)
{
    a.logits = static_cast<const T *>(a.logits) + t * a.ldl, a.ids += t * a.r.top_k, a.weights += t * a.r.top_k;
    return a;
}
template <typename T> MoeGradLaunch from_token(MoeGradLaunch a, int64_t t)
{
    a.logits = static_cast<const T *>(a.logits) + t * a.ldl, a.ids += t * a.r.top_k, a.dweights += t * a.r.top_k;
    a.dlogits = static_cast<T *>(a.dlogits) + t * a.r.experts;
    return a;
}

template <typename T, typename L> void by_experts(const L &a, hipStream_t s)
{
    const int wide = wide_rows(a.logits, a.ldl, (int)sizeof(T));
    const int e = a.r.experts;
    if (e <= 64) go<T, 16, 4>(a, wide, s);
    else if (e <= 128) go<T, 16, 8>(a, wide, s);
    else if (e <= 256) go<T, 16, 16>(a, wide, s);
    else if (e <= 512) go<T, 64, 8>(a, wide, s);
    else go<T, 64, 16>(a, wide, s);
}

// All tokens, as many at a time as a launch may have with the fewest tokens to a workgroup.
template <typename T, typename L> hipError_t by_tokens(const L &call, hipStream_t s)
{
    constexpr int64_t most = most_workgroups(kThreads) * (kThreads / 64);
    for (int64_t at = 0; at < call.tokens; at += most) {
        L a = from_token<T>(call, at);
        a.tokens = call.tokens - at < most ? call.tokens - at : most;
        by_experts<T>(a, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_moe_route(const MoeRouteLaunch &a, hipStream_t s)
{
    return a.x_dt == 0 ? by_tokens<float>(a, s) : by_tokens<bf16_bits>(a, s);
}

hipError_t launch_moe_route_grad(const MoeGradLaunch &a, hipStream_t s)
{
    return a.x_dt == 0 ? by_tokens<float>(a, s) : by_tokens<bf16_bits>(a, s);
}

}  // namespace nqk
