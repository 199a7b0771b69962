// Norms before and after a block with its gate and residual scale, and their
// gradient (contract in include/nq.h).
//
// Mathematics, for a row:
//   ry = 1 / sqrt(mean y^2 + eps),  u = y ry (post + offset)  (or u = y),
//   h' = h + scale gate u,
//   rh = 1 / sqrt(mean h'^2 + eps), z = h' rh (pre + offset).
// Gradient, from the stored h' and the gradients dh', dz that arrive:
//   v = dz (pre + offset),          D = dh' + rh (v - xh mean(v xh)),  xh = h' rh,
//   dh = D,  du = scale gate D,     w = du (post + offset),
//   dy = ry (w - yh mean(w yh))     (or dy = du),                      yh = y ry,
//   dpre = sum dz xh,  dpost = sum du yh,  dgate = scale sum D u,
// the sums over the rows that share the parameter.
//
// A row lies in the registers of one team of waves from its first load to its
// last store, so that each element is moved once; what teams exchange are the
// row's sums (one or two at a time, through LDS).  In the gradient a thread keeps its
// columns' parameter sums in registers over the rows of its workgroup's chunk; chunks
// write them to the workspace and a second kernel adds them in order.  All
// statistics and sums are fp32.
//
// What bounds it: memory, 4 moves of a row forward and 6 backward.
#include <algorithm>

#include "nq_kv.h"
#include "nq_layer.h"
#include "nq_vec.h"

namespace nqk {

namespace {

// Sums over a team of W waves, N at a time.  Slots alternate, so that one
// barrier per exchange is enough.
template <int W, int N> struct TeamSum {
    float (*sh)[W][N];      // two slots
    int slot;

    __device__ __forceinline__ void operator()(float *v, int lane, int wave)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lane_sum<64>(v[i], lane);
        if constexpr (W > 1) {
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < N; ++i) sh[slot][wave][i] = v[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float s = sh[slot][0][i];
#pragma unroll
                for (int w = 1; w < W; ++w) s += sh[slot][w][i];
                v[i] = s;
            }
            slot ^= 1;
        }
    }
};

// Teams of W waves; a row is V pieces of E elements for each thread.
template <int W> constexpr int teams() { return W == 1 ? 4 : 1; }

template <typename T, typename P, int E, int W, int V>
__global__ __launch_bounds__(64 * W * teams<W>()) void block_norm_kernel(BlockNormLaunch a)
{
    constexpr int TEAMS = teams<W>(), STRIDE = 64 * W * E;
    __shared__ float sh[2][W][1];
    const int lane = (int)(threadIdx.x & 63u), wave = W == 1 ? 0 : (int)(threadIdx.x >> 6);
    const int team = W == 1 ? (int)(threadIdx.x >> 6) : 0;
    TeamSum<W, 1> total{sh, 0};
    const int dim = (int)a.dim, col0 = (64 * wave + lane) * E;
    const float inv = 1.0f / (float)dim;
    const int64_t per_gate = a.gate ? a.rows / a.gates : 1;
    for (int64_t row = (int64_t)blockIdx.x * TEAMS + team; row < a.rows; row += (int64_t)gridDim.x * TEAMS) {
        const T *h = static_cast<const T *>(a.h) + row * a.ldh;
        float x[V][E];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = col0 + i * STRIDE;
            if (c < dim) load_run<T, E>(h + c, x[i]);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) x[i][e] = 0.0f;
        }
        if (a.y) {
            const T *y = static_cast<const T *>(a.y) + row * a.ldy;
            float u[V][E], s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = col0 + i * STRIDE;
                if (c < dim) load_run<T, E>(y + c, u[i]);
                else
#pragma unroll
                    for (int e = 0; e < E; ++e) u[i][e] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(u[i][e], u[i][e], s);
            }
            float f = a.scale;
            if (a.post) {
                total(&s, lane, wave);
                f *= rsqrtf(fmaf(s, inv, a.eps));
            }
            const P *gate = static_cast<const P *>(a.gate) + (a.gate ? row / per_gate * a.ldg : 0);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = col0 + i * STRIDE;
                if (c >= dim) continue;
                float w[E];
#pragma unroll
                for (int e = 0; e < E; ++e) u[i][e] *= f;
                if (a.post) {
                    load_run<P, E>(static_cast<const P *>(a.post) + c, w);
#pragma unroll
                    for (int e = 0; e < E; ++e) u[i][e] *= w[e] + a.offset;
                }
                if (a.gate) {
                    load_run<P, E>(gate + c, w);
#pragma unroll
                    for (int e = 0; e < E; ++e) u[i][e] *= w[e];
                }
#pragma unroll
                for (int e = 0; e < E; ++e) x[i][e] += u[i][e];
                store_run<T, E>(static_cast<T *>(a.h_out) + row * dim + c, x[i]);
            }
        }
        if (a.z) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(x[i][e], x[i][e], s);
            total(&s, lane, wave);
            const float r = rsqrtf(fmaf(s, inv, a.eps));
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = col0 + i * STRIDE;
                if (c >= dim) continue;
                float w[E], z[E];
                load_run<P, E>(static_cast<const P *>(a.pre) + c, w);
#pragma unroll
                for (int e = 0; e < E; ++e) z[e] = x[i][e] * r * (w[e] + a.offset);
                store_run<T, E>(static_cast<T *>(a.z) + row * dim + c, z);
            }
        }
    }
}

// How the gradient's rows are dealt to workgroups.  Rows that share a gate are
// kept together: where they are fewer than a chunk, a chunk is some whole
// gates' rows and adds their gate gradients itself; where they are more, each
// gate's rows are cut into `cuts` chunks.
struct Chunks {
    int64_t chunks;     // workgroups
    int64_t per_gate;   // rows that share a gate
    int64_t gates;      // gates of a chunk (0: the chunk is a part of one)
    int64_t cuts;       // chunks of a gate
    int64_t size;       // rows of a chunk
};

Chunks chunks_of(int64_t rows, int64_t gates)
{
    constexpr int64_t kMost = 1024, kLeast = 8;
    Chunks c{};
    if (rows == 0) return c;
    const int64_t want = std::max<int64_t>(kLeast, (rows + kMost - 1) / kMost);
    c.per_gate = rows / gates;
    if (c.per_gate < want) {
        c.gates = want / c.per_gate;
        c.cuts = 1;
        c.size = c.gates * c.per_gate;
        c.chunks = (gates + c.gates - 1) / c.gates;
    } else {
        c.cuts = (c.per_gate + want - 1) / want;
        c.size = (c.per_gate + c.cuts - 1) / c.cuts;
        c.cuts = (c.per_gate + c.size - 1) / c.size;
        c.chunks = gates * c.cuts;
    }
    return c;
}

template <typename T, typename P, int E, int W, int V>
__global__ __launch_bounds__(64 * W) void block_norm_grad_kernel(BlockNormGradLaunch a, Chunks ch, float *part_pre,
                                                                 float *part_post, float *part_gate)
{
    constexpr int STRIDE = 64 * W * E;
    __shared__ float sh3[2][W][3], sh1[2][W][1];
    const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
    TeamSum<W, 3> total3{sh3, 0};
    TeamSum<W, 1> total1{sh1, 0};
    const int dim = (int)a.dim, col0 = (64 * wave + lane) * E;
    const float inv = 1.0f / (float)dim;
    int64_t first, last;
    if (ch.gates) first = blockIdx.x * ch.size, last = first + ch.size < a.rows ? first + ch.size : a.rows;
    else {
        const int64_t g = blockIdx.x / ch.cuts, k = blockIdx.x - g * ch.cuts;
        first = g * ch.per_gate + k * ch.size;
        last = (k + 1) * ch.size < ch.per_gate ? first + ch.size : (g + 1) * ch.per_gate;
    }
    float dpre[V][E], dpost[V][E], dgate[V][E];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) dpre[i][e] = dpost[i][e] = dgate[i][e] = 0.0f;

    int64_t gate_row = a.gate ? first / ch.per_gate : 0, gate_end = (gate_row + 1) * ch.per_gate;
    for (int64_t row = first; row < last; ++row) {
        float x[V][E], y[V][E], d[V][E], t[V][E];
        float s[3] = {0.0f, 0.0f, 0.0f};    // of h'^2, v h', y^2
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = col0 + i * STRIDE;
            const bool in = c < dim;
            auto get = [&](const void *p, int64_t ld, float *v) {
                if (p && in) load_run<T, E>(static_cast<const T *>(p) + row * ld + c, v);
                else
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] = 0.0f;
            };
            get(a.h_out, a.ldh, x[i]);
            get(a.dz, a.ldz, t[i]);
            get(a.dh_out, a.ldd, d[i]);
            get(a.y, a.ldy, y[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = col0 + i * STRIDE;
            float w[E];
            if (a.pre && c < dim) load_run<P, E>(static_cast<const P *>(a.pre) + c, w);
            else
#pragma unroll
                for (int e = 0; e < E; ++e) w[e] = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s[0] = fmaf(x[i][e], x[i][e], s[0]);
                s[1] = fmaf(t[i][e] * (w[e] + a.offset), x[i][e], s[1]);
                s[2] = fmaf(y[i][e], y[i][e], s[2]);
            }
        }
        total3(s, lane, wave);
        if (a.dz) {
            const float rh = rsqrtf(fmaf(s[0], inv, a.eps));
            const float k = -(s[1] * inv * rh) * rh;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = col0 + i * STRIDE;
                float w[E];
                if (c < dim) load_run<P, E>(static_cast<const P *>(a.pre) + c, w);
                else
#pragma unroll
                    for (int e = 0; e < E; ++e) w[e] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float xh = x[i][e] * rh;
                    dpre[i][e] = fmaf(t[i][e], xh, dpre[i][e]);
                    d[i][e] += fmaf(k, xh, t[i][e] * rh * (w[e] + a.offset));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = col0 + i * STRIDE;
            if (c < dim) store_run<T, E>(static_cast<T *>(a.dh) + row * dim + c, d[i]);
        }
        if (a.y) {
            if (row >= gate_end) ++gate_row, gate_end += ch.per_gate;
            const P *gate = static_cast<const P *>(a.gate) + gate_row * a.ldg;
            const float ry = a.post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.0f;
            float sw = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = col0 + i * STRIDE;
                float g[E], p[E];
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 1.0f, p[e] = 1.0f;
                if (a.gate && c < dim) load_run<P, E>(gate + c, g);
                if (a.post && c < dim) {
                    load_run<P, E>(static_cast<const P *>(a.post) + c, p);
#pragma unroll
                    for (int e = 0; e < E; ++e) p[e] += a.offset;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float yh = y[i][e] * ry, sd = a.scale * d[i][e];
                    const float du = sd * g[e];
                    dgate[i][e] = fmaf(sd, yh * p[e], dgate[i][e]);
                    dpost[i][e] = fmaf(du, yh, dpost[i][e]);
                    t[i][e] = du * p[e];
                    sw = fmaf(t[i][e], y[i][e], sw);
                }
            }
            float k = 0.0f;
            if (a.post) {
                total1(&sw, lane, wave);
                k = -(sw * inv * ry) * ry;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = col0 + i * STRIDE;
                float v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = fmaf(k, y[i][e] * ry, t[i][e] * ry);
                if (c < dim) store_run<T, E>(static_cast<T *>(a.dy) + row * dim + c, v);
            }
            if (a.dgate && ch.gates && row + 1 == gate_end) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = col0 + i * STRIDE;
                    if (c < dim) store_run<P, E>(static_cast<P *>(a.dgate) + gate_row * dim + c, dgate[i]);
#pragma unroll
                    for (int e = 0; e < E; ++e) dgate[i][e] = 0.0f;
                }
            }
        }
    }
    const int64_t at = (int64_t)blockIdx.x * dim;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = col0 + i * STRIDE;
        if (c >= dim) continue;
        if (part_pre) store_run<float, E>(part_pre + at + c, dpre[i]);
        if (part_post) store_run<float, E>(part_post + at + c, dpost[i]);
        if (part_gate) store_run<float, E>(part_gate + at + c, dgate[i]);
    }
}

// out[g][c] = sum over the chunks g * cuts .. of part[chunk][c], in order within
// each of the workgroup's runs and over them.
constexpr int kSumRuns = 16, kSumCols = 64;
template <typename P>
__global__ __launch_bounds__(kSumRuns * kSumCols) void column_sum_kernel(const float *part, int64_t cuts, int dim, P *out,
                                                                         int64_t gate0)
{
    __shared__ float sh[kSumRuns][kSumCols];
    const int lane = (int)threadIdx.x % kSumCols, run = (int)threadIdx.x / kSumCols;
    const int c = (int)blockIdx.x * kSumCols + lane;
    const int64_t g = gate0 + blockIdx.y;
    float s = 0.0f;
    if (c < dim) {
        const float *p = part + g * cuts * dim + c;
#pragma unroll 8
        for (int64_t k = run; k < cuts; k += kSumRuns) s += p[k * dim];
    }
    sh[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < dim) {
#pragma unroll
        for (int r = 1; r < kSumRuns; ++r) s += sh[r][lane];
        Elt<P>::store(out, g * dim + c, s);
    }
}

template <typename P> hipError_t column_sum(const float *part, int64_t gates, int64_t cuts, int64_t dim, void *out, hipStream_t stream)
{
    for (int64_t g = 0; g < gates; g += 65535) {
        const dim3 grid((unsigned)((dim + kSumCols - 1) / kSumCols), (unsigned)std::min<int64_t>(65535, gates - g));
        column_sum_kernel<P><<<grid, kSumRuns * kSumCols, 0, stream>>>(part, cuts, (int)dim, static_cast<P *>(out), g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

bool aligned(const void *p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, typename P, int E, int W, int V> hipError_t forward(const BlockNormLaunch &a, hipStream_t stream)
{
    const int64_t groups = (a.rows + teams<W>() - 1) / teams<W>();
    const unsigned grid = (unsigned)std::min<int64_t>(groups, 1 << 20);
    block_norm_kernel<T, P, E, W, V><<<grid, 64 * W * teams<W>(), 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, typename P, int E, int W, int V> hipError_t backward(const BlockNormGradLaunch &a, hipStream_t stream)
{
    const Chunks ch = chunks_of(a.rows, a.gates);
    const int64_t part = ch.chunks * a.dim;
    float *at = a.partials, *pre = nullptr, *post = nullptr, *gate = nullptr;
    if (a.dpre) pre = at, at += part;
    if (a.dpost) post = at, at += part;
    if (a.dgate && !ch.gates) gate = at;
    hipError_t e = hipSuccess;
    if (ch.chunks) {
        block_norm_grad_kernel<T, P, E, W, V><<<(unsigned)ch.chunks, 64 * W, 0, stream>>>(a, ch, pre, post, gate);
        e = hipGetLastError();
    }
    if (e == hipSuccess && a.dpre) e = column_sum<P>(pre, 1, ch.chunks, a.dim, a.dpre, stream);
    if (e == hipSuccess && a.dpost) e = column_sum<P>(post, 1, ch.chunks, a.dim, a.dpost, stream);
    if (e == hipSuccess && a.dgate && !ch.gates) e = column_sum<P>(gate, a.gates, ch.cuts, a.dim, a.dgate, stream);
    return e;
}

// The smallest team that holds a row in 16 elements per thread (32 in fp32
// past 8192).
template <template <typename, typename, int, int, int> class Go, typename T, typename P, int E, typename A>
hipError_t by_width(const A &a, hipStream_t stream)
{
    constexpr int V = 16 / E;
    const int64_t dim = a.dim;
    if (dim <= 64 * E) return Go<T, P, E, 1, 1>::run(a, stream);
    if (dim <= 1024) return Go<T, P, E, 1, V>::run(a, stream);
    if (dim <= 2048) return Go<T, P, E, 2, V>::run(a, stream);
    if (dim <= 4096) return Go<T, P, E, 4, V>::run(a, stream);
    if (dim <= 8192) return Go<T, P, E, 8, V>::run(a, stream);
    return Go<T, P, E, 16, V>::run(a, stream);
}

template <typename T, typename P, int E, int W, int V> struct Forward {
    static hipError_t run(const BlockNormLaunch &a, hipStream_t s) { return forward<T, P, E, W, V>(a, s); }
};
template <typename T, typename P, int E, int W, int V> struct Backward {
    static hipError_t run(const BlockNormGradLaunch &a, hipStream_t s) { return backward<T, P, E, W, V>(a, s); }
};

// Whether all rows can be moved 16 bytes of T at a time.
bool wide(const BlockNormLaunch &a, int e)
{
    return a.dim % e == 0 && a.ldh % e == 0 && a.ldy % e == 0 && a.ldg % e == 0 && aligned(a.h) && aligned(a.y) &&
           aligned(a.post) && aligned(a.gate) && aligned(a.pre) && aligned(a.h_out) && aligned(a.z);
}
bool wide(const BlockNormGradLaunch &a, int e)
{
    return a.dim % e == 0 && a.ldh % e == 0 && a.ldy % e == 0 && a.ldd % e == 0 && a.ldz % e == 0 && a.ldg % e == 0 &&
           aligned(a.h_out) && aligned(a.y) && aligned(a.dh_out) && aligned(a.dz) && aligned(a.post) && aligned(a.gate) &&
           aligned(a.pre) && aligned(a.dh) && aligned(a.dy) && aligned(a.dpost) && aligned(a.dgate) && aligned(a.dpre);
}

template <template <typename, typename, int, int, int> class Go, typename T, typename P, typename A>
hipError_t by_alignment(const A &a, hipStream_t stream)
{
    constexpr int E = 16 / (int)sizeof(T);
    return wide(a, E) ? by_width<Go, T, P, E>(a, stream) : by_width<Go, T, P, 1>(a, stream);
}

template <template <typename, typename, int, int, int> class Go, typename A> hipError_t by_types(const A &a, hipStream_t stream)
{
    if (a.x_dt == 0)
        return a.p_dt == 0 ? by_alignment<Go, float, float>(a, stream) : by_alignment<Go, float, bf16_bits>(a, stream);
    return a.p_dt == 0 ? by_alignment<Go, bf16_bits, float>(a, stream) : by_alignment<Go, bf16_bits, bf16_bits>(a, stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormLaunch &a, hipStream_t stream) { return by_types<Forward>(a, stream); }

// A row of fp32 sums for each chunk and each of three parameters.
size_t block_norm_grad_ws_bytes(int64_t rows, int64_t dim, int64_t gates)
{
    return (size_t)(3 * chunks_of(rows, gates).chunks * dim) * sizeof(float);
}

hipError_t launch_block_norm_grad(const BlockNormGradLaunch &a, hipStream_t stream) { return by_types<Backward>(a, stream); }

}  // namespace nqk
