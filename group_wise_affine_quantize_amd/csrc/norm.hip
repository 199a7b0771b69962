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
// What bounds it: memory, 4 moves of a row forward and 6 backward.  8191 rows of
// 4096 in bf16: 40 to 44 us, 6.1 to 6.7 TB/s (some of the rows lie in the last
// cache); the gradient of 8192 rows of 2048 42 to 50 us, 4.1 to 4.8 TB/s, and 4.6 for the
// sums over the chunks: 30 vector instructions for each element, 13 us of them,
// and what is exchanged over a row's waves.
#include <algorithm>

#include "nq_kv.h"
#include "nq_layer.h"
#include "nq_norm_chunks.h"
#include "nq_tiles.h"
#include "nq_vec.h"

namespace nqk {

namespace {

// Sums over a team of W waves, N at a time.  Slots alternate, so that one
// barrier per exchange is enough; it leaves global loads in flight.
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
            lds_barrier();
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

template <typename T, typename P, int E, int W, int V, bool AL>
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
    const P *post = static_cast<const P *>(a.post), *pre = static_cast<const P *>(a.pre);
    for (int64_t row = (int64_t)blockIdx.x * TEAMS + team; row < a.rows; row += (int64_t)gridDim.x * TEAMS) {
        const T *h = static_cast<const T *>(a.h) + row * a.ldh;
        const T *y = static_cast<const T *>(a.y) + row * a.ldy;
        const P *gate = static_cast<const P *>(a.gate) + (a.gate ? row / per_gate * a.ldg : 0);
        // everything is asked for before the first sum is waited for
        Raw<T, E> hr[V], yr[V];
        Raw<P, E> wpost[V], wgate[V], wpre[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = col0 + i * STRIDE;
            hr[i] = load_cols<T, E, AL>(h, c, dim);
            if (a.y) yr[i] = load_cols<T, E, AL>(y, c, dim);
            if (a.gate) wgate[i] = load_cols<P, E, AL>(gate, c, dim);
            if (a.post) wpost[i] = load_cols<P, E, AL>(post, c, dim);
            if (a.z) wpre[i] = load_cols<P, E, AL>(pre, c, dim);
        }
        float x[V][E];
#pragma unroll
        for (int i = 0; i < V; ++i) unpack<T, E>(hr[i], x[i]);
        if (a.y) {
            float u[V][E], s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                unpack<T, E>(yr[i], u[i]);
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(u[i][e], u[i][e], s);
            }
            float f = a.scale;
            if (a.post) {
                total(&s, lane, wave);
                f *= rsqrtf(fmaf(s, inv, a.eps));
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float w[E];
#pragma unroll
                for (int e = 0; e < E; ++e) u[i][e] *= f;
                if (a.post) {
                    unpack<P, E>(wpost[i], w);
#pragma unroll
                    for (int e = 0; e < E; ++e) u[i][e] *= w[e] + a.offset;
                }
                if (a.gate) {
                    unpack<P, E>(wgate[i], w);
#pragma unroll
                    for (int e = 0; e < E; ++e) u[i][e] *= w[e];
                }
#pragma unroll
                for (int e = 0; e < E; ++e) x[i][e] += u[i][e];
                store_cols<T, E, AL>(static_cast<T *>(a.h_out) + row * dim, col0 + i * STRIDE, dim, pack<T, E>(x[i]));
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
                float w[E], z[E];
                unpack<P, E>(wpre[i], w);
#pragma unroll
                for (int e = 0; e < E; ++e) z[e] = x[i][e] * r * (w[e] + a.offset);
                store_cols<T, E, AL>(static_cast<T *>(a.z) + row * dim, col0 + i * STRIDE, dim, pack<T, E>(z));
            }
        }
    }
}

// Teams of a workgroup of the gradient (eight waves, or one team): they take the rows of a chunk (or its
// gates' runs of rows) by turns and add up their sums at the end.
template <int W> constexpr int grad_teams() { return W >= 8 ? 1 : 8 / W; }

template <typename T, typename P, int E, int W, int V, bool AL>
__global__ __launch_bounds__(64 * W * grad_teams<W>()) void block_norm_grad_kernel(BlockNormGradLaunch a, Chunks ch, float *part_pre,
                                                                                  float *part_post, float *part_gate)
{
    constexpr int TEAMS = grad_teams<W>(), STRIDE = 64 * W * E, COLS = STRIDE * V;
    // rows past 8192 columns leave 128 registers to each thread of their 16
    // waves: nothing is kept there over the rows but dpre's sums, the others'
    // are in LDS, each thread's columns its own (2048 rows of 16384 in bf16: 274 us with
    // all in registers, of which 127 spilled; 146 so, with 12)
    constexpr bool LEAN = V * E == 16;
    __shared__ float sh3[TEAMS][2][W][3], sh1[TEAMS][2][W][1];
    __shared__ float sh_sum[TEAMS > 1 ? TEAMS - 1 : 1][TEAMS > 1 ? COLS : 1];
    __shared__ float4 sh_own[LEAN ? 2 : 1][LEAN ? V * E / 4 : 1][LEAN ? 64 * W : 1];     // dpost, dgate
    const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6) % W;
    const int team = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / W);
    TeamSum<W, 3> total3{sh3[team], 0};
    TeamSum<W, 1> total1{sh1[team], 0};
    const int dim = (int)a.dim, col0 = (64 * wave + lane) * E;
    const float inv = 1.0f / (float)dim;

    // The team's rows: runs of `run` rows, its k-th starting `team` + k * TEAMS
    // runs behind `first`.  All teams take the same number of steps (they
    // meet at barriers), some past the chunk's end.
    int64_t first, last, run = 1;
    if (ch.gates) {
        first = blockIdx.x * ch.size, last = first + ch.size < a.rows ? first + ch.size : a.rows;
        run = ch.per_gate;
    } else {
        const int64_t g = blockIdx.x / ch.cuts, k = blockIdx.x - g * ch.cuts;
        first = g * ch.per_gate + k * ch.size;
        last = (k + 1) * ch.size < ch.per_gate ? first + ch.size : (g + 1) * ch.per_gate;
    }
    const int64_t steps = ((last - first) / run + TEAMS - 1) / TEAMS * run;
    int64_t gate_row = a.gate ? (ch.gates ? first / ch.per_gate + team : first / ch.per_gate) : 0;

    constexpr int HELD = LEAN ? 1 : V;      // pieces of dpost and dgate in registers
    float dpre[V][E], dpost[HELD][E], dgate[HELD][E];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) dpre[i][e] = dpost[i % HELD][e] = dgate[i % HELD][e] = 0.0f;
    auto get_own = [&](int which, int i, float *v) {
#pragma unroll
        for (int q = 0; q < E / 4; ++q) {
            const float4 s = sh_own[which][i * (E / 4) + q][threadIdx.x];
            v[4 * q] = s.x, v[4 * q + 1] = s.y, v[4 * q + 2] = s.z, v[4 * q + 3] = s.w;
        }
    };
    auto put_own = [&](int which, int i, const float *v) {
#pragma unroll
        for (int q = 0; q < E / 4; ++q)
            sh_own[which][i * (E / 4) + q][threadIdx.x] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    };
    if constexpr (LEAN)
#pragma unroll
        for (int i = 0; i < V; ++i) put_own(0, i, dpost[0]), put_own(1, i, dgate[0]);
    Raw<P, E> wpre[V], wpost[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = col0 + i * STRIDE;
        if constexpr (LEAN) continue;
        wpre[i] = a.pre ? load_cols<P, E, AL>(static_cast<const P *>(a.pre), c, dim) : raw_zero<P, E>();
        wpost[i] = a.post ? load_cols<P, E, AL>(static_cast<const P *>(a.post), c, dim) : raw_zero<P, E>();
    }

    Raw<T, E> x[V], t[V], d0[V], y[V];
    auto load = [&](const void *p, int64_t ld, int64_t row, Raw<T, E> *to) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            to[i] = p && row < last ? load_cols<T, E, AL, true>(static_cast<const T *>(p) + row * ld, col0 + i * STRIDE, dim) : raw_zero<T, E>();
    };
    int64_t row = first + team * run;
    auto load_all = [&](int64_t r) {
        load(a.h_out, a.ldh, r, x), load(a.dz, a.ldz, r, t), load(a.dh_out, a.ldd, r, d0), load(a.y, a.ldy, r, y);
    };
    if constexpr (!LEAN) load_all(row);
    auto weight = [&](const void *p, const Raw<P, E> &kept, int i, float *w) {
        if constexpr (LEAN) {
            if (p) unpack<P, E>(load_cols<P, E, AL>(static_cast<const P *>(p), col0 + i * STRIDE, dim), w);
            else unpack<P, E>(raw_zero<P, E>(), w);
        } else unpack<P, E>(kept, w);
    };
    int64_t in_run = 0;
    for (int64_t step = 0; step < steps; ++step) {
        const bool there = row < last;
        if constexpr (LEAN) load_all(row);
        Raw<P, E> wgate[V];
        auto load_gate = [&](int i) {
            wgate[i] = load_cols<P, E, AL>(static_cast<const P *>(a.gate) + gate_row * a.ldg, col0 + i * STRIDE, dim);
        };
        if constexpr (!LEAN)
            if (a.gate && there)
#pragma unroll
                for (int i = 0; i < V; ++i) load_gate(i);
        int64_t next = row + 1;
        if (++in_run == run) in_run = 0, next = row + 1 + (TEAMS - 1) * run;
        float s[3] = {0.0f, 0.0f, 0.0f};    // of h'^2, v h', y^2
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float w[E], xf[E], tf[E], yf[E];
            weight(a.pre, wpre[i], i, w);
            unpack<T, E>(x[i], xf), unpack<T, E>(t[i], tf), unpack<T, E>(y[i], yf);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s[0] = fmaf(xf[e], xf[e], s[0]);
                s[1] = fmaf(tf[e] * (w[e] + a.offset), xf[e], s[1]);
                s[2] = fmaf(yf[e], yf[e], s[2]);
            }
        }
        total3(s, lane, wave);
        const float rh = rsqrtf(fmaf(s[0], inv, a.eps)), kh = -(s[1] * inv * rh) * rh;
        float d[V][E];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float w[E], xf[E], tf[E];
            unpack<T, E>(d0[i], d[i]);
            if (a.dz) {
                weight(a.pre, wpre[i], i, w);
                unpack<T, E>(x[i], xf), unpack<T, E>(t[i], tf);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float xh = xf[e] * rh;
                    dpre[i][e] = fmaf(tf[e], xh, dpre[i][e]);
                    d[i][e] += fmaf(kh, xh, tf[e] * rh * (w[e] + a.offset));
                }
            }
            if (there) store_cols<T, E, AL>(static_cast<T *>(a.dh) + row * dim, col0 + i * STRIDE, dim, pack<T, E>(d[i]));
        }
        // the next row's, while this one's second half runs
        if constexpr (!LEAN) load(a.h_out, a.ldh, next, x), load(a.dz, a.ldz, next, t), load(a.dh_out, a.ldd, next, d0);
        if (a.y) {
            const float ry = a.post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.0f;
            float sw = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float g[E], p[E], yf[E];
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 1.0f, p[e] = 1.0f;
                if (a.gate && there) {
                    if constexpr (LEAN) load_gate(i);
                    unpack<P, E>(wgate[i], g);
                }
                if (a.post) {
                    weight(a.post, wpost[i], i, p);
#pragma unroll
                    for (int e = 0; e < E; ++e) p[e] += a.offset;
                }
                unpack<T, E>(y[i], yf);
                if constexpr (LEAN) get_own(0, i, dpost[0]), get_own(1, i, dgate[0]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float yh = yf[e] * ry, sd = a.scale * d[i][e];
                    const float du = sd * g[e];
                    dgate[i % HELD][e] = fmaf(sd, yh * p[e], dgate[i % HELD][e]);
                    dpost[i % HELD][e] = fmaf(du, yh, dpost[i % HELD][e]);
                    d[i][e] = du * p[e];
                    sw = fmaf(d[i][e], yf[e], sw);
                }
                if constexpr (LEAN) put_own(0, i, dpost[0]), put_own(1, i, dgate[0]);
            }
            float ky = 0.0f;
            if (a.post) {
                total1(&sw, lane, wave);
                ky = -(sw * inv * ry) * ry;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float v[E], yf[E];
                unpack<T, E>(y[i], yf);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = fmaf(ky, yf[e] * ry, d[i][e] * ry);
                if (there) store_cols<T, E, AL>(static_cast<T *>(a.dy) + row * dim, col0 + i * STRIDE, dim, pack<T, E>(v));
            }
            if (ch.gates && in_run == 0) {
                if (a.dgate && there)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if constexpr (LEAN) get_own(1, i, dgate[0]);
                        store_cols<P, E, AL>(static_cast<P *>(a.dgate) + gate_row * dim, col0 + i * STRIDE, dim, pack<P, E>(dgate[i % HELD]));
                    }
#pragma unroll
                for (int i = 0; i < HELD; ++i)
#pragma unroll
                    for (int e = 0; e < E; ++e) dgate[i][e] = 0.0f;
                if constexpr (LEAN)
#pragma unroll
                    for (int i = 0; i < V; ++i) put_own(1, i, dgate[0]);
                if (a.gate) gate_row += TEAMS;
            }
        }
        if constexpr (!LEAN) load(a.y, a.ldy, next, y);
        row = next;
    }

    // the chunk's sums, the teams' in their order: to `part`, or to `out` where they
    // are all there is to add
    auto finish = [&](float (*sum)[E], int own, float *part, P *out, bool all) {
        if (all ? !out : !part) return;
        if constexpr (TEAMS > 1) {
            __syncthreads();
            if (team > 0)
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < E; ++e) sh_sum[team - 1][col0 + i * STRIDE + e] = sum[i][e];
            __syncthreads();
            if (team > 0) return;
#pragma unroll
            for (int k = 0; k < TEAMS - 1; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[i][e] += sh_sum[k][col0 + i * STRIDE + e];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = sum[LEAN && own >= 0 ? 0 : i][e];
            if constexpr (LEAN)
                if (own >= 0) get_own(own, i, v);
            if (all) store_cols<P, E, AL>(out, col0 + i * STRIDE, dim, pack<P, E>(v));
            else store_cols<float, E, AL>(part + (int64_t)blockIdx.x * dim, col0 + i * STRIDE, dim, pack<float, E>(v));
        }
    };
    const bool alone = ch.chunks == 1;
    finish(dpre, -1, part_pre, static_cast<P *>(a.dpre), alone);
    finish(dpost, 0, part_post, static_cast<P *>(a.dpost), alone);
    // (gates of its own the chunk has written; one that it has all rows of is number blockIdx.x)
    P *of_gate = ch.gates ? nullptr : static_cast<P *>(a.dgate);
    if (TEAMS > 1 && of_gate) of_gate += (int64_t)blockIdx.x * dim;
    finish(dgate, 1, part_gate, of_gate, alone || (TEAMS > 1 && ch.cuts == 1));
}

// out[g][c] = sum over the chunks g * cuts .. of part[chunk][c], in order within
// each of the workgroup's runs and over them: of up to three parameters, of
// which the last may have many gates.
constexpr int kSumRuns = 16, kSumCols = 64;
struct ColumnSums {
    const float *part[3];
    void *out[3];
    int64_t cuts[3], gates[3];
    int dim;
};
template <typename P> __global__ __launch_bounds__(kSumRuns * kSumCols) void column_sum_kernel(ColumnSums a)
{
    __shared__ float sh[kSumRuns][kSumCols];
    const int lane = (int)threadIdx.x % kSumCols, run = (int)threadIdx.x / kSumCols;
    const int c = (int)blockIdx.x * kSumCols + lane, which = (int)blockIdx.z;
    P *out = static_cast<P *>(a.out[which]);
    if (!out) return;
    const int64_t cuts = a.cuts[which];
    for (int64_t g = blockIdx.y; g < a.gates[which]; g += gridDim.y) {
        float s = 0.0f;
        if (c < a.dim) {
            const float *p = a.part[which] + g * cuts * a.dim + c;
#pragma unroll 8
            for (int64_t k = run; k < cuts; k += kSumRuns) s += p[k * a.dim];
        }
        sh[run][lane] = s;
        __syncthreads();
        if (run == 0 && c < a.dim) {
#pragma unroll
            for (int r = 1; r < kSumRuns; ++r) s += sh[r][lane];
            Elt<P>::store(out, g * a.dim + c, s);
        }
        __syncthreads();
    }
}

bool aligned(const void *p) { return ((uintptr_t)p & 15) == 0; }

template <typename T, typename P, int E, int W, int V, bool AL> struct Forward {
    static hipError_t run(const BlockNormLaunch &a, hipStream_t stream)
    {
        const int64_t groups = (a.rows + teams<W>() - 1) / teams<W>();
        const unsigned grid = (unsigned)std::min<int64_t>(groups, 1 << 20);
        block_norm_kernel<T, P, E, W, V, AL><<<grid, 64 * W * teams<W>(), 0, stream>>>(a);
        return hipGetLastError();
    }
};
template <typename T, typename P, int E, int W, int V, bool AL> struct Backward {
    static hipError_t run(const BlockNormGradLaunch &a, hipStream_t stream)
    {
        const Chunks ch = norm_chunks(a.rows, a.gates, norm_grad_teams(a.dim));
        const int64_t part = ch.chunks * a.dim;
        float *at = a.partials, *pre = nullptr, *post = nullptr, *gate = nullptr;
        // the sums of a gate's parts; where workgroups have several teams, one that has all of
        // a gate's rows writes its gradient (a single team has whole gates when they are few
        // rows; and 16 waves would spill more: 2048 rows of 8192 in fp32 118 -> 128 us)
        const bool gates = a.dgate && !ch.gates && (grad_teams<W>() == 1 || ch.cuts != 1);
        if (ch.chunks > 1) {
            if (a.dpre) pre = at, at += part;
            if (a.dpost) post = at, at += part;
            if (gates) gate = at;
        }
        if (ch.chunks) {
            block_norm_grad_kernel<T, P, E, W, V, AL><<<(unsigned)ch.chunks, 64 * W * grad_teams<W>(), 0, stream>>>(a, ch, pre, post, gate);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        if (ch.chunks == 1) return hipSuccess;      // that workgroup wrote them
        if (!a.dpre && !a.dpost && !gates) return hipSuccess;
        const ColumnSums c{{pre, post, gate}, {a.dpre, a.dpost, gates ? a.dgate : nullptr}, {ch.chunks, ch.chunks, ch.cuts},
                           {1, 1, a.gates}, (int)a.dim};
        const dim3 grid((unsigned)((a.dim + kSumCols - 1) / kSumCols), (unsigned)(gates ? std::min<int64_t>(a.gates, 1024) : 1), gates ? 3 : 2);
        column_sum_kernel<P><<<grid, kSumRuns * kSumCols, 0, stream>>>(c);
        return hipGetLastError();
    }
};

// The smallest team that holds a row in `held` elements per thread.
template <template <typename, typename, int, int, int, bool> class Go, typename T, typename P, bool AL, int HELD, typename A>
hipError_t by_width(const A &a, hipStream_t stream)
{
    constexpr int E = 16 / (int)sizeof(T), V = HELD / E, W0 = 64 * HELD;
    const int64_t dim = a.dim;
    if (V > 1 && dim <= 64 * E) return Go<T, P, E, 1, 1, AL>::run(a, stream);
    if (dim <= W0) return Go<T, P, E, 1, V, AL>::run(a, stream);
    if (dim <= 2 * W0) return Go<T, P, E, 2, V, AL>::run(a, stream);
    if (dim <= 4 * W0) return Go<T, P, E, 4, V, AL>::run(a, stream);
    if (dim <= 8 * W0) return Go<T, P, E, 8, V, AL>::run(a, stream);
    if (dim <= 16 * W0) return Go<T, P, E, 16, V, AL>::run(a, stream);
    return Go<T, P, E, 16, 16 / E, AL>::run(a, stream);
}

// Whether all rows start at multiples of 16 bytes and end with a whole piece.
bool aligned_rows(const BlockNormLaunch &a, int e)
{
    return a.dim % e == 0 && a.ldh % e == 0 && a.ldy % e == 0 && a.ldg % e == 0 && aligned(a.h) && aligned(a.y) &&
           aligned(a.post) && aligned(a.gate) && aligned(a.pre) && aligned(a.h_out) && aligned(a.z);
}
bool aligned_rows(const BlockNormGradLaunch &a, int e)
{
    return a.dim % e == 0 && a.ldh % e == 0 && a.ldy % e == 0 && a.ldd % e == 0 && a.ldz % e == 0 && a.ldg % e == 0 &&
           aligned(a.h_out) && aligned(a.y) && aligned(a.dh_out) && aligned(a.dz) && aligned(a.post) && aligned(a.gate) &&
           aligned(a.pre) && aligned(a.dh) && aligned(a.dy) && aligned(a.dpost) && aligned(a.dgate) && aligned(a.dpre);
}

template <template <typename, typename, int, int, int, bool> class Go, int HELD, typename T, typename P, typename A>
hipError_t by_alignment(const A &a, hipStream_t stream)
{
    return aligned_rows(a, 8) ? by_width<Go, T, P, true, HELD>(a, stream) : by_width<Go, T, P, false, HELD>(a, stream);
}

template <template <typename, typename, int, int, int, bool> class Go, int HELD, typename A> hipError_t by_types(const A &a, hipStream_t stream)
{
    if (a.x_dt == 0)
        return a.p_dt == 0 ? by_alignment<Go, HELD, float, float>(a, stream) : by_alignment<Go, HELD, float, bf16_bits>(a, stream);
    return a.p_dt == 0 ? by_alignment<Go, HELD, bf16_bits, float>(a, stream) : by_alignment<Go, HELD, bf16_bits, bf16_bits>(a, stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormLaunch &a, hipStream_t stream) { return by_types<Forward, 16>(a, stream); }

// A row of fp32 sums for each chunk and each of three parameters; one chunk alone
// needs none.
size_t block_norm_grad_ws_bytes(int64_t rows, int64_t dim, int64_t gates)
{
    const int64_t chunks = norm_chunks(rows, gates, norm_grad_teams(dim)).chunks;
    return chunks == 1 ? 0 : (size_t)(3 * chunks * dim) * sizeof(float);
}

hipError_t launch_block_norm_grad(const BlockNormGradLaunch &a, hipStream_t stream) { return by_types<Backward, 8>(a, stream); }

}  // namespace nqk
