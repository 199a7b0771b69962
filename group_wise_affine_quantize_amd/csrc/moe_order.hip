// Tokens sorted by expert and back (contract in include/nq.h).
//
// Sorting is a stable counting sort of the pairs (token, choice) by their
// expert; experts that do not exist count as one more, behind the others.  A
// pair's place is
//   pairs of lower experts + earlier pairs of its own expert.
// Waves own runs of neighbouring pairs.  They count their experts (integer
// adds in LDS, whose order does not matter), the counts are summed over
// lower experts and earlier waves, and each wave then gives out places, 64
// pairs at a time: a ballot for each bit of the expert's number tells a lane
// which lanes have its expert, and how many of them come before it.
//
// Moving rows: a thread takes 16 bytes of a token's row.  Dispatch reads
// them once and writes top_k copies; combine reads top_k rows' and adds them in
// fp32 in the order of the choices; its gradient does both and adds
// the products for the weights over the row.
//
// What bounds it: sorting is latency (the ids are 4 bytes a pair); moving is
// memory, each row once.  Experts' rows are read past the caches, which they
// would fill in vain (8192 tokens of 8 rows of 8 KB, 30 % dropped, combined: 104
// -> 91 us, 5.6 TB/s; 6 rows of 4 KB and their gradients 86 -> 75 in a row of calls,
// 5.8 TB/s; 90 to 95 among a training step's other calls).  Rows off 16-byte
// alignment take more registers and share lines: the same gradient at 2047 columns
// takes 169 us for 78.
#include <algorithm>

#include "nq_kv_device.h"
#include "nq_layer.h"
#include "nq_vec.h"

namespace nqk {

namespace {

// ---------------------------------------------------------------- sorting
constexpr int kSortWaves = 16, kSortThreads = 64 * kSortWaves;
constexpr int kMaxBuckets = 1025;       // 1024 experts and those that do not exist
// Pairs up to which one workgroup sorts them all; more are cut into parts.
constexpr int64_t kOnePart = 8192;
constexpr int64_t kPart = 2048;
constexpr int kMostParts = 256;

int64_t sort_parts(int64_t pairs)
{
    return pairs <= kOnePart ? 1 : std::min<int64_t>(kMostParts, (pairs + kPart - 1) / kPart);
}
// Pairs of a part: whole rounds of 64 for each wave.
int64_t part_size(int64_t pairs, int64_t parts)
{
    const int64_t per = (pairs + parts - 1) / parts;
    return (per + kSortThreads - 1) / kSortThreads * kSortThreads;
}

__device__ __forceinline__ int bucket_of(uint32_t id, int experts) { return id < (uint32_t)experts ? (int)id : experts; }

// The run of pairs of a wave.
struct Run {
    int64_t first, last;
};
__device__ __forceinline__ Run run_of(const MoeSortLaunch &a, int64_t part, int64_t size, int wave)
{
    const int64_t each = size / kSortWaves;
    Run r;
    r.first = part * size + wave * each;
    r.last = r.first + each;
    if (r.last > a.pairs) r.last = a.pairs;
    return r;
}

// counts[part][bucket], for parts that several workgroups sort.
__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(MoeSortLaunch a, int64_t size)
{
    __shared__ int hist[kMaxBuckets];
    const int tid = (int)threadIdx.x, buckets = a.experts + 1;
    for (int b = tid; b < buckets; b += kSortThreads) hist[b] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * size, last = first + size < a.pairs ? first + size : a.pairs;
    for (int64_t p = first + tid; p < last; p += kSortThreads) atomicAdd(&hist[bucket_of(a.ids[p], a.experts)], 1);
    __syncthreads();
    for (int b = tid; b < buckets; b += kSortThreads) a.counts[(int64_t)blockIdx.x * buckets + b] = hist[b];
}

__global__ __launch_bounds__(kSortThreads) void moe_place_kernel(MoeSortLaunch a, int64_t size)
{
    __shared__ int hist[kSortWaves][kMaxBuckets];
    __shared__ int base[kMaxBuckets];
    __shared__ int sums[kSortWaves];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6, buckets = a.experts + 1;
    const int parts = (int)gridDim.x, part = (int)blockIdx.x;
    for (int b = lane; b < buckets; b += 64) hist[wave][b] = 0;
    __syncthreads();
    const Run run = run_of(a, part, size, wave);
    for (int64_t p = run.first + lane; p < run.last; p += 64) atomicAdd(&hist[wave][bucket_of(a.ids[p], a.experts)], 1);
    __syncthreads();
    // per bucket: waves' first places inside the part, the whole count, and the earlier parts'
    auto count = [&](int b, int &before, int &total) {
        int in_part = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const int n = hist[w][b];
            hist[w][b] = in_part;
            in_part += n;
        }
        before = 0, total = in_part;
        if (parts == 1) return;
        total = 0;
#pragma unroll 16
        for (int q = 0; q < parts; ++q) {
            const int n = a.counts[(int64_t)q * buckets + b];
            before += q < part ? n : 0;
            total += n;
        }
    };
    int before = 0, total = 0;
    if (tid < buckets) count(tid, before, total);
    // exclusive sums over the buckets; of 1025, the last comes behind all others
    const int upto = (int)wave_scan32((uint32_t)total);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int at = upto - total;
    for (int w = 0; w < wave; ++w) at += sums[w];
    if (tid < buckets) {
        base[tid] = at + before;
        if (part == 0) a.starts[tid] = at;
    }
    if (buckets > kSortThreads && tid == kSortThreads - 1) {
        at += total;
        count(kSortThreads, before, total);
        base[kSortThreads] = at + before;
        if (part == 0) a.starts[kSortThreads] = at;
    }
    __syncthreads();
    // places, in the order of the pairs
    const int bits = 32 - __clz(buckets - 1 | 1);
    volatile int *next = hist[wave];
    for (int64_t p0 = run.first; p0 < run.last; p0 += 64) {
        const int64_t p = p0 + lane;
        const bool in = p < run.last;
        const uint32_t id = in ? a.ids[p] : 0u;
        const int b = bucket_of(id, a.experts);
        uint64_t same = __ballot(in);
        for (int i = 0; i < bits; ++i) {
            const uint64_t set = __ballot((b >> i) & 1);
            same &= (b >> i) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
        const int first = next[b];
        __builtin_amdgcn_wave_barrier();
        if (in) {
            if (rank == 0) next[b] = first + __popcll(same);
            const int place = base[b] + first + rank;
            a.place[p] = place;
            a.row_token[place] = (uint32_t)p / (uint32_t)a.top_k;
            a.row_expert[place] = id;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ---------------------------------------------------------------- moving
constexpr int kRowThreads = 256;

// A row's place among `rows`, or -1 where there is none: places are read from
// memory that a caller may have filled with anything.
__device__ __forceinline__ int64_t checked(int place, int64_t rows) { return place >= 0 && place < rows ? place : -1; }

// Teams of 1 << shift threads take a token's row each, `pieces` runs of E elements.
struct Teams {
    int shift;
    int64_t pieces;
    int64_t token0;
};

// FAR: xs is more than the caches hold, and passes them by.
template <typename T, int E, bool AL, bool FAR> __global__ __launch_bounds__(kRowThreads) void moe_dispatch_kernel(MoeRowsLaunch a, Teams m)
{
    const int lane = (int)threadIdx.x & ((1 << m.shift) - 1);
    const int64_t t = m.token0 + ((int64_t)blockIdx.x << (8 - m.shift)) + ((int)threadIdx.x >> m.shift);
    if (t >= a.tokens) return;
    const int64_t rows = a.tokens * a.top_k;
    const int kept = *a.kept;
    const int32_t *place = a.place + t * a.top_k;
    const T *x = static_cast<const T *>(a.in) + t * a.ldi;
    T *out = static_cast<T *>(a.out);
    for (int64_t c = lane + ((int64_t)blockIdx.y << m.shift); c < m.pieces; c += (int64_t)gridDim.y << m.shift) {
        const Raw<T, E> v = load_cols<T, E, AL>(x, c * E, a.hidden);
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t r = checked(place[j], rows);
            if (r >= 0) store_cols<T, E, AL, FAR>(out + r * a.hidden, c * E, a.hidden, r < kept ? v : raw_zero<T, E>());
        }
    }
}

template <typename T, int E, bool AL> __global__ __launch_bounds__(kRowThreads) void moe_combine_kernel(MoeRowsLaunch a, Teams m)
{
    constexpr int K = 8;        // rows on the way at once
    const int lane = (int)threadIdx.x & ((1 << m.shift) - 1);
    const int64_t t = m.token0 + ((int64_t)blockIdx.x << (8 - m.shift)) + ((int)threadIdx.x >> m.shift);
    if (t >= a.tokens) return;
    const int64_t rows = std::min<int64_t>(a.tokens * a.top_k, *a.kept);
    const int32_t *place = a.place + t * a.top_k;
    const float *weights = a.weights ? a.weights + t * a.top_k : nullptr;
    const T *in = static_cast<const T *>(a.in);
    for (int64_t c = lane + ((int64_t)blockIdx.y << m.shift); c < m.pieces; c += (int64_t)gridDim.y << m.shift) {
        float sum[E];
        if (a.residual) unpack<T, E>(load_cols<T, E, AL>(static_cast<const T *>(a.residual) + t * a.ldr, c * E, a.hidden), sum);
        else
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] = 0.0f;
        for (int j0 = 0; j0 < a.top_k; j0 += K) {
            Raw<T, E> v[K];
            float w[K];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                v[j] = raw_zero<T, E>(), w[j] = 0.0f;
                if (j0 + j >= a.top_k) continue;
                const int64_t r = checked(place[j0 + j], rows);
                if (r < 0) continue;
                v[j] = load_cols<T, E, AL, true>(in + r * a.hidden, c * E, a.hidden);
                w[j] = weights ? weights[j0 + j] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float f[E];
                unpack<T, E>(v[j], f);
#pragma unroll
                for (int e = 0; e < E; ++e) sum[e] = fmaf(w[j], f[e], sum[e]);
            }
        }
        store_cols<T, E, AL>(static_cast<T *>(a.out) + t * a.hidden, c * E, a.hidden, pack<T, E>(sum));
    }
}

// A team takes a whole row here (its sums), TEAM threads.
template <typename T, int E, int TEAM, bool AL>
__global__ __launch_bounds__(kRowThreads) void moe_combine_grad_kernel(MoeRowsLaunch a, Teams m)
{
    constexpr int K = 8, WAVES = TEAM > 64 ? TEAM / 64 : 1;
    __shared__ float sh[WAVES][K];
    const int lane = (int)threadIdx.x % TEAM;
    const int64_t t = m.token0 + (int64_t)blockIdx.x * (kRowThreads / TEAM) + (int)threadIdx.x / TEAM;
    if (TEAM < kRowThreads && t >= a.tokens) return;    // whole waves or, in smaller teams, no exchange with these lanes
    const int64_t rows = a.tokens * a.top_k;
    const int kept = *a.kept;
    const int32_t *place = a.place + t * a.top_k;
    const T *dy = static_cast<const T *>(a.in) + t * a.ldi, *ys = static_cast<const T *>(a.ys);
    T *dys = static_cast<T *>(a.out);
    for (int j0 = 0; j0 < a.top_k; j0 += K) {
        int64_t at[K];
        float w[K], s[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const bool in = j0 + j < a.top_k;
            at[j] = in ? checked(place[in ? j0 + j : 0], rows) : -1;
            w[j] = in && a.weights ? a.weights[t * a.top_k + j0 + j] : 1.0f;
            s[j] = 0.0f;
        }
        for (int64_t c = lane; c < m.pieces; c += TEAM) {
            float g[E];
            unpack<T, E>(load_cols<T, E, AL>(dy, c * E, a.hidden), g);
            Raw<T, E> v[K];
            if (a.dweights) {
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    v[j] = raw_zero<T, E>();
                    if (at[j] >= 0 && at[j] < kept) v[j] = load_cols<T, E, AL, true>(ys + at[j] * a.hidden, c * E, a.hidden);
                }
            }
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (at[j] < 0) continue;
                const bool there = at[j] < kept;
                float f[E], d[E];
                if (a.dweights) {
                    unpack<T, E>(v[j], f);
#pragma unroll
                    for (int e = 0; e < E; ++e) s[j] = there ? fmaf(g[e], f[e], s[j]) : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] = there ? w[j] * g[e] : 0.0f;
                store_cols<T, E, AL>(dys + at[j] * a.hidden, c * E, a.hidden, pack<T, E>(d));
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int j = 0; j < K; ++j) s[j] = lane_sum<(TEAM < 64 ? TEAM : 64)>(s[j], (int)threadIdx.x & 63);
        if constexpr (WAVES > 1) {
            const int wave = lane >> 6;
            __syncthreads();
            if ((lane & 63) == 0)
#pragma unroll
                for (int j = 0; j < K; ++j) sh[wave][j] = s[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < K; ++j) {
                s[j] = sh[0][j];
#pragma unroll
                for (int i = 1; i < WAVES; ++i) s[j] += sh[i][j];
            }
        }
        if (lane == 0)
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (j0 + j < a.top_k) a.dweights[t * a.top_k + j0 + j] = s[j];
    }
}

bool aligned_rows(const MoeRowsLaunch &a, int e)
{
    const uintptr_t bits = (uintptr_t)a.in | (uintptr_t)a.out | (uintptr_t)a.residual | (uintptr_t)a.ys;
    return (bits & 15) == 0 && a.hidden % e == 0 && a.ldi % e == 0 && a.ldr % e == 0;
}

Teams teams_of(const MoeRowsLaunch &a, int e)
{
    Teams m;
    m.pieces = (a.hidden + e - 1) / e;
    m.shift = 0;
    while (m.shift < 8 && ((int64_t)1 << m.shift) < m.pieces) ++m.shift;
    m.token0 = 0;
    return m;
}

// Launches over all tokens, `y` workgroups to a row.
template <typename Kernel> hipError_t over_tokens(const MoeRowsLaunch &a, Teams m, unsigned y, Kernel kernel, hipStream_t stream)
{
    const int per = kRowThreads >> m.shift;
    const int64_t most = most_workgroups(kRowThreads) / y * per;
    for (m.token0 = 0; m.token0 < a.tokens; m.token0 += most) {
        const int64_t n = std::min<int64_t>(most, a.tokens - m.token0);
        kernel<<<dim3((unsigned)((n + per - 1) / per), y), kRowThreads, 0, stream>>>(a, m);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Workgroups to a row: one for every two rounds of its pieces.
unsigned rounds(const Teams &m) { return (unsigned)std::min<int64_t>(64, ((m.pieces >> m.shift) + 1) / 2 + (m.pieces >> m.shift == 0)); }

template <typename T, int E, bool AL> struct Dispatch {
    static hipError_t run(const MoeRowsLaunch &a, hipStream_t stream)
    {
        const Teams m = teams_of(a, E);
        // 65536 rows of 8 KB (537 MB): 116 -> 102 us; 49152 of 4 KB (201 MB): 35 without, 38 with
        const bool far = a.tokens * a.top_k * a.hidden * (int64_t)sizeof(T) > (int64_t)256 << 20;
        return far ? over_tokens(a, m, rounds(m), moe_dispatch_kernel<T, E, AL, true>, stream)
                   : over_tokens(a, m, rounds(m), moe_dispatch_kernel<T, E, AL, false>, stream);
    }
};
template <typename T, int E, bool AL> struct Combine {
    static hipError_t run(const MoeRowsLaunch &a, hipStream_t stream)
    {
        const Teams m = teams_of(a, E);
        return over_tokens(a, m, rounds(m), moe_combine_kernel<T, E, AL>, stream);
    }
};
template <typename T, int E, bool AL> struct CombineGrad {
    static hipError_t run(const MoeRowsLaunch &a, hipStream_t stream)
    {
        Teams m = teams_of(a, E);
        if (m.shift == 8) return over_tokens(a, m, 1, moe_combine_grad_kernel<T, E, 256, AL>, stream);
        if (m.shift > 4) {
            m.shift = 6;
            return over_tokens(a, m, 1, moe_combine_grad_kernel<T, E, 64, AL>, stream);
        }
        m.shift = 4;
        return over_tokens(a, m, 1, moe_combine_grad_kernel<T, E, 16, AL>, stream);
    }
};

template <template <typename, int, bool> class Go> hipError_t rows_go(const MoeRowsLaunch &a, hipStream_t stream)
{
    if (a.x_dt == 0) return aligned_rows(a, 4) ? Go<float, 4, true>::run(a, stream) : Go<float, 4, false>::run(a, stream);
    return aligned_rows(a, 8) ? Go<bf16_bits, 8, true>::run(a, stream) : Go<bf16_bits, 8, false>::run(a, stream);
}

}  // namespace

size_t moe_sort_ws_bytes(int64_t pairs, int experts)
{
    const int64_t parts = sort_parts(pairs);
    return parts == 1 ? 0 : (size_t)(parts * (experts + 1)) * sizeof(int32_t);
}

hipError_t launch_moe_sort(const MoeSortLaunch &a, hipStream_t stream)
{
    const int64_t parts = sort_parts(a.pairs), size = part_size(a.pairs, parts);
    if (parts > 1) {
        moe_count_kernel<<<(unsigned)parts, kSortThreads, 0, stream>>>(a, size);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    moe_place_kernel<<<(unsigned)parts, kSortThreads, 0, stream>>>(a, size);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch(const MoeRowsLaunch &a, hipStream_t stream) { return rows_go<Dispatch>(a, stream); }
hipError_t launch_moe_combine(const MoeRowsLaunch &a, hipStream_t stream) { return rows_go<Combine>(a, stream); }
hipError_t launch_moe_combine_grad(const MoeRowsLaunch &a, hipStream_t stream) { return rows_go<CombineGrad>(a, stream); }

}  // namespace nqk
