// Attention over the 8-bit key/value cache (contract in include/nq.h).
//
// Mathematics.  For a query row q and the visible tokens t of its sequence,
//   z_t = scale * q . k_t,   out = sum_t e^(z_t) v_t / sum_t e^(z_t),
// with k_t = sk_t * ck_t and v_t = sv_t * cv_t (block scales times codes).  In
// one pass over the tokens, in base 2 and with the value scale drawn into
// the exponent:
//   x_t = log2(e) * scale * sk_t * (q . ck_t) + log2(sv_t),
//   p_t = 2^(x_t - R),
//   O = sum_t p_t cv_t,      L = sum_t p_t / sv_t,      out = O / L.
// R, a column's reference, is set 14 below the maximum of x_t and moves (O and
// L are scaled) when a later maximum passes R + 14 by more than kSlack; the
// largest p_t lies in [2^14, 2^15.5).  Drawing sv into x makes p_t the whole
// weight of a code row, so that the second product runs on bare codes, and
// p_t fits fp16: 11 bits for weights within 2^-28 of the largest, an error of
// 2^-39 of it below (the tile kernel, whose weights start at 2^12: 2^-26 and
// 2^-37).  (bf16 would keep 8 bits, which shows in a bf16 result.)  Codes are exact in fp16.  A query row is taken times a power of
// two that brings its largest element to [2^14, 2^15); a bf16 element then is
// exact in fp16 down to 2^-28 of the largest.  fp32 rows and weights are the
// sum of two fp16 numbers and take two matrix products each: 22 bits while the
// second, at most 2^-11 of the number, is one of fp16's normal numbers (from
// 2^-14 up), that is for numbers from 2^-3 up -- 2^-17 of the largest, 2^-15 in
// the tile kernel's weights -- and an error of 2^-25 below.  Sums, references
// and the states O and L are fp32.
//
// p_t / sv_t is 2^(z_t - R) (z in base 2 here), whose range is not p_t's: a sum
// over tiny scales can pass fp32, and the p_t of a small scale beside a very
// large one be flushed though its weight in L is not small.  With scales in 2^-48 .. 2^16
// neither happens: p_t / sv_t is below 2^64, and p_t is only flushed for tokens
// whose weight is below 2^-60 of the largest.  From the first tile on that
// holds another scale, or a block of zeros (no logarithm: its tokens add to L
// alone), a wave keeps L = sum_t 2^(z_t - U) over a reference U of its own, by
// a second exponential of each score.
//
// Matrix products: S^T = K q^T and O^T = V^T P^T on 16x16x32 fp16 MFMA with
// the tokens in the rows of the first product.  Lane l (r = l % 16, g = l / 16)
// holds column (query row) r and, after the first product, tokens 16 g + 4 n +
// i of the 64-token tile (n the MFMA, i the register): the order in which K's
// rows are fed is free, and this one leaves each lane 16 neighbouring tokens,
// which are exactly the operand of the second product (16 bytes of a V^T row
// per lane).  No value moves between lanes but the running maximum.
//
// What bounds it: reading the codes.  64 sequences of 1k to 8k tokens, 8 heads of
// 128 in int8: 620 MB in 118 us, 5.2 TB/s (a 1 GiB copy moves 5.1), with two
// workgroups of four waves per compute unit, each wave with a tile of 16 KB on
// the way.  With more than 16 query columns two or four waves read the same tile, and
// less is on the way: 8 draft tokens over 131k tokens, 264 MB in 82 us.  One token at
// 333 is latency: 9.5 us.
#include <algorithm>

#include "nq_kv_attn.h"

namespace nqk {

namespace {

constexpr int kWorkers = 512;    // two workgroups of four waves per compute unit
constexpr int kJoinThreads = 512, kJoinCols = 4;
constexpr float kSlack = 1.5f;   // weights stay below 2^15.5, within fp16
constexpr int kWaves = 4;

// Units per worker.  At least two tiles for each wave, so that short contexts
// do not fall into parts that cost more to join than to read.
__device__ __forceinline__ uint32_t share_of(const AttnArgs &A, uint32_t total)
{
    return list_share(total, (uint32_t)A.workers, A.unit_shift ? 1u : 2u * kWaves);
}

// Finds the sequence of unit `at(share)` of the list: its number (-1: past the
// list's end), the unit's number inside it, the list's length and the share.
template <typename At>
__device__ __forceinline__ int stream_locate(const AttnArgs &A, int cols, At at, uint32_t *inside, uint32_t *total,
                                             uint32_t *share)
{
    const int batch = A.a.s.batch, lane = (int)(threadIdx.x & 63u);
    uint32_t work = lane < batch ? stream_seq(A, lane, cols).work : 0u;     // below 2^31
    uint32_t upto = wave_scan32_sat(work);
    uint32_t sum = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    *total = sum;
    for (int b = 64 + lane; b - lane < batch; b += 64)
        *total = add_sat(*total, (uint32_t)__builtin_amdgcn_readlane(
            (int)wave_scan32_sat(b < batch ? stream_seq(A, b, cols).work : 0u), 63));
    *total = list_total(*total);
    *share = share_of(A, *total);
    const uint32_t want = at(*share);
    if (want >= *total) return -1;
    uint32_t base = 0;      // at most `want`
    for (int b0 = 0; b0 < batch; b0 += 64) {
        if (b0) {
            work = b0 + lane < batch ? stream_seq(A, b0 + lane, cols).work : 0u;
            upto = wave_scan32_sat(work);
            sum = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
        }
        if (add_sat(base, sum) > want) {
            const int l = __ffsll((unsigned long long)__ballot(add_sat(base, upto) > want)) - 1;
            *inside = want - base - (uint32_t)__builtin_amdgcn_readlane((int)(upto - work), l);
            return b0 + l;
        }
        base += sum;
    }
    return -1;
}

// 16 bytes of codes.  ONCE: no other wave will want them, and they pass the
// caches by (64 sequences of 1k to 8k tokens 123 -> 121 us; with two column
// groups, which share them in the L1, it is 80 -> 104).
template <bool ONCE> __device__ __forceinline__ uint4 load_codes(const uint8_t *p)
{
    const uint4_t *q = reinterpret_cast<const uint4_t *>(p);
    uint4_t v;
    if constexpr (ONCE) v = __builtin_nontemporal_load(q);
    else v = *q;
    return __builtin_bit_cast(uint4, v);
}

// The state of a wave's 16 columns.
template <int D, int NP> struct State {
    half8_t q[D / 32][NP];
    float c;                     // log2(e) * scale / row power of two
    float m, l;                  // m: the reference, 14 below the maximum when set; weights are 2^(x - m)
    float u;                     // l's reference, where it is not m
    float4_t o[D / 16];
};

// CG groups of 16 columns; the waves of a group share its tiles.  A group's
// waves load the tiles of the other groups' waves too, out of the L1: two
// blocks of columns in one wave's registers would leave one wave per SIMD.
template <int D, int CG, int FMT, typename T>
__global__ __launch_bounds__(64 * kWaves, D <= 128 ? 2 : 1) void kv_stream_kernel(AttnArgs A)
{
    constexpr int NP = Parts<T>::n, COLS = 16 * CG, KS = D / 32, DT = D / 16, TL = kWaves / CG;
    constexpr int LDO = D + 4;
    __shared__ float2 sh_mu[TL][COLS];
    __shared__ float sh_l[TL][COLS];
    __shared__ float sh_o[TL > 1 ? TL / 2 : 1][COLS][LDO];
    const KvAttnLaunch &a = A.a;
    const int lane = (int)(threadIdx.x & 63u), wave = (int)(threadIdx.x >> 6);
    const int cg = wave % CG, turn = wave / CG;     // the wave's columns, its turn at their tiles
    const int r = lane & 15, g = lane >> 4, gk = r >> 2;
    const int sh = a.c.block_shift, bmask = (1 << sh) - 1;

    uint32_t inside, total, share;
    int b = stream_locate(A, COLS, [](uint32_t s) { return blockIdx.x * s; }, &inside, &total, &share);
    if (b < 0) return;
    uint32_t left = total - blockIdx.x * share < share ? total - blockIdx.x * share : share;
    StreamSeq s = stream_seq(A, b, COLS);

    while (left > 0) {
        while (inside >= s.work) {      // the next sequence with work
            inside -= s.work;
            if (++b >= a.s.batch) return;
            s = stream_seq(A, b, COLS);
        }
        const uint32_t seg = inside / s.units, unit0 = inside - seg * s.units;
        const int head = (int)(seg / s.ct);
        const int ctile = (int)(seg - (uint32_t)head * s.ct);
        const uint32_t units = s.units - unit0 < left ? s.units - unit0 : left;
        const bool whole = units == s.units;
        const int tile0 = (int)(unit0 << A.unit_shift);
        const int tile1 = unit0 + units == s.units ? s.nt : (int)((unit0 + units) << A.unit_shift);

        State<D, NP> st;
        uint32_t near = kNearScales;    // 0 where l has a reference of its own
        int col_lo, col_hi;
        {
            const Column c = column(A, s, ctile * COLS + 16 * cg + r, head);
            col_lo = c.lo, col_hi = c.hi;
            float f[KS][8], top = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (c.row >= 0)
                    load_f32x8<T>(static_cast<const T *>(a.q) + (int64_t)c.row * a.ldq + c.head * D + 64 * (ks >> 1) +
                                      16 * g + 8 * (ks & 1), f[ks]);
                else
                    for (int i = 0; i < 8; ++i) f[ks][i] = 0.0f;
                for (int i = 0; i < 8; ++i) top = larger(top, f[ks][i]);
            }
            float back;
            top = larger(top, xor_lane<16>(top, lane));
            const float up = row_scale(larger(top, xor_lane<32>(top, lane)), &back);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                for (int i = 0; i < 8; ++i) f[ks][i] *= up;
                split_half<NP>(f[ks], st.q[ks]);
            }
            st.c = a.scale * kLog2e * back;
            st.m = kNegInf, st.u = kNegInf;
            st.l = 0.0f;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) st.o[dt] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
        // tokens that some column sees, and tokens that every column sees
        const int count = s.n * A.group, last_col = (ctile + 1) * COLS < count ? (ctile + 1) * COLS - 1 : count - 1;
        const Column c0 = column(A, s, ctile * COLS, head), c1 = column(A, s, last_col, head);
        const int seg_lo = c0.lo, seg_hi = c1.hi, all_lo = c1.lo, all_hi = c0.hi;

        // A tile's blocks: of this lane's key rows, and of its value and score
        // tokens; -1 where no column sees the 16 tokens or no block holds them.
        const int *table = a.s.table + (int64_t)b * a.s.ldt;
        auto block_of = [&](int pos) -> int {
            if (pos >= seg_hi || pos + 16 <= seg_lo) return -1;     // also keeps pos inside the table
            const int id = table[pos >> sh];
            return id >= 0 && id < (int)a.c.blocks ? id : -1;
        };
        uint4 kw[4][D / 64], vw[DT];
        float sk, sv;
        auto load_keys = [&](int base, int idk) {
            const int pk = base + 16 * gk;
            const uint8_t *kp = a.c.k_codes + (int64_t)((((int64_t)(idk < 0 ? 0 : idk) * a.c.kv_heads + head) << sh) +
                                                        (pk & bmask) + (r & 3)) * D + 16 * g;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) kw[n][j] = load_codes<CG == 1>(kp + 4 * n * D + 64 * j);
        };
        auto load_values = [&](int base, int idv) {
            const int pv = base + 16 * g;
            const int64_t slab = (int64_t)(idv < 0 ? 0 : idv) * a.c.kv_heads + head;
            const uint8_t *vp = a.c.v_codes + ((slab * D + r) << sh) + (pv & bmask);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) vw[dt] = load_codes<CG == 1>(vp + ((16 * dt) << sh));
            sk = 0.0f, sv = 1.0f;
            if (idv >= 0) sk = a.c.k_scales[slab], sv = a.c.v_scales[slab];
        };

        // The loop keeps one tile's loads in flight: keys of the next tile go
        // out once this one's first product has read its registers, values
        // once the second has, block ids one tile before those.
        // Waves take tiles by turns; of blocks of 128 tokens, whose value rows
        // are two tiles long, both tiles, so that a wave uses whole lines.
        const int pair = sh == 7;
        auto after_of = [&](int t) {
            if (!pair) return t + TL;
            return ((s.t0 + t) & 1) ? t + 2 * TL - 1 : t + 1;
        };
        int ti = tile0 + turn;
        if (pair) ti = turn ? ((s.t0 + tile0) & ~1) + 2 * turn - s.t0 : tile0;
        int idk = -1, idv = -1, idk2 = -1, idv2 = -1;
        if (ti < tile1) {
            const int base = (s.t0 + ti) << 6;
            idk = block_of(base + 16 * gk), idv = block_of(base + 16 * g);
            if (after_of(ti) < tile1) {
                const int next = (s.t0 + after_of(ti)) << 6;
                idk2 = block_of(next + 16 * gk), idv2 = block_of(next + 16 * g);
            }
            load_keys(base, idk);
            load_values(base, idv);
        }
        for (; ti < tile1; ti = after_of(ti)) {
            const int base = (s.t0 + ti) << 6, pv = base + 16 * g;
            const int tn = after_of(ti);
            const bool more = tn < tile1, has = idv >= 0;
            const bool masked = base < all_lo || base + kTile > all_hi || __any(!has);

            float4_t S[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) S[n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const half8_t k0 = codes_to_half<FMT>(kw[n][j].x, kw[n][j].y);
                    const half8_t k1 = codes_to_half<FMT>(kw[n][j].z, kw[n][j].w);
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            S[n] = mfma(k0, st.q[2 * j][p], S[n]);
                            S[n] = mfma(k1, st.q[2 * j + 1][p], S[n]);
                        }
                }
            const int next = (s.t0 + tn) << 6;
            idk = idk2;
            if (more) load_keys(next, idk2);

            const bool zeros = sv == 0.0f;
            const float vs = zeros ? 1.0f : sv;
            const float lsv = fast_log2(vs);
            float isv = 1.0f / vs;
            half8_t P[2][NP];
            {
                const float f = st.c * sk;
                float x[16], mx = kNegInf;
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[4 * n + i] = fmaf(S[n][i], f, lsv);
                if (masked) {
                    const int lo = has ? col_lo - pv : 16, hi = col_hi - pv;
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = i < lo || i >= hi ? kNegInf : x[i];
                }
                if (__any(scale_place(sv) >= near)) {
                    if (near) st.u = st.m;
                    near = 0;
                    isv = 0.0f;
                    // a scale that is no number has made x NaN where tokens are seen
                    const float shift = lsv == lsv ? lsv : 0.0f;
                    add_weights(16, [&](int i) { return x[i] - shift; }, st.l, st.u);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = zeros ? kNegInf : x[i];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) mx = fmaxf(mx, x[i]);
                // the reference moves, and O with it, when a maximum passes it by kSlack
                const float over = group_max(mx, lane) - kPScale;
                if (__any(over > st.m + kSlack)) {
                    const float next = over > st.m + kSlack ? over : st.m;
                    const float alpha = next == kNegInf ? 0.0f : fast_exp2(st.m - next);
                    st.m = next;
                    if (near) st.l *= alpha;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) st.o[dt] *= alpha;
                }
                const float mref = st.m == kNegInf ? 0.0f : st.m;   // no token yet: every weight is 0
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] = fast_exp2(x[i] - mref);
                    sum += x[i];
                }
                st.l = fmaf(sum, isv, st.l);
                split_half<NP>(x, P[0]);
                split_half<NP>(x + 8, P[1]);
            }
            if constexpr (FMT == KV_FP8) {
                if (masked) {
                    // codes of tokens that no column sees are whatever memory
                    // holds, a NaN for instance: make them zeros
                    const int lo = has ? seg_lo - pv : 16, hi = seg_hi - pv;
                    uint32_t keep[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        keep[w] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (4 * w + e >= lo && 4 * w + e < hi) keep[w] |= 255u << (8 * e);
                    }
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt)
                        vw[dt].x &= keep[0], vw[dt].y &= keep[1], vw[dt].z &= keep[2], vw[dt].w &= keep[3];
                }
            }
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                const half8_t v0 = codes_to_half<FMT>(vw[dt].x, vw[dt].y);
                const half8_t v1 = codes_to_half<FMT>(vw[dt].z, vw[dt].w);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        st.o[dt] = mfma(v0, P[0][p], st.o[dt]);
                        st.o[dt] = mfma(v1, P[1][p], st.o[dt]);
                    }
            }
            idv = idv2;
            if (more) {
                load_values(next, idv2);
                if (after_of(tn) < tile1) {
                    const int after = (s.t0 + after_of(tn)) << 6;
                    idk2 = block_of(after + 16 * gk), idv2 = block_of(after + 16 * g);
                }
            }
        }

        // join the waves of a column group: references first, then sums by halves
        if (!near) {
            const float u = group_max(st.u, lane);
            st.l *= exp2_below(st.u, u);
            st.u = u;
        } else st.u = st.m;
        st.l = group_sum(st.l, lane);
        const int col = 16 * cg + r;
        if (g == 0) sh_mu[turn][col] = make_float2(st.m, st.u);
        __syncthreads();
        {
            float m = kNegInf, u = kNegInf;
            for (int w = 0; w < TL; ++w) m = fmaxf(m, sh_mu[w][col].x), u = fmaxf(u, sh_mu[w][col].y);
            const float f = exp2_below(st.m, m);
            st.l *= exp2_below(st.u, u);
            st.m = m, st.u = u;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) st.o[dt] *= f;
            if (g == 0) sh_l[turn][col] = st.l;
        }
        if (TL == 1) __syncthreads();
        for (int step = TL / 2; step >= 1; step >>= 1) {
            if (turn >= step && turn < 2 * step)
                for (int dt = 0; dt < DT; ++dt)
                    *reinterpret_cast<float4_t *>(&sh_o[turn - step][col][16 * dt + 4 * g]) = st.o[dt];
            __syncthreads();
            if (turn < step)
                for (int dt = 0; dt < DT; ++dt)
                    st.o[dt] += *reinterpret_cast<float4_t *>(&sh_o[turn][col][16 * dt + 4 * g]);
            __syncthreads();
        }
        const Column c = column(A, s, ctile * COLS + col, head);
        if (turn == 0 && c.row >= 0) {
            const int64_t slot = 2 * (int64_t)blockIdx.x + (unit0 == 0 ? 1 : 0);
            float l = sh_l[0][col];
            for (int w = 1; w < TL; ++w) l += sh_l[w][col];
            if (whole) {
                const float f = out_factor(l, st.m, st.u, 4 * DT, reinterpret_cast<float *>(st.o));
                T *out = static_cast<T *>(a.out) + ((int64_t)c.row * a.q_heads + c.head) * D;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    float v[4];
                    for (int i = 0; i < 4; ++i) v[i] = st.o[dt][i] * f;
                    store_f32x4<T>(out + 16 * dt + 4 * g, v);
                }
                if (a.lse && g == 0)
                    a.lse[(int64_t)c.row * a.q_heads + c.head] = log_sum(l, st.u);
            } else {
                float *po = A.part_o + (slot * COLS + col) * D;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) *reinterpret_cast<float4_t *>(po + 16 * dt + 4 * g) = st.o[dt];
                if (g == 0) A.part_s[slot * COLS + col] = make_float4(st.m, l, st.u, 0.0f);
            }
        }
        __syncthreads();
        left -= units;
        inside += units;
    }
}

// Workgroups per border: one for every kJoinCols columns, but with four column
// groups, whose parts are few, one for every 16 (most borders have nothing to
// join, and each workgroup has to find that out).
constexpr int join_blocks(int groups) { return groups == 4 ? 4 : 16 * groups / kJoinCols; }

// Joins the parts of the segments that several workgroups shared, in the
// order of the tokens.  Workgroup j looks at the border between workers j and
// j + 1; the one at the first border inside a segment joins it.  Two runs of
// threads or more take turns at the parts (7 us for 64 sequences of 8 heads, 13
// us where 8 segments of 32 columns have 64 parts each).
template <int D, int CG, typename T>
__global__ __launch_bounds__(kJoinThreads) void kv_join_kernel(AttnArgs A)
{
    constexpr int COLS = 16 * CG, QUADS = D / 4, LANES = kJoinCols * QUADS, RUNS = kJoinThreads / LANES;
    __shared__ float sh_f[kWorkers][kJoinCols];
    __shared__ float4 sh_s[kJoinCols];
    __shared__ float4 sh_o[RUNS][LANES];
    const KvAttnLaunch &a = A.a;
    const int tid = (int)threadIdx.x;
    uint32_t inside, total, share;
    const int b = stream_locate(A, COLS, [](uint32_t s) { return (blockIdx.x + 1) * s; }, &inside, &total, &share);
    if (b < 0) return;
    const StreamSeq s = stream_seq(A, b, COLS);
    const uint32_t seg = inside / s.units, unit = inside - seg * s.units;
    if (unit == 0 || unit > share) return;     // between segments, or not the first border inside
    const int head = (int)(seg / s.ct);
    // worker blockIdx.x has the first part, in its second slot; the others in their first
    const int w0 = (int)blockIdx.x, parts = list_parts(blockIdx.x + 1, share, total, unit, s.units);
    if (parts == 0) return;
    for (int turn = 0; turn < COLS / (kJoinCols * join_blocks(CG)); ++turn) {
        const int col0 = ((int)blockIdx.y + turn * join_blocks(CG)) * kJoinCols;
        const int idx0 = (int)(seg - (uint32_t)head * s.ct) * COLS + col0;
        if (idx0 >= s.n * A.group) return;
        auto slot = [&](int p) -> int64_t { return (2 * (int64_t)(w0 + p) + (p == 0 ? 1 : 0)) * COLS + col0; };

        // each part's factor of O: 2^(R_part - R); a wave to a column
        if (tid < 64 * kJoinCols) {
            const int c = tid >> 6, lane = tid & 63;
            float4 first = make_float4(kNegInf, 0.0f, kNegInf, 0.0f);
            if (lane < parts) first = A.part_s[slot(lane) + c];
            float m = first.x, u = first.z;
            for (int p = lane + 64; p < parts; p += 64) {
                const float4 t = A.part_s[slot(p) + c];
                m = fmaxf(m, t.x), u = fmaxf(u, t.z);
            }
            m = wave_max(m, lane), u = wave_max(u, lane);
            if (lane < parts) sh_f[lane][c] = exp2_below(first.x, m);
            float l = exp2_below(first.z, u) * first.y;
            for (int p = lane + 64; p < parts; p += 64) {
                const float4 t = A.part_s[slot(p) + c];
                sh_f[p][c] = exp2_below(t.x, m);
                l = fmaf(exp2_below(t.z, u), t.y, l);
            }
            l += xor_lane<1>(l, lane);
            l += xor_lane<2>(l, lane);
            l += xor_lane<4>(l, lane);
            l += xor_lane<8>(l, lane);
            l = group_sum(l, lane);
            if (lane == 0) sh_s[c] = make_float4(m, l, u, 0.0f);
        }
        __syncthreads();

        const int run = tid / LANES, i = tid % LANES, c = i / QUADS, d = (i % QUADS) * 4;
        if (run < RUNS) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float *o = A.part_o + (int64_t)c * D + d;
#pragma unroll 8
            for (int p = run; p < parts; p += RUNS) {
                const float f = sh_f[p][c];
                const float4 w = *reinterpret_cast<const float4 *>(o + slot(p) * D);
                v.x = fmaf(f, w.x, v.x), v.y = fmaf(f, w.y, v.y), v.z = fmaf(f, w.z, v.z), v.w = fmaf(f, w.w, v.w);
            }
            sh_o[run][i] = v;
        }
        __syncthreads();
        const Column q = column(A, s, idx0 + c, head);
        if (run == 0 && q.row >= 0) {
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = 0; k < RUNS; ++k) {
                const float4 w = sh_o[k][i];
                v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
            }
            const float4 t = sh_s[c];
            const float l = t.y, f = out_factor(l, t.x, t.z, 4, v);
            for (int e = 0; e < 4; ++e) v[e] *= f;
            store_f32x4<T>(static_cast<T *>(a.out) + ((int64_t)q.row * a.q_heads + q.head) * D + d, v);
            if (a.lse && d == 0)
                a.lse[(int64_t)q.row * a.q_heads + q.head] = log_sum(l, t.z);
        }
        __syncthreads();
    }
}

// The kernels a call takes, and their workspace: functions of sizes only.
//
// Sequences with up to kFew query columns per head go through the streaming
// kernel, which splits long contexts evenly; longer ones through the tile
// kernel, whose operands serve more columns.  Which of them a batch holds is
// only known on the device: both are launched, unless there is one sequence or
// there are at most two rows per sequence (then all of them are streamed).
// One sequence goes by the call's rows, of which it may own any number: the
// kernel that is launched takes it whatever it owns.  More sequences than a
// launch of the tile kernel has workgroups for are all streamed too.
constexpr int kFew = 64;
constexpr int kWholeShift = 4, kWholeTiles = 1 << kWholeShift;
// Tiles per part: a window of 2048 in fp32, 3 x 8 column tiles: 27 + 7 us at 5, 31 + 6 at 8.
constexpr int kPartTiles = 5;

struct Route {
    bool stream, tile;
    bool whole;         // the streaming kernel splits no segment
    int64_t tiles;      // of a context, at most
    int ct;             // 16-column groups of the streaming kernel
    int few;
    unsigned tile_bound;
    int tile_splits;
    size_t stream_floats, tile_floats;  // parts of O in the workspace
    size_t stream_cols, tile_cols;      // columns that these stand for
};

Route route_of(const KvAttnLaunch &a)
{
    Route r;
    const int64_t group = a.q_heads / a.c.kv_heads, cols = a.s.rows * group, D = a.c.head_dim;
    if (a.s.batch == 1) r.stream = cols <= kFew, r.tile = !r.stream, r.few = r.stream ? kFew : 0;
    else if (cols <= kFew || a.s.rows <= 2 * (int64_t)a.s.batch) r.stream = true, r.tile = false, r.few = INT32_MAX;
    else r.stream = r.tile = true, r.few = kFew;
    const int64_t per = std::max<int64_t>(1, (a.s.rows + a.s.batch - 1) / a.s.batch) * group;
    r.ct = per <= 16 ? 1 : per <= 32 ? 2 : 4;
    const int64_t M = prefill_columns(a), bound = std::min<int64_t>(cols / M + a.s.batch, cols);
    if (r.tile && bound * a.c.kv_heads > most_workgroups(512)) r.stream = true, r.tile = false, r.few = INT32_MAX;
    // Contexts that can have no more than 16 tiles are one unit: four tiles for
    // each wave, which take less than a second launch, and no parts.
    r.tiles = ((a.s.max_blocks << a.c.block_shift) >> 6) + 1;
    r.whole = r.tiles <= kWholeTiles;
    r.stream_cols = r.stream && !r.whole ? (size_t)2 * kWorkers * 16 * r.ct : 0;
    r.stream_floats = r.stream_cols * D;
    r.tile_bound = 0, r.tile_splits = 1, r.tile_cols = 0, r.tile_floats = 0;
    if (r.tile) {
        r.tile_bound = (unsigned)bound;
        // too few workgroups for 256 compute units: tokens are split, at least
        // kPartTiles tiles that a column tile can see to a part
        const int64_t segments = bound * a.c.kv_heads;
        int64_t tiles = r.tiles;
        if (a.window > 0) tiles = std::min<int64_t>(tiles, ((a.window + M / group) >> 6) + 2);
        if (segments < 192)
            r.tile_splits = (int)std::max<int64_t>(1, std::min<int64_t>(512 / segments, tiles / kPartTiles));
        if (r.tile_splits > 1) {
            r.tile_cols = (size_t)(segments * r.tile_splits * M);
            r.tile_floats = r.tile_cols * D;
        }
    }
    return r;
}

template <int D, int CG, int FMT, typename T> hipError_t stream_go(const AttnArgs &A, hipStream_t stream)
{
    kv_stream_kernel<D, CG, FMT, T><<<A.workers, 64 * kWaves, 0, stream>>>(A);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!A.splits) return e;
    kv_join_kernel<D, CG, T><<<dim3(A.workers - 1, join_blocks(CG)), kJoinThreads, 0, stream>>>(A);
    return hipGetLastError();
}

template <int D, int CG> hipError_t stream_types(const AttnArgs &A, hipStream_t stream)
{
    if (A.a.format == KV_INT8)
        return A.a.x_dt == 0 ? stream_go<D, CG, KV_INT8, float>(A, stream) : stream_go<D, CG, KV_INT8, bf16_bits>(A, stream);
    return A.a.x_dt == 0 ? stream_go<D, CG, KV_FP8, float>(A, stream) : stream_go<D, CG, KV_FP8, bf16_bits>(A, stream);
}

template <int D> hipError_t stream_groups(const AttnArgs &A, int groups, hipStream_t stream)
{
    return groups == 1 ? stream_types<D, 1>(A, stream) : groups == 2 ? stream_types<D, 2>(A, stream) : stream_types<D, 4>(A, stream);
}

}  // namespace

size_t kv_attn_ws_bytes(const KvAttnLaunch &a)
{
    // the two kernels run one after the other: they share the workspace
    const Route r = route_of(a);
    return std::max(r.stream_floats + 4 * r.stream_cols, r.tile_floats + 4 * r.tile_cols) * sizeof(float);
}

hipError_t launch_kv_attention(const KvAttnLaunch &a, hipStream_t stream)
{
    const Route r = route_of(a);
    AttnArgs A;
    A.a = a;
    A.workers = kWorkers;
    A.group = a.q_heads / a.c.kv_heads;
    A.few = r.few, A.tile_bound = r.tile_bound, A.tile_splits = r.tile_splits;
    A.unit_shift = 0, A.splits = false;
    A.part_o = static_cast<float *>(a.workspace);
    if (r.tile) {
        A.part_s = reinterpret_cast<float4 *>(A.part_o + r.tile_floats);
        const hipError_t e = launch_kv_prefill(A, stream);
        if (e != hipSuccess || !r.stream) return e;
    }
    // Units of one tile, unless the list could then pass 32 bits.  Only sequences
    // with rows have segments: with rows * q_heads below 2^30 there are fewer
    // than 2^31, and the loop ends, at the latest where each is one unit.
    const double segments =
        ((double)a.s.rows * A.group / (16 * r.ct) + (double)std::min<int64_t>(a.s.batch, a.s.rows)) * a.c.kv_heads;
    while (segments * (double)((r.tiles >> A.unit_shift) + 1) >= 0x1p31) ++A.unit_shift;
    if (r.whole) A.unit_shift = kWholeShift;
    A.splits = r.tiles > (int64_t)1 << A.unit_shift;
    A.part_s = reinterpret_cast<float4 *>(A.part_o + r.stream_floats);
    switch (a.c.head_dim) {
    case 64: return stream_groups<64>(A, r.ct, stream);
    case 128: return stream_groups<128>(A, r.ct, stream);
    case 192: return stream_groups<192>(A, r.ct, stream);
    default: return stream_groups<256>(A, r.ct, stream);
    }
}

}  // namespace nqk
