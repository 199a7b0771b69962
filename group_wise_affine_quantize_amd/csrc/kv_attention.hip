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
// SHARED: a pass of attention behind shared prefixes.
template <int D, int CG, int FMT, typename T, bool SHARED>
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
    int b = stream_locate<SHARED>(A, COLS, [](uint32_t s) { return blockIdx.x * s; }, &inside, &total, &share);
    if (b < 0) return;
    uint32_t left = total - blockIdx.x * share < share ? total - blockIdx.x * share : share;
    StreamSeq s = stream_seq<SHARED>(A, b, COLS);

    while (left > 0) {
        while (inside >= s.work) {      // the next sequence with work
            inside -= s.work;
            if (++b >= a.s.batch + (SHARED ? A.pre.batch : 0)) return;
            s = stream_seq<SHARED>(A, b, COLS);
        }
        const uint32_t span = SHARED ? s.slots : s.units;
        const uint32_t seg = inside / span, slot0 = inside - seg * span;
        const int head = (int)(seg / s.ct);
        const int ctile = (int)(seg - (uint32_t)head * s.ct);
        const uint32_t slots = span - slot0 < left ? span - slot0 : left;
        uint32_t unit0 = slot0, units = slots;
        if (SHARED) {       // what lies behind the slots of no units
            const ListUnits u = list_units(slot0, slots, A.extra);
            unit0 = u.first, units = u.count;
            if (units == 0) {
                left -= slots;
                inside += slots;
                continue;
            }
        }
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
        if (SHARED) table = s.prefix ? A.pre.table + (int64_t)b * A.pre.ldt : a.s.table + (int64_t)(b - A.pre.batch) * a.s.ldt;
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
            const int64_t slot = list_place(blockIdx.x, unit0 == 0);
            float l = sh_l[0][col];
            for (int w = 1; w < TL; ++w) l += sh_l[w][col];
            if (SHARED && whole) {
                const int64_t at = (int64_t)c.row * a.q_heads + c.head;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt)
                    *reinterpret_cast<float4_t *>((s.prefix ? A.pre_o : A.state_o) + at * D + 16 * dt + 4 * g) = st.o[dt];
                if (g == 0) (s.prefix ? A.pre_s : A.state_s)[at] = make_float4(st.m, l, st.u, 0.0f);
            } else if (whole) {
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
        left -= slots;
        inside += slots;
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

// Where the parts of a query column lie: part k at
//   k == 0 ? first : rest + 2 * k * cols
// of a pass's slots, or, where there is one part, at `first` of its states.
// parts 0: no sequence of the pass has the row.
struct ColumnParts {
    int parts, first, rest;
};

// The sequence of a pass that has `row`: the row's number in it, and where its
// segments are in the pass's list, whose length is counted on the way, 64
// sequences at a time.
struct Found {
    bool has;
    int row;
    uint32_t base, slots, ct;       // slots before it, of a segment; column tiles
};
// What a pass's share of its list goes by: its slots, and the units of its longest segment.
struct ListSize {
    uint32_t total, longest;
};
// `first`: the lane's sequence of the first 64.
__device__ __forceinline__ Found find_row(const Pass &p, const KvSeq &first, const KvCache &cache, int group, int row, ListSize *size)
{
    const int lane = (int)(threadIdx.x & 63u), batch = p.s.batch;
    Found f{false, 0, 0, 0, 0};
    uint32_t total = 0, longest = 0;
    for (int b0 = 0; b0 < batch; b0 += 64) {
        int r0 = 0, n = 0;
        uint32_t u = 0, c = 0;
        if (b0 + lane < batch) {
            const KvSeq q = b0 ? kv_seq(p.s, b0 + lane) : first;
            const int64_t cap = p.s.max_blocks << cache.block_shift, len = q.len < cap ? q.len : cap;
            const int tiles = len > 0 ? (int)((len + 63) >> 6) : 1;
            r0 = (int)q.r0, n = (int)q.n;
            u = (uint32_t)(tiles + (1 << p.unit_shift) - 1) >> p.unit_shift;
            c = n * group <= p.few ? (uint32_t)(n * group + p.cols - 1) / (uint32_t)p.cols : 0u;
            if (c && u > longest) longest = u;
            u += p.extra;
        }
        const uint32_t work = c * u * (uint32_t)cache.kv_heads, upto = wave_scan32_sat(work);
        const uint64_t has = __ballot(row >= r0 && row < r0 + n);
        if (has && !f.has) {
            const int at = __ffsll((unsigned long long)has) - 1;
            auto get = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, at); };
            f.has = true, f.row = row - (int)get((uint32_t)r0);
            f.base = add_sat(total, get(upto - work)), f.slots = get(u), f.ct = get(c);
        }
        total = add_sat(total, (uint32_t)__builtin_amdgcn_readlane((int)upto, 63));
    }
    *size = {total, wave_max32(longest)};
    return f;
}

// The parts of a row and head.
__device__ __forceinline__ ColumnParts parts_of(const Pass &p, const Found &f, ListSize size, int group, int q_heads, int row, int head)
{
    ColumnParts c{0, 0, 0};
    if (!f.has) return c;
    c.parts = 1, c.first = row * q_heads + head;
    if (f.ct == 0) return c;
    const uint32_t total = list_total(size.total), share = list_share(total, (uint32_t)p.workers, list_least(size.longest));
    const int kv_head = head / group, col = f.row * group + (head - kv_head * group);
    const uint32_t tile = (uint32_t)col / (uint32_t)p.cols, i = (uint32_t)col - tile * (uint32_t)p.cols;
    const ListParts at = list_segment((uint64_t)f.base + (uint64_t)((uint32_t)kv_head * f.ct + tile) * f.slots, f.slots, p.extra, share, total);
    c.parts = at.count;         // 0 past the list's end: not done
    c.rest = (int)(list_place(at.first, false) * (uint32_t)p.cols + i);
    if (c.parts > 1) c.first = (int)(list_place(at.first, true) * (uint32_t)p.cols + i);
    return c;
}

struct SharedJoin {
    KvAttnLaunch a;
    Pass prefix, own;
    int64_t first;  // row and head of the launch's first column
    int group;
    bool joint;     // one list: the prefixes' and the sequences' behind them
};

// Joins the two passes' parts of each row and head: the prefix's, then the
// sequence's own, each in the order of the tokens, with four threads for
// every 16 bytes of O: 64 rows of 32 heads of 128, two or more parts to each, 33.5 MB of them: 11.5
// us; 4 rows, 6.6 us of dependent loads.  A workgroup takes 1024 / D neighbouring heads and rows.  A wave to a column finds its parts and their
// factors, 64 at a time; then four runs of threads take turns at them.
constexpr int kSharedRuns = 4;
template <int D, typename T> __global__ __launch_bounds__(256 * kSharedRuns) void kv_shared_join_kernel(SharedJoin J)
{
    constexpr int COLS = 1024 / D, QUADS = D / 4;
    __shared__ const float *sh_p[COLS][64];
    __shared__ float sh_f[COLS][64];
    __shared__ float4 sh_s[COLS];       // m, l, u, and what O so far is scaled by
    __shared__ int sh_n[COLS];
    __shared__ float4 sh_o[kSharedRuns - 1][256];
    const KvAttnLaunch &a = J.a;
    const int64_t at0 = J.first + (int64_t)blockIdx.x * COLS, count = a.s.rows * a.q_heads;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = (int)threadIdx.x & 63;
    const int tid = (int)threadIdx.x & 255, run = (int)threadIdx.x >> 8, c = tid / QUADS, d = (tid % QUADS) * 4;

    ColumnParts p{0, 0, 0}, o{0, 0, 0};
    if (wave < COLS && at0 + wave < count) {
        const uint32_t at = (uint32_t)at0 + (uint32_t)wave;     // below 2^30
        const int row = (int)(at / (uint32_t)a.q_heads), head = (int)at - row * a.q_heads;
        ListSize its, mine;
        KvSeq qp{0, 0, 0, 0}, qo{0, 0, 0, 0};
        if (lane < J.prefix.s.batch) qp = kv_seq(J.prefix.s, lane);
        if (lane < J.own.s.batch) qo = kv_seq(J.own.s, lane);
        const Found fp = find_row(J.prefix, qp, a.c, J.group, row, &its);
        Found fo = find_row(J.own, qo, a.c, J.group, row, &mine);
        if (J.joint) {
            fo.base = add_sat(fo.base, its.total);
            its = mine = {add_sat(its.total, mine.total), its.longest > mine.longest ? its.longest : mine.longest};
        }
        p = parts_of(J.prefix, fp, its, J.group, a.q_heads, row, head);
        o = parts_of(J.own, fo, mine, J.group, a.q_heads, row, head);
        if (o.parts == 0) p.parts = 0;      // a row that no sequence has is left alone
    }
    const int parts = p.parts + o.parts;
    if (wave < COLS && lane == 0) sh_n[wave] = parts;
    float m = kNegInf, u = kNegInf, l = 0.0f;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0;; k0 += 64) {
        if (wave < COLS) {
            float4 t = make_float4(kNegInf, 0.0f, kNegInf, 0.0f);
            const int k = k0 + lane;
            if (k < parts) {
                const bool first = k < p.parts;
                const Pass &q = first ? J.prefix : J.own;
                const ColumnParts f = first ? p : o;
                const int i = first ? k : k - p.parts;
                const int64_t slot = i == 0 ? f.first : f.rest + 2 * (int64_t)i * q.cols;
                t = (f.parts == 1 ? q.state_s : q.part_s)[slot];
                sh_p[wave][lane] = (f.parts == 1 ? q.state_o : q.part_o) + slot * D;
            }
            const float mm = fmaxf(m, wave_max(t.x, lane)), uu = fmaxf(u, wave_max(t.z, lane));
            sh_f[wave][lane] = exp2_below(t.x, mm);
            float sum = exp2_below(t.z, uu) * t.y;
            sum += xor_lane<1>(sum, lane);
            sum += xor_lane<2>(sum, lane);
            sum += xor_lane<4>(sum, lane);
            sum += xor_lane<8>(sum, lane);
            sum = group_sum(sum, lane);
            l = fmaf(l, exp2_below(u, uu), sum);
            if (lane == 0) sh_s[wave] = make_float4(mm, l, uu, exp2_below(m, mm));
            m = mm, u = uu;
        }
        __syncthreads();
        int most = 0;
#pragma unroll
        for (int i = 0; i < COLS; ++i) most = sh_n[i] > most ? sh_n[i] : most;
        if (c < COLS) {
            const float again = sh_s[c].w;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= again;
            const int n = sh_n[c] - k0 < 64 ? sh_n[c] - k0 : 64;
#pragma unroll 8
            for (int k = run; k < n; k += kSharedRuns) {
                const float f = sh_f[c][k];
                const float4 x = *reinterpret_cast<const float4 *>(sh_p[c][k] + d);
                v[0] = fmaf(f, x.x, v[0]), v[1] = fmaf(f, x.y, v[1]), v[2] = fmaf(f, x.z, v[2]), v[3] = fmaf(f, x.w, v[3]);
            }
        }
        if (k0 + 64 >= most) break;
        __syncthreads();
    }
    if (run) sh_o[run - 1][tid] = make_float4(v[0], v[1], v[2], v[3]);
    __syncthreads();
    if (run || c >= COLS || sh_n[c] == 0) return;
    for (int k = 0; k < kSharedRuns - 1; ++k) {
        const float4 x = sh_o[k][tid];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    }
    const float4 t = sh_s[c];
    const float f = out_factor(t.y, t.x, t.z, 4, v);
    for (int e = 0; e < 4; ++e) v[e] *= f;
    store_f32x4<T>(static_cast<T *>(a.out) + (at0 + c) * D + d, v);
    if (a.lse && d == 0) a.lse[at0 + c] = log_sum(t.y, t.z);
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
// launch of the tile kernel has workgroups for are all streamed too, and behind shared
// prefixes batches of few rows to a sequence (list_streams_all).
constexpr int kFew = 64;
constexpr int kWholeShift = 4, kWholeTiles = 1 << kWholeShift;
// The tile kernel over a list of work: one workgroup per compute unit, which
// its registers fill.
constexpr int kTileWorkers = 256;
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

// `joined`: behind shared prefixes, where a call is three launches at least.
Route route_of(const KvAttnLaunch &a, bool joined = false)
{
    Route r;
    const int64_t group = a.q_heads / a.c.kv_heads, cols = a.s.rows * group, D = a.c.head_dim;
    if (a.s.batch == 1) r.stream = cols <= kFew, r.tile = !r.stream, r.few = r.stream ? kFew : 0;
    else if (cols <= kFew || a.s.rows <= 2 * (int64_t)a.s.batch) r.stream = true, r.tile = false, r.few = INT32_MAX;
    else r.stream = r.tile = true, r.few = kFew;
    const int64_t per = std::max<int64_t>(1, (a.s.rows + a.s.batch - 1) / a.s.batch) * group;
    r.ct = per <= 16 ? 1 : per <= 32 ? 2 : 4;
    if (joined && list_streams_all(a.s.batch, a.s.rows, group)) r.stream = true, r.tile = false, r.few = INT32_MAX;
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
    if (A.state_s) kv_stream_kernel<D, CG, FMT, T, true><<<A.workers, 64 * kWaves, 0, stream>>>(A);
    else kv_stream_kernel<D, CG, FMT, T, false><<<A.workers, 64 * kWaves, 0, stream>>>(A);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!A.splits || A.state_s) return e;
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

hipError_t stream_dims(const AttnArgs &A, int groups, hipStream_t stream)
{
    switch (A.a.c.head_dim) {
    case 64: return stream_groups<64>(A, groups, stream);
    case 128: return stream_groups<128>(A, groups, stream);
    case 192: return stream_groups<192>(A, groups, stream);
    default: return stream_groups<256>(A, groups, stream);
    }
}

// What a segment costs a workgroup besides its tiles, in tiles: a pass behind
// shared prefixes counts it in its list, so that workgroups with many short
// segments end when the others do (16 sequences of 64 tokens and 8 heads behind four
// prefixes of 16000 in one launch: 95 us at 0, 50 at 2, 42 at 4, 43 at 8; three
// prefixes' tiles for 40 sequences of 3 drafts, 83, 79, 77 and 77).  The segments of
// one prefix alone are as long as each other, and often whole numbers of shares, which
// it would spoil (64 sequences behind 16384 tokens 65 -> 69 us).
constexpr int kSegmentTiles = 4;

// Units of one tile, unless the list could then pass 32 bits.  Only sequences
// with rows have segments: with rows * q_heads below 2^30 there are fewer
// than 2^31, and the loop ends, at the latest where each is one unit.
int unit_shift_of(const KvAttnLaunch &a, int cols, int64_t tiles, int extra = 0)
{
    const double segments = ((double)a.s.rows * (a.q_heads / a.c.kv_heads) / cols +
                             (double)std::min<int64_t>(a.s.batch, a.s.rows)) * a.c.kv_heads;
    int shift = 0;
    while (segments * (double)((tiles >> shift) + 1 + (extra >> shift)) >= 0x1p31) ++shift;
    return shift;
}

}  // namespace

// The kernels over a.s.  `A` comes zeroed, or with a pass's states set.
static hipError_t launch_route(AttnArgs &A, const Route &r, const KvAttnLaunch &a, hipStream_t stream)
{
    A.a = a;
    A.workers = kWorkers;
    A.group = a.q_heads / a.c.kv_heads;
    A.few = r.few, A.tile_bound = r.tile_bound, A.tile_splits = r.tile_splits;
    A.part_o = static_cast<float *>(a.workspace);
    if (r.tile) {
        A.part_s = reinterpret_cast<float4 *>(A.part_o + r.tile_floats);
        const hipError_t e = launch_kv_prefill(A, stream);
        if (e != hipSuccess || !r.stream) return e;
    }
    A.unit_shift = r.whole ? kWholeShift : unit_shift_of(a, 16 * r.ct, r.tiles, A.state_s ? kSegmentTiles : 0);
    A.splits = r.tiles > (int64_t)1 << A.unit_shift;
    // at least two tiles for each wave, so that short contexts do not fall into
    // parts that cost more to join than to read
    A.least = A.unit_shift ? 1u : 2u * kWaves;
    if (A.state_s) A.extra = kSegmentTiles >> A.unit_shift;
    A.part_s = reinterpret_cast<float4 *>(A.part_o + r.stream_floats);
    return stream_dims(A, r.ct, stream);
}

static size_t route_floats(const Route &r) { return std::max(r.stream_floats + 4 * r.stream_cols, r.tile_floats + 4 * r.tile_cols); }

size_t kv_attn_ws_bytes(const KvAttnLaunch &a)
{
    // the two kernels run one after the other: they share the workspace
    return route_floats(route_of(a)) * sizeof(float);
}

hipError_t launch_kv_attention(const KvAttnLaunch &a, hipStream_t stream)
{
    AttnArgs A{};
    return launch_route(A, route_of(a), a, stream);
}

// The prefixes' pass takes one of the two kernels for all prefixes, by the mean
// of their query columns.
struct PrefixRoute {
    bool tile;
    int groups;         // 16-column groups of the streaming kernel
    int cols, workers;  // of a segment, of the list
    size_t slots;       // columns of all slots
};

// `groups`: those of the sequences' own pass, if one launch does both.
static PrefixRoute prefix_route(const KvAttnLaunch &a, const KvSeqs &prefix, int groups)
{
    PrefixRoute f;
    const int64_t mean = (a.s.rows + prefix.batch - 1) / prefix.batch * (a.q_heads / a.c.kv_heads);
    f.tile = !groups && mean > kFew;
    f.groups = groups ? groups : mean <= 16 ? 1 : mean <= 32 ? 2 : 4;
    f.cols = f.tile ? prefill_columns(a) : 16 * f.groups;
    f.workers = f.tile ? kTileWorkers : kWorkers;
    f.slots = (size_t)2 * f.workers * f.cols;
    return f;
}

// Both passes in one launch of the streaming kernel, over columns as the
// sequences' own pass has them: where that is streamed, where there are not very many
// segments, and where a prefix that more columns share is not read again too
// often.  32 heads of 128 over 8, 1500 own tokens, two launches -> one: 16 sequences
// behind 5000 tokens 43 -> 29 us (1900 tiles read again), 64 behind 1500 62 -> 46 (2900), 48
// behind 5000 60 -> 53 (7000), 24 behind 16000 54 -> 55 (10000), 64 behind
// 16000 81 -> 126 (30000); of 64, 100 of 8 over 2 behind 16000 47 -> 40
// (12000); of 256, 32 of 16 over 4 behind two of 5000 80 -> 56 (1900).  128 sequences
// behind 32 prefixes of 1500, 1280 segments, 92 -> 84; 256 behind 64, 2560, 163 -> 168.
static bool joint_route(const KvAttnLaunch &a, const KvSeqs &prefix, const Route &r)
{
    if (!r.stream || r.tile) return false;
    const int64_t group = a.q_heads / a.c.kv_heads, cols = 16 * r.ct;
    const int64_t own = std::min<int64_t>(a.s.batch, a.s.rows), its = std::min<int64_t>(prefix.batch, a.s.rows);
    const int64_t segments = (own + its + 2 * (a.s.rows * group / cols)) * a.c.kv_heads;
    const int64_t reads = ((a.s.rows + its - 1) / its * group + cols - 1) / cols;       // of a prefix
    const int64_t tiles = ((prefix.max_blocks << a.c.block_shift) >> 6) + 1;
    return segments <= 2048 && (double)((reads - 1) * its * a.c.kv_heads) * (double)tiles * a.c.head_dim <= 0x1p20;
}

// Workspace: the prefixes' slots and states, the sequences' states, and what
// their own kernels take.
size_t kv_shared_ws_bytes(const KvAttnLaunch &a, const KvSeqs &prefix)
{
    if (prefix.batch == 0) return kv_attn_ws_bytes(a);
    const Route r = route_of(a, true);
    const bool joint = joint_route(a, prefix, r);
    const size_t states = (size_t)a.s.rows * a.q_heads;
    return ((prefix_route(a, prefix, joint ? r.ct : 0).slots + 2 * states) * (a.c.head_dim + 4) +
            (joint ? 0 : route_floats(r))) * sizeof(float);
}

hipError_t launch_kv_shared(const KvAttnLaunch &a, const KvSeqs &prefix, hipStream_t stream)
{
    if (prefix.batch == 0) return launch_kv_attention(a, stream);
    const Route r = route_of(a, true);
    const bool joint = joint_route(a, prefix, r);
    const PrefixRoute f = prefix_route(a, prefix, joint ? r.ct : 0);
    const size_t D = (size_t)a.c.head_dim, states = (size_t)a.s.rows * a.q_heads;
    const int64_t tiles = ((prefix.max_blocks << a.c.block_shift) >> 6) + 1;
    float *at = static_cast<float *>(a.workspace);
    auto take = [&](size_t n) { float *p = at; at += n; return p; };

    AttnArgs A{};       // the prefixes' pass
    A.a = a;
    A.a.s = prefix, A.a.causal = 0, A.a.window = 0, A.a.out = nullptr, A.a.lse = nullptr;
    A.group = a.q_heads / a.c.kv_heads;
    A.few = INT32_MAX, A.workers = f.workers, A.listed = f.tile, A.tile_splits = 1;
    A.unit_shift = unit_shift_of(A.a, f.cols, tiles, kSegmentTiles);
    if (prefix.batch > 1) A.extra = kSegmentTiles >> A.unit_shift;
    A.part_o = take(f.slots * D), A.part_s = reinterpret_cast<float4 *>(take(f.slots * 4));
    A.state_o = take(states * D), A.state_s = reinterpret_cast<float4 *>(take(states * 4));
    AttnArgs O{};       // the sequences'
    O.state_o = take(states * D), O.state_s = reinterpret_cast<float4 *>(take(states * 4));
    hipError_t e;
    if (joint) {
        // twice the units of the longer of the two cannot pass 32 bits either
        const int64_t longer = std::max(tiles, r.tiles);
        KvAttnLaunch both = a;
        both.s.rows = 2 * a.s.rows, both.s.batch = a.s.batch + prefix.batch;
        O.a = a;
        O.group = A.group, O.few = INT32_MAX, O.workers = kWorkers;
        O.unit_shift = unit_shift_of(both, f.cols, longer, kSegmentTiles), O.extra = kSegmentTiles >> O.unit_shift;
        O.part_o = A.part_o, O.part_s = A.part_s;
        O.pre = prefix, O.pre_o = A.state_o, O.pre_s = A.state_s;
        A.unit_shift = O.unit_shift, A.extra = O.extra;
        e = stream_dims(O, f.groups, stream);
    } else {
        e = f.tile ? launch_kv_prefill(A, stream) : stream_dims(A, f.groups, stream);
        if (e != hipSuccess) return e;
        KvAttnLaunch own = a;
        own.workspace = at;
        e = launch_route(O, r, own, stream);
    }
    if (e != hipSuccess) return e;

    SharedJoin J;
    J.a = a;
    J.group = A.group, J.joint = joint;
    J.prefix = {prefix, A.few, f.cols, A.unit_shift, A.workers, A.extra, A.state_o, A.part_o, A.state_s, A.part_s};
    J.own = {a.s, r.stream ? O.few : 0, 16 * r.ct, O.unit_shift, O.workers, O.extra, O.state_o, O.part_o, O.state_s, O.part_s};
    const int cols = 1024 / (int)D;
    const int64_t most = most_workgroups(256 * kSharedRuns) * cols;     // columns of a launch
    auto go = [&](auto bf16, auto f32) {
        for (J.first = 0; J.first < (int64_t)states; J.first += most) {
            const int64_t n = std::min<int64_t>(most, (int64_t)states - J.first);
            (a.x_dt == 0 ? f32 : bf16)<<<(unsigned)((n + cols - 1) / cols), 256 * kSharedRuns, 0, stream>>>(J);
            if ((e = hipGetLastError()) != hipSuccess) return;
        }
    };
    switch (D) {
    case 64: go(kv_shared_join_kernel<64, bf16_bits>, kv_shared_join_kernel<64, float>); break;
    case 128: go(kv_shared_join_kernel<128, bf16_bits>, kv_shared_join_kernel<128, float>); break;
    case 192: go(kv_shared_join_kernel<192, bf16_bits>, kv_shared_join_kernel<192, float>); break;
    default: go(kv_shared_join_kernel<256, bf16_bits>, kv_shared_join_kernel<256, float>); break;
    }
    return e;
}

}  // namespace nqk
