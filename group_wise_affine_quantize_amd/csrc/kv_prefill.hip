// Attention over the 8-bit cache for many query rows (prompts and their
// chunks); the mathematics is at the head of kv_attention.hip.
//
// A workgroup takes 32 query columns per wave (a column is a row of the call
// and one of the head's queries) of one key/value head and runs over the
// tokens that they see, 64 at a time.  The tile's codes are converted to fp16
// once, into LDS, where all waves read them as operands of 32x32x16 MFMAs: S^T = K q^T,
// O^T = V^T P^T.  Eight waves (four for head_dim over 128, whose O and q take
// twice the registers): two per SIMD, so that one's softmax runs under the
// other's products.
//
// Lane l (r = l % 32, h = l / 32) holds column r of the wave's 32-column
// blocks and, after the first product, rows 8 a + 4 h + b of each 32-token
// half tile in register 4 a + b.  Token 16 h + 4 a + b of the half is put into
// that row, so that a lane's 16 weights are of neighbouring tokens -- of one
// block of the cache, with one scale -- and are the operand of the second
// product as they stand.
//
// The reference R of the weights 2^(x - R) only moves when a column's maximum
// passes it by kSlack: a move costs a pass over O, and weights may reach
// 2^(kTop + kSlack) in fp16.
//
// 3 prompts of 2530 to 4096 tokens, 32 heads of 128 over 8 int8 key/value
// heads: 370 to 380 us by itself (a call in a row of calls 341 to 352), 740 TFLOP/s of the
// visible products, where a large fp16 library product reaches 1131.  A tile
// takes about 4450 cycles at the 1.97 GHz that the card keeps up: 329 vector
// instructions for each of the two waves of a SIMD, and 2048 cycles of MFMA
// per SIMD, overlapped as far as the two waves' phases differ.  The LDS (256
// bytes a cycle with the placement below) is a quarter used.
#include "nq_kv_attn.h"
#include "nq_tiles.h"

namespace nqk {

namespace {

typedef float float16_t __attribute__((ext_vector_type(16)));

// Weights are at most 2^12 where R is set, and 2^15.5 before it moves again.
constexpr float kTop = 12.0f, kSlack = 3.5f;

// What sixteen tokens of a tile are; kLost: a scale is no number.
constexpr float kAbsent = 0.0f, kThere = 1.0f, kFar = 2.0f, kLost = 3.0f;

template <int D> struct Shape {
    static constexpr int W = D <= 128 ? 8 : 4;      // waves
    static constexpr int M = 32 * W;                // query columns
    static constexpr int THREADS = 64 * W;
    static constexpr int PIECES = 4 * D;            // 16-byte pieces of a tile's keys (and values)
    static constexpr int LD = (PIECES + THREADS - 1) / THREADS;
};

__device__ __forceinline__ float16_t mfma32(half8_t a, half8_t b, float16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// A row's 16-byte chunks are placed at their number xored with a key, so that
// sixteen neighbouring rows' chunks of one number -- what a phase of a 16-byte
// read takes -- lie in different quarters of the 64 banks.
template <int CHUNKS> __device__ __forceinline__ int key_of(int row)
{
    return CHUNKS % 16 == 0 ? row & 15 : (row >> 1) & 7;
}

// The column tiles of a sequence here.
template <int M> __device__ __forceinline__ uint32_t tile_count(const AttnArgs &A, int b)
{
    const KvSeq q = kv_seq(A.a.s, b);
    const int cols = (int)q.n * A.group;
    return cols > A.few ? (uint32_t)(cols + M - 1) / M : 0u;
}

// The workgroups start with the column tiles of the highest number (of all
// sequences), which see the most tokens of a causal prompt: the last ones to
// start are short.  Finds the sequence and number of tile `rank` in that
// order; -1 past the last.
template <int M> __device__ __forceinline__ int tile_locate(const AttnArgs &A, uint32_t rank, uint32_t *ctile)
{
    const int batch = A.a.s.batch, lane = (int)(threadIdx.x & 63u);
    const uint32_t mine = lane < batch ? tile_count<M>(A, lane) : 0u;     // of the first 64 sequences
    auto count = [&](int b) { return b < 64 ? mine : (b < batch ? tile_count<M>(A, b) : 0u); };
    // tiles numbered c or more
    auto from = [&](uint32_t c) -> uint32_t {
        uint32_t sum = 0;
        for (int b0 = 0; b0 < batch; b0 += 64) {
            const uint32_t n = count(b0 + lane);
            sum += (uint32_t)__builtin_amdgcn_readlane((int)wave_scan32(n > c ? n - c : 0u), 63);
        }
        return sum;
    };
    if (from(0) <= rank) return -1;
    uint32_t lo = 0, hi = A.tile_bound;     // from(lo) > rank >= from(hi)
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (from(mid) > rank) lo = mid;
        else hi = mid;
    }
    *ctile = lo;
    uint32_t left = rank - from(lo + 1);    // which of the sequences with more than lo tiles
    for (int b0 = 0; b0 < batch; b0 += 64) {
        const uint32_t upto = wave_scan32(count(b0 + lane) > lo ? 1u : 0u);
        const uint32_t sum = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
        if (sum > left) return b0 + __ffsll((unsigned long long)__ballot(upto > left)) - 1;
        left -= sum;
    }
    return -1;
}

// SHARED: a pass of attention behind shared prefixes.  The prefixes' runs
// over the list of work that the streaming kernel has (nq_kv_attn.h), an equal run
// of tiles for each workgroup; workgroups of one XCD take neighbouring runs.
template <int D, int FMT, typename T, bool SHARED>
__global__ __launch_bounds__(Shape<D>::THREADS) void kv_tile_kernel(AttnArgs A)
{
    constexpr int NP = Parts<T>::n, M = Shape<D>::M, THREADS = Shape<D>::THREADS, PIECES = Shape<D>::PIECES;
    constexpr int LD = Shape<D>::LD, KS = D / 16, DT = D / 32;
    constexpr int KC = D / 8;       // 16-byte chunks of a key row in LDS
    // keys [64 rows][D], values [D][64 tokens], fp16, chunks placed by key_of
    __shared__ uint4 sh_k[2][kTile * KC];
    __shared__ uint4 sh_v[2][D * 8];
    // of each 16 tokens: key scale, log2 and reciprocal of the value scale, and
    // kThere, kFar (L cannot share O's reference), kLost or kAbsent
    __shared__ float4 sh_s[2][4];
    const KvAttnLaunch &a = A.a;
    const int tid = (int)threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sh = a.c.block_shift, bmask = (1 << sh) - 1;

    const uint32_t heads = (uint32_t)a.c.kv_heads;
    int head, b, split = 0;
    uint32_t ctile, worker = 0, inside = 0, total = 0, share = 0, left = 0, unit0 = 0, units = 0, slots = 0;
    StreamSeq s;
    auto uniform = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); };
    if (SHARED && A.listed) {
        worker = (blockIdx.x & 7u) * (gridDim.x >> 3) + (blockIdx.x >> 3);
        b = stream_locate<SHARED>(A, M, [&](uint32_t w) { return worker * w; }, &inside, &total, &share);
        if (b < 0) return;
        b = (int)uniform((uint32_t)b), inside = uniform(inside), total = uniform(total), share = uniform(share);
        left = total - worker * share < share ? total - worker * share : share;
        s = stream_seq<SHARED>(A, b, M);
    } else {
        // workgroups of one head follow each other with the number of heads as
        // their distance: with eight heads an XCD keeps to one head's cache
        head = (int)(blockIdx.x % heads);
        const uint32_t rest = blockIdx.x / heads;
        split = (int)(rest % (uint32_t)A.tile_splits);
        b = tile_locate<M>(A, rest / (uint32_t)A.tile_splits, &ctile);
        if (b < 0) return;
        s = stream_seq(A, b, M);
    }
    do {
        if (SHARED && A.listed) {
            uint32_t seg;
            for (;;) {
                while (inside >= s.work) {      // the next sequence with work
                    inside -= s.work;
                    if (++b >= a.s.batch) return;
                    s = stream_seq<SHARED>(A, b, M);
                }
                const uint32_t span = uniform(s.slots);
                seg = inside / span;
                const uint32_t slot0 = inside - seg * span;
                slots = span - slot0 < left ? span - slot0 : left;
                const ListUnits u = list_units(slot0, slots, A.extra);
                unit0 = u.first, units = u.count;
                if (units) break;
                left -= slots, inside += slots;
                if (left == 0) return;
            }
            const uint32_t ct = uniform(s.ct);
            head = (int)(seg / ct);
            ctile = seg - (uint32_t)head * ct;
        }
        const int count = s.n * A.group, col0 = (int)ctile * M, end = col0 + M < count ? col0 + M : count;
        const Column c0 = column(A, s, col0, head), c1 = column(A, s, end - 1, head);
        const int seg_lo = __builtin_amdgcn_readfirstlane(c0.lo), seg_hi = __builtin_amdgcn_readfirstlane(c1.hi);
        const int first_tile = seg_lo >> 6, tiles = seg_hi > seg_lo ? ((seg_hi + 63) >> 6) - first_tile : 0;
        int t_begin = first_tile + (int)((int64_t)tiles * split / A.tile_splits);
        int t_end = first_tile + (int)((int64_t)tiles * (split + 1) / A.tile_splits);
        if (SHARED && A.listed) {
            t_begin = (int)(unit0 << A.unit_shift);
            t_end = unit0 + units == s.units ? tiles : (int)((unit0 + units) << A.unit_shift);
            t_begin = t_begin < t_end ? t_begin : t_end;
        }

        // the query rows are on their way while the first tile is asked for
        const int wcol = col0 + wave * 32;          // the wave's first column
        const Column mine = column(A, s, wcol + r, head);
        constexpr int RAW = 8 * (int)sizeof(T) / 16;
        uint4 raw[KS][RAW];
        {
            const T *src = static_cast<const T *>(a.q) + (int64_t)(mine.row < 0 ? 0 : mine.row) * a.ldq + mine.head * D + 8 * h;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < RAW; ++i) raw[ks][i] = reinterpret_cast<const uint4 *>(src + 16 * ks)[i];
        }
        float16_t o[DT];
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
            for (int i = 0; i < 16; ++i) o[dt][i] = 0.0f;
        // tokens that every column of the wave sees, and that some column sees
        const int wend = wcol + 32 < end ? wcol + 32 : end;
        const Column w0 = column(A, s, wcol, head), w1 = column(A, s, wend - 1, head);
        const int all_lo = __builtin_amdgcn_readfirstlane(w1.lo), all_hi = __builtin_amdgcn_readfirstlane(w0.hi);
        const int any_lo = __builtin_amdgcn_readfirstlane(w0.lo), any_hi = wcol >= end ? 0 : __builtin_amdgcn_readfirstlane(w1.hi);

        // Staging: this thread's 16-byte pieces of a tile's keys and values.  Block
        // ids are read a tile ahead of the codes, those a tile ahead of their
        // conversion.  A tile starts at a multiple of 64 tokens, so a piece's place
        // inside its block is the tile's plus the thread's own.
        const int *table = a.s.table + (int64_t)b * a.s.ldt;
        const int j_lo = seg_lo >> sh, j_hi = (seg_hi - 1) >> sh;      // table entries that may be read
        auto entry_of = [&](int j) -> int { return table[j < j_lo ? j_lo : (j > j_hi ? j_hi : j)]; };
        const int tg = tid & 3;
        const uint32_t stride = (uint32_t)heads * (uint32_t)(D << sh);  // bytes of a block's keys (and values)
        const uint8_t *kp[LD], *vp = a.c.v_codes + (int64_t)head * (D << sh) + ((tid >> 2) << sh) + ((16 * tg) & bmask);
        int kj[LD];
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const int piece = tid + i * THREADS, tok = piece / (D / 16), c16 = piece % (D / 16);
            kp[i] = a.c.k_codes + (int64_t)head * (D << sh) + (tok & bmask) * D + 16 * c16;
            kj[i] = tok >> sh;
        }
        const int vj = (16 * tg) >> sh;
        uint4 kw[LD], vw[LD];
        int kid[LD], vid;
        bool has = false;       // whether a column sees some of the 16 tokens, and a block holds them
        float sk = 1.0f, sv = 1.0f;
        auto load_ids = [&](int t) {
            const int j = (t << 6) >> sh;
#pragma unroll
            for (int i = 0; i < LD; ++i)
                if (PIECES % THREADS == 0 || tid + i * THREADS < PIECES) kid[i] = entry_of(j + kj[i]);
            vid = entry_of(j + vj);
        };
        auto load = [&](int t) {
            const int at = (t << 6) & bmask, pos = (t << 6) + 16 * tg;
            const bool there = (uint32_t)vid < (uint32_t)a.c.blocks;
            const uint32_t id = there ? (uint32_t)vid : 0u;
            has = there && pos < seg_hi && pos + 16 > seg_lo;
#pragma unroll
            for (int i = 0; i < LD; ++i)
                if (PIECES % THREADS == 0 || tid + i * THREADS < PIECES) {
                    const uint32_t k = (uint32_t)kid[i] < (uint32_t)a.c.blocks ? (uint32_t)kid[i] : 0u;
                    kw[i] = *reinterpret_cast<const uint4 *>(kp[i] + (uint64_t)k * stride + at * D);
                }
#pragma unroll
            for (int i = 0; i < LD; ++i)
                if (PIECES % THREADS == 0 || tid + i * THREADS < PIECES)
                    vw[i] = *reinterpret_cast<const uint4 *>(vp + (uint64_t)id * stride + (at + ((i * (THREADS / 4)) << sh)));
            if (wave == 0) {        // lanes 0 to 3 use them
                sk = a.c.k_scales[(int64_t)id * heads + head];
                sv = a.c.v_scales[(int64_t)id * heads + head];
            }
        };
        auto stage = [&](int t, int buf) {
#pragma unroll
            for (int i = 0; i < LD; ++i) {
                const int piece = tid + i * THREADS, tok = piece / (D / 16), c16 = piece % (D / 16);
                if (PIECES % THREADS == 0 || piece < PIECES) {
                    const int u = tok & 31, row = (tok & 32) + 8 * ((u >> 2) & 3) + 4 * (u >> 4) + (u & 3), key = key_of<KC>(row);
                    const half8_t x = codes_to_half<FMT>(kw[i].x, kw[i].y), y = codes_to_half<FMT>(kw[i].z, kw[i].w);
                    sh_k[buf][row * KC + ((2 * c16) ^ key)] = __builtin_bit_cast(uint4, x);
                    sh_k[buf][row * KC + ((2 * c16 + 1) ^ key)] = __builtin_bit_cast(uint4, y);
                }
            }
            const int pos = (t << 6) + 16 * tg;
            if constexpr (FMT == KV_FP8) {
                // codes of tokens that no column sees are whatever memory holds, a
                // NaN for instance: make them zeros
                if (!has || pos < seg_lo || pos + 16 > seg_hi) {
                    const int lo = !has ? 16 : seg_lo - pos, hi = seg_hi - pos;
                    uint32_t keep[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        keep[w] = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (4 * w + e >= lo && 4 * w + e < hi) keep[w] |= 255u << (8 * e);
                    }
#pragma unroll
                    for (int i = 0; i < LD; ++i) vw[i].x &= keep[0], vw[i].y &= keep[1], vw[i].z &= keep[2], vw[i].w &= keep[3];
                }
            }
#pragma unroll
            for (int i = 0; i < LD; ++i) {
                const int piece = tid + i * THREADS, d = piece >> 2;
                if (PIECES % THREADS == 0 || piece < PIECES) {
                    const half8_t x = codes_to_half<FMT>(vw[i].x, vw[i].y), y = codes_to_half<FMT>(vw[i].z, vw[i].w);
                    sh_v[buf][d * 8 + ((2 * tg) ^ key_of<8>(d))] = __builtin_bit_cast(uint4, x);
                    sh_v[buf][d * 8 + ((2 * tg + 1) ^ key_of<8>(d))] = __builtin_bit_cast(uint4, y);
                }
            }
            if (tid < 4) {
                // all-zero keys (or none): any scale will do for scores of zero, and one
                // keeps the factor of the scores above zero; all-zero values add to L alone
                const bool lost = has && !(sk - sk + (sv - sv) == 0.0f);
                const float k = !has || lost || sk == 0.0f ? 1.0f : sk, v = !has || lost ? 1.0f : sv, log = fast_log2(v);    // log2(0): -infinity
                const float kind = !has ? kAbsent : lost ? kLost : scale_place(v) >= kNearScales ? kFar : kThere;
                sh_s[buf][tid] = make_float4(k, log, v == 0.0f ? 0.0f : 1.0f / v, kind);
            }
        };

        const int t_last = t_end - 1;
        if (t_begin < t_end) {
            load_ids(t_begin);
            load(t_begin);
            load_ids(t_begin < t_last ? t_begin + 1 : t_last);
        }
        half8_t q[KS][NP];
        float cf = 1.0f, ref = kNegInf, l = 0.0f, lref = kNegInf;
        bool apart = false;     // whether l's reference is lref, not ref
        {
            float top = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float f[8];
                unpack_f32x8<T>(raw[ks], f);
                for (int i = 0; i < 8; ++i) top = larger(top, f[i]);
            }
            top = larger(top, xor_lane<32>(top, lane));
            float back;
            const float up = row_scale(top, &back);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float f[8];
                unpack_f32x8<T>(raw[ks], f);
                for (int i = 0; i < 8; ++i) f[i] = mine.row >= 0 ? f[i] * up : 0.0f;
                split_half<NP>(f, q[ks]);
            }
            if (mine.row >= 0) cf = a.scale * kLog2e * back;
        }
        if (t_begin < t_end) {
            stage(t_begin, 0);
            load(t_begin < t_last ? t_begin + 1 : t_last);
            load_ids(t_begin + 2 < t_last ? t_begin + 2 : t_last);
        }
        // The next tile goes into the other buffer, whose readers passed the last
        // barrier; then the loads of the one after.  The second four waves do
        // this first in a step and the others last: of the two waves of a SIMD,
        // one then is a phase behind the other, and they want the vector unit and
        // the matrix cores by turns.
        auto stage_next = [&](int t, int buf) {
            if (t >= t_last) return;
            stage(t + 1, buf ^ 1);
            load(t + 2 < t_last ? t + 2 : t_last);
            load_ids(t + 3 < t_last ? t + 3 : t_last);
        };
        const bool late = wave >= 4;
        lds_barrier();
        for (int t = t_begin; t < t_end; ++t) {
            const int buf = (t - t_begin) & 1, base = t << 6;
            const bool busy = base < any_hi && base + kTile > any_lo;
            if (late) stage_next(t, buf);
            float16_t S[2];
            if (busy) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    for (int i = 0; i < 16; ++i) S[u][i] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const half8_t k = __builtin_bit_cast(half8_t, sh_k[buf][(32 * u + r) * KC + ((2 * ks + h) ^ key_of<KC>(r))]);
#pragma unroll
                        for (int p = 0; p < NP; ++p) S[u] = mfma32(k, q[ks][p], S[u]);
                    }
            }
            if (busy) {
                const float4 s0 = sh_s[buf][h], s1 = sh_s[buf][2 + h];
                const bool special = __any(s0.w * s1.w != kThere);
                const bool masked = base < all_lo || base + kTile > all_hi || special;
                if (__builtin_amdgcn_readfirstlane((int)masked)) {
                    const int lo = mine.lo - base - 16 * h, hi = mine.hi - base - 16 * h;
                    const int hi0 = s0.w == kAbsent ? -64 : hi, hi1 = s1.w == kAbsent ? -64 : hi;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        S[0][i] = i < lo || i >= hi0 ? kNegInf : S[0][i];
                        S[1][i] = 32 + i < lo || 32 + i >= hi1 ? kNegInf : S[1][i];
                    }
                }
                if (special && __any(s0.w == kLost || s1.w == kLost)) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (s0.w == kLost && S[0][i] != kNegInf) S[0][i] = __builtin_nanf("");
                        if (s1.w == kLost && S[1][i] != kNegInf) S[1][i] = __builtin_nanf("");
                    }
                }
                // factors above zero, so that the maximum is that of S
                const float f0 = fmaxf(cf * s0.x, 1e-37f), f1 = fmaxf(cf * s1.x, 1e-37f);
                if (__builtin_expect(apart || (special && __any(s0.w == kFar || s1.w == kFar)), false)) {
                    if (!apart) lref = ref;
                    apart = true;
                    add_weights(16, [&](int i) { return S[0][i] * f0; }, l, lref);
                    add_weights(16, [&](int i) { return S[1][i] * f1; }, l, lref);
                }
                float m0 = S[0][0], m1 = S[1][0];
#pragma unroll
                for (int i = 1; i < 16; ++i) m0 = fmaxf(m0, S[0][i]), m1 = fmaxf(m1, S[1][i]);
                float m = fmaxf(fmaf(m0, f0, s0.y), fmaf(m1, f1, s1.y));
                m = fmaxf(m, xor_lane<32>(m, lane)) - kTop;
                if (__any(m > ref + kSlack)) {
                    const float next = m > ref + kSlack ? m : ref;
                    const float alpha = next == kNegInf ? 0.0f : fast_exp2(ref - next);
                    ref = next;
                    if (!apart) l *= alpha;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) o[dt] *= alpha;
                }
                const float at = ref == kNegInf ? 0.0f : ref;       // no token yet: every weight is 0
                const float a0 = s0.y - at, a1 = s1.y - at;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float f = u ? f1 : f0, add = u ? a1 : a0;
                    float x[16], sum = 0.0f;
                    half8_t P[2][NP];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[i] = fast_exp2(fmaf(S[u][i], f, add));
                        sum += x[i];    // in fp32: weights far below fp16's count, divided by a small value scale
                    }
                    split_half<NP>(x, P[0]);
                    split_half<NP>(x + 8, P[1]);
                    if (!apart) l = fmaf(sum, u ? s1.z : s0.z, l);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int dt = 0; dt < DT; ++dt) {
                            const half8_t v = __builtin_bit_cast(
                                half8_t, sh_v[buf][(32 * dt + r) * 8 + ((4 * u + 2 * h + e) ^ key_of<8>(r))]);
#pragma unroll
                            for (int p = 0; p < NP; ++p) o[dt] = mfma32(v, P[e][p], o[dt]);
                        }
                }
            }
            if (!late) stage_next(t, buf);
            lds_barrier();
        }

        if (apart) {
            const float top = fmaxf(lref, xor_lane<32>(lref, lane));
            l *= exp2_below(lref, top);
            lref = top;
        } else lref = ref;
        const float sum = l + xor_lane<32>(l, lane);
        if (SHARED && (A.listed || A.tile_splits == 1)) {
            if (mine.row >= 0) {
                const bool whole = !A.listed || units == s.units;
                const int64_t at = whole ? (int64_t)mine.row * a.q_heads + mine.head
                                         : (int64_t)list_place(worker, unit0 == 0) * M + wave * 32 + r;
                float *po = (whole ? A.state_o : A.part_o) + at * D;
#pragma unroll
                for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4 *>(po + 32 * dt + 2 * i + 4 * h) =
                            make_float4(o[dt][i], o[dt][i + 1], o[dt][i + 2], o[dt][i + 3]);
                if (h == 0) (whole ? A.state_s : A.part_s)[at] = make_float4(ref, sum, lref, 0.0f);
            }
            if (!A.listed) return;
            left -= slots;
            inside += slots;
            continue;
        }
        if (mine.row < 0) return;
        if (A.tile_splits == 1) {
            const float f = out_factor(sum, ref, lref, 16 * DT, reinterpret_cast<float *>(o));
            T *out = static_cast<T *>(a.out) + ((int64_t)mine.row * a.q_heads + mine.head) * D;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float v[4] = {o[dt][i] * f, o[dt][i + 1] * f, o[dt][i + 2] * f, o[dt][i + 3] * f};
                    store_f32x4<T>(out + 32 * dt + 2 * i + 4 * h, v);
                }
            if (a.lse && h == 0)
                a.lse[(int64_t)mine.row * a.q_heads + mine.head] = log_sum(sum, lref);
        } else {
            const int64_t at = (int64_t)blockIdx.x * M + wave * 32 + r;
            float *po = A.part_o + at * D;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4 *>(po + 32 * dt + 2 * i + 4 * h) =
                        make_float4(o[dt][i], o[dt][i + 1], o[dt][i + 2], o[dt][i + 3]);
            if (h == 0) A.part_s[at] = make_float4(ref, sum, lref, 0.0f);
        }
    } while (SHARED && left > 0);
}

// Joins the parts of a column tile's tokens, in their order; one workgroup
// takes 1024 / D columns.
template <int D, typename T, bool SHARED> __global__ __launch_bounds__(256) void kv_tile_join_kernel(AttnArgs A)
{
    constexpr int M = Shape<D>::M, COLS = 1024 / D, QUADS = D / 4;
    const KvAttnLaunch &a = A.a;
    const uint32_t heads = (uint32_t)a.c.kv_heads;
    const int head = (int)(blockIdx.x % heads);
    uint32_t ctile;
    const int b = tile_locate<M>(A, blockIdx.x / heads, &ctile);
    const int tid = (int)threadIdx.x, c = tid / QUADS, d = (tid % QUADS) * 4;
    if (b < 0 || c >= COLS) return;
    const StreamSeq s = stream_seq(A, b, M);
    const int col = (int)blockIdx.y * COLS + c;
    if (col >= M) return;
    const Column q = column(A, s, (int)ctile * M + col, head);
    if (q.row < 0) return;
    auto at = [&](int p) -> int64_t {
        return ((int64_t)(blockIdx.x / heads * (uint32_t)A.tile_splits + p) * heads + head) * M + col;
    };
    float m = kNegInf, u = kNegInf;
#pragma unroll 8
    for (int p = 0; p < A.tile_splits; ++p) {
        const float4 t = A.part_s[at(p)];
        m = fmaxf(m, t.x), u = fmaxf(u, t.z);
    }
    float l = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int p = 0; p < A.tile_splits; ++p) {
        const float4 t = A.part_s[at(p)];
        const float f = exp2_below(t.x, m);
        const float4 o = *reinterpret_cast<const float4 *>(A.part_o + at(p) * D + d);
        l = fmaf(exp2_below(t.z, u), t.y, l);
        v[0] = fmaf(f, o.x, v[0]), v[1] = fmaf(f, o.y, v[1]), v[2] = fmaf(f, o.z, v[2]), v[3] = fmaf(f, o.w, v[3]);
    }
    if constexpr (SHARED) {
        const int64_t row = (int64_t)q.row * a.q_heads + q.head;
        store_f32x4<float>(A.state_o + row * D + d, v);
        if (d == 0) A.state_s[row] = make_float4(m, l, u, 0.0f);
        return;
    }
    const float f = out_factor(l, m, u, 4, v);
    for (int e = 0; e < 4; ++e) v[e] *= f;
    store_f32x4<T>(static_cast<T *>(a.out) + ((int64_t)q.row * a.q_heads + q.head) * D + d, v);
    if (a.lse && d == 0)
        a.lse[(int64_t)q.row * a.q_heads + q.head] = log_sum(l, u);
}

template <int D, int FMT, typename T, bool SHARED> hipError_t tile_go(const AttnArgs &A, hipStream_t stream)
{
    const unsigned segments = A.tile_bound * (unsigned)A.a.c.kv_heads;
    const unsigned grid = A.listed ? (unsigned)A.workers : segments * (unsigned)A.tile_splits;
    kv_tile_kernel<D, FMT, T, SHARED><<<grid, Shape<D>::THREADS, 0, stream>>>(A);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || A.tile_splits == 1) return e;
    constexpr int cols = 1024 / D;
    kv_tile_join_kernel<D, T, SHARED><<<dim3(segments, (Shape<D>::M + cols - 1) / cols), 256, 0, stream>>>(A);
    return hipGetLastError();
}

template <int D, int FMT, typename T> hipError_t tile_shared(const AttnArgs &A, hipStream_t stream)
{
    return A.state_s ? tile_go<D, FMT, T, true>(A, stream) : tile_go<D, FMT, T, false>(A, stream);
}

template <int D> hipError_t tile_types(const AttnArgs &A, hipStream_t stream)
{
    if (A.a.format == KV_INT8)
        return A.a.x_dt == 0 ? tile_shared<D, KV_INT8, float>(A, stream) : tile_shared<D, KV_INT8, bf16_bits>(A, stream);
    return A.a.x_dt == 0 ? tile_shared<D, KV_FP8, float>(A, stream) : tile_shared<D, KV_FP8, bf16_bits>(A, stream);
}

}  // namespace

int prefill_columns(const KvAttnLaunch &a) { return a.c.head_dim <= 128 ? Shape<128>::M : Shape<256>::M; }

hipError_t launch_kv_prefill(const AttnArgs &A, hipStream_t stream)
{
    switch (A.a.c.head_dim) {
    case 64: return tile_types<64>(A, stream);
    case 128: return tile_types<128>(A, stream);
    case 192: return tile_types<192>(A, stream);
    default: return tile_types<256>(A, stream);
    }
}

}  // namespace nqk
