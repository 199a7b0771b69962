// Attention over the 8-bit cache for many query rows (prompts and their
// chunks); the mathematics is at the head of kv_attention.hip.
//
// A workgroup of four waves takes 128 * CQ query columns of one key/value head
// (a column is a row of the call and one of the head's queries) and runs over
// the tokens that they see, 64 at a time.  The tile's codes are converted to
// fp16 once, into LDS, where the four waves read them as operands of 32x32x16
// MFMAs: S^T = K q^T, O^T = V^T P^T.  CQ = 2 (head_dim up to 128): every
// operand read from LDS feeds two MFMAs, which keeps the LDS at half of its
// rate while the matrix cores run.
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
// 2^(14 + kSlack) in fp16.
#include "nq_kv_attn.h"
#include "nq_tiles.h"

namespace nqk {

namespace {

typedef float float16_t __attribute__((ext_vector_type(16)));

constexpr int kTileWaves = 4;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr float kSlack = 1.5f;

template <int D> struct Shape {
    static constexpr int CQ = D <= 128 ? 2 : 1;         // 32-column blocks per wave
    static constexpr int M = 32 * CQ * kTileWaves;      // columns per workgroup
};

__device__ __forceinline__ float16_t mfma32(half8_t a, half8_t b, float16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// The column tiles of a sequence here.
template <int M> __device__ __forceinline__ uint32_t tile_count(const AttnArgs &A, int b)
{
    const KvSeq q = kv_seq(A.a.s, b);
    const int cols = (int)q.n * A.group;
    return cols > A.few ? (uint32_t)(cols + M - 1) / M : 0u;
}

// Finds column tile `rank` counted from the end of the list (the last tiles of
// a causal sequence see the most tokens, and start first).
template <int M> __device__ __forceinline__ int tile_locate(const AttnArgs &A, uint32_t rank, uint32_t *ctile)
{
    const int batch = A.a.s.batch, lane = (int)(threadIdx.x & 63u);
    uint32_t base = 0;
    for (int b0 = 0; b0 < batch; b0 += 64) {
        const int b = batch - 1 - b0 - lane;
        const uint32_t c = b >= 0 ? tile_count<M>(A, b) : 0u;
        const uint32_t upto = wave_scan32(c);
        const uint32_t sum = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
        if (base + sum > rank) {
            const int l = __ffsll((unsigned long long)__ballot(base + upto > rank)) - 1;
            // tiles of this sequence after the wanted one
            *ctile = (uint32_t)__builtin_amdgcn_readlane((int)upto, l) + base - rank - 1;
            return batch - 1 - b0 - l;
        }
        base += sum;
    }
    return -1;
}

template <int D, int FMT, typename T>
__global__ __launch_bounds__(kTileThreads) void kv_tile_kernel(AttnArgs A)
{
    constexpr int NP = Parts<T>::n, CQ = Shape<D>::CQ, M = Shape<D>::M, KS = D / 16, DT = D / 32, LD = D / 64;
    constexpr int KC = D / 8;       // 16-byte chunks of a key row in LDS
    // keys [64 rows][D], values [D][64 tokens], fp16, 16-byte chunks xored with
    // the row's low bits: the eight lanes that a phase of a 16-byte read serves
    // then cover all banks
    __shared__ uint4 sh_k[2][kTile * KC];
    __shared__ uint4 sh_v[2][D * 8];
    __shared__ float4 sh_s[2][4];   // of each 16 tokens: key scale, log2 and reciprocal of the value scale, whether any is there
    const KvAttnLaunch &a = A.a;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 31, h = lane >> 5;
    const int sh = a.c.block_shift, bmask = (1 << sh) - 1;

    // workgroups of one head follow each other with the number of heads as
    // their distance: with eight heads an XCD keeps to one head's cache
    const uint32_t heads = (uint32_t)a.c.kv_heads;
    const int head = (int)(blockIdx.x % heads);
    const uint32_t rest = blockIdx.x / heads;
    const int split = (int)(rest % (uint32_t)A.tile_splits);
    uint32_t ctile;
    const int b = tile_locate<M>(A, rest / (uint32_t)A.tile_splits, &ctile);
    if (b < 0) return;
    const StreamSeq s = stream_seq(A, b, M);
    const int count = s.n * A.group, col0 = (int)ctile * M, end = col0 + M < count ? col0 + M : count;
    const Column c0 = column(A, s, col0, head), c1 = column(A, s, end - 1, head);
    const int seg_lo = c0.lo, seg_hi = c1.hi;
    const int first_tile = seg_lo >> 6, tiles = seg_hi > seg_lo ? ((seg_hi + 63) >> 6) - first_tile : 0;
    const int t_begin = first_tile + (int)((int64_t)tiles * split / A.tile_splits);
    const int t_end = first_tile + (int)((int64_t)tiles * (split + 1) / A.tile_splits);

    // queries
    half8_t q[CQ][KS][NP];
    float cf[CQ], ref[CQ], l[CQ];
    int col_lo[CQ], col_hi[CQ];
    float16_t o[CQ][DT];
    const int wcol = col0 + wave * 32 * CQ;     // the wave's first column
#pragma unroll
    for (int cq = 0; cq < CQ; ++cq) {
        const Column c = column(A, s, wcol + 32 * cq + r, head);
        col_lo[cq] = c.lo, col_hi[cq] = c.hi;
        float top = 0.0f;
        const T *src = static_cast<const T *>(a.q) + (int64_t)(c.row < 0 ? 0 : c.row) * a.ldq + c.head * D + 8 * h;
        // twice over the row (it stays in the cache): its maximum, then its parts
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            float f[8];
            load_f32x8<T>(src + 16 * ks, f);
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
        }
        top = fmaxf(top, xor_lane<32>(top, lane));
        float back;
        const float up = c.row < 0 ? 0.0f : row_scale(top, &back);
        if (c.row < 0) back = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            float f[8];
            load_f32x8<T>(src + 16 * ks, f);
            for (int i = 0; i < 8; ++i) f[i] = c.row < 0 ? 0.0f : f[i] * up;
            split_half<NP>(f, q[cq][ks]);
        }
        cf[cq] = a.scale * kLog2e * back;
        ref[cq] = kNegInf, l[cq] = 0.0f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
            for (int i = 0; i < 16; ++i) o[cq][dt][i] = 0.0f;
    }
    // tokens that every column of the wave sees, and that some column sees
    const int wend = wcol + 32 * CQ < end ? wcol + 32 * CQ : end;
    const Column w0 = column(A, s, wcol, head), w1 = column(A, s, wend - 1, head);
    const bool empty = wcol >= end;
    const int all_lo = w1.lo, all_hi = w0.hi, any_lo = empty ? 0 : w0.lo, any_hi = empty ? 0 : w1.hi;

    // staging: this thread's 16-byte pieces of a tile's keys and values
    const int *table = a.s.table + (int64_t)b * a.s.ldt;
    auto block_of = [&](int pos) -> int {
        if (pos >= seg_hi || pos + 16 <= seg_lo) return -1;     // also keeps pos inside the table
        const int id = table[pos >> sh];
        return id >= 0 && id < (int)a.c.blocks ? id : -1;
    };
    uint4 kw[LD], vw[LD];
    int vid;
    float sk = 0.0f, sv = 1.0f;
    auto load = [&](int t) {
        const int base = t << 6;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const int piece = tid + i * kTileThreads, tok = piece / (D / 16), c16 = piece % (D / 16);
            const int pos = base + tok, id = block_of(pos & ~15);
            kw[i] = *reinterpret_cast<const uint4 *>(
                a.c.k_codes + ((((int64_t)(id < 0 ? 0 : id) * a.c.kv_heads + head) << sh) + (pos & bmask)) * D + 16 * c16);
        }
        const int pos = base + 16 * (tid & 3);
        vid = block_of(pos);
        const int64_t slab = (int64_t)(vid < 0 ? 0 : vid) * a.c.kv_heads + head;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const int d = (tid >> 2) + i * (kTileThreads / 4);
            vw[i] = *reinterpret_cast<const uint4 *>(a.c.v_codes + ((slab * D + d) << sh) + (pos & bmask));
        }
        if (tid < 4) {
            sk = 0.0f, sv = 1.0f;
            if (vid >= 0) sk = a.c.k_scales[slab], sv = a.c.v_scales[slab];
        }
    };
    auto stage = [&](int t, int buf) {
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const int piece = tid + i * kTileThreads, tok = piece / (D / 16), c16 = piece % (D / 16);
            const int u = tok & 31, row = (tok & 32) + 8 * ((u >> 2) & 3) + 4 * (u >> 4) + (u & 3), key = row & 7;
            const half8_t x = codes_to_half<FMT>(kw[i].x, kw[i].y), y = codes_to_half<FMT>(kw[i].z, kw[i].w);
            sh_k[buf][row * KC + ((2 * c16) ^ key)] = __builtin_bit_cast(uint4, x);
            sh_k[buf][row * KC + ((2 * c16 + 1) ^ key)] = __builtin_bit_cast(uint4, y);
        }
        const int tg = tid & 3, pos = (t << 6) + 16 * tg;
        if constexpr (FMT == KV_FP8) {
            // codes of tokens that no column sees are whatever memory holds, a
            // NaN for instance: make them zeros
            if (vid < 0 || pos < seg_lo || pos + 16 > seg_hi) {
                const int lo = vid < 0 ? 16 : seg_lo - pos, hi = seg_hi - pos;
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
            const int d = (tid >> 2) + i * (kTileThreads / 4);
            const half8_t x = codes_to_half<FMT>(vw[i].x, vw[i].y), y = codes_to_half<FMT>(vw[i].z, vw[i].w);
            sh_v[buf][d * 8 + ((2 * tg) ^ (d & 7))] = __builtin_bit_cast(uint4, x);
            sh_v[buf][d * 8 + ((2 * tg + 1) ^ (d & 7))] = __builtin_bit_cast(uint4, y);
        }
        if (tid < 4) {
            const float v = sv == 0.0f ? kZeroBlockScale : sv;
            sh_s[buf][tid] = make_float4(sk, fast_log2(v), 1.0f / v, vid >= 0 ? 1.0f : 0.0f);
        }
    };

    if (t_begin < t_end) {
        load(t_begin);
        stage(t_begin, 0);
        if (t_begin + 1 < t_end) load(t_begin + 1);
    }
    lds_barrier();
    for (int t = t_begin; t < t_end; ++t) {
        const int buf = (t - t_begin) & 1, base = t << 6;
        if (base < any_hi && base + kTile > any_lo) {
            float16_t S[2][CQ];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int cq = 0; cq < CQ; ++cq)
                    for (int i = 0; i < 16; ++i) S[u][cq][i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const half8_t k = __builtin_bit_cast(half8_t, sh_k[buf][(32 * u + r) * KC + ((2 * ks + h) ^ (r & 7))]);
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int cq = 0; cq < CQ; ++cq) S[u][cq] = mfma32(k, q[cq][ks][p], S[u][cq]);
                }
            const float4 s0 = sh_s[buf][h], s1 = sh_s[buf][2 + h];
            const bool masked = base < all_lo || base + kTile > all_hi || __any(s0.w * s1.w == 0.0f);
            half8_t P[CQ][2][2][NP];
#pragma unroll
            for (int cq = 0; cq < CQ; ++cq) {
                if (masked) {
                    const int lo = col_lo[cq] - base - 16 * h, hi = col_hi[cq] - base - 16 * h;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        S[0][cq][i] = i < lo || i >= hi || s0.w == 0.0f ? kNegInf : S[0][cq][i];
                        S[1][cq][i] = 32 + i < lo || 32 + i >= hi || s1.w == 0.0f ? kNegInf : S[1][cq][i];
                    }
                }
                const float f0 = cf[cq] * s0.x, f1 = cf[cq] * s1.x;     // not negative: the maximum is that of S
                float m0 = S[0][cq][0], m1 = S[1][cq][0];
#pragma unroll
                for (int i = 1; i < 16; ++i) m0 = fmaxf(m0, S[0][cq][i]), m1 = fmaxf(m1, S[1][cq][i]);
                m0 = m0 == kNegInf ? kNegInf : fmaf(m0, f0, s0.y);
                m1 = m1 == kNegInf ? kNegInf : fmaf(m1, f1, s1.y);
                float m = fmaxf(m0, m1);
                m = fmaxf(m, xor_lane<32>(m, lane)) - kPScale;
                if (__any(m > ref[cq] + kSlack)) {
                    const float next = m > ref[cq] + kSlack ? m : ref[cq];
                    const float alpha = next == kNegInf ? 0.0f : fast_exp2(ref[cq] - next);
                    ref[cq] = next;
                    l[cq] *= alpha;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) o[cq][dt] *= alpha;
                }
                const float at = ref[cq] == kNegInf ? 0.0f : ref[cq];
                const float a0 = s0.y - at, a1 = s1.y - at;
                float x0[16], x1[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x0[i] = fmaf(S[0][cq][i], f0, a0);
                    x1[i] = fmaf(S[1][cq][i], f1, a1);
                }
                if (masked) {       // a zero factor times a masked score is no number
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x0[i] = S[0][cq][i] == kNegInf ? kNegInf : x0[i];
                        x1[i] = S[1][cq][i] == kNegInf ? kNegInf : x1[i];
                    }
                }
                float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x0[i] = fast_exp2(x0[i]), x1[i] = fast_exp2(x1[i]);
                    sum0 += x0[i], sum1 += x1[i];
                }
                l[cq] = fmaf(sum0, s0.z, fmaf(sum1, s1.z, l[cq]));
                split_half<NP>(x0, P[cq][0][0]);
                split_half<NP>(x0 + 8, P[cq][0][1]);
                split_half<NP>(x1, P[cq][1][0]);
                split_half<NP>(x1 + 8, P[cq][1][1]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt) {
                        const half8_t v = __builtin_bit_cast(
                            half8_t, sh_v[buf][(32 * dt + r) * 8 + ((4 * u + 2 * h + e) ^ (r & 7))]);
#pragma unroll
                        for (int p = 0; p < NP; ++p)
#pragma unroll
                            for (int cq = 0; cq < CQ; ++cq) o[cq][dt] = mfma32(v, P[cq][u][e][p], o[cq][dt]);
                    }
        }
        if (t + 1 < t_end) stage(t + 1, buf ^ 1);
        if (t + 2 < t_end) load(t + 2);
        lds_barrier();
    }

#pragma unroll
    for (int cq = 0; cq < CQ; ++cq) {
        const float sum = l[cq] + xor_lane<32>(l[cq], lane);
        const int col = wave * 32 * CQ + 32 * cq + r;
        const Column c = column(A, s, col0 + col, head);
        if (c.row < 0) continue;
        if (A.tile_splits == 1) {
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            T *out = static_cast<T *>(a.out) + ((int64_t)c.row * a.q_heads + c.head) * D;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float v[4] = {o[cq][dt][i] * inv, o[cq][dt][i + 1] * inv, o[cq][dt][i + 2] * inv, o[cq][dt][i + 3] * inv};
                    store_f32x4<T>(out + 32 * dt + 2 * i + 4 * h, v);
                }
            if (a.lse && h == 0)
                a.lse[(int64_t)c.row * a.q_heads + c.head] = sum > 0.0f ? (ref[cq] + fast_log2(sum)) * kLn2 : kNegInf;
        } else {
            const int64_t at = (int64_t)blockIdx.x * M + col;
            float *po = A.part_o + at * D;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4 *>(po + 32 * dt + 2 * i + 4 * h) =
                        make_float4(o[cq][dt][i], o[cq][dt][i + 1], o[cq][dt][i + 2], o[cq][dt][i + 3]);
            if (h == 0) A.part_ml[2 * at] = ref[cq], A.part_ml[2 * at + 1] = sum;
        }
    }
}

// Joins the parts of a column tile's tokens, in their order; one workgroup
// takes 1024 / D columns.
template <int D, typename T> __global__ __launch_bounds__(256) void kv_tile_join_kernel(AttnArgs A)
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
    float m = kNegInf;
    for (int p = 0; p < A.tile_splits; ++p) m = fmaxf(m, A.part_ml[2 * at(p)]);
    float l = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < A.tile_splits && m != kNegInf; ++p) {
        const float f = fast_exp2(A.part_ml[2 * at(p)] - m);
        const float4 o = *reinterpret_cast<const float4 *>(A.part_o + at(p) * D + d);
        l = fmaf(f, A.part_ml[2 * at(p) + 1], l);
        v[0] = fmaf(f, o.x, v[0]), v[1] = fmaf(f, o.y, v[1]), v[2] = fmaf(f, o.z, v[2]), v[3] = fmaf(f, o.w, v[3]);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    for (int e = 0; e < 4; ++e) v[e] *= inv;
    store_f32x4<T>(static_cast<T *>(a.out) + ((int64_t)q.row * a.q_heads + q.head) * D + d, v);
    if (a.lse && d == 0)
        a.lse[(int64_t)q.row * a.q_heads + q.head] = l > 0.0f ? (m + fast_log2(l)) * kLn2 : kNegInf;
}

template <int D, int FMT, typename T> hipError_t tile_go(const AttnArgs &A, hipStream_t stream)
{
    const unsigned segments = A.tile_bound * (unsigned)A.a.c.kv_heads;
    kv_tile_kernel<D, FMT, T><<<segments * (unsigned)A.tile_splits, kTileThreads, 0, stream>>>(A);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || A.tile_splits == 1) return e;
    constexpr int cols = 1024 / D;
    kv_tile_join_kernel<D, T><<<dim3(segments, (Shape<D>::M + cols - 1) / cols), 256, 0, stream>>>(A);
    return hipGetLastError();
}

template <int D> hipError_t tile_types(const AttnArgs &A, hipStream_t stream)
{
    if (A.a.format == KV_INT8)
        return A.a.x_dt == 0 ? tile_go<D, KV_INT8, float>(A, stream) : tile_go<D, KV_INT8, bf16_bits>(A, stream);
    return A.a.x_dt == 0 ? tile_go<D, KV_FP8, float>(A, stream) : tile_go<D, KV_FP8, bf16_bits>(A, stream);
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
