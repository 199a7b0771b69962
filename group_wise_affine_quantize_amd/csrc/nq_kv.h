// The 8-bit key/value cache: launch descriptors shared by the C-ABI layer and
// the kernels (kv_cache.hip, kv_attention.hip), and the expert router's
// (moe_route.hip).  Launchers assume validated arguments and only enqueue.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nqk {

// Workgroups that one launch may have along x: the runtime counts its threads
// in 32 bits, and takes more of them modulo 2^32 without an error.
constexpr int64_t most_workgroups(int threads) { return (((int64_t)1 << 32) - 1) / threads; }

enum { KV_INT8 = 1, KV_FP8 = 2 };

// The cache's arrays (layouts in include/nq.h).
struct KvCache {
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int64_t blocks;
    int kv_heads, head_dim, block_shift;   // block_tokens = 1 << block_shift
};

// The sequences of a call: device arrays, read by the kernels only.  Every
// value is clamped where it is read (see kv_seq), so no content of these
// arrays can lead a kernel out of the cache or of the rows.
struct KvSeqs {
    const int32_t *row_start, *lengths, *table;
    int64_t rows, max_blocks, ldt;
    int batch;
};

struct KvAppendLaunch {
    KvCache c;
    KvSeqs s;
    const void *k, *v;
    int64_t ldk, ldv;
    int64_t item0 = 0;      // first block of the launch (see max_items)
    int x_dt, format;
};
hipError_t launch_kv_append(const KvAppendLaunch &a, hipStream_t stream);

struct KvReadLaunch {
    KvCache c;
    KvSeqs s;
    void *k, *v;
    int64_t item0 = 0;
    int out_dt, format;
};
hipError_t launch_kv_read(const KvReadLaunch &a, hipStream_t stream);

struct KvAttnLaunch {
    KvCache c;
    KvSeqs s;
    const void *q;
    int64_t ldq;
    void *out;
    float *lse;      // or null
    void *workspace;
    int q_heads, x_dt, format, causal;
    int64_t window;  // 0: none
    float scale;
};
size_t kv_attn_ws_bytes(const KvAttnLaunch &a);
hipError_t launch_kv_attention(const KvAttnLaunch &a, hipStream_t stream);

enum { MOE_SOFTMAX = 1, MOE_SIGMOID = 2 };
struct MoeRoute {
    int experts, score, groups, top_groups, group_best, top_k, renormalise;
    float scale;
};
struct MoeRouteLaunch {
    MoeRoute r;
    const void *logits;
    const float *bias;       // or null
    int64_t tokens, ldl;
    uint32_t *ids;
    float *weights;
    int x_dt;
};
hipError_t launch_moe_route(const MoeRouteLaunch &a, hipStream_t stream);

struct MoeGradLaunch {
    MoeRoute r;
    const void *logits;
    const uint32_t *ids;
    const float *dweights;
    void *dlogits;
    int64_t tokens, ldl;
    int x_dt;
};
hipError_t launch_moe_route_grad(const MoeGradLaunch &a, hipStream_t stream);

}  // namespace nqk
