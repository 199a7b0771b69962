// The steps between a decoder layer's products: launch descriptors shared by
// the C-ABI layer and the kernels (norm.hip, rope.hip, moe_order.hip).
// Launchers assume validated arguments and only enqueue.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nqk {

// Widest row of the norm kernels: 1024 threads hold 16 elements each.
constexpr int kNormMaxDim = 16384;

struct BlockNormLaunch {
    const void *h, *y;                  // y null: no block, z from h
    const void *post, *gate, *pre;      // or null
    int64_t rows, dim, ldh, ldy, ldg, gates;
    void *h_out, *z;                    // z null without pre
    float eps, offset, scale;
    int x_dt, p_dt;
};
hipError_t launch_block_norm(const BlockNormLaunch &a, hipStream_t stream);

struct BlockNormGradLaunch {
    const void *h_out, *y, *dh_out, *dz;    // y, dh_out, dz or null
    const void *post, *gate, *pre;          // or null
    int64_t rows, dim, ldh, ldy, ldd, ldz, ldg, gates;
    void *dh, *dy;                          // dy null without y
    void *dpost, *dgate, *dpre;             // or null
    float *partials;                        // see block_norm_grad_ws_bytes
    float eps, offset, scale;
    int x_dt, p_dt;
};
size_t block_norm_grad_ws_bytes(int64_t rows, int64_t dim, int64_t gates);
hipError_t launch_block_norm_grad(const BlockNormGradLaunch &a, hipStream_t stream);

struct RopeLaunch {
    const void *x;
    void *out;
    const int32_t *positions;   // [axes][ldp]
    const double *freq;         // [rotary / 2]
    const int32_t *axis;        // [rotary / 2], or null: the first axis
    int64_t rows, ldx, ldo, ldp;
    int heads, head_dim, rotary, axes, pairs;   // pairs: neighbouring columns, not halves
    float cos_scale, sin_scale;                 // sin_scale negative: turned back
    int x_dt;
};
hipError_t launch_rope(const RopeLaunch &a, hipStream_t stream);

struct MoeSortLaunch {
    const uint32_t *ids;
    int64_t pairs;
    int top_k, experts;
    int32_t *starts, *place;
    uint32_t *row_token, *row_expert;
    int32_t *counts;            // see moe_sort_ws_bytes
};
size_t moe_sort_ws_bytes(int64_t pairs, int experts);
hipError_t launch_moe_sort(const MoeSortLaunch &a, hipStream_t stream);

// Rows between token order and expert order.
struct MoeRowsLaunch {
    const int32_t *kept;        // rows of experts that exist: starts[experts]
    const int32_t *place;       // [tokens][top_k]
    int64_t tokens, hidden;
    int top_k, x_dt;
    const void *in;             // dispatch: x; combine: ys; combine_grad: dy
    int64_t ldi;                // row stride of x, dy
    void *out;                  // xs; y; dys
    const float *weights;       // or null: ones
    const void *residual;       // combine, or null
    int64_t ldr;
    const void *ys;             // combine_grad
    float *dweights;            // combine_grad, or null
};
hipError_t launch_moe_dispatch(const MoeRowsLaunch &a, hipStream_t stream);
hipError_t launch_moe_combine(const MoeRowsLaunch &a, hipStream_t stream);
hipError_t launch_moe_combine_grad(const MoeRowsLaunch &a, hipStream_t stream);

}  // namespace nqk
