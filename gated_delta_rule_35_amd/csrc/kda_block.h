// Internal interface of what stands around the delta rule and the scan in a block: the short
// causal convolution (kda_conv, kda_conv_bwd, kda_conv_decode) and the norms after a block and
// before the next (kda_gated_norm, kda_add_norm and their gradients).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct ConvParams {
    const void* x;         // [B, T, C], strides sb and st in elements; decode [N, C], stride sb
    int64_t sb, st;
    const float* w;        // [C, W]
    const float* bias;     // [C] or nullptr
    const int32_t* cu;     // [N + 1] or nullptr
    const void* s_in;      // [N, W - 1, C] (decode [slots, W - 1, C]) or nullptr (zeros)
    void* s_out;           // likewise, or nullptr
    void* y;               // [B, T, C]; decode [N, C]
    int64_t T, total;      // tokens per row, of all rows
    int32_t N, C, W, silu;
    int32_t type;          // 0 bf16, 1 fp16, 2 fp32: x, y, states and their gradients
    // backward
    const void* dy;        // [B, T, C]
    const void* ds_out;    // [N, W - 1, C] or nullptr
    void* dx;              // [B, T, C]
    void* ds_in;           // [N, W - 1, C] or nullptr
    float* part;           // [tiles][W + 1][C]
    float *dw, *db;        // [C, W], [C] or nullptr
    // decode
    const int32_t* idx;    // [N] or nullptr
    int32_t slots;
};

// The split of a convolution's tokens and channels over threads: a thread takes eight channels
// of a run of `run` tokens; `lanes` neighbouring threads lie side by side along the channels, the
// others of a work-group's 256 along the tokens.
struct ConvSplit {
    int32_t run, lanes;
    int64_t tiles, cols;   // work-groups along the tokens and along the channels
};
ConvSplit conv_split(int64_t total, int64_t C, bool bwd);

hipError_t launch_conv(const ConvParams& p, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvParams& p, hipStream_t stream);
hipError_t launch_conv_decode(const ConvParams& p, hipStream_t stream);

struct BlockNormParams {
    const void* x;         // gated: the block's output; add: likewise; add's gradients: the sum h
    int64_t xb, xt, xh;    // strides of [B, T, H] in elements
    const void* z;         // gated: the gate; add: the residual
    int64_t zb, zt, zh;
    const float* w;        // [D], or [H, D] (per_head), or nullptr (ones)
    void* y;               // contiguous
    void* h;               // add: the sum; contiguous
    int64_t T, rows;       // rows = B * T * H
    int32_t H, D, per_head;
    int32_t type;          // of x, y, the gate and their gradients
    int32_t wide;          // add: residual and sum are fp32
    int32_t act, first;    // gated
    float eps, scale;
    // backward
    const void* dy;        // contiguous
    const void* dh;        // add: gradient of the sum from elsewhere, contiguous, or nullptr
    void *dx, *dz;         // contiguous
    float* part;           // [work-groups][D]
    float* dw;             // like w, or nullptr
};
hipError_t launch_gated_norm(const BlockNormParams& p, hipStream_t stream);
hipError_t launch_gated_norm_bwd(const BlockNormParams& p, hipStream_t stream);
hipError_t launch_add_norm(const BlockNormParams& p, hipStream_t stream);
hipError_t launch_add_norm_bwd(const BlockNormParams& p, hipStream_t stream);
// Most work-groups whose sums of the weights' gradients are left to add (of every head, for a
// weight per head, at least one).  1024 were 38 us and not 31 at 3001 x 4096: most of their time went into the sums' rows.
constexpr int BLOCK_DW_GROUPS = 512;

// Sums over the rows of part [n][cols], in a fixed order.  Column c < split goes to
// out[(c % inner) * outer + c / inner], a later one to out2[c - split].
struct SumParams {
    const float* part;
    int64_t n, cols, split, inner, outer;
    float *out, *out2;
};
hipError_t launch_sum_rows(const SumParams& p, hipStream_t stream);

}  // namespace kda
