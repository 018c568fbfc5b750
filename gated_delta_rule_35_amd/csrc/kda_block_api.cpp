// C-ABI front end of what stands around the delta rule and the scan in a block: the short
// causal convolution (kda_conv, kda_conv_bwd, kda_conv_decode) and the norms (kda_gated_norm,
// kda_add_norm and their gradients): argument checks and launch.  As in the rest of the
// library every check runs on the host before any HIP call, and the host never reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kda_block.h"
#include "kda_check.h"

namespace {

using namespace kda::check;

constexpr int64_t kMaxStride = int64_t(1) << 31;
constexpr int64_t kMaxGrid = int64_t(1) << 23;   // 256 threads each
constexpr int64_t kMaxConvChannels = int64_t(1) << 20, kMaxNormChannels = 8192;

bool any_type(kda_dtype_t d) { return d == KDA_BF16 || d == KDA_F16 || d == KDA_F32; }
int type_code(kda_dtype_t d) { return d == KDA_BF16 ? 0 : d == KDA_F16 ? 1 : 2; }

// A view whose last dimension is contiguous, a multiple of 8 elements, and whose other strides are non-negative multiples
// of 8 elements (those of dimensions of size 1 do not matter and come back as 0).
kda_status_t check_view(const kda_tensor_t* t, int ndim, int64_t (&stride)[3]) {
    if (!t) return KDA_ERR_NULL;
    if (!any_type(t->dtype)) return KDA_ERR_DTYPE;
    if (t->ndim != ndim || !sizes_ok(t)) return KDA_ERR_SHAPE;
    int64_t n = 1;
    for (int i = 0; i < ndim; ++i) {
        if (i < 3) stride[i] = 0;
        n = t->shape[i] == 0 ? 0 : n;
    }
    if (t->shape[ndim - 1] % 8 != 0) return KDA_ERR_UNSUPPORTED;
    if (n == 0) return KDA_OK;
    if (!t->data) return KDA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0) return KDA_ERR_LAYOUT;
    if (t->shape[ndim - 1] != 1 && t->stride[ndim - 1] != 1) return KDA_ERR_LAYOUT;
    for (int i = 0; i < ndim - 1; ++i) {
        if (t->shape[i] == 1) continue;
        if (t->stride[i] < 0 || t->stride[i] % 8 != 0 || t->stride[i] > kMaxStride * 256) return KDA_ERR_LAYOUT;
        stride[i] = t->stride[i];
    }
    return KDA_OK;
}
// A contiguous tensor of the given type and shape.
kda_status_t check_dense(const kda_tensor_t* t, kda_dtype_t type, int ndim, const int64_t* shape, size_t align) {
    const kda_status_t st = check_tensor(t, ndim, type, type, align);
    if (st != KDA_OK) return st;
    return same_shape(t, shape, ndim) ? KDA_OK : KDA_ERR_SHAPE;
}
// Whether an output shares memory with an input other than one that it may replace: `own` itself,
// contiguous and of the same type.
bool clashes(const kda_tensor_t* out, const kda_tensor_t* own, const kda_tensor_t* in) {
    if (in && in == own && in->data == out->data && in->dtype == out->dtype && contiguous(in)) return false;
    return overlaps(out, in);
}

// What the convolution's calls share: inputs, weights, activation.
kda_status_t prepare_conv(const kda_tensor_t* x, int ndim, const kda_tensor_t* weight, const kda_tensor_t* bias,
                          int32_t activation, kda::ConvParams& p) {
    kda_status_t st;
    p = kda::ConvParams{};
    int64_t s[3] = {0, 0, 0};
    if ((st = check_view(x, ndim, s)) != KDA_OK) return st;
    if ((st = check_tensor(weight, 2, KDA_F32, KDA_F32, 16)) != KDA_OK) return st;
    const int64_t C = x->shape[ndim - 1], W = weight->shape[1];
    if (weight->shape[0] != C || C < 1) return KDA_ERR_SHAPE;
    if (C > kMaxConvChannels || W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
    if (bias && (st = check_dense(bias, KDA_F32, 1, &C, 4)) != KDA_OK) return st;
    if (activation != 0 && activation != 1) return KDA_ERR_VALUE;
    p.x = x->data;
    p.sb = s[0];
    p.st = ndim == 3 ? s[1] : 0;
    p.w = static_cast<const float*>(weight->data);
    p.bias = bias ? static_cast<const float*>(bias->data) : nullptr;
    p.C = static_cast<int32_t>(C);
    p.W = static_cast<int32_t>(W);
    p.silu = activation;
    p.type = type_code(x->dtype);
    return KDA_OK;
}
// Batch, sequences and grid of the calls over sequences.
kda_status_t conv_batch(const kda_tensor_t* x, const kda_tensor_t* cu, kda::ConvParams& p) {
    kda_status_t st;
    const int64_t B = x->shape[0], T = x->shape[1];
    int64_t N = B;
    if (cu) {
        if ((st = check_tensor(cu, 1, KDA_I32, KDA_I32, 4)) != KDA_OK) return st;
        if (B != 1) return KDA_ERR_UNSUPPORTED;
        if (cu->shape[0] < 1) return KDA_ERR_SHAPE;
        N = cu->shape[0] - 1;
        p.cu = static_cast<const int32_t*>(cu->data);
    }
    if (N > (int64_t(1) << 24) || B * T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    p.N = static_cast<int32_t>(N);
    p.T = T;
    p.total = B * T;
    for (const bool bwd : {false, true}) {
        const kda::ConvSplit k = kda::conv_split(p.total, p.C, bwd);
        if (k.tiles * k.cols + (N * (p.W - 1) * (p.C / 8)) / 256 + 1 > kMaxGrid) return KDA_ERR_UNSUPPORTED;
    }
    return KDA_OK;
}
kda_status_t check_conv_state(const kda_tensor_t* t, const kda::ConvParams& p, kda_dtype_t type, int64_t n) {
    if (!t) return KDA_OK;
    const int64_t s[3] = {n, p.W - 1, p.C};
    return check_dense(t, type, 3, s, 16);
}
void* data_of(const kda_tensor_t* t) { return t ? t->data : nullptr; }

}  // namespace

extern "C" {

kda_status_t kda_conv(const kda_tensor_t* x, const kda_tensor_t* weight, const kda_tensor_t* bias, int32_t activation,
                      const kda_tensor_t* cu_seqlens, const kda_tensor_t* initial_state, const kda_tensor_t* out,
                      const kda_tensor_t* final_state, void* stream) {
    kda::ConvParams p;
    kda_status_t st = prepare_conv(x, 3, weight, bias, activation, p);
    if (st != KDA_OK) return st;
    if ((st = conv_batch(x, cu_seqlens, p)) != KDA_OK) return st;
    if ((st = check_conv_state(initial_state, p, x->dtype, p.N)) != KDA_OK) return st;
    if ((st = check_conv_state(final_state, p, x->dtype, p.N)) != KDA_OK) return st;
    if ((st = check_dense(out, x->dtype, 3, x->shape, 16)) != KDA_OK) return st;
    const kda_tensor_t* ins[] = {x, weight, bias, cu_seqlens, initial_state};
    const kda_tensor_t* outs[] = {out, final_state};
    if (any_overlap(outs, 2, ins, 5)) return KDA_ERR_LAYOUT;
    p.s_in = data_of(initial_state);
    p.s_out = data_of(final_state);
    p.y = out->data;
    if (p.N == 0) return KDA_OK;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return finish(kda::launch_conv(p, hs), hs);
}

int64_t kda_conv_bwd_workspace_size(int64_t total_tokens, int64_t channels, int64_t width) {
    if (total_tokens < 0 || total_tokens > kMaxTokens || channels < 0 || channels > kMaxConvChannels || width < 0 || width > 4)
        return -1;
    if (channels == 0) return 0;
    return kda::conv_split(total_tokens, channels, true).tiles * (width + 1) * channels * 4;
}

kda_status_t kda_conv_bwd(const kda_tensor_t* x, const kda_tensor_t* weight, const kda_tensor_t* bias, int32_t activation,
                          const kda_tensor_t* cu_seqlens, const kda_tensor_t* initial_state, const kda_tensor_t* d_out,
                          const kda_tensor_t* d_final_state, const kda_tensor_t* dx, const kda_tensor_t* dweight,
                          const kda_tensor_t* dbias, const kda_tensor_t* d_initial_state, void* workspace,
                          int64_t workspace_size, void* stream) {
    kda::ConvParams p;
    kda_status_t st = prepare_conv(x, 3, weight, bias, activation, p);
    if (st != KDA_OK) return st;
    if ((st = conv_batch(x, cu_seqlens, p)) != KDA_OK) return st;
    for (const kda_tensor_t* t : {initial_state, d_final_state, d_initial_state})
        if ((st = check_conv_state(t, p, x->dtype, p.N)) != KDA_OK) return st;
    if ((st = check_dense(d_out, x->dtype, 3, x->shape, 16)) != KDA_OK) return st;
    if ((st = check_dense(dx, x->dtype, 3, x->shape, 16)) != KDA_OK) return st;
    if ((st = check_dense(dweight, KDA_F32, 2, weight->shape, 4)) != KDA_OK) return st;
    if (dbias) {
        if (!bias) return KDA_ERR_NULL;
        if ((st = check_dense(dbias, KDA_F32, 1, bias->shape, 4)) != KDA_OK) return st;
    }
    const kda_tensor_t* ins[] = {x, weight, bias, cu_seqlens, initial_state, d_out, d_final_state};
    const kda_tensor_t* outs[] = {dx, dweight, dbias, d_initial_state};
    if (any_overlap(outs, 4, ins, 7)) return KDA_ERR_LAYOUT;
    const int64_t need = kda_conv_bwd_workspace_size(p.total, p.C, p.W);
    if (workspace && (workspace_size < need || reinterpret_cast<uintptr_t>(workspace) % 16 != 0)) return KDA_ERR_WORKSPACE;
    p.s_in = data_of(initial_state);
    p.dy = d_out->data;
    p.ds_out = data_of(d_final_state);
    p.dx = dx->data;
    p.ds_in = data_of(d_initial_state);
    p.dw = static_cast<float*>(dweight->data);
    p.db = static_cast<float*>(data_of(dbias));
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    void* ws = workspace;
    if (!ws && need > 0 && hipMallocAsync(&ws, (size_t)need, hs) != hipSuccess) return KDA_ERR_HIP;
    p.part = static_cast<float*>(ws);
    hipError_t e = kda::launch_conv_bwd(p, hs);
    if (!workspace && ws && hipFreeAsync(ws, hs) != hipSuccess && e == hipSuccess) e = hipErrorUnknown;
    return finish(e, hs);
}

kda_status_t kda_conv_decode(const kda_tensor_t* x, const kda_tensor_t* weight, const kda_tensor_t* bias,
                             int32_t activation, const kda_tensor_t* state_in, const kda_tensor_t* state_out,
                             const kda_tensor_t* state_indices, const kda_tensor_t* out, void* stream) {
    kda::ConvParams p;
    kda_status_t st = prepare_conv(x, 2, weight, bias, activation, p);
    if (st != KDA_OK) return st;
    const int64_t N = x->shape[0];
    if (state_indices) {
        if ((st = check_dense(state_indices, KDA_I32, 1, &N, 4)) != KDA_OK) return st;
        p.idx = static_cast<const int32_t*>(state_indices->data);
    }
    if (!state_out) return KDA_ERR_NULL;
    const int64_t slots = state_indices && state_out->ndim == 3 ? state_out->shape[0] : N;
    if ((st = check_conv_state(state_out, p, x->dtype, slots)) != KDA_OK) return st;
    if ((st = check_conv_state(state_in, p, x->dtype, slots)) != KDA_OK) return st;
    if ((st = check_dense(out, x->dtype, 2, x->shape, 16)) != KDA_OK) return st;
    if (N > (int64_t(1) << 24) || slots > kMaxTokens || N * (p.C / 1024 + 1) > kMaxGrid) return KDA_ERR_UNSUPPORTED;
    const kda_tensor_t* ins[] = {x, weight, bias, state_indices};
    const kda_tensor_t* outs[] = {out, state_out};
    if (any_overlap(outs, 2, ins, 4) || overlaps(out, state_in)) return KDA_ERR_LAYOUT;
    if (state_in && partly_overlap(state_in->data, state_out->data, span_of(state_out).bytes)) return KDA_ERR_LAYOUT;
    p.N = static_cast<int32_t>(N);
    p.slots = static_cast<int32_t>(slots);
    p.s_in = data_of(state_in);
    p.s_out = state_out->data;
    p.y = out->data;
    if (N == 0 || slots == 0) return KDA_OK;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return finish(kda::launch_conv_decode(p, hs), hs);
}

}  // extern "C"

// ---- the norms around a block ----
namespace {

// Rows [B, T, H, D] of x, or [B, T, D] with ndim 3; the weight; eps.
kda_status_t prepare_norm(const kda_tensor_t* x, int ndim, const kda_tensor_t* weight, float eps, kda::BlockNormParams& p) {
    kda_status_t st;
    p = kda::BlockNormParams{};
    int64_t s[3] = {0, 0, 0};
    if ((st = check_view(x, ndim, s)) != KDA_OK) return st;
    const int64_t B = x->shape[0], T = x->shape[1], H = ndim == 4 ? x->shape[2] : 1, D = x->shape[ndim - 1];
    if (H < 1 || D < 1) return KDA_ERR_SHAPE;
    if (D > kMaxNormChannels || H > (int64_t(1) << 16) || B * T > kMaxTokens || B * T * H > kMaxTokens)
        return KDA_ERR_UNSUPPORTED;
    if (weight) {
        const bool heads = ndim == 4 && weight->ndim == 2;
        const int64_t ws[2] = {heads ? H : D, D};
        if ((st = check_dense(weight, KDA_F32, heads ? 2 : 1, ws, 16)) != KDA_OK) return st;
        p.w = static_cast<const float*>(weight->data);
        p.per_head = heads;
    }
    if (!std::isfinite(eps) || !(eps > 0.f)) return KDA_ERR_VALUE;
    p.x = x->data;
    p.xb = s[0];
    p.xt = s[1];
    p.xh = ndim == 4 ? s[2] : 0;
    p.T = T;
    p.rows = B * T * H;
    p.H = static_cast<int32_t>(H);
    p.D = static_cast<int32_t>(D);
    p.type = type_code(x->dtype);
    p.eps = eps;
    // work-groups of a row up to 128 channels hold 16 of them, up to 2048 four
    if (p.rows / (D <= 128 ? 16 : D <= 2048 ? 4 : 1) + p.H > kMaxGrid) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
// The gate of x's shape and type.
kda_status_t prepare_gate(const kda_tensor_t* x, const kda_tensor_t* gate, int32_t activation, int32_t gate_first,
                          kda::BlockNormParams& p) {
    int64_t s[3] = {0, 0, 0};
    const kda_status_t st = check_view(gate, 4, s);
    if (st != KDA_OK) return st;
    if (gate->dtype != x->dtype) return KDA_ERR_DTYPE;
    if (!same_shape(gate, x->shape, 4)) return KDA_ERR_SHAPE;
    if (activation != 1 && activation != 2) return KDA_ERR_VALUE;
    p.z = gate->data;
    p.zb = s[0];
    p.zt = s[1];
    p.zh = s[2];
    p.act = activation;
    p.first = gate_first ? 1 : 0;
    return KDA_OK;
}
kda_status_t check_dweight(const kda_tensor_t* dweight, const kda_tensor_t* weight, kda::BlockNormParams& p) {
    if (!dweight) return KDA_OK;
    if (!weight) return KDA_ERR_NULL;
    const kda_status_t st = check_dense(dweight, KDA_F32, weight->ndim, weight->shape, 4);
    if (st != KDA_OK) return st;
    // their sums' launch takes 256 threads for 32 of them, and fewer than 2^32 in all
    if ((numel(weight) + 31) / 32 >= int64_t(1) << 24) return KDA_ERR_UNSUPPORTED;
    p.dw = static_cast<float*>(dweight->data);
    return KDA_OK;
}
// Runs a backward with its workspace, which only weight gradients need.
template <typename F>
kda_status_t with_workspace(kda::BlockNormParams& p, void* workspace, int64_t workspace_size, void* stream, F launch) {
    const int64_t need = p.dw ? kda_norm_bwd_workspace_size(p.per_head ? p.H : 1, p.D) : 0;
    if (need > 0 && workspace && (workspace_size < need || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
        return KDA_ERR_WORKSPACE;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    void* ws = need > 0 ? workspace : nullptr;
    if (need > 0 && !ws && hipMallocAsync(&ws, (size_t)need, hs) != hipSuccess) return KDA_ERR_HIP;
    p.part = static_cast<float*>(ws);
    hipError_t e = launch(p, hs);
    if (need > 0 && !workspace && hipFreeAsync(ws, hs) != hipSuccess && e == hipSuccess) e = hipErrorUnknown;
    return finish(e, hs);
}

}  // namespace

extern "C" {

int64_t kda_norm_bwd_workspace_size(int64_t heads, int64_t channels) {
    if (heads < 0 || heads > (int64_t(1) << 16) || channels < 0 || channels > kMaxNormChannels) return -1;
    return std::max<int64_t>(kda::BLOCK_DW_GROUPS, heads) * channels * 4;
}

kda_status_t kda_gated_norm(const kda_tensor_t* x, const kda_tensor_t* gate, const kda_tensor_t* weight,
                            int32_t activation, int32_t gate_first, float eps, const kda_tensor_t* out, void* stream) {
    kda::BlockNormParams p;
    kda_status_t st = prepare_norm(x, 4, weight, eps, p);
    if (st != KDA_OK) return st;
    if ((st = prepare_gate(x, gate, activation, gate_first, p)) != KDA_OK) return st;
    if ((st = check_dense(out, x->dtype, 4, x->shape, 16)) != KDA_OK) return st;
    if (clashes(out, x, x) || overlaps(out, gate) || overlaps(out, weight)) return KDA_ERR_LAYOUT;
    p.y = out->data;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return finish(kda::launch_gated_norm(p, hs), hs);
}

kda_status_t kda_gated_norm_bwd(const kda_tensor_t* x, const kda_tensor_t* gate, const kda_tensor_t* weight,
                                int32_t activation, int32_t gate_first, float eps, const kda_tensor_t* d_out,
                                const kda_tensor_t* dx, const kda_tensor_t* dgate, const kda_tensor_t* dweight,
                                void* workspace, int64_t workspace_size, void* stream) {
    kda::BlockNormParams p;
    kda_status_t st = prepare_norm(x, 4, weight, eps, p);
    if (st != KDA_OK) return st;
    if ((st = prepare_gate(x, gate, activation, gate_first, p)) != KDA_OK) return st;
    for (const kda_tensor_t* t : {d_out, dx, dgate})
        if ((st = check_dense(t, x->dtype, 4, x->shape, 16)) != KDA_OK) return st;
    if ((st = check_dweight(dweight, weight, p)) != KDA_OK) return st;
    const kda_tensor_t* ins[] = {x, gate, weight, d_out};
    const kda_tensor_t* outs[] = {dx, dgate, dweight};
    if (any_overlap(outs, 3, ins, 4)) return KDA_ERR_LAYOUT;
    p.dy = d_out->data;
    p.dx = dx->data;
    p.dz = dgate->data;
    return with_workspace(p, workspace, workspace_size, stream, kda::launch_gated_norm_bwd);
}

kda_status_t kda_add_norm(const kda_tensor_t* x, const kda_tensor_t* residual, const kda_tensor_t* weight, float scale,
                          float eps, const kda_tensor_t* out, const kda_tensor_t* sum, void* stream) {
    kda::BlockNormParams p;
    kda_status_t st = prepare_norm(x, 3, weight, eps, p);
    if (st != KDA_OK) return st;
    int64_t s[3] = {0, 0, 0};
    if ((st = check_view(residual, 3, s)) != KDA_OK) return st;
    if (residual->dtype != x->dtype && residual->dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (!same_shape(residual, x->shape, 3)) return KDA_ERR_SHAPE;
    if (!std::isfinite(scale)) return KDA_ERR_VALUE;
    if ((st = check_dense(out, x->dtype, 3, x->shape, 16)) != KDA_OK) return st;
    if ((st = check_dense(sum, residual->dtype, 3, x->shape, 16)) != KDA_OK) return st;
    if (clashes(out, x, x) || overlaps(out, residual) || overlaps(out, weight)) return KDA_ERR_LAYOUT;
    if (clashes(sum, residual, residual) || overlaps(sum, x) || overlaps(sum, weight) || overlaps(sum, out))
        return KDA_ERR_LAYOUT;
    p.z = residual->data;
    p.zb = s[0];
    p.zt = s[1];
    p.wide = residual->dtype == KDA_F32;
    p.scale = scale;
    p.y = out->data;
    p.h = sum->data;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return finish(kda::launch_add_norm(p, hs), hs);
}

kda_status_t kda_add_norm_bwd(const kda_tensor_t* sum, const kda_tensor_t* weight, float scale, float eps,
                              const kda_tensor_t* d_out, const kda_tensor_t* d_sum, const kda_tensor_t* dx,
                              const kda_tensor_t* dresidual, const kda_tensor_t* dweight, void* workspace,
                              int64_t workspace_size, void* stream) {
    kda::BlockNormParams p;
    kda_status_t st = prepare_norm(sum, 3, weight, eps, p);
    if (st != KDA_OK) return st;
    if (!std::isfinite(scale)) return KDA_ERR_VALUE;
    if (!d_out) return KDA_ERR_NULL;
    if (!any_type(d_out->dtype) || (sum->dtype != d_out->dtype && sum->dtype != KDA_F32)) return KDA_ERR_DTYPE;
    if ((st = check_dense(d_out, d_out->dtype, 3, sum->shape, 16)) != KDA_OK) return st;
    if (d_sum && (st = check_dense(d_sum, sum->dtype, 3, sum->shape, 16)) != KDA_OK) return st;
    if ((st = check_dense(dx, d_out->dtype, 3, sum->shape, 16)) != KDA_OK) return st;
    if ((st = check_dense(dresidual, sum->dtype, 3, sum->shape, 16)) != KDA_OK) return st;
    if ((st = check_dweight(dweight, weight, p)) != KDA_OK) return st;
    const kda_tensor_t* ins[] = {sum, weight, d_out, d_sum};
    const kda_tensor_t* outs[] = {dx, dresidual, dweight};
    if (any_overlap(outs, 3, ins, 4)) return KDA_ERR_LAYOUT;
    p.type = type_code(d_out->dtype);
    p.wide = sum->dtype == KDA_F32;
    p.scale = scale;
    p.dy = d_out->data;
    p.dh = data_of(d_sum);
    p.dx = dx->data;
    p.dz = dresidual->data;
    return with_workspace(p, workspace, workspace_size, stream, kda::launch_add_norm_bwd);
}

}  // extern "C"
