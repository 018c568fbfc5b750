// C-ABI front end of the gated delta rule with one decay per head (kda_gdr_fwd,
// kda_gdr_bwd, kda_gdr_decode) and of the per-head q/k norm (kda_qk_norm,
// kda_qk_norm_bwd): argument checks and launch.  As in the rest of the library every
// check runs on the host before any HIP call, and the host never reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kda_check.h"
#include "kda_gdr.h"

namespace {

using namespace kda::check;
using kda::Rows;

constexpr int64_t kMaxRowStride = int64_t(1) << 23;   // a chunk's byte offsets stay below 2^31

// Rows of 128 channels [B, T, H, 128], or [N, H, 128] with ndim 3: the channels are
// contiguous and rows start on multiples of 8 elements (16 bytes of bf16); tokens lie
// at least a row apart.  Strides of dimensions of size 1 do not matter.
kda_status_t check_rows(const kda_tensor_t* t, int ndim, bool any_type, Rows* out) {
    if (!t) return KDA_ERR_NULL;
    if (t->dtype != KDA_BF16 && !(any_type && (t->dtype == KDA_F16 || t->dtype == KDA_F32))) return KDA_ERR_DTYPE;
    if (t->ndim != ndim || !sizes_ok(t)) return KDA_ERR_SHAPE;
    if (t->shape[ndim - 1] != kHeadDim) return KDA_ERR_UNSUPPORTED;
    *out = Rows{static_cast<const uint16_t*>(t->data), 0, kHeadDim, 0};
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] == 0) return KDA_OK;
    if (!t->data) return KDA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0 || t->stride[ndim - 1] != 1) return KDA_ERR_LAYOUT;
    for (int i = 0; i < ndim - 1; ++i) {
        if (t->shape[i] == 1) continue;
        if (t->stride[i] < 0 || t->stride[i] % 8 != 0 || t->stride[i] > (int64_t(1) << 40)) return KDA_ERR_LAYOUT;
        if (i == ndim - 2) out->sh = t->stride[i];
        else if (i == 0) out->sb = t->stride[i];
        else out->st = t->stride[i];
    }
    if (ndim == 4 && (out->st < kHeadDim || out->st > kMaxRowStride)) return KDA_ERR_LAYOUT;
    return KDA_OK;
}

struct Sizes {
    int64_t B, T, Hq, Hv, N, nc, nslots;
};

// The checks that the forward and the backward share: inputs, shapes, grids.
kda_status_t prepare(const kda_tensor_t* q, const kda_tensor_t* k, const kda_tensor_t* v, const kda_tensor_t* g,
                     const kda_tensor_t* beta, float scale, const kda_tensor_t* cu, kda::GdrParams& p, Sizes& z) {
    kda_status_t st;
    p = kda::GdrParams{};
    if ((st = check_rows(q, 4, false, &p.q)) != KDA_OK) return st;
    if ((st = check_rows(k, 4, false, &p.k)) != KDA_OK) return st;
    if ((st = check_rows(v, 4, false, &p.v)) != KDA_OK) return st;
    if ((st = check_tensor(g, 3, KDA_F32, KDA_F32, 4)) != KDA_OK) return st;
    if (!beta) return KDA_ERR_NULL;
    if ((st = check_tensor(beta, 3, KDA_BF16, KDA_F32, elem_size(beta->dtype))) != KDA_OK) return st;
    if (cu && (st = check_tensor(cu, 1, KDA_I32, KDA_I32, 4)) != KDA_OK) return st;
    z = Sizes{q->shape[0], q->shape[1], q->shape[2], v->shape[2], q->shape[0], 0, 0};
    if (!same_shape(k, q->shape, 4)) return KDA_ERR_SHAPE;
    if (v->shape[0] != z.B || v->shape[1] != z.T) return KDA_ERR_SHAPE;
    const int64_t bs[3] = {z.B, z.T, z.Hv};
    if (!same_shape(g, bs, 3) || !same_shape(beta, bs, 3)) return KDA_ERR_SHAPE;
    if (z.Hq <= 0 || z.Hv <= 0) return KDA_ERR_SHAPE;
    if (z.Hv % z.Hq != 0) return KDA_ERR_UNSUPPORTED;
    if (cu) {
        if (z.B != 1) return KDA_ERR_UNSUPPORTED;
        if (cu->shape[0] < 1) return KDA_ERR_SHAPE;
        z.N = cu->shape[0] - 1;
    }
    if (!std::isfinite(scale) || !(scale > 0.f)) return KDA_ERR_VALUE;
    if (z.Hv > (int64_t(1) << 16) || z.N > (int64_t(1) << 24) || z.B * z.T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    z.nc = (z.T + 63) / 64;
    z.nslots = cu ? z.nc + z.N : z.B * z.nc;
    if (z.T == 0) z.nslots = 0;
    if (z.nslots * z.Hv > kMaxBlocks || z.N * z.Hv * 2 > kMaxBlocks) return KDA_ERR_UNSUPPORTED;
    p.g = static_cast<const float*>(g->data);
    p.beta = beta->data;
    p.beta_f32 = beta->dtype == KDA_F32 ? 1 : 0;
    p.cu = cu ? static_cast<const int32_t*>(cu->data) : nullptr;
    p.T = z.T;
    p.N = static_cast<int32_t>(z.N);
    p.Hq = static_cast<int32_t>(z.Hq);
    p.Hv = static_cast<int32_t>(z.Hv);
    p.nc = static_cast<int32_t>(z.nc);
    p.nslots = z.nslots;
    p.scale = scale;
    return KDA_OK;
}

kda_status_t check_state(const kda_tensor_t* t, int64_t n, int64_t Hv, bool needed) {
    if (!t) return needed ? KDA_ERR_NULL : KDA_OK;
    const kda_status_t st = check_tensor(t, 4, KDA_F32, KDA_F32, 16);
    if (st != KDA_OK) return st;
    const int64_t ss[4] = {n, Hv, kHeadDim, kHeadDim};
    return same_shape(t, ss, 4) ? KDA_OK : KDA_ERR_SHAPE;
}
// An output row tensor of `like`'s shape: contiguous bf16.
kda_status_t check_out(const kda_tensor_t* t, const kda_tensor_t* like) {
    const kda_status_t st = check_tensor(t, like ? like->ndim : 4, KDA_BF16, KDA_BF16, 16);
    if (st != KDA_OK) return st;
    return same_shape(t, like->shape, like->ndim) ? KDA_OK : KDA_ERR_SHAPE;
}

// Workspace of a call in units of one (chunk slot, value head): the records, then, for
// the backward, S, dS, u and dx.
int64_t fwd_bytes(int64_t units) { return units * kda::FWD_REC; }
struct BwdLayout {
    int64_t S, dS, u, dx, total;
};
BwdLayout bwd_layout(int64_t units) {
    BwdLayout L{};
    L.S = up256(units * kda::GDR_REC);
    L.dS = L.S + units * kHeadDim * kHeadDim * 4;
    L.u = L.dS + units * kHeadDim * kHeadDim * 4;
    L.dx = L.u + units * 64 * kHeadDim * 4;
    L.total = L.dx + units * 64 * kHeadDim * 4;
    return L;
}
int64_t units_of(int64_t tokens, int64_t N, int64_t Hv) { return tokens > 0 ? ((tokens + 63) / 64 + N) * Hv : 0; }

}  // namespace

extern "C" {

int64_t kda_gdr_fwd_workspace_size(int64_t total_tokens, int64_t num_sequences, int64_t num_value_heads) {
    if (total_tokens < 0 || num_sequences < 0 || num_value_heads < 0) return -1;
    return fwd_bytes(units_of(total_tokens, num_sequences, num_value_heads));
}

int64_t kda_gdr_bwd_workspace_size(int64_t total_tokens, int64_t num_sequences, int64_t num_value_heads) {
    if (total_tokens < 0 || num_sequences < 0 || num_value_heads < 0) return -1;
    return bwd_layout(units_of(total_tokens, num_sequences, num_value_heads)).total;
}

kda_status_t kda_gdr_fwd(const kda_tensor_t* q, const kda_tensor_t* k, const kda_tensor_t* v, const kda_tensor_t* g,
                         const kda_tensor_t* beta, float scale, const kda_tensor_t* cu_seqlens,
                         const kda_tensor_t* initial_state, const kda_tensor_t* out, const kda_tensor_t* final_state,
                         void* workspace, int64_t workspace_size, void* stream) {
    kda::GdrParams p;
    Sizes z;
    kda_status_t st = prepare(q, k, v, g, beta, scale, cu_seqlens, p, z);
    if (st != KDA_OK) return st;
    if ((st = check_out(out, v)) != KDA_OK) return st;
    if ((st = check_state(initial_state, z.N, z.Hv, false)) != KDA_OK) return st;
    if ((st = check_state(final_state, z.N, z.Hv, false)) != KDA_OK) return st;
    const kda_tensor_t* ins[] = {q, k, v, g, beta, cu_seqlens};
    const kda_tensor_t* outs[] = {out, final_state};
    if (any_overlap(outs, 2, ins, 6) || overlaps(out, initial_state)) return KDA_ERR_LAYOUT;
    if (initial_state && final_state &&
        partly_overlap(initial_state->data, final_state->data, z.N * z.Hv * kHeadDim * kHeadDim * 4))
        return KDA_ERR_LAYOUT;
    const int64_t need = fwd_bytes(units_of(z.B * z.T, z.N, z.Hv));
    if (workspace && (workspace_size < need || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
        return KDA_ERR_WORKSPACE;
    p.h0 = initial_state ? static_cast<const float*>(initial_state->data) : nullptr;
    p.o = static_cast<uint16_t*>(out->data);
    p.hT = final_state ? static_cast<float*>(final_state->data) : nullptr;
    if (z.N == 0 || (z.T == 0 && !final_state)) return KDA_OK;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    void* ws = workspace;
    if (!ws && need > 0 && hipMallocAsync(&ws, (size_t)need, hs) != hipSuccess) return KDA_ERR_HIP;
    p.rec = static_cast<char*>(ws);
    hipError_t e = kda::launch_gdr_fwd(p, std::max(device_cus(), 1), hs);
    if (!workspace && ws && hipFreeAsync(ws, hs) != hipSuccess && e == hipSuccess) e = hipErrorUnknown;
    return finish(e, hs);
}

kda_status_t kda_gdr_bwd(const kda_tensor_t* q, const kda_tensor_t* k, const kda_tensor_t* v, const kda_tensor_t* g,
                         const kda_tensor_t* beta, float scale, const kda_tensor_t* cu_seqlens,
                         const kda_tensor_t* initial_state, const kda_tensor_t* d_out,
                         const kda_tensor_t* d_final_state, const kda_tensor_t* dq, const kda_tensor_t* dk,
                         const kda_tensor_t* dv, const kda_tensor_t* dg, const kda_tensor_t* dbeta,
                         const kda_tensor_t* d_initial_state, void* workspace, int64_t workspace_size, void* stream) {
    kda::GdrParams p;
    Sizes z;
    kda_status_t st = prepare(q, k, v, g, beta, scale, cu_seqlens, p, z);
    if (st != KDA_OK) return st;
    if ((st = check_rows(d_out, 4, false, &p.dO)) != KDA_OK) return st;
    if (!same_shape(d_out, v->shape, 4)) return KDA_ERR_SHAPE;
    if ((st = check_out(dq, q)) != KDA_OK) return st;
    if ((st = check_out(dk, q)) != KDA_OK) return st;
    if ((st = check_out(dv, v)) != KDA_OK) return st;
    for (const kda_tensor_t* t : {dg, dbeta}) {
        if ((st = check_tensor(t, 3, KDA_F32, KDA_F32, 4)) != KDA_OK) return st;
        if (!same_shape(t, g->shape, 3)) return KDA_ERR_SHAPE;
    }
    if ((st = check_state(initial_state, z.N, z.Hv, false)) != KDA_OK) return st;
    if ((st = check_state(d_final_state, z.N, z.Hv, false)) != KDA_OK) return st;
    if ((st = check_state(d_initial_state, z.N, z.Hv, false)) != KDA_OK) return st;
    const kda_tensor_t* ins[] = {q, k, v, g, beta, cu_seqlens, initial_state, d_out, d_final_state};
    const kda_tensor_t* outs[] = {dq, dk, dv, dg, dbeta, d_initial_state};
    if (any_overlap(outs, 6, ins, 9)) return KDA_ERR_LAYOUT;
    const int64_t units = units_of(z.B * z.T, z.N, z.Hv);
    const BwdLayout L = bwd_layout(units);
    if (workspace && (workspace_size < L.total || reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
        return KDA_ERR_WORKSPACE;
    p.h0 = initial_state ? static_cast<const float*>(initial_state->data) : nullptr;
    p.dhT = d_final_state ? static_cast<const float*>(d_final_state->data) : nullptr;
    p.dh0 = d_initial_state ? static_cast<float*>(d_initial_state->data) : nullptr;
    p.dq = static_cast<uint16_t*>(dq->data);
    p.dk = static_cast<uint16_t*>(dk->data);
    p.dv = static_cast<uint16_t*>(dv->data);
    p.dg = static_cast<float*>(dg->data);
    p.dbeta = static_cast<float*>(dbeta->data);
    if (z.N == 0 || (z.T == 0 && !d_initial_state)) return KDA_OK;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    void* ws = workspace;
    if (!ws && L.total > 0 && hipMallocAsync(&ws, (size_t)L.total, hs) != hipSuccess) return KDA_ERR_HIP;
    if (char* base = static_cast<char*>(ws)) {
        p.rec = base;
        p.S = reinterpret_cast<float*>(base + L.S);
        p.dS = reinterpret_cast<float*>(base + L.dS);
        p.u = reinterpret_cast<float*>(base + L.u);
        p.dx = reinterpret_cast<float*>(base + L.dx);
    }
    hipError_t e = kda::launch_gdr_bwd(p, std::max(device_cus(), 1), hs);
    if (!workspace && ws && hipFreeAsync(ws, hs) != hipSuccess && e == hipSuccess) e = hipErrorUnknown;
    return finish(e, hs);
}

kda_status_t kda_gdr_decode(const kda_tensor_t* q, const kda_tensor_t* k, const kda_tensor_t* v, const kda_tensor_t* g,
                            const kda_tensor_t* beta, float scale, const kda_tensor_t* state_in,
                            const kda_tensor_t* state_out, const kda_tensor_t* state_indices, const kda_tensor_t* out,
                            void* stream) {
    kda_status_t st;
    kda::GdrDecodeParams p{};
    if ((st = check_rows(q, 3, false, &p.q)) != KDA_OK) return st;
    if ((st = check_rows(k, 3, false, &p.k)) != KDA_OK) return st;
    if ((st = check_rows(v, 3, false, &p.v)) != KDA_OK) return st;
    if ((st = check_tensor(g, 2, KDA_F32, KDA_F32, 4)) != KDA_OK) return st;
    if (!beta) return KDA_ERR_NULL;
    if ((st = check_tensor(beta, 2, KDA_BF16, KDA_F32, elem_size(beta->dtype))) != KDA_OK) return st;
    if (state_indices && (st = check_tensor(state_indices, 1, KDA_I32, KDA_I32, 4)) != KDA_OK) return st;
    const int64_t N = q->shape[0], Hq = q->shape[1], Hv = v->shape[1];
    if (!same_shape(k, q->shape, 3) || v->shape[0] != N) return KDA_ERR_SHAPE;
    const int64_t bs[2] = {N, Hv};
    if (!same_shape(g, bs, 2) || !same_shape(beta, bs, 2)) return KDA_ERR_SHAPE;
    if ((st = check_out(out, v)) != KDA_OK) return st;
    if (Hq <= 0 || Hv <= 0) return KDA_ERR_SHAPE;
    if (Hv % Hq != 0) return KDA_ERR_UNSUPPORTED;
    if (state_indices && state_indices->shape[0] != N) return KDA_ERR_SHAPE;
    if (!state_out) return KDA_ERR_NULL;
    const int64_t slots = state_indices && state_out->ndim == 4 ? state_out->shape[0] : N;
    if ((st = check_state(state_out, slots, Hv, true)) != KDA_OK) return st;
    if ((st = check_state(state_in, slots, Hv, false)) != KDA_OK) return st;
    if (!std::isfinite(scale) || !(scale > 0.f)) return KDA_ERR_VALUE;
    if (Hv > (int64_t(1) << 16) || N > (int64_t(1) << 24) || slots > kMaxTokens || N * Hv * 4 > kMaxBlocks)
        return KDA_ERR_UNSUPPORTED;
    const kda_tensor_t* ins[] = {q, k, v, g, beta, state_indices};
    const kda_tensor_t* outs[] = {out, state_out};
    if (any_overlap(outs, 2, ins, 6) || overlaps(out, state_in)) return KDA_ERR_LAYOUT;
    if (state_in && partly_overlap(state_in->data, state_out->data, slots * Hv * kHeadDim * kHeadDim * 4))
        return KDA_ERR_LAYOUT;
    p.g = static_cast<const float*>(g->data);
    p.beta = beta->data;
    p.beta_f32 = beta->dtype == KDA_F32 ? 1 : 0;
    p.idx = state_indices ? static_cast<const int32_t*>(state_indices->data) : nullptr;
    p.s_in = state_in ? static_cast<const float*>(state_in->data) : nullptr;
    p.s_out = static_cast<float*>(state_out->data);
    p.o = static_cast<uint16_t*>(out->data);
    p.N = static_cast<int32_t>(N);
    p.Hq = static_cast<int32_t>(Hq);
    p.Hv = static_cast<int32_t>(Hv);
    p.slots = static_cast<int32_t>(slots);
    p.scale = scale;
    if (N == 0 || slots == 0) return KDA_OK;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return finish(kda::launch_gdr_decode(p, device_cus(), hs), hs);
}

}  // extern "C"

// ---- per-head norm of queries and keys ----
namespace {

int dtype_code(kda_dtype_t d) { return d == KDA_BF16 ? 0 : d == KDA_F16 ? 1 : 2; }

// The checks that both directions share.
kda_status_t prepare_norm(const kda_tensor_t* const (&x)[2], const kda_tensor_t* const (&w)[2], int32_t mode, float eps,
                          const kda_tensor_t* cos, const kda_tensor_t* sin, const kda_tensor_t* positions,
                          int32_t interleaved, kda::NormParams& p) {
    kda_status_t st;
    p = kda::NormParams{};
    for (int i = 0; i < 2; ++i) {
        Rows r;
        if ((st = check_rows(x[i], 4, true, &r)) != KDA_OK) return st;
        if (x[i]->dtype != x[0]->dtype) return KDA_ERR_DTYPE;
        if (x[i]->shape[0] != x[0]->shape[0] || x[i]->shape[1] != x[0]->shape[1] || x[i]->shape[2] <= 0)
            return KDA_ERR_SHAPE;
        if (x[i]->shape[2] > (int64_t(1) << 16) || x[i]->shape[0] * x[i]->shape[1] > kMaxTokens)
            return KDA_ERR_UNSUPPORTED;
        if (w[i]) {
            if ((st = check_tensor(w[i], 1, KDA_F32, KDA_F32, 4)) != KDA_OK) return st;
            if (w[i]->shape[0] != kHeadDim) return KDA_ERR_SHAPE;
        }
        p.s[i].x = x[i]->data;
        p.s[i].sb = r.sb;
        p.s[i].st = r.st;
        p.s[i].sh = r.sh;
        p.s[i].w = w[i] ? static_cast<const float*>(w[i]->data) : nullptr;
        p.s[i].H = static_cast<int32_t>(x[i]->shape[2]);
        p.s[i].rows = x[i]->shape[0] * x[i]->shape[1] * x[i]->shape[2];
    }
    if (mode != 0 && mode != 1) return KDA_ERR_VALUE;
    if (!std::isfinite(eps) || !(eps > 0.f)) return KDA_ERR_VALUE;
    if (!cos != !sin || (positions && !cos)) return KDA_ERR_NULL;
    const int64_t B = x[0]->shape[0], T = x[0]->shape[1];
    if (B * T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    if (cos) {
        if ((st = check_tensor(cos, 2, KDA_F32, KDA_F32, 16)) != KDA_OK) return st;
        if ((st = check_tensor(sin, 2, KDA_F32, KDA_F32, 16)) != KDA_OK) return st;
        if (!same_shape(sin, cos->shape, 2) || cos->shape[0] < 1) return KDA_ERR_SHAPE;
        if (cos->shape[1] < 8 || cos->shape[1] > kHeadDim / 2 || cos->shape[1] % 8 != 0) return KDA_ERR_UNSUPPORTED;
        p.cos = static_cast<const float*>(cos->data);
        p.sin = static_cast<const float*>(sin->data);
        p.P = cos->shape[0];
        p.half = static_cast<int32_t>(cos->shape[1]);
        if (positions) {
            if ((st = check_tensor(positions, 2, KDA_I32, KDA_I32, 4)) != KDA_OK) return st;
            if (positions->shape[0] != B || positions->shape[1] != T) return KDA_ERR_SHAPE;
            p.pos = static_cast<const int32_t*>(positions->data);
        }
    }
    p.T = T;
    p.interleaved = interleaved ? 1 : 0;
    p.rms = mode == 1;
    p.xt = dtype_code(x[0]->dtype);
    p.eps = eps;
    return KDA_OK;
}

// Work-groups of both sides: one per 16 rows; with weight gradients at most
// NORM_DW_BLOCKS in proportion to the sides' rows (rounded up), which then loop.
kda_status_t norm_blocks(kda::NormParams& p, bool weights) {
    const int64_t total = p.s[0].rows + p.s[1].rows;
    if (total > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i) {
        int64_t b = (p.s[i].rows + kda::NORM_ROWS - 1) / kda::NORM_ROWS;
        if (weights && total > 0) b = std::min(b, (kda::NORM_DW_BLOCKS * p.s[i].rows + total - 1) / total);
        if (b > kMaxBlocks) return KDA_ERR_UNSUPPORTED;
        p.blocks[i] = static_cast<int32_t>(b);
    }
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_qk_norm(const kda_tensor_t* q, const kda_tensor_t* k, const kda_tensor_t* q_weight,
                         const kda_tensor_t* k_weight, int32_t mode, float eps, const kda_tensor_t* cos,
                         const kda_tensor_t* sin, const kda_tensor_t* positions, int32_t interleaved,
                         const kda_tensor_t* q_out, const kda_tensor_t* k_out, void* stream) {
    const kda_tensor_t *const x[2] = {q, k}, *const w[2] = {q_weight, k_weight}, *const y[2] = {q_out, k_out};
    kda::NormParams p;
    kda_status_t st = prepare_norm(x, w, mode, eps, cos, sin, positions, interleaved, p);
    if (st != KDA_OK) return st;
    const kda_tensor_t* ins[] = {q, k, q_weight, k_weight, cos, sin, positions};
    for (int i = 0; i < 2; ++i) {
        if ((st = check_out(y[i], x[i])) != KDA_OK) return st;
        for (const kda_tensor_t* t : ins) {
            // a contiguous bf16 input may be overwritten by its own output
            if (t == x[i] && t->data == y[i]->data && t->dtype == KDA_BF16 && contiguous(t)) continue;
            if (overlaps(y[i], t)) return KDA_ERR_LAYOUT;
        }
        p.s[i].y = y[i]->data;
    }
    if (overlaps(q_out, k_out)) return KDA_ERR_LAYOUT;
    if ((st = norm_blocks(p, false)) != KDA_OK) return st;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return finish(kda::launch_qk_norm(p, hs), hs);
}

int64_t kda_qk_norm_bwd_workspace_size(void) { return ((int64_t)kda::NORM_DW_BLOCKS + 2) * kHeadDim * 4; }

kda_status_t kda_qk_norm_bwd(const kda_tensor_t* q, const kda_tensor_t* k, const kda_tensor_t* d_q_out,
                             const kda_tensor_t* d_k_out, const kda_tensor_t* q_weight, const kda_tensor_t* k_weight,
                             int32_t mode, float eps, const kda_tensor_t* cos, const kda_tensor_t* sin,
                             const kda_tensor_t* positions, int32_t interleaved, const kda_tensor_t* dq,
                             const kda_tensor_t* dk, const kda_tensor_t* d_q_weight, const kda_tensor_t* d_k_weight,
                             void* workspace, int64_t workspace_size, void* stream) {
    const kda_tensor_t *const x[2] = {q, k}, *const w[2] = {q_weight, k_weight}, *const dy[2] = {d_q_out, d_k_out},
                       *const dx[2] = {dq, dk}, *const dw[2] = {d_q_weight, d_k_weight};
    kda::NormParams p;
    kda_status_t st = prepare_norm(x, w, mode, eps, cos, sin, positions, interleaved, p);
    if (st != KDA_OK) return st;
    for (int i = 0; i < 2; ++i) {
        if ((st = check_tensor(dy[i], 4, KDA_BF16, KDA_F32, 16)) != KDA_OK) return st;
        if (dy[i]->dtype != dy[0]->dtype) return KDA_ERR_DTYPE;
        if ((st = check_tensor(dx[i], 4, x[0]->dtype, x[0]->dtype, 16)) != KDA_OK) return st;
        if (!same_shape(dy[i], x[i]->shape, 4) || !same_shape(dx[i], x[i]->shape, 4)) return KDA_ERR_SHAPE;
        if (dw[i]) {
            if (!w[i]) return KDA_ERR_NULL;
            if ((st = check_tensor(dw[i], 1, KDA_F32, KDA_F32, 4)) != KDA_OK) return st;
            if (dw[i]->shape[0] != kHeadDim) return KDA_ERR_SHAPE;
        }
        p.s[i].dy = dy[i]->data;
        p.s[i].y = dx[i]->data;
        p.s[i].dw = dw[i] ? static_cast<float*>(dw[i]->data) : nullptr;
    }
    p.dt = dtype_code(dy[0]->dtype);
    const kda_tensor_t* ins[] = {q, k, d_q_out, d_k_out, q_weight, k_weight, cos, sin, positions};
    const kda_tensor_t* outs[] = {dq, dk, d_q_weight, d_k_weight};
    if (any_overlap(outs, 4, ins, 9)) return KDA_ERR_LAYOUT;
    const bool weights = d_q_weight || d_k_weight;
    if ((st = norm_blocks(p, weights)) != KDA_OK) return st;
    const int64_t need = weights ? kda_qk_norm_bwd_workspace_size() : 0;
    if (weights && workspace && (workspace_size < need || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
        return KDA_ERR_WORKSPACE;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    void* ws = weights ? workspace : nullptr;
    if (weights && !ws && hipMallocAsync(&ws, (size_t)need, hs) != hipSuccess) return KDA_ERR_HIP;
    p.part = static_cast<float*>(ws);
    hipError_t e = kda::launch_qk_norm_bwd(p, hs);
    if (weights && !workspace && hipFreeAsync(ws, hs) != hipSuccess && e == hipSuccess) e = hipErrorUnknown;
    return finish(e, hs);
}

}  // extern "C"
