// C-ABI front end of the selective state space scan (kda_ssm_fwd, kda_ssm_bwd, kda_ssm_decode):
// argument checks and launch.  As in the rest of the library every check runs on the host before
// any HIP call, and the host never reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kda_check.h"
#include "kda_ssm.h"

namespace {

using namespace kda::check;
using kda::Rows;

constexpr int64_t kMaxRowStride = int64_t(1) << 23;   // a chunk's byte offsets stay below 2^31
constexpr int64_t kMaxRowsStride = int64_t(1) << 40;

// Rows [B, T, H, D] (or [N, H, D] with ndim 3) of bf16, D 64 or 128: channels contiguous, data
// 16-byte aligned, strides non-negative multiples of 8, tokens at least a row apart.  Strides of
// dimensions of size 1 do not matter.
kda_status_t check_rows(const kda_tensor_t* t, int ndim, Rows* out) {
    if (!t) return KDA_ERR_NULL;
    if (t->dtype != KDA_BF16) return KDA_ERR_DTYPE;
    if (t->ndim != ndim || !sizes_ok(t)) return KDA_ERR_SHAPE;
    const int64_t D = t->shape[ndim - 1];
    if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
    *out = Rows{static_cast<const uint16_t*>(t->data), 0, D, 0};
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] == 0) return KDA_OK;
    if (!t->data) return KDA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0 || t->stride[ndim - 1] != 1) return KDA_ERR_LAYOUT;
    for (int i = 0; i < ndim - 1; ++i) {
        if (t->shape[i] == 1) continue;
        if (t->stride[i] < 0 || t->stride[i] % 8 != 0 || t->stride[i] > kMaxRowsStride) return KDA_ERR_LAYOUT;
        if (i == ndim - 2) out->sh = t->stride[i];
        else if (i == 0) out->sb = t->stride[i];
        else out->st = t->stride[i];
    }
    if (ndim == 4 && (out->st < D || out->st > kMaxRowStride)) return KDA_ERR_LAYOUT;
    return KDA_OK;
}

// dt [B, T, H] or [N, H], bf16 or fp32: heads contiguous, other strides any that are not negative.
kda_status_t check_dt(const kda_tensor_t* t, int ndim, int64_t* sb, int64_t* st) {
    if (!t) return KDA_ERR_NULL;
    if (t->dtype != KDA_BF16 && t->dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (t->ndim != ndim || !sizes_ok(t)) return KDA_ERR_SHAPE;
    *sb = *st = 0;
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] == 0) return KDA_OK;
    if (!t->data) return KDA_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(t->data) % elem_size(t->dtype) != 0) return KDA_ERR_LAYOUT;
    if (t->shape[ndim - 1] != 1 && t->stride[ndim - 1] != 1) return KDA_ERR_LAYOUT;
    for (int i = 0; i < ndim - 1; ++i) {
        if (t->shape[i] == 1) continue;
        if (t->stride[i] < 0 || t->stride[i] > kMaxRowsStride) return KDA_ERR_LAYOUT;
        (i == 0 ? *sb : *st) = t->stride[i];
    }
    return KDA_OK;
}

kda_status_t check_f32(const kda_tensor_t* t, int ndim, const int64_t* shape, size_t align) {
    const kda_status_t st = check_tensor(t, ndim, KDA_F32, KDA_F32, align);
    if (st != KDA_OK) return st;
    return same_shape(t, shape, ndim) ? KDA_OK : KDA_ERR_SHAPE;
}
kda_status_t check_bf16(const kda_tensor_t* t, const kda_tensor_t* like) {
    const kda_status_t st = check_tensor(t, like->ndim, KDA_BF16, KDA_BF16, 16);
    if (st != KDA_OK) return st;
    return same_shape(t, like->shape, like->ndim) ? KDA_OK : KDA_ERR_SHAPE;
}
const float* floats(const kda_tensor_t* t) { return t ? static_cast<const float*>(t->data) : nullptr; }
float* out_floats(const kda_tensor_t* t) { return t ? static_cast<float*>(t->data) : nullptr; }

struct Sizes {
    int64_t B, T, H, P, G, S, N;
};

// What every call shares: shapes of x, B and C, dt and the heads' numbers.
kda_status_t check_shapes(const kda_tensor_t* x, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* Bm,
                          const kda_tensor_t* Cm, const kda_tensor_t* D, const kda_tensor_t* bias, int lead, Sizes& z) {
    kda_status_t st;
    z = Sizes{x->shape[0], lead == 2 ? x->shape[1] : 1, x->shape[lead], x->shape[lead + 1], Bm->shape[lead],
              Bm->shape[lead + 1], x->shape[0]};
    if (!same_shape(Cm, Bm->shape, lead + 2)) return KDA_ERR_SHAPE;
    for (int i = 0; i < lead; ++i)
        if (Bm->shape[i] != x->shape[i]) return KDA_ERR_SHAPE;
    if (!same_shape(dt, x->shape, lead + 1)) return KDA_ERR_SHAPE;
    if (z.H <= 0 || z.G <= 0) return KDA_ERR_SHAPE;
    if (z.H % z.G != 0 || z.H > (int64_t(1) << 16)) return KDA_ERR_UNSUPPORTED;
    if ((st = check_f32(A, 1, &z.H, 4)) != KDA_OK) return st;
    for (const kda_tensor_t* t : {D, bias})
        if (t && (st = check_f32(t, 1, &z.H, 4)) != KDA_OK) return st;
    return KDA_OK;
}
kda_status_t check_state(const kda_tensor_t* t, int64_t n, const Sizes& z) {
    const int64_t s[4] = {n, z.H, z.S, z.P};
    return check_f32(t, 4, s, 16);
}

// Chunks of a segment and segments of a row.  Walks of whole sequences where they fill the compute units (one
// work-group each), else segments for that: of four chunks at least, since the walk that forms what they add reads
// their inputs again, or of two where half the units suffice (then a work-group takes half the columns).  They are
// chained one after the other: at most 4 sqrt(chunks).  S = 128, heads of 64: T = 1024 on 8 heads in 8 segments
// 33 us, in 4 45, in one 88; T = 16384 in 64 72 us, in 128 92; T = 2048 on 64 heads in 8 59 us, in 4 83, in 16 63.  Below 8
// chunks one walk is as fast.  The backward walks both ways at once: half as many segments each.
// Packed sequences are cut the same way from their own starts, as if they were one.
constexpr int64_t kUnits = 256;   // compute units: the workspace's size follows from the shapes alone
struct Segments {
    int64_t segc, nseg, slots;
};
Segments segments(int64_t tokens_per_row, int64_t N, bool packed, int64_t units) {
    const int64_t nc = (tokens_per_row + 63) / 64, walks = (packed ? 1 : N) * units;
    int64_t nseg = 1, most = 1;
    if (walks > 0 && nc >= 8) {
        while (most * most < 16 * nc) ++most;
        nseg = std::max<int64_t>({1, std::min(kUnits / walks, nc / 4), std::min(kUnits / 2 / walks, nc / 2)});
        nseg = std::min(nseg, most);
    }
    Segments s;
    s.segc = std::max<int64_t>(1, (nc + nseg - 1) / nseg);
    s.nseg = std::max<int64_t>(1, (nc + s.segc - 1) / s.segc);
    s.slots = packed ? tokens_per_row / (64 * s.segc) + N : N * s.nseg;
    return s;
}
// Work-groups that share a group's heads in a walk.
int64_t walk_units(int64_t H, int64_t G, int64_t P) { return G * ((H / G * P + kda::SSM_COLS - 1) / kda::SSM_COLS); }

// A workspace's parts, in bytes from its start.
struct Layout {
    int64_t seg, decay, dseg, ddecay, St, dSt, part, dB, dC, total, sets, slots;
    Segments s;
};
Layout layout(int64_t B, int64_t T, int64_t N, bool packed, int64_t H, int64_t G, int64_t P, int64_t S, bool bwd) {
    Layout L{};
    const int64_t state = S * P * 4;
    L.s = segments(T, N, packed, (bwd ? 2 : 1) * walk_units(H, G, P));
    L.slots = T == 0 ? 0 : packed ? (T + 63) / 64 + N : B * ((T + 63) / 64);
    const bool cut = packed ? (T + 63) / 64 > L.s.segc : L.s.nseg > 1;
    const int64_t segs = cut ? L.s.slots * H : 0;
    L.seg = up256(L.slots * H * kda::SSM_REC);
    L.decay = L.seg + segs * state;
    L.total = up256(L.decay + segs * 4);
    if (!bwd) return L;
    L.dseg = L.total;
    L.ddecay = L.dseg + segs * state;
    L.St = up256(L.ddecay + segs * 4);
    L.dSt = L.St + L.slots * H * state;
    L.part = L.dSt + L.slots * H * state;
    L.sets = 1;
    L.dB = L.dC = up256(L.part + L.slots * H * 12);
    L.total = L.dB;
    // Sets of a group's heads, so that chunks and groups fill the compute units, one work-group each: more sets only add sums to
    // join.  Heads of 64, S = 128, 64 of them: 512 tokens in 32 sets 90 us, in 64 102; 2048 tokens in 8 148 us, in 16 161;
    // 2 x 8192 in one 848 us, in two 860.
    const int64_t R = H / G, work = std::max<int64_t>(1, L.slots * G);
    while (L.sets * 2 <= R && work * L.sets < kUnits) L.sets *= 2;
    if (L.sets > 1) {
        const int64_t bytes = L.sets * L.slots * 64 * G * S * 4;
        L.dC = L.dB + bytes;
        L.total = L.dC + bytes;
    }
    return L;
}

// Bytes for `tokens` in N sequences, packed or (where they divide evenly) in N rows.
int64_t any_layout(int64_t tokens, int64_t N, int64_t H, int64_t G, int64_t P, int64_t S, bool bwd) {
    if (tokens < 0 || N < 0 || H < 1 || G < 1 || H % G != 0 || (P != 64 && P != 128) || (S != 64 && S != 128)) return -1;
    int64_t most = layout(1, tokens, N, true, H, G, P, S, bwd).total;
    if (N > 0 && tokens % N == 0) most = std::max(most, layout(N, tokens / N, N, false, H, G, P, S, bwd).total);
    return most;
}

// The checks and parameters that the forward and the backward share.
kda_status_t prepare(const kda_tensor_t* x, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* Bm,
                     const kda_tensor_t* Cm, const kda_tensor_t* D, const kda_tensor_t* bias, int32_t softplus,
                     const kda_tensor_t* cu, bool bwd, kda::SsmParams& p, Sizes& z, Layout& L) {
    kda_status_t st;
    p = kda::SsmParams{};
    if ((st = check_rows(x, 4, &p.x)) != KDA_OK) return st;
    if ((st = check_dt(dt, 3, &p.dtb, &p.dtt)) != KDA_OK) return st;
    if ((st = check_rows(Bm, 4, &p.B)) != KDA_OK) return st;
    if ((st = check_rows(Cm, 4, &p.C)) != KDA_OK) return st;
    if ((st = check_shapes(x, dt, A, Bm, Cm, D, bias, 2, z)) != KDA_OK) return st;
    if (cu) {
        if ((st = check_tensor(cu, 1, KDA_I32, KDA_I32, 4)) != KDA_OK) return st;
        if (z.B != 1) return KDA_ERR_UNSUPPORTED;
        if (cu->shape[0] < 1) return KDA_ERR_SHAPE;
        z.N = cu->shape[0] - 1;
    }
    if (softplus != 0 && softplus != 1) return KDA_ERR_VALUE;
    if (z.N > (int64_t(1) << 24) || z.B * z.T > kMaxTokens) return KDA_ERR_UNSUPPORTED;
    L = layout(z.B, z.T, z.N, cu != nullptr, z.H, z.G, z.P, z.S, bwd);
    // grids of at most 2^22 work-groups (of 768 threads at most: fewer than 2^32), segments rounded up to a multiple of 8;
    // the gradients' numbers take 1024 threads for 16 heads of a chunk
    if (L.slots * z.H > kMaxBlocks || 2 * (L.s.slots + 8) * walk_units(z.H, z.G, 2 * z.P) > kMaxBlocks ||
        2 * z.N * z.H * (z.S * z.P / 1024) > kMaxBlocks || L.slots * z.G * L.sets > kMaxBlocks ||
        (bwd && L.slots * ((z.H + 15) / 16) >= kMaxBlocks))
        return KDA_ERR_UNSUPPORTED;
    p.dt = dt->data;
    p.dt_f32 = dt->dtype == KDA_F32 ? 1 : 0;
    p.A = floats(A);
    p.D = floats(D);
    p.bias = floats(bias);
    p.cu = cu ? static_cast<const int32_t*>(cu->data) : nullptr;
    p.T = z.T;
    p.nslots = z.N > 0 ? L.slots : 0;
    p.segslots = z.N > 0 ? L.s.slots : 0;
    p.N = static_cast<int32_t>(z.N);
    p.H = static_cast<int32_t>(z.H);
    p.G = static_cast<int32_t>(z.G);
    p.P = static_cast<int32_t>(z.P);
    p.S = static_cast<int32_t>(z.S);
    p.nc = static_cast<int32_t>((z.T + 63) / 64);
    p.segc = static_cast<int32_t>(L.s.segc);
    p.nseg = static_cast<int32_t>(L.s.nseg);
    // half as many columns a work-group where a compute unit has no second one to take either way
    p.cols = z.H / z.G * z.P <= 128 || (bwd ? 4 : 2) * p.segslots * walk_units(z.H, z.G, z.P) <= kUnits ? kda::SSM_COLS / 2 : kda::SSM_COLS;
    p.softplus = softplus;
    p.sets = static_cast<int32_t>(L.sets);
    return KDA_OK;
}

}  // namespace

extern "C" {

int64_t kda_ssm_fwd_workspace_size(int64_t total_tokens, int64_t num_sequences, int64_t num_heads, int64_t num_groups,
                                   int64_t head_dim, int64_t state_dim) {
    return any_layout(total_tokens, num_sequences, num_heads, num_groups, head_dim, state_dim, false);
}

int64_t kda_ssm_bwd_workspace_size(int64_t total_tokens, int64_t num_sequences, int64_t num_heads, int64_t num_groups,
                                   int64_t head_dim, int64_t state_dim) {
    return any_layout(total_tokens, num_sequences, num_heads, num_groups, head_dim, state_dim, true);
}

kda_status_t kda_ssm_fwd(const kda_tensor_t* x, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* B,
                         const kda_tensor_t* C, const kda_tensor_t* D, const kda_tensor_t* dt_bias, int32_t softplus,
                         const kda_tensor_t* cu_seqlens, const kda_tensor_t* initial_state, const kda_tensor_t* out,
                         const kda_tensor_t* final_state, void* workspace, int64_t workspace_size, void* stream) {
    kda::SsmParams p;
    Sizes z;
    Layout L;
    kda_status_t st = prepare(x, dt, A, B, C, D, dt_bias, softplus, cu_seqlens, false, p, z, L);
    if (st != KDA_OK) return st;
    if ((st = check_bf16(out, x)) != KDA_OK) return st;
    if (initial_state && (st = check_state(initial_state, z.N, z)) != KDA_OK) return st;
    if (final_state && (st = check_state(final_state, z.N, z)) != KDA_OK) return st;
    const kda_tensor_t* ins[] = {x, dt, A, B, C, D, dt_bias, cu_seqlens};
    const kda_tensor_t* outs[] = {out, final_state};
    if (any_overlap(outs, 2, ins, 8) || overlaps(out, initial_state)) return KDA_ERR_LAYOUT;
    if (initial_state && final_state && partly_overlap(initial_state->data, final_state->data, span_of(final_state).bytes))
        return KDA_ERR_LAYOUT;
    if (workspace && (workspace_size < L.total || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)) return KDA_ERR_WORKSPACE;
    p.h0 = floats(initial_state);
    p.y = static_cast<uint16_t*>(out->data);
    p.hT = out_floats(final_state);
    if (z.N == 0 || (z.T == 0 && !final_state)) return KDA_OK;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    void* ws = workspace;
    if (!ws && L.total > 0 && hipMallocAsync(&ws, (size_t)L.total, hs) != hipSuccess) return KDA_ERR_HIP;
    if (char* base = static_cast<char*>(ws)) {
        p.rec = base;
        p.seg = reinterpret_cast<float*>(base + L.seg);
        p.decay = reinterpret_cast<float*>(base + L.decay);
    }
    hipError_t e = kda::launch_ssm_fwd(p, hs);
    if (!workspace && ws && hipFreeAsync(ws, hs) != hipSuccess && e == hipSuccess) e = hipErrorUnknown;
    return finish(e, hs);
}

kda_status_t kda_ssm_bwd(const kda_tensor_t* x, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* B,
                         const kda_tensor_t* C, const kda_tensor_t* D, const kda_tensor_t* dt_bias, int32_t softplus,
                         const kda_tensor_t* cu_seqlens, const kda_tensor_t* initial_state, const kda_tensor_t* d_out,
                         const kda_tensor_t* d_final_state, const kda_tensor_t* dx, const kda_tensor_t* ddt,
                         const kda_tensor_t* dA, const kda_tensor_t* dB, const kda_tensor_t* dC, const kda_tensor_t* dD,
                         const kda_tensor_t* ddt_bias, const kda_tensor_t* d_initial_state, void* workspace,
                         int64_t workspace_size, void* stream) {
    kda::SsmParams p;
    Sizes z;
    Layout L;
    kda_status_t st = prepare(x, dt, A, B, C, D, dt_bias, softplus, cu_seqlens, true, p, z, L);
    if (st != KDA_OK) return st;
    if ((st = check_rows(d_out, 4, &p.dO)) != KDA_OK) return st;
    if (!same_shape(d_out, x->shape, 4)) return KDA_ERR_SHAPE;
    if ((st = check_bf16(dx, x)) != KDA_OK) return st;
    if ((st = check_bf16(dB, B)) != KDA_OK) return st;
    if ((st = check_bf16(dC, B)) != KDA_OK) return st;
    if ((st = check_f32(ddt, 3, x->shape, 4)) != KDA_OK) return st;
    if ((st = check_f32(dA, 1, &z.H, 4)) != KDA_OK) return st;
    if ((dD && !D) || (ddt_bias && !dt_bias)) return KDA_ERR_NULL;
    for (const kda_tensor_t* t : {dD, ddt_bias})
        if (t && (st = check_f32(t, 1, &z.H, 4)) != KDA_OK) return st;
    for (const kda_tensor_t* t : {initial_state, d_final_state, d_initial_state})
        if (t && (st = check_state(t, z.N, z)) != KDA_OK) return st;
    const kda_tensor_t* ins[] = {x, dt, A, B, C, D, dt_bias, cu_seqlens, initial_state, d_out, d_final_state};
    const kda_tensor_t* outs[] = {dx, ddt, dA, dB, dC, dD, ddt_bias, d_initial_state};
    if (any_overlap(outs, 8, ins, 11)) return KDA_ERR_LAYOUT;
    if (workspace && (workspace_size < L.total || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)) return KDA_ERR_WORKSPACE;
    p.h0 = floats(initial_state);
    p.dhT = floats(d_final_state);
    p.dh0 = out_floats(d_initial_state);
    p.dx = static_cast<uint16_t*>(dx->data);
    p.dB = static_cast<uint16_t*>(dB->data);
    p.dC = static_cast<uint16_t*>(dC->data);
    p.ddt = out_floats(ddt);
    p.dA = out_floats(dA);
    p.dD = out_floats(dD);
    p.dbias = out_floats(ddt_bias);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    void* ws = workspace;
    if (!ws && L.total > 0 && hipMallocAsync(&ws, (size_t)L.total, hs) != hipSuccess) return KDA_ERR_HIP;
    if (char* base = static_cast<char*>(ws)) {
        auto part = [&](int64_t at) { return reinterpret_cast<float*>(base + at); };
        p.rec = base;
        p.seg = part(L.seg);
        p.decay = part(L.decay);
        p.dseg = part(L.dseg);
        p.ddecay = part(L.ddecay);
        p.St = part(L.St);
        p.dSt = part(L.dSt);
        p.part = part(L.part);
        if (L.sets > 1) {
            p.dBp = part(L.dB);
            p.dCp = part(L.dC);
        }
    }
    hipError_t e = kda::launch_ssm_bwd(p, hs);
    if (!workspace && ws && hipFreeAsync(ws, hs) != hipSuccess && e == hipSuccess) e = hipErrorUnknown;
    return finish(e, hs);
}

kda_status_t kda_ssm_decode(const kda_tensor_t* x, const kda_tensor_t* dt, const kda_tensor_t* A, const kda_tensor_t* B,
                            const kda_tensor_t* C, const kda_tensor_t* D, const kda_tensor_t* dt_bias, int32_t softplus,
                            const kda_tensor_t* state_in, const kda_tensor_t* state_out, const kda_tensor_t* state_indices,
                            const kda_tensor_t* out, void* stream) {
    kda_status_t st;
    kda::SsmDecodeParams p{};
    Sizes z;
    int64_t unused;
    if ((st = check_rows(x, 3, &p.x)) != KDA_OK) return st;
    if ((st = check_dt(dt, 2, &p.dtb, &unused)) != KDA_OK) return st;
    if ((st = check_rows(B, 3, &p.B)) != KDA_OK) return st;
    if ((st = check_rows(C, 3, &p.C)) != KDA_OK) return st;
    if ((st = check_shapes(x, dt, A, B, C, D, dt_bias, 1, z)) != KDA_OK) return st;
    if (softplus != 0 && softplus != 1) return KDA_ERR_VALUE;
    if ((st = check_bf16(out, x)) != KDA_OK) return st;
    if (state_indices) {
        if ((st = check_tensor(state_indices, 1, KDA_I32, KDA_I32, 4)) != KDA_OK) return st;
        if (state_indices->shape[0] != z.N) return KDA_ERR_SHAPE;
    }
    if (!state_out) return KDA_ERR_NULL;
    const int64_t slots = state_indices && state_out->ndim == 4 ? state_out->shape[0] : z.N;
    if ((st = check_state(state_out, slots, z)) != KDA_OK) return st;
    if (state_in && (st = check_state(state_in, slots, z)) != KDA_OK) return st;
    if (z.N > (int64_t(1) << 24) || slots > kMaxTokens || z.N * z.H * 4 > kMaxBlocks) return KDA_ERR_UNSUPPORTED;
    const kda_tensor_t* ins[] = {x, dt, A, B, C, D, dt_bias, state_indices};
    const kda_tensor_t* outs[] = {out, state_out};
    if (any_overlap(outs, 2, ins, 8) || overlaps(out, state_in)) return KDA_ERR_LAYOUT;
    if (state_in && partly_overlap(state_in->data, state_out->data, span_of(state_out).bytes)) return KDA_ERR_LAYOUT;
    p.dt = dt->data;
    p.dt_f32 = dt->dtype == KDA_F32 ? 1 : 0;
    p.A = floats(A);
    p.D = floats(D);
    p.bias = floats(dt_bias);
    p.idx = state_indices ? static_cast<const int32_t*>(state_indices->data) : nullptr;
    p.s_in = floats(state_in);
    p.s_out = out_floats(state_out);
    p.y = static_cast<uint16_t*>(out->data);
    p.N = static_cast<int32_t>(z.N);
    p.H = static_cast<int32_t>(z.H);
    p.G = static_cast<int32_t>(z.G);
    p.P = static_cast<int32_t>(z.P);
    p.S = static_cast<int32_t>(z.S);
    p.slots = static_cast<int32_t>(slots);
    p.softplus = softplus;
    if (z.N == 0 || slots == 0) return KDA_OK;
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return finish(kda::launch_ssm_decode(p, device_cus(), hs), hs);
}

}  // extern "C"
