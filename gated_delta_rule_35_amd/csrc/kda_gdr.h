// Internal interface of the gated delta rule with one decay per token and value
// head (kda_gdr_fwd, kda_gdr_bwd, kda_gdr_decode) and of the per-head q/k norm.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// A bf16 tensor [B, T, H, 128] whose last dimension is contiguous: strides in elements.
struct Rows {
    const uint16_t* p;
    int64_t sb, st, sh;
};

struct GdrParams {
    Rows q, k, v, dO;      // dO: gradient of the output (backward only)
    const float* g;        // [B, T, Hv] log-decay
    const void* beta;      // [B, T, Hv] bf16 bits or fp32
    const int32_t* cu;     // [N + 1] offsets of packed sequences (B = 1), or nullptr
    const float* h0;       // [N, Hv, 128, 128] or nullptr
    uint16_t* o;           // [B, T, Hv, 128] bf16 bits
    float* hT;             // [N, Hv, 128, 128] or nullptr
    char* rec;             // [nslots][Hv] chunk records of the prep kernel
    int64_t T;             // tokens per row
    int64_t nslots;        // chunk slots: N * nc, or with cu ceil(T / 64) + N
    int32_t N, Hq, Hv, nc; // nc = ceil(T / 64)
    int32_t beta_f32;
    float scale;
    // backward
    const float* dhT;      // [N, Hv, 128, 128] or nullptr
    float* dh0;            // [N, Hv, 128, 128] or nullptr
    uint16_t *dq, *dk, *dv;// [B, T, H, 128] bf16 bits
    float *dg, *dbeta;     // [B, T, Hv]
    float* S;              // [nslots][Hv][128][128] state entering each chunk
    float* dS;             // [nslots][Hv][128][128] gradient of the state leaving each chunk
    float* u;              // [nslots][Hv][64][128] corrected values of each chunk
    float* dx;             // [nslots][Hv][64][128] gradient of the right-hand side beta (v - e^G K S)
};

// Chunk records of the prep kernel (see kda_gdr_prep.hip): triangular operands as lists
// of six 1 KB fragments per part, and rows of 64 per-token numbers (fp32).
constexpr int GDR_FRAG = 1024;
// Place of lane l's 16 bytes in a fragment that is also read transposed: the sixteen lanes of
// a group four apart from the group's before, else such a read meets each bank four times.
__host__ __device__ constexpr int frag_piece(int l) { return 16 * (l ^ ((l >> 4) << 2)); }
constexpr int GDR_TRI = 6 * GDR_FRAG;              // one part of a triangular operand
// T in three bf16 parts (the forward's with its columns times beta) and the per-token rows; the
// backward also A (scale included) in three parts.
constexpr int GDR_T = 0, GDR_SC = 3 * GDR_TRI, FWD_REC = GDR_SC + 2048;
constexpr int GDR_A = GDR_SC + 1024, GDR_REC = GDR_A + 3 * GDR_TRI;

hipError_t launch_gdr_prep(const GdrParams& p, bool bwd, hipStream_t stream);
hipError_t launch_gdr_grads(const GdrParams& p, int cus, hipStream_t stream);
// cus: compute units of the current device.
hipError_t launch_gdr_fwd(const GdrParams& p, int cus, hipStream_t stream);
hipError_t launch_gdr_bwd(const GdrParams& p, int cus, hipStream_t stream);

struct GdrDecodeParams {
    Rows q, k, v;          // [N, H, 128]: sb is the stride of N, st is unused
    const float* g;        // [N, Hv]
    const void* beta;      // [N, Hv]
    const int32_t* idx;    // [N] state slots, or nullptr (slot n)
    const float* s_in;     // [slots, Hv, 128, 128] or nullptr (zero)
    float* s_out;          // [slots, Hv, 128, 128]; may equal s_in
    uint16_t* o;           // [N, Hv, 128]
    int32_t N, Hq, Hv, slots;
    int32_t beta_f32;
    float scale;
};
hipError_t launch_gdr_decode(const GdrDecodeParams& p, int cus, hipStream_t stream);

// One tensor of the per-head norm: rows [B, T, H, 128].
struct NormSide {
    const void* x;         // input, dtype NormParams::xt
    int64_t sb, st, sh;    // its strides in elements
    const void* dy;        // backward: gradient of the output, contiguous, dtype NormParams::dt
    void* y;               // forward: output bf16; backward: gradient of x, x's dtype; contiguous
    const float* w;        // [128] or nullptr
    float* dw;             // [128] or nullptr
    int32_t H;
    int64_t rows;          // B * T * H
};
struct NormParams {
    NormSide s[2];         // queries, keys
    const float *cos, *sin;// [P, half] or nullptr
    const int32_t* pos;    // [B, T] or nullptr (the token's index in its row)
    float* part;           // backward with weights: [blocks][128] partial sums
    int64_t T, P;
    int32_t half, interleaved, rms;
    int32_t xt, dt;        // 0 bf16, 1 fp16, 2 fp32
    float eps;
    int32_t blocks[2];     // work-groups of each side
};
hipError_t launch_qk_norm(const NormParams& p, hipStream_t stream);
hipError_t launch_qk_norm_bwd(const NormParams& p, hipStream_t stream);
constexpr int NORM_ROWS = 16;            // rows that a work-group takes at a time
// Most work-groups when weights have gradients, about: more of them leave more sums to add.
// 512, 1024 and 2048: 10.5, 11.0 and 14.5 us at 1024 tokens of 16 + 16 heads, 107, 105 and
// 103 us at 8192 of 64 + 16, 317, 305 and 324 us at 16,384 of 64 + 64.
constexpr int NORM_DW_BLOCKS = 1024;

}  // namespace kda
