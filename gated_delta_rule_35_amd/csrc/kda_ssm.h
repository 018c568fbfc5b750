// Internal interface of the selective state space scan (kda_ssm_fwd, kda_ssm_bwd, kda_ssm_decode).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_gdr.h"

namespace kda {

struct SsmParams {
    Rows x, B, C, dO;      // [B, T, H, P], [B, T, G, S] twice, [B, T, H, P] (backward only)
    const void* dt;        // [B, T, H] bf16 bits or fp32, heads contiguous
    int64_t dtb, dtt;      // its strides in elements
    const float *A, *D, *bias;   // [H]; D and bias may be nullptr (zeros)
    const int32_t* cu;     // [N + 1] offsets of packed sequences (B = 1), or nullptr
    const float* h0;       // [N, H, S, P] or nullptr
    uint16_t* y;           // [B, T, H, P] bf16 bits
    float* hT;             // [N, H, S, P] or nullptr
    char* rec;             // [nslots][H] records of per-token numbers
    float* seg;            // [segslots][H][S][P] states of segments: what each adds, then what enters it
    float* decay;          // [segslots][H] a segment's decay
    int64_t T;             // tokens per row
    int64_t nslots;        // chunk slots: N * nc, or with cu ceil(T / 64) + N
    int64_t segslots;      // segment slots: N * nseg, or with cu T / (64 segc) + N
    int32_t N, H, G, P, S, nc;   // nc = ceil(T / 64)
    int32_t segc, nseg;    // chunks of a segment; segments of a row (without cu)
    int32_t cols;          // value columns of a walking work-group: 256, or 128
    int32_t dt_f32, softplus;
    // backward
    const float* dhT;      // [N, H, S, P] or nullptr
    float* dh0;            // [N, H, S, P] or nullptr
    uint16_t *dx, *dB, *dC;
    float *ddt;            // [B, T, H]
    float *dA, *dD, *dbias;// [H]; dD and dbias may be nullptr
    float *dseg, *ddecay;  // seg and decay of the gradients' walk
    float *St, *dSt;       // [nslots][H][P S] states entering each chunk and gradients of those leaving it, as fragments
    float *dBp, *dCp;      // [sets][nslots 64][G][S] sums of dB and dC over each set of heads, or nullptr (one set)
    float* part;           // [nslots][3][H] sums over a chunk: dA, dD, dbias
    int32_t sets;          // sets of heads that a group's gradients are formed in
};

// A record's rows of 64 numbers (fp32), by token of the chunk: the step, e^G, e^{G_last - G}, G in
// units of log 2 as a value and its remainder, e^{G - G_s} with G_s of the token before its block of
// sixteen, e^{G_e - G} with G_e of its block's last token, the step times e^{G_last - G}.
enum { SSM_DT = 0, SSM_EG = 64, SSM_GA = 128, SSM_GH = 192, SSM_GL = 256, SSM_RI = 320, SSM_KA = 384, SSM_W = 448 };
constexpr int SSM_REC = 2048;

hipError_t launch_ssm_fwd(const SsmParams& p, hipStream_t stream);
hipError_t launch_ssm_bwd(const SsmParams& p, hipStream_t stream);
hipError_t launch_ssm_grads(const SsmParams& p, hipStream_t stream);
void launch_ssm_scan(const SsmParams& p, hipStream_t stream);
// What segments add to the state; `both`: and to its gradients.
void launch_ssm_adds(const SsmParams& p, bool both, hipStream_t stream);

// Value columns that a walking work-group takes at most.
constexpr int SSM_COLS = 256;

struct SsmDecodeParams {
    Rows x, B, C;          // [N, H, P], [N, G, S]: sb is the stride of N, st is unused
    const void* dt;        // [N, H], stride dtb
    int64_t dtb;
    const float *A, *D, *bias;
    const int32_t* idx;    // [N] state slots, or nullptr (slot n)
    const float* s_in;     // [slots, H, S, P] or nullptr (zero)
    float* s_out;          // [slots, H, S, P]; may equal s_in
    uint16_t* y;           // [N, H, P]
    int32_t N, H, G, P, S, slots;
    int32_t dt_f32, softplus;
};
hipError_t launch_ssm_decode(const SsmDecodeParams& p, int cus, hipStream_t stream);

}  // namespace kda
