// Chunk-parallel preparation of the gated delta rule with one decay per head, on
// gfx950 (MI355X).
//
// For a chunk of 64 tokens with G the running sum of g and Gam_ij = e^{G_i - G_j}:
//   M = beta_i (K K^T) Gam, j < i;   T = (I + M)^{-1};   backward also A = scale (Q K^T) Gam, j <= i
// The decay is one number per token, so the products are formed once per q/k head from
// the bf16 operands as they are, and every value head of the group only scales
// them: Gam_ij <= 1 is formed from the differences themselves, so no operand needs an
// anchor and no decay is out of range.
//
// One 256-thread work-group per (chunk slot, q/k head) walks the group's value heads.
// k (and q) come into LDS by DMA, where M (and A) go once the products are formed.  Wave w
// takes the diagonal tile (w, w) of both and one or two of the six below.  T in fp32: wave
// w inverts the diagonal block w by forward substitution, then forms block column w
// downwards on v_mfma_f32_16x16x4f32,
//   T_IJ = -T_II sum_{K=J}^{I-1} M_IK T_KJ,
// with the T_KJ of its column in registers (an accumulator tile is the next product's
// B operand).  T and A leave as operand fragments in three bf16 parts each, the forward's T
// with its columns times beta.  The forward's walk forms A itself, from the k and q that it
// holds anyway, so that q is not read here and records stay at 20 KB.
//
// At B=2 H=64 T=8192 (16,384 chunks of a head): forward 140 us, 0.66 GB at 4.7 TB/s; with the
// backward's records 203 us, 1.22 GB at 6.0 TB/s (part of what it writes stays in the
// last-level cache).  What brought the latter there: four work-groups a compute unit, k
// and q by DMA, and the tiles dealt evenly; a form that kept M and A beside k and q in LDS
// (two work-groups a unit) took 292 us of the forward's 200 then.  Forming T inside the walk
// instead, a work-group for both, took 848 us and more for 680 us of the two kernels then.
// Fragment (m, kk) holds in lane l rows 16 m + l % 16, columns 32 kk + 16 (s / 4) +
// 4 (l / 16) + s % 4, s < 8: the order in which accumulator tiles list a 32-wide k
// step.  The lists hold (0,0) (1,0) (2,0) (2,1) (3,0) (3,1), zeros above the diagonal.
#include "kda_gdr_device.h"

namespace kda {

namespace {
constexpr int SP = 68;   // row stride of the fp32 64x64 matrices (64 + 4: 16-byte aligned rows, spread banks)
}

template <bool BWD>
__global__ void __launch_bounds__(256, 4) kda_gdr_prep_kernel(const GdrParams p) {
    __shared__ __attribute__((aligned(1024))) float mats[2 * 64 * SP];
    float *const sM = mats, *const sA = mats + 64 * SP;   // M, then T in its place; A
    char *const tk = reinterpret_cast<char*>(mats), *const tq = tk + 16384;   // before them k and q
    static_assert(2 * 64 * SP * 4 >= 2 * 16384, "k and q fit where M and A go");
    __shared__ GSum sG[64];
    __shared__ __attribute__((aligned(16))) float sBeta[64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = (int)blockIdx.x / p.Hq, hq = (int)blockIdx.x % p.Hq, R = p.Hv / p.Hq;
    int64_t tok, row;
    const int rows = gdr_chunk(p, slot, tok, row);
    if (rows == 0) return;
    // g and beta of the value head at hand, token = lane (wave 0); tokens past the end
    // change nothing: g = 0, beta = 0
    const int64_t gi = (row * p.T + tok + lane) * p.Hv + hq * R;
    float gate = 0.f, beta = 0.f;
    if (w == 0 && lane < rows) {
        gate = p.g[gi];
        beta = gdr_beta(p.beta, p.beta_f32, gi);
    }

    {
        const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(tk));
        dma_tile(chunk_rsrc(p.k.p + row * p.k.sb + tok * p.k.st + hq * p.k.sh, p.k.st, rows, DK), lds, p.k.st, w, 4, lane);
        if (BWD)
            dma_tile(chunk_rsrc(p.q.p + row * p.q.sb + tok * p.q.st + hq * p.q.sh, p.q.st, rows, DK), lds + 16384, p.q.st,
                     w, 4, lane);
        if (w == 0) {
            sG[lane] = gate_sum(gate);
            sBeta[lane] = BWD ? beta_of_u(beta) : beta;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
    // The wave's tiles (I, J): the diagonal one, then (1,0) (3,0) | (2,0) (3,1) | (2,1) | (3,2).
    const int ti[3] = {w, w == 0 ? 1 : w == 3 ? 3 : 2, 3}, tj[3] = {w, w == 2 ? 1 : w == 3 ? 2 : 0, w};
    const int nt = w < 2 ? 3 : 2;
    f32x4 qk[3], kk[3];   // raw products: lane holds rows 16 I + 4 g + r of column 16 J + jj
    {
        const int g = lane >> 4, jj = lane & 15;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            qk[x] = kk[x] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (x >= nt) continue;
            bf16x8 aq[4], ak[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (BWD) aq[c] = lds_bf8(tq + tile_off(16 * ti[x] + jj, 4 * c + g));
                ak[c] = lds_bf8(tk + tile_off(16 * ti[x] + jj, 4 * c + g));
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bf16x8 b = x == 0 ? ak[c] : lds_bf8(tk + tile_off(16 * tj[x] + jj, 4 * c + g));
                if (BWD) qk[x] = mfma_bf(aq[c], b, qk[x]);
                kk[x] = mfma_bf(ak[c], b, kk[x]);
            }
        }
    }
    __syncthreads();   // k and q are read
    // tiles above the diagonal that fragments cover
    for (int e = tid; e < 512; e += 256) {
        const int t = e >> 8, x = e & 255, at = (32 * t + (x >> 4)) * SP + 32 * t + 16 + (x & 15);
        sM[at] = 0.f;
        if (BWD) sA[at] = 0.f;
    }

    for (int r = 0; r < R; ++r) {
        const int hv = hq * R + r;
        float own = 0.f;   // this value head's beta (wave 0)
        if (w == 0) {
            if (r > 0) {
                sG[lane] = gate_sum(gate);
                sBeta[lane] = BWD ? beta_of_u(beta) : beta;
            }
            own = beta;
            if (r + 1 < R && lane < rows) {
                gate = p.g[gi + r + 1];
                beta = gdr_beta(p.beta, p.beta_f32, gi + r + 1);
            }
        }
        if (r > 0) __syncthreads();
        char* rec = p.rec + ((int64_t)slot * p.Hv + hv) * (BWD ? GDR_REC : FWD_REC);
        if (w == 0) {
            float* sc = reinterpret_cast<float*>(rec + GDR_SC) + lane;
            const GSum G = sG[lane], GL = sG[63];
            sc[SC_EG] = gate_exp(G);
            sc[SC_GA] = gate_ratio(GL, G);
            sc[SC_BE] = own;
            if (BWD) {
                sc[SC_BU] = sBeta[lane];
            } else {
                sc[SC_GH] = G.hi;
                sc[SC_GL] = G.lo;
            }
        }
        {
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;   // formed anew: kept through the loop, addresses would spill
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            if (x < nt) {
                const int j = 16 * tj[x] + jj, i0 = 16 * ti[x] + 4 * g;
                const GSum Gj = sG[j];
                const f32x4 be = *reinterpret_cast<const f32x4*>(sBeta + i0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + e;
                    const float gam = j <= i ? gate_ratio(sG[i], Gj) : 0.f;
                    if (BWD) sA[i * SP + j] = j <= i ? p.scale * (qk[x][e] * gam) : 0.f;
                    sM[i * SP + j] = j < i ? be[e] * (kk[x][e] * gam) : 0.f;
                }
            }
        }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // this wave's tiles of M
        {   // diagonal block w, in its place: lane column jj (lane groups repeat each other)
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            const float* m = sM + 16 * w * SP + 16 * w;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = i == jj ? 1.f : 0.f;
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {   // four columns eliminated from the rows below them
                asm volatile("" : "+v"(x[15])::"memory");   // no earlier: all columns' loads at once would spill
                f32x4 r4[16];
#pragma unroll
                for (int i = 1; i < 16; ++i)
                    if (i > 4 * kb) r4[i] = *reinterpret_cast<const f32x4*>(m + i * SP + 4 * kb);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int i = 1; i < 16; ++i)
                        if (i > 4 * kb + e) x[i] = fmaf(-r4[i][e], x[4 * kb + e], x[i]);
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the block is read before it is overwritten
            if (g == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) sM[(16 * w + i) * SP + 16 * w + jj] = x[i];
            }
        }
        __syncthreads();
        f32x4 t[4];
        {   // block column w downwards
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
#pragma unroll
            for (int e = 0; e < 4; ++e) t[0][e] = sM[(16 * w + 4 * g + e) * SP + 16 * w + jj];
#pragma unroll
            for (int s = 1; s < 4; ++s) {   // row block I = w + s; t[n] is T_{w + n, w}
                const int I = w + s;
                if (I < 4) {
                    f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
#pragma unroll
                    for (int n = 0; n < s; ++n) {
                        const f32x4 a =
                            *reinterpret_cast<const f32x4*>(sM + (16 * I + jj) * SP + 16 * (w + n) + 4 * g);
                        x = __builtin_amdgcn_mfma_f32_16x16x4f32(a[0], t[n][0], x, 0, 0, 0);
                        y = __builtin_amdgcn_mfma_f32_16x16x4f32(a[1], t[n][1], y, 0, 0, 0);
                        x = __builtin_amdgcn_mfma_f32_16x16x4f32(a[2], t[n][2], x, 0, 0, 0);
                        y = __builtin_amdgcn_mfma_f32_16x16x4f32(a[3], t[n][3], y, 0, 0, 0);
                    }
                    x += y;
                    const f32x4 a = *reinterpret_cast<const f32x4*>(sM + (16 * I + jj) * SP + 16 * I + 4 * g);
                    f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 4; ++e) z = __builtin_amdgcn_mfma_f32_16x16x4f32(-a[e], x[e], z, 0, 0, 0);
                    t[s] = z;
                }
            }
        }
        __syncthreads();   // M is read
#pragma unroll
        for (int s = 1; s < 4; ++s) {
            const int I = w + s;
            if (I < 4) {
                const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
#pragma unroll
                for (int e = 0; e < 4; ++e) sM[(16 * I + 4 * g + e) * SP + 16 * w + jj] = t[s][e];
            }
        }
        __syncthreads();
        // fragments: six of T's and, for the backward, six of A's
#pragma unroll
        for (int f3 = 0; f3 < (BWD ? 3 : 2); ++f3) {
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            const int f = 4 * f3 + w, which = f >= 6, x = which ? f - 6 : f;
            if (!BWD && which) continue;
            const int m = x < 2 ? x : 2 + ((x - 2) >> 1), c = x < 2 ? 0 : x & 1;   // (m, kk)
            const float* a = (which ? sA : sM) + (16 * m + jj) * SP + 32 * c + 4 * g;
            f32x4 u0 = *reinterpret_cast<const f32x4*>(a), u1 = *reinterpret_cast<const f32x4*>(a + 16);
            if (!BWD) {   // T diag(beta)
                u0 *= *reinterpret_cast<const f32x4*>(sBeta + 32 * c + 4 * g);
                u1 *= *reinterpret_cast<const f32x4*>(sBeta + 32 * c + 16 + 4 * g);
            }
            char* dst = rec + (which ? GDR_A : GDR_T) + x * GDR_FRAG + frag_piece(ln);
            const Split<3> parts = split_acc<3>(u0, u1);
#pragma unroll
            for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8*>(dst + n * GDR_TRI) = parts.s[n];
        }
        __syncthreads();   // the matrices' reads before the next value head's writes
    }
}

hipError_t launch_gdr_prep(const GdrParams& p, bool bwd, hipStream_t stream) {
    const int64_t blocks = p.nslots * p.Hq;
    if (blocks == 0) return hipSuccess;
    if (bwd) hipLaunchKernelGGL(kda_gdr_prep_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(kda_gdr_prep_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
