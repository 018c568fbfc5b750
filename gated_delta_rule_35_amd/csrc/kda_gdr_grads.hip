// Token gradients of the gated delta rule with one decay per head, all chunks at once,
// on gfx950 (MI355X).
//
// From the walks: S the state entering the chunk, dS the gradient of the one leaving
// it, u the corrected values, dx the gradient of beta (v - e^G K S).  With Gam_ij =
// e^{G_i - G_j}, gam_i = e^{G_last - G_i}, P = scale Gam (do u^T) (j <= i),
// E = -beta_i Gam (dx u^T) (j < i), R1 = do S^T, R2 = u dS^T, R3 = dx S^T:
//   dq = scale e^G R1 + P K
//   dk = gam R2 - beta e^G R3 + P^T Q + (E + E^T) K
//   dbeta_i = dx_i . v_i - e^{G_i} k_i . R3_i - sum_j Gam_ij (dx_i . u_j) (k_i . k_j)
//   dG_i = scale e^{G_i} q_i . R1_i - beta_i e^{G_i} k_i . R3_i - t_i + (row i - column i
//          of P (QK^T) + E (KK^T)),   t_i = gam_i k_i . R2_i,
//   dG_last += sum t + e^{G_last} <S, dS>,   dg_t = sum_{i >= t} dG_i within the chunk.
//
// One 512-thread work-group per (chunk slot, q/k head) walks the group's value heads
// and sums their dq and dk in registers (so the sum's order is fixed).  It holds the
// chunk's do, u and dx (bf16 parts) and k, q in LDS; wave w owns channels 16 w .. + 15
// of R1, R2, R3, dq and dk, so S and dS are read once and split once; the ten lower
// 16x16 tiles of the token-by-token products are dealt to the eight waves.  All inputs
// that gradients of g and beta depend on enter in three bf16 parts (fp32's accuracy);
// P and E enter dq and dk, which are rounded to bf16, in two.
//   The kernel is bound by its reads: 64 KB each of S and dS and 32 KB each of u and dx
// per chunk and value head.
#include "kda_gdr_device.h"

namespace kda {

namespace {
constexpr int GT = 512;
constexpr int PS = 144;   // bytes per row of 64 bf16 (+16)
struct GL {
    static constexpr int K = 0, Q = 16384, DO = 32768, U = 49152, X = U + 3 * 16384;
    static constexpr int PL = 64 * PS;                  // one part of P or E, over U
    static constexpr int OUT = U, OS = 272;             // dq, dk on the way out: rows of 128 bf16 (+16)
    static constexpr int END = X + 3 * 16384;
    static_assert(4 * PL <= 3 * 16384 && 2 * 64 * OS <= 6 * 16384, "overlays");
};
struct GShared {
    GSum G[64];
    float eg[64], ga[64], be[64], vdot[64];
    float z[8][64], t[8][64], b[8][64];   // row dots by wave (channel sixteenths)
    float rowv[10][16], colv[10][16], rowb[10][16];   // row and column sums by tile
    float sdot[8];
};

// The lane's 16 x 16 tile piece: tokens 16 m + 4 g + r of channel 16 w + jj.
__device__ __forceinline__ u32x2 chan_frag(const char* tile, int m, int w, int g, int jj) {
    return lds_tr(tile + tile_off(16 * m + 4 * g + (jj >> 2), 2 * w + ((jj & 3) >> 1)) + 8 * (jj & 1));
}
__device__ __forceinline__ bf16x8 row_frag(const char* tile, int m, int kk, int g, int jj) {
    return lds_bf8(tile + tile_off(16 * m + jj, 4 * kk + g));
}
__device__ __forceinline__ f32x4 widen(u32x2 x) { return f32x4{bf_lo(x[0]), bf_hi(x[0]), bf_lo(x[1]), bf_hi(x[1])}; }
// A operand (m, kk) of a 64x64 plane, and of its transpose.
__device__ __forceinline__ bf16x8 plane_row(const char* pl, int m, int kk, int g, int jj) {
    const char* a = pl + (16 * m + jj) * PS + 64 * kk + 8 * g;
    return join(*reinterpret_cast<const u32x2*>(a), *reinterpret_cast<const u32x2*>(a + 32));
}
__device__ __forceinline__ bf16x8 plane_col(const char* pl, int m, int kk, int g, int jj) {
    const char* a = pl + (32 * kk + 4 * g + (jj >> 2)) * PS + 32 * m + 8 * (jj & 3);
    return join(lds_tr(a), lds_tr(a + 16 * PS));
}
}  // namespace

__global__ void __launch_bounds__(GT) kda_gdr_grads_kernel(const GdrParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[GL::END];
    __shared__ GShared sh;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, jj = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t slot = blockIdx.x / p.Hq;
    const int hq = blockIdx.x % p.Hq, R = p.Hv / p.Hq;
    int64_t tok, row;
    const int rows = gdr_chunk(p, slot, tok, row);
    if (rows == 0) return;
    const uint32_t lds = lds_addr(smem);
    dma_tile(chunk_rsrc(p.k.p + row * p.k.sb + tok * p.k.st + hq * p.k.sh, p.k.st, rows, DK), lds + GL::K, p.k.st, w, 8,
             lane);
    dma_tile(chunk_rsrc(p.q.p + row * p.q.sb + tok * p.q.st + hq * p.q.sh, p.q.st, rows, DK), lds + GL::Q, p.q.st, w, 8,
             lane);
    const f32x4 z4 = {0.f, 0.f, 0.f, 0.f};
    f32x4 dq[4], dk[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) dq[m] = dk[m] = z4;

    for (int r = 0; r < R; ++r) {
        const int hv = hq * R + r;
        const int64_t unit = slot * p.Hv + hv;
        const int64_t gi = (row * p.T + tok) * p.Hv + hv;
        dma_tile(chunk_rsrc(p.dO.p + row * p.dO.sb + tok * p.dO.st + hv * p.dO.sh, p.dO.st, rows, DK), lds + GL::DO,
                 p.dO.st, w, 8, lane);
        // u and dx in three parts, and dx . v
        {
            const __amdgpu_buffer_rsrc_t rv =
                chunk_rsrc(p.v.p + row * p.v.sb + tok * p.v.st + hv * p.v.sh, p.v.st, rows, DK);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 32 * h + (tid >> 4), pc = tid & 15;
                const float* us = p.u + unit * CH * DK + i * DK + 8 * pc;
                const float* xs = p.dx + unit * CH * DK + i * DK + 8 * pc;
                const f32x4 u0 = *reinterpret_cast<const f32x4*>(us), u1 = *reinterpret_cast<const f32x4*>(us + 4);
                const f32x4 x0 = *reinterpret_cast<const f32x4*>(xs), x1 = *reinterpret_cast<const f32x4*>(xs + 4);
                const i32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rv, (int)(i * p.v.st * 2) + 16 * pc, 0, 0);
                const Split<3> us3 = split_acc<3>(u0, u1), xs3 = split_acc<3>(x0, x1);
                const int at = tile_off(i, pc);
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    *reinterpret_cast<bf16x8*>(smem + GL::U + n * 16384 + at) = us3.s[n];
                    *reinterpret_cast<bf16x8*>(smem + GL::X + n * 16384 + at) = xs3.s[n];
                }
                float d = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t vv = (uint32_t)v[e];
                    const float xa = e < 2 ? x0[2 * e] : x1[2 * e - 4], xb = e < 2 ? x0[2 * e + 1] : x1[2 * e - 3];
                    d = fmaf(xa, bf_lo(vv), d);
                    d = fmaf(xb, bf_hi(vv), d);
                }
                d = sum16(d);
                if (pc == 0) sh.vdot[i] = d;
            }
        }
        if (w == 0) {
            const bool in = lane < rows;
            const GSum G = gate_sum(in ? p.g[gi + (int64_t)lane * p.Hv] : 0.f, lane);
            const GSum last = {__shfl(G.hi, 63), __shfl(G.lo, 63)};
            sh.G[lane] = G;
            sh.eg[lane] = gate_exp(G);
            sh.ga[lane] = gate_ratio(last, G);
            sh.be[lane] = in ? gdr_beta(p, gi + (int64_t)lane * p.Hv) : 0.f;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();

        // R1, R2, R3 for channels 16 w + jj
        {
            Split<3> sb[4], db[4];
            float sd = 0.f;
            const float* ss = p.S + unit * DK * DK + (16 * w + jj) * DK + 8 * g;
            const float* ds = p.dS + unit * DK * DK + (16 * w + jj) * DK + 8 * g;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const f32x4 a0 = *reinterpret_cast<const f32x4*>(ss + 32 * kk);
                const f32x4 a1 = *reinterpret_cast<const f32x4*>(ss + 32 * kk + 4);
                const f32x4 b0 = *reinterpret_cast<const f32x4*>(ds + 32 * kk);
                const f32x4 b1 = *reinterpret_cast<const f32x4*>(ds + 32 * kk + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) sd = fmaf(a0[e], b0[e], fmaf(a1[e], b1[e], sd));
                sb[kk] = split_acc<3>(a0, a1);
                db[kk] = split_acc<3>(b0, b1);
            }
            sd = sum16(sd);
            sd += __shfl_xor(sd, 16);
            sd += __shfl_xor(sd, 32);
            if (lane == 0) sh.sdot[w] = sd;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 r1 = z4, r2 = z4, r3 = z4;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const int at = tile_off(16 * m + jj, 4 * kk + g);
                    const bf16x8 fo[1] = {lds_bf8(smem + GL::DO + at)};
                    bf16x8 fu[3], fx[3];
#pragma unroll
                    for (int n = 0; n < 3; ++n) {
                        fu[n] = lds_bf8(smem + GL::U + n * 16384 + at);
                        fx[n] = lds_bf8(smem + GL::X + n * 16384 + at);
                    }
                    r1 = mfma_split<3>(fo, sb[kk], r1);
                    r2 = mfma_split<3>(fu, db[kk], r2);
                    r3 = mfma_split<3>(fx, sb[kk], r3);
                }
                const f32x4 eg = *reinterpret_cast<const f32x4*>(sh.eg + 16 * m + 4 * g);
                const f32x4 ga = *reinterpret_cast<const f32x4*>(sh.ga + 16 * m + 4 * g);
                const f32x4 be = *reinterpret_cast<const f32x4*>(sh.be + 16 * m + 4 * g);
                const f32x4 kv = widen(chan_frag(smem + GL::K, m, w, g, jj));
                const f32x4 qv = widen(chan_frag(smem + GL::Q, m, w, g, jj));
                r1 = (p.scale * eg) * r1;
                r2 = ga * r2;
                r3 = eg * r3;
                dq[m] += r1;
                dk[m] += r2 - be * r3;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float t = sum16(kv[e] * r2[e]), b = sum16(kv[e] * r3[e]), a = sum16(qv[e] * r1[e]);
                    if (jj == 0) {
                        const int i = 16 * m + 4 * g + e;
                        sh.t[w][i] = t;
                        sh.b[w][i] = b;
                        sh.z[w][i] = a - be[e] * b - t;
                    }
                }
            }
        }
        // token-by-token tiles w and w + 8 of the ten lower ones
        f32x4 P[2], E[2];
        int ti[2], tj[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int id = w + 8 * x;
            ti[x] = id >= 6 ? 3 : id >= 3 ? 2 : id >= 1 ? 1 : 0;
            tj[x] = id - ti[x] * (ti[x] + 1) / 2;
            P[x] = E[x] = z4;
            if (id >= 10) continue;
            f32x4 a = z4, mm = z4, qk = z4, kk2 = z4;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int ai = tile_off(16 * ti[x] + jj, 4 * kk + g), aj = tile_off(16 * tj[x] + jj, 4 * kk + g);
                Split<3> ub;
                bf16x8 fx[3];
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    ub.s[n] = lds_bf8(smem + GL::U + n * 16384 + aj);
                    fx[n] = lds_bf8(smem + GL::X + n * 16384 + ai);
                }
                const bf16x8 fo[1] = {lds_bf8(smem + GL::DO + ai)};
                a = mfma_split<3>(fo, ub, a);
                mm = mfma_split<3>(fx, ub, mm);
                const bf16x8 kb = lds_bf8(smem + GL::K + aj);
                qk = mfma_bf(lds_bf8(smem + GL::Q + ai), kb, qk);
                kk2 = mfma_bf(lds_bf8(smem + GL::K + ai), kb, kk2);
            }
            const int j = 16 * tj[x] + jj;
            const GSum Gj = sh.G[j];
            float cs = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * ti[x] + 4 * g + e;
                const float gam = j <= i ? gate_ratio(sh.G[i], Gj) : 0.f;
                const float pe = j <= i ? p.scale * (gam * a[e]) : 0.f;
                const float ge = j < i ? -(gam * mm[e]) : 0.f;   // Gam times dM
                const float ee = sh.be[i] * ge;
                P[x][e] = pe;
                E[x][e] = ee;
                const float val = pe * qk[e] + ee * kk2[e];
                cs += val;
                const float rs = sum16(val), rb = sum16(ge * kk2[e]);
                if (jj == 0) {
                    sh.rowv[id][4 * g + e] = rs;
                    sh.rowb[id][4 * g + e] = rb;
                }
            }
            cs += __shfl_xor(cs, 16);
            cs += __shfl_xor(cs, 32);
            if (g == 0) sh.colv[id][jj] = cs;
        }
        __syncthreads();   // u's parts read; the sums complete
        if (w == 7) {      // the wave with the fewest tiles
            const int i = lane, I = i >> 4;
            double dG = 0.0;
            float db = sh.vdot[i], ts = 0.f, sd = 0.f;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                dG += (double)sh.z[n][i];
                db -= sh.b[n][i];
                ts += sh.t[n][i];
                sd += sh.sdot[n];
            }
            for (int n = 0; n < 4; ++n) {
                if (n <= I) {
                    dG += (double)sh.rowv[I * (I + 1) / 2 + n][i & 15];
                    db += sh.rowb[I * (I + 1) / 2 + n][i & 15];
                }
                if (n >= I) dG -= (double)sh.colv[n * (n + 1) / 2 + I][i & 15];
            }
            double tsum = (double)ts;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) tsum += __shfl_xor(tsum, m);
            if (i == 63) dG += tsum + (double)(sh.eg[63] * sd);
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {   // suffix sums
                const double y = __shfl_down(dG, m);
                if (i + m < 64) dG += y;
            }
            if (i < rows) {
                p.dg[gi + (int64_t)i * p.Hv] = (float)dG;
                p.dbeta[gi + (int64_t)i * p.Hv] = db;
            }
        }
        // P and E as row-major planes of two bf16 parts
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (w + 8 * x >= 10) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = (16 * ti[x] + 4 * g + e) * PS + 2 * (16 * tj[x] + jj);
                const uint32_t h = pack_bf2(P[x][e], E[x][e]);
                const uint32_t l = pack_bf2(P[x][e] - bf_lo(h), E[x][e] - bf_hi(h));
                *reinterpret_cast<uint16_t*>(smem + GL::U + at) = (uint16_t)h;
                *reinterpret_cast<uint16_t*>(smem + GL::U + GL::PL + at) = (uint16_t)l;
                *reinterpret_cast<uint16_t*>(smem + GL::U + 2 * GL::PL + at) = (uint16_t)(h >> 16);
                *reinterpret_cast<uint16_t*>(smem + GL::U + 3 * GL::PL + at) = (uint16_t)(l >> 16);
            }
        }
        for (int e = tid; e < 2048; e += GT) {   // the tiles above the diagonal that operands cover
            const int x = e & 255, t = (e >> 8) & 1;
            *reinterpret_cast<uint16_t*>(smem + GL::U + (e >> 9) * GL::PL + (32 * t + (x >> 4)) * PS +
                                         2 * (32 * t + 16 + (x & 15))) = 0;
        }
        __syncthreads();
        {
            bf16x8 kb[2], qb[2];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                kb[kk] = join(chan_frag(smem + GL::K, 2 * kk, w, g, jj), chan_frag(smem + GL::K, 2 * kk + 1, w, g, jj));
                qb[kk] = join(chan_frag(smem + GL::Q, 2 * kk, w, g, jj), chan_frag(smem + GL::Q, 2 * kk + 1, w, g, jj));
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int n = 1; n >= 0; --n) {
                    const char* pp = smem + GL::U + n * GL::PL;
                    const char* pe = smem + GL::U + (2 + n) * GL::PL;
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        if (kk <= m / 2) {
                            dq[m] = mfma_bf(plane_row(pp, m, kk, g, jj), kb[kk], dq[m]);
                            dk[m] = mfma_bf(plane_row(pe, m, kk, g, jj), kb[kk], dk[m]);
                        }
                        if (kk >= m / 2) {
                            dk[m] = mfma_bf(plane_col(pp, m, kk, g, jj), qb[kk], dk[m]);
                            dk[m] = mfma_bf(plane_col(pe, m, kk, g, jj), kb[kk], dk[m]);
                        }
                    }
                }
            }
        }
        __syncthreads();   // the planes' reads before the next value head's parts
    }
    // dq and dk, rounded once
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t h = pack_bf2(dq[m][e], dk[m][e]);
            const int at = (16 * m + 4 * g + e) * GL::OS + 2 * (16 * w + jj);
            *reinterpret_cast<uint16_t*>(smem + GL::OUT + at) = (uint16_t)h;
            *reinterpret_cast<uint16_t*>(smem + GL::OUT + 64 * GL::OS + at) = (uint16_t)(h >> 16);
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const int i = 32 * (h & 1) + (tid >> 4), pc = tid & 15;
        if (i < rows) {
            uint16_t* dst = (h < 2 ? p.dq : p.dk) + ((row * p.T + tok + i) * p.Hq + hq) * DK + 8 * pc;
            *reinterpret_cast<u32x4*>(dst) =
                *reinterpret_cast<const u32x4*>(smem + GL::OUT + (h < 2 ? 0 : 64 * GL::OS) + i * GL::OS + 16 * pc);
        }
    }
}

hipError_t launch_gdr_grads(const GdrParams& p, hipStream_t stream) {
    const int64_t blocks = p.nslots * p.Hq;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(kda_gdr_grads_kernel, dim3((unsigned)blocks), dim3(GT), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
