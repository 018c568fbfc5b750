// The sequential walks of the backward of the gated delta rule with one decay per head,
// on gfx950 (MI355X), with the prep kernel's T and A:
// forwards once more, for the state that enters each chunk and the corrected values,
//   e = v - e^G (K S),  u = T (beta e),  S <- e^{G_last} S + K^T (e^{G_last - G} u),
// then chunks in reverse, dS the gradient of the state that leaves the chunk,
//   du = A^T do + e^{G_last - G} (K dS),  dx = T^T du,  dv = beta dx,
//   dS <- e^{G_last} dS + Q^T (scale e^G do) - K^T (beta e^G dx).
//
// Every product's right-hand side is a set of columns of S (value channels), and no
// product mixes columns: a wave owns 16 of them for the whole sequence and needs
// nothing from the others.  Its state is eight 16x16 accumulator tiles (32 registers a
// lane), and since an accumulator tile holds what a lane needs as B operand, the whole
// chain of a chunk stays in registers.  A work-group is four waves (64 columns) that
// share the chunk's left-hand operands in LDS: the K and Q tiles, read as they lie for
// K S and transposed (ds_read_b64_tr_b16) for K^T u, and the record's fragments.  The
// next chunk's come by DMA into the other buffer meanwhile; one barrier per chunk.
//   Tile t = 2 kk + h of the state holds key channel 32 kk + 8 g + 4 h + r in row
// 4 g + r (g = lane / 16), so that the two tiles of a 32-channel step list the lane's
// eight channels as they lie in K's rows.
//   fp32 operands go in as three bf16 parts, see kda_gdr_device.h.
#include "kda_gdr_device.h"

namespace kda {

namespace {

constexpr int SCAN_THREADS = 384;   // four waves that compute, two that load
// One LDS buffer: K, Q tiles (swizzled), the slice of v (or of do) [64][64] bf16, the record.
struct ScanL {
    static constexpr int K = 0, Q = 16384, V = 32768, REC = 40960, BYTES = REC + GDR_REC;
};

// The lane's eight (key channel, tile) rows: channel of row 4 g + r of tile t.
__device__ __forceinline__ int state_row(int t, int g, int r) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1) + r; }

// A operand (m, kk) of a tile [64][128]: rows 16 m + jj, channels 32 kk + 8 g ..
__device__ __forceinline__ bf16x8 row_frag(const char* tile, int m, int kk, int g, int jj) {
    return lds_bf8(tile + tile_off(16 * m + jj, 4 * kk + g));
}
// A operand of the transposed tile: state tile t's channels, tokens of k step kk.
__device__ __forceinline__ bf16x8 col_frag(const char* tile, int t, int kk, int g, int jj) {
    const int row = 32 * kk + 4 * g + (jj >> 2), piece = 4 * (t >> 1) + (jj & 3), b = 8 * (t & 1);
    return join(lds_tr(tile + tile_off(row, piece) + b), lds_tr(tile + tile_off(row + 16, piece) + b));
}
// Columns 16 w + jj of tokens 16 m + 4 g + r, r < 4, of the [64][64] slice, as packed bf16.
__device__ __forceinline__ u32x2 slice_frag(const char* v, int m, int w, int g, int jj) {
    return lds_tr(v + (16 * m + 4 * g + (jj >> 2)) * 128 + 32 * w + 8 * (jj & 3));
}
__device__ __forceinline__ f32x4 widen(u32x2 x) { return f32x4{bf_lo(x[0]), bf_hi(x[0]), bf_lo(x[1]), bf_hi(x[1])}; }

// Index of fragment (m, kk) in a record's lower triangular list.
__device__ __forceinline__ constexpr int tri_frag(int m, int kk) { return m < 2 ? m : 2 * m - 2 + kk; }
// Fragment (m, kk) of the transposed matrix (rows 16 m + jj, k step kk), kk >= m / 2.
__device__ __forceinline__ bf16x8 tri_col_frag(const char* part, int m, int kk, int g, int jj) {
    const int at = (jj & 3) * 256 + (4 * g + (jj >> 2)) * 16 + 8 * (m & 1);
    return join(lds_tr(part + tri_frag(2 * kk, m >> 1) * GDR_FRAG + at),
                lds_tr(part + tri_frag(2 * kk + 1, m >> 1) * GDR_FRAG + at));
}

// One loading wave's (ld = 0, 1) half of a chunk's DMA into a buffer: 32 pieces of
// tiles and slices, and nrec of the record.
template <int NREC, bool WITH_Q>
__device__ __forceinline__ void load_chunk(const GdrParams& p, const Rows& vsrc, uint32_t lds, int64_t row, int64_t tok,
                                           int rows, int hq, int hv, int sl, int64_t slot, int ld, int lane) {
    typedef ScanL L;
    const __amdgpu_buffer_rsrc_t rk =
        chunk_rsrc(p.k.p + row * p.k.sb + tok * p.k.st + hq * p.k.sh, p.k.st, rows, DK);
    const int l4 = lane >> 4, l16 = lane & 15;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int r = 4 * (8 * ld + u) + l4;
        dma_piece(rk, lds + L::K + (8 * ld + u) * 1024, (int)(r * p.k.st * 2) + ((l16 ^ tsw(4 * u + l4)) << 4));
    }
    if (WITH_Q) {
        const __amdgpu_buffer_rsrc_t rq =
            chunk_rsrc(p.q.p + row * p.q.sb + tok * p.q.st + hq * p.q.sh, p.q.st, rows, DK);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int r = 4 * (8 * ld + u) + l4;
            dma_piece(rq, lds + L::Q + (8 * ld + u) * 1024, (int)(r * p.q.st * 2) + ((l16 ^ tsw(4 * u + l4)) << 4));
        }
    }
    const __amdgpu_buffer_rsrc_t rv =
        chunk_rsrc(vsrc.p + row * vsrc.sb + tok * vsrc.st + hv * vsrc.sh + 64 * sl, vsrc.st, rows, 64);
#pragma unroll
    for (int u = 0; u < 4; ++u) {   // eight rows a piece
        const int x = 4 * ld + u;
        dma_piece(rv, lds + L::V + x * 1024, (int)((8 * x + (lane >> 3)) * vsrc.st * 2) + ((lane & 7) << 4));
    }
    const __amdgpu_buffer_rsrc_t rr =
        make_rsrc(p.rec + (slot * p.Hv + hv) * GDR_REC, GDR_REC);
#pragma unroll
    for (int u = 0; u < (NREC + 1) / 2; ++u) {
        const int x = 2 * u + ld;
        if (x < NREC) dma_piece(rr, lds + L::REC + x * 1024, x * 1024 + lane * 16);
    }
}

}  // namespace

__global__ void __launch_bounds__(SCAN_THREADS) kda_gdr_keep_kernel(const GdrParams p) {
    typedef ScanL L;
    __shared__ __attribute__((aligned(1024))) char smem[2 * L::BYTES];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, jj = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Walk walk = walk_of_block(p, (int)blockIdx.x, reinterpret_cast<int*>(smem));
    const int n = walk.n, hv = walk.hv, sl = walk.sl, hq = hv / (p.Hv / p.Hq);
    int64_t bos, len, row, slot0;
    gdr_seq(p, n, bos, len, row, slot0);
    const int nch = (int)((len + CH - 1) / CH);
    const int col = 64 * sl + 16 * w + jj;   // the lane's value channel
    auto rows_of = [&](int c) -> int {
        const int64_t r = len - (int64_t)c * CH;
        return r <= 0 ? 0 : (r >= CH ? CH : (int)r);
    };
    if (w >= 4) {   // loading waves: chunk c + 1 while the others are at chunk c
        constexpr int NREC = 19;   // pieces of the record that are read: T and the numbers
        const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));
        auto load = [&](int c) {
            load_chunk<NREC, false>(p, p.v, lds + (c & 1) * L::BYTES, row, bos + (int64_t)c * CH, rows_of(c), hq, hv,
                                        sl, slot0 + c, w - 4, lane);
        };
        if (nch > 0) load(0);
        for (int c = 0; c < nch; ++c) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's pieces of chunk c
            lds_barrier();
            if (c + 1 < nch) load(c + 1);
        }
        return;
    }

    f32x4 S[8];
    const int64_t so = ((int64_t)n * p.Hv + hv) * DK * DK + col;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = p.h0 ? p.h0[so + state_row(t, g, r) * DK] : 0.f;
    }
    for (int c = 0; c < nch; ++c) {
        lds_barrier();   // chunk c is in LDS, and the other buffer's reads are done
        char* buf = smem + (c & 1) * L::BYTES;
        const char *sK = buf + L::K, *sQ = buf + L::Q, *rec = buf + L::REC;
        const float* sc = reinterpret_cast<const float*>(rec + GDR_SC);
        {
            float* dst = p.S + ((slot0 + c) * p.Hv + hv) * DK * DK + col;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) dst[state_row(t, g, r) * DK] = S[t][r];
            }
        }
        Split<3> sb[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) sb[kk] = split_acc<3>(S[2 * kk], S[2 * kk + 1]);
        // x = beta (v - e^G K S)
        f32x4 x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const bf16x8 f[1] = {row_frag(sK, m, kk, g, jj)};
                a = mfma_split<3>(f, sb[kk], a);
            }
            const f32x4 eg = *reinterpret_cast<const f32x4*>(sc + SC_EG + 16 * m + 4 * g);
            const f32x4 be = *reinterpret_cast<const f32x4*>(sc + SC_BE + 16 * m + 4 * g);
            const f32x4 v = widen(slice_frag(buf + L::V, m, w, g, jj));
            x[m] = be * (v - eg * a);
        }
        // u = T x
        f32x4 u[4];
        {
            Split<3> xb[2];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) xb[kk] = split_acc<3>(x[2 * kk], x[2 * kk + 1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk <= m / 2; ++kk) {
                    const char* f = rec + GDR_T + tri_frag(m, kk) * GDR_FRAG + lane * 16;
                    const bf16x8 tp[3] = {lds_bf8(f), lds_bf8(f + GDR_TRI), lds_bf8(f + 2 * GDR_TRI)};
                    a = mfma_split<3>(tp, xb[kk], a);
                }
                u[m] = a;
            }
        }
        {
            float* dst = p.u + ((slot0 + c) * p.Hv + hv) * CH * DK + col;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int r = 0; r < 4; ++r) dst[(16 * m + 4 * g + r) * DK] = u[m][r];
            }
        }
        // S <- e^{G_last} S + K^T (e^{G_last - G} u)
        Split<3> wb[2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const f32x4 g0 = *reinterpret_cast<const f32x4*>(sc + SC_GA + 32 * kk + 4 * g);
            const f32x4 g1 = *reinterpret_cast<const f32x4*>(sc + SC_GA + 32 * kk + 16 + 4 * g);
            wb[kk] = split_acc<3>(g0 * u[2 * kk], g1 * u[2 * kk + 1]);
        }
        const float el = sc[SC_EL];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            f32x4 a = S[t] * el;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const bf16x8 f[1] = {col_frag(sK, t, kk, g, jj)};
                a = mfma_split<3>(f, wb[kk], a);
            }
            S[t] = a;
        }
    }
}

__global__ void __launch_bounds__(SCAN_THREADS) kda_gdr_rscan_kernel(const GdrParams p) {
    constexpr int NREC = 37;   // pieces of the record
    static_assert(NREC * 1024 == GDR_REC, "record");
    typedef ScanL L;
    __shared__ __attribute__((aligned(1024))) char smem[2 * L::BYTES];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, jj = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Walk walk = walk_of_block(p, (int)blockIdx.x, reinterpret_cast<int*>(smem));
    const int n = walk.n, hv = walk.hv, sl = walk.sl, hq = hv / (p.Hv / p.Hq);
    int64_t bos, len, row, slot0;
    gdr_seq(p, n, bos, len, row, slot0);
    const int nch = (int)((len + CH - 1) / CH);
    const int col = 64 * sl + 16 * w + jj;
    auto rows_of = [&](int c) -> int {
        const int64_t r = len - (int64_t)c * CH;
        return r <= 0 ? 0 : (r >= CH ? CH : (int)r);
    };
    if (w >= 4) {
        const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));
        auto load = [&](int c) {
            load_chunk<NREC, true>(p, p.dO, lds + (c & 1) * L::BYTES, row, bos + (int64_t)c * CH, rows_of(c),
                                              hq, hv, sl, slot0 + c, w - 4, lane);
        };
        if (nch > 0) load(nch - 1);
        for (int c = nch - 1; c >= 0; --c) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            lds_barrier();
            if (c > 0) load(c - 1);
        }
        return;
    }

    f32x4 S[8];   // dS
    const int64_t so = ((int64_t)n * p.Hv + hv) * DK * DK + col;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = p.dhT ? p.dhT[so + state_row(t, g, r) * DK] : 0.f;
    }
    for (int c = nch - 1; c >= 0; --c) {
        lds_barrier();
        char* buf = smem + (c & 1) * L::BYTES;
        const char *sK = buf + L::K, *sQ = buf + L::Q, *rec = buf + L::REC;
        const float* sc = reinterpret_cast<const float*>(rec + GDR_SC);
        {
            float* dst = p.dS + ((slot0 + c) * p.Hv + hv) * DK * DK + col;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) dst[state_row(t, g, r) * DK] = S[t][r];
            }
        }
        u32x2 d[4];   // do, as it is: accumulator order and, in pairs, B operand
#pragma unroll
        for (int m = 0; m < 4; ++m) d[m] = slice_frag(buf + L::V, m, w, g, jj);
        // du = e^{G_last - G} (K dS) + A^T do
        f32x4 du[4];
        {
            Split<3> sb[4];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) sb[kk] = split_acc<3>(S[2 * kk], S[2 * kk + 1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const bf16x8 f[1] = {row_frag(sK, m, kk, g, jj)};
                    a = mfma_split<3>(f, sb[kk], a);
                }
                a *= *reinterpret_cast<const f32x4*>(sc + SC_GA + 16 * m + 4 * g);
#pragma unroll
                for (int kk = m / 2; kk < 2; ++kk) {
                    const bf16x8 db = join(d[2 * kk], d[2 * kk + 1]);
#pragma unroll
                    for (int n3 = 2; n3 >= 0; --n3)
                        a = mfma_bf(tri_col_frag(rec + GDR_A + n3 * GDR_TRI, m, kk, g, jj), db, a);
                }
                du[m] = a;
            }
        }
        // dx = T^T du
        f32x4 dx[4];
        {
            Split<3> db[2];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) db[kk] = split_acc<3>(du[2 * kk], du[2 * kk + 1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = m / 2; kk < 2; ++kk) {
                    const bf16x8 tp[3] = {tri_col_frag(rec + GDR_T, m, kk, g, jj),
                                          tri_col_frag(rec + GDR_T + GDR_TRI, m, kk, g, jj),
                                          tri_col_frag(rec + GDR_T + 2 * GDR_TRI, m, kk, g, jj)};
                    a = mfma_split<3>(tp, db[kk], a);
                }
                dx[m] = a;
            }
        }
        const int rows = rows_of(c);
        {
            float* dst = p.dx + ((slot0 + c) * p.Hv + hv) * CH * DK + col;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int r = 0; r < 4; ++r) dst[(16 * m + 4 * g + r) * DK] = dx[m][r];
            }
        }
        // dv = beta dx, rounded once, through this wave's columns of the do slice
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 y = dx[m] * *reinterpret_cast<const f32x4*>(sc + SC_BE + 16 * m + 4 * g);
            const uint32_t p0 = pack_bf2(y[0], y[1]), p1 = pack_bf2(y[2], y[3]);
            char* dst = buf + L::V + (16 * m + 4 * g) * 128 + 2 * (16 * w + jj);
            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)p0;
            *reinterpret_cast<uint16_t*>(dst + 128) = (uint16_t)(p0 >> 16);
            *reinterpret_cast<uint16_t*>(dst + 256) = (uint16_t)p1;
            *reinterpret_cast<uint16_t*>(dst + 384) = (uint16_t)(p1 >> 16);
            dx[m] = y;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int i = 32 * q + (lane >> 1);
            const u32x4 y = *reinterpret_cast<const u32x4*>(buf + L::V + i * 128 + 32 * w + 16 * (lane & 1));
            if (i < rows)
                *reinterpret_cast<u32x4*>(p.dv + ((row * p.T + bos + (int64_t)c * CH + i) * p.Hv + hv) * DK + 64 * sl +
                                          16 * w + 8 * (lane & 1)) = y;
        }
        // dS <- e^{G_last} dS + Q^T (scale e^G do) - K^T (e^G dv)
        Split<3> qb[2], kb[2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const f32x4 e0 = *reinterpret_cast<const f32x4*>(sc + SC_EG + 32 * kk + 4 * g);
            const f32x4 e1 = *reinterpret_cast<const f32x4*>(sc + SC_EG + 32 * kk + 16 + 4 * g);
            qb[kk] = split_acc<3>((p.scale * e0) * widen(d[2 * kk]), (p.scale * e1) * widen(d[2 * kk + 1]));
            kb[kk] = split_acc<3>(-(e0 * dx[2 * kk]), -(e1 * dx[2 * kk + 1]));
        }
        const float el = sc[SC_EL];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            f32x4 a = S[t] * el;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const bf16x8 fq[1] = {col_frag(sQ, t, kk, g, jj)}, fk[1] = {col_frag(sK, t, kk, g, jj)};
                a = mfma_split<3>(fq, qb[kk], a);
                a = mfma_split<3>(fk, kb[kk], a);
            }
            S[t] = a;
        }
    }
    if (p.dh0) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) p.dh0[so + state_row(t, g, r) * DK] = S[t][r];
        }
    }
}

hipError_t launch_gdr_bwd(const GdrParams& p, int cus, hipStream_t stream) {
    const unsigned blocks = (unsigned)((int64_t)p.N * p.Hv * 2);
    hipError_t e = launch_gdr_prep(p, true, stream);
    if (e != hipSuccess) return e;
    if (p.nslots > 0) {
        hipLaunchKernelGGL(kda_gdr_keep_kernel, dim3(blocks), dim3(SCAN_THREADS), 0, stream, p);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kda_gdr_rscan_kernel, dim3(blocks), dim3(SCAN_THREADS), 0, stream, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    return launch_gdr_grads(p, cus, stream);
}

}  // namespace kda
