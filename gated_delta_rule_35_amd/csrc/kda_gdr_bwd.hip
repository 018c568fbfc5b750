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
//
// At B=2 H=64 T=8192 both walks are bound by HBM: forwards 487 us, 2.47 GB at 5.1 TB/s, of
// which 1.6 GB are S and u; reverse 675 us, 3.3 GB at 4.9 TB/s.  With few sequences and heads
// they are bound by the chain of a chunk: at T=1000 on 8 heads 44 and 61 us, 2.8 and 3.8 us
// a chunk.  There the order of the matrix instructions counts: four to six tiles side by
// side with the next operands read and split meanwhile took the reverse walk from 70 to 62
// us; T and A placed so that their transposed reads meet each bank twice instead of four
// times are part of it.
#include "kda_gdr_device.h"

namespace kda {

namespace {

constexpr int SCAN_THREADS = 384;   // four waves that compute, two that load
// One LDS buffer: K, Q tiles (swizzled), the slice of v (or of do) [64][64] bf16, the record.
struct ScanL {
    static constexpr int K = 0, Q = 16384, V = 32768, REC = 40960, BYTES = REC + GDR_REC;
};

// Fragment (m, kk) of the transposed matrix (rows 16 m + jj, k step kk), kk >= m / 2.
__device__ __forceinline__ bf16x8 tri_col_frag(const char* part, int m, int kk, int g, int jj) {
    const int at = frag_piece(16 * (jj & 3) + 4 * g + (jj >> 2)) + 8 * (m & 1);
    return join(lds_tr(part + tri_frag(2 * kk, m >> 1) * GDR_FRAG + at),
                lds_tr(part + tri_frag(2 * kk + 1, m >> 1) * GDR_FRAG + at));
}

// a[m] = rows 16 m .. of the tile times S, four tiles side by side, while the next step's
// operands are read and split; S is stored first, by all waves at once (two waves make up a
// 128-byte line): spread over the products, the stores cost the keeping walk at B=2 H=64
// T=8192 580 us for 460 to 500 and the reverse walk 735 for 680.
__device__ __forceinline__ void tile_times_state(const char* tile, const f32x4 (&S)[8], f32x4 (&a)[4], float* dst, int g,
                                                 int jj) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) dst[state_row(t, g, r) * DK] = S[t][r];
    }
    bf16x8 f[2][4];
    u32x4 sb[2][3];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        a[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        f[0][m] = row_frag(tile, m, 0, g, jj);
    }
    auto split = [&](int kk, int i) {
        const f32x4& s = S[2 * kk + (i >> 1)];
        split_pair<3>(sb[kk & 1], i, s[2 * (i & 1)], s[2 * (i & 1) + 1]);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) split(0, i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int n = 2; n >= 0; --n) {
            if (kk < 3) {
                if (n == 2) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) f[(kk + 1) & 1][m] = row_frag(tile, m, kk + 1, g, jj);
                    split(kk + 1, 0);
                } else {
                    split(kk + 1, 3 - n);
                }
                if (n == 0) split(kk + 1, 1);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) a[m] = mfma_bf(f[kk & 1][m], __builtin_bit_cast(bf16x8, sb[kk & 1][n]), a[m]);
            interleave<4, 5, 1, 1>();
        }
    }
}

// A choice made when compiling, as an argument.
template <bool X>
struct Bool {
    static constexpr bool value = X;
};

// One loading wave's (ld = 0, 1) half of a chunk's DMA into a buffer: 32 pieces of
// tiles and slices, and nrec of the record.
// PACED: with a pause of 64 clocks before each piece, so that the walking waves' stores need
// not wait for all of them (backward at T=1000 on 8 heads 157 -> 154 us; no change on full batches).
template <int NREC, bool WITH_Q, bool PACED>
__device__ __forceinline__ void load_chunk(const GdrParams& p, const Rows& vsrc, uint32_t lds, int64_t row, int64_t tok,
                                           int rows, int hq, int hv, int sl, int64_t slot, int ld, int lane) {
    typedef ScanL L;
    auto pause = [] {
        if (PACED) __builtin_amdgcn_s_sleep(1);
    };
    const __amdgpu_buffer_rsrc_t rk =
        chunk_rsrc(p.k.p + row * p.k.sb + tok * p.k.st + hq * p.k.sh, p.k.st, rows, DK);
    const int l4 = lane >> 4, l16 = lane & 15;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int r = 4 * (8 * ld + u) + l4;
        pause();
        dma_piece(rk, lds + L::K + (8 * ld + u) * 1024, (int)(r * p.k.st * 2) + ((l16 ^ tsw(4 * u + l4)) << 4));
    }
    if (WITH_Q) {
        const __amdgpu_buffer_rsrc_t rq =
            chunk_rsrc(p.q.p + row * p.q.sb + tok * p.q.st + hq * p.q.sh, p.q.st, rows, DK);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int r = 4 * (8 * ld + u) + l4;
            pause();
            dma_piece(rq, lds + L::Q + (8 * ld + u) * 1024, (int)(r * p.q.st * 2) + ((l16 ^ tsw(4 * u + l4)) << 4));
        }
    }
    const __amdgpu_buffer_rsrc_t rv =
        chunk_rsrc(vsrc.p + row * vsrc.sb + tok * vsrc.st + hv * vsrc.sh + 64 * sl, vsrc.st, rows, 64);
#pragma unroll
    for (int u = 0; u < 4; ++u) {   // eight rows a piece
        const int x = 4 * ld + u;
        pause();
        dma_piece(rv, lds + L::V + x * 1024, (int)((8 * x + (lane >> 3)) * vsrc.st * 2) + ((lane & 7) << 4));
    }
    const __amdgpu_buffer_rsrc_t rr =
        make_rsrc(p.rec + (slot * p.Hv + hv) * GDR_REC, GDR_REC);
#pragma unroll
    for (int u = 0; u < (NREC + 1) / 2; ++u) {
        const int x = 2 * u + ld;
        pause();
        if (x < NREC) dma_piece(rr, lds + L::REC + x * 1024, x * 1024 + lane * 16);
    }
}

}  // namespace

__global__ void __launch_bounds__(SCAN_THREADS) kda_gdr_keep_kernel(const GdrParams p) {
    typedef ScanL L;
    __shared__ __attribute__((aligned(1024))) char smem[2 * L::BYTES];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, jj = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Walk walk = walk_of_block<2>(p, (int)blockIdx.x, reinterpret_cast<int*>(smem));
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
        auto load = [&](int c, auto paced) {
            load_chunk<NREC, false, paced.value>(p, p.v, lds + (c & 1) * L::BYTES, row, bos + (int64_t)c * CH,
                                                 rows_of(c), hq, hv, sl, slot0 + c, w - 4, lane);
        };
        if (nch > 0) load(0, Bool<false>());
        for (int c = 0; c < nch; ++c) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's pieces of chunk c
            lds_barrier();
            if (c + 1 < nch) load(c + 1, Bool<true>());
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
        const char *sK = buf + L::K, *rec = buf + L::REC;
        const float* sc = reinterpret_cast<const float*>(rec + GDR_SC);
        // x = beta (v - e^G K S)
        f32x4 x[4];
        tile_times_state(sK, S, x, p.S + ((slot0 + c) * p.Hv + hv) * DK * DK + col, g, jj);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 eg = *reinterpret_cast<const f32x4*>(sc + SC_EG + 16 * m + 4 * g);
            const f32x4 be = *reinterpret_cast<const f32x4*>(sc + SC_BU + 16 * m + 4 * g);
            const f32x4 v = widen(slice_frag(buf + L::V, m, w, g, jj));
            x[m] = be * (v - eg * x[m]);
        }
        // u = T x
        const float el = sc[SC_EG + 63];
        f32x4 u[4];
        tri_times<false>(
            [&](int n3, int m, int kk) {
                return lds_bf8(rec + GDR_T + n3 * GDR_TRI + tri_frag(m, kk) * GDR_FRAG + frag_piece(lane));
            },
            x, u, [&](int n3) {
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    if (t % 3 == n3) S[t] *= el;
            });
        // S <- e^{G_last} S + K^T (e^{G_last - G} u)
        Split<3> wb[2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const f32x4 g0 = *reinterpret_cast<const f32x4*>(sc + SC_GA + 32 * kk + 4 * g);
            const f32x4 g1 = *reinterpret_cast<const f32x4*>(sc + SC_GA + 32 * kk + 16 + 4 * g);
            wb[kk] = split_acc<3>(g0 * u[2 * kk], g1 * u[2 * kk + 1]);
        }
        float* dst = p.u + ((slot0 + c) * p.Hv + hv) * CH * DK + col;
        bf16x8 f[2][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) f[0][t] = col_frag(sK, t, 0, g, jj);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // tiles 4 (i / 2) .., k step i & 1; u is stored meanwhile
            const int t0 = 4 * (i >> 1), kk = i & 1;
            if (i < 3) {
#pragma unroll
                for (int t = 0; t < 4; ++t) f[kk ^ 1][t] = col_frag(sK, 4 * ((i + 1) >> 1) + t, kk ^ 1, g, jj);
            }
#pragma unroll
            for (int n3 = 2; n3 >= 0; --n3) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r % 3 == n3) dst[(16 * i + 4 * g + r) * DK] = u[i][r];
#pragma unroll
                for (int t = 0; t < 4; ++t) S[t0 + t] = mfma_bf(f[kk][t], wb[kk].s[n3], S[t0 + t]);
                interleave<4, 2, 2, 1>();
            }
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
    const Walk walk = walk_of_block<2>(p, (int)blockIdx.x, reinterpret_cast<int*>(smem));
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
        auto load = [&](int c, auto paced) {
            load_chunk<NREC, true, paced.value>(p, p.dO, lds + (c & 1) * L::BYTES, row, bos + (int64_t)c * CH,
                                                 rows_of(c), hq, hv, sl, slot0 + c, w - 4, lane);
        };
        if (nch > 0) load(nch - 1, Bool<false>());
        for (int c = nch - 1; c >= 0; --c) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            lds_barrier();
            if (c > 0) load(c - 1, Bool<true>());
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
        u32x2 d[4];   // do, as it is: accumulator order and, in pairs, B operand
#pragma unroll
        for (int m = 0; m < 4; ++m) d[m] = slice_frag(buf + L::V, m, w, g, jj);
        // du = e^{G_last - G} (K dS) + A^T do, scale e^G do split meanwhile
        f32x4 du[4], eg[4], be[4];
        u32x4 qb[2][3], kb[2][3];
        tile_times_state(sK, S, du, p.dS + ((slot0 + c) * p.Hv + hv) * DK * DK + col, g, jj);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            du[m] *= *reinterpret_cast<const f32x4*>(sc + SC_GA + 16 * m + 4 * g);
            eg[m] = *reinterpret_cast<const f32x4*>(sc + SC_EG + 16 * m + 4 * g);
            be[m] = *reinterpret_cast<const f32x4*>(sc + SC_BE + 16 * m + 4 * g);
        }
        const float el = sc[SC_EG + 63];
        {
            const bf16x8 db[2] = {join(d[0], d[1]), join(d[2], d[3])};
            bf16x8 f[2][6];
            constexpr int M[6] = {0, 1, 2, 3, 0, 1}, KK[6] = {0, 0, 1, 1, 1, 1};
#pragma unroll
            for (int i = 0; i < 6; ++i) f[0][i] = tri_col_frag(rec + GDR_A + 2 * GDR_TRI, M[i], KK[i], g, jj);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n3 = 2; n3 >= 0; --n3) {
                if (n3) {
#pragma unroll
                    for (int i = 0; i < 6; ++i)
                        f[(n3 + 1) & 1][i] = tri_col_frag(rec + GDR_A + (n3 - 1) * GDR_TRI, M[i], KK[i], g, jj);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i % 3 != n3) continue;
                    const int m = i >> 1, e = 2 * (i & 1);
                    const f32x4 o = widen(d[m]);
                    split_pair<3>(qb[m >> 1], i & 3, (p.scale * eg[m][e]) * o[e], (p.scale * eg[m][e + 1]) * o[e + 1]);
                }
#pragma unroll
                for (int i = 0; i < 6; ++i) du[M[i]] = mfma_bf(f[n3 & 1][i], db[KK[i]], du[M[i]]);
                interleave<6, 7, 2, 0>();
            }
        }
        // dx = T^T du
        f32x4 dx[4];
        tri_times<true>([&](int n3, int m, int kk) { return tri_col_frag(rec + GDR_T + n3 * GDR_TRI, m, kk, g, jj); }, du,
                        dx, [&](int n3) {
#pragma unroll
                            for (int t = 0; t < 8; ++t)
                                if (t % 3 == n3) S[t] *= el;
                        });
        const int rows = rows_of(c);
        float* dst = p.dx + ((slot0 + c) * p.Hv + hv) * CH * DK + col;
        // dS <- e^{G_last} dS + Q^T (scale e^G do) - K^T (beta e^G dx), Q's part first;
        // dv = beta dx meanwhile, rounded once, through this wave's columns of the do slice
        bf16x8 f[2][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) f[0][t] = col_frag(sQ, t, 0, g, jj);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // Q's products, then K's; tiles 4 (i / 2 mod 2) .., k step i & 1
            const int t0 = 4 * ((i >> 1) & 1), kk = i & 1;
            if (i < 7) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    f[kk ^ 1][t] = col_frag(i + 1 < 4 ? sQ : sK, 4 * (((i + 1) >> 1) & 1) + t, kk ^ 1, g, jj);
            }
#pragma unroll
            for (int n3 = 2; n3 >= 0; --n3) {
                if (i < 4 && n3 == 2) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) dst[(16 * i + 4 * g + r) * DK] = dx[i][r];
                    dx[i] *= be[i];
                } else if (i < 4 && n3 == 1) {
                    const uint32_t p0 = pack_bf2(dx[i][0], dx[i][1]), p1 = pack_bf2(dx[i][2], dx[i][3]);
                    char* at = buf + L::V + (16 * i + 4 * g) * 128 + 2 * (16 * w + jj);
                    *reinterpret_cast<uint16_t*>(at) = (uint16_t)p0;
                    *reinterpret_cast<uint16_t*>(at + 128) = (uint16_t)(p0 >> 16);
                    *reinterpret_cast<uint16_t*>(at + 256) = (uint16_t)p1;
                    *reinterpret_cast<uint16_t*>(at + 384) = (uint16_t)(p1 >> 16);
                    split_pair<3>(kb[i >> 1], 2 * (i & 1), -(eg[i][0] * dx[i][0]), -(eg[i][1] * dx[i][1]));
                } else if (i < 4) {
                    split_pair<3>(kb[i >> 1], 2 * (i & 1) + 1, -(eg[i][2] * dx[i][2]), -(eg[i][3] * dx[i][3]));
                }
                if (i >= 4 && i < 6 && n3 == 2) {
                    asm volatile("" ::: "memory");   // the pieces written above, which LDS takes in order
                    const int j = 32 * (i - 4) + (lane >> 1);
                    const u32x4 y = *reinterpret_cast<const u32x4*>(buf + L::V + j * 128 + 32 * w + 16 * (lane & 1));
                    if (j < rows)
                        *reinterpret_cast<u32x4*>(p.dv + ((row * p.T + bos + (int64_t)c * CH + j) * p.Hv + hv) * DK +
                                                  64 * sl + 16 * w + 8 * (lane & 1)) = y;
                }
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    S[t0 + t] = mfma_bf(f[kk][t], __builtin_bit_cast(bf16x8, (i < 4 ? qb : kb)[kk][n3]), S[t0 + t]);
                interleave<4, 4, 2, 1>();
            }
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
