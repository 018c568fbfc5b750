// The forward's walk over the chunks of the gated delta rule with one decay per head, on
// gfx950 (MI355X).  With the prep kernel's T (its columns times beta) and per-token numbers:
//   x = v - e^G K S,  u = T x,  o = scale (e^G Q S + A u),  A = e^{G_i - G_j} Q K^T, j <= i
//   S <- e^{G_last} S + K^T (e^{G_last - G} u)
//
// Every product's right-hand side is a set of columns of S (value channels), and no
// product mixes columns: a wave owns 16 of them for the whole sequence and needs nothing
// from the others.  Its state is eight 16x16 accumulator tiles (32 registers a lane), and
// since an accumulator tile holds what a lane needs as B operand, the whole chain of a
// chunk stays in registers.  A work-group is four such waves (half a head, 64 value
// channels) or eight, and four more that bring the next chunk's k, q, v, T and numbers into
// LDS by DMA, store the last chunk's o and form this chunk's A: ten tiles, needed only
// once u is known, so that the walking waves meet them at a second barrier there.
// Tile t = 2 kk + h of the state holds key channel 32 kk + 8 g + 4 h + r in row 4 g + r
// (g = lane / 16), so that the two tiles of a 32-channel step list the lane's eight
// channels as they lie in K's rows.
//
// Precision.  fp32 operands enter as bf16 parts: S, x, u and T in three (24 bits at any
// size: nothing has to be scaled, and what overflows fp32 alone overflows), what A u adds to
// o, and S in Q S, in two parts of each (16 bits; o is rounded to bf16's eight).
//   fp16 parts, two of which hold 22 bits, need 132 matrix instructions a chunk for these
// 182 and two thirds of the vector ones, but k and q as fp16, whose range takes a power of
// two for each row, chunk and value channel, windows in which small entries lose bits, and
// waves that turn k and q: with A in two parts those were busy 7,500 of a chunk's 8,460 clocks.
//
// At B=2 H=64 T=8192 the walk takes 490 us (a warm kernel trace's median), 1.43 GB at 2.9 TB/s:
// 7,400 clocks a chunk at 1.95 GHz, matrix units busy 41%, LDS 50%.  It is bound by what one
// wave a SIMD can issue: 984 instructions a chunk, 182 of them matrix (9.7 clocks each with
// vector ones between), 563 vector (4.4 each, whether they depend on each other or not), 110
// LDS reads; 400 of the vector ones split S, x and u.  With 64 work-groups on the chip, no
// DMA, no A or neither, a chunk takes as long to within 5%.
#include "kda_gdr_device.h"

namespace kda {

namespace {

// A, and two slots of what comes by DMA: K, Q tiles (swizzled), the record, v's slices [64][64]
// (o's on the way out), one for each half of a head that the work-group walks.
template <int HALVES>
struct FL {
    static constexpr int A = 0, SLOTS = 2 * GDR_TRI;
    static constexpr int K = 0, Q = 16384, REC = 32768, V = REC + FWD_REC, SLOT = V + HALVES * 8192;
    static constexpr int BYTES = SLOTS + 2 * SLOT;
    static constexpr int THREADS = 256 * HALVES + 256;
};

template <int N>
struct Part {
    static constexpr int value = N;
};
__device__ __forceinline__ f32x4 sc4(const float* sc, int row, int m, int g) {
    return *reinterpret_cast<const f32x4*>(sc + row + 16 * m + 4 * g);
}
}  // namespace

template <int HALVES>
__global__ void __launch_bounds__(FL<HALVES>::THREADS) kda_gdr_scan_kernel(const GdrParams p) {
    typedef FL<HALVES> L;
    __shared__ __attribute__((aligned(1024))) char smem[L::BYTES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Walk walk = walk_of_block<2 / HALVES>(p, (int)blockIdx.x, reinterpret_cast<int*>(smem));
    const int n = walk.n, hv = walk.hv, sl = walk.sl, hq = hv / (p.Hv / p.Hq);
    int64_t bos, len, row, slot0;
    gdr_seq(p, n, bos, len, row, slot0);
    const int nch = (int)((len + CH - 1) / CH);
    auto rows_of = [&](int c) -> int {
        const int64_t r = len - (int64_t)c * CH;
        return r <= 0 ? 0 : (r >= CH ? CH : (int)r);
    };

    if (wave >= 4 * HALVES) {
        // ================= the waves that load, store and form A =================
        const int w = wave - 4 * HALVES, g = lane >> 4, jj = lane & 15;
        const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));
        // Rows 4 w + 16 x + lane / 16, x < 4, of k and q, and 8 (2 w + u) + lane / 8, u < 2, of v's
        // slices, whose o this wave also stores; a quarter of the record.
        auto dma = [&](int c) {
            const int rows = rows_of(c), r = 4 * w + g;
            const int64_t tok = bos + (int64_t)c * CH;
            const uint32_t to = lds + L::SLOTS + (c & 1) * L::SLOT;
            auto tile = [&](const Rows& t, uint32_t at) {
                const __amdgpu_buffer_rsrc_t rs = chunk_rsrc(t.p + row * t.sb + tok * t.st + hq * t.sh, t.st, rows, DK);
                const int st = (int)t.st * 2, off = r * st + ((jj ^ tsw(r)) << 4);   // 16 rows on, tsw is the same
#pragma unroll
                for (int x = 0; x < 4; ++x) dma_piece(rs, at + (w + 4 * x) * 1024, off + 16 * x * st);
            };
            tile(p.k, to + L::K);
            tile(p.q, to + L::Q);
            const __amdgpu_buffer_rsrc_t rv =
                chunk_rsrc(p.v.p + row * p.v.sb + tok * p.v.st + hv * p.v.sh + 64 * sl, p.v.st, rows, 64 * HALVES);
            const int st = (int)p.v.st * 2, off = (16 * w + (lane >> 3)) * st + ((lane & 7) << 4);
#pragma unroll
            for (int u = 0; u < 2 * HALVES; ++u)
                dma_piece(rv, to + L::V + (u >> 1) * 8192 + (2 * w + (u & 1)) * 1024, off + 8 * (u & 1) * st + 128 * (u >> 1));
            const __amdgpu_buffer_rsrc_t rr = make_rsrc(p.rec + ((slot0 + c) * p.Hv + hv) * FWD_REC, FWD_REC);
#pragma unroll
            for (int u = 0; u < FWD_REC / 4096; ++u)
                dma_piece(rr, to + L::REC + (4 * u + w) * 1024, (4 * u + w) * 1024 + lane * 16);
        };
        auto store_o = [&](int c) {   // 64 rows of 64 channels each where v was
            const int rows = rows_of(c);
            const char* tv = smem + L::SLOTS + (c & 1) * L::SLOT + L::V;
            u32x4 y[2 * HALVES];
#pragma unroll
            for (int u = 0; u < 2 * HALVES; ++u)
                y[u] = *reinterpret_cast<const u32x4*>(tv + (u >> 1) * 8192 + (2 * w + (u & 1)) * 1024 + lane * 16);
#pragma unroll
            for (int u = 0; u < 2 * HALVES; ++u) {
                const int i = 8 * (2 * w + (u & 1)) + (lane >> 3);
                if (i < rows)
                    *reinterpret_cast<u32x4*>(p.o + ((row * p.T + bos + (int64_t)c * CH + i) * p.Hv + hv) * DK + 64 * sl +
                                              64 * (u >> 1) + 8 * (lane & 7)) = y[u];
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the DMA of what comes there
        };
        // A of chunk c in two bf16 parts: wave 0 the tiles (3,0) (3,1), 1 (3,2) (3,3), 2 (2,0) (2,1)
        // (2,2), 3 (1,0) (1,1) (0,0).  Formed transposed, a lane holds one row and four columns, as
        // the operand fragments do.
        auto form_a = [&](int c) {
            const char *tk = smem + L::SLOTS + (c & 1) * L::SLOT + L::K, *tq = tk + L::Q;
            const float* sc = reinterpret_cast<const float*>(tk + L::REC + GDR_SC);
            auto raw = [&](const bf16x8 (&q)[4], const bf16x8 (&k)[4]) -> f32x4 {
                f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) a = mfma_bf(k[kk], q[kk], a);
                return a;
            };
            auto rows4 = [&](const char* tile, int m, bf16x8 (&to)[4]) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) to[kk] = row_frag(tile, m, kk, g, jj);
            };
            auto put = [&](int I, int J, f32x4 a) {
                const int i = 16 * I + jj;
                const float hi = sc[SC_GH + i], lo = sc[SC_GL + i];
                const f32x4 hj = sc4(sc, SC_GH, J, g), lj = sc4(sc, SC_GL, J, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] *= fexp2((hi - hj[e]) + (lo - lj[e]));
                if (I == J) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = 4 * g + e <= jj ? a[e] : 0.f;
                }
                char* to = smem + L::A + (I < 2 ? I : 2 * I - 2 + (J >> 1)) * GDR_FRAG + lane * 16 + 8 * (J & 1);
                const uint32_t h0 = pack_bf2(a[0], a[1]), h1 = pack_bf2(a[2], a[3]);
                *reinterpret_cast<u32x2*>(to) = u32x2{h0, h1};
                *reinterpret_cast<u32x2*>(to + GDR_TRI) =
                    u32x2{pack_bf2(a[0] - bf_lo(h0), a[1] - bf_hi(h0)), pack_bf2(a[2] - bf_lo(h1), a[3] - bf_hi(h1))};
            };
            const int I = w < 2 ? 3 : 4 - w, J = w == 1 ? 2 : 0;   // tiles (I, J), (I, J + 1), and one more of waves 2 and 3
            bf16x8 q[4], k0[4], k1[4];
            rows4(tq, I, q);
            rows4(tk, J, k0);
            rows4(tk, J + 1, k1);
            const f32x4 a0 = raw(q, k0), a1 = raw(q, k1);
            f32x4 a2;
            if (w == 2) rows4(tk, 2, k0);
            else rows4(tq, 0, q);
            if (w >= 2) a2 = raw(q, k0);
            put(I, J, a0);
            put(I, J + 1, a1);
            if (w >= 2) put(w == 2 ? 2 : 0, w == 2 ? 2 : 0, a2);
        };
        // what lies above the diagonal in fragments (0, 0) and (2, 1): columns 16 .. 31 of each
        *reinterpret_cast<u32x2*>(smem + L::A + (w >> 1) * GDR_TRI + 3 * (w & 1) * GDR_FRAG + lane * 16 + 8) = u32x2{0, 0};
        if (nch > 0) dma(0);
        for (int c = 0; c < nch; ++c) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's pieces of chunk c
            lds_barrier();
            form_a(c);
            if (c > 0) store_o(c - 1);
            if (c + 1 < nch) dma(c + 1);
            lds_barrier();   // A is in LDS
        }
        lds_barrier();
        if (nch > 0) store_o(nch - 1);
        return;
    }

    // ================= walking waves =================
    __builtin_amdgcn_s_setprio(3);
    const int w = wave & 3;   // sixteen columns of half wave / 4 of those that the work-group walks
    const int64_t so = ((int64_t)n * p.Hv + hv) * DK * DK + 64 * sl + 16 * wave + (lane & 15);
    f32x4 S[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = p.h0 ? p.h0[so + state_row(t, lane >> 4, r) * DK] : 0.f;
    }
    constexpr bool KEEP = HALVES == 1;
    u32x4 sb[KEEP ? 4 : 2][3];   // S's parts by k step
    auto split_s = [&](int kk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4& s = S[2 * kk + (i >> 1)];
            split_pair<3>(sb[kk & (KEEP ? 3 : 1)], i, s[2 * (i & 1)], s[2 * (i & 1) + 1]);
        }
    };
    if (KEEP) split_s(0);
    for (int c = 0; c < nch; ++c) {
        lds_barrier();   // chunk c is in LDS, and the other slot's reads are done
        const int ln = KEEP ? lane : opaque(lane), g = ln >> 4, jj = ln & 15;   // whole heads: addresses formed anew
        const char *tk = smem + L::SLOTS + (c & 1) * L::SLOT + L::K, *tq = tk + L::Q, *rec = tk + L::REC;
        char* tv = smem + L::SLOTS + (c & 1) * L::SLOT + L::V + (wave >> 2) * 8192;
        const float* sc = reinterpret_cast<const float*>(rec + GDR_SC);
        // x = v - e^G K S in parts, and Q S.  Half heads have the registers to keep S's parts:
        // K S first, and Q S while x is formed and split.  Whole heads' two walks a SIMD fill each
        // other's gaps: K S and Q S a k step at a time.
        f32x4 x[4], o[4];
        Split<3> xb[2];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = o[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto products = [&](auto top, const bf16x8 (&f)[4], const u32x4 (&parts)[3], f32x4 (&a)[4]) {
#pragma unroll
            for (int s = top.value; s >= 0; --s) {
#pragma unroll
                for (int m = 0; m < 4; ++m) a[m] = mfma_bf(f[m], __builtin_bit_cast(bf16x8, parts[s]), a[m]);
            }
        };
        auto rows4 = [&](const char* tile, int kk, bf16x8 (&f)[4]) {
#pragma unroll
            for (int m = 0; m < 4; ++m) f[m] = row_frag(tile, m, kk, g, jj);
        };
        auto form_x = [&](int m) {
            x[m] = widen(slice_frag(tv, m, w, g, jj)) - sc4(sc, SC_EG, m, g) * x[m];
        };
        auto split_x = [&](int h) { xb[h] = split_acc<3>(x[2 * h], x[2 * h + 1]); };
        if (KEEP) {
            bf16x8 f[2][4];
            rows4(tk, 0, f[0]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                if (kk < 3) {
                    rows4(tk, kk + 1, f[(kk + 1) & 1]);
                    split_s(kk + 1);
                } else {
                    rows4(tq, 0, f[0]);
                }
                products(Part<2>(), f[kk & 1], sb[kk & (KEEP ? 3 : 1)], x);
                interleave<12, 4, 1, 0>();
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                if (kk < 3) rows4(tq, kk + 1, f[(kk + 1) & 1]);
                if (kk & 1) {
                    split_x(kk >> 1);
                } else {
                    form_x(kk);
                    form_x(kk + 1);
                }
                products(Part<1>(), f[kk & 1], sb[kk & (KEEP ? 3 : 1)], o);
                interleave<8, 5, 1, 0>();
            }
        } else {
            bf16x8 fk[4], fq[4];
            rows4(tk, 0, fk);
            split_s(0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                rows4(tq, kk, fq);
                products(Part<2>(), fk, sb[kk & (KEEP ? 3 : 1)], x);
                interleave<12, 0, 1, 0>();
                if (kk < 3) {
                    rows4(tk, kk + 1, fk);
                    split_s(kk + 1);
                }
                products(Part<1>(), fq, sb[kk & (KEEP ? 3 : 1)], o);
                interleave<8, 5, 1, 0>();
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) form_x(m);
            split_x(0);
            split_x(1);
        }
        // u = T x: tiles of the parts' products of 2^-16 and more of the leading one's, the small
        // parts first, in two chains each; tokens 0 .. 31 first, so that what they become is split
        // beside the others' products
        const float el = sc[SC_EG + 63];
        auto t_frag = [&](int part, int m, int kk) {
            return lds_bf8(rec + GDR_T + part * GDR_TRI + tri_frag(m, kk) * GDR_FRAG + frag_piece(ln));
        };
        Split<3> wb[2];
        Split<2> ub[2];
        auto split_u = [&](int h, const f32x4& u0, const f32x4& u1) {   // u, and e^{G_last - G} u
            ub[h] = split_acc<2>(u0, u1);
            wb[h] = split_acc<3>(sc4(sc, SC_GA, 2 * h, g) * u0, sc4(sc, SC_GA, 2 * h + 1, g) * u1);
        };
        {
            f32x4 a[4], b[4];
            bf16x8 t[3][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = b[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int part = 0; part < 3; ++part) t[part][i] = t_frag(part, i, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            bf16x8 f[2][4];   // (2, 0) (3, 0) (2, 1) (3, 1)
            auto load = [&](int part) {
#pragma unroll
                for (int i = 0; i < 4; ++i) f[part & 1][i] = t_frag(part, 2 + (i & 1), i >> 1);
            };
            load(2);
#pragma unroll
            for (int y = 0; y < 6; ++y) {   // (2,0) (1,1) (0,2) in one chain, (1,0) (0,1) (0,0) in the other
                constexpr int TP[6] = {2, 1, 1, 0, 0, 0}, XP[6] = {0, 0, 1, 1, 2, 0};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f32x4& to = y == 1 || y == 3 || y == 5 ? b[i] : a[i];
                    to = mfma_bf(t[TP[y]][i], xb[0].s[XP[y]], to);
                }
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) S[n] *= el;
            interleave<12, 3, 1, 0>();
            const f32x4 u0 = a[0] + b[0], u1 = a[1] + b[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            split_u(0, u0, u1);
#pragma unroll
            for (int part = 2; part >= 0; --part) {
                if (part) load(part - 1);
#pragma unroll
                for (int d = 2 - part; d >= 0; --d) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = mfma_bf(f[part & 1][i], xb[i >> 1].s[d], a[i]);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) o[m] *= sc4(sc, SC_EG, m, g);
            interleave<24, 4, 1, 0>();
            x[2] = a[0] + a[2];
            x[3] = a[1] + a[3];
        }
        // S <- e^{G_last} S + K^T (e^{G_last - G} u), four tiles side by side; beside them A u, small
        // parts first, and o, rounded once, into this wave's columns of v's slice: the other waves
        // store it
        {
            bf16x8 f[2][4], fa[6];
            constexpr int TM[6] = {0, 1, 2, 3, 2, 3}, TK[6] = {0, 0, 0, 0, 1, 1};   // fragments (m, kk) of A
            auto a_frags = [&](int part) {
#pragma unroll
                for (int i = 0; i < 6; ++i)
                    fa[i] = lds_bf8(smem + L::A + part * GDR_TRI + tri_frag(TM[i], TK[i]) * GDR_FRAG + ln * 16);
            };
            auto a_times_u = [&](int part, int from, int to) {
#pragma unroll
                for (int y = from; y < to; ++y) o[TM[y]] = mfma_bf(fa[y], ub[TK[y]].s[part], o[TM[y]]);
            };
            auto columns = [&](int i, bf16x8 (&to)[4]) {   // of step i: tiles 4 (i & 1) .., k step i / 2
#pragma unroll
                for (int t = 0; t < 4; ++t) to[t] = col_frag(tk, 4 * (i & 1) + t, i >> 1, g, jj);
            };
            columns(0, f[0]);
            lds_barrier();   // A is in LDS
            a_frags(1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t0 = 4 * (i & 1), kk = i >> 1;
                if (i < 3) columns(i + 1, f[(i + 1) & 1]);
                if (i == 0) split_u(1, x[2], x[3]);
                if (i == 3) a_times_u(0, 0, 6);
#pragma unroll
                for (int s = 2; s >= 0; --s) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) S[t0 + t] = mfma_bf(f[i & 1][t], wb[kk].s[s], S[t0 + t]);
                }
                if (i == 0) {
                    a_times_u(0, 0, 4);
                    interleave<16, 5, 1, 0>();
                } else if (i == 1) {
                    a_times_u(0, 4, 6);
                    a_frags(0);
                    interleave<14, 1, 1, 0>();
                } else if (i == 2) {
                    a_times_u(1, 0, 6);
                    interleave<18, 1, 1, 0>();
                } else {
                    if (KEEP) split_s(0);   // for the next chunk
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        o[m] *= p.scale;
                        const uint32_t p0 = pack_bf2(o[m][0], o[m][1]), p1 = pack_bf2(o[m][2], o[m][3]);
                        char* dst = tv + (16 * m + 4 * g) * 128 + 2 * (16 * w + jj);
                        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)p0;
                        *reinterpret_cast<uint16_t*>(dst + 128) = (uint16_t)(p0 >> 16);
                        *reinterpret_cast<uint16_t*>(dst + 256) = (uint16_t)p1;
                        *reinterpret_cast<uint16_t*>(dst + 384) = (uint16_t)(p1 >> 16);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }
    lds_barrier();   // the last chunk's o is complete
    if (p.hT) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) p.hT[so + state_row(t, lane >> 4, r) * DK] = S[t][r];
        }
    }
}

hipError_t launch_gdr_fwd(const GdrParams& p, int cus, hipStream_t stream) {
    hipError_t e = launch_gdr_prep(p, false, stream);
    if (e != hipSuccess) return e;
    // Whole heads share the staging of k, q and T and A's tiles, and two of their walks a SIMD fill
    // each other's gaps: 1.8 times a half's time, worth it where heads alone fill the compute
    // units and no sequence is much longer than the others, for packed ones taken to be so with
    // four times as many.  Halves and whole heads: 596 and 542 us at B=4 H=64 T=4096, 162 and
    // 149 at B=32 H=16 T=512, 760 and 695 at 64 packed sequences of 256 tokens and 64 heads; but
    // 598 and 745 at B=2 H=64 T=8192, 574 and 611 at 11 of 16,384 tokens together and 64 heads, the
    // longest half of them.
    const int64_t heads = (int64_t)p.N * p.Hv;
    if (heads >= (p.cu ? 4 * (int64_t)cus : cus))
        hipLaunchKernelGGL(kda_gdr_scan_kernel<2>, dim3((unsigned)heads), dim3(FL<2>::THREADS), 0, stream, p);
    else
        hipLaunchKernelGGL(kda_gdr_scan_kernel<1>, dim3((unsigned)(2 * heads)), dim3(FL<1>::THREADS), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
