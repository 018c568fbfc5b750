// The forward's walk over the chunks of the gated delta rule with one decay per head, on
// gfx950 (MI355X).  With the prep kernel's T, A (fp16 fragments) and per-token numbers:
//   x = beta (v - e^G K S),  u = T x,  o = scale (e^G Q S + A u)
//   S <- e^{G_last} S + K^T (e^{G_last - G} u)
//
// Every product's right-hand side is a set of columns of S (value channels), and no
// product mixes columns: a wave owns 16 of them for the whole sequence and needs nothing
// from the others.  Its state is eight 16x16 accumulator tiles (32 registers a lane), and
// since an accumulator tile holds what a lane needs as B operand, the whole chain of a
// chunk stays in registers.  A work-group is four such waves (half a head, 64 value
// channels) or eight, and four that stage the next chunk's left-hand operands in LDS: k and
// q rows as fp16, v, T and A by DMA; one barrier a chunk.  Tile t = 2 kk + h of the state holds key channel
// 32 kk + 8 g + 4 h + r in row 4 g + r (g = lane / 16), so that the two tiles of a
// 32-channel step list the lane's eight channels as they lie in K's rows.
//
// Precision.  All products run on v_mfma_f32_16x16x32_f16.  k and q rows enter divided by
// a power of two that brings their largest entry into [1, 2): exact for entries down to
// 2^-14 of that, and off by 2^-25 of it below.  S, x, u and T enter as two fp16 parts, 22
// bits, so that the state keeps fp32's accuracy with two thirds of the matrix work of
// three bf16 parts and a fifth of fp32 instructions'; what only reaches the bf16 output
// (S in Q S, A, u in A u) enters as one part, eight times finer than o's own rounding.
// fp16's range is met by powers of two.  x and u are those of the rows times 2^ek / kap,
// 2^ek the power that divides the row's key and `kap` the chunk's largest, by which S is
// divided: what a key adds to S, and what it reads of it, then have S's units, and T's
// entries stay below 46 (kda_gdr_prep.hip).  One more for each value channel (each lane's
// column) keeps the largest |S| / kap and |beta v| 2^ek / kap within [2^2, 2^10] when a
// chunk starts; with beta |k|^2 <= 2, where the update does not expand the state,
// |x| <= 2^10 + beta 2^2ek |k^| |k^ . S| <= 2^10 + 2 128^{1/2} 2^10 < 2^15.  u can be 128 |k^|
// times larger where keys repeat (beta 2 and values of alternating signs: the state grows
// by 2 |v| a token): past 2^15 the column is scaled down, and what the chunk's end keeps is
// scaled up where it is far less than what it started with, before S is formed anew; all
// change rarely.  An entry keeps its 22 bits down to 2^-4 to 2^-12 of the largest, and is
// off by 2^-25 in these units below that, 2^-27 to 2^-35 of the largest.
//
// At B=2 H=64 T=8192 the walk takes 370 us, 1.43 GB at 3.9 TB/s: 5,300 clocks a chunk, the
// chain of its products (gate and window 900, K S and Q S 1,700, T x 700, S and o 2,000),
// where four waves' reads of the same operands keep LDS busy half of the time and splits and
// matrix instructions share the issue.  A chunk takes nearly as long when only 16 work-groups
// run, and 2% less without the staging waves' conversions.  Products of four tiles side by
// side, v, T and A by DMA two chunks ahead, the walking waves' priority and inverses of
// powers of two by integer subtraction brought 586 us of the whole call to 560.
#include "kda_gdr_device.h"

namespace kda {

namespace {

// Two slots of what passes through the staging waves' registers: K, Q tiles (fp16, swizzled)
// and per-token numbers; of what comes by DMA three, a chunk further ahead, or two where
// there is no room for more: T and A fragments, and v's slices [64][64] bf16 (o's on the way
// out), one for each half of a head that the work-group walks.
template <int HALVES>
struct FL {
    static constexpr int K = 0, Q = 16384, SC = 32768, STAGED = SC + FWD_ROWS * 256;
    static constexpr int T = 0, A = T + 2 * GDR_TRI, V = A + GDR_TRI, DMA = V + HALVES * 8192;
    static constexpr int SLOTS = HALVES == 1 ? 3 : 2, BYTES = 2 * STAGED + SLOTS * DMA;
    static constexpr int THREADS = 256 * HALVES + 256;
};

// Channel of row 4 g + r of state tile t.
__device__ __forceinline__ int state_row(int t, int g, int r) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1) + r; }
// A operand (m, kk) of a tile: rows 16 m + jj, channels 32 kk + 8 g ..
__device__ __forceinline__ half8 row_frag(const char* tile, int m, int kk, int g, int jj) {
    return *reinterpret_cast<const half8*>(tile + tile_off(16 * m + jj, 4 * kk + g));
}
// A operand of the transposed tile: state tile t's channels, tokens of k step kk.
__device__ __forceinline__ half8 col_frag(const char* tile, int t, int kk, int g, int jj) {
    const int row = 32 * kk + 4 * g + (jj >> 2), piece = 4 * (t >> 1) + (jj & 3), b = 8 * (t & 1);
    return __builtin_bit_cast(half8, join(lds_tr(tile + tile_off(row, piece) + b), lds_tr(tile + tile_off(row + 16, piece) + b)));
}
__device__ __forceinline__ constexpr int tri_frag(int m, int kk) { return m < 2 ? m : 2 * m - 2 + kk; }
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
    auto record = [&](int c) -> const char* { return p.rec + ((slot0 + c) * p.Hv + hv) * FWD_REC; };
    float kap = 1.f;   // of the chunk at hand; a chunk of zero keys keeps the one before

    if (wave >= 4 * HALVES) {
        // ================= staging waves =================
        const int w = wave - 4 * HALVES;
        const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));
        i32x4 kr[4], qr[4];   // rows 4 w + l / 16 (mod 16) of the next chunk: one 16-byte piece a lane
        float kp, qp, km, sc[2];
        // Rows 16 w + 4 x + lane / 16, piece lane % 16 of the next chunk's k and q, and (lane
        // for token) what they are divided by; two of the eight rows of numbers.
        auto fetch = [&](int c) {
            const int ln = opaque(lane), rows = rows_of(c);
            const int64_t tok = bos + (int64_t)c * CH;
            const __amdgpu_buffer_rsrc_t rk =
                chunk_rsrc(p.k.p + row * p.k.sb + tok * p.k.st + hq * p.k.sh, p.k.st, rows, DK);
            const __amdgpu_buffer_rsrc_t rq =
                chunk_rsrc(p.q.p + row * p.q.sb + tok * p.q.st + hq * p.q.sh, p.q.st, rows, DK);
            const int r = 16 * w + (ln >> 4), b = 16 * (ln & 15);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                kr[x] = __builtin_amdgcn_raw_buffer_load_b128(rk, (int)((r + 4 * x) * p.k.st * 2) + b, 0, 0);
                qr[x] = __builtin_amdgcn_raw_buffer_load_b128(rq, (int)((r + 4 * x) * p.q.st * 2) + b, 0, 0);
            }
            const float* s = reinterpret_cast<const float*>(record(c) + FWD_SC);
            kp = s[SC_KS + ln];
            qp = s[SC_QS + ln];
            km = s[SC_KP + ln];   // a vector load like the others: they are counted
            sc[0] = s[128 * w + ln];
            sc[1] = s[128 * w + 64 + ln];
        };
        auto dma = [&](int c, int slot) {   // v, T and A
            const int ln = opaque(lane);
            const uint32_t to = lds + 2 * L::STAGED + slot * L::DMA;
            const __amdgpu_buffer_rsrc_t rv =
                chunk_rsrc(p.v.p + row * p.v.sb + (bos + (int64_t)c * CH) * p.v.st + hv * p.v.sh + 64 * sl, p.v.st,
                           rows_of(c), 64 * HALVES);
#pragma unroll
            for (int u = 0; u < 2 * HALVES; ++u)
                dma_piece(rv, to + L::V + (u >> 1) * 8192 + (2 * w + (u & 1)) * 1024,
                          (int)((8 * (2 * w + (u & 1)) + (ln >> 3)) * p.v.st * 2) + 128 * (u >> 1) + ((ln & 7) << 4));
            const __amdgpu_buffer_rsrc_t rr = make_rsrc(record(c), FWD_SC);
#pragma unroll
            for (int u = 0; u < 5; ++u) {   // eighteen pieces
                const int x = 4 * u + w;
                if (x < 18) dma_piece(rr, to + L::T + x * 1024, x * 1024 + ln * 16);
            }
        };
        // 16 bytes of bf16 times `by` as fp16
        auto to_half = [&](const i32x4& raw, float by) -> u32x4 {
            u32x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t v = (uint32_t)raw[i];
                h[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{bf_lo(v) * by, bf_hi(v) * by}, half2v));
            }
            return h;
        };
        auto stage = [&](int c) {
            const int ln = opaque(lane), r = 16 * w + (ln >> 4);
            char* to = smem + (c & 1) * L::STAGED;
            float* out = reinterpret_cast<float*>(to + L::SC);
            const float kinv = kp > 0.f ? inverse2(kp) : 1.f, qinv = inverse2(qp);
            if (km > 0.f) kap = km;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int at = tile_off(r + 4 * x, ln & 15);
                *reinterpret_cast<u32x4*>(to + L::K + at) = to_half(kr[x], __shfl(kinv, r + 4 * x));
                *reinterpret_cast<u32x4*>(to + L::Q + at) = to_half(qr[x], __shfl(qinv, r + 4 * x));
            }
            out[128 * w + ln] = sc[0] * (w == 1 ? inverse2(kap) : 1.f);   // row 2: beta 2^ek / kap
            out[128 * w + 64 + ln] = sc[1];
        };
        if (nch > 0) {
            dma(0, 0);
            fetch(0);
            stage(0);
            if (nch > 1) {
                if (L::SLOTS == 3) dma(1, 1);
                fetch(1);
            }
        }
        // o of chunk c (64 rows of 64 channels where v was): the rows whose place this wave's DMA takes next
        auto store_o = [&](int c, int slot) {
            const int ln = opaque(lane), rows = rows_of(c);
            const char* tv = smem + 2 * L::STAGED + slot * L::DMA + L::V;
            u32x4 y[2 * HALVES];
#pragma unroll
            for (int u = 0; u < 2 * HALVES; ++u)
                y[u] = *reinterpret_cast<const u32x4*>(tv + (u >> 1) * 8192 + (2 * w + (u & 1)) * 1024 + ln * 16);
#pragma unroll
            for (int u = 0; u < 2 * HALVES; ++u) {
                const int i = 8 * (2 * w + (u & 1)) + (ln >> 3);
                if (i < rows)
                    *reinterpret_cast<u32x4*>(p.o + ((row * p.T + bos + (int64_t)c * CH + i) * p.Hv + hv) * DK + 64 * sl +
                                              64 * (u >> 1) + 8 * (ln & 7)) = y[u];
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        };
        constexpr int AHEAD = L::SLOTS - 1;
        int slot = AHEAD;   // of chunk c + AHEAD, and of c - 1
        for (int c = 0; c < nch; ++c) {
            // v, T and A of chunk c have landed; what was issued later may be on its way: thirteen loads
            // for chunk c + 1, before them with three slots six pieces or more of its v, T and A
            if (c + 1 == nch) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            else if (AHEAD == 2) asm volatile("s_waitcnt vmcnt(19)" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(13)" ::: "memory");
            lds_barrier();
            if (c > 0) store_o(c - 1, slot);
            if (c + 1 < nch) {
                stage(c + 1);   // before the DMA: what it reads is the only thing it waits for
                if (c + AHEAD < nch) dma(c + AHEAD, slot);
                if (c + 2 < nch) fetch(c + 2);
            }
            slot = slot == AHEAD ? 0 : slot + 1;
        }
        lds_barrier();
        if (nch > 0) store_o(nch - 1, slot);
        return;
    }

    // ================= scan waves =================
    __builtin_amdgcn_s_setprio(3);
    const int w = wave & 3;   // sixteen columns of half wave / 4 of those that the work-group walks
    const int64_t so = ((int64_t)n * p.Hv + hv) * DK * DK + 64 * sl + 16 * wave + (lane & 15);
    f32x4 S[8];                     // the state times down / kap
    float down = 1.f, up = 1.f;     // the lane's column: a power of two and its inverse
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = p.h0 ? p.h0[so + state_row(t, lane >> 4, r) * DK] : 0.f;
    }
    // Columns whose largest value lies below `least` or above `most` go back to [2^7, 2^8); top: the
    // lane's part of it.  Returns what the state was multiplied by: what is at hand in its units is too.
    auto rescale = [&](float top, float least, float most) -> float {
        top = max_groups(top);
        if (top > most || (top < least && top > 0.f)) {
            int e = (int)(__float_as_uint(top) >> 23) - 127 - 7;   // what its exponent has too many
            const int was = 127 - (int)(__float_as_uint(down) >> 23);
            e = max(-120 - was, min(120 - was, e));                // keep the power of two itself in range
            const float by = __uint_as_float((uint32_t)(127 - max(-126, min(126, e))) << 23);
#pragma unroll
            for (int t = 0; t < 8; ++t) S[t] *= by;
            down *= by;
            up = inverse2(down);
            return by;
        }
        return 1.f;
    };
    auto times = [](f32x4 (&x)[4], float by) {
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] *= by;
    };
    int at = 0;   // chunk c's slot of what comes by DMA
    for (int c = 0; c < nch; ++c) {
        lds_barrier();   // chunk c is in LDS, and the other slots' reads are done
        const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
        char* slot = smem + 2 * L::STAGED + at * L::DMA;
        at = at + 1 == L::SLOTS ? 0 : at + 1;
        const char *tk = smem + (c & 1) * L::STAGED + L::K, *tq = tk + L::Q;
        char* tv = slot + L::V + (wave >> 2) * 8192;
        const float* sc = reinterpret_cast<const float*>(tk + L::SC);
        const float km = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sc[SC_KP])));
        if (km > 0.f && km != kap) {   // powers of two: exact
#pragma unroll
            for (int t = 0; t < 8; ++t) S[t] *= kap * inverse2(km);
            kap = km;
        }
        f32x4 v[4];   // beta v 2^ek / kap
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const u32x2 b = lds_tr(tv + (16 * m + 4 * g + (jj >> 2)) * 128 + 32 * w + 8 * (jj & 3));
            v[m] = f32x4{bf_lo(b[0]), bf_hi(b[0]), bf_lo(b[1]), bf_hi(b[1])} * down * sc4(sc, SC_BE, m, g);
        }
        float top = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t) top = max_abs(top, S[t]);
#pragma unroll
        for (int m = 0; m < 4; ++m) top = max_abs(top, v[m]);
        if (__any(top > 1024.f || (top < 4.f && top > 0.f))) times(v, rescale(top, 4.f, 1024.f));
        // x = (beta v - beta e^G K S) 2^ek / kap and e^G Q S, eight tiles side by side; the next
        // step's operands are read and split meanwhile
        f32x4 x[4], o[4];
        {
            half8 fk[2][4], fq[2][4];
            HSplit<2> sb[2];
            sb[0] = hsplit<2>(S[0], S[1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                fk[0][m] = row_frag(tk, m, 0, g, jj);
                fq[0][m] = row_frag(tq, m, 0, g, jj);
                x[m] = o[m] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int now = kk & 1, next = now ^ 1;
                if (kk < 3) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        fk[next][m] = row_frag(tk, m, kk + 1, g, jj);
                        fq[next][m] = row_frag(tq, m, kk + 1, g, jj);
                    }
                    sb[next] = hsplit<2>(S[2 * kk + 2], S[2 * kk + 3]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) x[m] = mfma_h(fk[now][m], sb[now].s[1], x[m]);
#pragma unroll
                for (int m = 0; m < 4; ++m) o[m] = mfma_h(fq[now][m], sb[now].s[0], o[m]);
#pragma unroll
                for (int m = 0; m < 4; ++m) x[m] = mfma_h(fk[now][m], sb[now].s[0], x[m]);
                interleave<12, 3, 1, 0>();
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                x[m] = v[m] - sc4(sc, SC_EGK, m, g) * x[m];
                o[m] *= sc4(sc, SC_EG, m, g);
            }
        }
        // u = T x (of the rows times 2^ek / kap, as x is): six tiles side by side
        f32x4 u[4];
        constexpr int TM[6] = {0, 1, 2, 3, 2, 3}, TK[6] = {0, 0, 0, 0, 1, 1};   // fragments (m, kk)
        {
            half8 th[6], tl[6];
            f32x4 a[6];
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                const char* f = slot + L::T + tri_frag(TM[i], TK[i]) * GDR_FRAG + ln * 16;
                th[i] = *reinterpret_cast<const half8*>(f);
                tl[i] = *reinterpret_cast<const half8*>(f + GDR_TRI);
                a[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            const HSplit<2> xb[2] = {hsplit<2>(x[0], x[1]), hsplit<2>(x[2], x[3])};
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 6; ++i) a[i] = mfma_h(tl[i], xb[TK[i]].s[0], a[i]);
#pragma unroll
            for (int i = 0; i < 6; ++i) a[i] = mfma_h(th[i], xb[TK[i]].s[1], a[i]);
#pragma unroll
            for (int i = 0; i < 6; ++i) a[i] = mfma_h(th[i], xb[TK[i]].s[0], a[i]);
#pragma unroll
            for (int m = 0; m < 4; ++m) u[m] = m < 2 ? a[m] : a[m] + a[m + 2];
        }
        // repeated keys can make u up to 128 |k^| times what the chunk started with
        {
            float tu = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) tu = max_abs(tu, u[m]);
            if (__any(tu > 32768.f)) {
                const float by = rescale(tu, 0.f, 32768.f);
                times(u, by);
                times(o, by);
            }
        }
        const float whole = up * kap * p.scale;   // what o's sums are multiplied by
        // S <- e^{G_last} S + K^T (e^{G_last - G} u), four tiles side by side; between them
        // o's second part, rounded once, into this wave's columns of v's slice: the staging
        // waves store it
        {
            f32x4 wu[4];
            float tw = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) tw = max_abs(tw, wu[m] = sc4(sc, SC_GA, m, g) * u[m]);
            const float el = sc[SC_EL];
#pragma unroll
            for (int t = 0; t < 8; ++t) S[t] *= el;
            if (__any(tw < 4.f && tw > 0.f)) {   // what is left of the chunk may be far less than what it started with
#pragma unroll
                for (int t = 0; t < 8; ++t) tw = max_abs(tw, S[t]);
                times(wu, rescale(tw, 4.f, __builtin_inff()));
            }
            const HSplit<2> wb[2] = {hsplit<2>(wu[0], wu[1]), hsplit<2>(wu[2], wu[3])};
            const HSplit<1> ub[2] = {hsplit<1>(u[0], u[1]), hsplit<1>(u[2], u[3])};
            half8 f[2][4], fa[6];
#pragma unroll
            for (int t = 0; t < 4; ++t) f[0][t] = col_frag(tk, t, 0, g, jj);
#pragma unroll
            for (int i = 0; i < 6; ++i)
                fa[i] = *reinterpret_cast<const half8*>(slot + L::A + tri_frag(TM[i], TK[i]) * GDR_FRAG + ln * 16);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // tiles 4 (i / 2) .., k step i & 1
                const int t0 = 4 * (i >> 1), kk = i & 1;
                if (i < 3) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) f[kk ^ 1][t] = col_frag(tk, 4 * ((i + 1) >> 1) + t, kk ^ 1, g, jj);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) S[t0 + t] = mfma_h(f[kk][t], wb[kk].s[1], S[t0 + t]);
                if (i == 0) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) o[m] = mfma_h(fa[m], ub[0].s[0], o[m]);
                } else if (i == 1) {
#pragma unroll
                    for (int m = 2; m < 4; ++m) o[m] = mfma_h(fa[m + 2], ub[1].s[0], o[m]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) S[t0 + t] = mfma_h(f[kk][t], wb[kk].s[0], S[t0 + t]);
                if (i >= 2) {
#pragma unroll
                    for (int m = 2 * i - 4; m < 2 * i - 2; ++m) {
                        o[m] *= sc4(sc, SC_QS, m, g) * whole;
                        const uint32_t p0 = pack_bf2(o[m][0], o[m][1]), p1 = pack_bf2(o[m][2], o[m][3]);
                        char* dst = tv + (16 * m + 4 * g) * 128 + 2 * (16 * w + jj);
                        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)p0;
                        *reinterpret_cast<uint16_t*>(dst + 128) = (uint16_t)(p0 >> 16);
                        *reinterpret_cast<uint16_t*>(dst + 256) = (uint16_t)p1;
                        *reinterpret_cast<uint16_t*>(dst + 384) = (uint16_t)(p1 >> 16);
                    }
                }
                interleave<8, 4, 1, 0>();
            }
        }
    }
    lds_barrier();   // the last chunk's o is complete
    if (p.hT) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) p.hT[so + state_row(t, lane >> 4, r) * DK] = S[t][r] * up * kap;
        }
    }
}

hipError_t launch_gdr_fwd(const GdrParams& p, int cus, hipStream_t stream) {
    hipError_t e = launch_gdr_prep(p, false, stream);
    if (e != hipSuccess) return e;
    // Whole heads share the staging of k, q, T and A, and take 1.75 times a half's time: worth it
    // where heads alone fill the compute units and no sequence is much longer than the others,
    // for packed ones taken to be so with four times as many.  Halves and whole heads: 560 and
    // 502 us at B=4 H=64 T=4096, 152 and 130 at B=32 H=16 T=512, 656 and 484 at 64 packed
    // sequences of 256 tokens and 64 heads; but 519 and 581 at 11 of 16,384 tokens together, the
    // longest half of them.
    const int64_t heads = (int64_t)p.N * p.Hv;
    if (heads >= (p.cu ? 4 * (int64_t)cus : cus))
        hipLaunchKernelGGL(kda_gdr_scan_kernel<2>, dim3((unsigned)heads), dim3(FL<2>::THREADS), 0, stream, p);
    else
        hipLaunchKernelGGL(kda_gdr_scan_kernel<1>, dim3((unsigned)(2 * heads)), dim3(FL<1>::THREADS), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
