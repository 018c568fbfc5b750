// The token gradients of the selective state space scan, all chunks at once, on gfx950
// (MI355X).  For a chunk with S the state entering it, dS the gradient of the one leaving it, d the
// steps, L_ij = e^{G_i - G_j} (j <= i) and R = dy x^T:
//   V = x dS^T, W = dy S^T,  K_ij = L_ij R_ij d_j,  E_ij = L_ij (C B^T)_ij,  M = E R
//   dC = e^G W + K B,  dB = e^{G_last - G} d V + K^T C   (sums over a group's heads)
//   dx = d (e^{G_last - G} B dS + E^T dy) + D dy
//   u_j = e^{G_last - G_j} B_j . V_j,  w_i = e^{G_i} C_i . W_i,  q = e^{G_last} <S, dS>
//   da_t = sum_{j < t <= i} M_ij d_j + sum_{i >= t} w_i + sum_{j < t} u_j d_j + q
//   dd_t = A da_t + u_t + sum_{i >= t} M_it,  ddt = dd times the step's slope
// da_t adds only what passes token t, never differences of longer sums: it keeps fp32's accuracy
// where strong decays make it small.
//
// A work-group of eight waves takes a chunk and a group's heads, or some of them where that
// leaves compute units idle, one head after the other; C B^T, and dB and dC in accumulators, stay.
// Of the products with S and dS a wave takes sixteen state channels (with 64 of them half the
// tokens): the states come from memory as the operands that the walk left, and only dS goes
// through LDS, for dx.  The 64 x 64 matrices are ten tiles, dealt to the waves; they leave as
// operand fragments for the second half of a head's work.
//
// B = 2, H = 64, P = 64, S = 128, T = 8192: 499 us in a trace, 16,800 clocks a chunk and head.  Of those a SIMD spends 6,400 on
// vector and 3,900 on matrix instructions, the compute unit's LDS 8,400 and 2,500 on conflicts, and waves wait for 45% of
// theirs: LDS is the busiest pipe, the meetings keep the others from filling beside it.  The inputs of a head are asked for
// during the head before, S and dS apart from each other: all at once they waited for the memory's queue.
//
// Precision.  What multiplies x, dy, B and C enters in three bf16 parts, fp32's 24 bits: S and dS in V and W (in two parts,
// dA was off by 2 10^-6 at B = 2, H = 64, T = 8192, fp32's plain form by 4 10^-7), K, E and dS in dx.  The terms of dx, dB
// and dC may cancel: with two parts of the last three (the kernel 452 us in a trace there, not 499) they were off by up to 2^-18 of
// their terms, and by 9 10^-5 of their norm from a 32-bit form that is now 2 to 3 10^-5 away.
#include "kda_ssm_device.h"

namespace kda {

namespace {

constexpr int NT = 512;

template <int P>
struct GL {
    static constexpr int B = 0, C = 16384, X = 32768;            // [64][256 bytes] tiles, swizzled
    static constexpr int DY = P == 64 ? X : X + 16384;           // P = 64: beside x in its rows
    static constexpr int DS = DY + 16384;                        // [S][64 columns, two parts], swizzled
    static constexpr int DT = P == 64 ? DS + 32768 : DS;         // [64][64 columns of rows r and r + 64, the third part]
    static constexpr int KC = DS + (P == 64 ? 49152 : 32768), KB = KC + 3 * GDR_TRI, EX = KB + 3 * GDR_TRI;   // fragments, three parts each
    static constexpr int REC = EX + 3 * GDR_TRI;
    static constexpr int RS = REC + SSM_REC, CS = RS + 4 * 256, DR = CS + 4 * 256;   // sums of M's tiles by row, by column
    static constexpr int UP = DR + 256, YP = UP + 8 * 256, SD = YP + 8 * 256, BYTES = SD + 256;
};
static_assert(GL<64>::BYTES <= 163840 && GL<128>::BYTES <= 163840, "LDS");

// Byte of a 16-byte piece of a row of dS's tile: written from rows 8 a + b and read, two pieces of each, from four rows
// of 8 g, its pieces are permuted by the rows' bits 0, 1, 4 and 3, the last one so that neighbouring g do not meet.
__device__ __forceinline__ int ds_off(int row, int piece) {
    return row * 256 + ((piece ^ (((row & 3) << 2) | ((row >> 2) & 2) | ((row >> 4) & 1))) << 4);
}
__device__ __forceinline__ bf16x8 two8(const char* tile, int row, int at) {   // elements at .. + 3 and 16 more on
    const int q = at >> 3, b = 2 * (at & 7);
    return join(*reinterpret_cast<const u32x2*>(tile + tile_off(row, q) + b),
                *reinterpret_cast<const u32x2*>(tile + tile_off(row, q + 2) + b));
}
// Transposing reads of rows r0 + 0 .. 3 and r1 + 0 .. 3: column `at` + jj.
__device__ __forceinline__ bf16x8 two_tr(const char* tile, int r0, int r1, int at, int jj) {
    const int e = at + 4 * (jj & 3), q = e >> 3, b = 2 * (e & 7), r = jj >> 2;
    return join(lds_tr(tile + tile_off(r0 + r, q) + b), lds_tr(tile + tile_off(r1 + r, q) + b));
}
// Index of fragment (m, kk) in the lists whose rows are the pair matrices' columns.
__device__ __forceinline__ constexpr int upper_frag(int m, int kk) { return m < 2 ? 2 * m + kk : m + 2; }

// Inclusive sum over the lanes before this one, in its group of 16 or in the wave.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f32(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, true));
}
__device__ __forceinline__ float prefix16(float x) {
    x += dpp_f32<0x111, 0xf>(x);
    x += dpp_f32<0x112, 0xf>(x);
    x += dpp_f32<0x114, 0xf>(x);
    x += dpp_f32<0x118, 0xf>(x);
    return x;
}
__device__ __forceinline__ float prefix_wave(float x) {
    x = prefix16(x);
    x += dpp_f32<0x142, 0xa>(x);
    x += dpp_f32<0x143, 0xc>(x);
    return x;
}
__device__ __forceinline__ float suffix16(float x, int lane) { return __shfl(prefix16(__shfl(x, lane ^ 15)), lane ^ 15); }
__device__ __forceinline__ float suffix_wave(float x, int lane) { return __shfl(prefix_wave(__shfl(x, lane ^ 63)), lane ^ 63); }
// x of the lane before this one (0 for the first of each group of 16, or of the wave).
__device__ __forceinline__ float before16(float x) { return dpp_f32<0x111, 0xf>(x); }
__device__ __forceinline__ float before_wave(float x, int lane) {
    const float y = __shfl(x, lane - 1);
    return lane == 0 ? 0.f : y;
}
__device__ __forceinline__ float lane_f32(float x, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

}  // namespace

template <int S, int P>
__global__ void __launch_bounds__(NT) kda_ssm_grads_kernel(const SsmParams p) {
    typedef GL<P> L;
    constexpr int KT = S / 32, KP = P / 32, MW = S == 128 ? 4 : 2;   // k steps; row tiles of a wave's state channels
    constexpr int PX = P / 64;                                       // 16-byte pieces of x that a thread brings
    __shared__ __attribute__((aligned(1024))) char smem[L::BYTES];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, jj = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int R = uniform(p.H / p.G), hs = uniform((R + p.sets - 1) / p.sets);
    const int set = uniform((int)(blockIdx.x % p.sets)), group = uniform((int)(blockIdx.x / p.sets % p.G));
    const int64_t slot = uniform((int)(blockIdx.x / p.sets / p.G));
    const SsmChunk ch = ssm_chunk(p, slot);
    if (ch.rows == 0) return;
    const int h_from = group * R + set * hs, h_to = group * R + ((set + 1) * hs < R ? (set + 1) * hs : R);
    const char *tb = smem + L::B, *tc = smem + L::C, *tx = smem + L::X, *ty = smem + L::DY;
    constexpr int YO = P == 64 ? 64 : 0;   // dy's first element in its rows
    const float* rec = reinterpret_cast<const float*>(smem + L::REC);
    float *sRS = reinterpret_cast<float*>(smem + L::RS), *sCS = reinterpret_cast<float*>(smem + L::CS),
          *sDR = reinterpret_cast<float*>(smem + L::DR), *sU = reinterpret_cast<float*>(smem + L::UP),
          *sY = reinterpret_cast<float*>(smem + L::YP), *sS = reinterpret_cast<float*>(smem + L::SD);
    const int t = S == 128 ? wave : wave & 3, m0 = S == 128 ? 0 : 2 * (wave >> 2);   // state tile, first row tile

    {   // B and C
        const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));
        auto tile = [&](const Rows& w, uint32_t where) {
            const __amdgpu_buffer_rsrc_t rs = chunk_rsrc(w.p + ch.row * w.sb + ch.tok * w.st + group * w.sh, w.st, ch.rows, S);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = 4 * (wave + 8 * u) + g, piece = jj ^ tsw(r);
                const int off = (int)(r * w.st * 2) + 16 * piece;
                dma_piece(rs, where + (wave + 8 * u) * 1024, S == 128 || piece < 8 ? off : 0x7ffffff0);
            }
        };
        tile(p.B, lds + L::B);
        tile(p.C, lds + L::C);
    }
    // what no tile of the pair matrices covers in the fragments
    if (tid < 64) {
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            *reinterpret_cast<u32x2*>(smem + L::KC + n * GDR_TRI + tri_frag(0, 0) * GDR_FRAG + 16 * lane + 8) = u32x2{0, 0};
            *reinterpret_cast<u32x2*>(smem + L::KC + n * GDR_TRI + tri_frag(2, 1) * GDR_FRAG + 16 * lane + 8) = u32x2{0, 0};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                char* to = smem + (x ? L::EX : L::KB) + n * GDR_TRI + 16 * lane;
                *reinterpret_cast<u32x2*>(to + upper_frag(1, 0) * GDR_FRAG) = u32x2{0, 0};
                *reinterpret_cast<u32x2*>(to + upper_frag(3, 1) * GDR_FRAG) = u32x2{0, 0};
            }
        }
    }
    // A head's inputs, asked for ahead
    u32x4 nx[PX], ny[PX], nrec;
    uint32_t nskip = 0;
    f32x4 ns[KP][2], nds[KP][2];   // S and dS, 32 columns each
    const int lr = P == 64 ? tid >> 3 : tid >> 4, lp = P == 64 ? tid & 7 : tid & 15;   // row and piece of this thread
    // What a head reads and writes, from its first element: one head on at the end of each turn.  Behind the last
    // head the buffers are empty: loads that always stand there can be counted, and wait for less.
    const uint16_t *px = p.x.p + ch.row * p.x.sb + ch.tok * p.x.st + h_from * p.x.sh,
                   *py = p.dO.p + ch.row * p.dO.sb + ch.tok * p.dO.st + h_from * p.dO.sh;
    uint16_t* pdx = p.dx + ((ch.row * p.T + ch.tok) * p.H + h_from) * P;
    const float *ps = p.St + (slot * p.H + h_from) * S * P, *pds = p.dSt + (slot * p.H + h_from) * S * P;
    char* prec = p.rec + (slot * p.H + h_from) * SSM_REC;
    const float* pd = p.D ? p.D + h_from : nullptr;
    const int nx_bytes = (int)((ch.rows - 1) * p.x.st + P) * 2, ny_bytes = (int)((ch.rows - 1) * p.dO.st + P) * 2;
    const int skips = p.D ? 4 : 0;
    auto ask = [&](bool real, int on) {   // inputs `on` heads further
        const auto rx = make_rsrc(px + on * p.x.sh, real ? nx_bytes : 0), ry = make_rsrc(py + on * p.dO.sh, real ? ny_bytes : 0);
#pragma unroll
        for (int u = 0; u < PX; ++u) {   // rows past the chunk's end come as zeros
            const int r = lr + 32 * u;
            nx[u] = __builtin_amdgcn_raw_buffer_load_b128(rx, r * (int)p.x.st * 2 + 16 * lp, 0, 0);
            ny[u] = __builtin_amdgcn_raw_buffer_load_b128(ry, r * (int)p.dO.st * 2 + 16 * lp, 0, 0);
        }
        nrec = __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(prec + on * SSM_REC, real ? SSM_REC : 0), 16 * tid, 0, 0);
        nskip = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(pd + on, real ? skips : 0), 0, 0, 0);
    };
    auto ask_state = [&](const float* from, f32x4 (&to)[KP][2], bool real, int first, int end) {   // columns 32 first .. 32 end - 1
        const auto rs = make_rsrc(from, real ? S * P * 4 : 0);
#pragma unroll
        for (int pp = first; pp < end; ++pp) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct)
                to[pp][ct] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, 2048 * t + 1024 * ct + 16 * lane, pp * (S * 128), 0));
        }
    };
    ask(h_from < h_to, 0);
    ask_state(ps, ns, h_from < h_to, 0, 2);
    ask_state(pds, nds, h_from < h_to, 0, 2);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();

    // tiles (I, J) of the pair matrices: waves 0 .. 3 take those below the diagonal, (1,0) (2,0) | (2,1) (3,0) | (3,1) |
    // (3,2), and 4 .. 7 one on it
    const int nt = wave < 2 ? 2 : 1;
    const int tI[2] = {wave < 4 ? (wave < 2 ? wave + 1 : 3) : wave - 4, wave + 2};
    const int tJ[2] = {wave < 4 ? (wave < 1 ? 0 : wave < 3 ? 1 : 2) : wave - 4, 0};
    f32x4 cb[2];   // C B^T, rows 16 I + 4 g + r, column 16 J + jj
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        cb[x] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (x >= nt) continue;
#pragma unroll
        for (int kk = 0; kk < KT; ++kk)
            cb[x] = mfma_bf(row_frag(tc, tI[x], kk, g, jj), row_frag(tb, tJ[x], kk, g, jj), cb[x]);
    }
    f32x4 dB[MW], dC[MW];
#pragma unroll
    for (int m = 0; m < MW; ++m) dB[m] = dC[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    // token 16 m + jj's four channels of lane group g in the wave's state tile
    auto column = [&](const char* tile, int m, int g, int jj) {
        return widen(*reinterpret_cast<const u32x2*>(tile + tile_off(16 * m + jj, 4 * (t >> 1) + g) + 8 * (t & 1)));
    };

    for (int h = h_from; h < h_to; ++h) {
        // the head's inputs into LDS
#pragma unroll
        for (int u = 0; u < PX; ++u) {
            *reinterpret_cast<u32x4*>(smem + L::X + tile_off(lr + 32 * u, lp)) = nx[u];
            *reinterpret_cast<u32x4*>(smem + L::DY + tile_off(lr + 32 * u, lp + YO / 8)) = ny[u];
        }
        if (tid < SSM_REC / 16) *reinterpret_cast<u32x4*>(smem + L::REC + 16 * tid) = nrec;
        const float skip = __int_as_float(uniform((int)nskip));
        __syncthreads();
        const bool more = h + 1 < h_to;
        ask_state(ps, ns, true, 2, KP);
        ask_state(pds, nds, true, 2, KP);

        // ---- the pair matrices' tiles
        {
        const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;   // addresses formed anew: kept through the loop they would spill
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (x >= nt) continue;
            const int I = tI[x], J = tJ[x];
            f32x4 r = {0.f, 0.f, 0.f, 0.f}, rt = r;   // dy x^T, and transposed
#pragma unroll
            for (int pp = 0; pp < KP; ++pp) {
                const bf16x8 yf = two8(ty, 16 * I + jj, YO + 32 * pp + 4 * g), xf = two8(tx, 16 * J + jj, 32 * pp + 4 * g);
                r = mfma_bf(yf, xf, r);
                rt = mfma_bf(xf, yf, rt);
            }
            f32x4 l, lt;   // decays
            const float dj = rec[SSM_DT + 16 * J + jj];
            const f32x4 djt = num4(rec, SSM_DT, J, g);
            if (I == J) {
                const float hi = rec[SSM_GH + 16 * I + jj], lo = rec[SSM_GL + 16 * I + jj];
                const f32x4 h4 = num4(rec, SSM_GH, I, g), l4 = num4(rec, SSM_GL, I, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l[e] = formed(fexp2((h4[e] - hi) + (l4[e] - lo)));
                    lt[e] = formed(fexp2((hi - h4[e]) + (lo - l4[e])));
                }
            } else {
                float mid = 1.f;
                if (I > J + 1) mid = rec[SSM_RI + 16 * J + 31];
                if (I > J + 2) mid *= rec[SSM_RI + 16 * J + 47];
                l = num4(rec, SSM_RI, I, g) * (rec[SSM_KA + 16 * J + jj] * mid);
                lt = num4(rec, SSM_KA, J, g) * (rec[SSM_RI + 16 * I + jj] * mid);
            }
            f32x4 e = cb[x], m;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // above the diagonal nothing counts, not even NaN
                const bool on = I > J || jj <= 4 * g + i, ont = I > J || 4 * g + i <= jj;
                e[i] = on ? e[i] * l[i] : 0.f;
                m[i] = on ? e[i] * r[i] : 0.f;
                lt[i] = ont ? lt[i] * rt[i] * djt[i] : 0.f;
                l[i] = on ? l[i] * r[i] * dj : 0.f;
            }
            auto put = [&](int list, int frag, int half, const f32x4& a) {
                char* to = smem + list + frag * GDR_FRAG + 16 * lane + 8 * half;
                u32x4 part[3];
                split_pair<3>(part, 0, a[0], a[1]);
                split_pair<3>(part, 1, a[2], a[3]);
#pragma unroll
                for (int n = 0; n < 3; ++n) *reinterpret_cast<u32x2*>(to + n * GDR_TRI) = u32x2{part[n][0], part[n][1]};
            };
            put(L::KC, tri_frag(I, J >> 1), J & 1, lt);
            put(L::KB, upper_frag(J, I >> 1), I & 1, l);
            put(L::EX, upper_frag(J, I >> 1), I & 1, e);
            // M's sums: of a column over the tile's rows, of a row with each column's step
            const float cs = sum_groups((m[0] + m[1]) + (m[2] + m[3]));
            if (g == 0) sCS[64 * I + 16 * J + jj] = cs;
            f32x4 md = m * dj;
            if (I > J) {
#pragma unroll
                for (int i = 0; i < 4; ++i) md[i] = sum16(md[i]);
                if (jj == 0) *reinterpret_cast<f32x4*>(sRS + 64 * J + 16 * I + 4 * g) = md;
                if (I > J + 1) {   // (2, 0), (3, 0), (3, 1) whole
                    const float all = sum_groups((md[0] + md[1]) + (md[2] + md[3]));
                    if (ln == 0) sS[10 + I + J] = all;
                }
            } else {   // sum over j < t <= i of the tile, and the diagonal of dy x^T
                md[2] += md[3];
                md[1] += md[2];
                md[0] += md[1];
                // over the lane groups behind this one: pairs of groups come as the even and the odd, then the lower and the upper one
                const Pair two = across<16>(md[0]), halves = across<32>(two.a + two.b);
                const float above = (g & 1 ? 0.f : two.b) + (g < 2 ? halves.b : 0.f);
                float diag = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (jj == 4 * g + i) diag = r[i];
                    md[i] = sum16(jj < 4 * g + i ? md[i] + above : 0.f);
                }
                if (jj == 0) *reinterpret_cast<f32x4*>(sDR + 16 * I + 4 * g) = md;
                diag = sum64(diag);
                if (lane == 0) sS[8 + I] = diag;
            }
        }
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- V and W of the wave's state channels, 32 columns at a time, and dS's parts into LDS
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        // For P = 128 dS's tile holds by turns two parts of columns 0 .. 63, the third part of all, two parts of the others
        u32x4 later[PX > 1 ? 2 : 1][2], third[PX > 1 ? KP : 1];   // two parts of columns 64 ..; third parts
        auto put_ds = [&](int q, int n, u32x4 w, int row, int g, int base) {   // part n of 32 columns
            const int at = n == 2 ? 64 * (row >> 6) + 32 * q + 4 * g : 64 * n + 32 * q + 4 * g;
            char* to = smem + base + 2 * (at & 7);
            if (n == 2) row &= 63;
            *reinterpret_cast<u32x2*>(to + ds_off(row, at >> 3)) = u32x2{w[0], w[1]};
            *reinterpret_cast<u32x2*>(to + ds_off(row, (at >> 3) + 2)) = u32x2{w[2], w[3]};
        };
        {
            const int nrow = state_row(t, jj >> 2, jj & 3);
            f32x4 v[MW], w[MW];
#pragma unroll
            for (int mi = 0; mi < MW; ++mi) v[mi] = w[mi] = zero;
            float q = 0.f;
#pragma unroll
            for (int pp = 0; pp < KP; ++pp) {
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) q = fmaf(ns[pp][ct][i], nds[pp][ct][i], q);
                }
                {
                    const Split<3> dsp = split_acc<3>(nds[pp][0], nds[pp][1]);
#pragma unroll
                    for (int n = 0; n < 3; ++n) {
                        const u32x4 part = __builtin_bit_cast(u32x4, dsp.s[n]);
                        if (P == 128 && n == 2) third[pp] = part;
                        else if (pp >= 2) later[pp - 2][n] = part;
                        else if (S == 128 || wave < 4) put_ds(pp, n, part, nrow, g, n == 2 ? L::DT : L::DS);
                    }
                    bf16x8 f[MW];
#pragma unroll
                    for (int mi = 0; mi < MW; ++mi) f[mi] = two8(tx, 16 * (m0 + mi) + jj, 32 * pp + 4 * g);
#pragma unroll
                    for (int n = 2; n >= 0; --n) {
#pragma unroll
                        for (int mi = 0; mi < MW; ++mi) v[mi] = mfma_bf(dsp.s[n], f[mi], v[mi]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                {
                    const Split<3> sp = split_acc<3>(ns[pp][0], ns[pp][1]);
                    bf16x8 f[MW];
#pragma unroll
                    for (int mi = 0; mi < MW; ++mi) f[mi] = two8(ty, 16 * (m0 + mi) + jj, YO + 32 * pp + 4 * g);
#pragma unroll
                    for (int n = 2; n >= 0; --n) {
#pragma unroll
                        for (int mi = 0; mi < MW; ++mi) w[mi] = mfma_bf(sp.s[n], f[mi], w[mi]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            q = sum64(q);
            if (lane == 0) sS[wave] = S == 128 || wave < 4 ? q : 0.f;
#pragma unroll
            for (int mi = 0; mi < MW; ++mi) {
                const int m = m0 + mi;
                const int tok = 16 * m + jj;
                const f32x4 u = v[mi] * column(tb, m, g, jj), y = w[mi] * column(tc, m, g, jj);
                dB[mi] += (rec[SSM_GA + tok] * rec[SSM_DT + tok]) * v[mi];
                dC[mi] += rec[SSM_EG + tok] * w[mi];
                const float su = sum_groups((u[0] + u[1]) + (u[2] + u[3])), sy = sum_groups((y[0] + y[1]) + (y[2] + y[3]));
                if (g == 0) sU[64 * t + tok] = su;
                if (g == 1) sY[64 * t + tok] = sy;
            }
        }
        ask(more, 1);   // S and dS later: all at once would wait for the memory's queue
        __syncthreads();

        // ---- dB and dC from the pair matrices
        ask_state(ps + S * P, ns, more, 0, 2);
        {
            const int ln = P == 128 ? opaque(lane) : lane, g = ln >> 4, jj = ln & 15;
            bf16x8 bcol[2], ccol[2];   // channels of tile t, tokens of k step kk
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bcol[kk] = col_frag(tb, t, kk, g, jj);
                ccol[kk] = col_frag(tc, t, kk, g, jj);
            }
#pragma unroll
            for (int n = 2; n >= 0; --n) {
#pragma unroll
                for (int mi = 0; mi < MW; ++mi) {
                    const int m = m0 + mi;
                    const char *kc = smem + L::KC + n * GDR_TRI + 16 * ln, *kb = smem + L::KB + n * GDR_TRI + 16 * ln;
                    dC[mi] = mfma_bf(bcol[0], lds_bf8(kc + (m < 2 ? m : 2 * m - 2) * GDR_FRAG), dC[mi]);
                    if (m >= 2) dC[mi] = mfma_bf(bcol[1], lds_bf8(kc + (2 * m - 1) * GDR_FRAG), dC[mi]);
                    if (m < 2) dB[mi] = mfma_bf(ccol[0], lds_bf8(kb + 2 * m * GDR_FRAG), dB[mi]);
                    dB[mi] = mfma_bf(ccol[1], lds_bf8(kb + (m < 2 ? 2 * m + 1 : m + 2) * GDR_FRAG), dB[mi]);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- dx, transposed: a lane holds four channels of one token
        ask_state(pds + S * P, nds, more, 0, 2);
        const int dst = p.H * P;
        const auto rdx = chunk_rsrc(pdx, dst, ch.rows, P);
        const int pt = wave & 3, ma = 2 * (wave >> 2);   // columns 16 pt .. of 64; tokens of two tiles
        f32x4 ds[PX][2];   // B dS
#pragma unroll
        for (int half = 0; half < PX; ++half) ds[half][0] = ds[half][1] = zero;
        // a + B times parts `from` .. `to` - 1 of dS's columns 64 half .. in LDS
        auto times_ds = [&](f32x4 (&a)[2], int from, int to, int third_at) {
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                const bf16x8 b0 = row_frag(tb, ma, kk, g, jj), b1 = row_frag(tb, ma + 1, kk, g, jj);
#pragma unroll
                for (int n = to - 1; n >= from; --n) {
                    const int q = (n == 2 ? 8 * (kk >> 1) : 8 * n) + 2 * pt + ((jj & 3) >> 1), r = (n == 2 ? 32 * (kk & 1) : 32 * kk) + 8 * g + (jj >> 2);
                    const char* at = smem + (n == 2 ? third_at : L::DS) + 8 * (jj & 1);
                    const bf16x8 d = join(lds_tr(at + ds_off(r, q)), lds_tr(at + ds_off(r + 4, q)));
                    a[0] = mfma_bf(d, b0, a[0]);
                    a[1] = mfma_bf(d, b1, a[1]);
                }
            }
        };
        if (P == 64) {
            times_ds(ds[0], 0, 3, L::DT);
        } else {
            const int nrow = state_row(t, jj >> 2, jj & 3);
            const bool puts = S == 128 || wave < 4;
            times_ds(ds[0], 0, 2, 0);
            __syncthreads();
            if (puts) {
#pragma unroll
                for (int q = 0; q < KP; ++q) put_ds(q & 1, 2, third[PX > 1 ? q : 0], nrow, g, L::DT + 16384 * (q >> 1));
            }
            __syncthreads();
            times_ds(ds[0], 2, 3, L::DT);
            times_ds(ds[PX - 1], 2, 3, L::DT + 16384);
            __syncthreads();
            if (puts) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) put_ds(q, n, later[PX > 1 ? q : 0][n], nrow, g, L::DS);
                }
            }
            __syncthreads();
            times_ds(ds[PX - 1], 0, 2, 0);
        }
#pragma unroll
        for (int half = 0; half < PX; ++half) {
            const int col = 64 * half + 16 * pt;
            f32x4 b[2] = {zero, zero};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                if (kk == 0 && ma >= 2) continue;
                const bf16x8 yf = two_tr(ty, 32 * kk + 4 * g, 32 * kk + 16 + 4 * g, YO + col, jj);
                const char* ex = smem + L::EX + 16 * lane;
#pragma unroll
                for (int mi = 0; mi < 2; ++mi) {
                    const int f = ma < 2 ? 2 * mi + kk : 4 + mi;   // fragment (ma + mi, kk)
#pragma unroll
                    for (int n = 2; n >= 0; --n) b[mi] = mfma_bf(yf, lds_bf8(ex + f * GDR_FRAG + n * GDR_TRI), b[mi]);
                }
            }
#pragma unroll
            for (int mi = 0; mi < 2; ++mi) {
                const int tok = 16 * (ma + mi) + jj, at = YO + col + 4 * g;
                const f32x4 dy = widen(*reinterpret_cast<const u32x2*>(ty + tile_off(tok, at >> 3) + 2 * (at & 7)));
                const f32x4 d = rec[SSM_DT + tok] * (rec[SSM_GA + tok] * ds[half][mi] + b[mi]) + skip * dy;
                // rows past the chunk's end lie past the buffer's and are dropped
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(__attribute__((ext_vector_type(2))) unsigned int,
                                                                         u32x2{pack_bf2(d[0], d[1]), pack_bf2(d[2], d[3])}),
                                                      rdx, tok * dst * 2 + 2 * (col + 4 * g), 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- what the tokens' numbers are made of, into the head's record behind the steps: a wave a row
        {
            const int I = lane >> 4;
            float x = 0.f;
            if (wave == 0) {
#pragma unroll
                for (int j = 0; j < 3; ++j) x += j < I ? sRS[64 * j + lane] : 0.f;
            } else if (wave == 1) {
#pragma unroll
                for (int i = 1; i < 4; ++i) x += i > I ? sCS[64 * i + lane] : 0.f;
            } else if (wave == 2) {
                x = sCS[64 * I + lane];
            } else if (wave == 3) {
                x = sDR[lane];
            } else if (wave == 4 || wave == 5) {
                const float* s = wave == 4 ? sU : sY;
#pragma unroll
                for (int w = 0; w < S / 16; ++w) x += s[64 * w + lane];
                x *= rec[(wave == 4 ? SSM_GA : SSM_EG) + lane];
            } else if (wave == 6) {
                x = lane < 8 ? sS[lane] * rec[SSM_EG + 63] : lane < 15 ? sS[lane] : 0.f;
                const float q = sum16(lane < 8 ? x : 0.f), d = sum16(lane >= 8 && lane < 12 ? x : 0.f);
                x = lane == 0 ? q : lane == 1 ? d : x;
            }
            if (wave < 7) reinterpret_cast<float*>(prec)[64 * (wave + 1) + lane] = x;
        }
        px += p.x.sh;
        py += p.dO.sh;
        pdx += P;
        ps += S * P;
        pds += S * P;
        prec += SSM_REC;
        if (p.D) ++pd;
        __syncthreads();   // everything in LDS but B and C is read
    }

    // ---- dB and dC: a lane holds four channels of token 16 m + jj
    const int n = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
    const int64_t base = ((int64_t)set * p.nslots + slot) * 64;
#pragma unroll
    for (int mi = 0; mi < MW; ++mi) {
        const int tok = 16 * (m0 + mi) + jj;
        if (tok >= ch.rows) continue;
        if (p.sets > 1) {
            const int64_t at = ((base + tok) * p.G + group) * S + n;
            *reinterpret_cast<f32x4*>(p.dBp + at) = dB[mi];
            *reinterpret_cast<f32x4*>(p.dCp + at) = dC[mi];
        } else {
            const int64_t at = ((ch.row * p.T + ch.tok + tok) * p.G + group) * S + n;
            *reinterpret_cast<u32x2*>(p.dB + at) = u32x2{pack_bf2(dB[mi][0], dB[mi][1]), pack_bf2(dB[mi][2], dB[mi][3])};
            *reinterpret_cast<u32x2*>(p.dC + at) = u32x2{pack_bf2(dC[mi][0], dC[mi][1]), pack_bf2(dC[mi][2], dC[mi][3])};
        }
    }
}

// The tokens' numbers of a chunk: ddt, and the chunk's part of the heads' sums.  A wave for each head,
// lane = token, sixteen heads a work-group; ddt goes through LDS, so that the heads of a token are
// stored side by side.
__global__ void __launch_bounds__(1024) kda_ssm_numbers_kernel(const SsmParams p) {
    __shared__ float sh[64][17];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), I = lane >> 4;
    const int sixteens = (p.H + 15) / 16, h0 = (int)(blockIdx.x % sixteens) * 16, h = h0 + w;
    const int64_t slot = blockIdx.x / sixteens;
    const SsmChunk ch = ssm_chunk(p, slot);
    float sa = 0.f, sd = 0.f, own = 0.f;
    if (h < p.H && ch.rows > 0) {
        const float* r = reinterpret_cast<const float*>(p.rec + (slot * p.H + h) * SSM_REC) + lane;
        const float d = r[0], rs = r[64], cs = r[128], csd = r[192], dr = r[256], u = r[320], y = r[384], x = r[448];
        const float q = lane_f32(x, 0), t20 = lane_f32(x, 12), t30 = lane_f32(x, 13), t31 = lane_f32(x, 14);
        float slope = 1.f;
        if (p.softplus && lane < ch.rows)
            slope = sigmoid<true>(ssm_raw(p.dt, p.dt_f32, ch.row * p.dtb + (ch.tok + lane) * p.dtt + h, p.bias, h));
        float da = suffix16(rs, lane) + before16(prefix16(cs * d)) + dr + (I == 1 ? t20 + t30 : I == 2 ? t30 + t31 : 0.f);
        da += suffix_wave(y, lane) + before_wave(prefix_wave(u * d), lane) + q;
        if (lane < ch.rows) {
            own = (p.A[h] * da + (u + cs + csd)) * slope;
            sa = d * da;
        }
        sd = lane_f32(x, 1);
    }
    sh[lane][w] = own;
    own = sum64(own);
    sa = sum64(sa);
    if (lane < 3 && h < p.H) p.part[(slot * 3 + lane) * p.H + h] = lane == 0 ? sa : lane == 1 ? sd : own;
    __syncthreads();
    const int tok = threadIdx.x >> 4, i = threadIdx.x & 15;
    if (tok < ch.rows && h0 + i < p.H) p.ddt[(ch.row * p.T + ch.tok + tok) * p.H + h0 + i] = sh[tok][i];
}

// dB and dC of a chunk as sums over its sets of heads, in order; a thread takes four channels of one of them.
__global__ void __launch_bounds__(256) kda_ssm_join_kernel(const SsmParams p) {
    const int row = p.G * p.S, groups = row / 8;   // elements of a token; work-groups of a chunk
    const int64_t slot = blockIdx.x / groups;
    const int i = (int)(blockIdx.x % groups) * 256 + threadIdx.x;
    const bool c = i >= 16 * row;
    const int e = 4 * (c ? i - 16 * row : i);
    const SsmChunk ch = ssm_chunk(p, slot);
    if (e >= ch.rows * row) return;
    const float* from = (c ? p.dCp : p.dBp) + slot * 64 * row + e;
    const int64_t step = p.nslots * 64 * row;
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < p.sets; ++s) a += *reinterpret_cast<const f32x4*>(from + s * step);
    *reinterpret_cast<u32x2*>((c ? p.dC : p.dB) + (ch.row * p.T + ch.tok) * row + e) = u32x2{pack_bf2(a[0], a[1]), pack_bf2(a[2], a[3])};
}

// The heads' sums over the chunks: dA, dD, dbias.  A work-group takes one of them and 16 heads, 64
// threads each every 64th chunk, then in order.
__global__ void __launch_bounds__(1024) kda_ssm_sums_kernel(const SsmParams p) {
    __shared__ double sh[64][16];
    const int g = threadIdx.x >> 4, l = threadIdx.x & 15, which = blockIdx.x % 3, h = (int)(blockIdx.x / 3) * 16 + l;
    float* out = which == 0 ? p.dA : which == 1 ? p.dD : p.dbias;
    double x = 0.0;
    if (out && h < p.H)
        for (int64_t s = g; s < p.nslots; s += 64) x += (double)p.part[(s * 3 + which) * p.H + h];
    sh[g][l] = x;
    __syncthreads();
    if (g > 0 || !out || h >= p.H) return;
    for (int i = 1; i < 64; ++i) x += sh[i][l];
    out[h] = (float)x;
}

hipError_t launch_ssm_grads(const SsmParams& p, hipStream_t stream) {
    const int64_t blocks = p.nslots * p.G * p.sets;
    if (blocks > 0) {
        auto* f = p.S == 128 ? (p.P == 128 ? kda_ssm_grads_kernel<128, 128> : kda_ssm_grads_kernel<128, 64>)
                             : (p.P == 128 ? kda_ssm_grads_kernel<64, 128> : kda_ssm_grads_kernel<64, 64>);
        hipLaunchKernelGGL(f, dim3((unsigned)blocks), dim3(NT), 0, stream, p);
        if (p.sets > 1) hipLaunchKernelGGL(kda_ssm_join_kernel, dim3((unsigned)(p.nslots * (p.G * p.S / 8))), dim3(256), 0, stream, p);
        hipLaunchKernelGGL(kda_ssm_numbers_kernel, dim3((unsigned)(p.nslots * ((p.H + 15) / 16))), dim3(1024), 0, stream, p);
    }
    hipLaunchKernelGGL(kda_ssm_sums_kernel, dim3((unsigned)(3 * ((p.H + 15) / 16))), dim3(1024), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
