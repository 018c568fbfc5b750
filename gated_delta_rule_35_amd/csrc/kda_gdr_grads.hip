// Token gradients of the gated delta rule with one decay per head, all chunks at once,
// on gfx950 (MI355X).
//
// From the walks: S the state entering the chunk, dS the gradient of the one leaving
// it, u the corrected values, dx the gradient of beta (v - e^G K S).  With Gam_ij =
// e^{G_i - G_j}, gam_i = e^{G_last - G_i}, P = scale Gam (do u^T) (j <= i),
// E = -beta_i Gam (dx u^T) (j < i), R1 = do S^T, R2 = u dS^T, R3 = dx S^T:
//   dq = scale e^G R1 + P K
//   dk = gam R2 - beta e^G R3 + P^T Q + (E + E^T) K
//   dbeta_i = dx_i . u_i / beta_i           (u = beta times what it multiplies)
//   z_i = scale e^{G_i} q_i . R1_i - beta_i e^{G_i} k_i . R3_i
//         + (row i - column i of P (QK^T) + E (KK^T) below the diagonal)
//   dg_t = sum_{i >= t} z_i + sum_{i < t} gam_i k_i . R2_i + e^{G_last} <S, dS>, within the chunk
// (z_i - gam_i k_i . R2_i sums to do . o - dv . v per token, but every term above carries the
// decays that it passes, g_t's among them, but for the pairs behind t, whose rows and columns
// cancel: dg keeps its accuracy where the state is soon forgotten.  Summed as all tokens' k . R2
// less those from t on, what leaves the chunk without passing a decay left 2^-24 of itself.)
//
// One 512-thread work-group per compute unit takes items (chunk slot, q/k head), walks
// the group's value heads and sums their dq and dk in registers (so the sum's order is
// fixed); the next unit's S, u, dx and do are loaded into registers as soon as those of
// this one's are free, and dS while S's products run.  It holds the chunk's do, u and dx
// (u and dx in three bf16 parts) and k, q in LDS; wave w owns channels 16 w .. + 15 of R1, R2, R3, dq and
// dk, so S and dS are read once and split once; the ten lower 16x16 tiles of P and of E
// are dealt to the eight waves.  Every product is formed transposed (channels or the
// earlier token down, tokens across), so that a lane holds one token and four channels: a
// dot over channels is four products in the lane and two exchanges, per-token factors are
// one number, and results leave four at a time.
//   Precision: S, dS, u and dx enter in three bf16 parts each, which dg needs and which have
// fp32's range: value channels and tokens of any sizes beside each other; P and E enter dq and
// dk, which are rounded to bf16, in two.  (Rows of two fp16 parts, brought to one size by
// powers of two, took 1080 us and lost every channel far below its
// row's largest.)
//   The kernel reads 64 KB each of S and dS and 32 KB each of u and dx per chunk and value
// head.  At B=2 H=64 T=8192 it takes 1200 us, 4.7 GB at 3.9 TB/s; LDS, vector and matrix
// units are busy a quarter to a half of the time, with four barriers a unit.
// What brought it there from 2080 us: results formed transposed, inputs asked for in steps,
// arguments read anew instead of kept in spilled scalar registers (1600 -> 1440 us), the
// chains of four tiles side by side (1440 -> 1350 us), inputs asked for as soon as there are
// registers (-> 1320 us), sums across lane groups by v_permlane swaps instead of through LDS.
#include <type_traits>

#include "kda_gdr_device.h"

namespace kda {

namespace {
constexpr int GT = 512;
constexpr int PS = 144;   // bytes per row of 64 bf16 (+16)
struct GL {
    static constexpr int K = 0, Q = 16384, DO = 32768, U = 49152, X = U + 3 * 16384;   // U, X in three parts
    static constexpr int PL = 64 * PS;                  // one part of P or E, over U
    static constexpr int END = X + 3 * 16384;
    static_assert(4 * PL <= 3 * 16384, "overlay");
};
struct GShared {
    float hi[64], lo[64];  // G
    float eg[64], ga[64], be[64], xu[64];   // ga times beta's share of u; xu: dx . u
    float su[64];          // beta's share of u
    float z[8][64], k2[8][64];   // the row dots of z and k . R2 by wave (channel sixteenths)
    float row[20][16], col[20][16];   // row and column sums by tile: P (QK^T), then E (KK^T)
    float sd[8];           // <S, dS> by wave
};

// Operand of channels 16 w + jj: tokens 16 m + 4 g + r, r < 4.
__device__ __forceinline__ u32x2 chan_frag(const char* tile, int m, int w, int g, int jj) {
    return lds_tr(tile + tile_off(16 * m + 4 * g + (jj >> 2), 2 * w + ((jj & 3) >> 1)) + 8 * (jj & 1));
}
// Channels 16 w + 4 g + e, e < 4, of token 16 m + jj.
__device__ __forceinline__ f32x4 chan4(const char* tile, int m, int w, int g, int jj) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(tile + tile_off(16 * m + jj, 2 * w + (g >> 1)) + 8 * (g & 1));
    return f32x4{bf_lo(x[0]), bf_hi(x[0]), bf_lo(x[1]), bf_hi(x[1])};
}
// c += A B, both in parts, without the products below 2^-24 of the leading one; small ones first.
template <int NB>
__device__ __forceinline__ f32x4 mfma_parts(const Split<3>& a, const bf16x8 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int d = 2; d >= 0; --d) {
#pragma unroll
        for (int i = 0; i <= d; ++i)
            if (d - i < NB) c = mfma_bf(a.s[i], b[d - i], c);
    }
    return c;
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return fmaf(a[0], b[0], fmaf(a[1], b[1], fmaf(a[2], b[2], a[3] * b[3]))); }
// Operand (m, kk) of a 64x64 plane: rows 16 m + jj, columns of k step kk; and of its transpose.
__device__ __forceinline__ bf16x8 plane_row(const char* pl, int m, int kk, int g, int jj) {
    const char* a = pl + (16 * m + jj) * PS + 64 * kk + 8 * g;
    return join(*reinterpret_cast<const u32x2*>(a), *reinterpret_cast<const u32x2*>(a + 32));
}
__device__ __forceinline__ bf16x8 plane_col(const char* pl, int m, int kk, int g, int jj) {
    const char* a = pl + (32 * kk + 4 * g + (jj >> 2)) * PS + 32 * m + 8 * (jj & 3);
    return join(lds_tr(a), lds_tr(a + 16 * PS));
}
// The kernel's arguments, read anew at each use (a scalar load): kept in registers through
// the loop they would not fit the scalar ones.
typedef const __attribute__((address_space(4))) GdrParams Args;
__device__ __forceinline__ Args& args_again() {
    Args* a = (Args*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(a));
    return *a;
}
}  // namespace

__global__ void __launch_bounds__(GT) kda_gdr_grads_kernel(const GdrParams p, const int items) {
    __shared__ __attribute__((aligned(1024))) char smem[GL::END];
    __shared__ GShared sh;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int R = p.Hv / p.Hq;
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const f32x4 z4 = {0.f, 0.f, 0.f, 0.f};

    // The unit at hand, one value head r of an item (chunk slot, q/k head); item >= items: none.
    int item = blockIdx.x, r = 0, rows = 0, hq = 0;
    int64_t slot = 0, tok = 0, row = 0;
    auto find = [&]() {   // the first item from `item` on whose slot holds a chunk
        for (; item < items; item += gridDim.x) {
            slot = item / p.Hq;
            hq = item % p.Hq;
            rows = gdr_chunk(p, slot, tok, row);
            if (rows) break;
        }
    };
    f32x4 u[4], x[4], s[8];
    float gate = 0.f, beta = 0.f;
    // the unit's fp32 inputs into registers
    auto fetch_state = [&](const float* from, f32x4 (&to)[8]) {
        const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
        const float* at = from + (slot * p.Hv + hq * R + r) * DK * DK + (16 * w + jj) * DK + 8 * g;
#pragma unroll
        for (int n = 0; n < 8; ++n) to[n] = *reinterpret_cast<const f32x4*>(at + 32 * (n >> 1) + 4 * (n & 1));
    };
    auto fetch_tokens = [&]() {
        Args& p = args_again();
        const int t = opaque(tid), lane = t & 63;
        const int64_t unit = slot * p.Hv + hq * R + r;
        if (w == 6) {
            const int64_t gi = (row * p.T + tok + lane) * p.Hv + hq * R + r;
            gate = lane < rows ? p.g[gi] : 0.f;
            beta = lane < rows ? gdr_beta(p.beta, p.beta_f32, gi) : 0.f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = unit * CH * DK + (32 * h + (t >> 4)) * DK + 8 * (t & 15);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                u[2 * h + n] = *reinterpret_cast<const f32x4*>(p.u + at + 4 * n);
                x[2 * h + n] = *reinterpret_cast<const f32x4*>(p.dx + at + 4 * n);
            }
        }
    };
    auto dma_do = [&]() {
        Args& p = args_again();
        dma_tile(chunk_rsrc(p.dO.p + row * p.dO.sb + tok * p.dO.st + (hq * R + r) * p.dO.sh, p.dO.st, rows, DK),
                 lds + GL::DO, p.dO.st, w, 8, opaque(lane));
    };
    auto dma_kq = [&]() {
        Args& p = args_again();
        const int lane = opaque(tid & 63);
        dma_tile(chunk_rsrc(p.k.p + row * p.k.sb + tok * p.k.st + hq * p.k.sh, p.k.st, rows, DK), lds + GL::K, p.k.st, w,
                 8, lane);
        dma_tile(chunk_rsrc(p.q.p + row * p.q.sb + tok * p.q.st + hq * p.q.sh, p.q.st, rows, DK), lds + GL::Q, p.q.st, w,
                 8, lane);
    };
    find();
    if (item >= items) return;
    fetch_tokens();
    dma_do();
    dma_kq();
    fetch_state(args_again().S, s);
    f32x4 dq[4], dk[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) dq[m] = dk[m] = z4;

    while (item < items) {
        f32x4 ds[8];   // needed after S's products: in flight until then
        fetch_state(args_again().dS, ds);
        // u and dx in three parts, and dx . u
        const int t = opaque(tid);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pc = t & 15, i = 32 * h + (t >> 4), at = tile_off(i, pc);
            const Split<3> u3 = split_acc<3>(u[2 * h], u[2 * h + 1]);
            const Split<3> x3 = split_acc<3>(x[2 * h], x[2 * h + 1]);
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                *reinterpret_cast<bf16x8*>(smem + GL::U + n * 16384 + at) = u3.s[n];
                *reinterpret_cast<bf16x8*>(smem + GL::X + n * 16384 + at) = x3.s[n];
            }
            const f32x4 a = x[2 * h] * u[2 * h] + x[2 * h + 1] * u[2 * h + 1];
            const float xu = sum16((a[0] + a[1]) + (a[2] + a[3]));
            if (pc == 0) sh.xu[i] = xu;
        }
        if (w == 6) {
            const GSum G = gate_sum(gate);
            const GSum last = {__shfl(G.hi, 63), __shfl(G.lo, 63)};
            sh.hi[lane] = G.hi;
            sh.lo[lane] = G.lo;
            sh.eg[lane] = gate_exp(G);
            sh.su[lane] = beta_share(beta);
            sh.ga[lane] = gate_ratio(last, G) * beta_share(beta);
            sh.be[lane] = beta;
        }
        asm volatile("s_waitcnt vmcnt(8)" ::: "memory");   // this wave's pieces of do, k and q; dS may be on its way
        lds_barrier();

        const int rows0 = rows, hq0 = hq;
        const int64_t tok0 = tok, row0 = row, gi0 = (row * p.T + tok) * p.Hv + hq * R + r;
        const bool done = r == R - 1;   // the item's last value head
        // R1, R3, then R2, for channels 16 w + jj
        {
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            // k steps outermost: eight (then four) chains of products side by side, one step's parts at a time
            f32x4 r1[4], r3[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) r1[m] = r3[m] = z4;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const Split<3> sb = split_acc<3>(s[2 * kk], s[2 * kk + 1]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int at = tile_off(16 * m + jj, 4 * kk + g);
                    const bf16x8 fo[1] = {lds_bf8(smem + GL::DO + at)};
                    bf16x8 fx[3];
#pragma unroll
                    for (int n = 0; n < 3; ++n) fx[n] = lds_bf8(smem + GL::X + n * 16384 + at);
                    r1[m] = mfma_parts(sb, fo, r1[m]);
                    r3[m] = mfma_parts(sb, fx, r3[m]);
                }
            }
            float z[4];   // the lane's part of its tokens' row dots
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float eg = sh.eg[16 * m + jj];
                r1[m] *= p.scale * eg;
                r3[m] *= sh.be[16 * m + jj] * eg;
                dq[m] += r1[m];
                dk[m] -= r3[m];
                z[m] = dot4(chan4(smem + GL::Q, m, w, g, jj), r1[m]) - dot4(chan4(smem + GL::K, m, w, g, jj), r3[m]);
            }
            {
                f32x4 d4 = z4;
#pragma unroll
                for (int n = 0; n < 8; ++n) d4 += s[n] * ds[n];
                const float sd = sum64((d4[0] + d4[1]) + (d4[2] + d4[3]));
                if (lane == 0) sh.sd[w] = sd;
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) asm volatile("" : "+v"(ds[n]));   // dS's parts are formed after S's are done with
            // the next unit, whose inputs are asked for as soon as there are registers or LDS to put
            // them in: S now
            if (done) {
                r = 0;
                item += gridDim.x;
                find();
            } else {
                ++r;
            }
            if (item < items) fetch_state(args_again().S, s);
            f32x4 r2[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) r2[m] = z4;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const Split<3> sb = split_acc<3>(ds[2 * kk], ds[2 * kk + 1]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int at = tile_off(16 * m + jj, 4 * kk + g);
                    bf16x8 fu[3];
#pragma unroll
                    for (int n = 0; n < 3; ++n) fu[n] = lds_bf8(smem + GL::U + n * 16384 + at);
                    r2[m] = mfma_parts(sb, fu, r2[m]);
                }
            }
            float k2[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                r2[m] *= sh.ga[16 * m + jj];
                dk[m] += r2[m];
                k2[m] = sum_groups(dot4(chan4(smem + GL::K, m, w, g, jj), r2[m]));
                z[m] = sum_groups(z[m]);
            }
            sh.z[w][lane] = g == 0 ? z[0] : g == 1 ? z[1] : g == 2 ? z[2] : z[3];   // group m writes tokens 16 m ..
            sh.k2[w][lane] = g == 0 ? k2[0] : g == 1 ? k2[1] : g == 2 ? k2[2] : k2[3];
        }
        if (item < items) fetch_tokens();   // and u and dx now
        // lower tiles of P and E, transposed (lane: token i = 16 I + jj, j = 16 J + 4 g + e): wave w
        // has tile w of both; tiles 8 and 9 of P go to waves 0 and 1, of E to waves 2 and 3
        auto tile_rc = [&](int id, int& I, int& J) {
            I = id >= 6 ? 3 : id >= 3 ? 2 : id >= 1 ? 1 : 0;
            J = id - I * (I + 1) / 2;
        };
        // tile `id` of P, of E, or of both (u's and k's operands serve both), and the row and column
        // sums of their entries below the diagonal times QK^T and KK^T
        auto tile = [&](auto of_p, auto of_e, int id, f32x4& P, f32x4& E) {
            constexpr bool OF_P = decltype(of_p)::value, OF_E = decltype(of_e)::value;
            int I, J;
            tile_rc(id, I, J);
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            const int i = 16 * I + jj, j0 = 16 * J + 4 * g;
            f32x4 a = z4, ra = z4, b = z4, rb = z4;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                if (kk == 2) asm volatile("" ::: "memory");   // two steps' operands at a time: more would spill
                const int ai = tile_off(16 * I + jj, 4 * kk + g), aj = tile_off(16 * J + jj, 4 * kk + g);
                const Split<3> ua = {{lds_bf8(smem + GL::U + aj), lds_bf8(smem + GL::U + 16384 + aj),
                                      lds_bf8(smem + GL::U + 32768 + aj)}};
                const bf16x8 kj = lds_bf8(smem + GL::K + aj);
                if (OF_P) {
                    const bf16x8 fo[1] = {lds_bf8(smem + GL::DO + ai)};
                    a = mfma_parts(ua, fo, a);
                    ra = mfma_bf(kj, lds_bf8(smem + GL::Q + ai), ra);
                }
                if (OF_E) {
                    const bf16x8 fx[3] = {lds_bf8(smem + GL::X + ai), lds_bf8(smem + GL::X + 16384 + ai),
                                          lds_bf8(smem + GL::X + 32768 + ai)};
                    b = mfma_parts(ua, fx, b);
                    rb = mfma_bf(kj, lds_bf8(smem + GL::K + ai), rb);
                }
            }
            const GSum Gi = {sh.hi[i], sh.lo[i]};
            const f32x4 hj = *reinterpret_cast<const f32x4*>(sh.hi + j0), lj = *reinterpret_cast<const f32x4*>(sh.lo + j0);
            const f32x4 su = *reinterpret_cast<const f32x4*>(sh.su + j0);
            f32x4 gam;
#pragma unroll
            for (int e = 0; e < 4; ++e) gam[e] = j0 + e <= i ? gate_ratio(Gi, GSum{hj[e], lj[e]}) * su[e] : 0.f;
            auto finish = [&](auto is_p, const f32x4& a, const f32x4& raw) -> f32x4 {
                constexpr bool IS_P = decltype(is_p)::value;
                const float by = IS_P ? p.scale : -sh.be[i];
                f32x4 v, cs;
                float rs = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {   // what lies above the diagonal stays out, NaN and infinity too
                    v[e] = j0 + e < i + IS_P ? by * (gam[e] * a[e]) : 0.f;
                    const float y = j0 + e < i ? v[e] * raw[e] : 0.f;
                    rs += y;
                    cs[e] = sum16(y);
                }
                rs = sum_groups(rs);
                const int at = IS_P ? id : 10 + id;
                if (g == 0) sh.row[at][jj] = rs;
                if (jj == 0) *reinterpret_cast<f32x4*>(&sh.col[at][4 * g]) = cs;
                return v;
            };
            if (OF_P) P = finish(std::true_type{}, a, ra);
            if (OF_E) E = finish(std::false_type{}, b, rb);
        };
        f32x4 P, E, Z = z4;
        tile(std::true_type{}, std::true_type{}, w, P, E);
        if (w < 2) tile(std::true_type{}, std::false_type{}, 8 + w, Z, Z);
        else if (w < 4) tile(std::false_type{}, std::true_type{}, 6 + w, Z, Z);
        lds_barrier();   // u's parts read; the sums complete
        // P and E as row-major planes of two bf16 parts
        {
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            auto put = [&](f32x4 v, int id, int part) {
                int I, J;
                tile_rc(id, I, J);
                char* to = smem + GL::U + part * GL::PL + (16 * I + jj) * PS + 2 * (16 * J + 4 * g);
                const uint32_t h0 = pack_bf2(v[0], v[1]), h1 = pack_bf2(v[2], v[3]);
                *reinterpret_cast<u32x2*>(to) = u32x2{h0, h1};
                *reinterpret_cast<u32x2*>(to + GL::PL) =
                    u32x2{pack_bf2(v[0] - bf_lo(h0), v[1] - bf_hi(h0)), pack_bf2(v[2] - bf_lo(h1), v[3] - bf_hi(h1))};
            };
            put(P, w, 0);
            put(E, w, 2);
            if (w < 2) put(Z, 8 + w, 0);
            else if (w < 4) put(Z, 6 + w, 2);
            // the tiles above the diagonal that operands cover: 8 bytes a thread
            const int e = opaque(tid), t = (e >> 6) & 1;
            *reinterpret_cast<u32x2*>(smem + GL::U + (e >> 7) * GL::PL + (32 * t + ((e >> 2) & 15)) * PS +
                                      2 * (32 * t + 16 + 4 * (e & 3))) = u32x2{0, 0};
        }
        if (w == 5 && lane < rows0) args_again().dbeta[gi0 + (int64_t)lane * args_again().Hv] = sh.xu[lane] / beta_of_u(sh.be[lane]);
        if (w == 7) {   // dg
            const int i = lane, I = i >> 4;
            const int64_t gi = gi0 + (int64_t)i * p.Hv;
            double z = 0.0, k2 = 0.0;
            float sd = 0.f;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                z += (double)sh.z[n][i];
                k2 += (double)sh.k2[n][i];
                sd += sh.sd[n];
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int ra = I * (I + 1) / 2 + n, ca = n * (n + 1) / 2 + I;
                if (n <= I) z += (double)sh.row[ra][i & 15] + (double)sh.row[10 + ra][i & 15];
                if (n >= I) z -= (double)sh.col[ca][i & 15] + (double)sh.col[10 + ca][i & 15];
            }
            const double sum = prefix64(z), rest = lane_f64(sum, 63) - sum + z;
            const double upto = prefix64(k2), before = __shfl_up(upto, 1);
            if (i < rows0) {
                Args& p = args_again();
                p.dg[gi] = (float)(rest + (i > 0 ? before : 0.0) + (double)(sh.eg[63] * sd));
            }
        }
        if (item < items) dma_do();
        lds_barrier();
        {
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            bf16x8 kb[2], qb[2];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                kb[kk] = join(chan_frag(smem + GL::K, 2 * kk, w, g, jj), chan_frag(smem + GL::K, 2 * kk + 1, w, g, jj));
                qb[kk] = join(chan_frag(smem + GL::Q, 2 * kk, w, g, jj), chan_frag(smem + GL::Q, 2 * kk + 1, w, g, jj));
            }
#pragma unroll
            for (int n = 1; n >= 0; --n) {
                const char* pp = smem + GL::U + n * GL::PL;
                const char* pe = smem + GL::U + (2 + n) * GL::PL;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {   // four tiles of dq and of dk side by side
#pragma unroll
                    for (int m = 2 * kk; m < 4; ++m) {
                        dq[m] = mfma_bf(kb[kk], plane_row(pp, m, kk, g, jj), dq[m]);
                        dk[m] = mfma_bf(kb[kk], plane_row(pe, m, kk, g, jj), dk[m]);
                    }
#pragma unroll
                    for (int m = 0; m < 2 * kk + 2; ++m) dk[m] = mfma_bf(qb[kk], plane_col(pp, m, kk, g, jj), dk[m]);
#pragma unroll
                    for (int m = 0; m < 2 * kk + 2; ++m) dk[m] = mfma_bf(kb[kk], plane_col(pe, m, kk, g, jj), dk[m]);
                }
            }
        }
        if (done) {   // dq and dk, rounded once: eight bytes a lane, the waves' make up whole rows in L2
            Args& p = args_again();
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            const int64_t at = ((row0 * p.T + tok0 + jj) * p.Hq + hq0) * DK + 16 * w + 4 * g;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (16 * m + jj < rows0) {
                    const int64_t to = at + (int64_t)16 * m * p.Hq * DK;
                    *reinterpret_cast<u32x2*>(p.dq + to) = u32x2{pack_bf2(dq[m][0], dq[m][1]), pack_bf2(dq[m][2], dq[m][3])};
                    *reinterpret_cast<u32x2*>(p.dk + to) = u32x2{pack_bf2(dk[m][0], dk[m][1]), pack_bf2(dk[m][2], dk[m][3])};
                }
                dq[m] = dk[m] = z4;
            }
        }
        lds_barrier();   // k, q and the planes are read
        if (done && item < items) dma_kq();
    }
}

hipError_t launch_gdr_grads(const GdrParams& p, int cus, hipStream_t stream) {
    const int64_t items = p.nslots * p.Hq;
    if (items == 0) return hipSuccess;
    const int64_t blocks = items < cus ? items : cus;
    hipLaunchKernelGGL(kda_gdr_grads_kernel, dim3((unsigned)blocks), dim3(GT), 0, stream, p, (int)items);
    return hipGetLastError();
}

}  // namespace kda
