// Device helpers of the gated delta rule with one decay per head.
//
// Matrix products run on the 16x16x32 instructions for bf16 operands.  q, k, v and the
// output's gradient are bf16; an fp32 operand enters as the sum of bf16 parts, each the
// rounding of what the parts before it leave: three hold all 24 bits at any size, so that
// products keep fp32's accuracy and range at a third to a sixth of the 16-bit rate, several
// times that of the fp32 matrix instructions.  (Two fp16 parts hold 22 bits for less, of
// what powers of two keep in range: entries far below their row's largest lose theirs.)
#pragma once
#include "kda_device.h"
#include "kda_gdr.h"

namespace kda {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 mfma_bf(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Eight fp32 values as NS bf16 parts, packed as MFMA operands.
template <int NS>
struct Split {
    bf16x8 s[NS];
};
// Values 2 i and 2 i + 1 into word i of the parts.  What a part leaves is formed by plain
// subtractions (exact): v_dot2c would take one instruction for two, but it occupies the
// matrix unit, and these run beside it.
template <int NS>
__device__ __forceinline__ void split_pair(u32x4 (&w)[NS], int i, float a, float b) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        w[n][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2v));
        if (n + 1 < NS) {
            a -= bf_lo(w[n][i]);
            b -= bf_hi(w[n][i]);
        }
    }
}
template <int NS>
__device__ __forceinline__ Split<NS> split8(const float (&x)[8]) {
    u32x4 w[NS];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_pair<NS>(w, i, x[2 * i], x[2 * i + 1]);
    Split<NS> r;
#pragma unroll
    for (int n = 0; n < NS; ++n) r.s[n] = __builtin_bit_cast(bf16x8, w[n]);
    return r;
}
// Two accumulator tiles (rows 4 g + r of each, r < 4) as the B operand of a 32-wide
// k step whose index runs over tile 0's four rows of lane group g, then tile 1's.
template <int NS>
__device__ __forceinline__ Split<NS> split_acc(f32x4 a, f32x4 b) {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return split8<NS>(x);
}

// Per-token rows of a record's numbers, in elements: e^G (the last is e^{G_last}), e^{G_last - G},
// beta; backward also the beta that u is formed with; forward also G as an fp32 value and its
// remainder.
enum { SC_EG = 0, SC_GA = 64, SC_BE = 128, SC_BU = 192, SC_GH = 192, SC_GL = 256 };

// ---- swizzled [64][128] bf16 tiles in LDS: rows of 256 bytes, whose sixteen 16-byte
// pieces are permuted by tsw(row), so that both an operand read (sixteen consecutive
// rows at one piece) and a transposing read (four consecutive rows at four
// consecutive pieces) touch every bank once.
__device__ __forceinline__ int tsw(int row) { return ((row & 3) << 2) | ((row >> 2) & 3); }
__device__ __forceinline__ int tile_off(int row, int piece) { return row * 256 + ((piece ^ tsw(row)) << 4); }

__device__ __forceinline__ bf16x8 lds_bf8(const char* p) { return *reinterpret_cast<const bf16x8*>(p); }

// Transposing read: in each group of 16 lanes, lane 4 a + b receives element b of the
// 8-byte pieces addressed by lanes a, a + 4, a + 8, a + 12 of the group.
__device__ __forceinline__ u32x2 lds_tr(const char* p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) v4i16*)(p)));
}

// Two transposing reads as one operand.
__device__ __forceinline__ bf16x8 join(u32x2 a, u32x2 b) {
    return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
}

// One 1 KB piece by DMA: lane l's 16 bytes at `voff` of the buffer to byte 16 l of
// the LDS address.  Nothing waits for it here; offsets past the buffer's range
// arrive as zeros.
__device__ __forceinline__ void dma_piece(__amdgpu_buffer_rsrc_t r, uint32_t lds, int voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(r)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const char* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

// Rows of a chunk (64 rows, `rows` of them real) of a bf16 tensor: base of its first
// row and the bytes that the real rows span.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const uint16_t* base, int64_t st, int rows, int cols) {
    return make_rsrc(base, rows > 0 ? ((int64_t)(rows - 1) * st + cols) * 2 : 0);
}
// The swizzled tile of a chunk's rows by DMA: the sixteen pieces split over `nw` waves.
__device__ __forceinline__ void dma_tile(__amdgpu_buffer_rsrc_t r, uint32_t lds, int64_t st, int wave, int nw, int lane) {
    for (int u = wave; u < 16; u += nw) {
        const int row = 4 * u + (lane >> 4);
        dma_piece(r, __builtin_amdgcn_readfirstlane(lds + u * 1024),
                  (int)(row * st * 2) + (((lane & 15) ^ tsw(row)) << 4));
    }
}

// A copy of x that the compiler cannot see through: per-lane addresses derived from it
// are formed where they are used instead of being kept across a loop.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// The order of a stretch of code that ends here: after each of N matrix instructions up to
// VALU vector instructions, DS reads of LDS and VM stores.  Left to itself the compiler
// forms one tile after the other, each a chain of dependent matrix instructions that waits
// for its operands in between.
template <int N, int VALU, int DS, int VM>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (VALU) __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
        if (DS) __builtin_amdgcn_sched_group_barrier(0x100, DS, 0);
        if (VM) __builtin_amdgcn_sched_group_barrier(0x040, VM, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// ---- walks over the chunks: a wave owns sixteen columns of the state in eight accumulator tiles ----
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
// y = a triangular matrix in three parts times x, fragment(part, m, kk) its operands: the
// parts' products of 2^-16 and more of the leading one's, the small parts first, six tiles
// side by side.  work(n), n = 2, 1, 0, is done meanwhile.
template <bool UPPER, typename F, typename W>
__device__ __forceinline__ void tri_times(F fragment, const f32x4 (&x)[4], f32x4 (&y)[4], W work) {
    // the six (m, kk) of the triangle: lower kk <= m / 2, upper kk >= m / 2
    constexpr int M[6] = {0, 1, 2, 3, UPPER ? 0 : 2, UPPER ? 1 : 3};
    constexpr int KK[6] = {0, 0, UPPER ? 1 : 0, UPPER ? 1 : 0, 1, 1};
    bf16x8 f[2][6];
    f32x4 a[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        f[0][i] = fragment(2, M[i], KK[i]);
        a[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const Split<3> xb[2] = {split_acc<3>(x[0], x[1]), split_acc<3>(x[2], x[3])};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 2; n >= 0; --n) {
        if (n) {
#pragma unroll
            for (int i = 0; i < 6; ++i) f[(n + 1) & 1][i] = fragment(n - 1, M[i], KK[i]);
        }
        work(n);
#pragma unroll
        for (int d = 2 - n; d >= 0; --d) {
#pragma unroll
            for (int i = 0; i < 6; ++i) a[i] = mfma_bf(f[n & 1][i], xb[KK[i]].s[d], a[i]);
            if (d == 2 - n) interleave<6, 2, 2, 0>();
            else interleave<6, 2, 0, 0>();
        }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) y[m] = (M[4] == m) ? a[m] + a[4] : (M[5] == m) ? a[m] + a[5] : a[m];
}

// ---- chunks ----
// First token (in its row), length and row of sequence n, clamped to the row.
__device__ __forceinline__ void gdr_seq(const GdrParams& p, int n, int64_t& bos, int64_t& len, int64_t& row,
                                        int64_t& slot0) {
    if (p.cu) {
        int64_t a = p.cu[n], e = p.cu[n + 1];
        a = a < 0 ? 0 : (a > p.T ? p.T : a);
        e = e < a ? a : (e > p.T ? p.T : e);
        bos = a;
        len = e - a;
        row = 0;
        slot0 = a / CH + n;
    } else {
        bos = 0;
        len = p.T;
        row = n;
        slot0 = (int64_t)n * p.nc;
    }
}
// The chunk in slot s: its sequence, first token and real rows (0: the slot is empty).
// Packed sequence n's slots start at cu[n] / 64 + n, which grows with n.
__device__ __forceinline__ int gdr_chunk(const GdrParams& p, int64_t s, int64_t& tok, int64_t& row) {
    int n;
    if (p.cu) {
        int lo = 0, hi = p.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            int64_t a = p.cu[mid];
            a = a < 0 ? 0 : (a > p.T ? p.T : a);
            if (a / CH + mid <= s) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
    } else {
        n = (int)s / p.nc;
    }
    int64_t bos, len, slot0;
    gdr_seq(p, n, bos, len, row, slot0);
    const int64_t c = s - slot0;
    tok = bos + c * CH;
    const int64_t r = len - c * CH;
    return c < 0 || r <= 0 ? 0 : (r >= CH ? CH : (int)r);
}

// beta of element i.
__device__ __forceinline__ float gdr_beta(const void* beta, int f32, int64_t i) {
    return f32 ? reinterpret_cast<const float*>(beta)[i] : bf2f(reinterpret_cast<const uint16_t*>(beta)[i]);
}
// The beta that the backward forms u with: none nearer to zero than 2^-40.  dbeta is u's product
// with a gradient divided by it, and an update of 2^-40 is far below what the state's 24 bits
// hold.  The other gradients take u times beta_share: beta over the one it is formed with.
__device__ __forceinline__ float beta_of_u(float b) { return fabsf(b) < 0x1p-40f ? 0x1p-40f : b; }
__device__ __forceinline__ float beta_share(float b) { return fabsf(b) < 0x1p-40f ? b * 0x1p40f : 1.f; }

// x of the lane that a DPP control names, 0 where it names none (or the row is masked out).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double x) {
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROWS, 0xf, true),
                                            (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROWS, 0xf, true)});
}
// Sum of x over this lane and those before it in the wave: within rows of 16 lanes by
// shifts, then each row's total on to the rows after it.
__device__ __forceinline__ double prefix64(double x) {
    x += dpp_f64<0x111, 0xf>(x);   // row_shr 1, 2, 4, 8
    x += dpp_f64<0x112, 0xf>(x);
    x += dpp_f64<0x114, 0xf>(x);
    x += dpp_f64<0x118, 0xf>(x);
    x += dpp_f64<0x142, 0xa>(x);   // row_bcast 15 into rows 1 and 3
    x += dpp_f64<0x143, 0xc>(x);   // row_bcast 31 into rows 2 and 3
    return x;
}
// x of one lane, in every lane (to be called where all lanes are active).
__device__ __forceinline__ double lane_f64(double x, int lane) {
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)w[0], lane),
                                            (uint32_t)__builtin_amdgcn_readlane((int)w[1], lane)});
}

// Running sum of a chunk's log-decays in units of log 2, lane i holding token i's:
// summed in 64 bits and kept as an fp32 value and its remainder, so that differences
// of far sums keep fp32's relative accuracy.  Log-decays below -200 (minus infinity
// too) count as -200: their factor is 0 in fp32 either way, and sums stay finite.
struct GSum {
    float hi, lo;
};
__device__ __forceinline__ GSum gate_sum(float g) {
    const double x = prefix64((double)(g < -200.f ? -200.f : g) * 1.4426950408889634074);
    const float hi = (float)x;
    return {hi, (float)(x - (double)hi)};
}
// 2^(a - b)
__device__ __forceinline__ float gate_ratio(GSum a, GSum b) {
    const float d = a.hi - b.hi;
    return fexp2(d) * fmaf(a.lo - b.lo, LN2, 1.f);
}
__device__ __forceinline__ float gate_exp(GSum a) { return fexp2(a.hi) * fmaf(a.lo, LN2, 1.f); }

// x of the lane N places on in its group of 16 lanes (row_ror: no LDS access).
template <int N>
__device__ __forceinline__ float ror16(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + N, 0xf, 0xf, true));
}
// Sum over the 16 lanes of a group (lane & 15), the same bits in every lane.
__device__ __forceinline__ float sum16(float x) {
    x += ror16<8>(x);
    x += ror16<4>(x);
    x += ror16<2>(x);
    return x + ror16<1>(x);
}
// x of this lane and of the lane 16, or 32, places away (lane ^ N), in either order: for sums,
// the same bits in both lanes, without an LDS access.
struct Pair {
    float a, b;
};
template <int N>
__device__ __forceinline__ Pair across(float x) {
    const uint32_t v = __float_as_uint(x);
    const auto r = N == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
// Sum over the four lane groups, in every one.
__device__ __forceinline__ float sum_groups(float x) {
    const Pair p = across<16>(x), q = across<32>(p.a + p.b);
    return q.a + q.b;
}
// Sum over the wave.
__device__ __forceinline__ float sum64(float x) { return sum_groups(sum16(x)); }

// The (sequence, value head, 64-wide slice of value channels) of a walk's work-group.
// Work-groups start in order and are dealt to the 8 XCDs round robin.  An XCD takes an
// eighth of the heads of every sequence, both slices of a head and a group's heads
// together, so that they share k, q and the records in one L2.  Packed sequences are
// taken longest first (ties in order), so that the last work-groups to start are short:
// `sh` holds N + 1 words for that.  With more sequences than threads they keep their order.
//   Forward of 11 sequences of 16,384 tokens on 64 heads, 16 of q and k: longest first 594 us,
// in order 690; its gradients on 7 of 4096 tokens and 32 heads 371 and 405.  Heads dealt to
// the XCDs: the same forward 594 us, in order 614; at B=2 H=64 T=8192 608 and 618.
struct Walk {
    int n, hv, sl;
};
template <int SLICES>   // 2, or 1: whole heads
__device__ __forceinline__ Walk walk_of_block(const GdrParams& p, int b, int* sh) {
    Walk k;
    if ((p.Hv & 7) == 0) {
        const int per = p.Hv >> 3, rest = b / (8 * SLICES);
        k.sl = (b >> 3) % SLICES;
        k.n = rest / per;
        k.hv = (b & 7) * per + rest % per;
    } else {
        k.sl = b % SLICES;
        k.n = b / SLICES / p.Hv;
        k.hv = b / SLICES % p.Hv;
    }
    if (p.cu && p.N > 1 && p.N <= (int)blockDim.x) {
        const int t = threadIdx.x;
        if (t < p.N) {
            int64_t a = p.cu[t], e = p.cu[t + 1];
            a = a < 0 ? 0 : (a > p.T ? p.T : a);
            e = e < a ? a : (e > p.T ? p.T : e);
            sh[1 + t] = (int)(e - a);
        }
        __syncthreads();
        if (t < p.N) {
            const int mine = sh[1 + t];
            int rank = 0;
            for (int m = 0; m < p.N; ++m) rank += sh[1 + m] > mine || (sh[1 + m] == mine && m < t);
            if (rank == k.n) sh[0] = t;
        }
        __syncthreads();
        k.n = __builtin_amdgcn_readfirstlane(sh[0]);
        __syncthreads();   // read before the words are used for something else
    }
    return k;
}

}  // namespace kda
