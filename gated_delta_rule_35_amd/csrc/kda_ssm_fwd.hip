// The selective state space scan's walks over chunks of 64 tokens, on gfx950 (MI355X).  With
// d_t the steps, a_t = d_t A and G the running sum of a within a chunk:
//   y = e^G C S + (C B^T e^{G_i - G_j} d_j, j <= i, and D where i = j) x,   S <- e^{G_last} S + B^T (e^{G_last - G} d x)
// The state's transition is a number, so a sequence is cut into segments that are walked side by
// side: a first walk forms what each segment adds to the state, a small kernel chains them, and a second
// walk starts every segment from the state that enters it.  Where sequences and heads alone fill
// the compute units there is one segment and one walk.
//
// A work-group takes 256 of a group's value columns, or half of them where that leaves no compute unit with two (T = 195 on
// 8 heads 29 us and not 40, T = 2048 on 64 heads 59 and not 70: a SIMD then has one walk).  Eight waves walk, 32 columns each: their state is S / 16
// by 2 accumulator tiles, which as operands need no exchange (kda_gdr_fwd.hip has the order of their
// rows); two walks a SIMD fill each other's gaps.  Four more waves bring what the walks need into LDS and store y: a
// wave that waits for the memory's queue would keep its products waiting.  Three meetings a chunk:
//   1  C S                                                    | y of the last chunk out of LDS, x in its place
//   2  the pairs' products                                    | the next chunk's B, C and numbers (but e^G) into LDS
//   3  the state grows, and the pair matrix (C B^T with its   | e^G into LDS, y stored, x asked for a chunk ahead,
//      decays) of the next chunk, two waves half of it each   | B and C two
// B = 2, H = 64, P = 64, S = 128, T = 8192: 221 to 228 us a call (HBM alone 55).  In a trace, which parts the launches and where the
// clock is lower, a call takes 247: the numbers 14, the first walk 60, the chain 12, the second walk 161.  Of the second
// walk's 345,000 clocks, 21,600 a chunk, a SIMD spends 154,000 on vector and 127,000 on matrix instructions, a compute unit's LDS
// 153,000 and 51,000 on conflicts, and waves wait for 46% of theirs: no pipe is full, the meetings keep all walks
// in one phase.  T = 195 on 8 heads: 29 us, 25 of them the walk, 6.2 a chunk.
// y is formed transposed, so that a lane holds four channels of one token.  The decay between tokens of
// different blocks of sixteen is a product of a number of each token and one or two of the blocks,
// all at most 1 for A <= 0; within a block it is formed from the difference.
//
// Precision.  x, B and C are bf16, the state and all sums fp32, and what multiplies them enters in three bf16
// parts, fp32's 24 bits: the state in C S, the pair matrix with D, what enters the state.  y's terms may cancel: with
// two parts of the first two (200 us, not 221, at B = 2, H = 64, T = 8192) y was off by up to 2^-18 of its terms, and by
// 1.0 10^-4 of its norm from a 32-bit form that is now 2 10^-5 away.  Two parts of what enters the state would leave the
// final state 2^-19 of itself off.
#include "kda_ssm_device.h"

namespace kda {

namespace {

constexpr int WT = 768;   // eight walking and four loading waves

struct FL {   // LDS of the full walk; slots of B by chunk's parity
    static constexpr int C = 32768, X = C + 16384, PM = X + 32768, PARTS = 3 * GDR_TRI, REC = PM + 4 * PARTS, BYTES = REC + 4 * SSM_REC;
};
static_assert(FL::BYTES == 163840, "LDS");
struct AL {   // of the walk that forms what segments add: B, x and the records, all by chunk's parity
    static constexpr int X = 32768, REC = X + 65536, BYTES = REC + 4 * 2 * SSM_REC;
};

// Columns of x in LDS: rows of 128 bytes, whose eight 16-byte pieces are permuted in pairs by row / 2, so that
// neither transposing reads nor y's writes meet in a bank.  Byte of element c of row r.
__device__ __forceinline__ int x_off(int r, int c) { return r * 128 + (((c >> 3) ^ (((r >> 1) & 3) << 1)) << 4) + 2 * (c & 7); }
// Tokens 32 kk + 4 g + r and 16 more of columns c + jj, as an operand.
__device__ __forceinline__ bf16x8 x_frag(const char* x, int kk, int c, int ln) {
    const int r = 32 * kk + 4 * (ln >> 4) + ((ln & 15) >> 2);
    c += 4 * (ln & 3);
    return join(lds_tr(x + x_off(r, c)), lds_tr(x + x_off(r + 16, c)));
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Where a work-group is: a segment, 256 (or 128) columns of a group's heads, and of those the 64 of two walking
// waves and a loading one.
struct SsmWalk {
    SsmSegment sg;
    int64_t sslot, row, tok0, left;
    int group, head, pc, c0, nch;
    bool on;
    __device__ __forceinline__ int rows(int c) const {
        const int64_t r = left - (int64_t)c * CH;
        return r >= CH ? CH : (int)r;
    }
};
// Work-groups are dealt to the 8 XCDs round robin: a segment's go to one of them, since they share B and C.
__device__ __forceinline__ bool walk_place(const SsmParams& p, int block, int w, SsmWalk& k) {
    const int R = uniform(p.H / p.G), per = uniform((R * p.P + p.cols - 1) / p.cols), units = per * p.G;
    const int r = block >> 3, unit = uniform(r % units);
    k.sslot = uniform((int64_t)(r / units) * 8 + (block & 7));
    if (k.sslot >= p.segslots) return false;
    k.sg = ssm_segment(p, k.sslot);
    if (k.sg.index >= k.sg.count) return false;
    k.group = uniform(unit / per);
    const int col = uniform((unit % per) * p.cols + 64 * w);
    k.on = 64 * w < p.cols && col < R * p.P;
    k.head = uniform(k.group * R + (k.on ? col / p.P : 0));
    k.pc = uniform(col % p.P);
    k.c0 = k.sg.index * p.segc;
    k.left = k.sg.q.len - (int64_t)k.c0 * CH;
    const int64_t n = (k.left + CH - 1) / CH;
    k.nch = uniform(n <= 0 ? 0 : (n < p.segc ? (int)n : p.segc));
    k.row = k.sg.q.row;
    k.tok0 = k.sg.q.bos + (int64_t)k.c0 * CH;
    return true;
}

// What the loading waves hold on its way to LDS.  T tiles of [64][S] (B, or C and B), one after the
// other over the 256 lanes; 64 columns of x and a record for each wave.
template <int S, int T>
struct Tiles {
    static constexpr int PIECES = S / 8, N = T * 64 * PIECES / 256;   // 16-byte pieces of a row, of a lane
    u32x4 v[N];
    __device__ __forceinline__ void ask(const Rows* t, const SsmWalk& k, int c, int hl) {
        const int rows = k.rows(c);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const Rows& m = t[u * T / N];
            const int e = (u % (N / T)) * 256 + hl, r = e / PIECES;
            const __amdgpu_buffer_rsrc_t rs =
                chunk_rsrc(m.p + k.row * m.sb + (k.tok0 + (int64_t)c * CH) * m.st + k.group * m.sh, m.st, rows, S);
            v[u] = load16(rs, (int)(r * m.st * 2) + 16 * (e % PIECES));
        }
    }
    __device__ __forceinline__ void put(char* to, char* to2, int hl) const {   // to2: the second tile
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int e = (u % (N / T)) * 256 + hl;
            *reinterpret_cast<u32x4*>((u * T / N ? to2 : to) + tile_off(e / PIECES, e % PIECES)) = v[u];
        }
    }
};
struct Columns {
    u32x4 v[8];
    __device__ __forceinline__ void ask(const Rows& t, const SsmWalk& k, int c, int ln) {
        const __amdgpu_buffer_rsrc_t rs =
            chunk_rsrc(t.p + k.row * t.sb + (k.tok0 + (int64_t)c * CH) * t.st + k.head * t.sh + k.pc, t.st, k.rows(c), 64);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = load16(rs, (int)((8 * u + (ln >> 3)) * t.st * 2) + 16 * (ln & 7));
    }
    __device__ __forceinline__ void put(char* to, int ln) const {
#pragma unroll
        for (int u = 0; u < 8; ++u) *reinterpret_cast<u32x4*>(to + x_off(8 * u + (ln >> 3), 8 * (ln & 7))) = v[u];
    }
    __device__ __forceinline__ void get(const char* from, int ln) {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const u32x4*>(from + x_off(8 * u + (ln >> 3), 8 * (ln & 7)));
    }
    // y's rows; those past the chunk's end lie past the buffer's and are dropped
    __device__ __forceinline__ void store(const SsmParams& p, const SsmWalk& k, int c, int ln) const {
        const int st = p.H * p.P;
        const __amdgpu_buffer_rsrc_t rs =
            chunk_rsrc(p.y + ((k.row * p.T + k.tok0 + (int64_t)c * CH) * p.H + k.head) * p.P + k.pc, st, k.rows(c), 64);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(__attribute__((ext_vector_type(4))) unsigned int, v[u]), rs,
                                                   (8 * u + (ln >> 3)) * st * 2 + 16 * (ln & 7), 0, 0);
    }
};
struct Record {
    u32x4 v[2];
    __device__ __forceinline__ void ask(const SsmParams& p, const SsmWalk& k, int c, int ln) {
        const char* r = p.rec + ((k.sg.slot0 + k.c0 + c) * p.H + k.head) * SSM_REC + 16 * ln;
        v[0] = *reinterpret_cast<const u32x4*>(r);
        v[1] = *reinterpret_cast<const u32x4*>(r + 1024);
    }
    __device__ __forceinline__ void put(char* to, int ln) const {
        *reinterpret_cast<u32x4*>(to + 16 * ln) = v[0];
        *reinterpret_cast<u32x4*>(to + 1024 + 16 * ln) = v[1];
    }
    // The full walk's: one record for all chunks, since of the chunk at hand only e^G and SSM_W's row are read while the next
    // one's come in.  That row goes by the chunk's parity to its own place or to SSM_GA's, which is not used; e^G comes last.
    __device__ __forceinline__ void put_but_eg(char* to, int odd, int ln) const {
        if (ln < 16 || ln >= 48) *reinterpret_cast<u32x4*>(to + 16 * ln) = v[0];
        *reinterpret_cast<u32x4*>(to + (odd && ln >= 48 ? 4 * SSM_GA - 768 : 1024) + 16 * ln) = v[1];
    }
    __device__ __forceinline__ void put_eg(char* to, int ln) const {
        if (ln >= 16 && ln < 32) *reinterpret_cast<u32x4*>(to + 16 * ln) = v[0];
    }
};

// Row I of tiles of a chunk's pair matrix, in three parts, into the fragments (m, kk) of its lower triangle in
// LDS; D is added to its diagonal.  C B^T is formed transposed: tile (J, I) holds in a lane rows j = 16 J + 4 g + r of column i = 16 I + jj.
template <int S, int I>
__device__ __forceinline__ void pair_row(const char* tb, const char* tc, const float* rec, float skip, char* pm, int lane) {
    constexpr int KT = S / 32;
    const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
    f32x4 a[I + 1];
#pragma unroll
    for (int J = 0; J <= I; ++J) a[J] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < KT; ++kk) {
        const bf16x8 ck = row_frag(tc, I, kk, g, jj);
#pragma unroll
        for (int J = 0; J <= I; ++J) a[J] = mfma_bf(row_frag(tb, J, kk, g, jj), ck, a[J]);
    }
#pragma unroll
    for (int J = 0; J <= I; ++J) {
        const f32x4 d = num4(rec, SSM_DT, J, g);
        if (I == J) {
            const float hi = rec[SSM_GH + 16 * I + jj], lo = rec[SSM_GL + 16 * I + jj];
            const f32x4 hj = num4(rec, SSM_GH, J, g), lj = num4(rec, SSM_GL, J, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = formed(a[J][e] * fexp2((hi - hj[e]) + (lo - lj[e])));
                a[J][e] = 4 * g + e <= jj ? fmaf(v, d[e], 4 * g + e == jj ? skip : 0.f) : 0.f;
            }
        } else {
            float ri = rec[SSM_RI + 16 * I + jj];
            if (I > J + 1) ri *= rec[SSM_RI + 16 * J + 31];
            if (I > J + 2) ri *= rec[SSM_RI + 16 * J + 47];
            a[J] *= (num4(rec, SSM_KA, J, g) * d) * ri;
        }
        char* to = pm + tri_frag(I, J >> 1) * GDR_FRAG + 16 * ln + 8 * (J & 1);
        u32x4 part[3];
        split_pair<3>(part, 0, a[J][0], a[J][1]);
        split_pair<3>(part, 1, a[J][2], a[J][3]);
#pragma unroll
        for (int n = 0; n < 3; ++n) *reinterpret_cast<u32x2*>(to + n * GDR_TRI) = u32x2{part[n][0], part[n][1]};
    }
    __builtin_amdgcn_sched_barrier(0);
}
// Half of it: five tiles each.
template <int S>
__device__ __forceinline__ void pair_half(int half, const char* tb, const char* tc, const float* rec, float skip, char* pm, int lane) {
    if (half == 0) {
        pair_row<S, 3>(tb, tc, rec, skip, pm, lane);
        pair_row<S, 0>(tb, tc, rec, skip, pm, lane);
    } else {
        pair_row<S, 2>(tb, tc, rec, skip, pm, lane);
        pair_row<S, 1>(tb, tc, rec, skip, pm, lane);
    }
}

// A walking wave's state: tile t holds in a lane channels state_row(t, g, r) of columns 16 ct + jj.
template <int S>
struct State {
    static constexpr int NT = S / 16;
    f32x4 st[NT][2];
    __device__ __forceinline__ void load(const float* from, const SsmParams& p, int pc, int ln) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                st[t][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (!from) continue;
#pragma unroll
                for (int r = 0; r < 4; ++r) st[t][ct][r] = from[state_row(t, ln >> 4, r) * p.P + pc + 16 * ct + (ln & 15)];
            }
        }
    }
    __device__ __forceinline__ void store(float* to, const SsmParams& p, int pc, int ln) const {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
#pragma unroll
                for (int r = 0; r < 4; ++r) to[state_row(t, ln >> 4, r) * p.P + pc + 16 * ct + (ln & 15)] = st[t][ct][r];
            }
        }
    }
    // S <- el S + B^T (w x), el = e^{G_last}, w = e^{G_last - G} d (backwards e^G): 32 tokens at a time, the next ones' w x
    // formed beside the products.  c0: the wave's first column in x's rows; read() is called once x has been read.
    template <typename F>
    __device__ __forceinline__ void grow(const char* tb, const char* tx, int c0, float el, const float* w, int ln, F read) {
        constexpr int QS = NT / 2;
        const int g = ln >> 4, jj = ln & 15;
        Split<3> wx[2][2];
        auto weigh = [&](int kk, int c) {
            const u32x4 xx = __builtin_bit_cast(u32x4, x_frag(tx, kk, c0 + 16 * c, ln));
            wx[kk][c] = split_acc<3>(num4(w, 0, 2 * kk, g) * widen(u32x2{xx[0], xx[1]}),
                                     num4(w, 0, 2 * kk + 1, g) * widen(u32x2{xx[2], xx[3]}));
        };
        bf16x8 bq[2][2];
        auto columns = [&](int q) {   // of step q: k step q / QS, tiles 2 (q % QS) ..
#pragma unroll
            for (int t = 0; t < 2; ++t) bq[q & 1][t] = col_frag(tb, 2 * (q % QS) + t, q / QS, g, jj);
        };
        weigh(0, 0);
        weigh(0, 1);
        columns(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 2 * QS; ++q) {
            const int kk = q / QS, t0 = 2 * (q % QS);
            if (kk == 0) {
#pragma unroll
                for (int t = t0; t < t0 + 2; ++t) {
                    st[t][0] *= el;
                    st[t][1] *= el;
                }
            }
            if (q + 1 < 2 * QS) columns(q + 1);
            if (q == QS - 2) weigh(1, 0);
            if (q == QS - 1) weigh(1, 1);
#pragma unroll
            for (int n = 2; n >= 0; --n) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) st[t0 + t][c] = mfma_bf(bq[q & 1][t], wx[kk][c].s[n], st[t0 + t][c]);
                }
            }
            if (q == QS - 2 || q == QS - 1) interleave<12, 7, 1, 0>();
            else interleave<12, 2, 1, 0>();
            if (q == QS - 1) {
                read();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
};

}  // namespace

template <int S>
__global__ void __launch_bounds__(WT) kda_ssm_scan_kernel(const SsmParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[FL::BYTES];
    constexpr int KT = S / 32;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave < 8 ? wave >> 1 : wave - 8;   // 64 columns
    SsmWalk k;
    if (!walk_place(p, (int)blockIdx.x, w, k)) return;
    const int nch = k.nch;
    const int64_t state = (int64_t)S * p.P;
    char *tc = smem + FL::C, *tx = smem + FL::X + w * 8192, *pm = smem + FL::PM + w * FL::PARTS, *record = smem + FL::REC + w * SSM_REC;
    auto tile = [&](int i) { return smem + (i & 1) * 16384; };   // B

    if (wave >= 8) {
        // ================= the waves that load and store =================
        if (nch == 0) return;
        const int hl = tid - 512;
        const Rows bc[2] = {p.B, p.C};
        Tiles<S, 2> t;
        Columns x, y;
        Record r;
        if (k.on) {   // above the diagonal
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                *reinterpret_cast<u32x2*>(pm + n * GDR_TRI + tri_frag(0, 0) * GDR_FRAG + 16 * lane + 8) = u32x2{0, 0};
                *reinterpret_cast<u32x2*>(pm + n * GDR_TRI + tri_frag(2, 1) * GDR_FRAG + 16 * lane + 8) = u32x2{0, 0};
            }
        }
        t.ask(bc, k, 0, hl);
        if (k.on) {
            r.ask(p, k, 0, lane);
            x.ask(p.x, k, 0, lane);
        }
        t.put(tile(0), tc, hl);
        if (k.on) {
            r.put_but_eg(record, 0, lane);
            r.put_eg(record, lane);
        }
        if (nch > 1) {
            t.ask(bc, k, 1, hl);
            if (k.on) r.ask(p, k, 1, lane);
        }
        lds_barrier();   // B, C and the records of the first chunk
        for (int i = 0; i < nch; ++i) {
            lds_barrier();   // 1
            if (k.on) {
                const int ln = opaque(lane);   // addresses formed anew: kept through the loop they would spill
                if (i > 0) {
                    y.get(tx, ln);
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                }
                x.put(tx, ln);
            }
            lds_barrier();   // 2
            if (i + 1 < nch) {
                t.put(tile(i + 1), tc, opaque(hl));
                if (k.on) r.put_but_eg(record, (i + 1) & 1, opaque(lane));
            }
            lds_barrier();   // 3
            {
                const int ln = opaque(lane);
                if (k.on && i + 1 < nch) {
                    r.put_eg(record, ln);
                    x.ask(p.x, k, i + 1, ln);
                }
                if (k.on && i > 0) y.store(p, k, i - 1, ln);
                if (i + 2 < nch) {
                    t.ask(bc, k, i + 2, hl);
                    if (k.on) r.ask(p, k, i + 2, ln);
                }
            }
        }
        lds_barrier();
        if (k.on) {
            y.get(tx, lane);
            y.store(p, k, nch - 1, lane);
        }
        return;
    }

    // ================= walking waves =================
    const int x0 = 32 * (wave & 1), pc = k.pc + x0;   // the wave's first column in x's rows, in the head
    State<S> z;
    {
        const float* from = nullptr;
        if (k.sg.count > 1) from = p.seg + (k.sslot * p.H + k.head) * state;
        else if (p.h0) from = p.h0 + ((int64_t)k.sg.n * p.H + k.head) * state;
        z.load(k.on ? from : nullptr, p, pc, lane);
    }
    const float skip = k.on && p.D ? p.D[k.head] : 0.f;
    const float* rec = reinterpret_cast<const float*>(record);
    if (nch > 0) {
        lds_barrier();
        if (k.on) pair_half<S>(wave & 1, tile(0), tc, rec, skip, pm, lane);
    }
    for (int i = 0; i < nch; ++i) {
        lds_barrier();   // 1: B, C and the records, and the pair matrix at 2
        if (!k.on) {
            lds_barrier();
            lds_barrier();
            continue;
        }
        f32x4 y[4][2];   // channels 16 c + 4 g + r of token 16 m + jj
        {   // C S, 32 tokens at a time; the state's parts of a k step formed beside the products of the one before it
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            Split<3> sp[2][2];
            bf16x8 cf[2][2];
            auto parts = [&](int kk, int c) { sp[kk & 1][c] = split_acc<3>(z.st[2 * kk][c], z.st[2 * kk + 1][c]); };
            auto rows = [&](int q) {   // of step q: k step q / 2, tokens 32 (q % 2) ..
#pragma unroll
                for (int m = 0; m < 2; ++m) cf[q & 1][m] = row_frag(tc, 2 * (q & 1) + m, q >> 1, g, jj);
            };
            parts(0, 0);
            parts(0, 1);
            rows(0);
#pragma unroll
            for (int m = 0; m < 4; ++m) y[m][0] = y[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < 2 * KT; ++q) {
                const int kk = q >> 1, m0 = 2 * (q & 1);
                if (q + 1 < 2 * KT) rows(q + 1);
                if (kk + 1 < KT) parts(kk + 1, q & 1);
#pragma unroll
                for (int n = 2; n >= 0; --n) {
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        y[m0 + m][0] = mfma_bf(sp[kk & 1][0].s[n], cf[q & 1][m], y[m0 + m][0]);
                        y[m0 + m][1] = mfma_bf(sp[kk & 1][1].s[n], cf[q & 1][m], y[m0 + m][1]);
                    }
                }
                interleave<12, 4, 1, 0>();
            }
        }
        lds_barrier();   // 2: x
        u32x2 out[4][2];   // y as bf16
        const float el = __int_as_float(uniform(__float_as_int(rec[SSM_EG + 63])));
        {   // y = e^G C S, then the pairs' products
            const int ln = opaque(lane), g = ln >> 4, jj = ln & 15;
            bf16x8 xf[2][2], pf[6];
            constexpr int FM[6] = {0, 1, 2, 3, 2, 3}, FK[6] = {0, 0, 0, 0, 1, 1};
#pragma unroll
            for (int f = 0; f < 6; ++f) pf[f] = lds_bf8(pm + 2 * GDR_TRI + tri_frag(FM[f], FK[f]) * GDR_FRAG + 16 * ln);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                for (int c = 0; c < 2; ++c) xf[kk][c] = x_frag(tx, kk, x0 + 16 * c, ln);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float eg = rec[SSM_EG + 16 * m + jj];
#pragma unroll
                for (int c = 0; c < 2; ++c) y[m][c] *= eg;
            }
#pragma unroll
            for (int n = 2; n >= 0; --n) {
#pragma unroll
                for (int f = 0; f < 6; ++f) {
                    if (n < 2) pf[f] = lds_bf8(pm + n * GDR_TRI + tri_frag(FM[f], FK[f]) * GDR_FRAG + 16 * ln);
#pragma unroll
                    for (int c = 0; c < 2; ++c) y[FM[f]][c] = mfma_bf(xf[FK[f]][c], pf[f], y[FM[f]][c]);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int c = 0; c < 2; ++c) out[m][c] = u32x2{pack_bf2(y[m][c][0], y[m][c][1]), pack_bf2(y[m][c][2], y[m][c][3])};
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        lds_barrier();   // 3: the pair matrix is read
        // of a SIMD's two waves one grows first, the other forms its pairs first
        const bool pairs = i + 1 < nch;
        if (pairs && wave >= 4) pair_half<S>(wave & 1, tile(i + 1), tc, rec, skip, pm, lane);
        z.grow(tile(i), tx, x0, el, rec + (i & 1 ? SSM_GA : SSM_W), opaque(lane), [&]() {   // y in the place of x
            const int ln = opaque(lane);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    *reinterpret_cast<u32x2*>(tx + x_off(16 * m + (ln & 15), x0 + 16 * c + 4 * (ln >> 4))) = out[m][c];
            }
        });
        if (pairs && wave < 4) pair_half<S>(wave & 1, tile(i + 1), tc, rec, skip, pm, lane);
    }
    if (nch > 0) lds_barrier();   // the last chunk's y
    if (k.on && p.hT && k.sg.index == k.sg.count - 1)
        z.store(p.hT + ((int64_t)k.sg.n * p.H + k.head) * state, p, pc, lane);
}

// What a segment adds to the state (REV: to the gradient of the state that enters it), and its decay.
template <int S, bool REV>
__device__ __forceinline__ void ssm_adds(const SsmParams& p, char* smem, int block) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave < 8 ? wave >> 1 : wave - 8;   // 64 columns
    SsmWalk k;
    if (!walk_place(p, block, w, k)) return;
    if (k.sg.index == (REV ? 0 : k.sg.count - 1)) return;   // nothing starts from what it adds
    const int nch = k.nch;
    auto tile = [&](int i) { return smem + (i & 1) * 16384; };
    auto columns = [&](int i) { return smem + AL::X + ((i & 1) * 4 + w) * 8192; };
    auto record = [&](int i) { return smem + AL::REC + ((i & 1) * 4 + w) * SSM_REC; };
    auto at = [&](int i) { return REV ? nch - 1 - i : i; };
    if (wave >= 8) {
        const int hl = tid - 512;
        const Rows b[1] = {REV ? p.C : p.B};
        Tiles<S, 1> t;
        Columns x;
        Record r;
        auto ask = [&](int i) {
            t.ask(b, k, at(i), hl);
            if (!k.on) return;
            x.ask(REV ? p.dO : p.x, k, at(i), lane);
            r.ask(p, k, at(i), lane);
        };
        auto put = [&](int i) {
            t.put(tile(i), nullptr, hl);
            if (!k.on) return;
            x.put(columns(i), lane);
            r.put(record(i), lane);
        };
        ask(0);
        put(0);
        if (nch > 1) ask(1);
        for (int i = 0; i < nch; ++i) {
            lds_barrier();
            if (i + 1 < nch) put(i + 1);
            if (i + 2 < nch) ask(i + 2);
        }
        return;
    }
    const int x0 = 32 * (wave & 1), pc = k.pc + x0;
    State<S> z;
    z.load(nullptr, p, pc, lane);
    float total = 1.f;
    for (int i = 0; i < nch; ++i) {
        lds_barrier();
        if (!k.on) continue;
        const float* rec = reinterpret_cast<const float*>(record(i));
        total *= rec[SSM_EG + 63];
        z.grow(tile(i), columns(i), x0, rec[SSM_EG + 63], rec + (REV ? SSM_EG : SSM_W), lane, []() {});
    }
    if (!k.on) return;
    z.store((REV ? p.dseg : p.seg) + (k.sslot * p.H + k.head) * S * p.P, p, pc, lane);
    if (pc == 0 && lane == 0) (REV ? p.ddecay : p.decay)[k.sslot * p.H + k.head] = total;
}
// The backward's second half of the work-groups walks the gradients.
template <int S>
__global__ void __launch_bounds__(WT) kda_ssm_adds_kernel(const SsmParams p, const int half) {
    __shared__ __attribute__((aligned(1024))) char smem[AL::BYTES];
    if ((int)blockIdx.x < half) ssm_adds<S, false>(p, smem, (int)blockIdx.x);
    else ssm_adds<S, true>(p, smem, (int)blockIdx.x - half);
}

namespace {
unsigned walk_blocks(const SsmParams& p) {
    return (unsigned)((p.segslots + 7) / 8 * 8 * p.G * ((p.H / p.G * p.P + p.cols - 1) / p.cols));
}
}  // namespace

void launch_ssm_adds(const SsmParams& p, bool both, hipStream_t stream) {
    const unsigned half = walk_blocks(p);
    hipLaunchKernelGGL((p.S == 128 ? kda_ssm_adds_kernel<128> : kda_ssm_adds_kernel<64>), dim3(both ? 2 * half : half), dim3(WT), 0,
                       stream, p, (int)half);
}
void launch_ssm_scan(const SsmParams& p, hipStream_t stream) {
    hipLaunchKernelGGL((p.S == 128 ? kda_ssm_scan_kernel<128> : kda_ssm_scan_kernel<64>), dim3(walk_blocks(p)), dim3(WT), 0, stream, p);
}

}  // namespace kda
