// What the selective state space scan's walks share and the backward's own, on gfx950 (MI355X):
// the numbers of every token, the chaining of segments, and the walks that leave the states.
//
// Backward: the state that enters each chunk, S <- e^{G_last} S + B^T (e^{G_last - G} d x), and the gradient of the one
// that leaves it, last chunk first, dS <- e^{G_last} dS + C^T (e^G dy), both into memory in the order
// that the token gradients take as operands.  A wave owns 32 of a head's value columns: its state is S / 16 by 2 accumulator
// tiles, transposed (a lane holds four columns of a channel).  Four waves
// share the chunk's B or C in LDS, and each brings its own columns of x or dy there; the next chunk's come by DMA
// during this one's products.  Bound by HBM: B = 2, H = 64, T = 8192 leave 1.07 GB in 245 us, 4.4 TB/s.  Two work-groups share a compute unit (one of eight waves: 112 us, not 107, packed
// 4096 tokens of 32 heads of 128).
#include <algorithm>

#include "kda_ssm_device.h"

namespace kda {

// ---- per-token numbers ----
// 14 us at B = 2, H = 64, T = 8192, where 34 MB are written: a double's prefix sum and eight exponentials a token.
// One wave per (chunk slot, head), lane = token.  Tokens past the end change nothing: d = 0, a = 0.
__global__ void __launch_bounds__(256) kda_ssm_gates_kernel(const SsmParams p) {
    const int lane = threadIdx.x & 63, quads = (p.H + 3) / 4;
    const int64_t slot = blockIdx.x / quads;
    const int h = (int)(blockIdx.x % quads) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (h >= p.H) return;
    const SsmChunk c = ssm_chunk(p, slot);
    if (c.rows == 0) return;
    float d = 0.f;
    double a = 0.0;
    if (lane < c.rows) {
        d = ssm_step(ssm_raw(p.dt, p.dt_f32, c.row * p.dtb + (c.tok + lane) * p.dtt + h, p.bias, h), p.softplus);
        a = (double)d * p.A[h];
        a = a < -200.0 ? -200.0 : a;   // the factor is 0 in fp32 either way, and sums stay finite
    }
    const double x = prefix64(a * 1.4426950408889634074);
    const float hi = (float)x;
    const GSum G = {hi, (float)(x - (double)hi)};
    auto of = [&](int l) {
        const double y = lane_f64(x, l);
        const float f = (float)y;
        return GSum{f, (float)(y - (double)f)};
    };
    const GSum last = of(63), e0 = of(15), e1 = of(31), e2 = of(47);
    const int b = lane >> 4;
    const GSum s = b == 0 ? GSum{0.f, 0.f} : b == 1 ? e0 : b == 2 ? e1 : e2, e = b == 0 ? e0 : b == 1 ? e1 : b == 2 ? e2 : last;
    float* r = reinterpret_cast<float*>(p.rec + (slot * p.H + h) * SSM_REC) + lane;
    r[SSM_DT] = d;
    r[SSM_EG] = gate_exp(G);
    const float ga = gate_ratio(last, G);
    r[SSM_GA] = ga;
    r[SSM_W] = ga * d;
    r[SSM_GH] = G.hi;
    r[SSM_GL] = G.lo;
    r[SSM_RI] = gate_ratio(G, s);
    r[SSM_KA] = gate_ratio(e, G);
}

namespace {

constexpr int NW = 4;   // waves of a walk

struct SL {
    static constexpr int HEADS = NW / 2;   // at most, of 64 columns
    static constexpr int B = 0, X = 16384, REC = X + NW * 4096;
    static constexpr int SLOT = REC + HEADS * SSM_REC, BYTES = 2 * SLOT;
};

// Tokens 32 kk + 4 g + r and 16 more of the wave's columns 16 ct + jj, as an operand.
__device__ __forceinline__ bf16x8 x_frag(const char* x, int kk, int ct, int g, int jj) {
    const char* a = x + (32 * kk + 4 * g + (jj >> 2)) * 64 + 32 * ct + 8 * (jj & 3);
    return join(lds_tr(a), lds_tr(a + 16 * 64));
}

// A walk's work-group: a segment and a unit, the columns that it takes of a group of heads.  Work-groups
// are dealt to the 8 XCDs round robin: a segment's units go to one of them, since they share B and C.
__device__ __forceinline__ bool walk_place(int b, int units, int64_t segs, int64_t& seg, int& unit) {
    const int r = b >> 3;
    seg = (int64_t)(r / units) * 8 + (b & 7);
    unit = r % units;
    return seg < segs;
}

}  // namespace

// REV: the gradients' walk, with C, dy and e^G in the place of B, x and e^{G_last - G} d, last chunk first.
template <int S, bool REV>
__device__ __forceinline__ void ssm_walk(const SsmParams& p, char* smem, int block) {
    typedef SL L;
    constexpr int NT = S / 16;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, jj = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int R = p.H / p.G, per = (R * p.P + 32 * NW - 1) / (32 * NW);
    int64_t sslot;
    int unit;
    if (!walk_place(block, per * p.G, p.segslots, sslot, unit)) return;
    const SsmSegment sg = ssm_segment(p, sslot);
    if (sg.index >= sg.count) return;
    const int group = unit / per, h0 = (unit % per) * 32 * NW / p.P;      // first head (in the group) of the unit
    const int col = (unit % per) * 32 * NW + 32 * wave;                   // the wave's first column in the group
    const bool on = col < R * p.P;
    const int head = group * R + (on ? col / p.P : 0), pc = col % p.P;    // its head, its first column there
    const int myrec = (on ? col / p.P - h0 : 0) * SSM_REC;
    const int c0 = sg.index * p.segc;
    const int64_t left = sg.q.len - (int64_t)c0 * CH;
    const int nch = left <= 0 ? 0 : (int)((left + CH - 1) / CH < p.segc ? (left + CH - 1) / CH : p.segc);
    const int64_t row = sg.q.row, tok0 = sg.q.bos + (int64_t)c0 * CH;
    auto at = [&](int i) { return REV ? nch - 1 - i : i; };   // the i-th chunk of the walk
    auto rows_of = [&](int c) -> int {
        const int64_t r = left - (int64_t)c * CH;
        return r >= CH ? CH : (int)r;
    };
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));

    auto dma = [&](int i) {
        const int c = at(i), rows = rows_of(c);
        const int64_t tok = tok0 + (int64_t)c * CH;
        const uint32_t to = lds + (i & 1) * L::SLOT;
        auto tile = [&](const Rows& t, uint32_t where) {   // [64][S], rows of 256 bytes
            const __amdgpu_buffer_rsrc_t rs = chunk_rsrc(t.p + row * t.sb + tok * t.st + group * t.sh, t.st, rows, S);
#pragma unroll
            for (int u = 0; u < 16 / NW; ++u) {
                const int r = 4 * (wave + NW * u) + g, piece = jj ^ tsw(r);
                const int off = (int)(r * t.st * 2) + 16 * piece;
                dma_piece(rs, where + (wave + NW * u) * 1024, S == 128 || piece < 8 ? off : 0x7ffffff0);
            }
        };
        tile(REV ? p.C : p.B, to + L::B);
        if (on) {
            const Rows& t = REV ? p.dO : p.x;
            const __amdgpu_buffer_rsrc_t rs = chunk_rsrc(t.p + row * t.sb + tok * t.st + head * t.sh + pc, t.st, rows, 32);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                dma_piece(rs, to + L::X + wave * 4096 + u * 1024, (int)((16 * u + (lane >> 2)) * t.st * 2) + 16 * (lane & 3));
        }
        if (h0 + wave / 2 < R) {   // half of a head's record
            const __amdgpu_buffer_rsrc_t rs = make_rsrc(
                p.rec + ((sg.slot0 + c0 + c) * p.H + group * R + h0 + wave / 2) * SSM_REC, SSM_REC);
            dma_piece(rs, to + L::REC + wave * 1024, (wave & 1) * 1024 + 16 * lane);
        }
    };

    // The state that enters, transposed: a lane holds four columns of channel state_row(t, jj / 4, jj % 4) of tile t
    f32x4 st[NT][2];
    const int64_t state = (int64_t)p.S * p.P;
    const float *from = nullptr, *outer = REV ? p.dhT : p.h0;
    if (sg.count > 1) from = (REV ? p.dseg : p.seg) + (sslot * p.H + head) * state;
    else if (outer) from = outer + ((int64_t)sg.n * p.H + head) * state;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            st[t][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (from && on)
                st[t][ct] = *reinterpret_cast<const f32x4*>(from + (int64_t)state_row(t, jj >> 2, jj & 3) * p.P + pc + 16 * ct + 4 * g);
        }
    }

    if (nch > 0) dma(0);
    for (int i = 0; i < nch; ++i) {
        // this wave's pieces of the chunk; the 2 NT stores after them may still be under way
        if (i > 0 && on) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * NT) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_barrier();   // everyone's, and the other slot's reads are done
        if (i + 1 < nch) dma(i + 1);
        if (!on) continue;
        char* slot = smem + (i & 1) * L::SLOT;
        const char *tb = slot + L::B, *tx = slot + L::X + wave * 4096;
        const float* rec = reinterpret_cast<const float*>(slot + L::REC + myrec);
        const float el = rec[SSM_EG + 63];
        bf16x8 xf[2][2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) xf[kk][ct] = x_frag(tx, kk, ct, g, jj);
        }
        float* to = (REV ? p.dSt : p.St) + ((sg.slot0 + c0 + at(i)) * p.H + head) * state + (pc >> 5) * (S * 32) + lane * 4;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) *reinterpret_cast<f32x4*>(to + t * 512 + 256 * ct) = st[t][ct];
        }
        // S <- e^{G_last} S + B^T (w x)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            st[t][0] *= el;
            st[t][1] *= el;
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            f32x4 w0, w1;
            if (REV) {
                w0 = num4(rec, SSM_EG, 2 * kk, g);
                w1 = num4(rec, SSM_EG, 2 * kk + 1, g);
            } else {
                w0 = num4(rec, SSM_W, 2 * kk, g);
                w1 = num4(rec, SSM_W, 2 * kk + 1, g);
            }
            Split<3> wx[2];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                const u32x4 xx = __builtin_bit_cast(u32x4, xf[kk][ct]);
                wx[ct] = split_acc<3>(w0 * widen(u32x2{xx[0], xx[1]}), w1 * widen(u32x2{xx[2], xx[3]}));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const bf16x8 b = col_frag(tb, t, kk, g, jj);
#pragma unroll
                for (int n = 2; n >= 0; --n) {
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct)
                        st[t][ct] = mfma_bf(wx[ct].s[n], b, st[t][ct]);
                }
            }
        }
    }
    if (!REV || !on || !p.dh0 || sg.index != 0) return;
    float* dh0 = p.dh0 + ((int64_t)sg.n * p.H + head) * state;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
            *reinterpret_cast<f32x4*>(dh0 + (int64_t)state_row(t, jj >> 2, jj & 3) * p.P + pc + 16 * ct + 4 * g) = st[t][ct];
    }
}

// The second half of the work-groups walks the gradients.
template <int S>
__global__ void __launch_bounds__(64 * NW) kda_ssm_states_kernel(const SsmParams p, const int half) {
    __shared__ __attribute__((aligned(1024))) char smem[SL::BYTES];
    if ((int)blockIdx.x < half) ssm_walk<S, false>(p, smem, (int)blockIdx.x);
    else ssm_walk<S, true>(p, smem, (int)blockIdx.x - half);
}

// Chains a sequence's segments: what enters each from what the ones before it add (REV: after it).
// A thread takes four neighbouring entries of a head's state.  Bound by the states it reads and writes: 16 us for 97 MB, packed
// 4096 tokens of 32 heads of 128 x 128; eight segments asked for at a time were no faster.
template <bool REV>
__device__ __forceinline__ void ssm_chain(const SsmParams& p, int64_t block) {
    const int64_t state = (int64_t)p.S * p.P, parts = state / 1024;
    const int64_t e = (block % parts) * 1024 + threadIdx.x * 4, nh = block / parts;
    const int n = (int)(nh / p.H), h = (int)(nh % p.H);
    const SsmSeq q = ssm_seq(p, n);
    const int64_t unit = (int64_t)p.segc * CH, seg0 = p.cu ? q.bos / unit + n : (int64_t)n * p.nseg;
    const int64_t count = (q.len + unit - 1) / unit;
    float* seg = REV ? p.dseg : p.seg;
    const float *decay = REV ? p.ddecay : p.decay, *outer = REV ? p.dhT : p.h0;
    auto at = [&](int64_t i) { return (seg0 + (REV ? count - 1 - i : i)) * p.H + h; };
    auto load = [&](int64_t i) { return *reinterpret_cast<const f32x4*>(seg + at(i) * state + e); };
    if (count < 2) return;
    f32x4 run = {0.f, 0.f, 0.f, 0.f}, next = load(0);
    if (outer) run = *reinterpret_cast<const f32x4*>(outer + nh * state + e);
    // the first one's too: with several work-groups a sequence the last may write the final state where
    // the initial state is before the first has read it
    *reinterpret_cast<f32x4*>(seg + at(0) * state + e) = run;
    for (int64_t i = 0; i + 1 < count; ++i) {
        const f32x4 adds = next;
        if (i + 2 < count) next = load(i + 1);
        run = decay[at(i)] * run + adds;
        *reinterpret_cast<f32x4*>(seg + at(i + 1) * state + e) = run;
    }
}
__global__ void __launch_bounds__(256) kda_ssm_chain_kernel(const SsmParams p, const int64_t half) {
    if (blockIdx.x < half) ssm_chain<false>(p, blockIdx.x);
    else ssm_chain<true>(p, blockIdx.x - half);
}

namespace {

void states(const SsmParams& p, hipStream_t stream) {
    const int per = (p.H / p.G * p.P + 32 * NW - 1) / (32 * NW);
    const unsigned half = (unsigned)((p.segslots + 7) / 8 * 8 * per * p.G);
    auto* f = p.S == 128 ? kda_ssm_states_kernel<128> : kda_ssm_states_kernel<64>;
    hipLaunchKernelGGL(f, dim3(2 * half), dim3(64 * NW), 0, stream, p, (int)half);
}
bool segmented(const SsmParams& p) { return p.cu ? p.nc > p.segc : p.nseg > 1; }
void gates(const SsmParams& p, hipStream_t stream) {
    if (p.nslots > 0)
        hipLaunchKernelGGL(kda_ssm_gates_kernel, dim3((unsigned)(p.nslots * ((p.H + 3) / 4))), dim3(256), 0, stream, p);
}
// The states that enter the segments, and the gradients of those that leave them.
void enter(const SsmParams& p, bool both, hipStream_t stream) {
    if (!segmented(p)) return;
    launch_ssm_adds(p, both, stream);
    const int64_t half = (int64_t)p.N * p.H * (p.S * p.P / 1024);
    hipLaunchKernelGGL(kda_ssm_chain_kernel, dim3((unsigned)(both ? 2 * half : half)), dim3(256), 0, stream, p, half);
}

}  // namespace

hipError_t launch_ssm_fwd(const SsmParams& p, hipStream_t stream) {
    gates(p, stream);
    enter(p, false, stream);
    launch_ssm_scan(p, stream);
    return hipGetLastError();
}

hipError_t launch_ssm_bwd(const SsmParams& p, hipStream_t stream) {
    if (p.N > 0) {
        gates(p, stream);
        enter(p, true, stream);
        states(p, stream);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_ssm_grads(p, stream);
}

}  // namespace kda
