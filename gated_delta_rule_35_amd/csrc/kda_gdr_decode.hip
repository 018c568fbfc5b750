// One token per row of a batch for the gated delta rule with one decay per head, the
// states in a pool that a slot map indexes, on gfx950 (MI355X):
//   S~ = e^g S,  u = beta (v - S~^T k),  S' = S~ + k u^T,  o = scale S'^T q
// in fp32, o rounded to bf16 once.
//
// Bound by the state's 64 KB read and 64 KB written per row and value head.  Columns of
// S never mix, so a work-group takes CW of a head's 128 columns: all of them where rows
// and heads alone give every compute unit a work-group, 32 where they do not (four times
// the work-groups, a quarter of the work in each).  With 256 compute units, 128 and 32
// columns: 4.4 and 3.6 us at 16 rows and heads, 4.8 and 4.1 at 64, 6.6 and 6.9 at 256,
// 20.2 and 22.3 at 1024, 83 and 83 at 4096 (537 MB, 6.5 TB/s with part of the states in
// the last-level cache; 5.1 TB/s at 16,384, what a large copy reaches).  256 threads, each a
// quad of columns and every 256 / (CW / 4)-th row, so that loads and stores are 16 bytes
// a lane and CW columns of a row one run; S stays in registers.  The sums over rows go
// by lane exchange, then through LDS in wave order: runs are bitwise equal.
//
// Rows that name the same slot are tokens of one sequence in the order of the batch:
// the work-group of the first such row takes them all one after the other, and those of
// the later rows end at once.  Rows with a slot outside the pool are skipped.
#include "kda_gdr_device.h"

namespace kda {

namespace {
constexpr int DT = 256;
// Sum over the wave's lanes that are equal modulo N, in each of them.
template <int N>
__device__ __forceinline__ float sum_above(float x) {
    static_assert(N == 8 || N == 32, "rows of quads");
    if (N == 32) {
        const Pair p = across<32>(x);
        return p.a + p.b;
    }
    return sum_groups(x + ror16<8>(x));
}
}

template <int CW>
__global__ void __launch_bounds__(DT) kda_gdr_decode_kernel(const GdrDecodeParams p) {
    constexpr int NQ = CW / 4, RG = DT / NQ, NR = DK / RG;   // column quads, row groups, rows a thread
    constexpr int SL = DK / CW;
    __shared__ __attribute__((aligned(16))) float sU[4][CW], sQ[4][CW];
    __shared__ float sQK[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cq = tid % NQ, rg = tid / NQ;
    const int item = blockIdx.x / SL, sl = blockIdx.x % SL;
    const int n0 = item / p.Hv, hv = item % p.Hv, hq = hv / (p.Hv / p.Hq);
    const int slot = p.idx ? p.idx[n0] : n0;
    if (slot < 0 || slot >= p.slots) return;
    const int64_t so = ((int64_t)slot * p.Hv + hv) * DK * DK + CW * sl + 4 * cq;
    f32x4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        s[i] = p.s_in ? *reinterpret_cast<const f32x4*>(p.s_in + so + (int64_t)(rg + i * RG) * DK)
                      : f32x4{0.f, 0.f, 0.f, 0.f};
    bool more = false;   // a later row names this slot
    if (p.idx) {
        int f = 0;
        for (int m = tid; m < p.N; m += DT)
            if (m != n0 && p.idx[m] == slot) f |= m < n0 ? 1 : 2;
        f = __syncthreads_or(f & 1) ? 1 : (__syncthreads_or(f & 2) ? 2 : 0);
        if (f == 1) return;
        more = f == 2;
    }
    for (int n = n0;;) {
        const uint16_t* q = p.q.p + n * p.q.sb + hq * p.q.sh;
        const uint16_t* k = p.k.p + n * p.k.sb + hq * p.k.sh;
        const int64_t gi = (int64_t)n * p.Hv + hv;
        const float eg = fexp(p.g[gi]);
        const float beta = p.beta_f32 ? reinterpret_cast<const float*>(p.beta)[gi]
                                      : bf2f(reinterpret_cast<const uint16_t*>(p.beta)[gi]);
        f32x4 u = {0.f, 0.f, 0.f, 0.f}, o = u;
        float qk = 0.f, kk[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            kk[i] = bf2f(k[rg + i * RG]);
            const float qq = bf2f(q[rg + i * RG]);
            s[i] *= eg;
            u += kk[i] * s[i];
            o += qq * s[i];
            qk = fmaf(qq, kk[i], qk);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[e] = sum_above<NQ>(u[e]);
            o[e] = sum_above<NQ>(o[e]);
        }
        qk = sum_above<NQ>(qk);
        if (lane < NQ) {
            *reinterpret_cast<f32x4*>(&sU[wave][4 * lane]) = u;
            *reinterpret_cast<f32x4*>(&sQ[wave][4 * lane]) = o;
            if (lane == 0) sQK[wave] = qk;
        }
        __syncthreads();
        const uint16_t* v = p.v.p + n * p.v.sb + hv * p.v.sh + CW * sl + 4 * cq;
        const u32x2 vv = *reinterpret_cast<const u32x2*>(v);
        u = *reinterpret_cast<const f32x4*>(&sU[0][4 * cq]);
        o = *reinterpret_cast<const f32x4*>(&sQ[0][4 * cq]);
        qk = sQK[0];
#pragma unroll
        for (int m = 1; m < 4; ++m) {
            u += *reinterpret_cast<const f32x4*>(&sU[m][4 * cq]);
            o += *reinterpret_cast<const f32x4*>(&sQ[m][4 * cq]);
            qk += sQK[m];
        }
        u = beta * (f32x4{bf_lo(vv[0]), bf_hi(vv[0]), bf_lo(vv[1]), bf_hi(vv[1])} - u);
        if (rg == 0) {
            o = p.scale * (o + qk * u);
            *reinterpret_cast<u32x2*>(p.o + gi * DK + CW * sl + 4 * cq) =
                u32x2{pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3])};
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) s[i] += kk[i] * u;
        if (!more) break;
        do ++n;
        while (n < p.N && p.idx[n] != slot);
        if (n >= p.N) break;
        __syncthreads();   // the sums' reads before the next token's
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<f32x4*>(p.s_out + so + (int64_t)(rg + i * RG) * DK) = s[i];
}

hipError_t launch_gdr_decode(const GdrDecodeParams& p, int cus, hipStream_t stream) {
    const int64_t heads = (int64_t)p.N * p.Hv;
    if (heads == 0) return hipSuccess;
    if (heads >= cus)
        hipLaunchKernelGGL(kda_gdr_decode_kernel<128>, dim3((unsigned)heads), dim3(DT), 0, stream, p);
    else
        hipLaunchKernelGGL(kda_gdr_decode_kernel<32>, dim3((unsigned)(4 * heads)), dim3(DT), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
