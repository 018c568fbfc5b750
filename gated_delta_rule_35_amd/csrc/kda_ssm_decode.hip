// One token per row of a batch for the selective state space scan, the states in a pool that a
// slot map indexes, on gfx950 (MI355X):
//   d = softplus(dt + bias),  S' = e^{d A} S + B (d x)^T,  y = S'^T C + D x
// in fp32, y rounded to bf16 once.
//
// Bound by a state's 4 S P bytes read and written per row and head: 256 rows of 64 heads, S = 128, P = 64, take
// 207 us, 5.1 TB/s; one row 3.7 us.  A work-group takes a
// head's state, or CW of its columns where rows and heads alone do not fill the compute units;
// 256 threads, each a quad of columns of every 256 / (CW / 4)-th row, so that loads and stores are
// 16 bytes a lane.  The sums over rows go by lane exchange, then through LDS in wave order.
//
// Rows that name the same slot are tokens of one sequence in the order of the batch: the
// work-group of the first such row takes them all one after the other, and those of the later
// rows end at once.  Rows with a slot outside the pool are skipped.
#include "kda_ssm_device.h"

namespace kda {

namespace {
constexpr int DT = 256;
// Sum over the wave's lanes that are equal modulo N, in each of them.
template <int N>
__device__ __forceinline__ float sum_modulo(float x) {
    if (N <= 8) x += ror16<8>(x);
    if (N <= 16) {
        const Pair p = across<16>(x);
        x = p.a + p.b;
    }
    const Pair p = across<32>(x);
    return p.a + p.b;
}
}  // namespace

template <int S, int CW>
__global__ void __launch_bounds__(DT) kda_ssm_decode_kernel(const SsmDecodeParams p) {
    constexpr int NQ = CW / 4, RG = DT / NQ, NR = S / RG;   // column quads, row groups, rows a thread
    __shared__ __attribute__((aligned(16))) float sY[4][CW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cq = tid % NQ, rg = tid / NQ, SL = p.P / CW;
    const int item = blockIdx.x / SL, sl = blockIdx.x % SL;
    const int n0 = item / p.H, h = item % p.H, grp = h / (p.H / p.G);
    const int slot = p.idx ? p.idx[n0] : n0;
    if (slot < 0 || slot >= p.slots) return;
    const int col = CW * sl + 4 * cq;
    const int64_t so = ((int64_t)slot * p.H + h) * S * p.P + col;
    f32x4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        s[i] = p.s_in ? *reinterpret_cast<const f32x4*>(p.s_in + so + (int64_t)(rg + i * RG) * p.P) : f32x4{0.f, 0.f, 0.f, 0.f};
    bool more = false;   // a later row names this slot
    if (p.idx) {
        int f = 0;
        for (int m = tid; m < p.N; m += DT)
            if (m != n0 && p.idx[m] == slot) f |= m < n0 ? 1 : 2;
        if (__syncthreads_or(f & 1)) return;
        more = __syncthreads_or(f & 2);
    }
    const float A = p.A[h], skip = p.D ? p.D[h] : 0.f;
    for (int n = n0;;) {
        const float d = ssm_step(ssm_raw(p.dt, p.dt_f32, n * p.dtb + h, p.bias, h), p.softplus), ea = exp_of(d * A);
        const uint16_t *b = p.B.p + n * p.B.sb + grp * p.B.sh, *c = p.C.p + n * p.C.sb + grp * p.C.sh;
        const u32x2 xx = *reinterpret_cast<const u32x2*>(p.x.p + n * p.x.sb + h * p.x.sh + col);
        const f32x4 x = widen(xx), dx = d * x;
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            s[i] = ea * s[i] + bf2f(b[rg + i * RG]) * dx;
            y += bf2f(c[rg + i * RG]) * s[i];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = sum_modulo<NQ>(y[e]);
        if (lane < NQ) *reinterpret_cast<f32x4*>(&sY[wave][4 * lane]) = y;
        __syncthreads();
        if (rg == 0) {
            y = *reinterpret_cast<const f32x4*>(&sY[0][4 * cq]);
#pragma unroll
            for (int m = 1; m < 4; ++m) y += *reinterpret_cast<const f32x4*>(&sY[m][4 * cq]);
            y += skip * x;
            *reinterpret_cast<u32x2*>(p.y + ((int64_t)n * p.H + h) * p.P + col) = u32x2{pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3])};
        }
        if (!more) break;
        do ++n;
        while (n < p.N && p.idx[n] != slot);
        if (n >= p.N) break;
        __syncthreads();   // the sums' reads before the next token's
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<f32x4*>(p.s_out + so + (int64_t)(rg + i * RG) * p.P) = s[i];
}

hipError_t launch_ssm_decode(const SsmDecodeParams& p, int cus, hipStream_t stream) {
    const int64_t heads = (int64_t)p.N * p.H;
    if (heads == 0) return hipSuccess;
    // Whole states where they make two work-groups a compute unit, else 32 columns: 512 heads of 64 6.9 and 7.4 us; 256 heads
    // of 64 5.2 and 4.9, of 128 8.9 and 7.5.
    const int cw = heads >= 2 * cus ? p.P : 32;
    auto* f = p.S == 128 ? (cw == 128 ? kda_ssm_decode_kernel<128, 128> : cw == 64 ? kda_ssm_decode_kernel<128, 64> : kda_ssm_decode_kernel<128, 32>)
                         : (cw == 128 ? kda_ssm_decode_kernel<64, 128> : cw == 64 ? kda_ssm_decode_kernel<64, 64> : kda_ssm_decode_kernel<64, 32>);
    hipLaunchKernelGGL(f, dim3((unsigned)(heads * (p.P / cw))), dim3(DT), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
