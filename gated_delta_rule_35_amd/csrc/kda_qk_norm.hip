// Per-head norm of queries and keys with an optional weight and position rotation, and
// its gradients, on gfx950 (MI355X).
//
//   r = (sum x^2 [/ 128] + eps)^{-1/2},  z = x r w,  y = z with its first 2 half channels
//   rotated by the token's position: pairs (a, b) -> (a cos - b sin, b cos + a sin)
// Backward, with dz the rotation of dy the other way:
//   dw = sum over rows of dz x r,   dx = r (w dz - x r^2 [/ 128] <x, w dz>)
//
// Elementwise over rows of 128 channels, bound by HBM: a row is 16 lanes of eight
// channels, so that a wave's loads and stores are 16 bytes a lane (bf16) over four whole
// rows, and a work-group takes 16 rows at a time.  The sum over a row is four lane
// exchanges; a rotation's partner channel is in the same lane (adjacent pairs) or in the
// lane half / 8 away (half pairs).  Sums and products are fp32, rounded once at the end.
// At 16,384 tokens of 64 + 64 heads 175 us (1.07 GB, 6.1 TB/s, of which the last-level cache
// holds a part); gradients with weights and rotation at 8192 tokens of 64 + 16 heads 109 us
// (0.51 GB, 4.7 TB/s).  Small calls take 3 to 4 us on the device and are bound by their launch.
// Weight gradients: each lane sums its eight channels over the rows of its work-group's
// stride, work-groups leave 128 sums each, and a second launch adds those in a fixed
// order (no atomics).
#include "kda_elems.h"

namespace kda {

namespace {

constexpr int NT = 256;

// Row `i` of a side: its offset in x and its token (a side has fewer than 2^31 rows).
struct RowAt {
    int64_t x;
    uint32_t token;
};
__device__ __forceinline__ RowAt row_at(const NormParams& p, const NormSide& s, uint32_t i) {
    const uint32_t token = i / (uint32_t)s.H, h = i - token * (uint32_t)s.H, T = (uint32_t)p.T, b = token / T, t = token - b * T;
    return {b * s.sb + t * s.st + h * s.sh, token};
}

// The lane's cos and sin of a rotation: of its eight channels' angles (half pairs), or
// of its four pairs' (adjacent pairs).  Positions outside the tables take their nearest row.
struct Angles {
    f32x4 c[2], s[2];
};
__device__ __forceinline__ Angles angles(const NormParams& p, uint32_t token, int l) {
    Angles a;
    if (!p.cos) return a;
    int64_t pos = p.pos ? (int64_t)p.pos[token] : (int64_t)(token % (uint32_t)p.T);
    pos = pos < 0 ? 0 : (pos >= p.P ? p.P - 1 : pos);
    const int hl = p.half / 8, step = p.interleaved ? 4 : 8;
    // lanes past the rotated channels read the first angles and do not use them
    const int at = 8 * l >= 2 * p.half ? 0 : step * (p.interleaved || l < hl ? l : l - hl);
    const f32x4* c = reinterpret_cast<const f32x4*>(p.cos + pos * p.half + at);
    const f32x4* s = reinterpret_cast<const f32x4*>(p.sin + pos * p.half + at);
    a.c[0] = c[0];
    a.s[0] = s[0];
    if (!p.interleaved) {
        a.c[1] = c[1];
        a.s[1] = s[1];
    }
    return a;
}

// The rotation of the lane's eight channels 8 l .. + 7 (DIR 1), or back (DIR -1).
template <int DIR>
__device__ __forceinline__ void rotate(const NormParams& p, const Angles& a, int l, int lane, float (&x)[8]) {
    if (!p.cos) return;
    const bool in = 8 * l < 2 * p.half;
    if (p.interleaved) {
        if (!in) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float cc = a.c[0][i], ss = DIR * a.s[0][i], u = x[2 * i], v = x[2 * i + 1];
            x[2 * i] = u * cc - v * ss;
            x[2 * i + 1] = v * cc + u * ss;
        }
    } else {
        const int hl = p.half / 8;                      // lanes of the first members
        const int to = in ? lane - l + (l < hl ? l + hl : l - hl) : lane;
        const float sign = l < hl ? -DIR : DIR;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __shfl(x[i], to), cc = a.c[i >> 2][i & 3], ss = sign * a.s[i >> 2][i & 3];
            x[i] = in ? x[i] * cc + y * ss : x[i];
        }
    }
}

__device__ __forceinline__ float inverse_norm(const NormParams& p, float ss) {
    return 1.f / sqrtf((p.rms ? ss * (1.f / DK) : ss) + p.eps);
}

}  // namespace

template <int XT>
__global__ void __launch_bounds__(NT) kda_qk_norm_kernel(const NormParams p) {
    const int side = (int)blockIdx.x >= p.blocks[0];
    const NormSide& s = p.s[side];
    const int block = (int)blockIdx.x - (side ? p.blocks[0] : 0);
    const int lane = threadIdx.x & 63, l = lane & 15;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = s.w ? s.w[8 * l + i] : 1.f;
    const uint32_t row = (uint32_t)block * NORM_ROWS + (threadIdx.x >> 4), rows = (uint32_t)s.rows;
    const RowAt at = row_at(p, s, row < rows ? row : rows - 1);   // lanes past the end repeat the last row
    float x[8];
    Elems<XT>::widen(Elems<XT>::load(s.x, at.x + 8 * l), x);
    const Angles an = angles(p, at.token, l);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    const float r = inverse_norm(p, sum16(ss));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
    rotate<1>(p, an, l, lane, x);
    if (row < rows) Elems<0>::store(s.y, (int64_t)row * DK + 8 * l, x);
}

template <int XT, int DT>
__global__ void __launch_bounds__(NT) kda_qk_norm_bwd_kernel(const NormParams p) {
    __shared__ float part[NT / 16][DK];
    const int side = (int)blockIdx.x >= p.blocks[0];
    const NormSide& s = p.s[side];
    const int block = (int)blockIdx.x - (side ? p.blocks[0] : 0);
    const int lane = threadIdx.x & 63, l = lane & 15;
    float w[8], dw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = s.w ? s.w[8 * l + i] : 1.f;
        dw[i] = 0.f;
    }
    const uint32_t rows = (uint32_t)s.rows, stride = (uint32_t)p.blocks[side] * NORM_ROWS;
    // a work-group's rows are `stride` apart; every lane of a group takes the same number
    for (uint64_t base = (uint64_t)block * NORM_ROWS; base < rows; base += stride) {
        const uint64_t row = base + (threadIdx.x >> 4);
        const uint32_t i0 = row < rows ? (uint32_t)row : rows - 1;
        const RowAt at = row_at(p, s, i0);
        const auto rx = Elems<XT>::load(s.x, at.x + 8 * l);
        const auto rd = Elems<DT>::load(s.dy, (int64_t)i0 * DK + 8 * l);
        const Angles an = angles(p, at.token, l);
        float x[8], d[8];
        Elems<XT>::widen(rx, x);
        Elems<DT>::widen(rd, d);
        rotate<-1>(p, an, l, lane, d);
        float ss = 0.f, xd = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ss = fmaf(x[i], x[i], ss);
            xd = fmaf(x[i] * w[i], d[i], xd);
        }
        const float r = inverse_norm(p, sum16(ss));
        const float m = sum16(xd) * r * r * (p.rms ? 1.f / DK : 1.f);
        if (row < rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] = fmaf(d[i] * r, x[i], dw[i]);
                d[i] = r * (w[i] * d[i] - x[i] * m);
            }
            Elems<XT>::store(s.y, (int64_t)row * DK + 8 * l, d);
        }
    }
    if (!s.dw) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.x >> 4][8 * l + i] = dw[i];
    __syncthreads();
    if (threadIdx.x < DK) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 16; ++i) t += part[i][threadIdx.x];
        p.part[(int64_t)blockIdx.x * DK + threadIdx.x] = t;
    }
}

// dw of side blockIdx.x / 8, channels 16 (blockIdx.x % 8) .. + 15: the work-groups'
// sums, 64 of them side by side, then in order.
__global__ void __launch_bounds__(NT) kda_qk_norm_dw_kernel(const NormParams p) {
    __shared__ __attribute__((aligned(16))) float part[64][16];
    const int side = blockIdx.x >> 3, c = 4 * (threadIdx.x & 3), g = threadIdx.x >> 2, c0 = 16 * (blockIdx.x & 7);
    if (!p.s[side].dw) return;
    const float* src = p.part + (side ? (int64_t)p.blocks[0] * DK : 0) + c0 + c;
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int b = g; b < p.blocks[side]; b += 64) t += *reinterpret_cast<const f32x4*>(src + (int64_t)b * DK);
    *reinterpret_cast<f32x4*>(&part[g][c]) = t;
    __syncthreads();
    if (threadIdx.x < 16) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) y += part[i][threadIdx.x];
        p.s[side].dw[c0 + threadIdx.x] = y;
    }
}

hipError_t launch_qk_norm(const NormParams& p, hipStream_t stream) {
    const unsigned blocks = (unsigned)(p.blocks[0] + p.blocks[1]);
    if (blocks == 0) return hipSuccess;
    auto* f = p.xt == 0 ? kda_qk_norm_kernel<0> : p.xt == 1 ? kda_qk_norm_kernel<1> : kda_qk_norm_kernel<2>;
    hipLaunchKernelGGL(f, dim3(blocks), dim3(NT), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_qk_norm_bwd(const NormParams& p, hipStream_t stream) {
    const unsigned blocks = (unsigned)(p.blocks[0] + p.blocks[1]);
    typedef void (*Kernel)(NormParams);
    static const Kernel table[3][2] = {{kda_qk_norm_bwd_kernel<0, 0>, kda_qk_norm_bwd_kernel<0, 2>},
                                       {kda_qk_norm_bwd_kernel<1, 0>, kda_qk_norm_bwd_kernel<1, 2>},
                                       {kda_qk_norm_bwd_kernel<2, 0>, kda_qk_norm_bwd_kernel<2, 2>}};
    if (blocks) {
        hipLaunchKernelGGL(table[p.xt][p.dt == 2], dim3(blocks), dim3(NT), 0, stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (p.s[0].dw || p.s[1].dw) {
        hipLaunchKernelGGL(kda_qk_norm_dw_kernel, dim3(16), dim3(NT), 0, stream, p);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace kda
