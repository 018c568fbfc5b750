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
// Weight gradients: each lane sums its eight channels over the rows of its work-group's
// stride, work-groups leave 128 sums each, and a second launch adds those in a fixed
// order (no atomics).
#include "kda_gdr_device.h"

namespace kda {

namespace {

constexpr int NT = 256;

template <int XT>
struct NormType;
template <>
struct NormType<0> {   // bf16
    typedef uint16_t T;
    static __device__ __forceinline__ void load(const void* p, int64_t at, float (&x)[8]) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const T*>(p) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf_lo(v[i]);
            x[2 * i + 1] = bf_hi(v[i]);
        }
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, const float (&x)[8]) {
        *reinterpret_cast<u32x4*>(static_cast<T*>(p) + at) =
            u32x4{pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7])};
    }
};
template <>
struct NormType<1> {   // fp16
    typedef uint16_t T;
    static __device__ __forceinline__ void load(const void* p, int64_t at, float (&x)[8]) {
        const half8 v = *reinterpret_cast<const half8*>(static_cast<const T*>(p) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, const float (&x)[8]) {
        *reinterpret_cast<u32x4*>(static_cast<T*>(p) + at) =
            u32x4{pack_h2(x[0], x[1]), pack_h2(x[2], x[3]), pack_h2(x[4], x[5]), pack_h2(x[6], x[7])};
    }
};
template <>
struct NormType<2> {   // fp32
    typedef float T;
    static __device__ __forceinline__ void load(const void* p, int64_t at, float (&x)[8]) {
        const f32x4* s = reinterpret_cast<const f32x4*>(static_cast<const T*>(p) + at);
        const f32x4 a = s[0], b = s[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = a[i];
            x[4 + i] = b[i];
        }
    }
    static __device__ __forceinline__ void store(void* p, int64_t at, const float (&x)[8]) {
        f32x4* d = reinterpret_cast<f32x4*>(static_cast<T*>(p) + at);
        d[0] = f32x4{x[0], x[1], x[2], x[3]};
        d[1] = f32x4{x[4], x[5], x[6], x[7]};
    }
};

// Row `i` of a side: its offset in x, its token, and its offset in a contiguous tensor.
struct RowAt {
    int64_t x, token, flat;
};
__device__ __forceinline__ RowAt row_at(const NormParams& p, const NormSide& s, int64_t i) {
    const int64_t token = i / s.H, h = i - token * s.H, b = token / p.T, t = token - b * p.T;
    return {b * s.sb + t * s.st + h * s.sh, token, i * DK};
}

// The rotation of the lane's eight channels 8 l .. + 7 by the token's position (DIR 1),
// or back (DIR -1).  Positions outside the tables take their nearest row.
template <int DIR>
__device__ __forceinline__ void rotate(const NormParams& p, int64_t token, int l, int lane, float (&x)[8]) {
    if (!p.cos) return;
    int64_t pos = p.pos ? (int64_t)p.pos[token] : token % p.T;
    pos = pos < 0 ? 0 : (pos >= p.P ? p.P - 1 : pos);
    const bool in = 8 * l < 2 * p.half;
    if (p.interleaved) {
        if (!in) return;
        const float* c = p.cos + pos * p.half + 4 * l;
        const float* s = p.sin + pos * p.half + 4 * l;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float cc = c[i], ss = DIR * s[i], a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cc - b * ss;
            x[2 * i + 1] = b * cc + a * ss;
        }
    } else {
        const int hl = p.half / 8;                      // lanes of the first members
        const int to = lane - l + (l < hl ? l + hl : l - hl);
        const int at = l < hl ? 8 * l : 8 * (l - hl);
        const float* c = p.cos + pos * p.half + (in ? at : 0);
        const float* s = p.sin + pos * p.half + (in ? at : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __shfl(x[i], in ? to : lane);
            const float cc = c[i], ss = (l < hl ? -DIR : DIR) * s[i];
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
    const int64_t row = (int64_t)block * NORM_ROWS + (threadIdx.x >> 4);
    const RowAt at = row_at(p, s, row < s.rows ? row : s.rows - 1);   // lanes past the end repeat the last row
    float x[8];
    NormType<XT>::load(s.x, at.x + 8 * l, x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    const float r = inverse_norm(p, sum16(ss));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
    rotate<1>(p, at.token, l, lane, x);
    if (row < s.rows) NormType<0>::store(s.y, at.flat + 8 * l, x);
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
    for (int64_t base = (int64_t)block * NORM_ROWS; base < s.rows; base += (int64_t)p.blocks[side] * NORM_ROWS) {
        const int64_t row = base + (threadIdx.x >> 4);
        const bool in = row < s.rows;
        const RowAt at = row_at(p, s, in ? row : s.rows - 1);
        float x[8], d[8];
        NormType<XT>::load(s.x, at.x + 8 * l, x);
        NormType<DT>::load(s.dy, at.flat + 8 * l, d);
        rotate<-1>(p, at.token, l, lane, d);
        float ss = 0.f, xd = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ss = fmaf(x[i], x[i], ss);
            xd = fmaf(x[i] * w[i], d[i], xd);
        }
        const float r = inverse_norm(p, sum16(ss));
        const float m = sum16(xd) * r * r * (p.rms ? 1.f / DK : 1.f);
        if (in) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] = fmaf(d[i] * r, x[i], dw[i]);
                d[i] = r * (w[i] * d[i] - x[i] * m);
            }
            NormType<XT>::store(s.y, at.flat + 8 * l, d);
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

// dw of side blockIdx.x: the work-groups' sums, in order.
__global__ void __launch_bounds__(1024) kda_qk_norm_dw_kernel(const NormParams p) {
    __shared__ float part[8][DK];
    const int side = blockIdx.x, c = threadIdx.x & (DK - 1), g = threadIdx.x >> 7;
    if (!p.s[side].dw) return;
    const float* src = p.part + (side ? (int64_t)p.blocks[0] * DK : 0);
    float t = 0.f;
    for (int b = g; b < p.blocks[side]; b += 8) t += src[(int64_t)b * DK + c];
    part[g][c] = t;
    __syncthreads();
    if (g == 0) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += part[i][c];
        p.s[side].dw[c] = t;
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
        hipLaunchKernelGGL(kda_qk_norm_dw_kernel, dim3(2), dim3(1024), 0, stream, p);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace kda
