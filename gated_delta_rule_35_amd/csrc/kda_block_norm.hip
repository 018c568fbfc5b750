// The norms around a block and their gradients, on gfx950 (MI355X).  With r(v) = (mean v^2 +
// eps)^{-1/2} over a row of D channels:
//   gated   y = v r w act(z),  v = x,  or  y = v r w,  v = x act(z)  (the gate first)
//   add     h = residual + scale x,  y = h r w
// Backward, with dn the gradient of v r w times w, and m = <dn, v> r^2 / D:
//   dv = r (dn - v m),  dw = sum over rows of (gradient of v r w) v r
//   gated   dx = dv, dz = act'(z) dy v r w;  gate first dx = dv act(z), dz = act'(z) dv x
//   add     dh = dv + what reaches h from elsewhere;  dx = scale dh, d residual = dh
//
// Elementwise over rows, bound by HBM.  A row is L lanes of K pieces of eight channels each, so
// that loads and stores are 16 bytes a lane (bf16) and runs of L times that: 16 lanes up to 128
// channels, a wave up to 2048, a work-group of four waves up to 8192.  A row's sum is lane
// exchanges, and for four waves one exchange through LDS.  Everything is fp32, rounded once at
// the end; y is formed from the unrounded h.
// Weight gradients: a lane sums its channels over the rows of its work-group's stride, the
// work-group's lanes of equal channels are added in order and leave D sums, and a second launch
// adds those in a fixed order.  Measured: gated 2 x 8192 x 64 rows of 128 in bf16 154 us, 5.2 TB/s, their gradients at 4.0; gradients of
// 3001 x 4096 with the gate first 31 us, of 16384 x 4096 with an fp32 residual 210 us, 5.1 TB/s.  Each row's inputs are asked for before the row at hand is finished.
#include <algorithm>
#include <type_traits>

#include "kda_block.h"
#include "kda_elems.h"

namespace kda {

namespace {

constexpr int NT = 256;

// Sum over a row's L lanes, in every one of them.  For L = NT `sh` holds two sets of four
// words, used by turns, so that a row needs one barrier.
template <int L>
__device__ __forceinline__ float row_sum(float x, float* sh, int turn) {
    if (L == 16) return sum16(x);
    x = sum64(x);
    if (L == 64) return x;
    float* s = sh + 4 * (turn & 1);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

struct Row {
    int64_t i;      // row of [B, T, H]
    int64_t x, z;   // its offsets in x and z
};
template <bool FLAT>   // add: rows [B, T]
__device__ __forceinline__ Row row_of(const BlockNormParams& p, int64_t i) {
    const uint32_t r = (uint32_t)i, H = FLAT ? 1 : (uint32_t)p.H, T = (uint32_t)p.T;
    const uint32_t token = r / H, h = r - token * H, b = token / T, t = token - b * T;
    return {i, b * p.xb + t * p.xt + h * p.xh, b * p.zb + t * p.zt + h * p.zh};
}

}  // namespace

// Rows of work-group b: its first, the step to the next, and how many rows there are.  With a
// weight per head a work-group stays with one head, so that its sums are that head's.
struct RowWalk {
    int64_t first, step, end;
};
template <int L, bool SUMS>
__device__ __forceinline__ RowWalk row_walk(const BlockNormParams& p) {
    constexpr int R = NT / L;
    const int64_t k = threadIdx.x / L;
    if (SUMS && p.per_head) {
        const int64_t h = blockIdx.x % p.H, g = blockIdx.x / p.H, groups = gridDim.x / p.H;
        return {(g * R + k) * p.H + h, groups * R * p.H, p.rows};
    }
    return {(int64_t)blockIdx.x * R + k, (int64_t)gridDim.x * R, p.rows};
}

// GATED: y from x and the gate.  Otherwise h and y from the residual (fp32 where RT is 2) and x.
template <bool GATED, int XT, int RT, int L, int K>
__global__ void __launch_bounds__(NT) kda_block_norm_kernel(const BlockNormParams p) {
    __shared__ float sh[8];
    constexpr int ZT = GATED ? XT : RT;
    const int l = threadIdx.x % L;
    const int64_t i = (int64_t)blockIdx.x * (NT / L) + threadIdx.x / L;
    const bool real = i < p.rows;
    const Row at = row_of<!GATED>(p, real ? i : p.rows - 1);   // lanes past the end repeat the last row
    const int64_t wi = p.per_head ? (at.i % p.H) * p.D : 0;
    float v[K][8], g[K][8], ss = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (l + k * L);
        if (c < p.D) {
            Elems<XT>::widen(Elems<XT>::load(p.x, at.x + c), v[k]);
            Elems<ZT>::widen(Elems<ZT>::load(p.z, at.z + c), g[k]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = g[k][e] = 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (GATED) {
                g[k][e] = activation(p.act, g[k][e], sigmoid<XT == 2>(g[k][e]));
                if (p.first) v[k][e] *= g[k][e];
            } else {
                v[k][e] = fmaf(p.scale, v[k][e], g[k][e]);
            }
            ss = fmaf(v[k][e], v[k][e], ss);
        }
    }
    const float r = 1.f / sqrtf(row_sum<L>(ss, sh, 0) / (float)p.D + p.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (l + k * L);
        if (c >= p.D || !real) continue;
        float y[8];
        if (!GATED) Elems<RT>::store(p.h, i * p.D + c, v[k]);
        if (p.w) Elems<2>::widen(Elems<2>::load(p.w, wi + c), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = v[k][e] * r * (p.w ? y[e] : 1.f);
            if (GATED && !p.first) y[e] *= g[k][e];
        }
        Elems<XT>::store(p.y, i * p.D + c, y);
    }
}

// Gradients.  Gated: dx and dz from x, the gate and dy.  Otherwise dx and the residual's gradient from h
// (fp32 where RT is 2), dy and dh.
template <bool GATED, int XT, int RT, int L, int K>
__global__ void __launch_bounds__(NT) kda_block_norm_bwd_kernel(const BlockNormParams p) {
    constexpr int R = NT / L, VT = GATED ? XT : RT;   // rows at a time; type of x or h, and of z or dh
    __shared__ __attribute__((aligned(16))) float sh[8 + NT * 8];
    const int l = threadIdx.x % L;
    const RowWalk walk = row_walk<L, true>(p);
    const int64_t wi = p.per_head ? (int64_t)(blockIdx.x % p.H) * p.D : 0;
    float w[K][8], dw[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 8 * (l + k * L);
        const bool in = c < p.D;
        if (p.w && in) Elems<2>::widen(Elems<2>::load(p.w, wi + c), w[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!p.w || !in) w[k][e] = 1.f;
            dw[k][e] = 0.f;
        }
    }
    struct Inputs {
        typename Elems<VT>::Raw v[K], z[K];
        typename Elems<XT>::Raw dy[K];
    };
    auto load = [&](int64_t i, Inputs& in) {   // past the end the last row, past its channels the first piece
        const Row at = row_of<!GATED>(p, i < p.rows ? i : p.rows - 1);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = 8 * (l + k * L), cc = c < p.D ? c : 0;
            in.v[k] = Elems<VT>::load(p.x, at.x + cc);
            if (GATED) in.z[k] = Elems<VT>::load(p.z, at.z + cc);
            else if (p.dh) in.z[k] = Elems<VT>::load(p.dh, at.i * p.D + cc);
            in.dy[k] = Elems<XT>::load(p.dy, at.i * p.D + cc);
        }
    };
    // every lane of a work-group takes the same number of turns
    const int64_t first = walk.first - (int64_t)(threadIdx.x / L) * (p.per_head ? p.H : 1);
    Inputs next;
    if (first < walk.end) load(walk.first, next);
    int turn = 0;
    for (int64_t base = first, i = walk.first; base < walk.end; base += walk.step, i += walk.step, ++turn) {
        const Inputs in = next;
        if (base + walk.step < walk.end) load(i + walk.step, next);
        float v[K][8], s[K][8], sv = 0.f, sd = 0.f;   // s: sigmoid of the gate
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool on = 8 * (l + k * L) < p.D;
            float dy[8], z[8];
            Elems<VT>::widen(in.v[k], v[k]);
            Elems<XT>::widen(in.dy[k], dy);
            if (GATED) Elems<VT>::widen(in.z[k], z);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = v[k][e], d = dy[e];
                if (GATED) {
                    s[k][e] = sigmoid<XT == 2>(z[e]);
                    const float a = activation(p.act, z[e], s[k][e]);
                    x = p.first ? x * a : x;
                    d = p.first ? d : d * a;
                }
                if (!on) x = d = 0.f;
                sv = fmaf(x, x, sv);
                sd = fmaf(x, d * w[k][e], sd);
            }
        }
        const float rr = 1.f / sqrtf(row_sum<L>(sv, sh, 2 * turn) / (float)p.D + p.eps);
        const float m = row_sum<L>(sd, sh, 2 * turn + 1) / (float)p.D * rr * rr;
        if (i >= p.rows) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = 8 * (l + k * L);
            if (c >= p.D) continue;
            float dy[8], z[8], b[8];
            Elems<XT>::widen(in.dy[k], dy);
            if (GATED || p.dh) Elems<VT>::widen(in.z[k], z);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (GATED) {
                    const float g = activation(p.act, z[e], s[k][e]);
                    const float x = p.first ? v[k][e] * g : v[k][e];
                    const float d = p.first ? dy[e] : dy[e] * g;
                    dw[k][e] = fmaf(d * rr, x, dw[k][e]);
                    const float dv = rr * (d * w[k][e] - x * m);
                    b[e] = p.first ? dv * g : dv;
                    z[e] = slope(p.act, z[e], s[k][e]) * (p.first ? dv * v[k][e] : dy[e] * (x * rr * w[k][e]));
                } else {
                    dw[k][e] = fmaf(dy[e] * rr, v[k][e], dw[k][e]);
                    const float dv = rr * (dy[e] * w[k][e] - v[k][e] * m);
                    z[e] = p.dh ? z[e] + dv : dv;
                    b[e] = p.scale * z[e];
                }
            }
            Elems<XT>::store(p.dx, i * p.D + c, b);
            Elems<VT>::store(p.dz, i * p.D + c, z);
        }
    }
    if (!p.dw) return;
    // the work-group's rows, in the order of their lanes; work-group g of head h leaves row g of [..][H][D]
    float* part = p.part + (int64_t)blockIdx.x * p.D;
    float* sums = sh + 8;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[8 * threadIdx.x + e] = dw[k][e];
        __syncthreads();
        for (int c = threadIdx.x; c < 8 * L; c += NT) {
            float t = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) t += sums[8 * L * r + c];
            if (c + 8 * k * L < p.D) part[c + 8 * k * L] = t;
        }
    }
}

namespace {

template <int V>
using Int = std::integral_constant<int, V>;

// f(L, K) of the rows' split.  2^26 elements in bf16: 128 channels on 16 lanes 79 us gated, 133 their gradients, 213 the sum's
// with an fp32 residual, on 64 lanes 229, 451, 302; 512 channels on 64 lanes 79, 136, 213, on 256 156, 422, 346; 1024 on 64
// lanes of two pieces 79, 141, 202, on 256 95, 251, 205.  At 2048 four pieces on 64 lanes, whose gated gradients hold so many registers
// that a SIMD has one wave, and one on 256 are alike: 83, 143, 200 and 77, 138, 205.  4096 channels 82, 141, 210; 5120, where
// lanes of four pieces hold two and a half, 93, 177, 218; 8192 85, 150, 212.
template <typename F>
void by_width(int D, F f) {
    if (D <= 128) f(Int<16>(), Int<1>());
    else if (D <= 512) f(Int<64>(), Int<1>());
    else if (D <= 1024) f(Int<64>(), Int<2>());
    else if (D <= 2048) f(Int<64>(), Int<4>());
    else if (D <= 4096) f(Int<256>(), Int<2>());
    else f(Int<256>(), Int<4>());
}
template <typename F>
void by_type(int type, F f) {
    if (type == 0) f(Int<0>());
    else if (type == 1) f(Int<1>());
    else f(Int<2>());
}

template <bool GATED>
hipError_t forward(const BlockNormParams& p, hipStream_t stream) {
    if (p.rows == 0) return hipSuccess;
    by_type(p.type, [&](auto xt) {
        by_width(p.D, [&](auto l, auto k) {
            constexpr int XT = decltype(xt)::value, L = decltype(l)::value, K = decltype(k)::value, R = NT / L;
            const dim3 grid((unsigned)((p.rows + R - 1) / R));
            auto kernel = kda_block_norm_kernel<GATED, XT, XT, L, K>;
            if constexpr (!GATED)
                if (p.wide) kernel = kda_block_norm_kernel<GATED, XT, 2, L, K>;
            hipLaunchKernelGGL(kernel, grid, dim3(NT), 0, stream, p);
        });
    });
    return hipGetLastError();
}

template <bool GATED>
hipError_t backward(const BlockNormParams& p, hipStream_t stream) {
    int64_t groups = 0;   // work-groups, of each head with a weight per head
    if (p.rows > 0) {
        by_type(p.type, [&](auto xt) {
            by_width(p.D, [&](auto l, auto k) {
                constexpr int XT = decltype(xt)::value, L = decltype(l)::value, K = decltype(k)::value, R = NT / L;
                const int64_t per = p.per_head ? p.rows / p.H : p.rows, heads = p.per_head ? p.H : 1;
                groups = (per + R - 1) / R;
                if (p.dw) groups = std::min<int64_t>(groups, std::max<int64_t>(BLOCK_DW_GROUPS / heads, 1));
                const dim3 grid((unsigned)(groups * heads));
                auto kernel = kda_block_norm_bwd_kernel<GATED, XT, XT, L, K>;
                if constexpr (!GATED)
                    if (p.wide) kernel = kda_block_norm_bwd_kernel<GATED, XT, 2, L, K>;
                hipLaunchKernelGGL(kernel, grid, dim3(NT), 0, stream, p);
            });
        });
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!p.dw) return hipSuccess;
    const int64_t cols = (int64_t)(p.per_head ? p.H : 1) * p.D;
    return launch_sum_rows(SumParams{p.part, groups, cols, cols, cols, 1, p.dw, nullptr}, stream);
}

}  // namespace

hipError_t launch_gated_norm(const BlockNormParams& p, hipStream_t stream) { return forward<true>(p, stream); }
hipError_t launch_gated_norm_bwd(const BlockNormParams& p, hipStream_t stream) { return backward<true>(p, stream); }
hipError_t launch_add_norm(const BlockNormParams& p, hipStream_t stream) { return forward<false>(p, stream); }
hipError_t launch_add_norm_bwd(const BlockNormParams& p, hipStream_t stream) { return backward<false>(p, stream); }

}  // namespace kda
