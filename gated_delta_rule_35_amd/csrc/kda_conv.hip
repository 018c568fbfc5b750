// Short causal convolution over tokens, one filter of W = 2 .. 4 taps per channel, and its
// gradients, on gfx950 (MI355X):
//   z_t = bias + sum_i w_i x_{t-W+1+i},  y = z or z / (1 + e^-z)
// with the W - 1 inputs before a sequence's first token in an initial state.  Backward:
//   dz = dy act'(z),  dx_t = sum_d w_{W-1-d} dz_{t+d},  dw_i = sum_t dz_t x_{t-W+1+i}
//
// Bound by HBM: x is read and y written once (backward: x and dy, dx; there a token's 40 instructions a channel
// take as long).  16384 x 12288 in bf16: 158 us, 5.1 TB/s; gradients of 2 x 8192 x 12288 4.8 TB/s, of 2 x 4096 x 4352,
// where a SIMD's two waves have one run each, 47 us, 4.5 TB/s.  A thread takes eight
// channels of a run of tokens and walks it, the window of its last W inputs in registers, so
// that a run reads W - 1 rows that others read too (backward 2 (W - 1) of x, W - 1 of dy), from
// L2 as a rule.  Lanes lie along the channels: a wave's loads and stores are 16 bytes a lane
// and runs of up to 1 KB.  Eight rows are asked for at a time.  States are formed by
// work-groups of their own from the rows that make them up.  Sums are fp32, rounded once; the weights'
// gradients are summed over a run, then a work-group's runs, then the work-groups, each in order.
#include <algorithm>
#include <type_traits>

#include "kda_block.h"
#include "kda_elems.h"

namespace kda {

namespace {

constexpr int NT = 256;
constexpr int BATCH = 8;   // rows that are asked for at a time

// The sequence that holds token t (or, in no sequence, the next one): its bounds.
struct Seq {
    int n;
    int64_t a, e;
};
__device__ __forceinline__ Seq conv_seq(const ConvParams& p, int n) {
    Seq s{n, 0, 0};
    if (p.cu) {
        const int64_t a = p.cu[n], e = p.cu[n + 1];
        s.a = a < 0 ? 0 : (a > p.T ? p.T : a);
        s.e = e < s.a ? s.a : (e > p.T ? p.T : e);
    } else {
        s.a = n * p.T;
        s.e = s.a + p.T;
    }
    return s;
}
__device__ __forceinline__ int conv_find(const ConvParams& p, int64_t t) {
    if (!p.cu) return (int)(t / p.T);
    int lo = 0, hi = p.N;   // first sequence that ends behind t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
// Offset of token t (over all rows) of sequence s in x.
__device__ __forceinline__ int64_t x_at(const ConvParams& p, const Seq& s, int64_t t) {
    return p.cu ? t * p.st : s.n * p.sb + (t - s.a) * p.st;
}

template <int W>
struct Filter {
    float w[W][8], b[8];
    __device__ __forceinline__ Filter(const ConvParams& p, int c) {
        const f32x4* s = reinterpret_cast<const f32x4*>(p.w + (int64_t)c * W);
        f32x4 v[2 * W];
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) v[i] = s[i];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i][e] = v[(e * W + i) >> 2][(e * W + i) & 3];
            b[e] = p.bias ? p.bias[c + e] : 0.f;
        }
    }
    // z of the window's last row
    __device__ __forceinline__ float at(const float (&x)[W][8], int e) const {
        float z = b[e];
#pragma unroll
        for (int i = 0; i < W; ++i) z = fmaf(w[i][e], x[i][e], z);
        return z;
    }
};

// Row `r` of the inputs around sequence s: its token s.a + r, or for r < 0 the initial state's.
template <int XT, int W>
__device__ __forceinline__ void input_row(const ConvParams& p, const Seq& s, int64_t r, int c, float (&x)[8]) {
    if (r >= 0) {
        Elems<XT>::widen(Elems<XT>::load(p.x, x_at(p, s, s.a + r) + c), x);
    } else if (p.s_in) {
        Elems<XT>::widen(Elems<XT>::load(p.s_in, ((int64_t)s.n * (W - 1) + (W - 1 + r)) * p.C + c), x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
}
// The window before token s.a + r: its last row is left to be filled.
template <int XT, int W>
__device__ __forceinline__ void window_before(const ConvParams& p, const Seq& s, int64_t r, int c, float (&x)[W][8]) {
#pragma unroll
    for (int i = 1; i < W; ++i) input_row<XT, W>(p, s, r - W + i, c, x[i]);
}
template <int W>
__device__ __forceinline__ void shift(float (&x)[W][8]) {
#pragma unroll
    for (int i = 0; i + 1 < W; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = x[i + 1][e];
    }
}

// act(z) and its derivative, of results of type XT.
template <int XT, int ACT>
__device__ __forceinline__ float act_of(float z) {
    return ACT == ACT_NONE ? z : activation(ACT, z, sigmoid<XT == 2>(z));
}
template <int XT, int ACT>
__device__ __forceinline__ float slope_of(float z) {
    return ACT == ACT_NONE ? 1.f : slope(ACT, z, sigmoid<XT == 2>(z));
}

// The thread's channels and the first token of its run.
struct Place {
    int c, run;
    int64_t t0, t1;
    bool on;
};
__device__ __forceinline__ Place place_of(const ConvParams& p, const ConvSplit& k, int64_t block) {
    Place q;
    const int64_t tile = block / k.cols;
    const int col = (int)(block % k.cols), lane = threadIdx.x % k.lanes;
    q.run = threadIdx.x / k.lanes;
    q.c = 8 * (col * k.lanes + lane);
    q.on = q.c < p.C;
    q.t0 = (tile * (NT / k.lanes) + q.run) * k.run;
    q.t1 = q.t0 + k.run < p.total ? q.t0 + k.run : p.total;
    return q;
}

}  // namespace

template <int XT, int W, int ACT>
__global__ void __launch_bounds__(NT) kda_conv_kernel(const ConvParams p, const ConvSplit k) {
    const int64_t tiles = k.tiles * k.cols;
    if (blockIdx.x >= tiles) {   // final states, a thread eight channels of one row
        const int64_t i = ((int64_t)blockIdx.x - tiles) * NT + threadIdx.x, pieces = p.C / 8;
        const int64_t row = i / pieces;
        if (row >= (int64_t)p.N * (W - 1)) return;
        const Seq s = conv_seq(p, (int)(row / (W - 1)));
        const int c = 8 * (int)(i % pieces);
        float x[8];
        input_row<XT, W>(p, s, s.e - s.a - (W - 1) + row % (W - 1), c, x);
        Elems<XT>::store(p.s_out, row * p.C + c, x);
        return;
    }
    const Place q = place_of(p, k, blockIdx.x);
    if (!q.on || q.t0 >= q.t1) return;
    const Filter<W> f(p, q.c);
    for (int n = conv_find(p, q.t0); n < p.N; ++n) {
        const Seq s = conv_seq(p, n);
        if (s.a >= q.t1) break;
        int64_t t = s.a > q.t0 ? s.a : q.t0;
        const int64_t e1 = s.e < q.t1 ? s.e : q.t1;
        if (t >= e1) continue;
        float x[W][8];
        window_before<XT, W>(p, s, t - s.a, q.c, x);
        const int64_t base = x_at(p, s, t) + q.c;
        const int m = (int)(e1 - t);
        for (int i = 0; i < m; i += BATCH) {
            typename Elems<XT>::Raw raw[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) raw[u] = Elems<XT>::load(p.x, base + (i + u < m ? i + u : m - 1) * p.st);
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                shift(x);
                Elems<XT>::widen(raw[u], x[W - 1]);
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = act_of<XT, ACT>(f.at(x, e));
                if (i + u < m) Elems<XT>::store(p.y, (t + i + u) * p.C + q.c, y);
            }
        }
    }
}

// Gradients.  The walk goes W - 1 tokens past the run, within the sequence: dx of a token is whole
// once dz of the W - 1 tokens after it is known.
template <int XT, int W, int ACT>
__global__ void __launch_bounds__(NT, 2) kda_conv_bwd_kernel(const ConvParams p, const ConvSplit k) {
    constexpr int U = XT == 2 ? 2 : 4;   // rows that are asked for ahead, within the registers
    __shared__ __attribute__((aligned(16))) float sh[NT][8];
    const int64_t tiles = k.tiles * k.cols;
    if (blockIdx.x >= tiles) {   // gradients of the initial states, a thread eight channels of a sequence
        const int64_t i = ((int64_t)blockIdx.x - tiles) * NT + threadIdx.x, pieces = p.C / 8;
        if (i / pieces >= p.N) return;
        const Seq s = conv_seq(p, (int)(i / pieces));
        const int c = 8 * (int)(i % pieces);
        const int64_t len = s.e - s.a;
        const Filter<W> f(p, c);
        float x[W][8], g[W - 1][8];
        window_before<XT, W>(p, s, 0, c, x);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[r][e] = 0.f;
            if (r >= len && p.ds_out)
                Elems<XT>::widen(Elems<XT>::load(p.ds_out, ((int64_t)s.n * (W - 1) + (r - len)) * p.C + c), g[r]);
        }
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            if (t >= len) continue;
            float dy[8];
            shift(x);
            input_row<XT, W>(p, s, t, c, x[W - 1]);
            Elems<XT>::widen(Elems<XT>::load(p.dy, (s.a + t) * p.C + c), dy);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dz = dy[e] * slope_of<XT, ACT>(f.at(x, e));
#pragma unroll
                for (int r = t; r < W - 1; ++r) g[r][e] = fmaf(f.w[r - t][e], dz, g[r][e]);
            }
        }
#pragma unroll
        for (int r = 0; r < W - 1; ++r) Elems<XT>::store(p.ds_in, ((int64_t)s.n * (W - 1) + r) * p.C + c, g[r]);
        return;
    }
    const Place q = place_of(p, k, blockIdx.x);
    float dw[W + 1][8];   // the last one the bias's
#pragma unroll
    for (int i = 0; i <= W; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    }
    if (q.on && q.t0 < q.t1) {
        const Filter<W> f(p, q.c);
        for (int n = conv_find(p, q.t0); n < p.N; ++n) {
            const Seq s = conv_seq(p, n);
            if (s.a >= q.t1) break;
            const int64_t t = s.a > q.t0 ? s.a : q.t0, e1 = s.e < q.t1 ? s.e : q.t1;
            if (t >= e1) continue;
            float x[W][8], dz[W][8];
            window_before<XT, W>(p, s, t - s.a, q.c, x);
#pragma unroll
            for (int i = 0; i < W; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) dz[i][e] = 0.f;
            }
            const int64_t base = x_at(p, s, t) + q.c, left = s.e - t;
            const int m = (int)(e1 - t), real = left < m + W - 1 ? (int)left : m + W - 1;   // tokens whose dz counts
            typename Elems<XT>::Raw rx[U], rd[U];
            auto ask = [&](int u, int j) {
                const int at = j < real ? j : real - 1;
                rx[u] = Elems<XT>::load(p.x, base + at * p.st);
                rd[u] = Elems<XT>::load(p.dy, (t + at) * p.C + q.c);
            };
#pragma unroll
            for (int u = 0; u < U; ++u) ask(u, u);
            for (int i = 0; i < m + W - 1; i += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = i + u;
                    float dy[8], g[8];
                    shift(x);
                    shift(dz);
                    Elems<XT>::widen(rx[u], x[W - 1]);
                    Elems<XT>::widen(rd[u], dy);
                    ask(u, j + U);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float d = formed(dy[e] * slope_of<XT, ACT>(f.at(x, e)));
                        dz[W - 1][e] = j < real ? d : 0.f;
                        g[e] = 0.f;
#pragma unroll
                        for (int o = 0; o < W; ++o) g[e] = fmaf(f.w[W - 1 - o][e], dz[o][e], g[e]);
                    }
                    if (j < m) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
#pragma unroll
                            for (int o = 0; o < W; ++o) dw[o][e] = fmaf(dz[W - 1][e], x[o][e], dw[o][e]);
                            dw[W][e] += dz[W - 1][e];
                        }
                    }
                    const int64_t back = t + j - (W - 1);   // the token whose dx is whole
                    if (j >= W - 1 && j < m + W - 1) {
                        const int64_t last = back - (s.e - (W - 1));   // its row in the final state
                        if (last >= 0 && p.ds_out) {
                            float ds[8];
                            Elems<XT>::widen(Elems<XT>::load(p.ds_out, ((int64_t)s.n * (W - 1) + last) * p.C + q.c), ds);
#pragma unroll
                            for (int e = 0; e < 8; ++e) g[e] += ds[e];
                        }
                        Elems<XT>::store(p.dx, back * p.C + q.c, g);
                    }
                }
            }
        }
    }
    // the runs of the work-group's tile, in order
    const int nb = W + (p.db != nullptr), runs = NT / k.lanes;
    float* part = p.part + (int64_t)(blockIdx.x / k.cols) * nb * p.C;
#pragma unroll
    for (int i = 0; i <= W; ++i) {
        if (i < nb) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) sh[threadIdx.x][e] = dw[i][e];
            __syncthreads();
            const int col = (int)(blockIdx.x % k.cols) * 8 * k.lanes;
            for (int c = threadIdx.x; c < 8 * k.lanes; c += NT) {
                float sum = 0.f;
                for (int r = 0; r < runs; ++r) sum += sh[r * k.lanes + (c >> 3)][c & 7];
                if (col + c < p.C) part[(int64_t)i * p.C + col + c] = sum;
            }
        }
    }
}

// One token per row of a batch, the last W - 1 inputs of each sequence in a pool: a work-group
// takes 8 DT channels of a row.  Rows that name the same slot are tokens of one sequence in the
// order of the batch: the work-group of the first such row takes them all, those of the later
// ones end at once.  Rows with a slot outside the pool are skipped.
namespace {
constexpr int DT = 128;
}
template <int XT, int W, int ACT>
__global__ void __launch_bounds__(DT) kda_conv_decode_kernel(const ConvParams p) {
    const int pieces = p.C / 8, cols = (pieces + DT - 1) / DT;
    const int n0 = blockIdx.x / cols, piece = (int)(blockIdx.x % cols) * DT + threadIdx.x;
    const int slot = p.idx ? p.idx[n0] : n0;
    if (slot < 0 || slot >= p.slots) return;
    bool more = false;
    if (p.idx) {
        int f = 0;
        for (int m = threadIdx.x; m < p.N; m += DT)
            if (m != n0 && p.idx[m] == slot) f |= m < n0 ? 1 : 2;
        if (__syncthreads_or(f & 1)) return;
        more = __syncthreads_or(f & 2);
    }
    if (piece >= pieces) return;
    const int c = 8 * piece;
    const Filter<W> f(p, c);
    float x[W][8];
#pragma unroll
    for (int i = 1; i < W; ++i) {
        if (p.s_in) {
            Elems<XT>::widen(Elems<XT>::load(p.s_in, ((int64_t)slot * (W - 1) + i - 1) * p.C + c), x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
        }
    }
    int n = n0;
    do {
        shift(x);
        Elems<XT>::widen(Elems<XT>::load(p.x, n * p.sb + c), x[W - 1]);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = act_of<XT, ACT>(f.at(x, e));
        Elems<XT>::store(p.y, (int64_t)n * p.C + c, y);
        if (!more) break;
        do ++n;
        while (n < p.N && p.idx[n] != slot);
    } while (n < p.N);
#pragma unroll
    for (int i = 1; i < W; ++i) Elems<XT>::store(p.s_out, ((int64_t)slot * (W - 1) + i - 1) * p.C + c, x[i]);
}

// Sums over rows: a work-group takes 32 columns, eight threads each every eighth row, then in order.
__global__ void __launch_bounds__(256) kda_sum_rows_kernel(const SumParams p) {
    __shared__ double sh[8][32];
    const int g = threadIdx.x >> 5, l = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * 32 + l;
    double t = 0.0;   // the sums of a long batch keep fp32's accuracy
    if (c < p.cols) {
#pragma unroll 8
        for (int64_t r = g; r < p.n; r += 8) t += (double)p.part[r * p.cols + c];
    }
    sh[g][l] = t;
    __syncthreads();
    if (g == 0 && c < p.cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) t += sh[i][l];
        if (c < p.split) p.out[(c % p.inner) * p.outer + c / p.inner] = (float)t;
        else p.out2[c - p.split] = (float)t;
    }
}

hipError_t launch_sum_rows(const SumParams& p, hipStream_t stream) {
    if (p.cols == 0) return hipSuccess;
    hipLaunchKernelGGL(kda_sum_rows_kernel, dim3((unsigned)((p.cols + 31) / 32)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

ConvSplit conv_split(int64_t total, int64_t C, bool bwd) {
    const int64_t pieces = C / 8;
    ConvSplit k{};
    k.lanes = 64;
    while (k.lanes > 1 && k.lanes / 2 >= pieces) k.lanes /= 2;
    // fewer lanes side by side where the last column of them would be mostly empty
    while (k.lanes > 16 && (pieces + k.lanes - 1) / k.lanes * k.lanes - pieces > pieces / 32) k.lanes /= 2;
    k.cols = (pieces + k.lanes - 1) / k.lanes;
    auto tiles = [&](int run) { return (total + (int64_t)run * (NT / k.lanes) - 1) / ((int64_t)run * (NT / k.lanes)); };
    if (bwd) {   // Whole rounds of the 512 work-groups that the device holds at once, each as long as a run and the W - 1 tokens behind
                 // it: 8192 tokens x 4352 channels in runs of 36 (493 work-groups, one round) 47 us, of 32 (544) 61; 4096 x 4352 of 18
                 // (510) 32 us, of 16 (544) 40, of 32 (272) 39; 32768 x 1096 of 40 (468) 60 us, of 32 (576) 71; 16384 x 4352 of 36
                 // (986, two rounds) 101 us, of 32 (1088) 109, of 64 125; 8192 x 4096 of 32 (512) 44 us, of 36 (456) 47
        int64_t least = 0;
        for (int run = 8; run <= 40; run += 2) {
            const int64_t cost = (tiles(run) * k.cols + 511) / 512 * (run + 3);
            if (run == 8 || cost < least) {
                least = cost;
                k.run = run;
            }
        }
    } else {     // long runs read fewer rows twice, short ones fill the device: 8 and 32 tokens are 5.9 and 11.1 us at 512 x 4352, 29 and 31
                 // at 8192 x 4352, 62 and 56 at 16384 x 4352, 192 and 161 at 16384 x 12288.  fp16's four taps hold 169 registers, two waves a SIMD
                 // and not three: 33 and 32 us at 8192 x 4352, 237 and 161 at 16384 x 12288
        k.run = total * pieces >= (int64_t(3) << 21) ? 32 : 8;
    }
    k.tiles = tiles(k.run);
    return k;
}

namespace {
template <template <int, int, int> class K, typename... A>
void by_kind(const ConvParams& p, A... a) {
    auto act = [&](auto xt, auto w) {
        if (p.silu) K<decltype(xt)::value, decltype(w)::value, ACT_SILU>::run(p, a...);
        else K<decltype(xt)::value, decltype(w)::value, ACT_NONE>::run(p, a...);
    };
    auto width = [&](auto xt) {
        if (p.W == 2) act(xt, std::integral_constant<int, 2>());
        else if (p.W == 3) act(xt, std::integral_constant<int, 3>());
        else act(xt, std::integral_constant<int, 4>());
    };
    if (p.type == 0) width(std::integral_constant<int, 0>());
    else if (p.type == 1) width(std::integral_constant<int, 1>());
    else width(std::integral_constant<int, 2>());
}
template <int XT, int W, int ACT>
struct Forward {
    static void run(const ConvParams& p, const ConvSplit& k, unsigned blocks, hipStream_t s) {
        hipLaunchKernelGGL((kda_conv_kernel<XT, W, ACT>), dim3(blocks), dim3(NT), 0, s, p, k);
    }
};
template <int XT, int W, int ACT>
struct Backward {
    static void run(const ConvParams& p, const ConvSplit& k, unsigned blocks, hipStream_t s) {
        hipLaunchKernelGGL((kda_conv_bwd_kernel<XT, W, ACT>), dim3(blocks), dim3(NT), 0, s, p, k);
    }
};
template <int XT, int W, int ACT>
struct Decode {
    static void run(const ConvParams& p, unsigned blocks, hipStream_t s) {
        hipLaunchKernelGGL((kda_conv_decode_kernel<XT, W, ACT>), dim3(blocks), dim3(DT), 0, s, p);
    }
};
}  // namespace

hipError_t launch_conv(const ConvParams& p, hipStream_t stream) {
    const ConvSplit k = conv_split(p.total, p.C, false);
    const int64_t states = p.s_out ? ((int64_t)p.N * (p.W - 1) * (p.C / 8) + NT - 1) / NT : 0;
    const int64_t blocks = k.tiles * k.cols + states;
    if (blocks == 0) return hipSuccess;
    by_kind<Forward>(p, k, (unsigned)blocks, stream);
    return hipGetLastError();
}

hipError_t launch_conv_bwd(const ConvParams& p, hipStream_t stream) {
    const ConvSplit k = conv_split(p.total, p.C, true);
    const int64_t states = p.ds_in ? ((int64_t)p.N * (p.C / 8) + NT - 1) / NT : 0;
    const int64_t blocks = k.tiles * k.cols + states;
    if (blocks > 0) {
        by_kind<Backward>(p, k, (unsigned)blocks, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t nb = p.W + (p.db != nullptr);
    return launch_sum_rows(SumParams{p.part, k.tiles, nb * p.C, (int64_t)p.W * p.C, p.C, p.W, p.dw, p.db}, stream);
}

hipError_t launch_conv_decode(const ConvParams& p, hipStream_t stream) {
    const int64_t blocks = (int64_t)p.N * ((p.C / 8 + DT - 1) / DT);
    if (blocks == 0) return hipSuccess;
    by_kind<Decode>(p, (unsigned)blocks, stream);
    return hipGetLastError();
}

}  // namespace kda
