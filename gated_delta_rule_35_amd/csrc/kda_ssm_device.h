// Device helpers of the selective state space scan.
#pragma once
#include "kda_elems.h"
#include "kda_ssm.h"

namespace kda {

// x, which is the same in every lane, in scalar registers (what a division leaves in vector ones).
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x), hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}
// A token's step: dt + bias, or log(1 + e^{dt + bias}) of it.
__device__ __forceinline__ float ssm_raw(const void* dt, int f32, int64_t i, const float* bias, int h) {
    const float v = gdr_beta(dt, f32, i);
    return bias ? v + bias[h] : v;
}
__device__ __forceinline__ float ssm_step(float raw, int softplus) {
    if (!softplus) return raw;
    const float tail = log1pf(exp_of(-fabsf(raw)));
    return raw > 0.f ? raw + tail : tail;
}

// First token (in its row), length and row of sequence n, clamped to the row.
struct SsmSeq {
    int64_t bos, len, row;
};
__device__ __forceinline__ SsmSeq ssm_seq(const SsmParams& p, int n) {
    if (!p.cu) return {0, p.T, n};
    int64_t a = p.cu[n], e = p.cu[n + 1];
    a = a < 0 ? 0 : (a > p.T ? p.T : a);
    e = e < a ? a : (e > p.T ? p.T : e);
    return {a, e - a, 0};
}
// The packed sequence whose slots of `unit` tokens hold slot s: sequence n's start at
// cu[n] / unit + n, which grows with n.
__device__ __forceinline__ int ssm_find(const SsmParams& p, int64_t s, int64_t unit) {
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        int64_t a = p.cu[mid];
        a = a < 0 ? 0 : (a > p.T ? p.T : a);
        if (a / unit + mid <= s) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
// The chunk in slot s (the same in every lane): its sequence's row, first token and real rows (0: the slot is empty).
struct SsmChunk {
    int64_t tok, row;
    int rows;
};
__device__ __forceinline__ SsmChunk ssm_chunk(const SsmParams& p, int64_t s) {
    const int n = p.cu ? ssm_find(p, s, CH) : (int)(s / p.nc);
    const SsmSeq q = ssm_seq(p, n);
    const int64_t c = s - (p.cu ? q.bos / CH + n : (int64_t)n * p.nc), r = q.len - c * CH;
    return {uniform(q.bos + c * CH), uniform(q.row), uniform(c < 0 || r <= 0 ? 0 : (r >= CH ? CH : (int)r))};
}
// The segment in slot s: sequence, its segments (at least one), which of them it is (beyond them:
// the slot is empty), and the slot of the sequence's first segment and first chunk.
struct SsmSegment {
    SsmSeq q;
    int n, index, count;
    int64_t seg0, slot0;
};
__device__ __forceinline__ SsmSegment ssm_segment(const SsmParams& p, int64_t s) {
    const int64_t unit = (int64_t)p.segc * CH;
    SsmSegment g;
    g.n = p.cu ? ssm_find(p, s, unit) : (int)(s / p.nseg);
    g.q = ssm_seq(p, g.n);
    g.seg0 = p.cu ? g.q.bos / unit + g.n : (int64_t)g.n * p.nseg;
    g.slot0 = p.cu ? g.q.bos / CH + g.n : (int64_t)g.n * p.nc;
    g.index = (int)(s - g.seg0);
    const int64_t c = (g.q.len + unit - 1) / unit;
    g.count = c < 1 ? 1 : (int)c;
    return {{uniform(g.q.bos), uniform(g.q.len), uniform(g.q.row)}, uniform(g.n), uniform(g.index), uniform(g.count),
            uniform(g.seg0), uniform(g.slot0)};
}

// Row `row` of a record: the numbers of tokens 16 m + 4 g + r, r < 4.
__device__ __forceinline__ f32x4 num4(const float* rec, int row, int m, int g) {
    return *reinterpret_cast<const f32x4*>(rec + row + 16 * m + 4 * g);
}

}  // namespace kda
