// Host-side checks shared by the C-ABI front ends: no HIP call before a launch, and
// no device memory is read.
#pragma once
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdlib>

#include "../../include/kda.h"

namespace kda {
namespace check {

constexpr int64_t kHeadDim = 128;
constexpr int64_t kMaxBlocks = int64_t(1) << 22;  // 512 threads each: a grid stays below 2^31 work-items

inline int64_t numel(const kda_tensor_t* t) {
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
    return n;
}

inline size_t elem_size(kda_dtype_t d) { return (d == KDA_BF16 || d == KDA_F16) ? 2 : 4; }

inline bool contiguous(const kda_tensor_t* t) {
    int64_t expect = 1;
    for (int i = t->ndim - 1; i >= 0; --i) {
        if (t->shape[i] != 1 && t->stride[i] != expect) return false;
        expect *= t->shape[i];
    }
    return true;
}

inline kda_status_t check_tensor(const kda_tensor_t* t, int ndim, kda_dtype_t d0, kda_dtype_t d1, size_t align) {
    if (!t) return KDA_ERR_NULL;
    if (t->dtype != d0 && t->dtype != d1) return KDA_ERR_DTYPE;
    if (t->ndim != ndim) return KDA_ERR_SHAPE;
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] < 0) return KDA_ERR_SHAPE;
    const int64_t n = numel(t);
    if (n == 0) return KDA_OK;   // addresses no element: data and strides are not used
    if (!t->data) return KDA_ERR_NULL;
    if (!contiguous(t)) return KDA_ERR_LAYOUT;
    if ((reinterpret_cast<uintptr_t>(t->data) % align) != 0) return KDA_ERR_LAYOUT;
    return KDA_OK;
}

// Two state arrays of `bytes` each that share memory without starting at the
// same address.  A state may be updated in place, or written elsewhere; with a
// partial overlap one work-group's writes would land in tiles another has not
// read yet.
inline bool partly_overlap(const void* in, const void* out, int64_t bytes) {
    if (in == out || bytes <= 0) return false;
    const char* a = static_cast<const char*>(in);
    const char* b = static_cast<const char*>(out);
    return a < b + bytes && b < a + bytes;
}

// Two byte ranges that share memory (empty ranges share none).
inline bool ranges_overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    if (abytes <= 0 || bbytes <= 0 || !a || !b) return false;
    const char* x = static_cast<const char*>(a);
    const char* y = static_cast<const char*>(b);
    return x < y + bbytes && y < x + abytes;
}

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1;

// A tensor's bytes in memory, from its first element to past its last.
struct Span {
    const void* p;
    int64_t bytes;
};
inline Span span_of(const kda_tensor_t* t) {
    if (!t) return {nullptr, 0};
    int64_t last = 0;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->shape[i] <= 0) return {nullptr, 0};
        last += (t->shape[i] - 1) * t->stride[i];
    }
    return {t->data, (last + 1) * (int64_t)elem_size(t->dtype)};
}
inline bool overlaps(const kda_tensor_t* a, const kda_tensor_t* b) {
    const Span x = span_of(a), y = span_of(b);
    return ranges_overlap(x.p, x.bytes, y.p, y.bytes);
}
// Whether an output shares memory with an input or with another output.
inline bool any_overlap(const kda_tensor_t* const* outs, int no, const kda_tensor_t* const* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlaps(outs[i], ins[j])) return true;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}

inline bool sizes_ok(const kda_tensor_t* t) {
    for (int i = 0; i < t->ndim; ++i)
        if (t->shape[i] < 0 || t->shape[i] > kMaxTokens) return false;
    return true;
}

inline int64_t up256(int64_t x) { return (x + 255) & ~int64_t(255); }

inline bool same_shape(const kda_tensor_t* a, const int64_t* s, int nd) {
    for (int i = 0; i < nd; ++i)
        if (a->shape[i] != s[i]) return false;
    return true;
}

inline kda_status_t finish(hipError_t e, hipStream_t hs) {
    if (e != hipSuccess) return KDA_ERR_HIP;
    if (std::getenv("KDA_DEBUG_SYNC")) {
        if (hipStreamSynchronize(hs) != hipSuccess) return KDA_ERR_HIP;
        if (hipGetLastError() != hipSuccess) return KDA_ERR_HIP;
    }
    return KDA_OK;
}

// Compute units of the current device, read once per device (concurrent first
// reads store the same value).  0 if the runtime cannot tell.
inline int device_cus() {
    static std::atomic<int> cus[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
    int n = dev < 64 ? cus[dev].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) return 0;
    if (dev < 64) cus[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace check
}  // namespace kda
