// api_check.h -- argument checks shared by the extern "C" layers: size
// products with overflow detection, required / alignment / overlap checks,
// and the thread's last HIP error.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <vector>

#include "mss.h"

namespace mss {

inline thread_local int g_last_hip_error = 0;

inline int hip_fail(hipError_t e) {
    g_last_hip_error = static_cast<int>(e);
    return MSS_EHIP;
}

struct Span {
    const void* p;
    int64_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

// n1 * n2 * ... with overflow detection (all factors >= 0).
inline bool mul_ok(int64_t& acc, int64_t f) {
    if (f == 0 || acc == 0) {
        acc = 0;
        return true;
    }
    if (acc > INT64_MAX / f) return false;
    acc *= f;
    return true;
}

inline bool count(int64_t& out, std::initializer_list<int64_t> fs) {
    int64_t acc = 1;
    for (int64_t f : fs)
        if (!mul_ok(acc, f)) return false;
    if (acc > INT64_MAX / 16) return false;  // byte offsets (x4) plus headroom
    out = acc;
    return true;
}

struct Checker {
    int status = MSS_OK;
    std::vector<Span> ins, outs;

    // A dense tensor of `elems` fp32 values (16-byte aligned).  Required
    // tensors may be NULL only when they hold no elements.
    void in(const float* p, int64_t elems, bool required) { add(ins, p, elems * 4, required, 16); }
    void out(float* p, int64_t elems, bool required) { add(outs, p, elems * 4, required, 16); }
    // `rows` rows of `width` fp32 values, row r at p + r * stride (4-byte aligned).
    void in_rows(const float* p, int64_t rows, int64_t width, int64_t stride, bool required) {
        add(ins, p, rows_bytes(rows, width, stride), required, 4);
    }
    void out_rows(float* p, int64_t rows, int64_t width, int64_t stride, bool required) {
        add(outs, p, rows_bytes(rows, width, stride), required, 4);
    }

    int64_t rows_bytes(int64_t rows, int64_t width, int64_t stride) {
        if (rows <= 0 || width <= 0) return 0;
        int64_t span;
        if (stride < width || !count(span, {rows - 1, stride}) || span > INT64_MAX / 8 - width) {
            if (status == MSS_OK) status = MSS_EINVAL;
            return 0;
        }
        return (span + width) * 4;
    }

    void add(std::vector<Span>& v, const void* p, int64_t bytes, bool required, uintptr_t align) {
        if (status != MSS_OK) return;
        if (!p) {
            if (required && bytes > 0) status = MSS_EINVAL;
            return;
        }
        if (reinterpret_cast<uintptr_t>(p) % align != 0) {
            status = MSS_EALIGN;
            return;
        }
        v.push_back({p, bytes});
    }

    int finish() {
        if (status != MSS_OK) return status;
        for (size_t i = 0; i < outs.size(); i++) {
            for (const Span& s : ins)
                if (overlap(outs[i], s)) return MSS_EALIAS;
            for (size_t j = i + 1; j < outs.size(); j++)
                if (overlap(outs[i], outs[j])) return MSS_EALIAS;
        }
        return MSS_OK;
    }
};

}  // namespace mss
