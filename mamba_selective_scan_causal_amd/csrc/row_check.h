// row_check.h -- argument checks of the entry points whose tensors are
// row-strided and of several element types (block_api.hip, ends_api.hip).
#pragma once

#include <cstdint>

#include "api_check.h"
#include "mss.h"

namespace mss {

inline int64_t elem_size(int dtype) { return dtype == MSS_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == MSS_F32 || dtype == MSS_BF16 || dtype == MSS_F16; }

// `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t rows, width, stride;
};

inline int64_t span(const Rows& r) { return r.rows <= 0 || r.width <= 0 ? 0 : (r.rows - 1) * r.stride + r.width; }

// Whether two tensors share a byte.  Column ranges of one buffer (equal
// strides) that interleave without meeting do not.
inline bool overlap(const Rows& a, const Rows& b) {
    const Span sa{a.p, span(a)}, sb{b.p, span(b)};
    if (!overlap(sa, sb)) return false;
    if (a.stride != b.stride) return true;
    const intptr_t diff = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
    const int64_t off = ((diff % a.stride) + a.stride) % a.stride;
    return !(off >= a.width && off + b.width <= a.stride);
}

class Checks {
  public:
    explicit Checks(bool strided) : strided_(strided) {}

    // A row-strided activation tensor: the element's alignment when the call
    // gives strides, 16 bytes otherwise.
    void in(const void* p, int64_t rows, int64_t width, int64_t ld, int64_t elem, bool required) {
        add(ins_, n_ins_, p, rows, width, ld, elem, required, strided_ ? elem : 16);
    }
    void out(void* p, int64_t rows, int64_t width, int64_t ld, int64_t elem, bool required) {
        add(outs_, n_outs_, p, rows, width, ld, elem, required, strided_ ? elem : 16);
    }
    // A dense tensor (16-byte aligned).
    void in(const void* p, int64_t elems, int64_t elem, bool required) {
        add(ins_, n_ins_, p, elems > 0 ? 1 : 0, elems, elems, elem, required, 16);
    }
    void out(void* p, int64_t elems, int64_t elem, bool required) {
        add(outs_, n_outs_, p, elems > 0 ? 1 : 0, elems, elems, elem, required, 16);
    }
    // A dense tensor at its element's alignment (ids, values per row).
    void in_any(const void* p, int64_t elems, int64_t elem, bool required) {
        add(ins_, n_ins_, p, elems > 0 ? 1 : 0, elems, elems, elem, required, elem);
    }
    void out_any(void* p, int64_t elems, int64_t elem, bool required) {
        add(outs_, n_outs_, p, elems > 0 ? 1 : 0, elems, elems, elem, required, elem);
    }
    // Bytes of any alignment (the reset flags).
    void in_bytes(const void* p, int64_t n) { add(ins_, n_ins_, p, n > 0 ? 1 : 0, n, n, 1, false, 1); }
    void must(bool ok) {
        if (!ok && status_ == MSS_OK) status_ = MSS_EINVAL;
    }
    // The workspace: of the size the query reports, overlapping nothing.
    void workspace(void* p, size_t bytes, int64_t need) {
        if (need == 0) return;
        ws_status_ = !p || bytes < static_cast<uint64_t>(need) ? MSS_EWORKSPACE
                     : reinterpret_cast<uintptr_t>(p) % 256    ? MSS_EALIGN
                                                               : MSS_OK;
        if (p) outs_[n_outs_++] = {p, 1, need, need};
    }
    // The input added last, for finish.
    int last() const { return n_ins_ - 1; }
    // An output may be exactly the input number `in_place` (same pointer, width
    // and stride), updated in place.
    int finish(int in_place = -1) {
        if (status_ != MSS_OK) return status_;
        for (int i = 0; i < n_outs_; i++) {
            for (int j = 0; j < n_ins_; j++) {
                const Rows& s = ins_[j];
                if (j == in_place && outs_[i].p == s.p && outs_[i].width == s.width &&
                    outs_[i].stride == s.stride)
                    continue;
                if (overlap(outs_[i], s)) return MSS_EALIAS;
            }
            for (int j = i + 1; j < n_outs_; j++)
                if (overlap(outs_[i], outs_[j])) return MSS_EALIAS;
        }
        return ws_status_;
    }

  private:
    void add(Rows* v, int& used, const void* p, int64_t rows, int64_t width, int64_t ld,
             int64_t elem, bool required, int64_t align) {
        if (status_ != MSS_OK) return;
        int64_t all;
        if (ld < width || !count(all, {rows, ld, elem})) {
            status_ = MSS_EINVAL;
            return;
        }
        if (!p) {
            if (required && rows > 0 && width > 0) status_ = MSS_EINVAL;
            return;
        }
        if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(align) != 0) {
            status_ = MSS_EALIGN;
            return;
        }
        if (rows > 0 && width > 0) v[used++] = {p, rows, width * elem, ld * elem};
    }

    bool strided_;
    int status_ = MSS_OK, ws_status_ = MSS_OK;
    // the longest argument list has ten inputs and seven outputs
    Rows ins_[16], outs_[16];
    int n_ins_ = 0, n_outs_ = 0;
};

inline int launched(hipError_t e) { return e == hipSuccess ? MSS_OK : hip_fail(e); }

}  // namespace mss
