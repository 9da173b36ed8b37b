// abi_block_sanitized.cpp -- host-side argument validation of the gated
// recurrence and the block norms under AddressSanitizer and
// UndefinedBehaviorSanitizer.  Built by tests/test_block_abi_sanitized.py;
// every call is rejected, or is empty, before any HIP call, so it needs no GPU
// and the pointers are never dereferenced.  Sizes and strides are driven to
// the ends of int64.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "mss.h"

namespace {

int g_failed = 0;
void expect(int got, int want, const char* what, int64_t a, int64_t b, int64_t c) {
    if (got == want) return;
    std::printf("FAIL %s (%lld, %lld, %lld): status %d, expected %d\n", what, (long long)a,
                (long long)b, (long long)c, got, want);
    g_failed++;
}

float* at(int i) {
    return reinterpret_cast<float*>(static_cast<uintptr_t>(0x7f0000000000ull) +
                                    static_cast<uintptr_t>(i) * (64ull << 20));
}

mss_gated_dims gd(int64_t b, int64_t l, int64_t d) {
    return {sizeof(mss_gated_dims), 0, MSS_BF16, MSS_GATE_DECAY, b, l, d, 8.0f, 0};
}
mss_norm_dims nd(int64_t m, int64_t d, int64_t g) {
    return {sizeof(mss_norm_dims), 0, MSS_F16, MSS_F16, MSS_NORM_LAYER, MSS_GATE_AFTER_NORM,
            m, d, g, 1e-6f, 1.0f};
}

int scan(const mss_gated_dims& d, const mss_gated_strides* s, float* y) {
    return mss_gated_scan(&d, s, at(0), at(1), at(2), at(3), at(4), at(5),
                          reinterpret_cast<uint8_t*>(at(6)), y, at(8), at(9), at(10), SIZE_MAX, nullptr);
}
int scan_bwd(const mss_gated_dims& d, const mss_gated_strides* s, float* dx) {
    return mss_gated_scan_backward(&d, s, at(0), at(1), at(2), at(3), at(4),
                                   reinterpret_cast<uint8_t*>(at(5)), at(6), at(7), at(8), dx, at(10),
                                   at(11), at(12), at(13), at(14), at(15), SIZE_MAX, nullptr);
}
int step(const mss_gated_dims& d, const mss_gated_strides* s, float* y) {
    return mss_gated_step(&d, s, at(0), at(1), at(2), at(3), at(4), at(5), y, nullptr);
}
int norm(const mss_norm_dims& d, const mss_norm_strides* s, float* y) {
    return mss_gated_norm(&d, s, at(0), at(1), at(2), at(3), at(4), at(5), y, nullptr);
}
int norm_bwd(const mss_norm_dims& d, const mss_norm_strides* s, float* dx) {
    return mss_gated_norm_backward(&d, s, at(0), at(1), at(2), at(3), at(4), at(5), dx, at(7), at(8),
                                   at(9), at(10), at(11), SIZE_MAX, nullptr);
}

}  // namespace

int main() {
    const int64_t top = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
    const int64_t sizes[] = {low, -1, 1, 127, int64_t{1} << 20, int64_t{1} << 31, int64_t{1} << 40,
                             int64_t{1} << 62, top};
    for (int64_t b : sizes)
        for (int64_t l : sizes)
            for (int64_t d : sizes) {
                // an output on an input keeps what is not refused for its size from launching
                const mss_gated_dims g = gd(b, l, d);
                size_t bytes = 1;
                const int q = mss_gated_workspace_bytes(&g, MSS_OP_GATED_SCAN, &bytes);
                const bool fits = q == MSS_OK;
                const int got = scan(g, nullptr, at(0));
                expect(got, fits ? MSS_EALIAS : MSS_EINVAL, "scan", b, l, d);
                const int back = mss_gated_workspace_bytes(&g, MSS_OP_GATED_SCAN_BACKWARD, &bytes);
                expect(scan_bwd(g, nullptr, at(0)), back == MSS_OK ? MSS_EALIAS : MSS_EINVAL, "bwd", b, l, d);
                const int st = step(g, nullptr, at(0));
                if (st != MSS_EINVAL && st != MSS_EALIAS) expect(st, MSS_EALIAS, "step", b, l, d);
                const mss_norm_dims n = nd(b, d, l);
                const int nq = mss_norm_workspace_bytes(&n, MSS_OP_GATED_NORM_BACKWARD, &bytes);
                expect(norm(n, nullptr, at(0)), nq == MSS_OK ? MSS_EALIAS : MSS_EINVAL, "norm", b, d, l);
                expect(norm_bwd(n, nullptr, at(0)), nq == MSS_OK ? MSS_EALIAS : MSS_EINVAL, "norm bwd", b, d, l);
            }
    const mss_gated_dims g = gd(3, 100, 64);
    const mss_norm_dims n = nd(3, 64, 2);
    for (int64_t ld : {low, int64_t{-64}, int64_t{0}, int64_t{63}, top / 2, top}) {
        mss_gated_strides s{sizeof(mss_gated_strides), 0, ld, ld, ld, ld, ld, ld, ld, ld, ld};
        expect(scan(g, &s, at(7)), MSS_EINVAL, "scan stride", ld, 0, 0);
        expect(scan_bwd(g, &s, at(9)), MSS_EINVAL, "bwd stride", ld, 0, 0);
        expect(step(g, &s, at(7)), MSS_EINVAL, "step stride", ld, 0, 0);
        mss_norm_strides t{sizeof(mss_norm_strides), 0, ld, ld, ld, ld, ld, ld, ld, ld, ld};
        expect(norm(n, &t, at(6)), MSS_EINVAL, "norm stride", ld, 0, 0);
        expect(norm_bwd(n, &t, at(6)), MSS_EINVAL, "norm bwd stride", ld, 0, 0);
    }
    if (g_failed) return 1;
    std::printf("all checks passed\n");
    return 0;
}
