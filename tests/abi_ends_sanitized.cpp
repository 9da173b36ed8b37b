// abi_ends_sanitized.cpp -- host-side argument validation and planning of the
// embedding, the head's loss and clipping under AddressSanitizer and
// UndefinedBehaviorSanitizer.  Built by tests/test_ends_abi_sanitized.py; every
// call is rejected, or is empty, before any HIP call, so it needs no GPU and the
// pointers are never dereferenced.  Sizes and strides are driven to the ends of
// int64.
#include <cstdint>
#include <cstdio>
#include <limits>
#include <vector>

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

mss_embed_dims ed(int64_t m, int64_t v, int64_t d) {
    return {sizeof(mss_embed_dims), 0, MSS_BF16, MSS_F32, 8, 0, m, v, d, 1.0f, 0};
}
mss_head_dims hd(int64_t m, int64_t v, int64_t d) {
    return {sizeof(mss_head_dims), 0, MSS_F16, 4, m, v, d, 1.0f, 0};
}

int embed(const mss_embed_dims& d, const mss_embed_strides* s, float* y) {
    return mss_embedding(&d, s, at(0), at(1), y, nullptr);
}
int embed_bwd(const mss_embed_dims& d, const mss_embed_strides* s, float* dw) {
    return mss_embedding_backward(&d, s, at(0), at(1), dw, at(3), SIZE_MAX, nullptr);
}
int loss(const mss_head_dims& d, const mss_head_strides* s, float* out) {
    return mss_head_loss(&d, s, at(0), at(1), at(2), out, at(4), at(5), SIZE_MAX, nullptr);
}
int loss_bwd(const mss_head_dims& d, const mss_head_strides* s, float* dx) {
    return mss_head_loss_backward(&d, s, at(0), at(1), at(2), at(3), at(4), at(5), dx, at(7), at(8), SIZE_MAX,
                                  nullptr);
}

}  // namespace

int main() {
    const int64_t top = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
    const int64_t sizes[] = {low, -1, 1, 127, 5000, int64_t{1} << 20, (int64_t{1} << 26) - 1, int64_t{1} << 28,
                             int64_t{1} << 40, int64_t{1} << 62, top};
    for (int64_t m : sizes)
        for (int64_t v : sizes)
            for (int64_t d : sizes) {
                // an output on an input keeps what is not refused for its size from launching
                const mss_embed_dims e = ed(m, v, d);
                size_t bytes = 1;
                const int q = mss_embed_workspace_bytes(&e, &bytes);
                expect(embed_bwd(e, nullptr, at(0)), q == MSS_OK ? MSS_EALIAS : MSS_EINVAL, "embed bwd", m, v, d);
                const int st = embed(e, nullptr, at(0));
                if (st != MSS_EINVAL) expect(st, MSS_EALIAS, "embed", m, v, d);
                const mss_head_dims h = hd(m, v, d);
                const int f = mss_head_workspace_bytes(&h, MSS_OP_HEAD_LOSS, &bytes);
                expect(loss(h, nullptr, at(0)), f == MSS_OK ? MSS_EALIAS : MSS_EINVAL, "loss", m, v, d);
                const int b = mss_head_workspace_bytes(&h, MSS_OP_HEAD_LOSS_BACKWARD, &bytes);
                expect(loss_bwd(h, nullptr, at(0)), b == MSS_OK ? MSS_EALIAS : MSS_EINVAL, "loss bwd", m, v, d);
            }
    const mss_embed_dims e = ed(3, 100, 64);
    const mss_head_dims h = hd(3, 100, 64);
    for (int64_t ld : {low, int64_t{-64}, int64_t{0}, int64_t{63}, top / 2, top}) {
        const mss_embed_strides s{sizeof(mss_embed_strides), 0, ld, ld};
        expect(embed(e, &s, at(2)), MSS_EINVAL, "embed stride", ld, 0, 0);
        expect(embed_bwd(e, &s, at(2)), MSS_EINVAL, "embed bwd stride", ld, 0, 0);
        const mss_head_strides t{sizeof(mss_head_strides), 0, ld, ld, ld, ld};
        expect(loss(h, &t, at(3)), MSS_EINVAL, "loss stride", ld, 0, 0);
        expect(loss_bwd(h, &t, at(6)), MSS_EINVAL, "loss bwd stride", ld, 0, 0);
    }
    // lists: sizes to the end, and many tensors of which two meet
    for (int64_t n : {low, int64_t{-1}, int64_t{1} << 44, int64_t{1} << 62, top}) {
        const mss_tensor t[2] = {{at(0), at(0), n, MSS_F32, MSS_F32}, {at(1), at(1), 5, MSS_BF16, MSS_F32}};
        expect(mss_clip_grads(t, 2, 1.0f, 1.0f, at(90), at(91), SIZE_MAX, nullptr), MSS_EINVAL, "list", n, 0, 0);
        size_t bytes;
        if (n < 0 || n >= (int64_t{1} << 31)) expect(mss_clip_workspace_bytes(n, &bytes), MSS_EINVAL, "count", n, 0, 0);
    }
    std::vector<mss_tensor> many;
    for (int i = 0; i < 1000; i++) many.push_back({at(i + 100), at(i + 100), 16 << 20, MSS_F32, MSS_F32});
    many[700].in = many[700].out = at(200) + 3;
    expect(mss_clip_grads(many.data(), 1000, 1.0f, 1.0f, at(0), at(1), SIZE_MAX, nullptr), MSS_EALIAS, "many", 0, 0, 0);
    if (g_failed) return 1;
    std::printf("all checks passed\n");
    return 0;
}
