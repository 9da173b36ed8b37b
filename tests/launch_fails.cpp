// Stands in for the HIP runtime's launch and last-error calls (preloaded): no
// kernel runs, the launch number `fail_at` fails, and hipGetLastError returns
// an error once and clears it, as documented.
#include <cstddef>

namespace {
int fail_at = -1, launches = 0, last = 0;
}

struct Dim3 {
    unsigned x, y, z;
};

extern "C" {
void launch_fails_at(int n) {
    fail_at = n;
    launches = 0;
    last = 0;
}
int launches_seen() { return launches; }

int __hipPushCallConfiguration(Dim3, Dim3, size_t, void*) { return 0; }
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* lds, void** stream) {
    *grid = *block = {1, 1, 1};
    *lds = 0;
    *stream = nullptr;
    return 0;
}
int hipLaunchKernel(const void*, Dim3, Dim3, void**, size_t, void*) {
    if (launches++ != fail_at) return 0;
    return last = 719;   // hipErrorLaunchFailure
}
int hipGetLastError() {
    const int e = last;
    last = 0;
    return e;
}
}
