// clip_kernel.hip -- the norm of all gradients, and clipping by it.
//
// The list of tensors goes to the kernels in their arguments, kList tensors a
// launch (nothing is copied to the device, so that a captured graph holds it).
// Tensors are cut into chunks of kChunk elements, which the workgroups take in
// turn; a workgroup leaves one partial sum of squares.  Squares and sums are
// fp64: no square of a finite fp32 value overflows, and at two operations a
// value the sums hide behind the reads.  One workgroup adds the partial sums in
// order and writes the norm and the factor; the second pass scales.
#include "block_math.h"
#include "launch_ends.h"

namespace mss {
namespace {

constexpr int kList = 96;
constexpr int kThreads = 256;
constexpr int kChunk = 16384;
constexpr int kMostBlocks = 2048;               // all resident at once: 256 CUs x 8

struct List {
    const void* in[kList];
    void* out[kList];
    int64_t numel[kList];
    uint32_t first[kList];    // number of the tensor's first chunk
    uint8_t dtype[kList], out_dtype[kList];
    int32_t count;
    uint32_t chunks;
};
static_assert(sizeof(List) < 3584, "fits the kernel's arguments");

// The tensor that a chunk belongs to.
__device__ __forceinline__ int tensor_of(const List& l, uint32_t chunk) {
    int lo = 0, hi = l.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (l.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ double squares(const T* p, int64_t n) {
    constexpr int V = 16 / sizeof(T), kAhead = 4;
    double sum = 0.0;
    int64_t c = threadIdx.x * V;
    for (; c + (kAhead - 1) * kThreads * V + V <= n; c += kAhead * kThreads * V) {
        RowVec<T, V> r[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) r[i].t = *reinterpret_cast<const typename RowVec<T, V>::type*>(p + c + i * kThreads * V);
#pragma unroll
        for (int i = 0; i < kAhead; i++)
#pragma unroll
            for (int e = 0; e < V; e++) sum = __builtin_fma(static_cast<double>(r[i][e]), static_cast<double>(r[i][e]), sum);
    }
    for (; c < n; c += kThreads * V) {
        RowVec<T, V> r;
        r.load(p + c, 0, n - c < V ? static_cast<int>(n - c) : V);
#pragma unroll
        for (int e = 0; e < V; e++) sum = __builtin_fma(static_cast<double>(r[e]), static_cast<double>(r[e]), sum);
    }
    return sum;
}

__device__ __forceinline__ double group_sum(double v, double* lds) {
    for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kThreads / kWave; w++) v += lds[w];
    return v;
}

__global__ __launch_bounds__(kThreads) void square_kernel(List l, double* part) {
    __shared__ double lds[kThreads / kWave];
    double sum = 0.0;
    for (uint32_t chunk = blockIdx.x; chunk < l.chunks; chunk += gridDim.x) {
        const int i = tensor_of(l, chunk);
        const int64_t from = int64_t{chunk - l.first[i]} * kChunk;
        const int64_t n = l.numel[i] - from < kChunk ? l.numel[i] - from : kChunk;
        if (l.dtype[i] == MSS_F32) sum += squares(static_cast<const float*>(l.in[i]) + from, n);
        else if (l.dtype[i] == MSS_BF16) sum += squares(static_cast<const bf16*>(l.in[i]) + from, n);
        else sum += squares(static_cast<const f16*>(l.in[i]) + from, n);
    }
    sum = group_sum(sum, lds);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The factor as part 2^exponent, 1/2 <= part < 1, so that it keeps its digits where
// it is subnormal in fp32 (a norm near the end of the range).
struct Factor {
    float part;
    int exponent;
};

// The norm, and the factor of scale_kernel.
__global__ __launch_bounds__(kThreads) void norm_kernel(const double* part, int64_t n, float scale, float max_norm,
                                                        float* norm, Factor* factor) {
    __shared__ double lds[kThreads / kWave];
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += part[i];
    sum = group_sum(sum, lds);
    if (threadIdx.x != 0) return;
    const double total = scale * sqrt(sum);
    norm[0] = static_cast<float>(total);
    if (!factor) return;
    const bool finite = total < INFINITY;       // false for NaN too
    int exponent;
    const double most = frexp(!finite ? 1.0 : scale * (total > max_norm ? max_norm / total : 1.0), &exponent);
    *factor = {static_cast<float>(most), exponent};
}

template <typename TI, typename TO>
__device__ __forceinline__ void scaled(const TI* in, TO* out, int64_t n, Factor f) {
    constexpr int V = 16 / sizeof(TI);
    for (int64_t c = threadIdx.x * V; c < n; c += kThreads * V) {
        const int have = n - c < V ? static_cast<int>(n - c) : V;
        RowVec<TI, V> r;
        RowVec<TO, V> o;
        r.load(in + c, 0, have);
#pragma unroll
        for (int e = 0; e < V; e++) o.set(e, __builtin_ldexpf(r[e] * f.part, f.exponent));
        o.template store<false>(out + c, 0, have);
    }
}

template <typename TI>
__device__ __forceinline__ void scaled_to(const void* in, void* out, bool wide, int64_t from, int64_t n, Factor f) {
    const TI* p = static_cast<const TI*>(in) + from;
    if (wide) scaled(p, static_cast<float*>(out) + from, n, f);
    else scaled(p, static_cast<TI*>(out) + from, n, f);
}

__global__ __launch_bounds__(kThreads) void scale_kernel(List l, const Factor* factor) {
    const Factor f = *factor;
    for (uint32_t chunk = blockIdx.x; chunk < l.chunks; chunk += gridDim.x) {
        const int i = tensor_of(l, chunk);
        if (f.part == 0.5f && f.exponent == 1 && l.in[i] == l.out[i] && l.dtype[i] == l.out_dtype[i]) continue;     // as it is
        const int64_t from = int64_t{chunk - l.first[i]} * kChunk;
        const int64_t n = l.numel[i] - from < kChunk ? l.numel[i] - from : kChunk;
        const bool wide = l.out_dtype[i] == MSS_F32;
        if (l.dtype[i] == MSS_F32) scaled_to<float>(l.in[i], l.out[i], wide, from, n, f);
        else if (l.dtype[i] == MSS_BF16) scaled_to<bf16>(l.in[i], l.out[i], wide, from, n, f);
        else scaled_to<f16>(l.in[i], l.out[i], wide, from, n, f);
    }
}

// Calls f(list, workgroups) for every kList tensors.  (The entry points bound
// the elements of all tensors, so the chunks are counted in 31 bits.)
template <typename F>
hipError_t each_list(const mss_tensor* t, int64_t count, F&& f) {
    List l;
    l.count = 0;
    uint64_t chunks = 0;
    const auto send = [&]() -> hipError_t {
        if (l.count == 0) return hipSuccess;
        l.chunks = static_cast<uint32_t>(chunks);
        const hipError_t e = f(l, chunks < kMostBlocks ? static_cast<uint32_t>(chunks) : kMostBlocks);
        l.count = 0;
        chunks = 0;
        return e;
    };
    for (int64_t i = 0; i < count; i++) {
        if (t[i].numel == 0) continue;
        const uint64_t more = (static_cast<uint64_t>(t[i].numel) + kChunk - 1) / kChunk;
        if (l.count == kList)
            if (hipError_t e = send()) return e;
        l.in[l.count] = t[i].in;
        l.out[l.count] = t[i].out;
        l.numel[l.count] = t[i].numel;
        l.first[l.count] = static_cast<uint32_t>(chunks);
        l.dtype[l.count] = static_cast<uint8_t>(t[i].dtype);
        l.out_dtype[l.count] = static_cast<uint8_t>(t[i].out_dtype);
        l.count++;
        chunks += more;
    }
    return send();
}

}  // namespace

// The factor, and the partial sums of every list's launch.
int64_t clip_workspace(int64_t count) { return 256 + (count + kList - 1) / kList * (kMostBlocks * 8); }

hipError_t launch_clip(const mss_tensor* t, int64_t count, float scale, float max_norm, bool write, float* norm,
                       void* ws, hipStream_t st) {
    Factor* factor = static_cast<Factor*>(ws);
    double* part = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
    int64_t used = 0;
    hipError_t e = each_list(t, count, [&](const List& l, uint32_t blocks) {
        square_kernel<<<blocks, kThreads, 0, st>>>(l, part + used);
        used += blocks;
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    norm_kernel<<<1, kThreads, 0, st>>>(part, used, scale, max_norm, norm, write ? factor : nullptr);
    if ((e = hipGetLastError()) != hipSuccess || !write) return e;
    return each_list(t, count, [&](const List& l, uint32_t blocks) {
        scale_kernel<<<blocks, kThreads, 0, st>>>(l, factor);
        return hipGetLastError();
    });
}

}  // namespace mss
