// clip_kernel.hip -- the norm of all gradients, and clipping by it.
//
// The list of tensors goes to the kernels in their arguments, kList tensors a
// launch (nothing is copied to the device, so that a captured graph holds it).
// Tensors are cut into chunks, which the workgroups take in turn (neighbours at one
// time: a range of its own for each workgroup took 180 + 323 us in place of 173 + 298
// over 830 MB); a workgroup leaves one partial sum of squares.  Squares and sums are
// fp64: no square of a finite fp32 value overflows, and at two operations a
// value the sums hide behind the reads.  One workgroup adds the partial sums in
// order and writes the norm and the factor (or, of one list, every workgroup of the
// second pass for itself); the second pass scales.
#include "block_math.h"
#include "launch_ends.h"

namespace mss {
namespace {

constexpr int kList = 96;
constexpr int kThreads = 256;
constexpr int kLeastChunk = 2048, kMostChunk = 16384;      // elements; a power of two between them
constexpr int kMostBlocks = 2048;               // all resident at once: 256 CUs x 8

struct List {
    const void* in[kList];
    void* out[kList];
    int64_t numel[kList];
    uint32_t first[kList];    // number of the tensor's first chunk
    uint8_t dtype[kList], out_dtype[kList];
    int32_t count, chunk;     // tensors, elements of a chunk
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
    int i = tensor_of(l, blockIdx.x);
    for (uint32_t chunk = blockIdx.x; chunk < l.chunks; chunk += gridDim.x) {
        while (i + 1 < l.count && l.first[i + 1] <= chunk) i++;
        const int64_t from = int64_t{chunk - l.first[i]} * l.chunk;
        const int64_t n = l.numel[i] - from < l.chunk ? l.numel[i] - from : l.chunk;
        if (l.dtype[i] == MSS_F32) sum += squares(static_cast<const float*>(l.in[i]) + from, n);
        else if (l.dtype[i] == MSS_BF16) sum += squares(static_cast<const bf16*>(l.in[i]) + from, n);
        else sum += squares(static_cast<const f16*>(l.in[i]) + from, n);
    }
    sum = group_sum(sum, lds);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The factor, part 2^exponent: exponent 0 where it is a normal fp32 number (a value is then
// multiplied by it and rounded once, also a subnormal one: 1 leaves it as it is), else
// 1/2 <= part < 1, so that it keeps its digits (a norm near the end of the range).
struct Factor {
    float part;
    int exponent;
};

struct Clip {
    const double* part;       // partial sums of squares
    int64_t parts;
    float scale, max_norm;
    float* norm;
    Factor* factor;
};

// The norm, and the factor where it is asked for, from the partial sums.
__device__ __forceinline__ double norm_of(const Clip& c, double* lds) {
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < c.parts; i += kThreads) sum += c.part[i];
    return c.scale * sqrt(group_sum(sum, lds));
}

__device__ __forceinline__ Factor factor_of(const Clip& c, double norm) {
    const bool finite = norm < INFINITY;        // false for NaN too
    int exponent;
    const double part = frexp(!finite ? 1.0 : c.scale * (norm > c.max_norm ? c.max_norm / norm : 1.0), &exponent);
    if (exponent < -125) return {static_cast<float>(part), exponent};
    return {static_cast<float>(ldexp(part, exponent)), 0};
}

__global__ __launch_bounds__(kThreads) void norm_kernel(Clip c) {
    __shared__ double lds[kThreads / kWave];
    const double norm = norm_of(c, lds);
    if (threadIdx.x != 0) return;
    c.norm[0] = static_cast<float>(norm);
    if (c.factor) *c.factor = factor_of(c, norm);
}

// Stored past the caches, which keep more of what square_kernel read (830 MB of bf16:
// 168 + 295 -> 137 + 290 us; without the reversed order 142 + 306).
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
        o.template store<true>(out + c, 0, have);
    }
}

template <typename TI>
__device__ __forceinline__ void scaled_to(const void* in, void* out, bool wide, int64_t from, int64_t n, Factor f) {
    const TI* p = static_cast<const TI*>(in) + from;
    if (wide) scaled(p, static_cast<float*>(out) + from, n, f);
    else scaled(p, static_cast<TI*>(out) + from, n, f);
}

// OWN: every workgroup adds the partial sums up for itself, and the first writes
// the norm: a launch less (one block's gradients, 14 MB of fp32: 21.5 -> 16.9 us a call).
template <bool OWN>
__global__ __launch_bounds__(kThreads) void scale_kernel(List l, Clip c) {
    __shared__ double lds[kThreads / kWave];
    Factor f;
    if constexpr (OWN) {
        const double norm = norm_of(c, lds);
        if (blockIdx.x == 0 && threadIdx.x == 0) c.norm[0] = static_cast<float>(norm);
        f = factor_of(c, norm);
    } else {
        f = *c.factor;
    }
    // from the end, what square_kernel read last and the caches may still hold, each chunk on the XCD
    // that read it
    int64_t chunk = blockIdx.x + (l.chunks - 1 - blockIdx.x) / gridDim.x * gridDim.x;
    for (int i = tensor_of(l, static_cast<uint32_t>(chunk)); chunk >= 0; chunk -= gridDim.x) {
        while (l.first[i] > chunk) i--;
        if (f.part == 1.0f && f.exponent == 0 && l.in[i] == l.out[i] && l.dtype[i] == l.out_dtype[i]) continue;     // as it is
        const int64_t from = (chunk - l.first[i]) * l.chunk;
        const int64_t n = l.numel[i] - from < l.chunk ? l.numel[i] - from : l.chunk;
        const bool wide = l.out_dtype[i] == MSS_F32;
        if (l.dtype[i] == MSS_F32) scaled_to<float>(l.in[i], l.out[i], wide, from, n, f);
        else if (l.dtype[i] == MSS_BF16) scaled_to<bf16>(l.in[i], l.out[i], wide, from, n, f);
        else scaled_to<f16>(l.in[i], l.out[i], wide, from, n, f);
    }
}

// Calls f(list, workgroups) for every kList tensors that are not empty.  (The
// entry points bound the elements of all tensors, so the chunks are counted in 31
// bits.)
template <typename F>
hipError_t each_list(const mss_tensor* t, int64_t count, F&& f) {
    List l;
    for (int64_t i = 0; i < count;) {
        l.count = 0;
        int64_t total = 0;
        for (; i < count && l.count < kList; i++) {
            if (t[i].numel == 0) continue;
            l.in[l.count] = t[i].in;
            l.out[l.count] = t[i].out;
            l.numel[l.count] = t[i].numel;
            l.dtype[l.count] = static_cast<uint8_t>(t[i].dtype);
            l.out_dtype[l.count] = static_cast<uint8_t>(t[i].out_dtype);
            l.count++;
            total += t[i].numel;
        }
        if (l.count == 0) continue;
        // a few chunks to a workgroup where there is enough for all of them
        l.chunk = kLeastChunk;
        while (l.chunk < kMostChunk && total / l.chunk > 4 * kMostBlocks) l.chunk *= 2;
        int64_t chunks = 0;
        for (int k = 0; k < l.count; k++) {
            l.first[k] = static_cast<uint32_t>(chunks);
            chunks += (l.numel[k] + l.chunk - 1) / l.chunk;
        }
        l.chunks = static_cast<uint32_t>(chunks);
        const hipError_t e = f(l, chunks < kMostBlocks ? static_cast<uint32_t>(chunks) : kMostBlocks);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

// The factor, and the partial sums of every list's launch.
int64_t clip_workspace(int64_t count) { return 256 + (count + kList - 1) / kList * (kMostBlocks * 8); }

hipError_t launch_clip(const mss_tensor* t, int64_t count, float scale, float max_norm, bool write, float* norm,
                       void* ws, hipStream_t st) {
    double* part = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
    Clip c{part, 0, scale, max_norm, norm, write ? static_cast<Factor*>(ws) : nullptr};
    int lists = 0;
    hipError_t e = each_list(t, count, [&](const List& l, uint32_t blocks) {
        square_kernel<<<blocks, kThreads, 0, st>>>(l, part + c.parts);
        c.parts += blocks;
        lists++;
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    if (write && lists == 1)
        return each_list(t, count, [&](const List& l, uint32_t blocks) {
            scale_kernel<true><<<blocks, kThreads, 0, st>>>(l, c);
            return hipGetLastError();
        });
    norm_kernel<<<1, kThreads, 0, st>>>(c);
    if ((e = hipGetLastError()) != hipSuccess || !write) return e;
    return each_list(t, count, [&](const List& l, uint32_t blocks) {
        scale_kernel<false><<<blocks, kThreads, 0, st>>>(l, c);
        return hipGetLastError();
    });
}

}  // namespace mss
