// norm_kernel.hip -- the norms before and after a block (mss_add_norm,
// mss_gated_norm) and their backward passes.
//
// One workgroup per row: the row's groups are normalised one after the other,
// each in a pass for its moments and one that writes.  The backward adds its
// rows' shares of the parameter gradients to a row of the workspace that is
// its own, and a second kernel sums those rows in order.
#include "block_math.h"
#include "launch_block.h"

namespace mss {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kPartRows = 512;

// Sum of `v` over the workgroup, in every thread (two values at once).
__device__ __forceinline__ void block_sum2(float& a, float& b, float* lds) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        a += __shfl_xor(a, m, 64);
        b += __shfl_xor(b, m, 64);
    }
    const int wave = threadIdx.x / 64;
    __syncthreads();
    if (threadIdx.x % 64 == 0) {
        lds[2 * wave] = a;
        lds[2 * wave + 1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
    for (int w = 0; w < kThreads / 64; w++) {
        a += lds[2 * w];
        b += lds[2 * w + 1];
    }
}

// Mean (0 for RMS) and 1 / deviation of load(c), c in [0, n).
template <typename F>
__device__ __forceinline__ void moments(F load, int64_t n, int kind, float eps, float* lds,
                                        float& mean, float& rstd) {
    float sum = 0.0f, none = 0.0f;
    mean = 0.0f;
    if (kind == MSS_NORM_LAYER) {
        for (int64_t c = threadIdx.x; c < n; c += kThreads) sum += load(c);
        block_sum2(sum, none, lds);
        mean = sum / static_cast<float>(n);
    }
    float sq = 0.0f;
    for (int64_t c = threadIdx.x; c < n; c += kThreads) {
        const float v = load(c) - mean;
        sq = __builtin_fmaf(v, v, sq);
    }
    block_sum2(sq, none, lds);
    rstd = 1.0f / __builtin_sqrtf(sq / static_cast<float>(n) + eps);
}

template <typename T>
__device__ __forceinline__ T* row_of(const void* p, int64_t row, int64_t ld) {
    return const_cast<T*>(static_cast<const T*>(p)) + row * ld;
}

template <typename T, typename R>
__global__ __launch_bounds__(kThreads) void add_norm_kernel(NormArgs q) {
    __shared__ float lds[2 * kThreads / 64];
    for (int64_t m = blockIdx.x; m < q.M; m += gridDim.x) {
        const T* x = row_of<T>(q.x, m, q.ld_x);
        const R* res = row_of<R>(q.res, m, q.ld_res);
        R* s = row_of<R>(q.s, m, q.ld_s);
        T* y = row_of<T>(q.y, m, q.ld_y);
        for (int64_t c = threadIdx.x; c < q.D; c += kThreads) {
            const float k = q.alpha * (q.scale ? q.scale[c] : 1.0f);
            const float base = q.res ? static_cast<float>(res[c]) : 0.0f;
            s[c] = static_cast<R>(__builtin_fmaf(k, static_cast<float>(x[c]), base));
        }
        float mean, rstd;
        moments([&](int64_t c) { return static_cast<float>(s[c]); }, q.D, q.kind, q.eps, lds, mean,
                rstd);
        for (int64_t c = threadIdx.x; c < q.D; c += kThreads) {
            const float n = (static_cast<float>(s[c]) - mean) * rstd;
            y[c] = static_cast<T>(__builtin_fmaf(n, q.w[c], q.b ? q.b[c] : 0.0f));
        }
    }
}

template <typename T, typename R>
__global__ __launch_bounds__(kThreads) void add_norm_bwd_kernel(NormArgs q) {
    __shared__ float lds[2 * kThreads / 64];
    float* part = static_cast<float*>(q.ws) + blockIdx.x * 3 * q.D;
    for (int64_t c = threadIdx.x; c < q.D; c += kThreads)
        part[c] = part[q.D + c] = part[2 * q.D + c] = 0.0f;
    for (int64_t m = blockIdx.x; m < q.M; m += gridDim.x) {
        const R* s = row_of<R>(q.s, m, q.ld_s);
        const T* dy = row_of<T>(q.dy, m, q.ld_y);
        const R* ds = row_of<R>(q.ds, m, q.ld_ds);
        const T* x = row_of<T>(q.x, m, q.ld_x);
        float mean, rstd, c1 = 0.0f, c2 = 0.0f;
        moments([&](int64_t c) { return static_cast<float>(s[c]); }, q.D, q.kind, q.eps, lds, mean,
                rstd);
        for (int64_t c = threadIdx.x; c < q.D; c += kThreads) {
            const float g = static_cast<float>(dy[c]) * q.w[c];
            const float n = (static_cast<float>(s[c]) - mean) * rstd;
            c1 = __builtin_fmaf(g, n, c1);
            c2 += g;
        }
        block_sum2(c1, c2, lds);
        c1 /= static_cast<float>(q.D);
        c2 = q.kind == MSS_NORM_LAYER ? c2 / static_cast<float>(q.D) : 0.0f;
        for (int64_t c = threadIdx.x; c < q.D; c += kThreads) {
            const float gy = static_cast<float>(dy[c]);
            const float n = (static_cast<float>(s[c]) - mean) * rstd;
            float dres = rstd * (gy * q.w[c] - n * c1 - c2);
            if (q.ds) dres += static_cast<float>(ds[c]);
            const float k = q.alpha * (q.scale ? q.scale[c] : 1.0f);
            row_of<R>(q.dres, m, q.ld_dres)[c] = static_cast<R>(dres);
            if (q.dx) row_of<T>(q.dx, m, q.ld_dx)[c] = static_cast<T>(k * dres);
            part[c] += gy * n;
            part[q.D + c] += gy;
            if (q.x) part[2 * q.D + c] += dres * static_cast<float>(x[c]);
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_norm_kernel(NormArgs q) {
    __shared__ float lds[2 * kThreads / 64];
    const int64_t n = q.D / q.G;
    const bool before = q.order == MSS_GATE_BEFORE_NORM;
    for (int64_t m = blockIdx.x; m < q.M; m += gridDim.x) {
        for (int64_t g0 = 0; g0 < q.D; g0 += n) {
            const T* x = row_of<T>(q.x, m, q.ld_x) + g0;
            const T* z = row_of<T>(q.z, m, q.ld_z) + g0;
            const T* res = row_of<T>(q.res, m, q.ld_res) + g0;
            T* y = row_of<T>(q.y, m, q.ld_y) + g0;
            auto gate = [&](int64_t c) { return q.z ? silu(static_cast<float>(z[c])) : 1.0f; };
            auto v = [&](int64_t c) {
                return before ? static_cast<float>(x[c]) * gate(c) : static_cast<float>(x[c]);
            };
            float mean, rstd;
            moments(v, n, q.kind, q.eps, lds, mean, rstd);
            for (int64_t c = threadIdx.x; c < n; c += kThreads) {
                float o = __builtin_fmaf((v(c) - mean) * rstd, q.w[g0 + c], q.b ? q.b[g0 + c] : 0.0f);
                if (!before) o *= gate(c);
                o *= q.alpha * (q.scale ? q.scale[g0 + c] : 1.0f);
                if (q.res) o += static_cast<float>(res[c]);
                y[c] = static_cast<T>(o);
            }
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_norm_bwd_kernel(NormArgs q) {
    __shared__ float lds[2 * kThreads / 64];
    const int64_t n = q.D / q.G;
    const bool before = q.order == MSS_GATE_BEFORE_NORM;
    float* part = static_cast<float*>(q.ws) + blockIdx.x * 3 * q.D;
    for (int64_t c = threadIdx.x; c < q.D; c += kThreads)
        part[c] = part[q.D + c] = part[2 * q.D + c] = 0.0f;
    __syncthreads();
    for (int64_t m = blockIdx.x; m < q.M; m += gridDim.x) {
        for (int64_t g0 = 0; g0 < q.D; g0 += n) {
            const T* x = row_of<T>(q.x, m, q.ld_x) + g0;
            const T* z = row_of<T>(q.z, m, q.ld_z) + g0;
            const T* dout = row_of<T>(q.dy, m, q.ld_y) + g0;
            T* dx = row_of<T>(q.dx, m, q.ld_dx) + g0;
            T* dz = row_of<T>(q.dz, m, q.ld_dz) + g0;
            auto gate = [&](int64_t c) { return q.z ? silu(static_cast<float>(z[c])) : 1.0f; };
            auto v = [&](int64_t c) {
                return before ? static_cast<float>(x[c]) * gate(c) : static_cast<float>(x[c]);
            };
            // gradient of the normed row times w plus b
            auto dp = [&](int64_t c) {
                const float k = q.alpha * (q.scale ? q.scale[g0 + c] : 1.0f);
                const float dq = k * static_cast<float>(dout[c]);
                return before ? dq : dq * gate(c);
            };
            float mean, rstd, c1 = 0.0f, c2 = 0.0f;
            moments(v, n, q.kind, q.eps, lds, mean, rstd);
            for (int64_t c = threadIdx.x; c < n; c += kThreads) {
                const float g = dp(c) * q.w[g0 + c];
                c1 = __builtin_fmaf(g, (v(c) - mean) * rstd, c1);
                c2 += g;
            }
            block_sum2(c1, c2, lds);
            c1 /= static_cast<float>(n);
            c2 = q.kind == MSS_NORM_LAYER ? c2 / static_cast<float>(n) : 0.0f;
            for (int64_t c = threadIdx.x; c < n; c += kThreads) {
                const float nv = (v(c) - mean) * rstd;
                const float g = dp(c);
                const float p = __builtin_fmaf(nv, q.w[g0 + c], q.b ? q.b[g0 + c] : 0.0f);
                const float dv = rstd * (g * q.w[g0 + c] - nv * c1 - c2);
                const float k = q.alpha * (q.scale ? q.scale[g0 + c] : 1.0f);
                const float go = static_cast<float>(dout[c]);
                float f = 1.0f, slope = 0.0f;
                if (q.z) silu2(static_cast<float>(z[c]), f, slope);
                dx[c] = static_cast<T>(before ? dv * f : dv);
                if (q.z)
                    dz[c] = static_cast<T>(before ? dv * static_cast<float>(x[c]) * slope
                                                  : k * go * p * slope);
                part[g0 + c] += g * nv;
                part[q.D + g0 + c] += g;
                part[2 * q.D + g0 + c] += go * (before ? p : p * f);
            }
        }
    }
}

// dw, db and dscale from the workgroups' rows of partial sums.
__global__ __launch_bounds__(64) void norm_params_kernel(NormArgs q, int64_t rows) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (d >= q.D) return;
    const float* part = static_cast<const float*>(q.ws);
    float w = 0.0f, b = 0.0f, s = 0.0f;
    for (int64_t p = 0; p < rows; p++) {
        w += part[(3 * p) * q.D + d];
        b += part[(3 * p + 1) * q.D + d];
        s += part[(3 * p + 2) * q.D + d];
    }
    if (q.dw) q.dw[d] = w;
    if (q.db) q.db[d] = b;
    if (q.dscale) q.dscale[d] = q.alpha * s;
}

int64_t part_rows(int64_t M) { return M < kPartRows ? M : kPartRows; }
unsigned row_grid(int64_t M) { return static_cast<unsigned>(M < (1 << 20) ? M : (1 << 20)); }

hipError_t launch_params(const NormArgs& a, hipStream_t st) {
    if (!a.dw && !a.db && !a.dscale) return hipGetLastError();
    norm_params_kernel<<<static_cast<unsigned>((a.D + 63) / 64), 64, 0, st>>>(a, part_rows(a.M));
    return hipGetLastError();
}

template <typename F>
hipError_t dispatch(int dtype, F f) {
    switch (dtype) {
        case MSS_F32: f(float{}); break;
        case MSS_BF16: f(bf16{}); break;
        case MSS_F16: f(f16{}); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// f(activation, residual) for the call's types.
template <typename F>
hipError_t dispatch2(const NormArgs& a, F f) {
    return dispatch(a.dtype, [&](auto t) {
        if (a.res_dtype == MSS_F32)
            f(t, float{});
        else
            f(t, t);
    });
}

}  // namespace

bool norm_bwd_workspace(int64_t M, int64_t D, int64_t& bytes) {
    if (D > INT32_MAX) return false;
    bytes = (part_rows(M) * 3 * D * 4 + 255) / 256 * 256;
    return true;
}

hipError_t launch_add_norm(const NormArgs& a, hipStream_t st) {
    return dispatch2(a, [&](auto t, auto r) {
        add_norm_kernel<decltype(t), decltype(r)><<<row_grid(a.M), kThreads, 0, st>>>(a);
    });
}

hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t st) {
    const hipError_t e = dispatch2(a, [&](auto t, auto r) {
        add_norm_bwd_kernel<decltype(t), decltype(r)>
            <<<static_cast<unsigned>(part_rows(a.M)), kThreads, 0, st>>>(a);
    });
    return e == hipSuccess ? launch_params(a, st) : e;
}

hipError_t launch_gated_norm(const NormArgs& a, hipStream_t st) {
    return dispatch(a.dtype, [&](auto t) {
        gated_norm_kernel<decltype(t)><<<row_grid(a.M), kThreads, 0, st>>>(a);
    });
}

hipError_t launch_gated_norm_bwd(const NormArgs& a, hipStream_t st) {
    const hipError_t e = dispatch(a.dtype, [&](auto t) {
        gated_norm_bwd_kernel<decltype(t)>
            <<<static_cast<unsigned>(part_rows(a.M)), kThreads, 0, st>>>(a);
    });
    return e == hipSuccess ? launch_params(a, st) : e;
}

}  // namespace mss
