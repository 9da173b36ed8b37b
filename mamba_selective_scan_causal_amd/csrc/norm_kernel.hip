// norm_kernel.hip -- the norm before a block: s = residual + alpha scale x,
// y = norm(s) w + b, and its backward pass (mss_add_norm,
// mss_add_norm_backward); the sum of the parameter gradients' parts that
// gated_norm shares.
//
// Bound by HBM: the forward reads x and the residual and writes s and y, the
// backward reads s, dy, ds (and x) and writes dresidual and dx, each once.
// M 32768 D 2560 bf16 with an fp32 stream, a call of a row of calls (with the
// parameters' sums): forward 196 us (5.1 TB/s), backward with dscale 309 us (4.9
// TB/s).
// The outputs go through the cache: with the nontemporal hint the forward and
// backward of M 32768 D 2560 in turn take 561 us, without it 538.
#include "norm_common.h"

namespace mss {
namespace {

// s of one channel.  The product is rounded before the sum, as where the two
// are separate operations: with a half-precision stream and a scale like 0.7
// many sums lie next to the middle of two representable values, and a fused
// product would round them the other way.
__device__ __forceinline__ float scaled_sum(float res, float k, float x) {
#pragma clang fp contract(off)
    const float p = k * x;
    return res + p;
}

// A row as it was read: x and the residual, or s, dy, ds and x.
template <typename T, typename R, int NC>
struct AddRow {
    static constexpr int V = kVec<T>;
    RowVec<R, V> r[NC], ds[NC];
    RowVec<T, V> x[NC], dy[NC];
};

template <typename T, typename R, int TEAM, int NC, Ends ENDS>
__global__ __launch_bounds__((kMaxThreads<TEAM, NC>)) void add_norm_kernel(NormArgs q) {
    constexpr int V = kVec<T>;
    __shared__ float lds[kSumLds<TEAM>];
    const int n = static_cast<int>(q.D), lanes = team_lanes<TEAM>();
    const Spots<V, NC, ENDS> spots(team_lane<TEAM>(), lanes, n);
    const bool layer = q.kind == MSS_NORM_LAYER;
    const float inv_n = 1.0f / static_cast<float>(n);
    const int rows = TEAM == kGroup ? 1 : 256 / lanes;
    const int64_t step = gridDim.x * static_cast<int64_t>(rows);
    float w[NC][V], b[NC][V], k[NC][V];
#pragma unroll
    for (int j = 0; j < NC; j++) {
        const auto c = spots.s[j];
        load_param(q.w, c, n, 1.0f, w[j]);
        load_param(q.b, c, n, 0.0f, b[j]);
        load_param(q.scale, c, n, 1.0f, k[j]);
#pragma unroll
        for (int e = 0; e < V; e++) k[j][e] *= q.alpha;
    }
    auto read = [&](int64_t m, RowVec<R, V>(&res)[NC], RowVec<T, V>(&x)[NC]) {
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
            if (c.at < n && m < q.M) {
                if (q.res) res[j].load(row_of<R>(q.res, m, q.ld_res), c, n);
                x[j].load(row_of<T>(q.x, m, q.ld_x), c, n);
            }
        }
    };
    int turn = 0;
    int64_t m = blockIdx.x * static_cast<int64_t>(rows) + team_of<TEAM>();
    // (what lies past a row's end, or is not given, stays 0)
    RowVec<R, V> res[NC];
    RowVec<T, V> x[NC];
#pragma unroll
    for (int j = 0; j < NC; j++) {
        res[j].zero();
        x[j].zero();
    }
    clear_sums<TEAM>(lds);
    read(m, res, x);
    for (; m < q.M; m += step) {
        if (spots.shared) {
#pragma unroll
            for (int j = 0; j < NC; j++) {
                res[j].clear(spots.s[j]);
                x[j].clear(spots.s[j]);
            }
        }
        RowVec<R, V> s[NC];
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
#pragma unroll
            for (int e = 0; e < V; e++) s[j].set(e, scaled_sum(res[j][e], k[j][e], x[j][e]));
            if (c.at < n) s[j].template store<false>(row_of<R>(q.s, m, q.ld_s), c, n);
        }
        // the next row; this one has been read, so s may be the residual
        read(m + step, res, x);
        float mean = 0.0f;
        float sum[1] = {0.0f};
        if (layer) {
#pragma unroll
            for (int j = 0; j < NC; j++)
#pragma unroll
                for (int e = 0; e < V; e++) sum[0] += s[j][e];
            team_sum<TEAM>(sum, lds, turn);
            mean = sum[0] * inv_n;
            sum[0] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float v = spots.own(j, e, n) ? s[j][e] - mean : 0.0f;
                sum[0] = __builtin_fmaf(v, v, sum[0]);
            }
        team_sum<TEAM>(sum, lds, turn);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], inv_n, q.eps));
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
            RowVec<T, V> y;
#pragma unroll
            for (int e = 0; e < V; e++)
                y.set(e, __builtin_fmaf((s[j][e] - mean) * rstd, w[j][e], b[j][e]));
            if (c.at < n) y.template store<false>(row_of<T>(q.y, m, q.ld_y), c, n);
        }
    }
}

// EXTRA: db or dscale is wanted besides dw; either alone has the other summed as
// well (M 1551 D 1001 fp16 LAYER: 21.9 us a call with db, 20.3 without).
template <typename T, typename R, int TEAM, int NC, Ends ENDS, bool EXTRA>
__global__ __launch_bounds__((kMaxThreads<TEAM, NC>)) void add_norm_bwd_kernel(NormArgs q) {
    constexpr int V = kVec<T>, K = EXTRA ? 3 : 1;
    __shared__ float lds[kSumLds<TEAM>];
    __shared__ float part_lds[kPartLds<TEAM, NC, V>];
    const int n = static_cast<int>(q.D), lanes = team_lanes<TEAM>();
    const Spots<V, NC, ENDS> spots(team_lane<TEAM>(), lanes, n);
    const bool layer = q.kind == MSS_NORM_LAYER;
    const float inv_n = 1.0f / static_cast<float>(n);
    const int rows = TEAM == kGroup ? 1 : 256 / lanes;
    const int64_t step = gridDim.x * static_cast<int64_t>(rows);
    float w[NC][V], k[NC][V], acc[K][NC][V];
#pragma unroll
    for (int j = 0; j < NC; j++) {
        const auto c = spots.s[j];
        load_param(q.w, c, n, 1.0f, w[j]);
        load_param(q.scale, c, n, 1.0f, k[j]);
#pragma unroll
        for (int e = 0; e < V; e++) {
            k[j][e] *= q.alpha;
#pragma unroll
            for (int a = 0; a < K; a++) acc[a][j][e] = 0.0f;
        }
    }
    using Row = AddRow<T, R, NC>;
    auto read = [&](int64_t m, Row& r) {
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
            if (c.at < n && m < q.M) {
                r.r[j].load(row_of<R>(q.s, m, q.ld_s), c, n);
                r.dy[j].load(row_of<T>(q.dy, m, q.ld_y), c, n);
                if (q.ds) r.ds[j].load(row_of<R>(q.ds, m, q.ld_ds), c, n);
                if (EXTRA && q.x) r.x[j].load(row_of<T>(q.x, m, q.ld_x), c, n);
            }
        }
    };
    int turn = 0;
    int64_t m = blockIdx.x * static_cast<int64_t>(rows) + team_of<TEAM>();
    Row next;   // what lies past a row's end, or is not given, stays 0
#pragma unroll
    for (int j = 0; j < NC; j++) {
        next.r[j].zero();
        next.dy[j].zero();
        next.ds[j].zero();
        next.x[j].zero();
    }
    clear_sums<TEAM>(lds);
    read(m, next);
    for (; m < q.M; m += step) {
        Row r = next;
        read(m + step, next);
        if (spots.shared) {
#pragma unroll
            for (int j = 0; j < NC; j++) {
                r.r[j].clear(spots.s[j]);
                r.dy[j].clear(spots.s[j]);
            }
        }
        float mean = 0.0f;
        if (layer) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < NC; j++)
#pragma unroll
                for (int e = 0; e < V; e++) sum[0] += r.r[j][e];
            team_sum<TEAM>(sum, lds, turn);
            mean = sum[0] * inv_n;
        }
        // sums of (s - mean)^2, dy w (s - mean) and dy w (dy is 0 past the end)
        float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float v = spots.own(j, e, n) ? r.r[j][e] - mean : 0.0f;
                const float gw = r.dy[j][e] * w[j][e];
                sums[0] = __builtin_fmaf(v, v, sums[0]);
                sums[1] = __builtin_fmaf(gw, v, sums[1]);
                sums[2] += gw;
            }
        team_sum<TEAM>(sums, lds, turn);
#pragma unroll
        for (int j = 0; j < NC; j++) {
            r.r[j].narrow();
            r.dy[j].narrow();
        }
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(sums[0], inv_n, q.eps));
        const float c1 = sums[1] * inv_n * rstd;
        const float c2 = layer ? sums[2] * inv_n : 0.0f;
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
            RowVec<R, V> dres;
            RowVec<T, V> dx;
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float nv = (r.r[j][e] - mean) * rstd, g = r.dy[j][e];
                acc[0][j][e] = __builtin_fmaf(g, nv, acc[0][j][e]);
                const float t = __builtin_fmaf(g, w[j][e], -__builtin_fmaf(nv, c1, c2));
                const float d = __builtin_fmaf(rstd, t, r.ds[j][e]);
                if constexpr (EXTRA) {
                    acc[1][j][e] += g;
                    acc[2][j][e] = __builtin_fmaf(d, r.x[j][e], acc[2][j][e]);
                }
                dres.set(e, d);
                dx.set(e, d * k[j][e]);
            }
            if (c.at < n) {
                dres.template store<false>(row_of<R>(q.dres, m, q.ld_dres), c, n);
                if (q.dx) dx.template store<false>(row_of<T>(q.dx, m, q.ld_dx), c, n);
            }
        }
    }
    write_part<TEAM, NC, V, K, ENDS>(acc, part_lds, static_cast<float*>(q.ws) + blockIdx.x * K * q.D,
                               q.D, 0, n, spots);
}

// ---- rows too wide for the registers -------------------------------------------
// A pass over the row per round of sums, element by element, and parameter sums
// in memory: M 8192 D 8192 fp32 355 us forward and 826 us backward with dscale,
// where 1074 and 1611 MB would take 211 and 317 at a copy's rate (D 6144, held:
// 153 and 235).

constexpr int kWide = 1024;

template <typename T, typename R>
__global__ __launch_bounds__(kWide) void add_norm_wide_kernel(NormArgs q) {
    __shared__ float lds[kSumLds<kGroup>];
    int turn = 0;
    for (int64_t m = blockIdx.x; m < q.M; m += gridDim.x) {
        const T* x = row_of<T>(q.x, m, q.ld_x);
        const R* res = row_of<R>(q.res, m, q.ld_res);
        R* s = row_of<R>(q.s, m, q.ld_s);
        T* y = row_of<T>(q.y, m, q.ld_y);
        float sum[1] = {0.0f};
        for (int64_t c = threadIdx.x; c < q.D; c += kWide) {
            const float k = q.scale ? q.alpha * q.scale[c] : q.alpha;
            const float base = res ? static_cast<float>(res[c]) : 0.0f;
            s[c] = static_cast<R>(scaled_sum(base, k, static_cast<float>(x[c])));
            sum[0] += static_cast<float>(s[c]);
        }
        float mean = 0.0f;
        if (q.kind == MSS_NORM_LAYER) {
            team_sum<kGroup>(sum, lds, turn);
            mean = sum[0] / static_cast<float>(q.D);
        }
        sum[0] = 0.0f;
        for (int64_t c = threadIdx.x; c < q.D; c += kWide) {
            const float v = static_cast<float>(s[c]) - mean;
            sum[0] = __builtin_fmaf(v, v, sum[0]);
        }
        team_sum<kGroup>(sum, lds, turn);
        const float rstd = __builtin_amdgcn_rsqf(sum[0] / static_cast<float>(q.D) + q.eps);
        for (int64_t c = threadIdx.x; c < q.D; c += kWide) {
            const float nv = (static_cast<float>(s[c]) - mean) * rstd;
            y[c] = static_cast<T>(__builtin_fmaf(nv, q.w[c], q.b ? q.b[c] : 0.0f));
        }
    }
}

template <typename T, typename R>
__global__ __launch_bounds__(kWide) void add_norm_bwd_wide_kernel(NormArgs q) {
    __shared__ float lds[kSumLds<kGroup>];
    int turn = 0;
    float* part = static_cast<float*>(q.ws) + blockIdx.x * 3 * q.D;
    for (int64_t c = threadIdx.x; c < q.D; c += kWide)
        part[c] = part[q.D + c] = part[2 * q.D + c] = 0.0f;
    for (int64_t m = blockIdx.x; m < q.M; m += gridDim.x) {
        const R* s = row_of<R>(q.s, m, q.ld_s);
        const T* dy = row_of<T>(q.dy, m, q.ld_y);
        const R* ds = row_of<R>(q.ds, m, q.ld_ds);
        const T* x = row_of<T>(q.x, m, q.ld_x);
        R* dres = row_of<R>(q.dres, m, q.ld_dres);
        T* dx = row_of<T>(q.dx, m, q.ld_dx);
        float mean = 0.0f;
        if (q.kind == MSS_NORM_LAYER) {
            float sum[1] = {0.0f};
            for (int64_t c = threadIdx.x; c < q.D; c += kWide) sum[0] += static_cast<float>(s[c]);
            team_sum<kGroup>(sum, lds, turn);
            mean = sum[0] / static_cast<float>(q.D);
        }
        float sums[3] = {0.0f, 0.0f, 0.0f};
        for (int64_t c = threadIdx.x; c < q.D; c += kWide) {
            const float v = static_cast<float>(s[c]) - mean;
            const float gw = static_cast<float>(dy[c]) * q.w[c];
            sums[0] = __builtin_fmaf(v, v, sums[0]);
            sums[1] = __builtin_fmaf(gw, v, sums[1]);
            sums[2] += gw;
        }
        team_sum<kGroup>(sums, lds, turn);
        const float inv_n = 1.0f / static_cast<float>(q.D);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(sums[0], inv_n, q.eps));
        const float c1 = sums[1] * inv_n * rstd;
        const float c2 = q.kind == MSS_NORM_LAYER ? sums[2] * inv_n : 0.0f;
        for (int64_t c = threadIdx.x; c < q.D; c += kWide) {
            const float nv = (static_cast<float>(s[c]) - mean) * rstd;
            const float g = static_cast<float>(dy[c]);
            float d = ds ? static_cast<float>(ds[c]) : 0.0f;
            d = __builtin_fmaf(rstd, __builtin_fmaf(g, q.w[c], -__builtin_fmaf(nv, c1, c2)), d);
            part[c] = __builtin_fmaf(g, nv, part[c]);
            part[q.D + c] += g;
            if (x) part[2 * q.D + c] = __builtin_fmaf(d, static_cast<float>(x[c]), part[2 * q.D + c]);
            dres[c] = static_cast<R>(d);
            if (dx) dx[c] = static_cast<T>((q.scale ? q.alpha * q.scale[c] : q.alpha) * d);
        }
    }
}

// One workgroup sums 32 channels: 32 lanes side by side, 32 rows at a time, in
// a fixed order, all K sums at once.  4 to 13 us, most of it latency (768 rows of
// 3 x 2560 sums: 24 MB).  With 16 channels to a workgroup gated_norm forward and
// backward of M 32768 D 5120 take 521 us, like this 518; with 8 525.
template <int K>
__global__ __launch_bounds__(1024) void norm_params_kernel(NormArgs q, bool gated, int64_t rows) {
    __shared__ float lds[K][32][33];
    const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const float* part = static_cast<const float*>(q.ws);
    float S[3] = {0.0f, 0.0f, 0.0f};
    if (d < q.D) {
#pragma unroll 8
        for (int64_t p = group; p < rows; p += 32)
#pragma unroll
            for (int k = 0; k < K; k++) S[k] += part[(p * K + k) * q.D + d];
    }
#pragma unroll
    for (int k = 0; k < K; k++) lds[k][group][lane] = S[k];
    __syncthreads();
    if (group == 0) {
#pragma unroll
        for (int k = 0; k < K; k++) {
            S[k] = 0.0f;
#pragma unroll
            for (int g = 0; g < 32; g++) S[k] += lds[k][g][lane];
        }
    }
    if (group != 0 || d >= q.D) return;
    if (gated) {
        const float k = q.scale ? q.alpha * q.scale[d] : q.alpha;
        const float b = q.b ? q.b[d] : 0.0f;
        if (q.dw) q.dw[d] = k * S[0];
        if (q.db) q.db[d] = k * S[1];
        if (q.dscale) q.dscale[d] = q.alpha * __builtin_fmaf(q.w[d], S[0], b * S[1]);
    } else {
        if (q.dw) q.dw[d] = S[0];
        if (q.db) q.db[d] = S[1];
        if (q.dscale) q.dscale[d] = q.alpha * S[2];
    }
}

// f(activation, residual) for the call's types.
template <typename F>
hipError_t dispatch(const NormArgs& a, F f) {
    const bool wide = a.res_dtype == MSS_F32;
    switch (a.dtype) {
        case MSS_F32: f(float{}, float{}); break;
        case MSS_BF16: wide ? f(bf16{}, float{}) : f(bf16{}, bf16{}); break;
        case MSS_F16: wide ? f(f16{}, float{}) : f(f16{}, f16{}); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

bool norm_bwd_workspace(int64_t M, int64_t D, int64_t G, int64_t& bytes) {
    int64_t rows = (kMostParts + G - 1) / G;   // of partial sums, at most
    if (rows > M) rows = M;
    bytes = (rows * 3 * D * 4 + 255) / 256 * 256;
    return true;
}

hipError_t launch_norm_params(const NormArgs& a, bool gated, int64_t rows, int K, hipStream_t st) {
    if (!a.dw && !a.db && !a.dscale) return hipGetLastError();
    const unsigned grid = static_cast<unsigned>((a.D + 31) / 32);
    auto kernel = K == 1 ? norm_params_kernel<1> : K == 2 ? norm_params_kernel<2> : norm_params_kernel<3>;
    kernel<<<grid, 1024, 0, st>>>(a, gated, rows);
    return hipGetLastError();
}

hipError_t launch_add_norm(const NormArgs& a, hipStream_t st) {
    return dispatch(a, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        const bool held = by_width<T>(a.D, [&](auto s) {
            constexpr auto kernel = add_norm_kernel<T, R, s.TEAM, s.NC, s.ENDS>;
            const auto grid = row_groups<kernel>(a.M, 1, s.threads, s.rows);
            kernel<<<static_cast<unsigned>(grid), s.threads, 0, st>>>(a);
        });
        if (!held) {
            constexpr auto kernel = add_norm_wide_kernel<T, R>;
            const auto grid = row_groups<kernel>(a.M, 1, kWide, 1);
            kernel<<<static_cast<unsigned>(grid), kWide, 0, st>>>(a);
        }
    });
}

hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t st) {
    const bool extra = a.db || a.dscale;
    int64_t rows = 0;
    int K = extra ? 3 : 1;
    const hipError_t e = dispatch(a, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        const bool held = by_width<T>(a.D, [&](auto s) {
            auto go = [&](auto more) {
                constexpr auto kernel = add_norm_bwd_kernel<T, R, s.TEAM, s.NC, s.ENDS, more.value>;
                rows = row_groups<kernel>(a.M, 1, s.threads, s.rows, most_parts(a.M, s.threads));
                kernel<<<static_cast<unsigned>(rows), s.threads, 0, st>>>(a);
            };
            extra ? go(std::true_type{}) : go(std::false_type{});
        });
        if (!held) {
            constexpr auto kernel = add_norm_bwd_wide_kernel<T, R>;
            rows = row_groups<kernel>(a.M, 1, kWide, 1, most_parts(a.M, kWide));
            K = 3;
            kernel<<<static_cast<unsigned>(rows), kWide, 0, st>>>(a);
        }
    });
    return e == hipSuccess ? launch_norm_params(a, false, rows, K, st) : e;
}

}  // namespace mss
