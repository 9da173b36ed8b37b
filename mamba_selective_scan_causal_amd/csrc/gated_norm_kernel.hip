// gated_norm_kernel.hip -- the norm after a block with its gate and residual
// scale (mss_gated_norm) and its backward pass.
//
// Bound by HBM: the forward reads x, z (and the residual) and writes y, the
// backward reads x, z, dout and writes dx, dz, each once.  The outputs carry
// the nontemporal hint (M 32768 D 5120 bf16: forward 197 -> 188 us, backward
// 418 -> 405).  That size now, a call of a row of calls (with the parameters'
// sums): forward 209 us (4.8 TB/s), backward 318 us (5.3 TB/s; VALU busy 65 %).
#include "norm_common.h"

namespace mss {
namespace {

// The group of channels and the rows of a team: workgroup p of group g (the
// groups of a row side by side) takes rows p rows + team, and so on.
struct Place {
    int64_t g0, first, step;
};
template <int TEAM>
__device__ __forceinline__ Place place(const NormArgs& q) {
    const int rows = TEAM == kGroup ? 1 : 256 / team_lanes<TEAM>();
    const int64_t g = blockIdx.x % q.G, p = blockIdx.x / q.G;
    const int64_t team = team_of<TEAM>();
    return {g * (q.D / q.G), p * rows + team, gridDim.x / q.G * rows};
}

template <typename T, int TEAM, int NC, Ends ENDS, bool before, bool layer>
__global__ __launch_bounds__((kMaxThreads<TEAM, NC>)) void gated_norm_kernel(NormArgs q) {
    constexpr int V = kVec<T>;
    __shared__ float lds[kSumLds<TEAM>];
    const int n = static_cast<int>(q.D / q.G);
    const Spots<V, NC, ENDS> spots(team_lane<TEAM>(), team_lanes<TEAM>(), n);
    const float inv_n = 1.0f / static_cast<float>(n);
    const Place at = place<TEAM>(q);
    // k (norm w + b) with k = alpha scale folded into w and b
    float w[NC][V], b[NC][V];
#pragma unroll
    for (int j = 0; j < NC; j++) {
        const auto c = spots.s[j];
        float k[V];
        load_param(q.w + at.g0, c, n, 1.0f, w[j]);
        load_param(q.b ? q.b + at.g0 : nullptr, c, n, 0.0f, b[j]);
        load_param(q.scale ? q.scale + at.g0 : nullptr, c, n, 1.0f, k);
#pragma unroll
        for (int e = 0; e < V; e++) {
            w[j][e] *= q.alpha * k[e];
            b[j][e] *= q.alpha * k[e];
        }
    }
    struct Row {
        RowVec<T, V> x[NC], z[NC], res[NC];
    };
    auto read = [&](int64_t m, Row& r) {
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
            if (c.at < n && m < q.M) {
                r.x[j].load(row_of<T>(q.x, m, q.ld_x, at.g0), c, n);
                if (q.z) r.z[j].load(row_of<T>(q.z, m, q.ld_z, at.g0), c, n);
                if (q.res) r.res[j].load(row_of<T>(q.res, m, q.ld_res, at.g0), c, n);
            }
        }
    };
    int turn = 0;
    int64_t m = at.first;
    Row next;   // what lies past a row's end, or is not given, stays 0
#pragma unroll
    for (int j = 0; j < NC; j++) {
        next.x[j].zero();
        next.z[j].zero();
        next.res[j].zero();
    }
    clear_sums<TEAM>(lds);
    read(m, next);
    for (; m < q.M; m += at.step) {
        Row r = next;
        read(m + at.step, next);
        if (spots.shared) {
#pragma unroll
            for (int j = 0; j < NC; j++) {
                r.x[j].clear(spots.s[j]);
                r.z[j].clear(spots.s[j]);   // 0 times an infinite gate is NaN
            }
        }
        float v[NC][V];
        float mean = 0.0f;
        float sum[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int e = 0; e < V; e++) {
                v[j][e] = r.x[j][e];
                if (before && q.z) v[j][e] *= silu(r.z[j][e]);
                if constexpr (layer) sum[0] += v[j][e];
            }
        if constexpr (layer) {
            team_sum<TEAM>(sum, lds, turn);
            mean = sum[0] * inv_n;
            sum[0] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int e = 0; e < V; e++) {
                // (past the end an RMS norm's v is 0 already)
                if constexpr (layer)
                    v[j][e] = spots.own(j, e, n) ? v[j][e] - mean : 0.0f;
                sum[0] = __builtin_fmaf(v[j][e], v[j][e], sum[0]);
            }
        team_sum<TEAM>(sum, lds, turn);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], inv_n, q.eps));
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
            RowVec<T, V> y;
#pragma unroll
            for (int e = 0; e < V; e++) {
                v[j][e] = __builtin_fmaf(v[j][e] * rstd, w[j][e], b[j][e]);
                if (!before && q.z) v[j][e] *= silu(r.z[j][e]);
            }
            if (q.res) {
#pragma unroll
                for (int e = 0; e < V; e++) v[j][e] += r.res[j][e];
            }
#pragma unroll
            for (int e = 0; e < V; e++) y.set(e, v[j][e]);
            if (c.at < n) y.template store<true>(row_of<T>(q.y, m, q.ld_y, at.g0), c, n);
        }
    }
}

// EXTRA: the sum of the gradients alone is wanted too (for db, and for dscale
// where there is a bias).
template <typename T, int TEAM, int NC, Ends ENDS, bool before, bool layer, bool EXTRA>
__global__ __launch_bounds__((kMaxThreads<TEAM, NC>)) void gated_norm_bwd_kernel(NormArgs q) {
    constexpr int V = kVec<T>, K = EXTRA ? 2 : 1;
    __shared__ float lds[kSumLds<TEAM>];
    __shared__ float part_lds[kPartLds<TEAM, NC, V>];
    const int n = static_cast<int>(q.D / q.G);
    const Spots<V, NC, ENDS> spots(team_lane<TEAM>(), team_lanes<TEAM>(), n);
    const float inv_n = 1.0f / static_cast<float>(n);
    const Place at = place<TEAM>(q);
    float w[NC][V], acc[K][NC][V];   // w: k w, k = alpha scale
#pragma unroll
    for (int j = 0; j < NC; j++) {
        const auto c = spots.s[j];
        float k[V];
        load_param(q.w + at.g0, c, n, 1.0f, w[j]);
        load_param(q.scale ? q.scale + at.g0 : nullptr, c, n, 1.0f, k);
#pragma unroll
        for (int e = 0; e < V; e++) {
            w[j][e] *= q.alpha * k[e];
#pragma unroll
            for (int a = 0; a < K; a++) acc[a][j][e] = 0.0f;
        }
    }
    struct Row {
        RowVec<T, V> x[NC], z[NC], d[NC];
    };
    auto read = [&](int64_t m, Row& r) {
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
            if (c.at < n && m < q.M) {
                r.x[j].load(row_of<T>(q.x, m, q.ld_x, at.g0), c, n);
                if (q.z) r.z[j].load(row_of<T>(q.z, m, q.ld_z, at.g0), c, n);
                r.d[j].load(row_of<T>(q.dy, m, q.ld_y, at.g0), c, n);
            }
        }
    };
    int turn = 0;
    int64_t m = at.first;
    Row next;   // what lies past a row's end, or is not given, stays 0
#pragma unroll
    for (int j = 0; j < NC; j++) {
        next.x[j].zero();
        next.z[j].zero();
        next.d[j].zero();
    }
    clear_sums<TEAM>(lds);
    read(m, next);
    for (; m < q.M; m += at.step) {
        Row r = next;
        read(m + at.step, next);
        if (spots.shared) {
#pragma unroll
            for (int j = 0; j < NC; j++) {
                r.x[j].clear(spots.s[j]);
                r.z[j].clear(spots.s[j]);
                r.d[j].clear(spots.s[j]);
            }
        }
        // the gate's sigma(z), kept between the two halves of the row's work
        float sig[NC][V];
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int e = 0; e < V; e++) sig[j][e] = q.z ? sigmoid(r.z[j][e]) : 1.0f;
        auto gate = [&](int j, int e) { return q.z ? r.z[j][e] * sig[j][e] : 1.0f; };
        auto normed = [&](int j, int e) { return before ? r.x[j][e] * gate(j, e) : r.x[j][e]; };
        auto grad = [&](int j, int e) { return before ? r.d[j][e] : r.d[j][e] * gate(j, e); };
        float mean = 0.0f;
        if constexpr (layer) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < NC; j++)
#pragma unroll
                for (int e = 0; e < V; e++) sum[0] += normed(j, e);
            team_sum<TEAM>(sum, lds, turn);
            mean = sum[0] * inv_n;
        }
#pragma unroll
        for (int j = 0; j < NC; j++) {
            r.x[j].narrow();
            r.z[j].narrow();
            r.d[j].narrow();
        }
        constexpr int S = layer ? 3 : 2;
        float sums[S];
#pragma unroll
        for (int a = 0; a < S; a++) sums[a] = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int e = 0; e < V; e++) {
                float v = normed(j, e);
                if constexpr (layer) v = spots.own(j, e, n) ? v - mean : 0.0f;
                const float gw = grad(j, e) * w[j][e];
                sums[0] = __builtin_fmaf(v, v, sums[0]);
                sums[1] = __builtin_fmaf(gw, v, sums[1]);
                if constexpr (layer) sums[S - 1] += gw;
            }
        team_sum<TEAM>(sums, lds, turn);
#pragma unroll
        for (int j = 0; j < NC; j++) {
            r.x[j].narrow();
            r.z[j].narrow();
            r.d[j].narrow();
        }
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(sums[0], inv_n, q.eps));
        const float c1 = sums[1] * inv_n * rstd;
        const float c2 = layer ? sums[S - 1] * inv_n : 0.0f;
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const auto c = spots.s[j];
            RowVec<T, V> dx, dz;
            float kb[V], ks[V];
            if (!before && q.z) {   // k b, which enters dz
                load_param(q.b ? q.b + at.g0 : nullptr, c, n, 0.0f, kb);
                load_param(q.scale ? q.scale + at.g0 : nullptr, c, n, 1.0f, ks);
            }
#pragma unroll
            for (int e = 0; e < V; e++) {
                const float nv = (normed(j, e) - mean) * rstd, d = grad(j, e);
                acc[0][j][e] = __builtin_fmaf(d, nv, acc[0][j][e]);
                if constexpr (EXTRA) acc[1][j][e] += d;
                const float t =
                    __builtin_fmaf(d, w[j][e], -(layer ? __builtin_fmaf(nv, c1, c2) : nv * c1)) * rstd;
                dx.set(e, before ? t * gate(j, e) : t);
                if (q.z) {
                    // SiLU'(z) = sigma (1 + z (1 - sigma)); far below 0,
                    // where the sum cancels, sigma itself is as small
                    const float slope = sig[j][e] * __builtin_fmaf(r.z[j][e], 1.0f - sig[j][e], 1.0f);
                    dz.set(e, slope * (before ? t * r.x[j][e]
                                              : r.d[j][e] * __builtin_fmaf(nv, w[j][e],
                                                                           q.alpha * ks[e] * kb[e])));
                }
            }
            if (c.at < n) {
                dx.template store<true>(row_of<T>(q.dx, m, q.ld_dx, at.g0), c, n);
                if (q.z) dz.template store<true>(row_of<T>(q.dz, m, q.ld_dz, at.g0), c, n);
            }
        }
    }
    write_part<TEAM, NC, V, K, ENDS>(acc, part_lds,
                               static_cast<float*>(q.ws) + blockIdx.x / q.G * K * q.D, q.D, at.g0,
                               n, spots);
}

// ---- groups too wide for the registers -------------------------------------------
// A pass over the row per round of sums, element by element, and parameter sums
// in memory: M 8192 D 8192 fp32 301 us forward and 837 us backward, where 805 and
// 1342 MB would take 158 and 264 at a copy's rate (D 6144, held: 106 and 190).

constexpr int kWide = 1024;

template <typename T>
struct WideRow {
    const T* x;
    const T* z;
    bool before;
    __device__ __forceinline__ float gate(int64_t c) const {
        return z ? silu(static_cast<float>(z[c])) : 1.0f;
    }
    __device__ __forceinline__ float v(int64_t c) const {
        const float xv = static_cast<float>(x[c]);
        return before ? xv * gate(c) : xv;
    }
};

template <typename T>
__device__ __forceinline__ float wide_mean(const WideRow<T>& r, int64_t n, int kind, float* lds,
                                           int& turn) {
    if (kind != MSS_NORM_LAYER) return 0.0f;
    float sum[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < n; c += kWide) sum[0] += r.v(c);
    team_sum<kGroup>(sum, lds, turn);
    return sum[0] / static_cast<float>(n);
}

template <typename T>
__global__ __launch_bounds__(kWide) void gated_norm_wide_kernel(NormArgs q) {
    __shared__ float lds[kSumLds<kGroup>];
    const int64_t n = q.D / q.G;
    const float inv_n = 1.0f / static_cast<float>(n);
    const Place at = place<kGroup>(q);
    int turn = 0;
    for (int64_t m = at.first; m < q.M; m += at.step) {
        const WideRow<T> r{row_of<T>(q.x, m, q.ld_x, at.g0), row_of<T>(q.z, m, q.ld_z, at.g0),
                           q.order == MSS_GATE_BEFORE_NORM};
        const T* res = row_of<T>(q.res, m, q.ld_res, at.g0);
        T* y = row_of<T>(q.y, m, q.ld_y, at.g0);
        const float mean = wide_mean(r, n, q.kind, lds, turn);
        float sum[1] = {0.0f};
        for (int64_t c = threadIdx.x; c < n; c += kWide) {
            const float v = r.v(c) - mean;
            sum[0] = __builtin_fmaf(v, v, sum[0]);
        }
        team_sum<kGroup>(sum, lds, turn);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], inv_n, q.eps));
        for (int64_t c = threadIdx.x; c < n; c += kWide) {
            const int64_t d = at.g0 + c;
            float o = __builtin_fmaf((r.v(c) - mean) * rstd, q.w[d], q.b ? q.b[d] : 0.0f);
            if (!r.before) o *= r.gate(c);
            o *= q.scale ? q.alpha * q.scale[d] : q.alpha;
            y[c] = static_cast<T>(res ? o + static_cast<float>(res[c]) : o);
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kWide) void gated_norm_bwd_wide_kernel(NormArgs q) {
    __shared__ float lds[kSumLds<kGroup>];
    const int64_t n = q.D / q.G;
    const float inv_n = 1.0f / static_cast<float>(n);
    const Place at = place<kGroup>(q);
    int turn = 0;
    float* part = static_cast<float*>(q.ws) + blockIdx.x / q.G * 2 * q.D + at.g0;
    for (int64_t c = threadIdx.x; c < n; c += kWide) part[c] = part[q.D + c] = 0.0f;
    for (int64_t m = at.first; m < q.M; m += at.step) {
        const WideRow<T> r{row_of<T>(q.x, m, q.ld_x, at.g0), row_of<T>(q.z, m, q.ld_z, at.g0),
                           q.order == MSS_GATE_BEFORE_NORM};
        const T* dout = row_of<T>(q.dy, m, q.ld_y, at.g0);
        T* dx = row_of<T>(q.dx, m, q.ld_dx, at.g0);
        T* dz = row_of<T>(q.dz, m, q.ld_dz, at.g0);
        auto k = [&](int64_t c) { return q.scale ? q.alpha * q.scale[at.g0 + c] : q.alpha; };
        const float mean = wide_mean(r, n, q.kind, lds, turn);
        float sums[3] = {0.0f, 0.0f, 0.0f};
        for (int64_t c = threadIdx.x; c < n; c += kWide) {
            const float v = r.v(c) - mean;
            float g = k(c) * q.w[at.g0 + c] * static_cast<float>(dout[c]);
            if (!r.before) g *= r.gate(c);
            sums[0] = __builtin_fmaf(v, v, sums[0]);
            sums[1] = __builtin_fmaf(g, v, sums[1]);
            sums[2] += g;
        }
        team_sum<kGroup>(sums, lds, turn);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(sums[0], inv_n, q.eps));
        const float c1 = sums[1] * inv_n * rstd;
        const float c2 = q.kind == MSS_NORM_LAYER ? sums[2] * inv_n : 0.0f;
        for (int64_t c = threadIdx.x; c < n; c += kWide) {
            const float nv = (r.v(c) - mean) * rstd;
            const float w = q.w[at.g0 + c], go = static_cast<float>(dout[c]);
            float f = 1.0f, slope = 0.0f;
            if (r.z) silu2(static_cast<float>(r.z[c]), f, slope);
            const float d = r.before ? go : go * f;
            part[c] = __builtin_fmaf(d, nv, part[c]);
            part[q.D + c] += d;
            const float t = __builtin_fmaf(k(c) * w, d, -__builtin_fmaf(nv, c1, c2)) * rstd;
            if (r.z) {
                const float p = __builtin_fmaf(nv, w, q.b ? q.b[at.g0 + c] : 0.0f);
                dz[c] = static_cast<T>(slope * (r.before ? t * static_cast<float>(r.x[c])
                                                         : k(c) * go * p));
            }
            dx[c] = static_cast<T>(r.before ? t * f : t);
        }
    }
}

template <typename F>
hipError_t dispatch(const NormArgs& a, F f) {
    switch (a.dtype) {
        case MSS_F32: f(float{}); break;
        case MSS_BF16: f(bf16{}); break;
        case MSS_F16: f(f16{}); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// f(gate before norm, layer norm) for the call.
template <typename F>
void by_kind(const NormArgs& a, F f) {
    const bool layer = a.kind == MSS_NORM_LAYER;
    if (a.order == MSS_GATE_BEFORE_NORM)
        layer ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
    else
        layer ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

}  // namespace

hipError_t launch_gated_norm(const NormArgs& a, hipStream_t st) {
    return dispatch(a, [&](auto t) {
        using T = decltype(t);
        const bool held = by_width<T>(a.D / a.G, [&](auto s) {
            by_kind(a, [&](auto before, auto layer) {
                constexpr auto kernel = gated_norm_kernel<T, s.TEAM, s.NC, s.ENDS, before.value, layer.value>;
                const auto grid = a.G * row_groups<kernel>(a.M, a.G, s.threads, s.rows);
                kernel<<<static_cast<unsigned>(grid), s.threads, 0, st>>>(a);
            });
        });
        if (!held) {
            constexpr auto kernel = gated_norm_wide_kernel<T>;
            const auto grid = a.G * row_groups<kernel>(a.M, a.G, kWide, 1);
            kernel<<<static_cast<unsigned>(grid), kWide, 0, st>>>(a);
        }
    });
}

hipError_t launch_gated_norm_bwd(const NormArgs& a, hipStream_t st) {
    const bool extra = a.db || (a.dscale && a.b);
    int64_t rows = 0;
    int K = extra ? 2 : 1;
    const hipError_t e = dispatch(a, [&](auto t) {
        using T = decltype(t);
        const bool held = by_width<T>(a.D / a.G, [&](auto s) {
            by_kind(a, [&](auto before, auto layer) {
                auto go = [&](auto more) {
                    constexpr auto kernel = gated_norm_bwd_kernel<T, s.TEAM, s.NC, s.ENDS, before.value,
                                                                  layer.value, more.value>;
                    rows = row_groups<kernel>(a.M, a.G, s.threads, s.rows,
                                              most_parts(a.M, s.threads));
                    kernel<<<static_cast<unsigned>(rows * a.G), s.threads, 0, st>>>(a);
                };
                extra ? go(std::true_type{}) : go(std::false_type{});
            });
        });
        if (!held) {
            constexpr auto kernel = gated_norm_bwd_wide_kernel<T>;
            rows = row_groups<kernel>(a.M, a.G, kWide, 1, most_parts(a.M, kWide));
            K = 2;
            kernel<<<static_cast<unsigned>(rows * a.G), kWide, 0, st>>>(a);
        }
    });
    return e == hipSuccess ? launch_norm_params(a, true, rows, K, st) : e;
}

}  // namespace mss
