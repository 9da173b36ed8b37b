// gated_kernel.hip -- the gated linear recurrence h_t = v_t + a_t h_{t-1} of
// mss.h, its backward pass and its single-token step.
//
// One lane per (batch row, channel) walks the sequence; neighbouring lanes
// hold neighbouring channels, so every time row is read in whole lines.
#include "block_math.h"
#include "launch_block.h"

namespace mss {
namespace {

// The gates of one token and channel: a, v and what the backward pass needs.
template <int GATE>
struct Gates {
    float a, v;
    float c;          // SIGMOID: 1 - a;  DECAY: 1 - sigma(r)
    float s, m, g;    // DECAY: sigma(r), sqrt(1 - a^2), sigma(i)
    float gc;         // DECAY: 1 - sigma(i)

    // k = c softplus(decay) (DECAY)
    __device__ __forceinline__ void set(float x, float r, float i, float k) {
        if constexpr (GATE == MSS_GATE_SIGMOID) {
            sigmoid2(r, a, c);
            v = c * x;
        } else if constexpr (GATE == MSS_GATE_DECAY) {
            sigmoid2(r, s, c);
            sigmoid2(i, g, gc);
            const float l2 = -kLog2e * k * s;
            a = ex2(l2);
            m = decay_input_scale(l2, a);
            v = m * g * x;
        } else {
            a = ex2(kLog2e * r);
            v = x;
        }
    }

    // Gradients for G = dL/dh_t and p = the state carried into the step.
    // `ws` is w sigma(r), whose sum gives ddecay: sigma(r) goes into the
    // term over m first, so that it has its limit where both vanish.
    __device__ __forceinline__ void grads(float G, float p, float x, float k, float& dx, float& dr,
                                          float& di, float& ws) const {
        if constexpr (GATE == MSS_GATE_SIGMOID) {
            dx = G * c;
            dr = G * (p - x) * (a * c);
        } else if constexpr (GATE == MSS_GATE_DECAY) {
            dx = G * (m * g);
            di = dx * x * gc;
            const float q = m > 0.0f ? g * a * a * (s * rcp(m)) : 0.0f;
            ws = G * __builtin_fmaf(a * s, p, -x * q);
            dr = -k * ws * c;
        } else {
            dx = G;
            dr = G * a * p;
        }
    }
};

constexpr int kSeg = MSS_GATED_CKPT_STEPS;

template <typename T, int GATE>
__global__ __launch_bounds__(64) void gated_scan_kernel(GatedArgs q) {
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (j >= q.B * q.D) return;
    const int64_t b = j / q.D, d = j % q.D;
    const T* x = static_cast<const T*>(q.x) + b * q.L * q.ld_x + d;
    const T* r = static_cast<const T*>(q.r) + b * q.L * q.ld_r + d;
    const T* in = static_cast<const T*>(q.i) + b * q.L * q.ld_i + d;
    const T* z = static_cast<const T*>(q.z) + b * q.L * q.ld_z + d;
    T* y = static_cast<T*>(q.y) + b * q.L * q.ld_y + d;
    const float k = GATE == MSS_GATE_DECAY ? q.gate_scale * softplus(q.decay[d]) : 0.0f;
    const int64_t nck = (q.L + kSeg - 1) / kSeg;
    float h = q.h0 ? q.h0[j] : 0.0f;
    for (int64_t t = 0; t < q.L; t++) {
        if (q.h_ckpt && t % kSeg == 0) q.h_ckpt[(b * nck + t / kSeg) * q.D + d] = h;
        Gates<GATE> g;
        const float iv = GATE == MSS_GATE_DECAY ? static_cast<float>(in[t * q.ld_i]) : 0.0f;
        g.set(static_cast<float>(x[t * q.ld_x]), static_cast<float>(r[t * q.ld_r]), iv, k);
        h = q.reset && q.reset[b * q.L + t] ? g.v : __builtin_fmaf(g.a, h, g.v);
        const float out = q.z ? h * silu(static_cast<float>(z[t * q.ld_z])) : h;
        y[t * q.ld_y] = static_cast<T>(out);
    }
    if (q.h_last) q.h_last[j] = h;
}

template <typename T, int GATE>
__global__ __launch_bounds__(64) void gated_scan_bwd_kernel(GatedArgs q) {
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (j >= q.B * q.D) return;
    const int64_t b = j / q.D, d = j % q.D;
    const T* x = static_cast<const T*>(q.x) + b * q.L * q.ld_x + d;
    const T* r = static_cast<const T*>(q.r) + b * q.L * q.ld_r + d;
    const T* in = static_cast<const T*>(q.i) + b * q.L * q.ld_i + d;
    const T* z = static_cast<const T*>(q.z) + b * q.L * q.ld_z + d;
    const T* dout = static_cast<const T*>(q.dout) + b * q.L * q.ld_y + d;
    T* dx = static_cast<T*>(q.dx) + b * q.L * q.ld_dx + d;
    T* dr = static_cast<T*>(q.dr) + b * q.L * q.ld_dr + d;
    T* di = static_cast<T*>(q.di) + b * q.L * q.ld_di + d;
    T* dz = static_cast<T*>(q.dz) + b * q.L * q.ld_dz + d;
    const float k = GATE == MSS_GATE_DECAY ? q.gate_scale * softplus(q.decay[d]) : 0.0f;
    const int64_t nck = (q.L + kSeg - 1) / kSeg;
    float Q = q.dh_last ? q.dh_last[j] : 0.0f;   // what the step after passes to h_t
    float sum = 0.0f;
    for (int64_t s = nck - 1; s >= 0; s--) {
        const int64_t t0 = s * kSeg;
        const int n = static_cast<int>(q.L - t0 < kSeg ? q.L - t0 : kSeg);
        float before[kSeg];
        float h = q.h_ckpt[(b * nck + s) * q.D + d];
        for (int u = 0; u < n; u++) {
            const int64_t t = t0 + u;
            Gates<GATE> g;
            const float iv = GATE == MSS_GATE_DECAY ? static_cast<float>(in[t * q.ld_i]) : 0.0f;
            g.set(static_cast<float>(x[t * q.ld_x]), static_cast<float>(r[t * q.ld_r]), iv, k);
            before[u] = q.reset && q.reset[b * q.L + t] ? 0.0f : h;
            h = __builtin_fmaf(g.a, before[u], g.v);
        }
        for (int u = n - 1; u >= 0; u--) {
            const int64_t t = t0 + u;
            Gates<GATE> g;
            const float xv = static_cast<float>(x[t * q.ld_x]);
            const float iv = GATE == MSS_GATE_DECAY ? static_cast<float>(in[t * q.ld_i]) : 0.0f;
            g.set(xv, static_cast<float>(r[t * q.ld_r]), iv, k);
            float dy = static_cast<float>(dout[t * q.ld_y]);
            if (q.z) {
                float f, slope;
                silu2(static_cast<float>(z[t * q.ld_z]), f, slope);
                dz[t * q.ld_dz] = static_cast<T>(dy * __builtin_fmaf(g.a, before[u], g.v) * slope);
                dy *= f;
            }
            const float G = dy + Q;
            float gx, gr, gi = 0.0f, ws = 0.0f;
            g.grads(G, before[u], xv, k, gx, gr, gi, ws);
            dx[t * q.ld_dx] = static_cast<T>(gx);
            dr[t * q.ld_dr] = static_cast<T>(gr);
            if constexpr (GATE == MSS_GATE_DECAY) di[t * q.ld_di] = static_cast<T>(gi);
            sum += ws;
            Q = q.reset && q.reset[b * q.L + t] ? 0.0f : g.a * G;
        }
    }
    if (q.dh0) q.dh0[j] = Q;
    if constexpr (GATE == MSS_GATE_DECAY) static_cast<float*>(q.ws)[j] = sum;
}

// ddecay[d] = -c sigma(decay[d]) sum over the partial rows.
__global__ __launch_bounds__(64) void gated_ddecay_kernel(const float* __restrict__ part,
                                                          const float* __restrict__ decay,
                                                          float* __restrict__ ddecay, int64_t rows,
                                                          int64_t D, float scale) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (d >= D) return;
    float sum = 0.0f;
    for (int64_t p = 0; p < rows; p++) sum += part[p * D + d];
    ddecay[d] = -scale * sigmoid(decay[d]) * sum;
}

template <typename T, int GATE>
__global__ __launch_bounds__(64) void gated_step_kernel(GatedArgs q) {
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (j >= q.B * q.D) return;
    const int64_t b = j / q.D, d = j % q.D;
    const float k = GATE == MSS_GATE_DECAY ? q.gate_scale * softplus(q.decay[d]) : 0.0f;
    const float iv = GATE == MSS_GATE_DECAY
                         ? static_cast<float>(static_cast<const T*>(q.i)[b * q.ld_i + d])
                         : 0.0f;
    Gates<GATE> g;
    g.set(static_cast<float>(static_cast<const T*>(q.x)[b * q.ld_x + d]),
          static_cast<float>(static_cast<const T*>(q.r)[b * q.ld_r + d]), iv, k);
    const float h = __builtin_fmaf(g.a, q.h[j], g.v);
    q.h[j] = h;
    const float out =
        q.z ? h * silu(static_cast<float>(static_cast<const T*>(q.z)[b * q.ld_z + d])) : h;
    static_cast<T*>(q.y)[b * q.ld_y + d] = static_cast<T>(out);
}

template <typename T, typename F>
hipError_t by_gate(int gate, F f) {
    switch (gate) {
        case MSS_GATE_SIGMOID: f(T{}, std::integral_constant<int, MSS_GATE_SIGMOID>{}); break;
        case MSS_GATE_DECAY: f(T{}, std::integral_constant<int, MSS_GATE_DECAY>{}); break;
        case MSS_GATE_LOG: f(T{}, std::integral_constant<int, MSS_GATE_LOG>{}); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// f(element, gate) for the call's types.
template <typename F>
hipError_t dispatch(const GatedArgs& a, F f) {
    switch (a.dtype) {
        case MSS_F32: return by_gate<float>(a.gate, f);
        case MSS_BF16: return by_gate<bf16>(a.gate, f);
        case MSS_F16: return by_gate<f16>(a.gate, f);
        default: return hipErrorInvalidValue;
    }
}

unsigned blocks(int64_t n) { return static_cast<unsigned>((n + 63) / 64); }

}  // namespace

bool gated_scan_workspace(int64_t B, int64_t L, int64_t D, int gate, int64_t& bytes) {
    bytes = 0;
    return B * D <= (int64_t{INT32_MAX} - 1) * 64;
}

bool gated_scan_bwd_workspace(int64_t B, int64_t L, int64_t D, int gate, int64_t& bytes) {
    bytes = gate == MSS_GATE_DECAY ? (B * D * 4 + 255) / 256 * 256 : 0;
    return B * D <= (int64_t{INT32_MAX} - 1) * 64;
}

hipError_t launch_gated_scan(const GatedArgs& a, hipStream_t st) {
    return dispatch(a, [&](auto t, auto gate) {
        gated_scan_kernel<decltype(t), gate.value><<<blocks(a.B * a.D), 64, 0, st>>>(a);
    });
}

hipError_t launch_gated_scan_bwd(const GatedArgs& a, hipStream_t st) {
    const hipError_t e = dispatch(a, [&](auto t, auto gate) {
        gated_scan_bwd_kernel<decltype(t), gate.value><<<blocks(a.B * a.D), 64, 0, st>>>(a);
    });
    if (e != hipSuccess || a.gate != MSS_GATE_DECAY) return e;
    gated_ddecay_kernel<<<blocks(a.D), 64, 0, st>>>(static_cast<const float*>(a.ws), a.decay,
                                                    a.ddecay, a.B, a.D, a.gate_scale);
    return hipGetLastError();
}

hipError_t launch_gated_step(const GatedArgs& a, hipStream_t st) {
    return dispatch(a, [&](auto t, auto gate) {
        gated_step_kernel<decltype(t), gate.value><<<blocks(a.B * a.D), 64, 0, st>>>(a);
    });
}

}  // namespace mss
