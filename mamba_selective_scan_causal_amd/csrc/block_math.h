// block_math.h -- element types and gate functions of the gated recurrence and
// the block norms (gated_kernel.hip, norm_kernel.hip).
#pragma once

#include "device_math.h"

namespace mss {

using bf16 = __bf16;
using f16 = _Float16;

// How a row ends: with a whole vector (kWhole), with a partial one that is read
// as the V channels up to the row's end (kTail, rows of V channels or more), or
// with one that goes element by element (kEdge).
enum Ends { kWhole, kTail, kEdge };

// Where a lane's vector starts in a row, and how many of its first channels are
// another lane's.
template <Ends ENDS>
struct Spot {
    int at;
    static constexpr int lo = 0;
};
template <>
struct Spot<kTail> {
    int at, lo;
};

// Vector v of a row of n channels.
template <int V, Ends ENDS>
__device__ __forceinline__ Spot<ENDS> spot(int v, int n) {
    const int c = V * v;
    if constexpr (ENDS == kTail)
        return c < n && c + V > n ? Spot<kTail>{n - V, c + V - n} : Spot<kTail>{c, 0};
    else
        return {c};
}

// V channels as memory holds them.
template <typename T, int V>
struct RowVec {
    typedef T type __attribute__((ext_vector_type(V), aligned(alignof(T))));
    type t;

    // Channels c .. c + V - 1 of a row (group) of n; zeros past its end.
    __device__ __forceinline__ void load(const T* p, int c, int n) {
        if (c + V <= n) {
            t = *reinterpret_cast<const type*>(p + c);
        } else {
#pragma unroll
            for (int e = 0; e < V; e++) t[e] = c + e < n ? p[c + e] : static_cast<T>(0.0f);
        }
    }
    // STREAM: with the nontemporal hint, for what is not read again here.
    template <bool STREAM>
    __device__ __forceinline__ void store(T* p, int c, int n) const {
        if (c + V <= n) {
            if constexpr (STREAM)
                __builtin_nontemporal_store(t, reinterpret_cast<type*>(p + c));
            else
                *reinterpret_cast<type*>(p + c) = t;
        } else {
#pragma unroll
            for (int e = 0; e < V; e++)
                if (c + e < n) p[c + e] = t[e];
        }
    }
    // The same by spots.  In kTail no lane goes element by element when it
    // reads (2-byte elements would have to arrive before they are packed, and
    // hold up the loads behind them).
    template <Ends ENDS>
    __device__ __forceinline__ void load(const T* p, Spot<ENDS> s, int n) {
        if constexpr (ENDS == kEdge)
            load(p, s.at, n);
        else
            t = *reinterpret_cast<const type*>(p + s.at);
    }
    template <bool STREAM, Ends ENDS>
    __device__ __forceinline__ void store(T* p, Spot<ENDS> s, int n) const {
        if constexpr (ENDS == kEdge) {
            store<STREAM>(p, s.at, n);
        } else if (s.lo == 0) {
            store<STREAM>(p + s.at, 0, V);
        } else {
#pragma unroll
            for (int e = 1; e < V; e++)
                if (e >= s.lo) p[s.at + e] = t[e];
        }
    }
    // Zeroes the channels that are another lane's.
    template <Ends ENDS>
    __device__ __forceinline__ void clear(Spot<ENDS> s) {
#pragma unroll
        for (int e = 0; e < V; e++) t[e] = e >= s.lo ? t[e] : static_cast<T>(0.0f);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < V; e++) t[e] = static_cast<T>(0.0f);
    }
    // Tells the compiler nothing it computed from the vector still holds, so
    // that it keeps the 2-byte values across a round of sums and widens them
    // again afterwards, not their fp32 copies (twice the registers).
    __device__ __forceinline__ void narrow() {
        typedef unsigned int words __attribute__((ext_vector_type(V * sizeof(T) / 4)));
        words u = __builtin_bit_cast(words, t);
        asm volatile("" : "+v"(u));
        t = __builtin_bit_cast(type, u);
    }
    __device__ __forceinline__ float operator[](int e) const { return static_cast<float>(t[e]); }
    __device__ __forceinline__ void set(int e, float v) { t[e] = static_cast<T>(v); }
};

// sigma(v) and 1 - sigma(v), each to a few ulp of itself: the exponential of
// -|v| never overflows and neither result is formed by a subtraction.
// v = +-inf gives exactly 0 and 1.
__device__ __forceinline__ void sigmoid2(float v, float& s, float& c) {
    const float e = ex2(-kLog2e * __builtin_fabsf(v));
    const float big = rcp(1.0f + e);
    const float small = e * big;
    s = v >= 0.0f ? big : small;
    c = v >= 0.0f ? small : big;
}

__device__ __forceinline__ float sigmoid(float v) { return rcp(1.0f + ex2(-kLog2e * v)); }

// SiLU(v) = v sigma(v) and its slope sigma(v) (1 + v (1 - sigma(v))).
__device__ __forceinline__ void silu2(float v, float& f, float& slope) {
    float s, c;
    sigmoid2(v, s, c);
    f = v * s;
    slope = s * __builtin_fmaf(v, c, 1.0f);
}

// 1 - a^2 for a = 2^l2, l2 <= 0: -expm1(q) with q = 2 ln(2) l2, where q > -1/4
// (1 - a^2 would cancel) as q times a polynomial for expm1(q) / q, interpolated
// at the Chebyshev points of [-1/4, 0] (4.8e-9 off at most).
__device__ __forceinline__ float one_minus_square(float l2, float a) {
    const float q = (2.0f * kLn2) * l2;
    float p = __builtin_fmaf(q, 0.007514301221817732f, 0.04149100184440613f);
    p = __builtin_fmaf(q, p, 0.16665112972259521f);
    p = __builtin_fmaf(q, p, 0.4999995231628418f);
    p = __builtin_fmaf(q, p, 1.0f);
    const float near0 = -q * p;
    const float far0 = __builtin_fmaf(-a, a, 1.0f);
    return q > -0.25f ? near0 : far0;
}

}  // namespace mss
