// norm_common.h -- what the add_norm and gated_norm kernels share: rows held
// in registers by a team of lanes, and the team's sums.
//
// A team holds one group of n channels of one row: 16 lanes, a wave, or (TEAM
// = kGroup) a workgroup of as many waves as the row needs.  Lane l keeps the
// NC vectors of V channels that start at V (l + j lanes).  Every input is read
// once, in 16-byte pieces (2-byte types 8 channels, fp32 4) that stay in
// registers as they were read, the moments come from there, and one or two
// rounds of sums per row (RMS: one; LAYER: the mean first, so that the
// variance is that of the centred values) are all the lanes exchange.
// Vectors are read and written with the element's alignment (global memory
// takes unaligned vector accesses), so strided rows and odd widths run the
// same code and give the same bits.  A row's last, partial vector of a 2-byte
// type is read as the V channels up to the row's end, those of the lane before
// it set to 0, and written element by element; read by elements, they would
// hold up the loads behind them until they are packed (gated_norm forward and
// backward, M 16384 bf16: D 2559 265 us, like this 166; D 2560 132).  In fp32,
// with nothing to pack, it is read by elements (add_norm forward and backward,
// M 16384 D 1499: 187 us, the other way 210).  A team walks several rows, reading the next one while
// it works on this one; the per-channel parameters are read once, and the
// backward keeps its sums of the parameter gradients in registers.
#pragma once

#include <atomic>
#include <type_traits>

#include "block_math.h"
#include "launch_block.h"

namespace mss {

constexpr int kGroup = 0;   // TEAM: the workgroup

template <typename T>
constexpr int kVec = sizeof(T) == 4 ? 4 : 8;

// A per-channel parameter, or `otherwise` where it is not given; 0 past the end.
template <int V, Ends ENDS>
__device__ __forceinline__ void load_param(const float* p, Spot<ENDS> s, int n, float otherwise,
                                           float (&v)[V]) {
    RowVec<float, V> t;
    t.zero();
    if (p && s.at < n) t.load(p, s, n);
#pragma unroll
    for (int e = 0; e < V; e++) v[e] = p ? t[e] : s.at + (ENDS == kEdge ? e : 0) < n ? otherwise : 0.0f;
}

// The spots of a lane's vectors, and whether one of the wave's is shared.
template <int V, int NC, Ends ENDS>
struct Spots {
    Spot<ENDS> s[NC];
    bool shared = false;
    __device__ __forceinline__ Spots(int lane, int lanes, int n) {
#pragma unroll
        for (int j = 0; j < NC; j++) s[j] = spot<V, ENDS>(lane + j * lanes, n);
        if constexpr (ENDS == kTail) {
            bool p = false;
#pragma unroll
            for (int j = 0; j < NC; j++) p |= s[j].lo > 0;
            shared = __builtin_amdgcn_ballot_w64(p) != 0;
        }
    }
    // The lane's own channel of the row?
    __device__ __forceinline__ bool own(int j, int e, int n) const {
        return e >= s[j].lo && s[j].at + (ENDS == kEdge ? e : 0) < n;
    }
};

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL,
                                                                  0xf, 0xf, true));
}

__device__ __forceinline__ float read_lane(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

template <int TEAM>
__device__ __forceinline__ int team_lanes() {
    return TEAM == kGroup ? blockDim.x : TEAM;
}
template <int TEAM>
__device__ __forceinline__ int team_lane() {
    return TEAM == kGroup ? threadIdx.x : threadIdx.x % (TEAM ? TEAM : 1);
}

// The team's number in its workgroup, known to be the same for all lanes of a
// wave where it is, so that row addresses stay in scalar registers.
template <int TEAM>
__device__ __forceinline__ int team_of() {
    const int team = TEAM == kGroup ? 0 : threadIdx.x / (TEAM ? TEAM : 1);
    return TEAM == 64 ? __builtin_amdgcn_readfirstlane(team) : team;
}

// LDS floats of team_sum: twice up to three sums of sixteen waves.
constexpr int kSumHalf = 3 * 16;
template <int TEAM>
constexpr int kSumLds = TEAM == kGroup ? 2 * kSumHalf : 1;

// The sum over the team in each of its lanes, K sums at once, always in the
// same order.  The two halves of `lds` take turns from call to call, so that
// a wave that is a round ahead never writes what another still reads, with
// one barrier a round.
template <int TEAM, int K>
__device__ __forceinline__ void team_sum(float (&v)[K], float* lds, int& turn) {
#pragma unroll
    for (int k = 0; k < K; k++) {
        v[k] = dpp_add<0x128>(v[k]);   // rotations inside 16 lanes, by 8, 4, 2, 1
        v[k] = dpp_add<0x124>(v[k]);
        v[k] = dpp_add<0x122>(v[k]);
        v[k] = dpp_add<0x121>(v[k]);
        if constexpr (TEAM != 16)
            v[k] = (read_lane(v[k], 0) + read_lane(v[k], 16)) +
                   (read_lane(v[k], 32) + read_lane(v[k], 48));
    }
    if constexpr (TEAM == kGroup) {
        // one word of each wave (slots without a wave hold 0), summed by
        // every 16 lanes
        static_assert(K * 16 <= kSumHalf, "the halves do not overlap");
        float* at = lds + turn * kSumHalf;
        turn ^= 1;
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int k = 0; k < K; k++) at[k * 16 + threadIdx.x / 64] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; k++) {
            v[k] = at[k * 16 + threadIdx.x % 16];
            v[k] = dpp_add<0x128>(v[k]);
            v[k] = dpp_add<0x124>(v[k]);
            v[k] = dpp_add<0x122>(v[k]);
            v[k] = dpp_add<0x121>(v[k]);
        }
    }
}

// Zeroes the slots of team_sum that no wave writes; the first sum's barrier
// orders it.
template <int TEAM>
__device__ __forceinline__ void clear_sums(float* lds) {
    for (int i = threadIdx.x; i < kSumLds<TEAM>; i += blockDim.x)
        if (i % 16 >= static_cast<int>(blockDim.x) / 64) lds[i] = 0.0f;
}

// The workgroup's share of K sums per channel, in the row of the workspace
// that is its own: acc[k] of its teams added in order through `lds`.  Every
// thread of the workgroup calls it.
template <int TEAM, int NC, int V, int K, Ends ENDS>
__device__ __forceinline__ void write_part(float (&acc)[K][NC][V], float* lds, float* part,
                                           int64_t D, int64_t g0, int n,
                                           const Spots<V, NC, ENDS>& spots) {
#pragma unroll
    for (int k = 0; k < K; k++) {
        float* out = part + k * D + g0;
        if constexpr (TEAM == kGroup) {
#pragma unroll
            for (int j = 0; j < NC; j++) {
                RowVec<float, V> t;
#pragma unroll
                for (int e = 0; e < V; e++) t.set(e, acc[k][j][e]);
                if (spots.s[j].at < n) t.template store<false>(out, spots.s[j], n);
            }
        } else {
            constexpr int slots = TEAM * NC * V, teams = 256 / (TEAM ? TEAM : 1);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NC; j++)
#pragma unroll
                for (int e = 0; e < V; e++)
                    if (e >= spots.s[j].lo)
                        lds[team_of<TEAM>() * slots + spots.s[j].at + e] = acc[k][j][e];
            __syncthreads();
            for (int c = threadIdx.x; c < n; c += 256) {
                float s = 0.0f;
#pragma unroll
                for (int t = 0; t < teams; t++) s += lds[t * slots + c];
                out[c] = s;
            }
        }
    }
}

template <int TEAM, int NC, int V>
constexpr int kPartLds = TEAM == kGroup ? 1 : 256 * NC * V;

template <typename T>
__device__ __forceinline__ T* row_of(const void* p, int64_t row, int64_t ld, int64_t col = 0) {
    return p ? const_cast<T*>(static_cast<const T*>(p)) + row * ld + col : nullptr;
}

// dw, db and dscale from `rows` rows of K sums per channel in the workspace:
//   add_norm    S[0] = sum dy n, S[1] = sum dy, S[2] = sum dresidual x
//   gated_norm  S[0] = sum d n, S[1] = sum d, with d = dout (times the gate
//               where it comes after the norm): dw = k S[0], db = k S[1],
//               dscale = alpha (w S[0] + b S[1]), k = alpha scale
hipError_t launch_norm_params(const NormArgs& a, bool gated, int64_t rows, int K, hipStream_t st);

// ---- sizes -------------------------------------------------------------------

// A launch: the team, how rows end, its workgroup's threads, and the rows that
// a workgroup takes at a time.
template <int TEAM_, int NC_, Ends ENDS_>
struct Shape {
    static constexpr int TEAM = TEAM_, NC = NC_;
    static constexpr Ends ENDS = ENDS_;
    int threads, rows;
};

// Workgroups of `kernel` that a CU holds at once; asked for once per kernel and
// number of waves.
template <typename Kernel>
inline int resident(Kernel* kernel, std::atomic<int> (&known)[17], int threads) {
    std::atomic<int>& at = known[threads / 64];
    int n = at.load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, reinterpret_cast<const void*>(kernel),
                                                         threads, 0) != hipSuccess ||
            n < 1) {
            (void)hipGetLastError();
            return 1;
        }
        at.store(n, std::memory_order_relaxed);
    }
    return n;
}

// Workgroups per group of channels: what 256 CUs hold at once over all groups
// (they walk the rows, so a second, partly filled round only lengthens the
// launch: with 2048 lanes a CU whatever it holds, gated_norm forward and
// backward of M 32768 D 5120 bf16 took a tenth longer), none without a
// row of its own.
template <auto kernel>
inline int64_t row_groups(int64_t M, int64_t G, int threads, int rows, int64_t most = 1 << 20) {
    static std::atomic<int> known[17];
    int64_t p = 256 * static_cast<int64_t>(resident(kernel, known, threads));
    if (p > most) p = most;
    p = (p + G - 1) / G;
    const int64_t all = (M + rows - 1) / rows;
    return p < all ? p : all;
}

// The backward's workgroups each write a row of partial sums: at most 1024,
// and with few rows of input one for every four of them, but four waves for
// each CU (one for every eight, forward and backward, bf16: gated_norm M 1024
// D 5120 32.9 us, like this 25.8; add_norm M 1024 D 2560 23.4 and 20.8).
constexpr int64_t kMostParts = 1024;
inline int64_t most_parts(int64_t M, int threads) {
    int64_t most = 256 * 4 * 64 / threads;
    if (most < M / 4) most = M / 4;
    return most < kMostParts ? most : kMostParts;
}

// f(Shape) for groups of n channels, V to a vector: a quarter of a wave or a
// wave where one vector a lane is enough, else a workgroup with one (two past
// 1024 lanes, up to 1536 vectors).  One vector a lane keeps the backward
// passes at four waves or more on a SIMD (gated_norm's in bf16 takes 90
// registers with one vector and 150 with two, add_norm's 119 and over 168).
// False for wider groups.
template <int V, Ends ENDS, typename F>
bool by_width(int64_t n, F f) {
    const int64_t nv = (n + V - 1) / V;
    if (nv <= 16)
        f(Shape<16, 1, ENDS>{256, 16});
    else if (nv <= 64)
        f(Shape<64, 1, ENDS>{256, 4});
    else if (nv <= 1024)
        f(Shape<kGroup, 1, ENDS>{static_cast<int>((nv + 63) / 64 * 64), 1});
    else if (nv <= 1536)
        f(Shape<kGroup, 2, ENDS>{static_cast<int>((nv + 127) / 128 * 64), 1});
    else
        return false;
    return true;
}
template <typename T, typename F>
bool by_width(int64_t n, F f) {
    constexpr int V = kVec<T>;
    if (n % V == 0) return by_width<V, kWhole>(n, f);
    if constexpr (sizeof(T) == 4) {
        return by_width<V, kEdge>(n, f);
    } else {
        if (n >= V) return by_width<V, kTail>(n, f);
        f(Shape<16, 1, kEdge>{256, 16});
        return true;
    }
}

// Threads of a kernel's largest workgroup.
template <int TEAM, int NC>
constexpr int kMaxThreads = TEAM != kGroup ? 256 : NC == 1 ? 1024 : 768;

}  // namespace mss
