// gated_kernel.hip -- the gated linear recurrence h_t = v_t + a_t h_{t-1} of
// mss.h, its backward pass and its single-token step.
//
// Bound by HBM: per channel and step the forward reads x, r (i, z) and writes
// y, the backward reads those and dout and writes their gradients, and every
// tensor is read once.  One state per channel leaves too few channels to fill
// the chip, so time is cut into chunks that different workgroups hold at the
// same time:
//
//   A lane holds V neighbouring channels (2-byte types two, fp32 one, so that
//   a wave reads 256 bytes of a row) and S consecutive steps of them in
//   registers; the kWaves waves of a workgroup hold consecutive pieces of S
//   steps.  A piece is an affine map of the state that enters it, (A, H):
//   h -> A h + H, and so is a chunk, the pieces' composition.
//   A workgroup publishes its chunk's map as soon as its inputs are in, then
//   waits for the state entering its chunk, and only then steps through its
//   registers a second time, now with the true state, and writes the outputs.
//
// The state entering chunk c is formed from the state entering the group of 8
// (or 32) chunks that c lies in, published by the last chunk of the group
// before, and the maps of the group's chunks before c, in that order: a
// serial chain of one handover per group, and results that do not depend on
// which workgroup runs when.
//
// Workgroups take their chunk from a counter, time first, so a workgroup waits
// only for ones that have taken a lower number, and the lowest number that is
// not done never waits: every wait ends.  (The wait is bounded besides; past
// the bound, seconds, the outputs become NaN.)  What is handed over are
// 8-byte words that are written and read by single relaxed atomics of agent
// scope; all ones means not written yet, so that the words need no flags and
// no fences.  A first small kernel sets them, and the counter, in the
// workspace.
//
// Measured, a call of a row of calls (its other launches included) and the
// kernel's median in a trace: forward B1 L65536 D2560 bf16 decay + gate 319 and
// 328 us (5.3 TB/s), B4 L8192 D5120 fp32 sigmoid + gate 457 and 444 us (6.1
// TB/s), B8 L2048 D1536 bf16 decay 56 and 46 us (VALU busy 67 %); backward of the
// last two 839 and 811 us (5.8 TB/s), 97 and 86 us (VALU busy 86 %, its bound: 89
// instructions per element).  HBM traffic is 1.03 times what the tensors hold.
#include "block_math.h"
#include "launch_block.h"

namespace mss {
namespace {

// k of Gates: log2 of a where sigma(r) = 1.
__device__ __forceinline__ float decay_rate(float scale, float decay) {
    return -kLog2e * (scale * softplus(decay));
}

// The gates of one token and channel: a and v.  The backward works in two
// halves, with `er` and `ei` kept in between in the place of r and i, which
// saves their exponentials the second time.  Keeping 1 - a^2 too spills
// (B8 L2048 D1536 bf16 decay, forward and backward: 154 -> 164 us), keeping a
// for the gradients gains nothing (155).
template <int GATE>
struct Gates {
    float a, v;
    float er, ei;     // DECAY: e^-r, e^-i, at most 2^126 so that their sigmoids stay normal
                      // numbers (what that adds to a closed gate is below 2^-60);
                      // SIGMOID: r itself;  LOG: a
    static constexpr float kMost = 8.507059173023462e37f;   // 2^126

    // k = -log2(e) c softplus(decay) (DECAY);  KEEP: er and ei are used later
    template <bool KEEP>
    __device__ __forceinline__ void set(float x, float r, float i, float k) {
        if constexpr (GATE == MSS_GATE_SIGMOID) {
            float c;
            sigmoid2(r, a, c);
            v = c * x;
            er = r;
        } else if constexpr (GATE == MSS_GATE_DECAY) {
            er = ex2(-kLog2e * r);
            ei = ex2(-kLog2e * i);
            if constexpr (KEEP) {
                // (minimum hands a NaN on, fmin would make it the bound: a closed gate)
                er = __builtin_elementwise_minimum(er, kMost);
                ei = __builtin_elementwise_minimum(ei, kMost);
            }
            const float l2 = k * rcp(1.0f + er);
            a = ex2(l2);
            v = __builtin_amdgcn_sqrtf(one_minus_square(l2, a)) * rcp(1.0f + ei) * x;
        } else {
            a = ex2(kLog2e * r);
            v = x;
            er = a;
        }
    }

    // Gradients for G = dL/dh_t and p = the state carried into the step, from
    // the kept er and ei.  `ws` is w sigma(r), whose sum gives ddecay.
    static __device__ __forceinline__ void grads(float er, float ei, float G, float p, float x,
                                                 float k, float& dx, float& dr, float& di,
                                                 float& ws) {
        if constexpr (GATE == MSS_GATE_SIGMOID) {
            float a, c;
            sigmoid2(er, a, c);
            dx = G * c;
            dr = G * (p - x) * (a * c);
        } else if constexpr (GATE == MSS_GATE_DECAY) {
            const float s = rcp(1.0f + er), c = er * s;   // sigma(r), 1 - sigma(r)
            const float g = rcp(1.0f + ei), gc = ei * g;
            const float l2 = k * s;
            const float a = ex2(l2);
            // m = sqrt(1 - a^2) and 1 / m; where m vanishes, so do sigma(r) or
            // k, and k sigma(r) / m (all that 1 / m enters) is below 2^-60
            // with the bound on 1 / m (a NaN in mm is one in a as well)
            const float mm = one_minus_square(l2, a);
            const float rm = __builtin_amdgcn_rsqf(__builtin_fmaxf(mm, 0x1p-126f));
            const float as = a * s;
            dx = G * (mm * rm * g);
            di = dx * x * gc;
            ws = G * __builtin_fmaf(-x, (g * a) * (as * rm), as * p);
            dr = kLn2 * k * ws * c;
        } else {
            dx = G;
            dr = G * er * p;
        }
    }
};

constexpr int kWaves = 8;                        // waves of a workgroup
// S of the forward.  Half of it leaves room for three workgroups on a CU
// instead of two, and measures slower for the handovers it adds: 480 -> 568 us
// on B4 L8192 D5120 fp32 with a gate, 59 -> 60 us on B8 L2048 D1536 bf16.
constexpr int kSteps = 16;
constexpr int kChunk = kWaves * kSteps;
constexpr int kBwdSteps = 8;                     // S of the backward: twice the inputs per step
constexpr int kBwdChunk = kWaves * kBwdSteps;
static_assert(kChunk % MSS_GATED_CKPT_STEPS == 0, "checkpoints lie between a chunk's waves");
static_assert(kBwdChunk == MSS_GATED_CKPT_STEPS, "a backward chunk starts from a checkpoint");

typedef unsigned long long Word;
constexpr Word kUnset = ~0ull;

// What a launch's workgroups share (chain: chunks > 1).
struct Chain {
    unsigned tiles, ctiles;    // B * ctiles tiles of 64 V channels
    unsigned sets, each;       // 1 or 8 sets of `each` neighbouring tiles
    int64_t chunks, groups;
    unsigned* ticket;          // a counter per set, 8 words apart
    int per;                   // chunks of a group for each wave: a group is kWaves * per
    Word* maps;                // [tile][chunk][V][64]: (A, H)
    Word* states;              // [tile][group][V][64]: the state entering a group
};

// The affine map h -> A h + H.  A = -0, which no product of the factors is (all
// are >= 0), marks a map that drops what was carried whatever it is: rows on the
// other side of a reset may hold anything, NaN among it.  A product that only
// underflows is +0: it leaves a finite state behind, but not a NaN.
constexpr float kDrop = -0.0f;
struct Map {
    float A, H;
    __device__ __forceinline__ bool drops() const {
        return __builtin_bit_cast(unsigned, A) == 0x80000000u;
    }
    __device__ __forceinline__ float operator()(float h) const {
        return drops() ? H : __builtin_fmaf(A, h, H);
    }
    // this after first
    __device__ __forceinline__ Map after(const Map& first) const {
        return {drops() || first.drops() ? kDrop : A * first.A, (*this)(first.H)};
    }
};

__device__ __forceinline__ void put(Word* p, float lo, float hi) {
    Word w = static_cast<Word>(__builtin_bit_cast(unsigned, lo)) |
             static_cast<Word>(__builtin_bit_cast(unsigned, hi)) << 32;
    if (w == kUnset) w = 0x7fc000007fc00000ull;   // two NaNs, but not the mark
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Each lane's V words at p (64 words apart), once all of the wave's are there.
template <int V>
__device__ __forceinline__ void wait_for(Word* p, Map (&m)[V]) {
    Word w[V];
    for (int tries = 0;; tries++) {
        bool unset = false;
#pragma unroll
        for (int v = 0; v < V; v++) {
            w[v] = __hip_atomic_load(p + 64 * v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            unset |= w[v] == kUnset;
        }
        if (!wave_any(unset)) break;
        if (tries > (1 << 22)) {
#pragma unroll
            for (int v = 0; v < V; v++) w[v] = 0x7fc000007fc00000ull;
            break;
        }
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int v = 0; v < V; v++)
        m[v] = {__builtin_bit_cast(float, static_cast<unsigned>(w[v])),
                __builtin_bit_cast(float, static_cast<unsigned>(w[v] >> 32))};
}

// 2 us for 0.2 MB, 6 us for 24 MB.  ws holds n words, an even number: 32 for the
// counters, then the handed over.
__global__ __launch_bounds__(256) void gated_unset_kernel(ulonglong2* ws, int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n / 2;
         i += static_cast<int64_t>(gridDim.x) * 256)
        ws[i] = i < 16 ? make_ulonglong2(0, 0) : make_ulonglong2(kUnset, kUnset);
}

// This workgroup's turn (the chunk, or in the backward its distance from the
// last) and tile.  Workgroup i works for set i % sets, which with eight sets
// puts a set on one XCD, where neighbouring tiles that share cache lines meet in
// one L2.  A set counts its own workgroups, so each waits only for some of its
// set that started before it.
__device__ __forceinline__ unsigned take(const Chain& g, unsigned* lds, unsigned& tile) {
    const unsigned set = blockIdx.x & (g.sets - 1);   // 1 or 8 sets
    unsigned n = g.sets == 1 ? blockIdx.x : blockIdx.x >> 3;
    if (g.chunks > 1) {
        if (threadIdx.x == 0) *lds = atomicAdd(g.ticket + 8 * set, 1u);
        __syncthreads();
        n = *lds;
    }
    n = __builtin_amdgcn_readfirstlane(n);
    const unsigned turn = n / g.each;
    tile = __builtin_amdgcn_readfirstlane(set * g.each + n - turn * g.each);
    return __builtin_amdgcn_readfirstlane(turn);
}

// Waits for the maps of the group's chunks that this wave looks after, those of
// [per wave, per (wave + 1)) that come before the group's `mate`-th, and leaves
// their composition in `mates`.
template <int V>
__device__ __forceinline__ void meet(const Chain& g, Word* first, int wave, int mate, int lane,
                                     Map (*mates)[V][64]) {
    const int from = wave * g.per;
    if (from >= mate) return;
    const int to = from + g.per < mate ? from + g.per : mate;
    Map all[V], e[V];
    wait_for<V>(first + int64_t{from} * (64 * V) + lane, all);
    for (int m = from + 1; m < to; m++) {
        wait_for<V>(first + int64_t{m} * (64 * V) + lane, e);
#pragma unroll
        for (int v = 0; v < V; v++) all[v] = e[v].after(all[v]);
    }
#pragma unroll
    for (int v = 0; v < V; v++) mates[wave][v][lane] = all[v];
}

// Takes h, the state entering the group (or what the adjoint carries into it), to
// the group's `mate`-th chunk, by the waves' compositions.  With growing states
// (GATE_LOG, r > 0) the factor of one of several chunks can overflow although h
// and what becomes of it do not: then by the chunks' own maps, one after another.
template <int GATE, int V>
__device__ __forceinline__ void carry(const Chain& g, Word* first, int mate, int lane,
                                      const Map (*mates)[V][64], float (&h)[V]) {
    float start[V], most = 0.0f;   // most: inf or NaN where a factor is
#pragma unroll
    for (int v = 0; v < V; v++) start[v] = h[v];
    for (int w = 0; w * g.per < mate; w++)
#pragma unroll
        for (int v = 0; v < V; v++) {
            const Map m = mates[w][v][lane];
            h[v] = m(h[v]);
            if constexpr (GATE == MSS_GATE_LOG) most = __builtin_elementwise_maximum(most, m.A);
        }
    if constexpr (GATE == MSS_GATE_LOG) {
        if (g.per == 1 || !wave_any(!(most < __builtin_inff()))) return;
#pragma unroll
        for (int v = 0; v < V; v++) h[v] = start[v];
        for (int m = 0; m < mate; m++) {
            Map e[V];
            wait_for<V>(first + int64_t{m} * (64 * V) + lane, e);
#pragma unroll
            for (int v = 0; v < V; v++) h[v] = e[v](h[v]);
        }
    }
}

// V channels of one row; an odd row's last lane takes the last V channels, so
// its first is its neighbour's too, computed twice to the same bits.
template <typename T, int V>
struct Piece {
    typename std::conditional<V == 1, T, typename RowVec<T, V == 1 ? 2 : V>::type>::type t;
    // `row` is the same for all lanes and `at` the lane's byte offset in it,
    // below 2^31: one register pair and one register of address.
    __device__ __forceinline__ void load(const T* row, unsigned at) {
        t = *reinterpret_cast<const decltype(t)*>(reinterpret_cast<const char*>(row) + at);
    }
    // Outputs carry the nontemporal hint: B4 L8192 D5120 fp32 with a gate,
    // forward 469 -> 441 us, backward 832 -> 813; B8 L2048 D1536 bf16 decay,
    // forward 60 -> 54 us, backward 98 -> 87.
    __device__ __forceinline__ void store(T* row, unsigned at) const {
        __builtin_nontemporal_store(t, reinterpret_cast<decltype(t)*>(reinterpret_cast<char*>(row) + at));
    }
    __device__ __forceinline__ float get(int v) const {
        if constexpr (V == 1)
            return static_cast<float>(t);
        else
            return static_cast<float>(t[v]);
    }
    __device__ __forceinline__ void set(int v, float f) {
        if constexpr (V == 1)
            t = static_cast<T>(f);
        else
            t[v] = static_cast<T>(f);
    }
    // The compiler keeps the value as it was read, not what it made of it.
    __device__ __forceinline__ void keep() {
        typename std::conditional<sizeof(t) == 2, unsigned short, unsigned>::type u;
        __builtin_memcpy(&u, &t, sizeof(t));
        asm volatile("" : "+v"(u));
        __builtin_memcpy(&t, &u, sizeof(t));
    }
};

template <typename T>
__device__ __forceinline__ T* at_row(const void* p, int64_t row, int64_t ld) {
    return const_cast<T*>(static_cast<const T*>(p)) + row * ld;
}

// The offset is widened to 64 bits where it is used, which lets the access
// take the row's address from scalar registers; known from another block it
// would be added up in vector registers for every row.
__device__ __forceinline__ void own_block(unsigned& at) { asm volatile("" : "+v"(at)); }

// A piece's S rows from `row` on, of which n are there (the others read the
// last one again, or the row given when none is).
template <int S, typename T, int V>
__device__ __forceinline__ void load_rows(Piece<T, V> (&p)[S], const void* base, int64_t row, int64_t ld,
                                          int n, unsigned at) {
    const T* from = at_row<T>(base, row, ld);
#pragma unroll
    for (int s = 0; s < S; s++) {
        own_block(at);
        p[s].load(from, at);
        from += s + 1 < n ? ld : 0;
    }
}

// Bit s: step t0 + s (of S) drops what is carried into it.
template <int S>
__device__ __forceinline__ unsigned reset_bits(const uint8_t* reset, int64_t row0, int64_t t0, int64_t L,
                                               int lane) {
    if (!reset) return 0;
    const int64_t t = t0 + lane;
    return static_cast<unsigned>(
        __builtin_amdgcn_ballot_w64(lane < S && t < L && reset[row0 + t] != 0));
}

// Steps past the end of the sequence carry the state as it is.
template <int S, int V>
__device__ __forceinline__ void end_at(float (&a)[S][V], float (&u)[S][V], int n) {
    if (n == S) return;
#pragma unroll
    for (int s = 0; s < S; s++)
#pragma unroll
        for (int v = 0; v < V; v++) {
            a[s][v] = s < n ? a[s][v] : 1.0f;
            u[s][v] = s < n ? u[s][v] : 0.0f;
        }
}

// A piece's map of the state, f, and (REVERSE) of the adjoint, w, in which
// dy(s, v) enters at step s.  With resets (a branch that is the same for all
// lanes and rarely taken) the steps on either side of one are kept apart by
// selection, not by a factor 0.
template <bool REVERSE, int S, int V, typename F>
__device__ __forceinline__ void maps_of(const float (&a)[S][V], const float (&u)[S][V],
                                        unsigned resets, Map (&f)[V], Map (&w)[V], F dy) {
    auto run = [&](auto some) {
        constexpr bool SOME = decltype(some)::value;
#pragma unroll
        for (int v = 0; v < V; v++) {
            f[v] = {1.0f, 0.0f};
            w[v].H = 0.0f;
#pragma unroll
            for (int s = 0; s < S; s++) {
                const bool drop = SOME && (resets >> s & 1);
                f[v].A = f[v].A * a[s][v];
                f[v].H = drop ? u[s][v] : __builtin_fmaf(a[s][v], f[v].H, u[s][v]);
                // nothing from a reset on reaches what is before the piece
                if constexpr (REVERSE)
                    if (!SOME || !(resets & ((2u << s) - 1)))
                        w[v].H = __builtin_fmaf(f[v].A, dy(s, v), w[v].H);
            }
            if (SOME && resets) f[v].A = kDrop;
            w[v].A = f[v].A;
        }
    };
    if (resets)
        run(std::true_type{});
    else
        run(std::false_type{});
}

// The states after each step in the place of the input terms, from the state
// h that enters; h: the last.
template <int S, int V>
__device__ __forceinline__ void states(const float (&a)[S][V], float (&u)[S][V], float (&h)[V],
                                       unsigned resets) {
    if (resets) {
#pragma unroll
        for (int s = 0; s < S; s++)
#pragma unroll
            for (int v = 0; v < V; v++)
                h[v] = u[s][v] = resets >> s & 1 ? u[s][v] : __builtin_fmaf(a[s][v], h[v], u[s][v]);
    } else {
#pragma unroll
        for (int s = 0; s < S; s++)
#pragma unroll
            for (int v = 0; v < V; v++) h[v] = u[s][v] = __builtin_fmaf(a[s][v], h[v], u[s][v]);
    }
}

template <typename T, int V, int GATE, bool Z>
__global__ __launch_bounds__(64 * kWaves) void gated_scan_kernel(GatedArgs q, Chain g) {
    constexpr int S = kSteps;
    __shared__ Map own[kWaves][V][64], mates[kWaves][V][64];
    __shared__ float entering[V][64];
    __shared__ unsigned ticket;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    unsigned tile;
    const int64_t chunk = take(g, &ticket, tile);
    const unsigned b = tile / g.ctiles;
    unsigned c = tile % g.ctiles * (64 * V) + lane * V;
    const bool live = c < q.D;
    c = live && c + V <= q.D ? c : static_cast<unsigned>(q.D - V);
    const int64_t t0 = chunk * kChunk + wave * S, row0 = int64_t{b} * q.L;
    const int n = t0 >= q.L ? 0 : q.L - t0 < S ? static_cast<int>(q.L - t0) : S;

    const int64_t row = row0 + (n > 0 ? t0 : q.L - 1);
    const unsigned at = c * sizeof(T);

    Piece<T, V> x[S], r[S], in[S], z[S];
    load_rows<S>(r, q.r, row, q.ld_r, n, at);
    if constexpr (GATE == MSS_GATE_DECAY) load_rows<S>(in, q.i, row, q.ld_i, n, at);
    load_rows<S>(x, q.x, row, q.ld_x, n, at);
    const unsigned resets = reset_bits<S>(q.reset, row0, t0, q.L, lane);
    float k[V];
#pragma unroll
    for (int v = 0; v < V; v++)
        k[v] = GATE == MSS_GATE_DECAY ? decay_rate(q.gate_scale, q.decay[c + v]) : 0.0f;

    float a[S][V], u[S][V];
    Map m[V];
#pragma unroll
    for (int s = 0; s < S; s++) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            Gates<GATE> e;
            e.template set<false>(x[s].get(v), r[s].get(v), GATE == MSS_GATE_DECAY ? in[s].get(v) : 0.0f, k[v]);
            a[s][v] = e.a;
            u[s][v] = e.v;
        }
    }
    // z is not needed before the wait: read with the rest it makes 64 loads in
    // flight in a wave, one more than can be counted (B1 L65536 D2560 bf16
    // decay: 399 us, here 316)
    if constexpr (Z) load_rows<S>(z, q.z, row, q.ld_z, n, at);
    end_at<S, V>(a, u, n);
    {
        Map none[V];
        maps_of<false, S, V>(a, u, resets, m, none, 0);
    }
#pragma unroll
    for (int v = 0; v < V; v++) own[wave][v][lane] = m[v];
    __syncthreads();

    float h[V];
    const int group = kWaves * g.per, mate = static_cast<int>(chunk % group);
    if (g.chunks > 1) {
        const int64_t first = chunk - mate, words = 64 * V;
        if (wave == 0 && mate != group - 1 && chunk + 1 < g.chunks) {
#pragma unroll
            for (int v = 0; v < V; v++) {
                Map all = own[0][v][lane];
#pragma unroll
                for (int w = 1; w < kWaves; w++) all = own[w][v][lane].after(all);
                put(g.maps + (int64_t{tile} * g.chunks + chunk) * words + 64 * v + lane, all.A, all.H);
            }
        }
        Word* maps = g.maps + (int64_t{tile} * g.chunks + first) * words;
        meet<V>(g, maps, wave, mate, lane, mates);
        if (wave == kWaves - 1) {
            Map e[V];
            if (first > 0)
                wait_for<V>(g.states + (int64_t{tile} * g.groups + first / group) * words + lane, e);
            else
#pragma unroll
                for (int v = 0; v < V; v++) e[v].H = q.h0 ? q.h0[int64_t{b} * q.D + c + v] : 0.0f;
#pragma unroll
            for (int v = 0; v < V; v++) entering[v][lane] = e[v].H;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; v++) h[v] = entering[v][lane];
        carry<GATE, V>(g, maps, mate, lane, mates, h);
    } else {
#pragma unroll
        for (int v = 0; v < V; v++) h[v] = q.h0 ? q.h0[int64_t{b} * q.D + c + v] : 0.0f;
    }
    for (int w = 0; w < wave; w++)
#pragma unroll
        for (int v = 0; v < V; v++) h[v] = own[w][v][lane](h[v]);
    if (wave == kWaves - 1 && mate == group - 1 && chunk + 1 < g.chunks) {
#pragma unroll
        for (int v = 0; v < V; v++)
            put(g.states + (int64_t{tile} * g.groups + chunk / group + 1) * (64 * V) + 64 * v + lane, 0.0f,
                m[v](h[v]));
    }
    if (q.h_ckpt && t0 % MSS_GATED_CKPT_STEPS == 0 && n > 0 && live) {
        const int64_t per = (q.L + MSS_GATED_CKPT_STEPS - 1) / MSS_GATED_CKPT_STEPS;
        float* out = q.h_ckpt + (int64_t{b} * per + t0 / MSS_GATED_CKPT_STEPS) * q.D;
#pragma unroll
        for (int v = 0; v < V; v++) out[c + v] = h[v];
    }
    states<S, V>(a, u, h, resets);
    T* y_row = at_row<T>(q.y, row, q.ld_y);
#pragma unroll
    for (int s = 0; s < S; s++, y_row += q.ld_y) {
        if (s >= n) continue;
        Piece<T, V> y;
#pragma unroll
        for (int v = 0; v < V; v++) {
            if constexpr (Z)
                y.set(v, u[s][v] * silu(z[s].get(v)));
            else
                y.set(v, u[s][v]);
        }
        if (live) {
            unsigned to = at;
            own_block(to);
            y.store(y_row, to);
        }
    }
    if (q.h_last && n > 0 && t0 + n == q.L && live) {
#pragma unroll
        for (int v = 0; v < V; v++) q.h_last[int64_t{b} * q.D + c + v] = h[v];
    }
}

// The adjoint runs through the chunks from the last to the first: a piece maps
// what the steps after it pass to its last state, Q, to A Q + R, with the same
// A as the forward's map.  The states inside a chunk come from its checkpoint
// and the pieces' forward maps.
template <typename T, int V, int GATE, bool Z>
__global__ __launch_bounds__(64 * kWaves, 4) void gated_scan_bwd_kernel(GatedArgs q, Chain g,
                                                                     float* part) {
    constexpr int S = kBwdSteps;
    __shared__ Map fwd[kWaves][V][64], rev[kWaves][V][64], mates[kWaves][V][64];
    __shared__ float entering[V][64];
    __shared__ unsigned ticket;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int waves = blockDim.x / 64;   // kWaves, or fewer where they hold all steps
    unsigned tile;
    const int64_t turn = take(g, &ticket, tile);   // 0: the last chunk
    const int64_t chunk = g.chunks - 1 - turn;
    const unsigned b = tile / g.ctiles;
    unsigned c = tile % g.ctiles * (64 * V) + lane * V;
    const bool live = c < q.D;
    c = live && c + V <= q.D ? c : static_cast<unsigned>(q.D - V);
    const int64_t t0 = chunk * kBwdChunk + wave * S, row0 = int64_t{b} * q.L;
    const int n = t0 >= q.L ? 0 : q.L - t0 < S ? static_cast<int>(q.L - t0) : S;

    const int64_t row = row0 + (n > 0 ? t0 : q.L - 1);
    const unsigned at = c * sizeof(T);

    Piece<T, V> x[S], r[S], in[S], z[S], dout[S];
    load_rows<S>(r, q.r, row, q.ld_r, n, at);
    if constexpr (GATE == MSS_GATE_DECAY) load_rows<S>(in, q.i, row, q.ld_i, n, at);
    load_rows<S>(x, q.x, row, q.ld_x, n, at);
    if constexpr (Z) load_rows<S>(z, q.z, row, q.ld_z, n, at);
    load_rows<S>(dout, q.dout, row, q.ld_y, n, at);
    const unsigned resets = reset_bits<S>(q.reset, row0, t0, q.L, lane);
    float k[V], h[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        k[v] = GATE == MSS_GATE_DECAY ? decay_rate(q.gate_scale, q.decay[c + v]) : 0.0f;
        h[v] = q.h_ckpt[(int64_t{b} * g.chunks + chunk) * q.D + c + v];
    }

    float a[S][V], u[S][V];     // u: the input term, later the state
    float er[S][V], ei[S][V];   // what the gradients take of r and i
    Map f[V], w[V];
#pragma unroll
    for (int s = 0; s < S; s++) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            Gates<GATE> e;
            e.template set<true>(x[s].get(v), r[s].get(v), GATE == MSS_GATE_DECAY ? in[s].get(v) : 0.0f, k[v]);
            a[s][v] = e.a;
            u[s][v] = e.v;
            er[s][v] = e.er;
            if constexpr (GATE == MSS_GATE_DECAY) ei[s][v] = e.ei;
        }
    }
    end_at<S, V>(a, u, n);
    if (n < S) {
#pragma unroll
        for (int s = 0; s < S; s++)
#pragma unroll
            for (int v = 0; v < V; v++)
                if (s >= n) dout[s].set(v, 0.0f);
    }
    maps_of<true, S, V>(a, u, resets, f, w, [&](int s, int v) {
        const float dy = dout[s].get(v);
        if constexpr (Z)
            return dy * silu(z[s].get(v));
        else
            return dy;
    });
#pragma unroll
    for (int v = 0; v < V; v++) {
        fwd[wave][v][lane] = f[v];
        rev[wave][v][lane] = w[v];
    }
    __syncthreads();

    float Q[V];
    const int group = kWaves * g.per, mate = static_cast<int>(turn % group);
    const int64_t first = turn - mate, words = 64 * V;
    if (wave == 0 && mate != group - 1 && turn + 1 < g.chunks) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            Map all = rev[kWaves - 1][v][lane];
#pragma unroll
            for (int p = kWaves - 2; p >= 0; p--) all = rev[p][v][lane].after(all);
            put(g.maps + (int64_t{tile} * g.chunks + turn) * words + 64 * v + lane, all.A, all.H);
        }
    }
    Word* maps = g.maps + (int64_t{tile} * g.chunks + first) * words;
    meet<V>(g, maps, wave, mate, lane, mates);
    if (wave == waves - 1) {
        Map e[V];
        if (first > 0)
            wait_for<V>(g.states + (int64_t{tile} * g.groups + first / group) * words + lane, e);
        else
#pragma unroll
            for (int v = 0; v < V; v++) e[v].H = q.dh_last ? q.dh_last[int64_t{b} * q.D + c + v] : 0.0f;
#pragma unroll
        for (int v = 0; v < V; v++) entering[v][lane] = e[v].H;
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; v++) Q[v] = entering[v][lane];
    carry<GATE, V>(g, maps, mate, lane, mates, Q);
    for (int p = waves - 1; p > wave; p--)
#pragma unroll
        for (int v = 0; v < V; v++) Q[v] = rev[p][v][lane](Q[v]);
    if (wave == 0 && mate == group - 1 && turn + 1 < g.chunks) {
#pragma unroll
        for (int v = 0; v < V; v++)
            put(g.states + (int64_t{tile} * g.groups + turn / group + 1) * words + 64 * v + lane, 0.0f,
                w[v](Q[v]));
    }
    for (int p = 0; p < wave; p++)
#pragma unroll
        for (int v = 0; v < V; v++) h[v] = fwd[p][v][lane](h[v]);

    float before[V];   // the state entering the piece
#pragma unroll
    for (int v = 0; v < V; v++) before[v] = h[v];
#pragma unroll
    for (int s = 0; s < S; s++) {
        x[s].keep();
        dout[s].keep();
        if constexpr (Z) z[s].keep();
#pragma unroll
        for (int v = 0; v < V; v++) {
            // nothing but these is kept of the gates
            asm volatile("" : "+v"(er[s][v]));
            if constexpr (GATE == MSS_GATE_DECAY) asm volatile("" : "+v"(ei[s][v]));
        }
    }
    states<S, V>(a, u, h, resets);
    float sum[V];
#pragma unroll
    for (int v = 0; v < V; v++) sum[v] = 0.0f;
    T* dx_row = at_row<T>(q.dx, row + n, q.ld_dx);
    T* dr_row = at_row<T>(q.dr, row + n, q.ld_dr);
    T* di_row = at_row<T>(q.di, row + n, q.ld_di);
    T* dz_row = at_row<T>(q.dz, row + n, q.ld_dz);
#pragma unroll
    for (int s = S - 1; s >= 0; s--) {
        if (s >= n) continue;
        dx_row -= q.ld_dx;
        dr_row -= q.ld_dr;
        di_row -= q.ld_di;
        dz_row -= q.ld_dz;
        Piece<T, V> dx, dr, di, dz;
        const bool drop = resets >> s & 1;
#pragma unroll
        for (int v = 0; v < V; v++) {
            const float xv = x[s].get(v);
            const float p = drop ? 0.0f : s > 0 ? u[s > 0 ? s - 1 : 0][v] : before[v];
            float dy = dout[s].get(v);
            if constexpr (Z) {
                float gate, slope;
                silu2(z[s].get(v), gate, slope);
                dz.set(v, dy * u[s][v] * slope);
                dy *= gate;
            }
            const float G = dy + Q[v];
            float gx, gr, gi = 0.0f, ws = 0.0f;
            Gates<GATE>::grads(er[s][v], GATE == MSS_GATE_DECAY ? ei[s][v] : 0.0f, G, p, xv, k[v], gx,
                               gr, gi, ws);
            Q[v] = drop ? 0.0f : a[s][v] * G;
            sum[v] += ws;
            dx.set(v, gx);
            dr.set(v, gr);
            di.set(v, gi);
        }
        if (live) {
            unsigned to = at;
            own_block(to);
            dx.store(dx_row, to);
            dr.store(dr_row, to);
            if constexpr (GATE == MSS_GATE_DECAY) di.store(di_row, to);
            if constexpr (Z) dz.store(dz_row, to);
        }
    }
    if (q.dh0 && t0 == 0 && live) {
#pragma unroll
        for (int v = 0; v < V; v++) q.dh0[int64_t{b} * q.D + c + v] = Q[v];
    }
    if constexpr (GATE == MSS_GATE_DECAY) {
        // the chunk's share of sum w sigma(r), its waves in order
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; v++) fwd[wave][v][lane].A = sum[v];
        __syncthreads();
        if (wave == 0 && live) {
#pragma unroll
            for (int v = 0; v < V; v++) {
                float all = 0.0f;
                for (int p = 0; p < waves; p++) all += fwd[p][v][lane].A;
                part[(int64_t{b} * g.chunks + chunk) * q.D + c + v] = all;
            }
        }
    }
}

// ddecay[d] = -c sigma(decay[d]) sum over the partial rows: 32 channels a
// workgroup, 32 rows at a time, in a fixed order.  Latency: 4.8 us for 256
// rows of D 1536.
__global__ __launch_bounds__(1024) void gated_ddecay_kernel(const float* __restrict__ part,
                                                            const float* __restrict__ decay,
                                                            float* __restrict__ ddecay,
                                                            int64_t rows, int64_t D, float scale) {
    __shared__ float lds[32][33];
    const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float sum = 0.0f;
    if (d < D) {
#pragma unroll 8
        for (int64_t p = group; p < rows; p += 32) sum += part[p * D + d];
    }
    lds[group][lane] = sum;
    __syncthreads();
    if (group != 0 || d >= D) return;
    sum = 0.0f;
#pragma unroll
    for (int p = 0; p < 32; p++) sum += lds[p][lane];
    ddecay[d] = -scale * sigmoid(decay[d]) * sum;
}

// One token: lanes side by side over (sequence, vector of 4 channels), every
// access 8 or 16 bytes.  B4 D1536 bf16 3.3 us (a launch's latency), B256 D5120
// fp32 4.8 us (31 MB from the last-level cache).
constexpr int kStepVec = 4;
template <typename T, int GATE>
__global__ __launch_bounds__(64) void gated_step_kernel(GatedArgs q, unsigned per) {
    constexpr int V = kStepVec;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    const int64_t b = j / per;
    if (b >= q.B) return;
    const int c = V * static_cast<int>(j - b * per), n = static_cast<int>(q.D);
    RowVec<T, V> x, r, in, z, y;
    RowVec<float, V> h, decay;
    x.load(at_row<T>(q.x, b, q.ld_x), c, n);
    r.load(at_row<T>(q.r, b, q.ld_r), c, n);
    h.load(q.h + b * q.D, c, n);
    if constexpr (GATE == MSS_GATE_DECAY) {
        in.load(at_row<T>(q.i, b, q.ld_i), c, n);
        decay.load(q.decay, c, n);
    }
    if (q.z) z.load(at_row<T>(q.z, b, q.ld_z), c, n);
#pragma unroll
    for (int v = 0; v < V; v++) {
        Gates<GATE> e;
        const float k = GATE == MSS_GATE_DECAY ? decay_rate(q.gate_scale, decay[v]) : 0.0f;
        e.template set<false>(x[v], r[v], GATE == MSS_GATE_DECAY ? in[v] : 0.0f, k);
        h.set(v, __builtin_fmaf(e.a, h[v], e.v));
        y.set(v, q.z ? h[v] * silu(z[v]) : h[v]);
    }
    h.template store<true>(q.h + b * q.D, c, n);
    y.template store<true>(at_row<T>(q.y, b, q.ld_y), c, n);
}

template <typename T, int V, typename F>
hipError_t by_gate(int gate, F f) {
    constexpr std::integral_constant<int, V> v{};
    switch (gate) {
        case MSS_GATE_SIGMOID: return f(T{}, v, std::integral_constant<int, MSS_GATE_SIGMOID>{});
        case MSS_GATE_DECAY: return f(T{}, v, std::integral_constant<int, MSS_GATE_DECAY>{});
        case MSS_GATE_LOG: return f(T{}, v, std::integral_constant<int, MSS_GATE_LOG>{});
        default: return hipErrorInvalidValue;
    }
}

// f(element, channels per lane, gate) for the call's types; f returns what its
// launches reported (hipGetLastError() clears an error, so each is asked for
// once).  A single channel is no pair.
template <typename F>
hipError_t dispatch(const GatedArgs& a, F f) {
    switch (a.dtype) {
        case MSS_F32: return by_gate<float, 1>(a.gate, f);
        case MSS_BF16: return a.D > 1 ? by_gate<bf16, 2>(a.gate, f) : by_gate<bf16, 1>(a.gate, f);
        case MSS_F16: return a.D > 1 ? by_gate<f16, 2>(a.gate, f) : by_gate<f16, 1>(a.gate, f);
        default: return hipErrorInvalidValue;
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Threads of a workgroup: eight waves, or as many as a single chunk has pieces.
unsigned threads_of(int64_t L, int64_t steps) {
    const int64_t waves = cdiv(L, steps);
    return static_cast<unsigned>(64 * (waves < kWaves ? waves : kWaves));
}

// A launch's threads are counted in 32 bits.
constexpr int64_t kMaxThreads = int64_t{UINT32_MAX};

// Words handed over for chunks of `len` steps, over tiles of whole pairs of
// waves' channels (what either V needs).
int64_t chain_words(int64_t B, int64_t L, int64_t D, int64_t len) {
    const int64_t chunks = cdiv(L, len);
    return chunks <= 1 ? 0 : B * cdiv(D, 128) * 128 * (chunks + cdiv(chunks, kWaves));
}

bool chain_bytes(int64_t B, int64_t L, int64_t D, int64_t len, int64_t& bytes) {
    // a workgroup per chunk and tile; the word counts stay far below 2^63
    // (8 bytes for every `len` steps of a channel whose elements were counted)
    // byte offsets in a row stay below 2^31
    if (D > MSS_MAX_WIDTH || cdiv(L, len) > kMaxThreads / (64 * kWaves) / (B * cdiv(D, 64))) return false;
    const int64_t words = chain_words(B, L, D, len);
    bytes = words == 0 ? 0 : align256(256 + 8 * words);
    return true;
}

Chain chain_of(const GatedArgs& a, int V, int64_t len) {
    Chain g;
    g.ctiles = static_cast<unsigned>(cdiv(a.D, 64 * V));
    g.tiles = static_cast<unsigned>(a.B * g.ctiles);
    // Sets of tiles that stay on an XCD let neighbouring tiles meet in one L2,
    // where they share lines if rows start inside one (a stride that is no
    // multiple of 128 bytes), but move the XCDs' places in the tensors apart,
    // which costs once a tensor is as large as the last-level cache.  Forward and
    // backward in us, without / with sets (sigmoid gate but where said), for
    // strides that end inside a line: fp32 B4 D5119 277 / 244 (126 MB a tensor)
    // and 1293 / 1178 (598 MB), B8 D511 1391 / 1207 (600 MB), bf16 B8 D2047 279 /
    // 256 (130 MB) and 1389 / 1228 (599 MB); for whole lines: fp32 B8 L1920 D2048
    // 200 / 183, B8 L12160 D512 303 / 302 (199 MB), B8 L16384 D512 390 / 408 (268
    // MB), B4 L8192 D5120 935 / 967 (671 MB), B8 L4096 D4096 768 / 833 (537 MB);
    // bf16 B8 D1536 decay L2048 147 / 141 and L8128 488 / 489 (200 MB), L16384 623
    // / 651 (403 MB).  (Beyond 200 MB some gain: fp32 B8 L9152 D2048 903 / 863.)
    // A tensor that only begins inside a line, or one of several with such a
    // stride, is within 3 % either way.  Only equal sets, so that the XCDs end
    // together, of eight tiles or more.
    const int64_t elem = a.dtype == MSS_F32 ? 4 : 2;
    const bool off_line = (a.ld_x | a.ld_r | a.ld_y) * elem % 128 != 0;
    const bool small = a.B * a.L * a.D * elem <= int64_t{200} << 20;
    g.sets = g.tiles % 8 == 0 && g.tiles >= 64 && (off_line || small) ? 8 : 1;
    g.each = g.tiles / g.sets;
    g.chunks = cdiv(a.L, len);
    // With few tiles the handovers between groups are what takes the time, and
    // groups of 32 chunks have a quarter of them; with many, the words that a
    // chunk then reads cost more.  Forward and backward in bf16, groups of 8 /
    // of 32: 2 tiles L12294 72.8 / 39.8 us, 8 tiles L65536 408 / 390, 12 tiles
    // L4096 67.9 / 65.8, 16 tiles L8192 75.4 / 80.2, 20 tiles L16384 251 / 260.
    g.per = g.tiles <= 12 ? 4 : 1;
    g.groups = cdiv(g.chunks, kWaves * g.per);
    g.ticket = static_cast<unsigned*>(a.ws);
    g.maps = static_cast<Word*>(a.ws) + 32;
    g.states = g.maps + int64_t{g.tiles} * g.chunks * 64 * V;
    return g;
}

// Marks the words of a chain as not written and zeroes its counters.
hipError_t unset(const Chain& g, int V, hipStream_t st) {
    if (g.chunks == 1) return hipSuccess;
    const int64_t n = 32 + g.tiles * (g.chunks + g.groups) * 64 * V;
    const int64_t blocks = cdiv(n, 512);
    gated_unset_kernel<<<static_cast<unsigned>(blocks < 8192 ? blocks : 8192), 256, 0, st>>>(
        static_cast<ulonglong2*>(static_cast<void*>(g.ticket)), n);
    return hipGetLastError();
}

}  // namespace

bool gated_step_fits(int64_t B, int64_t D) {
    return D <= MSS_MAX_WIDTH && (B == 0 || cdiv(D, kStepVec) <= (kMaxThreads - 63) / B);
}

bool gated_scan_workspace(int64_t B, int64_t L, int64_t D, int64_t& bytes) {
    return chain_bytes(B, L, D, kChunk, bytes);
}

bool gated_scan_bwd_workspace(int64_t B, int64_t L, int64_t D, int gate, int64_t& bytes) {
    if (!chain_bytes(B, L, D, kBwdChunk, bytes)) return false;
    if (gate == MSS_GATE_DECAY) bytes += align256(B * cdiv(L, kBwdChunk) * D * 4);
    return true;
}

hipError_t launch_gated_scan(const GatedArgs& a, hipStream_t st) {
    return dispatch(a, [&](auto t, auto v, auto gate) {
        using T = decltype(t);
        const Chain g = chain_of(a, v.value, kChunk);
        if (const hipError_t e = unset(g, v.value, st); e != hipSuccess) return e;
        const unsigned grid = g.tiles * static_cast<unsigned>(g.chunks);
        const unsigned threads = threads_of(a.L, kSteps);
        if (a.z)
            gated_scan_kernel<T, v.value, gate.value, true><<<grid, threads, 0, st>>>(a, g);
        else
            gated_scan_kernel<T, v.value, gate.value, false><<<grid, threads, 0, st>>>(a, g);
        return hipGetLastError();
    });
}

hipError_t launch_gated_scan_bwd(const GatedArgs& a, hipStream_t st) {
    const int64_t rows = a.B * cdiv(a.L, kBwdChunk);
    int64_t bytes = 0;
    chain_bytes(a.B, a.L, a.D, kBwdChunk, bytes);
    float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + bytes);
    const hipError_t e = dispatch(a, [&](auto t, auto v, auto gate) {
        using T = decltype(t);
        const Chain g = chain_of(a, v.value, kBwdChunk);
        if (const hipError_t e = unset(g, v.value, st); e != hipSuccess) return e;
        const unsigned grid = g.tiles * static_cast<unsigned>(g.chunks);
        const unsigned threads = threads_of(a.L, kBwdSteps);
        if (a.z)
            gated_scan_bwd_kernel<T, v.value, gate.value, true><<<grid, threads, 0, st>>>(a, g, part);
        else
            gated_scan_bwd_kernel<T, v.value, gate.value, false><<<grid, threads, 0, st>>>(a, g, part);
        return hipGetLastError();
    });
    if (e != hipSuccess || a.gate != MSS_GATE_DECAY) return e;
    gated_ddecay_kernel<<<static_cast<unsigned>(cdiv(a.D, 32)), 1024, 0, st>>>(
        part, a.decay, a.ddecay, rows, a.D, a.gate_scale);
    return hipGetLastError();
}

hipError_t launch_gated_step(const GatedArgs& a, hipStream_t st) {
    return dispatch(a, [&](auto t, auto, auto gate) {
        const int64_t per = cdiv(a.D, kStepVec);
        gated_step_kernel<decltype(t), gate.value>
            <<<static_cast<unsigned>(cdiv(a.B * per, 64)), 64, 0, st>>>(a, static_cast<unsigned>(per));
        return hipGetLastError();
    });
}

}  // namespace mss
