// embed_kernel.hip -- rows of a table by token id, and the table's gradient.
//
// Forward: y_m = scale W[id_m].  A wave copies a row, 16 bytes of the wider type
// to a lane, four of them in flight.  HBM: M32768 V65536 D2560 bf16 to fp32 63 us, 6.2
// TB/s (y stored through the caches: 98 us).
//
// Backward: dW_v = scale sum over the m with id_m = v of dy_m.  No sum goes
// through float atomics, so its order is fixed:
//   1. The positions m are sorted by id, stably, by a radix sort of up to ten
//      bits a pass (ids that mark a padded place sort as V, to the end).
//   2. The sorted positions are cut into runs of kRun.  A workgroup sums a
//      run's rows of dy in that order, for a slice of the columns, and writes
//      every token's sum that begins and ends within it.  What reaches over
//      its ends goes to two rows of partial sums.
//   3. The workgroup in whose run a token begins that goes on beyond it adds
//      up the partial sums.
// The work is cut by position, so a token that makes up much of the batch costs
// no more than any others.  Rows of tokens that do not occur are zeroed by
// further workgroups of step 2, which look each row up in the sorted ids.
// M32768 V65536 D2560, fp32 to bf16, a Zipf distribution: 183 us, of which 135 are step
// 2 (671 MB, 5.0 TB/s), 19 the join and 32 the sort, whose launches wait for memory and
// for each other; M16384 V32768 D1536 added to the head's: 50 us (19, 7 and 23).
#include <type_traits>

#include "block_math.h"
#include "launch_ends.h"

namespace mss {
namespace {

constexpr int kSortThreads = 256;
constexpr int kMostTiles = 64;
constexpr int kMaxBits = 10;
constexpr int kMaxBins = 1 << kMaxBits;
constexpr bool kStream = true;            // y and dW pass the caches by
constexpr int kSumThreads = 512;
constexpr int kRun = 16;
constexpr int kZeroRows = 16;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The sort key of an id: the id, or V where it marks a padded place.
__device__ __forceinline__ uint32_t key_of(const void* ids, bool wide, int64_t m, int64_t V) {
    const int64_t id = wide ? static_cast<const int64_t*>(ids)[m] : static_cast<const int32_t*>(ids)[m];
    return static_cast<uint32_t>(id >= 0 && id < V ? id : V);
}

// ---- forward -----------------------------------------------------------------

// Values to a lane: 16 bytes of the wider type, so that its lines are read or
// written whole by one instruction.
template <typename TW, typename TY>
constexpr int kVec = sizeof(TW) == 4 || sizeof(TY) == 4 ? 4 : 8;

template <typename TW, typename TY>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a) {
    constexpr int V = kVec<TW, TY>;
    const int64_t m = blockIdx.x * int64_t{4} + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (m >= a.M) return;
    const uint32_t key = key_of(a.ids, a.wide_ids, m, a.V);
    const int n = static_cast<int>(a.D);
    TY* y = static_cast<TY*>(a.y) + m * a.ld_y;
    const bool in = key < static_cast<uint64_t>(a.V);
    const TW* w = static_cast<const TW*>(a.w) + (in ? key * a.ld_w : 0);
    constexpr int kAhead = 4;
    for (int c0 = (threadIdx.x % kWave) * V; c0 < n; c0 += kAhead * kWave * V) {
        RowVec<TW, V> r[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int c = c0 + i * kWave * V;
            if (in && c < n) r[i].load(w, c, n);
            else r[i].zero();
        }
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int c = c0 + i * kWave * V;
            RowVec<TY, V> o;
#pragma unroll
            for (int e = 0; e < V; e++) o.set(e, in ? a.scale * r[i][e] : 0.0f);
            if (c < n) o.template store<kStream>(y, c, n);
        }
    }
}

// ---- the sort ------------------------------------------------------------------
// A pass over one digit: every workgroup takes a tile of the positions, of the
// same size, and counts[tile][digit] says how many of the tile's keys have the
// digit.  The counts of the first pass are made by a launch of their own; a pass
// counts for the next one as it places its keys.  A workgroup works out where its
// keys go from the counts of all tiles (at most kMostTiles), so that no launch
// between only adds them up.

struct SortArgs {
    const void* ids;          // first pass
    bool wide;
    int64_t M, V;
    const uint32_t* key_in;   // later passes
    const uint32_t* pos_in;
    uint32_t* key_out;
    uint32_t* pos_out;
    uint32_t* counts;         // [tiles][1 << bits]
    uint32_t* next;           // of the next pass (right behind); null in the last
    int later;                // passes behind the first, whose counts sort_count_kernel zeroes
    int64_t tiles;
    int tile;                 // positions, a multiple of kSortThreads
    int shift, bits;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int64_t m) {
    return a.ids ? key_of(a.ids, a.wide, m, a.V) : a.key_in[m];
}

// The lanes of a wave whose keys have the same digit.
struct Peers {
    uint64_t same, below;     // of them, those in lower lanes
    uint32_t digit;
    bool in;
    __device__ __forceinline__ Peers(uint32_t digit_, bool in_, int bits, int lane)
        : same(__builtin_amdgcn_ballot_w64(in_)), digit(digit_), in(in_) {
        for (int b = 0; b < bits; b++) {
            const uint64_t ones = __builtin_amdgcn_ballot_w64(digit >> b & 1);
            same &= digit >> b & 1 ? ones : ~ones;
        }
        below = same & ((uint64_t{1} << lane) - 1);
    }
    // The key's place: next[digit] says where the digit's next key goes, and moves on by the wave's.
    // (The lanes of a digit have all read it before the first of them writes: one instruction
    // after the other for the whole wave.)
    __device__ __forceinline__ uint32_t place(volatile uint32_t* next) const {
        const uint32_t first = next[digit];
        __builtin_amdgcn_wave_barrier();
        if (below == 0) next[digit] = first + __builtin_popcountll(same);
        __builtin_amdgcn_wave_barrier();
        return first + __builtin_popcountll(below);
    }
};

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
    __shared__ uint32_t bins[kMaxBins];
    const int n = 1 << a.bits;
    for (int b = threadIdx.x; b < n; b += kSortThreads) {
        bins[b] = 0;
        for (int p = 0; p < a.later; p++) a.next[(p * a.tiles + blockIdx.x) * n + b] = 0;
    }
    __syncthreads();
    const int64_t m0 = blockIdx.x * int64_t{a.tile}, end = m0 + a.tile < a.M ? m0 + a.tile : a.M;
    for (int64_t m = m0 + threadIdx.x; m < end; m += kSortThreads)
        atomicAdd(&bins[sort_key(a, m) >> a.shift & (n - 1)], 1u);
    __syncthreads();
    for (int b = threadIdx.x; b < n; b += kSortThreads) a.counts[blockIdx.x * n + b] = bins[b];
}

// Each wave takes a quarter of the tile in a row; a key's place is that of its
// digit, plus the keys of that digit in earlier tiles, in the tile's earlier
// waves, in the wave's earlier rounds and in the lanes before it.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
    constexpr int kWaves = kSortThreads / kWave, kEach = kMaxBins / kSortThreads, kTogether = 16;
    __shared__ uint32_t at[kWaves][kMaxBins];
    __shared__ uint32_t sums[kWaves];
    const int n = 1 << a.bits, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (int b = threadIdx.x; b < kWaves * n; b += kSortThreads) at[b / n][b % n] = 0;
    __syncthreads();
    const int quarter = a.tile / kWaves;
    const int64_t m0 = blockIdx.x * int64_t{a.tile} + wave * quarter;
    const int64_t end = m0 + quarter < a.M ? m0 + quarter : a.M;
    for (int64_t m = m0 + lane; m < end; m += kWave) atomicAdd(&at[wave][sort_key(a, m) >> a.shift & (n - 1)], 1u);
    // digits kEach t .. of thread t: all tiles' keys, and those of the tiles before
    uint32_t all[kEach] = {}, before[kEach] = {}, sum = 0;
    const int each = n > kSortThreads ? n / kSortThreads : 1, d0 = threadIdx.x * each;
    if (d0 < n) {
        for (int64_t t0 = 0; t0 < a.tiles; t0 += kTogether) {
            uint32_t c[kTogether][kEach];
#pragma unroll
            for (int k = 0; k < kTogether; k++)
#pragma unroll
                for (int i = 0; i < kEach; i++)
                    c[k][i] = t0 + k < a.tiles && i < each ? a.counts[(t0 + k) * n + d0 + i] : 0;
#pragma unroll
            for (int k = 0; k < kTogether; k++)
#pragma unroll
                for (int i = 0; i < kEach; i++) {
                    all[i] += c[k][i];
                    before[i] += t0 + k < blockIdx.x ? c[k][i] : 0;
                }
        }
#pragma unroll
        for (int i = 0; i < kEach; i++) sum += all[i];
    }
    uint32_t upto = sum;                          // of the digits of this and the lower lanes
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t below = __shfl_up(upto, d);
        if (lane >= d) upto += below;
    }
    if (lane == kWave - 1) sums[wave] = upto;
    __syncthreads();
    uint32_t first = upto - sum;
    for (int w = 0; w < wave; w++) first += sums[w];
    if (d0 < n)
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            if (i >= each) break;
            uint32_t to = first + before[i];
            for (int w = 0; w < kWaves; w++) {
                const uint32_t c = at[w][d0 + i];
                at[w][d0 + i] = to;
                to += c;
            }
            first += all[i];
        }
    __syncthreads();
    volatile uint32_t* mine = at[wave];      // this wave's alone from here on
    for (int64_t base = m0; base < end; base += kWave) {
        const int64_t m = base + lane;
        const bool in = m < end;
        const uint32_t key = in ? sort_key(a, m) : 0;
        const uint32_t pos = !in ? 0 : a.ids ? static_cast<uint32_t>(m) : a.pos_in[m];
        const Peers peers(key >> a.shift & (n - 1), in, a.bits, lane);
        if (in) {
            const uint32_t to = peers.place(mine);
            a.key_out[to] = key;
            a.pos_out[to] = pos;
            if (a.next) atomicAdd(&a.next[to / a.tile * n + (key >> (a.shift + a.bits) & (n - 1))], 1u);
        }
    }
}

// All passes of few positions in one workgroup and one launch, in LDS: what the
// launches above take for so few is their start (a gradient added to a table, M 2048
// V32768 D1536 bf16: 22 us a call in place of 30).  With more, the rounds of one CU take
// longer than they save (M 16384: 50 us against 23).
constexpr int kSmallThreads = 1024;
constexpr int kSmallRounds = 2;
constexpr int kSmallRows = kSmallThreads * kSmallRounds;

struct SmallSortArgs {
    const void* ids;
    bool wide;
    int M, bits, passes;
    int64_t V;
    uint32_t* key_out;
    uint32_t* pos_out;
};

__global__ __launch_bounds__(kSmallThreads) void sort_small_kernel(SmallSortArgs a) {
    constexpr int kWaves = kSmallThreads / kWave;
    static_assert(kMaxBins <= kSmallThreads, "a thread to a digit");
    __shared__ uint32_t keys[kSmallRows], places[kSmallRows];
    __shared__ uint32_t at[kWaves][kMaxBins];       // per wave: keys of a digit, then the place of the next one
    __shared__ uint32_t sums[kWaves];
    const int n = 1 << a.bits, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int m0 = wave * kSmallRounds * kWave + lane;          // a wave's positions lie in a row
    uint32_t key[kSmallRounds], pos[kSmallRounds];
#pragma unroll
    for (int i = 0; i < kSmallRounds; i++) {
        const int m = m0 + i * kWave;
        key[i] = m < a.M ? key_of(a.ids, a.wide, m, a.V) : 0;
        pos[i] = m;
    }
    for (int p = 0; p < a.passes; p++) {
        const int shift = p * a.bits;
        for (int b = threadIdx.x; b < kWaves * n; b += kSmallThreads) at[b / n][b % n] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSmallRounds; i++)
            if (m0 + i * kWave < a.M) atomicAdd(&at[wave][key[i] >> shift & (n - 1)], 1u);
        __syncthreads();
        const int d = threadIdx.x;
        uint32_t all = 0;
        if (d < n)
            for (int w = 0; w < kWaves; w++) all += at[w][d];
        uint32_t upto = all;
        for (int k = 1; k < kWave; k *= 2) {
            const uint32_t below = __shfl_up(upto, k);
            if (lane >= k) upto += below;
        }
        if (lane == kWave - 1) sums[wave] = upto;
        __syncthreads();
        if (d < n) {
            uint32_t to = upto - all;
            for (int w = 0; w < wave; w++) to += sums[w];
            for (int w = 0; w < kWaves; w++) {
                const uint32_t c = at[w][d];
                at[w][d] = to;
                to += c;
            }
        }
        __syncthreads();
        volatile uint32_t* mine = at[wave];
#pragma unroll
        for (int i = 0; i < kSmallRounds; i++)
            if (const Peers peers(key[i] >> shift & (n - 1), m0 + i * kWave < a.M, a.bits, lane); peers.in) {
                const uint32_t to = peers.place(mine);
                keys[to] = key[i];
                places[to] = pos[i];
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSmallRounds; i++) {
            key[i] = keys[m0 + i * kWave];
            pos[i] = places[m0 + i * kWave];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kSmallRounds; i++) {
        const int m = m0 + i * kWave;
        if (m >= a.M) break;
        a.key_out[m] = key[i];
        a.pos_out[m] = pos[i];
    }
}

// ---- sums of the sorted rows -------------------------------------------------------

struct SumArgs {
    int64_t M, V, D, ld_dy, ld_dw;
    float scale;
    bool accumulate;
    const void* dy;
    void* dw;
    const uint32_t* key;      // sorted
    const uint32_t* pos;
    float* head;              // [run][D]: of the token that came in from the run before
    float* tail;              // [run][D]: of the token that goes on in the next run
    int64_t runs, slices;
    int64_t joins;            // slices of embed_join_kernel
};

// `o`: what dW holds there, where it is added to.
template <typename TW, int V>
__device__ __forceinline__ void write_sum(const SumArgs& a, uint32_t key, int c, const float (&sum)[V], RowVec<TW, V> o) {
    const int n = static_cast<int>(a.D);
    TW* dw = static_cast<TW*>(a.dw) + key * a.ld_dw;
#pragma unroll
    for (int e = 0; e < V; e++) {
        const float v = a.scale * sum[e];
        o.set(e, a.accumulate ? o[e] + v : v);
    }
    o.template store<kStream>(dw, c, n);
}

template <typename TW, typename TD, int V>
__device__ __forceinline__ void zero_rows(const SumArgs& a, int64_t block, bool* found) {
    const int64_t v0 = block * kZeroRows;
    if (threadIdx.x < kZeroRows) {
        const int64_t v = v0 + threadIdx.x;
        int64_t lo = 0, hi = a.M;             // the first place whose key is v or more
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (a.key[mid] < v) lo = mid + 1;
            else hi = mid;
        }
        found[threadIdx.x] = v >= a.V || (lo < a.M && a.key[lo] == v);
    }
    __syncthreads();
    const int n = static_cast<int>(a.D);
    RowVec<TW, V> z;
    z.zero();
    for (int i = 0; i < kZeroRows; i++) {
        if (found[i]) continue;
        TW* dw = static_cast<TW*>(a.dw) + (v0 + i) * a.ld_dw;
        for (int c = threadIdx.x * V; c < n; c += blockDim.x * V) z.template store<kStream>(dw, c, n);
    }
}

template <typename TW, typename TD>
__global__ __launch_bounds__(kSumThreads) void embed_sum_kernel(SumArgs a) {
    constexpr int V = kVec<TW, TD>;
    constexpr int kAhead = 16;
    __shared__ uint32_t keys[kRun + 2], places[kRun];
    __shared__ bool found[kZeroRows];
    const int64_t sums = a.runs * a.slices;
    if (blockIdx.x >= sums) {
        zero_rows<TW, TD, V>(a, blockIdx.x - sums, found);
        return;
    }
    const int64_t run = blockIdx.x / a.slices;
    const int n = static_cast<int>(a.D);
    const int c = (static_cast<int>(blockIdx.x % a.slices) * blockDim.x + threadIdx.x) * V;
    // keys[1 + i] is the run's i-th; the places beyond the ends hold V, a key without a row
    const int64_t m0 = run * kRun;
    if (threadIdx.x < kRun + 2) {
        const int64_t m = m0 + threadIdx.x - 1;
        keys[threadIdx.x] = m >= 0 && m < a.M ? a.key[m] : static_cast<uint32_t>(a.V);
        if (threadIdx.x < kRun) places[threadIdx.x] = m + 1 < a.M ? a.pos[m + 1] : 0;
    }
    __syncthreads();
    if (c >= n || keys[1] >= a.V) return;
    const TD* dy = static_cast<const TD*>(a.dy);
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; e++) sum[e] = 0.0f;
    bool first = keys[0] != keys[1];            // the current token begins in this run
    for (int i0 = 0; i0 < kRun; i0 += kAhead) {
        RowVec<TD, V> r[kAhead];
        RowVec<TW, V> old[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const uint32_t key = keys[1 + i0 + i];
            if (key >= a.V) continue;
            r[i].load(dy + places[i0 + i] * a.ld_dy, c, n);
            if (a.accumulate && key != keys[2 + i0 + i]) old[i].load(static_cast<const TW*>(a.dw) + key * a.ld_dw, c, n);
        }
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const uint32_t key = keys[1 + i0 + i], next = keys[2 + i0 + i];
            if (key >= a.V) return;
#pragma unroll
            for (int e = 0; e < V; e++) sum[e] += r[i][e];
            const bool last = i0 + i == kRun - 1;
            if (key == next && !last) continue;
            if (first && key != next) {
                write_sum<TW, V>(a, key, c, sum, old[i]);
            } else {
                RowVec<float, V> o;
#pragma unroll
                for (int e = 0; e < V; e++) o.set(e, sum[e]);
                o.template store<false>((first ? a.tail : a.head) + run * a.D, c, n);
            }
            first = true;
#pragma unroll
            for (int e = 0; e < V; e++) sum[e] = 0.0f;
        }
    }
}

// The tokens that reach over the end of the run they begin in, for 64 V columns: a
// wave looks at one end, and adds up a token's parts if they are few.  Those of a
// token in many runs are added up by the workgroup, in equal shares in order, and
// the shares in order.
constexpr int kJoinThreads = 512;
constexpr int kEnds = kJoinThreads / kWave;

template <typename TW, typename TD>
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(SumArgs a) {
    constexpr int V = kVec<TW, TD>, kAhead = 8;
    __shared__ float parts[kEnds][kWave * V];
    __shared__ int64_t many[kEnds];              // one past the last run of a token in many, or 0
    const int n = static_cast<int>(a.D), lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int c = (static_cast<int>(blockIdx.x % a.joins) * kWave + lane) * V;
    const int64_t run0 = blockIdx.x / a.joins * kEnds;
    // adds head[from .. to)
    const auto add = [&](float (&sum)[V], int64_t from, int64_t to) {
        for (int64_t r = from; r < to; r += kAhead) {
            RowVec<float, V> p[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; i++)
                if (r + i < to && c < n) p[i].load(a.head + (r + i) * a.D, c, n);
                else p[i].zero();
#pragma unroll
            for (int i = 0; i < kAhead; i++)
#pragma unroll
                for (int e = 0; e < V; e++) sum[e] += p[i][e];
        }
    };
    const auto begin = [&](float (&sum)[V], RowVec<TW, V>& old, int64_t run, uint32_t key) {
        if (a.accumulate && c < n) old.load(static_cast<const TW*>(a.dw) + key * a.ld_dw, c, n);
#pragma unroll
        for (int e = 0; e < V; e++) sum[e] = c + e < n ? a.tail[run * a.D + c + e] : 0.0f;
    };
    float sum[V];
    RowVec<TW, V> old;
    int64_t last = 0;
    {
        const int64_t run = run0 + wave, m0 = run * kRun, end = m0 + kRun;
        const bool inside = end < a.M;
        const uint32_t before = inside && m0 > 0 ? a.key[m0 - 1] : static_cast<uint32_t>(a.V);
        const uint32_t first = inside ? a.key[m0] : 0, key = inside ? a.key[end - 1] : 0;
        const uint32_t next = inside ? a.key[end] : 1;
        if (key == next && key < a.V && !(first == key && before == key)) {
            // one past the last run that starts with the token: doubling steps, then halving ones
            int64_t lo = run + 1, hi = run + 2;
            while (hi < a.runs && a.key[hi * kRun] == key) {
                lo = hi;
                hi += hi - run;
            }
            if (hi > a.runs) hi = a.runs;
            lo++;
            while (lo < hi) {
                const int64_t mid = (lo + hi) / 2;
                if (a.key[mid * kRun] == key) lo = mid + 1;
                else hi = mid;
            }
            if (lo - run - 1 > 2 * kAhead) {
                last = lo;
            } else {
                begin(sum, old, run, key);
                add(sum, run + 1, lo);
                if (c < n) write_sum<TW, V>(a, key, c, sum, old);
            }
        }
    }
    if (lane == 0) many[wave] = last;
    __syncthreads();
    for (int i = 0; i < kEnds; i++) {
        if (many[i] == 0) continue;
        const int64_t run = run0 + i, each = (many[i] - run - 1 + kEnds - 1) / kEnds;
        const int64_t from = run + 1 + wave * each, to = from + each < many[i] ? from + each : many[i];
        const uint32_t key = a.key[run * kRun + kRun - 1];
        if (wave == 0) {
            begin(sum, old, run, key);
        } else {
#pragma unroll
            for (int e = 0; e < V; e++) sum[e] = 0.0f;
        }
        add(sum, from, to);
#pragma unroll
        for (int e = 0; e < V; e++) parts[wave][lane * V + e] = sum[e];
        __syncthreads();
        if (wave == 0 && c < n) {
            for (int w = 1; w < kEnds; w++)
#pragma unroll
                for (int e = 0; e < V; e++) sum[e] += parts[w][lane * V + e];
            write_sum<TW, V>(a, key, c, sum, old);
        }
        __syncthreads();
    }
}

// ---- host ------------------------------------------------------------------------

struct Plan {
    int passes, bits;         // bits per pass
    int64_t tiles, runs;
    int tile;
    int64_t key[2], pos[2], counts, head, tail, bytes;   // offsets
};

bool plan_of(int64_t M, int64_t V, int64_t D, Plan& p) {
    int bits = 1;
    while (V >> bits) bits++;
    p.passes = (bits + kMaxBits - 1) / kMaxBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    // enough tiles to spread the work, few enough to add their counts up in every one of them
    p.tile = static_cast<int>(ceil_div(ceil_div(M, kMostTiles), 2 * kSortThreads) * 2 * kSortThreads);
    if (p.tile < 2 * kSortThreads) p.tile = 2 * kSortThreads;
    p.tiles = ceil_div(M, p.tile);
    p.runs = ceil_div(M, kRun);
    int64_t at = 0;
    const auto take = [&](int64_t n) {
        const int64_t here = at;
        at += ceil_div(n * 4, 256) * 256;
        return here;
    };
    for (int i = 0; i < 2; i++) p.key[i] = take(M), p.pos[i] = take(M);
    p.counts = take((p.tiles << p.bits) * p.passes);
    if (p.runs > (int64_t{1} << 60) / (D > 0 ? D : 1)) return false;
    p.head = take(p.runs * D);
    p.tail = take(p.runs * D);
    p.bytes = at;
    // grids: every launch below 2^32 threads
    const int64_t sums = p.runs * ceil_div(D, 4 * kSumThreads) + ceil_div(V, kZeroRows);
    const int64_t joins = ceil_div(p.runs, kEnds) * ceil_div(D, 4 * kWave);
    const int64_t blocks = sums > joins ? sums : joins;
    return p.runs < (int64_t{1} << 23) && D <= MSS_MAX_WIDTH && blocks < (int64_t{1} << 32) / kSumThreads;
}

template <typename F>
hipError_t by_types(int table, int rows, F&& f) {
    const auto second = [&](auto w) {
        using TW = decltype(w);
        if (rows == MSS_F32) return f(w, 0.0f);
        if constexpr (!std::is_same_v<TW, f16>)
            if (rows == MSS_BF16) return f(w, bf16{});
        if constexpr (!std::is_same_v<TW, bf16>)
            if (rows == MSS_F16) return f(w, f16{});
        return hipErrorInvalidValue;
    };
    return table == MSS_F32 ? second(0.0f) : table == MSS_BF16 ? second(bf16{}) : second(f16{});
}

}  // namespace

bool embed_bwd_workspace(int64_t M, int64_t V, int64_t D, int64_t& bytes) {
    Plan p;
    if (!plan_of(M, V, D, p)) return false;
    bytes = p.bytes;
    return true;
}

hipError_t launch_embed(const EmbedArgs& all, hipStream_t st) {
    constexpr int64_t kMost = int64_t{1} << 25;      // rows of a launch, below 2^32 threads
    return by_types(all.dtype, all.out_dtype, [&](auto w, auto y) {
        for (int64_t m0 = 0; m0 < all.M; m0 += kMost) {
            EmbedArgs a = all;
            a.M = all.M - m0 < kMost ? all.M - m0 : kMost;
            a.ids = static_cast<const char*>(all.ids) + m0 * (all.wide_ids ? 8 : 4);
            a.y = static_cast<decltype(y)*>(all.y) + m0 * all.ld_y;
            embed_kernel<decltype(w), decltype(y)><<<static_cast<uint32_t>(ceil_div(a.M, 4)), 256, 0, st>>>(a);
            if (hipError_t e = hipGetLastError()) return e;
        }
        return hipSuccess;
    });
}

hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t st) {
    Plan p;
    if (!plan_of(a.M, a.V, a.D, p)) return hipErrorInvalidValue;
    char* ws = static_cast<char*>(a.ws);
    const auto words = [&](int64_t at) { return reinterpret_cast<uint32_t*>(ws + at); };
    int from = 1;
    const bool small = a.M <= kSmallRows;
    if (small && a.M > 0) {
        from = 0;
        sort_small_kernel<<<1, kSmallThreads, 0, st>>>({a.ids, a.wide_ids, static_cast<int>(a.M), p.bits, p.passes, a.V,
                                                        words(p.key[0]), words(p.pos[0])});
        if (hipError_t e = hipGetLastError()) return e;
    }
    for (int i = 0; i < p.passes && !small; i++) {
        SortArgs s{};
        s.ids = i == 0 ? a.ids : nullptr;
        s.wide = a.wide_ids;
        s.M = a.M;
        s.V = a.V;
        s.key_in = words(p.key[from]);
        s.pos_in = words(p.pos[from]);
        s.key_out = words(p.key[from ^ 1]);
        s.pos_out = words(p.pos[from ^ 1]);
        s.counts = words(p.counts) + i * (p.tiles << p.bits);
        s.next = i + 1 < p.passes ? s.counts + (p.tiles << p.bits) : nullptr;
        s.later = p.passes - 1;
        s.tiles = p.tiles;
        s.tile = p.tile;
        s.shift = i * p.bits;
        s.bits = p.bits;
        from ^= 1;
        if (i == 0) {
            sort_count_kernel<<<static_cast<uint32_t>(p.tiles), kSortThreads, 0, st>>>(s);
            if (hipError_t e = hipGetLastError()) return e;
        }
        sort_place_kernel<<<static_cast<uint32_t>(p.tiles), kSortThreads, 0, st>>>(s);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return by_types(a.dtype, a.out_dtype, [&](auto w, auto y) {
        using TW = decltype(w);
        using TD = decltype(y);
        const int64_t vecs = ceil_div(a.D, kVec<TW, TD>);
        const int64_t slices = ceil_div(vecs, kSumThreads);
        const int threads = static_cast<int>(ceil_div(ceil_div(vecs, slices), 64) * 64);
        SumArgs s{};
        s.M = a.M;
        s.V = a.V;
        s.D = a.D;
        s.ld_dy = a.ld_y;
        s.ld_dw = a.ld_w;
        s.scale = a.scale;
        s.accumulate = a.accumulate;
        s.dy = a.y;
        s.dw = a.dw;
        s.key = words(p.key[from]);
        s.pos = words(p.pos[from]);
        s.head = reinterpret_cast<float*>(ws + p.head);
        s.tail = reinterpret_cast<float*>(ws + p.tail);
        s.runs = p.runs;
        s.slices = slices;
        const int64_t zeros = a.accumulate ? 0 : ceil_div(a.V, kZeroRows);
        embed_sum_kernel<TW, TD><<<static_cast<uint32_t>(s.runs * s.slices + zeros), threads, 0, st>>>(s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.M == 0) return e;
        s.joins = ceil_div(vecs, kWave);
        const uint32_t groups = static_cast<uint32_t>(ceil_div(s.runs, kEnds) * s.joins);
        embed_join_kernel<TW, TD><<<groups, kJoinThreads, 0, st>>>(s);
        return hipGetLastError();
    });
}

}  // namespace mss
