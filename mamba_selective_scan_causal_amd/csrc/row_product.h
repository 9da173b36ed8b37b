// row_product.h -- products of rows on the matrix cores of gfx950:
//   C[l][r] = sum_k L[l][k] R[r][k]
// with L (nl, K) and R (nr, K) row-major (K contiguous), as the head's logits
// and both of its gradients are computed.
//
// A workgroup computes a BL x BR tile of C.  128 bytes of every row (64 values
// of two bytes, 32 of four) go to LDS per stage, one stage ahead of the matrix
// instructions: by direct loads where the rows lie at multiples of 16 bytes,
// through registers otherwise.  Chunk c (16 bytes) of row i lies at chunk
// c ^ (i & 7) of the row's 128 bytes: the 16 rows that a fragment reads at one
// c then fall on different banks.  R is the instruction's row operand, so that a
// lane ends up with four neighbouring r of one l: runs of C's rows.
#pragma once

#include <type_traits>

#include "block_math.h"

namespace mss {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kStage = 128;                       // bytes of a row per stage
constexpr int kXcds = 8;
constexpr int kNoLoads = 0x0f70;                  // s_waitcnt: vmcnt 0, the other counters as they are

// Fragments of 16 rows by 32 values of K, and the products of two of them.  A
// lane's chunks c and c + 4 of its row are what it holds of a fragment's row in
// fp32; in two-byte types each chunk is of a fragment of its own.  (Which k goes
// where does not matter as long as both operands agree.)
template <typename T>
struct Mma;
template <>
struct Mma<bf16> {
    typedef bf16 frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ v4f run(v4i r, v4i l, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, r),
                                                       __builtin_bit_cast(frag, l), c, 0, 0, 0);
    }
};
template <>
struct Mma<f16> {
    typedef f16 frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ v4f run(v4i r, v4i l, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, r),
                                                      __builtin_bit_cast(frag, l), c, 0, 0, 0);
    }
};

// fp32 values as three bf16 each, high to low, 8 bits of the significand in each
// (cut off, not rounded: the parts add up to the value exactly, and none overflows).
// A product is the six of the nine partial products that are not below 2^-22 of it:
// six instructions at a sixteenth of the fp32 instruction's time each, and the
// splitting (M2048 V32768 D768: 211 TFLOP/s against 139 with the fp32 instruction).
// An infinity has no such parts (inf - inf is NaN, and so is inf times the other operand's
// empty lower parts): sums that are not finite are computed again (RowProduct::mend).
struct Parts {
    v4i p[3];
    __device__ __forceinline__ void of(v4i a_, v4i b_) {
        const v4f a = __builtin_bit_cast(v4f, a_), b = __builtin_bit_cast(v4f, b_);
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = a[e], v[4 + e] = b[e];
#pragma unroll
        for (int k = 0; k < 3; k++) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                p[k][e] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, v[2 * e + 1]),
                                                __builtin_bit_cast(uint32_t, v[2 * e]), 0x07060302);
            if (k == 2) break;
#pragma unroll
            for (int e = 0; e < 8; e++)
                v[e] -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v[e]) & 0xffff0000u);
        }
    }
};

struct ProductArgs {
    const char* l;            // row-strided operands
    const char* r;
    int64_t ld_l, ld_r;       // bytes
    int64_t nl, nr;           // rows of each (at least 1)
    int64_t kbytes;           // bytes of a row that count
    const int* off;           // rows of l that count as zeros: off[row] < 0 (null: none)
    int64_t tiles_l, tiles_r;
};

// The tile of C that workgroup b computes.  Neighbouring workgroups go to
// different XCDs, so each XCD gets a contiguous part of the tiles; within it
// GL tiles along l share their r tile, so that the tiles computed at one time
// on an XCD form a block, whose operands its L2 holds.
template <int GL>
__device__ __forceinline__ void tile_of(int64_t b, int64_t n, int64_t tiles_l, int64_t tiles_r, int64_t& tl,
                                        int64_t& tr) {
    const int64_t xcd = b % kXcds, per = n / kXcds, rest = n % kXcds;
    const int64_t t = xcd * per + (xcd < rest ? xcd : rest) + b / kXcds;
    const int64_t group = t / (GL * tiles_r), first = group * GL;
    const int64_t high = tiles_l - first < GL ? tiles_l - first : GL;
    const int64_t in = t - group * (GL * tiles_r);
    tl = first + in % high;
    tr = in / high;
}

typedef const __attribute__((address_space(1))) void* gmem;
typedef __attribute__((address_space(3))) void* lmem;

static __device__ const v4i kZeros = {0, 0, 0, 0};

// A stage of ROWS rows of one operand: where this lane's chunks come from.
template <int ROWS, int WAVES>
struct StageRows {
    static constexpr int kLoads = ROWS / 8 / WAVES;
    const char* p[kLoads];
    int64_t at;               // this lane's byte of the row
    bool on[kLoads];          // whether the row counts

    __device__ __forceinline__ void init(const char* base, int64_t ld, int64_t row0, int64_t n, int wave, int lane,
                                         const int* off) {
        at = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
        for (int s = 0; s < kLoads; s++) {
            // rows past the last read the last one again: their products are not used
            int64_t row = row0 + (s * WAVES + wave) * 8 + (lane >> 3);
            row = row < n ? row : n - 1;
            p[s] = base + row * ld;
            on[s] = !off || off[row] >= 0;
        }
    }
    static __device__ __forceinline__ char* place(char* lds, int s, int wave) { return lds + (s * WAVES + wave) * 1024; }
};

// Rows that start at multiples of 16 bytes and are a multiple of 16 long: straight
// to LDS, once load() is called.
template <typename T, int ROWS, int WAVES>
struct DirectStage : StageRows<ROWS, WAVES> {
    using Rows = StageRows<ROWS, WAVES>;
    // The chunks of the stage that starts at byte k of the rows.  Past the end of a
    // row both operands read zeros.
    __device__ __forceinline__ void load(char* lds, int64_t k, int64_t kbytes, int wave) {
        const bool in = k + this->at < kbytes;
#pragma unroll
        for (int s = 0; s < Rows::kLoads; s++) {
            const char* q = in && this->on[s] ? this->p[s] + k + this->at : reinterpret_cast<const char*>(&kZeros);
            __builtin_amdgcn_global_load_lds((gmem)q, (lmem)Rows::place(lds, s, wave), 16, 0, 0);
        }
    }
    __device__ __forceinline__ void keep(char*, int, int) {}
};

// Rows at any element: to registers when load() is called, to LDS by keep().
template <typename T, int ROWS, int WAVES>
struct ThroughStage : StageRows<ROWS, WAVES> {
    using Rows = StageRows<ROWS, WAVES>;
    static constexpr int V = 16 / sizeof(T);
    RowVec<T, V> r[Rows::kLoads];
    __device__ __forceinline__ void load(char*, int64_t k, int64_t kbytes, int) {
        const int64_t c = (k + this->at) / static_cast<int>(sizeof(T)), n = kbytes / static_cast<int>(sizeof(T));
        if (c + V <= n) {
#pragma unroll
            for (int s = 0; s < Rows::kLoads; s++)
                r[s].t = *reinterpret_cast<const typename RowVec<T, V>::type*>(this->p[s] + k + this->at);
        } else {
            const int have = c < n ? static_cast<int>(n - c) : 0;
#pragma unroll
            for (int s = 0; s < Rows::kLoads; s++)
                r[s].load(reinterpret_cast<const T*>(this->p[s]) + (have ? c : 0), 0, have);
        }
    }
    __device__ __forceinline__ void keep(char* lds, int wave, int lane) {
#pragma unroll
        for (int s = 0; s < Rows::kLoads; s++)
            *reinterpret_cast<v4i*>(Rows::place(lds, s, wave) + lane * 16) =
                this->on[s] ? __builtin_bit_cast(v4i, r[s].t) : v4i{0, 0, 0, 0};
    }
};

// A stage of COLS columns of an operand that lies with K down its rows: 128 bytes'
// worth of rows of the tile's columns, straight to LDS.  Row k's values at columns
// 16 b .. 16 b + 15 lie at block b ^ swap(k): the rows that are read at one b at one
// time (eight by half a wave in two-byte types, four by a wave in fp32) are then on
// different banks.
template <typename T>
__device__ __forceinline__ int swap_of(int k) {
    return sizeof(T) == 2 ? (k & 3) | (k >> 1 & 4) : k >> 2 & 3;
}

template <typename T, int COLS, int WAVES>
struct ColumnStage {
    static_assert(COLS % 128 == 0, "whole groups of blocks");
    static constexpr int kSize = sizeof(T), kLoads = COLS / 8 / WAVES, kPitch = COLS * kSize;
    static constexpr int kDown = 1024 / kPitch;                 // rows of a load
    const char* p;
    int64_t ld;
    int first;                // this lane's row of the wave's first load
    bool in[kLoads];          // whether its columns are the operand's
    int64_t at[kLoads];       // bytes from p

    // n columns, whole pieces of 16 bytes, at multiples of 16 bytes.
    __device__ __forceinline__ void init(const char* base, int64_t ld_, int64_t col0, int64_t n, int wave, int lane,
                                         const int*) {
        p = base + col0 * kSize;
        ld = ld_;
        const int piece = lane * 16 % kPitch / 16;
        first = wave * kDown + lane * 16 / kPitch;
#pragma unroll
        for (int s = 0; s < kLoads; s++) {
            const int k = first + s * WAVES * kDown;
            const int col = ((piece / kSize) ^ swap_of<T>(k)) * 16 + piece % kSize * (16 / kSize);
            in[s] = col0 + col < n;
            at[s] = k * ld + col * kSize;
        }
    }
    // The rows that start at byte k of what would be a row; zeros past kbytes.
    __device__ __forceinline__ void load(char* lds, int64_t k, int64_t kbytes, int wave) {
        const int64_t row = k / kSize, rows = kbytes / kSize;
        const char* base = p + row * ld;
#pragma unroll
        for (int s = 0; s < kLoads; s++) {
            const char* q = in[s] && row + first + s * WAVES * kDown < rows ? base + at[s]
                                                                            : reinterpret_cast<const char*>(&kZeros);
            __builtin_amdgcn_global_load_lds((gmem)q, (lmem)(lds + (s * WAVES + wave) * 1024), 16, 0, 0);
        }
    }
    __device__ __forceinline__ void keep(char*, int, int) {}
};

// How an operand lies: K along its rows, at multiples of 16 bytes or anywhere; or
// down its columns (which takes 1.35 times as long: M16384 N1536 K8192 in bf16 564 us
// against 418; the transposing load reads half as many bytes at a time).
enum Layout { kDirect, kThrough, kColumns };
template <typename T, int ROWS, int WAVES, Layout LAYOUT>
struct StageOf {
    using type = DirectStage<T, ROWS, WAVES>;
};
template <typename T, int ROWS, int WAVES>
struct StageOf<T, ROWS, WAVES, kThrough> {
    using type = ThroughStage<T, ROWS, WAVES>;
};
template <typename T, int ROWS, int WAVES>
struct StageOf<T, ROWS, WAVES, kColumns> {
    using type = ColumnStage<T, ROWS, WAVES>;
};

// A lane's part of an operand's stage in LDS: of tile i (16 rows of the operand
// from `first` on), 16 bytes of the row lane % 16.  In two-byte types those are K =
// 8 (lane / 16) + 0..7 of half kk of the stage, in fp32 4 (lane / 16) + 0..3.
template <typename T, int ROWS, Layout LAYOUT>
struct Fragments {
    static constexpr int kReads = 1;
    const char* p;
    int c;
    __device__ __forceinline__ Fragments(const char* stage, int first, int lane)
        : p(stage + (first + lane % 16) * kStage), c((lane / 16 ^ (lane & 7)) * 16) {}
    __device__ __forceinline__ v4i at(int i, int kk) const {
        return *reinterpret_cast<const v4i*>(p + i * 16 * kStage + (c ^ kk * 64));
    }
};
// Columns of two-byte types are read with the transposing load: of 16 lanes, lane l
// reads 8 bytes of row l / 4, and gets column l of the four rows.
template <typename T, int ROWS>
struct Fragments<T, ROWS, kColumns> {
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s* lds4;
    static constexpr int kReads = 2, kPitch = ROWS * 2;
    const char* p;
    int block, swap;
    __device__ __forceinline__ Fragments(const char* stage, int first, int lane)
        : p(stage + (lane / 16 * 8 + lane % 16 / 4) * kPitch + lane % 4 * 8),
          block(first / 16),
          swap(swap_of<T>(lane / 16 * 8 + lane % 16 / 4)) {}
    __device__ __forceinline__ v4i at(int i, int kk) const {
        const char* q = p + ((block + i) ^ swap) * 32 + kk * 32 * kPitch;
        struct {
            v4s a, b;
        } both = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)q),
                  __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(q + 4 * kPitch))};
        return __builtin_bit_cast(v4i, both);
    }
};
template <int ROWS>
struct Fragments<float, ROWS, kColumns> {
    static constexpr int kPitch = ROWS * 4;
    const char* p;
    int block, swap;
    __device__ __forceinline__ Fragments(const char* stage, int first, int lane)
        : p(stage + lane / 16 * 4 * kPitch + lane % 16 * 4), block(first / 16), swap(lane / 16) {}
    __device__ __forceinline__ v4i at(int i, int kk) const {
        const char* q = p + ((block + i) ^ swap) * 64 + kk * 16 * kPitch;
        v4i v;
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = *reinterpret_cast<const int*>(q + e * kPitch);
        return v;
    }
};

// acc[i][j]: the 16 x 16 tile of C at r = 16 i, l = 16 j of the wave's part; a
// lane holds r = 4 (lane / 16) + 0..3, l = lane % 16 of it.
//
// LL, LR: how L and R lie; the products are the same, in the same order.
template <typename T, int BL, int BR, int WL, int WR, Layout LL = kDirect, Layout LR = kDirect>
struct RowProduct {
    static constexpr int kWaves = WL * WR, kThreads = kWaves * kWave;
    static constexpr int kTL = BL / WL / 16, kTR = BR / WR / 16;
    static constexpr int kLds = 2 * (BL + BR) * kStage;

    // The products of a stage in two-byte types, its first and its second half.
    //
    // The order of LDS reads and matrix instructions: the reads that the first
    // kTL products need, then two reads for every kTL products, so that the first
    // half's fragments arrive as they are used, and the second half's while the
    // first is multiplied.  (Left to the compiler, with a wait after every two
    // reads: 1277 against 1316 TFLOP/s at 8192^3 in bf16; one read for two
    // products, or three for four, 1315 and 1298.)
    static __device__ __forceinline__ void narrow(const Fragments<T, BL, LL>& l, const Fragments<T, BR, LR>& r,
                                                  v4f (&acc)[kTR][kTL]) {
        v4i fl[2][kTL], fr[2][kTR];
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
#pragma unroll
            for (int j = 0; j < kTL; j++) fl[kk][j] = l.at(j, kk);
#pragma unroll
            for (int i = 0; i < kTR; i++) fr[kk][i] = r.at(i, kk);
        }
#pragma unroll
        for (int kk = 0; kk < 2; kk++)
#pragma unroll
            for (int i = 0; i < kTR; i++)
#pragma unroll
                for (int j = 0; j < kTL; j++) acc[i][j] = Mma<T>::run(fr[kk][i], fl[kk][j], acc[i][j]);
        constexpr int kRead = 0x100, kMfma = 0x8, nl = Fragments<T, BL, LL>::kReads;
        constexpr int nr = Fragments<T, BR, LR>::kReads;
        __builtin_amdgcn_sched_group_barrier(kRead, kTL * nl + nr, 0);
#pragma unroll
        for (int q = 0; q < kTR - 1; q++) {
            __builtin_amdgcn_sched_group_barrier(kMfma, kTL, 0);
            __builtin_amdgcn_sched_group_barrier(kRead, 2 * nr, 0);
        }
        __builtin_amdgcn_sched_group_barrier(kMfma, kTL, 0);
        __builtin_amdgcn_sched_group_barrier(kRead, kTL * nl + nr, 0);
        __builtin_amdgcn_sched_group_barrier(kMfma, kTR * kTL, 0);
    }

    // The same in fp32: L's fragments are split once for the stage, R's one by one,
    // ahead of the products of the one before.
    static __device__ __forceinline__ void wide(const Fragments<T, BL, LL>& l, const Fragments<T, BR, LR>& r,
                                                v4f (&acc)[kTR][kTL]) {
        Parts fl[kTL], fr;
#pragma unroll
        for (int j = 0; j < kTL; j++) fl[j].of(l.at(j, 0), l.at(j, 1));
        fr.of(r.at(0, 0), r.at(0, 1));
#pragma unroll
        for (int i = 0; i < kTR; i++) {
            Parts next;
            if (i + 1 < kTR) next.of(r.at(i + 1, 0), r.at(i + 1, 1));
            // small products first; the sum of 32 values of K is rounded to acc's size once
            v4f sums[kTL];
#pragma unroll
            for (int j = 0; j < kTL; j++) sums[j] = v4f{0, 0, 0, 0};
#pragma unroll
            for (int sum = 2; sum >= 0; sum--)
#pragma unroll
                for (int k = 0; k <= sum; k++)
#pragma unroll
                    for (int j = 0; j < kTL; j++) sums[j] = Mma<bf16>::run(fr.p[k], fl[j].p[sum - k], sums[j]);
#pragma unroll
            for (int j = 0; j < kTL; j++) acc[i][j] += sums[j];
            fr = next;
        }
    }

    // The 16 x 16 tiles of the wave at l, l + 16, .. (where asked for) and r with the fp32
    // instruction, straight from memory: this lane's rows of L and its row of R at value k0 + lane / 16
    // of K, in steps of four.
    static __device__ __forceinline__ void exact(const ProductArgs& a, int64_t l, int64_t r, int64_t kbegin,
                                                 int64_t kend, int lane, const bool (&asked)[kTL], v4f (&sum)[kTL]) {
        constexpr int kAhead = 4;
        const int64_t down_l = LL == kColumns ? a.ld_l : 4, down_r = LR == kColumns ? a.ld_r : 4;
        r = r < a.nr ? r : a.nr - 1;
        const char* pr = a.r + r * (LR == kColumns ? 4 : a.ld_r);
        const char* pl[kTL];
        bool on[kTL];
#pragma unroll
        for (int j = 0; j < kTL; j++) {
            const int64_t row = l + 16 * j < a.nl ? l + 16 * j : a.nl - 1;
            pl[j] = a.l + row * (LL == kColumns ? 4 : a.ld_l);
            on[j] = !a.off || a.off[row] >= 0;
            sum[j] = v4f{0, 0, 0, 0};
        }
        for (int64_t k0 = kbegin / 4; k0 < kend / 4; k0 += 4 * kAhead) {
            float x[kTL][kAhead], y[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; i++) {
                const int64_t k = k0 + 4 * i + lane / 16;
                y[i] = k < kend / 4 ? *reinterpret_cast<const float*>(pr + k * down_r) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kTL; j++)
                if (asked[j])
#pragma unroll
                    for (int i = 0; i < kAhead; i++) {
                        const int64_t k = k0 + 4 * i + lane / 16;
                        x[j][i] = on[j] && k < kend / 4 ? *reinterpret_cast<const float*>(pl[j] + k * down_l) : 0.0f;
                    }
#pragma unroll
            for (int j = 0; j < kTL; j++)
                if (asked[j])
#pragma unroll
                    for (int i = 0; i < kAhead; i++)
                        sum[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(y[i], x[j][i], sum[j], 0, 0, 0);
        }
    }

    // fp32: the sums that are infinite or NaN, as the fp32 instruction has them. The others stay as they
    // are, so that no sum depends on what else is in its tile. Slow, and rare: an infinity is a mask or
    // the end of a run that has diverged (M2048 V32768 D768: forward 0.59 ms, with 100 tokens masked by
    // -inf 1.23, all of it NaN 7.0; looking for them costs 0.5 to 1 %).
    static __device__ __forceinline__ void mend(const ProductArgs& a, int64_t l0, int64_t r0, int64_t kbegin,
                                                int64_t kend, int lane, v4f (&acc)[kTR][kTL]) {
        float zero = 0.0f;            // 0 times each sum: NaN where one is not finite
#pragma unroll
        for (int i = 0; i < kTR; i++)
#pragma unroll
            for (int j = 0; j < kTL; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) zero = __builtin_fmaf(acc[i][j][e], 0.0f, zero);
        if (!wave_any(!(zero == 0.0f))) return;
        const auto finite = [](float v) { return __builtin_fabsf(v) < INFINITY; };
#pragma unroll
        for (int i = 0; i < kTR; i++) {
            bool asked[kTL], some = false;
#pragma unroll
            for (int j = 0; j < kTL; j++) {
                bool all = true;
#pragma unroll
                for (int e = 0; e < 4; e++) all &= finite(acc[i][j][e]);
                asked[j] = wave_any(!all);
                some |= asked[j];
            }
            if (!some) continue;
            v4f sum[kTL];
            exact(a, l0 + lane % 16, r0 + 16 * i + lane % 16, kbegin, kend, lane, asked, sum);
#pragma unroll
            for (int j = 0; j < kTL; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][j][e] = finite(acc[i][j][e]) ? acc[i][j][e] : sum[j][e];
        }
    }

    static __device__ __forceinline__ void run(const ProductArgs& a, int64_t l0, int64_t r0, int64_t kbegin,
                                               int64_t kend, char* lds, v4f (&acc)[kTR][kTL]) {
        const int lane = threadIdx.x % kWave;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const int wl = wave % WL, wr = wave / WL;
        typename StageOf<T, BL, kWaves, LL>::type sl;
        typename StageOf<T, BR, kWaves, LR>::type sr;
        sl.init(a.l, a.ld_l, l0, a.nl, wave, lane, a.off);
        sr.init(a.r, a.ld_r, r0, a.nr, wave, lane, nullptr);
#pragma unroll
        for (int i = 0; i < kTR; i++)
#pragma unroll
            for (int j = 0; j < kTL; j++) acc[i][j] = v4f{0, 0, 0, 0};
        if (kbegin >= kend) return;
        sl.load(lds, kbegin, kend, wave);
        sr.load(lds + BL * kStage, kbegin, kend, wave);
        sl.keep(lds, wave, lane);
        sr.keep(lds + BL * kStage, wave, lane);
        int buf = 0;
        for (int64_t k = kbegin; k < kend; k += kStage) {
            // this stage has landed for every wave, and every wave has read the other one
            __builtin_amdgcn_s_waitcnt(kNoLoads);
            __syncthreads();
            char* next = lds + (buf ^ 1) * (BL + BR) * kStage;
            if (k + kStage < kend) {
                sl.load(next, k + kStage, kend, wave);
                sr.load(next + BL * kStage, k + kStage, kend, wave);
            }
            const char* pl = lds + buf * (BL + BR) * kStage;
            const char* pr = pl + BL * kStage;
            if constexpr (sizeof(T) == 4)
                wide({pl, wl * (BL / WL), lane}, {pr, wr * (BR / WR), lane}, acc);
            else
                narrow({pl, wl * (BL / WL), lane}, {pr, wr * (BR / WR), lane}, acc);
            if (k + kStage < kend) {
                sl.keep(next, wave, lane);
                sr.keep(next + BL * kStage, wave, lane);
            }
            buf ^= 1;
        }
        if constexpr (sizeof(T) == 4) mend(a, l0 + wl * (BL / WL), r0 + wr * (BR / WR), kbegin, kend, lane, acc);
    }
};

// Orders a wave's LDS writes before its lanes' reads of them (the hardware
// does; this is for the compiler).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 16 bytes of T's to p, which may lie at any element, n of them.
template <typename T>
__device__ __forceinline__ void store_piece(T* p, v4i piece, int64_t n) {
    constexpr int V = 16 / sizeof(T);
    RowVec<T, V> r;
    r.t = __builtin_bit_cast(typename RowVec<T, V>::type, piece);
    if (n > 0) r.template store<false>(p, 0, n < V ? static_cast<int>(n) : V);
}

// A wave's part of C, 16 * TR values along r for 16 * TL along l, to memory
// through LDS, so that whole lines are written: a lane's own four values are 8
// bytes of a row, and rows are far apart.
//
// Rows of l: out[l * ld + r], l < nl, r < nr, from the wave's first l and r;
// get(i, j) gives the four values of acc[i][j].  `lds` is the wave's own.
template <typename T, int TR, int TL>
struct RowStore {
    static constexpr int kRow = 16 * TR * sizeof(T) + 16;       // 16 bytes apart from a multiple of all banks
    static constexpr int kBytes = 16 * kRow;
    template <typename F>
    static __device__ __forceinline__ void run(char* lds, int lane, T* out, int64_t ld, int64_t nl, int64_t nr, F get) {
        typedef T quad __attribute__((ext_vector_type(4)));
        constexpr int kPieces = TR * sizeof(T);                  // of a row
#pragma unroll
        for (int j = 0; j < TL; j++) {
#pragma unroll
            for (int i = 0; i < TR; i++) {
                const quad v = get(i, j);
                *reinterpret_cast<quad*>(lds + lane % 16 * kRow + (16 * i + lane / 16 * 4) * sizeof(T)) = v;
            }
            wave_lds_fence();
#pragma unroll
            for (int k = 0; k < (16 * kPieces + kWave - 1) / kWave; k++) {
                const int at = k * kWave + lane, row = at / kPieces, c = at % kPieces;
                const int64_t l = 16 * j + row, r = c * (16 / sizeof(T));
                if (row < 16 && l < nl)
                    store_piece(out + l * ld + r, *reinterpret_cast<const v4i*>(lds + row * kRow + c * 16), nr - r);
            }
            wave_lds_fence();
        }
    }
};

// Rows of r: out[r * ld + l], GROUP tiles along r at a time.
template <typename T, int TR, int TL, int GROUP>
struct ColStore {
    static_assert(TR % GROUP == 0, "whole groups");
    static constexpr int kRow = 16 * TL * sizeof(T) + 16, kRows = 16 * GROUP;
    static constexpr int kBytes = kRows * kRow;
    template <typename F>
    static __device__ __forceinline__ void run(char* lds, int lane, T* out, int64_t ld, int64_t nl, int64_t nr, F get) {
        constexpr int kPieces = TL * sizeof(T);
#pragma unroll
        for (int i0 = 0; i0 < TR; i0 += GROUP) {
#pragma unroll
            for (int i = 0; i < GROUP; i++)
#pragma unroll
                for (int j = 0; j < TL; j++) {
                    const auto v = get(i0 + i, j);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        *reinterpret_cast<T*>(lds + (16 * i + lane / 16 * 4 + e) * kRow +
                                              (16 * j + lane % 16) * sizeof(T)) = v[e];
                }
            wave_lds_fence();
#pragma unroll
            for (int k = 0; k < (kRows * kPieces + kWave - 1) / kWave; k++) {
                const int at = k * kWave + lane, row = at / kPieces, c = at % kPieces;
                const int64_t r = 16 * i0 + row, l = c * (16 / sizeof(T));
                if (row < kRows && r < nr)
                    store_piece(out + r * ld + l, *reinterpret_cast<const v4i*>(lds + row * kRow + c * 16), nl - l);
            }
            wave_lds_fence();
        }
    }
};

}  // namespace mss
