// head_kernel.hip -- softmax cross entropy of x W^T over a large vocabulary, and
// its gradients, without keeping the logits.
//
// Forward: each tile of logits l leaves, for each of its rows, the largest logit
// and the sum of e^(l - largest) of the columns of one wave; a second kernel joins
// those of a row and takes the target's logit, which the tile that has it wrote.
// The exponentials are powers of 2 whose argument is one fused multiply-add of the
// product; where its rounding could matter (kFar) logits are subtracted first.
//
// Backward, a piece of the vocabulary at a time:
//   dl = (dloss + dlse) p - dloss [v = t],  p = e^(l - lse),  recomputed from
// the logits' tiles, in the operands' type, as dl (rows, piece) and its
// transpose; then dx += dl W and dW = dl^T x, in one launch.  All three are
// products of rows (row_product.h), for which x and the piece of W are transposed
// first: that reads and writes each once, against products that take hundreds of
// operations for each of their values.  With few rows dx's product reads W down
// its columns instead (kColumnRows).
//
// What bounds it, by a trace: M8192 V32768 D1536 bf16 takes 751 us forward (1099
// TFLOP/s, a library product of the size 583 us; 669 us and 1232 TFLOP/s in a run of
// forwards alone), 883 for dl with its two stores of 537 MB, 1384 for both gradients (1192
// TFLOP/s): matrix instructions, with 10 to 15 % in the start and end of tiles.
// M8 V65536 D2560 reads W at 5.9 TB/s (57 us).
//
// dl is held times a factor that brings the largest |dloss| + |dlse| to just
// below 2^13: fp16 would lose what a mean over many rows leaves of it, and right
// below a power of two a value's rounding is smallest against it -- where a mean
// gives all rows one factor, the dl of unlikely targets, which weigh most, all lie
// there (bf16, M8192 V32768 D1536: dx is off by 0.0020 of its norm, of which 0.0017
// is its own rounding; with the same dl right above a power of two, 0.0028).  dx and
// dW are scaled back in fp32.  In fp16 the rows of dl, which make dx, have each a
// further power of 2 (RowGrads::lift), so that a row's digits do not depend on how
// large the others' dloss is (V32768 D256, a row of 2^-26 of the largest: its dx
// off by 0.1 % of its norm in place of 3 %).  dl^T, which sums over the rows, has
// none: what lies below 2^-38 of the largest is lost to dW.
#include <algorithm>

#include "launch_ends.h"
#include "row_product.h"

namespace mss {
namespace {

// Tiles along l that share their r tile in an XCD's L2 (both gradients, M8192 V32768 D1536 bf16:
// 2, 4, 5, 8 and 16 tiles take 2306, 2290, 2368, 2355 and 2385 us; the forward changes by
// 1 %).
constexpr int kGroup = 4;
constexpr int kPadRows = 64;                 // dl^T and x^T have rows of a multiple of this many values

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile shapes, rows of the operand whose rows are C's first.  With 256 x 256
// and 192 x 320 one workgroup of eight waves fills a CU's LDS, of the others' four
// waves two do (four of the last, which reads the vocabulary for a few rows: 8 rows
// of 65536 x 2560 in bf16 take 63.0 us a call with it, 64.5 with 128 x 128 and 86 with
// 256 x 256).
enum TileShape { kLarge, kTall, kWide, kSmall, kFew };
template <bool DIRECT>
constexpr Layout kLies = DIRECT ? kDirect : kThrough;
template <typename T, int SHAPE, bool DIRECT>
struct Tile;
template <typename T, bool DIRECT>
struct Tile<T, kLarge, DIRECT> {
    using type = RowProduct<T, 256, 256, 4, 2, kLies<DIRECT>, kLies<DIRECT>>;
};
template <typename T, bool DIRECT>
struct Tile<T, kTall, DIRECT> {
    using type = RowProduct<T, 192, 320, 4, 2, kLies<DIRECT>, kLies<DIRECT>>;
};
template <typename T, bool DIRECT>
struct Tile<T, kWide, DIRECT> {
    using type = RowProduct<T, 128, 160, 2, 2, kLies<DIRECT>, kLies<DIRECT>>;
};
template <typename T, bool DIRECT>
struct Tile<T, kSmall, DIRECT> {
    using type = RowProduct<T, 128, 128, 2, 2, kLies<DIRECT>, kLies<DIRECT>>;
};
template <typename T, bool DIRECT>
struct Tile<T, kFew, DIRECT> {
    using type = RowProduct<T, 32, 128, 1, 4, kLies<DIRECT>, kLies<DIRECT>>;
};
template <typename P>
struct Tag {
    using type = P;
};

// f(Tag of the shape's RowProduct).  Through registers kTall and kWide are slower than
// the other shapes, and so is kLarge in fp32 (its registers spill).  FEW: where kFew may
// be the shape.
// A column product has the shapes whose columns are groups of 128, without kLarge in
// fp32 (spills too).
constexpr bool has_columns(int shape, int64_t elem) { return shape == kSmall || (shape == kLarge && elem == 2); }
constexpr bool has_tile(int shape, bool direct, int64_t elem) {
    return direct || shape == kSmall || shape == kFew || (shape == kLarge && elem == 2);
}
template <typename T, bool DIRECT, bool FEW, typename F>
void with_tile(int shape, F&& f) {
    const auto as = [&](auto s) {
        if constexpr (has_tile(s, DIRECT, sizeof(T))) f(Tag<typename Tile<T, s, DIRECT>::type>{});
    };
    switch (shape) {
        case kLarge: return as(std::integral_constant<int, kLarge>{});
        case kTall: return as(std::integral_constant<int, kTall>{});
        case kWide: return as(std::integral_constant<int, kWide>{});
        case kSmall: return as(std::integral_constant<int, kSmall>{});
    }
    if constexpr (FEW) as(std::integral_constant<int, kFew>{});
}
template <typename T, typename F>
void with_tile(int shape, bool direct, F&& f) {
    if (direct) with_tile<T, true, true>(shape, f);
    else with_tile<T, false, true>(shape, f);
}

template <typename P>
struct Shape;
template <typename T, int BL_, int BR_, int WL_, int WR_, Layout LL, Layout LR>
struct Shape<RowProduct<T, BL_, BR_, WL_, WR_, LL, LR>> {
    using type = T;
    using columns = RowProduct<T, BL_, BR_, WL_, WR_, kDirect, kColumns>;
    static constexpr int BL = BL_, BR = BR_, WL = WL_, WR = WR_;
    static constexpr int kSlab = BR / WR;    // columns of one wave
    static constexpr bool kDirectRows = LL == kDirect;
    static constexpr int kShape = BL == 256 ? kLarge : BL == 192 ? kTall : BL == 32 ? kFew : BR == 160 ? kWide : kSmall;
};

// Where a wave's part of the tile lies.
template <typename P>
struct Part {
    using S = Shape<P>;
    // workgroup b of n
    int64_t l, r;             // the lane's: l of acc[.][0], r of acc[0][.] element 0
    int64_t l0, r0;           // the tile's
    int64_t lw, rw;           // the wave's
    int lane, wave;
    __device__ __forceinline__ Part(const ProductArgs& a, int64_t b, int64_t n) {
        int64_t tl, tr;
        tile_of<kGroup>(b, n, a.tiles_l, a.tiles_r, tl, tr);
        lane = threadIdx.x % kWave;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        l0 = tl * S::BL;
        r0 = tr * S::BR;
        lw = l0 + wave % S::WL * (S::BL / S::WL);
        rw = r0 + wave / S::WL * S::kSlab;
        l = lw + lane % 16;
        r = rw + 4 * (lane / 16);
    }
    // The place of column v (any number) from the lane's r on: 16 i + e of acc[i][.][e], or one
    // that no e has.
    __device__ __forceinline__ int place(int64_t v) const {
        return v >= r && v < r + S::kSlab ? static_cast<int>(v - r) : -1;
    }
    // Whether the lane's tiles hold column v of nr.
    __device__ __forceinline__ bool holds(int64_t v, int64_t nr) const {
        return v >= r && v < rw + S::kSlab && v < nr && (v - r) % 16 < 4;
    }
};

// ---- forward -----------------------------------------------------------------

// With |l| in units of log2 below this, fma(product, c, -l') is off by 2^-5 at most where l' is l
// rounded. Beyond, that error grows until the power overflows (from 2^31 on, where half a step is
// 2^7), and c times a product may overflow where the logit does not: there logits are subtracted
// before they are scaled.
constexpr float kFar = 0x1p20f;
__device__ __forceinline__ bool is_far(float l) { return !(__builtin_fabsf(l) < kFar); }      // NaN too

struct LossArgs {
    float s, c;               // logit_scale, and times log2(e)
    int64_t first;            // vocabulary row of the piece's first
    int64_t m0;               // row of the rows' first
    const void* targets;
    bool wide;
    float2* part;             // [slab][nl]
    float* at_target;         // [M]
};

__device__ __forceinline__ int64_t target_of(const void* t, bool wide, int64_t m) {
    return wide ? static_cast<const int64_t*>(t)[m] : static_cast<const int32_t*>(t)[m];
}

__device__ __forceinline__ float over_quads_max(float v) {
    v = __builtin_fmaxf(v, __shfl_xor(v, 16));
    return __builtin_fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float over_quads_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <typename P>
__global__ __launch_bounds__(P::kThreads) void head_loss_kernel(ProductArgs a, LossArgs h) {
    using S = Shape<P>;
    __shared__ __align__(1024) char lds[P::kLds];
    const Part<P> at(a, blockIdx.x, gridDim.x);
    v4f acc[P::kTR][P::kTL];
    P::run(a, at.l0, at.r0, 0, a.kbytes, lds, acc);
    if (at.rw >= a.nr) return;
    const bool whole = at.rw + S::kSlab <= a.nr;
    float s = h.s, c = h.c;
    // s > 0 below, and every value counts: the few waves that are not so make it so
    if (!whole || !(s > 0.0f)) {
        const int valid = whole ? S::kSlab : static_cast<int>(a.nr - at.r);       // from the lane's r on
#pragma unroll
        for (int j = 0; j < P::kTL; j++)
#pragma unroll
            for (int i = 0; i < P::kTR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][j][e] = 16 * i + e < valid ? acc[i][j][e] * s : -INFINITY;
        s = 1.0f;
        c = kLog2e;
    }
#pragma unroll
    for (int j = 0; j < P::kTL; j++) {
        const int64_t m = at.l + 16 * j;
        const bool in = m < a.nl;
        const int64_t v = in ? target_of(h.targets, h.wide, h.m0 + m) - h.first : -1;
        float most = acc[0][j][0];
#pragma unroll
        for (int i = 0; i < P::kTR; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) most = __builtin_fmaxf(most, acc[i][j][e]);
        most = over_quads_max(most);
        // one wave in V / kSlab has a row's target
        if (const bool here = at.holds(v, a.nr); wave_any(here)) {
            const int hit = at.place(v);
            float own = 0.0f;
#pragma unroll
            for (int i = 0; i < P::kTR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) own = hit == 16 * i + e ? acc[i][j][e] : own;
            if (here) h.at_target[h.m0 + m] = own * s;
        }
        const float top = most * s, top2 = most * c;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < P::kTR; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) sum += ex2(__builtin_fmaf(acc[i][j][e], c, -top2));
        // from the roundings of top2 to those of top
        sum *= ex2(__builtin_fmaf(__builtin_fmaf(most, s, -top), kLog2e, -__builtin_fmaf(most, c, -top2)));
        if (const bool far = is_far(top2); wave_any(far)) {
            // equal ones count 1, infinite ones too: a slab of logits -inf leaves (-inf, their number),
            // which the join takes as nothing beside a finite one
            float apart = 0.0f;
#pragma unroll
            for (int i = 0; i < P::kTR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    apart += ex2(acc[i][j][e] == most ? 0.0f : (acc[i][j][e] - most) * c);
            sum = far ? apart : sum;
        }
        sum = over_quads_sum(sum);
        if (at.lane < 16 && in) h.part[at.rw / S::kSlab * a.nl + m] = make_float2(top, sum);
    }
}

struct JoinArgs {
    const float2* part;       // [slabs][rows]
    int64_t slabs, rows, m0, V;
    const float* at_target;
    const void* targets;
    bool wide;
    float* loss;
    float* lse;
};

__device__ __forceinline__ void join(float& top, float& sum, float2 p) {
    const float t = __builtin_fmaxf(top, p.x);
    // equal infinities, whose difference is NaN, are taken as they are
    const float from = top == t ? sum : sum * ex2((top - t) * kLog2e);
    const float add = p.x == t ? p.y : p.y * ex2((p.x - t) * kLog2e);
    sum = from + add;
    top = t;
}

// ROWS rows to a workgroup of 256 / ROWS threads each.
template <int ROWS>
__global__ __launch_bounds__(256) void head_join_kernel(JoinArgs h) {
    constexpr int kTeam = 256 / ROWS;
    __shared__ float2 team[kTeam][ROWS];
    const int row = threadIdx.x % ROWS, member = threadIdx.x / ROWS;
    const int64_t m = blockIdx.x * int64_t{ROWS} + row;
    float top = -INFINITY, sum = 0.0f;
    if (m < h.rows) {
        int64_t s = member;
        for (; s + 3 * kTeam < h.slabs; s += 4 * kTeam) {
            float2 p[4];
#pragma unroll
            for (int i = 0; i < 4; i++) p[i] = h.part[(s + i * kTeam) * h.rows + m];
#pragma unroll
            for (int i = 0; i < 4; i++) join(top, sum, p[i]);
        }
        for (; s < h.slabs; s += kTeam) join(top, sum, h.part[s * h.rows + m]);
    }
    team[member][row] = make_float2(top, sum);
    for (int d = kTeam / 2; d > 0; d /= 2) {
        __syncthreads();
        if (member < d) {
            join(top, sum, team[member + d][row]);
            team[member][row] = make_float2(top, sum);
        }
    }
    if (member != 0 || m >= h.rows) return;
    const float lse = __builtin_fmaf(log2f(sum), kLn2, top);
    const int64_t at = h.m0 + m, t = target_of(h.targets, h.wide, at);
    h.lse[at] = lse;
    h.loss[at] = t >= 0 && t < h.V ? lse - h.at_target[at] : 0.0f;
}

// ---- copies ---------------------------------------------------------------------

// A wave to a row, four waves to a workgroup, workgroups in turn where there are more rows.
__device__ __forceinline__ int64_t first_row() { return blockIdx.x * int64_t{4} + threadIdx.x / kWave; }
__device__ __forceinline__ int64_t rows_apart() { return gridDim.x * int64_t{4}; }
uint32_t row_groups(int64_t rows) {
    return static_cast<uint32_t>(rows < (int64_t{1} << 22) ? ceil_div(rows, 4) : int64_t{1} << 20);
}

// Rows of n values to rows of ld_out values, zeros behind.
template <typename T>
__global__ __launch_bounds__(256) void pad_rows_kernel(const T* in, int64_t ld_in, int64_t rows, int64_t n, T* out,
                                                       int64_t ld_out) {
    constexpr int V = 16 / sizeof(T);           // ld_out is a multiple
    for (int64_t row = first_row(); row < rows; row += rows_apart())
        for (int64_t c = threadIdx.x % kWave * V; c < ld_out; c += kWave * V) {
            RowVec<T, V> v;
            v.load(in + row * ld_in, static_cast<int>(c), static_cast<int>(n));
            v.template store<false>(out + row * ld_out + c, 0, V);
        }
}

// in (rows, n) to out (n, ld_out), ld_out >= rows, zeros behind and in the
// columns of rows that are off (t < 0).  A tile of 64 x 64 values goes through
// LDS, read and written in pieces of 16 bytes (at any element in `in`, whole lines
// of out, whose rows are a multiple of 64 values long).
template <typename T>
__global__ __launch_bounds__(256) void transpose_kernel(const T* in, int64_t ld_in, int64_t rows, int64_t n, T* out,
                                                        int64_t ld_out, const int* t) {
    constexpr int kTile = 64, V = 16 / sizeof(T), kPieces = kTile / V;
    // one word (or a half) more than a multiple of the banks: neighbours along r are in different ones
    __shared__ T tile[kTile][kTile + 4 / sizeof(T)];
    const int64_t across = (n + kTile - 1) / kTile;
    const int64_t r0 = blockIdx.x / across * kTile, c0 = blockIdx.x % across * kTile;
#pragma unroll
    for (int k = 0; k < kTile * kPieces / 256; k++) {
        const int at = k * 256 + threadIdx.x, y = at / kPieces, x = at % kPieces * V;
        const int64_t r = r0 + y, c = c0 + x;
        RowVec<T, V> v;
        v.zero();
        if (r < rows && c < n && (!t || t[r] >= 0)) v.load(in + r * ld_in + c, 0, n - c < V ? static_cast<int>(n - c) : V);
#pragma unroll
        for (int e = 0; e < V; e++) tile[y][x + e] = v.t[e];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTile * kPieces / 256; k++) {
        const int at = k * 256 + threadIdx.x, y = at / kPieces, x = at % kPieces * V;
        const int64_t c = c0 + y, r = r0 + x;
        RowVec<T, V> v;
#pragma unroll
        for (int e = 0; e < V; e++) v.t[e] = tile[x + e][y];
        if (c < n && r < ld_out) v.template store<false>(out + c * ld_out + r, 0, V);
    }
}

// ---- backward --------------------------------------------------------------------

// What a row brings to dl: a = (dloss + dlse) s, b = dloss s, its lse and its
// target (-1: a padded row, all zeros); and the power of 2 that brings its own
// |dloss| + |dlse| times s to 2^12 .. 2^13 (1 for the largest).
struct RowGrads {
    float* a;
    float* b;
    float* lse;
    int* t;
    float* lift;
    float* back;              // [0]: logit_scale / s
};

constexpr float kMostDl = 8190.0f;       // rounds to less than 2^13 in every type

constexpr int kTops = 256;
constexpr int64_t kRowsEach = 16384;

// Of a workgroup's 1024 threads.
__device__ __forceinline__ float largest_of_all(float top, float* most) {
    for (int d = 32; d > 0; d /= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d));
    if (threadIdx.x % kWave == 0) most[threadIdx.x / kWave] = top;
    __syncthreads();
    for (int w = 0; w < 16; w++) top = __builtin_fmaxf(top, most[w]);
    return top;
}

// The largest |dloss| + |dlse| of the rows that count, for all threads of the workgroup:
// the `first` 1024 rows and every `apart` times 1024 behind them.
__device__ __forceinline__ float largest(const HeadArgs& h, int64_t first, int64_t apart) {
    constexpr int kAhead = 8;
    __shared__ float most[16];
    float top = 0.0f;
    for (int64_t m0 = first * 1024 + threadIdx.x; m0 < h.M; m0 += 1024 * kAhead * apart) {
        int64_t t[kAhead];
        float up[kAhead], more[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int64_t m = m0 + 1024 * apart * i;
            const bool in = m < h.M;
            t[i] = in ? target_of(h.targets, h.wide_ids, m) : -1;
            up[i] = in ? h.dloss[m] : 0.0f;
            more[i] = in && h.dlse ? h.dlse[m] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; i++)
            if (t[i] >= 0 && t[i] < h.V)
                top = __builtin_fmaxf(top, __builtin_fabsf(up[i]) + __builtin_fabsf(more[i]));
    }
    return largest_of_all(top, most);
}

// Of many rows, for row_grads_kernel: kTops workgroups leave a value each.
__global__ __launch_bounds__(1024) void row_tops_kernel(HeadArgs h, float* tops) {
    const float top = largest(h, blockIdx.x, kTops);
    if (threadIdx.x == 0) tops[blockIdx.x] = top;
}

// 1024 rows to a workgroup.  Up to kRowsEach rows each workgroup finds the largest factor
// of all for itself (12 to 16 bytes a row, from L2): one launch, and no wait between
// workgroups.  With more it takes it from `tops` (8192 rows: 5.2 us against 3.6 + 3.2 and
// the launch; 32768: 10.9 and 3.6 + 3.4).
__global__ __launch_bounds__(1024) void row_grads_kernel(HeadArgs h, RowGrads g, const float* tops) {
    __shared__ float most[16];
    const float top = tops ? largest_of_all(threadIdx.x < kTops ? tops[threadIdx.x] : 0.0f, most) : largest(h, 0, 1);
    // 1 where nothing or not a number would come of it; bounded, so that 1 / s is a normal number
    float s = 1.0f;
    if (top > 0.0f && top < INFINITY) s = __builtin_fminf(kMostDl / top, 0x1p120f);
    if (blockIdx.x == 0 && threadIdx.x == 0) g.back[0] = h.logit_scale / s;
    const int64_t m = blockIdx.x * int64_t{1024} + threadIdx.x;
    if (m >= h.M) return;
    const int64_t t = target_of(h.targets, h.wide_ids, m);
    const bool on = t >= 0 && t < h.V;
    const float up = on ? h.dloss[m] : 0.0f;
    g.a[m] = on ? (up + (h.dlse ? h.dlse[m] : 0.0f)) * s : 0.0f;
    g.b[m] = up * s;
    const float size = on ? (__builtin_fabsf(up) + (h.dlse ? __builtin_fabsf(h.dlse[m]) : 0.0f)) * s : 0.0f;
    int e = 12;
    if (size > 0.0f && size < INFINITY) e = ilogbf(size);
    g.lift[m] = ldexpf(1.0f, e < -88 ? 100 : 12 - e);
    g.lse[m] = on ? h.lse[m] : 0.0f;
    g.t[m] = on ? static_cast<int>(t) : -1;
}

template <typename T>
constexpr bool kLifted = std::is_same_v<T, f16>;      // the others have fp32's exponents

struct DlArgs {
    float s, c;               // logit_scale, and times log2(e)
    int64_t first;
    RowGrads g;
    void* dl;                 // (M, ld_dl)
    void* dlt;                // (piece, ld_dlt)
    int64_t ld_dl, ld_dlt;
};

// The store of dl^T: the tiles along r that fit the stages' LDS at a time.
template <typename P>
using Transposed = ColStore<typename Shape<P>::type, P::kTR, P::kTL,
                            P::kTR % 4 == 0 && sizeof(typename Shape<P>::type) == 2 ? 4 : P::kTR % 2 == 0 ? 2 : 1>;

template <typename P>
__global__ __launch_bounds__(P::kThreads) void head_dl_kernel(ProductArgs a, DlArgs h) {
    using T = typename Shape<P>::type;
    using Rows = RowStore<T, P::kTR, P::kTL>;
    using Cols = Transposed<P>;
    typedef T quad __attribute__((ext_vector_type(4)));
    constexpr int kStore = Rows::kBytes > Cols::kBytes ? Rows::kBytes : Cols::kBytes;
    static_assert(P::kWaves * kStore <= P::kLds, "stored through the stages' LDS");
    __shared__ __align__(1024) char lds[P::kLds];
    const Part<P> at(a, blockIdx.x, gridDim.x);
    constexpr int kPadded = -2;
    int hit[P::kTL];
    float up[P::kTL], own[P::kTL], lse[P::kTL], lift[P::kTL];
    // ahead of the product where its registers leave room
    constexpr bool kAhead = sizeof(T) == 2 && Shape<P>::kDirectRows;
    const auto read_rows = [&] {
#pragma unroll
        for (int j = 0; j < P::kTL; j++) {
            const int64_t m = at.l + 16 * j;
            const bool in = m < a.nl;
            const int t = in ? h.g.t[m] : -1;
            hit[j] = t < 0 ? kPadded : at.place(t - h.first);
            up[j] = in ? h.g.a[m] : 0.0f;
            own[j] = in ? h.g.b[m] : 0.0f;
            lse[j] = in ? h.g.lse[m] : 0.0f;
        }
    };
    const auto read_lift = [&] {
#pragma unroll
        for (int j = 0; j < P::kTL; j++) lift[j] = at.l + 16 * j < a.nl ? h.g.lift[at.l + 16 * j] : 0.0f;
    };
    if constexpr (kAhead) read_rows();
    if constexpr (kAhead && kLifted<T>) read_lift();
    v4f acc[P::kTR][P::kTL];
    P::run(a, at.l0, at.r0, 0, a.kbytes, lds, acc);
    if constexpr (!kAhead) read_rows();
#pragma unroll
    for (int j = 0; j < P::kTL; j++) {
        if (const bool far = is_far(lse[j]); wave_any(far)) {
            // the logit is rounded as the forward rounds it, and not into the difference
#pragma clang fp contract(off)
#pragma unroll
            for (int i = 0; i < P::kTR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float l = acc[i][j][e] * h.s;
                    const float x = far ? (l - lse[j]) * kLog2e : __builtin_fmaf(acc[i][j][e], h.c, -lse[j] * kLog2e);
                    acc[i][j][e] = ex2(x) * up[j];
                }
        } else {
            const float lse2 = lse[j] * kLog2e;
#pragma unroll
            for (int i = 0; i < P::kTR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][j][e] = ex2(__builtin_fmaf(acc[i][j][e], h.c, -lse2)) * up[j];
        }
        if (wave_any(hit[j] >= 0)) {
#pragma unroll
            for (int i = 0; i < P::kTR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][j][e] -= hit[j] == 16 * i + e ? own[j] : 0.0f;
        }
        // a padded row's x counts as zeros (ProductArgs::off) and its up is 0, but 0 times an infinite
        // weight is NaN
        if (wave_any(hit[j] == kPadded)) {
#pragma unroll
            for (int i = 0; i < P::kTR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][j][e] = hit[j] == kPadded ? 0.0f : acc[i][j][e];
        }
    }
    if (at.rw + 16 * P::kTR > a.nr || at.lw + 16 * P::kTL > a.nl) {
        // zeros past the piece and past the rows, where the last ones were read again
#pragma unroll
        for (int j = 0; j < P::kTL; j++)
#pragma unroll
            for (int i = 0; i < P::kTR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (at.r + 16 * i + e >= a.nr || at.l + 16 * j >= a.nl) acc[i][j][e] = 0.0f;
    }
    const auto get = [&](int i, int j) {
        quad v;
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = static_cast<T>(acc[i][j][e]);
        return v;
    };
    if constexpr (!kAhead && kLifted<T>) read_lift();
    __syncthreads();          // the last stage is read
    char* mine = lds + at.wave * kStore;
    Rows::run(mine, at.lane, static_cast<T*>(h.dl) + at.lw * h.ld_dl + at.rw, h.ld_dl, a.nl - at.lw, h.ld_dl - at.rw,
              [&](int i, int j) {
                  if constexpr (!kLifted<T>) return get(i, j);
                  quad v;
#pragma unroll
                  for (int e = 0; e < 4; e++) v[e] = static_cast<T>(acc[i][j][e] * lift[j]);
                  return v;
              });
    Cols::run(mine, at.lane, static_cast<T*>(h.dlt) + at.rw * h.ld_dlt + at.lw, h.ld_dlt, h.ld_dlt - at.lw, a.nr - at.rw,
              get);
}

struct GradArgs {
    const float* back;
    void* out;                // (nl, ld) of T; or null:
    int64_t ld;
    float* acc;               // [split][nl][ld] fp32, ld a multiple of 4; added to unless it is the first piece
    bool first;
    int split;                // of K
    const int* t;             // rows of out with t < 0 are zeros, whatever the weight (null: none)
    const float* lift;        // out's rows are to be divided by (null: 1)
};

// The products of a piece, dx's and dW's, in one launch, the tiles of the longer K
// first: those of the other fill the CUs that a last, partial round would leave idle.
struct TwoProducts {
    ProductArgs a[2];
    GradArgs g[2];
    int64_t first;            // workgroups of the first
    bool dx;                  // which of them is dx's
};

// COLUMNS: dx's product reads W as it lies, K down its rows.
template <typename P, bool COLUMNS>
__global__ __launch_bounds__(P::kThreads) void head_grad_kernel(TwoProducts two) {
    using T = typename Shape<P>::type;
    using Rows = RowStore<T, P::kTR, P::kTL>;
    typedef T quad __attribute__((ext_vector_type(4)));
    static_assert(P::kWaves * Rows::kBytes <= P::kLds, "stored through the stages' LDS");
    __shared__ __align__(1024) char lds[P::kLds];
    const bool second = blockIdx.x >= two.first;
    const ProductArgs a = two.a[second];
    const GradArgs h = two.g[second];
    // a product's workgroups: the tiles, for every part of K
    const int64_t b = second ? blockIdx.x - two.first : blockIdx.x, tiles = a.tiles_l * a.tiles_r;
    const int64_t part = b / tiles;
    const Part<P> at(a, b - part * tiles, tiles);
    v4f acc[P::kTR][P::kTL];
    // this workgroup's part of K, whole stages
    const int64_t stages = (a.kbytes + kStage - 1) / kStage;
    const int64_t k0 = stages * part / h.split * kStage, k1 = stages * (part + 1) / h.split * kStage;
    if (COLUMNS && second == two.dx) {
        if constexpr (COLUMNS) Shape<P>::columns::run(a, at.l0, at.r0, k0, k1 < a.kbytes ? k1 : a.kbytes, lds, acc);
    } else {
        P::run(a, at.l0, at.r0, k0, k1 < a.kbytes ? k1 : a.kbytes, lds, acc);
    }
    if (!h.out) {
        // fp32 sums: a lane's four are 16 bytes of a row
        float* to = h.acc + (part * a.nl + at.l) * h.ld + at.r;
#pragma unroll
        for (int j = 0; j < P::kTL; j++) {
            if (at.l + 16 * j >= a.nl) continue;
#pragma unroll
            for (int i = 0; i < P::kTR; i++) {
                if (at.r + 16 * i >= a.nr) continue;
                v4f* p = reinterpret_cast<v4f*>(to + 16 * j * h.ld + 16 * i);
                *p = h.first ? acc[i][j] : *p + acc[i][j];
            }
        }
        return;
    }
    float back[P::kTL];
    bool on[P::kTL];
#pragma unroll
    for (int j = 0; j < P::kTL; j++) {
        const int64_t l = at.l + 16 * j;
        on[j] = !h.t || (l < a.nl && h.t[l] >= 0);
        back[j] = h.back[0];
        if constexpr (kLifted<T>) back[j] /= h.lift && l < a.nl ? h.lift[l] : 1.0f;
    }
    __syncthreads();          // the last stage is read
    Rows::run(lds + at.wave * Rows::kBytes, at.lane, static_cast<T*>(h.out) + at.lw * h.ld + at.rw, h.ld, a.nl - at.lw,
              a.nr - at.rw, [&](int i, int j) {
                  quad v;
#pragma unroll
                  for (int e = 0; e < 4; e++) v[e] = static_cast<T>(on[j] ? acc[i][j][e] * back[j] : 0.0f);
                  return v;
              });
}

// out = back * the sum of the parts of K, 16 bytes of them to a lane; zeros in rows with t < 0,
// other rows divided by their lift.
template <typename T>
__global__ __launch_bounds__(256) void head_finish_kernel(const float* acc, int64_t ld_acc, int split, int64_t rows,
                                                          int64_t n, const float* back, const int* t,
                                                          const float* lift, T* out, int64_t ld) {
    for (int64_t row = first_row(); row < rows; row += rows_apart()) {
        const bool on = !t || t[row] >= 0;
        const float s = lift ? back[0] / lift[row] : back[0];
        for (int64_t c = threadIdx.x % kWave * 4; c < n; c += kWave * 4) {
            v4f v = {0, 0, 0, 0};
            for (int k = 0; k < split; k++) v += *reinterpret_cast<const v4f*>(acc + (k * rows + row) * ld_acc + c);
            RowVec<T, 4> o;
#pragma unroll
            for (int e = 0; e < 4; e++) o.set(e, on ? v[e] * s : 0.0f);
            o.template store<false>(out + row * ld, static_cast<int>(c), static_cast<int>(n));
        }
    }
}

// ---- plans -------------------------------------------------------------------------

constexpr int64_t kPartBytes = int64_t{256} << 20;      // partial sums of the forward at a time
// dl and its transpose take 1 GiB, with many rows what 3328 vocabulary rows take, up to 8:
// every piece reads and writes dx's sums (both gradients, M262144 V32768 D1536 bf16: 79 ms,
// with 1 GiB 96; M400000 V10000 D768 fp16 22 and 32).
constexpr int64_t kDlBytes = int64_t{1} << 30, kMostDlBytes = int64_t{8} << 30, kDlColumns = 3328;

int64_t align_up(int64_t n, int64_t a) { return ceil_div(n, a) * a; }

// What the tile shapes take on this card, in microseconds: a value of K of one
// tile, with as many workgroups on a CU as `slots` says for all of them, and a
// tile's start and end.  Measured in bf16 with 8192 x 32768 x 1536: 1218, 1123, 1063
// and 1006 TFLOP/s; in fp32 (4096 x 32768 x 1024) 213, 200, 189 and 181.  The best shape
// changes with the size: fp16, 1551 x 10007 x 1001 take 76, 78, 66 and 75 us.  kFew is
// bound by what it reads, and is taken by the number of rows.
struct TileCost {
    int64_t nl, nr, slots;
    double each, fixed;
};
TileCost tile_cost(int shape, int64_t elem) {
    constexpr TileCost costs[] = {{256, 256, 256, 0.0274, 5.0}, {192, 320, 256, 0.0274, 5.0},
                                  {128, 160, 512, 0.0192, 4.0}, {128, 128, 512, 0.0161, 4.0},
                                  {32, 128, 1024, 0.0161, 4.0}};
    TileCost c = costs[shape];
    if (elem == 4) c.each *= 5.8;
    return c;
}
constexpr int64_t kFewRows = 32;

// `n` tiles that take `us` each, on CUs that took `m` tiles of `first` each before.
double spread(int64_t slots, int64_t m, double first, int64_t n, double us) {
    const int64_t q = m / slots, r = m % slots;
    double most = q * first + (r ? first : 0.0);
    // slots - r are free at q first, r of them a tile later: k tiles to each of the earlier ones
    for (int64_t k = n / slots; n > 0; k++) {
        const double end = q * first + k * us;
        const int64_t later = end > (q + 1) * first ? static_cast<int64_t>((end - (q + 1) * first) / us + 1e-9) : 0;
        if ((slots - r) * k + r * later >= n) return end > most ? end : most;
    }
    return most;
}

struct Choice {
    double us;
    int shape;
};
// A product of nl x nr with K = k.
Choice product_us(int64_t elem, int64_t nl, int64_t nr, int64_t k, bool direct = true) {
    Choice best{0, -1};
    for (int shape = 0; shape < kFew; shape++) {
        if (!has_tile(shape, direct, elem)) continue;
        const TileCost c = tile_cost(shape, elem);
        const double us = spread(c.slots, 0, 0, ceil_div(nl, c.nl) * ceil_div(nr, c.nr), c.each * k + c.fixed);
        if (best.shape < 0 || us < best.us) best = {us, shape};
    }
    if (nl <= kFewRows) best.shape = kFew;
    return best;
}

// dx (M, D) with K = n in `split` parts, and dW (n, D) with K = M in split_w.
Choice gradients_us(int64_t elem, int64_t M, int64_t n, int64_t D, int64_t split, int64_t split_w, bool columns) {
    Choice best{0, -1};
    for (int shape = 0; shape < kFew; shape++) {
        if (columns && !has_columns(shape, elem)) continue;
        const TileCost c = tile_cost(shape, elem);
        const int64_t wide = ceil_div(D, c.nr), x = ceil_div(M, c.nl) * wide * split,
                      w = ceil_div(n, c.nl) * wide * split_w;
        const double ux = (!columns ? 1.0 : elem == 2 ? 1.35 : 2.3) * c.each * n / split + c.fixed,
                     uw = c.each * M / split_w + c.fixed;
        const double us = ux >= uw ? spread(c.slots, x, ux, w, uw) : spread(c.slots, w, uw, x, ux);
        if (best.shape < 0 || us < best.us) best = {us, shape};
    }
    return best;
}

// Rows that are not a multiple of 16 bytes long are copied to rows that are where
// there are so many that the copy of W costs less than reading it through registers
// (bf16, V32768, forward: M8192 D1535 880 us through registers, 741 copied; M2048 D769
// 130 and 131; fp16 M1551 V10007 D1001 85 and 66).
constexpr int64_t kCopyRows = 1024;
// Below as many rows dx's product reads W as it lies, down its columns: slower, but W
// is not transposed first (bf16, both gradients: M16 V65536 D2560 292 us against 428, M517
// V50021 D1536 380 and 399, M1000 V32768 D1536 359 and 387, M1100 441 and 461, M1536 540
// and 535, M2048 719 and 681; M1280 V50304 D768 420 and 396).  In fp32 its 4-byte LDS reads
// take 2.3 times as long: below 256 rows (M128 V65536 D2560 949 us against 1158, M250 V50021
// D1536 782 and 876, M517 1623 and 1611).
constexpr int64_t kColumnRows = 1024, kColumnRowsWide = 256;

struct Plan {
    bool copied, columns;     // columns: where W's rows lie at multiples of 16 bytes
    int64_t Dk;               // values in a row that the products read
    int64_t piece;            // vocabulary rows at a time
    int64_t chunk;            // rows at a time (forward)
    int split, split_w;       // parts of dx's K and of dW's
    bool accumulate;          // dx goes through fp32 partial sums (and dW where split_w > 1)
    int64_t ld_m;             // values in a row of dl^T and x^T
    int64_t ld_acc;           // and of the partial sums
    int64_t x, w, part, at_target, dl, dlt, xt, wt, acc, acc_w, rows, bytes;
};

bool plan_of(int dtype, int64_t M, int64_t V, int64_t D, bool backward, Plan& p) {
    const int64_t e = dtype == MSS_F32 ? 4 : 2;
    p = Plan{};
    p.copied = D * e % 16 != 0 && M >= kCopyRows;
    p.Dk = p.copied ? align_up(D, 16 / e) : D;
    p.columns = M < (e == 2 ? kColumnRows : kColumnRowsWide) && D * e % 16 == 0;
    p.ld_m = align_up(M, kPadRows);
    bool fits = true;
    const auto take = [&](int64_t a, int64_t b, int64_t c) {
        const int64_t here = p.bytes;
        int64_t n = a;
        for (int64_t f : {b, c}) {
            if (f > 0 && n > (int64_t{1} << 60) / f) fits = false;
            else n *= f;
        }
        if (fits) p.bytes += align_up(n, 256);
        if (p.bytes > (int64_t{1} << 60)) fits = false;
        return here;
    };
    if (!backward) {
        p.piece = p.copied ? align_up((int64_t{64} << 20) / (p.Dk * e) + 1, 256) : int64_t{1} << 18;
        if (p.piece > (int64_t{1} << 18)) p.piece = int64_t{1} << 18;
        if (p.piece > V) p.piece = V;
        // the narrowest slab is 32 columns, of few rows, 64 otherwise; each piece ends in one of its own
        const int64_t slabs = ceil_div(V, M <= kFewRows ? 32 : 64) + ceil_div(V, p.piece);
        p.chunk = kPartBytes / (slabs * 8) / 256 * 256;
        if (p.chunk < 256) p.chunk = 256;
        if (p.chunk > M) p.chunk = M;
        p.part = take(slabs, p.chunk, 8);
        p.at_target = take(M, 4, 1);
        if (p.copied) {
            p.x = take(M, p.Dk, e);
            p.w = take(p.piece, p.Dk, e);
        }
        return fits;
    }
    // The piece, in steps of 256 vocabulary rows, and the parts of both K: what takes the least
    // time by the costs above, the traffic of the partial sums (5 TB/s) and launches counted in.
    // dW's K is split where a small vocabulary leaves it few tiles (bf16, M65536 V256 D1024: both
    // gradients 288 us, with K whole 1085; M4096 V1000 D512 50 and 74).
    const int64_t steps = ceil_div(V, 256);
    int64_t most = std::clamp(2 * e * p.ld_m * kDlColumns, kDlBytes, kMostDlBytes) / (2 * 256 * e * p.ld_m);
    for (int64_t bound : {int64_t{1024}, steps})
        if (most > bound) most = bound;
    if (most < 1) most = 1;
    const double pass = 4.0 * D / 5e6;              // of a row of sums, one part
    double best = 0;
    const int64_t stride = ceil_div(most, 32);
    for (int64_t n = most; n > 0 && n > most / 3; n -= stride) {
        const int64_t full = steps / n, rest = steps % n, pieces = full + (rest > 0);
        const int64_t tiles_w = ceil_div(256 * n, 128) * ceil_div(D, 128);
        const double before = full * product_us(e, M, 256 * n, D).us + 10.0 * pieces +
                              (rest ? product_us(e, M, 256 * rest, D).us : 0.0);
        for (int split_w = 1; split_w == 1 || (M / split_w >= 512 && tiles_w * split_w <= 1024); split_w *= 2)
            for (int split : {1, 2, 3, 4, 6, 8, 12, 16}) {
                if (split > 1 && 256 * n / split < 512) break;
                const bool sums = split > 1 || pieces > 1;
                double us = before + full * gradients_us(e, M, 256 * n, D, split, split_w, p.columns).us +
                            (sums ? pass * M * split * 2 * pieces : 0.0) +
                            (split_w > 1 ? (pass * 256 * n * split_w * 2 + 5.0) * pieces : 0.0);
                if (best != 0 && us >= best) continue;
                if (rest) us += gradients_us(e, M, 256 * rest, D, split, split_w, p.columns).us;
                if (best == 0 || us < best) best = us, p.piece = 256 * n, p.split = split, p.split_w = split_w;
            }
    }
    p.accumulate = p.split > 1 || p.piece < V;
    p.dl = take(M, p.piece, e);
    p.dlt = take(p.piece, p.ld_m, e);
    p.xt = take(D, p.ld_m, e);
    p.wt = take(D, p.piece, e);
    if (p.copied) {
        p.x = take(M, p.Dk, e);
        p.w = take(p.piece, p.Dk, e);
    }
    p.ld_acc = align_up(D, 4);
    if (p.accumulate) p.acc = take(M * int64_t{4}, p.ld_acc, p.split);
    if (p.split_w > 1) p.acc_w = take((V < p.piece ? V : p.piece) * int64_t{4}, p.ld_acc, p.split_w);
    p.rows = take(align_up(M, 64) * int64_t{20} + 256 + 4 * kTops, 1, 1);
    // the workgroups of the transposes are counted in 32 bits of threads
    return fits && (p.ld_m > p.piece ? p.ld_m : p.piece) / 64 * ceil_div(D, 64) < (int64_t{1} << 24);
}

template <typename F>
hipError_t by_type(int dtype, F&& f) {
    return dtype == MSS_F32 ? f(0.0f) : dtype == MSS_BF16 ? f(bf16{}) : f(f16{});
}

ProductArgs product(const void* l, int64_t ld_l, int64_t nl, const void* r, int64_t ld_r, int64_t nr, int64_t kbytes,
                    int shape, const int* off = nullptr) {
    const TileCost t = tile_cost(shape, 2);
    return {static_cast<const char*>(l), static_cast<const char*>(r), ld_l, ld_r, nl, nr, kbytes, off,
            ceil_div(nl, t.nl), ceil_div(nr, t.nr)};
}

// Whether rows of a product's operand can go straight to LDS.
bool direct(const void* p, int64_t ld, int64_t rows, int64_t n, int64_t e) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && n * e % 16 == 0 && (rows == 1 || ld * e % 16 == 0);
}

// Rows as the products read them: as they lie, or copied to `to`.
template <typename T>
hipError_t rows_of(const Plan& p, const T*& in, int64_t& ld, int64_t rows, int64_t n, char* to, hipStream_t st) {
    if (!p.copied) return hipSuccess;
    T* out = reinterpret_cast<T*>(to);
    pad_rows_kernel<T><<<row_groups(rows), 256, 0, st>>>(in, ld, rows, n, out, p.Dk);
    in = out;
    ld = p.Dk;
    return hipGetLastError();
}

template <typename T>
hipError_t transpose(const T* in, int64_t ld, int64_t rows, int64_t n, T* out, int64_t ld_out, const int* t,
                     hipStream_t st) {
    const int64_t blocks = ceil_div(ld_out, 64) * ceil_div(n, 64);
    transpose_kernel<T><<<static_cast<uint32_t>(blocks), 256, 0, st>>>(in, ld, rows, n, out, ld_out, t);
    return hipGetLastError();
}

template <typename T>
hipError_t finish(const float* acc, int64_t ld_acc, int split, int64_t rows, int64_t n, const float* back,
                  const int* t, const float* lift, T* out, int64_t ld, hipStream_t st) {
    head_finish_kernel<T><<<row_groups(rows), 256, 0, st>>>(acc, ld_acc, split, rows, n, back, t, lift, out, ld);
    return hipGetLastError();
}

template <typename T>
hipError_t forward(const HeadArgs& h, const Plan& p, hipStream_t st) {
    char* ws = static_cast<char*>(h.ws);
    constexpr int64_t e = sizeof(T);
    const T* x = static_cast<const T*>(h.x);
    int64_t ld_x = h.ld_x;
    const bool straight = p.copied || (direct(x, ld_x, h.M, h.D, e) && direct(h.w, h.ld_w, h.V, h.D, e));
    if (hipError_t r = rows_of(p, x, ld_x, h.M, h.D, ws + p.x, st)) return r;
    float* at_target = reinterpret_cast<float*>(ws + p.at_target);
    float2* part = reinterpret_cast<float2*>(ws + p.part);
    for (int64_t m0 = 0; m0 < h.M; m0 += p.chunk) {
        const int64_t rows = h.M - m0 < p.chunk ? h.M - m0 : p.chunk;
        const int shape = product_us(e, rows, h.V < p.piece ? h.V : p.piece, h.D, straight).shape;
        int64_t slabs = 0;
        for (int64_t v0 = 0; v0 < h.V; v0 += p.piece) {
            const int64_t n = h.V - v0 < p.piece ? h.V - v0 : p.piece;
            const T* w = static_cast<const T*>(h.w) + v0 * h.ld_w;
            int64_t ld_w = h.ld_w;
            if (hipError_t r = rows_of(p, w, ld_w, n, h.D, ws + p.w, st)) return r;
            const ProductArgs a = product(x + m0 * ld_x, ld_x * e, rows, w, ld_w * e, n, p.Dk * e, shape);
            const LossArgs l{h.logit_scale, h.logit_scale * kLog2e, v0, m0, h.targets, h.wide_ids,
                             part + slabs * rows, at_target};
            with_tile<T>(shape, straight, [&](auto tag) {
                using P = typename decltype(tag)::type;
                head_loss_kernel<P><<<static_cast<uint32_t>(a.tiles_l * a.tiles_r), P::kThreads, 0, st>>>(a, l);
                slabs += ceil_div(n, Shape<P>::kSlab);
            });
            if (hipError_t r = hipGetLastError()) return r;
        }
        const JoinArgs j{part, slabs, rows, m0, h.V, at_target, h.targets, h.wide_ids, h.loss, h.lse};
        if (rows < 1024) head_join_kernel<1><<<static_cast<uint32_t>(rows), 256, 0, st>>>(j);
        else head_join_kernel<16><<<static_cast<uint32_t>(ceil_div(rows, 16)), 256, 0, st>>>(j);
        if (hipError_t r = hipGetLastError()) return r;
    }
    return hipSuccess;
}

template <typename T>
hipError_t backward(const HeadArgs& h, const Plan& p, hipStream_t st) {
    char* ws = static_cast<char*>(h.ws);
    constexpr int64_t e = sizeof(T);
    const int64_t M = h.M, D = h.D;
    RowGrads g;
    const int64_t padded = align_up(M, 64);
    g.a = reinterpret_cast<float*>(ws + p.rows);
    g.b = g.a + padded;
    g.lse = g.b + padded;
    g.t = reinterpret_cast<int*>(g.lse + padded);
    g.lift = reinterpret_cast<float*>(g.t + padded);
    g.back = g.lift + padded;
    const float* lift = kLifted<T> ? g.lift : nullptr;
    float* tops = M > kRowsEach ? g.back + 64 : nullptr;
    if (tops) {
        row_tops_kernel<<<kTops, 1024, 0, st>>>(h, tops);
        if (hipError_t r = hipGetLastError()) return r;
    }
    row_grads_kernel<<<static_cast<uint32_t>(ceil_div(M, 1024)), 1024, 0, st>>>(h, g, tops);
    if (hipError_t r = hipGetLastError()) return r;
    const T* x = static_cast<const T*>(h.x);
    int64_t ld_x = h.ld_x;
    const bool straight = p.copied || (direct(x, ld_x, M, D, e) && direct(h.w, h.ld_w, h.V, D, e));
    if (hipError_t r = rows_of(p, x, ld_x, M, D, ws + p.x, st)) return r;
    T* xt = reinterpret_cast<T*>(ws + p.xt);
    T* wt = reinterpret_cast<T*>(ws + p.wt);
    T* dl = reinterpret_cast<T*>(ws + p.dl);
    T* dlt = reinterpret_cast<T*>(ws + p.dlt);
    if (h.dw)
        if (hipError_t r = transpose(x, ld_x, M, D, xt, p.ld_m, g.t, st)) return r;
    for (int64_t v0 = 0; v0 < h.V; v0 += p.piece) {
        const int64_t n = h.V - v0 < p.piece ? h.V - v0 : p.piece;
        const int64_t ld_n = align_up(n, kPadRows);      // at most the piece, a multiple of 256
        const T* w = static_cast<const T*>(h.w) + v0 * h.ld_w;
        int64_t ld_w = h.ld_w;
        if (hipError_t r = rows_of(p, w, ld_w, n, D, ws + p.w, st)) return r;
        int shape = product_us(e, M, n, D, straight).shape;
        const ProductArgs a = product(x, ld_x * e, M, w, ld_w * e, n, p.Dk * e, shape, g.t);
        const DlArgs d{h.logit_scale, h.logit_scale * kLog2e, v0, g, dl, dlt, ld_n, p.ld_m};
        with_tile<T>(shape, straight, [&](auto tag) {
            using P = typename decltype(tag)::type;
            head_dl_kernel<P><<<static_cast<uint32_t>(a.tiles_l * a.tiles_r), P::kThreads, 0, st>>>(a, d);
        });
        if (hipError_t r = hipGetLastError()) return r;
        const bool columns = p.columns && straight;
        if (h.dx && !columns)
            if (hipError_t r = transpose(w, ld_w, n, D, wt, ld_n, static_cast<const int*>(nullptr), st)) return r;
        shape = gradients_us(e, M, n, D, p.split, p.split_w, columns).shape;
        // whole 16 bytes of K: head_dl_kernel's tiles reach so far, and write zeros there
        const ProductArgs px = columns ? product(dl, ld_n * e, M, w, ld_w * e, D, n * e, shape)
                                       : product(dl, ld_n * e, M, wt, ld_n * e, D, align_up(n * e, 16), shape);
        const ProductArgs pw = product(dlt, p.ld_m * e, n, xt, p.ld_m * e, D, align_up(M * e, 16), shape);
        const GradArgs gx{g.back, p.accumulate ? nullptr : h.dx, p.accumulate ? p.ld_acc : h.ld_dx,
                          reinterpret_cast<float*>(ws + p.acc), v0 == 0, p.split, g.t, lift};
        T* dw = h.dw ? static_cast<T*>(h.dw) + v0 * h.ld_dw : nullptr;
        float* acc_w = reinterpret_cast<float*>(ws + p.acc_w);
        const bool sums_w = p.split_w > 1;
        const GradArgs gw{g.back, sums_w ? nullptr : dw, sums_w ? p.ld_acc : h.ld_dw, acc_w, true, p.split_w,
                          nullptr, nullptr};
        const int64_t nx = h.dx ? px.tiles_l * px.tiles_r * p.split : 0,
                      nw = dw ? pw.tiles_l * pw.tiles_r * p.split_w : 0;
        const TwoProducts two =
            n / p.split >= M / p.split_w ? TwoProducts{{px, pw}, {gx, gw}, nx, false} : TwoProducts{{pw, px}, {gw, gx}, nw, true};
        with_tile<T, true, false>(shape, [&](auto tag) {
            using P = typename decltype(tag)::type;
            const uint32_t grid = static_cast<uint32_t>(nx + nw);
            if constexpr (has_columns(Shape<P>::kShape, sizeof(T)))
                if (columns) return head_grad_kernel<P, true><<<grid, P::kThreads, 0, st>>>(two);
            head_grad_kernel<P, false><<<grid, P::kThreads, 0, st>>>(two);
        });
        if (hipError_t r = hipGetLastError()) return r;
        if (dw && sums_w)
            if (hipError_t r = finish(acc_w, p.ld_acc, p.split_w, n, D, g.back, nullptr, nullptr, dw, h.ld_dw, st))
                return r;
    }
    if (h.dx && p.accumulate)
        return finish(reinterpret_cast<const float*>(ws + p.acc), p.ld_acc, p.split, M, D, g.back, g.t, lift,
                      static_cast<T*>(h.dx), h.ld_dx, st);
    return hipSuccess;
}

__global__ __launch_bounds__(256) void zero_rows_kernel(char* p, int64_t rows, int64_t width, int64_t ld) {
    // bytes, in pieces of two: every element type's size is a multiple
    for (int64_t row = first_row(); row < rows; row += rows_apart())
        for (int64_t c = threadIdx.x % kWave * 2; c < width; c += kWave * 2)
            *reinterpret_cast<uint16_t*>(p + row * ld + c) = 0;
}

}  // namespace

bool head_workspace(int dtype, int64_t M, int64_t V, int64_t D, bool bwd, int64_t& bytes) {
    Plan p;
    bytes = 0;
    if (M == 0) return true;
    if (!plan_of(dtype, M, V, D, bwd, p)) return false;
    // every launch below 2^32 threads: 256 to a tile of 128 x 128 or more (or 32 x 128 of few rows), to
    // 64 x 64 values of a transposition and to four rows (of at most 2^26) of the others
    const int64_t across = ceil_div(bwd ? M : p.chunk, 128), down = ceil_div(p.piece, 128), wide = ceil_div(D, 128);
    const int64_t most = int64_t{1} << 24;
    if (across * down >= most || across * wide * (bwd ? p.split : 1) + down * wide >= most ||
        ceil_div(p.ld_m, 64) * ceil_div(D, 64) >= most || ceil_div(p.piece, 64) * ceil_div(D, 64) >= most)
        return false;
    bytes = p.bytes;
    return true;
}

hipError_t launch_head(const HeadArgs& a, hipStream_t st) {
    Plan p;
    if (!plan_of(a.dtype, a.M, a.V, a.D, false, p)) return hipErrorInvalidValue;
    return by_type(a.dtype, [&](auto t) { return forward<decltype(t)>(a, p, st); });
}

hipError_t launch_head_bwd(const HeadArgs& a, hipStream_t st) {
    if (a.M == 0) {
        if (!a.dw) return hipSuccess;
        const int64_t e = a.dtype == MSS_F32 ? 4 : 2;
        zero_rows_kernel<<<row_groups(a.V), 256, 0, st>>>(static_cast<char*>(a.dw), a.V, a.D * e, a.ld_dw * e);
        return hipGetLastError();
    }
    if (!a.dx && !a.dw) return hipSuccess;
    Plan p;
    if (!plan_of(a.dtype, a.M, a.V, a.D, true, p)) return hipErrorInvalidValue;
    return by_type(a.dtype, [&](auto t) { return backward<decltype(t)>(a, p, st); });
}

}  // namespace mss
