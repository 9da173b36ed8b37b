/*
 * mss.h -- C ABI of libmss: the data-parallel core of a Mamba-1 (S6) block on
 * AMD Instinct MI355X (gfx950), hand-written HIP.
 *
 * The operation is the one the pages of the npm package
 * "@seanhogg/builderforce-memory-engine" define in the diff
 * 2026.7.12 -> 2026.9.27, file src/training/mamba1_cpu.ts, function
 * mamba1CpuForward, steps 4 (causal depthwise conv1d), 5 (SiLU), 8 (selective
 * scan with softplus(delta), A = -exp(clamp(A_log, -10, 5)), exponential
 * discretisation, recurrence, y = sum_n C h + D u) and 9 (gate by SiLU(z)),
 * with the layouts listed in that file's header comment.  The GPU dispatch
 * of the same computation (conv1d_forward, forward_scan, forward_reduce and
 * the h_cache binding) is in the diff 2026.7.14 -> 2026.9.28, file
 * src/model/mamba1_block.ts, Mamba1Block.forward.
 *
 * Symbols: B = batch, L = seq_len, M = B * L, D = d_inner, N = d_state,
 * K = d_conv.  Row r = b * L + t.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers to dense, row-major fp32 arrays
 *     (the activations of the gated recurrence and the block norms, and the
 *     tables, rows and gradients at the ends of a model may be bf16 or fp16)
 *     on the current HIP device, allocated and owned by the caller.
 *     The library allocates nothing and never frees a caller buffer; the
 *     backward passes, mss_gated_scan, mss_head_loss and the calls on lists
 *     of gradients take a caller workspace.  Its only device state is the
 *     static scratch array of mss_selective_scan_backward_noalloc (and
 *     constants).
 *   - Every pointer must be 16-byte aligned (MSS_EALIGN otherwise), except
 *     the activation and B/C tensors of the *_strided entry points (4 bytes),
 *     the activations of the gated recurrence and the block norms when strides
 *     are given (their element), the tensors at the ends of a model as said
 *     there, reset flags (any) and workspaces (256).
 *   - Outputs may not overlap any input (MSS_EALIAS), except the state
 *     buffers of mss_selective_step and mss_gated_step, which are updated in
 *     place by design, and the residual stream of mss_add_norm and the tensors
 *     of mss_clip_grads, which may be.
 *   - Work is enqueued on `stream` (NULL = the null stream) and the call
 *     returns without synchronising.  Arguments are validated before any
 *     launch; a call that returns an error has written nothing.
 *   - A zero size (B, L or D = 0) is valid and launches nothing, except that
 *     a sequence of length 0 still defines h_last (= h0, or zeros).
 *   - Limits: 1 <= N <= 16; 1 <= K <= 8.  Dimensions are int64; element
 *     offsets are computed in 64 bits.
 *   - NaN or Inf inputs are outside the contract: the kernels terminate and
 *     write every output, but the values are unspecified.
 *   - Calls on different streams may run concurrently; they share nothing.
 */
#ifndef MSS_H
#define MSS_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MSS_VERSION 4

/* Status codes. */
#define MSS_OK 0
#define MSS_EINVAL (-1)     /* null required pointer, bad size or limit, bad struct_size, bad disc */
#define MSS_EALIGN (-2)     /* a pointer is not 16-byte aligned */
#define MSS_EALIAS (-3)     /* an output overlaps an input */
#define MSS_EWORKSPACE (-4) /* workspace NULL or smaller than mss_workspace_bytes */
#define MSS_EHIP (-5)       /* a HIP runtime call or kernel launch failed; see mss_last_hip_error */
#define MSS_ESCRATCH (-6)   /* needs more than MSS_NOALLOC_SCRATCH_BYTES (the *_noalloc entry point) */

/* Problem sizes.  `struct_size` must be sizeof(mss_dims): it guards against a
 * caller built against a different layout of this struct.
 *
 * Time split.  The recurrence of every (b, d) column runs sequentially in
 * time, and a Mamba-1 problem has few enough columns that the scans split
 * time into segments processed in parallel.  A segment that starts at
 * t0 > 0 rebuilds the state it starts from, h(t0-1), by replaying the
 * recurrence from h = 0 over a window [tw, t0): tw is the latest step from
 * which every state of the segment's columns has decayed by at least
 * 2^-MSS_REPLAY_DECAY_BITS (prod aBar = exp(A sum dv), decided from delta
 * alone), or tw = 0.  (A state that decays faster than the slowest one
 * joins the replay later, at the 8-step block from which its own decay
 * reaches the same bound.)  Relative to the plain sequential recurrence the
 * state at t >= t0 then lacks exactly
 *     prod_{s=tj..t} aBar_s[n] * h_{tj-1}[n]   <=   2^-MSS_REPLAY_DECAY_BITS |h_{tj-1}[n]|
 * per state n, where tj is the step its replay started from, and an output
 * y_t lacks sum_n C_t[n] times that (times SiLU(z_t)).  So the difference
 * from the sequential recurrence is bounded by 2^-MSS_REPLAY_DECAY_BITS
 * times the magnitude of the state at the replay start: only a state far
 * above the scale of the outputs shortly before a segment start could make
 * it visible.  Segment lengths depend on the shape (and flags) alone, never
 * on the device or the environment: mss_time_split reports them, and the
 * output bits are a function of the inputs and the shape.
 * MSS_FLAG_EXACT turns the split off: each channel tile scans its whole
 * sequence in one wave, so there is no replay and the result is the plain
 * recurrence in fp32, at the cost of parallelism (B * ceil(D/64) waves for
 * the scans, B * ceil(D/32) for the scan backward, B * H workgroups for the
 * SSD scan). */
#define MSS_REPLAY_DECAY_BITS 24
#define MSS_FLAG_EXACT 1
/* MSS_FLAG_CKPT8: state checkpoints every 8 steps, for the backward pass.
 * Forward calls: h_cache is (B, ceil(L/8), D, N) and holds the state entering
 * steps 0, 8, 16, ... (entry k = h_{8k-1}; entry 0 = h0, or 0) instead of
 * every step's state -- 8 bytes per (m, d) instead of 64.
 * mss_selective_scan_backward: the flag says that h_ckpt carries those
 * checkpoints (from a forward call with the same inputs); the backward then
 * starts every 8-step block from them instead of rebuilding the states, and
 * needs no checkpoint workspace (mss_workspace_bytes with the flag set
 * reports the smaller size).  Without the flag h_ckpt must be NULL. */
#define MSS_FLAG_CKPT8 2
typedef struct mss_dims {
    int32_t struct_size;
    int32_t flags;          /* 0, or MSS_FLAG_EXACT (any other bit: MSS_EINVAL) */
    int64_t batch;          /* B */
    int64_t seq_len;        /* L (ignored by mss_selective_step) */
    int64_t d_inner;        /* D */
    int64_t d_state;        /* N, 1..16 */
    int64_t d_conv;         /* K, 1..8 (ignored by mss_selective_scan) */
} mss_dims;

/* Discretisation of the input term (the caller must choose; no default).
 *   MSS_DISC_ZOH:   bBar = ((exp(dv*A) - 1) / A) * B, as the pages' scan
 *                   computes it (mamba1CpuForward step 8; its backward pass
 *                   differentiates the same form).
 *   MSS_DISC_EULER: bBar = dv * B (the simplified form). */
#define MSS_DISC_ZOH 0
#define MSS_DISC_EULER 1

/* Steps 4 + 5: u = SiLU(b_conv[d] + sum_{k<K, k<=t} w_conv[d*K + k] * x[b, t-k, d]).
 * Tap k = 0 multiplies the current step; there is no contribution from
 * before t = 0 of each batch row, and none across batch rows.
 *   x      (M, D)  in
 *   w_conv (D, K)  in
 *   b_conv (D)     in, may be NULL (= 0)
 *   u      (M, D)  out                                                      */
int mss_conv1d_silu(const mss_dims* dims, const float* x, const float* w_conv,
                    const float* b_conv, float* u, hipStream_t stream);

/* Steps 8 + 9 on a given u:
 *   dv = softplus(delta) = max(delta, 0) + log1p(exp(-|delta|))
 *   A[d,n] = -exp(clamp(A_log[d,n], -10, 5)),  aBar = exp(dv * A)
 *   h_t = aBar * h_{t-1} + bBar(disc) * u_t      (h_{-1} = h0, or 0)
 *   y_t = (D_vec[d] * u_t + sum_n C[r,n] * h_t[n]) * SiLU(z_t)
 *   u, delta, z, y (M, D);  A_log (D, N);  B, C (M, N);  D_vec (D);
 *   h0, h_last (B, D, N);  h_cache (B, L, D, N) = h_t after the update of step t.
 *   Optional (NULL allowed): D_vec (= 0), z (ungated output), h0 (= 0),
 *   h_cache, h_last.  Required: u, delta, A_log, B, C, y.
 *   Time is split into segments processed in parallel (see "Time split"
 *   above for what that drops, and MSS_FLAG_EXACT for the path without it);
 *   the result is otherwise the plain recurrence in fp32.                  */
int mss_selective_scan(const mss_dims* dims, int disc, const float* u, const float* delta,
                       const float* A_log, const float* B, const float* C, const float* D_vec,
                       const float* z, const float* h0, float* y, float* h_cache,
                       float* h_last, hipStream_t stream);

/* Steps 4, 5, 8 and 9 fused into one kernel: mss_conv1d_silu followed by
 * mss_selective_scan, without materialising u.  Same arguments and layouts;
 * x (M, D), w_conv (D, K), b_conv (D, may be NULL) replace u.             */
int mss_mamba1_core(const mss_dims* dims, int disc, const float* x, const float* w_conv,
                    const float* b_conv, const float* delta, const float* A_log,
                    const float* B, const float* C, const float* D_vec, const float* z,
                    const float* h0, float* y, float* h_cache, float* h_last,
                    hipStream_t stream);

/* Row strides (in elements) of the activation-shaped tensors, for reading
 * them in place as column slices of wider buffers: x and z as the two halves
 * of the (M, 2D) input-projection output, delta / B / C as column ranges of
 * the (M, R+2N) x-projection output.  The pages split these with a strided
 * column gather (COL_SLICE_WGSL / dispatchColumnSlice, which replaced a
 * prefix copy that was wrong for more than one row; builderforce-memory-engine
 * 2026.7.14 -> 2026.9.28, src/model/mamba1_block.ts); the strided entry
 * points make that gather unnecessary.
 * Row r of tensor T starts at T + r * T_stride.  Each stride must be at least
 * the row width (D for x, z, delta, y; N for B, C).  In the strided entry
 * points x (or u), z, delta, B, C and y need only 4-byte alignment; the
 * remaining tensors keep the 16-byte rule. */
typedef struct mss_strides {
    int32_t struct_size;    /* sizeof(mss_strides) */
    int32_t reserved;       /* must be 0 */
    int64_t x;              /* x (core) or u (scan) */
    int64_t z;
    int64_t delta;
    int64_t B;
    int64_t C;
    int64_t y;
} mss_strides;

/* mss_selective_scan with row strides; same semantics otherwise. */
int mss_selective_scan_strided(const mss_dims* dims, const mss_strides* strides, int disc,
                               const float* u, const float* delta, const float* A_log,
                               const float* B, const float* C, const float* D_vec,
                               const float* z, const float* h0, float* y, float* h_cache,
                               float* h_last, hipStream_t stream);

/* mss_mamba1_core with row strides; same semantics otherwise. */
int mss_mamba1_core_strided(const mss_dims* dims, const mss_strides* strides, int disc,
                            const float* x, const float* w_conv, const float* b_conv,
                            const float* delta, const float* A_log, const float* B,
                            const float* C, const float* D_vec, const float* z,
                            const float* h0, float* y, float* h_cache, float* h_last,
                            hipStream_t stream);

/* One single-token recurrent step (decode) with carried state; the plainest
 * reading of steps 4-9 for L = 1 with the conv window and h carried over.
 *   x, z, delta, y (B, D);  B, C (B, N);  A_log (D, N);  D_vec (D);
 *   w_conv (D, K);  b_conv (D);
 *   conv_state (B, K-1, D) in/out: the K-1 previous inputs, oldest first;
 *     tap k >= 1 multiplies conv_state[K-1-k]; afterwards the window is
 *     shifted by one and x appended.  May be NULL only when K == 1.
 *   h (B, D, N) in/out: the scan state, updated in place.
 *   Optional: D_vec, z, b_conv (NULL = 0 / ungated / 0).              */
int mss_selective_step(const mss_dims* dims, int disc, const float* x, const float* z,
                       const float* delta, const float* A_log, const float* B, const float* C,
                       const float* D_vec, const float* w_conv, const float* b_conv,
                       float* conv_state, float* h, float* y, hipStream_t stream);

/* ---- Backward passes ------------------------------------------------------
 * The reverse-time adjoint of the pages' CPU mirror (same diff and file,
 * function mamba1CpuBackward: its gate, reverse-time selective-scan, A_log
 * clamp mask, softplus, SiLU and depthwise conv1d parts).
 * Gradients are written, not accumulated.  Both entry points take a caller
 * workspace of at least mss_workspace_bytes bytes for the same dims and
 * device (256-byte aligned, overlapping nothing else; MSS_EWORKSPACE if
 * missing or too small); its contents on entry do not matter and it may be
 * reused once the call's work on `stream` has finished.  Results are
 * deterministic: every sum runs in a fixed order, no atomics.            */

#define MSS_OP_SELECTIVE_SCAN_BACKWARD 1
#define MSS_OP_CONV1D_SILU_BACKWARD 2

/* Workspace size in bytes for `op` (one of MSS_OP_*) on the current device;
 * 0 for empty problems. */
int mss_workspace_bytes(const mss_dims* dims, int op, size_t* bytes);

/* Gradients of the selective scan + gate (the forward of mss_selective_scan,
 * same inputs and layouts) against dout (M, D), the gradient of y:
 *   dY = dout * SiLU(z) (dout when z is NULL), with h the forward states and
 *   g the adjoint carried from step t+1, dh = C[r,:] dY + g:
 *   du (M, D)      = D_vec dY + sum_n dh bBar      (through the scan only:
 *                    the caller adds what u receives elsewhere)
 *   ddelta (M, D)  = sigmoid(delta) sum_n (dh h_{t-1} A aBar + dh u dbBar/ddv)
 *   dA_log (D, N)  = A sum_{b,t} (dh h_{t-1} dv aBar + dh u dbBar/dA),
 *                    0 where A_log <= -10 or A_log >= 5 (outside the clamp)
 *   dB, dC (M, N)  = sum_d dh u dbBar/dB,  sum_d dY h_t
 *   dD_vec (D)     = sum_{b,t} dY u                 (NULL: not computed)
 *   dz (M, D)      = dout y SiLU'(z), y ungated     (required iff z given)
 *   dh0 (B, D, N)  = the adjoint after step 0       (NULL: not computed)
 * Time segments are processed in parallel as in the forward: each rebuilds
 * the forward state entering it and the adjoint leaving it by replays whose
 * starting point has decayed by 2^-MSS_REPLAY_DECAY_BITS (see "Time split";
 * for the adjoint the window runs forward in time from the segment end).
 * MSS_FLAG_EXACT: no split, no replay.                                      */
/* h_ckpt (B, ceil(L/8), D, N): the forward's states entering every 8th step
 * (MSS_FLAG_CKPT8 in dims->flags; NULL otherwise).                        */
int mss_selective_scan_backward(const mss_dims* dims, int disc, const float* u,
                                const float* delta, const float* A_log, const float* B,
                                const float* C, const float* D_vec, const float* z,
                                const float* h0, const float* h_ckpt, const float* dout,
                                float* du, float* ddelta, float* dA_log, float* dB, float* dC,
                                float* dD_vec, float* dz, float* dh0, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

/* For callers that cannot allocate device memory -- code under HIP graph
 * capture, tight serving or training loops, harnesses that forbid hipMalloc:
 * mss_selective_scan_backward with the workspace taken from a static device
 * array inside the library instead of from the caller.  Same arguments and
 * results (the same kernels), minus the workspace.
 *   - The array holds MSS_NOALLOC_SCRATCH_BYTES (256 MiB) on every GPU the
 *     library runs on, from the time its code is loaded until the process
 *     ends.  A problem whose mss_workspace_bytes(MSS_OP_SELECTIVE_SCAN_BACKWARD)
 *     exceeds it is refused with MSS_ESCRATCH before anything is launched
 *     (B2 L512 D256 needs 3.3 MiB, B4 L2048 D1024 101 MiB, B8 L2048 D1536
 *     294 MiB: refused).  With the forward's checkpoints (MSS_FLAG_CKPT8)
 *     the backward needs no checkpoint workspace: B8 L2048 D1536 then needs
 *     102 MiB.
 *   - The call allocates nothing: no hipMalloc, no hipFree, no allocating
 *     library routine.  Its first call on a device looks up the array's
 *     device address (hipGetSymbolAddress, with that device current).
 *   - All calls on one GPU share the one array, which keeps the last call's
 *     contents (nothing in it needs to start at zero).  Calls that overlap
 *     in time on one GPU -- on two streams, or from two threads -- race on
 *     it: order them on one stream or use the workspace entry point.      */
#define MSS_NOALLOC_SCRATCH_BYTES (256ull << 20)
int mss_selective_scan_backward_noalloc(const mss_dims* dims, int disc, const float* u,
                                        const float* delta, const float* A_log, const float* B,
                                        const float* C, const float* D_vec, const float* z,
                                        const float* h0, const float* h_ckpt, const float* dout,
                                        float* du, float* ddelta, float* dA_log, float* dB,
                                        float* dC, float* dD_vec, float* dz, float* dh0,
                                        hipStream_t stream);

/* Gradients of u = SiLU(conv1d(x)) (mss_conv1d_silu) against du (M, D), the
 * total gradient reaching u:  dc = du * SiLU'(c),
 *   dx (M, D)         = sum_{k, t+k<L} dc[t+k] w_conv[d,k]
 *   dw_conv (D, K)    = sum_{b, t>=k} dc[t] x[t-k]
 *   db_conv (D)       = sum_{b,t} dc[t]            (NULL: not computed)   */
int mss_conv1d_silu_backward(const mss_dims* dims, const float* x, const float* w_conv,
                             const float* b_conv, const float* du, float* dx, float* dw_conv,
                             float* db_conv, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* ---- Mamba-2 SSD scan --------------------------------------------------------
 * The recurrence that the pages' Mamba2Block dispatches as ssd_chunk_forward
 * (diff 2026.7.14 -> 2026.9.28, src/model/mamba2_block.ts: x (M, D = H*P),
 * dt (M, H), B and C (M, G*N) split from the projections).  The pages do not
 * show its arithmetic; this is the plainest reading consistent with the
 * Mamba-1 path: per batch row and head h of group g = h / (H/G),
 *   dv = softplus(dt[r, h] + dt_bias[h]),  A_h = -exp(clamp(A_log[h], -10, 5))
 *   S_h[p, n] <- exp(dv A_h) S_h[p, n] + f x[r, h*P + p] B[r, g*N + n]
 *   y[r, h*P + p] = sum_n C[r, g*N + n] S_h[p, n] + D_vec[h] x[r, h*P + p]
 * with f = dv (MSS_DISC_EULER, the Mamba-2 form) or expm1(dv A_h) / A_h
 * (MSS_DISC_ZOH, the discretisation of the pages' Mamba-1 path).
 * Computed in chunks on the matrix cores (fp32 MFMA); time segments are
 * processed in parallel, each rebuilding its initial state by a replay whose
 * start has decayed by 2^-MSS_REPLAY_DECAY_BITS (see "Time split"; here the
 * decay is the head's scalar exp(A_h sum dv)).  MSS_FLAG_EXACT: no split. */
typedef struct mss_ssd_dims {
    int32_t struct_size;    /* sizeof(mss_ssd_dims) */
    int32_t flags;          /* 0, or MSS_FLAG_EXACT (any other bit: MSS_EINVAL) */
    int64_t batch;          /* B */
    int64_t seq_len;        /* L */
    int64_t n_heads;        /* H */
    int64_t head_dim;       /* P: 16, 32, 64 or 128 */
    int64_t d_state;        /* N: 16, 32, 64 or 128 */
    int64_t n_groups;       /* G: divides H */
} mss_ssd_dims;

/*   x, y (M, H*P);  dt (M, H);  A_log (H);  B, C (M, G*N);
 *   D_vec, dt_bias (H), may be NULL (= 0);
 *   h0, h_last (B, H, P, N), may be NULL (h0 = 0 / not written).
 * A sequence of length 0 still defines h_last (= h0, or zeros).          */
int mss_ssd_scan(const mss_ssd_dims* dims, int disc, const float* x, const float* dt, const float* A_log,
                 const float* B, const float* C, const float* D_vec, const float* dt_bias,
                 const float* h0, float* y, float* h_last, hipStream_t stream);

/* ---- Time split ----------------------------------------------------------
 * The segment length, in steps, that a call with these dims (flags
 * included) uses, for callers and tests that need to know where segments
 * start.  op: MSS_OP_SELECTIVE_SCAN (mss_selective_scan, mss_mamba1_core and
 * their strided forms) or MSS_OP_SELECTIVE_SCAN_BACKWARD.  The scans cut the
 * flattened (tile, t) space, tile = b * ceil(D/T) + d / T with T = 64
 * channels (forward) or 32 (backward) and t running fastest, into pieces of
 * *segment_steps steps (a multiple of 8); a segment starts wherever
 * (tile * Lp + t) is a multiple of *segment_steps, with Lp = L rounded up to
 * a multiple of 8 (so segments start at multiples of 8).  0 for empty
 * problems.                                                                 */
#define MSS_OP_SELECTIVE_SCAN 3
int mss_time_split(const mss_dims* dims, int op, int64_t* segment_steps);

/* The same for mss_ssd_scan: every (batch row, head) sequence is cut into
 * segments of *segment_steps steps starting at t = 0.                       */
int mss_ssd_time_split(const mss_ssd_dims* dims, int64_t* segment_steps);

/* ---- Gated linear recurrence ---------------------------------------------------
 * One state per channel instead of d_state of them, with gates that every
 * token brings along.  Per batch row b and channel d:
 *   h_t = v_t + (reset_t ? 0 : a_t h_{t-1})        (h_{-1} = h0, or 0)
 *   y_t = h_t SiLU(z_t)                             (h_t when z is NULL)
 * with the carry factor a and the input term v by `gate`:
 *   MSS_GATE_SIGMOID  a = sigma(r),                   v = (1 - a) x
 *   MSS_GATE_DECAY    a = exp(-c softplus(decay[d]) sigma(r)),
 *                     v = sqrt(1 - a^2) sigma(i) x    (c = gate_scale)
 *   MSS_GATE_LOG      a = exp(r),                     v = x
 * r = -inf is valid: it means a = 0 (a = 1 for MSS_GATE_DECAY).  reset_t != 0
 * drops the state carried into step t (the start of another document packed
 * into the same row, or the end of a row's left padding).  What lies on one
 * side of a reset, NaN and infinities included, does not reach the outputs
 * and gradients of rows on the other (ddecay, a sum over all rows, excepted).
 * Time is cut into chunks of up to 128 steps that are combined as affine maps
 * of the state: with MSS_GATE_LOG and r > 0 (growing states) the product of a
 * chunk's factors must stay finite.  A chunk waits for the state that enters it
 * from the one before: the wait ends by itself (a launch hands its chunks out in
 * order), and is bounded besides.  Past the bound, seconds for what takes
 * microseconds, the call's outputs are NaN from there on, although it returned
 * MSS_OK.
 * The activations x, r, i, z, y and their gradients are of type dims->dtype;
 * the states, decay and its gradient are fp32.  States are carried in fp32
 * and results are rounded once, to the nearest even.                       */
#define MSS_F32 0
#define MSS_BF16 1
#define MSS_F16 2
#define MSS_GATE_SIGMOID 0
#define MSS_GATE_DECAY 1
#define MSS_GATE_LOG 2
/* h_ckpt holds the state entering steps 0, 64, 128, ... */
#define MSS_GATED_CKPT_STEPS 64
/* Most channels of these calls and of the norms below; a call whose kernel
 * would have 2^32 threads or more is refused as well (MSS_EINVAL). */
#define MSS_MAX_WIDTH (1 << 28)
typedef struct mss_gated_dims {
    int32_t struct_size;    /* sizeof(mss_gated_dims) */
    int32_t flags;          /* must be 0 */
    int32_t dtype;          /* MSS_F32, MSS_BF16 or MSS_F16 */
    int32_t gate;           /* MSS_GATE_*; no default */
    int64_t batch;          /* B */
    int64_t seq_len;        /* L (ignored by mss_gated_step) */
    int64_t d_inner;        /* D */
    float gate_scale;       /* c of MSS_GATE_DECAY: finite, > 0 (ignored otherwise) */
    int32_t reserved;       /* must be 0 */
} mss_gated_dims;

/* Row strides in elements, each at least D; NULL in a call means dense rows
 * (stride D).  With strides given the activation tensors need only their
 * element's alignment (x and z as the two halves of a projection's output,
 * dx and dz as the halves of its gradient); outputs may then interleave with
 * each other inside one buffer as long as no element is shared.  Fields of
 * tensors that a call does not take are ignored. */
typedef struct mss_gated_strides {
    int32_t struct_size;    /* sizeof(mss_gated_strides) */
    int32_t reserved;       /* must be 0 */
    int64_t x, r, i, z;
    int64_t y;              /* y (forward, step) or dout (backward) */
    int64_t dx, dr, di, dz;
} mss_gated_strides;

#define MSS_OP_GATED_SCAN 4
#define MSS_OP_GATED_SCAN_BACKWARD 5
/* Workspace size in bytes of mss_gated_scan / mss_gated_scan_backward: a
 * function of the sizes alone, 0 for empty problems and for calls that need
 * none.  256-byte aligned; its contents on entry do not matter; it may be
 * reused, by a captured graph's replay too, once the call's work has
 * finished (calls that overlap in time need one each). */
int mss_gated_workspace_bytes(const mss_gated_dims* dims, int op, size_t* bytes);

/* The recurrence over a sequence.
 *   x, r, y (M, D);  i (M, D) and decay (D): required for MSS_GATE_DECAY,
 *   NULL otherwise;  z (M, D), h0 (B, D), reset (M) bytes: may be NULL;
 *   h_ckpt (B, ceil(L/64), D), h_last (B, D): outputs, may be NULL.
 * Deterministic: the output bits are a function of the inputs and sizes.
 * A sequence of length 0 still defines h_last (= h0, or zeros).            */
int mss_gated_scan(const mss_gated_dims* dims, const mss_gated_strides* strides, const void* x,
                   const void* r, const void* i, const float* decay, const void* z,
                   const float* h0, const uint8_t* reset, void* y, float* h_ckpt, float* h_last,
                   void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Its gradients, against dout (M, D), the gradient of y, and dh_last (B, D),
 * the gradient of h_last (NULL = 0).  h_ckpt: the forward's, from a call with
 * the same inputs.  With dy = dout SiLU(z), G_t = dy_t + (reset_{t+1} ? 0 :
 * a_{t+1} G_{t+1}) and p_t = (reset_t ? 0 : h_{t-1}):
 *   SIGMOID  dx = G (1 - a),  dr = G (p - x) a (1 - a)
 *   DECAY    dx = G m s,  di = G m x s (1 - s)     (s = sigma(i), m = sqrt(1 - a^2))
 *            w = G (a p - x s a^2 / m),  dr = -w c softplus(decay) q (1 - q),
 *            ddecay = -c sigma(decay) sum_{b,t} w q     (q = sigma(r); the
 *            terms over m take their limit, 0, where m = 0)
 *   LOG      dx = G,  dr = G a p
 *   dz = dout h SiLU'(z);  dh0 (B, D) = (reset_0 ? 0 : a_0 G_0)
 * Required: dx, dr; di and ddecay for MSS_GATE_DECAY (NULL otherwise); dz iff
 * z is given; dh0 may be NULL.  For L = 0 dh0 is dh_last (or zeros) and
 * ddecay zeros.  Gradients are written, not accumulated; deterministic.    */
int mss_gated_scan_backward(const mss_gated_dims* dims, const mss_gated_strides* strides,
                            const void* x, const void* r, const void* i, const float* decay,
                            const void* z, const uint8_t* reset, const float* h_ckpt,
                            const void* dout, const float* dh_last, void* dx, void* dr, void* di,
                            float* ddecay, void* dz, float* dh0, void* workspace,
                            size_t workspace_bytes, hipStream_t stream);

/* One token per sequence: x, r, i, z, y (B, D), h (B, D) updated in place. */
int mss_gated_step(const mss_gated_dims* dims, const mss_gated_strides* strides, const void* x,
                   const void* r, const void* i, const float* decay, const void* z, float* h,
                   void* y, hipStream_t stream);

/* ---- Norms before and after a block ---------------------------------------------
 * norm(v) over `width` channels in `groups` equal contiguous groups:
 *   MSS_NORM_RMS    v / sqrt(mean(v^2) + eps)
 *   MSS_NORM_LAYER  (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps)
 * (RMSNorm with eps 1e-6 is the pages' pre-block norm: cpu_ops.ts
 * rmsNormForward, RMSNORM_EPS.)  Activations are of type dims->dtype, the
 * residual stream of res_dtype (dtype, or fp32); w, b, scale and their
 * gradients fp32; statistics and sums fp32.                                */
#define MSS_NORM_RMS 0
#define MSS_NORM_LAYER 1
#define MSS_GATE_BEFORE_NORM 0
#define MSS_GATE_AFTER_NORM 1
typedef struct mss_norm_dims {
    int32_t struct_size;    /* sizeof(mss_norm_dims) */
    int32_t flags;          /* must be 0 */
    int32_t dtype;          /* MSS_F32, MSS_BF16 or MSS_F16 */
    int32_t res_dtype;      /* add_norm: dtype or MSS_F32; gated_norm: dtype */
    int32_t kind;           /* MSS_NORM_*; no default */
    int32_t order;          /* gated_norm: MSS_GATE_*_NORM; add_norm: 0 */
    int64_t rows;           /* M */
    int64_t width;          /* D */
    int64_t groups;         /* divides D, at most 2^20 (add_norm: 1) */
    float eps;              /* > 0, a normal number (2^-126 or more, finite) */
    float alpha;            /* scalar factor of the residual scale, finite */
} mss_norm_dims;

/* Row strides in elements, as in mss_gated_strides (NULL: dense rows). */
typedef struct mss_norm_strides {
    int32_t struct_size;    /* sizeof(mss_norm_strides) */
    int32_t reserved;       /* must be 0 */
    int64_t x, z, residual;
    int64_t s;              /* add_norm: the new residual stream */
    int64_t y;              /* y (forward) or dy / dout (backward) */
    int64_t ds;             /* add_norm backward: gradient of s */
    int64_t dx, dz, dresidual;
} mss_norm_strides;

#define MSS_OP_ADD_NORM_BACKWARD 6
#define MSS_OP_GATED_NORM_BACKWARD 7
/* Workspace size in bytes of the norm backward passes (partial sums of the
 * parameter gradients), under the rules of mss_gated_workspace_bytes. */
int mss_norm_workspace_bytes(const mss_norm_dims* dims, int op, size_t* bytes);

/* Before a block: s = residual + alpha scale[d] x, rounded to res_dtype, and
 * y = norm(s) w + b of the rounded s (so that the backward, which reads s,
 * differentiates the same numbers).
 *   x, y (M, D) dtype;  residual, s (M, D) res_dtype;  w, b, scale (D).
 *   Optional: residual (= 0), b (= 0), scale (= 1).  s may be residual itself
 *   (same pointer and stride): the stream is then updated in place.         */
int mss_add_norm(const mss_norm_dims* dims, const mss_norm_strides* strides, const void* x,
                 const void* residual, const float* w, const float* b, const float* scale, void* s,
                 void* y, hipStream_t stream);

/* Its gradients against dy (M, D) dtype and ds (M, D) res_dtype, what else
 * reaches the stream (NULL = 0):
 *   dresidual = ds + (norm backward of dy w at s)   res_dtype
 *   dx        = alpha scale[d] dresidual            dtype
 *   dw, db, dscale (D) = sum dy n,  sum dy,  alpha sum dresidual x
 * Required: s, w, dy, dresidual; x when dscale is wanted; dx, dw, db, dscale
 * are computed where given.                                                */
int mss_add_norm_backward(const mss_norm_dims* dims, const mss_norm_strides* strides,
                          const void* s, const float* w, const void* dy, const void* ds,
                          const void* x, const float* scale, void* dx, void* dresidual, float* dw,
                          float* db, float* dscale, void* workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* After a block: with the gate SiLU(z) (1 when z is NULL),
 *   MSS_GATE_BEFORE_NORM  n = norm(x SiLU(z)) w + b
 *   MSS_GATE_AFTER_NORM   n = (norm(x) w + b) SiLU(z)
 *   y = alpha scale[d] n, plus residual when given.
 *   x, z, residual, y (M, D) dtype;  w, b, scale (D).
 *   Optional: z, b (= 0), residual (= 0), scale (= 1).                     */
int mss_gated_norm(const mss_norm_dims* dims, const mss_norm_strides* strides, const void* x,
                   const void* z, const float* w, const float* b, const void* residual,
                   const float* scale, void* y, hipStream_t stream);

/* Its gradients against dout (M, D) (the residual's is dout itself):
 *   dx, dz (M, D) dtype;  dw, db, dscale (D) where given (b: the forward's;
 *   it enters dz of MSS_GATE_AFTER_NORM and dscale).
 * Required: x, w, dout, dx; dz iff z is given.                             */
int mss_gated_norm_backward(const mss_norm_dims* dims, const mss_norm_strides* strides,
                            const void* x, const void* z, const float* w, const float* b,
                            const float* scale, const void* dout, void* dx, void* dz, float* dw,
                            float* db, float* dscale, void* workspace, size_t workspace_bytes,
                            hipStream_t stream);

/* ---- The ends of a model ------------------------------------------------------
 * What stands before the first block and after the last one (the pages'
 * cpuModelForward / cpuModelLoss / cpuModelBackward: token rows of a table,
 * the head on the final norm and its cross entropy), and the clipping of the
 * gradients before the update (the trainer's maxGradNorm).  Tables, rows and
 * their gradients are of type MSS_F32, MSS_BF16 or MSS_F16; losses, log sums
 * and norms are fp32, sums at least that.  Results are deterministic (every
 * sum runs in a fixed order), gradients are written once and rounded once.
 *
 * Token ids and targets are int32 or int64 (id_bytes 4 or 8).  One outside
 * 0 .. vocab-1 is no error: it marks a padded place (for the embedding also a
 * token that another shard of the table holds; for the head see
 * mss_head_loss_backward).
 *
 * Row strides in elements, as in mss_gated_strides (NULL: dense rows).  With
 * strides given the tensors need only their element's alignment; ids, targets
 * and tensors of one value per row always do.                              */
#define MSS_EMBED_ACCUMULATE 1
typedef struct mss_embed_dims {
    int32_t struct_size;    /* sizeof(mss_embed_dims) */
    int32_t flags;          /* 0, or MSS_EMBED_ACCUMULATE (backward only) */
    int32_t dtype;          /* of the table and its gradient */
    int32_t out_dtype;      /* of y and dy: dtype or MSS_F32; any where dtype is MSS_F32 */
    int32_t id_bytes;       /* 4 or 8 */
    int32_t reserved;       /* must be 0 */
    int64_t rows;           /* M, below 2^26 */
    int64_t vocab;          /* V, below 2^26 */
    int64_t width;          /* D, at most MSS_MAX_WIDTH */
    float scale;            /* finite */
    int32_t reserved2;      /* must be 0 */
} mss_embed_dims;

typedef struct mss_embed_strides {
    int32_t struct_size;    /* sizeof(mss_embed_strides) */
    int32_t reserved;       /* must be 0 */
    int64_t weight;         /* the table, or its gradient */
    int64_t y;              /* y, or dy */
} mss_embed_strides;

/* y_m = scale weight[id_m]; zeros where id_m marks a padded place.
 *   ids (M);  weight (V, D) dtype;  y (M, D) out_dtype                     */
int mss_embedding(const mss_embed_dims* dims, const mss_embed_strides* strides, const void* ids,
                  const void* weight, void* y, hipStream_t stream);

/* Its gradient: dweight_v = scale sum_{m: id_m = v} dy_m, in the order of m.
 * Every row of dweight is written (zeros where v does not occur); with
 * MSS_EMBED_ACCUMULATE the sums are added to what dweight holds, and only the
 * rows that occur are touched (a table tied to the head: after
 * mss_head_loss_backward has written its part).
 *   ids (M);  dy (M, D) out_dtype;  dweight (V, D) dtype                    */
int mss_embedding_backward(const mss_embed_dims* dims, const mss_embed_strides* strides,
                           const void* ids, const void* dy, void* dweight, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);

/* Workspace size in bytes of mss_embedding_backward, under the rules of
 * mss_gated_workspace_bytes. */
int mss_embed_workspace_bytes(const mss_embed_dims* dims, size_t* bytes);

typedef struct mss_head_dims {
    int32_t struct_size;    /* sizeof(mss_head_dims) */
    int32_t flags;          /* must be 0 */
    int32_t dtype;          /* of x, weight and their gradients */
    int32_t id_bytes;       /* of the targets: 4 or 8 */
    int64_t rows;           /* M, below 2^26; backward: M D below about 2^36 as well */
    int64_t vocab;          /* V, 1 .. 2^26 - 1 */
    int64_t width;          /* D, 1 .. MSS_MAX_WIDTH */
    float logit_scale;      /* finite */
    int32_t reserved;       /* must be 0 */
} mss_head_dims;

typedef struct mss_head_strides {
    int32_t struct_size;    /* sizeof(mss_head_strides) */
    int32_t reserved;       /* must be 0 */
    int64_t x, weight, dx, dweight;
} mss_head_strides;

#define MSS_OP_HEAD_LOSS 8
#define MSS_OP_HEAD_LOSS_BACKWARD 9
/* Workspace size in bytes of the head calls, under the rules of
 * mss_gated_workspace_bytes. */
int mss_head_workspace_bytes(const mss_head_dims* dims, int op, size_t* bytes);

/* Softmax cross entropy of the logits l_mv = logit_scale x_m . weight_v,
 * which are never stored (the vocabulary goes by in tiles):
 *   lse_m  = log sum_v exp(l_mv)
 *   loss_m = lse_m - l_{m, t_m}; 0 where t_m marks a padded place
 *   x (M, D), weight (V, D) dtype;  targets (M);  loss, lse (M) fp32
 * Logits are fp32 sums of exact products of 2-byte operands.  fp32 operands
 * are split in three parts of 8 bits each, and of their nine products the six
 * largest are summed: what is left out is below 2^-21 of each product (of
 * operands of 2^-100 and more, whose last part is no subnormal); a sum with an
 * infinite or NaN operand is that of the fp32 products.
 * A logit may have any value of fp32: one far below a row's largest, down to
 * -inf, adds 0 to the sum (masked tokens).  lse is inf where a logit is, and
 * -inf (and the loss NaN) where every logit is.                             */
int mss_head_loss(const mss_head_dims* dims, const mss_head_strides* strides, const void* x,
                  const void* weight, const void* targets, float* loss, float* lse,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Its gradients against dloss (M) and dlse (M) (NULL = 0), with the forward's
 * lse:
 *   dl_mv = (dloss_m + dlse_m) exp(l_mv - lse_m) - dloss_m [v = t_m]
 *   dx = logit_scale dl weight,  dweight = logit_scale dl^T x
 * A padded row takes no part: its dx is 0, and its x, dloss and dlse are not
 * used (they may be NaN).  dl is computed a piece of the vocabulary at a time
 * and held in dtype for the two products, times a factor that brings the
 * largest |dloss| + |dlse| to just below 2^13 (fp16 would lose the small
 * ones, and bf16 rounds least there): in 2-byte types each of its values is
 * rounded once.  In fp16 a row of dl has for dx a further power of 2 of its own,
 * so that its dx does not depend on the others' size; to dweight what is below
 * 2^-38 of the largest is lost.  dx and dweight are summed in fp32.
 *   dx (M, D), dweight (V, D) dtype: each computed where given.
 * A vocabulary in shards: with LSE, the log of the sum of the shards' exp(lse),
 * the loss is LSE - (lse - loss) with lse and loss of the shard that has the
 * target.  Backwards every shard is given LSE as lse.  A row whose target is in
 * another shard takes part in this one by dlse: any token of the shard as its
 * target, dloss 0 and dlse the row's dloss + dlse.  (Left as a padded row it
 * would lose the shard's part of its gradients.)  dx is the sum over the
 * shards.                                                                   */
int mss_head_loss_backward(const mss_head_dims* dims, const mss_head_strides* strides,
                           const void* x, const void* weight, const void* targets,
                           const float* lse, const float* dloss, const float* dlse, void* dx,
                           void* dweight, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* One of a list of tensors: numel elements, dense, at their element's
 * alignment.  The list itself is host memory, read before the call returns. */
typedef struct mss_tensor {
    const void* in;
    void* out;              /* mss_clip_grads: may be `in` (updated in place) */
    int64_t numel;
    int32_t dtype;          /* MSS_F32, MSS_BF16 or MSS_F16 */
    int32_t out_dtype;      /* dtype or MSS_F32 */
} mss_tensor;

/* Workspace size in bytes of the two calls below for `count` tensors, under
 * the rules of mss_gated_workspace_bytes. */
int mss_clip_workspace_bytes(int64_t count, size_t* bytes);

/* norm[0] = scale sqrt(sum of all elements' squares); squares and sums are
 * fp64.  `out` and `out_dtype` are ignored; scale is finite and > 0.
 * An empty list has norm 0.                                                */
int mss_grad_norm(const mss_tensor* tensors, int64_t count, float scale, float* norm,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The norm, and out = in * scale * min(1, max_norm / norm).  Where a value is
 * infinite or NaN out = in: nothing is lost, and the caller sees it in norm[0]
 * (where finite values' norm exceeds fp32, norm[0] is infinite as well, but they
 * are clipped).  max_norm is finite and >= 0.  No tensor may overlap another, in place apart.  */
int mss_clip_grads(const mss_tensor* tensors, int64_t count, float scale, float max_norm,
                   float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Human-readable text for a status code (static storage). */
const char* mss_strerror(int status);

/* MSS_VERSION of the library that was loaded. */
int mss_version(void);

/* The hipError_t of the last MSS_EHIP returned on the calling thread. */
int mss_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MSS_H */
