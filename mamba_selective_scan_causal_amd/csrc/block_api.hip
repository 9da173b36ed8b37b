// block_api.hip -- the extern "C" entry points of the gated linear recurrence
// and the block norms: argument validation and dispatch on the caller's
// stream, under the same rules as mss_api.hip (everything is checked before
// any launch; a rejected call writes nothing).
#include <cmath>
#include <cstdint>

#include "api_check.h"
#include "launch.h"
#include "launch_block.h"
#include "mss.h"

namespace {

using mss::count;
using mss::hip_fail;

int64_t elem_size(int dtype) { return dtype == MSS_F32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype == MSS_F32 || dtype == MSS_BF16 || dtype == MSS_F16; }

// `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t rows, width, stride;
};

int64_t span(const Rows& r) { return r.rows <= 0 || r.width <= 0 ? 0 : (r.rows - 1) * r.stride + r.width; }

// Whether two tensors share a byte.  Column ranges of one buffer (equal
// strides) that interleave without meeting do not.
bool overlap(const Rows& a, const Rows& b) {
    const mss::Span sa{a.p, span(a)}, sb{b.p, span(b)};
    if (!mss::overlap(sa, sb)) return false;
    if (a.stride != b.stride) return true;
    const intptr_t diff = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
    const int64_t off = ((diff % a.stride) + a.stride) % a.stride;
    return !(off >= a.width && off + b.width <= a.stride);
}

class Checks {
  public:
    explicit Checks(bool strided) : strided_(strided) {}

    // A row-strided activation tensor: the element's alignment when the call
    // gives strides, 16 bytes otherwise.
    void in(const void* p, int64_t rows, int64_t width, int64_t ld, int64_t elem, bool required) {
        add(ins_, n_ins_, p, rows, width, ld, elem, required, strided_ ? elem : 16);
    }
    void out(void* p, int64_t rows, int64_t width, int64_t ld, int64_t elem, bool required) {
        add(outs_, n_outs_, p, rows, width, ld, elem, required, strided_ ? elem : 16);
    }
    // A dense tensor (16-byte aligned).
    void in(const void* p, int64_t elems, int64_t elem, bool required) {
        add(ins_, n_ins_, p, elems > 0 ? 1 : 0, elems, elems, elem, required, 16);
    }
    void out(void* p, int64_t elems, int64_t elem, bool required) {
        add(outs_, n_outs_, p, elems > 0 ? 1 : 0, elems, elems, elem, required, 16);
    }
    // Bytes of any alignment (the reset flags).
    void in_bytes(const void* p, int64_t n) { add(ins_, n_ins_, p, n > 0 ? 1 : 0, n, n, 1, false, 1); }
    void must(bool ok) {
        if (!ok && status_ == MSS_OK) status_ = MSS_EINVAL;
    }
    // The workspace: of the size the query reports, overlapping nothing.
    void workspace(void* p, size_t bytes, int64_t need) {
        if (need == 0) return;
        ws_status_ = !p || bytes < static_cast<uint64_t>(need) ? MSS_EWORKSPACE
                     : reinterpret_cast<uintptr_t>(p) % 256    ? MSS_EALIGN
                                                               : MSS_OK;
        if (p) outs_[n_outs_++] = {p, 1, need, need};
    }
    // The input added last, for finish.
    int last() const { return n_ins_ - 1; }
    // An output may be exactly the input number `in_place` (same pointer, width
    // and stride), updated in place.
    int finish(int in_place = -1) {
        if (status_ != MSS_OK) return status_;
        for (int i = 0; i < n_outs_; i++) {
            for (int j = 0; j < n_ins_; j++) {
                const Rows& s = ins_[j];
                if (j == in_place && outs_[i].p == s.p && outs_[i].width == s.width &&
                    outs_[i].stride == s.stride)
                    continue;
                if (overlap(outs_[i], s)) return MSS_EALIAS;
            }
            for (int j = i + 1; j < n_outs_; j++)
                if (overlap(outs_[i], outs_[j])) return MSS_EALIAS;
        }
        return ws_status_;
    }

  private:
    void add(Rows* v, int& used, const void* p, int64_t rows, int64_t width, int64_t ld,
             int64_t elem, bool required, int64_t align) {
        if (status_ != MSS_OK) return;
        int64_t all;
        if (ld < width || !count(all, {rows, ld, elem})) {
            status_ = MSS_EINVAL;
            return;
        }
        if (!p) {
            if (required && rows > 0 && width > 0) status_ = MSS_EINVAL;
            return;
        }
        if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(align) != 0) {
            status_ = MSS_EALIGN;
            return;
        }
        if (rows > 0 && width > 0) v[used++] = {p, rows, width * elem, ld * elem};
    }

    bool strided_;
    int status_ = MSS_OK, ws_status_ = MSS_OK;
    // the longest argument list has ten inputs and seven outputs
    Rows ins_[16], outs_[16];
    int n_ins_ = 0, n_outs_ = 0;
};

int launched(hipError_t e) { return e == hipSuccess ? MSS_OK : hip_fail(e); }

int state_init(const float* from, float* to, int64_t n, hipStream_t stream) {
    return to && n > 0 ? launched(mss::launch_state_init(from, to, n, stream)) : MSS_OK;
}

// ---- gated recurrence --------------------------------------------------------

bool gated_ok(const mss_gated_dims* d, const mss_gated_strides* s, bool need_l) {
    if (!d || d->struct_size != static_cast<int32_t>(sizeof(mss_gated_dims)) || d->flags != 0 ||
        d->reserved != 0 || !dtype_ok(d->dtype))
        return false;
    if (d->gate != MSS_GATE_SIGMOID && d->gate != MSS_GATE_DECAY && d->gate != MSS_GATE_LOG)
        return false;
    if (d->gate == MSS_GATE_DECAY && !(std::isfinite(d->gate_scale) && d->gate_scale > 0.0f))
        return false;
    if (d->batch < 0 || d->d_inner < 0 || (need_l && d->seq_len < 0)) return false;
    if (d->d_inner > MSS_MAX_WIDTH) return false;
    return !s || (s->struct_size == static_cast<int32_t>(sizeof(mss_gated_strides)) &&
                  s->reserved == 0);
}

mss::GatedArgs gated_args(const mss_gated_dims* d, const mss_gated_strides* s, int64_t L) {
    mss::GatedArgs a{};
    a.dtype = d->dtype;
    a.gate = d->gate;
    a.B = d->batch;
    a.L = L;
    a.D = d->d_inner;
    a.gate_scale = d->gate_scale;
    const int64_t D = a.D;
    a.ld_x = s ? s->x : D;
    a.ld_r = s ? s->r : D;
    a.ld_i = s ? s->i : D;
    a.ld_z = s ? s->z : D;
    a.ld_y = s ? s->y : D;
    a.ld_dx = s ? s->dx : D;
    a.ld_dr = s ? s->dr : D;
    a.ld_di = s ? s->di : D;
    a.ld_dz = s ? s->dz : D;
    return a;
}

int64_t ckpt_rows(int64_t L) { return L / MSS_GATED_CKPT_STEPS + (L % MSS_GATED_CKPT_STEPS != 0); }

// The inputs that every entry point takes.
void gated_inputs(Checks& ck, const mss::GatedArgs& a, int64_t M) {
    const int64_t e = elem_size(a.dtype);
    const bool decay = a.gate == MSS_GATE_DECAY;
    ck.must(decay || (!a.i && !a.decay));
    ck.in(a.x, M, a.D, a.ld_x, e, true);
    ck.in(a.r, M, a.D, a.ld_r, e, true);
    if (decay) {
        ck.in(a.i, M, a.D, a.ld_i, e, true);
        ck.in(a.decay, a.D, 4, true);
    }
    if (a.z) ck.in(a.z, M, a.D, a.ld_z, e, false);
}

// ---- norms ---------------------------------------------------------------------

bool norm_ok(const mss_norm_dims* d, const mss_norm_strides* s, bool add) {
    if (!d || d->struct_size != static_cast<int32_t>(sizeof(mss_norm_dims)) || d->flags != 0 ||
        !dtype_ok(d->dtype))
        return false;
    if (d->kind != MSS_NORM_RMS && d->kind != MSS_NORM_LAYER) return false;
    if (d->rows < 0 || d->width < 0 || d->groups < 1 || d->width % d->groups != 0) return false;
    if (d->width > MSS_MAX_WIDTH || d->groups > (1 << 20)) return false;
    if (!(std::isnormal(d->eps) && d->eps > 0.0f) || !std::isfinite(d->alpha)) return false;
    if (add) {
        if (d->groups != 1 || d->order != 0) return false;
        if (d->res_dtype != d->dtype && d->res_dtype != MSS_F32) return false;
    } else {
        if (d->order != MSS_GATE_BEFORE_NORM && d->order != MSS_GATE_AFTER_NORM) return false;
        if (d->res_dtype != d->dtype) return false;
    }
    return !s || (s->struct_size == static_cast<int32_t>(sizeof(mss_norm_strides)) &&
                  s->reserved == 0);
}

mss::NormArgs norm_args(const mss_norm_dims* d, const mss_norm_strides* s) {
    mss::NormArgs a{};
    a.dtype = d->dtype;
    a.res_dtype = d->res_dtype;
    a.kind = d->kind;
    a.order = d->order;
    a.M = d->rows;
    a.D = d->width;
    a.G = d->groups;
    a.eps = d->eps;
    a.alpha = d->alpha;
    const int64_t D = a.D;
    a.ld_x = s ? s->x : D;
    a.ld_z = s ? s->z : D;
    a.ld_res = s ? s->residual : D;
    a.ld_s = s ? s->s : D;
    a.ld_y = s ? s->y : D;
    a.ld_ds = s ? s->ds : D;
    a.ld_dx = s ? s->dx : D;
    a.ld_dz = s ? s->dz : D;
    a.ld_dres = s ? s->dresidual : D;
    return a;
}

// Parameter gradients of no rows are zero.
int zero_params(const mss::NormArgs& a, hipStream_t stream) {
    int st = state_init(nullptr, a.dw, a.D, stream);
    if (st == MSS_OK) st = state_init(nullptr, a.db, a.D, stream);
    return st == MSS_OK ? state_init(nullptr, a.dscale, a.D, stream) : st;
}

// Bytes of the norm backward's workspace for these sizes.
bool norm_need(const mss::NormArgs& a, int64_t& need) {
    need = 0;
    return a.M == 0 || a.D == 0 || mss::norm_bwd_workspace(a.M, a.D, a.G, need);
}

}  // namespace

extern "C" {

int mss_gated_workspace_bytes(const mss_gated_dims* dims, int op, size_t* bytes) {
    if (!bytes) return MSS_EINVAL;
    *bytes = 0;
    if (!gated_ok(dims, nullptr, true)) return MSS_EINVAL;
    int64_t n, need = 0;
    if (!count(n, {dims->batch, dims->seq_len, dims->d_inner, 4})) return MSS_EINVAL;
    if (op != MSS_OP_GATED_SCAN && op != MSS_OP_GATED_SCAN_BACKWARD) return MSS_EINVAL;
    if (n == 0) return MSS_OK;
    const bool ok = op == MSS_OP_GATED_SCAN
                        ? mss::gated_scan_workspace(dims->batch, dims->seq_len, dims->d_inner,
                                                    need)
                        : mss::gated_scan_bwd_workspace(dims->batch, dims->seq_len, dims->d_inner,
                                                        dims->gate, need);
    if (!ok) return MSS_EINVAL;
    *bytes = static_cast<size_t>(need);
    return MSS_OK;
}

int mss_gated_scan(const mss_gated_dims* dims, const mss_gated_strides* strides, const void* x,
                   const void* r, const void* i, const float* decay, const void* z,
                   const float* h0, const uint8_t* reset, void* y, float* h_ckpt, float* h_last,
                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!gated_ok(dims, strides, true)) return MSS_EINVAL;
    mss::GatedArgs a = gated_args(dims, strides, dims->seq_len);
    a.x = x;
    a.r = r;
    a.i = i;
    a.decay = decay;
    a.z = z;
    a.h0 = h0;
    a.reset = reset;
    a.y = y;
    a.h_ckpt = h_ckpt;
    a.h_last = h_last;
    a.ws = workspace;
    int64_t M, MD, BD, BKD, need = 0;
    if (!count(M, {a.B, a.L}) || !count(MD, {M, a.D, 4}) || !count(BD, {a.B, a.D}) ||
        !count(BKD, {a.B, ckpt_rows(a.L), a.D, 4}))
        return MSS_EINVAL;
    if (MD > 0 && !mss::gated_scan_workspace(a.B, a.L, a.D, need)) return MSS_EINVAL;
    Checks ck(strides != nullptr);
    gated_inputs(ck, a, M);
    ck.in(h0, BD, 4, false);
    ck.in_bytes(reset, M);
    ck.out(y, M, a.D, a.ld_y, elem_size(a.dtype), true);
    ck.out(h_ckpt, BKD / 4, 4, false);
    ck.out(h_last, BD, 4, false);
    ck.workspace(workspace, workspace_bytes, need);
    const int st = ck.finish();
    if (st != MSS_OK) return st;
    if (BD == 0) return MSS_OK;
    if (a.L == 0) return state_init(h0, h_last, BD, stream);
    return launched(mss::launch_gated_scan(a, stream));
}

int mss_gated_scan_backward(const mss_gated_dims* dims, const mss_gated_strides* strides,
                            const void* x, const void* r, const void* i, const float* decay,
                            const void* z, const uint8_t* reset, const float* h_ckpt,
                            const void* dout, const float* dh_last, void* dx, void* dr, void* di,
                            float* ddecay, void* dz, float* dh0, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    if (!gated_ok(dims, strides, true)) return MSS_EINVAL;
    mss::GatedArgs a = gated_args(dims, strides, dims->seq_len);
    a.x = x;
    a.r = r;
    a.i = i;
    a.decay = decay;
    a.z = z;
    a.reset = reset;
    a.h_ckpt = const_cast<float*>(h_ckpt);
    a.dout = dout;
    a.dh_last = dh_last;
    a.dx = dx;
    a.dr = dr;
    a.di = di;
    a.ddecay = ddecay;
    a.dz = dz;
    a.dh0 = dh0;
    a.ws = workspace;
    int64_t M, MD, BD, BKD, need = 0;
    if (!count(M, {a.B, a.L}) || !count(MD, {M, a.D, 4}) || !count(BD, {a.B, a.D}) ||
        !count(BKD, {a.B, ckpt_rows(a.L), a.D, 4}))
        return MSS_EINVAL;
    if (MD > 0 && !mss::gated_scan_bwd_workspace(a.B, a.L, a.D, a.gate, need)) return MSS_EINVAL;
    const bool has_decay = a.gate == MSS_GATE_DECAY;
    const int64_t e = elem_size(a.dtype);
    Checks ck(strides != nullptr);
    gated_inputs(ck, a, M);
    ck.must(has_decay || (!di && !ddecay));
    ck.must(MD == 0 || (z != nullptr) == (dz != nullptr));
    ck.in_bytes(reset, M);
    ck.in(h_ckpt, BKD / 4, 4, true);
    ck.in(dout, M, a.D, a.ld_y, e, true);
    ck.in(dh_last, BD, 4, false);
    ck.out(dx, M, a.D, a.ld_dx, e, true);
    ck.out(dr, M, a.D, a.ld_dr, e, true);
    if (has_decay) {
        ck.out(di, M, a.D, a.ld_di, e, true);
        ck.out(ddecay, a.D, 4, true);
    }
    if (dz) ck.out(dz, M, a.D, a.ld_dz, e, false);
    ck.out(dh0, BD, 4, false);
    ck.workspace(workspace, workspace_bytes, need);
    int st = ck.finish();
    if (st != MSS_OK) return st;
    if (MD == 0) {
        if (has_decay && (st = state_init(nullptr, ddecay, a.D, stream)) != MSS_OK) return st;
        return state_init(dh_last, dh0, BD, stream);
    }
    return launched(mss::launch_gated_scan_bwd(a, stream));
}

int mss_gated_step(const mss_gated_dims* dims, const mss_gated_strides* strides, const void* x,
                   const void* r, const void* i, const float* decay, const void* z, float* h,
                   void* y, hipStream_t stream) {
    if (!gated_ok(dims, strides, false)) return MSS_EINVAL;
    mss::GatedArgs a = gated_args(dims, strides, 1);
    a.x = x;
    a.r = r;
    a.i = i;
    a.decay = decay;
    a.z = z;
    a.h = h;
    a.y = y;
    int64_t BD;
    if (!count(BD, {a.B, a.D, 4}) || !mss::gated_step_fits(a.B, a.D)) return MSS_EINVAL;
    BD /= 4;
    Checks ck(strides != nullptr);
    gated_inputs(ck, a, a.B);
    ck.out(h, BD, 4, true);
    ck.out(y, a.B, a.D, a.ld_y, elem_size(a.dtype), true);
    const int st = ck.finish();
    if (st != MSS_OK || BD == 0) return st;
    return launched(mss::launch_gated_step(a, stream));
}

int mss_norm_workspace_bytes(const mss_norm_dims* dims, int op, size_t* bytes) {
    if (!bytes) return MSS_EINVAL;
    *bytes = 0;
    if (op != MSS_OP_ADD_NORM_BACKWARD && op != MSS_OP_GATED_NORM_BACKWARD) return MSS_EINVAL;
    if (!norm_ok(dims, nullptr, op == MSS_OP_ADD_NORM_BACKWARD)) return MSS_EINVAL;
    const mss::NormArgs a = norm_args(dims, nullptr);
    int64_t n, need;
    if (!count(n, {a.M, a.D, 4}) || !norm_need(a, need)) return MSS_EINVAL;
    *bytes = static_cast<size_t>(need);
    return MSS_OK;
}

int mss_add_norm(const mss_norm_dims* dims, const mss_norm_strides* strides, const void* x,
                 const void* residual, const float* w, const float* b, const float* scale, void* s,
                 void* y, hipStream_t stream) {
    if (!norm_ok(dims, strides, true)) return MSS_EINVAL;
    mss::NormArgs a = norm_args(dims, strides);
    a.x = x;
    a.res = residual;
    a.w = w;
    a.b = b;
    a.scale = scale;
    a.s = s;
    a.y = y;
    const int64_t e = elem_size(a.dtype), er = elem_size(a.res_dtype);
    int64_t n;
    if (!count(n, {a.M, a.D, 4})) return MSS_EINVAL;
    Checks ck(strides != nullptr);
    ck.in(x, a.M, a.D, a.ld_x, e, true);
    if (residual) ck.in(residual, a.M, a.D, a.ld_res, er, false);
    const int in_place = residual && residual == s ? ck.last() : -1;
    ck.in(w, a.D, 4, true);
    ck.in(b, a.D, 4, false);
    ck.in(scale, a.D, 4, false);
    ck.out(s, a.M, a.D, a.ld_s, er, true);
    ck.out(y, a.M, a.D, a.ld_y, e, true);
    const int st = ck.finish(in_place);
    if (st != MSS_OK || n == 0) return st;
    return launched(mss::launch_add_norm(a, stream));
}

int mss_add_norm_backward(const mss_norm_dims* dims, const mss_norm_strides* strides,
                          const void* s, const float* w, const void* dy, const void* ds,
                          const void* x, const float* scale, void* dx, void* dresidual, float* dw,
                          float* db, float* dscale, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
    if (!norm_ok(dims, strides, true)) return MSS_EINVAL;
    mss::NormArgs a = norm_args(dims, strides);
    a.s = const_cast<void*>(s);
    a.w = w;
    a.dy = dy;
    a.ds = ds;
    a.x = dscale ? x : nullptr;
    a.scale = scale;
    a.dx = dx;
    a.dres = dresidual;
    a.dw = dw;
    a.db = db;
    a.dscale = dscale;
    a.ws = workspace;
    const int64_t e = elem_size(a.dtype), er = elem_size(a.res_dtype);
    int64_t n, need;
    if (!count(n, {a.M, a.D, 4}) || !norm_need(a, need)) return MSS_EINVAL;
    Checks ck(strides != nullptr);
    ck.in(s, a.M, a.D, a.ld_s, er, true);
    ck.in(w, a.D, 4, true);
    ck.in(dy, a.M, a.D, a.ld_y, e, true);
    if (ds) ck.in(ds, a.M, a.D, a.ld_ds, er, false);
    if (dscale) ck.in(x, a.M, a.D, a.ld_x, e, true);
    ck.in(scale, a.D, 4, false);
    if (dx) ck.out(dx, a.M, a.D, a.ld_dx, e, false);
    ck.out(dresidual, a.M, a.D, a.ld_dres, er, true);
    ck.out(dw, a.D, 4, false);
    ck.out(db, a.D, 4, false);
    ck.out(dscale, a.D, 4, false);
    ck.workspace(workspace, workspace_bytes, need);
    const int st = ck.finish();
    if (st != MSS_OK) return st;
    return n == 0 ? zero_params(a, stream) : launched(mss::launch_add_norm_bwd(a, stream));
}

int mss_gated_norm(const mss_norm_dims* dims, const mss_norm_strides* strides, const void* x,
                   const void* z, const float* w, const float* b, const void* residual,
                   const float* scale, void* y, hipStream_t stream) {
    if (!norm_ok(dims, strides, false)) return MSS_EINVAL;
    mss::NormArgs a = norm_args(dims, strides);
    a.x = x;
    a.z = z;
    a.w = w;
    a.b = b;
    a.res = residual;
    a.scale = scale;
    a.y = y;
    const int64_t e = elem_size(a.dtype);
    int64_t n;
    if (!count(n, {a.M, a.D, 4})) return MSS_EINVAL;
    Checks ck(strides != nullptr);
    ck.in(x, a.M, a.D, a.ld_x, e, true);
    if (z) ck.in(z, a.M, a.D, a.ld_z, e, false);
    if (residual) ck.in(residual, a.M, a.D, a.ld_res, e, false);
    ck.in(w, a.D, 4, true);
    ck.in(b, a.D, 4, false);
    ck.in(scale, a.D, 4, false);
    ck.out(y, a.M, a.D, a.ld_y, e, true);
    const int st = ck.finish();
    if (st != MSS_OK || n == 0) return st;
    return launched(mss::launch_gated_norm(a, stream));
}

int mss_gated_norm_backward(const mss_norm_dims* dims, const mss_norm_strides* strides,
                            const void* x, const void* z, const float* w, const float* b,
                            const float* scale, const void* dout, void* dx, void* dz, float* dw,
                            float* db, float* dscale, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
    if (!norm_ok(dims, strides, false)) return MSS_EINVAL;
    mss::NormArgs a = norm_args(dims, strides);
    a.x = x;
    a.z = z;
    a.w = w;
    a.b = b;
    a.scale = scale;
    a.dy = dout;
    a.dx = dx;
    a.dz = dz;
    a.dw = dw;
    a.db = db;
    a.dscale = dscale;
    a.ws = workspace;
    const int64_t e = elem_size(a.dtype);
    int64_t n, need;
    if (!count(n, {a.M, a.D, 4}) || !norm_need(a, need)) return MSS_EINVAL;
    Checks ck(strides != nullptr);
    ck.must(n == 0 || (z != nullptr) == (dz != nullptr));
    ck.in(x, a.M, a.D, a.ld_x, e, true);
    if (z) ck.in(z, a.M, a.D, a.ld_z, e, false);
    ck.in(w, a.D, 4, true);
    ck.in(b, a.D, 4, false);
    ck.in(scale, a.D, 4, false);
    ck.in(dout, a.M, a.D, a.ld_y, e, true);
    ck.out(dx, a.M, a.D, a.ld_dx, e, true);
    if (dz) ck.out(dz, a.M, a.D, a.ld_dz, e, false);
    ck.out(dw, a.D, 4, false);
    ck.out(db, a.D, 4, false);
    ck.out(dscale, a.D, 4, false);
    ck.workspace(workspace, workspace_bytes, need);
    const int st = ck.finish();
    if (st != MSS_OK) return st;
    return n == 0 ? zero_params(a, stream) : launched(mss::launch_gated_norm_bwd(a, stream));
}

}  // extern "C"
