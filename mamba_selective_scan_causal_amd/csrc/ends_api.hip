// ends_api.hip -- the extern "C" entry points of the embedding, the head's loss
// and gradient clipping: argument validation and dispatch on the caller's
// stream, under the same rules as mss_api.hip (everything is checked before
// any launch; a rejected call writes nothing).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "launch_ends.h"
#include "mss.h"
#include "row_check.h"

namespace {

using mss::Checks;
using mss::count;
using mss::dtype_ok;
using mss::elem_size;
using mss::launched;

constexpr int64_t kMostRows = int64_t{1} << 26;
constexpr int64_t kMostElements = int64_t{1} << 44;      // of all tensors of a list

// ---- embedding -----------------------------------------------------------------

bool embed_ok(const mss_embed_dims* d, const mss_embed_strides* s, bool backward) {
    if (!d || d->struct_size != static_cast<int32_t>(sizeof(mss_embed_dims)) || d->reserved != 0 ||
        d->reserved2 != 0 || (d->flags & ~(backward ? MSS_EMBED_ACCUMULATE : 0)) != 0)
        return false;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->out_dtype)) return false;
    if (d->dtype != d->out_dtype && d->dtype != MSS_F32 && d->out_dtype != MSS_F32) return false;
    if ((d->id_bytes != 4 && d->id_bytes != 8) || !std::isfinite(d->scale)) return false;
    if (d->rows < 0 || d->vocab < 0 || d->width < 0) return false;
    if (d->rows >= kMostRows || d->vocab >= kMostRows || d->width > MSS_MAX_WIDTH) return false;
    return !s || (s->struct_size == static_cast<int32_t>(sizeof(mss_embed_strides)) && s->reserved == 0);
}

mss::EmbedArgs embed_args(const mss_embed_dims* d, const mss_embed_strides* s) {
    mss::EmbedArgs a{};
    a.dtype = d->dtype;
    a.out_dtype = d->out_dtype;
    a.wide_ids = d->id_bytes == 8;
    a.accumulate = (d->flags & MSS_EMBED_ACCUMULATE) != 0;
    a.M = d->rows;
    a.V = d->vocab;
    a.D = d->width;
    a.ld_w = s ? s->weight : a.D;
    a.ld_y = s ? s->y : a.D;
    a.scale = d->scale;
    return a;
}

bool embed_need(const mss::EmbedArgs& a, int64_t& need) {
    need = 0;
    return a.V == 0 || a.D == 0 || mss::embed_bwd_workspace(a.M, a.V, a.D, need);
}

// ---- head ------------------------------------------------------------------------

bool head_ok(const mss_head_dims* d, const mss_head_strides* s) {
    if (!d || d->struct_size != static_cast<int32_t>(sizeof(mss_head_dims)) || d->flags != 0 || d->reserved != 0 ||
        !dtype_ok(d->dtype))
        return false;
    if ((d->id_bytes != 4 && d->id_bytes != 8) || !std::isfinite(d->logit_scale)) return false;
    if (d->rows < 0 || d->rows >= kMostRows || d->vocab < 1 || d->vocab >= kMostRows || d->width < 1 ||
        d->width > MSS_MAX_WIDTH)
        return false;
    return !s || (s->struct_size == static_cast<int32_t>(sizeof(mss_head_strides)) && s->reserved == 0);
}

mss::HeadArgs head_args(const mss_head_dims* d, const mss_head_strides* s) {
    mss::HeadArgs a{};
    a.dtype = d->dtype;
    a.wide_ids = d->id_bytes == 8;
    a.M = d->rows;
    a.V = d->vocab;
    a.D = d->width;
    a.ld_x = s ? s->x : a.D;
    a.ld_w = s ? s->weight : a.D;
    a.ld_dx = s ? s->dx : a.D;
    a.ld_dw = s ? s->dweight : a.D;
    a.logit_scale = d->logit_scale;
    return a;
}

void head_inputs(Checks& ck, const mss::HeadArgs& a) {
    const int64_t e = elem_size(a.dtype);
    ck.in(a.x, a.M, a.D, a.ld_x, e, true);
    ck.in(a.w, a.V, a.D, a.ld_w, e, true);
    ck.in_any(a.targets, a.M, a.wide_ids ? 8 : 4, true);
}

// ---- lists of tensors ----------------------------------------------------------------

struct Range {
    uintptr_t from, to;
    bool out;
};

// The status of a list's tensors; `write`: with their outputs.  norm and the
// workspace are outputs beside them.
int list_status(const mss_tensor* t, int64_t n, bool write, const float* norm, const void* ws, int64_t need) {
    int64_t all = 0;
    for (int64_t i = 0; i < n; i++) {
        if (t[i].numel < 0 || t[i].numel >= kMostElements || !dtype_ok(t[i].dtype)) return MSS_EINVAL;
        if ((all += t[i].numel) >= kMostElements) return MSS_EINVAL;
        if (write && t[i].out_dtype != t[i].dtype && t[i].out_dtype != MSS_F32) return MSS_EINVAL;
        if (t[i].numel == 0) continue;
        if (!t[i].in || (write && !t[i].out)) return MSS_EINVAL;
    }
    const int64_t most = n * (write ? 2 : 1) + 2;
    const std::unique_ptr<Range[]> r(new (std::nothrow) Range[most]);
    if (!r) return MSS_EINVAL;
    int64_t used = 0;
    const auto add = [&](const void* p, int64_t bytes, bool out) {
        const uintptr_t from = reinterpret_cast<uintptr_t>(p);
        r[used++] = {from, from + static_cast<uintptr_t>(bytes), out};
    };
    for (int64_t i = 0; i < n; i++) {
        if (t[i].numel == 0) continue;
        const int64_t e = elem_size(t[i].dtype), eo = elem_size(t[i].out_dtype);
        if (reinterpret_cast<uintptr_t>(t[i].in) % e != 0) return MSS_EALIGN;
        if (write && reinterpret_cast<uintptr_t>(t[i].out) % eo != 0) return MSS_EALIGN;
        const bool in_place = write && t[i].in == t[i].out && e == eo;
        if (!in_place) add(t[i].in, t[i].numel * e, false);
        if (write) add(t[i].out, t[i].numel * eo, true);
    }
    add(norm, 4, true);
    if (ws && need > 0) add(ws, need, true);
    // an output may not reach into what starts at or after it, nor anything into an output
    std::sort(r.get(), r.get() + used, [](const Range& a, const Range& b) { return a.from < b.from; });
    uintptr_t end = 0, out_end = 0;              // of all before, and of the outputs before
    for (int64_t i = 0; i < used; i++) {
        if (r[i].from < out_end || (r[i].out && r[i].from < end)) return MSS_EALIAS;
        end = std::max(end, r[i].to);
        if (r[i].out) out_end = std::max(out_end, r[i].to);
    }
    return MSS_OK;
}

int clip(const mss_tensor* t, int64_t n, float scale, float max_norm, bool write, float* norm, void* ws,
         size_t ws_bytes, hipStream_t stream) {
    if (n < 0 || n >= (int64_t{1} << 31) || (n > 0 && !t) || !norm) return MSS_EINVAL;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return MSS_EINVAL;
    if (write && !(std::isfinite(max_norm) && max_norm >= 0.0f)) return MSS_EINVAL;
    if (reinterpret_cast<uintptr_t>(norm) % 4 != 0) return MSS_EALIGN;
    const int64_t need = mss::clip_workspace(n);
    const int st = list_status(t, n, write, norm, ws, need);
    if (st != MSS_OK) return st;
    if (!ws || ws_bytes < static_cast<uint64_t>(need)) return MSS_EWORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MSS_EALIGN;
    return launched(mss::launch_clip(t, n, scale, max_norm, write, norm, ws, stream));
}

}  // namespace

extern "C" {

int mss_embedding(const mss_embed_dims* dims, const mss_embed_strides* strides, const void* ids,
                  const void* weight, void* y, hipStream_t stream) {
    if (!embed_ok(dims, strides, false)) return MSS_EINVAL;
    mss::EmbedArgs a = embed_args(dims, strides);
    a.ids = ids;
    a.w = weight;
    a.y = y;
    Checks ck(strides != nullptr);
    ck.in_any(ids, a.M, dims->id_bytes, true);
    ck.in(weight, a.V, a.D, a.ld_w, elem_size(a.dtype), true);
    ck.out(y, a.M, a.D, a.ld_y, elem_size(a.out_dtype), true);
    const int st = ck.finish();
    if (st != MSS_OK || a.M == 0 || a.D == 0) return st;
    return launched(mss::launch_embed(a, stream));
}

int mss_embed_workspace_bytes(const mss_embed_dims* dims, size_t* bytes) {
    if (!bytes) return MSS_EINVAL;
    *bytes = 0;
    if (!embed_ok(dims, nullptr, true)) return MSS_EINVAL;
    int64_t need;
    if (!embed_need(embed_args(dims, nullptr), need)) return MSS_EINVAL;
    *bytes = static_cast<size_t>(need);
    return MSS_OK;
}

int mss_embedding_backward(const mss_embed_dims* dims, const mss_embed_strides* strides,
                           const void* ids, const void* dy, void* dweight, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    if (!embed_ok(dims, strides, true)) return MSS_EINVAL;
    mss::EmbedArgs a = embed_args(dims, strides);
    a.ids = ids;
    a.y = const_cast<void*>(dy);
    a.dw = dweight;
    a.ws = workspace;
    int64_t need;
    if (!embed_need(a, need)) return MSS_EINVAL;
    Checks ck(strides != nullptr);
    ck.in_any(ids, a.M, dims->id_bytes, true);
    ck.in(dy, a.M, a.D, a.ld_y, elem_size(a.out_dtype), true);
    ck.out(dweight, a.V, a.D, a.ld_w, elem_size(a.dtype), true);
    ck.workspace(workspace, workspace_bytes, need);
    const int st = ck.finish();
    if (st != MSS_OK || a.V == 0 || a.D == 0 || (a.M == 0 && a.accumulate)) return st;
    return launched(mss::launch_embed_bwd(a, stream));
}

int mss_head_workspace_bytes(const mss_head_dims* dims, int op, size_t* bytes) {
    if (!bytes) return MSS_EINVAL;
    *bytes = 0;
    if (op != MSS_OP_HEAD_LOSS && op != MSS_OP_HEAD_LOSS_BACKWARD) return MSS_EINVAL;
    if (!head_ok(dims, nullptr)) return MSS_EINVAL;
    int64_t need;
    if (!mss::head_workspace(dims->dtype, dims->rows, dims->vocab, dims->width,
                             op == MSS_OP_HEAD_LOSS_BACKWARD, need))
        return MSS_EINVAL;
    *bytes = static_cast<size_t>(need);
    return MSS_OK;
}

int mss_head_loss(const mss_head_dims* dims, const mss_head_strides* strides, const void* x,
                  const void* weight, const void* targets, float* loss, float* lse,
                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!head_ok(dims, strides)) return MSS_EINVAL;
    mss::HeadArgs a = head_args(dims, strides);
    a.x = x;
    a.w = weight;
    a.targets = targets;
    a.loss = loss;
    a.lse = lse;
    a.ws = workspace;
    int64_t need;
    if (!mss::head_workspace(a.dtype, a.M, a.V, a.D, false, need)) return MSS_EINVAL;
    Checks ck(strides != nullptr);
    head_inputs(ck, a);
    ck.out_any(loss, a.M, 4, true);
    ck.out_any(lse, a.M, 4, true);
    ck.workspace(workspace, workspace_bytes, need);
    const int st = ck.finish();
    if (st != MSS_OK || a.M == 0) return st;
    return launched(mss::launch_head(a, stream));
}

int mss_head_loss_backward(const mss_head_dims* dims, const mss_head_strides* strides,
                           const void* x, const void* weight, const void* targets,
                           const float* lse, const float* dloss, const float* dlse, void* dx,
                           void* dweight, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
    if (!head_ok(dims, strides)) return MSS_EINVAL;
    mss::HeadArgs a = head_args(dims, strides);
    a.x = x;
    a.w = weight;
    a.targets = targets;
    a.lse = const_cast<float*>(lse);
    a.dloss = dloss;
    a.dlse = dlse;
    a.dx = dx;
    a.dw = dweight;
    a.ws = workspace;
    int64_t need;
    if (!mss::head_workspace(a.dtype, a.M, a.V, a.D, true, need)) return MSS_EINVAL;
    const int64_t e = elem_size(a.dtype);
    Checks ck(strides != nullptr);
    head_inputs(ck, a);
    ck.in_any(lse, a.M, 4, true);
    ck.in_any(dloss, a.M, 4, true);
    ck.in_any(dlse, a.M, 4, false);
    if (dx) ck.out(dx, a.M, a.D, a.ld_dx, e, false);
    if (dweight) ck.out(dweight, a.V, a.D, a.ld_dw, e, false);
    ck.workspace(workspace, workspace_bytes, need);
    const int st = ck.finish();
    if (st != MSS_OK) return st;
    return launched(mss::launch_head_bwd(a, stream));
}

int mss_clip_workspace_bytes(int64_t n, size_t* bytes) {
    if (!bytes) return MSS_EINVAL;
    *bytes = 0;
    if (n < 0 || n >= (int64_t{1} << 31)) return MSS_EINVAL;
    *bytes = static_cast<size_t>(mss::clip_workspace(n));
    return MSS_OK;
}

int mss_grad_norm(const mss_tensor* tensors, int64_t n, float scale, float* norm,
                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return clip(tensors, n, scale, 0.0f, false, norm, workspace, workspace_bytes, stream);
}

int mss_clip_grads(const mss_tensor* tensors, int64_t n, float scale, float max_norm,
                   float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return clip(tensors, n, scale, max_norm, true, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
