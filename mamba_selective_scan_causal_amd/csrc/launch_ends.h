// launch_ends.h -- internal interface between ends_api.hip and the kernels of
// the embedding, the head's loss and gradient clipping.  Arguments arrive
// validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mss.h"

namespace mss {

struct EmbedArgs {
    int dtype, out_dtype;     // table, rows
    bool wide_ids;            // int64
    bool accumulate;
    int64_t M, V, D;
    int64_t ld_w, ld_y;       // elements
    float scale;
    const void* ids;
    const void* w;
    void* y;                  // y, or dy (read)
    void* dw;
    void* ws;
};

// Workspace bytes (sizes only); false when a size overflows or a launch would
// not fit a grid.
bool embed_bwd_workspace(int64_t M, int64_t V, int64_t D, int64_t& bytes);
hipError_t launch_embed(const EmbedArgs& a, hipStream_t st);
hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t st);

struct HeadArgs {
    int dtype;
    bool wide_ids;
    int64_t M, V, D;
    int64_t ld_x, ld_w, ld_dx, ld_dw;   // elements
    float logit_scale;
    const void* x;
    const void* w;
    const void* targets;
    float* loss;
    float* lse;               // also the backward's input
    const float* dloss;
    const float* dlse;
    void* dx;
    void* dw;
    void* ws;
};

bool head_workspace(int dtype, int64_t M, int64_t V, int64_t D, bool backward, int64_t& bytes);
hipError_t launch_head(const HeadArgs& a, hipStream_t st);
hipError_t launch_head_bwd(const HeadArgs& a, hipStream_t st);

// `count` validated tensors, none of them empty.
int64_t clip_workspace(int64_t count);
hipError_t launch_clip(const mss_tensor* t, int64_t count, float scale, float max_norm, bool write, float* norm,
                       void* ws, hipStream_t st);

}  // namespace mss
