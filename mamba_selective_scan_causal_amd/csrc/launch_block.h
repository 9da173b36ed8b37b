// launch_block.h -- internal interface between block_api.hip and the kernels
// of the gated recurrence and the block norms.  Arguments arrive validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mss.h"

namespace mss {

// Row strides (ld_*) are in elements.
struct GatedArgs {
    int dtype, gate;
    int64_t B, L, D;
    float gate_scale;
    int64_t ld_x, ld_r, ld_i, ld_z, ld_y, ld_dx, ld_dr, ld_di, ld_dz;   // ld_y: y or dout
    const void* x;
    const void* r;
    const void* i;
    const float* decay;
    const void* z;
    const uint8_t* reset;
    // forward
    const float* h0;
    void* y;
    float* h_ckpt;           // also the backward's input
    float* h_last;
    // backward
    const void* dout;
    const float* dh_last;
    void* dx;
    void* dr;
    void* di;
    float* ddecay;
    void* dz;
    float* dh0;
    // step
    float* h;
    void* ws;
};

// Workspace bytes (sizes and gate only; never the pointers or strides).
// False when a size overflows or the launch would not fit a grid.
bool gated_scan_workspace(int64_t B, int64_t L, int64_t D, int64_t& bytes);
bool gated_scan_bwd_workspace(int64_t B, int64_t L, int64_t D, int gate, int64_t& bytes);
bool gated_step_fits(int64_t B, int64_t D);
hipError_t launch_gated_scan(const GatedArgs& a, hipStream_t st);
hipError_t launch_gated_scan_bwd(const GatedArgs& a, hipStream_t st);
hipError_t launch_gated_step(const GatedArgs& a, hipStream_t st);

struct NormArgs {
    int dtype, res_dtype, kind, order;
    int64_t M, D, G;
    float eps, alpha;
    int64_t ld_x, ld_z, ld_res, ld_s, ld_y, ld_ds, ld_dx, ld_dz, ld_dres;   // ld_y: y, dy or dout
    const void* x;
    const void* z;
    const void* res;
    const float* w;
    const float* b;
    const float* scale;
    void* s;                 // new residual stream (input of the backward)
    void* y;
    // backward
    const void* dy;          // dy or dout
    const void* ds;
    void* dx;
    void* dz;
    void* dres;
    float* dw;
    float* db;
    float* dscale;
    void* ws;
};

bool norm_bwd_workspace(int64_t M, int64_t D, int64_t G, int64_t& bytes);
hipError_t launch_add_norm(const NormArgs& a, hipStream_t st);
hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t st);
hipError_t launch_gated_norm(const NormArgs& a, hipStream_t st);
hipError_t launch_gated_norm_bwd(const NormArgs& a, hipStream_t st);

}  // namespace mss
